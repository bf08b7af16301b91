"""The token operators' calls through ctypes, as they are made where the module of quick calls is
missing: every one gives what the module's gives."""
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from test_gpu_kv4 import Cache
from test_gpu_qk_norm_rope import Heads

pytestmark = pytest.mark.gpu


def everything(dev):
    a = Heads(dev, T=7, grad=torch.float32, fused=True)
    a.fwd()
    a.bwd()
    c = Cache(dev, B=2, Hq=4, Hkv=2, D=64, N=128)
    k = torch.randn(2, 3, 2, 64, generator=c.g).to(torch.bfloat16).to(dev)
    rows = torch.empty(2, 2, 3, dtype=torch.int32, device=dev)
    P.pbsa_kv4_evict(c.cfg, c.pos, c.mass, 2, c.i32([200, 200]), rows, c.status)
    P.pbsa_kv4_append(c.cfg, c.cache, k, k.flip(1), c.i32([[256, 257, 258], [256, -1, -1]]), rows, c.mass, c.status)
    out, lse = c.attend(c.queries(3), c.i32([[256, 257, 258], [256, -1, -1]]), c.i32([128, 100]), c.mass)
    ko, vo = (torch.empty(2, 2, 3, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    P.pbsa_kv4_read(c.cfg, c.cache, rows, ko, vo, c.status)
    assert int(c.status.item()) == 0 and int(a.status.item()) == 0
    return [a.q_out, a.k_out, a.dq, a.dk, a.dwq, a.dwk, rows, out, lse, c.mass, c.pos, ko, vo, c.kc, c.ks, c.vc, c.vs]


def test_calls_through_ctypes(cuda_dev, monkeypatch):
    made = []
    real = P._calls
    spy = {n: (lambda f: lambda *a: made.append(1) or f(*a))(getattr(real, n)) for n in vars(P._NO_CALLS)}
    monkeypatch.setattr(P, "_calls", type(P._NO_CALLS)(**spy))
    want = everything(cuda_dev)
    assert len(made) == 6
    monkeypatch.setattr(P, "_calls", P._NO_CALLS)
    assert all(torch.equal(x, y) for x, y in zip(everything(cuda_dev), want))

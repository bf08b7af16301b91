"""Norm and rotation of heads on the GPU, through the C ABI, against the fp64 oracle.

Tolerances.  u = 2^-24 is the fp32 half step and e half a step of the output's type (finfo.eps / 2
relative to the value: bf16 2^-8, fp16 2^-11, fp32 2^-24).  Every output is a
handful of fp32 operations on x r w, r a sum of D squares (relative error of the sum at most
(log2 D + 8) u, since eight are added in a lane and the rest in a tree) and a reciprocal root
(2 ulp): 32 u of the magnitudes that enter covers them.
  forward   |err| <= e |y| + 32 u (|a| + |b|), a and b the pair before it is turned
  dx        |err| <= e |dx| + 64 u r (|g w| + |x| r^2 mean |g w x| D), the magnitudes of its two
            terms with the sum's terms taken absolute (sum of D terms: (log2 D + 8) u of it)
  dw        |err| <= (n_lane + 40) u sum |g x r|, n_lane the terms one lane adds in a row; the
            cases here stay below 64 of them
fp16 outputs below its smallest normal number are off by at most 2^-25 absolutely."""
import numpy as np
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from block_sparse_attention_35_b200.attention import SparseForcingAttention, rope_table
from block_sparse_attention_35_b200.synth import WORKLOADS, decode_inputs
from oracle import token_oracle as orc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Heads:
    """Inputs of one call, on the GPU."""

    def __init__(self, dev, B=2, T=5, Hq=4, Hkv=2, D=128, dtype=torch.bfloat16, rot=None, interleaved=False,
                 pairs=None, grad=None, fused=False, eps=1e-6, length=61, seed=0, weights=True):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)
        self.rot = D if rot is None else rot
        self.pairs = (self.rot // 2,) if pairs is None else pairs
        self.cfg = P.make_qk_config(B, T, Hq, Hkv, D, dtype, self.rot, interleaved, self.pairs, length, eps, grad)
        H = Hq + Hkv
        if fused:
            qkv = (2 * rn(B, T, H + Hkv, D)).to(dtype).to(dev)
            self.q, self.k = qkv[:, :, :Hq], qkv[:, :, Hq:H]
        else:
            self.q, self.k = (2 * rn(B, T, Hq, D)).to(dtype).to(dev), (2 * rn(B, T, Hkv, D)).to(dtype).to(dev)
        self.wq = (1 + 0.3 * rn(D)).to(dev) if weights else None
        self.wk = (1 + 0.3 * rn(D)).to(dev) if weights else None
        self.cos = self.sin = self.pos = None
        if self.rot:
            self.cos, self.sin = rope_table(self.pairs, length, 100.0, dev)
            self.pos = torch.randint(0, length, (B, T, len(self.pairs)), generator=g, dtype=torch.int32).to(dev)
        gt = dtype if grad is None else grad
        self.gq, self.gk = rn(B, T, Hq, D).to(gt).to(dev), rn(B, T, Hkv, D).to(gt).to(dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        nan = lambda t: torch.full(t.shape, float("nan"), dtype=dtype, device=dev)
        self.q_out, self.k_out, self.dq, self.dk = nan(self.q), nan(self.k), nan(self.q), nan(self.k)
        self.dwq, self.dwk = torch.full((D,), float("nan"), device=dev), torch.full((D,), float("nan"), device=dev)
        self.ws = torch.full((P.pbsa_qk_workspace_size(self.cfg),), 255, dtype=torch.uint8, device=dev)

    def fwd(self, **kw):
        P.pbsa_qk_norm_rope(self.cfg, self.q, self.k, self.wq, self.wk, self.cos, self.sin, self.pos,
                            self.q_out, self.k_out, self.status, **kw)

    def bwd(self, **kw):
        P.pbsa_qk_norm_rope_bwd(self.cfg, self.q, self.k, self.wq, self.wk, self.cos, self.sin, self.pos,
                                self.gq, self.gk, self.dq, self.dk, self.dwq, self.dwk, self.ws, self.status, **kw)

    def oracle(self):
        rotation = (None if self.cos is None else f64(self.cos), None if self.sin is None else f64(self.sin),
                    None if self.pos is None else self.pos.cpu().numpy(), self.rot, bool(self.cfg.interleaved),
                    self.pairs, self.cfg.eps)
        one = np.ones(self.cfg.D)
        for x, w, gy in ((self.q, self.wq, self.gq), (self.k, self.wk, self.gk)):
            yield f64(x), one if w is None else f64(w), f64(gy), rotation

    def check(self, tokens=None, grads=True):
        D, eps = self.cfg.D, self.cfg.eps
        e = torch.finfo(self.q.dtype).eps / 2
        tiny = 2.0 ** -25 if self.q.dtype == torch.float16 else 0.0
        at = (slice(None), slice(None)) if tokens is None else tokens
        for (x, w, gy, rotation), y, dx, dw in zip(self.oracle(), (self.q_out, self.k_out), (self.dq, self.dk),
                                                   (self.dwq, self.dwk)):
            want = orc.norm_rope(x, w, *rotation)
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            big = np.abs(x * r * w).max(-1, keepdims=True)
            assert (np.abs(f64(y) - want) <= e * np.abs(want) + 64 * U * big + tiny)[at].all()
            if not grads:
                continue
            wdx, wdw = orc.norm_rope_bwd(x, w, *rotation, gy)
            g = orc._turn(gy, *rotation[:6], back=True)
            gb = np.abs(gy).max(-1, keepdims=True) * 2          # bound of every |a| + |b| turned
            mag = r * (gb * np.abs(w) + np.abs(x) * r * r * (gb * np.abs(w * x)).sum(-1, keepdims=True) / D * 16)
            assert (np.abs(f64(dx) - wdx) <= e * np.abs(wdx) + 64 * U * mag + tiny)[at].all()
            if tokens is None:
                bound = (np.maximum(np.abs(g), gb / 2) * np.abs(x) * r).reshape(-1, D).sum(0)
                assert (np.abs(f64(dw) - wdw) <= 104 * U * bound).all()
        assert int(self.status.item()) == 0 or tokens is not None


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                        (torch.float16, torch.float16), (torch.float16, torch.float32),
                                        (torch.float32, torch.float32)])
def test_types_and_pairings(cuda_dev, D, interleaved, dtype, grad):
    a = Heads(cuda_dev, D=D, interleaved=interleaved, dtype=dtype, grad=grad, seed=1)
    a.fwd()
    a.bwd()
    a.check()


@pytest.mark.parametrize("D,rot,pairs", [(128, 0, (0,)), (128, 16, (8,)), (128, 48, (24,)), (64, 48, (10, 7, 7)),
                                         (128, 128, (22, 21, 21)), (64, 64, (31, 1)), (128, 64, (0, 32, 0))])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_channels_and_axes(cuda_dev, D, rot, pairs, interleaved):
    a = Heads(cuda_dev, D=D, rot=rot, pairs=pairs, interleaved=interleaved, seed=2)
    if rot == 0:
        a.cos = a.sin = a.pos = None
    a.fwd()
    a.bwd()
    a.check()


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 12, 12), (3, 1, 5, 1), (1, 7, 40, 3), (2, 333, 7, 7),
                                        (1, 2, 3, 0), (1, 1300, 9, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_counts_and_lengths(cuda_dev, B, T, Hq, Hkv, D):
    """One token to many, more heads than a warp's step and fewer, queries alone."""
    a = Heads(cuda_dev, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, grad=torch.float32, seed=3)
    a.fwd()
    a.bwd()
    if Hkv == 0:
        assert (a.dwk == 0).all()
    a.check()


def test_views_of_one_projection_and_in_place(cuda_dev):
    for dtype, D in ((torch.bfloat16, 128), (torch.float32, 64), (torch.float16, 128)):
        a = Heads(cuda_dev, T=9, Hq=6, Hkv=2, D=D, dtype=dtype, fused=True, seed=4)
        assert not a.q.is_contiguous()
        # gradients written into views of one buffer as well
        dqkv = torch.full((2, 9, 10, D), 7.0, dtype=dtype, device=cuda_dev)
        a.dq, a.dk = dqkv[:, :, :6], dqkv[:, :, 6:8]
        a.fwd()
        a.bwd()
        a.check()
        assert (dqkv[:, :, 8:] == 7).all()
        # head-major storage: [B, H, T, D] seen as [B, T, H, D]
        qt = a.q.transpose(1, 2).contiguous().transpose(1, 2)
        out = torch.empty_like(a.k_out).transpose(1, 2).contiguous().transpose(1, 2)
        ref_q, ref_k, q0, ref_dq = a.q_out.clone(), a.k_out.clone(), a.q, a.dq.clone()
        a.q, a.k_out = qt, out
        a.fwd()
        assert torch.equal(a.q_out, ref_q) and torch.equal(a.k_out, ref_k)
        # in place: the outputs over the inputs, the gradients over the outputs' gradients
        a.q, a.q_out = q0.clone(), None
        a.q_out = a.q
        a.fwd()
        assert torch.equal(a.q, ref_q)
        a.q, a.dq = q0, a.gq
        a.bwd()
        assert torch.equal(a.dq, ref_dq)


def test_no_weights_and_broadcast_gradients(cuda_dev):
    a = Heads(cuda_dev, weights=False, T=6, seed=5)
    a.gq = a.gq[:, :1, :1].expand(a.gq.shape)          # one gradient for every token and head
    a.fwd()
    a.bwd()
    a.check()
    want = a.dq.clone()
    a.dwq = a.dwk = a.ws = None                        # no weights' gradients: no workspace
    a.dq.fill_(float("nan"))
    a.bwd()
    assert torch.equal(a.dq, want)


def test_zero_rows_tiny_and_large_values(cuda_dev):
    a = Heads(cuda_dev, dtype=torch.float32, T=4, eps=1e-6, seed=6)
    a.q[0, 0] = 0
    a.q[0, 1] *= 1e-18
    a.q[1, 2] *= 1e15
    a.fwd()
    a.bwd()
    a.check()
    assert (a.q_out[0, 0] == 0).all()


def test_position_out_of_the_table_leaves_its_token_alone(cuda_dev):
    for bad in (-1, 61, 2 ** 31 - 1):
        a = Heads(cuda_dev, pairs=(30, 30, 4), T=5, seed=7)
        a.pos[1, 3, 2] = bad
        a.fwd()
        a.bwd()
        assert int(a.status.item()) == P.PBSA_ERR_DEVICE_CHECK
        for t in (a.q_out, a.k_out, a.dq, a.dk):
            assert t[1, 3].isnan().all()
        a.pos[1, 3, 2] = 0
        keep = np.ones((2, 5), bool)
        keep[1, 3] = False
        a.check(tokens=keep)
        # its gradients do not enter the weights': the same sums with that token's gradient zero
        got = a.dwq.clone()
        a.gq[1, 3] = 0
        a.gk[1, 3] = 0
        a.bwd()
        assert torch.equal(got, a.dwq)


def test_what_does_not_fit_is_refused_and_odd_strides_of_one_element_are_not(cuda_dev):
    B, T, Hq, Hkv, D = 1, 1, 2, 1, 64
    cfg = P.make_qk_config(B, T, Hq, Hkv, D, torch.bfloat16, table_len=4)
    f32 = dict(dtype=torch.float32, device=cuda_dev)
    good = dict(q=torch.randn(B, T, Hq, D, device=cuda_dev).bfloat16(), k=torch.randn(B, T, Hkv, D, device=cuda_dev).bfloat16(),
                q_weight=torch.rand(D, **f32), k_weight=torch.rand(D, **f32), cos=torch.rand(4, D // 2, **f32),
                sin=torch.rand(4, D // 2, **f32), pos=torch.zeros(B, T, 1, dtype=torch.int32, device=cuda_dev),
                q_out=torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device=cuda_dev),
                k_out=torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=cuda_dev),
                status=torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    order = list(good)
    grads = lambda g: (g["q_out"], g["k_out"], torch.empty_like(good["q"]), torch.empty_like(good["k"]), None, None, None)
    for name in order:
        x = good[name]
        bad = [x.cpu(), x.double(), x[None], x[..., :-1], None]
        if name in ("q_out", "k_out"):
            bad.append(x[..., :1, :].expand(B, T, 2, D) if name == "q_out" else x.transpose(-1, -2))
        if name in ("q_weight", "k_weight"):
            bad.pop()   # None: all ones
        for y in bad:
            g = dict(good, **{name: y})
            with pytest.raises((P.PBSAError, AttributeError)):
                P.pbsa_qk_norm_rope(cfg, *g.values())
            if name not in ("q_out", "k_out"):
                with pytest.raises((P.PBSAError, AttributeError)):
                    P.pbsa_qk_norm_rope_bwd(cfg, *[g[n] for n in order[:7]], *grads(g), g["status"])
    assert int(good["status"].item()) == 0 and not good["q_out"].any() and not good["k_out"].any()
    P.pbsa_qk_norm_rope(cfg, *good.values())
    odd = dict(good, q=good["q"].as_strided((1, 1, 2, 64), (3, 5, 64, 1)), k=good["k"].as_strided((1, 1, 1, 64), (1, 7, 9, 1)),
               q_out=torch.zeros_like(good["q_out"]).as_strided((1, 1, 2, 64), (1, 1, 64, 1)), k_out=torch.zeros_like(good["k_out"]))
    P.pbsa_qk_norm_rope(cfg, *odd.values())
    assert torch.equal(odd["q_out"], good["q_out"]) and torch.equal(odd["k_out"], good["k_out"]) and good["q_out"].any()


def test_no_tokens(cuda_dev):
    a = Heads(cuda_dev, T=0)
    a.fwd()
    a.bwd()
    assert (a.dwq == 0).all() and (a.dwk == 0).all()


def test_runs_repeat_bit_for_bit_and_on_another_stream(cuda_dev):
    a = Heads(cuda_dev, B=2, T=700, Hq=8, Hkv=8, grad=torch.float32, seed=8)
    a.fwd()
    a.bwd()
    want = [t.clone() for t in (a.q_out, a.k_out, a.dq, a.dk, a.dwq, a.dwk)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a.fwd()
        a.bwd()
    a.fwd(stream=s)
    s.synchronize()
    for t, w in zip((a.q_out, a.k_out, a.dq, a.dk, a.dwq, a.dwk), want):
        assert torch.equal(t, w)


def test_captured_and_replayed(cuda_dev):
    a = Heads(cuda_dev, T=33, grad=torch.float32, seed=9)
    a.fwd()
    a.bwd()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.fwd()
        a.bwd()
    b = Heads(cuda_dev, T=33, grad=torch.float32, seed=10)
    for x, y in ((a.q, b.q), (a.k, b.k), (a.wq, b.wq), (a.wk, b.wk), (a.pos, b.pos), (a.gq, b.gq), (a.gk, b.gk)):
        x.copy_(y)
    for _ in range(2):
        g.replay()
    a.check()


def test_gradient_against_differences(cuda_dev):
    """The GPU's fp32 gradient against central differences of the fp64 forward: 2 directions."""
    a = Heads(cuda_dev, B=1, T=3, Hq=2, Hkv=1, D=64, dtype=torch.float32, pairs=(12, 10, 10), seed=11)
    a.bwd()
    rng = np.random.default_rng(0)
    (x, w, gy, rotation), _ = a.oracle()
    h = 1e-6
    for _ in range(8):
        u, v = rng.normal(size=x.shape), rng.normal(size=w.shape)
        f = lambda s: (orc.norm_rope(x + s * u, w + s * v, *rotation) * gy).sum()
        want = (f(h) - f(-h)) / (2 * h)
        got = (f64(a.dq) * u).sum() + (f64(a.dwq) * v).sum()
        size = (np.abs(f64(a.dq) * u)).sum() + (np.abs(f64(a.dwq) * v)).sum()
        assert abs(got - want) <= 1e-6 * size


def test_heads_feed_the_block_attention(cuda_dev):
    """norm_rope -> append -> select + attend -> backward -> norm_rope_backward on the tiny
    workload: positions continue from chunk to chunk, gradients come back in fp32."""
    wl = WORKLOADS["tiny"]
    a = SparseForcingAttention(wl.B, wl.H, wl.D, wl.frame_h, wl.frame_w, wl.total_cache_size,
                               wl.local_cache_size, wl.persistent_cache_size, max_seq_len=wl.max_seq_len,
                               local_block_sparse_topk_ratio=wl.topk_ratio, chunk_frames=wl.q_frames,
                               device=cuda_dev)
    inp = decode_inputs(wl)
    q = inp["q"].to(cuda_dev)
    g = torch.Generator().manual_seed(1)
    k, v, dout = (torch.randn(q.shape, generator=g).to(torch.bfloat16).to(cuda_dev) for _ in range(3))
    wq, wk = (1 + 0.1 * torch.randn(wl.D, generator=g).to(cuda_dev) for _ in range(2))
    first = wl.q_frames
    qn, kn = a.norm_rope(q, k, wq, wk, first)
    a.append(kn, v)
    out = a(qn)
    dq, _, _, dk_ring, _ = a.backward(qn, dout)
    dk = dk_ring[:, :q.shape[1]]
    gq, gk, gwq, gwk = a.norm_rope_backward(q, k, wq, wk, first, dq, dk)
    assert int(a.status.item()) == 0 and torch.isfinite(out).all()
    p = wl.D // 2
    pairs = (p - 2 * (p // 3), p // 3, p // 3)
    n = torch.arange(q.shape[1])
    pos = torch.stack((n // a.tf + first, n % a.tf // wl.frame_w, n % wl.frame_w), -1).expand(wl.B, -1, -1).numpy()
    cos, sin = rope_table(pairs, a._rope[0].shape[0], device="cpu")
    rotation = (f64(cos), f64(sin), pos, wl.D, True, pairs, 1e-6)
    for x, w, y, gy, gx, gw in ((q, wq, qn, dq, gq, gwq), (k, wk, kn, dk, gk, gwk)):
        want = orc.norm_rope(f64(x), f64(w), *rotation)
        # half a bf16 step, and the table's fp32 angles times the size of a pair
        assert (np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max()).all()
        dx, dw = orc.norm_rope_bwd(f64(x), f64(w), *rotation, f64(gy))
        assert (np.abs(f64(gx) - dx) <= 2.0 ** -8 * np.abs(dx) + 2.0 ** -16 * np.abs(dx).max()).all()
        assert np.abs(f64(gw) - dw).max() <= 2.0 ** -16 * np.abs(dw).max()

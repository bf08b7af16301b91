"""Edges of the token operators that need no GPU: sources, refusals, the binding and its build."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

from block_sparse_attention_35_b200 import build as B
from block_sparse_attention_35_b200 import pbsa as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_attention_35_b200", "csrc")


@pytest.mark.parametrize("name", ["kv4_attn.cu", "kv4_chunk.cu"])
def test_warps_agree_on_what_a_wait_returned(name):
    """Where a whole warp waits and goes on with shuffles, votes or matrix instructions, its lanes
    share one answer: nothing stores a single lane's."""
    src = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"\bmbar_wait_warp\(", src)) >= 1
    assert not re.findall(r"\bok\w*\s*=[^;]*\bmbar_wait\(", src)
    # what is left are the waits of one elected lane that asks for copies
    for m in re.finditer(r"\bmbar_wait\(", src):
        before = src[:m.start()]
        assert before.rfind("if (lane == 0)") > before.rfind("} else"), src[m.start() - 80:m.end() + 40]



def test_products_end_before_tensor_memory_is_released():
    """A softmax warp whose wait gives up leaves products in flight that the warp which issued them
    has no reason to doubt: every release stands behind the block's barrier and, where any warp
    raised the abort flag, behind a bounded wait for all products."""
    src = open(os.path.join(CSRC, "kv4_chunk.cu")).read()
    ends = [m.start() for m in re.finditer(r"\btmem_dealloc\(tmem", src)]
    assert len(ends) == 2
    for at in ends:
        tail = src[:at]
        barrier = tail.rfind("    tc_fence_before();\n    __syncthreads();")
        drain = tail[barrier:]
        assert "if (s_abort)" in drain and "umma_commit(&s_drain" in drain and "mbar_wait_drain(&s_drain" in drain


def test_the_package_imports_without_the_module_of_quick_calls():
    """Block attention and the token operators do not depend on the module that reads torch's
    tensors: without it, or with another torch's, ctypes makes the calls."""
    code = """
import sys, types, warnings
warnings.simplefilter("error")
name = "block_sparse_attention_35_b200.token_calls"
sys.modules[name] = {stand_in}
try:
    import block_sparse_attention_35_b200.pbsa
except UserWarning as w:
    assert "ctypes" in str(w), w
else:
    raise SystemExit("no warning")
warnings.simplefilter("ignore")
import torch
import block_sparse_attention_35_b200.pbsa as P
import block_sparse_attention_35_b200.attention, block_sparse_attention_35_b200.token_cache
c = P.make_kv4_config(1, 2, 2, 64, 64)
pos, mass = torch.zeros(1, 2, 64, dtype=torch.int32), torch.zeros(1, 2, 64)
try:
    P.pbsa_kv4_evict(c, pos, mass, 0, None, pos[..., :1].contiguous(), torch.zeros(1, dtype=torch.int32))
except P.PBSAError as e:
    assert "not on a CUDA device" in str(e), e
else:
    raise SystemExit("not refused")
"""
    for stand_in in ("None", "types.SimpleNamespace(torch_version='1.0')"):
        r = subprocess.run([sys.executable, "-c", code.replace("{stand_in}", stand_in)], cwd=ROOT,
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr


def test_another_torch_means_another_build(monkeypatch):
    monkeypatch.setattr(B.os.path, "getmtime", lambda path: 0.0)
    assert P._calls.torch_version == torch.__version__ and B.calls_up_to_date()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert not B.calls_up_to_date() and not B.up_to_date()


def test_a_module_that_cannot_be_built_is_left_out(monkeypatch, tmp_path):
    stale = tmp_path / "token_calls.so"
    stale.write_bytes(b"of another torch")
    monkeypatch.setattr(B, "CALLS", str(stale))
    monkeypatch.setattr(B, "calls_command", lambda: [sys.executable, "-c", "raise SystemExit(1)"])
    monkeypatch.setattr(B, "library_up_to_date", lambda: True)
    with pytest.warns(UserWarning, match="could not be built"):
        assert B.build() == B.LIB
    assert not stale.exists()


@pytest.mark.parametrize("bad", [
    (0, 128, 64), (512, 0, 64), (512, 128, 0),        # broadcast
    (512, 128, 56), (512, 120, 64), (448, 128, 64),   # a head, a token, a sequence over the one before
    (64, 512, 64), (128, 64, 256),                   # in another order
    (2 ** 62, 64, 2 ** 62),
])
def test_outputs_whose_elements_share_memory_are_refused(bad):
    """[2, 4, 2, 64] outputs: the good strides are (512, 128, 64)."""
    lib, qc, good = P.library(), P.make_qk_config(2, 4, 2, 2, 64, table_len=8), (512, 128, 64)
    for call, n, outputs in ((lib.pbsa_qk_norm_rope, 4, (2, 3)), (lib.pbsa_qk_norm_rope_bwd, 6, (4, 5))):
        for i in outputs:
            strides = [s for j in range(n) for s in (bad if j == i else good)]
            args = [256, 256, (ctypes.c_int64 * len(strides))(*strides)] + [256] * (8 if n == 4 else 12)
            rc = call(ctypes.byref(qc), *args, *((None,) if n == 4 else (1 << 20, 256, None)))
            assert rc == P.PBSA_ERR_ARG and "share memory" in P.pbsa_last_error()


def test_a_call_without_tokens_divides_by_none(tmp_path):
    """The split of the heads divides by the tokens, which an optimising compiler may hide: the host
    code of a call without tokens is run as it is written."""
    src = open(os.path.join(CSRC, "qk_norm_rope.cu")).read()
    body = src[src.index("int heads_per_item("):]
    split = body[:body.index("\n}\n") + 3]
    blocks = src[src.index("int qk_bwd_blocks("):]
    blocks = blocks[:blocks.index("\n}\n") + 3]
    run = src[src.index("cudaError_t run_bwd("):]
    run = run[run.index("{") + 1:run.index("\n}\n")]
    run = re.sub(r"qk_\w+<[^;]*;", ";", run)           # no launches
    (tmp_path / "t.cpp").write_text("""
#include "pbsa.h"
typedef int cudaError_t; enum { cudaSuccess = 0 }; int cudaGetLastError() { return 0; }
constexpr int kSMs = 148, kWarps = 8, kFwdCtas = 4, kBwdCtas = 2, D = 64;
struct QkArgs { pbsa_qk_config c; float* dw[2]; };
""" + split + blocks + "int run(const QkArgs& a) {" + run + """}
int main() {
    QkArgs a{};
    a.c.B = 1, a.c.T = 0, a.c.Hq = 2, a.c.Hkv = 2, a.c.D = D;
    return run(a);
}
""")
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-O0", "-w", "-I", os.path.join(ROOT, "include"), "-o", exe, str(tmp_path / "t.cpp")], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0

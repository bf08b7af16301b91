"""Token operators without a GPU: pins of their oracle, host-only queries and refusals (every
refused call returns before anything is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from oracle import token_oracle as orc


# ------------------------------------------------------------------------- oracle pins
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,pairs", [(32, (16,)), (16, (4, 3, 1)), (0, (0,))])
def test_norm_rope_gradient_matches_differences(interleaved, rot, pairs):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(2, 3, 2, 32))
    w = 1 + 0.2 * rng.normal(size=32)
    dy = rng.normal(size=x.shape)
    ang = rng.normal(size=(9, max(rot // 2, 1)))
    pos = rng.integers(0, 9, size=(2, 3, len(pairs)))
    args = (np.cos(ang), np.sin(ang), pos, rot, interleaved, pairs, 1e-3)
    dx, dw = orc.norm_rope_bwd(x, w, *args, dy)
    f = lambda xx, ww: (orc.norm_rope(xx, ww, *args) * dy).sum()
    h = 1e-6
    for _ in range(20):
        u, v = rng.normal(size=x.shape), rng.normal(size=32)
        want = (f(x + h * u, w + h * v) - f(x - h * u, w - h * v)) / (2 * h)
        assert abs((dx * u).sum() + (dw * v).sum() - want) < 1e-6 * (1 + abs(want))


def test_rotation_keeps_lengths_and_relative_angles():
    """A rotation by positions p and q leaves the product depending on p - q alone."""
    rng = np.random.default_rng(4)
    ang = np.arange(40)[:, None] * (100.0 ** (-np.arange(8) / 8))
    a, b = rng.normal(size=(2, 1, 1, 1, 16))
    one = np.ones(16)

    def at(x, p):
        return orc.norm_rope(x, one, np.cos(ang), np.sin(ang), np.full((1, 1, 1), p), 16, True, (8,), 1e-6)

    assert np.allclose((at(a, 7) * at(b, 3)).sum(), (at(a, 31) * at(b, 27)).sum())
    assert np.allclose((at(a, 7) ** 2).sum(), 16, rtol=1e-4)


def test_quantiser_against_all_neighbours():
    """Every code is the nearest level; ties go to the even code; scales are e4m3(amax / 6)."""
    assert [orc.LEVELS[orc.nearest(t, orc.LEVELS)] for t in
            (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0)] == [0, 1, 1, 2, 2, 4, 4, 6]
    assert orc.E4M3[126] == 448 and orc.E4M3[8] == 2.0 ** -6 and orc.E4M3[1] == 2.0 ** -9
    v = torch.tensor(orc.E4M3).to(torch.float8_e4m3fn)
    assert v.view(torch.uint8).tolist() == list(range(127))
    rng = np.random.default_rng(5)
    x = rng.normal(size=64) * 3
    codes, scales = orc.quantise_row(x, 1.0)
    packed = np.array([codes[i] | codes[i + 1] << 4 for i in range(0, 64, 2)], np.uint8)
    y = orc.values(packed, np.array(scales, np.uint8), 1.0)
    step = np.repeat([orc.E4M3[s] for s in scales], 16)
    # at most half the widest gap (4 to 6), a little more where the scale rounded down
    assert (np.abs(x - y) <= step * 1.4).all()


def test_attention_oracle_is_the_softmax_of_torch():
    rng = np.random.default_rng(6)
    B, T, Hq, Hkv, D, N = 2, 3, 4, 2, 16, 10
    q, k, v = rng.normal(size=(B, T, Hq, D)), rng.normal(size=(B, Hkv, N, D)), rng.normal(size=(B, Hkv, N, D))
    pos = np.tile(np.arange(N), (B, Hkv, 1))
    q_pos = np.array([[7, 8, 9], [7, 8, -1]])
    out, lse, mass, _, _ = orc.kv4_attn(q, k, v, pos, q_pos, [N, N])
    kk, vv = (torch.tensor(t).repeat_interleave(2, 1) for t in (k, v))
    mask = torch.tensor(q_pos)[:, None, :, None] >= torch.arange(N)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).transpose(1, 2), kk, vv, attn_mask=mask).transpose(1, 2).numpy()
    assert np.allclose(out[0], want[0]) and np.allclose(out[1, :2], want[1, :2])
    assert (out[1, 2] == 0).all() and np.isneginf(lse[1, :, 2]).all()
    assert np.allclose(mass.sum(-1), [[6, 6], [4, 4]])     # one per query token and head


def test_eviction_oracle_by_hand():
    pos = np.array([[[0, 5, -1, 9, 3, 8, 4, -1]]])
    mass = np.array([[[0.0, 2.0, 9.0, 0.0, 1.0, 0.5, 1.0, 0.1]]])
    # row 0 is a first token, rows 3 and 5 are recent; empties 2 and 7, then 4 and 6 (tie), 1
    for n, want in ((1, [2]), (2, [2, 7]), (3, [2, 4, 7]), (5, [1, 2, 4, 6, 7])):
        rows, short = orc.kv4_evict(pos, mass, n, 1, [8])
        assert rows[0, 0].tolist() == want and not short
    rows, short = orc.kv4_evict(pos, mass, 6, 1, [8])
    assert rows[0, 0].tolist() == [1, 2, 4, 6, 7, -1] and short


# --------------------------------------------------------------------- host-only queries
def test_workspace_sizes():
    assert P.pbsa_qk_workspace_size(P.make_qk_config(1, 0, 2, 2, 64, table_len=1)) == 2 * 64 * 4
    assert P.pbsa_qk_workspace_size(P.make_qk_config(4, 4096, 12, 12, 128, table_len=1)) >= 148 * 2 * 128 * 4
    c = P.make_kv4_config(1, 8, 8, 128, 65536)
    assert P.pbsa_kv4_workspace_size(c, 0) == 0
    assert P.pbsa_kv4_workspace_size(c, 1) >= 8 * 2 * 128 * 4      # at least two splits


@pytest.mark.parametrize("over,code", [
    (dict(D=96), P.PBSA_ERR_UNSUPPORTED), (dict(B=0), P.PBSA_ERR_ARG), (dict(T=-1), P.PBSA_ERR_ARG),
    (dict(Hq=0), P.PBSA_ERR_ARG), (dict(Hkv=-1), P.PBSA_ERR_ARG), (dict(eps=0.0), P.PBSA_ERR_ARG),
    (dict(eps=float("nan")), P.PBSA_ERR_ARG), (dict(rot_dim=24), P.PBSA_ERR_UNSUPPORTED),
    (dict(rot_dim=144), P.PBSA_ERR_ARG), (dict(table_len=0), P.PBSA_ERR_ARG),
    (dict(axis_pairs=(64, 1)), P.PBSA_ERR_ARG), (dict(axis_pairs=(65, -1)), P.PBSA_ERR_ARG),
    (dict(grad_dtype=torch.float16), P.PBSA_ERR_UNSUPPORTED),
    (dict(B=65536, T=65536, Hq=65535), P.PBSA_ERR_UNSUPPORTED),
    # 65535 heads of 2^62 - 2^32 + 1 tokens: in 64 bits a negative number
    (dict(B=2 ** 31 - 1, T=2 ** 31 - 1, Hq=65533), P.PBSA_ERR_UNSUPPORTED),
])
def test_bad_head_configs_are_refused(over, code):
    kw = dict(B=1, T=4, Hq=2, Hkv=2, D=128, table_len=8)
    kw.update(over)
    with pytest.raises(P.PBSAError) as e:
        P._check(P.library().pbsa_qk_norm_rope(
            ctypes.byref(P.make_qk_config(**kw)), 256, 256, None, 256, 256, 256, 256, 256, 256, 256,
            256, None))
    assert e.value.code == code and P.pbsa_last_error()


@pytest.mark.parametrize("over,code", [
    (dict(D=80), P.PBSA_ERR_UNSUPPORTED), (dict(Hq=6, Hkv=4), P.PBSA_ERR_ARG),
    (dict(B=0), P.PBSA_ERR_ARG), (dict(Hkv=0), P.PBSA_ERR_ARG), (dict(capacity=0), P.PBSA_ERR_ARG),
    (dict(capacity=100), P.PBSA_ERR_ARG), (dict(dtype=torch.float32), P.PBSA_ERR_UNSUPPORTED),
    (dict(k_unit=3.0), P.PBSA_ERR_ARG), (dict(v_unit=0.0), P.PBSA_ERR_ARG),
    (dict(v_unit=-1.0), P.PBSA_ERR_ARG), (dict(k_unit=2.0 ** 41), P.PBSA_ERR_ARG),
    (dict(k_unit=2.0 ** -41), P.PBSA_ERR_ARG), (dict(v_unit=math.inf), P.PBSA_ERR_ARG),
    (dict(v_unit=math.nan), P.PBSA_ERR_ARG),
    (dict(B=65535, Hq=65535, Hkv=65535), P.PBSA_ERR_UNSUPPORTED),
])
def test_bad_cache_configs_are_refused(over, code):
    kw = dict(B=1, Hq=4, Hkv=4, D=128, capacity=64)
    kw.update(over)
    with pytest.raises(P.PBSAError) as e:
        P.pbsa_validate_kv4_config(P.make_kv4_config(**kw))
    assert e.value.code == code
    P.pbsa_validate_kv4_config(P.make_kv4_config(1, 4, 4, 128, 64, k_unit=2.0 ** 40, v_unit=2.0 ** -40))


def _cache(**over):
    c = P.pbsa_kv4_cache(256, 256, 256, 256, 256)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def test_bad_pointers_and_sizes_are_refused_before_any_launch():
    lib, ref = P.library(), ctypes.byref
    qc, kc, ok = P.make_qk_config(1, 4, 2, 2, 64, table_len=8), P.make_kv4_config(1, 4, 2, 64, 64), _cache()

    def refused(rc, word, code=P.PBSA_ERR_ARG):
        assert rc == code, rc
        assert word in P.pbsa_last_error(), P.pbsa_last_error()

    fwd = [256] * 2 + [None] + [256] * 8 + [None]
    for i, name in ((0, "q"), (1, "k"), (5, "cos"), (6, "sin"), (7, "pos"), (8, "q_out"), (9, "k_out"),
                    (10, "status")):
        for bad, word in ((None, "NULL"), (264, "aligned")):
            refused(lib.pbsa_qk_norm_rope(ref(qc), *fwd[:i], bad, *fwd[i + 1:]), f"{name} is {'NULL' if bad is None else 'not'}")
    refused(lib.pbsa_qk_norm_rope(ref(qc), *fwd[:3], 264, *fwd[4:]), "wq")
    strides = (ctypes.c_int64 * 12)(*([512, 128, 64] * 4))
    for i, bad in ((1, 130), (4, -128), (9, 4)):
        s = (ctypes.c_int64 * 12)(*strides)
        s[i] = bad
        refused(lib.pbsa_qk_norm_rope(ref(qc), 256, 256, s, *fwd[3:]), "stride")
    bwd = [256] * 2 + [None] + [256] * 12
    refused(lib.pbsa_qk_norm_rope_bwd(ref(qc), *bwd, 16, 256, None), "workspace", P.PBSA_ERR_WORKSPACE)
    refused(lib.pbsa_qk_norm_rope_bwd(ref(qc), *bwd[:8], None, *bwd[9:], 1 << 20, 256, None), "dq_out")
    refused(lib.pbsa_qk_norm_rope_bwd(ref(qc), *bwd[:-1], None, 1 << 20, 256, None), "workspace")
    for name, _ in P.pbsa_kv4_cache._fields_:
        for bad in (None, 8):
            refused(lib.pbsa_kv4_append(ref(kc), ref(_cache(**{name: bad})), 256, 256, None, 4, 256, 256,
                                        256, 256, None), name)
    for i, name in ((0, "k_new"), (1, "v_new"), (4, "pos_new"), (7, "status")):
        args = [256, 256, None, 4, 256, 256, 256, 256]
        args[i] = None
        refused(lib.pbsa_kv4_append(ref(kc), ref(ok), *args, None), name)
    refused(lib.pbsa_kv4_append(ref(kc), ref(ok), 256, 256, None, -1, 256, 256, 256, 256, None), "T -1")
    refused(lib.pbsa_kv4_append(ref(kc), None, 256, 256, None, 1, 256, 256, 256, 256, None), "cache")
    refused(lib.pbsa_kv4_read(ref(kc), ref(ok), None, 65, 256, 256, 256, None), "capacity")
    refused(lib.pbsa_kv4_read(ref(kc), ref(ok), 256, -1, 256, 256, 256, None), "n -1")
    refused(lib.pbsa_kv4_read(ref(kc), ref(ok), 256, 1, None, 256, 256, None), "k_out")
    need = P.pbsa_kv4_workspace_size(kc, 3)
    attn = [256, None, 3, 256, 256, 256, 256, 256, 256, need, 256]
    for i, name in ((0, "q"), (4, "kv_len"), (5, "out"), (6, "lse"), (8, "workspace"), (10, "status")):
        args = list(attn)
        args[i] = None
        refused(lib.pbsa_kv4_attn(ref(kc), ref(ok), *args, None), name)
    args = list(attn)
    args[9] = need - 1
    refused(lib.pbsa_kv4_attn(ref(kc), ref(ok), *args, None), "workspace", P.PBSA_ERR_WORKSPACE)
    args = list(attn)
    args[2] = 1 << 20
    refused(lib.pbsa_kv4_attn(ref(kc), ref(ok), *args, None), "too many", P.PBSA_ERR_UNSUPPORTED)
    # a call whose pieces of work cannot be counted in 31 bits
    big = P.make_kv4_config(1024, 64, 1, 128, 131072)
    assert P.library().pbsa_kv4_workspace_size(ref(big), 16384) == 0 and "too many" in P.pbsa_last_error()
    for n, sink, word in ((-1, 0, "n -1"), (65, 0, "n 65"), (1, -1, "n_sink")):
        refused(lib.pbsa_kv4_evict(ref(kc), 256, 256, n, sink, None, 256, 256, None), word)
    for i, name in ((0, "pos"), (1, "mass"), (5, "rows"), (6, "status")):
        args = [256, 256, 1, 0, 256, 256, 256]
        args[i] = None
        refused(lib.pbsa_kv4_evict(ref(kc), *args, None), name)


def test_empty_calls_need_no_tensors():
    lib, ref = P.library(), ctypes.byref
    qc, kc = P.make_qk_config(1, 0, 2, 2, 64, table_len=8), P.make_kv4_config(1, 4, 2, 64, 64)
    assert lib.pbsa_qk_norm_rope(ref(qc), *[None] * 12) == P.PBSA_OK
    assert lib.pbsa_qk_norm_rope_bwd(ref(qc), *[None] * 15, 0, None, None) == P.PBSA_OK
    assert lib.pbsa_kv4_append(ref(kc), None, None, None, None, 0, None, None, None, None, None) == P.PBSA_OK
    assert lib.pbsa_kv4_read(ref(kc), None, None, 0, None, None, None, None) == P.PBSA_OK
    assert lib.pbsa_kv4_attn(ref(kc), None, None, None, 0, None, None, None, None, None, None, 0, None, None) == P.PBSA_OK
    assert lib.pbsa_kv4_evict(ref(kc), None, None, 0, 0, None, None, None, None) == P.PBSA_OK


def test_binding_refuses_tensors_that_do_not_fit():
    """Shapes, types, layouts and devices, seen on CPU tensors: the call itself never happens."""
    kc = P.make_kv4_config(2, 4, 2, 64, 64)
    u8 = dict(dtype=torch.uint8)
    t = dict(k_codes=torch.zeros(2, 2, 64, 32, **u8), k_scales=torch.zeros(2, 2, 64, 4, **u8),
             v_codes=torch.zeros(2, 2, 64, 32, **u8), v_scales=torch.zeros(2, 2, 64, 4, **u8),
             pos=torch.zeros(2, 2, 64, dtype=torch.int32))
    for name, bad in (("k_codes", torch.zeros(2, 2, 64, 64, **u8)), ("v_scales", t["v_scales"].int()),
                      ("pos", t["pos"].long()), ("k_scales", torch.zeros(2, 2, 4, 64, **u8).transpose(2, 3))):
        with pytest.raises(P.PBSAError, match=name):
            P.make_kv4_cache(kc, **{**t, name: bad})
    cache = P.make_kv4_cache(kc, **t)
    st = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(P.PBSAError, match="not on a CUDA device"):
        P.pbsa_kv4_append(kc, cache, k, k, pos, None, None, st)
    for args, name in (((k.half(), k, pos, None, None), "k_new"), ((k, k[:, :2], pos, None, None), "v_new"),
                       ((k, k, pos.long(), None, None), "pos_new"), ((k, k, pos, pos, None), "rows"),
                       ((k, k, pos, None, t["pos"].float()[:1]), "mass"),
                       ((k.transpose(2, 3).contiguous().transpose(2, 3), k, pos, None, None), "channels")):
        with pytest.raises(P.PBSAError, match=name):
            P.pbsa_kv4_append(kc, cache, *args, st)
    with pytest.raises(P.PBSAError, match="does not belong"):
        P.pbsa_kv4_append(P.make_kv4_config(2, 4, 2, 64, 128), cache, k, k, pos, None, None, st)
    qc = P.make_qk_config(2, 3, 2, 2, 64, table_len=8)
    table = torch.zeros(8, 32)
    xyz = torch.zeros(2, 3, 1, dtype=torch.int32)
    w = torch.ones(64)
    good = [k, k, w, w, table, table, xyz, k, k]
    for i, bad, name in ((0, k[:1], "q"), (2, w.double(), "q_weight"), (4, table[:7], "cos"),
                         (5, None, "needed"), (6, xyz.expand(2, 3, 3), "pos"), (8, k.float(), "k_out")):
        args = list(good)
        args[i] = bad
        with pytest.raises(P.PBSAError, match=name):
            P.pbsa_qk_norm_rope(qc, *args, st)
    with pytest.raises(P.PBSAError, match="share memory"):
        P.pbsa_qk_norm_rope(qc, *good[:7], k[:, :1].expand(2, 3, 2, 64), k, st)
    with pytest.raises(P.PBSAError):
        P.make_qk_config(2, 3, 2, 2, 64, axis_pairs=(8, 8, 8, 8))


def test_quick_calls_leave_alone_what_is_not_on_the_device():
    """The module behind the binding makes no call over CPU tensors, and none for no device."""
    from block_sparse_attention_35_b200 import token_calls as C
    cfg = P.make_qk_config(1, 1, 1, 1, 64, rot_dim=0)
    x, st = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    args = (x, x, None, None, None, None, None, x, x, st)
    for dev in (-1, 0):
        assert C.qk_norm_rope(ctypes.addressof(cfg), dev, 0, *args) is None
    assert C.qk_norm_rope(ctypes.addressof(cfg), 0, "stream", *args) is None
    assert C.qk_norm_rope(ctypes.addressof(cfg), 0, 0, *([None] * 10)) is None
    for f in (C.qk_norm_rope, C.qk_norm_rope_bwd, C.kv4_append, C.kv4_read, C.kv4_attn, C.kv4_evict):
        with pytest.raises(TypeError):
            f(ctypes.addressof(cfg), 0)

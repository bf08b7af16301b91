"""The cases that the token-cache operators are timed and compared on, with their plain forms.

Four operators (include/pbsa.h):

* ``qk``     - RMS norm of every query and key head with the position rotation in the same
               pass (pbsa_qk_norm_rope), and in training its backward pass too;
* ``append`` - new keys and values quantised to 4 bits and written into given rows of a
               cache (pbsa_kv4_append), then read back as the values they stand for
               (pbsa_kv4_read);
* ``attn``   - attention of a few or many query tokens over such a cache, with the
               probability that every cached row drew (pbsa_kv4_attn);
* ``evict``  - the rows that the next tokens will take: empty ones, then those with the least
               accumulated probability (pbsa_kv4_evict).

The 4-bit format: 16 consecutive channels share one scale.  scale = e4m3(amax / 6 / unit), a
channel is the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} to x / unit / scale (ties to the even
code), unit a power of two per cache; channel 2i of a row is the low nibble of byte i.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_FRAME_H, _FRAME_W = 30, 52          # token grid of one video frame
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one generated token: 12 query and key heads, where only latency counts
        dict(name="qk_step", op="qk", train=False, B=1, T=1, Hq=12, Hkv=12, D=128, dtype="bf16",
             rot=128, interleaved=False, axes=1, fused=False),
        # a training batch of an odd length, queries and keys views of one projection's
        # output, five key heads for twenty query heads, half of each head rotated
        dict(name="qk_train_odd", op="qk", train=True, B=3, T=777, Hq=20, Hkv=5, D=64,
             dtype="fp16", rot=32, interleaved=False, axes=1, fused=True),
        # the longest training sequence (21 frames of 30 x 52 tokens), rotated by frame, row
        # and column, with the attention's fp32 gradients coming back
        dict(name="qk_train", op="qk", train=True, B=1, T=32760, Hq=12, Hkv=12, D=128,
             dtype="bf16", rot=128, interleaved=True, axes=3, fused=False),
        # one token of each of 32 sequences enters their caches
        dict(name="append_step", op="append", B=32, T=1, Hkv=8, D=128, dtype="bf16", N=8192,
             unit=1.0, padded=False),
        # a chunk of three frames enters the cache
        dict(name="append_chunk", op="append", B=1, T=4680, Hkv=12, D=128, dtype="bf16", N=18752,
             unit=0.25, padded=False),
        # one token over a short cache: latency
        dict(name="attn_one", op="attn", B=1, T=1, Hq=12, Hkv=12, D=128, dtype="bf16", N=4096,
             causal=False, mass=False, ragged=False),
        # five drafted tokens a sequence, a causal mask among them, ragged lengths
        dict(name="attn_draft", op="attn", B=8, T=5, Hq=20, Hkv=5, D=64, dtype="fp16", N=1600,
             causal=True, mass=True, ragged=True),
        # a serving batch of ragged lengths that also keeps the accounts for eviction
        dict(name="attn_batch", op="attn", B=32, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", N=8192,
             causal=False, mass=True, ragged=True),
        # one sequence with a long cache
        dict(name="attn_long", op="attn", B=1, T=1, Hq=32, Hkv=4, D=128, dtype="bf16", N=131072,
             causal=False, mass=False, ragged=False),
        # one frame's queries over the whole video cache
        dict(name="attn_chunk", op="attn", B=1, T=1560, Hq=12, Hkv=12, D=128, dtype="bf16",
             N=18752, causal=False, mass=True, ragged=False),
        # room for one token in each of 32 full caches
        dict(name="evict_step", op="evict", B=32, Hkv=8, N=8192, n=1, n_sink=4, n_recent=64),
        # room for a frame in the video cache
        dict(name="evict_chunk", op="evict", B=1, Hkv=12, N=18752, n=1560, n_sink=1560,
             n_recent=4680),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk", "append", "attn", "attn", "evict"])
    D = rng.choice([64, 128])
    if op == "qk":
        Hq, Hkv = rng.choice([(12, 12), (20, 5), (32, 8), (8, 1), (7, 7), (24, 2)])
        B = rng.randint(1, 8)
        T = _log_int(rng, 1, max(1, 32760 * 24 * 128 // (B * (Hq + Hkv) * D)))
        return dict(op="qk", train=rng.random() < 0.6, B=B, T=min(T, 32760), Hq=Hq, Hkv=Hkv, D=D,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    rot=rng.choice([D, D, D // 2, 48, 0]), interleaved=rng.random() < 0.5,
                    axes=rng.choice([1, 3]), fused=rng.random() < 0.4)
    if op == "append":
        B, Hkv = _log_int(rng, 1, 32), rng.choice([1, 5, 8, 12])
        N = 64 * _log_int(rng, 1, 293)
        T = min(N, _log_int(rng, 1, max(1, 4680 * 12 // (B * Hkv))))
        return dict(op="append", B=B, T=T, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "fp16"]), N=N,
                    unit=rng.choice([1.0, 0.25, 2.0 ** -6]), padded=rng.random() < 0.5)
    if op == "attn":
        Hq, Hkv = rng.choice([(12, 12), (20, 5), (32, 8), (32, 4), (8, 1), (7, 7), (48, 2)])
        B = _log_int(rng, 1, 32)
        N = 64 * _log_int(rng, 1, max(1, 2097152 // (64 * B * Hkv)))
        N = min(N, 131072)
        T = _log_int(rng, 1, max(1, min(1560, 1560 * 12 * 18752 // (B * Hq * N))))
        return dict(op="attn", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "fp16"]),
                    N=N, causal=rng.random() < 0.5, mass=rng.random() < 0.5,
                    ragged=rng.random() < 0.6)
    B, Hkv = _log_int(rng, 1, 32), rng.choice([1, 5, 8, 12])
    N = min(64 * _log_int(rng, 1, max(1, 2097152 // (64 * B * Hkv))), 131072)
    n = _log_int(rng, 1, max(1, min(1560, N // 4)))
    return dict(op="evict", B=B, Hkv=Hkv, N=N, n=n, n_sink=rng.choice([0, 4, N // 16]),
                n_recent=rng.choice([0, 16, N // 8]))


def lengths(case):
    """Rows in use of every sequence's cache: ragged ones shrink towards the last sequence,
    which is empty in a batch of four or more."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    out = [max(1, N * (B - b) // B - (37 * b) % 61) for b in range(B)]
    if B >= 4:
        out[-1] = 0
    return out


def _axis_pairs(case):
    p = case["rot"] // 2
    return (p,) if case["axes"] == 1 else (p - 2 * (p // 3), p // 3, p // 3)


def _table_len(case):
    return 40960 if case["axes"] == 1 else 64


def work(case):
    op = case["op"]
    if op == "qk":
        es = _BYTES[case["dtype"]]
        x = case["B"] * case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        pos = case["B"] * case["T"] * case["axes"] * 4 if case["rot"] else 0
        rows = _table_len(case) if case["axes"] == 3 else min(_table_len(case), case["B"] * case["T"])
        small = pos + rows * case["rot"] * 4 + 8 * case["D"]
        if not case["train"]:
            return dict(bytes=2 * x * es + small, flops=8 * x)
        ge = 4 if case["dtype"] == "bf16" else es
        return dict(bytes=3 * x * es + x * ge + small + 8 * case["D"], flops=26 * x)
    D = case.get("D", 128)
    row = D + D // 8                     # codes and scales of one row's key and value
    if op == "append":
        n = case["B"] * case["Hkv"] * case["T"]
        es = _BYTES[case["dtype"]]
        return dict(bytes=n * (2 * D * es + row + 2 * D * es + 12) + 4 * case["B"] * case["T"],
                    flops=8 * n * D)
    if op == "attn":
        rows = sum(lengths(case))
        es = _BYTES[case["dtype"]]
        q = case["B"] * case["T"] * case["Hq"]
        return dict(bytes=rows * case["Hkv"] * (row + 4 + (8 if case["mass"] else 0)) +
                    q * (2 * D * es + 4), flops=4 * rows * case["T"] * case["Hq"] * D)
    n = case["B"] * case["Hkv"]
    return dict(bytes=n * (case["N"] * 8 + case["n"] * 4), flops=4 * n * case["N"])


# ----------------------------------------------------------------------------- the format
def _quantise(x, unit):
    """Codes (one a channel) and e4m3 scale bytes of x [..., D], in 32-bit arithmetic."""
    g = x.float().reshape(*x.shape[:-1], -1, 16) / unit
    scale = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    r = torch.where(s > 0, g.abs() / s, torch.zeros_like(g))
    # nearest level; the ties go to the even code: up at 0.75, 1.75, 3.5
    code = ((r > 0.25).int() + (r >= 0.75).int() + (r > 1.25).int() + (r >= 1.75).int() +
            (r > 2.5).int() + (r >= 3.5).int() + (r > 5.0).int())
    code = code + 8 * (g < 0).int()
    return code.reshape(x.shape), scale.view(torch.uint8)


def _pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)


def _dequantise(codes, scales, unit):
    lut = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float32,
                       device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    v = lut[c].reshape(*scales.shape, 16)
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * unit


# ----------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_qk(case, seed):
    g = _gen(seed)
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    dt = _DT[case["dtype"]]
    H = Hq + Hkv
    gain = 0.5 + 1.5 * torch.rand(H, 1, generator=g, device="cuda")
    if case["fused"]:     # the projection's output: queries, keys and values of a token together
        qkv = (_randn(g, B, T, H + Hkv, D) * torch.cat((gain, gain[Hq:]))).to(dt)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:H]
    else:
        q = (_randn(g, B, T, Hq, D) * gain[:Hq]).to(dt)
        k = (_randn(g, B, T, Hkv, D) * gain[Hq:]).to(dt)
    s = dict(case=case, q=q, k=k, wq=1 + 0.1 * _randn(g, D), wk=1 + 0.1 * _randn(g, D))
    s["cos"] = s["sin"] = s["pos"] = None
    if case["rot"]:
        n = _table_len(case)
        inv = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64, device="cuda") / max(p, 1))
                         for p in _axis_pairs(case)])
        ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        t = torch.arange(T, device="cuda")
        if case["axes"] == 1:
            start = torch.randint(0, n - T, (B, 1, 1), generator=g, device="cuda")
            s["pos"] = (t[None, :, None] + start).int()
        else:
            start = torch.randint(0, 40, (B, 1), generator=g, device="cuda")
            tf = _FRAME_H * _FRAME_W
            xyz = (t // tf + start, (t % tf // _FRAME_W).expand(B, T), (t % _FRAME_W).expand(B, T))
            s["pos"] = torch.stack(xyz, -1).int().contiguous()
    if case["train"]:     # the attention backward's gradients; fp32 beside bf16
        gt = torch.float32 if case["dtype"] == "bf16" else dt
        s["dq_out"] = (0.1 * _randn(g, B, T, Hq, D)).to(gt)
        s["dk_out"] = (0.1 * _randn(g, B, T, Hkv, D)).to(gt)
    if own:
        from block_sparse_attention_35_b200 import pbsa as P
        c = P.make_qk_config(B, T, Hq, Hkv, D, dtype=dt, rot_dim=case["rot"],
                             interleaved=case["interleaved"],
                             axis_pairs=_axis_pairs(case) if case["rot"] else (0,),
                             table_len=_table_len(case) if case["rot"] else 0, eps=1e-6,
                             grad_dtype=s["dq_out"].dtype if case["train"] else dt)
        s.update(cfg=c, q_out=torch.empty_like(q, memory_format=torch.contiguous_format),
                 k_out=torch.empty_like(k, memory_format=torch.contiguous_format),
                 status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if case["train"]:
            s.update(dq=torch.empty_like(s["q_out"]), dk=torch.empty_like(s["k_out"]),
                     dwq=torch.empty(D, device="cuda"), dwk=torch.empty(D, device="cuda"),
                     ws=torch.empty(P.pbsa_qk_workspace_size(c), dtype=torch.uint8, device="cuda"))
    return s


def _random_cache(case, g):
    """A cache with plausible contents: codes of a sixteen-channel block, scales around 1/4."""
    B, Hkv, N, D = (case[k] for k in ("B", "Hkv", "N", "D"))
    u8 = dict(generator=g, device="cuda", dtype=torch.uint8)
    return dict(k_codes=torch.randint(0, 256, (B, Hkv, N, D // 2), **u8),
                k_scales=torch.randint(32, 56, (B, Hkv, N, D // 16), **u8),
                v_codes=torch.randint(0, 256, (B, Hkv, N, D // 2), **u8),
                v_scales=torch.randint(32, 56, (B, Hkv, N, D // 16), **u8))


def _kv4(case, s, Hq, dt, unit):
    """The configuration and cache handle that a program keeps beside the cache's tensors."""
    from block_sparse_attention_35_b200 import pbsa as P
    s["cfg"] = P.make_kv4_config(case["B"], Hq, case["Hkv"], case["D"], case["N"], dtype=dt,
                                 k_unit=unit, v_unit=unit)
    s["cache"] = P.make_kv4_cache(s["cfg"], s["k_codes"], s["k_scales"], s["v_codes"],
                                  s["v_scales"], s["pos"])
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return P


def _prepare_append(case, seed):
    g = _gen(seed)
    B, Hkv, N, D, T = (case[k] for k in ("B", "Hkv", "N", "D", "T"))
    dt = _DT[case["dtype"]]
    s = dict(case=case, **_random_cache(case, g))
    # keys after norm and rotation have a few strong channels, values are small
    strong = 1 + 4 * (torch.rand(Hkv, D, generator=g, device="cuda") > 0.95)
    s["k_new"] = (_randn(g, B, T, Hkv, D) * strong).to(dt)
    s["v_new"] = (0.5 * _randn(g, B, T, Hkv, D) * torch.rand(B, T, 1, 1, generator=g, device="cuda")).to(dt)
    s["pos"] = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, Hkv, N).contiguous()
    s["mass"] = torch.rand(B, Hkv, N, generator=g, device="cuda")
    order = torch.rand(B, Hkv, N, generator=g, device="cuda").argsort(-1)
    s["rows"] = order[..., :T].sort(-1).values.int().contiguous()
    pos = (N + torch.arange(T, device="cuda")).expand(B, T).int().contiguous()
    if case["padded"]:    # sequences of different lengths: their last places hold no token
        n = torch.randint(0, T + 1, (B, 1), generator=g, device="cuda")
        pos = torch.where(torch.arange(T, device="cuda") < n, pos, torch.full_like(pos, -1))
    s["pos_new"] = pos
    if own:
        _kv4(case, s, Hkv, dt, case["unit"])
        s["k_read"] = torch.empty(B, Hkv, T, D, dtype=dt, device="cuda")
        s["v_read"] = torch.empty_like(s["k_read"])
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, Hq, Hkv, N, D, T = (case[k] for k in ("B", "Hq", "Hkv", "N", "D", "T"))
    dt = _DT[case["dtype"]]
    s = dict(case=case)
    strong = 1 + 2 * (torch.rand(Hkv, 1, D, generator=g, device="cuda") > 0.95)
    for x in "kv":
        codes = torch.empty(B, Hkv, N, D // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(B, Hkv, N, D // 16, dtype=torch.uint8, device="cuda")
        for b in range(B):
            data = _randn(g, Hkv, N, D) * (strong if x == "k" else 0.5)
            c, scales[b] = _quantise(data, 1.0)
            codes[b] = _pack(c)
        s[x + "_codes"], s[x + "_scales"] = codes, scales
    s["q"] = _randn(g, B, T, Hq, D).to(dt)
    lens = torch.tensor(lengths(case), device="cuda")
    s["kv_len"] = lens.int()
    # after evictions the rows are in no order and a few are empty
    seen = 2 * N
    pos = torch.rand(B, Hkv, seen, generator=g, device="cuda").argsort(-1)[..., :N].int()
    gone = torch.rand(B, Hkv, N, generator=g, device="cuda") < 0.02
    s["pos"] = torch.where(gone, torch.full_like(pos, -1), pos).contiguous()
    s["q_pos"] = None
    if case["causal"]:
        # the last rows in use hold the T newest tokens, which are the queries
        qp = (seen + torch.arange(T, device="cuda")).expand(B, T).int().contiguous()
        for b, n in enumerate(lengths(case)):
            m = min(n, T)
            if m:
                s["pos"][b, :, n - m:n] = qp[b, T - m:]
        if T > 2:         # a shorter draft in the first sequence: its last place is no token
            qp[0, -1] = -1
        s["q_pos"] = qp
    if case["mass"]:
        s["mass"] = torch.rand(B, Hkv, N, generator=g, device="cuda")
    if own:
        P = _kv4(case, s, Hq, dt, 1.0)
        s["out"] = torch.empty(B, T, Hq, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(B, Hq, T, device="cuda")
        s["ws"] = torch.empty(P.pbsa_kv4_workspace_size(s["cfg"], T), dtype=torch.uint8, device="cuda")
    return s


def _prepare_evict(case, seed):
    g = _gen(seed)
    B, Hkv, N = (case[k] for k in ("B", "Hkv", "N"))
    # most rows drew next to nothing, a few a lot; new rows draw nothing yet
    mass = torch.exp(3 * _randn(g, B, Hkv, N) - 6)
    mass[torch.rand(B, Hkv, N, generator=g, device="cuda") < 0.01] = 0
    pos = torch.rand(B, Hkv, 2 * N, generator=g, device="cuda").argsort(-1)[..., :N].int()
    empty = torch.rand(B, Hkv, N, generator=g, device="cuda") < 1.0 / N
    s = dict(case=case, mass=mass,
             pos=torch.where(empty, torch.full_like(pos, -1), pos).contiguous())
    s["keep_from"] = torch.full((B,), 2 * N - case["n_recent"], dtype=torch.int32, device="cuda")
    if own:
        from block_sparse_attention_35_b200 import pbsa as P
        s["cfg"] = P.make_kv4_config(B, Hkv, Hkv, 128, N, dtype=torch.bfloat16)
        s["rows"] = torch.empty(B, Hkv, case["n"], dtype=torch.int32, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    return {"qk": _prepare_qk, "append": _prepare_append, "attn": _prepare_attn,
            "evict": _prepare_evict}[case["op"]](case, seed)


# --------------------------------------------------------------------------- the operators
def _angles(s):
    """cos and sin of every token's pairs [B, T, 1, rot / 2]."""
    case = s["case"]
    axis = torch.cat([torch.full((p,), a, device="cuda") for a, p in enumerate(_axis_pairs(case))])
    row = s["pos"].long()[..., axis]                          # [B, T, rot / 2]
    col = torch.arange(case["rot"] // 2, device="cuda")
    return s["cos"][row, col].unsqueeze(2), s["sin"][row, col].unsqueeze(2)


def _pairs(x, case):
    r = case["rot"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2]
    return x[..., :r // 2], x[..., r // 2:r]


def _unpairs(a, b, x, case):
    r = case["rot"]
    head = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((head, x[..., r:]), -1)


def _plain_qk(s):
    case = s["case"]
    rot = case["rot"] > 0
    if rot:
        c, sn = _angles(s)
    outs, dxs, dws = [], [], []
    for x, w, gy in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        xn = xf * r
        y = xn * w
        if rot:
            a, b = _pairs(y, case)
            y = _unpairs(a * c - b * sn, b * c + a * sn, y, case)
        outs.append(y.to(x.dtype))
        if case["train"]:
            gn = gy.float()
            if rot:
                a, b = _pairs(gn, case)
                gn = _unpairs(a * c + b * sn, b * c - a * sn, gn, case)
            dws.append((gn * xn).sum((0, 1, 2)))
            gw = gn * w
            dxs.append((r * (gw - xn * (gw * xn).mean(-1, keepdim=True))).to(x.dtype))
    return outs + dxs + dws


def _own_qk(s):
    from block_sparse_attention_35_b200 import pbsa as P
    P.pbsa_qk_norm_rope(s["cfg"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                        s["q_out"], s["k_out"], s["status"])
    if not s["case"]["train"]:
        return [s["q_out"], s["k_out"]]
    P.pbsa_qk_norm_rope_bwd(s["cfg"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
                            s["pos"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["dwq"],
                            s["dwk"], s["ws"], s["status"])
    return [s["q_out"], s["k_out"], s["dq"], s["dk"], s["dwq"], s["dwk"]]


def _plain_append(s):
    case, unit = s["case"], s["case"]["unit"]
    dt = _DT[case["dtype"]]
    rows = s["rows"].long()
    live = (s["pos_new"] >= 0)[:, None, :].expand(rows.shape)
    out = []
    for x in "kv":
        code, scale = _quantise(s[x + "_new"].transpose(1, 2), unit)
        new = (_pack(code), scale)
        for t, n in zip((s[x + "_codes"], s[x + "_scales"]), new):
            at = rows.unsqueeze(-1).expand(n.shape)
            t.scatter_(2, at, torch.where(live.unsqueeze(-1), n, t.gather(2, at)))
        codes, scales = (t.gather(2, rows.unsqueeze(-1).expand(n.shape))
                         for t, n in zip((s[x + "_codes"], s[x + "_scales"]), new))
        out.append(_dequantise(codes, scales, unit).to(dt))
    s["pos"].scatter_(2, rows, torch.where(live, s["pos_new"][:, None, :].expand(rows.shape),
                                           s["pos"].gather(2, rows)))
    s["mass"].scatter_(2, rows, torch.where(live, torch.zeros_like(s["mass"][:, :, :1]),
                                            s["mass"].gather(2, rows)))
    return out + [s["pos"], s["mass"]]


def _own_append(s):
    from block_sparse_attention_35_b200 import pbsa as P
    P.pbsa_kv4_append(s["cfg"], s["cache"], s["k_new"], s["v_new"], s["pos_new"], s["rows"],
                      s["mass"], s["status"])
    P.pbsa_kv4_read(s["cfg"], s["cache"], s["rows"], s["k_read"], s["v_read"], s["status"])
    return [s["k_read"], s["v_read"], s["pos"], s["mass"]]


def _visible(s):
    """[B, Hkv, 1 or T, N]: the rows that a query token sees."""
    N = s["case"]["N"]
    pos = s["pos"]
    see = (pos >= 0) & (torch.arange(N, device="cuda") < s["kv_len"][:, None, None])
    see = see.unsqueeze(2)
    if s["q_pos"] is not None:
        see = see & (pos.unsqueeze(2) <= s["q_pos"][:, None, :, None])
    return see


def _plain_attn(s):
    case = s["case"]
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    k = _dequantise(s["k_codes"], s["k_scales"], 1.0)
    q = s["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    sc = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)).view(B, Hkv, G, T, -1)
    del k
    see = _visible(s).unsqueeze(2)
    sc = torch.where(see, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(sc - m)
    del sc
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    v = _dequantise(s["v_codes"], s["v_scales"], 1.0)
    o = torch.matmul(p.view(B, Hkv, G * T, -1), v).view(B, Hkv, G, T, D)
    out = [o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(_DT[case["dtype"]]),
           lse.reshape(B, Hq, T)]
    if case["mass"]:
        out.append(s["mass"] + p.sum((2, 3)))
    return out


def _own_attn(s):
    from block_sparse_attention_35_b200 import pbsa as P
    # the pass adds to a copy, so that it can be repeated on the same inputs
    mass = s["mass"].clone() if s["case"]["mass"] else None
    P.pbsa_kv4_attn(s["cfg"], s["cache"], s["q"], s["q_pos"], s["kv_len"], s["out"], s["lse"],
                    mass, s["ws"], s["status"])
    return [s["out"], s["lse"]] + ([mass] if mass is not None else [])


def _plain_evict(s):
    case = s["case"]
    pos, mass = s["pos"], s["mass"].clamp(min=0)
    # 0: empty, 1: may go, 2: stays
    kind = torch.where(pos < 0, 0, torch.where(
        (pos < case["n_sink"]) | (pos >= s["keep_from"][:, None, None]), 2, 1))
    mass = torch.where(kind == 1, mass, torch.zeros_like(mass))
    by_mass = torch.sort(mass, dim=-1, stable=True).indices
    by_kind = torch.sort(kind.gather(-1, by_mass), dim=-1, stable=True)
    rows = by_mass.gather(-1, by_kind.indices)[..., :case["n"]]
    free = by_kind.values[..., :case["n"]] < 2
    rows = torch.where(free, rows, torch.full_like(rows, case["N"])).sort(-1).values
    return [torch.where(rows < case["N"], rows, torch.full_like(rows, -1)).int()]


def _own_evict(s):
    from block_sparse_attention_35_b200 import pbsa as P
    P.pbsa_kv4_evict(s["cfg"], s["pos"], s["mass"], s["case"]["n_sink"], s["keep_from"],
                     s["rows"], s["status"])
    return [s["rows"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"qk": _own_qk, "append": _own_append, "attn": _own_attn, "evict": _own_evict}[op](state)
    return {"qk": _plain_qk, "append": _plain_append, "attn": _plain_attn,
            "evict": _plain_evict}[op](state)


# ------------------------------------------------------------------ the definitions, 64 bits
def _exact_qk(case, s):
    outs, dxs, dws = [], [], []
    r = case["rot"]
    if r:
        pairs = _axis_pairs(case)
        cs = torch.complex(s["cos"].double(), s["sin"].double())
        cols = torch.split(torch.arange(r // 2, device="cuda"), pairs)
        turn = torch.cat([cs[s["pos"][..., a].long()][..., c] for a, c in enumerate(cols)], -1)
    for x, w, gy in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
        xd = x.double().requires_grad_(case["train"])
        wd = w.double().requires_grad_(case["train"])
        y = xd / torch.sqrt(xd.square().sum(-1, keepdim=True) / case["D"] + 1e-6) * wd
        if r:
            if case["interleaved"]:
                z = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous())
                z = torch.view_as_real(z * turn.unsqueeze(2)).flatten(-2)
            else:
                z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * turn.unsqueeze(2)
                z = torch.cat((z.real, z.imag), -1)
            y = torch.cat((z, y[..., r:]), -1)
        outs.append(y.detach())
        if case["train"]:
            gx, gw = torch.autograd.grad(y, (xd, wd), gy.double())
            dxs.append(gx)
            dws.append(gw)
    return outs + dxs + dws


def _e4m3_values():
    v = np.arange(127)                       # 0x00 .. 0x7e, the finite non-negative codes
    e, m = v >> 3, v & 7
    return torch.tensor(np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0)), device="cuda")


def _nearest(x, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    hi = torch.searchsorted(table, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dh, dl = (table[hi] - x).abs(), (x - table[lo]).abs()
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _exact_append(case, s):
    rows, unit = s["rows"].long(), case["unit"]
    live = (s["pos_new"] >= 0)[:, None, :].expand(rows.shape)
    e4m3 = _e4m3_values()
    levels = torch.tensor(_LEVELS, dtype=torch.float64, device="cuda")
    out = []
    for x in "kv":
        g = s[x + "_new"].double().transpose(1, 2).unflatten(-1, (-1, 16)) / unit
        sc = e4m3[_nearest(g.abs().amax(-1, keepdim=True) / 6, e4m3)]
        mag = levels[_nearest(g.abs() / torch.where(sc > 0, sc, torch.ones_like(sc)), levels)]
        new = (torch.sign(g) * mag * sc * unit).flatten(-2)
        codes, scales = s[x + "_codes"], s[x + "_scales"]
        codes = codes.gather(2, rows.unsqueeze(-1).expand(*rows.shape, codes.shape[-1])).long()
        scales = scales.gather(2, rows.unsqueeze(-1).expand(*rows.shape, scales.shape[-1])).long()
        nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
        old = levels[nib % 8] * (1 - 2 * (nib // 8)) * e4m3[scales].repeat_interleave(16, -1) * unit
        out.append(torch.where(live.unsqueeze(-1), new, old))
    pos, mass = s["pos"].clone(), s["mass"].double()
    b, h, t = torch.nonzero(live, as_tuple=True)
    pos[b, h, rows[b, h, t]] = s["pos_new"][b, t]
    mass[b, h, rows[b, h, t]] = 0
    return out + [pos, mass]


def _exact_attn(case, s):
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    e4m3 = _e4m3_values()
    levels = torch.tensor(_LEVELS, dtype=torch.float64, device="cuda")
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if case["mass"] else None

    def values(codes, scales):
        c = codes.long()
        nib = torch.stack((c % 16, c // 16), -1).flatten(-2)
        return levels[nib % 8] * (1 - 2 * (nib // 8)) * e4m3[scales.long()].repeat_interleave(16, -1)

    for b, n in enumerate(lengths(case)):
        for h in range(Hkv):
            at = torch.nonzero(s["pos"][b, h, :n] >= 0).flatten()
            if not len(at):
                continue
            k = values(s["k_codes"][b, h, at], s["k_scales"][b, h, at])
            v = values(s["v_codes"][b, h, at], s["v_scales"][b, h, at])
            hide = None
            if s["q_pos"] is not None:
                hide = s["pos"][b, h, at][None, :] > s["q_pos"][b][:, None]
            for j in range(h * G, (h + 1) * G):
                sc = s["q"][b, :, j].double() @ k.T / math.sqrt(D)
                if hide is not None:
                    sc = sc.masked_fill(hide, -math.inf)
                lse[b, j] = torch.logsumexp(sc, -1)
                p = torch.exp(sc - lse[b, j].unsqueeze(-1)).nan_to_num(0.0)
                out[b, :, j] = p @ v
                if mass is not None:
                    mass[b, h, at] += p.sum(0)
    return [out, lse] + ([mass] if mass is not None else [])


def _exact_evict(case, s):
    pos, mass = s["pos"].cpu().numpy(), s["mass"].cpu().numpy().astype(np.float64)
    keep = s["keep_from"].cpu().numpy()
    rows = np.full((case["B"], case["Hkv"], case["n"]), -1, np.int32)
    for b in range(case["B"]):
        for h in range(case["Hkv"]):
            p = pos[b, h]
            empty = np.flatnonzero(p < 0)[:case["n"]]
            may = np.flatnonzero((p >= case["n_sink"]) & (p < keep[b]))
            order = may[np.lexsort((may, np.maximum(mass[b, h, may], 0)))]
            got = np.sort(np.concatenate((empty, order[:case["n"] - len(empty)])))
            rows[b, h, :len(got)] = got
    return [torch.from_numpy(rows).cuda()]


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "append": _exact_append, "attn": _exact_attn,
            "evict": _exact_evict}[case["op"]](case, s)

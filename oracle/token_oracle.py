"""Plain fp64 numpy forms of the token operators: norm and rotation of heads, the 4-bit token
cache (quantise, attend, choose rows to evict).  Written from the formulas of include/pbsa.h
with loops where a loop is clearest; it shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

# ------------------------------------------------------------------ norm and rotation
def _turn(x, cos, sin, pos, rot_dim, interleaved, axis_pairs, back=False):
    """Rotates the first rot_dim channels of x [B, T, H, D] by every token's angles."""
    if rot_dim == 0:
        return x.copy()
    out = x.copy()
    p = rot_dim // 2
    i = 0
    for axis, n in enumerate(axis_pairs):
        for _ in range(n):
            c = cos[pos[..., axis], i][..., None]
            s = sin[pos[..., axis], i][..., None]
            s = -s if back else s
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + p)
            out[..., a] = x[..., a] * c - x[..., b] * s
            out[..., b] = x[..., b] * c + x[..., a] * s
            i += 1
    return out


def norm_rope(x, w, cos, sin, pos, rot_dim, interleaved, axis_pairs, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, cos, sin, pos, rot_dim, interleaved, axis_pairs)


def norm_rope_bwd(x, w, cos, sin, pos, rot_dim, interleaved, axis_pairs, eps, dy):
    """(dx, dw) of sum(norm_rope(x) * dy)."""
    D = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = _turn(dy, cos, sin, pos, rot_dim, interleaved, axis_pairs, back=True)
    dw = (g * x * r).reshape(-1, D).sum(0)
    dx = r * (g * w - x * r * r * (g * w * x).mean(-1, keepdims=True))
    return dx, dw


# ------------------------------------------------------------------------ 4-bit format
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def nearest(x: float, table) -> int:
    """Index of the nearest table entry to x >= 0, ties to the even index, saturating."""
    best = 0
    for i, t in enumerate(table):
        d, db = abs(t - x), abs(table[best] - x)
        if d < db or (d == db and i % 2 == 0):
            best = i
    return best


def quantise_row(x, unit):
    """(codes, scale bytes) of one row of D channels."""
    codes, scales = [], []
    for g in range(0, len(x), 16):
        v = [0.0 if math.isnan(t) else t / unit for t in x[g:g + 16]]
        amax = max(abs(t) for t in v)
        sb = 126 if math.isinf(amax) else nearest(amax / 6, E4M3)
        scales.append(sb)
        for t in v:
            c = nearest(min(abs(t) / E4M3[sb], 1e30), LEVELS) if E4M3[sb] > 0 else 0
            codes.append(c + 8 if t < 0 and E4M3[sb] > 0 else c)
    return codes, scales


def values(codes, scales, unit):
    """Values [..., D] of packed codes [..., D/2] and e4m3 scale bytes [..., D/16]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.asarray(LEVELS)[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    table = np.full(256, np.nan)
    table[:127] = E4M3
    table[128:255] = [-t for t in E4M3]
    return v * np.repeat(table[scales], 16, -1) * unit


# --------------------------------------------------------------------------- attention
def kv4_attn(q, k, v, pos, q_pos, kv_len):
    """q [B, T, Hq, D]; k, v [B, Hkv, N, D] values; returns out, lse, mass [B, Hkv, N] and, for
    tolerances, vabs = sum_j p |v| like out and qk = max_j sum_d |q k| / sqrt(D) like lse."""
    B, T, Hq, D = q.shape
    Hkv, N = k.shape[1:3]
    G = Hq // Hkv
    out = np.zeros(q.shape)
    vabs = np.zeros(q.shape)
    lse = np.full((B, Hq, T), -np.inf)
    qk = np.zeros((B, Hq, T))
    mass = np.zeros((B, Hkv, N))
    for b in range(B):
        for h in range(Hq):
            kh = h // G
            for t in range(T):
                see = (pos[b, kh] >= 0) & (np.arange(N) < kv_len[b])
                if q_pos is not None:
                    see &= pos[b, kh] <= q_pos[b, t]
                j = np.flatnonzero(see)
                if len(j) == 0:
                    continue
                s = k[b, kh, j] @ q[b, t, h] / math.sqrt(D)
                qk[b, h, t] = (np.abs(k[b, kh, j]) @ np.abs(q[b, t, h])).max() / math.sqrt(D)
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, t] = m + math.log(p.sum())
                p /= p.sum()
                out[b, t, h] = p @ v[b, kh, j]
                vabs[b, t, h] = p @ np.abs(v[b, kh, j])
                mass[b, kh, j] += p
    return out, lse, mass, vabs, qk


# ---------------------------------------------------------------------------- eviction
def kv4_evict(pos, mass, n, n_sink, keep_from):
    """rows [B, Hkv, n] and whether some sequence had fewer than n rows to give."""
    B, H, N = pos.shape
    rows = np.full((B, H, n), -1, np.int64)
    short = False
    for b in range(B):
        for h in range(H):
            order = []
            for j in range(N):
                p = pos[b, h, j]
                if p < 0:
                    order.append((0, 0.0, j))
                elif p >= n_sink and (keep_from is None or p < keep_from[b]):
                    m = mass[b, h, j]
                    order.append((1, math.inf, j) if math.isinf(m) and m > 0 else
                                 (2, 0.0, j) if math.isnan(m) else (1, max(m, 0.0), j))
            got = sorted(j for _, _, j in sorted(order)[:n])
            rows[b, h, :len(got)] = got
            short |= len(got) < n
    return rows, short

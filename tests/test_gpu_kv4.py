"""The 4-bit token cache on the GPU, through the C ABI, against the fp64 oracle.

The quantiser, the read-back and the eviction are exact.  Attention's tolerances, with A_r =
max_j sum_d |q_d k_jd| / sqrt(D) of a query row:
  E_r = 2^-19 A_r     error of a logit: products of fp16 operands are exact, 2 D / 16 <= 16
                      accumulating tensor-core steps lose at most 2^-23 of the partial sum each
  lse   |err| <= E_r + 2^-20 (1 + |lse|): exponentials and logarithm to 2 ulp, fp32 sums
  mass  |err| <= sum over rows of p (2 E_r + 2^-19 (1 + |lse|)) <= mass (2 max E + ...)
  out   |err| <= e |o| + (2 E_r + 2^-11 + 2^-18) sum_j p_j |v_j|: each probability is rounded to
        fp16 (2^-11), e = finfo.eps / 2 of the output's type; plus N 2^-32 max |v|: fp16 keeps
        multiples of 2^-24 of 2^(s - m + 7), so a probability is off by at most 2^-25 / 2^7 =
        2^-32 of its row's largest where it is too small for 11 bits."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from block_sparse_attention_35_b200.attention import rope_table
from block_sparse_attention_35_b200.token_cache import TokenCache
from oracle import token_oracle as orc

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Cache:
    """A cache with random contents (finite scales around 1/4)."""

    def __init__(self, dev, B=2, Hq=4, Hkv=2, D=128, N=64, dtype=torch.bfloat16, ku=1.0, vu=1.0, seed=0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.dev, self.B, self.Hq, self.Hkv, self.D, self.N, self.dtype = dev, B, Hq, Hkv, D, N, dtype
        self.cfg = P.make_kv4_config(B, Hq, Hkv, D, N, dtype, ku, vu)
        ri = lambda lo, hi, w: torch.randint(lo, hi, (B, Hkv, N, w), generator=g, dtype=torch.uint8).to(dev)
        self.kc, self.ks, self.vc, self.vs = ri(0, 256, D // 2), ri(30, 56, D // 16), ri(0, 256, D // 2), ri(30, 56, D // 16)
        self.pos = torch.stack([torch.randperm(2 * N, generator=g)[:N] for _ in range(B * Hkv)]).view(B, Hkv, N).int().to(dev)
        self.mass = torch.rand(B, Hkv, N, generator=g).to(dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cache = P.make_kv4_cache(self.cfg, self.kc, self.ks, self.vc, self.vs, self.pos)

    def values(self):
        k = orc.values(self.kc.cpu().numpy(), self.ks.cpu().numpy(), self.cfg.k_unit)
        return k, orc.values(self.vc.cpu().numpy(), self.vs.cpu().numpy(), self.cfg.v_unit)

    def attend(self, q, q_pos, kv_len, mass=None, ws=None, stream=None):
        T = q.shape[1]
        out = torch.full((self.B, T, self.Hq, self.D), float("nan"), dtype=self.dtype, device=self.dev)
        lse = torch.full((self.B, self.Hq, T), float("nan"), device=self.dev)
        if ws is None:
            ws = torch.full((P.pbsa_kv4_workspace_size(self.cfg, T),), 255, dtype=torch.uint8, device=self.dev)
        P.pbsa_kv4_attn(self.cfg, self.cache, q, q_pos, kv_len, out, lse, mass, ws, self.status, stream=stream)
        return out, lse

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def queries(self, T, size=1.0):
        return (size * torch.randn(self.B, T, self.Hq, self.D, generator=self.g)).to(self.dtype).to(self.dev)


def check_attention(c, q, q_pos, kv_len, out, lse, mass=None, mass0=None, k=None, v=None):
    k0, v0 = c.values()
    k, v = (k0 if k is None else k), (v0 if v is None else v)
    wo, wl, wm, vabs, qk = orc.kv4_attn(f64(q), k, v, c.pos.cpu().numpy(),
                                        None if q_pos is None else q_pos.cpu().numpy(), kv_len)
    E = 2.0 ** -19 * qk
    lg = f64(lse)
    none = np.isneginf(wl)
    assert np.isneginf(lg[none]).all() and (f64(out).transpose(0, 2, 1, 3)[none] == 0).all()
    some = ~none
    al = np.abs(np.where(none, 0, wl))
    assert (np.abs(lg[some] - wl[some]) <= (E + 2.0 ** -20 * (1 + al))[some]).all()
    e = torch.finfo(c.dtype).eps / 2
    tol = e * np.abs(wo) + (2 * E + 2.0 ** -11 + 2.0 ** -18).transpose(0, 2, 1)[..., None] * vabs
    tol += c.N * 2.0 ** -32 * np.abs(v).max(initial=0, where=np.isfinite(v))
    tol += 2.0 ** -25 if c.dtype == torch.float16 else 0
    assert (np.abs(f64(out) - wo) <= tol).all(), np.abs(f64(out) - wo).max()
    if mass is not None:
        rel = 2 * E.max() + 2.0 ** -19 * (1 + al.max())
        want = f64(mass0) + wm
        assert (np.abs(f64(mass) - want) <= rel * wm + 2.0 ** -23 * want).all()


# --------------------------------------------------------------------------- quantiser
def border_rows(D):
    """Rows whose channels sit on and beside every border between codes, for several scales."""
    rows = []
    for s in (1.0, 0.34375, 448.0, 2.0 ** -9, 0.0625):
        base = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
        rows.append([t * s for t in base] + [-t * s for t in base])
        rows.append([t * s * (1 + 2.0 ** -7) for t in base[:-1]] + [6 * s] + [-t * s * (1 - 2.0 ** -7) for t in base])
    rows.append([0.0] * 16)
    rows.append([6 * 2.0 ** -10] * 16)             # amax / 6 on the border between scale 0 and 1
    rows.append([6 * 2.0 ** -10 * 1.01] * 16)
    rows.append([3e4] * 16)                        # beyond the largest value: saturates
    rows.append([-0.0, 1e-7] * 8)
    for m in range(8):                             # amax / 6 on the borders of e4m3
        rows.append([6 * (8.5 + m) / 8] * 8 + [1.0] * 8)
    flat = [t for r in rows for t in r]
    flat += [0.0] * (-len(flat) % D)
    return torch.tensor(flat).view(-1, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ku,vu", [(1.0, 1.0), (0.25, 2.0 ** -6)])
def test_append_is_exact(cuda_dev, D, dtype, ku, vu):
    rows = border_rows(D)
    extra = torch.randn(9, D, generator=torch.Generator().manual_seed(1)) * 3
    x = torch.cat((rows, extra)).to(dtype)
    T = len(x)
    c = Cache(cuda_dev, B=1, Hq=2, Hkv=2, D=D, N=128, dtype=dtype, ku=ku, vu=vu)
    k = torch.stack((x, x.flip(0)), 1)[None].to(cuda_dev)
    v = k.flip(2).contiguous()
    perm = torch.stack([torch.randperm(128, generator=c.g)[:T] for _ in range(2)])[None].int().to(cuda_dev)
    pos = (1000 + torch.arange(T, dtype=torch.int32, device=cuda_dev))[None]
    before = [t.clone() for t in (c.kc, c.ks, c.vc, c.vs, c.pos, c.mass)]
    P.pbsa_kv4_append(c.cfg, c.cache, k, v, pos, perm, c.mass, c.status)
    assert int(c.status.item()) == 0
    for h in range(2):
        for t in range(T):
            r = int(perm[0, h, t])
            for src, codes, scales, unit in ((k, c.kc, c.ks, ku), (v, c.vc, c.vs, vu)):
                wc, ws = orc.quantise_row(f64(src[0, t, h]).tolist(), unit)
                assert scales[0, h, r].tolist() == ws
                got = codes[0, h, r].cpu()
                nib = torch.stack((got & 15, got >> 4), -1).flatten().tolist()
                assert [n if n != 8 else 0 for n in nib] == [n if n != 8 else 0 for n in wc], (t, h)
            assert int(c.pos[0, h, r]) == 1000 + t and float(c.mass[0, h, r]) == 0
        keep = torch.ones(128, dtype=torch.bool)
        keep[perm[0, h].cpu().long()] = False
        for t, b in zip((c.kc, c.ks, c.vc, c.vs, c.pos, c.mass), before):
            assert torch.equal(t[0, h].cpu()[keep], b[0, h].cpu()[keep])
    # and back: exactly the values, in the given order; -1 asks for none
    rows = perm.clone()
    rows[0, 0, 3] = -1
    ko, vo = (torch.full((1, 2, T, D), float("nan"), dtype=dtype, device=cuda_dev) for _ in range(2))
    P.pbsa_kv4_read(c.cfg, c.cache, rows, ko, vo, c.status)
    for got, want in zip((ko, vo), c.values()):
        for h in range(2):
            w = want[0, h, perm[0, h].cpu().numpy()]
            if h == 0:
                w[3] = 0
            assert np.array_equal(f64(got[0, h]), w.astype(np.float32).astype(np.float64))
    assert int(c.status.item()) == 0
    all_k = torch.empty(1, 2, 100, D, dtype=dtype, device=cuda_dev)
    all_v = torch.empty_like(all_k)
    P.pbsa_kv4_read(c.cfg, c.cache, None, all_k, all_v, c.status)
    assert np.array_equal(f64(all_k), c.values()[0][:, :, :100])
    rows[0, 1, 0] = 128
    P.pbsa_kv4_read(c.cfg, c.cache, rows, ko, vo, c.status)
    assert int(c.status.item()) == P.PBSA_ERR_DEVICE_CHECK and (ko[0, 1, 0] == 0).all()


def test_append_padding_views_bad_rows_and_non_finite(cuda_dev):
    c = Cache(cuda_dev, B=3, Hq=5, Hkv=5, D=64, N=64)
    qkv = torch.randn(3, 4, 15, 64, generator=c.g).to(torch.bfloat16).to(cuda_dev)
    k, v = qkv[:, :, 5:10], qkv[:, :, 10:]
    pos = c.i32([[0, 1, 2, 3], [7, -1, -1, -1], [-1, -5, -1, 60]])
    before = c.kc.clone()
    # no rows: a token goes to the row of its position
    P.pbsa_kv4_append(c.cfg, c.cache, k, v, pos, None, None, c.status)
    assert int(c.status.item()) == 0
    written = torch.zeros(3, 64, dtype=torch.bool)
    for b, t, r in ((0, 0, 0), (0, 1, 1), (0, 2, 2), (0, 3, 3), (1, 0, 7), (2, 3, 60)):
        written[b, r] = True
        for h in range(5):
            wc, ws = orc.quantise_row(f64(k[b, t, h]).tolist(), 1.0)
            assert c.ks[b, h, r].tolist() == ws and int(c.pos[b, h, r]) == r
    keep = ~written[:, None].expand(3, 5, 64).to(cuda_dev)
    assert torch.equal(c.kc[keep], before[keep])
    # a row out of the cache is skipped and reported, the others are written
    rows = torch.arange(4, dtype=torch.int32, device=cuda_dev).expand(3, 5, 4).contiguous()
    rows[1, 2] = c.i32([64, -1, 2 ** 31 - 1, 5])
    pos = c.i32([[100, 101, 102, 103]] * 3)
    P.pbsa_kv4_append(c.cfg, c.cache, k, v, pos, rows, c.mass, c.status)
    assert int(c.status.item()) == P.PBSA_ERR_DEVICE_CHECK
    assert int(c.pos[1, 2, 5]) == 103 and int(c.pos[0, 0, 3]) == 103
    # infinities saturate, a NaN is stored as zero and reported
    c.status.zero_()
    bad = k.contiguous()
    bad[0, 0, 0, 1], bad[0, 0, 0, 2] = float("inf"), -float("inf")
    rows[1, 2] = c.i32([0, 1, 2, 3])
    P.pbsa_kv4_append(c.cfg, c.cache, bad, v, pos, rows, None, c.status)
    assert int(c.status.item()) == 0
    assert c.values()[0][0, 0, 0, 1:3].tolist() == [2688.0, -2688.0]
    bad[0, 0, 0, 3] = float("nan")
    P.pbsa_kv4_append(c.cfg, c.cache, bad, v, pos, rows, None, c.status)
    assert int(c.status.item()) == P.PBSA_ERR_DEVICE_CHECK
    assert np.isfinite(c.values()[0]).all() and c.values()[0][0, 0, 0, 3] == 0


def test_append_skips_the_last_position(cuda_dev):
    """2^31 - 1 stands for no token inside the kernels."""
    c = Cache(cuda_dev, B=1, Hq=1, Hkv=1, D=64, N=64)
    k = torch.randn(1, 2, 1, 64, generator=c.g).to(torch.bfloat16).to(cuda_dev)
    rows, pos, before = c.i32([[[3, 4]]]), c.i32([[2 ** 31 - 1, 2 ** 31 - 2]]), c.pos.clone()
    P.pbsa_kv4_append(c.cfg, c.cache, k, k, pos, rows, None, c.status)
    assert int(c.status.item()) == P.PBSA_ERR_DEVICE_CHECK
    assert int(c.pos[0, 0, 3]) == int(before[0, 0, 3]) and int(c.pos[0, 0, 4]) == 2 ** 31 - 2


# --------------------------------------------------------------------------- attention
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (4, 2, 1), (8, 1, 1), (12, 1, 1), (6, 2, 3), (5, 5, 7), (9, 1, 2),
                                      (32, 1, 1), (7, 1, 5), (3, 1, 11), (4, 1, 8), (2, 1, 40)])
def test_rows_of_every_count(cuda_dev, D, dtype, Hq, Hkv, T):
    """1 to 80 query rows to a key head: all variants, full groups of rows and ragged ones."""
    N = 192
    c = Cache(cuda_dev, B=2, Hq=Hq, Hkv=Hkv, D=D, N=N, dtype=dtype, seed=T + Hq)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.1] = -1
    q = c.queries(T)
    lens = [N, 77]
    mass = c.mass.clone()
    out, lse = c.attend(q, None, c.i32(lens), mass)
    check_attention(c, q, None, lens, out, lse, mass, c.mass)
    q_pos = torch.randint(0, 2 * N, (2, T), generator=c.g, dtype=torch.int32).to(cuda_dev)
    q_pos[1, -1] = -1                                    # a padded place
    mass = c.mass.clone()
    out, lse = c.attend(q, q_pos, c.i32(lens), mass)
    check_attention(c, q, q_pos, lens, out, lse, mass, c.mass)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 65), (2, 1, 64), (3, 1, 43), (8, 2, 65), (1, 1, 300), (4, 2, 257)])
@pytest.mark.parametrize("N,lens", [(64, [64, 33]), (448, [448, 129])])
def test_chunks(cuda_dev, D, dtype, Hq, Hkv, T, N, lens):
    """65 to 514 query rows to a key head: one side of 128 and two, ragged groups, several
    segments a CTA and several CTAs a segment."""
    c = Cache(cuda_dev, B=2, Hq=Hq, Hkv=Hkv, D=D, N=N, dtype=dtype, seed=T + Hq)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.05] = -1
    q = c.queries(T)
    mass = c.mass.clone()
    out, lse = c.attend(q, None, c.i32(lens), mass)
    check_attention(c, q, None, lens, out, lse, mass, c.mass)
    q_pos = torch.randint(0, 2 * N, (2, T), generator=c.g, dtype=torch.int32).to(cuda_dev)
    q_pos[1, -3:] = -1                                   # padded places
    q_pos[0, :40] = 2                                    # rows that see next to nothing
    mass = c.mass.clone()
    out, lse = c.attend(q, q_pos, c.i32(lens), mass)
    check_attention(c, q, q_pos, lens, out, lse, mass, c.mass)
    again = c.mass.clone()
    out2, lse2 = c.attend(q, q_pos, c.i32(lens), again)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(mass, again)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("Hkv,G,T", [(8, 1, 128), (4, 1, 300), (2, 3, 256), (12, 2, 390)])
def test_chunks_of_many_tiles(cuda_dev, D, dtype, Hkv, G, T):
    """Many 128-key tiles a CTA, in segments of one side and of two; against torch in fp64 on the
    GPU, and three runs bit for bit."""
    N = 4096
    c = Cache(cuda_dev, B=2, Hq=Hkv * G, Hkv=Hkv, D=D, N=N, dtype=dtype, seed=T + Hkv)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.02] = -1
    lens = [N, 3000]
    q = c.queries(T, 1.5)
    runs = []
    for _ in range(3):
        mass = c.mass.clone()
        runs.append((*c.attend(q, None, c.i32(lens), mass), mass))
    assert int(c.status.item()) == 0
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))
    out, lse, mass = runs[0]
    k, v = (torch.tensor(t, device=cuda_dev) for t in c.values())
    e = torch.finfo(dtype).eps / 2
    for b in range(2):
        for h in range(Hkv):
            j = torch.nonzero(c.pos[b, h, :lens[b]] >= 0).flatten()
            x = q[b, :, h * G:(h + 1) * G].double()                       # [T, G, D]
            s = x @ k[b, h, j].T / math.sqrt(D)
            E = 2.0 ** -19 * (x.abs() @ k[b, h, j].abs().T).amax(-1) / math.sqrt(D)
            wl = torch.logsumexp(s, -1)
            p = torch.exp(s - wl[..., None])
            al = lse[b, h * G:(h + 1) * G].T.double()
            assert ((al - wl).abs() <= E + 2.0 ** -20 * (1 + wl.abs())).all()
            wo, vabs = p @ v[b, h, j], p @ v[b, h, j].abs()
            got = out[b, :, h * G:(h + 1) * G].double()
            tol = e * wo.abs() + (2 * E + 2.0 ** -11 + 2.0 ** -18)[..., None] * vabs
            tol = tol + N * 2.0 ** -32 * v[b, h, j].abs().max() + 2.0 ** -25
            assert ((got - wo).abs() <= tol).all()
            wm = p.sum((0, 1))
            rel = 2 * E.max() + 2.0 ** -19 * (1 + wl.abs().max())
            want = c.mass[b, h, j].double() + wm
            assert ((mass[b, h, j].double() - want).abs() <= rel * wm + T * G * 2.0 ** -24 * wm + 2.0 ** -23 * want).all()


def test_chunk_of_a_long_cache(cuda_dev):
    """Parts of one head on many CTAs, an empty sequence and garbage in rows without a token."""
    c = Cache(cuda_dev, B=3, Hq=2, Hkv=1, D=128, N=4096, seed=21)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.02] = -1
    lens = [4096, 0, 1500]
    gone = (c.pos < 0) | (torch.arange(4096, device=cuda_dev) >= c.i32(lens)[:, None, None])
    q = c.queries(70, 2.0)
    mass = c.mass.clone()
    out, lse = c.attend(q, None, c.i32(lens), mass)
    k, v = c.values()
    check_attention(c, q, None, lens, out, lse, mass, c.mass, k=k, v=v)
    for t, x in ((c.kc, 255), (c.ks, 127), (c.vc, 255), (c.vs, 127)):
        t[gone] = x
    again = c.mass.clone()
    out2, lse2 = c.attend(q, None, c.i32(lens), again)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(mass, again)


@pytest.mark.parametrize("N,lens", [(64, [0, 1, 2, 15]), (64, [16, 17, 63, 64]), (1088, [1088, 1073, 257, 0]),
                                    (4096, [4096, 1, 2049, 0])])
@pytest.mark.parametrize("G", [1, 10])
def test_lengths(cuda_dev, N, lens, G):
    """Empty caches, one row, lengths around a step of sixteen; one split and several."""
    c = Cache(cuda_dev, B=4, Hq=G, Hkv=1, D=128, N=N, seed=N)
    q = c.queries(1)
    mass = c.mass.clone()
    out, lse = c.attend(q, None, c.i32(lens), mass)
    check_attention(c, q, None, lens, out, lse, mass, c.mass)
    for b, n in enumerate(lens):
        assert torch.equal(mass[b, :, n:], c.mass[b, :, n:])


def test_long_splits_join(cuda_dev):
    """A long cache of one head, its largest logits far apart from split to split."""
    c = Cache(cuda_dev, B=1, Hq=2, Hkv=1, D=64, N=32768, seed=5)
    c.ks[0, 0, ::4099] = 90                               # a few keys 2^5 times larger
    q = c.queries(1, 2.0)
    mass = c.mass.clone()
    out, lse = c.attend(q, None, c.i32([32768]), mass)
    check_attention(c, q, None, [32768], out, lse, mass, c.mass)
    again, lse2 = c.attend(q, None, c.i32([32768]))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D,T,Hq", [(64, 3, 4), (128, 5, 4), (64, 4, 8)])
def test_masses_of_many_cached_rows(cuda_dev, D, T, Hq):
    """Enough rows that a warp of the mass kernel takes several units; lengths end inside them."""
    c = Cache(cuda_dev, B=3, Hq=Hq, Hkv=1, D=D, N=51200, seed=23)
    lens, q = [51200, 20011, 1], c.queries(T)
    q_pos = torch.randint(30000, 90000, (3, T), generator=c.g, dtype=torch.int32).to(cuda_dev)
    mass = c.mass.clone()
    out, lse = c.attend(q, q_pos, c.i32(lens), mass)
    check_attention(c, q, q_pos, lens, out, lse, mass, c.mass)


def test_causal_steps_equal_single_tokens(cuda_dev):
    """T tokens under the causal mask give what they give one at a time."""
    N, T = 128, 6
    c = Cache(cuda_dev, B=1, Hq=4, Hkv=2, N=N, seed=6)
    c.pos.copy_(torch.arange(N, dtype=torch.int32, device=cuda_dev).expand(1, 2, N))
    q = c.queries(T)
    q_pos = c.i32([list(range(N - T, N))])
    out, lse = c.attend(q, q_pos, c.i32([N]))
    check_attention(c, q, q_pos, [N], out, lse)
    for t in range(T):
        o, l = c.attend(q[:, t:t + 1].contiguous(), None, c.i32([N - T + t + 1]))
        assert torch.allclose(l[..., 0], lse[..., t], rtol=0, atol=2e-6)
        assert (o[:, 0].float() - out[:, t].float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()


def test_garbage_in_rows_without_a_token_changes_nothing(cuda_dev):
    """Empty rows and rows past the length may hold anything, NaN scales and infinities of
    masked logits among it."""
    c = Cache(cuda_dev, B=2, Hq=4, Hkv=2, N=128, seed=7)
    empty = torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.3
    c.pos[empty] = -1
    lens = [100, 37]
    gone = empty | (torch.arange(128, device=cuda_dev) >= c.i32(lens)[:, None, None])
    q = c.queries(3)
    k, v = c.values()
    mass = c.mass.clone()
    want = c.attend(q, None, c.i32(lens), mass)
    for code, scale in ((255, 127), (119, 126), (0, 255)):
        for t, x in ((c.kc, code), (c.ks, scale), (c.vc, code), (c.vs, scale)):
            t[gone] = x
        again = c.mass.clone()
        got = c.attend(q, None, c.i32(lens), again)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(again, mass)
    check_attention(c, q, None, lens, *want, k=k, v=v)


def test_large_small_and_uneven_queries(cuda_dev):
    """Queries far from 1 in both directions keep their logits (bf16 reaches beyond fp16), zero
    queries give the plain mean."""
    c = Cache(cuda_dev, B=1, Hq=4, Hkv=1, D=64, N=64, ku=2.0 ** -6, seed=8)
    q = c.queries(5)
    q[0, 0] *= 2.0 ** 18
    q[0, 1] *= 2.0 ** -30
    q[0, 2] = 0
    q[0, 3, :, 0] *= 2.0 ** 9
    out, lse = c.attend(q, None, c.i32([64]))
    check_attention(c, q, None, [64], out, lse)
    mean = c.values()[1][0, 0].mean(0)
    assert np.abs(f64(out[0, 2, 0]) - mean).max() <= 2.0 ** -8 * np.abs(mean).max() + 2.0 ** -11


def test_units(cuda_dev):
    c = Cache(cuda_dev, B=1, Hq=2, Hkv=2, D=128, N=64, ku=0.25, vu=2.0 ** -7, seed=9)
    q = c.queries(2)
    out, lse = c.attend(q, None, c.i32([64]))
    check_attention(c, q, None, [64], out, lse)


def test_length_out_of_the_cache_is_clamped_and_reported(cuda_dev):
    c = Cache(cuda_dev, B=2, Hq=2, Hkv=2, D=64, N=64, seed=10)
    q = c.queries(1)
    out, lse = c.attend(q, None, c.i32([65, -3]))
    assert int(c.status.item()) == P.PBSA_ERR_DEVICE_CHECK
    check_attention(c, q, None, [64, 0], out, lse)


def test_strided_queries_streams_and_workspaces(cuda_dev):
    """Views of a projection's output; two calls at once on two streams, each its workspace."""
    c = Cache(cuda_dev, B=2, Hq=6, Hkv=2, D=128, N=2048, seed=11)
    qkv = torch.randn(2, 3, 10, 128, generator=c.g).to(torch.bfloat16).to(cuda_dev)
    q, lens = qkv[:, :, :6], c.i32([2048, 900])
    want = c.attend(q.contiguous(), None, lens)
    torch.cuda.synchronize()
    got = c.attend(q, None, lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    q2 = c.queries(3)
    want2 = c.attend(q2, None, lens)
    torch.cuda.synchronize()
    res = []
    for s, x in zip(streams, (q, q2)):
        with torch.cuda.stream(s):
            for _ in range(5):
                r = c.attend(x, None, lens)
            res.append(r)
    torch.cuda.synchronize()
    assert torch.equal(res[0][0], want[0]) and torch.equal(res[1][0], want2[0])


def test_attention_captured_and_replayed(cuda_dev):
    """A graph sees the lengths, positions and rows of the moment it is replayed."""
    c = Cache(cuda_dev, B=2, Hq=8, Hkv=2, D=128, N=1024, seed=12)
    q, lens = c.queries(1), c.i32([10, 20])
    ws = torch.empty(P.pbsa_kv4_workspace_size(c.cfg, 1), dtype=torch.uint8, device=cuda_dev)
    mass = c.mass.clone()
    c.attend(q, None, lens, mass, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = c.attend(q, None, lens, mass, ws)
    for n in ([1024, 3], [500, 1000]):
        lens.copy_(c.i32(n))
        q.copy_(c.queries(1))
        mass.copy_(c.mass)
        g.replay()
        check_attention(c, q, None, n, out, lse, mass, c.mass)


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_captured_and_replayed(cuda_dev, D):
    """Many rows: new lengths (one of them 0), positions, queries and rows without a token."""
    c = Cache(cuda_dev, B=2, Hq=4, Hkv=2, D=D, N=320, seed=21)
    q, lens, q_pos = c.queries(150), c.i32([10, 20]), torch.zeros(2, 150, dtype=torch.int32, device=cuda_dev)
    ws = torch.empty(P.pbsa_kv4_workspace_size(c.cfg, 150), dtype=torch.uint8, device=cuda_dev)
    mass = c.mass.clone()
    c.attend(q, q_pos, lens, mass, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = c.attend(q, q_pos, lens, mass, ws)
    for n in ([320, 0], [77, 300]):
        lens.copy_(c.i32(n))
        q.copy_(c.queries(150))
        q_pos.copy_(torch.randint(-1, 640, (2, 150), generator=c.g, dtype=torch.int32))
        c.pos[:, :, 5:60:7] = -1
        mass.copy_(c.mass)
        g.replay()
        check_attention(c, q, q_pos, n, out, lse, mass, c.mass)


@pytest.mark.parametrize("D", [64, 128])
def test_calls_of_all_kinds_at_once(cuda_dev, D):
    """Streams that run one row, a few and many, with masses, beside each other: every call is
    the same as alone, bit for bit."""
    c = Cache(cuda_dev, B=3, Hq=6, Hkv=3, D=D, N=1984, seed=22)
    lens = c.i32([1984, 700, 0])
    qs = [c.queries(T) for T in (1, 9, 130, 300)]
    wss = [torch.empty(P.pbsa_kv4_workspace_size(c.cfg, q.shape[1]), dtype=torch.uint8, device=cuda_dev) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]

    def run(q, ws):
        mass = c.mass.clone()
        return (*c.attend(q, None, lens, mass, ws), mass)

    want = []
    for q, ws in zip(qs, wss):
        want.append(run(q, ws))
        torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for q, ws, st in zip(qs, wss, streams):
            with torch.cuda.stream(st):
                got.append(run(q, ws))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(r, want[i % len(qs)]))


def test_offsets_past_32_bits(cuda_dev):
    """A cache of more than 2^31 bytes of codes and 2^31 values: its last rows are reached."""
    B, Hkv, N, D = 33, 8, 131072, 128
    u8 = dict(dtype=torch.uint8, device=cuda_dev)
    kc = torch.zeros(B, Hkv, N, D // 2, **u8)
    ks = torch.zeros(B, Hkv, N, D // 16, **u8)
    pos = torch.full((B, Hkv, N), -1, dtype=torch.int32, device=cuda_dev)
    assert kc.numel() > 2 ** 31
    c = Cache(cuda_dev, B=1, Hq=Hkv, Hkv=Hkv, D=D, N=64, seed=13)       # for its helpers
    c.B, c.N, c.pos = B, N, pos
    c.cfg = P.make_kv4_config(B, Hkv, Hkv, D, N)
    c.cache = P.make_kv4_cache(c.cfg, kc, ks, kc, ks, pos)              # keys and values alike
    k = torch.randn(B, 2, Hkv, D, generator=c.g).to(torch.bfloat16).to(cuda_dev)
    new = torch.full((B, 2), -1, dtype=torch.int32, device=cuda_dev)
    new[-1] = c.i32([N - 2, N - 1])
    P.pbsa_kv4_append(c.cfg, c.cache, k, k, new, None, None, c.status)
    lens = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    lens[-1] = N
    q = torch.randn(B, 1, Hkv, D, generator=c.g).to(torch.bfloat16).to(cuda_dev)
    mass = torch.zeros(B, Hkv, N, device=cuda_dev)
    out, lse = c.attend(q, None, lens, mass)
    assert int(c.status.item()) == 0
    assert (out[:-1] == 0).all() and torch.isneginf(lse[:-1]).all()
    vals = orc.values(kc[-1:, :, -2:].cpu().numpy(), ks[-1:, :, -2:].cpu().numpy(), 1.0)
    wo, wl, wm, vabs, qk = orc.kv4_attn(f64(q[-1:]), vals, vals, pos[-1:, :, -2:].cpu().numpy(), None, [2])
    assert np.abs(f64(lse[-1:]) - wl).max() <= 2.0 ** -19 * qk.max() + 2.0 ** -17
    assert (np.abs(f64(out[-1:]) - wo) <= 2.0 ** -8 * np.abs(wo) + 2.0 ** -10 * vabs).all()
    assert np.abs(f64(mass[-1:, :, -2:]) - wm).max() <= 2.0 ** -14
    rows = c.i32([[[N - 1]] * Hkv] * B)
    ko = torch.empty(B, Hkv, 1, D, dtype=torch.bfloat16, device=cuda_dev)
    vo = torch.empty_like(ko)
    P.pbsa_kv4_read(c.cfg, c.cache, rows, ko, vo, c.status)
    assert np.array_equal(f64(ko[-1:]), vals[:, :, 1:]) and (ko[:-1] == 0).all()
    got = torch.empty(B, Hkv, 1, dtype=torch.int32, device=cuda_dev)
    mass[:] = 1
    pos[:] = 5
    mass[-1, :, -1] = 0.5
    P.pbsa_kv4_evict(c.cfg, pos, mass, 0, None, got, c.status)
    assert (got[-1] == N - 1).all() and (got[:-1] == 0).all()


# ---------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("B,Hkv,N", [(1, 1, 64), (2, 3, 192), (1, 2, 1088), (2, 1, 4160), (1, 1, 40000 // 64 * 64),
                                     (1, 1, 131072), (5, 8, 9280), (5, 8, 20032), (1, 1, 200064)])
@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "odd"])
def test_evicted_rows(cuda_dev, B, Hkv, N, kind):
    g = torch.Generator().manual_seed(N)
    pos = torch.stack([torch.randperm(2 * N, generator=g)[:N] for _ in range(B * Hkv)]).view(B, Hkv, N).int()
    mass = torch.exp(3 * torch.randn(B, Hkv, N, generator=g) - 6)
    if kind == "ties":
        mass = (mass * 8).floor() / 8
    elif kind == "zeros":
        mass.zero_()
    elif kind == "odd":
        pick = lambda p: torch.rand(mass.shape, generator=g) < p
        mass[pick(0.1)], mass[pick(0.1)], mass[pick(0.1)] = float("nan"), float("inf"), -1.0
        mass[pick(0.1)], mass[pick(0.1)] = -0.0, 1e-42
        pos[pick(0.05)] = -1
    c = P.make_kv4_config(B, Hkv, Hkv, 64, N)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    keep = torch.tensor([2 * N - N // 8 - b for b in range(B)], dtype=torch.int32)
    for n, n_sink, kf in ((1, 0, None), (1, N // 8, keep), (17, 4, keep), (N // 3, N // 8, keep), (N, 0, None),
                          (N, N // 8, keep)):
        rows = torch.full((B, Hkv, n), -9, dtype=torch.int32, device=cuda_dev)
        st.zero_()
        P.pbsa_kv4_evict(c, pos.to(cuda_dev), mass.to(cuda_dev), n_sink, None if kf is None else kf.to(cuda_dev),
                         rows, st)
        want, short = orc.kv4_evict(pos.numpy(), mass.double().numpy(), n, n_sink, None if kf is None else kf.numpy())
        assert np.array_equal(rows.cpu().numpy(), want), (kind, n, n_sink)
        assert int(st.item()) == (P.PBSA_ERR_DEVICE_CHECK if short else 0)


def test_eviction_captured_and_replayed(cuda_dev):
    c = Cache(cuda_dev, B=2, Hkv=2, N=256, seed=14)
    rows = torch.empty(2, 2, 5, dtype=torch.int32, device=cuda_dev)
    keep = c.i32([400, 500])
    P.pbsa_kv4_evict(c.cfg, c.pos, c.mass, 3, keep, rows, c.status)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.pbsa_kv4_evict(c.cfg, c.pos, c.mass, 3, keep, rows, c.status)
    for _ in range(3):
        c.mass.copy_(torch.rand(c.mass.shape, generator=c.g))
        g.replay()
        want, _ = orc.kv4_evict(c.pos.cpu().numpy(), f64(c.mass), 5, 3, keep.cpu().numpy())
        assert np.array_equal(rows.cpu().numpy(), want)


# ---------------------------------------------------------------- all of them, as used
@pytest.mark.parametrize("graph", [False, True])
def test_generation_with_a_bounded_cache(cuda_dev, graph):
    """Norm and rotation -> rows -> append -> attention, token by token past the capacity, then
    padded steps of three: every step against the oracle on the GPU's own state before it."""
    B, Hq, Hkv, D, N = 2, 4, 2, 64, 64
    tc = TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=8, device=cuda_dev)
    gen = torch.Generator().manual_seed(15)
    cos, sin = rope_table((D // 2,), 512, device=cuda_dev)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    graphs, buffers = {}, {}

    def heads(q, k, pos):
        T = q.shape[1]
        c = P.make_qk_config(B, T, Hq, Hkv, D, table_len=512)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        P.pbsa_qk_norm_rope(c, q, k, None, None, cos, sin, pos, qo, ko, st)
        return qo, ko

    def one(T, n_new):
        q, k, v = (torch.randn(B, T, h, D, generator=gen).to(torch.bfloat16).to(cuda_dev) for h in (Hq, Hkv, Hkv))
        pos = (tc.seen[:, None] + torch.arange(T, dtype=torch.int32, device=cuda_dev))[..., None].contiguous()
        qn, kn = heads(q, k, pos)
        before = dict(pos=tc.pos.cpu().numpy(), mass=f64(tc.mass), seen=tc.seen.cpu().numpy(), len=tc.kv_len.cpu().numpy())
        if T not in buffers:
            buffers[T] = [torch.empty_like(t) for t in (qn, kn, v)] + [torch.empty(B, dtype=torch.int32, device=cuda_dev)]
        b = buffers[T]
        for x, y in zip(b, (qn, kn, v)):
            x.copy_(y)
        b[3].copy_(torch.tensor(n_new, dtype=torch.int32))
        if graph and T in graphs:
            graphs[T].replay()
            out = tc._steps[T]["out"]
        else:
            out = tc.step(b[0], b[1], b[2], b[3])
            if graph:
                graphs[T] = torch.cuda.CUDAGraph()
                keep = [t.clone() for t in (tc.k_codes, tc.k_scales, tc.v_codes, tc.v_scales, tc.pos, tc.mass, tc.seen, tc.kv_len)]
                with torch.cuda.graph(graphs[T]):
                    tc.step(b[0], b[1], b[2], b[3])
                for x, y in zip((tc.k_codes, tc.k_scales, tc.v_codes, tc.v_scales, tc.pos, tc.mass, tc.seen, tc.kv_len), keep):
                    assert torch.equal(x, y)           # capturing ran nothing
        assert int(tc.status.item()) == 0 and int(st.item()) == 0
        rows, short = orc.kv4_evict(before["pos"], before["mass"], T, tc.n_sink, before["seen"] - tc.n_recent)
        assert not short
        pos0, mass0 = before["pos"].copy(), before["mass"].copy()
        q_pos = np.full((B, T), -1)
        for i in range(B):
            for t in range(n_new[i]):
                q_pos[i, t] = before["seen"][i] + t
                for h in range(Hkv):
                    r = rows[i, h, t]
                    pos0[i, h, r], mass0[i, h, r] = q_pos[i, t], 0
                    wc, ws = orc.quantise_row(f64(kn[i, t, h]).tolist(), 1.0)
                    assert tc.k_scales[i, h, r].tolist() == ws
        assert np.array_equal(tc.pos.cpu().numpy(), pos0)
        lens = np.minimum(before["len"] + np.array(n_new), N)
        assert tc.kv_len.tolist() == lens.tolist()
        k_val = orc.values(tc.k_codes.cpu().numpy(), tc.k_scales.cpu().numpy(), 1.0)
        v_val = orc.values(tc.v_codes.cpu().numpy(), tc.v_scales.cpu().numpy(), 1.0)
        wo, wl, wm, vabs, qk = orc.kv4_attn(f64(qn), k_val, v_val, pos0, q_pos, lens)
        E = 2.0 ** -19 * qk
        assert (np.abs(f64(out) - wo) <= 2.0 ** -8 * np.abs(wo) + (2 * E + 2.0 ** -10).transpose(0, 2, 1)[..., None] * vabs).all()
        assert np.abs(f64(tc.mass) - (mass0 + wm)).max() <= 1e-4

    for i in range(70):
        one(1, [1, 1 if i < 50 else 0])
    for n in ([3, 1], [0, 3], [2, 2], [3, 3]):
        one(3, n)
    assert tc.seen.tolist() == [78, 59]


def test_calls_refuse_tensors_that_do_not_fit(cuda_dev):
    c = Cache(cuda_dev, B=2, Hq=4, Hkv=2, D=64, N=128)
    bf = dict(dtype=torch.bfloat16, device=cuda_dev)
    rows, pos = torch.zeros(2, 2, 1, dtype=torch.int32, device=cuda_dev), c.i32([[1], [2]])
    kv, out = torch.zeros(2, 1, 2, 64, **bf), torch.zeros(2, 2, 1, 64, **bf)
    ws = torch.empty(P.pbsa_kv4_workspace_size(c.cfg, 1), dtype=torch.uint8, device=cuda_dev)
    calls = [
        (P.pbsa_kv4_append, [kv, kv.clone(), pos, rows, c.mass, c.status], (3, 4)),
        (P.pbsa_kv4_read, [rows, out, out.clone(), c.status], (0,)),
        (P.pbsa_kv4_attn, [c.queries(1), pos, c.i32([5, 6]), torch.zeros(2, 1, 4, 64, **bf),
                           torch.zeros(2, 4, 1, device=cuda_dev), c.mass, ws, c.status], (1, 5)),
        (lambda cfg, cache, *a: P.pbsa_kv4_evict(cfg, a[0], a[1], 0, *a[2:]), [c.pos, c.mass, c.i32([0, 0]), rows, c.status], (2,)),
    ]
    before = [x.clone() for x in (c.kc, c.ks, c.vc, c.vs, c.pos, c.mass, rows, out)]
    for call, args, may_be_none in calls:
        for i, x in enumerate(args):
            # (a longer or wider workspace, a batch of one more dimension of new tokens fit)
            bad = [x.cpu()] if x is ws else [x.cpu(), x.double(), x[None], x.expand(3, *x.shape[1:]) if x.shape[0] == 1 else x[:1]]
            for y in bad + ([] if i in may_be_none else [None]):
                with pytest.raises((P.PBSAError, AttributeError)):
                    call(c.cfg, c.cache, *args[:i], y, *args[i + 1:])
    assert int(c.status.item()) == 0
    assert all(torch.equal(x, y) for x, y in zip(before, (c.kc, c.ks, c.vc, c.vs, c.pos, c.mass, rows, out)))


def test_cache_class_refuses_what_cannot_work(cuda_dev):
    tc = TokenCache(1, 2, 2, 64, 64, n_sink=30, n_recent=30, device=cuda_dev)
    z = lambda T: torch.zeros(1, T, 2, 64, dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(ValueError):
        tc.step(z(5), z(5), z(5))
    with pytest.raises(ValueError):
        TokenCache(1, 2, 2, 64, 64, n_sink=-1, device=cuda_dev)
    with pytest.raises(P.PBSAError):
        tc.step(z(1), z(1).cpu(), z(1))
    tc.step(z(4), z(4), z(4))
    assert int(tc.status.item()) == 0

"""Edges of the 4-bit token cache's attention: queries that hold no number, against the same call on
harmless inputs, and logits far beyond and far below one, against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from oracle import token_oracle as orc
from test_gpu_kv4 import Cache, check_attention, f64

pytestmark = pytest.mark.gpu

# query rows a key head: kept logits, the groups of up to 32 rows, one side of 128 and two
ROWS = [(1, 1), (2, 3), (4, 5), (5, 6), (1, 70), (3, 60)]      # (G, T)
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("junk", [NAN, INF, -INF])
def test_queries_that_see_nothing_may_hold_anything(cuda_dev, D, G, T, junk):
    """Padded places hold NaN or infinities: their output is zero, their lse -infinity, and
    everything else, masses among it, is bit for bit what it is with zeros there."""
    N, Hkv = 448, 2
    c = Cache(cuda_dev, B=4, Hq=G * Hkv, Hkv=Hkv, D=D, N=N, seed=G + T)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.1] = -1
    c.pos[1] = -1                                          # a sequence of empty rows
    c.pos[3, :, 128:256] = -1                              # whole tiles without a token
    lens = [N, N, 0, 300]
    q = c.queries(T)
    q_pos = torch.randint(N // 2, 2 * N, (4, T), generator=c.g, dtype=torch.int32).to(cuda_dev)
    q_pos[:, T // 2:] = -1
    none = q_pos < 0
    none[1:3] = True                                       # no row to see
    for pos in (q_pos, None):
        hide = none if pos is not None else torch.stack([torch.full_like(none[0], b in (1, 2)) for b in range(4)])
        q[hide] = 0
        mass = c.mass.clone()
        want = c.attend(q, pos, c.i32(lens), mass)
        q[hide] = junk
        again = c.mass.clone()
        got = c.attend(q, pos, c.i32(lens), again)
        assert (got[0][hide] == 0).all() and torch.isneginf(got[1].transpose(1, 2)[hide]).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(again, mass)
        q[hide] = 0
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", ROWS)
def test_a_query_without_a_number_leaves_the_masses_of_rows_it_does_not_see(cuda_dev, D, G, T):
    N = 256
    c = Cache(cuda_dev, B=1, Hq=G, Hkv=1, D=D, N=N, seed=3)
    q = c.queries(T)
    q[:, -1] = NAN
    q_pos = torch.full((1, T), 2 * N, dtype=torch.int32, device=cuda_dev)
    q_pos[:, -1] = N // 2
    mass = c.mass.clone()
    out, _ = c.attend(q, q_pos, c.i32([N]), mass)
    unseen = c.pos > N // 2
    assert torch.isfinite(mass[unseen]).all() and unseen.any()
    assert out[:, -1].isnan().all() and torch.isfinite(out[:, :-1]).all()


def one_channel_cache(dev, D, N, steps, base_scale, base_code):
    """Keys that hold base in channel 0 and, in channel 16, one of the codes `steps` (scale 1):
    with q = (a, 0.., b at 16, 0..) a logit is a base + b step, and fp32 holds it exactly."""
    c = Cache(dev, B=1, Hq=1, Hkv=1, D=D, N=N, dtype=torch.float16, seed=1)
    c.kc.zero_()
    c.ks.zero_()
    c.kc[..., 0] = base_code
    c.ks[..., 0] = base_scale
    c.kc[0, 0, :, 8] = torch.tensor(steps, dtype=torch.uint8, device=dev)
    c.ks[..., 1] = 56                                      # e4m3 of 1
    return c


def fine_steps(order, N):
    steps = np.arange(N) * 8 // N                          # codes 0 .. 7: 0, .5, 1, 1.5, 2, 3, 4, 6
    if order == "down":
        steps = steps[::-1].copy()
    elif order == "mixed":
        steps = np.random.default_rng(0).permutation(steps)
    return steps.astype(np.uint8)


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("T", [1, 20, 100])
def test_large_logits_keep_their_differences(cuda_dev, order, T):
    """Logits near 2^23.4 that differ by 1 to 12, all held exactly by fp32: 32768 x 2688 lies between
    2^26 and 2^27, where its steps are 8, and 16 x step is a multiple of 8.  So no logit's error
    enters (E = 0): the probabilities are good to the rounding of fp16 and the exponentials, the
    lse to 2^-22 of itself."""
    D, N = 64, 512
    c = one_channel_cache(cuda_dev, D, N, fine_steps(order, N), 126, 7)
    q = torch.zeros(1, T, 1, D, dtype=torch.float16, device=cuda_dev)
    q[..., 0], q[..., 16] = 32768.0, 16.0
    mass = torch.zeros_like(c.mass)
    out, lse = c.attend(q, None, c.i32([N]), mass)
    k, v = c.values()
    wo, wl, wm, vabs, _ = orc.kv4_attn(f64(q), k, v, c.pos.cpu().numpy(), None, [N])
    assert (np.abs(f64(lse) - wl) <= 2.0 ** -22 * wl).all()
    tol = 2.0 ** -11 * np.abs(wo) + (2.0 ** -11 + 2.0 ** -18) * vabs + N * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25
    assert (np.abs(f64(out) - wo) <= tol).all(), np.abs(f64(out) - wo).max()
    assert (np.abs(f64(mass) - wm) <= 2.0 ** -17 * wm).all(), np.abs(f64(mass) / wm - 1).max()


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("T", [1, 20, 100])
def test_large_logits_between_the_steps_of_fp32(cuda_dev, order, T):
    """The same with 8 x step, which falls between fp32's steps of 8: a product may be off by a step
    (8, so a logit by 1), and its probability by a factor e^2.  The output is still a mean of the
    values, the masses still add to the queries, and the lse is off by no more than 1."""
    D, N = 64, 512
    c = one_channel_cache(cuda_dev, D, N, fine_steps(order, N), 126, 7)
    q = torch.zeros(1, T, 1, D, dtype=torch.float16, device=cuda_dev)
    q[..., 0], q[..., 16] = 32768.0, 8.0
    mass = torch.zeros_like(c.mass)
    out, lse = c.attend(q, None, c.i32([N]), mass)
    k, v = c.values()
    _, wl, wm, _, _ = orc.kv4_attn(f64(q), k, v, c.pos.cpu().numpy(), None, [N])
    assert (np.abs(f64(lse) - wl) <= 1 + 2.0 ** -22 * wl).all()
    o, lo, hi = f64(out)[0, :, 0], v[0, 0].min(0), v[0, 0].max(0)
    slack = 2.0 ** -9 * np.abs(v).max()
    assert (o >= lo - slack).all() and (o <= hi + slack).all()
    m = f64(mass)
    assert (m <= math.e ** 2 * 1.001 * wm).all() and (m >= wm / (math.e ** 2 * 1.001)).all()
    assert abs(m.sum() - T) <= 2.0 ** -17 * T


@pytest.mark.parametrize("D,dtype,size", [(128, torch.float16, 65504.0), (64, torch.float16, 30000.0),
                                          (128, torch.bfloat16, 2.0 ** 100), (64, torch.bfloat16, 2.0 ** 20)])
@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("N", [64, 4096])
def test_far_logits_pick_the_largest(cuda_dev, D, dtype, size, G, T, N):
    """Queries up to their type's largest against keys of the largest scales: the softmax is a
    choice of one row, or the mean of rows with the same key.  Rows whose two largest logits are
    nearer than twice the error of a logit (2^-19 A_r each) plus 40 are left out."""
    c = Cache(cuda_dev, B=1, Hq=G, Hkv=1, D=D, N=N, dtype=dtype, seed=T)
    c.ks.fill_(126)
    c.kc[:, :, N // 2:] = c.kc[:, :, :N // 2]              # every key twice
    q = c.queries(T).sign() * size
    mass = torch.zeros_like(c.mass)
    out, lse = c.attend(q, None, c.i32([N]), mass)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all() and int(c.status.item()) == 0
    k, v = c.values()
    x = f64(q)[0].reshape(T * G, D)                        # row t G + g
    s = x @ k[0, 0, :N // 2].T / math.sqrt(D)
    err = 2.0 ** -19 * (np.abs(x) @ np.abs(k[0, 0, :N // 2]).T).max(-1) / math.sqrt(D)
    top = s.argmax(-1)
    two = np.sort(s, -1)
    clear = two[:, -1] - two[:, -2] > 2 * err + 40
    assert clear.any()
    wo = (v[0, 0, top] + v[0, 0, top + N // 2]) / 2
    got = f64(out)[0].reshape(T * G, D)
    e = torch.finfo(dtype).eps / 2
    va = (np.abs(v[0, 0, top]) + np.abs(v[0, 0, top + N // 2])) / 2
    assert (np.abs(got - wo) <= e * np.abs(wo) + 2.0 ** -18 * va + 2.0 ** -25)[clear].all()
    assert (np.abs(f64(lse)[0].T.reshape(-1) - s.max(-1)) <= err + 2.0 ** -20 * np.abs(s.max(-1)))[clear].all()
    if clear.all():
        want = np.zeros(N)
        for j in top:
            want[j] += 0.5
            want[j + N // 2] += 0.5
        assert np.abs(f64(mass)[0, 0] - want).max() <= 2.0 ** -18 * T * G
    assert abs(float(mass.double().sum()) - T * G) <= 2.0 ** -18 * T * G


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("ku,size", [(2.0 ** -40, 2.0 ** -100), (2.0 ** -40, 2.0 ** -126), (2.0 ** -28, 2.0 ** -120),
                                     (2.0 ** -40, 2.0 ** -60), (2.0 ** 40, 2.0 ** -126)])
def test_tiny_queries_and_units_give_the_mean(cuda_dev, D, G, T, ku, size):
    """Logits that are nearly zero: hidden and padded rows stay hidden, the others weigh alike."""
    c = Cache(cuda_dev, B=2, Hq=G, Hkv=1, D=D, N=192, ku=ku, seed=5)
    c.pos[torch.rand(c.pos.shape, generator=c.g).to(cuda_dev) < 0.2] = -1
    q = (c.queries(T).float().clamp(-2, 2) * size).to(torch.bfloat16)
    q_pos = torch.randint(0, 384, (2, T), generator=c.g, dtype=torch.int32).to(cuda_dev)
    lens = [192, 70]
    for pos in (None, q_pos):
        mass = c.mass.clone()
        out, lse = c.attend(q, pos, c.i32(lens), mass)
        check_attention(c, q, pos, lens, out, lse, mass, c.mass)


@pytest.mark.parametrize("G,T", ROWS)
def test_logits_past_fp32_still_pick_the_largest(cuda_dev, G, T):
    """A unit of 2^40 and queries of 2^120: the logits are beyond fp32, the choice is not."""
    c = Cache(cuda_dev, B=1, Hq=G, Hkv=1, D=64, N=64, ku=2.0 ** 40, seed=6)
    q = c.queries(T) * 2.0 ** 120
    out, lse = c.attend(q, None, c.i32([64]))
    k, v = c.values()
    x = f64(q)[0].reshape(T * G, 64)
    s = x @ k[0, 0].T
    two, err = np.sort(s, -1), 2.0 ** -19 * (np.abs(x) @ np.abs(k[0, 0]).T).max(-1)
    clear = two[:, -1] - two[:, -2] > 4 * err
    wo = v[0, 0, s.argmax(-1)]
    got = f64(out)[0].reshape(T * G, 64)
    assert clear.any() and (np.abs(got - wo) <= 2.0 ** -8 * np.abs(wo))[clear].all()
    assert (lse == INF).all()

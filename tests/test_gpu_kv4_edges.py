"""Edges of the 4-bit token cache's attention: queries that hold no number, against the same call on
harmless inputs, and logits far below one, against the fp64 oracle."""
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

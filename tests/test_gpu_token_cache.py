"""TokenCache at its edges: refused and padded steps, many lengths, streams and graphs."""
import pytest
import torch

from block_sparse_attention_35_b200 import pbsa as P
from block_sparse_attention_35_b200.token_cache import TokenCache

pytestmark = pytest.mark.gpu


def tokens(dev, g, B, T, Hq, Hkv, D, dtype=torch.bfloat16):
    return tuple(torch.randn(B, T, h, D, generator=g).to(dtype).to(dev) for h in (Hq, Hkv, Hkv))


def state(tc):
    return [t.clone() for t in (tc.k_codes, tc.k_scales, tc.v_codes, tc.v_scales, tc.pos, tc.mass, tc.seen,
                                tc.kv_len, tc.status)]


def test_a_refused_step_changes_nothing(cuda_dev):
    """Every argument that does not fit, on a full cache whose rows are being given up."""
    B, Hq, Hkv, D, N = 2, 4, 2, 64, 64
    tc = TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=4, device=cuda_dev)
    g = torch.Generator().manual_seed(0)
    tc.step(*tokens(cuda_dev, g, B, 50, Hq, Hkv, D))
    tc.step(*tokens(cuda_dev, g, B, 40, Hq, Hkv, D))
    good = tokens(cuda_dev, g, B, 3, Hq, Hkv, D)
    want = state(tc)
    n_new = torch.tensor([3, 1], dtype=torch.int32, device=cuda_dev)
    odd = lambda t: torch.zeros(t.numel() + 8, dtype=t.dtype, device=cuda_dev)[1:1 + t.numel()].view(t.shape)
    wide = lambda t: torch.zeros(*t.shape[:3], D + 4, dtype=t.dtype, device=cuda_dev)[..., :D]
    for i in range(3):
        x = good[i]
        for bad in (x.cpu(), x.half(), x.float(), x[:, :, :1], x[..., :32], x[:1], x[:, :2] if i else x[None],
                    x.transpose(2, 3).contiguous().transpose(2, 3), odd(x), wide(x)):
            args = list(good)
            args[i] = bad
            for n in (None, n_new):
                with pytest.raises((P.PBSAError, ValueError)):
                    tc.step(*args, n)
    assert all(torch.equal(a, b) for a, b in zip(state(tc), want))
    tc.step(*good, n_new)
    assert tc.seen.tolist() == [93, 91] and int(tc.status.item()) == 0


def test_counts_beyond_the_step_are_held_to_it(cuda_dev):
    """n_new below 0 counts as 0 and above T as T: positions never repeat and never skip."""
    B, Hq, Hkv, D, N = 3, 2, 1, 64, 64
    a, b = (TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=4, device=cuda_dev) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    for given, meant in (([9, -3, 2], [3, 0, 2]), ([2 ** 31 - 1, -2 ** 31, 1], [3, 0, 1]), ([3, 3, 0], [3, 3, 0])):
        x = tokens(cuda_dev, g, B, 3, Hq, Hkv, D)
        i = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt, device=cuda_dev)
        oa, ob = a.step(*x, i(given)), b.step(*x, i(meant, torch.int64))
        assert torch.equal(oa, ob) and all(torch.equal(u, v) for u, v in zip(state(a), state(b)))
    assert a.seen.tolist() == [9, 3, 3] and a.kv_len.tolist() == [9, 3, 3] and int(a.status.item()) == 0


def test_counts_of_another_kind_are_refused(cuda_dev):
    tc = TokenCache(2, 2, 1, 64, 64, n_sink=2, n_recent=4, device=cuda_dev)
    x = tokens(cuda_dev, torch.Generator().manual_seed(2), 2, 3, 2, 1, 64)
    n = torch.tensor([1, 2], dtype=torch.int32, device=cuda_dev)
    for bad in (n.cpu(), n[:1], n[:, None], n.float(), n.bool()):
        with pytest.raises(ValueError):
            tc.step(*x, bad)
    assert (tc.pos == -1).all() and tc.seen.tolist() == [0, 0]


@pytest.mark.parametrize("n", [[2, 1], [1, 0], [0, 2], [3, 3]])
def test_padded_steps_take_empty_rows_before_rows_in_use(cuda_dev, n):
    """Two rows are empty, a step of three asks for one more: a sequence that has no more than two
    tokens in it gives up nothing."""
    B, Hq, Hkv, D, N = 2, 4, 2, 64, 64
    tc = TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=4, device=cuda_dev)
    g = torch.Generator().manual_seed(3)
    tc.step(*tokens(cuda_dev, g, B, 40, Hq, Hkv, D))
    tc.step(*tokens(cuda_dev, g, B, 22, Hq, Hkv, D))
    assert (tc.pos[:, :, :62] >= 0).all() and (tc.pos[:, :, 62:] == -1).all()
    before = tc.pos.clone()
    tc.step(*tokens(cuda_dev, g, B, 3, Hq, Hkv, D), torch.tensor(n, dtype=torch.int32, device=cuda_dev))
    for b, m in enumerate(n):
        kept = (tc.pos[b] == before[b])[:, :62].sum(-1)
        assert kept.tolist() == [62 - max(0, m - 2)] * Hkv
        held = tc.pos[b].sort(-1).values[:, N - min(m, 3):] if m else tc.pos[b][:, :0]
        assert held.tolist() == [list(range(62, 62 + m))] * Hkv
        assert (tc.pos[b] == -1).sum(-1).tolist() == [max(0, 2 - m)] * Hkv
    assert tc.kv_len.tolist() == [min(N, 62 + m) for m in n] and int(tc.status.item()) == 0


def test_buffers_of_many_lengths_do_not_pile_up(cuda_dev):
    """Steps of thirty lengths hold the buffers of a few; a captured step keeps its own, and its
    replay between them gives what an eager step gives."""
    B, Hq, Hkv, D, N = 1, 8, 2, 64, 1024
    a, b = (TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=8, device=cuda_dev) for _ in range(2))
    g = torch.Generator().manual_seed(4)
    static = [torch.zeros_like(t) for t in tokens(cuda_dev, g, B, 2, Hq, Hkv, D)]
    for tc in (a, b):
        tc.step(*static)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = a.step(*static)
    sizes, held, outs = [], [torch.cuda.memory_allocated()], []
    for T in [*range(60, 90), 3]:
        x = tokens(cuda_dev, g, B, T, Hq, Hkv, D)
        oa, ob = a.step(*x), b.step(*x)
        assert torch.equal(oa, ob)
        outs.append((oa, oa.clone()))
        del outs[:-3]
        assert all(torch.equal(x, y) for x, y in outs)     # nothing writes to an output of another length
        for s, t in zip(static, tokens(cuda_dev, g, B, 2, Hq, Hkv, D)):
            s.copy_(t)
        graph.replay()
        assert torch.equal(replayed, b.step(*static))
        sizes.append(len(a._steps))
        held.append(torch.cuda.memory_allocated())
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert max(sizes) <= 5 and 2 in a._steps
    # Each of the two caches keeps four lengths and makes a fifth; outs holds six outputs and a
    # step's inputs and comparisons are smaller than a length's buffers.  Buffers grow with T (from
    # 65 tokens on, 260 query rows a head are two groups and the parts' count doubles), so the
    # largest length bounds them all: 2 (4 + 1) + 1 of it, of thirty.
    most = P.pbsa_kv4_workspace_size(a.cfg, 89) + 89 * Hq * (D * 2 + 4) + 89 * (Hkv + 1) * 4 + 5 * 512
    assert max(held) - held[0] <= 11 * most


@pytest.mark.parametrize("replay", [False, True])
def test_a_length_that_was_captured_first(cuda_dev, replay):
    """Buffers that a capture allocated serve eager steps too, before any replay and after."""
    B, Hq, Hkv, D, N = 2, 4, 2, 64, 64
    a, b = (TokenCache(B, Hq, Hkv, D, N, n_sink=2, n_recent=4, device=cuda_dev) for _ in range(2))
    g = torch.Generator().manual_seed(5)
    x = tokens(cuda_dev, g, B, 1, Hq, Hkv, D)
    a.step(*x), b.step(*x)
    n = torch.tensor([3, 2], dtype=torch.int32, device=cuda_dev)
    x = tokens(cuda_dev, g, B, 3, Hq, Hkv, D)
    torch.full((64,), -7, dtype=torch.int32, device=cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a.step(*x, n)
    if replay:
        graph.replay()
        assert torch.equal(out, b.step(*x, n))
    for _ in range(2):
        y = tokens(cuda_dev, g, B, 3, Hq, Hkv, D)
        assert torch.equal(a.step(*y, n), b.step(*y, n))
    assert all(torch.equal(u, v) for u, v in zip(state(a), state(b)))

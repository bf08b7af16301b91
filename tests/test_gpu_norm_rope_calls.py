"""SparseForcingAttention.norm_rope as a function of its inputs: on several streams, captured, and
at the ends of its table."""
import pytest
import torch

from block_sparse_attention_35_b200.attention import SparseForcingAttention

pytestmark = pytest.mark.gpu


def attention(dev, B=1, H=12, D=128, fh=16, fw=16, frames=8):
    return SparseForcingAttention(B, H, D, fh, fw, total_cache_size=4 * fh * fw, local_cache_size=2 * fh * fw,
                                  persistent_cache_size=2 * fh * fw, max_seq_len=frames * fh * fw, chunk_frames=1,
                                  device=dev)


def heads(dev, g, a, n):
    x = lambda dt: torch.randn(a.B, n * a.tf, a.H, a.D, generator=g).to(dt).to(dev)
    w = lambda: (1 + 0.2 * torch.randn(a.D, generator=g)).to(dev)
    return x(torch.bfloat16), x(torch.bfloat16), w(), w(), x(torch.float32), x(torch.float32)


def test_calls_on_two_streams_do_not_share_their_sums(cuda_dev):
    a = attention(cuda_dev)
    g = torch.Generator().manual_seed(0)
    ins = [heads(cuda_dev, g, a, 8) for _ in range(2)]
    run = lambda x: a.norm_rope_backward(*x[:4], 0, *x[4:])
    want = []
    for x in ins:
        want.append(run(x))
        torch.cuda.synchronize()
    streams, graphs, got = [torch.cuda.Stream() for _ in ins], [], []
    for x in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append([run(x) for _ in range(20)])
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for rs, w in zip(got, want):
        for r in rs:
            assert all(torch.equal(u, v) for u, v in zip(r, w))


@pytest.mark.parametrize("B", [1, 2])
def test_a_first_call_that_is_captured(cuda_dev, B):
    """Neither the table nor the positions are made by the first call."""
    a, b = (attention(cuda_dev, B=B, H=2, D=64) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    x = heads(cuda_dev, g, a, 2)
    want = [*b.norm_rope(*x[:4], 3), *b.norm_rope_backward(*x[:4], 3, *x[4:])]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [*a.norm_rope(*x[:4], 3), *a.norm_rope_backward(*x[:4], 3, *x[4:])]
    eager = [*a.norm_rope(*x[:4], 3), *a.norm_rope_backward(*x[:4], 3, *x[4:])]
    assert all(torch.equal(u, v) for u, v in zip(eager, want))
    graph.replay()
    assert all(torch.equal(u, v) for u, v in zip(out, want))
    assert int(a.status.item()) == 0


def test_frames_past_the_table_are_refused(cuda_dev):
    """Their outputs would be left unwritten.  The last frames of the table are not refused."""
    a = attention(cuda_dev, H=2, D=64, fh=4, fw=8, frames=10)
    g = torch.Generator().manual_seed(2)
    x = heads(cuda_dev, g, a, 2)
    for first in (-1, 9, 10, 10 ** 9):
        with pytest.raises(ValueError):
            a.norm_rope(*x[:4], first)
        with pytest.raises(ValueError):
            a.norm_rope_backward(*x[:4], first, *x[4:])
    q, k = a.norm_rope(*x[:4], 8)
    assert torch.isfinite(q).all() and int(a.status.item()) == 0
    # what a table starts with does not depend on its length
    b = attention(cuda_dev, H=2, D=64, fh=4, fw=8, frames=40)
    assert all(torch.equal(u, v) for u, v in zip((q, k), b.norm_rope(*x[:4], 8)))


@pytest.mark.parametrize("B", [1, 2])
@pytest.mark.parametrize("fh,fw", [(3, 5), (2, 3), (9, 7)])
def test_frames_of_odd_sizes(cuda_dev, B, fh, fw):
    """Positions of a later frame begin at any multiple of 12 bytes; two frames at once are the two
    one by one."""
    a = attention(cuda_dev, B=B, H=2, D=64, fh=fh, fw=fw, frames=12)
    g = torch.Generator().manual_seed(3)
    q, k, wq, wk, gq, gk = heads(cuda_dev, g, a, 2)
    one = lambda t, i: t[:, i * a.tf:(i + 1) * a.tf]
    for first in range(5):
        both = (*a.norm_rope(q, k, wq, wk, first), *a.norm_rope_backward(q, k, wq, wk, first, gq, gk)[:2])
        for i in range(2):
            x = [one(t, i) for t in (q, k, gq, gk)]
            got = (*a.norm_rope(*x[:2], wq, wk, first + i),
                   *a.norm_rope_backward(*x[:2], wq, wk, first + i, *x[2:])[:2])
            assert all(torch.equal(u, one(v, i)) for u, v in zip(got, both))
    assert int(a.status.item()) == 0

"""la2_state_copy and la2_state_compact against plain loops: exact moves."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_la2_b200 import build

    build.build()
    from linear_attention_la2_b200 import la2 as lib

    return lib


def pool_of(S, H, d, dv, offset=0):
    """A pool with a margin in front and behind; offset: floats off 16-byte alignment."""
    n = S * H * d * dv
    buf = torch.randn(n + 64 + offset, generator=torch.Generator().manual_seed(S + d)).cuda()
    return buf, buf[32 + offset:32 + offset + n].view(S, H, d, dv)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("shape,offset", [((6, 2, 64, 64), 0), ((6, 3, 128, 128), 0), ((6, 1, 1, 1), 0),
                                          ((6, 3, 7, 5), 0), ((6, 2, 64, 64), 1), ((6, 1, 33, 4), 0)])
def test_copy(la2, shape, offset):
    buf, pool = pool_of(*shape, offset)
    before = buf.clone()
    ref = pool.cpu().numpy().copy()
    src, dst = [0, 0, -1, 3, 1], [2, 5, 4, 3, -1]
    la2.state_copy(pool, ints(src), ints(dst))
    la2.check()
    assert np.array_equal(pool.cpu().numpy(), oracle.state_copy(ref, src, dst))
    n = pool.numel()
    assert torch.equal(buf[:32 + offset], before[:32 + offset])
    assert torch.equal(buf[32 + offset + n:], before[32 + offset + n:])


@pytest.mark.parametrize("src,dst,done", [
    ([0, 1], [1, 2], [1]),          # 1 is read by the second entry: the first is refused
    ([0, 1], [2, 2], [0]),          # 2 is written twice: the later entry is refused
    ([0, 1], [1, 0], []),           # a swap: both are
    ([0, 9], [1, 2], [0]),
    ([0, 1], [3, 9], [0]),
    ([0, -2], [3, 2], [0]),
    ([0, 1], [3, -2], [0]),
    ([9, 0], [9, 3], [1]),
])
def test_refused_copies_are_skipped_and_reported(la2, src, dst, done):
    _, pool = pool_of(4, 2, 16, 16)
    ref = pool.cpu().numpy().copy()
    la2.state_copy(pool, ints(src), ints(dst))
    assert la2.la2_check(la2._stream_handle(None)) == la2.LA2_ERR_INVALID_ARG
    assert la2.la2_check(la2._stream_handle(None)) == la2.LA2_OK
    assert np.array_equal(pool.cpu().numpy(), oracle.state_copy(ref, [src[i] for i in done], [dst[i] for i in done]))


@pytest.mark.parametrize("S,H,d,dv,p", [(1, 1, 4, 4, 0.5), (7, 2, 16, 8, 0.0), (7, 2, 16, 8, 1.0),
                                        (33, 1, 7, 3, 0.5), (64, 4, 32, 32, 0.3), (1500, 1, 4, 4, 0.5),
                                        (5000, 1, 2, 3, 0.9), (14000, 1, 4, 1, 0.5), (32768, 1, 1, 1, 0.4)])
def test_compact(la2, S, H, d, dv, p):
    buf, pool = pool_of(S, H, d, dv)
    before = buf.clone()
    live = (np.random.default_rng(S).random(S) < p).astype(np.int32)
    want, moved = oracle.state_compact(pool.cpu().numpy(), live)
    got = la2.state_compact(pool, ints(live.tolist()) * 3)
    la2.check()
    assert got.cpu().tolist() == moved.tolist()
    n = int(live.sum())
    assert np.array_equal(pool.cpu().numpy()[:n], want[:n])
    assert np.array_equal(pool.cpu().numpy()[n:], want[n:])
    m = pool.numel()
    assert torch.equal(buf[:32], before[:32]) and torch.equal(buf[32 + m:], before[32 + m:])


def test_replayed_from_a_graph_with_other_lists(la2):
    _, pool = pool_of(5, 2, 32, 32)
    src, dst, live = ints([0, 1]), ints([2, 3]), ints([1, 1, 1, 1, 1])
    moved = torch.empty_like(live)
    la2.state_copy(pool, src, dst)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la2.state_copy(pool, src, dst)
        la2.state_compact(pool, live, moved)
    src.copy_(ints([4, -1]))
    live.copy_(ints([0, 1, 0, 1, 1]))
    ref = pool.cpu().numpy().copy()
    graph.replay()
    la2.check()
    want, m = oracle.state_compact(oracle.state_copy(ref, [4, -1], [2, 3]), [0, 1, 0, 1, 1])
    assert np.array_equal(pool.cpu().numpy(), want) and moved.cpu().tolist() == m.tolist()


@pytest.mark.parametrize("S", [2, 3, 31, 1023, 1024, 1025])
@pytest.mark.parametrize("front", [True, False])
def test_compact_around_one_launch(la2, S, front):
    """Pools up to and beyond those that are compacted by one launch: the dead slots all
    in front (every live one moves that can), or spread."""
    _, pool = pool_of(S, 1, 4, 5)
    live = np.arange(S) >= (S + 1) // 2 if front else np.random.default_rng(S).random(S) < 0.6
    live = live.astype(np.int32)
    want, moved = oracle.state_compact(pool.cpu().numpy(), live)
    got = la2.state_compact(pool, ints(live.tolist()))
    la2.check()
    assert got.cpu().tolist() == moved.tolist() and np.array_equal(pool.cpu().numpy(), want)

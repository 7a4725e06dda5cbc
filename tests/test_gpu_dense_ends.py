"""The dense layer's operators at the ends of their ranges: positions up to the type's last value, caches
without tokens, the largest and smallest BF16 values, NaN in every kind of step, many rows of 4-bit
projections.  References and bounds are those of tests/dense_ref.py; tolerances count roundings."""
import numpy as np
import pytest
import torch

import long_context_sparse_softmax_b200 as lc
from tests import dense_ref as R
from tests.test_gpu_dense_layer import BF16, GpuCache, check_attn, gpu, make_cache, np64, p, rng_for, run_attn

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 1


# ------------------------------------------------------------ windows that have left the cache
@pytest.mark.parametrize("D,bt,g,nq", [(128, 64, 8, 1), (64, 16, 5, 1), (128, 16, 3, 4), (64, 16, 4, 40), (128, 32, 8, 70), (64, 128, 1, 200)])
@pytest.mark.parametrize("W", [1, 5, 37])
def test_attn_windows_behind_the_cache(D, bt, g, nq, W):
    """Every query of a sequence past the end of its cache by more than the window, up to the last
    position there is; one sequence whose window still reaches the cache for its first queries, one whose
    first queries lie before the cache."""
    r = rng_for(D, g, nq, W)
    kv = np.array([40, 333, 300, 0, 100, 90, 200])
    pos = np.array([1000, 10 ** 9 + 7, LAST - (nq - 1), 77, LAST - (nq - 1) - 300, 88, -3])
    c = make_cache(r, kv, 2, D, bt)
    q = gpu(r.standard_normal((len(kv) * nq, 2 * g, D)) * 2.0 ** -8, BF16)
    start = np.arange(len(kv) + 1) * nq
    for sink in (None, r.standard_normal(2 * g).astype(np.float32)):
        for decode in ([True, False] if nq == 1 else [False]):
            got = run_attn(GpuCache(c), q, start, pos, kv, 2 * g, decode, W=W, sink=sink)
            assert got[2] == 0
            check_attn(c, np64(q), start, pos, kv, 2 * g, got[0], got[1], W=W, sink=sink)
            gone = np.arange(5 * nq)  # of the first five: nothing visible
            assert not got[0][gone].any()
            assert np.array_equal(got[1][gone], np.broadcast_to(-np.inf if sink is None else sink.astype(np.float64), (5 * nq, 2 * g)))


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_attn_positions_at_the_types_last_value(nq):
    """Without a window, and with one as wide: the whole cache, bit by bit as from its end."""
    r = rng_for(nq, 3)
    kv = np.array([700])
    c = make_cache(r, kv, 1, 128, 32)
    q = gpu(r.standard_normal((nq, 4, 128)) * 2.0 ** -8, BF16)
    far = LAST - (nq - 1)
    want = run_attn(GpuCache(c), q, [0, nq], np.array([kv[0] + 10]), kv, 4, nq == 1)
    check_attn(c, np64(q), np.array([0, nq]), np.array([kv[0] + 10]), kv, 4, want[0], want[1])
    for W in (0, LAST):
        got = run_attn(GpuCache(c), q, [0, nq], np.array([far]), kv, 4, nq == 1, W=W)
        assert got[2] == 0
        if W == 0:
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        else:  # the last positions no longer see the first tokens
            check_attn(c, np64(q), np.array([0, nq]), np.array([far]), kv, 4, got[0], got[1], W=W)


# ------------------------------------------------------------------ caches that hold nothing
@pytest.mark.parametrize("nq", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_without_a_cache(D, nq):
    """max_kv 0 with no arrays behind the cache, and a pool of no blocks whose tables name none: every query
    gets o = 0 and the sink's logit (-inf without one)."""
    S, H = 3, 6
    q = gpu(rng_for(D, nq).standard_normal((S * nq, H, D)), BF16)
    start, pos, kv = np.arange(S + 1) * nq, np.array([0, 5, 100]), np.array([0, 50, 64])

    class Pool:
        pass
    none = Pool()
    none.args = lc.Kv8Cache(H_kv=2, D=D, bt=16, n_blocks=0, table_cols=0)
    empty = Pool()
    table = torch.full((S, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 3] = 0, 7  # outside a pool of no blocks
    room = torch.zeros(256, dtype=torch.uint8, device="cuda")
    empty.args = lc.Kv8Cache(H_kv=2, D=D, bt=16, n_blocks=0, table_cols=4, k=p(room), v=p(room), k_scale=p(room), v_scale=p(room), table=p(table))
    for sink in (None, np.float32([-3, 0, 1, 2, 90, -np.inf])):
        for decode in ([True, False] if nq == 1 else [False]):
            for pool, max_kv, status in ((none, 0, 0), (empty, 0, 0), (empty, 64, lc.LC_DEV_BAD_BLOCK)):
                got = run_attn(pool, q, start, pos, kv, H, decode, sink=sink, max_kv=max_kv)
                assert got[2] == status
                assert not got[0].any()
                assert np.array_equal(got[1], np.broadcast_to(-np.inf if sink is None else sink.astype(np.float64), (S * nq, H)))

"""The dense layer's operators at the ends of their ranges: positions up to the type's last value, caches
without tokens, the largest and smallest BF16 values, NaN in every kind of step, many rows of 4-bit
projections.  References and bounds are those of tests/dense_ref.py; tolerances count roundings."""
import numpy as np
import pytest
import torch

import long_context_sparse_softmax_b200 as lc
from tests import dense_ref as R
from tests.test_gpu_dense_layer import (BF16, F32, GpuCache, check_attn, gpu, make_cache, make_w4, np64, p, rng_for, run_attn, run_w4,
                                        w4_reference)

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


# ---------------------------------------------------------------- the two terms of a BF16 row
SPLIT = 2.0 ** -14 / 224  # of a block's largest value: half of the second term's step, where that value is 224 X


def bf16(bits):
    """BF16 bit patterns -> float64."""
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("n", [1, 8, 20, 40])
@pytest.mark.parametrize("end", ["largest", "smallest"])
def test_w4_at_the_ends_of_bf16(n, end):
    """Rows of the largest finite values (up to 0x7f7f, which needs the scale 2^120) under small weight
    scales, and rows of subnormal ones under large scales: the bound of every other row, relative to what the
    row holds.  FP32 sums of K products, the split, the output's rounding."""
    r = rng_for(n, end == "largest")
    G, K, dg = 2, 160, 70
    codes, scales = make_w4(r, G, dg, K)
    if end == "largest":
        bits = r.choice([0x7f7f, 0xff7f, 0x7f70, 0xff6f, 0x7f6e, 0x7e80, 0x3f80, 0x0001], (n, G * K))
        scales = scales - 100
    else:
        bits = r.integers(0, 0x0400, (n, G * K)) | r.integers(0, 2, (n, G * K)) << 15  # below 2^-119
        bits[0, :32] = 1                        # a block of the smallest value there is
        bits[0, 32:64] = r.integers(0, 128, 32)  # subnormals alone
        scales = scales + 100
    x64 = bf16(bits)
    xt = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).cuda().view(torch.bfloat16)
    ref, mag, top = w4_reference(x64, codes, scales.astype(np.uint8), G, K, dg)
    got = run_w4(xt, None, codes, scales.astype(np.uint8), G, K, dg, F32)
    lim = (K + 1) * 2.0 ** -24 * mag + SPLIT * top
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / lim)


@pytest.mark.parametrize("n", [8, 16, 32])
def test_w4_split_of_every_significand(n):
    """Against the identity an output is what the two terms make of one value: exact from 1 / 14336 of the
    block's largest value on, within the bound below.  Every significand as the largest of a block, with 31
    values of any significand over 24 octaves below it, at exponents whose
    outputs stay FP32's normal numbers."""
    r = rng_for(n, 14336)
    K = 32 * 128
    x = np.empty((n, 128, 32))
    for i in range(n):
        big = bf16(((128 + r.integers(-95, 127, 128)) << 7) | np.arange(128))
        low = bf16(r.integers(126 << 7, 127 << 7, (128, 31))) * np.exp2(r.integers(-24, 1, (128, 31)).astype(float))  # below 1
        x[i, :, 0] = big
        x[i, :, 1:] = big[:, None] * low * r.choice([-1, 1], (128, 31))
    xt = torch.from_numpy(x.reshape(n, K).astype(np.float32)).cuda().to(torch.bfloat16)
    x64 = np64(xt)
    codes = np.zeros((1, K, K // 2), np.uint8)
    k = np.arange(K)
    codes[0, k, k // 2] = np.where(k % 2, 0x20, 0x02)  # 1.0
    got = run_w4(xt, None, codes, np.full((1, K, K // 32), 127, np.uint8), 1, K, K, F32)
    err = np.abs(got - x64).reshape(n, 128, 32)
    a = np.abs(x64).reshape(n, 128, 32)
    top = a.max(2, keepdims=True)
    assert not err[a * 14336 >= top].any()
    assert np.all(err <= SPLIT * top), np.max(err / top) * 2.0 ** 21.8

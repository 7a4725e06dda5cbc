"""The dense layer's operators at the ends of their ranges: positions up to the type's last value, caches
without tokens, the largest and smallest BF16 values, NaN in every kind of step, many rows of 4-bit
projections.  References and bounds are those of tests/dense_ref.py; tolerances count roundings."""
import numpy as np
import pytest
import torch

import long_context_sparse_softmax_b200 as lc
from tests import dense_ref as R
from tests.test_gpu_dense_layer import (BF16, F32, GpuCache, attn_args, check_attn, gpu, make_cache, make_w4, np64, p, rng_for, run_attn, run_w4,
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


# --------------------------------------------------------------------- NaN among keys and values
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("W", [0, 45])
@pytest.mark.parametrize("D,bt,g,nq,kv", [
    (128, 32, 3, 4, 200), (64, 16, 5, 3, 150),      # few rows, one split
    (128, 64, 3, 9, 3000), (64, 16, 14, 2, 2900),   # few rows, split keys (the second: two row tiles' worth of heads)
    (128, 32, 4, 70, 900), (64, 64, 3, 100, 700),   # many rows
    (128, 16, 2, 150, 5000), (64, 128, 7, 40, 4500)])  # many rows behind a long prefix, split keys
def test_attn_nan_in_every_kind_of_step(D, bt, g, nq, kv, W, where):
    """A NaN at the last token, among the last queries, right before them, at the start of the first query's
    window, in front of it (seen by none with a window), in the middle and at token 0: the queries that see
    it are NaN (from a value: in that dim alone), and the others as without it."""
    r = rng_for(D, g, nq, W, where == "k")
    c = make_cache(r, [kv], 1, D, bt)
    q = gpu(r.standard_normal((nq, g, D)) * 2.0 ** -8, BF16)
    sees_from = max(0, kv - nq - W + 1) if W else 0
    for t in sorted({kv - 1, kv - 1 - nq // 2, kv - nq - 1, sees_from, max(sees_from - 1, 0), kv // 2, 0}):
        bad = R.Cache(c.k.copy(), c.ks, c.v.copy(), c.vs, c.table)
        dim = int(r.integers(0, D))
        getattr(bad, where)[c.table[0, t // bt], 0, t % bt, dim] = 0x7f if t % 2 else 0xff
        got = run_attn(GpuCache(bad), q, [0, nq], [kv - nq], [kv], g, False, W=W)
        assert got[2] == 0
        check_attn(bad, np64(q), np.array([0, nq]), [kv - nq], [kv], g, got[0], got[1], W=W)
        p_ = kv - nq + np.arange(nq)
        hit = (t <= p_) & ((t > p_ - W) if W else True)
        nan = np.isnan(got[0])
        assert nan[hit].all() if where == "k" else (nan[hit][..., dim].all() and nan.sum() == hit.sum() * g)
        assert not nan[~hit].any()


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("D,bt,g,kv", [(128, 32, 8, 203), (64, 16, 3, 37), (128, 64, 16, 2501)])
def test_attn_decode_nan_in_the_last_step(D, bt, g, kv, where):
    """The last 16-key step is partial, and the rows of its block behind the cache are NaN anyway: only a NaN
    at a token reaches the query, and with a window only one inside it."""
    r = rng_for(D, g, kv, where == "k")
    c = make_cache(r, [kv], 2, D, bt)
    q = gpu(r.standard_normal((1, 2 * g, D)) * 2.0 ** -8, BF16)
    for t, W in ((kv - 1, 0), (kv & ~15, 0), (kv - 10, 10), (kv - 11, 10), (kv - 10, 9)):
        bad = R.Cache(c.k.copy(), c.ks, c.v.copy(), c.vs, c.table)
        getattr(bad, where)[c.table[0, t // bt], 1, t % bt, 5] = 0x7f
        got = run_attn(GpuCache(bad), q, [0, 1], [kv - 1], [kv], 2 * g, True, W=W)
        check_attn(bad, np64(q), np.array([0, 1]), [kv - 1], [kv], 2 * g, got[0], got[1], W=W)
        hit = W == 0 or t > kv - 1 - W
        nan = np.isnan(got[0])
        assert nan.sum() == (0 if not hit else g * (D if where == "k" else 1)) and not nan[:, :g].any()


def test_attn_nan_behind_a_long_prefix_costs_no_more():
    """Where a replaced value code is looked for again is the tiles that not every row sees: what a NaN in the
    last tile costs does not grow with the cache (a scan of all of it would cost 16 times as much here)."""
    r = rng_for(65536)
    Hkv, g, D, bt, nq = 8, 8, 64, 64, 640

    def extra(kv):
        c = make_cache(r, [kv], Hkv, D, bt)
        q = gpu(r.standard_normal((nq, Hkv * g, D)) * 2.0 ** -8, BF16)
        gc = GpuCache(c)
        a, out, lse, status, keep = attn_args(gc, q, [0, nq], [kv - nq], [kv], Hkv * g, False)
        assert a.workspace_bytes == 0  # the keys are not split

        def took():
            ms = []
            for _ in range(5):
                e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
                e[0].record()
                lc.lc_kv8_attn_prefill(a)
                e[1].record()
                torch.cuda.synchronize()
                ms.append(e[0].elapsed_time(e[1]))
            return min(ms)
        clean = took()
        gc.t[2][int(c.table[0, (kv - 20) // bt]), :, (kv - 20) % bt, 3] = 0x7f
        bad = took()
        nan = torch.isnan(out[-20:, :, 3])
        assert nan.all() and not torch.isnan(out[-20:, :, :3]).any()
        return bad - clean
    assert extra(65536) < 4 * extra(4096)


# ------------------------------------------------------------------------------ many rows
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("n,G,K,dg", [(131, 2, 160, 40), (300, 1, 1056, 300), (1000, 3, 64, 129), (2113, 1, 256, 128)])
def test_w4_rows_of_a_prompt(n, G, K, dg, mx):
    """Accepted, if slow: every 32 (64) rows read the weights again.  The bound of test_w4 with the split's own
    constant."""
    r = rng_for(n, K, mx)
    codes, scales = make_w4(r, G, dg, K)
    x = r.standard_normal((n, G * K)) * np.exp2(r.integers(-12, 13, (n, G * K)))
    if mx:
        e = R.scale_exp(R.finite_amax(x.reshape(n, -1, 32), 2), -127, 127, 0)
        xc = R.e4m3_codes(x * np.repeat(np.exp2(-e.astype(float)), 32, 1))
        sc = (e + 127).astype(np.uint8)
        x64, xt, xs = R.mxfp8_rows(xc, sc), torch.from_numpy(xc).cuda(), torch.from_numpy(sc).cuda()
    else:
        xt, xs = gpu(x, BF16), None
        x64 = np64(xt)
    ref, mag, top = w4_reference(x64, codes, scales, G, K, dg)
    got = run_w4(xt, xs, codes, scales, G, K, dg, F32)
    lim = (K + 1) * 2.0 ** -24 * mag + (0 if mx else SPLIT * top)
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / lim)


def test_w4_tiny_rows_next_to_others():
    """A row of 1e-37 among rows of zeros, of 1e30, of NaN and infinities, under weights large enough that its
    outputs are normal numbers: held to its own size."""
    r = rng_for(78)
    G, K, dg = 2, 128, 70
    codes, scales = make_w4(r, G, dg, K)
    scales = (scales + 90).astype(np.uint8)
    x = r.standard_normal((8, G * K))
    x[0] = 0
    x[1] *= 1e-37
    x[2] *= 1e-30
    x[3, 3], x[4, K + 9] = np.nan, np.inf
    x[5] *= 1e-20
    xt = gpu(x, BF16)
    got = run_w4(xt, None, codes, scales, G, K, dg, F32)
    x64 = np.where(np.isfinite(np64(xt)), np64(xt), 0)
    ref, mag, top = w4_reference(x64, codes, scales, G, K, dg)
    ok = np.abs(got - ref) <= (K + 1) * 2.0 ** -24 * mag + SPLIT * top
    assert np.isnan(got[3, :dg]).all() and np.isnan(got[4, dg:]).all()
    ok[3, :dg] = ok[4, dg:] = True
    assert ok.all() and np.abs(got[1]).max() > 1e-10 and not got[0].any()

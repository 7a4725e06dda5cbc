"""The operators around a dense attention layer with an 8-bit cache, through the C ABI, against
their 64-bit definitions (tests/dense_ref.py): at the sizes, masks and values where they can go
wrong, and as a layer's step runs them.  Tolerances count roundings (half a step: BF16 2^-8, F16
2^-11, FP32 2^-24, E4M3 2^-4) and are derived beside each check."""
import numpy as np
import pytest
import torch

import long_context_sparse_softmax_b200 as lc
from oracle import lc_oracle as O
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, MXFP8 = lc.LC_FMT_F32, lc.LC_FMT_BF16, lc.LC_FMT_MXFP8
DT = {F32: torch.float32, BF16: torch.bfloat16}


def p(t):
    return None if t is None else t.data_ptr()


def np64(t):
    return t.detach().double().cpu().numpy()


def rng_for(*seed):
    return np.random.default_rng([int(x) for x in seed])


def gpu(a, fmt):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(DT[fmt])


# ------------------------------------------------------------------------------ add_rms_norm
def run_norm(x, res, w, out_fmt, eps=1e-6, res_out=None, stream=None):
    n, d = x.shape
    fmt = F32 if x.dtype == torch.float32 else BF16
    y = torch.empty(n, d, device="cuda", dtype=DT.get(out_fmt, torch.uint8))
    ys = torch.empty(n, max(d // 32, 1), device="cuda", dtype=torch.uint8)
    a = lc.AddRmsNormArgs(n_rows=n, d=d, in_fmt=fmt, x=p(x), res=p(res), res_out=p(res_out), w=p(w),
                          w_fmt=F32 if w is not None and w.dtype == torch.float32 else BF16, out_fmt=out_fmt, y=p(y),
                          y_scale=p(ys), eps=eps)
    lc.lc_add_rms_norm(a, stream)
    torch.cuda.synchronize()
    return y, ys


def check_norm(x64, res64, w64, out_fmt, y, ys, eps=1e-6):
    """FP32 terms: the sum of squares is a tree of at most 8 kV + 5 + 16 + 1 adds of one rounding
    each (kV <= 4: 54), halved by the square root; the quotient, root, reciprocal, two products
    and the residual's sum add 2^-24 each: 40 * 2^-24 in all.  The residual's own rounding is
    relative to r, which the 64-bit r has without it: one more 2^-24 of |r|."""
    _, ref = R.add_rms_norm(x64, res64, w64, eps)
    fine = np.isfinite(ref)
    tol = 40 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -149
    if out_fmt == MXFP8:
        codes, sc = y.cpu().numpy(), ys.cpu().numpy()
        n, d = ref.shape
        blk = ref.reshape(n, -1, 32)
        # the scale: that of the 64-bit maximum, or of one within the FP32 error of it
        am = R.finite_amax(blk, 2)
        lo = R.scale_exp(am * (1 - 2.0 ** -18), -127, 127, 0)
        hi = R.scale_exp(am * (1 + 2.0 ** -18), -127, 127, 0)
        e = sc.astype(np.int64) - 127
        bad_rows = ~fine.all(1)
        assert np.all(((e >= lo) & (e <= hi)) | bad_rows[:, None])
        got = R.mxfp8_rows(codes, sc)
        X = np.repeat(np.exp2(e.astype(float)), 32, 1)
        tol = tol + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * X
    else:
        got = np64(y)
        if out_fmt == BF16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got - ref)
    assert np.all((err <= tol) | ~fine), np.max((err / tol)[fine])
    assert np.all(~np.isfinite(got[~fine]) | (out_fmt == MXFP8))


@pytest.mark.parametrize("out_fmt", [F32, BF16, MXFP8], ids=["f32", "bf16", "mxfp8"])
@pytest.mark.parametrize("fmt", [F32, BF16], ids=["xf32", "xbf16"])
@pytest.mark.parametrize("rows,d", [(1, 32), (3, 64), (5, 2880), (2, 7168), (7, 8192), (3, 8224), (2, 16384), (130, 576), (1, 1024)])
def test_norm(rows, d, fmt, out_fmt):
    r = rng_for(rows, d, fmt, out_fmt)
    x, res = gpu(r.standard_normal((rows, d)), fmt), gpu(3 * r.standard_normal((rows, d)), fmt)
    w = gpu(1 + 0.3 * r.standard_normal(d), BF16 if d % 3 else F32)
    ro = torch.empty_like(res)
    y, ys = run_norm(x, res, w, out_fmt, res_out=ro)
    check_norm(np64(x), np64(res), np64(w), out_fmt, y, ys)
    s = np64(x) + np64(res)
    assert np.all(np.abs(np64(ro) - s) <= (2.0 ** -24 if fmt == F32 else 2.0 ** -8) * np.abs(s) + 2.0 ** -149)
    # in place over either input, and without residual or weight
    for into in ("res", "x"):
        x2, res2 = x.clone(), res.clone()
        y2, _ = run_norm(x2, res2, w, out_fmt, res_out=res2 if into == "res" else x2)
        assert torch.equal(res2 if into == "res" else x2, ro) and torch.equal(y2, y)
    y3, ys3 = run_norm(x, None, None, out_fmt)
    check_norm(np64(x), None, None, out_fmt, y3, ys3)


def test_norm_width_of_eight():
    x = gpu(rng_for(1).standard_normal((9, 8)), BF16)
    y, ys = run_norm(x, None, None, F32)
    check_norm(np64(x), None, None, F32, y, ys)
    x = gpu(rng_for(2).standard_normal((9, 40)), F32)
    y, ys = run_norm(x, None, None, BF16)
    check_norm(np64(x), None, None, BF16, y, ys)


def test_norm_special_values():
    """Zero rows, tiny and huge rows, NaN and infinities: each row on its own; blocks of zeros
    take the scale 2^0; infinities saturate, NaN stays NaN."""
    r = rng_for(5)
    x = r.standard_normal((8, 128))
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 5] = np.nan
    x[4, 40:72] = 0
    x[5, 7] = np.inf
    xt = gpu(x, F32)
    for fmt in (F32, BF16, MXFP8):
        y, ys = run_norm(xt, None, None, fmt, eps=1e-6)
        fine = [0, 1, 2, 4, 6, 7]
        check_norm(np64(xt)[fine], None, None, fmt, y[fine], ys[fine])
        got = R.mxfp8_rows(y.cpu().numpy(), ys.cpu().numpy()) if fmt == MXFP8 else np64(y)
        assert np.isnan(got[3]).all()
        assert np.isnan(got[5, 7]) and np.all(got[5, :7] == 0)  # finite / inf
        assert np.all(got[0] == 0)
    assert ys[0].eq(127).all()
    # the weight brings infinities into a finite row
    w = np.ones(128)
    w[3] = np.inf
    y, ys = run_norm(xt[6:], None, gpu(w, F32), MXFP8)
    got = y.cpu().numpy()
    assert np.all((got[:, 3] & 0x7f) == 0x7e)  # +-448
    _, ref = R.add_rms_norm(np64(xt)[6:], None, None, 1e-6)
    keep = np.arange(128) != 3
    v = R.mxfp8_rows(got, ys.cpu().numpy())
    X = np.repeat(np.exp2(ys.cpu().numpy().astype(float) - 127), 32, 1)
    assert np.all((np.abs(v - ref) <= 2.0 ** -4 * np.abs(ref) * 1.01 + 2.0 ** -10 * X)[:, keep])


def test_norm_scale_borders():
    """Maxima exactly at 448 2^k take 2^k, the next FP32 value above takes 2^(k+1)."""
    d = 32
    for k in (-3, 0, 4):
        for over in (False, True):
            top = np.float32(448 * 2.0 ** k)
            if over:
                top = np.nextafter(top, np.float32(np.inf))
            # y = r * rstd * w with rstd = 1 / sqrt(1 + 0): r = +-1, so y = w exactly
            x = torch.ones(1, d, device="cuda")
            w = torch.full((d,), float(top) / 4, device="cuda")
            w[7] = float(top)
            y, ys = run_norm(x, None, w, MXFP8, eps=0.0)
            assert int(ys[0, 0]) - 127 == k + over
            assert (int(y[0, 7]) & 0x7f) == (0x76 if over else 0x7e)


# ----------------------------------------------------------------------------------- w4_proj
def make_w4(r, G, dg, K):
    codes = r.integers(0, 256, (G, dg, K // 2), dtype=np.uint8)
    scales = (127 + r.integers(-9, 4, (G, dg, K // 32))).astype(np.uint8)
    return codes, scales


def run_w4(x, xs, codes, scales, G, K, dg, out_fmt):
    n = x.shape[0]
    ct, st = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    y = torch.full((n + 1, G * dg), float("nan"), device="cuda", dtype=DT[out_fmt])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = lc.W4ProjArgs(n_q=n, G=G, K=K, d_g=dg, in_fmt=BF16 if xs is None else MXFP8, out_fmt=out_fmt, x=p(x), x_scale=p(xs),
                      w=p(ct), w_scale=p(st), y=p(y), status=p(status))
    lc.lc_w4_proj(a)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.isnan(y[n]).all()  # nothing behind the last row
    return np64(y[:n])


def w4_reference(x64, codes, scales, G, K, dg):
    w = R.mxfp4_rows(codes, scales)  # [G, dg, K]
    xg = x64.reshape(-1, G, K).transpose(1, 0, 2)
    y = np.einsum("gnk,gck->ngc", xg, w).reshape(-1, G * dg)
    mag = np.einsum("gnk,gck->ngc", np.abs(xg), np.abs(w)).reshape(-1, G * dg)
    # the largest value of each 32-block of x, against the same weights
    top = np.repeat(R.finite_amax(xg.reshape(G, -1, K // 32, 32), 3), 32, 2)
    return y, mag, np.einsum("gnk,gck->ngc", top, np.abs(w)).reshape(-1, G * dg)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("n,G,K,dg", [
    (1, 1, 32, 1), (1, 1, 4096, 300), (2, 3, 96, 17), (7, 1, 160, 128), (8, 1, 128, 129), (9, 2, 1056, 100), (16, 1, 512, 257),
    (17, 1, 7168, 130), (33, 8, 256, 64), (64, 1, 384, 40), (65, 2, 224, 31), (130, 1, 2080, 200), (5, 1, 20480, 128), (3, 40, 64, 512)])
def test_w4(n, G, K, dg, mx):
    """FP32 accumulation of K exact products (K 2^-24 of the sum of magnitudes), the split of BF16
    rows (2^-22 of a block's largest value; twice that allows for the scale's clamp), and the
    rounding of the output."""
    r = rng_for(n, G, K, dg, mx)
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
    tol = K * 2.0 ** -24 * mag + (0 if mx else 2.0 ** -21 * top) + 1e-30
    for fmt in (F32, BF16):
        got = run_w4(xt, xs, codes, scales, G, K, dg, fmt)
        err = np.abs(got - ref)
        lim = tol + (2.0 ** -8 * np.abs(ref) if fmt == BF16 else 2.0 ** -24 * np.abs(ref))
        assert np.all(err <= lim), np.max(err / lim)


def test_w4_extreme_rows_stay_apart():
    """Rows of zeros, of subnormal and of huge values, NaN and infinities: each affects itself only."""
    r = rng_for(77)
    G, K, dg = 2, 128, 70
    codes, scales = make_w4(r, G, dg, K)
    x = r.standard_normal((8, G * K))
    x[0] = 0
    x[1] *= 1e-37
    x[2] *= 1e30
    x[3, 3] = np.nan     # group 0 only
    x[4, K + 9] = np.inf  # group 1 only
    xt = gpu(x, BF16)
    x64 = np64(xt)
    got = run_w4(xt, None, codes, scales, G, K, dg, F32)
    assert np.isnan(got[3, :dg]).all() and np.isnan(got[4, dg:]).all()
    x64 = np.where(np.isfinite(x64), x64, 0)
    ref, mag, top = w4_reference(x64, codes, scales, G, K, dg)
    # 1e-37 rows: the scale's exponent is clamped at 2^-120, so values keep 2^-129 absolute
    tol = K * 2.0 ** -24 * mag + 2.0 ** -21 * top + 1e-30 + (2.0 ** -129 * 6 * 16 * K) * (np.arange(8) == 1)[:, None]
    ok = np.abs(got - ref) <= tol
    ok[3, :dg] = ok[4, dg:] = True
    assert ok.all()


@pytest.mark.parametrize("n", [1, 20, 40])
def test_w4_scales_at_the_ends_of_e8m0(n):
    """Weight scales 2^-127 .. 2^127 against x scales that bring the products back; the sums as in
    test_w4.  x at 2^-127 of a block's scale next to weights at 2^127."""
    r = rng_for(31, n)
    K, dg = 224, 40
    codes, _ = make_w4(r, 1, dg, K)
    we = np.repeat(np.array([[-127, 127, -126, 126, 0, 100, -100]]), dg, 0)  # per block of 32, the same in every row
    scales = (we + 127).astype(np.uint8)[None]
    xc = r.integers(0, 256, (n, K), dtype=np.uint8)
    xc = np.where((xc & 0x7f) == 0x7f, xc ^ 1, xc).astype(np.uint8)
    xs = np.repeat((127 - we[:1]).astype(np.uint8), n, 0)
    x64 = R.mxfp8_rows(xc, xs)
    ref, mag, _ = w4_reference(x64, codes, scales, 1, K, dg)
    got = run_w4(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), codes, scales, 1, K, dg, F32)
    assert np.all(np.abs(got - ref) <= K * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(ref) + 1e-30)


def test_w4_reads_what_the_quantiser_writes():
    r = rng_for(9)
    K, dg, n = 256, 96, 4
    wf = gpu(r.standard_normal((dg, K)), BF16)
    codes = torch.empty(dg, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(dg, K // 32, dtype=torch.uint8, device="cuda")
    lc.lc_mxfp4_quantize(lc.Mxfp4QuantArgs(dg, K, BF16, p(wf), p(codes), p(scales)))
    xt = gpu(r.standard_normal((n, K)), BF16)
    got = run_w4(xt, None, codes.cpu().numpy()[None], scales.cpu().numpy()[None], 1, K, dg, F32)
    w = O.mxfp4_to_f64(codes.cpu().numpy(), scales.cpu().numpy())
    ref = np64(xt) @ w.T
    assert np.all(np.abs(got - ref) <= K * 2.0 ** -23 * (np.abs(np64(xt)) @ np.abs(w).T) + 2.0 ** -21 * np.abs(w).sum(1) * np.abs(np64(xt)).max())


# ------------------------------------------------------------------------------------ cache
def make_cache(r, lens, Hkv, D, bt, spare=2, spread=6, cols=None):
    """Random valid codes everywhere (stale rows NaN), scales spread over 2 * spread octaves."""
    nb = [(int(n) + bt - 1) // bt for n in lens]
    n_blocks = sum(nb) + spare
    table = np.full((len(lens), cols or max(max(nb), 1)), -1, np.int32)
    perm = r.permutation(n_blocks)
    at = 0
    for s, c in enumerate(nb):
        table[s, :c] = perm[at:at + c]
        at += c

    def codes():
        c = r.integers(0, 256, (n_blocks, Hkv, bt, D), dtype=np.uint8)
        return np.where((c & 0x7f) == 0x7f, c ^ 1, c).astype(np.uint8)

    def scales():
        return (127 + r.integers(-spread, spread + 1, (n_blocks, Hkv))).astype(np.uint8)
    c = R.Cache(codes(), scales(), codes(), scales(), table)
    for s, n in enumerate(lens):  # rows past the end hold NaN codes
        if n % bt:
            blk = table[s, n // bt]
            c.k[blk, :, n % bt:] = 0x7f
            c.v[blk, :, n % bt:] = 0xff
    return c


class GpuCache:
    def __init__(self, c):
        self.t = [torch.from_numpy(x.copy()).cuda() for x in (c.k, c.ks, c.v, c.vs, c.table)]
        k, ks, v, vs, table = self.t
        self.args = lc.Kv8Cache(H_kv=c.Hkv, D=c.D, bt=c.bt, n_blocks=c.n_blocks, table_cols=table.shape[1], k=p(k), v=p(v),
                                k_scale=p(ks), v_scale=p(vs), table=p(table))

    def host(self):
        return [x.cpu().numpy() for x in self.t[:4]]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def run_append(gc, kx, vx, start, pos0, k_stride=0, v_stride=0, max_tok=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st, ps = i32(start), i32(pos0)
    n = int(np.max(np.diff(start))) if max_tok is None else max_tok
    a = lc.Kv8AppendArgs(cache=gc.args, num_seqs=len(pos0), in_fmt=F32 if kx.dtype == torch.float32 else BF16, max_tok=n,
                         k=p(kx), v=p(vx), k_stride=k_stride, v_stride=v_stride, tok_start=p(st), pos0=p(ps), status=p(status))
    lc.lc_kv8_append(a)
    torch.cuda.synchronize()
    return int(status.item())


@pytest.mark.parametrize("fmt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Hkv,D,bt", [(1, 64, 16), (3, 128, 16), (2, 64, 32), (8, 128, 64), (2, 128, 128), (1, 64, 128)])
def test_append_is_bit_exact(Hkv, D, bt, fmt):
    """Lengths 0 and 1, blocks entered in the middle, whole blocks, several at once; scales that
    grow and that stay; NaN and infinities; other rows untouched."""
    r = rng_for(Hkv, D, bt, fmt)
    old = [0, 0, 5, bt - 1, bt, 3 * bt + 7, 2, 40]
    new = [0, 1, 1, 2, bt, 2 * bt + 3, 5 * bt, 1]
    c = make_cache(r, [o + n for o, n in zip(old, new)], Hkv, D, bt)
    c.ks[:], c.vs[:] = 127 + r.integers(-9, -2, c.ks.shape), 127 + r.integers(-9, -2, c.vs.shape)
    n = sum(new)
    kx, vx = (r.standard_normal((n, Hkv, D)) * np.exp2(r.integers(-6, 7, (n, 1, 1))) for _ in range(2))
    kx[0, 0, 3], vx[n // 2, :, 5], kx[n - 1, :, 1] = np.nan, np.inf, 0.0
    kt, vt = gpu(kx, fmt), gpu(vx, fmt)
    gc = GpuCache(c)
    start = np.concatenate([[0], np.cumsum(new)])
    assert run_append(gc, kt, vt, start, old) == 0
    R.append(c, np64(kt), np64(vt), start, old)
    for got, ref, name in zip(gc.host(), (c.k, c.ks, c.v, c.vs), ("k", "k_scale", "v", "v_scale")):
        if name in ("k", "v"):  # a NaN keeps its sign bit free
            got, ref = (np.where((x & 0x7f) == 0x7f, 0x7f, x) for x in (got, ref))
        assert np.array_equal(got, ref), f"{name}: {np.argwhere(got != ref)[:5]}"


def test_append_extremes_of_the_scale():
    """Zeros take 2^-32, values beyond 448 2^31 saturate, exact borders do not move up."""
    D, bt = 64, 16
    c = make_cache(rng_for(3), [bt] * 5, 1, D, bt)
    x = np.zeros((5, bt, 1, D))
    x[1] = 1e-20
    x[2] = 3e12
    x[3, 2, 0, 9] = 448 * 2.0 ** 5
    x[4, 2, 0, 9] = np.nextafter(np.float32(448 * 2.0 ** 5), np.float32(1e9))
    kt = gpu(x.reshape(-1, 1, D), F32)
    gc = GpuCache(c)
    run_append(gc, kt, kt, np.arange(6) * bt, [0] * 5)
    R.append(c, np64(kt), np64(kt), np.arange(6) * bt, [0] * 5)
    k, ks, v, vs = gc.host()
    assert np.array_equal(k, c.k) and np.array_equal(ks, c.ks) and np.array_equal(v, c.v) and np.array_equal(vs, c.vs)
    assert [int(ks[c.table[s, 0], 0]) - 127 for s in range(5)] == [-32, -32, 31, 5, 6]


def test_append_token_by_token_and_strided():
    """Single tokens from slices of a fused projection, one call a token."""
    Hkv, D, bt, S, T = 2, 128, 16, 3, 20
    r = rng_for(4)
    c = make_cache(r, [T + 11, T, T + 5], Hkv, D, bt)
    gc = GpuCache(c)
    pos = np.array([11, 0, 5])
    row = Hkv * D
    for t in range(T):
        fused = gpu(r.standard_normal((S, 3 * row)) * 2.0 ** r.integers(-4, 5, (S, 1)), BF16)
        k, v = fused[:, row:2 * row], fused[:, 2 * row:]
        assert run_append(gc, k, v, np.arange(S + 1), pos, k_stride=3 * row, v_stride=3 * row) == 0
        R.append(c, np64(k).reshape(S, Hkv, D), np64(v).reshape(S, Hkv, D), np.arange(S + 1), pos)
        pos = pos + 1
    for got, ref in zip(gc.host(), (c.k, c.ks, c.v, c.vs)):
        assert np.array_equal(got, ref)


def test_append_skips_and_reports_bad_blocks():
    Hkv, D, bt = 1, 64, 16
    c = make_cache(rng_for(6), [40, 40], Hkv, D, bt)
    c.table[0, 1] = -1
    c.table[1, 2] = c.n_blocks
    kt = gpu(rng_for(7).standard_normal((2 * 64, Hkv, D)), BF16)
    gc = GpuCache(c)
    # the second sequence also runs past the table's columns
    assert run_append(gc, kt, kt, [0, 40, 104], [0, 0]) == lc.LC_DEV_BAD_BLOCK
    assert R.append(c, np64(kt), np64(kt), np.array([0, 40, 104]), [0, 0])
    for got, ref in zip(gc.host(), (c.k, c.ks, c.v, c.vs)):
        assert np.array_equal(got, ref)


# -------------------------------------------------------------------------------- attention
def attn_args(gc, q, start, pos0, kv, H, decode, W=0, scale=None, sink=None, q_stride=0, max_kv=None, max_q=None):
    n_q = q.shape[0]
    keep = [i32(start), i32(pos0), i32(kv), None if sink is None else torch.tensor(sink, dtype=torch.float32, device="cuda")]
    out = torch.full((n_q, H, gc.args.D), float("nan"), device="cuda", dtype=torch.bfloat16)
    lse = torch.full((n_q, H), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = lc.Kv8AttnArgs(cache=gc.args, H=H, num_seqs=len(kv), n_q=n_q,
                       max_q=max(int(np.max(np.diff(start))), 0) if max_q is None else max_q,
                       max_kv=int(np.max(kv)) if max_kv is None else max_kv, W=W, scale=scale if scale is not None else gc.args.D ** -0.5,
                       q=p(q), q_stride=q_stride, q_start=p(keep[0]), q_pos0=p(keep[1]), kv_len=p(keep[2]), sink=p(keep[3]),
                       out=p(out), lse=p(lse), status=p(status))
    ws = lc.lc_kv8_attn_workspace_bytes(a, decode)
    work = torch.full((max(ws, 16),), 0xff, dtype=torch.uint8, device="cuda")  # NaN: every word read was written
    a.workspace, a.workspace_bytes = p(work), ws
    return a, out, lse, status, keep + [work]


def run_attn(gc, q, start, pos0, kv, H, decode, **kw):
    a, out, lse, status, keep = attn_args(gc, q, start, pos0, kv, H, decode, **kw)
    (lc.lc_kv8_attn_decode if decode else lc.lc_kv8_attn_prefill)(a)
    torch.cuda.synchronize()
    return np64(out), np64(lse), int(status.item())


def check_attn(c, q64, start, pos0, kv, H, got_o, got_l, W=0, scale=None, sink=None, rows=None):
    scale = scale if scale is not None else c.D ** -0.5
    o, lse, bo, bl = R.attn(c, q64, start, pos0, kv, H, W, scale, sink)
    sel = slice(0, int(start[-1])) if rows is None else rows
    with np.errstate(invalid="ignore"):
        eo, el = np.abs(got_o - o)[sel], np.abs(got_l - lse)[sel]
    eo = np.where(np.isnan(got_o[sel]) & np.isnan(o[sel]), 0, eo)  # a NaN the query sees
    el = np.where((got_l[sel] == lse[sel]) | (np.isnan(got_l[sel]) & np.isnan(lse[sel])), 0, el)  # equal infinities
    bo, bl = np.where(np.isnan(o), 0, bo), np.where(np.isnan(lse), 0, bl)
    assert np.all(eo <= bo[sel]), f"o: worst error / bound {np.nanmax(eo / bo[sel])}, NaN {np.isnan(eo).sum()}"
    assert np.all(el <= bl[sel]), f"lse: worst error / bound {np.nanmax(el / bl[sel])}"


DECODE_LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 700, 1025]


@pytest.mark.parametrize("W", [0, 1, 100])
@pytest.mark.parametrize("Hkv,g,D,bt", [(1, 1, 128, 64), (2, 8, 128, 16), (1, 3, 64, 128), (3, 9, 64, 32), (1, 16, 128, 128),
                                        (1, 20, 128, 64), (2, 7, 64, 16), (1, 64, 64, 64)])
def test_attn_decode(Hkv, g, D, bt, W):
    r = rng_for(Hkv, g, D, bt, W)
    H, S = Hkv * g, len(DECODE_LENS)
    c = make_cache(r, DECODE_LENS, Hkv, D, bt)
    q = gpu(r.standard_normal((S, H, D)) * 2.0 ** r.integers(-8, 0, (S, H, 1)) * 2.0 ** -8, BF16)
    kv = np.array(DECODE_LENS)
    for sink in (None, r.standard_normal(H).astype(np.float32)):
        got = run_attn(GpuCache(c), q, np.arange(S + 1), np.maximum(kv - 1, 0), kv, H, True, W=W, sink=sink)
        assert got[2] == 0
        check_attn(c, np64(q), np.arange(S + 1), np.maximum(kv - 1, 0), kv, H, got[0], got[1], W=W, sink=sink)


@pytest.mark.parametrize("D,bt,g", [(128, 64, 8), (64, 16, 5)])
def test_attn_decode_long(D, bt, g):
    """Past 32768 keys the splits grow; scales wander over 60 octaves between blocks."""
    r = rng_for(D, bt, g)
    lens = [33000, 70001, 4]
    c = make_cache(r, lens, 1, D, bt, spread=3)
    c.vs[:] = 127 + r.integers(-30, 31, c.vs.shape)
    q = gpu(r.standard_normal((3, g, D)) * 0.02, BF16)
    kv = np.array(lens)
    got = run_attn(GpuCache(c), q, np.arange(4), kv - 1, kv, g, True)
    check_attn(c, np64(q), np.arange(4), kv - 1, kv, g, got[0], got[1])


PREFILL = [
    # (queries, cached) per sequence
    [(1, 1), (3, 3), (0, 40), (17, 200), (130, 130)],
    [(300, 300)],
    [(5, 700), (257, 513), (1, 16), (64, 64)],
]


@pytest.mark.parametrize("W", [0, 1, 77])
@pytest.mark.parametrize("case", range(len(PREFILL)))
@pytest.mark.parametrize("Hkv,g,D,bt", [(2, 1, 128, 64), (1, 8, 128, 16), (1, 3, 64, 128), (2, 5, 64, 32), (1, 16, 128, 32)])
def test_attn_prefill(Hkv, g, D, bt, case, W):
    r = rng_for(Hkv, g, D, bt, case, W)
    H = Hkv * g
    nq, kv = (np.array(x) for x in zip(*PREFILL[case]))
    c = make_cache(r, kv, Hkv, D, bt)
    start = np.concatenate([[0], np.cumsum(nq)])
    q = gpu(r.standard_normal((int(start[-1]) + 3, H, D)) * 2.0 ** -8, BF16)  # three rows behind the last sequence
    sink = r.standard_normal(H).astype(np.float32) if case else None
    got = run_attn(GpuCache(c), q, start, kv - nq, kv, H, False, W=W, sink=sink)
    assert got[2] == 0
    check_attn(c, np64(q), start, kv - nq, kv, H, got[0], got[1], W=W, sink=sink)
    assert np.isnan(got[0][start[-1]:]).all() and np.isnan(got[1][start[-1]:]).all()


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
def test_attn_nothing_visible_and_far_positions(decode):
    """Positions before the first token, past the cache, a window that has left the cache."""
    r = rng_for(12)
    D, bt, H = 64, 16, 4
    kv = np.array([40, 40, 0, 40])
    pos = np.array([-1, 1000, 3, 39])
    c = make_cache(r, kv, 2, D, bt)
    q = gpu(r.standard_normal((4, H, D)), BF16)
    for W in (0, 5):
        for sink in (None, np.float32([-2, 0, 1, 90])):
            got = run_attn(GpuCache(c), q, np.arange(5), pos, kv, H, decode, W=W, sink=sink)
            check_attn(c, np64(q), np.arange(5), pos, kv, H, got[0], got[1], W=W, sink=sink)


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
def test_attn_extreme_queries_and_sinks(decode):
    r = rng_for(13)
    D, bt, g, n = 128, 32, 8, 300
    c = make_cache(r, [n], 1, D, bt, spread=0)
    q = r.standard_normal((1, g, D))
    q[0, 0] = 0
    q[0, 1] *= 1e-36
    q[0, 2] *= 1e-3
    q[0, 3, 1:] = 0
    q[0, 4, 0] = 30.0
    q[0, 5] *= 0.1
    qt = gpu(q, BF16)
    sink = np.float32([0, -np.inf, 80, -80, 0, 1e4, -1e4, 3])
    got = run_attn(GpuCache(c), qt, [0, 1], [n - 1], [n], g, decode, sink=sink)
    check_attn(c, np64(qt), np.array([0, 1]), [n - 1], [n], g, got[0], got[1], sink=sink)


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
def test_attn_scales_far_apart(decode):
    """One block holds nearly all of the weight and tiny values, another huge values and next to no
    weight; scale bytes outside the range are read as its ends."""
    r = rng_for(14)
    D, bt, g, n = 64, 16, 2, 64
    c = make_cache(r, [n], 1, D, bt, spread=0)
    c.vs[c.table[0]] = np.array([[127 - 32], [127 + 31], [0], [255]], np.uint8)
    c.ks[c.table[0]] = np.array([[127], [119], [127], [100]], np.uint8)
    q = gpu(r.standard_normal((1, g, D)) * 0.05, BF16)
    got = run_attn(GpuCache(c), q, [0, 1], [n - 1], [n], g, decode)
    check_attn(c, np64(q), np.array([0, 1]), [n - 1], [n], g, got[0], got[1])


@pytest.mark.parametrize("where", ["k", "v"])
def test_attn_nan_reaches_only_who_sees_it(where):
    """A NaN at token 37 of a prefill: queries before it are as without it, those that see it are NaN."""
    r = rng_for(15)
    D, bt, g, n = 128, 16, 3, 120
    for W in (0, 20):
        c = make_cache(r, [n], 1, D, bt)
        q = gpu(r.standard_normal((n, g, D)) * 2.0 ** -8, BF16)
        bad = R.Cache(c.k.copy(), c.ks, c.v.copy(), c.vs, c.table)
        getattr(bad, where)[c.table[0, 37 // bt], 0, 37 % bt, 70] = 0x7f
        got = run_attn(GpuCache(bad), q, [0, n], [0], [n], g, False, W=W)
        sees = (np.arange(n) >= 37) & ((np.arange(n) < 37 + W) if W else True)
        check_attn(c, np64(q), np.array([0, n]), [0], [n], g, got[0], got[1], W=W, rows=np.where(~sees)[0])
        hit = got[0][sees]
        assert np.isnan(hit[..., 70] if where == "v" else hit).all()
        if where == "k":
            assert np.isnan(got[1][sees]).all()
        # decode at token 20 of the same cache: the NaN lies behind it
        got = run_attn(GpuCache(bad), q[:1], [0, 1], [20], [n], g, True, W=W)
        check_attn(c, np64(q[:1]), np.array([0, 1]), [20], [n], g, got[0], got[1], W=W)


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "prefill"])
def test_attn_bad_blocks_are_skipped_and_reported(decode):
    r = rng_for(16)
    D, bt, g, n = 128, 32, 8, 400
    c = make_cache(r, [n, n], 1, D, bt)
    c.table[0, 3], c.table[1, 0], c.table[1, 12] = -7, c.n_blocks, 2 ** 31 - 1
    q = gpu(r.standard_normal((2, g, D)) * 2.0 ** -8, BF16)
    got = run_attn(GpuCache(c), q, [0, 1, 2], [n - 1] * 2, [n] * 2, g, decode)
    assert got[2] == lc.LC_DEV_BAD_BLOCK
    check_attn(c, np64(q), np.array([0, 1, 2]), [n - 1] * 2, [n] * 2, g, got[0], got[1])
    # a length past the table's columns: read to its end, and reported
    got = run_attn(GpuCache(c), q, [0, 1, 2], [10 ** 6] * 2, [10 ** 6] * 2, g, decode)
    assert got[2] == lc.LC_DEV_BAD_BLOCK
    full = R.Cache(c.k, c.ks, c.v, c.vs, c.table)
    m = c.table.shape[1] * bt
    check_attn(full, np64(q), np.array([0, 1, 2]), [10 ** 6] * 2, [m] * 2, g, got[0], got[1])


def test_attn_strided_queries_and_max_kv():
    r = rng_for(17)
    D, bt, H, n = 64, 64, 6, 500
    c = make_cache(r, [n, n], 2, D, bt)
    fused = gpu(r.standard_normal((2, H * D + 256)) * 2.0 ** -8, BF16)
    q = fused[:, 128:128 + H * D]
    for decode in (True, False):
        got = run_attn(GpuCache(c), q.view(2, -1), [0, 1, 2], [n - 1] * 2, [n] * 2, H, decode, q_stride=H * D + 256, max_kv=300)
        check_attn(c, np64(q).reshape(2, H, D), np.array([0, 1, 2]), [n - 1] * 2, [300] * 2, H, got[0], got[1])


def test_attn_is_independent_of_the_batch():
    """A sequence's result is the same bits alone and in a batch, and from call to call."""
    r = rng_for(18)
    D, bt, H = 128, 64, 16
    kv = np.array([5000, 300, 20000, 64])
    c = make_cache(r, kv, 2, D, bt)
    gc = GpuCache(c)
    q = gpu(r.standard_normal((4, H, D)) * 2.0 ** -7, BF16)
    a = run_attn(gc, q, np.arange(5), kv - 1, kv, H, True)
    for _ in range(3):
        b = run_attn(gc, q, np.arange(5), kv - 1, kv, H, True)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    for s in range(4):
        one = R.Cache(c.k, c.ks, c.v, c.vs, c.table[s:s + 1])
        b = run_attn(GpuCache(one), q[s:s + 1], [0, 1], kv[s:s + 1] - 1, kv[s:s + 1], H, True)
        assert np.array_equal(a[0][s], b[0][0]) and np.array_equal(a[1][s], b[1][0])


@pytest.mark.parametrize("decode,nq", [(True, 1), (False, 2), (False, 40)])
def test_attn_window_of_the_types_last_value(decode, nq):
    """Wider than any context: the same answer as without a window, bit by bit."""
    r = rng_for(decode, nq, 99)
    kv = np.array([2600])
    c = make_cache(r, kv, 1, 64, 64)
    q = gpu(r.standard_normal((nq, 4, 64)) * 2.0 ** -8, BF16)
    want = run_attn(GpuCache(c), q, [0, nq], kv - nq, kv, 4, decode)
    check_attn(c, np64(q), np.array([0, nq]), kv - nq, kv, 4, want[0], want[1])
    for W in (2600, (1 << 31) - nq, (1 << 31) - 1):
        got = run_attn(GpuCache(c), q, [0, nq], kv - nq, kv, 4, decode, W=W)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0


@pytest.mark.parametrize("D,decode,nq", [(128, True, 1), (128, False, 3), (64, True, 1), (64, False, 3), (128, False, 50), (64, False, 50)])
def test_attn_cache_that_starts_16_bytes_in(D, decode, nq):
    """The cache's arrays need 16-byte alignment and no more: the same bits as from an allocation's start."""
    r = rng_for(D, decode, nq, 16)
    kv = np.array([1900])
    c = make_cache(r, kv, 2, D, 32)
    q = gpu(r.standard_normal((nq, 6, D)) * 2.0 ** -8, BF16)
    want = run_attn(GpuCache(c), q, [0, nq], kv - nq, kv, 6, decode)
    check_attn(c, np64(q), np.array([0, nq]), kv - nq, kv, 6, want[0], want[1])
    gc = GpuCache(c)
    moved = []
    for name, i in (("k", 0), ("v", 2)):
        x = gc.t[i].reshape(-1)
        y = torch.full((x.numel() + 32,), 0x7f, dtype=torch.uint8, device="cuda")
        y[16:-16] = x
        moved.append(y)
        setattr(gc.args, name, p(y) + 16)
    got = run_attn(gc, q, [0, nq], kv - nq, kv, 6, decode)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0


@pytest.mark.parametrize("nq", [1, 2, 24])
def test_attn_block_slots_past_2_31_bytes(nq):
    """Blocks whose codes lie past 2^31 and 2^32 bytes of the arrays."""
    r = rng_for(nq, 31)
    kv, H, D, bt = np.array([500]), 4, 128, 128
    c = make_cache(r, kv, 2, D, bt, spare=0)
    n_blocks = (1 << 32) // (2 * D * bt) + 40
    small = GpuCache(c)
    want_q = gpu(r.standard_normal((nq, H, D)) * 2.0 ** -8, BF16)
    want = run_attn(small, want_q, [0, nq], kv - nq, kv, H, nq == 1)
    far = np.array([n_blocks - 1, n_blocks // 2 + 3, 7, n_blocks - 33])  # of the sequence's four blocks
    gc = GpuCache(c)
    big = []
    for x, fill in zip(gc.t[:4], (0x7f, 127, 0x7f, 127)):
        y = torch.full((n_blocks, *x.shape[1:]), fill, dtype=torch.uint8, device="cuda")
        y[torch.from_numpy(far).cuda()] = x[gc.t[4][0].long()]
        big.append(y)
    table = i32(far[None])
    gc.args = lc.Kv8Cache(H_kv=2, D=D, bt=bt, n_blocks=n_blocks, table_cols=4, k=p(big[0]), v=p(big[2]), k_scale=p(big[1]),
                          v_scale=p(big[3]), table=p(table))
    got = run_attn(gc, want_q, [0, nq], kv - nq, kv, H, nq == 1)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0

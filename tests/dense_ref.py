"""The dense-layer operators in 64 bits (numpy on the CPU), straight from their definitions in
include/lc.h; shared by the CPU and the GPU tests.  Codecs come from the oracle."""
import numpy as np

from oracle import lc_oracle as O

E_MIN, E_MAX = -32, 31


def scale_exp(amax, lo, hi, zero):
    """The smallest e in lo..hi with amax <= 448 2^e; `zero` where amax is 0."""
    amax = np.asarray(amax, np.float64)
    m, x = np.frexp(amax)
    e = np.clip(np.where(m <= 0.875, x - 9, x - 8), lo, hi)
    return np.where(amax > 0, e, zero).astype(np.int64)


def finite_amax(x, axis):
    a = np.abs(x)
    return np.where(np.isfinite(a), a, 0.0).max(axis=axis)


def e4m3_codes(v):
    """Nearest E4M3 code, ties to even, saturating; NaN is 0x7F (with the sign bit free).  The sign
    stays where a value rounds to zero, as in any IEEE rounding (the oracle's codec drops it)."""
    nan = np.isnan(v)
    c = O.f64_to_e4m3(np.clip(np.where(nan, 0.0, np.abs(v)), 0.0, 448.0))
    return np.where(nan, 0x7F, c | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def e4m3_values(codes):
    return O.e4m3_to_f64(codes)


def add_rms_norm(x, res, w, eps):
    r = x + res if res is not None else x
    with np.errstate(all="ignore"):
        y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        return r, y * w if w is not None else y


def mxfp4_rows(codes, scales):
    """[.., K/2] codes, [.., K/32] scale bytes -> float64 [.., K]."""
    v = np.stack([O.e2m1_to_f64(codes & 15), O.e2m1_to_f64(codes >> 4)], -1).reshape(*codes.shape[:-1], -1)
    return v * np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, -1)


def mxfp8_rows(codes, scales):
    return e4m3_values(codes) * np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, -1)


class Cache:
    """A cache on the CPU: codes [n_blocks, H_kv, bt, D], scale bytes [n_blocks, H_kv], a table."""

    def __init__(self, k, ks, v, vs, table):
        self.k, self.ks, self.v, self.vs, self.table = k, ks, v, vs, table
        self.n_blocks, self.Hkv, self.bt, self.D = k.shape

    def rows(self, s, h, n):
        """Keys and values of tokens 0..n-1 and whether each lies in a valid block."""
        t = np.arange(n)
        blk = self.table[s, t // self.bt] if n else np.zeros(0, np.int64)
        ok = (blk >= 0) & (blk < self.n_blocks)
        b = np.where(ok, blk, 0)

        def get(c, sc):
            e = np.clip(sc[b, h].astype(np.int64) - 127, E_MIN, E_MAX)
            return e4m3_values(c[b, h, t % self.bt]) * np.exp2(e.astype(np.float64))[:, None]
        return get(self.k, self.ks), get(self.v, self.vs), ok


def append(cache, kx, vx, tok_start, pos0):
    """In place; returns whether a block was skipped."""
    bad = False
    bt = cache.bt
    for s in range(len(pos0)):
        p0, n = int(pos0[s]), int(tok_start[s + 1] - tok_start[s])
        if n <= 0:
            continue
        for col in range(p0 // bt, (p0 + n - 1) // bt + 1):
            blk = int(cache.table[s, col]) if col < cache.table.shape[1] else -1
            if not 0 <= blk < cache.n_blocks:
                bad = True
                continue
            lo, hi = max(p0, col * bt), min(p0 + n, (col + 1) * bt)
            r0, r1 = lo - col * bt, hi - col * bt
            src = slice(tok_start[s] + lo - p0, tok_start[s] + hi - p0)
            for x, codes, scales in ((kx, cache.k, cache.ks), (vx, cache.v, cache.vs)):
                new = x[src].transpose(1, 0, 2)  # [H_kv, rows, D]
                e = scale_exp(finite_amax(new, (1, 2)), E_MIN, E_MAX, E_MIN)
                if r0 > 0:
                    old = np.clip(scales[blk].astype(np.int64) - 127, E_MIN, E_MAX)
                    e = np.maximum(e, old)
                    again = e4m3_codes(e4m3_values(codes[blk, :, :r0]) * np.exp2((old - e).astype(float))[:, None, None])
                    grown = (e > old)[:, None, None]
                    codes[blk, :, :r0] = np.where(grown, again, codes[blk, :, :r0])
                with np.errstate(all="ignore"):
                    codes[blk, :, r0:r1] = e4m3_codes(new * np.exp2(-e.astype(float))[:, None, None])
                scales[blk] = (e + 127).astype(np.uint8)
    return bad


def attn(cache, q, q_start, q_pos0, kv_len, H, W, scale, sink):
    """(o, lse, bound_o, bound_lse): float64 results and the error that the arithmetic allows.

    Weights: rounded to F16 (2^-11 relative; absolute 2^-25 of the largest weight, of which at
    least one is >= 1/2, on a code of at most 448); logits: FP32 sums of D exact products and two
    FP32 factors ((D + 8) 2^-24 of the sum of magnitudes), 2^x within 2^-21 plus the rounding of
    its FP32 argument (2^-23 of its magnitude); sums over n keys in FP32.  A factor between
    references (a sink far above every logit) below 2^-126 is flushed to 0: it multiplies a sum of
    at most n weights of 2^8 on codes of 448, over Z >= 1/2."""
    n_q, _, D = q.shape
    g = H // cache.Hkv
    o = np.zeros((n_q, H, D))
    lse = np.full((n_q, H), -np.inf)
    bo, bl = np.zeros((n_q, H, D)), np.zeros((n_q, H))
    for s in range(len(kv_len)):
        n = min(int(kv_len[s]), cache.table.shape[1] * cache.bt)
        for h in range(cache.Hkv):
            k, v, ok = cache.rows(s, h, n)
            e = np.clip(cache.vs[np.where(ok, cache.table[s, np.arange(n) // cache.bt], 0), h].astype(int) - 127, E_MIN, E_MAX) if n else np.zeros(0)
            for i in range(q_start[s], q_start[s + 1]):
                p = int(q_pos0[s]) + i - int(q_start[s])
                t = np.arange(n)
                see = (t <= p) & ok
                if W:
                    see &= t > p - W
                kk, vv, ee = k[see], v[see], e[see]
                for hh in range(h * g, (h + 1) * g):
                    sk = sink[hh] if sink is not None else -np.inf
                    if not see.any():
                        lse[i, hh] = sk
                        continue
                    with np.errstate(all="ignore"):
                        lg = scale * (kk @ q[i, hh])
                        mag = abs(scale) * (np.abs(kk) @ np.abs(q[i, hh]))
                        M = max(lg.max(), sk)
                        w = np.exp(lg - M)
                        z = w.sum() + np.exp(sk - M)
                        pr = w / z
                        o[i, hh] = pr @ vv
                        lse[i, hh] = M + np.log(z)
                        d = (D + 8) * 2.0 ** -24 * mag.max() + 2.0 ** -21 + 2.0 ** -22 * (np.abs(lg).max() * 1.5 + 40) + len(lg) * 2.0 ** -24
                        pv = pr @ np.abs(vv)
                        under = len(lg) * 2.0 ** -24 * (pr * np.exp2(ee) * 448).max()
                        bo[i, hh] = 2.0 ** -8 * np.abs(o[i, hh]) + (2.0 ** -11 + 2 * d) * pv + under + 2.0 ** -133 + len(lg) * 448 * 2.0 ** (8 - 125)
                        bl[i, hh] = d + 2.0 ** -22 * (abs(lse[i, hh]) + 1)
    return o, lse, bo, bl

"""The dense layer's operators together, as a serving loop runs them: a prefill chunk, then decode steps
over the growing cache, each stage against 64 bits on the library's own previous stage; the step as a
CUDA graph, on side streams, with a shared prefix; arrays past 2^32 bytes."""
import numpy as np
import pytest
import torch

import long_context_sparse_softmax_b200 as lc
from tests import dense_ref as R
from tests.test_gpu_dense_layer import (BF16, F32, MXFP8, GpuCache, attn_args, check_attn, check_norm, gpu, i32, make_cache, make_w4, np64, p,
                                        rng_for, run_append, run_attn, run_w4, w4_reference)

pytestmark = pytest.mark.gpu


class Layer:
    """norm -> fused projection -> query / key preparation -> append -> attention -> grouped projection."""

    def __init__(self, seed, S, H, Hkv, D, bt, hidden, max_kv, W=0):
        self.S, self.H, self.Hkv, self.D, self.bt, self.hidden, self.max_kv, self.W = S, H, Hkv, D, bt, hidden, max_kv, W
        r = rng_for(seed)
        self.n_out = (H + 2 * Hkv) * D
        c1, s1 = make_w4(r, 1, self.n_out, hidden)
        c2, s2 = make_w4(r, Hkv, hidden // Hkv, H // Hkv * D)
        self.host = (c1, s1 - 3, c2, s2 - 3)  # outputs of moderate size
        self.w = [torch.from_numpy(x).cuda() for x in self.host]
        self.nw = gpu(1 + 0.2 * r.standard_normal(hidden), BF16)
        self.sink = gpu(r.standard_normal(H), F32)
        self.cache = make_cache(r, [max_kv] * S, Hkv, D, bt)
        self.gc = GpuCache(self.cache)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self, n, max_q, decode):
        """Everything a step of n rows writes, and its argument structs."""
        b = dict(n=n, decode=decode)
        H, Hkv, D, hid = self.H, self.Hkv, self.D, self.hidden

        def empty(*s, dtype=torch.bfloat16):
            return torch.empty(*s, device="cuda", dtype=dtype)
        b["x"], b["res"] = empty(n, hid), empty(n, hid)
        b["codes"], b["scales"] = empty(n, hid, dtype=torch.uint8), empty(n, hid // 32, dtype=torch.uint8)
        b["qkv"] = empty(n, self.n_out)
        b["q"], b["k"] = empty(n, H, D), empty(n, Hkv, D)
        b["q2"], b["k2"] = empty(n, H, D), empty(n, Hkv, D)
        b["pos"], b["start"], b["pos0"], b["kv"] = i32(np.zeros(n)), i32(np.zeros(self.S + 1)), i32(np.zeros(self.S)), i32(np.zeros(self.S))
        b["o"], b["lse"] = empty(n, H, D), empty(n, H, dtype=torch.float32)
        b["y"] = empty(n, hid)
        b["norm"] = lc.AddRmsNormArgs(n_rows=n, d=hid, in_fmt=BF16, x=p(b["x"]), res=p(b["res"]), res_out=p(b["res"]), w=p(self.nw), w_fmt=BF16,
                                      out_fmt=MXFP8, y=p(b["codes"]), y_scale=p(b["scales"]), eps=1e-6, status=p(self.status))
        b["qkv_proj"] = lc.W4ProjArgs(n_q=n, G=1, K=hid, d_g=self.n_out, in_fmt=MXFP8, out_fmt=BF16, x=p(b["codes"]), x_scale=p(b["scales"]),
                                      w=p(self.w[0]), w_scale=p(self.w[1]), y=p(b["qkv"]), status=p(self.status))
        b["prep"] = [lc.QkPrepArgs(dims=lc.Dims(D, 64, 0, h), n_tok=n, in_fmt=BF16, x=p(b[i]), pos=p(b["pos"]), out=lc.Rows(BF16, 0, p(b[o]), None),
                                   rope_base=10000.0, eps=1e-6) for i, o, h in (("q", "q2", H), ("k", "k2", Hkv))]
        v = b["qkv"][:, (H + Hkv) * D:]
        b["append"] = lc.Kv8AppendArgs(cache=self.gc.args, num_seqs=self.S, in_fmt=BF16, max_tok=max_q, k=p(b["k2"]), v=p(v), v_stride=self.n_out,
                                       tok_start=p(b["start"]), pos0=p(b["pos0"]), status=p(self.status))
        a = lc.Kv8AttnArgs(cache=self.gc.args, H=H, num_seqs=self.S, n_q=n, max_q=max_q, max_kv=self.max_kv, W=self.W, scale=D ** -0.5,
                           q=p(b["q2"]), q_start=p(b["start"]), q_pos0=p(b["pos0"]), kv_len=p(b["kv"]), sink=p(self.sink), out=p(b["o"]),
                           lse=p(b["lse"]), status=p(self.status))
        ws = lc.lc_kv8_attn_workspace_bytes(a, decode)
        b["ws"] = torch.full((max(ws, 16),), 0xff, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = p(b["ws"]), ws
        b["attn"] = a
        b["out_proj"] = lc.W4ProjArgs(n_q=n, G=Hkv, K=H // Hkv * D, d_g=hid // Hkv, in_fmt=BF16, out_fmt=BF16, x=p(b["o"]), w=p(self.w[2]),
                                      w_scale=p(self.w[3]), y=p(b["y"]), status=p(self.status))
        return b

    def fill(self, b, x, res, new, pos0):
        pos = np.concatenate([np.arange(q, q + n) for q, n in zip(pos0, new)])
        for k, v in (("pos", pos), ("start", np.concatenate([[0], np.cumsum(new)])), ("pos0", pos0), ("kv", np.asarray(pos0) + new)):
            b[k].copy_(torch.from_numpy(np.asarray(v, np.int32)))
        b["x"].copy_(x)
        b["res"].copy_(res)

    def run(self, b):
        H, Hkv, D = self.H, self.Hkv, self.D
        lc.lc_add_rms_norm(b["norm"])
        lc.lc_w4_proj(b["qkv_proj"])
        b["q"].copy_(b["qkv"][:, :H * D].view(-1, H, D))
        b["k"].copy_(b["qkv"][:, H * D:(H + Hkv) * D].view(-1, Hkv, D))
        for a in b["prep"]:
            (lc.lc_qk_prep_decode if b["decode"] else lc.lc_qk_prep_prefill)(a)
        lc.lc_kv8_append(b["append"])
        (lc.lc_kv8_attn_decode if b["decode"] else lc.lc_kv8_attn_prefill)(b["attn"])
        lc.lc_w4_proj(b["out_proj"])

    def check(self, b, x, res, new, pos0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        H, Hkv, D = self.H, self.Hkv, self.D
        check_norm(np64(x), np64(res), np64(self.nw), MXFP8, b["codes"], b["scales"])
        s = np64(x) + np64(res)
        assert np.all(np.abs(np64(b["res"]) - s) <= 2.0 ** -8 * np.abs(s))
        hn = R.mxfp8_rows(b["codes"].cpu().numpy(), b["scales"].cpu().numpy())
        self.check_w4(hn, 0, 1, self.hidden, self.n_out, b["qkv"], False)
        start = np.concatenate([[0], np.cumsum(new)])
        v = np64(b["qkv"])[:, (H + Hkv) * D:].reshape(-1, Hkv, D)
        R.append(self.cache, np64(b["k2"]), v, start, pos0)
        for got, ref in zip(self.gc.host(), (self.cache.k, self.cache.ks, self.cache.v, self.cache.vs)):
            assert np.array_equal(got, ref)
        check_attn(self.cache, np64(b["q2"]), start, pos0, np.asarray(pos0) + new, H, np64(b["o"]), np64(b["lse"]), W=self.W, sink=np64(self.sink))
        self.check_w4(np64(b["o"]).reshape(b["n"], -1), 2, Hkv, H // Hkv * D, self.hidden // Hkv, b["y"], True)

    def check_w4(self, x64, at, G, K, dg, y, bf16):
        ref, mag, top = w4_reference(x64, self.host[at], self.host[at + 1], G, K, dg)
        tol = K * 2.0 ** -24 * mag + (2.0 ** -21 * top if bf16 else 0) + 2.0 ** -8 * np.abs(ref) + 1e-30
        assert np.all(np.abs(np64(y) - ref) <= tol)


@pytest.mark.parametrize("H,Hkv,D,bt,W", [(8, 2, 128, 32, 0), (12, 4, 64, 16, 50)])
def test_prefill_then_decode_steps(H, Hkv, D, bt, W):
    r = rng_for(H, D)
    S, hidden = 3, 256 * Hkv // 2
    layer = Layer(71, S, H, Hkv, D, bt, hidden, 256, W)
    new, pos0 = np.array([40, 1, 150]), np.array([0, 0, 0])
    for step in range(4):
        n = int(new.sum())
        b = layer.buffers(n, int(new.max()), step > 0)
        x, res = gpu(r.standard_normal((n, hidden)), BF16), gpu(2 * r.standard_normal((n, hidden)), BF16)
        layer.fill(b, x, res, new, pos0)
        layer.run(b)
        layer.check(b, x, res, new, pos0)
        pos0, new = pos0 + new, np.ones(S, int)


def test_decode_step_as_a_graph():
    """Captured once and replayed while the positions, lengths and inputs in its buffers change; two
    graphs over one workspace, replayed in turn; an eager step between them."""
    S, H, Hkv, D, hidden = 4, 16, 2, 128, 256
    r = rng_for(5)
    a, e = (Layer(72, S, H, Hkv, D, 64, hidden, 900) for _ in range(2))
    ba, be = a.buffers(S, 1, True), e.buffers(S, 1, True)
    pos0 = np.array([3, 64, 500, 895])
    x, res = gpu(r.standard_normal((S, hidden)), BF16), gpu(r.standard_normal((S, hidden)), BF16)
    a.fill(ba, x, res, np.ones(S, int), np.zeros(S, int))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a.run(ba)
        graphs.append(g)
    a.gc.t[0].copy_(e.gc.t[0]), a.gc.t[1].copy_(e.gc.t[1]), a.gc.t[2].copy_(e.gc.t[2]), a.gc.t[3].copy_(e.gc.t[3])
    for step in range(4):
        x, res = gpu(r.standard_normal((S, hidden)), BF16), gpu(r.standard_normal((S, hidden)), BF16)
        a.fill(ba, x, res, np.ones(S, int), pos0)
        e.fill(be, x, res, np.ones(S, int), pos0)
        graphs[step % 2].replay()
        e.run(be)
        torch.cuda.synchronize()
        for k in ("codes", "scales", "res", "qkv", "o", "lse", "y"):
            assert torch.equal(ba[k].view(torch.uint8), be[k].view(torch.uint8)), (step, k)
        for t, u in zip(a.gc.t, e.gc.t):
            assert torch.equal(t, u)
        pos0 = pos0 + 1
    assert int(a.status.item()) == 0


def test_two_streams_at_once():
    """Calls that overlap in time, each with its own outputs and workspace, give what they give alone."""
    r = rng_for(6)
    H, Hkv, D, bt = 16, 2, 128, 64
    kv = np.array([9000, 20000])
    c = make_cache(r, kv, Hkv, D, bt)
    gc = GpuCache(c)
    q = gpu(r.standard_normal((2, H, D)) * 0.05, BF16)
    nq = np.array([300, 64])
    qp = gpu(r.standard_normal((int(nq.sum()), H, D)) * 0.05, BF16)
    calls = []
    for _ in range(3):
        calls.append((lc.lc_kv8_attn_decode, attn_args(gc, q, np.arange(3), kv - 1, kv, H, True)))
        calls.append((lc.lc_kv8_attn_prefill, attn_args(gc, qp, np.concatenate([[0], np.cumsum(nq)]), kv - nq, kv, H, False)))
    codes, scales = make_w4(r, 2, 500, 1024)
    ct, st = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    x = gpu(r.standard_normal((9, 2048)), BF16)
    ys = [torch.empty(9, 1000, device="cuda") for _ in range(3)]
    for y in ys:
        calls.append((lc.lc_w4_proj, (lc.W4ProjArgs(n_q=9, G=2, K=1024, d_g=500, in_fmt=BF16, out_fmt=F32, x=p(x), w=p(ct), w_scale=p(st), y=p(y)), y, y)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for s, (f, a) in zip(streams, calls):
            f(a[0], s)
    torch.cuda.synchronize()
    for kind in (lc.lc_kv8_attn_decode, lc.lc_kv8_attn_prefill, lc.lc_w4_proj):
        same = [a for f, a in calls if f is kind]
        for a in same[1:]:
            assert torch.equal(a[1].view(torch.uint8), same[0][1].view(torch.uint8)) and torch.equal(a[2], same[0][2])
    start = np.concatenate([[0], np.cumsum(nq)])
    a = calls[1][1]
    check_attn(c, np64(qp), start, kv - nq, kv, H, np64(a[1]), np64(a[2]))


def test_shared_prefix():
    """Two sequences whose tables name the same blocks."""
    r = rng_for(7)
    c = make_cache(r, [640, 640, 700], 2, 64, 32)
    c.table[1, :20] = c.table[0, :20]
    c.table[2, 3:6] = c.table[0, 7]  # and one block three times
    q = gpu(r.standard_normal((3, 8, 64)) * 0.1, BF16)
    kv = np.array([640, 640, 700])
    for decode in (True, False):
        got = run_attn(GpuCache(c), q, np.arange(4), kv - 1, kv, 8, decode)
        check_attn(c, np64(q), np.arange(4), kv - 1, kv, 8, got[0], got[1])


def test_cache_past_32_bits():
    """Blocks whose bytes lie past 2^32 of the arrays: written, read by decode and by both prefill kernels."""
    Hkv, D, bt, H = 8, 128, 128, 16
    n_blocks = 2 ** 32 // (Hkv * bt * D) + 40
    kv = np.array([700, 300])
    small = make_cache(rng_for(8), kv, Hkv, D, bt)
    k, v = (torch.empty(n_blocks, Hkv, bt, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_blocks, Hkv, dtype=torch.uint8, device="cuda") for _ in range(2))
    shift = n_blocks - small.n_blocks
    for big, part in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        big[shift:] = torch.from_numpy(part).cuda()
    table = np.where(small.table >= 0, small.table + shift, -1).astype(np.int32)
    tt = torch.from_numpy(table).cuda()
    gc = GpuCache(small)
    gc.args = lc.Kv8Cache(H_kv=Hkv, D=D, bt=bt, n_blocks=n_blocks, table_cols=table.shape[1], k=p(k), v=p(v), k_scale=p(ks), v_scale=p(vs), table=p(tt))
    r = rng_for(9)
    new, pos0 = np.array([130, 5]), np.array([560, 290])
    kx, vx = (gpu(r.standard_normal((135, Hkv, D)), BF16) for _ in range(2))
    start = np.array([0, 130, 135])
    assert run_append(gc, kx, vx, start, pos0) == 0
    R.append(small, np64(kx), np64(vx), start, pos0)
    for big, part in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        assert np.array_equal(big[shift:].cpu().numpy(), part)
    kv = pos0 + new
    for nq in ([1, 1], [3, 2], [100, 60]):
        nq = np.array(nq)
        st = np.concatenate([[0], np.cumsum(nq)])
        q = gpu(r.standard_normal((int(nq.sum()), H, D)) * 0.1, BF16)
        for decode in ([True, False] if nq.max() == 1 else [False]):
            got = run_attn(gc, q, st, kv - nq, kv, H, decode)
            assert got[2] == 0
            check_attn(small, np64(q), st, kv - nq, kv, H, got[0], got[1])


def test_rows_past_32_bits():
    """The norm's last rows of 2^31 values and more; weights past 2^32 bytes."""
    d, rows = 8192, 2 ** 31 // 8192 + 5
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    last = gpu(rng_for(10).standard_normal((3, d)), BF16)
    x[-3:] = last
    y = torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    ys = torch.empty(rows, d // 32, dtype=torch.uint8, device="cuda")
    ro = torch.empty_like(x)
    lc.lc_add_rms_norm(lc.AddRmsNormArgs(n_rows=rows, d=d, in_fmt=BF16, x=p(x), res_out=p(ro), out_fmt=MXFP8, y=p(y), y_scale=p(ys), eps=1e-6))
    torch.cuda.synchronize()
    check_norm(np64(last), None, None, MXFP8, y[-3:], ys[-3:])
    assert torch.equal(ro[-3:], last) and not y[:-3].any()
    del x, y, ys, ro
    K, dg, n = 4096, 2 ** 21 + 70, 2
    w = torch.zeros(1, dg, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.full((1, dg, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes, scales = make_w4(rng_for(11), 1, 100, K)
    w[:, -100:], ws[:, -100:] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    xt = gpu(rng_for(12).standard_normal((n, K)), BF16)
    out = torch.empty(n, dg, device="cuda")
    lc.lc_w4_proj(lc.W4ProjArgs(n_q=n, G=1, K=K, d_g=dg, in_fmt=BF16, out_fmt=F32, x=p(xt), w=p(w), w_scale=p(ws), y=p(out)))
    torch.cuda.synchronize()
    ref, mag, top = w4_reference(np64(xt), codes, scales, 1, K, 100)
    got = np64(out[:, -100:])
    assert np.all(np.abs(got - ref) <= K * 2.0 ** -24 * mag + 2.0 ** -21 * top + 2.0 ** -24 * np.abs(ref))
    assert not out[:, :-100].any()


def test_empty_and_single():
    """Sequences without tokens or queries among others; one token in all."""
    r = rng_for(13)
    c = make_cache(r, [0, 1, 200, 0], 1, 128, 16, cols=14)
    gc = GpuCache(c)
    q = gpu(r.standard_normal((75, 5, 128)) * 0.1, BF16)
    nq, kv = np.array([0, 1, 70, 0]), np.array([0, 1, 200, 0])
    st = np.concatenate([[0], np.cumsum(nq)])
    got = run_attn(gc, q, st, kv - nq, kv, 5, False)
    assert got[2] == 0
    check_attn(c, np64(q), st, kv - nq, kv, 5, got[0], got[1])
    assert np.isnan(got[0][71:]).all()
    one = make_cache(r, [1], 1, 64, 16)
    q1 = gpu(r.standard_normal((1, 1, 64)), BF16)
    for decode in (True, False):
        got = run_attn(GpuCache(one), q1, [0, 1], [0], [1], 1, decode)
        check_attn(one, np64(q1), np.array([0, 1]), [0], [1], 1, got[0], got[1])
    codes, scales = make_w4(r, 1, 1, 32)
    assert run_w4(gpu(r.standard_normal((1, 32)), BF16), None, codes, scales, 1, 32, 1, F32).shape == (1, 1)


@pytest.mark.parametrize("g,D,nq,kv,W", [(1, 64, 2, 6000, 0), (8, 128, 9, 5000, 0), (8, 128, 20, 9000, 0), (4, 64, 33, 3000, 1000), (2, 128, 500, 2500, 200)])
def test_prefill_with_few_rows_splits_the_keys(g, D, nq, kv, W):
    """A short chunk on a long cache: the keys are split, by either kernel."""
    r = rng_for(g, nq)
    c = make_cache(r, [kv, kv // 3], 1, D, 64)
    n = np.array([nq, 1])
    st = np.array([0, nq, nq + 1])
    lens = np.array([kv, kv // 3])
    q = gpu(r.standard_normal((nq + 1, g, D)) * 0.05, BF16)
    sink = r.standard_normal(g).astype(np.float32)
    got = run_attn(GpuCache(c), q, st, lens - n, lens, g, False, W=W, sink=sink)
    assert got[2] == 0
    check_attn(c, np64(q), st, lens - n, lens, g, got[0], got[1], W=W, sink=sink)


def test_calls_between_other_kernels_without_waiting():
    """The kernels start before the one in front of them ends: chains with torch's kernels in front, between
    and behind, sent without a pause, give what the same chain gives with a pause after every call."""
    r = rng_for(14)
    n, d, dg = 9, 512, 384
    codes, scales = make_w4(r, 1, dg, d)
    ct, st = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    S, H, Hkv, D, bt = n, 6, 3, 64, 16
    start = np.arange(S + 1)

    def chain(pause):
        gen = torch.Generator(device="cuda").manual_seed(5)
        c = make_cache(rng_for(15), [600] * S, Hkv, D, bt)
        gc = GpuCache(c)
        x, y8, ys = (torch.empty(n, d, device="cuda"), torch.empty(n, d, dtype=torch.uint8, device="cuda"),
                     torch.empty(n, d // 32, dtype=torch.uint8, device="cuda"))
        y = torch.empty(n, dg, device="cuda", dtype=torch.bfloat16)
        kv, pos = i32(np.full(S, 301)), i32(np.full(S, 300))
        q0 = gpu(np.zeros((S, H, D)), BF16)
        a, out, lse, status, keep = attn_args(gc, q0, start, np.full(S, 300), np.full(S, 301), H, True, max_kv=600)
        a.q, a.q_pos0, a.kv_len = p(y), p(pos), p(kv)
        ap = lc.Kv8AppendArgs(cache=gc.args, num_seqs=S, in_fmt=BF16, max_tok=1, k=p(y), v=p(y), k_stride=dg, v_stride=dg, tok_start=p(keep[0]), pos0=p(pos))
        got = []
        for _ in range(40):
            for f in (lambda: x.normal_(generator=gen),
                      lambda: lc.lc_add_rms_norm(lc.AddRmsNormArgs(n_rows=n, d=d, in_fmt=F32, x=p(x), out_fmt=MXFP8, y=p(y8), y_scale=p(ys), eps=1e-6)),
                      lambda: lc.lc_w4_proj(lc.W4ProjArgs(n_q=n, G=1, K=d, d_g=dg, in_fmt=MXFP8, out_fmt=BF16, x=p(y8), x_scale=p(ys), w=p(ct), w_scale=p(st), y=p(y))),
                      lambda: y.mul_(0.125),
                      lambda: lc.lc_kv8_append(ap),
                      lambda: lc.lc_kv8_attn_decode(a),
                      lambda: pos.add_(1), lambda: kv.add_(1),
                      lambda: got.append((out.clone(), lse.clone(), y8.clone()))):
                f()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got, [t.clone() for t in gc.t]
    (a, ca), (b, cb) = chain(False), chain(True)
    for u, v in zip(a, b):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(u, v))
    assert all(torch.equal(s, t) for s, t in zip(ca, cb))

"""Cases of the operators around a dense attention layer served from an 8-bit cache.

A decode or prefill step of such a layer runs, in this order: the residual's addition with
the root-mean-square norm (output in 8 bits with scales), projections with 4-bit weights,
the append of the new keys and values to the 8-bit cache, and the attention over that cache.

  norm    lc_add_rms_norm: r = x + res, y = r / sqrt(mean(r^2) + eps) * w; y in BF16, FP32 or
          MXFP8 (E4M3 codes, one E8M0 scale per 32 values: the smallest power of two X with
          max |y| <= 448 X).
  w4      lc_w4_proj: y[n, g d_g + c] = sum_k x[n, g K + k] W_g[c, k], W in MXFP4 (E2M1 codes,
          element 2i in the low nibble of byte i, one E8M0 scale per 32), x in BF16 or MXFP8.
  append  lc_kv8_append: new key and value rows into blocks of bt tokens; each (block, head)
          holds E4M3 codes and one E8M0 scale, the smallest power of two in 2^-32 .. 2^31 that
          covers its tokens; a block that already holds tokens keeps its scale unless the new
          ones need a larger one, and then its codes are rounded again to the larger scale.
  attn    lc_kv8_attn_{decode,prefill}: softmax attention of H query heads over that cache
          (H / H_kv heads share one), causal, optionally with a window and a sink logit.

Sizes: hidden sizes, head counts, sequence lengths and batches of this library's workloads
(7168 / 4096 hidden, 64 and 128 heads, batches of 32 and 8, contexts up to 2^18 here), grouped
heads with 8 shared heads of 128 dims, and generic odd ones.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
E_MIN, E_MAX = -32, 31  # scale exponents of the cache
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's norm before an MXFP4 projection: 32 rows of a 7168-wide model
        dict(name="norm_decode", op="norm", rows=32, d=7168, x="bf16", res=True, y="mxfp8"),
        # a prefill chunk's norm, the same model
        dict(name="norm_prefill", op="norm", rows=16384, d=7168, x="bf16", res=True, y="mxfp8"),
        # odd row count, FP32 stream, BF16 output: the norm in front of a BF16 product
        dict(name="norm_ragged", op="norm", rows=1003, d=4096, x="f32", res=True, y="bf16"),
        # one token through a hidden-to-hidden projection: the latency case
        dict(name="w4_token", op="w4", n=1, G=1, K=7168, dg=4096, x="bf16"),
        # a decode batch through the grouped output projection of 64 heads (8 groups)
        dict(name="w4_grouped", op="w4", n=32, G=8, K=4096, dg=1024, x="bf16"),
        # an odd batch from the norm's MXFP8 output, ragged output width
        dict(name="w4_mxfp8", op="w4", n=17, G=1, K=7168, dg=7000, x="mxfp8"),
        # a decode batch appends one token to each sequence
        dict(name="append_decode", op="append", S=32, new=1, old=5000, Hkv=8, D=128, bt=64, x="bf16"),
        # a prefill chunk appends 16384 tokens behind an unfinished block
        dict(name="append_prefill", op="append", S=1, new=16384, old=1037, Hkv=8, D=128, bt=64, x="bf16"),
        # a decode batch, ragged contexts up to 16384
        dict(name="attn_decode", op="attn", S=32, q=1, kv=16384, H=64, Hkv=8, D=128, bt=64, W=0, sink=False),
        # one long context alone: the keys have to be split to fill the device
        dict(name="attn_long", op="attn", S=1, q=1, kv=262144, H=64, Hkv=8, D=128, bt=128, W=0, sink=True),
        # a prefill chunk of 2048 queries at the end of an 8192-token cache
        dict(name="attn_prefill", op="attn", S=1, q=2048, kv=8192, H=64, Hkv=8, D=128, bt=64, W=0, sink=False),
        # ragged prefill of several sequences, odd head group, 64 dims, a window and small blocks
        dict(name="attn_ragged", op="attn", S=5, q=777, kv=2500, H=28, Hkv=4, D=64, bt=16, W=1024, sink=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "w4", "append", "attn"])
    if op == "norm":
        d = 32 * _log(rng, 8, 256)
        rows = min(_log(rng, 1, 32768), 16384 * 7168 // d)
        return dict(op=op, rows=rows, d=d, x=rng.choice(["bf16", "f32"]), res=rng.random() < 0.8,
                    y=rng.choice(["mxfp8", "bf16", "f32"]))
    if op == "w4":
        G = rng.choice([1, 1, 2, 4, 8])
        K = 32 * _log(rng, 8, 320)
        dg = _log(rng, 16, 8192)
        while G * K * dg > 8 * 4096 * 1024 * 2:
            dg = dg // 2 + 1
        return dict(op=op, n=_log(rng, 1, 64), G=G, K=K, dg=dg, x=rng.choice(["bf16", "mxfp8"]))
    if op == "append":
        S = _log(rng, 1, 64)
        return dict(op=op, S=S, new=min(_log(rng, 1, 16384), max(1, 16384 // S)), old=_log(rng, 1, 8192) - 1,
                    Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), bt=rng.choice([16, 32, 64, 128]),
                    x=rng.choice(["bf16", "f32"]))
    Hkv, D, g = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    c = dict(op=op, H=Hkv * g, Hkv=Hkv, D=D, bt=rng.choice([16, 32, 64, 128]), W=rng.choice([0, 0, 128, 1000, 4096]),
             sink=rng.random() < 0.5)
    if rng.random() < 0.5:  # decode
        S = _log(rng, 1, 64)
        return dict(c, S=S, q=1, kv=min(_log(rng, 1, 131072), max(1, 32 * 16384 // S)))
    S = _log(rng, 1, 8)
    kv = _log(rng, 16, 8192)
    return dict(c, S=S, q=max(2, min(_log(rng, 2, 2048), kv, 2048 * 64 * 8192 // (S * kv * c["H"]))), kv=kv)


# ------------------------------------------------------------------- formats, as plain torch
def _scale_exp(amax, lo, hi, zero):
    """The smallest e in lo..hi with amax <= 448 2^e (zero where amax is 0)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(lo, hi)
    return torch.where(amax > 0, e, torch.full_like(e, zero))


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _finite_amax(x, dim):
    a = x.abs()
    return torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(dim)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _mxfp8(y):
    """FP32 rows -> (E4M3 codes, E8M0 scales per 32)."""
    b = y.unflatten(-1, (-1, 32))
    e = _scale_exp(_finite_amax(b, -1), -127, 127, 0)
    # two exact factors: 2^-e alone can leave the range of FP32
    codes = _e4m3(torch.ldexp(torch.ldexp(b, -(e // 2).unsqueeze(-1)), -(e - e // 2).unsqueeze(-1)))
    return codes.flatten(-2), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _dequant_w4(codes, scale, dtype=torch.float32):
    lut = torch.tensor(E2M1, device=codes.device, dtype=dtype)
    w = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    s = torch.ldexp(torch.ones((), device=codes.device, dtype=dtype), scale.to(torch.int32) - 127)
    return (w.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _dequant_x8(codes, scale, dtype=torch.float32):
    s = torch.ldexp(torch.ones((), device=codes.device, dtype=dtype), scale.view(torch.uint8).to(torch.int32) - 127)
    return (codes.to(dtype).unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- inputs
def _cache(gen, n_blocks, Hkv, bt, D):
    """A filled cache: heads and dims of different size, an outlier dim in each key head."""
    out = []
    for outlier in (True, False):
        mul = torch.exp(torch.randn(Hkv, 1, D, device="cuda", generator=gen) * 0.5)
        if outlier:
            mul[:, 0, D // 3] *= 8
        codes = torch.empty(n_blocks, Hkv, bt, D, device="cuda", dtype=torch.float8_e4m3fn)
        exps = torch.empty(n_blocks, Hkv, device="cuda", dtype=torch.int32)
        for b in range(0, n_blocks, 4096):  # in pieces: the FP32 rows are four times the codes
            x = torch.randn(min(4096, n_blocks - b), Hkv, bt, D, device="cuda", generator=gen) * mul
            e = _scale_exp(x.abs().amax((2, 3)), E_MIN, E_MAX, E_MIN)
            codes[b:b + 4096] = _e4m3(x * _pow2(-e)[:, :, None, None])
            exps[b:b + 4096] = e
        out += [codes.view(torch.uint8), (exps + 127).to(torch.uint8)]
    return dict(k=out[0], ks=out[1], v=out[2], vs=out[3])


def _lengths(S, top, low):
    """Ragged lengths, the same for every seed (the outputs' shapes follow from them): the
    longest is `top`, the others spread below it."""
    fixed = torch.Generator().manual_seed(S * 1000003 + top)
    n = torch.randint(min(low, top), top + 1, (S,), generator=fixed)
    n[int(torch.randint(0, S, (1,), generator=fixed))] = top
    return n.to(torch.int32)


def _table(cpu, lengths, bt):
    """Blocks of every sequence at shuffled places of a pool with a few spare ones."""
    nb = (lengths.long() + bt - 1) // bt
    n_blocks = int(nb.sum()) + 3
    perm = torch.randperm(n_blocks, generator=cpu)
    cols = max(1, int(nb.max()))
    table = torch.zeros(len(lengths), cols, dtype=torch.int32)
    mask = torch.arange(cols)[None, :] < nb[:, None]
    table[mask] = perm[:int(nb.sum())].to(torch.int32)
    return table, n_blocks


def prepare(case, seed):
    c, op = case, case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    st = dict(c=c)
    if op == "norm":
        st["x"] = (randn(c["rows"], c["d"]) * 0.5).to(DT[c["x"]])
        st["res"] = (randn(c["rows"], c["d"]) * 4).to(DT[c["x"]]) if c["res"] else None
        st["w"] = (1 + 0.2 * randn(c["d"])).to(torch.bfloat16)
    elif op == "w4":
        n, G, K, dg = c["n"], c["G"], c["K"], c["dg"]
        st["w"] = torch.randint(0, 256, (G, dg, K // 2), device="cuda", generator=gen, dtype=torch.uint8)
        e = torch.randint(-2, 3, (G, dg, K // 32), device="cuda", generator=gen) - int(round(math.log2(3 * K ** 0.5)))
        st["ws"] = (e + 127).to(torch.uint8)
        x = randn(n, G * K) * torch.exp(randn(1, G * K))
        if c["x"] == "bf16":
            st["x"], st["xs"] = x.to(torch.bfloat16), None
        else:
            st["x"], st["xs"] = _mxfp8(x)
    elif op == "append":
        S, Hkv, D, bt = c["S"], c["Hkv"], c["D"], c["bt"]
        new = _lengths(S, c["new"], 1)
        old = _lengths(S, c["old"], 0)
        table, n_blocks = _table(cpu, old + new, bt)
        st.update(_cache(gen, n_blocks, Hkv, bt, D))
        n = int(new.sum())
        mul = torch.exp(0.5 * randn(n, Hkv, 1))  # tokens of different size: some blocks need a larger scale
        st["kx"], st["vx"] = ((randn(n, Hkv, D) * mul).to(DT[c["x"]]) for _ in range(2))
        st["start"] = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).to(torch.int32)]).cuda()
        st["pos0"], st["table"], st["max_new"] = old.cuda(), table.cuda(), int(new.max())
    else:
        S, H, Hkv, D, bt = c["S"], c["H"], c["Hkv"], c["D"], c["bt"]
        kv = _lengths(S, c["kv"], 1 if c["q"] == 1 else max(1, c["kv"] // 4))
        nq = torch.ones(S, dtype=torch.int32) if c["q"] == 1 else torch.minimum(_lengths(S, c["q"], 1), kv)
        table, n_blocks = _table(cpu, kv, bt)
        st.update(_cache(gen, n_blocks, Hkv, bt, D))
        st["q"] = randn(int(nq.sum()), H, D).to(torch.bfloat16)
        st["start"] = torch.cat([torch.zeros(1, dtype=torch.int32), nq.cumsum(0).to(torch.int32)]).cuda()
        st["pos0"], st["kv"], st["table"] = (kv - nq).cuda(), kv.cuda(), table.cuda()
        st["sink"] = randn(H) if c["sink"] else None
        st["max_q"], st["max_kv"] = int(nq.max()), int(kv.max())
    if own:
        _plan(st)
    return st


# -------------------------------------------------------------------- the framework's calls
def _plan(st):
    """Output buffers, workspace and argument structs, as a serving loop keeps them."""
    import long_context_sparse_softmax_b200 as lc
    c, op = st["c"], st["c"]["op"]
    fmt = {"bf16": lc.LC_FMT_BF16, "f32": lc.LC_FMT_F32, "mxfp8": lc.LC_FMT_MXFP8}

    def p(t):
        return None if t is None else t.data_ptr()

    def empty(*s, dtype):
        return torch.empty(*s, device="cuda", dtype=dtype)

    if op == "norm":
        n, d = c["rows"], c["d"]
        st["r_out"] = empty(n, d, dtype=DT[c["x"]]) if c["res"] else None
        st["y"] = empty(n, d, dtype=DT.get(c["y"], torch.float8_e4m3fn))
        st["ys"] = empty(n, d // 32, dtype=torch.uint8) if c["y"] == "mxfp8" else None
        a = lc.AddRmsNormArgs(n_rows=n, d=d, in_fmt=fmt[c["x"]], x=p(st["x"]), res=p(st["res"]), res_out=p(st["r_out"]),
                              w=p(st["w"]), w_fmt=lc.LC_FMT_BF16, out_fmt=fmt[c["y"]], y=p(st["y"]), y_scale=p(st["ys"]),
                              eps=EPS)
        st["call"] = lambda: lc.lc_add_rms_norm(a)
    elif op == "w4":
        st["y"] = empty(c["n"], c["G"] * c["dg"], dtype=torch.bfloat16)
        a = lc.W4ProjArgs(n_q=c["n"], G=c["G"], K=c["K"], d_g=c["dg"], in_fmt=fmt[c["x"]], out_fmt=lc.LC_FMT_BF16,
                          x=p(st["x"]), x_scale=p(st["xs"]), w=p(st["w"]), w_scale=p(st["ws"]), y=p(st["y"]))
        st["call"] = lambda: lc.lc_w4_proj(a)
    else:
        cache = lc.Kv8Cache(H_kv=c["Hkv"], D=c["D"], bt=c["bt"], n_blocks=st["k"].shape[0], table_cols=st["table"].shape[1],
                            k=p(st["k"]), v=p(st["v"]), k_scale=p(st["ks"]), v_scale=p(st["vs"]), table=p(st["table"]))
        if op == "append":
            a = lc.Kv8AppendArgs(cache=cache, num_seqs=c["S"], in_fmt=fmt[c["x"]], max_tok=st["max_new"], k=p(st["kx"]),
                                 v=p(st["vx"]), tok_start=p(st["start"]), pos0=p(st["pos0"]))
            st["call"] = lambda: lc.lc_kv8_append(a)
        else:
            decode = c["q"] == 1
            st["o"] = torch.empty_like(st["q"])
            st["lse"] = empty(st["q"].shape[0], c["H"], dtype=torch.float32)
            a = lc.Kv8AttnArgs(cache=cache, H=c["H"], num_seqs=c["S"], n_q=st["q"].shape[0], max_q=st["max_q"],
                               max_kv=st["max_kv"], W=c["W"], scale=c["D"] ** -0.5, q=p(st["q"]), q_start=p(st["start"]),
                               q_pos0=p(st["pos0"]), kv_len=p(st["kv"]), sink=p(st["sink"]), out=p(st["o"]),
                               lse=p(st["lse"]))
            ws = lc.lc_kv8_attn_workspace_bytes(a, decode)
            st["ws"] = empty(max(ws, 16), dtype=torch.uint8)
            a.workspace, a.workspace_bytes = p(st["ws"]), ws
            f = lc.lc_kv8_attn_decode if decode else lc.lc_kv8_attn_prefill
            st["call"] = lambda: f(a)


def _outputs(st):
    op, c = st["c"]["op"], st["c"]
    if op == "norm":
        out = [st["r_out"]] if c["res"] else []
        return out + [st["y"]] + ([st["ys"].view(torch.float8_e8m0fnu)] if c["y"] == "mxfp8" else [])
    if op == "w4":
        return [st["y"]]
    if op == "append":
        return [st["k"].view(torch.float8_e4m3fn), st["ks"], st["v"].view(torch.float8_e4m3fn), st["vs"]]
    return [st["o"], st["lse"]]


def run(st):
    if own:
        st["call"]()
        return _outputs(st)
    return dict(norm=_run_norm, w4=_run_w4, append=_run_append, attn=_run_attn)[st["c"]["op"]](st)


# ------------------------------------------------------------------------- the plain forms
def _run_norm(st):
    c = st["c"]
    r = st["x"].float()
    out = []
    if c["res"]:
        r = r + st["res"].float()
        out.append(r.to(DT[c["x"]]))
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * st["w"].float()
    return out + (list(_mxfp8(y)) if c["y"] == "mxfp8" else [y.to(DT[c["y"]])])


def _run_w4(st):
    c = st["c"]
    x = st["x"].float() if st["xs"] is None else _dequant_x8(st["x"], st["xs"])
    w = _dequant_w4(st["w"], st["ws"])
    x = x.view(c["n"], c["G"], c["K"]).transpose(0, 1)
    return [torch.bmm(x, w.transpose(1, 2)).transpose(0, 1).reshape(c["n"], -1).to(torch.bfloat16)]


def _run_append(st):
    c = st["c"]
    S, bt = c["S"], c["bt"]
    start, pos0 = st["start"].long(), st["pos0"].long()
    new = start[1:] - start[:-1]
    b0 = pos0 // bt
    j = torch.arange((st["max_new"] + bt - 1) // bt + 1, device="cuda")
    blk = b0[:, None] + j  # [S, J]: the blocks that the new tokens can touch
    pos = blk[:, :, None] * bt + torch.arange(bt, device="cuda")
    is_new = (pos >= pos0[:, None, None]) & (pos < (pos0 + new)[:, None, None])
    is_old = pos < pos0[:, None, None]
    touched = is_new.any(-1)
    row = (start[:-1, None, None] + pos - pos0[:, None, None]).clamp(0, st["kx"].shape[0] - 1)
    page = st["table"].long().gather(1, blk.clamp(max=st["table"].shape[1] - 1))
    for x, codes, scales in ((st["kx"], st["k"], st["ks"]), (st["vx"], st["v"], st["vs"])):
        xb = x.float()[row].transpose(2, 3) * is_new[:, :, None, :, None]  # [S, J, Hkv, bt, D]
        e = _scale_exp(_finite_amax(xb, (-1, -2)), E_MIN, E_MAX, E_MIN)
        e_old = scales[page].to(torch.int32) - 127
        e = torch.where(is_old.any(-1)[:, :, None], torch.maximum(e, e_old), e)
        fresh = _e4m3(xb * _pow2(-e)[..., None, None])
        have = codes.view(torch.float8_e4m3fn)[page]
        again = _e4m3(have.float() * _pow2(e_old - e)[..., None, None])
        new_codes = torch.where(is_new[:, :, None, :, None], fresh.view(torch.uint8), torch.where(
            is_old[:, :, None, :, None], again.view(torch.uint8), have.view(torch.uint8)))
        codes[page[touched]] = new_codes[touched]
        scales[page[touched]] = (e + 127).to(torch.uint8)[touched]
    return [st["k"].view(torch.float8_e4m3fn), st["ks"], st["v"].view(torch.float8_e4m3fn), st["vs"]]


def _run_attn(st):
    c = st["c"]
    S, H, Hkv, D, bt = c["S"], c["H"], c["Hkv"], c["D"], c["bt"]
    table, start, pos0, kv = st["table"].long(), st["start"].long(), st["pos0"].long(), st["kv"].long()

    def rows(codes, scales):  # [S, Hkv, T, D]
        x = codes.view(torch.float8_e4m3fn)[table].float() * _pow2(scales[table].to(torch.int32) - 127)[..., None, None]
        return x.transpose(1, 2).reshape(S, Hkv, -1, D)

    k, v = rows(st["k"], st["ks"]), rows(st["v"], st["vs"])
    T = k.shape[2]
    i = torch.arange(st["max_q"], device="cuda")
    real = i < (start[1:] - start[:-1])[:, None]  # [S, Q]
    q = st["q"].float()[(start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)]  # [S, Q, H, D]
    q = q.view(S, -1, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)
    s = (q @ k.transpose(2, 3)).view(S, Hkv, H // Hkv, -1, T) * D ** -0.5
    p = pos0[:, None] + i
    t = torch.arange(T, device="cuda")
    see = (t <= p[..., None]) & (t < kv[:, None, None])
    if c["W"]:
        see &= t > p[..., None] - c["W"]
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    if c["sink"]:
        sink = st["sink"].view(1, Hkv, H // Hkv, 1, 1)
        m = torch.maximum(m, sink)
    e = s.sub_(m.masked_fill(m == -math.inf, 0)).exp_()
    z = e.sum(-1, keepdim=True)
    if c["sink"]:
        z = z + torch.exp(sink - m)
    o = (e.view(S, Hkv, -1, T) @ v).view(S, Hkv, H // Hkv, -1, D) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + torch.log(z)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, -1, H, D)[real]
    return [o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(S, -1, H)[real]]


# ---------------------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    if op == "norm":
        b = 4 if c["x"] == "f32" else 2
        n = c["rows"] * c["d"]
        by = n * b * (3 if c["res"] else 1) + c["d"] * 2 + n * {"mxfp8": 33 / 32, "bf16": 2, "f32": 4}[c["y"]]
        return dict(bytes=by, flops=6 * n)
    if op == "w4":
        w = c["G"] * c["dg"] * c["K"]
        x = c["n"] * c["G"] * c["K"] * (2 if c["x"] == "bf16" else 33 / 32)
        return dict(bytes=w * 17 / 32 + x + c["n"] * c["G"] * c["dg"] * 2, flops=2 * w * c["n"])
    if op == "append":
        tok = c["new"] * (1 + (c["S"] - 1) * 0.5)
        n = 2 * tok * c["Hkv"] * c["D"]
        return dict(bytes=n * ((2 if c["x"] == "bf16" else 4) + 1), flops=2 * n)
    # decode: the mean of the ragged lengths below the longest; prefill: the same, causal
    S, q, W = c["S"], c["q"], c["W"]
    tot_kv = c["kv"] * (1 + (S - 1) * (0.5 if q == 1 else 0.625))
    seen = min(tot_kv, S * (W + q - 1)) if W else tot_kv
    tot_q = S if q == 1 else q * (1 + (S - 1) * 0.5)
    per_q = tot_kv / S - (q - 1) / 2
    per_q = min(per_q, W) if W else per_q
    by = 2 * seen * c["Hkv"] * c["D"] + tot_q * c["H"] * (4 * c["D"] + 4)
    return dict(bytes=by, flops=4 * tot_q * per_q * c["H"] * c["D"])


# ------------------------------------------------------------------ the definition in 64 bits
def _round_e4m3_64(x):
    """FP64 values to the nearest E4M3 value, ties to even, saturating: by steps of the grid."""
    a = x.abs().clamp(max=448.0)
    _, ex = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _ceil_exp_64(a, lo, hi):
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448.0))
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(a <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return e.clamp(lo, hi)


def exact(case, seed):
    c, op = case, case["op"]
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(norm=_exact_norm, w4=_exact_w4, append=_exact_append, attn=_exact_attn)[op](c, st)


def _exact_norm(c, st):
    rs, ys, ss = [], [], []
    for a in range(0, c["rows"], 2048):
        r = st["x"][a:a + 2048].double()
        if c["res"]:
            r = r + st["res"][a:a + 2048].double()
            rs.append(r)
        y = r / torch.sqrt(r.pow(2).sum(1, keepdim=True) / c["d"] + EPS) * st["w"].double()
        if c["y"] == "mxfp8":
            b = y.reshape(y.shape[0], -1, 32)
            x = torch.exp2(_ceil_exp_64(b.abs().amax(2), -127, 127))
            ss.append(x)
            y = _round_e4m3_64(b / x[:, :, None]).reshape(y.shape)
        ys.append(y)
    return [torch.cat(v) for v in (rs, ys, ss) if v]


def _exact_w4(c, st):
    K, out = c["K"], []
    for g in range(c["G"]):
        nib = torch.stack([st["w"][g] & 15, st["w"][g] >> 4], 2).reshape(c["dg"], K).int()
        mag, ex = (nib & 1).double(), (nib >> 1) & 3
        val = torch.where(ex == 0, mag * 0.5, (1 + 0.5 * mag) * torch.exp2(ex.double() - 1))
        val = torch.where(nib >= 8, -val, val) * torch.exp2(st["ws"][g].double() - 127).repeat_interleave(32, 1)
        x = st["x"][:, g * K:(g + 1) * K].double()
        if st["xs"] is not None:
            x = x * torch.exp2(st["xs"].view(torch.uint8)[:, g * K // 32:(g + 1) * K // 32].double() - 127).repeat_interleave(32, 1)
        out.append(x @ val.t())
    return [torch.cat(out, 1)]


def _exact_append(c, st):
    """One sequence and one block row at a time, from the definition."""
    bt = c["bt"]
    start, pos0, table = st["start"].tolist(), st["pos0"].tolist(), st["table"].long()
    out = []
    for x, codes, scales in ((st["kx"], st["k"], st["ks"]), (st["vx"], st["v"], st["vs"])):
        val, sc = codes.view(torch.float8_e4m3fn).double(), scales.clone()
        for s in range(c["S"]):
            lo, hi = pos0[s], pos0[s] + start[s + 1] - start[s]
            if hi == lo:
                continue
            new = x[start[s]:start[s + 1]].double()
            first, last = lo // bt, (hi - 1) // bt
            cuts = [lo] + [b * bt for b in range(first + 1, last + 1)] + [hi]
            whole = [i for i in range(len(cuts) - 1) if cuts[i] % bt == 0 and cuts[i + 1] - cuts[i] == bt]
            if whole:  # complete new blocks, together
                w = torch.stack([new[cuts[i] - lo:cuts[i + 1] - lo] for i in whole]).transpose(1, 2)
                e = _ceil_exp_64(w.abs().amax((2, 3)), E_MIN, E_MAX)
                page = table[s, torch.tensor([cuts[i] // bt for i in whole], device="cuda")]
                val[page] = _round_e4m3_64(w / torch.exp2(e)[:, :, None, None])
                sc[page] = (e + 127).to(torch.uint8)
            for i in range(len(cuts) - 1):
                if i in whole:
                    continue
                page, r0 = table[s, cuts[i] // bt], cuts[i] % bt
                w = new[cuts[i] - lo:cuts[i + 1] - lo].transpose(0, 1)
                e = _ceil_exp_64(w.abs().amax((1, 2)), E_MIN, E_MAX)
                if r0:
                    was = sc[page].double() - 127
                    e = torch.maximum(e, was)
                    val[page, :, :r0] = _round_e4m3_64(val[page, :, :r0] * torch.exp2(was - e)[:, None, None])
                val[page, :, r0:r0 + w.shape[1]] = _round_e4m3_64(w / torch.exp2(e)[:, None, None])
                sc[page] = (e + 127).to(torch.uint8)
        out += [val, sc]
    return out


def _exact_attn(c, st):
    H, Hkv, D, bt, W = c["H"], c["Hkv"], c["D"], c["bt"], c["W"]
    g = H // Hkv
    o = torch.zeros(st["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(o.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    start, pos0, kv = st["start"].tolist(), st["pos0"].tolist(), st["kv"].tolist()
    for s in range(c["S"]):
        q0, q1 = start[s], start[s + 1]
        pages = st["table"][s, :(kv[s] + bt - 1) // bt].long()
        for h in range(Hkv):
            key, val = ((st[x].view(torch.float8_e4m3fn)[pages, h].double() *
                         torch.exp2(st[x + "s"][pages, h].double() - 127)[:, None, None]).reshape(-1, D)[:kv[s]]
                        for x in ("k", "v"))
            pos = torch.arange(pos0[s], pos0[s] + q1 - q0, device="cuda")
            t = torch.arange(kv[s], device="cuda")
            hide = t[None, :] > pos[:, None]
            if W:
                hide = hide | (t[None, :] <= pos[:, None] - W)
            for hh in range(h * g, (h + 1) * g):
                lg = (st["q"][q0:q1, hh].double() @ key.t()) / math.sqrt(D)
                lg[hide] = -math.inf
                if c["sink"]:
                    all_lg = torch.cat([lg, st["sink"][hh].double().expand(q1 - q0, 1)], 1)
                else:
                    all_lg = lg
                z = torch.logsumexp(all_lg, 1)
                lse[q0:q1, hh] = z
                o[q0:q1, hh] = torch.exp(lg - z[:, None]) @ val
    return [o, lse]

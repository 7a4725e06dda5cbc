"""Host-side checks of the dense-layer entry points: what they refuse, and what they accept without
a launch (no GPU needed: a refused or empty call touches no device memory)."""
import ctypes

import pytest

import long_context_sparse_softmax_b200 as lc

OK, ARG, ALIGN, UNSUP, WS = lc.LC_OK, lc.LC_ERR_ARG, lc.LC_ERR_ALIGN, lc.LC_ERR_UNSUPPORTED, lc.LC_ERR_WORKSPACE
P = 1 << 20  # an aligned address that is never read


def call(name, a):
    return getattr(lc.lib, name)(ctypes.byref(a), None)


def norm(**kw):
    a = dict(n_rows=4, d=64, in_fmt=lc.LC_FMT_BF16, x=P, res=P, res_out=P, w=P, w_fmt=lc.LC_FMT_BF16,
             out_fmt=lc.LC_FMT_MXFP8, y=P, y_scale=P, eps=1e-6)
    a.update(kw)
    return call("lc_add_rms_norm", lc.AddRmsNormArgs(**a))


@pytest.mark.parametrize("kw,want", [
    (dict(n_rows=-1), ARG), (dict(d=0), ARG), (dict(d=12), ARG), (dict(d=16392), ARG), (dict(d=40), ARG),  # 40: not a multiple of 32
    (dict(in_fmt=lc.LC_FMT_E4M3_BF16), ARG), (dict(in_fmt=lc.LC_FMT_MXFP8), ARG), (dict(w_fmt=7), ARG), (dict(out_fmt=2), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(x=None), ARG), (dict(y=None), ARG), (dict(y_scale=None), ARG),
    (dict(x=P + 8), ALIGN), (dict(res=P + 2), ALIGN), (dict(res_out=P + 4), ALIGN), (dict(w=P + 8), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(y_scale=P + 2), ALIGN), (dict(n_rows=1 << 31), ARG), (dict(n_rows=0), OK), (dict(n_rows=0, x=None, y=None), OK)])
def test_add_rms_norm(kw, want):
    assert norm(**kw) == want


def w4(**kw):
    a = dict(n_q=4, G=2, K=64, d_g=8, in_fmt=lc.LC_FMT_BF16, out_fmt=lc.LC_FMT_F32, x=P, x_scale=P, w=P, w_scale=P, y=P)
    a.update(kw)
    return call("lc_w4_proj", lc.W4ProjArgs(**a))


@pytest.mark.parametrize("kw,want", [
    (dict(n_q=-1), ARG), (dict(G=0), ARG), (dict(K=0), ARG), (dict(K=48), ARG), (dict(d_g=0), ARG), (dict(in_fmt=lc.LC_FMT_F32), ARG),
    (dict(out_fmt=lc.LC_FMT_MXFP8), ARG), (dict(x=None), ARG), (dict(w=None), ARG), (dict(w_scale=None), ARG), (dict(y=None), ARG),
    (dict(in_fmt=lc.LC_FMT_MXFP8, x_scale=None), ARG), (dict(x=P + 8), ALIGN), (dict(w=P + 8), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(w_scale=P + 2), ALIGN), (dict(G=1 << 20, K=1 << 20), UNSUP), (dict(G=1 << 16, d_g=1 << 16), UNSUP),
    (dict(n_q=2147483647), UNSUP), (dict(n_q=0), OK)])
def test_w4_proj(kw, want):
    assert w4(**kw) == want


def cache(**kw):
    a = dict(H_kv=2, D=128, bt=64, n_blocks=8, table_cols=4, k=P, v=P, k_scale=P, v_scale=P, table=P)
    a.update(kw)
    return lc.Kv8Cache(**a)


CACHE = [(dict(H_kv=0), ARG), (dict(n_blocks=-1), ARG), (dict(table_cols=-1), ARG), (dict(D=96), UNSUP), (dict(D=256), UNSUP),
         (dict(bt=8), UNSUP), (dict(bt=48), UNSUP), (dict(bt=256), UNSUP), (dict(table_cols=1 << 26, bt=64), ARG),
         (dict(n_blocks=1 << 30, H_kv=4), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG),
         (dict(table=None), ARG), (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN)]


def append(c=None, **kw):
    a = dict(cache=c or cache(), num_seqs=2, in_fmt=lc.LC_FMT_BF16, max_tok=3, k=P, v=P, tok_start=P, pos0=P)
    a.update(kw)
    return call("lc_kv8_append", lc.Kv8AppendArgs(**a))


@pytest.mark.parametrize("kw,want", [
    (dict(in_fmt=lc.LC_FMT_MXFP8), ARG), (dict(num_seqs=-1), ARG), (dict(max_tok=-1), ARG), (dict(k_stride=128), ARG), (dict(k_stride=260), ARG),
    (dict(v_stride=-256), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(tok_start=None), ARG), (dict(pos0=None), ARG),
    (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN), (dict(num_seqs=0), OK), (dict(max_tok=0), OK)])
def test_kv8_append(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", CACHE)
def test_kv8_cache(kw, want):
    assert append(cache(**kw)) == want
    a = dict(cache=cache(**kw), workspace=P, workspace_bytes=1 << 40)
    if "H_kv" in kw and kw["H_kv"]:
        a["H"] = 4 * kw["H_kv"]
    assert attn("decode", **a) == want and attn("prefill", **a) == want


def attn(which, **kw):
    d = which == "decode"
    a = dict(cache=cache(), H=8, num_seqs=3, n_q=3 if d else 40, max_q=1 if d else 20, max_kv=256, W=0, scale=0.1, q=P, q_start=P, q_pos0=P,
             kv_len=P, out=P, lse=P, workspace=P, workspace_bytes=1 << 40)
    a.update(kw)
    return call("lc_kv8_attn_" + which, lc.Kv8AttnArgs(**a))


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("kw,want", [
    (dict(H=0), ARG), (dict(H=7), ARG), (dict(num_seqs=-1), ARG), (dict(n_q=-1), ARG), (dict(max_q=-1), ARG), (dict(max_kv=-1), ARG), (dict(W=-1), ARG),
    (dict(q_stride=512), ARG), (dict(q_stride=1028), ARG), (dict(q=None), ARG), (dict(q_start=None), ARG), (dict(q_pos0=None), ARG),
    (dict(kv_len=None), ARG), (dict(out=None), ARG), (dict(q=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(num_seqs=0, n_q=0), OK), (dict(max_q=0), OK)])
def test_kv8_attn(which, kw, want):
    assert attn(which, **kw) == want


def test_kv8_attn_decode_takes_one_query_a_sequence():
    assert attn("decode", n_q=4) == ARG and attn("decode", max_q=2) == ARG


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_kv8_attn_workspace(which):
    d = which == "decode"
    a = lc.Kv8AttnArgs(cache=cache(table_cols=1024), H=8, num_seqs=1, n_q=1 if d else 2, max_q=1 if d else 2, max_kv=60000)
    need = lc.lc_kv8_attn_workspace_bytes(a, d)
    assert need > 0
    kw = dict(cache=cache(table_cols=1024), num_seqs=1, n_q=a.n_q, max_q=a.max_q, max_kv=60000)
    assert attn(which, workspace_bytes=need - 1, **kw) == WS and attn(which, workspace=None, **kw) == WS
    assert attn(which, workspace=P + 8, **kw) == ALIGN
    for bad in (dict(H=7), dict(max_kv=0), dict(n_q=0), dict(cache=cache(D=96))):
        b = lc.Kv8AttnArgs(cache=bad.get("cache", a.cache), H=bad.get("H", 8), num_seqs=1, n_q=bad.get("n_q", a.n_q), max_q=a.max_q,
                           max_kv=bad.get("max_kv", 60000))
        assert lc.lc_kv8_attn_workspace_bytes(b, d) == 0


def test_workspace_covers_every_shorter_sequence():
    """The split of a sequence follows from its own length: the workspace of a call holds the splits of
    every length up to max_kv (the number of splits does not grow steadily with the length)."""
    for hkv in (1, 2, 8, 16):
        c = cache(H_kv=hkv, table_cols=1 << 20)

        def need(n):
            return lc.lc_kv8_attn_workspace_bytes(lc.Kv8AttnArgs(cache=c, H=hkv, num_seqs=1, n_q=1, max_q=1, max_kv=n), True)
        most = 0
        for n in [*range(1, 12000, 61), *range(12000, 1500000, 9973)]:
            assert need(n) >= most
            most = need(n)


@pytest.mark.parametrize("which", ["prefill", "decode"])
def test_a_window_wider_than_the_context_needs_the_same_workspace(which):
    """A window up to the type's last value is no window: no sum with it may pass 32 bits."""
    d = which == "decode"
    for max_q in (1,) if d else (1, 2, 3, 4000):
        def need(W, max_kv=60000):
            return lc.lc_kv8_attn_workspace_bytes(lc.Kv8AttnArgs(
                cache=cache(table_cols=1024), H=8, num_seqs=1, n_q=max_q, max_q=max_q, max_kv=max_kv, W=W), d)
        for W in (60000, (1 << 31) - max_q, (1 << 31) - 17, (1 << 31) - 16, (1 << 31) - 1):
            assert need(W) == need(0)
        # no more keys than the table has columns for: 65536
        assert need(0, (1 << 31) - 1) == need(0, 65536)


def test_cache_of_at_most_2_30_tokens():
    for bt in (16, 32, 64, 128):
        assert append(cache(table_cols=(1 << 30) // bt, bt=bt), num_seqs=0) == OK
        assert append(cache(table_cols=(1 << 30) // bt + 1, bt=bt), num_seqs=0) == ARG
        assert attn("prefill", cache=cache(table_cols=(1 << 30) // bt + 1, bt=bt)) == ARG


def test_w4_proj_launch_limits():
    assert w4(n_q=65535 * 32 + 1) == UNSUP and w4(n_q=65535 * 64 + 1, in_fmt=lc.LC_FMT_MXFP8) == UNSUP
    assert w4(G=1, K=32, d_g=(1 << 31) - 1) == UNSUP and w4(G=1, K=32, d_g=(1 << 31) - 127) == UNSUP

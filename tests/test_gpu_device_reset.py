"""The library keeps no state that a device reset makes false: after cudaDeviceReset, which ends the calling
process's own context alone, every call works as before it.  In a process of its own, without torch."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, glob, sys
import numpy as np
import long_context_sparse_softmax_b200 as lc
so = lc.load()
path = [p for d in sys.path for p in glob.glob(d + "/nvidia/cuda_runtime/lib/libcudart.so*")] + glob.glob("/usr/local/cuda/lib64/libcudart.so*")
rt = ctypes.CDLL(path[0])

def ok(e):
    assert e == 0, e

def malloc(n):
    p = ctypes.c_void_p()
    ok(rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(n)))
    ok(rt.cudaMemset(p, 0, ctypes.c_size_t(n)))
    return p.value

def put(a):
    p = malloc(a.nbytes)
    ok(rt.cudaMemcpy(ctypes.c_void_p(p), a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes), 1))
    return p

def get(p, like):
    a = np.empty_like(like)
    ok(rt.cudaMemcpy(a.ctypes.data_as(ctypes.c_void_p), ctypes.c_void_p(p), ctypes.c_size_t(a.nbytes), 2))
    return a

def calls(stream=None, check=True):
    # a norm whose ring needs more than 48 KB, a projection, decode and prefill over an 8-bit cache
    n, d, K = 8, 16384, 512
    x = np.arange(n * d, dtype=np.float32).reshape(n, d) % 7 - 3
    y, z, o, o2 = malloc(x.nbytes), malloc(8 * K * 4), malloc(1 << 16), malloc(1 << 16)
    w, ws, big = put(np.full((K, K // 2), 0x22, np.uint8)), put(np.full((K, K // 32), 127, np.uint8)), put(np.full((8, K), 0x3f80, np.uint16))
    codes, scale = put(np.full((4, 1, 64, 64), 0x38, np.uint8)), put(np.full(4, 127, np.uint8))  # ones
    i32 = lambda *v: put(np.array(v, np.int32))
    cache = lc.Kv8Cache(H_kv=1, D=64, bt=64, n_blocks=4, table_cols=4, k=codes, v=codes, k_scale=scale, v_scale=scale, table=i32(0, 1, 2, 3))
    q = put(np.full((40, 1, 64), 0x3f80, np.uint16))
    dec = lc.Kv8AttnArgs(cache=cache, H=1, num_seqs=1, n_q=1, max_q=1, max_kv=200, scale=0.125, q=q, q_start=i32(0, 1), q_pos0=i32(199),
                         kv_len=i32(200), out=o)
    pre = lc.Kv8AttnArgs(cache=cache, H=1, num_seqs=1, n_q=40, max_q=40, max_kv=200, scale=0.125, q=q, q_start=i32(0, 40), q_pos0=i32(160),
                         kv_len=i32(200), out=o2)
    assert lc.lc_kv8_attn_workspace_bytes(dec, True) == lc.lc_kv8_attn_workspace_bytes(pre, False) == 0
    xp, r = put(x), ctypes.byref
    def run():
        return [so.lc_add_rms_norm(r(lc.AddRmsNormArgs(n_rows=n, d=d, in_fmt=0, x=xp, res=xp, out_fmt=0, y=y, eps=0.0)), stream),
                so.lc_w4_proj(r(lc.W4ProjArgs(n_q=8, G=1, K=K, d_g=K, in_fmt=1, out_fmt=0, x=big, w=w, w_scale=ws, y=z)), stream),
                so.lc_kv8_attn_decode(r(dec), stream), so.lc_kv8_attn_prefill(r(pre), stream)]
    def good():
        ok(rt.cudaDeviceSynchronize())
        ref = x / np.sqrt((x.astype(np.float64) ** 2).mean(1, keepdims=True))
        assert np.all(np.abs(get(y, x) - ref) <= 40 * 2.0 ** -24 * np.abs(ref))
        assert np.all(get(z, np.empty((8, K), np.float32)) == K)
        assert np.all(get(o, np.empty(64, np.uint16)) == 0x3f80) and np.all(get(o2, np.empty((40, 64), np.uint16)) == 0x3f80)
    return run, good

def eager():
    run, good = calls()
    assert run() == [0] * 4, "a call failed"
    good()

def captured():
    st, graph, exe = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    ok(rt.cudaStreamCreate(ctypes.byref(st)))
    run, good = calls(st)
    ok(rt.cudaStreamBeginCapture(st, 0))
    assert run() == [0] * 4, "a captured call failed"
    ok(rt.cudaStreamEndCapture(st, ctypes.byref(graph)))
    ok(rt.cudaGraphInstantiate(ctypes.byref(exe), graph, ctypes.c_ulonglong(0)))
    ok(rt.cudaGraphLaunch(exe, st))
    ok(rt.cudaStreamSynchronize(st))
    good()
    ok(rt.cudaGraphExecDestroy(exe))
    ok(rt.cudaGraphDestroy(graph))

for first in (eager, eager, captured, eager):
    first()
    eager()
    ok(rt.cudaDeviceReset())
print("fine")
"""


@pytest.mark.gpu
def test_calls_after_a_device_reset():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), (r.stdout + r.stderr)[-2000:]

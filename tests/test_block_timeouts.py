"""Failure detection of the operators around the layer without a fault: in the debug build a
wait budget of 0 makes the first wait of every pipelined kernel run out. The kernel then issues
no more work, lets what is in flight land, frees its tensor memory and returns; the error word
reports NMOE_ERR_TIMEOUT, and the next call is right."""

import ctypes as C
import os
import subprocess
import sys
from pathlib import Path

import pytest

import diffusion_transformer_moe_b200 as nm

ROOT = Path(__file__).resolve().parents[1]
DEBUG_LIB = ROOT / "diffusion_transformer_moe_b200" / "libnmoe_debug.so"


def test_only_the_debug_build_sets_the_budget():
    assert hasattr(C.CDLL(str(DEBUG_LIB)), "nmoe_debug_block_wait_ns")
    assert not hasattr(nm.lib(), "nmoe_debug_block_wait_ns") or "debug" in nm.build_info()


_RUN = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import diffusion_transformer_moe_b200 as nm
import ctypes
assert "debug checks" in nm.build_info()
budget = nm.lib().nmoe_debug_block_wait_ns
budget.argtypes, budget.restype = [ctypes.c_uint64], None
g = torch.Generator("cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)

def linear(M, K, N, **kw):
    x, w, b = r(M, K), r(K, N), r(N)
    return lambda: (nm.linear(x, w, b, **kw),)

def fp8(M, K, N):
    x, w = nm.quantize_rows(r(M, K)), nm.quantize_rows(r(N, K))
    return lambda: (nm.linear_fp8(*x, *w),)

def grads(M, K, N, **kw):
    x, w, dy = r(M, K), r(K, N), r(M, N)
    return lambda: [t for t in nm.linear_backward(dy, x, w, **kw) if t is not None]

def norm(T, d):
    h, dy, w, dh = r(T, d), r(T, d), r(d), r(T, d)
    rstd = nm.rms_norm(h, w).rstd
    return lambda: nm.rms_norm_backward(dy, h, rstd, w, dh=dh)

cases = dict(
    swapped=linear(8, 64, 128), swapped_parts=linear(16, 2048, 512), whole=linear(200, 256, 136),
    parts=linear(100, 4096, 72, act="silu"), long_ring=linear(391, 7936, 1824),
    pairs=linear(8192, 64, 2048), pairs_act=linear(4700, 264, 1800, act="gelu"),
    fp8_tiles=fp8(300, 2048, 1000), fp8_pairs=fp8(4700, 272, 1800),
    two_tiles=grads(33, 72, 104), sums_beside=grads(2001, 1032, 64),
    two_pairs=grads(2100, 1032, 2056), apart=grads(600, 4096, 3000, need_dx=False),
    norm=norm(1000, 2048), norm_cluster=norm(100, 256), norm_wide=norm(300, 16384))
for name, call in cases.items():
    want = call()
    torch.cuda.synchronize()
    assert nm.get_last_error() == 0, name
    budget(0)
    call()
    budget(2_000_000_000)
    torch.cuda.synchronize()
    assert nm.get_last_error() == 5, name          # NMOE_ERR_TIMEOUT
    assert nm.get_last_error() == 0, name          # read and cleared
    got = call()
    torch.cuda.synchronize()
    assert nm.get_last_error() == 0, name
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    print(name, "ok", flush=True)
"""


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    r = subprocess.run([sys.executable, "-c", _RUN, str(ROOT)], capture_output=True, text=True,
                       timeout=240, env=dict(os.environ, NMOE_DEBUG="1"))
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
    assert r.stdout.count(" ok") == 16

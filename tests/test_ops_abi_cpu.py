"""include/fp4mi_ops.h: the header compiles as C99, every entry point it
declares is exported and bound, and host-side validation returns the documented
status without touching a GPU -- also under AddressSanitizer and UBSan (host
code only)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4mi_ops.h")
CSRC = os.path.join(ROOT, "block_scaled_fp4_amd", "csrc")
SANITIZED = os.environ.get("FP4MI_SANITIZED_OPS_LIB")
LIB = SANITIZED or os.path.join(ROOT, "block_scaled_fp4_amd", "libfp4mi.so")
P, I, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
OK, EINVAL, ESHAPE, EALIGN, EDTYPE, EHIP, EOVERLAP = range(7)
G = 1 << 30
A = 0x7F0000000000                      # never dereferenced: validation comes first


def declared():
    return re.findall(r"^(?:int|int64_t)\s+(\w+)\(", open(HEADER).read(), flags=re.M)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("libfp4mi.so is not built (python __graft_entry__.py)")
    h = ctypes.CDLL(LIB)
    h.mxfp4_matmul.argtypes = [P, I, P, P, P, P, I64, I64, I64, P, I, P]
    h.mxfp4_matmul_grouped.argtypes = [P, I, P, P, P, P, P, I32, I64, I64, I64, P, I, P]
    h.fp8_matmul_tokblk.argtypes = [P, P, P, P, P, I32, I64, I64, I64, P, I, P]
    h.rmsnorm_quantize.argtypes = [P, P, I, P, I, I64, I64, F32, I, P, P, P, P, P]
    h.rmsnorm_backward.argtypes = [P, P, P, I, P, I, P, I64, I64, P, P, P, I64, P]
    h.rmsnorm_backward_workspace.argtypes = [I64, I64]
    h.rmsnorm_backward_workspace.restype = I64
    return h


def test_exported_and_bound(lib):
    names = declared()
    assert len(names) == 6
    for n in names:
        assert hasattr(lib, n), n
    if not SANITIZED:
        import block_scaled_fp4_amd as m
        for n in names:
            assert callable(getattr(m, n)), n


def dense(lib, a=A, fmt=0, sa=A + G, row=A + 2 * G, b=A + 3 * G, sb=A + 4 * G, m=4, n=8, k=256, out=A + 5 * G, dt=1):
    return lib.mxfp4_matmul(a, fmt, sa, row, b, sb, m, n, k, out, dt, None)


def grouped(lib, a=A, fmt=0, sa=A + G, row=A + 2 * G, b=A + 3 * G, sb=A + 4 * G, off=A + 6 * G, e=3, t=4, n=8, k=256,
            out=A + 5 * G, dt=1):
    return lib.mxfp4_matmul_grouped(a, fmt, sa, row, b, sb, off, e, t, n, k, out, dt, None)


@pytest.mark.parametrize("call", [dense, grouped])
def test_products(lib, call):
    rows = "m" if call is dense else "t"
    assert call(lib, fmt=2) == EINVAL
    assert call(lib, dt=2) == EDTYPE
    assert call(lib, k=48) == ESHAPE
    assert call(lib, fmt=1, k=160) == ESHAPE                # FP8 rows need K % 128
    assert call(lib, k=0) == ESHAPE
    assert call(lib, k=1 << 21) == ESHAPE
    assert call(lib, n=-1) == ESHAPE
    assert call(lib, n=1 << 26) == ESHAPE
    assert call(lib, **{rows: -1}) == ESHAPE
    assert call(lib, **{rows: 1 << 26}) == ESHAPE
    assert call(lib, **{rows: 0}, a=None, out=None) == OK   # empty output
    assert call(lib, n=0, b=None) == OK
    for p in ("a", "sa", "b", "sb", "out"):
        assert call(lib, **{p: None}) == EINVAL, p
    assert call(lib, a=A + 8) == EALIGN
    assert call(lib, sa=A + G + 2) == EALIGN
    assert call(lib, row=A + 2 * G + 2) == EALIGN
    assert call(lib, b=A + 3 * G + 8) == EALIGN
    assert call(lib, out=A + 5 * G + 8) == EALIGN
    for p in (A, A + G, A + 2 * G, A + 3 * G, A + 4 * G):
        assert call(lib, out=p) == EOVERLAP
    if call is grouped:
        assert call(lib, e=0) == EINVAL
        assert call(lib, e=1 << 23) == ESHAPE
        assert call(lib, off=None) == EINVAL
        assert call(lib, off=A + 6 * G + 4) == EALIGN
        assert call(lib, out=A + 6 * G) == EOVERLAP
        assert call(lib, e=1 << 22, n=1 << 25, k=1 << 20) == ESHAPE     # E N K past 2^46


def wgrad(lib, a=A, sa=A + G, b=A + 2 * G, sb=A + 3 * G, off=A + 4 * G, e=3, t=300, m=128, n=256, out=A + 5 * G, dt=0):
    return lib.fp8_matmul_tokblk(a, sa, b, sb, off, e, t, m, n, out, dt, None)


def test_weight_gradient(lib):
    assert wgrad(lib, e=0) == EINVAL
    assert wgrad(lib, dt=5) == EDTYPE
    assert wgrad(lib, m=100) == ESHAPE
    assert wgrad(lib, n=64) == ESHAPE
    assert wgrad(lib, t=-1) == ESHAPE
    assert wgrad(lib, t=1 << 24) == ESHAPE
    assert wgrad(lib, m=1 << 21) == ESHAPE
    assert wgrad(lib, e=1 << 23) == ESHAPE
    assert wgrad(lib, off=None) == EINVAL
    assert wgrad(lib, m=0) == OK
    for p in ("a", "sa", "b", "sb", "out"):
        assert wgrad(lib, **{p: None}) == EINVAL, p
    assert wgrad(lib, a=A + 2) == EALIGN
    assert wgrad(lib, out=A + 5 * G + 4) == EALIGN
    assert wgrad(lib, off=A + 4 * G + 4) == EALIGN
    for p in (A, A + G, A + 2 * G, A + 3 * G, A + 4 * G):
        assert wgrad(lib, out=p) == EOVERLAP


def norm(lib, x=A, res=A + G, dt=1, w=A + 2 * G, wdt=0, rows=4, cols=256, eps=1e-6, fmt=1, q=A + 3 * G, s=A + 4 * G,
         r=A + 5 * G, h=A + 6 * G):
    return lib.rmsnorm_quantize(x, res, dt, w, wdt, rows, cols, eps, fmt, q, s, r, h, None)


def test_norm(lib):
    assert norm(lib, fmt=3) == EINVAL
    assert norm(lib, dt=4) == EDTYPE
    assert norm(lib, wdt=4) == EDTYPE
    assert norm(lib, eps=-1.0) == EINVAL
    assert norm(lib, eps=float("inf")) == EINVAL
    assert norm(lib, eps=float("nan")) == EINVAL
    assert norm(lib, cols=160) == ESHAPE
    assert norm(lib, cols=48, fmt=0) == ESHAPE
    assert norm(lib, cols=0) == ESHAPE
    assert norm(lib, cols=1 << 21) == ESHAPE
    assert norm(lib, rows=-1) == ESHAPE
    assert norm(lib, rows=1 << 40) == ESHAPE
    assert norm(lib, rows=0, x=None, q=None) == OK
    for p in ("x", "w", "q", "s", "r"):
        assert norm(lib, **{p: None}) == EINVAL, p
    for p, at in (("x", 0), ("res", G), ("w", 2 * G), ("q", 3 * G), ("h", 6 * G)):
        assert norm(lib, **{p: A + at + 8}) == EALIGN, p
    for p in ("q", "s", "r"):
        for at in (A, A + G, A + 2 * G):
            assert norm(lib, **{p: at}) == EOVERLAP, p
    assert norm(lib, h=A + 16) == EOVERLAP                  # inside x, not x itself
    assert norm(lib, h=A + 2 * G) == EOVERLAP
    assert norm(lib, s=A + 3 * G) == EOVERLAP               # two outputs
    assert norm(lib, h=A + 5 * G) == EOVERLAP


def norm_grad(lib, dy=A, h=A + G, dh=A + 2 * G, dt=1, w=A + 3 * G, wdt=0, r=A + 4 * G, rows=4, cols=96, dx=A + 5 * G,
              dw=A + 6 * G, ws=A + 7 * G, nws=None):
    nws = lib.rmsnorm_backward_workspace(rows, cols) if nws is None else nws
    return lib.rmsnorm_backward(dy, h, dh, dt, w, wdt, r, rows, cols, dx, dw, ws, nws, None)


def test_norm_gradient(lib):
    assert lib.rmsnorm_backward_workspace(4, 96) > 0
    for bad in ((-1, 96), (4, 95), (4, 0), (1 << 40, 1 << 20), (4, 1 << 21)):
        assert lib.rmsnorm_backward_workspace(*bad) == 0
    assert norm_grad(lib, dt=4) == EDTYPE
    assert norm_grad(lib, wdt=4) == EDTYPE
    assert norm_grad(lib, cols=95) == ESHAPE
    assert norm_grad(lib, rows=-1) == ESHAPE
    assert norm_grad(lib, nws=lib.rmsnorm_backward_workspace(4, 96) - 1) == ESHAPE
    for p in ("dy", "h", "w", "r", "dx", "dw", "ws"):
        assert norm_grad(lib, **{p: None}) == EINVAL, p
    for p, at in (("dy", 0), ("h", G), ("dh", 2 * G), ("w", 3 * G), ("dx", 5 * G), ("dw", 6 * G), ("ws", 7 * G)):
        assert norm_grad(lib, **{p: A + at + 8}) == EALIGN, p
    for at in (A + G, A + 3 * G, A + 4 * G, A + 16):
        assert norm_grad(lib, dx=at) == EOVERLAP
    for p in ("dw", "ws"):
        for at in (A, A + G, A + 2 * G, A + 3 * G, A + 4 * G, A + 5 * G):
            assert norm_grad(lib, **{p: at}) == EOVERLAP, p


def test_random_invalid_calls(lib):
    """Random sizes, pointers and enums with one rule broken in each call:
    never FP4_OK, never a launch."""
    rng = np.random.default_rng(0)
    breaks = [
        lambda: dense(lib, fmt=int(rng.integers(2, 99)), m=int(rng.integers(1, 1 << 20))),
        lambda: dense(lib, k=32 * int(rng.integers(1, 9)) + int(rng.integers(1, 32))),
        lambda: dense(lib, a=A + int(rng.integers(1, 16))),
        lambda: grouped(lib, e=-int(rng.integers(0, 99))),
        lambda: grouped(lib, n=int(rng.integers(1 << 26, 1 << 60))),
        lambda: grouped(lib, t=-int(rng.integers(1, 1 << 62))),
        lambda: wgrad(lib, m=128 * int(rng.integers(1, 9)) + int(rng.integers(1, 128))),
        lambda: wgrad(lib, t=int(rng.integers(1 << 24, 1 << 62))),
        lambda: norm(lib, rows=int(rng.integers(1 << 46, 1 << 62))),
        lambda: norm(lib, cols=int(rng.integers(1 << 21, 1 << 62))),
        lambda: norm_grad(lib, rows=int(rng.integers(1 << 46, 1 << 62)), nws=1 << 62),
        lambda: norm_grad(lib, nws=-int(rng.integers(1, 1 << 62))),
    ]
    for _ in range(200):
        for f in breaks:
            assert f() in (EINVAL, ESHAPE, EALIGN)


C_PROGRAM = r"""
#include <stdio.h>
#include "fp4mi_ops.h"
int main(void) {
  int (*mm)(const void*, int, const void*, const float*, const uint8_t*, const uint8_t*, int64_t, int64_t, int64_t,
            void*, int, void*) = mxfp4_matmul;
  int (*mg)(const void*, int, const void*, const float*, const uint8_t*, const uint8_t*, const int64_t*, int32_t,
            int64_t, int64_t, int64_t, void*, int, void*) = mxfp4_matmul_grouped;
  int (*wg)(const uint8_t*, const float*, const uint8_t*, const float*, const int64_t*, int32_t, int64_t, int64_t,
            int64_t, void*, int, void*) = fp8_matmul_tokblk;
  int (*rq)(const void*, const void*, int, const void*, int, int64_t, int64_t, float, int, void*, void*, float*, void*,
            void*) = rmsnorm_quantize;
  int (*rb)(const void*, const void*, const void*, int, const void*, int, const float*, int64_t, int64_t, void*, float*,
            void*, int64_t, void*) = rmsnorm_backward;
  if (mm(0, FP4_ROWS_MXFP4, 0, 0, 0, 0, 1, 1, 33, 0, FP4_DTYPE_F32, 0) != FP4_ESHAPE) return 1;
  if (mg(0, FP4_ROWS_FP8, 0, 0, 0, 0, 0, 0, 1, 1, 128, 0, FP4_DTYPE_F32, 0) != FP4_EINVAL) return 2;
  if (wg(0, 0, 0, 0, 0, 1, 1, 1, 1, 0, FP4_DTYPE_F32, 0) != FP4_ESHAPE) return 3;
  if (rq(0, 0, FP4_DTYPE_BF16, 0, FP4_DTYPE_F32, 0, 128, 0.0f, FP4_ROWS_FP8, 0, 0, 0, 0, 0) != FP4_OK) return 4;
  if (rb(0, 0, 0, FP4_DTYPE_BF16, 0, FP4_DTYPE_F32, 0, 1, 32, 0, 0, 0, 0, 0) != FP4_EINVAL) return 5;
  if (rmsnorm_backward_workspace(1, 31) != 0) return 6;
  puts("c abi ok");
  return 0;
}
"""


@pytest.mark.skipif(bool(SANITIZED), reason="already inside the sanitized run")
def test_header_is_c99(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.exists(LIB):
        pytest.skip("no C compiler or no library")
    src, exe, libdir = tmp_path / "ops.c", tmp_path / "ops", os.path.dirname(LIB)
    src.write_text(C_PROGRAM)
    b = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                        str(src), "-o", str(exe), "-L", libdir, "-l:libfp4mi.so", "-Wl,-rpath," + libdir,
                        "-Wl,--allow-shlib-undefined"], capture_output=True, text=True)
    assert b.returncode == 0, b.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "c abi ok" in r.stdout, (r.returncode, r.stdout, r.stderr)


@pytest.mark.skipif(bool(SANITIZED), reason="already inside the sanitized run")
def test_host_validation_under_asan_and_ubsan(tmp_path):
    hipcc = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    clang = "/opt/rocm/llvm/bin/clang++"
    if hipcc is None or not os.path.exists(clang):
        pytest.skip("hipcc / clang++ not available")
    rt = subprocess.run([clang, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isfile(rt):
        pytest.skip("the ASan runtime is not available")
    lib = str(tmp_path / "libops_sanitized.so")
    cmd = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-Wno-unused-command-line-argument",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer", "-shared-libsan",
           "-I", os.path.join(ROOT, "include"),
           *[os.path.join(CSRC, s) for s in ("matmul.hip", "wgrad.hip", "rmsnorm.hip", "abi.hip")], "-o", lib]
    b = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert b.returncode == 0, b.stderr[-2000:]
    env = dict(os.environ, LD_PRELOAD=rt, FP4MI_SANITIZED_OPS_LIB=lib, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=900)
    out = p.stdout + p.stderr
    assert p.returncode == 0, out[-3000:]
    assert "runtime error:" not in out and "AddressSanitizer" not in out, out[-3000:]

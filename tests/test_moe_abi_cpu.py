"""include/fp4mi_moe.h: the header compiles as C99, every entry point it declares
is exported and bound, and host-side validation returns the documented status
without touching a GPU -- also under AddressSanitizer and UBSan (host code only).
The binding's own refusals run on CPU and fake tensors."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4mi_moe.h")
CSRC = os.path.join(ROOT, "block_scaled_fp4_amd", "csrc")
SANITIZED = os.environ.get("FP4MI_SANITIZED_MOE_LIB")
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
    h.fp8_quantize.argtypes = [P, I, I64, I64, P, P, P]
    h.fp8_quantize_blocks.argtypes = [P, I, I64, I64, I64, P, P, P, P, P]
    h.fp8_matmul.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, I, P]
    h.fp8_matmul_grouped.argtypes = [P, P, P, P, P, I, P, I32, I64, I64, I64, P, I, P]
    h.swiglu_quantize.argtypes = [P, I, I64, I64, I, P, P, P, P, P]
    h.swiglu_backward.argtypes = [P, I, P, P, I64, I64, P, I, P, P, P]
    h.router_balance.argtypes = [P, I, P, I, P, I64, I32, I32, F32, P, P, P, P, P, I64, P]
    h.router_balance_workspace.argtypes = [I64, I32]
    h.router_balance_workspace.restype = I64
    h.router_balance_backward.argtypes = [P, I, P, P, P, P, I64, I32, P, P]
    return h


def test_exported_and_bound(lib):
    names = declared()
    assert len(names) == 9
    for n in names:
        assert hasattr(lib, n), n
    if not SANITIZED:
        import block_scaled_fp4_amd as m
        for n in names:
            assert callable(getattr(m, n)), n


def rows(lib, x=A, dt=1, r=4, c=256, q=A + G, s=A + 2 * G):
    return lib.fp8_quantize(x, dt, r, c, q, s, None)


def blocks(lib, x=A, dt=1, b=2, r=256, c=256, q=A + G, s=A + 2 * G, qt=A + 3 * G, st=A + 4 * G):
    return lib.fp8_quantize_blocks(x, dt, b, r, c, q, s, qt, st, None)


def test_quantizers(lib):
    for call in (rows, blocks):
        assert call(lib, dt=2) == EDTYPE
        assert call(lib, c=160) == ESHAPE
        assert call(lib, c=-128) == ESHAPE
        assert call(lib, r=-128) == ESHAPE
        assert call(lib, r=1 << 40, c=1 << 10) == ESHAPE
        assert call(lib, r=0, x=None, q=None) == OK
        assert call(lib, c=0, x=None) == OK
        for p in ("x", "q", "s"):
            assert call(lib, **{p: None}) == EINVAL, p
        for p, at in (("x", 8), ("q", G + 8), ("s", 2 * G + 2)):
            assert call(lib, **{p: A + at}) == EALIGN, p
        assert call(lib, q=A + 16) == EOVERLAP
        assert call(lib, s=A + 4) == EOVERLAP
        assert call(lib, s=A + G) == EOVERLAP
    assert blocks(lib, r=200) == ESHAPE                     # the copy needs whole tiles
    assert blocks(lib, b=-1) == ESHAPE
    assert blocks(lib, b=1 << 40) == ESHAPE
    assert blocks(lib, st=None) == EINVAL
    assert blocks(lib, qt=None) == EINVAL
    assert blocks(lib, qt=A + 3 * G + 8) == EALIGN
    assert blocks(lib, st=A + 4 * G + 1) == EALIGN
    assert blocks(lib, qt=A + 32) == EOVERLAP
    assert blocks(lib, qt=A + G) == EOVERLAP
    assert blocks(lib, st=A + 2 * G) == EOVERLAP


def dense(lib, a=A, sa=A + G, row=A + 2 * G, b=A + 3 * G, sb=A + 4 * G, blk=1, m=4, n=8, k=256, out=A + 5 * G, dt=1):
    return lib.fp8_matmul(a, sa, row, b, sb, blk, m, n, k, out, dt, None)


def grouped(lib, a=A, sa=A + G, row=A + 2 * G, b=A + 3 * G, sb=A + 4 * G, blk=128, off=A + 6 * G, e=3, m=4, n=8, k=256,
            out=A + 5 * G, dt=1):
    return lib.fp8_matmul_grouped(a, sa, row, b, sb, blk, off, e, m, n, k, out, dt, None)


@pytest.mark.parametrize("call", [dense, grouped])
def test_products(lib, call):
    assert call(lib, blk=0) == EINVAL
    assert call(lib, blk=64) == EINVAL
    assert call(lib, dt=2) == EDTYPE
    assert call(lib, k=160) == ESHAPE
    assert call(lib, k=0) == ESHAPE
    assert call(lib, k=1 << 21) == ESHAPE
    assert call(lib, n=-1) == ESHAPE
    assert call(lib, n=1 << 26) == ESHAPE
    assert call(lib, m=-1) == ESHAPE
    assert call(lib, m=1 << 26) == ESHAPE
    assert call(lib, m=0, a=None, out=None) == OK
    assert call(lib, n=0, b=None) == OK
    for p in ("a", "sa", "b", "sb", "out"):
        assert call(lib, **{p: None}) == EINVAL, p
    assert call(lib, a=A + 8) == EALIGN
    assert call(lib, sa=A + G + 2) == EALIGN
    assert call(lib, row=A + 2 * G + 2) == EALIGN
    assert call(lib, b=A + 3 * G + 8) == EALIGN
    assert call(lib, sb=A + 4 * G + 1) == EALIGN
    assert call(lib, out=A + 5 * G + 8) == EALIGN
    for p in (A, A + G, A + 2 * G, A + 3 * G, A + 4 * G):
        assert call(lib, out=p) == EOVERLAP
    if call is grouped:
        assert call(lib, e=0) == EINVAL
        assert call(lib, e=1 << 23) == ESHAPE
        assert call(lib, off=None) == EINVAL
        assert call(lib, off=A + 6 * G + 4) == EALIGN
        assert call(lib, out=A + 6 * G) == EOVERLAP
        assert call(lib, e=1 << 22, n=1 << 25, k=1 << 20) == ESHAPE


def swiglu(lib, x=A, dt=1, r=4, f=256, fmt=1, q=A + G, s=A + 2 * G, c=A + 3 * G, cs=A + 4 * G):
    return lib.swiglu_quantize(x, dt, r, f, fmt, q, s, c, cs, None)


def swiglu_grad(lib, dy=A, dt=1, c=A + G, cs=A + 2 * G, r=4, f=256, dx=A + 3 * G, fmt=1, q=A + 4 * G, s=A + 5 * G):
    return lib.swiglu_backward(dy, dt, c, cs, r, f, dx, fmt, q, s, None)


def test_swiglu(lib):
    for call in (swiglu, swiglu_grad):
        assert call(lib, dt=2) == EDTYPE
        assert call(lib, fmt=2) == EINVAL
        for f in (0, -128, 1 << 20, 160):
            assert call(lib, f=f) == ESHAPE, f
        assert call(lib, r=-1) == ESHAPE
        assert call(lib, r=1 << 40) == ESHAPE
        assert call(lib, r=0, q=None, s=None) == OK
        assert call(lib, s=None) == EINVAL
    assert swiglu(lib, fmt=0, f=160) == ESHAPE              # a checkpoint needs whole blocks
    assert swiglu(lib, fmt=0, f=48, c=None, cs=None) == ESHAPE
    assert swiglu(lib, r=0, x=None) == OK
    assert swiglu(lib, cs=None) == EINVAL
    for p in ("x", "q"):
        assert swiglu(lib, **{p: None, **({"s": None} if p == "q" else {})}) == EINVAL
    for p, at in (("x", 8), ("q", G + 8), ("s", 2 * G + 1), ("c", 3 * G + 8), ("cs", 4 * G + 2)):
        assert swiglu(lib, **{p: A + at}) == EALIGN, p
    for p in ("q", "s", "c", "cs"):
        assert swiglu(lib, **{p: A + 2048}) == EOVERLAP, p  # inside x
    assert swiglu(lib, c=A + G) == EOVERLAP
    assert swiglu(lib, cs=A + 2 * G) == EOVERLAP
    assert swiglu_grad(lib, dx=None, q=None, s=None) == EINVAL
    assert swiglu_grad(lib, q=None) == EINVAL
    for p in ("dy", "c", "cs"):
        assert swiglu_grad(lib, **{p: None}) == EINVAL, p
    for p, at in (("dy", 8), ("c", G + 8), ("cs", 2 * G + 2), ("dx", 3 * G + 8), ("q", 4 * G + 4), ("s", 5 * G + 1)):
        assert swiglu_grad(lib, **{p: A + at}) == EALIGN, p
    for p in ("dx", "q", "s"):
        for at in (A, A + G, A + 2 * G):
            assert swiglu_grad(lib, **{p: at}) == EOVERLAP, p
    assert swiglu_grad(lib, q=A + 3 * G) == EOVERLAP


def balance(lib, x=A, dt=1, idx=A + G, isz=8, mask=A + 2 * G, t=40, e=8, k=2, coef=1.0, loss=A + 3 * G, c=A + 4 * G,
            off=A + 5 * G, v=A + 6 * G, ws=A + 7 * G, wn=1 << 20):
    return lib.router_balance(x, dt, idx, isz, mask, t, e, k, coef, loss, c, off, v, ws, wn, None)


def balance_grad(lib, x=A, dt=1, v=A + G, dl=A + 2 * G, mask=A + 3 * G, add=A + 4 * G, t=40, e=8, out=A + 5 * G):
    return lib.router_balance_backward(x, dt, v, dl, mask, add, t, e, out, None)


def test_router(lib):
    for call in (balance, balance_grad):
        assert call(lib, dt=2) == EDTYPE
        for e in (0, -1, 4097):
            assert call(lib, e=e) == ESHAPE, e
        assert call(lib, t=-1) == ESHAPE
        assert call(lib, t=1 << 31) == ESHAPE
    for isz in (0, 2, 16):
        assert balance(lib, isz=isz) == EINVAL
    for coef in (float("inf"), float("-inf"), float("nan")):
        assert balance(lib, coef=coef) == EINVAL
    assert balance(lib, k=0) == ESHAPE
    assert balance(lib, t=1 << 30, k=2, wn=1 << 40) == ESHAPE
    need = lib.router_balance_workspace(40, 8)
    assert need > 0 and balance(lib, wn=need - 1) == ESHAPE
    for t, e in ((-1, 8), (1 << 31, 8), (4, 0), (4, 4097)):
        assert lib.router_balance_workspace(t, e) == 0
    for p in ("x", "idx", "loss", "c", "off", "v", "ws"):
        assert balance(lib, **{p: None}) == EINVAL, p
    for p, at in (("x", 1), ("idx", G + 4), ("loss", 3 * G + 2), ("c", 4 * G + 2), ("off", 5 * G + 4), ("v", 6 * G + 2),
                  ("ws", 7 * G + 8)):
        assert balance(lib, **{p: A + at}) == EALIGN, p
    for p in ("loss", "c", "off", "v", "ws"):
        for at in (A, A + G):
            assert balance(lib, **{p: at}) == EOVERLAP, p
    assert balance(lib, loss=A + 2 * G + 36) == EOVERLAP    # the mask's last bytes
    assert balance(lib, v=A + 4 * G + 16) == EOVERLAP
    assert balance(lib, ws=A + 6 * G) == EOVERLAP
    assert balance_grad(lib, t=0, x=None, v=None, out=None) == OK
    for p in ("x", "v", "out"):
        assert balance_grad(lib, **{p: None}) == EINVAL, p
    for p, at in (("x", 1), ("v", G + 2), ("dl", 2 * G + 2), ("add", 4 * G + 1), ("out", 5 * G + 1)):
        assert balance_grad(lib, **{p: A + at}) == EALIGN, p
    assert balance_grad(lib, out=A + 2) == EOVERLAP         # neither x itself
    assert balance_grad(lib, out=A + 4 * G + 16) == EOVERLAP
    for at in (G, 2 * G, 3 * G):
        assert balance_grad(lib, out=A + at) == EOVERLAP


def test_header_compiles_as_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "h.c"
    src.write_text('#include "fp4mi_moe.h"\nint main(void) { return router_balance_workspace(0, 0) != 0; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), LIB, "-o", str(tmp_path / "h")], check=True)


@pytest.mark.skipif(SANITIZED is not None, reason="already the sanitized run")
def test_validation_under_sanitizers(tmp_path):
    """The same validation tests against host code built with AddressSanitizer and
    UBSan (device code compiled as usual and never run)."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    lib = str(tmp_path / "libmoe_san.so")
    env = dict(os.environ)
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared", "-ffp-contract=off",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-command-line-argument",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
                    "-fno-sanitize-recover=all", "-shared-libsan", "-I", os.path.join(ROOT, "include"),
                    *[os.path.join(CSRC, s) for s in ("fp8quant.hip", "fp8mat.hip", "swiglu.hip", "router.hip", "abi.hip")],
                    "-o", lib], check=True, capture_output=True, env=env)
    clang = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "clang")
    rt = subprocess.run([clang, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(rt):
        rt = subprocess.run([clang, "-print-file-name=libclang_rt.asan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.exists(rt):
        pytest.skip("no shared ASan runtime")
    env.update(FP4MI_SANITIZED_MOE_LIB=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__), "-k",
                        "test_quantizers or test_products or test_swiglu or test_router"], capture_output=True, text=True, env=env)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]


@pytest.mark.skipif(SANITIZED is not None, reason="the plain library's run")
def test_the_binding_refuses():
    import block_scaled_fp4_amd as m
    u8, f32, i64 = torch.uint8, torch.float32, torch.int64
    cpu = lambda dt, *shape: torch.zeros(shape, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="on the GPU"):
        m.fp8_quantize(cpu(f32, 4, 128))
    with pytest.raises(ValueError, match="on the GPU"):
        m.fp8_quantize_blocks(cpu(f32, 4, 128))
    with pytest.raises(ValueError, match="on the GPU"):
        m.fp8_matmul(cpu(u8, 4, 128), cpu(f32, 4, 1), cpu(u8, 8, 128), cpu(f32, 8, 1))
    with pytest.raises(ValueError, match="on the GPU"):
        m.swiglu_quantize(cpu(f32, 4, 256))
    with pytest.raises(ValueError, match="on the GPU"):
        m.swiglu_backward(cpu(f32, 4, 128), cpu(u8, 4, 256), cpu(f32, 4, 2))
    with pytest.raises(ValueError, match="on the GPU"):
        m.router_balance(cpu(f32, 4, 8), cpu(i64, 4, 2))
    with pytest.raises(ValueError, match="on the GPU"):
        m.router_balance_backward(cpu(f32, 4, 8), cpu(f32, 8))
    with pytest.raises(ValueError, match="columns"):
        m.fp8_matmul(cpu(u8, 4, 128), cpu(f32, 4, 1), cpu(u8, 8, 256), cpu(f32, 8, 2))
    with pytest.raises(ValueError, match="rows of blocks"):
        m.fp8_matmul(cpu(u8, 4, 128), cpu(f32, 4, 1), cpu(u8, 300, 128), cpu(f32, 2, 1))
    with pytest.raises(ValueError, match="b must be"):
        m.fp8_matmul(cpu(u8, 4, 128), cpu(f32, 4, 1), cpu(u8, 1, 8, 128), cpu(f32, 8, 1))
    with pytest.raises(ValueError, match="token_offsets"):
        m.fp8_matmul_grouped(cpu(u8, 4, 128), cpu(f32, 4, 1), cpu(u8, 1, 8, 128), cpu(f32, 1, 8, 1), None)
    with pytest.raises(ValueError, match="2 ffn"):
        m.swiglu_quantize(cpu(f32, 4, 257))
    with pytest.raises(ValueError, match="fmt is required"):
        m.swiglu_backward(cpu(f32, 4, 128), cpu(u8, 4, 256), cpu(f32, 4, 2), q=cpu(u8, 4, 256))


@pytest.mark.skipif(SANITIZED is not None, reason="the plain library's run")
def test_the_binding_checks_each_tensor(monkeypatch):
    """Types, sizes, strides and devices, on fake tensors of a GPU, with no launch."""
    import block_scaled_fp4_amd as m
    monkeypatch.setattr(m, "_lib", type("Stub", (), {"__getattr__": lambda s, n: (lambda *a: 4096 if "workspace" in n else pytest.fail(n))})())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 4096)
    u8, f32, i64 = torch.uint8, torch.float32, torch.int64
    with FakeTensorMode(allow_non_fake_inputs=True):
        t = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda:0")  # noqa: E731
        x, a, s, w, ws = t(f32, 4, 256), t(u8, 4, 256), t(f32, 4, 2), t(u8, 8, 256), t(f32, 8, 2)
        bad = [
            (TypeError, lambda: m.fp8_quantize(x, q=t(f32, 4, 256))),
            (ValueError, lambda: m.fp8_quantize(x, scales=t(f32, 4, 1))),
            (ValueError, lambda: m.fp8_quantize(t(f32, 256, 4).t())),
            (ValueError, lambda: m.fp8_quantize_blocks(t(f32, 256, 256), q_t=t(u8, 256, 255))),
            (ValueError, lambda: m.fp8_matmul(a, t(f32, 4, 1), w, ws)),
            (TypeError, lambda: m.fp8_matmul(a, t(u8, 4, 2), w, ws)),
            (ValueError, lambda: m.fp8_matmul(a, s, w, ws, a_row_scale=t(f32, 3))),
            (ValueError, lambda: m.fp8_matmul(a, s, w, ws, out=t(f32, 4, 7))),
            (ValueError, lambda: m.fp8_matmul(t(u8, 256, 4).t(), s, w, ws)),
            (TypeError, lambda: m.fp8_matmul_grouped(a, s, w.view(2, 4, 256), ws.view(2, 4, 2), t(torch.int32, 3))),
            (ValueError, lambda: m.fp8_matmul_grouped(a, s, w.view(2, 4, 256), ws.view(2, 4, 2), t(i64, 2))),
            (ValueError, lambda: m.swiglu_quantize(x, ckpt=t(u8, 4, 255))),
            (TypeError, lambda: m.swiglu_quantize(x, "mxfp4", scales=t(f32, 4, 4))),
            (ValueError, lambda: m.swiglu_backward(x, t(u8, 4, 256), t(f32, 4, 4))),
            (TypeError, lambda: m.swiglu_backward(x, t(u8, 4, 512), t(f32, 4, 4), dx=t(torch.bfloat16, 4, 512))),
            (ValueError, lambda: m.router_balance(x, t(i64, 3, 2))),
            (TypeError, lambda: m.router_balance(x, t(torch.int16, 4, 2))),
            (ValueError, lambda: m.router_balance(x, t(i64, 4, 2), mask=t(torch.bool, 3))),
            (TypeError, lambda: m.router_balance(x, t(i64, 4, 2), mask=t(f32, 4))),
            (TypeError, lambda: m.router_balance_backward(x, t(f32, 256), add=t(torch.bfloat16, 4, 256))),
            (ValueError, lambda: m.router_balance_backward(x, t(f32, 255))),
        ]
        for kind, call in bad:
            with pytest.raises(kind):
                call()
        for call in (lambda: m.fp8_quantize(x), lambda: m.fp8_quantize_blocks(x), lambda: m.fp8_matmul(a, s, w, ws),
                     lambda: m.swiglu_quantize(x), lambda: m.router_balance(x, t(i64, 4, 2)),
                     lambda: m.router_balance_backward(x, t(f32, 256))):
            with pytest.raises(ValueError, match="not the current one"):
                call()

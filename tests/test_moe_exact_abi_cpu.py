"""FP4_EXACT of the FP8 products: what the library accepts and refuses, and what the
binding hands it."""
import ctypes
import os
import re

import torch
from torch._subclasses.fake_tensor import FakeTensorMode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, G = 0x7F0000000000, 1 << 30
OK, EINVAL, ESHAPE, EALIGN, EDTYPE, EHIP, EOVERLAP = range(7)


def test_header_and_binding_agree():
    import block_scaled_fp4_amd as m
    text = open(os.path.join(ROOT, "include", "fp4mi_moe.h")).read()
    assert int(re.search(r"#define FP4_EXACT (0x[0-9a-f]+)", text).group(1), 16) == m.EXACT == 0x100


def test_status():
    lib = ctypes.CDLL(os.path.join(ROOT, "block_scaled_fp4_amd", "libfp4mi.so"))
    P, I, I32, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64
    lib.fp8_matmul.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, I, P]
    lib.fp8_matmul_grouped.argtypes = [P, P, P, P, P, I, P, I32, I64, I64, I64, P, I, P]

    def dense(dt, m=4, out=A + 5 * G):
        return lib.fp8_matmul(A, A + G, A + 2 * G, A + 3 * G, A + 4 * G, 1, m, 8, 256, out, dt, None)

    def grouped(dt, m=4, out=A + 5 * G):
        return lib.fp8_matmul_grouped(A, A + G, A + 2 * G, A + 3 * G, A + 4 * G, 128, A + 6 * G, 3, m, 8, 256, out, dt, None)
    for call in (dense, grouped):
        for dt in (0x100, 0x101):
            assert call(dt, m=0) == OK                       # nothing to do, everything checked
            assert call(dt, out=None) == EINVAL
            assert call(dt, out=A + 5 * G + 8) == EALIGN
            assert call(dt, out=A + G) == EOVERLAP
        for dt in (0x102, 0x201, 0x200, 0x80, 0x11, -1):
            assert call(dt, m=0) == EDTYPE, dt
    # the last of the output's 4 x 8 x 2 bytes
    assert dense(0x101, out=A + G - 4 * 8 * 2 + 16) == EOVERLAP


def test_binding_passes_it_on(monkeypatch):
    import block_scaled_fp4_amd as m
    seen = []

    class Stub:
        def fp8_matmul(self, *a):
            seen.append(a[-2])
            return 0

        def fp8_matmul_grouped(self, *a):
            seen.append(a[-2])
            return 0
    monkeypatch.setattr(m, "_lib", Stub())
    monkeypatch.setattr(m, "_stream_on", lambda gpu, stream: None)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 4096)
    with FakeTensorMode(allow_non_fake_inputs=True):
        t = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda:0")  # noqa: E731
        a, s, w, ws = t(torch.uint8, 4, 256), t(torch.float32, 4, 2), t(torch.uint8, 8, 256), t(torch.float32, 8, 2)
        off = t(torch.int64, 3)
        for out, code in ((torch.bfloat16, 1), (torch.float32, 0)):
            m.fp8_matmul(a, s, w, ws, out_dtype=out)
            m.fp8_matmul(a, s, w, ws, out_dtype=out, exact=True)
            m.fp8_matmul_grouped(a, s, w.view(2, 4, 256), ws.view(2, 4, 2), off, out_dtype=out)
            m.fp8_matmul_grouped(a, s, w.view(2, 4, 256), ws.view(2, 4, 2), off, out_dtype=out, exact=True)
            assert seen[-4:] == [code, code | 0x100] * 2
        m.fp8_matmul(a, s, w, ws, out_dtype=torch.float16, exact=True)
        assert seen[-1] & ~0x100 not in (0, 1)               # no type of the library's with the flag either

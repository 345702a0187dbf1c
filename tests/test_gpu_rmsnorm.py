"""rmsnorm_quantize and rmsnorm_backward: codes and block scales bit for bit
against the oracle's quantizer on z = fl32(h w), row factors and gradients
against 64 bits within derived bounds, and against differences.

Bounds: a sum of n fp32 terms in any order errs by at most n 2^-24 of the sum
of magnitudes.  row_scale = (s/n + eps)^-1/2 then errs by (n + 8) 2^-24 / 2
relatively; the bound used is (n + 8) 2^-24.  dx: the mean of g h errs by
(n + 8) 2^-24 mean|g h|, times r^3 |h|, and a few roundings of each term.
dweight: (rows + 8) 2^-24 sum|dy h r|."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import Guarded, dev_bf16, dev_f32, host, host_bf16, need_gpu
from oracle import formats as F
from oracle import mxfp4

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def dev(x, dt):
    return dev_bf16(F.f32_to_bf16_bits(x)) if dt == "bf16" else dev_f32(x)


def rounded(x, dt):
    return F.bf16_bits_to_f32(F.f32_to_bf16_bits(x)) if dt == "bf16" else x.astype(np.float32)


def back(t):
    return F.bf16_bits_to_f32(host_bf16(t)) if t.dtype == torch.bfloat16 else host(t)


def inputs(rng, rows, cols, dt, wdt):
    x = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, 1)))
    x[:, rng.integers(0, cols, max(1, cols // 300))] *= 40.0
    x[rng.random((rows, cols)) < 0.02] = 0.0
    if rows > 2:
        x[rows // 2] = 0.0                                # a row of zeros
    if cols >= 256:
        x[0, :128] = 0.0                                  # a block of zeros
    w = 1.0 + 0.3 * rng.standard_normal(cols)
    return rounded(x.astype(np.float32), dt), rounded(w.astype(np.float32), wdt)


def check_forward(m, x, w, res, dt, wdt, fmt, eps=1e-6, h_over=None):
    rows, cols = x.shape
    print(f"norm {rows}x{cols} {dt} w {wdt} {fmt} res={res is not None} {h_over}", flush=True)
    h = x if res is None else rounded(x + res, dt)
    z = h * w
    if fmt == "fp8":
        q_ref, s_ref = R.fp8_block_quantize(z)
        gq, gs = Guarded(rows * cols), Guarded(rows * cols // 128 * 4)
        q, s = gq.view(torch.uint8, (rows, cols)), gs.view(torch.float32, (rows, cols // 128))
    else:
        q_ref, s_ref = mxfp4.quantize_packed(z)
        gq, gs = Guarded(rows * cols // 2), Guarded(rows * cols // 32)
        q, s = gq.view(torch.uint8, (rows, cols // 2)), gs.view(torch.uint8, (rows, cols // 32))
    gr = Guarded(rows * 4)
    xd, rd = dev(x, dt), None if res is None else dev(res, dt)
    hd = {"x": xd, "res": rd, None: None}[h_over]
    q, s, r, ho = m.rmsnorm_quantize(xd, dev(w, wdt), residual=rd, eps=eps, fmt=fmt, q=q, scales=s,
                                     row_scale=gr.view(torch.float32, (rows,)), h=hd)
    torch.cuda.synchronize()
    for g in (gq, gs, gr):
        g.check()
    np.testing.assert_array_equal(back(ho), h)
    np.testing.assert_array_equal(host(q), q_ref)
    np.testing.assert_array_equal(host(s), s_ref)
    want = (np.square(h.astype(np.float64)).mean(-1) + np.float64(np.float32(eps))) ** -0.5
    assert (np.abs(host(r) - want) <= (cols + 8) * E * want).all()


@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 7168), (3, 256), (4, 512), (5, 640), (37, 2048), (130, 1152), (3, 16512),
                                       (2, 33024)])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_forward(rows, cols, fmt, dt, wdt):
    m = need_gpu()
    rng = np.random.default_rng(rows + cols)
    x, w = inputs(rng, rows, cols, dt, wdt)
    res = rounded(rng.standard_normal((rows, cols)).astype(np.float32), dt) if (rows + cols) % 3 else None
    if res is not None and cols >= 256:
        res[0, :128] = 0.0
    check_forward(m, x, w, res, dt, wdt, fmt)


@pytest.mark.parametrize("rows,cols", [(1, 32), (2, 96), (7, 160), (9, 2080)])
def test_forward_mxfp4_odd_widths(rows, cols):
    m = need_gpu()
    rng = np.random.default_rng(cols)
    x, w = inputs(rng, rows, cols, "bf16", "f32")
    check_forward(m, x, w, x[::-1].copy(), "bf16", "f32", "mxfp4")


@pytest.mark.parametrize("h_over", ["x", "res"])
def test_forward_sum_in_place(h_over):
    m = need_gpu()
    rng = np.random.default_rng(12)
    x, w = inputs(rng, 9, 1024, "bf16", "f32")
    check_forward(m, x, w, x[:, ::-1].copy(), "bf16", "f32", "fp8", h_over=h_over)


def test_forward_many_rows():
    m = need_gpu()
    rng = np.random.default_rng(13)
    x, w = inputs(rng, 4100, 384, "bf16", "f32")
    check_forward(m, x, w, None, "bf16", "f32", "fp8")
    check_forward(m, x, w, x[::-1].copy(), "bf16", "f32", "mxfp4")


def test_forward_scale_boundaries():
    """Block maxima just below, at and just above 448 * 2^k and 2^k."""
    m = need_gpu()
    rows, cols = 64, 256
    x = np.full((rows, cols), 1.0, np.float32) * np.float32(1e-3)
    for i in range(rows):
        k = i - 32
        for b, v in enumerate((448.0, 512.0)):
            t = np.float32(v * 2.0 ** k)
            x[i, 128 * b + i] = (np.nextafter(t, np.float32(0)), t, np.nextafter(t, np.float32(np.inf)))[i % 3]
    w = np.ones(cols, np.float32)
    check_forward(m, x, w, None, "f32", "f32", "fp8")
    check_forward(m, x, w, None, "f32", "f32", "mxfp4")


def test_forward_tiny_and_huge():
    """Values near both ends of fp32's exponents (squares of the row may leave
    fp32's range, so only codes and block scales are compared)."""
    m = need_gpu()
    rng = np.random.default_rng(14)
    x = rng.standard_normal((6, 256))
    x *= np.exp2(np.array([-140, -126, -100, 60, 110, 124]))[:, None]
    x = x.astype(np.float32)
    w = np.ones(256, np.float32)
    for fmt in ("fp8", "mxfp4"):
        q, s, _, _ = m.rmsnorm_quantize(dev_f32(x), dev_f32(w), fmt=fmt)
        torch.cuda.synchronize()
        qr, sr = R.fp8_block_quantize(x) if fmt == "fp8" else mxfp4.quantize_packed(x)
        np.testing.assert_array_equal(host(s), sr)
        np.testing.assert_array_equal(host(q), qr)


def check_backward(m, rng, rows, cols, dt, wdt, with_dh, dx_over=None):
    print(f"norm grad {rows}x{cols} {dt} w {wdt} dh={with_dh} {dx_over}", flush=True)
    h, w = inputs(rng, rows, cols, dt, wdt)
    dy = rounded((1e-2 * rng.standard_normal((rows, cols))).astype(np.float32), dt)
    dh = rounded((1e-2 * rng.standard_normal((rows, cols))).astype(np.float32), dt) if with_dh else None
    r = ((np.square(h.astype(np.float64)).mean(-1) + 1e-6) ** -0.5).astype(np.float32)
    sz = 2 if dt == "bf16" else 4
    gx, gw, gs = Guarded(rows * cols * sz), Guarded(cols * 4), Guarded(m.rmsnorm_backward_workspace(rows, cols))
    dyd, dhd = dev(dy, dt), None if dh is None else dev(dh, dt)
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    dxd = {"dy": dyd, "dh": dhd, None: gx.view(tdt, (rows, cols))}[dx_over]
    dx, dw = m.rmsnorm_backward(dyd, dev(h, dt), dev(w, wdt), dev_f32(r), dh=dhd, dx=dxd,
                                dweight=gw.view(torch.float32, (cols,)), workspace=gs.view(torch.uint8, (gs.nbytes,)))
    torch.cuda.synchronize()
    for g in (gx, gw, gs):
        g.check()
    dx_ref, dw_ref = R.rmsnorm_backward(dy, h, w, r, dh)
    g64, h64, r64 = dy.astype(np.float64) * w, h.astype(np.float64), r.astype(np.float64)[:, None]
    size = r64 * (np.abs(g64) + np.abs(h64) * r64 ** 2 * np.abs(g64 * h64).mean(-1, keepdims=True))
    tol = (cols + 16) * E * r64 ** 3 * np.abs(h64) * np.abs(g64 * h64).mean(-1, keepdims=True) + 8 * E * size
    tol += (2.0 ** -8 if dt == "bf16" else 2 * E) * np.abs(dx_ref) + 2 * E * (0 if dh is None else np.abs(dh))
    assert (np.abs(back(dx) - dx_ref) <= tol + 2.0 ** -126).all()
    tol_w = (rows + 8) * E * np.abs(dy * h64 * r64).sum(0)
    assert (np.abs(host(dw) - dw_ref) <= tol_w + 2.0 ** -126).all()


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (2, 96), (3, 512), (33, 2048), (130, 1056), (333, 256), (600, 640),
                                       (3, 16512), (2, 33024)])
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(rows, cols, dt, wdt, with_dh):
    m = need_gpu()
    check_backward(m, np.random.default_rng(rows + cols), rows, cols, dt, wdt, with_dh)


@pytest.mark.parametrize("dx_over", ["dy", "dh"])
def test_backward_in_place(dx_over):
    m = need_gpu()
    check_backward(m, np.random.default_rng(1), 70, 1024, "bf16", "f32", True, dx_over)


def test_backward_many_rows():
    m = need_gpu()
    check_backward(m, np.random.default_rng(2), 5001, 384, "bf16", "f32", True)


def test_backward_against_differences():
    """Central differences of L = sum(c * h * w / rms(h)) in 64 bits."""
    m = need_gpu()
    rng = np.random.default_rng(3)
    rows, cols = 3, 64
    h = rng.standard_normal((rows, cols)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    c = rng.standard_normal((rows, cols)).astype(np.float32)

    def loss(h, w):
        return (c * h * w * (np.square(h).mean(-1, keepdims=True) + 1e-6) ** -0.5).sum()

    r = ((np.square(h.astype(np.float64)).mean(-1) + 1e-6) ** -0.5).astype(np.float32)
    dx, dw = m.rmsnorm_backward(dev_f32(c), dev_f32(h), dev_f32(w), dev_f32(r))
    torch.cuda.synchronize()
    dx, dw, d = host(dx), host(dw), 1e-5
    h64, w64 = h.astype(np.float64), w.astype(np.float64)
    for i in range(rows):
        for j in range(0, cols, 7):
            e = np.zeros_like(h64)
            e[i, j] = d
            assert abs((loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * d) - dx[i, j]) < 2e-5
    for j in range(cols):
        e = np.zeros(cols)
        e[j] = d
        assert abs((loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * d) - dw[j]) < 2e-5


def test_backward_no_rows_gives_zero_dweight():
    m = need_gpu()
    z = torch.empty((0, 64), device="cuda")
    dx, dw = m.rmsnorm_backward(z, z, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_forward_no_rows():
    m = need_gpu()
    z = torch.empty((0, 128), device="cuda")
    q, s, r, h = m.rmsnorm_quantize(z, torch.ones(128, device="cuda"))
    assert q.shape == (0, 128) and s.shape == (0, 1) and r.shape == (0,) and h is z


def test_binding_refuses():
    m = need_gpu()
    x = torch.zeros((4, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    r = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        m.rmsnorm_quantize(x, w[:128].contiguous())
    with pytest.raises(TypeError):
        m.rmsnorm_quantize(x, w, residual=x.to(torch.bfloat16))
    with pytest.raises(m.Fp4Error):
        m.rmsnorm_quantize(x, w, fmt="int8")
    with pytest.raises(m.Fp4Error):
        m.rmsnorm_quantize(x, w, eps=float("nan"))
    with pytest.raises(m.Fp4Error):
        m.rmsnorm_quantize(x, w, eps=-1.0)
    with pytest.raises(m.Fp4Error):                                 # 192 is no multiple of 128
        m.rmsnorm_quantize(x[:, :192].contiguous(), w)
    with pytest.raises(m.Fp4Error):
        m.rmsnorm_quantize(x.half(), w)
    with pytest.raises(ValueError):
        m.rmsnorm_backward(x, x, w, r, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        m.rmsnorm_backward(x, x[:2].contiguous(), w, r)
    with pytest.raises(m.Fp4Error):                                 # dx over h
        m.rmsnorm_backward(x, r.new_zeros((4, 256)), w, r, dx=w.new_zeros(1030)[6:].view(4, 256))

"""SwiGLU into quantized rows with its FP8 checkpoint, and the gradient from it.

y passes through an exponential of 2 last places, a sum, a reciprocal and two
products: under 6 of fp32's last places (2^-24 each), SLACK allows 16.  In dx the
two terms of 1 + g (1 - s) may cancel, so its bound is on their sizes."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import Guarded, dev_f32, dev_u8, host, need_gpu
from oracle import formats as F

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -20
TINY = 2.0 ** -100                # exp(-g) past fp32 makes y zero below this


def inputs(rng, rows, ffn, bf16, size=2.0):
    x = rng.standard_normal((rows, 2 * ffn)) * size * np.exp(rng.standard_normal((rows, 1)))
    x[:, ::37] *= 20
    x[rows // 2, :ffn] = 0
    if rows > 4:
        x[1, :ffn], x[2, :ffn], x[3, ffn:] = -200.0, 90.0, 0.0
    t = torch.from_numpy(x.astype(np.float32))
    t = t.to(torch.bfloat16) if bf16 else t
    return t.cuda(), t.double().numpy()


def row_bufs(rows, width, fmt):
    n = rows * width
    if fmt == "fp8":
        return Guarded(n), Guarded(n // 32), (torch.uint8, (rows, width)), (torch.float32, (rows, width // 128))
    return Guarded(n // 2), Guarded(n // 32), (torch.uint8, (rows, width // 2)), (torch.uint8, (rows, width // 32))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("rows,ffn", [(1, 128), (1, 2048), (3, 8192), (5, 384), (33, 640), (300, 256), (17, 8320), (2, 393344)])
def test_forward(rows, ffn, fmt, bf16):
    m = need_gpu()
    x, v = inputs(np.random.default_rng(rows + ffn), rows, ffn, bf16)
    qb, sb, qv, sv = row_bufs(rows, ffn, fmt)
    cb, tb = Guarded(rows * 2 * ffn), Guarded(rows * 2 * ffn // 32)
    q, s, c, t = m.swiglu_quantize(x, fmt, True, qb.view(*qv), sb.view(*sv), cb.view(torch.uint8, (rows, 2 * ffn)),
                                   tb.view(torch.float32, (rows, 2 * ffn // 128)))
    torch.cuda.synchronize()
    for b in (qb, sb, cb, tb):
        b.check()
    rc, rt = R.fp8_quantize(v)
    np.testing.assert_array_equal(host(t), rt)
    np.testing.assert_array_equal(host(c), rc)
    R.assert_rows(host(q), host(s), R.swiglu(v), fmt, SLACK, TINY)
    q2, s2, c2, t2 = m.swiglu_quantize(x, fmt, checkpoint=False)          # nothing kept, the same rows
    assert c2 is None and t2 is None and torch.equal(q2, q) and torch.equal(s2, s)


def test_forward_mxfp4_width():
    """Without a checkpoint MXFP4 rows take widths of 32."""
    m = need_gpu()
    x, v = inputs(np.random.default_rng(0), 7, 160, True)
    q, s, _, _ = m.swiglu_quantize(x, "mxfp4", checkpoint=False)
    R.assert_rows(host(q), host(s), R.swiglu(v), "mxfp4", SLACK, TINY)


def kept(rng, rows, ffn):
    _, v = inputs(rng, rows, ffn, False)
    c, s = R.fp8_quantize(v)
    return c, s, R.values(c, s)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("fmt", [None, "fp8", "mxfp4"])
@pytest.mark.parametrize("rows,ffn", [(1, 128), (1, 2048), (3, 8192), (5, 384), (33, 640), (300, 256), (17, 8320), (2, 393344)])
def test_backward(rows, ffn, fmt, bf16):
    m = need_gpu()
    rng = np.random.default_rng(rows * ffn)
    c, s, x = kept(rng, rows, ffn)
    dy = torch.from_numpy((1e-3 * rng.standard_normal((rows, ffn))).astype(np.float32))
    dy = dy.to(torch.bfloat16) if bf16 else dy
    dx, size = R.swiglu_backward(x, dy.double().numpy())
    dxb = Guarded(rows * 2 * ffn * (2 if bf16 else 4))
    dxv = dxb.view(dy.dtype, (rows, 2 * ffn))
    args = dy.cuda(), dev_u8(c), dev_f32(s)
    if fmt is None:
        m.swiglu_backward(*args, dx=dxv)
    else:
        qb, sb, qv, sv = row_bufs(rows, 2 * ffn, fmt)
        _, q, t = m.swiglu_backward(*args, fmt, dxv, qb.view(*qv), sb.view(*sv))
        torch.cuda.synchronize()
        qb.check()
        sb.check()
        # the rows' own bound allows for cancellation: floor is the largest of it
        R.assert_rows(host(q), host(t), dx, fmt, SLACK, float((SLACK * size).max()) + TINY)
        none, q2, t2 = m.swiglu_backward(*args, fmt)
        assert none is None and torch.equal(q2, q) and torch.equal(t2, t)
    torch.cuda.synchronize()
    dxb.check()
    got = dxv.double().cpu().numpy()
    tol = SLACK * size + TINY + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(dx)
    assert (np.abs(got - dx) <= tol).all(), float((np.abs(got - dx) / tol).max())


def test_gradient_against_differences():
    """Central differences of the formula in 64 bits at the checkpoint's values:
    error h^2/6 of a third derivative (below 0.3 |u|), rounding eps/h."""
    m = need_gpu()
    rng = np.random.default_rng(5)
    c, s, x = kept(rng, 6, 256)
    dy = rng.standard_normal((6, 256)).astype(np.float32)
    got = m.swiglu_backward(dev_f32(dy), dev_u8(c), dev_f32(s))[0].double().cpu().numpy()
    h = 1e-4
    for half in (0, 1):
        d = np.zeros_like(x)
        d[:, 256 * half:256 * (half + 1)] = h
        slope = dy * (R.swiglu(x + d) - R.swiglu(x - d)) / (2 * h)
        _, size = R.swiglu_backward(x, dy)
        part = slice(256 * half, 256 * (half + 1))
        tol = SLACK * size[:, part] + np.abs(dy) * (np.abs(x[:, 256:]) * h * h + 1e-11 * (1 + np.abs(x[:, :256] * x[:, 256:])))
        assert (np.abs(got[:, part] - slope) <= tol).all()


def test_forward_then_backward():
    """The forward's checkpoint into the backward: off by the checkpoint's 2^-4."""
    m = need_gpu()
    x = torch.randn((40, 512), device="cuda").to(torch.bfloat16)
    dy = torch.randn((40, 256), device="cuda").to(torch.bfloat16)
    _, _, c, s = m.swiglu_quantize(x)
    dx = m.swiglu_backward(dy, c, s)[0]
    v = x.double().requires_grad_()
    (torch.nn.functional.silu(v[:, :256]) * v[:, 256:]).backward(dy.double())
    assert float((dx.double() - v.grad).norm() / v.grad.norm()) < 0.05
    assert float((dx.double() - v.grad).norm() / v.grad.norm()) > 0      # from the checkpoint, not from x


def test_nan_stays_in_its_place():
    m = need_gpu()
    x = torch.randn((2, 512), device="cuda")
    x[0, 3], x[1, 256 + 130] = float("nan"), float("nan")
    q, s, c, t = m.swiglu_quantize(x)
    assert torch.isnan(q.view(torch.float8_e4m3fn).float()).nonzero().tolist() == [[0, 3], [1, 130]]
    assert torch.isnan(c.view(torch.float8_e4m3fn).float()).nonzero().tolist() == [[0, 3], [1, 386]]
    dx = m.swiglu_backward(torch.ones((2, 256), device="cuda"), c, t)[0]
    assert torch.isnan(dx).nonzero().tolist() == [[0, 3], [0, 259], [1, 130]]    # u does not reach its own gradient


def test_empty():
    m = need_gpu()
    q, s, c, t = m.swiglu_quantize(torch.empty((0, 512), device="cuda"))
    assert q.shape == (0, 256) and c.shape == (0, 512)
    assert m.swiglu_backward(torch.empty((0, 256), device="cuda"), c, t)[0].shape == (0, 512)

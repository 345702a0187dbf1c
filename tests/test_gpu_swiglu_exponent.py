"""SwiGLU's exponential over the whole range of a gate: bf16 gradients and rows are the
nearest values, unless the formula comes within 16 of fp32's last places (2^-24 each) of a
border: exp 5 (exp2 itself 2, its correction and that one's square 3), the sum 1, the
reciprocal 2, three or four products and 1 + g (1 - s) one each.  An argument of exp2 that is
rounded once is off by |g| 2^-24, 60 of these last places."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import dev_f32, dev_u8, host, need_gpu

pytestmark = pytest.mark.gpu
NEAR = 16 * 2.0 ** -24


def bf16_border(x):
    """Relative distance of |x| (normal) from the nearest middle between two bf16 values."""
    m, e = np.frexp(np.abs(x))
    q = m * 256                                    # 8 significant bits: [128, 256)
    return np.abs(q / (np.floor(q) + 0.5) - 1)


def nearest_bf16(x):
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)       # to even


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_gradient_is_the_nearest_bf16_value(sign):
    """Every E4M3 mantissa of g from 2^-3 to 87, of u, and every bf16 mantissa of dy.  The term
    of dg where 1 + g (1 - s) cancels is left out: its error is relative to the terms."""
    m = need_gpu()
    mant = 1 + np.arange(8) / 8
    g = np.concatenate([mant * 2.0 ** e for e in range(-3, 7)])
    g = sign * g[g <= 80]
    dy = (1 + np.arange(128) / 128).astype(np.float32)
    rows = len(g) * 8
    gg, uu = np.repeat(g, 8), np.tile(mant, len(g))
    x = np.concatenate([np.repeat(gg[:, None], 128, 1), np.repeat(uu[:, None], 128, 1)], 1)
    # a row has one g: its codes and scale hold it exactly
    c, s = R.fp8_quantize(x)
    np.testing.assert_array_equal(R.values(c, s), x)
    d = np.repeat(dy[None], rows, 0)
    got = m.swiglu_backward(dev_f32(d).to(torch.bfloat16), dev_u8(c), dev_f32(s))[0].double().cpu().numpy()
    dx, size = R.swiglu_backward(x, d)
    sure = (bf16_border(dx) > NEAR) & (size < 1.5 * np.abs(dx))
    assert sure.mean() > 0.75                      # below -5 all but those near a border
    bad = sure & (got != nearest_bf16(dx))
    assert not bad.any(), (int(bad.sum()), [(x[i, 0], x[i, 255], d[i, j % 128]) for i, j in np.argwhere(bad)[:4]])


def test_rows_hold_the_nearest_codes():
    """Forward: every bf16 gate from 2^-6 to 87 of either sign beside one mantissa of u a row; y
    alone is the largest of its block, and its code the nearest unless y lies within
    16 last places of a border."""
    m = need_gpu()
    bits = np.arange(0x3C80, 0x42AF, dtype=np.uint32) << 16
    g = bits.view(np.float32)
    g = np.concatenate([g, -g])
    for mant in range(0, 128, 5):
        x = np.zeros((len(g), 256), np.float32)
        x[:, 7], x[:, 128 + 7] = g, 1 + mant / 128
        q, s, _, _ = m.swiglu_quantize(dev_f32(x).to(torch.bfloat16), checkpoint=False)
        y = R.swiglu(x)[:, 7]
        a = np.abs(y)
        k = R.least_exponent(a)
        t = a * np.exp2(-k.astype(np.float64))     # (224, 448]
        step = np.exp2(np.floor(np.log2(t)) - 3)
        sure = (np.abs(t / ((np.floor(t / step) + 0.5) * step) - 1) > NEAR) & (np.abs(t / 448 - 1) > NEAR) & (np.abs(t / 224 - 1) > NEAR)
        rq, rs = R.fp8_quantize(np.where(np.arange(128) == 7, y[:, None], 0.0))
        assert sure.mean() > 0.99
        np.testing.assert_array_equal(host(q)[sure], rq[sure])
        np.testing.assert_array_equal(host(s)[sure], rs[sure])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_infinite_gates(dt):
    """silu(inf) u is infinite: a NaN code, and the block's scale 2^120; silu(-inf) is 0 times
    infinity, NaN, which no scale sees.  Gates past the exponent's range end at u g or 0."""
    m = need_gpu()
    x = torch.ones((4, 256), device="cuda")
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = float("inf"), -float("inf"), 3e4, -3e4
    q, s, _, _ = m.swiglu_quantize(x.to(dt))
    q, s = host(q), host(s)
    assert (q[0, 3] & 0x7F) == 0x7F and s[0, 0] == 2.0 ** 120
    assert (q[1, 3] & 0x7F) == 0x7F and s[1, 0] < 1
    v = R.values(q[2:], s[2:])
    assert abs(v[0, 3] / 3e4 - 1) <= 2.0 ** -4 and v[1, 3] == 0

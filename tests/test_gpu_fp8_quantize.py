"""fp8_quantize and fp8_quantize_blocks, bit for bit against 64-bit references:
codes and scales are exact functions of the inputs."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import Guarded, dev_bf16, dev_f32, host, need_gpu

pytestmark = pytest.mark.gpu


def inputs(rng, shape, bf16):
    """Rows of widely differing size with zeros, ties and the ends of the range ->
    (device tensor, float64 values)."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-30, 30, (*shape[:-1], 1)).astype(float))
    flat = x.reshape(-1, 128)
    flat[:: 5] = 0.0
    flat[1:: 7] = np.exp2(rng.integers(-3, 4, flat[1:: 7].shape).astype(float)) * rng.choice([1.0625, 1.1875, 1.75, -1.4375], flat[1:: 7].shape)
    if len(flat) > 8:
        flat[2] = 3e38
        flat[3] = 1e-40
        flat[8, :] = -0.0
    x = x.astype(np.float32)
    if bf16:
        t = torch.from_numpy(x).to(torch.bfloat16)
        return t.cuda(), t.double().numpy()
    return dev_f32(x), x.astype(np.float64)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 7168), (3, 640), (33, 1920), (257, 384), (1025, 128)])
def test_rows(rows, cols, bf16):
    m = need_gpu()
    x, v = inputs(np.random.default_rng(rows * cols), (rows, cols), bf16)
    q, s = Guarded(rows * cols), Guarded(rows * cols // 32)
    m.fp8_quantize(x, q=q.view(torch.uint8, (rows, cols)), scales=s.view(torch.float32, (rows, cols // 128)))
    torch.cuda.synchronize()
    rq, rs = R.fp8_quantize(v)
    np.testing.assert_array_equal(host(s.view(torch.float32, (rows, cols // 128))), rs)
    np.testing.assert_array_equal(host(q.view(torch.uint8, (rows, cols))), rq)
    q.check()
    s.check()
    a, b = m.fp8_quantize(x.view(1, rows, cols))
    assert a.shape == (1, rows, cols) and b.shape == (1, rows, cols // 128) and np.array_equal(host(a)[0], rq)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("batch,rows,cols", [(1, 128, 128), (3, 256, 640), (1, 1, 128), (2, 130, 384), (2, 1, 256), (1, 1001, 256)])
def test_blocks(batch, rows, cols, bf16):
    m = need_gpu()
    x, v = inputs(np.random.default_rng(batch * rows * cols), (batch, rows, cols), bf16)
    pad = -rows % 128
    full = np.concatenate([v, np.zeros((batch, pad, cols))], 1)
    ref = [R.fp8_quantize(full[i], 128) for i in range(batch)]
    rq, rs = np.stack([r[0][:rows] for r in ref]), np.stack([r[1] for r in ref])
    n, tiles = batch * rows * cols, rs.size
    copy = rows % 128 == 0
    bufs = [Guarded(n), Guarded(4 * tiles)] + ([Guarded(n), Guarded(4 * tiles)] if copy else [])
    views = [bufs[0].view(torch.uint8, v.shape), bufs[1].view(torch.float32, rs.shape)]
    if copy:
        views += [bufs[2].view(torch.uint8, (batch, cols, rows)), bufs[3].view(torch.float32, (batch, cols // 128, rows // 128))]
    got = m.fp8_quantize_blocks(x, copy, *views)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(got[1]), rs)
    np.testing.assert_array_equal(host(got[0]), rq)
    if copy:
        np.testing.assert_array_equal(host(got[2]), rq.transpose(0, 2, 1))
        np.testing.assert_array_equal(host(got[3]), rs.transpose(0, 2, 1))
    else:
        assert got[2] is None and got[3] is None
    for b in bufs:
        b.check()


@pytest.mark.parametrize("bf16", [True, False])
def test_infinities_and_nan(bf16):
    """Their codes are NaN; NaN leaves the block's other values alone, an infinity
    sets its scale to 2^120."""
    m = need_gpu()
    x = np.random.default_rng(1).standard_normal((4, 128)).astype(np.float32)
    x[1, 5], x[2, 7], x[2, 9], x[3, 3] = np.nan, np.inf, 1e37, -np.inf
    t = torch.from_numpy(x)
    t = (t.to(torch.bfloat16) if bf16 else t).cuda()
    v = t.double().cpu().numpy()
    q, s = (host(a) for a in m.fp8_quantize(t))
    fine = v.copy()
    fine[1, 5] = 0
    rq, rs = R.fp8_quantize(fine[:2])
    np.testing.assert_array_equal(s[:2], rs)
    keep = np.ones(256, bool)
    keep[128 + 5] = False
    np.testing.assert_array_equal(q[:2].reshape(-1)[keep], rq.reshape(-1)[keep])
    assert (q[1, 5] & 0x7F) == 0x7F and (q[2, 7] & 0x7F) == 0x7F and (q[3, 3] & 0x7F) == 0x7F
    assert (s[2:] == 2.0 ** 120).all()
    assert q[2, 9] == R.F.e4m3_encode(np.array([v[2, 9] / 2.0 ** 120]))[0]
    qb, sb, _, _ = m.fp8_quantize_blocks(t)
    assert float(sb) == 2.0 ** 120 and int((host(qb) & 0x7F == 0x7F).sum()) == 3


def test_every_bf16_value():
    """All finite bf16 values, each the largest of its block and beside larger ones."""
    m = need_gpu()
    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    for up in (0, 1, 9):
        x = np.zeros((bits.size, 128), np.uint16)
        x[:, 17] = bits
        if up:                                   # a neighbour 2^up times as large, where there is one
            e = np.minimum(((bits >> 7) & 0xFF) + up, 254).astype(np.uint16)
            x[:, 100] = e << 7
        t = dev_bf16(x)
        q, s = m.fp8_quantize(t)
        rq, rs = R.fp8_quantize(t.double().cpu().numpy()[:, :])
        np.testing.assert_array_equal(host(s), rs)
        np.testing.assert_array_equal(host(q), rq)


def test_empty():
    m = need_gpu()
    q, s = m.fp8_quantize(torch.empty((0, 256), device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    q, s, t, u = m.fp8_quantize_blocks(torch.empty((0, 128, 256), device="cuda"), transposed=True)
    assert q.shape == (0, 128, 256) and t.shape == (0, 256, 128)

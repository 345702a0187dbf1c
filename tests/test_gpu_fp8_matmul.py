"""Products of FP8 by FP8 against 64 bits: fp32 outputs within the error of fp32
sums of exact products, bf16 outputs within that and what the matrix instruction
drops (moe_ref.product_bounds)."""
import numpy as np
import pytest
import torch

import moe_ref as M
import ops_ref as R
from gpu_util import Guarded, dev_f32, dev_i64, dev_u8, host, host_bf16, need_gpu
from oracle import formats as F

pytestmark = pytest.mark.gpu


def weights(rng, n, k, tile, lo=-9, hi=3):
    q, s = R.random_fp8(rng, n, k, lo, hi)
    if tile:
        s = s[:-(-n // 128)]
    return q, s, M.values(q, s, 128 if tile else 1)


def got(t, bf16):
    return F.bf16_bits_to_f32(host_bf16(t)) if bf16 else host(t)


def run(m, a, sa, w, sw, row, bf16, off=None):
    T, N = a.shape[0], w.shape[-2]
    out = Guarded(T * N * (2 if bf16 else 4))
    v = out.view(torch.bfloat16 if bf16 else torch.float32, (T, N))
    args = dev_u8(a), dev_f32(sa), dev_u8(w), dev_f32(sw)
    row = None if row is None else dev_f32(row)
    if off is None:
        m.fp8_matmul(*args, a_row_scale=row, out=v)
    else:
        m.fp8_matmul_grouped(*args, dev_i64(off), a_row_scale=row, out=v)
    torch.cuda.synchronize()
    out.check()
    return got(v, bf16)


# few rows, then tiles: sides around each tile's, lengths around each stage
SHAPES = [(1, 1, 128), (1, 130, 256), (3, 16, 1152), (16, 33, 384), (17, 65, 640), (77, 1001, 2176), (130, 260, 128),
          (257, 5000, 384), (600, 2311, 256), (255, 8200, 1024), (513, 4097, 640), (1300, 1284, 896),
          (1100, 4100, 128), (1100, 4101, 256), (1027, 4102, 384)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_dense(m, n, k, tile, bf16):
    mod = need_gpu()
    rng = np.random.default_rng(m * n + k)
    a, sa = R.random_fp8(rng, m, k)
    w, sw, wv = weights(rng, n, k, tile)
    row = np.exp(rng.standard_normal(m)).astype(np.float32) if k % 256 else None
    c, bound = M.product_bounds(M.values(a, sa), wv, row, bf16)
    R.assert_product(run(mod, a, sa, w, sw, row, bf16), c, bound, bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,n,k", [
    ([1], 128, 128), ([3, 0, 1, 2], 200, 384), ([0, 0, 5], 64, 256), ([40, 0, 100, 1, 60], 300, 512),
    ([300, 0, 129, 1], 700, 640), ([256, 512, 0, 255, 257], 513, 384), ([1000, 24], 260, 1152),
    ([700, 0, 90, 513], 3001, 384), ([60, 0, 75, 41] * 33, 300, 128), ([200, 300, 0, 129, 1, 256] * 12, 200, 256)])
def test_grouped(counts, n, k, bf16):
    mod = need_gpu()
    rng = np.random.default_rng(sum(counts) + n)
    off = R.offsets_of(counts)
    T, E = int(off[-1]), len(counts)
    a, sa = R.random_fp8(rng, T, k)
    row = np.exp(rng.standard_normal(T)).astype(np.float32)
    for tile in (True, False):
        ws = [weights(rng, n, k, tile) for _ in range(E)]
        o = run(mod, a, sa, np.stack([w[0] for w in ws]), np.stack([w[1] for w in ws]), row, bf16, off)
        av = M.values(a, sa)
        for e in range(E):
            t = slice(int(off[e]), int(off[e + 1]))
            if counts[e]:
                c, bound = M.product_bounds(av[t], ws[e][2], row[t], bf16)
                R.assert_product(o[t], c, bound, bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("m,n", [(5, 40), (700, 2500), (1100, 4100)])
def test_far_scales_and_nan(m, n, bf16):
    """Scales at both ends of their range beside blocks of zeros, and NaN codes and
    scales, which reach the outputs that read them and no others."""
    mod = need_gpu()
    rng = np.random.default_rng(m)
    k = 512
    a, sa = R.random_fp8(rng, m, k)
    w, sw, _ = weights(rng, n, k, False)
    sa[:, 1], sw[:, 1] = 2.0 ** -120, 2.0 ** 115
    sa[:, 2], sw[:, 2] = 2.0 ** 112, 2.0 ** -126
    a[::3, 384:], sa[::3, 3] = 0, 2.0 ** -127
    c, bound = M.product_bounds(M.values(a, sa), M.values(w, sw), None, bf16)
    R.assert_product(run(mod, a, sa, w, sw, None, bf16), c, bound, bf16)
    a[1, 7] = 0x7F
    w[2, 300] = 0xFF
    sa = sa.copy()
    sa[3, 0] = np.inf                       # exponent field 255
    o = run(mod, a, sa, w, sw, None, bf16)
    bad = np.zeros((m, n), bool)
    bad[1], bad[:, 2], bad[3] = True, True, True
    assert np.isnan(o[bad]).all()
    ok = (~bad).nonzero()
    R.assert_product(o[ok][None], c[ok][None], bound[ok][None], bf16)


@pytest.mark.parametrize("m,n", [(4, 64), (520, 4200)])
def test_what_bf16_outputs_drop(m, n):
    """One product of 2^16 beside seven near its 13th bit down, in every run of 8."""
    mod = need_gpu()
    k = 256
    a, w = np.zeros((m, k), np.float64), np.zeros((n, k), np.float64)
    a[:], w[:] = 1.875, 1.625
    a[:, ::8], w[:, ::8] = 256.0, 256.0
    a[:, 1::16] = -448.0
    w[::2, 4::8] = 2.0 ** -9
    qa, qw = (F.e4m3_encode(np.abs(v)) | np.where(v < 0, 0x80, 0).astype(np.uint8) for v in (a, w))
    one = np.ones((m, k // 128), np.float32)
    c, bound = M.product_bounds(a, w, None, True)
    R.assert_product(run(mod, qa.astype(np.uint8), one, qw.astype(np.uint8), np.ones((n, k // 128), np.float32), None, True), c, bound, True)
    c, bound = M.product_bounds(a, w, None, False)
    R.assert_product(run(mod, qa.astype(np.uint8), one, qw.astype(np.uint8), np.ones((n, k // 128), np.float32), None, False), c, bound, False)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,n", [
    ([3], 200), ([5], 4200), ([16], 8300), ([40], 3000), ([130], 2100), ([300], 2500), ([900], 4700),
    ([1, 2, 0] * 20, 256), ([10] * 12, 1024), ([35] * 4, 2100), ([300, 0, 200, 520], 1030)])
def test_long_rows(counts, n, bf16):
    """K past what a wave or a stage group takes at once, for each kernel; reference
    in fp64 on the GPU, the dropped products bounded by sum|a b|."""
    mod = need_gpu()
    k, E, T = 8448, len(counts), sum(counts)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + n)
    a, sa = mod.fp8_quantize(torch.randn((T, k), generator=g, device="cuda"))
    w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((E, n, k), generator=g, device="cuda"))
    off = dev_i64(R.offsets_of(counts))
    dt = torch.bfloat16 if bf16 else torch.float32
    c = mod.fp8_matmul_grouped(a, sa, w, sw, off, out_dtype=dt) if E > 1 else mod.fp8_matmul(a, sa, w[0], sw[0], out_dtype=dt)

    def wide(q, s):
        return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
    av = wide(a, sa)
    for e in range(E):
        t = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            b = wide(w[e], sw[e].repeat_interleave(128, 0)[:n])
            ref, mag = av[t] @ b.t(), av[t].abs() @ b.t().abs()
            tol = ((k + 16) * R.U + (7 * 2.0 ** -13 if bf16 else 0)) * mag + (2.0 ** -8 if bf16 else R.U) * ref.abs()
            assert bool(((c[t].double() - ref).abs() <= tol).all()), e
            rms = float((c[t].double() - ref).norm() / ref.norm())      # Gaussian rows: what is dropped averages out
            assert rms < (2.0 ** -8 if bf16 else 1e-6), rms


def test_malformed_offsets_stay_inside():
    """Clamped on the device: rows outside every shard are not written."""
    mod = need_gpu()
    rng = np.random.default_rng(3)
    for T, n in ((20, 64), (400, 600), (1400, 4200)):
        a, sa = R.random_fp8(rng, T, 256)
        ws = [weights(rng, n, 256, True) for _ in range(3)]
        for off in ([-5, 3, 2, T + 9], [0, T, T, T - 4], [4, 6, 9, 11]):
            for dt, size in ((torch.float32, 4), (torch.bfloat16, 2)):
                out = Guarded(T * n * size)
                v = out.view(dt, (T, n))
                mod.fp8_matmul_grouped(dev_u8(a), dev_f32(sa), dev_u8(np.stack([w[0] for w in ws])),
                                       dev_f32(np.stack([w[1] for w in ws])), dev_i64(np.array(off)), out=v)
                torch.cuda.synchronize()
                out.check()
                if off[0] == 4:                      # rows before the first shard keep what they held
                    assert bool((v[:4].view(torch.uint8) == 0xA5).all())


def test_float8_views_and_leading_shapes():
    mod = need_gpu()
    x = torch.randn((2, 3, 256), device="cuda")
    w = torch.randn((200, 256), device="cuda")
    q, s = mod.fp8_quantize(x)
    b, t = mod.fp8_quantize(w)
    b2, t2, _, _ = mod.fp8_quantize_blocks(w)
    y = mod.fp8_matmul(q.view(torch.float8_e4m3fn), s, b.view(torch.float8_e4m3fn), t, out_dtype=torch.float32)
    assert y.shape == (2, 3, 200)
    ref = x.double() @ w.double().t()
    assert float((y.double() - ref).norm() / ref.norm()) < 0.05        # two roundings of 2.6% each
    y = mod.fp8_matmul(q, s, b2, t2)
    assert y.dtype == torch.bfloat16 and float((y.double() - ref).norm() / ref.norm()) < 0.05


def test_empty():
    mod = need_gpu()
    u8, f = torch.uint8, torch.float32
    w, ws = torch.zeros((8, 128), dtype=u8, device="cuda"), torch.ones((8, 1), device="cuda")
    assert mod.fp8_matmul(torch.empty((0, 128), dtype=u8, device="cuda"), torch.empty((0, 1), device="cuda"), w, ws).shape == (0, 8)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    y = mod.fp8_matmul_grouped(torch.empty((0, 128), dtype=u8, device="cuda"), torch.empty((0, 1), device="cuda"),
                               w.view(2, 4, 128), ws.view(2, 4, 1), off, out_dtype=f)
    assert y.shape == (0, 4)

"""mxfp4_matmul and mxfp4_matmul_grouped against 64-bit products of the decoded
operands, within the derived bounds of ops_ref, with guard bands."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import Guarded, dev_f32, dev_i64, dev_u8, host, host_bf16, need_gpu
from oracle import formats as F
from oracle import mxfp4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def operand(rng, act, rows, k):
    """(device codes, device scales, float64 values)."""
    if act == "fp8":
        q, s = R.random_fp8(rng, rows, k)
        return dev_u8(q), dev_f32(s), R.fp8_values(q, s)
    q, s = R.random_mx(rng, rows, k)
    return dev_u8(q), dev_u8(s), R.mx_values(q, s)


def numbers(t):
    return F.bf16_bits_to_f32(host_bf16(t)) if t.dtype == torch.bfloat16 else host(t)


def check_dense(m, rng, M, N, K, act, out, row):
    print(f"dense M={M} N={N} K={K} {act} {out} row={row}", flush=True)
    a, sa, va = operand(rng, act, M, K)
    b, sb, vb = operand(rng, "mxfp4", N, K)
    r = np.exp(rng.standard_normal(M)).astype(np.float32) if row else None
    g = Guarded(M * N * (2 if out == "bf16" else 4))
    c = m.mxfp4_matmul(a, sa, b, sb, a_row_scale=None if r is None else dev_f32(r),
                       out=g.view(DT[out], (M, N)))
    torch.cuda.synchronize()
    g.check()
    R.assert_product(numbers(c), *R.product(va, vb, r), out == "bf16")


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 16, 128), (2, 5, 64), (3, 7, 96), (16, 16, 160), (17, 33, 288), (31, 130, 1056),
    (64, 100, 416), (65, 257, 2080), (130, 129, 512), (300, 515, 1120), (513, 260, 768), (1, 300, 4128)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_mxfp4_rows(M, N, K, out):
    m = need_gpu()
    check_dense(m, np.random.default_rng(M * 7 + N + K), M, N, K, "mxfp4", out, (M + N) % 2 == 0)


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 40, 7168), (5, 33, 256), (16, 64, 384), (77, 101, 2176),
                                   (129, 260, 640), (400, 512, 1152)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_fp8_rows(M, N, K, out):
    m = need_gpu()
    check_dense(m, np.random.default_rng(M * 3 + N + K), M, N, K, "fp8", out, (M + N) % 2 == 1)


@pytest.mark.parametrize("M,N,K,act", [(256, 256, 8192, "mxfp4"), (1024, 768, 2048, "mxfp4"), (777, 1030, 1184, "mxfp4"),
                                       (1024, 512, 1024, "fp8"), (770, 1029, 896, "fp8"), (2100, 1300, 512, "mxfp4")])
def test_large_tiles(M, N, K, act):
    m = need_gpu()
    check_dense(m, np.random.default_rng(M + N + K), M, N, K, act, "f32", True)


def test_one_hot_positions():
    """A one in one place of either operand lands in exactly one place of the
    product: every k of a step and every row and column of a tile."""
    m = need_gpu()
    K = 288
    for act in ("mxfp4", "fp8"):
        k_all = K if act == "mxfp4" else 256
        codes = np.zeros((k_all, k_all), np.uint8)
        np.fill_diagonal(codes, 2)                       # 1.0
        b = F.pack_codes(codes)
        sb = np.full((k_all, k_all // 32), 127, np.uint8)
        rng = np.random.default_rng(3)
        a, sa, va = operand(rng, act, k_all, k_all)
        c = m.mxfp4_matmul(a, sa, dev_u8(b), dev_u8(sb), out_dtype=torch.float32)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host(c).astype(np.float64), va)


def test_extreme_scales():
    """Scale bytes from 0 to 254: small and large products, in range of fp32."""
    m = need_gpu()
    rng = np.random.default_rng(11)
    M, N, K = 20, 24, 256
    for sa_lo, sa_hi, sb_lo, sb_hi in [(0, 3, 240, 254), (240, 250, 0, 10), (0, 20, 127, 140), (200, 230, 120, 126)]:
        qa, sa = R.random_mx(rng, M, K, sa_lo, sa_hi)
        qb, sb = R.random_mx(rng, N, K, sb_lo, sb_hi)
        c = m.mxfp4_matmul(dev_u8(qa), dev_u8(sa), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32)
        torch.cuda.synchronize()
        R.assert_product(host(c), *R.product(R.mx_values(qa, sa), R.mx_values(qb, sb)), False)


def test_smallest_fp8_scale_and_zero_rows():
    m = need_gpu()
    q = np.zeros((3, 256), np.uint8)
    q[1] = 0x38                                          # 1.0
    s = np.array([[2.0 ** -127] * 2, [2.0 ** -127, 2.0 ** -126], [1.0, 2.0 ** -127]], np.float32)
    qb, sb = R.random_mx(np.random.default_rng(1), 5, 256, 200, 210)
    c = m.mxfp4_matmul(dev_u8(q), dev_f32(s), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32)
    torch.cuda.synchronize()
    R.assert_product(host(c), *R.product(R.fp8_values(q, s), R.mx_values(qb, sb)), False)
    assert (host(c)[[0, 2]] == 0).all()


def test_fp8_rows_with_far_apart_scales():
    """Block scales of one row 2^200 apart, the large ones over zero codes of
    either side, so that the small blocks make the result."""
    m = need_gpu()
    rng = np.random.default_rng(21)
    q, s = R.random_fp8(rng, 18, 256)
    qb, sb = R.random_mx(rng, 20, 256, 60, 70)
    s[::2] = 2.0 ** -60
    sb[:, 1] = 250
    sb[:, 6] = 3
    codes = F.unpack_codes(qb)
    codes[:9, 32:64] = 0
    q[:, 32:64] = 0
    qb = F.pack_codes(codes)
    c = m.mxfp4_matmul(dev_u8(q), dev_f32(s), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32)
    torch.cuda.synchronize()
    R.assert_product(host(c), *R.product(R.fp8_values(q, s), R.mx_values(qb, sb)), False)


def test_nan_scale_and_code():
    """A UE8M0 byte of 0xFF or an E4M3 NaN code makes the outputs that read it
    NaN, and no others."""
    m = need_gpu()
    rng = np.random.default_rng(5)
    for act in ("mxfp4", "fp8"):
        K = 384
        a, sa, _ = operand(rng, act, 40, K)
        qb, sb = R.random_mx(rng, 50, K)
        if act == "mxfp4":
            sa[7, 5] = 255
        else:
            a[7, 200] = 0x7F
        sb[33, 2] = 255
        c = m.mxfp4_matmul(a, sa, dev_u8(qb), dev_u8(sb), out_dtype=torch.float32)
        torch.cuda.synchronize()
        want = np.zeros((40, 50), bool)
        want[7, :] = True
        want[:, 33] = True
        np.testing.assert_array_equal(np.isnan(host(c)), want)


def test_empty_outputs():
    m = need_gpu()
    a = torch.empty((0, 64), dtype=torch.uint8, device="cuda")
    sa = torch.empty((0, 4), dtype=torch.uint8, device="cuda")
    b = torch.zeros((5, 64), dtype=torch.uint8, device="cuda")
    sb = torch.zeros((5, 4), dtype=torch.uint8, device="cuda")
    assert m.mxfp4_matmul(a, sa, b, sb).shape == (0, 5)
    assert m.mxfp4_matmul(b, sb, a, sa).shape == (5, 0)


def check_grouped(m, rng, counts, N, K, act, out, row):
    print(f"grouped {counts if len(counts) < 20 else len(counts)} N={N} K={K} {act} {out}", flush=True)
    off = R.offsets_of(counts)
    T, E = int(off[-1]), len(counts)
    a, sa, va = operand(rng, act, T, K)
    qw, sw = R.random_mx(rng, E * N, K)
    r = np.exp(rng.standard_normal(T)).astype(np.float32) if row else None
    g = Guarded(T * N * (2 if out == "bf16" else 4))
    c = m.mxfp4_matmul_grouped(a, sa, dev_u8(qw.reshape(E, N, -1)), dev_u8(sw.reshape(E, N, -1)), dev_i64(off),
                               a_row_scale=None if r is None else dev_f32(r), out=g.view(DT[out], (T, N)))
    torch.cuda.synchronize()
    g.check()
    got = numbers(c)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            vw = R.mx_values(qw[e * N:(e + 1) * N], sw[e * N:(e + 1) * N])
            R.assert_product(got[lo:hi], *R.product(va[lo:hi], vw, None if r is None else r[lo:hi]), out == "bf16")


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [5, 0, 17, 1], [16, 16], [33, 0, 0, 200, 7], [0, 0, 129], [300, 1, 260]])
@pytest.mark.parametrize("act,K", [("mxfp4", 224), ("fp8", 384)])
def test_ragged_shards(counts, act, K):
    m = need_gpu()
    rng = np.random.default_rng(sum(counts) + K)
    check_grouped(m, rng, counts, 72, K, act, "bf16" if sum(counts) % 2 else "f32", True)


@pytest.mark.parametrize("E", [64, 65, 130])
def test_many_experts(E):
    m = need_gpu()
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 4, E) * rng.integers(0, 9, E)
    counts[-1] = 5
    check_grouped(m, rng, counts.tolist(), 40, 128, "mxfp4", "f32", False)


@pytest.mark.parametrize("act", ["mxfp4", "fp8"])
def test_long_ragged_shards(act):
    m = need_gpu()
    rng = np.random.default_rng(9)
    check_grouped(m, rng, [700, 0, 1, 255, 256, 257, 90, 513], 520, 768, act, "f32", True)


def test_equal_to_the_dense_product_per_shard():
    """The same rows and weights through either entry point agree within the
    two sums' bounds."""
    m = need_gpu()
    rng = np.random.default_rng(2)
    qa, sa = R.random_mx(rng, 90, 512)
    qw, sw = R.random_mx(rng, 64, 512)
    off = dev_i64(np.array([0, 90]))
    c = m.mxfp4_matmul_grouped(dev_u8(qa), dev_u8(sa), dev_u8(qw[None]), dev_u8(sw[None]), off, out_dtype=torch.float32)
    d = m.mxfp4_matmul(dev_u8(qa), dev_u8(sa), dev_u8(qw), dev_u8(sw), out_dtype=torch.float32)
    torch.cuda.synchronize()
    _, bound = R.product(R.mx_values(qa, sa), R.mx_values(qw, sw))
    assert (np.abs(host(c).astype(np.float64) - host(d)) <= 2 * bound + 1e-300).all()


def test_malformed_offsets_stay_inside():
    """Descending, negative and too large offsets: the call completes and the
    guard bands hold (the outputs are unspecified)."""
    m = need_gpu()
    rng = np.random.default_rng(8)
    T, N, K = 50, 48, 128
    qa, sa = R.random_mx(rng, T, K)
    qw, sw = R.random_mx(rng, 3 * N, K)
    for off in ([0, 40, 10, 50], [-5, 20, 90, 1 << 40], [50, 0, 50, 0], [0, -(1 << 50), 25, 50]):
        g = Guarded(T * N * 4)
        m.mxfp4_matmul_grouped(dev_u8(qa), dev_u8(sa), dev_u8(qw.reshape(3, N, -1)), dev_u8(sw.reshape(3, N, -1)),
                               dev_i64(np.array(off)), out=g.view(torch.float32, (T, N)))
        torch.cuda.synchronize()
        g.check()


def test_other_stream_and_repeatable():
    m = need_gpu()
    rng = np.random.default_rng(4)
    a, sa, va = operand(rng, "mxfp4", 200, 1024)
    b, sb, vb = operand(rng, "mxfp4", 300, 1024)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = m.mxfp4_matmul(a, sa, b, sb, out_dtype=torch.float32)
    s.synchronize()
    R.assert_product(host(c), *R.product(va, vb), False)
    d = m.mxfp4_matmul(a, sa, b, sb, out_dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(c, d)


def test_binding_refuses():
    m = need_gpu()
    a = torch.zeros((4, 64), dtype=torch.uint8, device="cuda")
    sa = torch.zeros((4, 4), dtype=torch.uint8, device="cuda")
    w = torch.zeros((2, 4, 64), dtype=torch.uint8, device="cuda")
    sw = torch.zeros((2, 4, 4), dtype=torch.uint8, device="cuda")
    off = dev_i64(np.array([0, 1, 4]))
    with pytest.raises(ValueError):
        m.mxfp4_matmul(a, sa, a[:, :48].contiguous(), sa)           # another K
    with pytest.raises(ValueError):
        m.mxfp4_matmul(a, sa[:2].contiguous(), a, sa)               # too few scales
    with pytest.raises(ValueError):
        m.mxfp4_matmul(a.t(), sa, a, sa)                            # not contiguous
    with pytest.raises(TypeError):
        m.mxfp4_matmul(a, sa, a, sa.float())                        # FP8 weights
    with pytest.raises(ValueError):
        m.mxfp4_matmul(a, sa, w, sw)                                # 3-d weights
    with pytest.raises(ValueError):
        m.mxfp4_matmul_grouped(a, sa, w, sw, off[:2].contiguous())  # offsets too short
    with pytest.raises(ValueError):
        m.mxfp4_matmul_grouped(a, sa, a, sa, off)                   # 2-d weights
    with pytest.raises(m.Fp4Error):
        m.mxfp4_matmul(a, sa, a, sa, out_dtype=torch.float16)
    with pytest.raises(m.Fp4Error):                                 # out over an input
        m.mxfp4_matmul(a, sa, a, sa, out=a.view(-1)[:64].view(torch.float32).view(4, 4))


def test_large_fp8_tiles_with_scales_out_of_window():
    """Shapes that take the tiles: blocks of zeros with the smallest scale,
    a far smaller and a far larger scale over codes, and NaN scales."""
    m = need_gpu()
    rng = np.random.default_rng(31)
    M, N, K = 300, 330, 512
    q, s = R.random_fp8(rng, M, K)
    qb, sb = R.random_mx(rng, N, K)
    q[5] = 0
    s[5] = 2.0 ** -127
    codes = F.unpack_codes(qb)
    codes[7, 64:96] = 8                                  # negative zeros
    qb = F.pack_codes(codes)
    sb[7, 2] = 0
    for step in range(3):
        if step == 1:
            s[140, 1] = 2.0 ** -120
            sb[9, 3] = 240
        if step == 2:
            sb[200, 4] = 255
        c = m.mxfp4_matmul(dev_u8(q), dev_f32(s), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32)
        torch.cuda.synchronize()
        got = host(c)
        if step == 2:
            assert np.isnan(got[:, 200]).all() and not np.isnan(np.delete(got, 200, 1)).any()
        sb2 = np.where(sb == 255, 127, sb).astype(np.uint8)
        want, bound = R.product(R.fp8_values(q, s), R.mx_values(qb, sb2))
        keep = np.arange(N) != 200 if step == 2 else np.ones(N, bool)
        R.assert_product(got[:, keep], want[:, keep], bound[:, keep], False)


@pytest.mark.parametrize("M,N,K,act", [(1000, 1100, 256, "mxfp4"), (1030, 4100, 160, "mxfp4"), (4099, 2050, 224, "mxfp4"),
                                       (4200, 2100, 1568, "mxfp4"), (1500, 1300, 128, "fp8"), (1700, 1290, 384, "fp8"),
                                       (900, 1025, 2080, "mxfp4"), (16, 515, 1056, "mxfp4"), (13, 200, 1152, "fp8")])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_every_kernel(M, N, K, act, out):
    """Shapes on both sides of each choice of kernel, with odd edges and short
    last steps and stages."""
    m = need_gpu()
    check_dense(m, np.random.default_rng(M + K), M, N, K, act, out, M % 2 == 0)


@pytest.mark.parametrize("counts,N,K,act", [([300, 0, 20, 700, 1], 260, 288, "mxfp4"), ([1200, 3, 800], 4100, 160, "mxfp4"),
                                            ([100, 0, 200, 17], 300, 256, "fp8"), ([30] * 9, 100, 1152, "fp8")])
def test_grouped_kernels(counts, N, K, act):
    m = need_gpu()
    check_grouped(m, np.random.default_rng(K), counts, N, K, act, "f32", True)

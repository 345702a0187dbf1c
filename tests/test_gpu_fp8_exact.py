"""bf16 outputs of exact products (exact=True) from each kernel of the products of FP8 by FP8:
sums that the default drops are there to the last bit, and random ones are the nearest
bf16 value of an fp32 sum.

An fp32 sum of exact products is off by less than 1e-6 of a Gaussian sum's size (fp32
outputs are held to that), which takes a bf16 output to its neighbour, 2^-7 relative away
at most, so seldom that the root mean square of these steps is at most sqrt(1e-6 * 2^-7)."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import Guarded, dev_f32, dev_i64, dev_u8, need_gpu
from oracle import formats as F
from test_gpu_fp8_tiles import check, wide
from test_gpu_graphs import _replay_check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NEAR = (1e-6 * 2.0 ** -7) ** 0.5

# tokens of each expert, N: 16 x 16 to 64 x 64 workgroups, tiles of 128 rows, of 256
KINDS = [([1], 130), ([3], 4200), ([16], 8300), ([40], 3000), ([130], 2100), ([300], 2500), ([2100], 4200), ([3585], 4100),
         ([1, 2, 0] * 20, 256), ([10] * 12, 1024), ([35] * 4, 2100), ([300, 0, 200, 520], 1030), ([700, 0, 257, 1300], 4100)]


def codes(v):
    return dev_u8(F.e4m3_encode(np.abs(v)) | np.where(v < 0, 0x80, 0).astype(np.uint8))


def product(mod, a, sa, w, sw, counts, off=None, **kw):
    if len(counts) == 1:
        return mod.fp8_matmul(a, sa, w[0], sw[0], **kw)
    return mod.fp8_matmul_grouped(a, sa, w, sw, dev_i64(R.offsets_of(counts)) if off is None else off, **kw)


@pytest.mark.parametrize("counts,n", KINDS)
def test_what_is_left_where_large_products_cancel(counts, n):
    """In every run of 8 one product of +-2^12, which cancel, and seven of 2^-2: every
    partial sum is a whole number of quarters below 2^20, so fp32 holds it, and the sum
    itself, 7 K / 32, is a bf16 value.  The default drops the small ones, each below 2^-13
    of the large one, or not, within its stated bound."""
    mod = need_gpu()
    E, T, k = len(counts), sum(counts), 1024
    a, w = np.full((1, k), 0.5), np.full((1, k), 0.5)
    a[:, ::8], w[:, ::8] = 256.0, 16.0
    a[:, ::16] = -256.0
    av, wv = (np.broadcast_to(v, (rows, k)) for v, rows in ((a, T), (w, E * n)))
    qa, qw = codes(av), codes(wv).view(E, n, k)
    one = (dev_f32(np.ones((T, k // 128))), dev_f32(np.ones((E, n, k // 128))))
    got = product(mod, qa, one[0], qw, one[1], counts, exact=True)
    assert got.dtype is BF and bool((got == 7 * k / 32).all())
    assert bool((product(mod, qa, one[0], qw, one[1], counts, out_dtype=F32) == 7 * k / 32).all())
    plain = product(mod, qa, one[0], qw, one[1], counts)
    assert bool(((plain.double() - 7 * k / 32).abs() <= k / 8 * 7 * 2.0 ** -13 * 4096).all())


@pytest.mark.parametrize("counts,n", KINDS)
def test_the_nearest_bf16_value(counts, n):
    mod = need_gpu()
    E, T, k = len(counts), sum(counts), 1152
    g = torch.Generator(device="cuda")
    g.manual_seed(T + n)
    a, sa = mod.fp8_quantize(torch.randn((T, k), generator=g, device="cuda"))
    w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((E, n, k), generator=g, device="cuda"))
    row = torch.exp(torch.randn(T, generator=g, device="cuda"))
    out = Guarded(T * n * 2)
    v = out.view(BF, (T, n))
    assert product(mod, a, sa, w, sw, counts, a_row_scale=row, out=v, exact=True) is v
    torch.cuda.synchronize()
    out.check()
    av, off, apart, size = wide(a, sa), R.offsets_of(counts), 0.0, 0.0
    for e in range(E):
        t = slice(int(off[e]), int(off[e + 1]))
        b = wide(w[e], sw[e], True)
        if not counts[e]:
            continue
        c, mag = av[t] @ b.t() * row[t].double()[:, None], av[t].abs() @ b.abs().t() * row[t].double()[:, None]
        err = (v[t].double() - c).abs()
        assert bool((err <= (k + 16) * R.U * mag + 2.0 ** -8 * c.abs()).all()), e
        apart += float((v[t].double() - c.to(BF).double()).square().sum())
        size += float(c.square().sum())
    assert (apart / size) ** 0.5 <= NEAR, (apart / size) ** 0.5
    # fp32 outputs are exact with it and without
    assert torch.equal(product(mod, a, sa, w, sw, counts, out_dtype=F32, exact=True), product(mod, a, sa, w, sw, counts, out_dtype=F32))


@pytest.mark.parametrize("m,n", [(5, 40), (300, 2500), (2100, 4200), (3585, 4100)])
def test_far_scales_and_nan(m, n):
    """Scales outside the window of bf16 products: the path that takes them apart writes
    bf16 too.  A NaN scale has the four blocks of 32 k of its step, for the 16 x 16 outputs
    that read it, multiplied one by one and added then: the same exact products in
    another order.  So the outputs beside it are held to the bound of an fp32 sum in any
    order, (K + 16) U sum|a b|, and not to the bits that they had without it."""
    mod = need_gpu()
    rng = np.random.default_rng(m)
    k = 512
    a, sa = R.random_fp8(rng, m, k)
    w, sw = R.random_fp8(rng, n, k)
    sa[:, 1], sw[:, 1] = 2.0 ** -120, 2.0 ** 115
    sa[:, 2], sw[:, 2] = 2.0 ** 112, 2.0 ** -126
    args = dev_u8(a), dev_f32(sa), dev_u8(w), dev_f32(sw)
    av, wv = wide(*args[:2]), wide(*args[2:])
    out = mod.fp8_matmul(*args, exact=True)
    c, mag = av @ wv.t(), av.abs() @ wv.abs().t()
    tol = (k + 16) * (R.U * mag + 2.0 ** -126) + 2.0 ** -8 * c.abs()
    assert bool(((out.double() - c).abs() <= tol).all())
    check(mod.fp8_matmul(*args, out_dtype=F32), av, wv, None, False, "fp32")
    args[0][1, 7], args[3][2, 0] = 0x7F, float("inf")
    got = mod.fp8_matmul(*args, exact=True)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[1], bad[:, 2] = True, True
    assert bool(torch.isnan(got[bad]).all()) and bool(((got.double() - c).abs() <= tol)[~bad].all())


def test_in_a_graph_and_on_a_stream():
    mod = need_gpu()
    side = torch.cuda.Stream()
    for counts, n in (([3], 4200), ([300], 2500), ([3585], 4100), ([700, 0, 257, 1300], 4100)):
        E, T, k = len(counts), sum(counts), 384
        a, sa = mod.fp8_quantize(torch.randn((T, k), device="cuda"))
        w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((E, n, k), device="cuda"))
        off = dev_i64(R.offsets_of(counts))
        out = product(mod, a, sa, w, sw, counts, off, exact=True)
        torch.cuda.synchronize()
        apart = product(mod, a, sa, w, sw, counts, off, exact=True, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(apart, out)
        _replay_check(lambda: product(mod, a, sa, w, sw, counts, off, out=out, exact=True), [out])

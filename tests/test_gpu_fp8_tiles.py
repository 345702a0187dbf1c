"""Products of FP8 by FP8 whose launches take row tiles of 256 (more than 192 tiles of 256 x
256), alone and mixed with the halves of 128 rows that shards leave, against 64 bits on
the GPU.

A sum is off by (K + 16) U sum|a b| at most (ops_ref), a bf16 output also by 7 * 2^-13 of the
largest product in each run of 8 k, which is at most the product of the run's largest
a and largest b (`dropped`).  On Gaussian rows what is dropped is 2e-5 of the sum's size: a
bf16 output then differs from the nearest bf16 value only where the sum comes so near to
a border, by one step of 2^-7 relative or less, with a chance of the error over the
step, so the root mean square of these differences is at most sqrt(2e-5 * 2^-7) = 4.0e-4
of the outputs'; rounding itself is 1.1e-3."""
import numpy as np
import pytest
import torch

import moe_ref as M
import ops_ref as R
from gpu_util import Guarded, dev_f32, dev_i64, dev_u8, need_gpu
from test_gpu_graphs import _replay_check

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
NEAR = (2e-5 * 2.0 ** -7) ** 0.5


def wide(q, s, tile=False):
    """Codes and scales on the GPU -> fp64 values there (scales by way of the CPU, which
    keeps subnormal ones)."""
    s = s.cpu().double().to(q.device).repeat_interleave(128, 1)
    if tile:
        s = s.repeat_interleave(128, 0)[:q.shape[0]]
    return q.view(torch.float8_e4m3fn).double() * s


def dropped(a, b):
    """7 * 2^-13 of what the largest product of each run of 8 k can be, summed."""
    x, y = (v.abs().view(v.shape[0], -1, 8).amax(-1) for v in (a, b))
    return 7 * 2.0 ** -13 * (x @ y.t())


def check(got, a, b, row, bf16, what):
    """Every output of a . b^T times row within its bound; returns the reference."""
    c, mag = a @ b.t(), a.abs() @ b.abs().t()
    bound = (a.shape[1] + 16) * (R.U * mag + 2.0 ** -126)
    if bf16:
        bound += dropped(a, b)
    if row is not None:
        r = row.double()[:, None]
        c, bound = c * r, bound * r.abs()
    tol = bound + (2.0 ** -8 if bf16 else R.U) * c.abs()
    bad = ~((got.double() - c).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist())
    return c


def check_gaussian(got, c, bf16):
    """The relative root mean square of the error: fp32's last places, or of what is not the
    nearest bf16 value."""
    near = c.to(BF).double() if bf16 else c
    rms = float((got.double() - near).norm() / c.norm())
    assert rms <= (NEAR if bf16 else 1e-6), rms


def gaussian(mod, g, rows, k):
    return mod.fp8_quantize(torch.randn((rows, k), generator=g, device="cuda"))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("m,n,k", [
    # 14 or 15 row tiles by 16 or 17 of columns: a rest of 172 rows, 129 (whole tiles), 128, 16 and 1 (halves)
    (3500, 4100, 128), (3713, 4001, 256), (3712, 4096, 640), (3600, 4353, 1152), (3585, 4100, 8448),
    (3500, 4100, 384), (3713, 4100, 512), (3600, 4096, 896)])
def test_dense(m, n, k, bf16):
    mod = need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    a, sa = gaussian(mod, g, m, k)
    tile = k % 256 == 0
    if tile:
        w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((n, k), generator=g, device="cuda"))
    else:
        w, sw = gaussian(mod, g, n, k)
    row = torch.exp(torch.randn(m, generator=g, device="cuda")) if k % 384 == 0 else None
    out = Guarded(m * n * (2 if bf16 else 4))
    v = out.view(BF if bf16 else F32, (m, n))
    mod.fp8_matmul(a, sa, w, sw, a_row_scale=row, out=v)
    torch.cuda.synchronize()
    out.check()
    check_gaussian(v, check(v, wide(a, sa), wide(w, sw, tile), row, bf16, (m, n, k)), bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,n,k", [
    ([129, 255, 0, 256, 257, 400, 0] * 2, 4100, 640), ([400, 0, 257, 1, 128, 513, 1200], 4609, 384),
    ([3000, 0, 700], 4100, 1152), ([256, 384, 640, 0, 127] * 3, 4097, 8448)])
def test_whole_tiles_and_halves(counts, n, k, bf16):
    """Shards of every rest: whole tiles of all of them come before the halves."""
    mod = need_gpu()
    E, T = len(counts), sum(counts)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + n)
    a, sa = gaussian(mod, g, T, k)
    w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((E, n, k), generator=g, device="cuda"))
    row = torch.exp(torch.randn(T, generator=g, device="cuda"))
    off = R.offsets_of(counts)
    out = Guarded(T * n * (2 if bf16 else 4))
    v = out.view(BF if bf16 else F32, (T, n))
    mod.fp8_matmul_grouped(a, sa, w, sw, dev_i64(off), a_row_scale=row, out=v)
    torch.cuda.synchronize()
    out.check()
    av = wide(a, sa)
    for e in range(E):
        if counts[e]:
            t = slice(int(off[e]), int(off[e + 1]))
            check_gaussian(v[t], check(v[t], av[t], wide(w[e], sw[e], True), row[t], bf16, e), bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("m,n", [(3500, 4100), (3600, 4353)])
def test_far_scales_and_nan(m, n, bf16):
    """Every code, scales at both ends of their range beside blocks of zeros; then NaN codes
    and scales, which reach the outputs that read them and no others."""
    mod = need_gpu()
    rng = np.random.default_rng(m)
    k = 640
    a, sa = R.random_fp8(rng, m, k)
    w, sw = R.random_fp8(rng, n, k)
    sa[:, 1], sw[:, 1] = 2.0 ** -120, 2.0 ** 115
    sa[:, 2], sw[:, 2] = 2.0 ** 112, 2.0 ** -126
    a[::3, 384:512], sa[::3, 3] = 0, 2.0 ** -127
    da, dsa, dw, dsw = dev_u8(a), dev_f32(sa), dev_u8(w), dev_f32(sw)
    av, wv = wide(da, dsa), wide(dw, dsw)
    out = mod.fp8_matmul(da, dsa, dw, dsw, out_dtype=BF if bf16 else F32)
    check(out, av, wv, None, bf16, "far scales")
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    for i in (1, 300, m - 1):                       # the first row tile, the second, the rest
        da[i, 7], bad[i] = 0x7F, True
    for i in (2, 259, n - 2):
        dw[i, 300], bad[:, i] = 0xFF, True
    dsa[3, 0], bad[3] = float("inf"), True          # exponent field 255
    dsw[700, 4], bad[:, 700] = float("nan"), True
    got = mod.fp8_matmul(da, dsa, dw, dsw, out_dtype=BF if bf16 else F32)
    assert bool(torch.isnan(got[bad]).all())
    check(torch.where(bad, out, got), av, wv, None, bf16, "beside NaN")


def test_what_bf16_outputs_drop():
    """One product of 2^16 beside seven near its 13th bit down, in every run of 8: within
    the stated bound, and exact where the output is fp32."""
    mod = need_gpu()
    m, n, k = 3500, 4100, 256
    a, w = np.full((m, k), 1.875), np.full((n, k), 1.625)
    a[:, ::8], w[:, ::8] = 256.0, 256.0
    a[:, 1::16] = -448.0
    w[::2, 4::8] = 2.0 ** -9
    one, (qa, qw) = np.ones, (M.F.e4m3_encode(np.abs(v)) | np.where(v < 0, 0x80, 0).astype(np.uint8) for v in (a, w))
    args = dev_u8(qa), dev_f32(one((m, 2))), dev_u8(qw), dev_f32(one((n, 2)))
    av, wv = wide(*args[:2]), wide(*args[2:])
    for dt in (BF, F32):
        check(mod.fp8_matmul(*args, out_dtype=dt), av, wv, None, dt is BF, dt)


def operands(mod):
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    a, sa = gaussian(mod, g, 3585, 384)
    w, sw, _, _ = mod.fp8_quantize_blocks(torch.randn((2, 4100, 384), generator=g, device="cuda"))
    return a, sa, w, sw, dev_i64(np.array([0, 1900, 3585]))


def calls(mod):
    a, sa, w, sw, off = operands(mod)
    for dt in (BF, F32):
        yield lambda dt=dt, **kw: mod.fp8_matmul(a, sa, w[0], sw[0], out_dtype=dt, **kw)
        yield lambda dt=dt, **kw: mod.fp8_matmul_grouped(a, sa, w, sw, off, out_dtype=dt, **kw)


def test_captured_and_replayed():
    mod = need_gpu()
    for call in calls(mod):
        out = call()
        _replay_check(lambda: call(out=out), [out])


def test_on_a_delayed_stream_and_two_at_once():
    mod = need_gpu()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for call in calls(mod):
        want = call()
        torch.cuda.synchronize()
        for s in sides:
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
        got = [call(stream=s) for s in sides]
        junk = [torch.full((want.numel() * want.element_size(),), 0xA5, dtype=U8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(t.view(U8), want.view(U8)) for t in got)
        del junk

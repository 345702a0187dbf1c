"""Blocks of zeros under the smallest scale (tokens masked out of a loss, padding
rows) in the products of FP8 operands: exact beside blocks that do need the
careful path, and not sent through it themselves.

A tile that holds zero blocks reads its scales again and the codes of those
blocks, at most its operands once more without any product: less than the
tile's own time again, with a margin 3 times the time without zeros in all."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import dev_f32, dev_i64, dev_u8, host, need_gpu

pytestmark = pytest.mark.gpu


def gradient(m, cols_a, cols_b, off, M, N):
    return m.fp8_matmul_tokblk(dev_u8(cols_a[0]), dev_f32(cols_a[1]), dev_u8(cols_b[0]), dev_f32(cols_b[1]),
                               dev_i64(off), M, N, out_dtype=torch.float32)


def mask_tokens(cols, off, ch, spans):
    """Codes of tokens in spans to zero, and the scales of blocks that are all zero to 2^-127."""
    q, s = cols[0].copy(), cols[1].copy()
    for e, at in enumerate(R.column_scale_start(off, ch)):
        lo, hi = int(off[e]), int(off[e + 1])
        n, nb = hi - lo, -(-(hi - lo) // 128)
        v, sc = q[ch * lo:ch * hi].reshape(ch, n), s[at:at + ch * nb].reshape(ch, nb)
        for a, b in spans:
            v[:, max(a - lo, 0):max(b - lo, 0)] = 0
        for k in range(nb):
            sc[:, k] = np.where((v[:, 128 * k:128 * k + 128] & 0x7F).any(1), sc[:, k], 2.0 ** -127)
    return q, s


@pytest.mark.parametrize("counts", [[300], [256, 0, 131], [7, 140, 15], [129, 1000], [1]])
@pytest.mark.parametrize("M,N", [(128, 256), (384, 128)])
def test_masked_tokens(counts, M, N):
    m = need_gpu()
    rng = np.random.default_rng(sum(counts) + M)
    off = R.offsets_of(counts)
    t = int(off[-1])
    for spans in ([(0, 128)], [(t - min(t, 44), t)], [(0, t)], [(128, 256), (t - 1, t)]):
        a = mask_tokens(R.random_columns(rng, off, M), off, M, spans)
        b = R.random_columns(rng, off, N)
        got = host(gradient(m, a, b, off, M, N))
        va, vb = R.column_values(*a, off, M), R.column_values(*b, off, N)
        for e, n in enumerate(counts):
            if n:
                R.assert_product(got[e], *R.product(va[e], vb[e]), False)
            else:
                assert not got[e].any()


@pytest.mark.parametrize("count", [1, 15, 16, 17, 129, 143, 300])
@pytest.mark.parametrize("side", ["a", "b"])
def test_one_code_under_a_tiny_scale(count, side):
    """One code alone in its block, at every place where the search for it could
    end, under a scale that bf16 products cannot hold."""
    m = need_gpu()
    rng = np.random.default_rng(count)
    M, N, off = 128, 256, R.offsets_of([count])
    nb, last = -(-count // 128), count - 1
    for t in sorted({0, last, max(last - 15, 0), max(last - 16, 0), 128 * (nb - 1)}):
        ch_tiny, ch_big = (M, N) if side == "a" else (N, M)
        q = np.zeros((ch_tiny, count), np.uint8)
        s = np.full((ch_tiny, nb), 2.0 ** -127, np.float32)
        q[5, t], s[5, t // 128] = 0x01, 2.0 ** -118                      # 2^-9 times 2^-118
        s_all = np.zeros(ch_tiny * (nb + 1), np.float32)
        s_all[:ch_tiny * nb] = s.reshape(-1)
        tiny = (q.reshape(-1), s_all)
        big = R.random_columns(rng, off, ch_big, 80, 90)
        a, b = (tiny, big) if side == "a" else (big, tiny)
        got = host(gradient(m, a, b, off, M, N))[0]
        want, bound = R.product(R.column_values(*a, off, M)[0], R.column_values(*b, off, N)[0])
        assert np.abs(want).max() > 0
        R.assert_product(got, want, bound, False)


@pytest.mark.parametrize("at", [0, 31, 32, 127, 128, 1151])
@pytest.mark.parametrize("side", ["a", "b"])
def test_one_code_under_a_tiny_scale_in_rows(at, side):
    """The same for FP8 rows by MXFP4 on the tiles."""
    m = need_gpu()
    rng = np.random.default_rng(at)
    M, N, K = 1400, 1290, 1152
    if side == "a":
        q, s = np.zeros((M, K), np.uint8), np.full((M, K // 128), 2.0 ** -127, np.float32)
        q[200, at], s[200, at // 128] = 0x01, 2.0 ** -118
        qb, sb = R.random_mx(rng, N, K, 200, 210)
    else:
        q, s = R.random_fp8(rng, M, K, 80, 90)
        qb, sb = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 32), np.uint8)
        qb[300, at // 2], sb[300, at // 32] = 1 << (4 * (at & 1)), 8     # 0.5 times 2^-119
    c = host(m.mxfp4_matmul(dev_u8(q), dev_f32(s), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32))
    va, vb = (torch.from_numpy(v).cuda() for v in (R.fp8_values(q, s), R.mx_values(qb, sb)))
    want = (va @ vb.t().contiguous()).cpu().numpy()
    size = (va.abs() @ vb.abs().t().contiguous()).cpu().numpy()
    assert np.abs(want).max() > 0
    R.assert_product(c, want, (K + 16) * (R.U * size + 2.0 ** -126), False)


def median_us(f):
    t = []
    for _ in range(9):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        t.append(a.elapsed_time(b) * 1e3)
    return sorted(t)[4]


def test_zero_blocks_do_not_take_the_careful_path():
    m = need_gpu()
    rng = np.random.default_rng(1)
    off = R.offsets_of([8192])
    M = N = 2048
    a, b = R.random_columns(rng, off, M), R.random_columns(rng, off, N)
    z = mask_tokens(a, off, M, [(0, 128), (4096, 6144)])
    offd, b = dev_i64(off), (dev_u8(b[0]), dev_f32(b[1]))
    times = {}
    for name, c in (("full", a), ("masked", z)):
        c = (dev_u8(c[0]), dev_f32(c[1]))
        times[name] = median_us(lambda: m.fp8_matmul_tokblk(*c, *b, offd, M, N))
    print("weight gradient", times, flush=True)
    assert times["masked"] < 3 * times["full"]
    q, s = R.random_fp8(rng, 4096, 4096)
    w = tuple(dev_u8(v) for v in R.random_mx(rng, 4096, 4096))
    for name in ("full", "masked"):
        c = (dev_u8(q), dev_f32(s))
        times[name] = median_us(lambda: m.mxfp4_matmul(*c, *w))
        q[::50] = 0
        s[::50] = 2.0 ** -127
    print("rows", times, flush=True)
    assert times["masked"] < 3 * times["full"]

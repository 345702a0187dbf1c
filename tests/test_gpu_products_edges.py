"""The products' tile kernels where the smaller tests do not reach them:
malformed offsets, NaN scales and scale bytes at both ends beside a last stage
that ends inside K, one token by a very wide weight; and the precision of
their sums, which bounds proportional to K cannot see.

Precision, derived:
  cancelling blocks: two products of +-P in one block of 32, and n small ones
  (sum S of magnitudes) in another.  In any order at most n + 2 additions are
  made, each off by at most 2^-23 of a partial sum of at most P + S:
  (n + 2) 2^-23 (P + S).  Operands lined up with the largest of them 14 bits
  deep would lose up to 2^-14 P.
  random rows: with independent products of mean zero and n additions rounded by
  at most 2^-24 of partial sums that grow as sqrt(i), the errors' RMS is at most
  2^-24 sqrt(n / 2) of the results' RMS (1.9e-6 at 2048); dropping what lies 14
  bits below a neighbour costs E4M3 about 2e-5."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import CANARY, Guarded, dev_f32, dev_i64, dev_u8, host, need_gpu
from oracle import formats as F

pytestmark = pytest.mark.gpu


def operand(rng, act, rows, k):
    if act == "fp8":
        q, s = R.random_fp8(rng, rows, k)
        return q, s, R.fp8_values(q, s)
    q, s = R.random_mx(rng, rows, k)
    return q, s, R.mx_values(q, s)


def dev(q, s):
    return dev_u8(q), dev_f32(s) if s.dtype == np.float32 else dev_u8(s)


def f64(a, b):
    """a . b^T and |a| . |b|^T in 64 bits, on the GPU."""
    a, b = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    return (a @ b.t().contiguous()).cpu().numpy(), (a.abs() @ b.abs().t().contiguous()).cpu().numpy()


# ------------------------------------------------------------- malformed offsets
@pytest.mark.parametrize("act,T,N,K", [("mxfp4", 600, 300, 160),      # 256 x 128 tiles
                                       ("mxfp4", 2000, 4100, 160),    # 256 x 256 tiles
                                       ("fp8", 600, 300, 128)])
def test_malformed_offsets_on_tiles(act, T, N, K):
    """Every access stays inside (guard bands), and rows outside every clamped
    shard are not written."""
    m = need_gpu()
    rng = np.random.default_rng(T)
    q, s, _ = operand(rng, act, T, K)
    qw, sw = R.random_mx(rng, 3 * N, K)
    args = (*dev(q, s), dev_u8(qw.reshape(3, N, -1)), dev_u8(sw.reshape(3, N, -1)))
    for off in ([0, T - 100, 100, T], [-5, 20, 9 * T, 1 << 40], [T, 0, T, 0], [0, -(1 << 50), T // 2, T],
                [130, 300, 300, 500], [1 << 40, T, 3, -7]):
        print(act, T, off, flush=True)
        g = Guarded(T * N * 4)
        out = g.view(torch.float32, (T, N))
        m.mxfp4_matmul_grouped(*args, dev_i64(np.array(off)), out=out)
        torch.cuda.synchronize()
        g.check()
        inside = np.zeros(T, bool)
        for a, b in zip(off, off[1:]):
            lo = min(max(a, 0), T)
            inside[lo:min(max(b, lo), T)] = True
        left = host(out).view(np.uint8)[~inside]
        assert (left == CANARY).all()


@pytest.mark.parametrize("T,M,N", [(300, 128, 256), (300, 4096, 3968)])
def test_malformed_offsets_on_gradient_tiles(T, M, N):
    m = need_gpu()
    rng = np.random.default_rng(8)
    E = 3
    nb = -(-T // 128) + E
    args = [dev_u8(rng.integers(0, 120, T * M, dtype=np.uint8)), dev_f32(np.ones(M * nb)),
            dev_u8(rng.integers(0, 120, T * N, dtype=np.uint8)), dev_f32(np.ones(N * nb))]
    for off in ([0, 200, 100, 300], [-5, 3, 900, 1 << 40], [300, 0, 300, 0], [299, 300, 300, 290]):
        print(T, M, N, off, flush=True)
        g = Guarded(E * M * N * 4)
        out = g.view(torch.float32, (E, M, N))
        m.fp8_matmul_tokblk(*args, dev_i64(np.array(off)), M, N, out=out)
        torch.cuda.synchronize()
        g.check()
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if min(max(b, 0), T) <= min(max(a, 0), T):
                assert not out[e].any()


# ----------------------------------------------------- scales on the tile kernel
@pytest.mark.parametrize("K", [256, 288, 416, 800])
@pytest.mark.parametrize("M", [1024, 1100])
def test_nan_scales_on_tiles(M, K):
    """A NaN scale makes its row or column NaN and nothing else, the last block
    of a row among them: its byte is also what the tail past K is read as."""
    m = need_gpu()
    rng = np.random.default_rng(M + K)
    N = 1030
    qa, sa, va = operand(rng, "mxfp4", M, K)
    qb, sb, vb = operand(rng, "mxfp4", N, K)
    sa[7, 5] = sa[M - 1, -1] = sb[33, -1] = sb[N - 1, 0] = 255
    c = host(m.mxfp4_matmul(dev_u8(qa), dev_u8(sa), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32))
    rows, cols = np.isin(np.arange(M), [7, M - 1]), np.isin(np.arange(N), [33, N - 1])
    np.testing.assert_array_equal(np.isnan(c), rows[:, None] | cols[None])
    want, s = f64(va[~rows], vb[~cols])
    R.assert_product(c[~rows][:, ~cols], want, (K + 16) * (R.U * s + 2.0 ** -126), False)


def test_nan_of_one_shard_stays_there():
    """The last row of a shard fills up its last tile; a NaN there reaches no
    row of the next shard."""
    m = need_gpu()
    rng = np.random.default_rng(3)
    counts, N, K = [130, 257, 1, 300], 270, 288
    off = R.offsets_of(counts)
    qa, sa, _ = operand(rng, "mxfp4", int(off[-1]), K)
    qw, sw = R.random_mx(rng, 4 * N, K)
    bad = off[1:] - 1
    sa[bad[[0, 2]], -1] = 255
    c = host(m.mxfp4_matmul_grouped(dev_u8(qa), dev_u8(sa), dev_u8(qw.reshape(4, N, -1)), dev_u8(sw.reshape(4, N, -1)),
                                    dev_i64(off), out_dtype=torch.float32))
    np.testing.assert_array_equal(np.isnan(c).all(1), np.isin(np.arange(off[-1]), bad[[0, 2]]))
    np.testing.assert_array_equal(np.isnan(c).any(1), np.isnan(c).all(1))


@pytest.mark.parametrize("K", [256, 288, 416])
@pytest.mark.parametrize("lo,hi,lo2,hi2", [(0, 3, 240, 254), (240, 250, 0, 10), (0, 20, 127, 140), (200, 230, 120, 126)])
def test_extreme_scales_on_tiles(K, lo, hi, lo2, hi2):
    m = need_gpu()
    rng = np.random.default_rng(K + lo)
    qa, sa = R.random_mx(rng, 1024, K, lo, hi)
    qb, sb = R.random_mx(rng, 1030, K, lo2, hi2)
    c = host(m.mxfp4_matmul(dev_u8(qa), dev_u8(sa), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32))
    want, s = f64(R.mx_values(qa, sa), R.mx_values(qb, sb))
    R.assert_product(c, want, (K + 16) * (R.U * s + 2.0 ** -126), False)


@pytest.mark.parametrize("M,N", [(5, 20), (40, 40), (1024, 1030)])
@pytest.mark.parametrize("K", [64, 256, 288])
def test_zero_codes_under_the_largest_scales(M, N, K):
    """Zeros times 2^127 on both sides are zero."""
    m = need_gpu()
    rng = np.random.default_rng(M + K)
    qa, sa = R.random_mx(rng, M, K)
    qb, sb = R.random_mx(rng, N, K)
    qa[:, -16:], qb[:, -16:] = 0, 0x88                    # +0 and -0
    sa[:, -1], sb[:, -1] = 254, 254
    c = host(m.mxfp4_matmul(dev_u8(qa), dev_u8(sa), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32))
    want, s = f64(R.mx_values(qa, sa), R.mx_values(qb, sb))
    R.assert_product(c, want, (K + 16) * (R.U * s + 2.0 ** -126), False)


# --------------------------------------------------------- few tokens, wide weight
@pytest.mark.parametrize("M,N,K,act", [(1, 25000, 160, "mxfp4"), (3, 24640, 288, "mxfp4"), (1, 51300, 128, "fp8")])
def test_few_tokens_by_a_wide_weight(M, N, K, act):
    m = need_gpu()
    rng = np.random.default_rng(N)
    q, s, va = operand(rng, act, M, K)
    qb, sb, vb = operand(rng, "mxfp4", N, K)
    g = Guarded(M * N * 4)
    c = m.mxfp4_matmul(*dev(q, s), dev_u8(qb), dev_u8(sb), out=g.view(torch.float32, (M, N)))
    torch.cuda.synchronize()
    g.check()
    R.assert_product(host(c), *R.product(va, vb), False)


# ---------------------------------------------------------------------- precision
@pytest.mark.parametrize("M,N,K", [(4, 16, 64), (20, 40, 128), (1024, 1024, 256)])
def test_blocks_that_cancel(M, N, K):
    """A block whose two large products cancel, up to 2^40 above its neighbour,
    leaves the neighbour's sum."""
    m = need_gpu()
    for d in range(0, 41, 4):
        for big, small in ((0, 1), (1, 0), (0, K // 32 - 1)):
            for at in ((0, 1), (0, 31), (3, 16)):
                ca, cb = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
                ca[:, 32 * big + at[0]], ca[:, 32 * big + at[1]] = 7, 15          # 6 and -6
                cb[:, 32 * big + at[0]] = cb[:, 32 * big + at[1]] = 7
                ca[:, 32 * small:32 * small + 32] = 3                             # 1.5
                cb[:, 32 * small:32 * small + 32] = 1                             # 0.5
                cb[:, 32 * small + 7] = 5                                         # 3
                sa, sb = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
                sa[:, big], sb[:, big] = 127 + d // 2, 127 + d // 2
                c = host(m.mxfp4_matmul(dev_u8(F.pack_codes(ca)), dev_u8(sa), dev_u8(F.pack_codes(cb)), dev_u8(sb),
                                        out_dtype=torch.float32)).astype(np.float64)
                want = 1.5 * (31 * 0.5 + 3)
                assert np.abs(c - want).max() <= 34 * 2.0 ** -23 * (36 * 2.0 ** d + want), (d, big, small, at)


@pytest.mark.parametrize("M,N", [(8, 64), (64, 64), (300, 300), (1024, 1024), (1700, 1290)])
@pytest.mark.parametrize("act", ["mxfp4", "fp8"])
def test_random_rows(M, N, act):
    """Relative RMS error of fp32 outputs at K = 2048, codes over their whole range."""
    m = need_gpu()
    rng = np.random.default_rng(M)
    K = 2048
    q, s, va = operand(rng, act, M, K)
    qb, sb, vb = operand(rng, "mxfp4", N, K)
    c = host(m.mxfp4_matmul(*dev(q, s), dev_u8(qb), dev_u8(sb), out_dtype=torch.float32))
    want, _ = f64(va, vb)
    assert np.sqrt(np.square(c - want).sum() / np.square(want).sum()) <= 2.0 ** -24 * (K / 2) ** 0.5


@pytest.mark.parametrize("M,N,E", [(256, 384, 1), (2048, 2048, 8)])
def test_random_columns(M, N, E):
    """The same of the weight gradient over 2048 tokens an expert: 128- and 256-row tiles."""
    m = need_gpu()
    rng = np.random.default_rng(M)
    K = 2048
    off = R.offsets_of([K] + [0] * (E - 1))
    (qa, sa), (qb, sb) = R.random_columns(rng, off, M), R.random_columns(rng, off, N)
    c = host(m.fp8_matmul_tokblk(dev_u8(qa), dev_f32(sa), dev_u8(qb), dev_f32(sb), dev_i64(off), M, N,
                                 out_dtype=torch.float32))[0]
    want, _ = f64(R.column_values(qa, sa, off, M)[0], R.column_values(qb, sb, off, N)[0])
    assert np.sqrt(np.square(c - want).sum() / np.square(want).sum()) <= 2.0 ** -24 * (K / 2) ** 0.5

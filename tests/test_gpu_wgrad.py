"""fp8_matmul_tokblk against 64-bit products of the decoded columns, within the
derived bounds of ops_ref, with guard bands."""
import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import Guarded, dev_f32, dev_i64, dev_u8, host, host_bf16, need_gpu
from oracle import formats as F

pytestmark = pytest.mark.gpu


def check(m, rng, counts, M, N, out, cols=None):
    print(f"wgrad {counts} M={M} N={N} {out}", flush=True)
    off = R.offsets_of(counts)
    E = len(counts)
    qa, sa = cols[0] if cols else R.random_columns(rng, off, M)
    qb, sb = cols[1] if cols else R.random_columns(rng, off, N)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    g = Guarded(E * M * N * (2 if out == "bf16" else 4))
    c = m.fp8_matmul_tokblk(dev_u8(qa), dev_f32(sa), dev_u8(qb), dev_f32(sb), dev_i64(off), M, N,
                            out=g.view(dt, (E, M, N)))
    torch.cuda.synchronize()
    g.check()
    got = F.bf16_bits_to_f32(host_bf16(c)) if out == "bf16" else host(c)
    va, vb = R.column_values(qa, sa, off, M), R.column_values(qb, sb, off, N)
    for e in range(E):
        if counts[e] == 0:
            assert (got[e] == 0).all()
        else:
            R.assert_product(got[e], *R.product(va[e], vb[e]), out == "bf16")


@pytest.mark.parametrize("counts", [[1], [0, 2, 0], [3, 0, 31, 32, 33], [127, 128, 129], [16, 256, 5, 0], [500, 1, 383]])
@pytest.mark.parametrize("M,N,out", [(128, 128, "f32"), (256, 384, "bf16"), (384, 128, "f32")])
def test_ragged_shards(counts, M, N, out):
    m = need_gpu()
    check(m, np.random.default_rng(sum(counts) + M + N), counts, M, N, out)


@pytest.mark.parametrize("counts,M,N", [([700, 3, 1029], 512, 640), ([2048], 768, 256), ([1, 1, 1, 1, 1, 90] * 12, 128, 256)])
def test_more_shapes(counts, M, N):
    m = need_gpu()
    check(m, np.random.default_rng(sum(counts)), counts, M, N, "f32")


def test_from_converted_rows():
    """Columns that mxfp4_row_to_fp8_col_tokblk made from MXFP4 rows."""
    m = need_gpu()
    rng = np.random.default_rng(6)
    counts = [140, 0, 61, 300]
    off = R.offsets_of(counts)
    cols = []
    for ch in (256, 384):
        q, s = R.random_mx(rng, int(off[-1]), ch, 110, 135)
        o, sc = m.mxfp4_row_to_fp8_col_tokblk(dev_u8(q), dev_u8(s), dev_i64(off), ch)
        torch.cuda.synchronize()
        cols.append((host(o), host(sc)))
    check(m, rng, counts, 256, 384, "f32", cols)


def test_smallest_scale():
    m = need_gpu()
    rng = np.random.default_rng(7)
    off = R.offsets_of([130])
    a = R.random_columns(rng, off, 128, -127, -125)
    b = R.random_columns(rng, off, 128, 110, 112)
    check(m, rng, [130], 128, 128, "f32", [a, b])


def test_no_tokens_gives_zeros():
    m = need_gpu()
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    s = torch.zeros(128 * 3, dtype=torch.float32, device="cuda")
    c = m.fp8_matmul_tokblk(e, s, e, s, dev_i64(np.zeros(4, np.int64)), 128, 128)
    torch.cuda.synchronize()
    assert c.shape == (3, 128, 128) and (c == 0).all()


def test_malformed_offsets_stay_inside():
    m = need_gpu()
    rng = np.random.default_rng(8)
    T, E, M, N = 300, 3, 128, 256
    nb = -(-T // 128) + E
    qa, qb = (rng.integers(0, 120, T * x, dtype=np.uint8) for x in (M, N))
    sa, sb = (np.ones(x * nb, np.float32) for x in (M, N))
    for off in ([0, 200, 100, 300], [-5, 20, 900, 1 << 40], [300, 0, 300, 0]):
        g = Guarded(E * M * N * 4)
        m.fp8_matmul_tokblk(dev_u8(qa), dev_f32(sa), dev_u8(qb), dev_f32(sb), dev_i64(np.array(off)), M, N,
                            out=g.view(torch.float32, (E, M, N)))
        torch.cuda.synchronize()
        g.check()


def test_binding_refuses():
    m = need_gpu()
    off = dev_i64(np.array([0, 4]))
    q = torch.zeros(4 * 128, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2 * 128, dtype=torch.float32, device="cuda")
    with pytest.raises(ValueError):
        m.fp8_matmul_tokblk(q, s, q, s, off, 128, 256)              # b too short
    with pytest.raises(ValueError):
        m.fp8_matmul_tokblk(q, s[:128].contiguous(), q, s, off, 128, 128)
    with pytest.raises(TypeError):
        m.fp8_matmul_tokblk(q, s, q, s, off.int(), 128, 128)
    with pytest.raises(m.Fp4Error):
        m.fp8_matmul_tokblk(q, s, q, s, off, 128, 128, out_dtype=torch.float16)


def test_zero_blocks_and_far_apart_scales():
    m = need_gpu()
    rng = np.random.default_rng(9)
    counts = [200, 300]
    off = R.offsets_of(counts)
    qa, sa = R.random_columns(rng, off, 128)
    qb, sb = R.random_columns(rng, off, 256)
    at = R.column_scale_start(off, 128)
    qa[3 * 200:4 * 200] = 0
    sa[at[0] + 6:at[0] + 8] = 2.0 ** -127                # a channel of zeros
    check(m, rng, counts, 128, 256, "f32", [(qa, sa), (qb, sb)])
    sa[at[1] + 30] = 2.0 ** 102                          # outside the window; products stay below 2^125
    check(m, rng, counts, 128, 256, "f32", [(qa, sa), (qb, sb)])


@pytest.mark.parametrize("counts,M,N", [([130, 0, 300, 65] * 8, 1024, 1152), ([1100, 5], 4096, 4224)])
def test_larger_outputs(counts, M, N):
    """Enough tiles for the larger of the two tile shapes, with a half tile at
    the end of either side."""
    m = need_gpu()
    check(m, np.random.default_rng(M), counts, M - 128, N, "f32" if M < 2000 else "bf16")


@pytest.mark.parametrize("last", list(range(1, 18)))
def test_few_tokens_at_the_end(last):
    """Shards of 1 to 17 tokens in the middle and at the end of the operands:
    every byte alignment, and loads that would pass the end."""
    m = need_gpu()
    check(m, np.random.default_rng(last), [3, last, 0, 20 - last, 1, last], 128, 384, "f32")
    check(m, np.random.default_rng(last), [last], 256, 128, "f32")

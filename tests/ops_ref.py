"""64-bit references of the operators over quantized rows, and the error bounds
their tests use.

Products of decoded values are exact in fp64 here (at most 8 significant bits
times a power of two), so the reference sums carry only fp64 rounding.  The
kernels add K exact products in fp32 in some order; with u = 2^-23 per
addition (truncation allowed for) the error of a sum is at most
(K + 16) u sum|a b|, 16 for the joins of partial sums and the row factor.
Rounding to bf16 adds 2^-8 |c|, to fp32 2^-23 |c|.  Results below the smallest normal fp32
may be flushed: an absolute 2^-126 (K + 16) covers that."""
import numpy as np

from oracle import formats as F
from oracle import mxfp4

U = 2.0 ** -23


def mx_values(packed, sb):
    codes = F.unpack_codes(packed)
    v = F.e2m1_decode(codes).astype(np.float64)
    return v * np.repeat(np.exp2(sb.astype(np.float64) - 127.0), 32, axis=-1)


def fp8_values(q, s):
    return F.e4m3_decode(q).astype(np.float64) * np.repeat(s.astype(np.float64), 128, axis=-1)


def product(a, b, row=None):
    """(c, bound on the fp32 sums' error) of a [M, K] . b [N, K]^T times row."""
    c, s = a @ b.T, np.abs(a) @ np.abs(b).T
    bound = (a.shape[1] + 16) * (U * s + 2.0 ** -126)
    if row is not None:
        r = row.astype(np.float64)[:, None]
        c, bound = c * r, bound * np.abs(r)
    return c, bound


def assert_product(got, c, bound, bf16):
    got = got.astype(np.float64)
    tol = bound + (2.0 ** -8 if bf16 else U) * np.abs(c)
    bad = ~(np.abs(got - c) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.max(np.abs(got - c) / np.maximum(tol, 1e-300))))


def random_mx(rng, rows, k, lo=118, hi=130):
    return (rng.integers(0, 256, (rows, k // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (rows, k // 32), dtype=np.uint8))


def random_fp8(rng, rows, k, lo=-9, hi=3):
    q = rng.integers(0, 256, (rows, k), dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] ^= 1                       # no NaN codes
    return q, np.exp2(rng.integers(lo, hi + 1, (rows, k // 128))).astype(np.float32)


def fp8_block_quantize(z):
    """fp32 z [rows, cols] -> (E4M3 bytes, scales): the least power of two 2^k,
    k >= -126, with amax <= 448 * 2^k; 2^-127 for a block of zeros."""
    b = z.astype(np.float64).reshape(z.shape[0], -1, 128)
    am = np.abs(b).max(-1)
    k = np.full(am.shape, -126, dtype=np.int64)
    for e in range(-126, 128):
        k = np.where(am > 448.0 * 2.0 ** e, e + 1, k)
    q = b * np.exp2(-k.astype(np.float64))[..., None]
    code = F.e4m3_encode(np.abs(q)) | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)
    s = np.where(am > 0, np.exp2(k.astype(np.float64)), 2.0 ** -127).astype(np.float32)
    return code.reshape(z.shape).astype(np.uint8), s


def column_scale_start(offsets, ch):
    return [ch * (-(-int(offsets[e]) // 128) + e) for e in range(len(offsets) - 1)]


def column_values(q, s, offsets, ch):
    """FP8 columns with 128-token blocks -> list of float64 [ch, n_e]."""
    out = []
    for e, at in enumerate(column_scale_start(offsets, ch)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        nb = -(-(hi - lo) // 128)
        v = F.e4m3_decode(q[ch * lo:ch * hi]).astype(np.float64).reshape(ch, hi - lo)
        sc = s[at:at + ch * nb].astype(np.float64).reshape(ch, nb)
        out.append(v * np.repeat(sc, 128, axis=1)[:, :hi - lo] if hi > lo else v)
    return out


def random_columns(rng, offsets, ch, lo=-9, hi=3):
    """Random FP8 columns; scale slots that no block uses hold NaN."""
    t, e = int(offsets[-1]), len(offsets) - 1
    q = rng.integers(0, 256, t * ch, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] ^= 1
    s = np.full(ch * (-(-t // 128) + e), np.nan, dtype=np.float32)
    for x, at in enumerate(column_scale_start(offsets, ch)):
        n = ch * -(-(int(offsets[x + 1]) - int(offsets[x])) // 128)
        s[at:at + n] = np.exp2(rng.integers(lo, hi + 1, n))
    return q, s


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def rmsnorm_backward(dy, h, w, r, dh=None):
    """float64 gradient of r h w with r held as given."""
    dy, h, w, r = (np.asarray(v, dtype=np.float64) for v in (dy, h, w, r))
    g, rr = dy * w, r[:, None]
    dx = rr * (g - h * rr * rr * (g * h).mean(-1, keepdims=True))
    return (dx if dh is None else dx + dh), (dy * h * rr).sum(0)

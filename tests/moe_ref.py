"""64-bit references of the FP8 step's operators, and the bounds their tests use.

Rounding to E4M3 is off by half a step at most: 2^-4 relative, 2^-10 absolute
below 2^-6.  Where the value that is rounded went through fp32 operations, `slack`
is their relative error, which moves a value across a boundary at most by itself.
"""
import numpy as np
import torch

from ops_ref import U
from oracle import formats as F


def fp8_quantize(z, rows=1):
    """z [R, C] (R % rows == 0) -> E4M3 bytes, scales [R/rows, C/128], one for
    rows x 128 values: the least 2^k, k >= -126, with amax <= 448 2^k; 2^-127 for
    zeros."""
    z = np.asarray(z, dtype=np.float64)
    r, c = z.shape
    b = z.reshape(r // rows, rows, c // 128, 128)
    am = np.abs(b).max((1, 3))
    k = least_exponent(am)
    q = (b * np.exp2(-k.astype(np.float64))[:, None, :, None]).reshape(r, c)
    code = F.e4m3_encode(np.abs(q)) | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)
    return code.astype(np.uint8), np.where(am > 0, np.exp2(k.astype(np.float64)), 2.0 ** -127).astype(np.float32)


def least_exponent(am):
    m, e = np.frexp(am)                       # am = m 2^e, 448 = 0.875 * 2^9
    return np.where(am > 0, np.clip(np.where(m <= 0.875, e - 9, e - 8), -126, 127), -126)


def values(q, s, rows=1):
    v = F.e4m3_decode(q).astype(np.float64)
    s = np.repeat(np.repeat(s.astype(np.float64), 128, axis=-1), rows, axis=-2)
    return v * s[..., :v.shape[-2], :]


def assert_rows(q, s, y, fmt, slack, floor=0.0):
    """Codes (bytes) and scales hold y [R, C] rounded to rows of fmt, y being known
    to `slack` relative (and `floor` absolute)."""
    y = np.asarray(y, dtype=np.float64)
    block = 128 if fmt == "fp8" else 32
    am = np.abs(y).reshape(y.shape[0], -1, block).max(-1)
    lo, hi = np.maximum(am * (1 - slack) - floor, 0), am * (1 + slack) + floor
    if fmt == "fp8":
        assert ((s >= np.exp2(least_exponent(lo).astype(float))) | (s == np.float32(2.0 ** -127))).all()
        assert (s <= np.exp2(least_exponent(hi).astype(float))).all()
        assert ((s > 2.0 ** -127) | (lo == 0)).all()
        k = np.log2(s.astype(np.float64))
        got = F.e4m3_decode(q).astype(np.float64)
    else:
        def byte(a):
            return np.clip(np.frexp(a)[1] - 1 - 2 + 127, 0, 254) * (a > 0)
        assert ((s >= byte(lo)) & (s <= byte(hi))).all()
        k = s.astype(np.float64) - 127
        got = F.e2m1_decode(F.unpack_codes(q)).astype(np.float64)
    t = y * np.exp2(-np.repeat(k, block, axis=-1))
    e = np.floor(np.log2(np.maximum(np.abs(t), 1e-300)))
    if fmt == "fp8":
        half = np.exp2(np.maximum(e, -6) - 4)
    else:                                      # magnitudes 0 .5 1 1.5 2 3 4 6; 8 - 6 saturates
        half = np.exp2(np.clip(e, 0, 2) - 2) + np.maximum(np.abs(t) - 7, 0)
    bad = np.abs(got - t) > half + slack * np.abs(t) * 1.01 + floor * np.exp2(-np.repeat(k, block, axis=-1))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], t[bad][:4])


def product_bounds(a, b, row, bf16):
    """(c, bound) of a [M, K] . b [N, K]^T: fp32 sums in any order, (K + 16) U
    sum|a b|, and for bf16 outputs 7 * 2^-13 of the largest product in each run of 8
    k beside the rounding."""
    c, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    bound = (a.shape[1] + 16) * (U * mag + 2.0 ** -126)
    if bf16:
        x, y = (torch.from_numpy(np.ascontiguousarray(np.abs(v))).view(v.shape[0], -1, 8) for v in (a, b))
        for i in range(a.shape[0]):
            bound[i] += 7 * 2.0 ** -13 * (x[i] * y).amax(-1).sum(-1).numpy()
    if row is not None:
        r = row.astype(np.float64)[:, None]
        c, bound = c * r, bound * np.abs(r)
    return c, bound


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


def swiglu(x):
    f = x.shape[-1] // 2
    g, u = x[:, :f].astype(np.float64), x[:, f:].astype(np.float64)
    return g * sigmoid(g) * u


def swiglu_backward(x, dy):
    """(dx, size of the terms it is a sum of) at x = [g | u]."""
    f = x.shape[-1] // 2
    g, u, dy = (np.asarray(v, dtype=np.float64) for v in (x[:, :f], x[:, f:], dy))
    s, r = sigmoid(g), sigmoid(-g)
    dx = np.concatenate([dy * u * s * (1 + g * r), dy * g * s], 1)
    return dx, np.concatenate([np.abs(dy * u * s) * (1 + np.abs(g) * r), np.abs(dy * g * s)], 1)


def balance(logits, experts, coef, mask=None):
    """(loss, counts, prob_grad, p) with p the softmax rows (0 for a row of -inf)."""
    x = np.asarray(logits, dtype=np.float64)
    t, e = x.shape
    keep = np.ones(t, bool) if mask is None else mask.astype(bool)
    p = softmax(x)
    idx = experts[keep].reshape(-1)
    counts = np.bincount(idx[(idx >= 0) & (idx < e)], minlength=e)
    n = int(keep.sum())
    if n == 0:
        return 0.0, counts, np.zeros(e), p
    v = coef * e * counts / (experts.shape[1] * float(n) ** 2)
    return float((v * p[keep].sum(0)).sum()), counts, v, p


def softmax(x):
    with np.errstate(invalid="ignore"):
        top = x.max(-1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0, top))
        s = e.sum(-1, keepdims=True)
        return np.where(s == 0, 0, e / np.where(s == 0, 1, s))

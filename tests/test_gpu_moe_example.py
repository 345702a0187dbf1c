"""examples/moe_train_step.py against the same step in 64 bits on unquantized
weights, and the operators in captured graphs.

Bounds: MXFP4 rounds Gaussian values by about 11% (relative RMS), so a product
of two rounded operands is off by about 16%; `out` holds h unrounded beside one
such chain of two products (below 25%, and h is larger), each weight gradient
is two roundings beside the forward's own error and one more on the way back
(below 35%), dx holds dout unrounded beside three products (below 35%)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import ops_ref as R
from gpu_util import dev_f32, dev_i64, dev_u8, need_gpu
from test_gpu_graphs import _replay_check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,hidden,ffn,experts", [(300, 512, 256, 8), (1, 256, 128, 4), (1000, 1024, 384, 40)])
def test_train_step(tokens, hidden, ffn, experts):
    need_gpu()
    spec = importlib.util.spec_from_file_location("moe_train_step", os.path.join(ROOT, "examples", "moe_train_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    off_by = ex.main(tokens, hidden, ffn, experts)
    assert off_by["out"] < 0.25, off_by
    for n in ("dx", "dgamma", "dw1", "dw2"):
        assert off_by[n] < 0.35, off_by


def test_operators_in_graphs():
    """Each operator captured and replayed, bit for bit like the eager call."""
    m = need_gpu()
    rng = np.random.default_rng(0)
    off = R.offsets_of([300, 0, 212, 500])
    T, K, N = int(off[-1]), 512, 384
    qa, sa = (dev_u8(t) for t in R.random_mx(rng, T, K))
    q8, s8 = R.random_fp8(rng, T, K)
    q8, s8 = dev_u8(q8), dev_f32(s8)
    qw, sw = R.random_mx(rng, 4 * N, K)
    qw, sw = dev_u8(qw.reshape(4, N, -1)), dev_u8(sw.reshape(4, N, -1))
    offd = dev_i64(off)
    c = torch.empty((T, N), device="cuda")
    for rows in (1, 100, T):
        o = c[:rows]
        _replay_check(lambda: m.mxfp4_matmul(qa[:rows], sa[:rows], qw[0], sw[0], out=o), [o])
        _replay_check(lambda: m.mxfp4_matmul(q8[:rows], s8[:rows], qw[0], sw[0], out=o), [o])
    _replay_check(lambda: m.mxfp4_matmul_grouped(qa, sa, qw, sw, offd, out=c), [c])
    _replay_check(lambda: m.mxfp4_matmul_grouped(q8, s8, qw, sw, offd, out=c), [c])
    ca, cb = R.random_columns(rng, off, 256), R.random_columns(rng, off, 128)
    args = [dev_u8(ca[0]), dev_f32(ca[1]), dev_u8(cb[0]), dev_f32(cb[1])]
    dw = torch.empty((4, 256, 128), device="cuda")
    _replay_check(lambda: m.fp8_matmul_tokblk(*args, offd, 256, 128, out=dw), [dw])
    x = torch.randn((700, 1024), device="cuda").to(torch.bfloat16)
    w = torch.randn(1024, device="cuda")
    q, s, r, h = m.rmsnorm_quantize(x, w, residual=x)
    _replay_check(lambda: m.rmsnorm_quantize(x, w, residual=x, q=q, scales=s, row_scale=r, h=h), [q, s, r, h])
    dx, dweight = m.rmsnorm_backward(x, h, w, r)
    ws = torch.empty(m.rmsnorm_backward_workspace(700, 1024), dtype=torch.uint8, device="cuda")
    _replay_check(lambda: m.rmsnorm_backward(x, h, w, r, dx=dx, dweight=dweight, workspace=ws), [dx, dweight])


def test_offsets_past_32_bits():
    """Operands and outputs over 4 GiB: the last rows of a product, the last
    expert's weights and gradient, the last rows of the norm."""
    m = need_gpu()
    rng = np.random.default_rng(5)
    # output of 2^32 + elements: 1.2e6 tokens x 4096 in bf16 (9.8 GB); MXFP4 rows of K = 64
    T, N, K = 1_200_000, 4096, 64
    qb, sb = R.random_mx(rng, N, K)
    qa, sa = R.random_mx(rng, 640, K)
    a = torch.zeros((T, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((T, K // 32), 127, dtype=torch.uint8, device="cuda")
    a[-640:], s[-640:] = dev_u8(qa), dev_u8(sa)
    c = m.mxfp4_matmul(a, s, dev_u8(qb), dev_u8(sb))
    torch.cuda.synchronize()
    want, bound = R.product(R.mx_values(qa, sa), R.mx_values(qb, sb))
    R.assert_product(c[-640:].float().cpu().numpy(), want, bound, True)
    assert not c[:1000].any()
    del a, s, c
    # weights of 4.3 GB: 9 experts x 16384 x 58368
    E, N, K = 9, 16384, 58368
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    qb, sb = R.random_mx(rng, 48, K)
    w[-1, -48:], ws[-1, -48:] = dev_u8(qb), dev_u8(sb)
    for rows in (5, 300):
        qa, sa = R.random_mx(rng, rows, K)
        off = dev_i64(np.array([0] * E + [rows]))
        c = m.mxfp4_matmul_grouped(dev_u8(qa), dev_u8(sa), w, ws, off, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want, bound = R.product(R.mx_values(qa, sa), R.mx_values(qb, sb))
        R.assert_product(c[:, -48:].cpu().numpy(), want, bound, False)
    del w, ws
    # gradient of 4.8 GB in fp32: 9 x 11520 x 11520; only the last expert has tokens
    E, M = 9, 11520
    off = np.array([0] * E + [40], np.int64)
    ca, cb = R.random_columns(rng, off, M), R.random_columns(rng, off, M)
    c = m.fp8_matmul_tokblk(dev_u8(ca[0]), dev_f32(ca[1]), dev_u8(cb[0]), dev_f32(cb[1]), dev_i64(off), M, M,
                            out_dtype=torch.float32)
    torch.cuda.synchronize()
    va, vb = R.column_values(*ca, off, M)[-1], R.column_values(*cb, off, M)[-1]
    want, bound = R.product(va[-200:], vb[-300:])
    R.assert_product(c[-1, -200:, -300:].cpu().numpy(), want, bound, False)
    assert not c[:-1].any()
    del c
    # norm over 2^32 + elements of bf16
    rows, cols = 1_100_000, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((64, cols), device="cuda").to(torch.bfloat16)
    x[-64:] = tail
    wt = torch.ones(cols, device="cuda")
    q, s, r, _ = m.rmsnorm_quantize(x, wt)
    q2, s2, r2, _ = m.rmsnorm_quantize(tail, wt)
    torch.cuda.synchronize()
    assert torch.equal(q[-64:], q2) and torch.equal(s[-64:], s2) and torch.equal(r[-64:], r2)
    dx, dw = m.rmsnorm_backward(x, x, wt, r)
    dx2, dw2 = m.rmsnorm_backward(tail, tail, wt, r2)
    torch.cuda.synchronize()
    assert torch.equal(dx[-64:], dx2)
    assert torch.allclose(dw, dw2, rtol=2e-5, atol=0)

"""From the norm's rows to a weight gradient, as fp4mi_ops.h says it has to be
done: the rows lack row_scale, so dY's rows take it before they are quantized.

dW in 64 bits from unquantized data; MXFP4 rounds Gaussian values by about 11%
(relative RMS), so a product of two rounded operands is off by about 16%
(bound 25%).  Rows differ in size by up to e^4, so that a gradient without the
factor is another one."""
import numpy as np
import pytest
import torch

from gpu_util import dev_i64, need_gpu

pytestmark = pytest.mark.gpu


def test_row_scale_goes_into_dy():
    m = need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    T, H, N, off = 700, 512, 256, [0, 300, 300, 700]
    x = torch.randn(T, H, generator=g, device="cuda") * torch.exp(4 * torch.rand(T, 1, generator=g, device="cuda"))
    x, gamma = x.to(torch.bfloat16), 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    dy = torch.randn(T, N, generator=g, device="cuda").to(torch.bfloat16)
    q, s, r, _ = m.rmsnorm_quantize(x, gamma, fmt="mxfp4")
    offd = dev_i64(np.array(off))
    qc, qcs = m.mxfp4_row_to_fp8_col_tokblk(q, s, offd, H)

    def gradient(rows):
        p, ps, _ = m.fp4_quantize(rows.to(torch.bfloat16), "mxfp4")
        return m.fp8_matmul_tokblk(*m.mxfp4_row_to_fp8_col_tokblk(p, ps, offd, N), qc, qcs, offd, N, H,
                                   out_dtype=torch.float32).double()

    h = x.double()
    y = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma.double()
    want = torch.stack([dy[a:b].double().t().contiguous() @ y[a:b] for a, b in zip(off, off[1:])])
    assert (gradient(dy * r.unsqueeze(-1)) - want).norm() < 0.25 * want.norm()
    assert (gradient(dy) - want).norm() > want.norm()

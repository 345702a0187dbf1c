"""One training step of a mixture-of-experts layer on quantized operands.

    out = h + sum_k gate_k W2[e_k] silu(W1[e_k] norm(h)),   h = x + residual

Every product reads MXFP4 rows or FP8 columns; the norm writes MXFP4 rows with
its row factor apart; the gradients of both products come from MXFP4 rows
(data) and from FP8 columns over each expert's tokens (weights).  Routing and
gates count as constants in the backward pass.

    python examples/moe_train_step.py [tokens hidden ffn experts]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_amd as fp4  # noqa: E402


def mx(w, **kw):
    """MXFP4 rows of [.., rows, cols], in the shape of w."""
    p, s, _ = fp4.fp4_quantize(w.contiguous(), "mxfp4", **kw)
    return p.view(*w.shape[:-1], -1), s.view(*w.shape[:-1], -1)


class MoELayer:
    def __init__(self, hidden, ffn, experts, top_k=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.experts, self.top_k, self.hidden, self.ffn = experts, top_k, hidden, ffn
        self.gamma = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)
        self.router = draw(experts, hidden)
        self.w1, self.w2 = draw(experts, ffn, hidden), draw(experts, hidden, ffn)
        # quantized along the axis that each product contracts
        self.router_q = mx(self.router)
        self.w1_q, self.w2_q = mx(self.w1), mx(self.w2)
        self.w1t_q, self.w2t_q = mx(self.w1.transpose(1, 2)), mx(self.w2.transpose(1, 2))

    def forward(self, x, residual):
        q, s, r, h = fp4.rmsnorm_quantize(x, self.gamma, residual=residual, fmt="mxfp4")
        logits = fp4.mxfp4_matmul(q, s, *self.router_q, a_row_scale=r, out_dtype=torch.float32)
        gate, expert = torch.softmax(logits, -1).topk(self.top_k, -1)
        order = expert.flatten().argsort(stable=True)                # tokens by expert
        tok, gate = order // self.top_k, gate.flatten()[order].unsqueeze(-1)
        off = torch.zeros(self.experts + 1, dtype=torch.int64, device=x.device)
        off[1:] = torch.bincount(expert.flatten(), minlength=self.experts).cumsum(0)
        qx, sx, rx = q[tok], s[tok], r[tok]
        u = fp4.mxfp4_matmul_grouped(qx, sx, *self.w1_q, off, a_row_scale=rx)
        qa, sa = mx(torch.nn.functional.silu(u))
        y = fp4.mxfp4_matmul_grouped(qa, sa, *self.w2_q, off)
        out = h.float().index_add_(0, tok, gate * y.float()).to(x.dtype)
        return out, (h, r, tok, gate, off, qx, sx, rx, u, qa, sa)

    def backward(self, dout, saved, step=0):
        """-> (dx, dgamma, dw1, dw2); dx is the residual's gradient too."""
        h, r, tok, gate, off, qx, sx, rx, u, qa, sa = saved
        H, F = self.hidden, self.ffn

        def cols(q, s, width):
            return fp4.mxfp4_row_to_fp8_col_tokblk(q, s, off, width)

        dy = mx((gate * dout[tok].float()).to(torch.bfloat16), rounding="sr", seed=1, step=step)
        dw2 = fp4.fp8_matmul_tokblk(*cols(*dy, H), *cols(qa, sa, F), off, H, F)
        da = fp4.mxfp4_matmul_grouped(*dy, *self.w2t_q, off)
        sig = torch.sigmoid(u.float())
        du = da.float() * sig * (1 + u.float() * (1 - sig))
        # the rows of the norm lack their factor, so the gradient's rows take it
        dur = mx((du * rx.unsqueeze(-1)).to(torch.bfloat16), rounding="sr", seed=2, step=step)
        dw1 = fp4.fp8_matmul_tokblk(*cols(*dur, F), *cols(qx, sx, H), off, F, H)
        duq = mx(du.to(torch.bfloat16), rounding="sr", seed=3, step=step)
        dn = fp4.mxfp4_matmul_grouped(*duq, *self.w1t_q, off, out_dtype=torch.float32)
        dn = torch.zeros(h.shape, device=h.device).index_add_(0, tok, dn).to(h.dtype)
        dx, dgamma = fp4.rmsnorm_backward(dn, h, self.gamma, r, dh=dout)
        return dx, dgamma, dw1, dw2


def plain_step(layer, x, residual, dout, routing):
    """The same step from the unquantized weights in 64 bits, on the routing
    that the quantized forward chose."""
    tok, gate, off = routing
    d = torch.float64
    v = {k: t.to(d).requires_grad_() for k, t in (("x", x), ("gamma", layer.gamma), ("w1", layer.w1), ("w2", layer.w2))}
    h = v["x"] + residual.to(d)
    n = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * v["gamma"]
    out = h
    for e in range(layer.experts):
        t = slice(int(off[e]), int(off[e + 1]))
        y = torch.nn.functional.silu(n[tok[t]] @ v["w1"][e].t()) @ v["w2"][e].t()
        out = out.index_add(0, tok[t], gate[t].to(d) * y)
    out.backward(dout.to(d))
    return out.detach(), [v[k].grad for k in ("x", "gamma", "w1", "w2")]


def main(tokens=4096, hidden=2048, ffn=1024, experts=16):
    layer = MoELayer(hidden, ffn, experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, res, dout = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    out, saved = layer.forward(x, res)
    grads = layer.backward(dout, saved)
    ref, ref_grads = plain_step(layer, x, res, dout, (saved[2], saved[3], saved[4]))
    off_by = {n: float((a.double() - b).norm() / b.norm())
              for n, a, b in zip(("out", "dx", "dgamma", "dw1", "dw2"), (out, *grads), (ref, *ref_grads))}
    print("relative difference from 64 bits:", ", ".join(f"{n} {e:.3f}" for n, e in off_by.items()))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for step in range(20):
        out, saved = layer.forward(x, res)
        layer.backward(dout, saved, step)
    torch.cuda.synchronize()
    print(f"{tokens} tokens, {hidden} -> {ffn}, {experts} experts: {(time.perf_counter() - t) / 20 * 1e3:.2f} ms a step")
    return off_by


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))

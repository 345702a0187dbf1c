"""One training step of a mixture-of-experts layer with FP8 weights, an 8-bit
checkpoint of the experts' hidden rows, and the router's balance loss.

    out = h + sum_k gate_k W2[e_k] (silu(g) * u),   [g | u] = W1[e_k] norm(h),
    h = x + residual;   loss = balance loss of the router's logits Wr norm(h)

The norm writes FP8 rows with its row factor apart; both products of an expert, and
their gradients with respect to the rows, read FP8 rows and FP8 blocks of weights
(the gradients their transposed copy).  Of the hidden rows only the FP8 checkpoint is
kept.  The weights' gradients go through MXFP4 rows into FP8 columns.  Gates count as
constants in the backward pass; the router learns from the balance loss.

    python examples/moe_fp8_train_step.py [tokens hidden ffn experts]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_amd as fp4  # noqa: E402


def mx(w, **kw):
    """MXFP4 rows of [rows, cols]."""
    p, s, _ = fp4.fp4_quantize(w.contiguous(), "mxfp4", **kw)
    return p, s


def values(q, s):
    """bf16 values of FP8 rows."""
    v = q.view(torch.float8_e4m3fn).float().view(*s.shape, 128) * s.unsqueeze(-1)
    return v.view(q.shape).to(torch.bfloat16)


class MoELayer:
    def __init__(self, hidden, ffn, experts, top_k=2, coef=0.01, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.experts, self.top_k, self.hidden, self.ffn, self.coef = experts, top_k, hidden, ffn, coef
        self.gamma = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)
        self.router = draw(experts, hidden)
        self.w1, self.w2 = draw(experts, 2 * ffn, hidden), draw(experts, hidden, ffn)
        self.quantize()

    def quantize(self):
        """FP8 weights, after each update of the masters."""
        self.router_q = fp4.fp8_quantize(self.router)
        q, s, qt, st = fp4.fp8_quantize_blocks(self.w1, transposed=True)
        self.w1_q, self.w1t_q = (q, s), (qt, st)
        q, s, qt, st = fp4.fp8_quantize_blocks(self.w2, transposed=True)
        self.w2_q, self.w2t_q = (q, s), (qt, st)

    def forward(self, x, residual, mask=None):
        """-> (out, balance loss, what the backward pass takes)."""
        q, s, r, h = fp4.rmsnorm_quantize(x, self.gamma, residual=residual, fmt="fp8")
        logits = fp4.fp8_matmul(q, s, *self.router_q, a_row_scale=r, out_dtype=torch.float32)
        gate, expert = torch.softmax(logits, -1).topk(self.top_k, -1)
        loss, counts, off, prob_grad = fp4.router_balance(logits, expert, self.coef, mask)
        if mask is not None:                                # slots of tokens that do not count go nowhere
            expert = expert.masked_fill(~mask.unsqueeze(-1), self.experts)
        order = expert.flatten().argsort(stable=True)       # slots by expert
        if mask is not None:
            order = order[:int(off[-1])]
        tok, gate = order // self.top_k, gate.flatten()[order].unsqueeze(-1)
        qx, sx, rx = q[tok], s[tok], r[tok]
        u = fp4.fp8_matmul_grouped(qx, sx, *self.w1_q, off, a_row_scale=rx)
        qa, sa, kept, kept_s = fp4.swiglu_quantize(u, "fp8")
        y = fp4.fp8_matmul_grouped(qa, sa, *self.w2_q, off)
        out = h.float().index_add_(0, tok, gate * y.float()).to(x.dtype)
        return out, loss, (h, r, q, s, logits, prob_grad, mask, tok, gate, off, qx, sx, rx, qa, sa, kept, kept_s)

    def backward(self, dout, dloss, saved, step=0):
        """-> (dx, dgamma, drouter, dw1, dw2); dx is the residual's gradient too."""
        h, r, q, s, logits, prob_grad, mask, tok, gate, off, qx, sx, rx, qa, sa, kept, kept_s = saved
        H, F = self.hidden, self.ffn

        def cols(rows, width):
            return fp4.mxfp4_row_to_fp8_col_tokblk(*rows, off, width)

        dy = (gate * dout[tok].float()).to(torch.bfloat16)
        dw2 = fp4.fp8_matmul_tokblk(*cols(mx(dy, rounding="sr", seed=1, step=step), H), *cols(mx(values(qa, sa)), F), off, H, F)
        da = fp4.fp8_matmul_grouped(*fp4.fp8_quantize(dy), *self.w2t_q, off)
        du = torch.empty(kept.shape, dtype=da.dtype, device=da.device)
        _, duq, dus = fp4.swiglu_backward(da, kept, kept_s, fmt="fp8", dx=du)
        # the rows of the norm lack their factor, so the gradient's rows take it
        dur = mx((du * rx.unsqueeze(-1)).to(torch.bfloat16), rounding="sr", seed=2, step=step)
        dw1 = fp4.fp8_matmul_tokblk(*cols(dur, 2 * F), *cols(mx(values(qx, sx)), H), off, 2 * F, H)
        dn = fp4.fp8_matmul_grouped(duq, dus, *self.w1t_q, off, out_dtype=torch.float32)
        dlogits = fp4.router_balance_backward(logits, prob_grad, dloss, mask)
        drouter = dlogits.t() @ (values(q, s).float() * r.unsqueeze(-1))
        dn = (dlogits @ self.router.float()).index_add_(0, tok, dn).to(h.dtype)
        dx, dgamma = fp4.rmsnorm_backward(dn, h, self.gamma, r, dh=dout)
        return dx, dgamma, drouter, dw1, dw2


def plain_step(layer, x, residual, dout, dloss, mask, saved):
    """The same step from the unquantized weights in 64 bits, on the routing that the
    quantized forward chose."""
    tok, gate, off, prob_grad = saved[7], saved[8], saved[9], saved[5].double()
    d = torch.float64
    names = ("gamma", "router", "w1", "w2")
    v = {"x": x.to(d).requires_grad_(), **{n: getattr(layer, n).to(d).requires_grad_() for n in names}}
    h = v["x"] + residual.to(d)
    n = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * v["gamma"]
    p = torch.softmax(n @ v["router"].t(), -1)
    loss = (prob_grad * (p if mask is None else p[mask]).sum(0)).sum()
    out = h
    for e in range(layer.experts):
        t = slice(int(off[e]), int(off[e + 1]))
        u = n[tok[t]] @ v["w1"][e].t()
        y = (torch.nn.functional.silu(u[:, :layer.ffn]) * u[:, layer.ffn:]) @ v["w2"][e].t()
        out = out.index_add(0, tok[t], gate[t].to(d) * y)
    torch.autograd.backward([out, loss], [dout.to(d), dloss.to(d).reshape(())])
    return out.detach(), loss.detach(), [v[k].grad for k in ("x", *names)]


def main(tokens=4096, hidden=2048, ffn=1024, experts=16, masked=False):
    layer = MoELayer(hidden, ffn, experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, res, dout = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    mask = (torch.rand(tokens, generator=g, device="cuda") < 0.9) if masked else None
    dloss = torch.full((1,), 300.0, device="cuda")
    out, loss, saved = layer.forward(x, res, mask)
    grads = layer.backward(dout, dloss, saved)
    ref, ref_loss, ref_grads = plain_step(layer, x, res, dout, dloss, mask, saved)
    off_by = {n: float((a.double() - b).norm() / b.norm())
              for n, a, b in zip(("out", "loss", "dx", "dgamma", "drouter", "dw1", "dw2"), (out, loss, *grads),
                                 (ref, ref_loss.reshape(1), *ref_grads))}
    print("relative difference from 64 bits:", ", ".join(f"{n} {e:.3f}" for n, e in off_by.items()))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for step in range(20):
        out, loss, saved = layer.forward(x, res, mask)
        layer.backward(dout, dloss, saved, step)
    torch.cuda.synchronize()
    print(f"{tokens} tokens, {hidden} -> {ffn}, {experts} experts: {(time.perf_counter() - t) / 20 * 1e3:.2f} ms a step")
    return off_by


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))

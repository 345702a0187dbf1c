"""The router's balance loss and its gradient over more rows than the launches hold at
once: every lane goes round several times, with the next rows on their way, at each
width of a row, and the workgroups' parts are joined.  References in 64 bits on the GPU.

p_te is off by (16 + |x - max|) U relative (exponential, its argument's rounding, the sum
over lanes, the division).  The loss adds p in fp32, a lane's rows one after another,
then 64 / L rows of a wave and 16 waves at most, and what follows in fp64: at most (rounds +
24) U of the sum."""
import pytest
import torch

from gpu_util import Guarded, need_gpu
from ops_ref import U
from test_gpu_graphs import _replay_check

pytestmark = pytest.mark.gpu

# tokens, experts, k: a width of each kind, four rounds or more of the forward launch
# and two or more of the gradient's
SIZES = [(150001, 16, 2), (90001, 50, 4), (50001, 100, 3), (20001, 256, 8), (20001, 255, 1), (20001, 400, 2),
         (18001, 1000, 3), (17001, 1500, 2), (17001, 2048, 2), (17001, 2500, 2), (9001, 4096, 3)]


def rounds(t, e):
    """Rows that a lane of the forward launch takes at most."""
    rows = 128 if e <= 32 else 64 if e <= 64 else 32 if e <= 128 else 16 if e <= 512 else 8 if e <= 2048 else 4
    return -(-t // (256 * rows))


def inputs(t, e, k, bf16, masked):
    g = torch.Generator(device="cuda")
    g.manual_seed(t + e)
    x = 2 * torch.randn((t, e), generator=g, device="cuda") + torch.randn(e, generator=g, device="cuda")
    x[::3, 1] = -float("inf")
    x[5] = -float("inf")
    x[t - 2] *= 50.0
    x = x.to(torch.bfloat16) if bf16 else x
    idx = torch.randint(0, e, (t, k), generator=g, device="cuda")
    idx[3, 0], idx[t - 1, k - 1], idx[t // 2] = -1, e, e // 2
    mask = torch.rand(t, generator=g, device="cuda") < 0.5 if masked else None
    if masked:
        x[~mask & (torch.arange(t, device="cuda") % 5 == 0)] = float("nan")     # not counted, whatever it holds
    return x, idx, mask


def softmax(x):
    """(p, (16 + |x - max|) U) in fp64; 0 for a row of -inf."""
    x = x.double()
    top = x.amax(-1, keepdim=True)
    far = x - torch.where(top == -float("inf"), 0.0, top)
    p = torch.exp(far)
    s = p.sum(-1, keepdim=True)
    return p / torch.where(s == 0, 1.0, s), U * (16 + torch.where(far == -float("inf"), 0.0, -far))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("t,e,k", SIZES)
def test_forward_and_gradient(t, e, k, masked, bf16):
    m = need_gpu()
    assert rounds(t, e) >= 4
    x, idx, mask = inputs(t, e, k, bf16, masked)
    keep = torch.ones(t, dtype=torch.bool, device="cuda") if mask is None else mask
    n = int(keep.sum())
    flat = idx[keep].reshape(-1)
    counts = torch.bincount(flat[(flat >= 0) & (flat < e)], minlength=e)
    v = 0.01 * e * counts.double() / (k * float(n) ** 2)
    p, off_by = softmax(torch.where(keep[:, None], x, 0.0))
    size = (p * keep[:, None]).sum(0)
    want = float((v * size).sum())
    tol = float((v * (p * off_by * keep[:, None]).sum(0)).sum()) + (rounds(t, e) + 24) * U * want
    bufs = [Guarded(4), Guarded(4 * e), Guarded(8 * (e + 1)), Guarded(4 * e), Guarded(m.router_balance_workspace(t, e))]
    views = [bufs[0].view(torch.float32, (1,)), bufs[1].view(torch.int32, (e,)), bufs[2].view(torch.int64, (e + 1,)),
             bufs[3].view(torch.float32, (e,)), bufs[4].view(torch.uint8, (bufs[4].nbytes,))]
    for it in (torch.int64, torch.int32):
        loss, c, o, grad = m.router_balance(x, idx.to(it), 0.01, mask, *views)
        torch.cuda.synchronize()
        for b in bufs:
            b.check()
        assert torch.equal(c.long(), counts) and torch.equal(o[1:], torch.cumsum(counts, 0)) and int(o[0]) == 0
        assert bool(((grad.double() - v).abs() <= 2.0 ** -22 * v).all())
        assert abs(float(loss) - want) <= tol, (float(loss), want, tol)

    # the gradient, beside another one
    gen = torch.Generator(device="cuda")
    gen.manual_seed(e)
    add = (1e-3 * float(v.max()) * torch.randn((t, e), generator=gen, device="cuda")).to(x.dtype)
    dl = torch.tensor([0.37], device="cuda")
    v = grad.double()
    dot = (p * v).sum(-1, keepdim=True)
    ref = float(dl) * p * (v - dot) * keep[:, None]
    tol = 4 * float(dl) * (off_by.amax(-1, keepdim=True) + 16 * U) * p * (v + dot) + 1e-38
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    out = Guarded(t * e * x.element_size())
    got = m.router_balance_backward(x, grad, dl, mask, add, out.view(x.dtype, (t, e)))
    torch.cuda.synchronize()
    out.check()
    want = ref + add.double()
    assert bool(((got.double() - want).abs() <= tol + half * want.abs() * 1.01 + U * ref.abs()).all())
    del want
    alone = m.router_balance_backward(x, grad, dl, mask)
    assert bool(((alone.double() - ref).abs() <= tol + half * ref.abs() * 1.01).all())
    if mask is not None:
        assert not bool(alone[~mask].any()) and torch.equal(got[~mask], add[~mask])
    del p, off_by, ref, tol
    assert torch.equal(m.router_balance_backward(x, grad, dl, mask, add, add), got)      # in place of either
    assert torch.equal(m.router_balance_backward(x, grad, dl, mask, None, x), alone)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("t,e,k", [(90001, 50, 4), (20001, 256, 8), (17001, 2500, 2)])
def test_captured_and_replayed(t, e, k, bf16):
    m = need_gpu()
    x, idx, mask = inputs(t, e, k, bf16, True)
    o = m.router_balance(x, idx, 0.1, mask)
    work = torch.empty(m.router_balance_workspace(t, e), dtype=torch.uint8, device="cuda")
    _replay_check(lambda: m.router_balance(x, idx, 0.1, mask, *o, work), list(o))
    grad = torch.empty_like(x)
    _replay_check(lambda: m.router_balance_backward(x, o[3], None, mask, None, grad), [grad])

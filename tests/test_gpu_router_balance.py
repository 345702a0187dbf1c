"""The router's balance loss, counts and gradient against 64 bits.

p_te is off by the exponential (2 last places), its argument (x - max, rounded: its
size in last places), the sum of E terms over lanes, and a division: (16 + |x - max|)
of fp32's 2^-23 relative.  Sums of p over tokens in fp32 add at most one such a row
that a workgroup's lane takes, tokens / 256 + 64 here."""
import numpy as np
import pytest
import torch

import moe_ref as R
from gpu_util import Guarded, host, need_gpu
from ops_ref import U

pytestmark = pytest.mark.gpu


def inputs(rng, t, e, k, bf16, masked, wild=True):
    x = torch.from_numpy((2 * rng.standard_normal((t, e)) + rng.standard_normal(e)).astype(np.float32))
    if wild and e > 2:
        x[::3, 1] = -float("inf")
        if t > 8:
            x[5], x[7] = -float("inf"), 50.0 * x[7]
    x = x.to(torch.bfloat16) if bf16 else x
    idx = rng.integers(0, e, (t, k))
    if wild and t > 4:
        idx[3, 0], idx[4, k - 1], idx[2] = -1, e, e // 2         # out of range, and one expert k times
    mask = rng.random(t) < 0.7 if masked else None
    return x, idx, mask


def p_tol(x):
    x = x.double().numpy()
    with np.errstate(invalid="ignore"):
        far = np.where(np.isneginf(x), 0, x.max(-1, keepdims=True) - x)
    return U * (16 + np.nan_to_num(far, nan=0.0))


def dev_mask(mask):
    return None if mask is None else torch.from_numpy(mask).cuda()


SIZES = [(1, 1, 1), (1, 8, 2), (2, 3, 3), (7, 33, 4), (100, 61, 8), (513, 64, 1), (300, 130, 6), (1000, 256, 8),
         (77, 257, 2), (50, 511, 8), (40, 1000, 3), (9, 1025, 2), (11, 4096, 2), (20000, 16, 2),
         (700, 100, 3), (200, 400, 2), (150, 1000, 3), (100, 3000, 4), (3000, 5, 40),
         (300, 1100, 3), (70, 2048, 2), (70, 2049, 2)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("t,e,k", SIZES)
def test_forward(t, e, k, masked, bf16):
    m = need_gpu()
    x, idx, mask = inputs(np.random.default_rng(t + e), t, e, k, bf16, masked)
    loss, counts, v, p = R.balance(x.double().numpy(), idx, 0.01, mask)
    bufs = [Guarded(4), Guarded(4 * e), Guarded(8 * (e + 1)), Guarded(4 * e), Guarded(m.router_balance_workspace(t, e))]
    views = [bufs[0].view(torch.float32, (1,)), bufs[1].view(torch.int32, (e,)), bufs[2].view(torch.int64, (e + 1,)),
             bufs[3].view(torch.float32, (e,)), bufs[4].view(torch.uint8, (bufs[4].nbytes,))]
    for it in (torch.int64, torch.int32):
        got = m.router_balance(x.cuda(), torch.from_numpy(idx).to(it).cuda(), 0.01, dev_mask(mask), *views)
        torch.cuda.synchronize()
        for b in bufs:
            b.check()
        np.testing.assert_array_equal(host(got[1]), counts)
        np.testing.assert_array_equal(host(got[2]), np.concatenate([[0], np.cumsum(counts)]))
        np.testing.assert_allclose(host(got[3]).astype(np.float64), v, rtol=2.0 ** -22, atol=0)
        tol = float(p_tol(x).max()) + U * (t / 256 + 64)
        assert abs(float(got[0]) - loss) <= tol * loss, (float(got[0]), loss)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("t,e,k", SIZES)
def test_backward(t, e, k, masked, bf16):
    m = need_gpu()
    rng = np.random.default_rng(t * e)
    x, idx, mask = inputs(rng, t, e, k, bf16, masked)
    _, _, v, p = R.balance(x.double().numpy(), idx, 1.0, mask)
    v = v.astype(np.float32).astype(np.float64)
    add = torch.from_numpy((1e-4 * rng.standard_normal((t, e))).astype(np.float32)).to(x.dtype)
    dl = np.float32(0.37)
    keep = np.ones(t) if mask is None else mask.astype(np.float64)
    dot = (p * v).sum(-1, keepdims=True)
    ref = dl * p * (v - dot) * keep[:, None]
    tol = p_tol(x).max(-1, keepdims=True) + U * 16
    tol = 4 * tol * dl * p * (v + dot) + 1e-38
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    dev = dict(prob_grad=torch.from_numpy(v.astype(np.float32)).cuda(), dloss=torch.tensor([dl], device="cuda"), mask=dev_mask(mask))
    out = Guarded(t * e * x.element_size())
    o = out.view(x.dtype, (t, e))
    m.router_balance_backward(x.cuda(), add=add.cuda(), dlogits=o, **dev)
    torch.cuda.synchronize()
    out.check()
    want = ref + add.double().numpy()
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= tol + half * np.abs(want) * 1.01 + U * np.abs(ref)).all(), float((err / (tol + half * np.abs(want) + 1e-30)).max())
    alone = m.router_balance_backward(x.cuda(), **dev)
    err = np.abs(alone.double().cpu().numpy() - ref)
    assert (err <= tol + half * np.abs(ref) * 1.01).all()
    if mask is not None:
        assert (host(alone.float())[~mask] == 0).all()
    y = add.cuda()                                                 # in place
    assert torch.equal(m.router_balance_backward(x.cuda(), add=y, dlogits=y, **dev), o)
    z = x.cuda()
    assert torch.equal(m.router_balance_backward(z, dlogits=z, **dev), alone)


def test_gradient_against_autograd_and_differences():
    m = need_gpu()
    rng = np.random.default_rng(2)
    x, idx, mask = inputs(rng, 64, 12, 3, False, True, wild=False)
    loss, counts, _, v = m.router_balance(x.cuda(), torch.from_numpy(idx).cuda(), 0.5, dev_mask(mask))
    got = m.router_balance_backward(x.cuda(), v, mask=dev_mask(mask)).double().cpu().numpy()
    z = x.double().requires_grad_()
    n = int(mask.sum())
    p = torch.softmax(z, -1)[torch.from_numpy(mask)]
    c = counts.double().cpu()
    ref = 0.5 * 12 / (3 * n * n) * (c * p.sum(0)).sum()
    ref.backward()
    assert abs(float(loss) - float(ref.detach())) < 2e-6 * float(loss)
    np.testing.assert_allclose(got, z.grad.numpy(), rtol=0, atol=64 * U * float(v.max()))
    h = 1e-4
    for t, e in ((0, 0), (5, 11), (63, 4)):
        d = np.zeros((64, 12))
        d[t, e] = h
        x0 = x.double().numpy()
        slope = (R.balance(x0 + d, idx, 0.5, mask)[0] - R.balance(x0 - d, idx, 0.5, mask)[0]) / (2 * h)
        assert abs(got[t, e] - slope) <= 64 * U * float(v.max()) + 1e-10


def test_even_routing_costs_coef():
    m = need_gpu()
    loss, counts, off, v = m.router_balance(torch.zeros((64, 8), device="cuda"), torch.arange(128, device="cuda").view(64, 2) % 8, 0.25)
    assert float(loss) == 0.25 and host(counts).tolist() == [16] * 8 and host(off).tolist() == list(range(0, 129, 16))


def test_nobody_counts():
    m = need_gpu()
    x = torch.full((10, 5), float("nan"), device="cuda")
    idx = torch.zeros((10, 2), dtype=torch.int64, device="cuda")
    mask = torch.zeros(10, dtype=torch.bool, device="cuda")
    loss, counts, off, v = m.router_balance(x, idx, 1.0, mask)
    assert float(loss) == 0 and not counts.any() and not off.any() and not v.any()
    assert not m.router_balance_backward(x, v, mask=mask).any()
    loss, counts, off, v = m.router_balance(x[:0], idx[:0], 1.0)
    assert float(loss) == 0 and not counts.any() and not off.any() and not v.any()
    assert m.router_balance_backward(x[:0], v).shape == (0, 5)


def test_nan_and_infinity_in_counted_rows():
    m = need_gpu()
    for bad in (float("nan"), float("inf")):
        x = torch.randn((6, 10), device="cuda")
        idx = torch.topk(x, 2).indices
        x[4, 3] = bad
        loss, counts, _, v = m.router_balance(x, idx)
        assert torch.isnan(loss).item() and int(counts.sum()) == 12
        d = m.router_balance_backward(x, v)
        assert torch.isnan(d[4]).all() and torch.isfinite(d[[0, 1, 2, 3, 5]]).all()
        mask = torch.ones(6, dtype=torch.bool, device="cuda")
        mask[4] = False
        loss, _, _, v = m.router_balance(x, idx, mask=mask)
        assert torch.isfinite(loss).item() and torch.isfinite(m.router_balance_backward(x, v, mask=mask)).all()


def huge_rows(dt, e):
    """Rows of masks and values far past any exponent, with p known exactly: even over
    the places of the largest value."""
    low, rows, top = torch.finfo(dt).min, [], []

    def add(base, places, value):
        r = torch.full((e,), base, dtype=dt)
        r[places] = value
        rows.append(r)
        top.append(r == r.max())

    for base in (low, -1e30, -3e9, 3e9, 1e30, torch.finfo(dt).max):   # one value throughout
        add(base, [], 0.0)
    for base in (low, -1e30, -3e9):                                   # a few places left
        add(base, [0, e - 1], 2.5)
        add(base, [1], 0.0)
    add(-float("inf"), [0, 2], low)
    add(-float("inf"), [2], 3e9)
    add(low, [1, 2], torch.finfo(dt).max)
    return torch.stack(rows), torch.stack(top).double() / torch.stack(top).sum(-1, keepdim=True)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [3, 8, 61, 100, 256, 400, 1000, 1500])
def test_masks_of_the_lowest_value_and_huge_logits(e, dt):
    """A place of p is 1 / n, off by the exponential, the sum and the division, as p_tol
    with x = max; every other place lies
    10^9 or more below the largest, and its p is 0."""
    m = need_gpu()
    x, p = huge_rows(dt, e)
    t = x.shape[0]
    idx = np.random.default_rng(e).integers(0, e, (t, 2))
    c = np.bincount(idx.reshape(-1), minlength=e)
    v = 0.5 * e * c / (2.0 * t * t)
    loss, counts, _, grad = m.router_balance(x.cuda(), torch.from_numpy(idx).cuda(), 0.5)
    np.testing.assert_array_equal(host(counts), c)
    want = float((v * p.numpy().sum(0)).sum())
    assert abs(float(loss) - want) <= U * (16 + 64) * want, (float(loss), want)
    got = m.router_balance_backward(x.cuda(), grad).double().cpu().numpy()
    v = host(grad).astype(np.float64)
    p = p.numpy()
    dot = (p * v).sum(-1, keepdims=True)
    ref = p * (v - dot)
    half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    tol = 4 * U * 32 * p * (v + dot) + 1e-38 + half * np.abs(ref) * 1.01
    assert (np.abs(got - ref) <= tol).all(), np.argwhere(~(np.abs(got - ref) <= tol))[:4].tolist()


def test_unaligned_rows_and_repeatability():
    """Rows that begin at any element, and the same bits from call to call."""
    m = need_gpu()
    for dt in (torch.float32, torch.bfloat16):
        base = torch.randn(501 * 37 + 1, device="cuda").to(dt)
        x = base[1:].view(501, 37)
        idx = torch.topk(x.float(), 4).indices
        a, b = m.router_balance(x, idx), m.router_balance(x.clone(), idx)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert torch.equal(m.router_balance_backward(x, a[3]), m.router_balance_backward(x.clone(), a[3]))

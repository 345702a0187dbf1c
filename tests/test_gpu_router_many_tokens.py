"""The balance loss of so many tokens that a fp32 sum of their probabilities, one after
another, would be off by far more than fp32's last places."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
def test_rows_alike(masked):
    """Logits of zero: p = 1 / 160 everywhere, so the loss is coef, and every addition of p to
    a sum of its own size errs the same way.  p is off by 2^-24 of itself, each of 128
    additions at most and of those of 16 waves by 2^-24 of the sum, and the loss' rounding by
    2^-24: 146 of these, 8.7e-6.  A sum of 4000 of them is off by 4e-5."""
    m = need_gpu()
    t, e = 16_400_001, 160
    x = torch.zeros((t, e), dtype=torch.bfloat16, device="cuda")
    idx = torch.randint(0, e, (t, 1), dtype=torch.int32, device="cuda")
    mask = torch.ones(t, dtype=torch.bool, device="cuda") if masked else None
    if masked:
        mask[::1000] = False
        x[::1000] = float("nan")
    loss, counts, off, v = m.router_balance(x, idx, 1.0, mask)
    n = t if mask is None else int(mask.sum())
    want = torch.bincount(idx.reshape(-1) if mask is None else idx.reshape(-1)[mask], minlength=e)
    assert torch.equal(counts.long(), want) and int(off[-1]) == n
    assert abs(float(loss) - 1) <= 146 * 2.0 ** -24, float(loss)
    assert bool(((v.double() - e * want.double() / float(n) ** 2).abs() <= 2.0 ** -22 * v).all())
    again = m.router_balance(x, idx, 1.0, mask)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, off, v)))


def test_workspace_follows_the_tokens():
    m = need_gpu()
    for e in (1, 8, 64, 160, 500, 1000, 2000, 4096):
        sizes = [m.router_balance_workspace(t, e) for t in (0, 1, 1000, 65536, 1 << 20, 1 << 24, (1 << 31) - 1)]
        assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
        assert sizes[-1] <= 1 << 20 or sizes[-1] <= ((1 << 31) - 1) * e * 2 / 100      # under a hundredth of bf16 logits

"""The norm and its gradient at widths around each change of a workgroup's shape
(4096 and 16384 columns, octets that leave a part of the last wave idle), in
both types and row formats.  Bounds as in test_gpu_rmsnorm."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_rmsnorm import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols,fmt", [(4064, "mxfp4"), (4096, "fp8"), (4128, "mxfp4"), (4224, "fp8"), (7168, "mxfp4"),
                                      (8192, "fp8"), (16352, "mxfp4"), (16384, "fp8"), (16416, "mxfp4")])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 2051])
def test_forward(rows, cols, fmt, dt):
    m = need_gpu()
    if rows > 1000 and cols > 5000:
        rows = 70
    rng = np.random.default_rng(rows + cols)
    x, w = inputs(rng, rows, cols, dt, "f32")
    check_forward(m, x, w, x[::-1].copy(), dt, "f32", fmt)


@pytest.mark.parametrize("cols", [4064, 4096, 4128, 7168, 16352, 16384, 16416])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows", [1, 2, 70])
def test_backward(rows, cols, dt, wdt):
    m = need_gpu()
    check_backward(m, np.random.default_rng(rows + cols), rows, cols, dt, wdt, True)

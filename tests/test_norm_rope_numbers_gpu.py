"""The gradient of norms with rotation for numbers near the ends of fp32's range, against float64.
Tolerances as in test_norm_rope_gpu."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_norm_rope_gpu import handle, near, status  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def compare(handle, x, d, eps, aligned=True):
    from bit_weight_quantized_int4_gb300 import q4lin
    tokens, heads, dim = x.shape
    wide = ops.to_device(np.zeros((tokens, heads * dim + 1), np.float32))
    q = wide[:, 0 if aligned else 1:][:, :heads * dim].unflatten(1, (heads, dim))
    q.copy_(ops.to_device(x.astype(np.float32)))
    dq = ops.to_device(d.astype(np.float32))
    weight = np.ones(dim, np.float32)
    got = q4lin.norm_rope_backward(handle, q, q[:, :0], ops.to_device(weight), None, None, None, dq, dq[:, :0], eps=eps)
    want, want_w, size, size_w = kv4.norm_rope_backward(ops.to_host(q), weight.astype(np.float64), None, None,
                                                        float(np.float32(eps)), False, ops.to_host(dq))
    near(got.d_q, want, 2.0**-19 * size + ops.ROUND["f32"] * np.abs(want) + ops.TINY["f32"])
    near(got.d_q_weight, want_w, 400 * 2.0**-24 * size_w + 1e-37)
    assert status(handle) == 0
    return got.d_q


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_products_that_leave_the_range(handle, dim, aligned):
    """Rows and gradients whose products pass fp32's range, or are lost below it, where their gradient is an
    ordinary number; beside them ordinary rows and a row of zeros."""
    rng = np.random.default_rng(91)
    x, d = rng.standard_normal((6, 3, dim)), rng.uniform(1, 3, (6, 3, dim))
    for i, (a, b) in enumerate(((1e18 * (64 / dim)**0.5, 1e20), (3e-15, 1e-31), (1, 1), (1e-14, 1e-28), (1e17, 1e21))):
        x[i] *= a
        d[i] *= b
    x[5], d[5, 1] = 1e-3, 0
    d[:, 2, 5:] = 0  # one lane's channels alone
    compare(handle, x, d, 1e-31, aligned)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_of_the_smallest_numbers(handle, dim, aligned):
    """Rows below 2^-126, without eps: zeros where the gradient that comes in is, ordinary numbers where it
    is small."""
    rng = np.random.default_rng(92)
    x, d = rng.standard_normal((4, 2, dim)) * 1e-42, rng.standard_normal((4, 2, dim)) * 1e-25
    x[x == 0] = 1e-42
    d[1] = 0
    x[2] *= 1e-2
    x[2, :, 0] = 1.5e-45
    d[3] = 0
    x[3] *= 1e60
    got = compare(handle, x, d, 0.0, aligned)
    assert bool((got[[1, 3]] == 0).all())

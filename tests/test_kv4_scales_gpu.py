"""Attention over the 4-bit cache where neighbouring tokens' scales are far apart, against float64.

Tolerances as in test_kv4_attention_gpu: relative to the largest value that a row sees, whatever the
scales of the tokens that it does not see."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_attention_gpu import check, status
from tests.test_kv4_attention_gpu import BOTH, attend, handle, split  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,dim", [(1, 64), (2, 128), (5, 256), (100, 64), (130, 128), (70, 256)])
def test_scales_of_minus_zero(handle, split, tokens, dim, dtype):
    """A scale of -0 is a zero: the same bits as with +0, and right beside the other tokens' scales."""
    import torch
    rng = np.random.default_rng(71)
    host = kv4.Cache(rng, [230], 2, 16, dim)
    zero = np.zeros(host.vs.shape, bool)
    zero[host.table[0, 0], :, 4:8] = zero[host.table[0, 3], :, 8:12] = zero[host.table[0, 7]] = True
    zero |= rng.random(zero.shape) < 0.1
    q = ops.to_device(rng.standard_normal((tokens, 4, dim)).astype(np.float32), dtype)
    results = []
    for sign in (1.0, -1.0):
        host.vs[zero], host.ks[zero] = sign * np.float32(0), sign * np.float32(0)
        want = ops.attention(host, ops.to_host(q), [0, tokens], [230], 0.125)
        for rows in BOTH:
            split(rows)
            results.append(attend(handle, host, q, [tokens], [230], 0.125))
            check(*results[-1], want, dtype)
    for plus, minus in zip(results[:2], results[2:]):
        assert all(torch.equal(a, b) for a, b in zip(plus, minus))
    assert status(handle) == 0

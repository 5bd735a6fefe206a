"""Attention over the 4-bit cache with numbers near the ends of fp32's range, against float64.
Tolerances as in test_kv4_attention_gpu."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_attention_gpu import check, status
from tests.test_kv4_attention_gpu import BOTH, attend, check_rows, handle, some, split  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_keys_under_a_small_scale(handle, split, dim, rotated, dtype):
    """Keys of 2^110 and a scale of 2^-113: ordinary scores."""
    rng = np.random.default_rng(81)
    host = kv4.Cache(rng, [300], 2, 32, dim)
    host.ks *= np.float32(2.0**110)
    q = ops.to_device(rng.standard_normal((70, 4, dim)).astype(np.float32), dtype)
    rope = ops.rope_tables(rng, 300, dim) if rotated else None
    want = ops.attention(host, ops.to_host(q), [0, 70], [300], 2.0**-113, rope)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [70], [300], 2.0**-113, rope=rope and tuple(map(ops.to_device, rope))), want, dtype)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_keys_that_are_not_seen(handle, split, dim, dtype):
    """A prompt whose last key is of 2^120: the rows before it are as without it."""
    rng = np.random.default_rng(83)
    host = kv4.Cache(rng, [130], 1, 16, dim)
    q = ops.to_device((rng.standard_normal((130, 2, dim)) * 30).astype(np.float32), dtype)
    results = []
    for power in (0, 120):
        host.ks[host.table[0, 8], :, 1] = 2.0**power
        for rows in BOTH:
            split(rows)
            results.append([t[:129] for t in attend(handle, host, q, [130], [130], 0.125)])
    want = [w[:129] for w in ops.attention(host, ops.to_host(q), [0, 130], [130], 0.125)]
    for plain, large in zip(results[:2], results[2:]):
        check(*plain, want, dtype)
        check(*large, want, dtype)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,tokens", [(300, 70), (5000, 3), (5000, 40)])
@pytest.mark.parametrize("power", [-100, 100, 126])
def test_values_near_the_ends_of_the_range(handle, split, power, n, tokens, dim, dtype):
    """Values up to 2^127, and of 2^-100: whole walks and cut ones."""
    rng = np.random.default_rng(82)
    host = kv4.Cache(rng, [n], 2, 32, dim)
    host.vs *= np.float32(2.0**power)
    q = ops.to_device(rng.standard_normal((tokens, 4, dim)).astype(np.float32), dtype)
    for rows in BOTH:
        split(rows)
        out, lse = attend(handle, host, q, [tokens], [n], 0.125)
        check_rows(out, lse, host, q, n, 0.125, some(rng, tokens, 4, 40), dtype)
    assert status(handle) == 0

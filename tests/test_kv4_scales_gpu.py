"""Attention over the 4-bit cache where neighbouring tokens' scales are far apart, against float64.

Tolerances as in test_kv4_attention_gpu: relative to the largest value that a row sees, whatever the
scales of the tokens that it does not see."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_attention_gpu import check, status
from tests.test_kv4_attention_gpu import BOTH, attend, check_rows, handle, some, split  # noqa: F401 (fixtures)

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


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("apart", [12, 20, 30, 60])
@pytest.mark.parametrize("tokens,n,window", [(300, 300, 1), (40, 300, 2), (300, 300, 8), (3, 200, 2), (9, 130, 3)])
def test_rows_that_see_small_values_only(handle, split, tokens, n, window, apart, dim, dtype):
    """Every other four tokens' values are 2^apart smaller, so that some rows' windows see those only."""
    rng = np.random.default_rng(72)
    host = kv4.Cache(rng, [n], 1, 32, dim)
    small = np.arange(host.vs.shape[2]) // 4 % 2 == 0
    host.vs[..., small] *= np.float32(2.0**-apart)
    q = ops.to_device(rng.standard_normal((tokens, 2, dim)).astype(np.float32), dtype)
    want = ops.attention(host, ops.to_host(q), [0, tokens], [n], 0.125, window=window)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [tokens], [n], 0.125, window=window), want, dtype)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("apart", [9, 20, 30, 60])
@pytest.mark.parametrize("tokens", [7, 300])
def test_small_values_before_large_ones(handle, split, tokens, apart, dim, dtype):
    """A prompt whose first half has small values: its rows must not depend on the ones behind them."""
    rng = np.random.default_rng(73)
    host = kv4.Cache(rng, [tokens], 2, 16, dim)
    slots = host.table[0, :-(-tokens // 16)]
    at = np.arange(len(slots) * 16).reshape(len(slots), 1, 16)
    host.vs[slots] *= np.where(at < tokens // 2, 2.0**-apart, 1.0).astype(np.float32)
    host.vs[slots] *= np.where(at % 11 == 5, 0.0, 1.0).astype(np.float32)
    q = ops.to_device(rng.standard_normal((tokens, 6, dim)).astype(np.float32), dtype)
    want = ops.attention(host, ops.to_host(q), [0, tokens], [tokens], 0.125)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [tokens], [tokens], 0.125), want, dtype)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype,dim,tokens,n,heads", [
    ("f32", 64, 3000, 3000, 16), ("bf16", 64, 3000, 3000, 16), ("f16", 128, 300, 3000, 4),  # whole walks, cut ones
    ("bf16", 128, 300, 3000, 4), ("f32", 256, 40, 5000, 2), ("bf16", 256, 40, 5000, 2)])
def test_values_that_grow(handle, split, dtype, dim, tokens, n, heads):
    """Values that grow by 2^50 along the sequence, so that every row's largest one is among its last; and
    shrink, so that the last rows' windows see small ones."""
    rng = np.random.default_rng(74)
    host = kv4.Cache(rng, [n], heads, 64, dim)
    slots = host.table[0, :-(-n // 64)]
    at = np.arange(len(slots) * 64).reshape(len(slots), 1, 64)
    base = host.vs.copy()
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    pairs = some(rng, tokens, heads, 40)
    for grows, window in ((True, 0), (False, 60), (True, 60)):
        power = at / n * 50 - 50 if grows else -at / n * 50
        host.vs[slots] = base[slots] * (2.0**power).astype(np.float32)
        for rows in BOTH:
            split(rows)
            out, lse = attend(handle, host, q, [tokens], [n], 0.125, window=window)
            check_rows(out, lse, host, q, n, 0.125, pairs, dtype, window=window)
    assert status(handle) == 0


def test_small_values_and_outputs_taken_out(handle, split):
    """fp16 rows over a table so long that their outputs are taken out on the way, in whole walks."""
    split(1)
    rng = np.random.default_rng(75)
    n, tokens, heads = 33000, 2600, 16
    host = kv4.Cache(rng, [n], heads, 64, 64)
    slots = host.table[0, :-(-n // 64)]
    at = np.arange(len(slots) * 64).reshape(len(slots), 1, 64)
    host.vs[slots] *= np.where(at // 1000 % 2 == 0, 2.0**-30, 1.0).astype(np.float32)
    host.vs[slots] *= np.where(at < 31500, 2.0**-12, 1.0).astype(np.float32)
    q = ops.to_device(rng.standard_normal((tokens, heads, 64)).astype(np.float32), "f16")
    out, lse = attend(handle, host, q, [tokens], [n], 0.125)
    check_rows(out, lse, host, q, n, 0.125, some(rng, tokens, heads, 40), "f16")
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_log_sums_of_few_keys_with_values_far_apart(handle, split, seed, dim, dtype):
    """Each row sees one key, whose value is up to 2^40 smaller than the largest, in whole walks and cut ones."""
    rng = np.random.default_rng(76 + seed)
    n = (300, 77, 500, 230)[seed]
    host = kv4.Cache(rng, [n], 1, 32, dim)
    host.vs *= (2.0**rng.integers(-40, 1, host.vs.shape)).astype(np.float32)
    host.ks *= np.float32(0.3)
    q = ops.to_device((rng.standard_normal((n, 7, dim)) * (1, 0.3, 0.1, 0.05)[seed]).astype(np.float32), dtype)
    want = ops.attention(host, ops.to_host(q), [0, n], [n], dim**-0.5, window=1)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [n], [n], dim**-0.5, window=1), want, dtype)
    assert status(handle) == 0

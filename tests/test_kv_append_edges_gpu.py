"""Appending with offsets that are no offsets."""
import numpy as np
import pytest

from tests import _operators as ops
from tests.test_kv_append_gpu import same, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


@pytest.mark.parametrize("tokens", [1, 4, 9, 200])
@pytest.mark.parametrize("sequences,bad", [(1, 0), (2, 0), (2, 1), (3, 1), (40, 17), (40, 39), (2000, 1234)])
def test_offsets_that_decrease_are_reported(handle, sequences, bad, tokens):
    """Sequence `bad` ends before it begins; the others take the tokens in order, or none."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = ops.Cache(np.random.default_rng(61), [64] * sequences, 1, 64, 64, filled=False)
    cache = host.device()
    k = torch.randn(tokens, 1, 64, device="cuda")
    starts = ops.to_device(np.zeros(sequences, np.int32))
    rising = np.minimum(np.arange(sequences + 1), tokens).astype(np.int32)
    wrong = rising.copy()
    wrong[bad:] = 1
    wrong[bad + 1:] = 0
    q4lin.kv_append(handle, cache, k, k, ops.to_device(wrong), starts)
    assert status(handle) == 4
    q4lin.kv_append(handle, cache, k, k, ops.to_device(rising), starts)
    assert status(handle) == 0


@pytest.mark.parametrize("tokens", [3, 300])
@pytest.mark.parametrize("wrong", [-1, 301])
def test_offsets_outside_the_tokens_are_reported(handle, tokens, wrong):
    """Anywhere among the sequences; nothing is written for that sequence."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    for at in (0, 5, 99):
        host = ops.Cache(np.random.default_rng(62), [64] * 100, 1, 64, 64, filled=False)
        cache = host.device()
        k = torch.randn(tokens, 1, 64, device="cuda")
        offsets = np.zeros(101, np.int32)
        offsets[at + (wrong > 0):] = wrong
        q4lin.kv_append(handle, cache, k, k, ops.to_device(offsets), ops.to_device(np.zeros(100, np.int32)))
        assert status(handle) == 4
        same(cache, host)


@pytest.mark.parametrize("tokens", [1, 2, 300])
def test_a_sequence_without_new_tokens_may_start_anywhere(handle, tokens):
    """A place in the batch that nobody holds, with a start of -1 or past its pages: nothing is
    written for it, and nothing reported, whichever kernel runs."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(63)
    counts = [0, tokens, 0, 0, tokens, 0]
    host = ops.Cache(rng, [0, tokens + 5, 0, 0, tokens, 0], 2, 16, 64)
    cache = host.device()
    starts = np.array([-1, 5, -1, 1 << 30, 0, -2**31], np.int32)
    k, v = (rng.standard_normal((2 * tokens, 2, 64)).astype(np.float32) for _ in range(2))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ops.append(host, k, v, offsets, starts)
    q4lin.kv_append(handle, cache, ops.to_device(k), ops.to_device(v), ops.to_device(offsets), ops.to_device(starts))
    same(cache, host)
    assert status(handle) == 0

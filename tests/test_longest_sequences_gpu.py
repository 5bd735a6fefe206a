"""Attention over the longest sequence that positions of 32 bits allow, whose page table names a few pages over
and over: every key counts as often as its page is named, so the sums over the pages, weighted, are the answer.

Tolerance: a part of the 64 has 2^18 steps of 128 keys, whose products add 16 keys at a time to a sum that
grows evenly, 2^21 additions that each cut off up to 2^-23 of it: 2^21 / 2 x 2^-23 = 2^-3 of the largest value.  The
weights' sums add a step at a time, rounded: 2^18 / 2 x 2^-24 = 2^-7 of the sum; over the 8-bit cache 16 keys at
a time, 2^-4.  (The kernel for few rows has shorter chains.)"""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_attention_gpu import status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("few", [False, True])
def test_a_sequence_of_all_positions(few, bits, dtype):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(95)
    page, named = 16, 4
    pages = (2**31 - 1 - 64) // page
    n = pages * page
    host = (kv4 if bits == 4 else ops).Cache(rng, [named * page], 1, page, 64, spare=0)
    cache = host.device()
    own = cache.page_table[:, :named]
    cache = type(cache)(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales,
                        own.repeat(1, -(-pages // named))[:, :pages].contiguous())
    times = np.array([pages // named + (i < pages % named) for i in range(named)], float).repeat(page)
    q = ops.to_device(rng.standard_normal((3, 2, 64)).astype(np.float32), dtype)
    h = q4lin.Handle(0)
    h.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 1 << 40 if few else 1)
    out, lse = q4lin.attention(h, cache, q, ops.to_device(np.array([0, 3], np.int32)),
                               ops.to_device(np.array([n], np.int32)), 0.125, causal=False)
    torch.cuda.synchronize()
    k, v, x = host.keys(0, named * page, 0), host.values(0, named * page, 0), ops.to_host(q)
    s = 0.125 * np.einsum("thd,nd->thn", x, k)
    w = np.exp(s - s.max(-1, keepdims=True)) * times
    want, want_lse = np.einsum("thn,nd->thd", w, v) / w.sum(-1, keepdims=True), s.max(-1) + np.log(w.sum(-1))
    assert np.all(np.abs(ops.to_host(out) - want) <= 2.0**-3 * np.abs(v).max())
    assert np.all(np.abs(ops.to_host(lse) - want_lse) <= 2.0**(-7 if bits == 4 else -4))
    assert status(h) == 0
    h.close()

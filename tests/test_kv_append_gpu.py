"""Appending to the paged 8-bit cache: bytes and scales are fixed by the definition, so they
have to equal the host's, bit for bit."""
import numpy as np
import pytest

from tests import _operators as ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


def draw(rng, tokens, heads, dim, dtype):
    """Inputs as the type holds them, float32 on the host."""
    x = rng.standard_normal((tokens, heads, dim)) * np.exp(rng.standard_normal((1, heads, dim)) * 0.5)
    t = ops.to_device(x.astype(np.float32), dtype)
    return t, t.float().cpu().numpy()


def same(device_cache, host):
    for got, want, what in ((device_cache.k_scales, host.ks, "key scales"),
                            (device_cache.v_scales, host.vs, "value scales"),
                            (device_cache.k_codes, host.k, "key codes"),
                            (device_cache.v_codes, host.v, "value codes")):
        got = got.cpu().numpy()
        assert np.array_equal(got, want), f"{what}: {np.sum(got != want)} of {want.size} differ"


def status(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    return q4lin.q4lin_check_device_status(handle.ptr, torch.cuda.current_stream().cuda_stream)[1]


CASES = [
    # lengths before, new tokens, heads, page, dim, dtype, rotated, interleaved
    ([0], [1], 1, 16, 64, "f32", 64, False),
    ([15], [1], 2, 16, 64, "f16", 64, False),
    ([16], [1], 2, 16, 64, "bf16", 32, False),
    ([63, 5, 64, 0], [1, 1, 1, 1], 8, 64, 128, "bf16", 128, False),
    ([63, 5, 64, 0], [2, 0, 3, 1], 8, 64, 128, "f32", 128, True),
    ([0, 0, 0], [130, 64, 1], 3, 64, 128, "f32", 128, False),
    ([7, 100, 31], [57, 97, 33], 2, 32, 64, "f16", 16, True),
    ([40, 0], [300, 17], 5, 16, 256, "f32", 256, False),
    ([33], [129], 1, 64, 256, "bf16", 128, False),
    ([1], [62], 4, 64, 64, "f32", 0, False),
    ([0] * 40 + [70], [0] * 39 + [3, 65], 2, 32, 128, "f32", 8, False),
    ([i % 70 for i in range(150)], [i % 3 for i in range(150)], 1, 16, 64, "f32", 64, False),
]


@pytest.mark.parametrize("starts,counts,heads,page,dim,dtype,rotated,interleaved", CASES)
def test_bytes(handle, starts, counts, heads, page, dim, dtype, rotated, interleaved):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(len(starts) * 1000 + dim + page)
    host = ops.Cache(rng, [s + n for s, n in zip(starts, counts)], heads, page, dim)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k, k_host = draw(rng, offsets[-1], heads, dim, dtype)
    v, v_host = draw(rng, offsets[-1], heads, dim, dtype)
    rope = ops.rope_tables(rng, max(s + n for s, n in zip(starts, counts)), rotated) if rotated else None
    cache = host.device()
    ops.append(host, k_host, v_host, offsets, np.array(starts), rope, interleaved)
    q4lin.kv_append(handle, cache, k, v, ops.to_device(offsets),
                    ops.to_device(np.array(starts, np.int32)),
                    rope=None if rope is None else tuple(map(ops.to_device, rope)),
                    interleaved=interleaved)
    same(cache, host)
    assert status(handle) == 0


@pytest.mark.parametrize("page", [16, 64])
def test_token_by_token_rounds_the_open_page_again(handle, page):
    """Growing tokens: the page's scale grows with nearly every one of them."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(3)
    host = ops.Cache(rng, [70], 2, page, 64, filled=False)
    cache = host.device()
    offsets = np.array([0, 1], np.int32)
    for i in range(70):
        k, v = (rng.standard_normal((1, 2, 64)).astype(np.float32) * (1 + 0.1 * i) for _ in range(2))
        ops.append(host, k, v, offsets, np.array([i]))
        q4lin.kv_append(handle, cache, ops.to_device(k), ops.to_device(v), ops.to_device(offsets),
                        ops.to_device(np.array([i], np.int32)))
    same(cache, host)
    # What the cache stands for is near what went in: half a step of each rounding.
    assert np.all(np.abs(host.keys(0, 70, 0)) < 127.5 * host.ks.max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_slices_of_one_projection(handle, dtype, shift):
    """k and v as slices of a wider array, at any alignment of its elements."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(5)
    heads, dim, tokens = 2, 64, 37
    host = ops.Cache(rng, [50], heads, 32, dim)
    wide = rng.standard_normal((tokens, 3 * heads * dim + 5)).astype(np.float32)
    t = ops.to_device(wide, dtype)
    k = t[:, shift:shift + heads * dim].unflatten(1, (heads, dim))
    v = t[:, shift + heads * dim + 1:shift + 2 * heads * dim + 1].unflatten(1, (heads, dim))
    cache = host.device()
    offsets, starts = np.array([0, tokens], np.int32), np.array([13], np.int32)
    ops.append(host, k.float().cpu().numpy(), v.float().cpu().numpy(), offsets, starts)
    q4lin.kv_append(handle, cache, k, v, ops.to_device(offsets), ops.to_device(starts))
    same(cache, host)


def test_zeros_infinities_and_nan(handle):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(6)
    host = ops.Cache(rng, [20], 2, 16, 64, filled=False)
    k = rng.standard_normal((20, 2, 64)).astype(np.float32)
    k[:, 1] = 0
    k[3, 0, :4] = np.inf, -np.inf, np.nan, 1e-45
    v = np.zeros_like(k)
    v[18] = 1e-40  # below what a scale can hold
    cache = host.device()
    offsets, starts = np.array([0, 20], np.int32), np.array([0], np.int32)
    ops.append(host, k, v, offsets, starts)
    q4lin.kv_append(handle, cache, ops.to_device(k), ops.to_device(v), ops.to_device(offsets),
                    ops.to_device(starts))
    same(cache, host)
    assert status(handle) == 3
    assert status(handle) == 0


def test_indices_out_of_range_touch_nothing(handle):
    """A page outside the cache, positions past the page table and the rotation table."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(7)
    k = torch.randn(4, 2, 64, device="cuda")
    for table, starts, offsets, rope_rows in (([[7, -1]], [0], [0, 4], 100), ([[-1, 1]], [0], [0, 4], 100),
                                              ([[0, 1]], [30], [0, 4], 100), ([[0, 1]], [2], [0, 4], 5),
                                              ([[0, 1]], [-3], [0, 4], 100), ([[0, 1]], [0], [0, 9], 100)):
        host = ops.Cache(rng, [32], 2, 16, 64, spare=0)
        host.table = np.array(table, np.int32)
        cache = host.device()
        rope = tuple(map(ops.to_device, ops.rope_tables(rng, rope_rows, 64)))
        before = {n: getattr(cache, n).clone() for n in ("k_codes", "k_scales")}
        q4lin.kv_append(handle, cache, k, k.clone(), ops.to_device(np.array(offsets, np.int32)),
                        ops.to_device(np.array(starts, np.int32)), rope=rope)
        assert status(handle) == 4
        if starts != [30]:  # (there the two tokens that fit are appended)
            assert all(torch.equal(getattr(cache, n), t) for n, t in before.items())


def test_other_stream_and_nothing_to_do(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(8)
    host = ops.Cache(rng, [40], 2, 32, 128)
    cache = host.device()
    k, k_host = draw(rng, 40, 2, 128, "f32")
    offsets, starts = np.array([0, 40], np.int32), np.array([0], np.int32)
    ops.append(host, k_host, k_host, offsets, starts)
    o, s = ops.to_device(offsets), ops.to_device(starts)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q4lin.kv_append(handle, cache, k, k, o, s, stream=stream.cuda_stream)
    stream.synchronize()
    same(cache, host)
    q4lin.kv_append(handle, cache, k[:0], k[:0], o, s)
    torch.cuda.synchronize()
    same(cache, host)


def test_refusals(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = ops.Cache(np.random.default_rng(9), [40], 2, 32, 64)
    cache = host.device()
    o, s = (ops.to_device(np.array(a, np.int32)) for a in ([0, 4], [0]))
    k = torch.randn(4, 2, 64, device="cuda")
    bad = [dict(k=k[:, :1]), dict(v=k[:3]), dict(k=k.double(), v=k.double()), dict(v=k.half()),
           dict(k=k.transpose(1, 2)), dict(offsets=s), dict(starts=o), dict(starts=s.long()),
           dict(k=k.cpu()), dict(rope=(k[0], k[0, :1])), dict(rope=(k[0].half(), k[0].half()))]
    for change in bad:
        args = dict(dict(k=k, v=k, offsets=o, starts=s), **change)
        with pytest.raises(ValueError):
            q4lin.kv_append(handle, cache, **args)
    # The C entry's own checks: sizes and types it does not take, overlaps, null pointers.
    fields = lambda: q4lin.q4lin_kv_append_t(k.data_ptr(), k.data_ptr(), 128, 64, 128, 64, 0, 4,
                                             o.data_ptr(), s.data_ptr(), q4lin.q4lin_rope_t())
    def call(change_args=(), change_cache=()):
        a, c = fields(), q4lin.q4lin_kv_cache_t.from_buffer_copy(cache.args)
        for n, x in change_args:
            setattr(a, n, x)
        for n, x in change_cache:
            setattr(c, n, x)
        return q4lin.q4lin_run_kv_append(handle.ptr, c, a, 0)
    assert call() == q4lin.Q4LIN_OK
    inv, uns = q4lin.Q4LIN_ERR_INVALID_ARG, q4lin.Q4LIN_ERR_UNSUPPORTED
    rope = q4lin.q4lin_rope_t
    for change, want in (([("k", None)], inv), ([("dtype", 3)], inv), ([("tokens", -1)], inv),
                         ([("offsets", None)], inv), ([("k_token_stride", -128)], inv),
                         ([("v_head_stride", 1 << 62)], inv), ([("k", k.data_ptr() + 2)], inv),
                         ([("v", cache.args.k_codes)], inv),
                         ([("rope", rope(k.data_ptr(), None, 4, 64, 0))], inv),
                         ([("rope", rope(k.data_ptr(), k.data_ptr(), 4, 12, 0))], inv),
                         ([("rope", rope(k.data_ptr(), k.data_ptr(), 4, 72, 0))], inv),
                         ([("rope", rope(k.data_ptr(), k.data_ptr(), 0, 64, 0))], inv)):
        assert call(change_args=change) == want, change
    for change, want in (([("page_size", 48)], uns), ([("page_size", 128)], uns), ([("head_dim", 96)], uns),
                         ([("num_pages", 0)], inv), ([("page_table", None)], inv),
                         ([("k_codes", cache.args.k_codes + 8)], inv),
                         ([("v_codes", cache.args.k_codes)], inv), ([("table_stride", 1)], inv),
                         ([("num_pages", 1 << 60)], inv)):
        assert call(change_cache=change) == want, change
    assert q4lin.q4lin_run_kv_append(None, cache.args, fields(), 0) == inv
    torch.cuda.synchronize()

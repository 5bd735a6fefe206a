"""Refusals of the norms with rotation and of the 4-bit cache's entry points: the host checks its
arguments before any device work, so they need no GPU.  The pointers are never followed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def q():
    from bit_weight_quantized_int4_gb300 import build
    build.build()
    from bit_weight_quantized_int4_gb300 import q4lin
    return q4lin


@pytest.fixture(scope="module")
def handle():
    """Something that is not NULL; a call that is refused reads nothing of it."""
    memory = ctypes.create_string_buffer(4096)
    yield ctypes.addressof(memory)


MB = 1 << 20


def norm(lib, **change):
    """64 tokens of 8 + 2 heads of 128 in fp32, everything in megabytes of its own."""
    a = lib.q4lin_norm_rope_t(16 * MB, 32 * MB, 1024, 128, 256, 128, 1 * MB, 2 * MB, 48 * MB, 64 * MB, 1024, 128,
                            256, 128, lib.Q4LIN_DTYPE_F32, 64, 8, 2, 128, 3 * MB,
                            lib.q4lin_rope_t(4 * MB, 5 * MB, 100, 128, 0), 1e-6)
    return changed(a, change)


def changed(a, change):
    for name, value in change.items():
        at = a
        *path, last = name.split("__")
        for p in path:
            at = getattr(at, p)
        setattr(at, last, value)
    return a


NORM = [
    dict(dtype=3), dict(dtype=-1), dict(tokens=-1), dict(heads=-1), dict(heads=0, kv_heads=0), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None), dict(k=None), dict(q_out=None), dict(q=16 * MB + 2),
    dict(q_out=48 * MB + 1), dict(positions=None), dict(positions=3 * MB + 2), dict(q_weight=MB + 1),
    dict(rope__sin=None), dict(rope__positions=0), dict(rope__rotated=12), dict(rope__rotated=136),
    dict(rope__interleaved=2), dict(q_token_stride=-1), dict(k_head_stride=-128), dict(q_token_stride=1 << 62),
    dict(q_out_token_stride=0), dict(q_out_head_stride=64), dict(q_out_token_stride=1000), dict(k_out_head_stride=0),
    dict(q_out=16 * MB + 512), dict(q_out=32 * MB), dict(k_out=48 * MB + 4096), dict(q_out=16 * MB, q_token_stride=2048),
    dict(q_out=MB), dict(k_out=2 * MB), dict(q_out=3 * MB), dict(k_out=4 * MB), dict(k_out=5 * MB),
]


@pytest.mark.parametrize("change", NORM)
def test_norm_rope(q, handle, change):
    assert q.q4lin_run_norm_rope(handle, norm(q, **change), None) == q.Q4LIN_ERR_INVALID_ARG
    # The gradient checks the same, and its own.
    b = q.q4lin_norm_rope_backward_t(norm(q, **change), 80 * MB, 96 * MB, 1024, 128, 256, 128, 6 * MB, 7 * MB)
    assert q.q4lin_run_norm_rope_backward(handle, b, None) == q.Q4LIN_ERR_INVALID_ARG


BACKWARD = [
    dict(d_q_out=None), dict(d_k_out=None), dict(d_q_out=80 * MB + 2), dict(d_q_out_token_stride=-1),
    dict(d_q_weight=6 * MB + 2), dict(d_k_weight=6 * MB), dict(d_k_weight=6 * MB + 256), dict(d_q_weight=16 * MB),
    dict(d_q_weight=48 * MB), dict(d_q_weight=80 * MB), dict(d_k_weight=MB), dict(d_k_weight=3 * MB),
    dict(d_k_weight=4 * MB), dict(d_q_out=48 * MB + 512), dict(d_q_out=64 * MB), dict(d_k_out=48 * MB),
    dict(d_q_out=48 * MB, d_q_out_token_stride=0),
]


@pytest.mark.parametrize("change", BACKWARD)
def test_norm_rope_backward(q, handle, change):
    b = q.q4lin_norm_rope_backward_t(norm(q), 80 * MB, 96 * MB, 1024, 128, 256, 128, 6 * MB, 7 * MB)
    assert q.q4lin_run_norm_rope_backward(handle, changed(b, change), None) == q.Q4LIN_ERR_INVALID_ARG


def test_norm_rope_sizes(q, handle):
    for dim in (0, 32, 96, 512):
        assert q.q4lin_run_norm_rope(handle, norm(q, head_dim=dim), None) == q.Q4LIN_ERR_UNSUPPORTED
    assert q.q4lin_run_norm_rope(None, norm(q), None) == q.Q4LIN_ERR_INVALID_ARG
    assert q.q4lin_run_norm_rope(handle, None, None) == q.Q4LIN_ERR_INVALID_ARG
    assert q.q4lin_run_norm_rope_backward(handle, None, None) == q.Q4LIN_ERR_INVALID_ARG
    assert q.q4lin_run_norm_rope(handle, norm(q, tokens=0), None) == q.Q4LIN_OK


def cache(q, **change):
    """256 pages of 64 tokens, 8 heads of 128: 8 MB of codes and 512 KB of scales each."""
    c = q.q4lin_kv_cache_t(16 * MB, 1 * MB, 32 * MB, 2 * MB, 3 * MB, 256, 8, 64, 128, 4, 64, 64)
    return changed(c, change)


CACHE = [
    dict(k_codes=None), dict(v_scales=None), dict(page_table=None), dict(k_codes=16 * MB + 8), dict(k_scales=MB + 4),
    dict(v_scales=2 * MB + 8), dict(page_table=3 * MB + 2), dict(v_codes=16 * MB + 4 * MB), dict(v_scales=MB + 4096),
    dict(k_scales=16 * MB), dict(num_pages=0), dict(kv_heads=0), dict(batch=-1), dict(table_stride=63),
    dict(num_pages=1 << 60), dict(pages_per_sequence=0),
]


def calls(q):
    append = q.q4lin_kv_append_t(48 * MB, 64 * MB, 1024, 128, 1024, 128, 0, 100, 4 * MB, 5 * MB, q.q4lin_rope_t())
    read = q.q4lin_kv_read_t(48 * MB, 64 * MB, 0, 100, 4 * MB, 5 * MB)
    attend = q.q4lin_attention_t(48 * MB, 4096, 128, 64 * MB, 80 * MB, 0, 100, 32, 100, 4 * MB, 5 * MB, 0.1, 1, 0,
                                 q.q4lin_rope_t())
    return ((q.q4lin_run_kv4_append, append), (q.q4lin_run_kv4_read, read), (q.q4lin_run_kv4_attention, attend))


@pytest.mark.parametrize("change", CACHE)
def test_caches(q, handle, change):
    for run, args in calls(q):
        assert run(handle, cache(q, **change), args, None) == q.Q4LIN_ERR_INVALID_ARG


def test_cache_sizes(q, handle):
    for run, args in calls(q):
        for change in (dict(page_size=8), dict(page_size=128), dict(head_dim=32), dict(head_dim=192)):
            assert run(handle, cache(q, **change), args, None) == q.Q4LIN_ERR_UNSUPPORTED
        for change in (dict(kv_heads=65536, num_pages=1), dict(pages_per_sequence=1 << 30, table_stride=1 << 30)):
            far = dict(k_codes=1 << 44, v_codes=1 << 45, k_scales=1 << 46, v_scales=1 << 47, page_table=1 << 50)
            assert run(handle, cache(q, **change, **far), args, None) in (q.Q4LIN_ERR_TOO_LARGE, q.Q4LIN_ERR_INVALID_ARG)
        assert run(None, cache(q), args, None) == q.Q4LIN_ERR_INVALID_ARG
        assert run(handle, None, args, None) == q.Q4LIN_ERR_INVALID_ARG
        assert run(handle, cache(q), None, None) == q.Q4LIN_ERR_INVALID_ARG
        assert run(handle, cache(q), changed(args, dict(tokens=0)), None) == q.Q4LIN_OK
        assert run(handle, cache(q, batch=0), args, None) == q.Q4LIN_OK


@pytest.mark.parametrize("which,change", [
    (0, dict(dtype=3)), (0, dict(tokens=-1)), (0, dict(k=None)), (0, dict(k=48 * MB + 2)), (0, dict(k_token_stride=-1)),
    (0, dict(offsets=None)), (0, dict(k=17 * MB)), (0, dict(v=MB)), (0, dict(starts=2 * MB)),
    (0, dict(rope__cos=6 * MB)),
    (1, dict(dtype=3)), (1, dict(tokens=-1)), (1, dict(k=None, v=None)), (1, dict(k=48 * MB + 8)), (1, dict(v=None, k=17 * MB)),
    (1, dict(k=64 * MB + 64)), (1, dict(k=2 * MB)), (1, dict(k=3 * MB)), (1, dict(k=4 * MB)), (1, dict(v=5 * MB)),
    (1, dict(starts=None)), (1, dict(offsets=4 * MB + 2)), (1, dict(tokens=1 << 61)),
    (2, dict(dtype=3)), (2, dict(heads=30)), (2, dict(heads=0)), (2, dict(window=-1)), (2, dict(causal=2)),
    (2, dict(max_query=0)), (2, dict(query=None)), (2, dict(out=48 * MB)), (2, dict(out=16 * MB)), (2, dict(lse=64 * MB)),
    (2, dict(out=64 * MB + 8)), (2, dict(lse=MB)), (2, dict(lengths=None)), (2, dict(q_head_stride=-1)),
])
def test_arguments(q, handle, which, change):
    run, args = calls(q)[which]
    assert run(handle, cache(q), changed(args, change), None) == q.Q4LIN_ERR_INVALID_ARG


def test_binding(q):
    """What the convenience layer checks by itself, on tensors of the CPU."""
    import torch
    codes, scales = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    good = codes, scales, codes.clone(), scales.clone(), table
    assert q.KVCache4(*good).args.head_dim == 64
    for at, bad in ((0, codes[0]), (0, codes.int()), (1, scales.half()), (1, scales[..., :8]), (2, codes[:3]),
                    (3, scales.transpose(0, 1)), (4, table.long()), (4, table[0])):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            q.KVCache4(*args)
    empty = q.KVCache4.empty(4, 2, 16, 64, table)
    assert (empty.k_codes == 0x88).all() and empty.v_scales.shape == (4, 2, 16)
    with pytest.raises(ValueError):
        q.KVCache4.empty(4, 2, 16, 63, table)
    with pytest.raises(ValueError):
        q.KVCache4.empty(4, 2, 16, 64, table[0])

"""Attention over the paged 8-bit cache where its walks, masks and indices are at their limits:
selected rows against float64, with the tolerance of test_attention_gpu."""
import numpy as np
import pytest

from tests import _operators as ops
from tests.test_attention_gpu import check, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


def attend(handle, host, q, counts, lengths, scale, cache=None, **more):
    from bit_weight_quantized_int4_gb300 import q4lin
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return q4lin.attention(handle, host.device() if cache is None else cache, q, ops.to_device(offsets),
                           ops.to_device(np.array(lengths, np.int32)), scale, **more)


def check_rows(out, lse, host, q, n, scale, rows, dtype="f32", b=0, first=0, count=None, causal=True, window=0):
    """Pairs (token, head) of `rows`, of sequence b of n tokens, whose `count` queries begin at row
    `first`."""
    x, want = ops.to_host(q), [[], [], [], []]
    count = q.shape[0] if count is None else count
    heads, group = q.shape[1], q.shape[1] // host.heads
    kept = {}
    for i, h in rows:
        if h // group not in kept:
            kept[h // group] = host.keys(b, n, h // group), host.values(b, n, h // group)
        position = n - count + i
        seen = slice(max(0, position - window + 1) if window else 0, position + 1 if causal else n)
        k, v = (a[seen] for a in kept[h // group])
        s = scale * (k @ x[first + i, h])
        p = np.exp(s - s.max())
        for one, value in zip(want, (p @ v / p.sum(), s.max() + np.log(p.sum()), np.abs(v).max(),
                                     abs(scale) * (np.abs(k) @ np.abs(x[first + i, h])).max())):
            one.append(value)
    at = [first + i for i, _ in rows], [h for _, h in rows]
    check(out[at], lse[at], [np.array(w) for w in want], dtype)


def some(rng, count, heads, n=40):
    """Tokens at both ends and anywhere, of any head."""
    ends = [(0, 0), (0, heads - 1), (count - 1, 0), (count - 1, heads - 1)]
    return ends + [(int(rng.integers(count)), int(rng.integers(heads))) for _ in range(n)]


@pytest.mark.parametrize("dim", [64, 128])
def test_maxima_that_grow_as_outputs_are_taken_out(handle, dim):
    """Scores that rise by 14 every 1024 keys, so that a row's maximum moves by far more than 2^8
    just where fp32 outputs leave tensor memory; whole walks (168 of them)."""
    rng = np.random.default_rng(41)
    n, tokens, heads, kv_heads = 5300, 1300, 32, 8
    host = ops.Cache(rng, [n], kv_heads, 64, dim)
    way = np.sign(rng.standard_normal(dim))
    rise = np.arange(host.table.shape[1]) * 64 // 1024
    for j, page in enumerate(host.table[0, :-(-n // 64)]):
        host.k[page] = np.clip(100 * way + rng.integers(-9, 10, host.k[page].shape), -127, 127) + 128
        host.ks[page] = 0.14 * (rise[j] + 1) / dim
    q = ops.to_device(np.broadcast_to(way, (tokens, heads, dim)).astype(np.float32))
    out, lse = attend(handle, host, q, [tokens], [n], 1.0)
    # A row whose last keys are the first few of a higher block weighs both blocks.
    rows = some(rng, tokens, heads) + [(1024 * j + e - (n - tokens), h) for j in (4, 5) for e in range(-2, 4)
                                       for h in (0, 7, 31)]
    check_rows(out, lse, host, q, n, 1.0, rows)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sequences", [3, 64, 1500])
def test_offsets_that_rise_and_fall(handle, sequences, dtype):
    """0, n, 0, n, ...: every other sequence looks like all of the tokens.  More row tiles than the
    call's tokens have are not taken (of three sequences, one or two are), and nothing past the
    workspace is touched: the call after it is right."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(42)
    n = 700
    host = ops.Cache(rng, [n], 1, 64, 64)
    host.table = np.repeat(host.table, sequences, 0)
    cache = host.device()
    q = ops.to_device(rng.standard_normal((n, 8, 64)).astype(np.float32), dtype)
    offsets = ops.to_device((np.arange(sequences + 1) % 2 * n).astype(np.int32))
    lengths = ops.to_device(np.full(sequences, n, np.int32))
    out = torch.full_like(q, 7.0)
    q4lin.attention(handle, cache, q, offsets, lengths, 0.125, out=out)
    assert status(handle) == 4
    if sequences > 3:
        assert bool((out == 7.0).all())
    host.table = host.table[:1]
    got = attend(handle, host, q, [n], [n], 0.125)
    check_rows(*got, host, q, n, 0.125, some(rng, n, 8), dtype)
    assert status(handle) == 0


BEHIND_A_WINDOW = [
    # tokens, keys, heads, kv heads, dim, dtype, window
    (600, 600, 4, 1, 64, "f32", 50),
    (600, 600, 4, 1, 128, "bf16", 1),
    (600, 900, 3, 1, 128, "f32", 256),
    (1000, 1000, 1, 1, 64, "f16", 33),
    (1000, 1000, 4, 1, 64, "f32", 33),
    (2048, 2048, 1, 1, 64, "bf16", 256),
    (2048, 2048, 4, 2, 64, "f32", 50),
    (1024, 3000, 4, 1, 64, "f32", 1),
    (2048, 2100, 8, 2, 64, "f32", 256),
    (1100, 1100, 40, 10, 64, "f32", 50),    # whole walks
    (1100, 1100, 40, 10, 128, "bf16", 256),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tokens,n,heads,kv_heads,dim,dtype,window", BEHIND_A_WINDOW)
def test_a_window_without_an_end(handle, tokens, n, heads, kv_heads, dim, dtype, window, causal):
    """Not causal, a query sees its window and everything after it: walks as long as the queries'
    count and the window together.  Both kernels; and the causal form of the same sizes."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(43)
    host = ops.Cache(rng, [n], kv_heads, 32, dim)
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    rows, scale = some(rng, tokens, heads), float(np.float32(1 / np.sqrt(dim)))
    try:
        for split in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, split)
            out, lse = attend(handle, host, q, [tokens], [n], scale, causal=causal, window=window)
            check_rows(out, lse, host, q, n, scale, rows, dtype, causal=causal, window=window)
            assert status(handle) == 0
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens,n,heads,kv_heads", [(1, 3000, 4, 1), (5, 40, 4, 2), (1100, 1100, 40, 10),
                                                     (700, 1500, 4, 1)])
def test_windows_wider_than_any_sequence(handle, tokens, n, heads, kv_heads, causal):
    """As if there were none, up to the largest number that the argument holds."""
    import torch
    rng = np.random.default_rng(44)
    host = ops.Cache(rng, [n], kv_heads, 16, 64)
    q = ops.to_device(rng.standard_normal((tokens, heads, 64)).astype(np.float32))
    want = attend(handle, host, q, [tokens], [n], 0.125, causal=causal)
    check_rows(*want, host, q, n, 0.125, some(rng, tokens, heads), causal=causal)
    for window in (n, n + 1, n + 100, 2**31, 2**62, 2**63 - 300, 2**63 - 1):
        got = attend(handle, host, q, [tokens], [n], 0.125, causal=causal, window=window)
        check_rows(*got, host, q, n, 0.125, some(rng, tokens, heads), causal=causal)
        if window > n + 16:  # (no page fewer than without)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert status(handle) == 0


def wide_cache(host, width):
    """The host's cache with a page table of `width` pages a sequence, -1 past what is there."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    narrow = host.device()
    table = torch.full((host.table.shape[0], width), -1, dtype=torch.int32, device="cuda")
    table[:, :host.table.shape[1]] = narrow.page_table
    return q4lin.KVCache(narrow.k_codes, narrow.k_scales, narrow.v_codes, narrow.v_scales, table)


MANY = [
    # new tokens of each sequence (the first, the others), sequences, heads, kv heads, dim, page, pages of a table row
    (1, 1, 1024, 32, 8, 64, 64, 2048),       # single tokens, and no max_query given
    (1024, 1, 256, 32, 8, 64, 64, 2048),     # a prompt among single tokens
    (300, 1, 64, 16, 4, 128, 16, 200000),
    (2000, 1, 1, 32, 8, 64, 64, 1 << 20),    # one prompt, a table for 2^26 tokens
    (300, 1, 64, 8, 8, 256, 64, 2048),
]


@pytest.mark.parametrize("first,others,sequences,heads,kv_heads,dim,page,width", MANY)
def test_many_sequences_and_wide_tables(handle, first, others, sequences, heads, kv_heads, dim, page, width):
    """Calls whose page table is wide for more than they hold."""
    rng = np.random.default_rng(45)
    counts = [first] + [others] * (sequences - 1)
    lengths = [t + i * 37 % 400 for i, t in enumerate(counts)]
    host = ops.Cache(rng, lengths, kv_heads, page, dim)
    q = ops.to_device(rng.standard_normal((sum(counts), heads, dim)).astype(np.float32), "bf16")
    scale = float(np.float32(1 / np.sqrt(dim)))
    out, lse = attend(handle, host, q, counts, lengths, scale, cache=wide_cache(host, width))
    for b in sorted({0, 1 % sequences, 255 % sequences, sequences // 2, sequences - 1}):
        check_rows(out, lse, host, q, lengths[b], scale, some(rng, counts[b], heads, 8), "bf16", b=b,
                   first=sum(counts[:b]), count=counts[b])
    assert status(handle) == 0


def test_too_many_tiles_are_refused(handle):
    """More tiles than the list of the kernel for few rows counts, which with 256 channels takes
    prompts too; the same call by the prompts' kernel is above."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = ops.Cache(np.random.default_rng(46), [4096], 8, 64, 256)
    q = torch.randn(4096, 32, 256, device="cuda")
    out = torch.full_like(q, 7.0)
    with pytest.raises(q4lin.Q4LinError) as e:
        attend(handle, host, q, [4096], [4096], 0.1, cache=wide_cache(host, 1 << 18), out=out)
    assert e.value.status == q4lin.Q4LIN_ERR_TOO_LARGE
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and status(handle) == 0


@pytest.mark.parametrize("dim", [64, 256])
def test_overlapping_sequences_do_not_outgrow_the_list(handle, dim):
    """128 sequences that claim the same tokens, by offsets that rise and fall: with 256 channels
    2^31 tiles.  Nothing is run, and the next call is right."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(47)
    tokens, n = (2048, 131072) if dim == 256 else (10, 131072)
    host = ops.Cache(rng, [64], 8, 64, dim)
    page = int(host.table[0, 0])
    host.table = np.full((256, n // 64), page, np.int32)
    cache = host.device()
    q = torch.randn(tokens, 32, dim, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((tokens, 32), 7.0, device="cuda")
    offsets = ops.to_device((np.arange(257) % 2 * tokens).astype(np.int32))
    q4lin.attention(handle, cache, q, offsets, ops.to_device(np.full(256, n, np.int32)), 0.1, out=out, lse=lse)
    assert status(handle) == 4
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    host.table = np.full((1, 2), page, np.int32)
    got = attend(handle, host, q[:9], [9], [64], 0.125)
    check_rows(*got, host, q[:9], 64, 0.125, some(rng, 9, 32))
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_near_the_largest_number(handle, dim, dtype):
    """Finite queries of up to 2^128, whose scores are of ordinary size by the scale.  Both kernels."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(48)
    host = ops.Cache(rng, [300], 2, 32, dim)
    host.ks /= 64
    q = rng.uniform(-1, 1, (70, 4, dim)) * 2.0**rng.integers(120, 128, (70, 4, 1))
    q = ops.to_device(q.astype(np.float32), dtype)
    q[q.isinf()] = 0
    try:
        for split in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, split)
            out, lse = attend(handle, host, q, [70], [300], 2.0**-124)
            check_rows(out, lse, host, q, 300, 2.0**-124, some(rng, 70, 4, 80), dtype)
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,tokens", [(1, 1), (200, 130)])
def test_an_infinite_query_gives_nan(handle, n, tokens, dim, dtype, rotated):
    """Also where every key has the same sign in its channel, so that all scores are infinities of
    one sign.  The other rows are as they were.  Both kernels."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(49)
    host = ops.Cache(rng, [n], 1, 16, dim)
    host.k[..., 3] = 1 + host.k[..., 3] % 100    # codes below 128
    host.k[..., 5] = 255 - host.k[..., 5] % 100  # and above
    cache = host.device()
    angle = np.zeros((n, dim // 2), np.float32)
    rope = (ops.to_device(angle + 1), ops.to_device(angle)) if rotated else None
    q = ops.to_device(rng.standard_normal((tokens, 4, dim)).astype(np.float32), dtype)
    try:
        for split in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, split)
            want, want_lse = attend(handle, host, q, [tokens], [n], 0.1, cache=cache, rope=rope)
            assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
            for channel, value in ((3, float("inf")), (3, -float("inf")), (5, float("inf")), (5, -float("inf"))):
                x = q.clone()
                x[-1, 2, channel] = value
                out, lse = attend(handle, host, x, [tokens], [n], 0.1, cache=cache, rope=rope)
                assert torch.isnan(out[-1, 2]).all() and torch.isnan(lse[-1, 2])
                out[-1, 2], lse[-1, 2] = want[-1, 2], want_lse[-1, 2]
                assert torch.equal(out, want) and torch.equal(lse, want_lse)
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [5000, 3200])
def test_sums_over_many_keys_lean_to_neither_side(handle, tokens, dim, dtype):
    """131072 keys, in whole walks (5000 tokens) and cut ones.  The tensor cores cut off what a sum
    has no room for: on average 2^-24 of it in each of the 16 additions of a step of 128 keys,
    an error of one sign that grows with the steps until outputs are taken out (8 steps for fp32,
    64 for f16).  What the outputs lack along their own direction is at most 16 x 64 x 2^-24 =
    6.1e-5; the rounding to f16 (1.6e-4 of an output, in no direction) leaves 5 x 1.6e-4 / sqrt(48
    rows of 64) = 1.5e-5 there."""
    rng = np.random.default_rng(50)
    n, heads = 131072, 8
    host = ops.Cache(rng, [n], 1, 64, dim)
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    scale = float(np.float32(1 / np.sqrt(dim)))
    out, lse = attend(handle, host, q, [tokens], [n], scale)
    rows = some(rng, tokens, heads, 44)
    check_rows(out, lse, host, q, n, scale, rows, dtype)
    x, k, v = ops.to_host(q), host.keys(0, n, 0), host.values(0, n, 0)
    got, want = [], []
    for i, h in rows:
        s = scale * (k[:n - tokens + i + 1] @ x[i, h])
        p = np.exp(s - s.max())
        want.append(p @ v[:len(p)] / p.sum())
        got.append(ops.to_host(out[i, h]))
    got, want = np.array(got), np.array(want)
    assert abs(((got - want) * want).sum()) <= (6.1e-5 + (1.5e-5 if dtype == "f16" else 0)) * (want * want).sum()
    assert status(handle) == 0


@pytest.mark.parametrize("entry", [-2**31, -1, 2**31 - 1, 3])
@pytest.mark.parametrize("tokens", [1, 100])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_every_page_outside_the_cache_is_reported(handle, at, tokens, entry):
    """Any number that is none of the three pages, and no row of another sequence suffers."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(52)
    host = ops.Cache(rng, [100], 1, 64, 64, spare=1)
    host.table = np.stack([host.table[0], host.table[0]])[:, [0, 1, 1]]
    good = host.table.copy()
    host.table[0, at] = entry
    q = ops.to_device(rng.standard_normal((2 * tokens, 2, 64)).astype(np.float32))
    out, lse = attend(handle, host, q, [tokens] * 2, [180, 100], 0.125)
    assert status(handle) == 4
    host.table = good
    check_rows(out, lse, host, q, 100, 0.125, some(rng, tokens, 2), b=1, first=tokens, count=tokens)


def test_a_sequence_alone_and_in_a_batch(handle):
    """Where a walk is cut goes by everything that a call is given, so a sequence's rows may differ
    in their last bits with the rest of the batch; both are within the tolerance of the exact."""
    rng = np.random.default_rng(54)
    counts, lengths = [1, 70, 3, 1], [3000, 900, 1500, 64]
    host = ops.Cache(rng, lengths, 2, 32, 128)
    table = host.table
    q = ops.to_device(rng.standard_normal((75, 8, 128)).astype(np.float32))
    out, lse = attend(handle, host, q, counts, lengths, 0.1)
    scale = float(np.float32(0.1))
    for b in range(4):
        first = sum(counts[:b])
        rows = some(rng, counts[b], 8, 20)
        check_rows(out, lse, host, q, lengths[b], scale, rows, b=b, first=first, count=counts[b])
        host.table = table[b:b + 1]
        x = q[first:first + counts[b]]
        alone = attend(handle, host, x, counts[b:b + 1], lengths[b:b + 1], 0.1)
        check_rows(*alone, host, x, lengths[b], scale, rows)
        host.table = table
    assert status(handle) == 0


@pytest.mark.parametrize("window", [0, 2, 5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_before_the_sequence_that_are_not_causal(handle, dtype, window):
    """More queries than tokens: the first ones have negative positions and see what their window
    leaves, like any other; those of an empty sequence see nothing.  Both kernels."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(55)
    lengths, counts = [3, 0, 20], [7, 2, 30]
    host = ops.Cache(rng, lengths, 1, 16, 64)
    q = ops.to_device(rng.standard_normal((39, 2, 64)).astype(np.float32), dtype)
    offsets = np.array([0, 7, 9, 39], np.int32)
    want = ops.attention(host, ops.to_host(q), offsets, lengths, 0.125, causal=False, window=window)
    try:
        for split in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, split)
            check(*attend(handle, host, q, counts, lengths, 0.125, causal=False, window=window), want, dtype)
            assert status(handle) == 0
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_log_sums_of_a_few_keys(handle, dim, dtype):
    """Small scores of 1 to 20 keys: a log sum's own error, without the scores' share.  The logarithm
    of a sum up to 32 is off by 5 x 2^-22 in powers of two, or 2^-20.2 in its own unit, and each
    of the three roundings after it by 2^-24 of at most 8: 2^-20 + 2^-22 in all, beside 2^-20 of
    the scores' sums of products.  Both kernels."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(56)
    lengths = [1 + i % 20 for i in range(120)]
    host = ops.Cache(rng, lengths, 2, 16, dim)
    q = ops.to_device((rng.standard_normal((240, 8, dim)) * 0.05).astype(np.float32), dtype)
    offsets = np.arange(121, dtype=np.int32) * 2
    want = ops.attention(host, ops.to_host(q), offsets, lengths, 0.125)
    some_key = ~np.isneginf(want[1])
    try:
        for split in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, split)
            _, lse = attend(handle, host, q, [2] * 120, lengths, 0.125)
            error = np.abs(ops.to_host(lse)[some_key] - want[1][some_key])
            assert np.all(error <= (2.0**-20 * want[3] + 2.0**-20 + 2.0**-22)[some_key])
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)

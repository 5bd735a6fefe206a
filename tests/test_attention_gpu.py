"""Attention over the paged 8-bit cache against float64.

Tolerance of a row: the query's two fp16 terms leave 2^-22 of its largest element, so a score
is off by at most 2^-21 S, S = scale sum |q k| (doubled for the fp32 sums), the weights
relatively by twice that, and the weights' own terms, exponentials and sums add 2^-19 at
most for these lengths.  The outputs are means of values no larger than A, so they are off by
A (2^-19 S + 2^-18); then comes the rounding to the output's type."""
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


def status(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    return q4lin.q4lin_check_device_status(handle.ptr, torch.cuda.current_stream().cuda_stream)[1]


def check(out, lse, want, dtype):
    ref, ref_lse, vmax, smax = want
    one_term = 2.0**-11 if dtype == "bf16" else 0.0
    bound = (vmax * (2.0**-19 * smax + 2.0**-18 + one_term))[..., None] + ops.ROUND[dtype] * np.abs(ref) + ops.TINY[dtype]
    err = np.abs(ops.to_host(out) - ref)
    assert np.all(err <= bound), f"out: {np.max(err / bound):.3g} times the tolerance"
    got = ops.to_host(lse)
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got), empty)
    err = np.abs(got[~empty] - ref_lse[~empty])
    bound = (2.0**-20 * smax + 2.0**-20 + 2.0**-22 * np.abs(np.where(empty, 0, ref_lse)))[~empty]
    assert np.all(err <= bound), f"lse: {np.max(err / bound):.3g} times the tolerance"


def run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, rotated=None, interleaved=False,
        causal=True, window=0, seed=0, gain=1.5, q=None, **more):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(seed + dim + page + sum(lengths))
    host = ops.Cache(rng, lengths, kv_heads, page, dim)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    if q is None:
        q = ops.to_device((rng.standard_normal((offsets[-1], heads, dim)) * gain).astype(np.float32), dtype)
    rotated = dim if rotated is None else rotated
    rope = ops.rope_tables(rng, max(max(lengths), 1), rotated) if rotated else None
    scale = 1 / np.sqrt(dim)
    out, lse = q4lin.attention(handle, host.device(), q, ops.to_device(offsets),
                               ops.to_device(np.array(lengths, np.int32)), scale,
                               rope=None if rope is None else tuple(map(ops.to_device, rope)),
                               interleaved=interleaved, causal=causal, window=window, **more)
    want = ops.attention(host, ops.to_host(q), offsets, lengths, float(np.float32(scale)), rope,
                         interleaved, causal, window)
    return out, lse, want, dtype


SINGLE = [
    # lengths, heads, kv heads, page, dim, dtype
    ([1], 1, 1, 16, 64, "f32"),
    ([2], 4, 1, 64, 128, "f32"),
    ([63, 64, 65], 4, 2, 64, 128, "f32"),
    ([15, 16, 17, 33], 6, 2, 16, 64, "bf16"),
    ([511, 512, 513, 700], 8, 2, 32, 128, "f16"),
    ([701], 32, 8, 16, 64, "f32"),
    ([4097, 1, 900, 0, 31], 8, 8, 64, 64, "f32"),
    ([1300, 77], 14, 2, 32, 128, "bf16"),
    ([650, 3], 8, 1, 16, 256, "f32"),
    ([300], 12, 1, 64, 128, "f32"),
    ([200, 210], 34, 2, 64, 64, "f16"),
    ([9000], 4, 4, 64, 128, "f32"),
    ([i * 7 % 130 for i in range(300)], 2, 1, 16, 64, "f32"),
]


@pytest.mark.parametrize("lengths,heads,kv_heads,page,dim,dtype", SINGLE)
def test_one_token(handle, lengths, heads, kv_heads, page, dim, dtype):
    check(*run(handle, lengths, [1] * len(lengths), heads, kv_heads, page, dim, dtype, max_query=1))
    assert status(handle) == 0


SEVERAL = [
    # lengths, query tokens, heads, kv heads, page, dim, dtype, causal, window
    ([5], [5], 4, 2, 16, 64, "f32", True, 0),
    ([70, 9, 128], [3, 0, 5], 4, 1, 32, 128, "f32", True, 0),
    ([70, 9, 128], [3, 2, 5], 4, 1, 32, 128, "bf16", False, 0),
    ([200, 130], [17, 4], 6, 2, 64, 128, "f16", True, 50),
    ([100, 3, 0], [2, 5, 2], 2, 2, 16, 64, "f32", True, 0),   # queries before the sequence: empty rows
    ([100, 3], [2, 5], 2, 2, 16, 64, "f32", True, 1),
    ([333], [70], 7, 1, 64, 256, "f32", True, 100),
    ([333], [70], 8, 2, 64, 128, "f32", False, 33),
    ([260, 40, 600], [150, 1, 90], 4, 2, 16, 128, "bf16", True, 0),
    ([260, 40, 600], [150, 1, 90], 4, 2, 64, 64, "f32", True, 0),
    ([400], [400], 3, 1, 32, 64, "f16", True, 0),
    ([129], [129], 2, 1, 64, 128, "f32", True, 0),
    ([640, 2], [200, 2], 5, 1, 64, 128, "f32", True, 64),
]


@pytest.mark.parametrize("lengths,counts,heads,kv_heads,page,dim,dtype,causal,window", SEVERAL)
def test_several_tokens(handle, lengths, counts, heads, kv_heads, page, dim, dtype, causal, window):
    check(*run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, causal=causal, window=window))
    assert status(handle) == 0


PROMPTS = [
    # lengths, query tokens, heads, kv heads, page, dim, dtype, causal, window
    ([1], [1], 1, 1, 16, 64, "f32", True, 0),
    ([5], [5], 4, 2, 64, 128, "f32", True, 0),
    ([130, 9, 128], [3, 0, 5], 4, 1, 32, 128, "bf16", True, 0),
    ([129, 300], [129, 2], 3, 1, 16, 128, "f16", True, 0),
    ([200, 130], [17, 4], 6, 2, 64, 64, "bf16", False, 50),
    ([700, 3, 0], [90, 5, 2], 7, 1, 32, 128, "f32", True, 100),
    ([400], [400], 3, 1, 64, 64, "f32", True, 0),
    ([513], [513], 2, 2, 16, 64, "bf16", True, 0),
    ([640, 2], [200, 2], 5, 1, 64, 128, "bf16", True, 64),
    ([3], [7], 2, 1, 64, 128, "f32", True, 0),
    ([1500], [40], 8, 1, 32, 128, "f16", False, 0),
]


CUT = [
    # Few rows over many keys: walks in parts, some shorter than others, and a tile without rows.
    ([5000], [3], 4, 1, 64, 128, "f32", True, 0),
    ([4097, 130, 1], [40, 40, 1], 4, 2, 16, 64, "bf16", True, 0),
    ([3000, 2900], [100, 7], 3, 1, 32, 128, "f16", False, 0),
    ([6000], [150], 2, 1, 64, 64, "f32", True, 2000),
    ([2500, 0, 700], [2, 3, 300], 8, 2, 64, 128, "bf16", True, 300),
]


@pytest.mark.parametrize("lengths,counts,heads,kv_heads,page,dim,dtype,causal,window", PROMPTS + CUT)
def test_prompt_kernel(handle, lengths, counts, heads, kv_heads, page, dim, dtype, causal, window):
    """Every size through the prompts' kernel, then the same call by the other one."""
    from bit_weight_quantized_int4_gb300 import q4lin
    try:
        for rows in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, rows)
            check(*run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, causal=causal, window=window))
            assert status(handle) == 0
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,window", [(5120, 0), (7700, 0), (7700, 3000), (10000, 0)])
def test_more_walks_than_sms(handle, tokens, window, dtype):
    """Whole walks and those of a last round that are cut; rows all over it, the last ones too."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(tokens)
    heads, dim = 8, 64
    host = ops.Cache(rng, [tokens], heads, 64, dim)
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    offsets = np.array([0, tokens], np.int32)
    out, lse = q4lin.attention(handle, host.device(), q, ops.to_device(offsets),
                               ops.to_device(np.array([tokens], np.int32)), 0.125, window=window)
    rows = np.concatenate([[0, 1, 255, 256, tokens - 1], rng.integers(0, tokens, 120)])
    at = np.concatenate([np.arange(5) % heads, rng.integers(0, heads, 120)])
    want = [[], [], [], []]
    keys = [(host.keys(0, tokens, h), host.values(0, tokens, h)) for h in range(heads)]
    x = ops.to_host(q)
    for i, h in zip(rows, at):
        seen = slice(max(0, i - window + 1) if window else 0, i + 1)
        k, v = keys[h][0][seen], keys[h][1][seen]
        s = 0.125 * (k @ x[i, h])
        p = np.exp(s - s.max())
        for one, value in zip(want, (p @ v / p.sum(), s.max() + np.log(p.sum()), np.abs(v).max(),
                                     (0.125 * (np.abs(k) @ np.abs(x[i, h]))).max())):
            one.append(value)
    check(out[rows, at], lse[rows, at], [np.array(w) for w in want], dtype)
    assert status(handle) == 0


def test_long_fp32_prompt(handle):
    """Sums over 16384 keys.  The tensor cores cut off instead of rounding: at most 2^-24 of a sum
    on average for each of the 256 additions (2048 keys in steps of 16, two terms) between two
    roundings to memory, 1.5e-5 of the outputs' norm."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(31)
    n, tokens, heads, dim = 16384, 2048, 8, 64
    host = ops.Cache(rng, [n], heads, 16, dim)
    q = ops.to_device((rng.standard_normal((tokens, heads, dim)) * 1.2).astype(np.float32))
    q = q.repeat_interleave(3, 1)  # 192 walks
    out, _ = q4lin.attention(handle, host.device(), q, ops.to_device(np.array([0, tokens], np.int32)),
                             ops.to_device(np.array([n], np.int32)), 0.125)
    x, got, want = ops.to_host(q), ops.to_host(out), []
    rows = [(int(i), h) for h in range(heads) for i in rng.integers(0, tokens, 6)]
    for i, h in rows:
        k, v = host.keys(0, n, h)[:n - tokens + i + 1], host.values(0, n, h)[:n - tokens + i + 1]
        s = 0.125 * (k @ x[i, 3 * h])
        p = np.exp(s - s.max())
        want.append(p @ v / p.sum())
    want = np.array(want)
    error = np.array([got[i, 3 * h] for i, h in rows]) - want
    assert np.linalg.norm(error) <= 1.5e-5 * np.linalg.norm(want)


def test_values_of_very_different_pages(handle):
    """Pages whose values are 2^12 apart, and one of zeros: rows that see only small ones."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(17)
    host = ops.Cache(rng, [256], 1, 64, 128)
    for i, s in enumerate((2.0**-12, 0.0, 1.0, 2.0**-12)):
        host.vs[host.table[0, i]] = s
    offsets = np.array([0, 256], np.int32)
    q = torch.randn(256, 2, 128, device="cuda")
    out, lse = q4lin.attention(handle, host.device(), q, ops.to_device(offsets),
                               ops.to_device(np.array([256], np.int32)), 0.1)
    check(out, lse, ops.attention(host, ops.to_host(q), offsets, [256], float(np.float32(0.1))), "f32")


@pytest.mark.parametrize("rotated,interleaved", [(0, False), (32, False), (32, True), (128, True)])
def test_rotation(handle, rotated, interleaved):
    check(*run(handle, [100, 40], [1, 3], 4, 2, 32, 128, "f32", rotated=rotated, interleaved=interleaved))


def test_more_sequences_than_one_launch_takes(handle):
    """1100 sequences of 0 to 40 tokens, one query each; then prompts among them."""
    lengths = [i * 7 % 41 for i in range(1100)]
    check(*run(handle, lengths, [1] * 1100, 2, 1, 16, 64, "f32", max_query=1))
    counts = [min(n, 30) if i % 100 == 0 else 1 for i, n in enumerate(lengths)]
    check(*run(handle, lengths, counts, 2, 1, 16, 64, "f32"))
    assert status(handle) == 0


def test_negative_and_zero_scale(handle):
    """The smallest scores weigh most, or all keys alike; both kernels."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(19)
    host = ops.Cache(rng, [300], 1, 32, 64)
    q = ops.to_device(rng.standard_normal((40, 2, 64)).astype(np.float32))
    offsets = np.array([0, 40], np.int32)
    for scale in (-0.25, 0.0):
        for rows in (1, 1 << 40):
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, rows)
            out, lse = q4lin.attention(handle, host.device(), q, ops.to_device(offsets),
                                       ops.to_device(np.array([300], np.int32)), scale)
            handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)
            ref = ops.attention(host, ops.to_host(q), offsets, [300], scale)
            check(out, lse, (*ref[:3], np.abs(ref[3])), "f32")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("count", [1, 5, 200])
def test_pages_before_the_window_may_be_gone(handle, count, page):
    """A window of 50 keys behind each query: the pages before the first query's hold NaN scales
    and have left the table."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(21)
    n, window = 500, 50
    host = ops.Cache(rng, [n], 2, page, 64)
    gone = host.table[0, :(n - count - window + 1) // page]
    host.ks[gone], host.vs[gone] = np.nan, np.nan
    device = host.device()
    device.page_table[0, :len(gone)] = -1
    q = ops.to_device(rng.standard_normal((count, 4, 64)).astype(np.float32))
    offsets = np.array([0, count], np.int32)
    out, lse = q4lin.attention(handle, device, q, ops.to_device(offsets),
                               ops.to_device(np.array([n], np.int32)), 0.125, window=window)
    check(out, lse, ops.attention(host, ops.to_host(q), offsets, [n], 0.125, window=window), "f32")
    assert status(handle) == 0


def test_a_wait_that_runs_out_is_reported(handle):
    """Keys that do not come: the kernels give up, leave, and work again afterwards."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = ops.Cache(np.random.default_rng(20), [3000], 2, 64, 128)
    cache, q = host.device(), torch.randn(200, 4, 128, device="cuda")
    n = ops.to_device(np.array([3000], np.int32))
    for tokens in (1, 200):
        o = ops.to_device(np.array([0, tokens], np.int32))
        want = q4lin.attention(handle, cache, q[:tokens], o, n, 0.1)[0]
        handle.set_option(q4lin.Q4LIN_OPT_WAIT_LIMIT, 1000000)  # 1 ms
        handle.set_option(q4lin.Q4LIN_OPT_TC_SKIP_FIRST_COPY, 1)
        q4lin.attention(handle, cache, q[:tokens], o, n, 0.1)
        handle.set_option(q4lin.Q4LIN_OPT_TC_SKIP_FIRST_COPY, 0)
        handle.set_option(q4lin.Q4LIN_OPT_WAIT_LIMIT, 0)
        assert status(handle) == 1
        assert torch.equal(q4lin.attention(handle, cache, q[:tokens], o, n, 0.1)[0], want)
        assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 40.0])
def test_tiny_and_large_scores(handle, dtype, size):
    """Scores all alike, and one weight that takes everything."""
    check(*run(handle, [150], [2], 4, 2, 16, 64, dtype, gain=size))


def test_slices_of_one_projection(handle):
    import torch
    wide = torch.randn(3, 1 + 8 * 64 + 64, device="cuda")
    for shift in (0, 1, 4):
        q = wide[:, shift:shift + 512].unflatten(1, (8, 64))
        check(*run(handle, [50, 20], [2, 1], 8, 2, 16, 64, "f32", q=q))


def test_results_do_not_depend_on_the_rest_of_the_batch_or_the_run(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(4)
    host = ops.Cache(rng, [3000, 50, 700], 2, 64, 128)
    cache = host.device()
    q = torch.randn(3, 8, 128, device="cuda")
    o, n = (ops.to_device(np.array(a, np.int32)) for a in ([0, 1, 2, 3], [3000, 50, 700]))
    first = q4lin.attention(handle, cache, q, o, n, 0.1, max_query=1)
    for _ in range(5):
        again = q4lin.attention(handle, cache, q, o, n, 0.1, max_query=1)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("counts", [[1], [200]])
def test_a_nan_stays_in_its_row_and_unseen_pages_are_not_read(handle, counts):
    """A NaN in one query; NaN scales of pages that no sequence has."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(11)
    host = ops.Cache(rng, [230], 2, 64, 128)
    used = host.table[0, :4]
    for s in (host.ks, host.vs):
        spare = np.setdiff1d(np.arange(host.total), used)
        s[spare] = np.nan
    q = torch.randn(counts[0], 4, 128, device="cuda")
    q[0, 1, 7] = float("nan")
    offsets = np.array([0, counts[0]], np.int32)
    out, lse = q4lin.attention(handle, host.device(), q, ops.to_device(offsets),
                               ops.to_device(np.array([230], np.int32)), 0.1)
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[0, 1] = True
    assert torch.equal(bad, want) and torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    q[0, 1, 7] = 0
    ref = ops.attention(host, ops.to_host(q), offsets, [230], float(np.float32(0.1)))
    ok = ~want.cpu().numpy()
    err = np.abs(ops.to_host(out) - ref[0])[ok]
    assert np.all(err <= (ref[2] * (2.0**-19 * ref[3] + 2.0**-18))[ok][:, None] + 1e-7)


def test_masked_places_may_hold_anything(handle):
    """Bytes of a page past the sequence's end change nothing."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(12)
    host = ops.Cache(rng, [70], 1, 64, 64)
    q = torch.randn(70, 2, 64, device="cuda")
    results = []
    for fill in (0, 255):
        last = host.table[0, 1]
        host.k[last, 0, 6:] = fill
        host.v[last, 0, :, 6:] = fill
        cache = host.device()
        for n in (1, 70):
            results.append(q4lin.attention(handle, cache, q[:n], ops.to_device(np.array([0, n], np.int32)),
                                           ops.to_device(np.array([70], np.int32)), 0.125)[0])
    assert torch.equal(results[0], results[2]) and torch.equal(results[1], results[3])


def test_append_then_attend(handle):
    """The two together, token by token, against attention over unquantised keys."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(13)
    table = ops.to_device(np.arange(8, dtype=np.int32).reshape(2, 4))
    cache = q4lin.KVCache.empty(8, 2, 16, 64, table)
    rope = tuple(map(ops.to_device, ops.rope_tables(rng, 64, 64)))
    offsets = ops.to_device(np.array([0, 1, 2], np.int32))
    x = rng.standard_normal((3, 40, 2, 2, 64)).astype(np.float32)  # k, v, q of each step
    k_all, v_all = [], []
    for i in range(40):
        k, v, q = (ops.to_device(x[j, i]) for j in range(3))
        at = torch.full((2,), i, dtype=torch.int32, device="cuda")
        q4lin.kv_append(handle, cache, k, v, offsets, at, rope=rope)
        out, _ = q4lin.attention(handle, cache, q, offsets, at + 1, 0.125, max_query=1, rope=rope)
        position = np.full(2, i)
        host_rope = tuple(t.cpu().numpy() for t in rope)
        k_all.append(ops.rotate(x[0, i], position, host_rope, False))
        v_all.append(x[1, i])
        qr = ops.rotate(x[2, i], position, host_rope, False)
        for b in range(2):
            for h in range(2):
                kk, vv = np.array(k_all)[:, b, h], np.array(v_all)[:, b, h]
                p = np.exp(0.125 * kk @ qr[b, h])
                ref = p @ vv / p.sum()
                # A code is within half a step, and each growth of the scale adds half of one:
                # some steps of 1/127 of the largest element, which are averaged.
                assert np.max(np.abs(ops.to_host(out)[b, h] - ref)) < 0.1
    assert status(handle) == 0


def test_indices_out_of_range_are_reported(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(14)
    host = ops.Cache(rng, [100], 1, 64, 64, spare=0)
    q = torch.randn(2, 2, 64, device="cuda")
    for table, lengths, offsets, most in (([[0, 9]], [100], [0, 2], 2), ([[0, -1]], [100], [0, 2], 2),
                                          ([[0, 1]], [129], [0, 2], 2), ([[0, 1]], [100], [0, 3], 2),
                                          ([[0, 1]], [100], [0, 2], 1), ([[0, 1]], [100], [1, 0], 2)):
        host.table = np.array(table, np.int32)
        q4lin.attention(handle, host.device(), q, ops.to_device(np.array(offsets, np.int32)),
                        ops.to_device(np.array(lengths, np.int32)), 0.1, max_query=most)
        assert status(handle) == 4


def test_other_stream_and_nothing_to_do(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = ops.Cache(np.random.default_rng(15), [100], 1, 64, 64)
    cache, q = host.device(), torch.randn(1, 2, 64, device="cuda")
    o, n = (ops.to_device(np.array(a, np.int32)) for a in ([0, 1], [100]))
    want = q4lin.attention(handle, cache, q, o, n, 0.1)[0]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(q, 7.0)
    stream.wait_stream(torch.cuda.current_stream())
    q4lin.attention(handle, cache, q, o, n, 0.1, out=out, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(out, want)
    empty, _ = q4lin.attention(handle, cache, q[:0], o, n, 0.1)
    assert empty.shape == (0, 2, 64)


def test_refusals(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    cache = ops.Cache(np.random.default_rng(16), [100], 2, 64, 64).device()
    q = torch.randn(1, 4, 64, device="cuda")
    o, n = (ops.to_device(np.array(a, np.int32)) for a in ([0, 1], [100]))
    for change in (dict(query=q[:, :3]), dict(query=q[..., :32]), dict(query=q.double()), dict(offsets=n),
                   dict(lengths=n.long()), dict(out=q.half()), dict(lse=q[..., 0].half()),
                   dict(query=q.transpose(1, 2)), dict(query=q.cpu())):
        args = dict(dict(query=q, offsets=o, lengths=n), **change)
        with pytest.raises(ValueError):
            q4lin.attention(handle, cache, scale=0.1, **args)
    inv = q4lin.Q4LIN_ERR_INVALID_ARG
    for change in (dict(window=-1), dict(max_query=0), dict(causal=2), dict(out=q)):
        with pytest.raises(q4lin.Q4LinError) as e:
            q4lin.attention(handle, cache, q, o, n, 0.1, **change)
        assert e.value.status == inv
    wide = q4lin.q4lin_kv_cache_t.from_buffer_copy(cache.args)
    wide.pages_per_sequence = wide.table_stride = 1 << 40
    a = q4lin.q4lin_attention_t(q.data_ptr(), 256, 64, torch.empty_like(q).data_ptr(), None, 0, 1, 4, 1,
                                o.data_ptr(), n.data_ptr(), 0.1, 1, 0, q4lin.q4lin_rope_t())
    assert q4lin.q4lin_run_attention(handle.ptr, wide, a, 0) == q4lin.Q4LIN_ERR_TOO_LARGE
    assert q4lin.q4lin_run_attention(handle.ptr, cache.args, None, 0) == inv
    torch.cuda.synchronize()

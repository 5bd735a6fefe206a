"""Attention over the paged 4-bit cache against float64.

Tolerance of a row as in test_attention_gpu: the query's two fp16 terms leave 2^-22 of its largest
element, so a score is off by at most 2^-21 S, S = scale sum |q k| (doubled for the fp32 sums); a
key's scale rounds once more in fp32, which the same factor covers.  The weights and their
products with the values' scales are off relatively by twice that and 2^-19 for terms, exponentials
and sums.  Outputs are means of values no larger than A: A (2^-19 S + 2^-18), and the rounding to
the type; bf16 outputs may take weights of one term, 2^-11."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_attention_gpu import CUT, PROMPTS, SEVERAL, SINGLE, check, status

pytestmark = pytest.mark.gpu
BOTH = (1, 1 << 40)  # rows a head up to which the kernel for few rows takes a sequence: either kernel


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


@pytest.fixture
def split(handle):
    """Sets which kernel takes what, and the rule again afterwards."""
    from bit_weight_quantized_int4_gb300 import q4lin
    yield lambda rows: handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, rows)
    handle.set_option(q4lin.Q4LIN_OPT_ATTENTION_SPLIT_ROWS, 0)


def attend(handle, host, q, counts, lengths, scale, cache=None, **more):
    from bit_weight_quantized_int4_gb300 import q4lin
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return q4lin.attention(handle, host.device() if cache is None else cache, q, ops.to_device(offsets),
                           ops.to_device(np.array(lengths, np.int32)), scale, **more)


def run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, rotated=0, interleaved=False,
        causal=True, window=0, seed=0, gain=1.5, q=None, **more):
    rng = np.random.default_rng(seed + dim + page + sum(lengths))
    host = kv4.Cache(rng, lengths, kv_heads, page, dim)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    if q is None:
        q = ops.to_device((rng.standard_normal((offsets[-1], heads, dim)) * gain).astype(np.float32), dtype)
    rope = ops.rope_tables(rng, max(max(lengths), 1), rotated) if rotated else None
    scale = float(np.float32(1 / np.sqrt(dim)))
    out, lse = attend(handle, host, q, counts, lengths, scale, rope=rope and tuple(map(ops.to_device, rope)),
                      interleaved=interleaved, causal=causal, window=window, **more)
    return out, lse, ops.attention(host, ops.to_host(q), offsets, lengths, scale, rope, interleaved, causal, window), dtype


def check_rows(out, lse, host, q, n, scale, rows, dtype="f32", b=0, first=0, count=None, causal=True, window=0):
    """Pairs (token, head) of `rows`, of sequence b of n tokens, whose queries begin at row `first`."""
    x, want = ops.to_host(q), [[], [], [], []]
    count = q.shape[0] if count is None else count
    group, kept = q.shape[1] // host.heads, {}
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
    ends = [(0, 0), (0, heads - 1), (count - 1, 0), (count - 1, heads - 1)]
    return ends + [(int(rng.integers(count)), int(rng.integers(heads))) for _ in range(n)]


@pytest.mark.parametrize("lengths,heads,kv_heads,page,dim,dtype", SINGLE)
def test_one_token(handle, lengths, heads, kv_heads, page, dim, dtype):
    check(*run(handle, lengths, [1] * len(lengths), heads, kv_heads, page, dim, dtype, max_query=1))
    assert status(handle) == 0


@pytest.mark.parametrize("lengths,counts,heads,kv_heads,page,dim,dtype,causal,window", SEVERAL)
def test_several_tokens(handle, lengths, counts, heads, kv_heads, page, dim, dtype, causal, window):
    check(*run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, rotated=dim, causal=causal, window=window))
    assert status(handle) == 0


@pytest.mark.parametrize("lengths,counts,heads,kv_heads,page,dim,dtype,causal,window", PROMPTS + CUT)
def test_both_kernels(handle, split, lengths, counts, heads, kv_heads, page, dim, dtype, causal, window):
    for rows in BOTH:
        for rotated in (0, dim):
            split(rows)
            check(*run(handle, lengths, counts, heads, kv_heads, page, dim, dtype, rotated=rotated, causal=causal,
                       window=window))
            assert status(handle) == 0


@pytest.mark.parametrize("rotated,interleaved", [(32, False), (32, True), (128, True), (8, False)])
@pytest.mark.parametrize("counts", [[1, 3], [100, 3]])
def test_rotation(handle, split, counts, rotated, interleaved):
    for rows in BOTH:
        split(rows)
        check(*run(handle, [100, 40], counts, 4, 2, 32, 128, "f32", rotated=rotated, interleaved=interleaved))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,window,dim", [(5120, 0, 64), (7700, 3000, 64), (6000, 0, 128)])
def test_more_walks_than_sms(handle, tokens, window, dim, dtype):
    rng = np.random.default_rng(tokens)
    host = kv4.Cache(rng, [tokens], 8, 64, dim)
    q = ops.to_device(rng.standard_normal((tokens, 8, dim)).astype(np.float32), dtype)
    out, lse = attend(handle, host, q, [tokens], [tokens], 0.125, window=window)
    check_rows(out, lse, host, q, tokens, 0.125, some(rng, tokens, 8, 80), dtype, window=window)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 200])
def test_scales_that_are_far_apart(handle, split, tokens, dtype):
    """Neighbouring tokens whose scales are up to 2^30 apart, and some of zero; the smallest ones' rows
    are those whose window sees nothing else."""
    rng = np.random.default_rng(17)
    host = kv4.Cache(rng, [300], 1, 32, 64)
    host.vs *= (2.0**rng.integers(-30, 1, host.vs.shape)).astype(np.float32)
    host.ks *= (2.0**rng.integers(-30, 1, host.ks.shape)).astype(np.float32)
    host.vs[rng.random(host.vs.shape) < 0.1] = 0
    host.ks[rng.random(host.ks.shape) < 0.1] = 0
    q = ops.to_device(rng.standard_normal((tokens, 2, 64)).astype(np.float32), dtype)
    offsets = np.array([0, tokens], np.int32)
    want = ops.attention(host, ops.to_host(q), offsets, [300], 0.125)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [tokens], [300], 0.125), want, dtype)
    host.vs[:] = 0
    want = ops.attention(host, ops.to_host(q), offsets, [300], 0.125)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, [tokens], [300], 0.125), want, dtype)


@pytest.mark.parametrize("tokens", [1, 9, 200])
def test_slots_behind_a_sequence_may_hold_anything(handle, split, tokens):
    """Codes, and scales of infinity and NaN, behind the last token, in the same page and in pages of
    no sequence."""
    import torch
    rng = np.random.default_rng(12)
    host = kv4.Cache(rng, [230], 2, 64, 128)
    q = torch.randn(tokens, 4, 128, device="cuda")
    for rows in BOTH:
        split(rows)
        results = []
        for fill in (0.0, float("nan"), float("inf"), -float("inf")):
            last, spare = host.table[0, 3], np.setdiff1d(np.arange(host.total), host.table[0, :4])
            for s, c in ((host.ks, host.k), (host.vs, host.v)):
                s[last, :, 230 - 192:] = fill
                s[spare] = fill
                c[last, :, 230 - 192:] = 0 if fill == 0 else 15
            results.append(attend(handle, host, q, [tokens], [230], 0.1))
        for out, lse in results[1:]:
            assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    assert status(handle) == 0


def test_more_sequences_than_one_launch_takes(handle):
    lengths = [i * 7 % 41 for i in range(1100)]
    check(*run(handle, lengths, [1] * 1100, 2, 1, 16, 64, "f32", max_query=1))
    counts = [min(n, 30) if i % 100 == 0 else 1 for i, n in enumerate(lengths)]
    check(*run(handle, lengths, counts, 2, 1, 16, 64, "f32"))
    assert status(handle) == 0


def test_negative_and_zero_scale(handle, split):
    rng = np.random.default_rng(19)
    host = kv4.Cache(rng, [300], 1, 32, 64)
    q = ops.to_device(rng.standard_normal((40, 2, 64)).astype(np.float32))
    for scale in (-0.25, 0.0):
        for rows in BOTH:
            split(rows)
            ref = ops.attention(host, ops.to_host(q), [0, 40], [300], scale)
            check(*attend(handle, host, q, [40], [300], scale), (*ref[:3], np.abs(ref[3])), "f32")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("count", [1, 5, 200])
def test_pages_before_the_window_may_be_gone(handle, count, page):
    rng = np.random.default_rng(21)
    n, window = 500, 50
    host = kv4.Cache(rng, [n], 2, page, 64)
    gone = host.table[0, :(n - count - window + 1) // page]
    host.ks[gone], host.vs[gone] = np.nan, np.nan
    device = host.device()
    device.page_table[0, :len(gone)] = -1
    q = ops.to_device(rng.standard_normal((count, 4, 64)).astype(np.float32))
    out, lse = attend(handle, host, q, [count], [n], 0.125, cache=device, window=window)
    check(out, lse, ops.attention(host, ops.to_host(q), [0, count], [n], 0.125, window=window), "f32")
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 40.0])
def test_tiny_and_large_scores(handle, split, dtype, size):
    for rows in BOTH:
        split(rows)
        check(*run(handle, [150], [2], 4, 2, 16, 64, dtype, gain=size))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_near_the_largest_number(handle, split, dim, dtype):
    rng = np.random.default_rng(48)
    host = kv4.Cache(rng, [300], 2, 32, dim)
    host.ks /= 64
    q = rng.uniform(-1, 1, (70, 4, dim)) * 2.0**rng.integers(120, 128, (70, 4, 1))
    q = ops.to_device(q.astype(np.float32), dtype)
    q[q.isinf()] = 0
    for rows in BOTH:
        split(rows)
        out, lse = attend(handle, host, q, [70], [300], 2.0**-124)
        check_rows(out, lse, host, q, 300, 2.0**-124, some(rng, 70, 4, 80), dtype)


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n,tokens", [(1, 1), (200, 130)])
def test_an_infinite_query_gives_nan(handle, split, n, tokens, dim, dtype, rotated):
    """Also where every key has the same sign in its channel; the other rows are as they were."""
    import torch
    rng = np.random.default_rng(49)
    host = kv4.Cache(rng, [n], 1, 16, dim)
    host.k[..., 3] = host.k[..., 3] % 8      # codes below 8
    host.k[..., 5] = 9 + host.k[..., 5] % 7  # and above
    cache = host.device()
    angle = np.zeros((n, dim // 2), np.float32)
    rope = (ops.to_device(angle + 1), ops.to_device(angle)) if rotated else None
    q = ops.to_device(rng.standard_normal((tokens, 4, dim)).astype(np.float32), dtype)
    for rows in BOTH:
        split(rows)
        want, want_lse = attend(handle, host, q, [tokens], [n], 0.1, cache=cache, rope=rope)
        assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
        for channel, value in ((3, float("inf")), (3, -float("inf")), (5, float("inf")), (5, -float("inf")),
                               (0, float("nan"))):
            x = q.clone()
            x[-1, 2, channel] = value
            out, lse = attend(handle, host, x, [tokens], [n], 0.1, cache=cache, rope=rope)
            assert torch.isnan(out[-1, 2]).all() and torch.isnan(lse[-1, 2])
            out[-1, 2], lse[-1, 2] = want[-1, 2], want_lse[-1, 2]
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_slices_of_one_projection(handle):
    import torch
    wide = torch.randn(3, 1 + 8 * 64 + 64, device="cuda")
    for shift in (0, 1, 4):
        q = wide[:, shift:shift + 512].unflatten(1, (8, 64))
        check(*run(handle, [50, 20], [2, 1], 8, 2, 16, 64, "f32", q=q))


def test_the_same_call_gives_the_same_bits(handle):
    import torch
    rng = np.random.default_rng(4)
    host = kv4.Cache(rng, [3000, 50, 700], 2, 64, 128)
    cache = host.device()
    for counts in ([1, 1, 1], [100, 1, 300]):
        q = torch.randn(sum(counts), 8, 128, device="cuda")
        first = attend(handle, host, q, counts, [3000, 50, 700], 0.1, cache=cache)
        for _ in range(5):
            again = attend(handle, host, q, counts, [3000, 50, 700], 0.1, cache=cache)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tokens,n,heads,kv_heads,dim,dtype,window", [
    (600, 600, 4, 1, 64, "f32", 50), (600, 900, 3, 1, 128, "f32", 256), (1000, 1000, 1, 1, 64, "f16", 33),
    (1024, 3000, 4, 1, 64, "f32", 1), (1100, 1100, 40, 10, 128, "bf16", 256)])
def test_a_window_without_an_end(handle, split, tokens, n, heads, kv_heads, dim, dtype, window, causal):
    rng = np.random.default_rng(43)
    host = kv4.Cache(rng, [n], kv_heads, 32, dim)
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    rows, scale = some(rng, tokens, heads), float(np.float32(1 / np.sqrt(dim)))
    for r in BOTH:
        split(r)
        out, lse = attend(handle, host, q, [tokens], [n], scale, causal=causal, window=window)
        check_rows(out, lse, host, q, n, scale, rows, dtype, causal=causal, window=window)
        assert status(handle) == 0


@pytest.mark.parametrize("window", [0, 2, 5, 2**63 - 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_before_the_sequence_that_are_not_causal(handle, split, dtype, window):
    rng = np.random.default_rng(55)
    lengths, counts = [3, 0, 20], [7, 2, 30]
    host = kv4.Cache(rng, lengths, 1, 16, 64)
    q = ops.to_device(rng.standard_normal((39, 2, 64)).astype(np.float32), dtype)
    want = ops.attention(host, ops.to_host(q), [0, 7, 9, 39], lengths, 0.125, causal=False,
                         window=window if window < 100 else 0)
    for rows in BOTH:
        split(rows)
        check(*attend(handle, host, q, counts, lengths, 0.125, causal=False, window=window), want, dtype)
        assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_log_sums_of_a_few_keys(handle, split, dim, dtype):
    """As in test_attention_edges_gpu: 2^-20 + 2^-22 in all, beside 2^-20 of the scores' sums."""
    rng = np.random.default_rng(56)
    lengths = [1 + i % 20 for i in range(120)]
    host = kv4.Cache(rng, lengths, 2, 16, dim)
    q = ops.to_device((rng.standard_normal((240, 8, dim)) * 0.05).astype(np.float32), dtype)
    want = ops.attention(host, ops.to_host(q), np.arange(121) * 2, lengths, 0.125)
    seen = ~np.isneginf(want[1])
    for rows in BOTH:
        split(rows)
        _, lse = attend(handle, host, q, [2] * 120, lengths, 0.125)
        error = np.abs(ops.to_host(lse)[seen] - want[1][seen])
        assert np.all(error <= (2.0**-20 * want[3] + 2.0**-20 + 2.0**-22)[seen])


@pytest.mark.parametrize("dtype,tokens", [("f32", 1), ("f32", 3200), ("f16", 5000)])
def test_many_keys(handle, tokens, dtype):
    """131072 keys: single tokens, whole walks and cut ones.  Means of as many values are small beside
    the values, and what the sums lack along the outputs' own direction is at most 6.1e-5 of them
    (16 additions of 2^-24 a step of 128 keys, up to 64 steps between roundings; beside it the
    rounding to f16)."""
    rng = np.random.default_rng(50)
    n, heads, dim = 131072, 8, 128
    host = kv4.Cache(rng, [n], 1, 64, dim)
    q = ops.to_device(rng.standard_normal((tokens, heads, dim)).astype(np.float32), dtype)
    scale = float(np.float32(1 / np.sqrt(dim)))
    out, lse = attend(handle, host, q, [tokens], [n], scale)
    rows = some(rng, tokens, heads, 30)
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


@pytest.mark.parametrize("tokens", [1, 100])
def test_indices_out_of_range_are_reported(handle, tokens):
    rng = np.random.default_rng(14)
    host = kv4.Cache(rng, [100], 1, 64, 64, spare=1)
    good = np.stack([host.table[0], host.table[0]])[:, [0, 1, 1]]
    q = ops.to_device(rng.standard_normal((2 * tokens, 2, 64)).astype(np.float32))
    for at in (0, 1, 2):
        for entry in (-2**31, -1, 2**31 - 1, 3):
            host.table = good.copy()
            host.table[0, at] = entry
            out, lse = attend(handle, host, q, [tokens] * 2, [180, 100], 0.125)
            assert status(handle) == 4
            host.table = good
            check_rows(out, lse, host, q, 100, 0.125, some(rng, tokens, 2), b=1, first=tokens, count=tokens)
    for lengths, counts, most in (([200, 100], [tokens] * 2, 200), ([100, 100], [tokens, 3 * tokens], 200),
                                  ([100, 100], [3 * tokens, -2 * tokens], 200)):
        attend(handle, host, q, counts, lengths, 0.1, max_query=most)
        assert status(handle) == 4
    if tokens > 1:
        attend(handle, host, q, [tokens] * 2, [180, 100], 0.1, max_query=tokens - 1)
        assert status(handle) == 4


@pytest.mark.parametrize("sequences", [3, 1500])
def test_offsets_that_rise_and_fall(handle, sequences):
    """0, n, 0, n, ...: every other sequence looks like all of the tokens; the call after it is right."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(42)
    n = 700
    host = kv4.Cache(rng, [n], 1, 64, 64)
    host.table = np.repeat(host.table, sequences, 0)
    q = ops.to_device(rng.standard_normal((n, 8, 64)).astype(np.float32))
    q4lin.attention(handle, host.device(), q, ops.to_device((np.arange(sequences + 1) % 2 * n).astype(np.int32)),
                    ops.to_device(np.full(sequences, n, np.int32)), 0.125)
    assert status(handle) == 4
    host.table = host.table[:1]
    got = attend(handle, host, q, [n], [n], 0.125)
    check_rows(*got, host, q, n, 0.125, some(rng, n, 8))
    assert status(handle) == 0


def test_other_stream_nothing_to_do_and_graph(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = kv4.Cache(np.random.default_rng(15), [100, 900], 2, 64, 64)
    cache, q = host.device(), torch.randn(301, 4, 64, device="cuda")
    call = lambda **more: attend(handle, host, q, [1, 300], [100, 900], 0.1, cache=cache, **more)
    want = [t.clone() for t in call()]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=stream.cuda_stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    o, n = (ops.to_device(np.array(a, np.int32)) for a in ([0, 1, 301], [100, 900]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = q4lin.attention(handle, cache, q, o, n, 0.1)
    x = q.clone()
    q.normal_()
    n.copy_(ops.to_device(np.array([77, 850], np.int32)))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, q4lin.attention(handle, cache, q, o, n, 0.1)))
    q.copy_(x)
    n.copy_(ops.to_device(np.array([100, 900], np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert attend(handle, host, q[:0], [0, 0], [100, 900], 0.1)[0].shape == (0, 4, 64)


def test_a_wait_that_runs_out_is_reported(handle):
    """Keys that do not come: the kernels give up, leave, and work again afterwards."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    host = kv4.Cache(np.random.default_rng(20), [3000], 2, 64, 128)
    cache = host.device()
    for dtype in (torch.float32, torch.bfloat16):
        for tokens in (1, 200):
            q = torch.randn(tokens, 4, 128, device="cuda").to(dtype)
            want = attend(handle, host, q, [tokens], [3000], 0.1, cache=cache)[0]
            handle.set_option(q4lin.Q4LIN_OPT_WAIT_LIMIT, 1000000)  # 1 ms
            handle.set_option(q4lin.Q4LIN_OPT_TC_SKIP_FIRST_COPY, 1)
            attend(handle, host, q, [tokens], [3000], 0.1, cache=cache)
            handle.set_option(q4lin.Q4LIN_OPT_TC_SKIP_FIRST_COPY, 0)
            handle.set_option(q4lin.Q4LIN_OPT_WAIT_LIMIT, 0)
            assert status(handle) == 1
            assert torch.equal(attend(handle, host, q, [tokens], [3000], 0.1, cache=cache)[0], want)
            assert status(handle) == 0


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_a_scale_that_is_no_number(handle, split, scale):
    """Every row becomes NaN; the next call is right."""
    import torch
    host = kv4.Cache(np.random.default_rng(21), [200], 1, 32, 64)
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn(100, 2, 64, device="cuda").to(dtype)
        for rows in BOTH:
            split(rows)
            out, lse = attend(handle, host, q, [100], [200], scale)
            assert torch.isnan(out).all() and torch.isnan(lse).all()
            assert torch.isfinite(attend(handle, host, q, [100], [200], 0.1)[0]).all()


def test_two_heads_apart_and_padded_batches(handle):
    """One query head a key head, a batch with sequences of no queries among others, rows behind the last
    sequence left as they were, and offsets that do not begin at 0."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(22)
    lengths, counts = [40, 300, 0, 129, 7], [1, 0, 0, 100, 7]
    for heads, dim, dtype in ((3, 64, "f32"), (6, 128, "bf16"), (3, 256, "f16")):
        host = kv4.Cache(rng, lengths, 3, 16, dim)
        q = ops.to_device(rng.standard_normal((120, heads, dim)).astype(np.float32), dtype)
        offsets = np.concatenate([[2], 2 + np.cumsum(counts)]).astype(np.int32)
        out, lse = torch.full_like(q, 7.0), torch.full((120, heads), 7.0, device="cuda")
        q4lin.attention(handle, host.device(), q, ops.to_device(offsets), ops.to_device(np.array(lengths, np.int32)),
                        0.125, out=out, lse=lse)
        want = ops.attention(host, ops.to_host(q), offsets, lengths, 0.125)
        rows = slice(2, offsets[-1])
        check(out[rows], lse[rows], [w[rows] for w in want], dtype)
        for edge in (slice(0, 2), slice(offsets[-1], None)):
            assert bool((out[edge] == 7).all()) and bool((lse[edge] == 7).all())
        assert status(handle) == 0


def test_a_layer(handle):
    """Norm and rotation, append, attention token by token and in one call, as a decoder runs them,
    against float64 over what the cache then holds; the whole captured into a graph."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(13)
    table = ops.to_device(np.arange(8, dtype=np.int32).reshape(2, 4))
    rope = ops.rope_tables(rng, 64, 64)
    device_rope = tuple(map(ops.to_device, rope))
    weights = [ops.to_device((1 + 0.2 * rng.standard_normal(64)).astype(np.float32)) for _ in range(2)]
    x = ops.to_device(rng.standard_normal((40, 2, 8, 64)).astype(np.float32))  # 4 queries, 2 keys, 2 values

    def step(cache, y, positions, offsets, starts, lengths):
        q, k, v = y.split([4, 2, 2], 1)
        q, k = q4lin.norm_rope(handle, q, k, *weights, positions, device_rope)
        q4lin.kv_append(handle, cache, k, v, offsets, starts)
        return q4lin.attention(handle, cache, q, offsets, lengths, 0.125, max_query=y.shape[0])[0], q

    one, whole = (q4lin.KVCache4.empty(8, 2, 16, 64, table) for _ in range(2))
    offsets = ops.to_device(np.array([0, 1, 2], np.int32))
    outs = []
    for i in range(40):
        at = torch.full((2,), i, dtype=torch.int32, device="cuda")
        outs.append(step(one, x[i], at, offsets, at, at + 1)[0])
    flat = x.transpose(0, 1).reshape(80, 8, 64).contiguous()
    args = [ops.to_device(np.array(a, np.int32)) for a in (list(range(40)) * 2, [0, 40, 80], [0, 0], [40, 40])]
    out, q = step(whole, flat, *args)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(whole, name))
    host = kv4.DeviceCache(whole)
    want = ops.attention(host, ops.to_host(q), [0, 40, 80], [40, 40], 0.125)
    check(out, torch.from_numpy(want[1]), want, "f32")
    check(torch.stack(outs, 1).flatten(0, 1), torch.from_numpy(want[1]), want, "f32")
    graph, cache = torch.cuda.CUDAGraph(), q4lin.KVCache4.empty(8, 2, 16, 64, table)
    with torch.cuda.graph(graph):
        held = step(cache, flat, *args)[0]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, out)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype,window", [("f16", 0), ("f32", 9001), ("bf16", 0)])
def test_walks_cut_where_the_last_round_is_short(handle, dtype, window):
    """More walks than SMs, by few, over so many keys that they are cut; another sequence beside them."""
    rng = np.random.default_rng(34)
    lengths, counts = [34000, 300], [5100, 200]
    host = kv4.Cache(rng, lengths, 8, 64, 64)
    q = ops.to_device(rng.standard_normal((5300, 8, 64)).astype(np.float32), dtype)
    out, lse = attend(handle, host, q, counts, lengths, 0.125, window=window)
    check_rows(out, lse, host, q, 34000, 0.125, some(rng, 5100, 8, 30), dtype, count=5100, window=window)
    check_rows(out, lse, host, q, 300, 0.125, some(rng, 200, 8, 30), dtype, b=1, first=5100, count=200, window=window)
    again = attend(handle, host, q, counts, lengths, 0.125, window=window)
    assert out.equal(again[0]) and lse.equal(again[1])
    assert status(handle) == 0


WIDE = [  # heads of 256 in the prompts' kernel: lengths, counts, heads, kv heads, page, dtype, rotated, causal, window
    ([130, 700, 64], [130, 333, 64], 6, 2, 16, "f32", 256, True, 0),
    ([401, 5, 130], [129, 5, 130], 8, 8, 64, "bf16", 0, True, 0),
    ([900, 0, 333], [64, 0, 200], 7, 1, 32, "f16", 64, True, 100),
    ([257, 1], [100, 1], 4, 4, 64, "bf16", 256, False, 0),
    ([3000], [70], 4, 1, 64, "bf16", 0, True, 0),       # walks that are cut
    ([3100], [40], 8, 2, 16, "f32", 128, True, 2500),
    ([2500], [129], 2, 1, 32, "f16", 0, True, 0),
    ([1300, 1200], [50, 1200], 2, 2, 64, "f32", 0, True, 0),  # outputs taken out on the way
]


@pytest.mark.parametrize("lengths,counts,heads,kv_heads,page,dtype,rotated,causal,window", WIDE)
def test_prompts_of_wide_heads(handle, split, lengths, counts, heads, kv_heads, page, dtype, rotated, causal, window):
    results = []
    for rows in BOTH:
        split(rows)
        results.append(run(handle, lengths, counts, heads, kv_heads, page, 256, dtype, rotated=rotated, causal=causal,
                           window=window))
        check(*results[-1])
        assert status(handle) == 0


@pytest.mark.parametrize("dtype,n,tokens", [("f16", 34000, 90), ("f32", 9000, 2600), ("bf16", 9000, 2600)])
def test_many_keys_of_wide_heads(handle, split, dtype, n, tokens):
    """Few walks in parts, and more walks than SMs; with outputs taken out."""
    split(1)
    rng = np.random.default_rng(n)
    host = kv4.Cache(rng, [n], 8, 64, 256)
    q = ops.to_device(rng.standard_normal((tokens, 8, 256)).astype(np.float32), dtype)
    out, lse = attend(handle, host, q, [tokens], [n], 0.0625)
    check_rows(out, lse, host, q, n, 0.0625, some(rng, tokens, 8, 30), dtype)
    again = attend(handle, host, q, [tokens], [n], 0.0625)
    assert out.equal(again[0]) and lse.equal(again[1])
    assert status(handle) == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rotated", [False, True])
def test_rows_that_begin_while_others_maxima_grow(handle, split, dim, rotated):
    """bf16 prompts with a window, whose rows first see a key in a step in which scores of others grow by
    2^12 and more: outputs are rescaled twice there."""
    split(1)
    rng = np.random.default_rng(61)
    n, window = 600, 150
    host = kv4.Cache(rng, [n], 2, 32, dim)
    slots = host.table[0, :-(-n // 32)]
    at = np.arange(len(slots) * 32).reshape(len(slots), 1, 32)
    host.k[..., 0], host.ks[slots] = 15, np.where(at % 128 < 40, 0.02, 2.0)
    host.ks[slots] *= (1 + at / 200).astype(np.float32)
    q = rng.standard_normal((n, 2, dim)) * 0.1
    q[..., 0] = 4
    q = ops.to_device(q.astype(np.float32), "bf16")
    angle = np.zeros((n, dim // 2), np.float32)
    rope = (ops.to_device(angle + 1), ops.to_device(angle)) if rotated else None
    want = ops.attention(host, ops.to_host(q), [0, n], [n], 0.125, window=window)
    check(*attend(handle, host, q, [n], [n], 0.125, window=window, rope=rope), want, "bf16")
    assert status(handle) == 0

"""Appending to the paged 4-bit cache, bit for bit against its definition, and reading it back."""
import numpy as np
import pytest

from tests import _kv4 as kv4
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


def ints(*values):
    return ops.to_device(np.array(values, np.int32))


def draw(rng, shape, dtype):
    x = rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal(shape[1:]))
    return ops.to_device(x.astype(np.float32), dtype)


def same(device, host):
    got = kv4.DeviceCache(device)
    for name in ("k", "ks", "v", "vs"):
        assert np.array_equal(getattr(got, name), getattr(host, name)), name


CASES = [
    # starts, counts, heads, page, dim, dtype, rotated, interleaved
    ([0], [1], 1, 16, 64, "f32", 64, False),
    ([5, 16, 31], [1, 1, 1], 8, 16, 64, "bf16", 64, False),
    ([0, 3], [70, 0], 2, 32, 128, "f32", 128, False),
    ([0, 100, 63], [130, 1, 2], 4, 64, 128, "f16", 64, True),
    ([7], [200], 5, 16, 256, "bf16", 256, True),
    ([0, 0, 0], [0, 33, 0], 3, 16, 64, "f32", 8, False),
    ([15, 1], [17, 300], 9, 32, 64, "f16", 0, False),
    ([1000], [513], 8, 64, 128, "f32", 128, False),
    ([i % 50 for i in range(100)], [i % 4 for i in range(100)], 2, 16, 128, "bf16", 24, False),
    ([0], [2100], 17, 64, 64, "f32", 0, False),
]


@pytest.mark.parametrize("starts,counts,heads,page,dim,dtype,rotated,interleaved", CASES)
def test_bytes_and_back(handle, starts, counts, heads, page, dim, dtype, rotated, interleaved):
    """What is written is the definition's, nothing else in the cache moves, and it reads back as
    what the codes stand for, rounded once."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(sum(counts) + dim)
    ends = [s + n for s, n in zip(starts, counts)]
    host = kv4.Cache(rng, ends, heads, page, dim)
    device = host.device()
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k, v = (draw(rng, (offsets[-1], heads, dim), dtype) for _ in range(2))
    rope = ops.rope_tables(rng, max(ends), rotated) if rotated else None
    q4lin.kv_append(handle, device, k, v, ops.to_device(offsets), ints(*starts),
                    rope=rope and tuple(map(ops.to_device, rope)), interleaved=interleaved)
    f32 = lambda t: t.float().cpu().numpy()
    kv4.append(host, f32(k), f32(v), offsets, starts, rope, interleaved)
    same(device, host)
    # Half a step, amax / 15, is the most that a value is off, but for roundings: scale (twice), inverse
    # and product leave x / s off by 4 x 2^-24 of at most 7.5 steps, so a value that close to a tie
    # may go the other way, 1.8e-6 steps or 2^-18 of half a step further; the value read back rounds
    # once more.
    for got, x in zip(q4lin.kv_read(handle, device, ops.to_device(offsets), ints(*starts), int(offsets[-1])),
                      (f32(k) if rope is None else None, f32(v))):
        if x is not None:
            bound = np.abs(x).max(-1, keepdims=True) / 15 * (1 + 2.0**-17)
            assert (np.abs(got.cpu().numpy() - x) / bound).max() <= 1
    for to in ("f32", "f16", "bf16"):
        kind = ops.torch_dtype(to)
        got = q4lin.kv_read(handle, device, ops.to_device(offsets), ints(*starts), int(offsets[-1]), dtype=kind)
        for t, codes, scales in zip(got, (host.k, host.v), (host.ks, host.vs)):
            want = np.zeros(t.shape, np.float32)
            for b, n in enumerate(counts):
                at = np.arange(starts[b], starts[b] + n)
                p, s = host.table[b, at // page], at % page
                want[offsets[b]:offsets[b + 1]] = (codes[p, :, s].astype(np.float32) - 8) * scales[p, :, s][..., None]
            assert torch.equal(t, torch.from_numpy(want).to(kind).cuda())
    assert status(handle) == 0


def test_token_by_token_is_all_at_once(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(1)
    table = ints(2, 0, 1).view(1, 3)
    one, all_of_them = (q4lin.KVCache4.empty(3, 2, 16, 64, table) for _ in range(2))
    k, v = (draw(rng, (40, 2, 64), "f32") for _ in range(2))
    q4lin.kv_append(handle, all_of_them, k, v, ints(0, 40), ints(0))
    for i in range(40):
        q4lin.kv_append(handle, one, k[i:i + 1], v[i:i + 1], ints(0, 1), ints(i))
    for a in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, a), getattr(all_of_them, a))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_slices_of_one_projection(handle, dtype, shift):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(2)
    wide = ops.to_device(rng.standard_normal((20, 5 * 64 + 3)).astype(np.float32), dtype)
    k, v = (wide[:, shift + a:shift + a + 128].unflatten(1, (2, 64)) for a in (0, 190))
    table = ints(0, 1).view(1, 2)
    caches = [q4lin.KVCache4.empty(2, 2, 16, 64, table) for _ in range(2)]
    q4lin.kv_append(handle, caches[0], k, v, ints(0, 20), ints(0))
    q4lin.kv_append(handle, caches[1], k.contiguous(), v.contiguous(), ints(0, 20), ints(0))
    for a in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(*(getattr(c, a) for c in caches))


def test_zeros_infinities_nan_and_tiny(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    inf, nan = float("inf"), float("nan")
    x = torch.randn(6, 1, 64, device="cuda")
    x[0] = 0
    x[1, 0, :3] = torch.tensor([inf, -inf, nan])
    x[2] = inf
    x[3] *= 1e-39
    x[4] *= 1e38
    host = kv4.Cache(np.random.default_rng(3), [6], 1, 16, 64)
    device = host.device()
    q4lin.kv_append(handle, device, x[:1], x[:1], ints(0, 1), ints(0))
    assert status(handle) == 0
    q4lin.kv_append(handle, device, x[1:], x[1:], ints(0, 5), ints(1))
    assert status(handle) == 3
    kv4.append(host, x.cpu().numpy(), x.cpu().numpy(), [0, 6], [0])
    same(device, host)
    p = host.table[0, 0]
    assert host.k[p, 0, 1, :3].tolist() == [15, 0, 8] and (host.k[p, 0, [0, 2, 3]] == 8).all()


def test_indices_out_of_range_touch_nothing(handle):
    """Bad pages, positions and offsets: what they would have touched stays, the rest is done."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(4)
    k, v = (draw(rng, (6, 2, 64), "f32") for _ in range(2))
    for table, offsets, starts, positions in (
            ([[0, 1], [3, 2]], [0, 3, 6], [0, 0], 99), ([[0, 1], [-1, 2]], [0, 3, 6], [0, 0], 99),
            ([[0, 1], [2, -2**31]], [0, 3, 6], [0, 15], 99), ([[0, 1], [2, 2]], [0, 3, 6], [0, 40], 99),
            ([[0, 1], [2, 2]], [0, 3, 6], [0, -1], 99), ([[0, 1], [2, 2]], [0, 3, 9], [0, 0], 99),
            ([[0, 1], [2, 2]], [0, 3, 2], [0, 0], 99), ([[0, 1], [2, 2]], [-1, 3, 6], [0, 0], 99),
            ([[0, 1], [2, 2]], [0, 3, 6], [0, 0], 2), ([[0, 1], [2, 2]], [0, 3, 6], [0, 2**31 - 1], 99)):
        host = kv4.Cache(rng, [16, 16], 2, 16, 64, spare=1)
        host.table = np.array(table, np.int32)
        device = host.device()
        rope = tuple(map(ops.to_device, ops.rope_tables(rng, positions, 64)))
        before = kv4.DeviceCache(device)
        q4lin.kv_append(handle, device, k, v, ints(*offsets), ints(*starts), rope=rope)
        assert status(handle) == 4
        after = kv4.DeviceCache(device)
        # Only the pages of good tokens: the first sequence's page 0, and the second's first page.
        for name in ("k", "v", "ks", "vs"):
            a, b = getattr(after, name), getattr(before, name)
            assert np.array_equal(a[1], b[1])
            assert np.array_equal(a[0][:, 3:], b[0][:, 3:])
        out = [torch.full((6, 2, 64), 7.0, device="cuda") for _ in range(2)]
        if positions > 2:
            q4lin.kv_read(handle, device, ints(*offsets), ints(*starts), 6, k=out[0], v=out[1])
            assert status(handle) == 4
            if offsets[0] == 0:
                assert not (out[0][:3] == 7.0).any()
            if starts[1] != 15 and offsets[0] == 0:  # (the second sequence is bad in its first page)
                assert (out[0][3:] == 7.0).all() and (out[1][3:] == 7.0).all()


def test_rows_of_no_sequence_stay(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    device = kv4.Cache(np.random.default_rng(5), [40], 2, 16, 64).device()
    out = [torch.full((10, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    q4lin.kv_read(handle, device, ints(2, 7), ints(30), 10, k=out[0], v=out[1])
    for t in out:
        assert (t[:2] == 7).all() and (t[7:] == 7).all() and not (t[2:7] == 7).all()
    assert status(handle) == 0


def test_other_stream_nothing_to_do_and_graph(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(6)
    host = kv4.Cache(rng, [200, 90], 4, 32, 128)
    k, v = (draw(rng, (30, 4, 128), "bf16") for _ in range(2))
    o, s = ints(0, 20, 30), ints(180, 80)
    a, b = host.device(), host.device()
    q4lin.kv_append(handle, a, k, v, o, s)
    want = [t.clone() for t in q4lin.kv_read(handle, a, o, s, 30)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q4lin.kv_append(handle, b, k, v, o, s, stream=stream.cuda_stream)
    got = q4lin.kv_read(handle, b, o, s, 30, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(a.k_codes, b.k_codes) and all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4lin.kv_append(handle, a, k, v, o, s)
        held = q4lin.kv_read(handle, a, o, s, 30)
    k.neg_(), v.mul_(2)
    graph.replay()
    q4lin.kv_append(handle, b, k, v, o, s)
    assert all(torch.equal(x, y) for x, y in zip(held, q4lin.kv_read(handle, b, o, s, 30)))
    q4lin.kv_append(handle, a, k[:0], v[:0], ints(0, 0, 0), s)
    assert q4lin.kv_read(handle, a, ints(0, 0, 0), s, 0)[0].shape == (0, 4, 128)
    assert status(handle) == 0

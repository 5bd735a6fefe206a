"""Queries and keys normalised per head and rotated, and the gradient of that, against float64.

Tolerances.  The sum of squares of up to 256 channels goes through 8 additions in a lane and 5 between
lanes, each off by 2^-24 of it, so r is off by 7 x 2^-24 of itself, the two products and the
rotation's three operations by as much as 2^-24 each: under 2^-20 of the terms' sizes, then the
rounding to the type.  The gradient adds the same kind of sum for the mean and three more operations:
2^-19 of the sizes of its terms.  The weights' gradients add up rows in chains of at most 400
additions for the sizes here (a warp's, a CTA's, the CTAs'): 400 x 2^-24 of the terms' sizes."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


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


def inputs(tokens, heads, kv_heads, dim, dtype, rotated, gain=1.0, seed=0):
    """Slices of one array, weights, positions, tables; the slices as float64 too."""
    rng = np.random.default_rng(seed + tokens + heads + dim)
    x = rng.standard_normal((tokens, heads + 2 * kv_heads, dim)) * gain
    x = ops.to_device(x.astype(np.float32), dtype)
    q, k = x[:, :heads], x[:, heads:heads + kv_heads]
    weights = [(1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2)]
    positions = rng.integers(0, 300, tokens).astype(np.int32)
    rope = ops.rope_tables(rng, 300, rotated) if rotated else None
    return rng, q, k, weights, positions, rope


def near(got, want, bound):
    err = np.abs(ops.to_host(got) - want)
    assert np.all(err <= bound), f"{np.max(err / bound):.3g} times the tolerance"


CASES = [
    # tokens, heads, kv heads, dim, dtype, rotated, interleaved
    (1, 32, 8, 64, "f32", 64, False),
    (1, 1, 1, 128, "bf16", 128, True),
    (3, 5, 2, 64, "f16", 32, False),
    (7, 28, 4, 128, "f32", 128, False),
    (33, 7, 1, 256, "bf16", 64, True),
    (65, 3, 3, 256, "f32", 256, False),
    (129, 9, 5, 64, "bf16", 8, False),
    (200, 14, 2, 128, "f16", 24, True),
    (500, 32, 8, 128, "bf16", 128, False),
    (40, 6, 2, 128, "f32", 0, False),
    (17, 4, 0, 64, "f32", 64, False),
    (17, 0, 3, 128, "f32", 40, False),
]


@pytest.mark.parametrize("tokens,heads,kv_heads,dim,dtype,rotated,interleaved", CASES)
def test_forward(handle, tokens, heads, kv_heads, dim, dtype, rotated, interleaved):
    from bit_weight_quantized_int4_gb300 import q4lin
    _, q, k, weights, positions, rope = inputs(tokens, heads, kv_heads, dim, dtype, rotated)
    out = q4lin.norm_rope(handle, q, k, *map(ops.to_device, weights), ops.to_device(positions),
                          rope and tuple(map(ops.to_device, rope)), eps=EPS, interleaved=interleaved)
    for x, w, got in zip((q, k), weights, out):
        want, size = kv4.norm_rope(ops.to_host(x), w.astype(np.float64), positions, rope, EPS, interleaved)
        assert got.dtype == x.dtype and got.shape == x.shape
        near(got, want, 2.0**-20 * size + ops.ROUND[dtype] * np.abs(want) + ops.TINY[dtype])
    assert status(handle) == 0


@pytest.mark.parametrize("tokens,heads,kv_heads,dim,dtype,rotated,interleaved", CASES)
def test_backward(handle, tokens, heads, kv_heads, dim, dtype, rotated, interleaved):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(tokens, heads, kv_heads, dim, dtype, rotated)
    d = [ops.to_device(rng.standard_normal(x.shape).astype(np.float32), dtype) for x in (q, k)]
    call = lambda: q4lin.norm_rope_backward(handle, q, k, *map(ops.to_device, weights), ops.to_device(positions),
                                            rope and tuple(map(ops.to_device, rope)), *d, eps=EPS,
                                            interleaved=interleaved)
    got = call()
    for x, w, dy, dx, dw in zip((q, k), weights, d, got[:2], got[2:]):
        want, want_w, size, size_w = kv4.norm_rope_backward(ops.to_host(x), w.astype(np.float64), positions, rope,
                                                            EPS, interleaved, ops.to_host(dy))
        near(dx, want, 2.0**-19 * size + ops.ROUND[dtype] * np.abs(want) + ops.TINY[dtype])
        near(dw, want_w, 400 * 2.0**-24 * size_w + 1e-37)
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert status(handle) == 0


def test_gradient_against_differences(handle):
    """The sum of squares of the outputs, differenced in float64 along random directions of q, k and
    the weights; the kernel's gradients are within 2^-19 of their terms (under 3 per element here)."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(5, 3, 2, 64, "f32", 32)
    args = [ops.to_host(q), ops.to_host(k), *(w.astype(np.float64) for w in weights)]
    aim = [rng.standard_normal(x.shape) for x in args[:2]]
    forward = lambda a: [kv4.norm_rope(x, w, positions, rope, EPS, True)[0] for x, w in zip(a[:2], a[2:])]
    loss = lambda a: sum(((y - t)**2).sum() / 2 for y, t in zip(forward(a), aim))
    d = [ops.to_device((y - t).astype(np.float32)) for y, t in zip(forward(args), aim)]
    got = q4lin.norm_rope_backward(handle, q, k, *map(ops.to_device, weights), ops.to_device(positions),
                                   tuple(map(ops.to_device, rope)), *d, eps=EPS, interleaved=True)
    for i in range(4):
        way = [rng.standard_normal(a.shape) if j == i else np.zeros(a.shape) for j, a in enumerate(args)]
        step = 1e-5
        ends = [loss([a + s * step * w for a, w in zip(args, way)]) for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        terms = ops.to_host(got[i]) * way[i]
        assert abs(terms.sum() - slope) <= 1e-5 * np.abs(terms).sum()


@pytest.mark.parametrize("dim", [64, 256])
def test_sizes_of_numbers(handle, dim):
    """Rows of zeros, rows near the largest number, tiny ones, and a NaN that stays in its row."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 2, dim))
    x[0] = 0
    x[1] *= 1e37
    x[2] *= 1e-30
    x[3] *= 1e19
    q = ops.to_device(x.astype(np.float32))
    q[4, 1, 5] = float("nan")
    k, d = q[:, :1].contiguous(), torch.ones_like(q)
    out, _ = q4lin.norm_rope(handle, q, k, eps=EPS)
    got = q4lin.norm_rope_backward(handle, q, k, None, None, None, None, d, d[:, :1], eps=EPS)
    assert got.d_q_weight is None and got.d_k_weight is None
    fine = [0, 1, 2, 3, 5]
    x = ops.to_host(q)[fine]
    want, size = kv4.norm_rope(x, np.ones(dim), None, None, EPS, False)
    near(out[fine], want, 2.0**-20 * size + 1e-37)
    want, _, size, _ = kv4.norm_rope_backward(x, np.ones(dim), None, None, EPS, False, np.ones(x.shape))
    near(got.d_q[fine], want, 2.0**-19 * size + 2e-37)
    assert torch.isnan(out[4, 1]).all() and torch.isfinite(out[4, 0]).all()
    assert torch.isnan(got.d_q[4, 1]).all() and torch.isfinite(got.d_q[4, 0]).all()
    # Without eps, rows as large as the type holds and as small as fp32 does: like any other.
    x = rng.standard_normal((5, 2, dim)) * np.array([3e37, 1e-18, 1e-25, 1e-38, 1])[:, None, None]
    q = ops.to_device(x.astype(np.float32))
    out, _ = q4lin.norm_rope(handle, q, q[:, :1], eps=0.0)
    x = ops.to_host(q)
    want, size = kv4.norm_rope(x, np.ones(dim), None, None, 0.0, False)
    near(out, want, 2.0**-20 * size)
    d = torch.ones_like(q) * torch.tensor([1e10, 1e-10, 1e-10, 1e-10, 1], device="cuda")[:, None, None]
    got = q4lin.norm_rope_backward(handle, q, q[:, :1], None, None, None, None, d, d[:, :1], eps=0.0)
    want, _, size, _ = kv4.norm_rope_backward(x, np.ones(dim), None, None, 0.0, False, ops.to_host(d))
    near(got.d_q, want, 2.0**-19 * size + 1e-37)
    # An infinity: its row alone.
    q[4, 0, 3] = float("inf")
    out, _ = q4lin.norm_rope(handle, q, q[:, :1], eps=EPS)
    assert torch.isnan(out[4, 0, 3]) and torch.isfinite(out[4, 1]).all() and torch.isfinite(out[:4]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_strides_and_in_place(handle, dtype, shift):
    """Slices that begin anywhere, outputs in heads-first order, and outputs in the inputs' place."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(37, 6, 2, 64, dtype, 64)
    wide = torch.zeros(37, 9 * 64 + 8, device="cuda", dtype=q.dtype)
    wide[:, shift:shift + 384], wide[:, shift + 384:shift + 512] = q.flatten(1), k.flatten(1)
    q2, k2 = (wide[:, shift + a:shift + b].unflatten(1, (-1, 64)) for a, b in ((0, 384), (384, 512)))
    more = [*map(ops.to_device, weights), ops.to_device(positions), tuple(map(ops.to_device, rope))]
    want = q4lin.norm_rope(handle, q, k, *more)
    first = torch.zeros(6, 40, 64, device="cuda", dtype=q.dtype)
    got = q4lin.norm_rope(handle, q2, k2, *more, q_out=first.transpose(0, 1)[2:39])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not first[:, :2].any() and not first[:, 39:].any()
    d = [ops.to_device(rng.standard_normal(x.shape).astype(np.float32), dtype) for x in (q, k)]
    grads = q4lin.norm_rope_backward(handle, q2, k2, *more, *d)
    kept = wide.clone()
    inside = q4lin.norm_rope_backward(handle, q2, k2, *more, *d, d_q=q2, d_k=d[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, inside))
    wide.copy_(kept)
    d[1] = grads.d_k.clone()
    q4lin.norm_rope(handle, q2, k2, *more, q_out=q2, k_out=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert not wide[:, :shift].any() and torch.equal(wide[:, shift + 512:], kept[:, shift + 512:])
    # One gradient for all tokens (heads): strides of 0.
    one = torch.randn(1, 6, 64, device="cuda").to(q.dtype)
    same = one.expand(37, 6, 64)
    a = q4lin.norm_rope_backward(handle, q, k, *more, same, d[1])
    b = q4lin.norm_rope_backward(handle, q, k, *more, same.contiguous(), d[1])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    one = torch.randn(37, 1, 64, device="cuda").to(q.dtype)
    a = q4lin.norm_rope_backward(handle, q, k, *more, one.expand(37, 6, 64), d[1])
    b = q4lin.norm_rope_backward(handle, q, k, *more, one.expand(37, 6, 64).contiguous(), d[1])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_positions_out_of_range_are_reported(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(20, 4, 2, 64, "f32", 64)
    more = [*map(ops.to_device, weights)], tuple(map(ops.to_device, rope))
    d = [torch.randn_like(x) for x in (q.contiguous(), k.contiguous())]
    keep = np.ones(20, bool)
    want = q4lin.norm_rope(handle, q, k, *more[0], ops.to_device(positions), more[1])
    for at, bad in ((3, 300), (0, -1), (19, 2**31 - 1), (7, -2**31)):
        p = positions.copy()
        p[at] = bad
        keep[:] = True
        keep[at] = False
        outs = [torch.full_like(x, 7.0) for x in d]
        q4lin.norm_rope(handle, q, k, *more[0], ops.to_device(p), more[1], q_out=outs[0], k_out=outs[1])
        assert status(handle) == 4
        for got, w in zip(outs, want):
            assert torch.equal(got[keep], w[keep]) and bool((got[at] == 7.0).all())
        outs = [torch.full_like(x, 7.0) for x in d]
        got = q4lin.norm_rope_backward(handle, q, k, *more[0], ops.to_device(p), more[1], *d, d_q=outs[0], d_k=outs[1])
        assert status(handle) == 4
        rest = q4lin.norm_rope_backward(handle, q[keep], k[keep], *more[0], ops.to_device(positions[keep]), more[1],
                                        d[0][keep], d[1][keep])
        for g, r in zip(outs, rest[:2]):
            assert torch.equal(g[keep], r) and bool((g[at] == 7.0).all())
        for g, r, x in zip(got[2:], rest[2:], d):
            # The same rows in another order of warps: 400 x 2^-24 of terms of size up to 30 each.
            assert float((g - r).abs().max()) <= 400 * 2.0**-24 * 30 * x.shape[1] * 20


def test_no_tokens(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    q, w = torch.zeros(0, 4, 64, device="cuda"), torch.ones(64, device="cuda")
    out, _ = q4lin.norm_rope(handle, q, q, w, w)
    assert out.shape == (0, 4, 64)
    got = q4lin.norm_rope_backward(handle, q, q, w, w, None, None, q, q)
    assert not got.d_q_weight.any() and not got.d_k_weight.any() and got.d_q_weight.shape == (64,)


def test_other_stream_and_graph(handle):
    """On another stream, and captured and replayed on new inputs."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(300, 8, 2, 128, "bf16", 128)
    q, k = q.contiguous(), k.contiguous()
    more = [*map(ops.to_device, weights), ops.to_device(positions), tuple(map(ops.to_device, rope))]
    d = torch.randn_like(q), torch.randn_like(k)
    both = lambda stream=None: [*q4lin.norm_rope(handle, q, k, *more, stream=stream),
                                *q4lin.norm_rope_backward(handle, q, k, *more, *d, stream=stream)]
    want = [t.clone() for t in both()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = both(stream.cuda_stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    x = q.clone()
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], -want[0]) and torch.equal(held[3], want[3])
    q.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("tokens,heads,kv_heads,dim,dtype,rotated,shift", [
    (5003, 6, 2, 64, "bf16", 64, 0),     # rows of a pass that are not all heads
    (2500, 7, 5, 128, "f32", 32, 0),     # an odd last pass of every token
    (2600, 3, 1, 256, "f16", 256, 0),    # a pass a head
    (5003, 6, 2, 64, "bf16", 64, 1),     # rows that no copy takes
    (2500, 7, 5, 128, "f32", 0, 1),
])
def test_gradient_of_many_tokens(handle, tokens, heads, kv_heads, dim, dtype, rotated, shift):
    """Shares of a warp that begin and end inside a token, some positions out of range among them."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng, q, k, weights, positions, rope = inputs(tokens, heads, kv_heads, dim, dtype, rotated)
    if shift:
        wide = torch.zeros(tokens, heads + kv_heads, dim + shift, dtype=q.dtype, device="cuda")
        wide[..., shift:] = torch.cat([q, k], 1)
        q, k = wide[:, :heads, shift:], wide[:, heads:, shift:]
    d = [ops.to_device(rng.standard_normal(x.shape).astype(np.float32), dtype) for x in (q, k)]
    kept = np.ones(tokens, bool)
    if rope:
        kept[[0, 7, tokens // 2, tokens - 1]] = False
    at = np.where(kept, positions, 300).astype(np.int32)
    outs = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (q, k)]
    got = q4lin.norm_rope_backward(handle, q, k, *map(ops.to_device, weights), ops.to_device(at),
                                   rope and tuple(map(ops.to_device, rope)), *d, eps=EPS, d_q=outs[0], d_k=outs[1])
    for x, w, dy, dx, dw in zip((q, k), weights, d, got[:2], got[2:]):
        x, dy, dx = ops.to_host(x), ops.to_host(dy), ops.to_host(dx)
        assert np.all(dx[~kept] == 7)  # nothing is written for a position that is not in the table
        want, want_w, size, size_w = kv4.norm_rope_backward(x[kept], w.astype(np.float64), positions[kept], rope, EPS,
                                                            False, dy[kept])
        near(torch.from_numpy(dx[kept]), want, 2.0**-19 * size + ops.ROUND[dtype] * np.abs(want) + ops.TINY[dtype])
        near(dw, want_w, 400 * 2.0**-24 * size_w)
    assert (status(handle) != 0) == (rope is not None)

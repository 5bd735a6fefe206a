"""Log probabilities, entropy and top entries of rows of logits, and their gradient, against
float64.

Tolerances.  lse and a log probability: differences x - m are rounded once (2^-24 of |x| +
|m|), each exponential is off by 2^-21 relatively, and sums of 128 k terms, partial by
thread, by 2^-19: 2^-18 + 2^-22 (|x| + |lse|).  The entropy weighs differences of up to W =
max(m - x where p counts) with those: (2^-18) (1 + H) + 2^-22 |m|.  A gradient: p to 2^-20 +
2^-22 (|x| + |lse|), times |d_lp| + |d_H| (|ln p| + H), then the rounding to its type."""
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


def draw(rng, rows, size, dtype, peak=9.0):
    x = rng.standard_normal((rows, size)) * 2
    x[np.arange(rows)[:, None], rng.integers(0, size, (rows, 4))] += peak
    return ops.to_device(x.astype(np.float32), dtype)


def check(r, x, tokens, top):
    lp, entropy, lse, ids, best = ops.logprobs(x, tokens, top)
    with np.errstate(all="ignore"):
        size = np.where(np.isfinite(lse), np.abs(lse), 0) + np.abs(np.where(np.isfinite(x), x, 0)).max(1)
    tol = 2.0**-18 + 2.0**-22 * size
    for got, want, bound, what in ((r.lse, lse, tol, "lse"), (r.logprob, lp, tol, "logprob"),
                                   (r.entropy, entropy, tol * (1 + entropy), "entropy")):
        got = ops.to_host(got)
        finite = np.isfinite(want)
        assert np.array_equal(got[~finite], want[~finite]), what
        err = np.abs(got[finite] - want[finite])
        assert np.all(err <= bound[finite]), f"{what}: {np.max(err / bound[finite]):.3g} times the tolerance"
    if top:
        assert np.array_equal(r.top_tokens.cpu().numpy(), ids)
        got = ops.to_host(r.top_logprobs)
        finite = np.isfinite(best)
        assert np.array_equal(got[~finite], best[~finite])
        assert np.all(np.abs(got[finite] - best[finite]) <= np.broadcast_to(tol[:, None], best.shape)[finite])


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 5, 3), (1, 31, 31), (2, 33, 32), (7, 100, 5), (2, 1000, 20), (5, 1003, 32),
          (400, 777, 5), (1, 4097, 1), (3, 5000, 0), (1, 128256, 5), (2, 128257, 32), (310, 2049, 20),
          (40, 70001, 20)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size,top", SHAPES)
def test_rows(handle, rows, size, top, dtype):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(rows * 7 + size)
    x = draw(rng, rows, size, dtype)
    tokens = rng.integers(-1, size, rows).astype(np.int32)
    r = q4lin.logprobs(handle, x, ops.to_device(tokens), top=top)
    check(r, ops.to_host(x), tokens, top)
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift,extra", [(0, 0), (1, 0), (0, 3), (3, 5)])
def test_strides(handle, dtype, shift, extra):
    """Rows that start at any element, with a stride of their own."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(21)
    x = draw(rng, 6, 3001 + shift + extra, dtype)[:, shift:shift + 3001]
    tokens = rng.integers(0, 3001, 6).astype(np.int32)
    check(q4lin.logprobs(handle, x, ops.to_device(tokens), top=7), ops.to_host(x), tokens, 7)
    one = x[:1].expand(5, -1)  # stride 0: the same row five times
    check(q4lin.logprobs(handle, one, ops.to_device(tokens[:5]), top=7), ops.to_host(one), tokens[:5], 7)


LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("fill", [-np.inf, LOWEST, -1e4])
@pytest.mark.parametrize("rows,size,allowed", [(1, 128256, 3), (2, 128256, 0), (300, 3000, 1), (2, 5000, 40)])
def test_masked_vocabulary(handle, fill, rows, size, allowed):
    """A few words allowed (or none): the rest of the top entries are the first masked ones."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(22)
    x = np.full((rows, size), fill, np.float32)
    for r in range(rows):
        x[r, rng.choice(size, allowed, replace=False)] = rng.standard_normal(allowed)
    tokens = np.array([int(np.argmax(x[r])) if r % 2 == 0 else 17 for r in range(rows)], np.int32)
    r = q4lin.logprobs(handle, ops.to_device(x), ops.to_device(tokens), top=8)
    x64 = x.astype(np.float64)
    if fill == LOWEST and allowed:
        # exp of the difference is 0 in any precision; the log probability itself is the number.
        lp, entropy, lse, ids, best = ops.logprobs(x64, tokens, 8)
        assert np.array_equal(r.top_tokens.cpu().numpy(), ids)
        assert np.allclose(ops.to_host(r.lse), lse, rtol=1e-6, atol=1e-5)
        assert np.allclose(ops.to_host(r.logprob), lp, rtol=1e-6, atol=1e-5)
        assert np.allclose(ops.to_host(r.entropy), entropy, rtol=1e-5, atol=1e-5)
    elif fill == LOWEST:
        lp, entropy, lse, ids, best = ops.logprobs(np.zeros_like(x64), tokens, 8)
        assert np.array_equal(r.top_tokens.cpu().numpy(), ids)
        assert np.allclose(ops.to_host(r.entropy), entropy, rtol=1e-5)
        assert np.allclose(ops.to_host(r.logprob), lp, rtol=1e-5)
    else:
        check(r, x64, tokens, 8)


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "few values", "zeros of both signs"])
@pytest.mark.parametrize("rows,size", [(1, 50000), (400, 6000)])
def test_order_of_equal_and_sorted_entries(handle, kind, rows, size):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(23)
    x = {"equal": np.full(size, 1.5), "rising": np.linspace(-4, 4, size), "falling": np.linspace(4, -4, size),
         "few values": rng.integers(0, 3, size).astype(np.float64),
         "zeros of both signs": np.where(rng.random(size) < 0.5, -0.0, 0.0)}[kind]
    x = np.repeat(x.astype(np.float32)[None], rows, 0)
    tokens = np.zeros(rows, np.int32)
    r = q4lin.logprobs(handle, ops.to_device(x), ops.to_device(tokens), top=32)
    check(r, x.astype(np.float64), tokens, 32)


@pytest.mark.parametrize("rows", [1, 310])
def test_infinity_and_nan(handle, rows):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(rows, 3000, device="cuda")
    x[0, 2500] = float("nan")
    x[-1, 100] = float("inf") if rows > 1 else x[-1, 100]
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    r = q4lin.logprobs(handle, x, tokens, top=3)
    assert torch.isnan(r.lse[0]) and torch.isnan(r.entropy[0]) and torch.isnan(r.logprob[0])
    assert r.top_tokens[0, 0] == 2500
    rest = torch.argsort(torch.nan_to_num(x[0], nan=-100.0), descending=True)[:2]
    assert torch.equal(r.top_tokens[0, 1:].long(), rest)
    if rows > 1:
        assert r.top_tokens[-1, 0] == 100 and torch.isinf(r.lse[-1]) and torch.isnan(r.entropy[-1])
        assert not torch.isnan(r.lse[1:-1]).any()


def test_tokens_out_of_range_are_reported(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(3, 100, device="cuda")
    bad = torch.tensor([5, 100, -2], dtype=torch.int32, device="cuda")
    r = q4lin.logprobs(handle, x, bad)
    assert status(handle) == 4 and r.logprob[1] == 0 and r.logprob[2] == 0
    d = torch.ones(3, device="cuda")
    g = q4lin.logprobs_backward(handle, x, bad, r.lse, r.entropy, d)
    assert status(handle) == 4 and not g[1:].any() and g[0].any()


def gradient_bound(x, lse, entropy, d_lp, d_h, ref, dtype):
    with np.errstate(all="ignore"):
        lp = np.where(np.isfinite(x), x - lse[:, None], 0)
        p = np.where(np.isfinite(x), np.exp(lp), 0)
        rel = 2.0**-20 + 2.0**-22 * (np.abs(np.where(np.isfinite(x), x, 0)) + np.abs(lse)[:, None])
        size = np.abs(d_lp)[:, None] + np.abs(d_h)[:, None] * (np.abs(lp) + np.abs(entropy)[:, None])
    return p * rel * 2 * size + 2.0**-23 * np.abs(ref) + ops.ROUND[dtype] * np.abs(ref) + ops.TINY[dtype]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(1, 1), (2, 7), (3, 1003), (1, 128257), (310, 2050), (2, 128256)])
def test_gradient(handle, rows, size, dtype):
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(rows + size)
    x = draw(rng, rows, size, dtype)
    tokens = rng.integers(-1, size, rows).astype(np.int32)
    r = q4lin.logprobs(handle, x, ops.to_device(tokens))
    d_lp, d_h = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))
    for use_lp, use_h in ((1, 1), (1, 0), (0, 1)):
        got = q4lin.logprobs_backward(handle, x, ops.to_device(tokens) if use_lp else None, r.lse,
                                      r.entropy if use_h else None,
                                      ops.to_device(d_lp) if use_lp else None,
                                      ops.to_device(d_h) if use_h else None)
        x64, lse, entropy = (ops.to_host(t) for t in (x, r.lse, r.entropy))
        a, b = d_lp.astype(np.float64) * use_lp, d_h.astype(np.float64) * use_h
        ref = ops.logprobs_backward(x64, tokens, lse, entropy, a, b)
        bound = gradient_bound(x64, lse, entropy, a, b, ref, dtype)
        err = np.abs(ops.to_host(got) - ref)
        assert np.all(err <= bound), f"{np.max(err / bound):.3g} times the tolerance"


def test_gradient_against_differences(handle):
    """d(sum w logprob + u entropy) along a direction, by central differences in float64."""
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(31)
    x = rng.standard_normal((4, 50)).astype(np.float32)
    tokens = np.array([3, -1, 49, 0], np.int32)
    w, u = (rng.standard_normal(4).astype(np.float32) for _ in range(2))
    dx = ops.to_device(x)
    r = q4lin.logprobs(handle, dx, ops.to_device(tokens))
    g = ops.to_host(q4lin.logprobs_backward(handle, dx, ops.to_device(tokens), r.lse, r.entropy,
                                            ops.to_device(w), ops.to_device(u)))

    def f(y):
        lp, entropy = ops.logprobs(y, tokens, 0)[:2]
        return float(w @ lp + u @ entropy)

    for _ in range(5):
        v = rng.standard_normal(x.shape)
        h = 1e-5
        slope = (f(x + h * v) - f(x - h * v)) / (2 * h)
        # Differences: h^2 times third derivatives (below 1e-8 here), rounding 1e-16 / h; the
        # gradient: 200 entries of up to 3, each to 2^-20.
        assert abs(slope - float((g * v).sum())) < 200 * 3 * 2.0**-20 + 1e-8


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_strides_and_in_place(handle, dtype):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(32)
    x = draw(rng, 5, 2000, dtype)
    tokens = ops.to_device(rng.integers(0, 2000, 5).astype(np.int32))
    d = torch.randn(5, device="cuda")
    for shift in (0, 1, 8):
        y = x[:, shift:shift + 1900]
        r = q4lin.logprobs(handle, y, tokens.clamp(max=1899))
        want = q4lin.logprobs_backward(handle, y.contiguous(), tokens.clamp(max=1899), r.lse, r.entropy, d, d)
        wide = torch.full((5, 1917), 9.0, dtype=x.dtype, device="cuda")
        got = q4lin.logprobs_backward(handle, y, tokens.clamp(max=1899), r.lse, r.entropy, d, d,
                                      out=wide[:, 3:1903])
        assert torch.equal(got, want)
        assert (wide[:, :3] == 9).all() and (wide[:, 1903:] == 9).all()
        z = x.clone()[:, shift:shift + 1900]
        assert torch.equal(q4lin.logprobs_backward(handle, z, tokens.clamp(max=1899), r.lse, r.entropy, d, d,
                                                   out=z), want)


def test_gradient_of_masked_rows(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(3, 1000, device="cuda")
    x[0, 10:] = float("-inf")
    x[1] = float("-inf")
    x[2, 10:] = LOWEST
    tokens = torch.tensor([2, 5, 3], dtype=torch.int32, device="cuda")
    r = q4lin.logprobs(handle, x, tokens)
    d = torch.ones(3, device="cuda")
    g = q4lin.logprobs_backward(handle, x, tokens, r.lse, r.entropy, d, d)
    assert torch.isfinite(g).all()
    assert not g[1].any() and not g[0, 10:].any() and not g[2, 10:].any()
    ref = ops.logprobs_backward(ops.to_host(x), tokens.cpu().numpy(), ops.to_host(r.lse),
                                ops.to_host(r.entropy), np.ones(3), np.ones(3))
    assert np.max(np.abs(ops.to_host(g) - ref)[[0, 2], :10]) < 1e-5


def test_head_loss_and_its_gradient_through_the_4_bit_head(handle):
    """logits by the 4-bit head, the loss's gradient back through it: the operators of a
    training step that reach the hidden state."""
    import torch
    import oracle
    from bit_weight_quantized_int4_gb300 import q4lin, synth
    c = synth.make_case(3, 1000, 256, 32, seed=41)
    x, w, s = (ops.to_device(a) for a in (c.x, c.qweight, c.scales))
    tokens = torch.tensor([1, 999, 500], dtype=torch.int32, device="cuda")
    logits = q4lin.linear(handle, x, w, s, None, 32)
    r = q4lin.logprobs(handle, logits, tokens)
    d = torch.full((3,), -1.0 / 3, device="cuda")
    d_logits = q4lin.logprobs_backward(handle, logits, tokens, r.lse, None, d, out=logits)
    d_x = torch.empty_like(x)
    st = q4lin.q4lin_run_backward_dx(handle.ptr, d_logits.data_ptr(), w.data_ptr(), s.data_ptr(),
                                     d_x.data_ptr(), 3, 1000, 256, 32, q4lin.Q4LIN_SCALE_F32,
                                     torch.cuda.current_stream().cuda_stream)
    assert st == q4lin.Q4LIN_OK
    ref, _ = oracle.linear(c.x, c.qweight, c.scales, None, c.K, 32)
    lse = np.log(np.exp(ref - ref.max(1, keepdims=True)).sum(1)) + ref.max(1)
    g = ops.logprobs_backward(ref, tokens.cpu().numpy(), lse, np.zeros(3), np.full(3, -1.0 / 3), np.zeros(3))
    want, mag = oracle.backward_dx(g.astype(np.float32), c.qweight, c.scales, 256, 32)
    # The fp32 logits are off by 1e-5 of their sums of products (about 2e-4 here), and so are
    # the probabilities, relatively.
    assert np.all(np.abs(ops.to_host(d_x) - want) <= 1e-3 * mag + 1e-7)


def test_refusals(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(4, 100, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    for change in (dict(logits=x.double()), dict(logits=x.t()), dict(tokens=t[:3]), dict(tokens=t.long()),
                   dict(logits=x.cpu()), dict(logits=x[0])):
        with pytest.raises(ValueError):
            q4lin.logprobs(handle, **dict(dict(logits=x, tokens=t), **change))
    inv = q4lin.Q4LIN_ERR_INVALID_ARG
    for top in (-1, 33):
        with pytest.raises((q4lin.Q4LinError, RuntimeError)):
            q4lin.logprobs(handle, x, t, top=top)
    with pytest.raises(q4lin.Q4LinError) as e:
        q4lin.logprobs(handle, x[:, :5], t, top=6)
    assert e.value.status == inv
    for change in (dict(lse=f[:3]), dict(d_logprob=f.half()), dict(out=x.half()), dict(out=x[:, :50])):
        with pytest.raises(ValueError):
            q4lin.logprobs_backward(handle, **dict(dict(logits=x, tokens=t, lse=f, entropy=f, d_logprob=f),
                                                   **change))
    for change in (dict(lse=None), dict(tokens=None), dict(d_entropy=f, entropy=None),
                   dict(out=torch.empty_like(x)[:1].expand(4, -1))):
        with pytest.raises(q4lin.Q4LinError) as e:
            q4lin.logprobs_backward(handle, **dict(dict(logits=x, tokens=t, lse=f, entropy=f, d_logprob=f),
                                                   **change))
        assert e.value.status == inv
    big = torch.randn(401, device="cuda")
    with pytest.raises(q4lin.Q4LinError):  # overlapping, but not in place
        q4lin.logprobs_backward(handle, big[:400].view(4, 100), t, f, f, f, out=big[1:].view(4, 100))
    assert q4lin.logprobs(handle, x[:0], t[:0], top=3).top_tokens.shape == (0, 3)
    torch.cuda.synchronize()

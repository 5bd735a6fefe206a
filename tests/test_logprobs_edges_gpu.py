"""Log probabilities and their gradient where rows hold NaN and infinities, strides say nothing,
and outputs lie on other streams."""
import numpy as np
import pytest

from tests import _operators as ops
from tests.test_logprobs_gpu import status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size,top", [(1, 7, 7), (2, 1, 1), (3, 32, 32), (400, 500, 5), (2, 70001, 20),
                                           (1, 128256, 32)])
def test_nan_at_both_ends(handle, rows, size, top, dtype):
    """A NaN counts as the largest entry wherever it stands, the first and the last place too, and
    of several the first comes first; one row split over CTAs and not."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(51)
    x = rng.standard_normal((rows, size)).astype(np.float32)
    every = np.full((rows, size), np.nan, np.float32)
    first, both = x.copy(), x.copy()
    first[:, 0] = np.nan
    both[:, [0, -1]] = np.nan
    for y in (first, both, every):
        y = ops.to_host(ops.to_device(y, dtype))
        r = q4lin.logprobs(handle, ops.to_device(y.astype(np.float32), dtype),
                           torch.zeros(rows, dtype=torch.int32, device="cuda"), top=top)
        order = np.argsort(np.where(np.isnan(y), -np.inf, -y), axis=1, kind="stable")[:, :top]
        assert np.array_equal(r.top_tokens.cpu().numpy(), order)
        assert torch.isnan(r.top_logprobs).all() and torch.isnan(r.lse).all()
        assert torch.isnan(r.entropy).all() and torch.isnan(r.logprob).all()
    assert status(handle) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(1, 40), (3, 5000), (400, 1000), (1, 128256), (20, 70001)])
def test_infinities_and_nan_in_one_row(handle, rows, size, dtype):
    """+infinity alone: lse is +infinity; with a NaN before or after it, near or far: NaN."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    rng = np.random.default_rng(53)
    x = ops.to_device(rng.standard_normal((rows, size)).astype(np.float32), dtype)
    tokens = torch.full((rows,), 3, dtype=torch.int32, device="cuda")
    for at, nan in ((5, None), (0, 1), (1, 0), (5, size - 1), (size - 1, 5), (size // 2, size // 2 + 1)):
        y = x.clone()
        y[:, at] = float("inf")
        if nan is not None:
            y[:, nan] = float("nan")
        r = q4lin.logprobs(handle, y, tokens, top=3)
        assert torch.isnan(r.lse).all() if nan is not None else bool((r.lse == float("inf")).all())
        assert torch.isnan(r.entropy).all() and torch.isnan(r.logprob).all()
        assert torch.isnan(r.top_logprobs).all()
        assert bool((r.top_tokens[:, 0] == (at if nan is None else nan)).all())
    # An excluded token's log probability is -infinity beside +infinity too, but not beside a NaN.
    y = x.clone()
    y[:, 3], y[:, 7] = -float("inf"), float("inf")
    assert bool((q4lin.logprobs(handle, y, tokens).logprob == -float("inf")).all())
    y[:, 8] = float("nan")
    assert torch.isnan(q4lin.logprobs(handle, y, tokens).logprob).all()


def test_one_row_has_no_stride(handle):
    """One row as a transposed column or a broadcast row, whose strides are 1 and 0: logits, the
    gradient, and both in one place."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(1, 1003, device="cuda")
    tokens, d = torch.tensor([7], dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    want = q4lin.logprobs(handle, x, tokens, top=5)
    gradient = q4lin.logprobs_backward(handle, x, tokens, want.lse, want.entropy, d, d)
    column = torch.empty(1003, 1, device="cuda").copy_(x.t()).t()
    assert column.stride() == (1, 1)
    for y in (column, x[0].expand(1, -1), x.as_strided((1, 1003), (0, 1))):
        assert all(torch.equal(a, b) for a, b in zip(q4lin.logprobs(handle, y, tokens, top=5), want))
        for out in (None, torch.empty(1003, 1, device="cuda").t(), torch.empty(1, 1003, device="cuda")):
            got = q4lin.logprobs_backward(handle, y, tokens, want.lse, want.entropy, d, d, out=out)
            assert torch.equal(got, gradient)
    got = q4lin.logprobs_backward(handle, column, tokens, want.lse, want.entropy, d, d, out=column)
    assert got is column and torch.equal(column, gradient)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(1, 128257), (300, 20001), (2, 37)])
def test_gradient_in_place_is_the_same(handle, rows, size, dtype):
    """Over all CTAs of a row and all rows at once, vectors and single entries."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(rows, size, device="cuda").to(ops.torch_dtype(dtype))
    tokens = torch.randint(size, (rows,), device="cuda", dtype=torch.int32)
    d = torch.randn(rows, device="cuda")
    r = q4lin.logprobs(handle, x, tokens)
    want = q4lin.logprobs_backward(handle, x, tokens, r.lse, r.entropy, d, d)
    assert torch.equal(q4lin.logprobs_backward(handle, x, tokens, r.lse, r.entropy, d, d, out=x), want)


def test_refusals_of_the_c_entries(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    x = torch.randn(4, 100, device="cuda")
    f, i = torch.zeros(40, device="cuda"), torch.zeros(40, dtype=torch.int32, device="cuda")
    top = torch.zeros(4, 3, device="cuda")
    d = torch.zeros(4, 100, device="cuda")
    at = lambda t, k=0: t.data_ptr() + 4 * k
    inv, large = q4lin.Q4LIN_ERR_INVALID_ARG, q4lin.Q4LIN_ERR_TOO_LARGE

    def forward(**change):
        a = q4lin.q4lin_logprobs_t(at(x), 100, 0, 4, 100, at(i), at(f), at(f, 4), at(f, 8), 3, at(i, 8), at(top))
        for n, v in change.items():
            setattr(a, n, v)
        return q4lin.q4lin_run_logprobs(handle.ptr, a, 0)

    def backward(**change):
        a = q4lin.q4lin_logprobs_backward_t(at(x), 100, 0, 4, 100, at(i), at(f), at(f, 4), at(f, 8), at(f, 12),
                                            at(d), 100)
        for n, v in change.items():
            setattr(a, n, v)
        return q4lin.q4lin_run_logprobs_backward(handle.ptr, a, 0)

    assert forward() == q4lin.Q4LIN_OK and backward() == q4lin.Q4LIN_OK
    assert forward(tokens=None, logprob=None, entropy=None, lse=None) == q4lin.Q4LIN_OK
    assert forward(rows=0) == q4lin.Q4LIN_OK and backward(rows=0) == q4lin.Q4LIN_OK
    for change in (dict(logits=None), dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocabulary=0),
                   dict(row_stride=-1), dict(top=-1), dict(top=33), dict(vocabulary=2), dict(top_tokens=None),
                   dict(top_logprobs=None), dict(logits=at(x) + 2), dict(tokens=at(i) + 1), dict(lse=at(f) + 2),
                   dict(entropy=at(f)), dict(lse=at(f, 1)), dict(logprob=at(x, 399)), dict(lse=at(i)),
                   dict(top_tokens=at(i, 2)), dict(row_stride=1 << 61)):
        assert forward(**change) == inv, change
    none = dict(tokens=None, logprob=None, entropy=None, lse=None, top=0)
    assert forward(vocabulary=1 << 31, rows=1, **none) == large  # (no output can overlap so many)
    for change in (dict(logits=None), dict(d_logits=None), dict(lse=None), dict(tokens=None), dict(entropy=None),
                   dict(dtype=7), dict(rows=-1), dict(vocabulary=0), dict(row_stride=-1), dict(d_row_stride=99),
                   dict(d_logits=at(d) + 2), dict(d_logits=at(x, 1)), dict(d_logits=at(x), d_row_stride=101),
                   dict(lse=at(d, 9)), dict(d_entropy=at(d, 399)), dict(d_row_stride=1 << 61)):
        assert backward(**change) == inv, change
    assert q4lin.q4lin_run_logprobs(None, q4lin.q4lin_logprobs_t(), 0) == inv
    assert q4lin.q4lin_run_logprobs(handle.ptr, None, 0) == inv
    assert q4lin.q4lin_run_logprobs_backward(None, q4lin.q4lin_logprobs_backward_t(), 0) == inv
    assert q4lin.q4lin_run_logprobs_backward(handle.ptr, None, 0) == inv
    torch.cuda.synchronize()
    assert status(handle) == 0

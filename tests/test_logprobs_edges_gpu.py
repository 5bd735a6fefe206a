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

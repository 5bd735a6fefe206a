"""The example decoder against float64: its last step over the caches that it built, and the
gradient that it takes back through the head."""
import os
import sys

import numpy as np
import pytest

import _operators as ops

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _weights(linear):
    codes = linear.codes.cpu().numpy()
    both = np.stack([codes & 15, codes >> 4], -1).reshape(linear.rows, linear.columns)
    scales = linear.scales.double().cpu().numpy().T  # [rows, groups]
    return (both.astype(np.float64) - 8) * np.repeat(scales, 32, 1)


def _norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


class HostCache(ops.Cache):
    """A device cache's contents after a call."""

    def __init__(self, cache):
        self.k, self.v = cache.k_codes.cpu().numpy(), cache.v_codes.cpu().numpy()
        self.ks, self.vs = cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()
        self.table = cache.page_table.cpu().numpy()
        self.heads, self.page, self.dim = self.k.shape[1:]


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import generate
    finally:
        sys.path.pop(0)
    return generate


def test_last_step_and_gradient(example):
    """Tolerances: a linear of these sizes is within 1e-5 sum |x w| (at most 4e-3 of it where the
    tensor cores multiply in tf32: not the rows here), which is up to sqrt(2 K / pi) ~ 18 times its
    outputs' size, so 2e-4 of them; ten products in a row, with the attention's 1e-5 between,
    give 2e-3 of the logits' size, and 1e-2 leaves room for what the norms and exponentials
    multiply.  The gradient is the formula's for the logits' gradient that it was given
    (1e-5 sum |d w|), and that one within the logits' 1e-2 of p."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin

    handle = q4lin.Handle(0)
    c = example.Config(layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024,
                       vocabulary=1001, page=16)
    model = example.Model(c, handle, 120)
    g = torch.Generator("cuda").manual_seed(3)
    prompts = [torch.randint(c.vocabulary, (n,), device="cuda", generator=g) for n in (70, 1, 33)]
    taken, scores, caches, logits = example.generate(model, prompts, 6)
    lengths = [len(p) + 5 for p in prompts]
    rope = tuple(t.cpu().numpy() for t in model.rope)
    x = model.embedding[taken[:, -2].long()].double().cpu().numpy()
    for cache, (qkv, o, up, down) in zip(caches, model.layers):
        y = (_norm(x) @ _weights(qkv).T).reshape(3, -1, c.head_dim)
        y = ops.attention(HostCache(cache), y[:, :c.heads], [0, 1, 2, 3], lengths, c.head_dim**-0.5,
                          rope)[0]
        x = x + y.reshape(3, -1) @ _weights(o).T
        gate, value = np.split(_norm(x) @ _weights(up).T, 2, 1)
        x = x + (gate / (1 + np.exp(-gate)) * value) @ _weights(down).T
    want = _norm(x) @ _weights(model.head).T
    got = logits.double().cpu().numpy()
    assert np.abs(got - want).max() <= 1e-2 * np.abs(want).max()
    # The last token's score is that of these logits.
    lp = ops.logprobs(got, taken[:, -1].cpu().numpy(), 1)[0]
    assert np.abs(scores[:, -1].double().cpu().numpy() - lp).max() <= 1e-5

    advantages = torch.tensor([1.0, -0.5, 2.0], device="cuda")
    gradient, again = example.policy_gradient(model, prompts, taken, advantages)
    assert gradient.shape == (18, c.hidden) and bool(torch.isfinite(gradient).all())
    # What an 8-bit cache loses differs between the two ways of filling it: 1/254 of a page's
    # largest value per key and value, so log probabilities of size 10 agree to a few percent.
    assert float((again - scores).abs().max()) <= 0.5
    status, code = q4lin.q4lin_check_device_status(handle.ptr, torch.cuda.current_stream().cuda_stream)
    assert (status, code) == (q4lin.Q4LIN_OK, 0)
    handle.close()


def test_gradient_of_the_head(example):
    """The loss in float64, differenced along random directions of the hidden states."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin

    handle = q4lin.Handle(0)
    g = torch.Generator("cuda").manual_seed(5)
    head = example.Linear(501, 256, g)
    x = torch.randn(6, 256, device="cuda", generator=g)
    tokens = torch.tensor([3, 500, 0, -1, 77, 77], dtype=torch.int32, device="cuda")
    a = torch.randn(6, device="cuda", generator=g)
    e = torch.randn(6, device="cuda", generator=g)
    logits = head(handle, x)
    got = q4lin.logprobs(handle, logits, tokens)
    q4lin.logprobs_backward(handle, logits, tokens, got.lse, got.entropy, a, e, out=logits)
    d_x = head.gradient(handle, logits).double().cpu().numpy()

    w, xs = _weights(head), x.double().cpu().numpy()
    weights = [t.double().cpu().numpy() for t in (a, e)]

    def loss(at):
        lp, entropy = ops.logprobs(at @ w.T, tokens.cpu().numpy(), 1)[:2]
        return weights[0] @ lp + weights[1] @ entropy

    rng = np.random.default_rng(0)
    for _ in range(4):
        way = rng.standard_normal(xs.shape)
        step = 1e-5
        slope = (loss(xs + step * way) - loss(xs - step * way)) / (2 * step)
        # Differences: step^2 of the third derivative; the gradient: 1e-5 of each product's terms
        # (256 x 501 of them, of random signs) against a slope of the size of their sum.
        assert abs((d_x * way).sum() - slope) <= 1e-4 * np.abs(d_x * way).sum()
    handle.close()

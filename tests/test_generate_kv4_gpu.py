"""The example decoder with normalised heads over the 4-bit cache: its last step against float64 over
the caches that it built."""
import numpy as np
import pytest

from tests import _kv4 as kv4
from tests import _operators as ops
from tests.test_generate_gpu import _norm, _weights, example  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_norm", [0, 1])
def test_last_step(example, head_norm):
    """Tolerance as in test_generate_gpu: linears of these sizes leave 2e-3 of the logits' size behind
    ten products in a row, and 1e-2 leaves room for what norms and exponentials multiply.  (What the
    cache holds is read from it, so its codes do not count.)"""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin

    handle = q4lin.Handle(0)
    c = example.Config(layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024,
                       vocabulary=1001, page=16, cache_bits=4, head_norm=head_norm)
    model = example.Model(c, handle, 120)
    g = torch.Generator("cuda").manual_seed(3)
    prompts = [torch.randint(c.vocabulary, (n,), device="cuda", generator=g) for n in (70, 1, 33)]
    taken, scores, caches, logits = example.generate(model, prompts, 6)
    lengths = [len(p) + 5 for p in prompts]
    position = np.array(lengths) - 1
    rope = tuple(t.cpu().numpy() for t in model.rope)
    x = model.embedding[taken[:, -2].long()].double().cpu().numpy()
    for layer, (cache, (qkv, o, up, down)) in enumerate(zip(caches, model.layers)):
        y = (_norm(x) @ _weights(qkv).T).reshape(3, -1, c.head_dim)
        q = y[:, :c.heads]
        if head_norm:
            q, _ = kv4.norm_rope(q, model.head_norms[layer][0].double().cpu().numpy(), position, rope, 1e-6, False)
        y = ops.attention(kv4.DeviceCache(cache), q, [0, 1, 2, 3], lengths, c.head_dim**-0.5,
                          None if head_norm else rope)[0]
        x = x + y.reshape(3, -1) @ _weights(o).T
        gate, value = np.split(_norm(x) @ _weights(up).T, 2, 1)
        x = x + (gate / (1 + np.exp(-gate)) * value) @ _weights(down).T
    want = _norm(x) @ _weights(model.head).T
    got = logits.double().cpu().numpy()
    assert np.abs(got - want).max() <= 1e-2 * np.abs(want).max()
    # One pass over prompts and generated tokens, and its gradient: finite, and of the right shape.
    gradient, again = example.policy_gradient(model, prompts, taken, torch.tensor([1.0, -0.5, 2.0], device="cuda"))
    assert gradient.shape == (18, c.hidden) and bool(torch.isfinite(gradient).all())
    assert again.shape == scores.shape and bool(torch.isfinite(again).all())
    status, code = q4lin.q4lin_check_device_status(handle.ptr, torch.cuda.current_stream().cuda_stream)
    assert (status, code) == (q4lin.Q4LIN_OK, 0)
    handle.close()

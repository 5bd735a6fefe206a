"""Outputs of calls on another stream than torch's current one."""
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


def calls(handle):
    """name -> a call on a stream, which returns its outputs."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin, synth
    c = synth.make_case(8, 1024, 256, 32, seed=71)
    x, w, s = (ops.to_device(a) for a in (c.x, c.qweight, c.scales))
    host = ops.Cache(np.random.default_rng(72), [200, 90], 2, 32, 64)
    cache, q = host.device(), torch.randn(40, 8, 64, device="cuda")
    o, n = (ops.to_device(np.array(a, np.int32)) for a in ([0, 30, 40], [200, 90]))
    logits, tokens = torch.randn(16, 3001, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")
    got, d = q4lin.logprobs(handle, logits, tokens), torch.randn(16, device="cuda")
    torch.cuda.synchronize()
    return {"linear": lambda t: [q4lin.linear(handle, x, w, s, None, 32, stream=t)],
            "attention": lambda t: list(q4lin.attention(handle, cache, q, o, n, 0.125, stream=t)),
            "logprobs": lambda t: list(q4lin.logprobs(handle, logits, tokens, top=7, stream=t)),
            "gradient": lambda t: [q4lin.logprobs_backward(handle, logits, tokens, got.lse, got.entropy, d, d,
                                                           stream=t)]}


@pytest.mark.parametrize("name", ["linear", "attention", "logprobs", "gradient"])
@pytest.mark.parametrize("default", [False, True])
def test_memory_that_the_current_stream_still_writes(handle, name, default):
    """The current stream has freed memory of the outputs' sizes that it is yet to write: the
    call's outputs lie elsewhere.  On a stream of its own, and on the default one from another."""
    import torch
    call = calls(handle)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    current, other = (side, torch.cuda.default_stream()) if default else (torch.cuda.current_stream(), side)
    with torch.cuda.stream(current):
        waste = [torch.empty_like(t) for t in want for _ in range(3)]
        torch.cuda._sleep(40_000_000)  # (about 20 ms)
        for t in waste:
            t.fill_(77)
        del waste, t
        got = call(other.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_outlive_their_use_on_the_current_stream(handle):
    """Freed while the current stream is yet to read them, they are not given to the next call."""
    import torch
    call = calls(handle)["attention"]
    want = call(None)[0].clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    out = call(other.cuda_stream)[0]
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(40_000_000)
    kept = out.clone()
    del out
    with torch.cuda.stream(other):
        waste = [torch.full_like(want, 55) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(waste) == 4

"""Calls of a decoder layer over a 4-bit cache one right after the other: launches that overlap the end of
what the stream ran before give the bits of calls that wait for one another, whatever the last kernel wrote
(positions, lengths, a linear's weights).  And what the binding refuses by itself."""
import numpy as np
import pytest

from tests import _operators as ops

pytestmark = pytest.mark.gpu
STEPS = 40


@pytest.fixture(scope="module")
def handle():
    from bit_weight_quantized_int4_gb300 import q4lin
    h = q4lin.Handle(0)
    yield h
    h.close()


class Layer:
    """A sequence of each length, one token more a step; everything that changes is on the device."""

    def __init__(self, handle, heads, kv_heads, dim, dtype, lengths):
        import torch
        rng = np.random.default_rng(heads + dim)
        self.handle, self.n = handle, len(lengths)
        pages = (max(lengths) + STEPS) // 16 + 1
        table = rng.permutation(self.n * pages).astype(np.int32).reshape(self.n, pages)
        from bit_weight_quantized_int4_gb300 import q4lin
        self.q4lin = q4lin
        self.cache = q4lin.KVCache4.empty(self.n * pages, kv_heads, 16, dim, ops.to_device(table))
        self.offsets = ops.to_device(np.arange(self.n + 1, dtype=np.int32))
        self.starts = ops.to_device(np.array(lengths, np.int32))
        self.first = self.starts.clone()
        self.rope = tuple(map(ops.to_device, ops.rope_tables(rng, max(lengths) + STEPS + 1, dim)))
        self.weight = ops.to_device(rng.uniform(0.5, 1.5, dim).astype(np.float32))
        self.x = ops.to_device(rng.standard_normal((self.n, heads + 2 * kv_heads, dim)).astype(np.float32), dtype)
        self.x0, self.split, self.scale = self.x.clone(), [heads, kv_heads, kv_heads], dim**-0.5

    def reset(self):
        self.x.copy_(self.x0)
        self.starts.copy_(self.first)
        self.cache.k_codes.fill_(0x88), self.cache.v_codes.fill_(0x88)
        self.cache.k_scales.zero_(), self.cache.v_scales.zero_()

    def step(self, wait=lambda: None):
        q, k, v = self.x.split(self.split, 1)
        q, k = self.q4lin.norm_rope(self.handle, q, k, self.weight, self.weight, self.starts, self.rope)
        wait()
        self.q4lin.kv_append(self.handle, self.cache, k, v, self.offsets, self.starts)
        wait()
        out, lse = self.q4lin.attention(self.handle, self.cache, q, self.offsets, self.starts + 1, self.scale, max_query=1)
        wait()
        back = self.q4lin.kv_read(self.handle, self.cache, self.offsets, self.starts, self.n, dtype=q.dtype)
        wait()
        grads = self.q4lin.norm_rope_backward(self.handle, q, k, self.weight, self.weight, self.starts, self.rope, out, back[1])
        wait()
        self.starts.add_(1)
        self.x.mul_(0.5).add_(out.repeat(1, 3, 1)[:, :self.x.shape[1]]).add_(grads.d_q_weight.to(self.x.dtype) * 0.01)
        wait()
        return out, lse, *back, *grads


@pytest.mark.parametrize("heads,kv_heads,dim,dtype,lengths", [(8, 2, 128, "bf16", [0, 1, 500, 63, 17]),
                                                              (4, 4, 64, "f32", [300])])
def test_steps_without_a_pause(handle, heads, kv_heads, dim, dtype, lengths):
    import torch
    layer = Layer(handle, heads, kv_heads, dim, dtype, lengths)
    layer.reset()
    want = [layer.step(torch.cuda.synchronize) for _ in range(STEPS)]
    torch.cuda.synchronize()
    layer.reset()
    got = [layer.step() for _ in range(STEPS)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    layer.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer.step()
    layer.reset()
    for _ in range(STEPS):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want[-1]))
    assert all(bool(torch.isfinite(t).all()) for t in want[-1])


@pytest.mark.parametrize("early", [0, 1])
def test_weights_that_were_just_written(handle, early):
    """A linear whose codes the stream wrote two kernels ago, a norm between them; the linear may begin
    while the norm runs, but not before the codes are there."""
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    torch.manual_seed(2)
    n, k, tokens = 4096, 2048, 1
    latents = [torch.randn(n, k, device="cuda") for _ in range(2)]
    scales = torch.full((n, 1), 0.25, device="cuda")
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    x = torch.randn(tokens, k // 64, 64, device="cuda")
    none = x[:, :0]

    def step(latent, wait):
        stream = torch.cuda.current_stream().cuda_stream
        assert q4lin.q4lin_run_requant(handle.ptr, latent.data_ptr(), scales.data_ptr(), codes.data_ptr(), n, k, k, 0,
                                       stream) == q4lin.Q4LIN_OK
        wait()
        y, _ = q4lin.norm_rope(handle, x, none)
        wait()
        return q4lin.linear(handle, y.view(tokens, k), codes, scales, None, k)

    want = [step(latent, torch.cuda.synchronize) for latent in latents]
    assert not torch.equal(*want)
    handle.set_option(q4lin.Q4LIN_OPT_PDL, early)
    try:
        got = [step(latents[i % 2], lambda: None) for i in range(60)]
    finally:
        handle.set_option(q4lin.Q4LIN_OPT_PDL, 0)
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


def test_binding_refuses(handle):
    import torch
    from bit_weight_quantized_int4_gb300 import q4lin
    q, k = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda")
    w, at = torch.ones(64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    rope = torch.ones(5, 32, device="cuda"), torch.zeros(5, 32, device="cuda")
    good = dict(q=q, k=k, q_weight=w, k_weight=w, positions=at, rope=rope)
    q4lin.norm_rope(handle, **good)
    for change in (dict(q=q.cpu()), dict(q=q.half()), dict(q=q.double(), k=k.double()), dict(k=k[:2]), dict(k=k[..., :32]),
                   dict(q=q.transpose(1, 2)), dict(q_weight=w.half()), dict(k_weight=w[:32]), dict(q_weight=w.cpu()),
                   dict(positions=at.long()), dict(positions=at[:2]), dict(positions=None), dict(rope=(rope[0], rope[1][:4])),
                   dict(rope=(rope[0].half(), rope[1])), dict(q_out=q.half()), dict(k_out=q), dict(q_out=q[:2])):
        with pytest.raises(ValueError):
            q4lin.norm_rope(handle, **{**good, **change})
    more = dict(good, d_q_out=q, d_k_out=k)
    q4lin.norm_rope_backward(handle, **more)
    for change in (dict(d_q_out=q[:2]), dict(d_k_out=k.half()), dict(d_q_out=q.cpu()), dict(d_q=q.half()), dict(d_k=q)):
        with pytest.raises(ValueError):
            q4lin.norm_rope_backward(handle, **{**more, **change})
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    cache, one = q4lin.KVCache4.empty(2, 2, 16, 64, table), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    read = dict(cache=cache, offsets=one, starts=starts, tokens=3)
    q4lin.kv_read(handle, **read)
    for change in (dict(offsets=one.long()), dict(offsets=one[:1]), dict(starts=starts.cpu()), dict(dtype=torch.float64),
                   dict(k=k[:2]), dict(k=k.half(), v=k), dict(k=k.transpose(0, 1)),
                   dict(cache=q4lin.KVCache.empty(2, 2, 64, 64, table))):
        with pytest.raises(ValueError):
            q4lin.kv_read(handle, **{**read, **change})
    for change in (dict(q=q.expand(3, 4, 64)[:, :1].expand(3, 4, 64), q_out=q[:, :1].expand(3, 4, 64)), dict(eps=float("nan")),
                   dict(eps=-1.0)):
        with pytest.raises(q4lin.Q4LinError):
            q4lin.norm_rope(handle, **{**good, **change})

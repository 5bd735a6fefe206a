"""A decoder of 4-bit linears that generates text tokens, scores them and takes the policy
gradient of what it generated back to its last hidden states.

    python examples/generate.py [--layers 16 --hidden 2048 --heads 32 --kv-heads 8 ...]

The weights are random (the shapes are what counts here), activations are fp32.  Every layer
keeps its keys and values in a paged 8-bit cache; all layers share one page table.

    prompts    one call for all of them: kv_append rotates and stores the keys, attention
               reads them back (many query rows per sequence)
    steps      the same two calls with one token per sequence
    logits     logprobs gives the alternatives that the next token is drawn from, and the
               log probability of the drawn one
    learning   logprobs_backward turns advantages into the logits' gradient (in the logits'
               own memory), and the head's input gradient takes it to the hidden states
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_quantized_int4_gb300 import q4lin  # noqa: E402

GROUP = 32  # weights per scale


@dataclass
class Config:
    layers: int = 4
    hidden: int = 1024
    heads: int = 16
    kv_heads: int = 4
    head_dim: int = 64
    inner: int = 4096
    vocabulary: int = 32000
    page: int = 32


class Linear:
    """Packed 4-bit weights [rows, columns] with one fp16 scale per 32 of a row."""

    def __init__(self, rows, columns, generator):
        device = generator.device
        self.rows, self.columns = rows, columns
        low, high = (torch.randint(1, 16, (rows, columns // 2), dtype=torch.uint8, device=device,
                                   generator=generator) for _ in range(2))
        self.codes = low + 16 * high
        gain = 1 / (4.3 * math.sqrt(columns))  # codes - 8: mean 0, standard deviation 4.3
        self.scales = gain * (0.5 + torch.rand(columns // GROUP, rows, device=device,
                                               generator=generator))
        self.scales = self.scales.half()

    def __call__(self, handle, x):
        return q4lin.linear(handle, x, self.codes, self.scales, None, GROUP)

    def gradient(self, handle, d_out):
        """Of its input, given that of its output."""
        d_x = torch.empty(d_out.shape[0], self.columns, device=d_out.device)
        status = q4lin.q4lin_run_backward_dx(
            handle.ptr, d_out.data_ptr(), self.codes.data_ptr(), self.scales.data_ptr(),
            d_x.data_ptr(), d_out.shape[0], self.rows, self.columns, GROUP, q4lin.Q4LIN_SCALE_F16,
            torch.cuda.current_stream().cuda_stream)
        if status != q4lin.Q4LIN_OK:
            raise q4lin.Q4LinError(status, "q4lin_run_backward_dx")
        return d_x


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self, config, handle, positions, seed=0):
        c, device = config, torch.device("cuda", handle.device)
        g = torch.Generator(device).manual_seed(seed)
        self.config, self.handle = c, handle
        self.embedding = torch.randn(c.vocabulary, c.hidden, device=device, generator=g)
        width = (c.heads + 2 * c.kv_heads) * c.head_dim  # queries, keys and values in one product
        self.layers = [(Linear(width, c.hidden, g), Linear(c.hidden, c.heads * c.head_dim, g),
                        Linear(2 * c.inner, c.hidden, g), Linear(c.hidden, c.inner, g))
                       for _ in range(c.layers)]
        self.head = Linear(c.vocabulary, c.hidden, g)
        rate = 10000.0 ** (-torch.arange(0, c.head_dim, 2, device=device) / c.head_dim)
        angle = torch.arange(positions, device=device)[:, None] * rate
        self.rope = angle.cos().contiguous(), angle.sin().contiguous()

    def caches(self, sequences, tokens):
        """Empty caches of all layers, with room for `tokens` tokens of each sequence."""
        c = self.config
        pages = -(-tokens // c.page)
        table = torch.randperm(sequences * pages, device=self.embedding.device)
        table = table.to(torch.int32).view(sequences, pages)
        return [q4lin.KVCache.empty(sequences * pages, c.kv_heads, c.page, c.head_dim, table)
                for _ in self.layers]

    def hidden(self, caches, tokens, offsets, held, most):
        """Last hidden states [len(tokens), hidden] of the new tokens, rows offsets[b] to
        offsets[b + 1] of sequence b, which holds held[b] before and no more than `most` new
        ones; the caches grow by them."""
        c, handle = self.config, self.handle
        lengths = held + offsets[1:] - offsets[:-1]
        x = self.embedding[tokens]
        for cache, (qkv, o, up, down) in zip(caches, self.layers):
            y = qkv(handle, norm(x)).view(-1, c.heads + 2 * c.kv_heads, c.head_dim)
            q, k, v = y.split([c.heads, c.kv_heads, c.kv_heads], 1)
            q4lin.kv_append(handle, cache, k, v, offsets, held, rope=self.rope)
            y, _ = q4lin.attention(handle, cache, q, offsets, lengths, c.head_dim**-0.5,
                                   max_query=most, rope=self.rope)
            x = x + o(handle, y.view(-1, c.heads * c.head_dim))
            gate, value = up(handle, norm(x)).chunk(2, 1)
            x = x + down(handle, torch.nn.functional.silu(gate) * value)
        return norm(x)


def offsets_of(counts):
    """[0, counts[0], counts[0] + counts[1], ...] for the device."""
    return torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)


def generate(model, prompts, steps, top=16, seed=0):
    """`steps` tokens for each prompt, each drawn from the `top` most likely ones.  Returns
    (tokens [prompts, steps], their log probabilities, caches, the last step's logits)."""
    handle, device = model.handle, model.embedding.device
    g = torch.Generator(device).manual_seed(seed)
    counts = torch.tensor([len(p) for p in prompts], device=device)
    caches = model.caches(len(prompts), max(map(len, prompts)) + steps)
    held = torch.zeros(len(prompts), dtype=torch.int32, device=device)
    x = model.hidden(caches, torch.cat(prompts), offsets_of(counts), held, max(map(len, prompts)))
    x = x[counts.cumsum(0) - 1]  # each prompt's last token
    held = counts.to(torch.int32)
    one = torch.arange(len(prompts) + 1, dtype=torch.int32, device=device)
    taken, scores = [], []
    for step in range(steps):
        logits = model.head(handle, x)
        best = q4lin.logprobs(handle, logits, top=top)
        at = torch.multinomial(best.top_logprobs.exp(), 1, generator=g)
        taken.append(best.top_tokens.gather(1, at)[:, 0])
        scores.append(best.top_logprobs.gather(1, at)[:, 0])
        if step + 1 < steps:
            x = model.hidden(caches, taken[-1], one, held, 1)
            held += 1
    return torch.stack(taken, 1), torch.stack(scores, 1), caches, logits


def policy_gradient(model, prompts, taken, advantages, entropy_weight=0.01):
    """Of -mean(advantage * log probability + entropy_weight * entropy) over the generated
    tokens, for the hidden states that predicted them; and the log probabilities."""
    handle, device = model.handle, model.embedding.device
    steps = taken.shape[1]
    rows = [torch.cat([p, t[:-1].to(p.dtype)]) for p, t in zip(prompts, taken)]
    counts = torch.tensor([len(r) for r in rows], device=device)
    held = torch.zeros(len(rows), dtype=torch.int32, device=device)
    caches = model.caches(len(rows), max(map(len, rows)))
    x = model.hidden(caches, torch.cat(rows), offsets_of(counts), held, max(map(len, rows)))
    last = torch.arange(1 - steps, 1, device=device)  # the tokens that predict taken ones
    x = x[(counts.cumsum(0)[:, None] - 1 + last).flatten()]
    logits, tokens = model.head(handle, x), taken.flatten()
    got = q4lin.logprobs(handle, logits, tokens)
    d_logprob = -advantages.repeat_interleave(steps) / tokens.numel()
    d_entropy = torch.full_like(d_logprob, -entropy_weight / tokens.numel())
    q4lin.logprobs_backward(handle, logits, tokens, got.lse, got.entropy, d_logprob, d_entropy,
                            out=logits)
    return model.head.gradient(handle, logits), got.logprob.view_as(taken)


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in vars(Config()).items():
        parser.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    parser.add_argument("--sequences", type=int, default=8)
    parser.add_argument("--prompt", type=int, default=700, help="longest prompt")
    parser.add_argument("--steps", type=int, default=64)
    args = vars(parser.parse_args())
    sequences, longest, steps = (args.pop(n) for n in ("sequences", "prompt", "steps"))
    config, handle = Config(**args), q4lin.Handle(0)
    model = Model(config, handle, longest + steps)
    g = torch.Generator("cuda").manual_seed(1)
    prompts = [torch.randint(config.vocabulary, (max(1, longest * (b + 1) // sequences),),
                             device="cuda", generator=g) for b in range(sequences)]
    generate(model, prompts, 2)  # (the library loads its kernels at their first use)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    taken, scores, _, _ = generate(model, prompts, steps)
    end.record()
    gradient, again = policy_gradient(model, prompts, taken, torch.randn(sequences, device="cuda"))
    status, code = q4lin.q4lin_check_device_status(handle.ptr, torch.cuda.current_stream().cuda_stream)
    if status != q4lin.Q4LIN_OK:
        raise SystemExit(f"device status {code}")
    print(f"{sequences} prompts of {len(prompts[0])} to {len(prompts[-1])} tokens, {steps} tokens each: "
          f"{start.elapsed_time(end):.1f} ms")
    print(f"mean log probability {scores.mean():.4f} generated, {again.mean():.4f} scored in one pass "
          f"(largest difference {(scores - again).abs().max():.4f})")
    print(f"gradient at the hidden states: {list(gradient.shape)}, norm {gradient.norm():.4g}")


if __name__ == "__main__":
    main()

"""Plain float64 (numpy) forms of the operators around the linears, written from their
definitions, and the inputs of their tests."""
import numpy as np

DTYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
# Unit roundoff of an output's type (half an ulp, relative), and the spacing below which the
# type has no more bits.
ROUND = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f32": 1e-37, "f16": 2.0**-24, "bf16": 1e-37}


def torch_dtype(name):
    import torch
    return getattr(torch, DTYPES[name])


def to_device(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(torch_dtype(dtype))


def to_host(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rope_tables(rng, positions, rotated):
    angle = rng.uniform(0, 6.3, size=(positions, rotated // 2))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def rotate(x, position, rope, interleaved, dtype=np.float64):
    """x [tokens, heads, dim], each product and sum rounded to dtype once."""
    if rope is None:
        return x.astype(dtype)
    x = x.astype(dtype)
    cos, sin = (t[position][:, None].astype(dtype) for t in rope)
    half = cos.shape[-1]
    out = x.copy()
    a_at = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b_at = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., a_at], x[..., b_at]
    out[..., a_at] = a * cos - b * sin
    out[..., b_at] = b * cos + a * sin
    return out


class Cache:
    """A cache on the host; values [page, head, dim, slot] as on the device."""

    def __init__(self, rng, lengths, kv_heads, page, dim, spare=2, filled=True):
        need = [-(-n // page) for n in lengths]
        total = max(1, sum(need) + spare)
        order = rng.permutation(total)
        self.page, self.dim, self.heads, self.total = page, dim, kv_heads, total
        self.table = np.full((len(lengths), max(need + [0]) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape_k, shape_v = (total, kv_heads, page, dim), (total, kv_heads, dim, page)
        if filled:
            draw = lambda s: np.clip(np.rint(rng.standard_normal(s) * 36), -127, 127)
            self.k = (draw(shape_k) + 128).astype(np.uint8)
            self.v = (draw(shape_v) + 128).astype(np.uint8)
            self.ks = rng.uniform(0.01, 0.06, (total, kv_heads)).astype(np.float32)
            self.vs = rng.uniform(0.004, 0.03, (total, kv_heads)).astype(np.float32)
        else:
            self.k, self.v = np.full(shape_k, 128, np.uint8), np.full(shape_v, 128, np.uint8)
            self.ks, self.vs = (np.zeros((total, kv_heads), np.float32) for _ in range(2))

    def device(self):
        from bit_weight_quantized_int4_gb300 import q4lin
        return q4lin.KVCache(to_device(self.k), to_device(self.ks), to_device(self.v),
                             to_device(self.vs), to_device(self.table))

    def keys(self, b, n, h):
        """[n, dim] of head h of sequence b, in float64."""
        p = self.table[b, :-(-n // self.page)]
        k = (self.k[p, h].astype(np.float64) - 128) * self.ks[p, h].astype(np.float64)[:, None, None]
        return k.reshape(-1, self.dim)[:n]

    def values(self, b, n, h):
        p = self.table[b, :-(-n // self.page)]
        v = (self.v[p, h].astype(np.float64) - 128) * self.vs[p, h].astype(np.float64)[:, None, None]
        return v.transpose(0, 2, 1).reshape(-1, self.dim)[:n]


def append(cache, k, v, offsets, starts, rope=None, interleaved=False):
    """The append's definition on the host cache, in the fp32 steps that fix its bytes.
    k, v: float32 arrays of the (exactly held) inputs."""
    f = np.float32
    with np.errstate(all="ignore"):
        for b in range(len(starts)):
            n = offsets[b + 1] - offsets[b]
            if n <= 0:
                continue
            position = np.arange(starts[b], starts[b] + n)
            rows = slice(offsets[b], offsets[b + 1])
            new = {"k": rotate(k[rows], position, rope, interleaved, f), "v": v[rows].astype(f)}
            for p in range(starts[b] // cache.page, (starts[b] + n - 1) // cache.page + 1):
                at = position[(position // cache.page) == p]
                held = max(0, min(starts[b] - p * cache.page, cache.page))
                page = cache.table[b, p]
                for name in ("k", "v"):
                    x = new[name][at - starts[b]]  # [tokens, heads, dim]
                    codes = cache.k if name == "k" else cache.v
                    scales = cache.ks if name == "k" else cache.vs
                    for h in range(cache.heads):
                        c = codes[page, h] if name == "k" else codes[page, h].T  # [slot, dim], views
                        y = x[:, h]
                        finite = np.abs(y)[np.isfinite(y)]
                        amax = f(finite.max()) if finite.size else f(0)
                        s0 = scales[page, h] if held else f(0)
                        s = max(s0, f(amax * f(1.0 / 127.0)))
                        if not s >= f(2.0**-126):
                            s = f(0)
                        if s > s0 and s0 > 0:
                            old = c[:held].astype(f) - f(128)
                            c[:held] = (np.rint(old * f(s0 / s)) + 128).astype(np.uint8)
                        inv = f(1) / s if s > 0 else f(0)
                        z = np.rint(y * inv)
                        z = np.where(np.isnan(z), 0, np.clip(z, -127, 127))
                        c[at % cache.page] = (z + 128).astype(np.uint8)
                        scales[page, h] = s


def attention(cache, q, offsets, lengths, scale, rope=None, interleaved=False, causal=True, window=0):
    """(out, lse, the largest |value| and the largest sum of |q k| behind each row)."""
    tokens, heads, dim = q.shape
    group = heads // cache.heads
    out = np.zeros((tokens, heads, dim))
    lse = np.full((tokens, heads), -np.inf)
    vmax, smax = np.zeros((tokens, heads)), np.zeros((tokens, heads))
    for b in range(len(lengths)):
        t, n = offsets[b + 1] - offsets[b], lengths[b]
        if t <= 0 or n <= 0:
            continue
        position = np.arange(n - t, n)
        x = rotate(q[offsets[b]:offsets[b + 1]], np.maximum(position, 0), rope, interleaved)
        key = np.arange(n)
        for i in range(t):
            seen = np.ones(n, bool)
            if causal:
                seen &= key <= position[i]
            if window:
                seen &= key > position[i] - window
            if not seen.any():
                continue
            for h in range(heads):
                k, v = cache.keys(b, n, h // group)[seen], cache.values(b, n, h // group)[seen]
                s = scale * (k @ x[i, h])
                m = s.max()
                p = np.exp(s - m)
                row = offsets[b] + i
                out[row, h] = p @ v / p.sum()
                lse[row, h] = m + np.log(p.sum())
                vmax[row, h] = np.abs(v).max()
                smax[row, h] = (scale * (np.abs(k) @ np.abs(x[i, h]))).max()
    return out, lse, vmax, smax


def logprobs(x, tokens, top):
    """Of float64 logits: logprob, entropy, lse, top tokens, top log probabilities."""
    rows, size = x.shape
    with np.errstate(all="ignore"):
        m = x.max(1)
        safe = np.where(np.isfinite(m), m, 0)
        e = np.exp(x - safe[:, None])
        lse = np.where(m == -np.inf, -np.inf, safe + np.log(e.sum(1)))
        lp = np.where(x == -np.inf, -np.inf, x - lse[:, None])
        p = np.where(x == -np.inf, 0, np.exp(lp))
        entropy = -np.where(p > 0, p * lp, 0).sum(1)
    logprob = np.array([0.0 if t < 0 else lp[r, t] for r, t in enumerate(tokens)])
    order = np.argsort(-x, axis=1, kind="stable")[:, :top]
    return logprob, entropy, lse, order.astype(np.int32), np.take_along_axis(lp, order, 1)


def logprobs_backward(x, tokens, lse, entropy, d_logprob, d_entropy):
    """The gradient's definition in float64; lse and entropy as the call is given them."""
    with np.errstate(all="ignore"):
        lp = x - lse[:, None]
        p = np.where((x == -np.inf) | (lse == -np.inf)[:, None], 0, np.exp(lp))
        d = -p * (d_logprob * (tokens >= 0))[:, None]
        d -= np.where(p > 0, p * (lp + entropy[:, None]), 0) * d_entropy[:, None]
    for r, t in enumerate(tokens):
        if t >= 0 and lse[r] != -np.inf:
            d[r, t] += d_logprob[r]
    return d

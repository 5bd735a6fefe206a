"""The operators of a decoder layer whose cache is held in 4 bits, as they are measured: what
goes into each, what comes out, and the same results from elementary torch operations.

  norm      queries and keys normalised per head and rotated, in one pass
  gradient  the gradient of that for queries, keys and both weights
  append    keys and values quantised into a paged 4-bit cache as they are written, and what
            was written read back
  read      stretches of such a cache as dense keys and values
  attend    attention over such a cache: one token a sequence, a few, or a prompt's chunk

With `own` false, run() computes them in plain torch, in 32 bits; with `own` true it calls
the framework.  A 4-bit cache holds, for each page of `page` tokens and each key-value head,
keys and values [page, dim / 2] as bytes, two codes each (the even channel in the low half),
and one scale per token, head and kind: a code c stands for (c - 8) * scale.  The codes are
whole numbers that the definition fixes (every step rounds once, in a given order), so the
values read back are equal bit for bit.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROPE_BASE = 500000.0
EPS = 1e-6
_handles = []


def _norm(name, op, tokens, heads, kv_heads, dim, dtype, rotated=None, interleaved=False):
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "rotated": dim if rotated is None else rotated,
            "interleaved": interleaved}


def _stretch(name, op, batch, start, tokens, kv_heads, dim, page, dtype, rotated=0):
    return {"name": name, "op": op, "batch": batch, "start": start, "tokens": tokens,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "rotated": rotated}


def _attend(name, batch, length, tokens, heads, kv_heads, dim, page, dtype, window=0, rotated=0):
    return {"name": name, "op": "attend", "batch": batch, "length": length, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "window": window, "rotated": rotated}


def listed():
    return [
        # One new token of one conversation, the 1B shape (32 + 8 heads of 64): latency.
        _norm("norm_one", "norm", 1, 32, 8, 64, "f32"),
        # A prompt of 8192 tokens, the 8B shape, slices of the one q/k/v product.
        _norm("norm_prompt", "norm", 8192, 32, 8, 128, "bf16"),
        # Training on a short text: odd tokens, seven query heads a key head, half of each
        # head rotated, neighbouring channels in pairs.
        _norm("gradient_odd", "gradient", 701, 28, 4, 128, "f16", rotated=64, interleaved=True),
        # Training on 8192 tokens, the 8B shape.
        _norm("gradient_rows", "gradient", 8192, 32, 8, 128, "bf16"),
        # A decode step of 64 conversations of different lengths, the 8B shape.
        _stretch("append_step", "append", 64, 4095, 1, 8, 128, 64, "bf16"),
        # Seven prompts of odd lengths written in one call, rotated on the way, as the
        # framework's linears give them (fp32).
        _stretch("append_prompts", "append", 7, 0, 2047, 8, 128, 64, "f32", rotated=128),
        # The last few tokens of three short conversations, the 1B shape.
        _stretch("read_few", "read", 3, 700, 17, 8, 64, 16, "f32"),
        # A document of 65531 tokens out of the cache, the 8B shape.
        _stretch("read_long", "read", 1, 0, 65531, 8, 128, 64, "bf16"),
        # One token over a short conversation, the 1B shape: latency.
        _attend("attend_one", 1, 701, 1, 32, 8, 64, 16, "f32"),
        # One token over one very long document, the 8B shape: the long axis is all there is.
        _attend("attend_long", 1, 131071, 1, 32, 8, 128, 64, "bf16"),
        # A decode step of 64 conversations of up to 8192 tokens, the 8B shape.
        _attend("attend_batch", 64, 8192, 1, 32, 8, 128, 64, "f32"),
        # The last 2048 tokens of an 8192-token prompt that is read in chunks, the 8B shape.
        _attend("attend_prompt", 1, 8192, 2048, 32, 8, 128, 64, "bf16"),
    ]


def _between(rng, low, high):
    """A whole number spread evenly over the logarithm of [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "gradient", "append", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 256])
    group, page = rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([16, 32, 64])
    if op in ("norm", "gradient"):
        heads = kv_heads * group
        most = 8192 * 40 * 128 // ((heads + kv_heads) * dim * (2 if dtype == "f32" else 1))
        c = _norm("", op, _between(rng, 1, min(16384, most)), heads, kv_heads, dim, dtype,
                  rng.choice([dim, dim, dim // 2, dim // 4]), rng.choice([False, True]))
    elif op == "append":
        batch = _between(rng, 1, 64)
        tokens = rng.choice([1, _between(rng, 1, 8), _between(rng, 1, max(1, 8192 // batch))])
        c = _stretch("", op, batch, rng.choice([0, _between(rng, 1, 8191)]), tokens, kv_heads, dim,
                     page, dtype, rng.choice([0, dim, dim // 2]))
    elif op == "read":
        batch = _between(rng, 1, 64)
        tokens = _between(rng, 1, max(1, 65536 * 1024 // (batch * kv_heads * dim * (2 if dtype == "f32" else 1))))
        c = _stretch("", op, batch, rng.choice([0, _between(rng, 1, 8191)]), min(tokens, 65536),
                     kv_heads, dim, page, dtype)
    else:
        batch = _between(rng, 1, 64)
        length = _between(rng, 1, min(131072, 524288 * 1024 // (batch * kv_heads * dim)))
        # Chunks stay below the work of the largest listed one.
        most = int(2.2e11 / (4.0 * dim * kv_heads * group * batch * length))
        tokens = rng.choice([1, 1, _between(rng, 1, 8), _between(rng, 1, 2048)])
        c = _attend("", batch, length, max(1, min(tokens, length, most)), kv_heads * group, kv_heads,
                    dim, page, dtype, rng.choice([0, 0, 0, _between(rng, 16, 8192)]),
                    rng.choice([0, dim]))
    c.pop("name", None)
    return c


def _spread(n, low, high):
    """n whole numbers over [low, high], the first one `high`; the same in every run."""
    return [high - (high - low) * (i * 7919 % 997) // 997 for i in range(n)]


def _counts(case):
    """Tokens of each sequence that the call takes, and how many the sequence holds before
    them (append, read) or with them (attend)."""
    n = case["batch"]
    tokens = _spread(n, 1, case["tokens"])
    if case["op"] != "attend":
        return tokens, _spread(n, case["start"] // 4, case["start"])
    return tokens, [max(t, v) for t, v in zip(tokens, _spread(n, (case["length"] + 3) // 4, case["length"]))]


def _pairs(case):
    """Pairs of a query and a key that it reads, summed over the sequences (one head)."""
    total, window = 0, case["window"]
    for t, length in zip(*_counts(case)):
        first = length - t + 1  # keys that the first of the t queries sees
        if not window or window >= length:
            total += t * (first + length) // 2
        else:
            total += sum(min(window, first + i) for i in range(t))
    return total


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op, dim, heads = case["op"], case["dim"], case["kv_heads"]
    if op in ("norm", "gradient"):
        tokens, all_heads = case["tokens"], case["heads"] + heads
        elements, passes = tokens * all_heads * dim, 2 if op == "norm" else 3
        angles = tokens * (case["rotated"] * 4 + 4)
        weights = 2 * dim * 4 * (1 if op == "norm" else 2)
        return {"bytes": elements * size * passes + angles + weights,
                "flops": elements * (7 if op == "norm" else 16)}
    held = dim // 2 + 4  # bytes of a token's keys (values) of one head
    tokens, counts = _counts(case)
    if op == "append":
        rows = sum(tokens) * heads * 2
        return {"bytes": rows * (2 * dim * size + held) + sum(tokens) * case["rotated"] * 4,
                "flops": rows * dim * 8}
    if op == "read":
        rows = sum(tokens) * heads * 2
        return {"bytes": rows * (dim * size + held), "flops": rows * dim * 2}
    window = case["window"]
    read = sum(min(n, window + t - 1) if window else n for t, n in zip(tokens, counts))
    return {"bytes": read * heads * 2 * held + sum(tokens) * case["heads"] * (dim * 2 * size + 4)
            + sum(tokens) * case["rotated"] * 4,
            "flops": 4 * dim * case["heads"] * _pairs(case)}


# ------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _rope_table(positions, rotated):
    """cos and sin of position * base^(-2i / rotated), [positions, rotated / 2]."""
    i = torch.arange(0, rotated, 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * ROPE_BASE ** (-i / rotated)
    return a.cos().float(), a.sin().float()


def _index(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(g, case, lengths):
    """A cache in use: its pages in no order, codes and scales as they are there."""
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table, at = torch.full((len(lengths), max(need) + 1), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    shape = total, heads, page, dim // 2
    codes = []
    for _ in range(2):
        low, high = ((_randn(g, *shape, dtype=torch.float16) * 2.8 + 8).round_().clamp_(0, 15).to(torch.uint8)
                     for _ in range(2))
        codes.append(low + high * 16)
    scales = [(torch.rand(total, heads, page, generator=g, device="cuda") + 0.5) * c for c in (0.4, 0.1)]
    return {"k_codes": codes[0], "k_scales": scales[0], "v_codes": codes[1], "v_scales": scales[1],
            "page_table": table.cuda()}


def _prepare_norm(s, g, dtype):
    case = s["case"]
    tokens, heads, kv_heads, dim = (case[n] for n in ("tokens", "heads", "kv_heads", "dim"))
    # Slices of the q/k/v product; some channels are larger than the others in every model.
    gain = _randn(g, heads + 2 * kv_heads, dim).mul(0.4).exp()
    x = (_randn(g, tokens, heads + 2 * kv_heads, dim) * gain).to(dtype)
    s["q"], s["k"] = x[:, :heads], x[:, heads:heads + kv_heads]
    s["q_weight"], s["k_weight"] = (1 + 0.2 * _randn(g, dim) for _ in range(2))
    # Texts packed one behind the other, each from position 0 or from a held prefix.
    first = int(torch.randint(0, 1024, (1,), generator=g, device="cuda"))
    s["positions"] = ((torch.arange(tokens, device="cuda") + first) % 5000).int()
    s["rope"] = _rope_table(5000, case["rotated"])
    if case["op"] == "gradient":
        s["d_q"] = (_randn(g, tokens, heads, dim) * 0.01).to(dtype)
        s["d_k"] = (_randn(g, tokens, kv_heads, dim) * 0.03).to(dtype)


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("norm", "gradient"):
        _prepare_norm(s, g, dtype)
    else:
        tokens, counts = _counts(case)
        offsets = [0]
        for t in tokens:
            offsets.append(offsets[-1] + t)
        ends = counts if case["op"] == "attend" else [c + t for c, t in zip(counts, tokens)]
        s.update(_cache(g, case, ends))
        s.update(offsets=_index(offsets), most=max(tokens), total=offsets[-1], rope=None)
        if case["rotated"]:
            s["rope"] = _rope_table(max(ends), case["rotated"])
        if case["op"] == "attend":
            # Normalised queries: about one per channel, some channels larger than others.
            gain = _randn(g, case["heads"], case["dim"]).mul(0.3).exp()
            s["query"] = (_randn(g, offsets[-1], case["heads"], case["dim"]) * gain).to(dtype)
            s["lengths"] = _index(counts)
        else:
            s["starts"] = _index(counts)
        if case["op"] == "append":
            gain = _randn(g, case["kv_heads"], case["dim"]).mul(0.4).exp()
            s["k"] = (_randn(g, offsets[-1], case["kv_heads"], case["dim"]) * gain).to(dtype)
            s["v"] = (_randn(g, offsets[-1], case["kv_heads"], case["dim"]) * 0.4).to(dtype)
    if own:
        from bit_weight_quantized_int4_gb300 import q4lin
        if not _handles:
            _handles.append(q4lin.Handle(0))
        s["handle"] = _handles[0]
        if "k_codes" in s:
            s["cache"] = q4lin.KVCache4(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                        s["page_table"])
    return s


# --------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, interleaved=False):
    """Channel i of the first half with channel i of the second (or neighbours); the rest
    as it is."""
    half = cos.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turned[..., ::2], turned[..., 1::2]) if interleaved else (turned[..., :half], turned[..., half:])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, rest], -1)


def _angles(s):
    position = s["positions"].long()
    return s["rope"][0][position][:, None], s["rope"][1][position][:, None]


def _plain_norm(s):
    cos, sin = _angles(s)
    out = {}
    for n in ("q", "k"):
        x = s[n].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[n + "_weight"]
        out[n] = _rotate(x, cos, sin, s["case"]["interleaved"]).to(s[n].dtype)
    return out


def _plain_gradient(s):
    cos, sin = _angles(s)
    out = {}
    for n in ("q", "k"):
        x = s[n].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        g = _rotate(s["d_" + n].float(), cos, -sin, s["case"]["interleaved"])
        unit = x * r
        out["d_" + n + "_weight"] = (g * unit).sum(0).sum(0)
        g = g * s[n + "_weight"]
        out["d_" + n] = (r * (g - unit * (g * unit).mean(-1, keepdim=True))).to(s[n].dtype)
    return out


def _places(offsets, count):
    """Of each token: its sequence, and its place among the sequence's tokens of the call."""
    token = torch.arange(count, device="cuda")
    sequence = torch.searchsorted(offsets[1:].contiguous(), token.int(), right=True)
    return sequence, token - offsets[sequence].long()


def _slots(s):
    """Of each token: its page, its slot there and its position."""
    page = s["case"]["page"]
    sequence, place = _places(s["offsets"], s["total"])
    position = s["starts"].long()[sequence] + place
    return s["page_table"].long()[sequence, position // page], position % page, position


def _values(codes, scales):
    """What codes [..., dim / 2] with scales [...] stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return (c.float() - 8) * scales[..., None]


def _plain_append(s):
    pages, slot, position = _slots(s)
    k, v = s["k"].float(), s["v"].float()
    if s["rope"] is not None:
        cos, sin = s["rope"]
        k = _rotate(k, cos[position][:, None], sin[position][:, None])
    result = {}
    for n, x in (("k", k), ("v", v)):
        scale = x.abs().amax(-1) * (1.0 / 7.5)
        inverse = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
        c = (torch.round(x * inverse[..., None]).clamp(-8, 7) + 8).to(torch.uint8)
        s[n + "_codes"][pages, :, slot] = c[..., ::2] + c[..., 1::2] * 16
        s[n + "_scales"][pages, :, slot] = scale
        result[n + "_scales"] = s[n + "_scales"]
    result.update(_plain_read(s, pages, slot))
    return result


def _plain_read(s, pages=None, slot=None):
    if pages is None:
        pages, slot, _ = _slots(s)
    dtype = DTYPES[s["case"]["dtype"]]
    return {n: _values(s[n + "_codes"][pages, :, slot], s[n + "_scales"][pages, :, slot]).to(dtype)
            for n in ("k", "v")}


def _plain_attend(s):
    case = s["case"]
    batch, page, heads, dim = case["batch"], case["page"], case["kv_heads"], case["dim"]
    group, most, window = case["heads"] // heads, s["most"], case["window"]
    sequence, place = _places(s["offsets"], s["total"])
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    counts = offsets[1:] - offsets[:-1]
    position = (lengths - counts)[sequence] + place
    q = s["query"].float()
    if s["rope"] is not None:
        q = _rotate(q, s["rope"][0][position][:, None], s["rope"][1][position][:, None])
    dense = torch.zeros(batch, most, heads, group, dim, device="cuda")
    dense[sequence, place] = q.view(-1, heads, group, dim)
    dense = dense.permute(0, 2, 1, 3, 4).reshape(batch, heads, most * group, dim)
    pages = s["page_table"].long().clamp(min=0)
    span = pages.shape[1] * page
    k = _values(s["k_codes"][pages], s["k_scales"][pages])
    k = k.permute(0, 2, 1, 3, 4).reshape(batch, heads, span, dim)
    score = torch.matmul(dense, k.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    del k
    key = torch.arange(span, device="cuda")[None, None]
    at = ((lengths - counts)[:, None] + torch.arange(most, device="cuda")[None])[:, :, None]
    seen = (key <= at) & (key < lengths[:, None, None])
    if window:
        seen = seen & (key > at - window)
    score = score.view(batch, heads, most, group, span)
    score = torch.where(seen[:, None, :, None], score, torch.full((), -math.inf, device="cuda"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = (score - top).exp()
    del score
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    v = _values(s["v_codes"][pages], s["v_scales"][pages])
    v = v.permute(0, 2, 1, 3, 4).reshape(batch, heads, span, dim)
    o = torch.matmul(p.view(batch, heads, most * group, span), v).view(batch, heads, most, group, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    out = o.permute(0, 2, 1, 3, 4).reshape(batch, most, heads * group, dim)[sequence, place]
    lse = lse.permute(0, 2, 1, 3).reshape(batch, most, heads * group)[sequence, place]
    return {"out": out.to(s["query"].dtype), "lse": lse}


_PLAIN = {"norm": _plain_norm, "gradient": _plain_gradient, "append": _plain_append,
          "read": _plain_read, "attend": _plain_attend}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](s)
    from bit_weight_quantized_int4_gb300 import q4lin
    handle = s["handle"]
    if op == "norm":
        q, k = q4lin.norm_rope(handle, s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                               s["rope"], eps=EPS, interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "gradient":
        r = q4lin.norm_rope_backward(handle, s["q"], s["k"], s["q_weight"], s["k_weight"],
                                     s["positions"], s["rope"], s["d_q"], s["d_k"], eps=EPS,
                                     interleaved=case["interleaved"])
        return {"d_q_weight": r.d_q_weight, "d_q": r.d_q, "d_k_weight": r.d_k_weight, "d_k": r.d_k}
    if op == "attend":
        out, lse = q4lin.attention(handle, s["cache"], s["query"], s["offsets"], s["lengths"],
                                   1.0 / math.sqrt(case["dim"]), max_query=s["most"],
                                   rope=s["rope"], window=case["window"])
        return {"out": out, "lse": lse}
    result = {}
    if op == "append":
        q4lin.kv_append(handle, s["cache"], s["k"], s["v"], s["offsets"], s["starts"], rope=s["rope"])
        result = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    k, v = q4lin.kv_read(handle, s["cache"], s["offsets"], s["starts"], s["total"],
                         dtype=DTYPES[case["dtype"]])
    result.update(k=k, v=v)
    return result


# ----------------------------------------------------------------- the definitions, 64 bits
def _turn(x, position, rope, interleaved=False):
    """Rotation of x [tokens, heads, dim] as the product of complex numbers, in 64 bits."""
    half = rope[0].shape[1]
    turn = torch.complex(rope[0].double(), rope[1].double())[position][:, None]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., 2 * half:]], -1)
    z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
    return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)


def _exact_norm(s):
    return {n: _turn(_normed(s[n].double(), s[n + "_weight"].double()), s["positions"].long(), s["rope"],
                     s["case"]["interleaved"]) for n in ("q", "k")}


def _normed(x, weight):
    return x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / x.shape[-1] + EPS) * weight


def _exact_gradient(s):
    # By differentiating the definition, in stretches of tokens that fit.
    parts = {n: [] for n in ("d_q", "d_k")}
    result = {}
    for n in ("q", "k"):
        weight = s[n + "_weight"].double().requires_grad_()
        for x, d, position in zip(s[n].split(1024), s["d_" + n].split(1024), s["positions"].split(1024)):
            x = x.double().requires_grad_()
            y = _turn(_normed(x, weight), position.long(), s["rope"], s["case"]["interleaved"])
            y.backward(d.double())
            parts["d_" + n].append(x.grad)
        result["d_" + n + "_weight"] = weight.grad
        result["d_" + n] = torch.cat(parts["d_" + n])
    return result


def _exact_append(s):
    # A scale is defined for every value; a code follows from the rounded steps alone.
    case = s["case"]
    offsets, starts, table = s["offsets"].tolist(), s["starts"].tolist(), s["page_table"].long()
    scales = {n: s[n + "_scales"].double() for n in ("k", "v")}
    for b in range(case["batch"]):
        position = torch.arange(starts[b], starts[b] + offsets[b + 1] - offsets[b], device="cuda")
        new = {n: s[n][offsets[b]:offsets[b + 1]].double() for n in ("k", "v")}
        if s["rope"] is not None:
            new["k"] = _turn(new["k"], position, s["rope"])
        for n, x in new.items():
            scales[n][table[b, position // case["page"]], :, position % case["page"]] = x.abs().amax(-1) / 7.5
    return {"k_scales": scales["k"], "v_scales": scales["v"], "k": None, "v": None}


def _unpacked(codes, scales):
    c = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    c[..., ::2], c[..., 1::2] = codes % 16, torch.div(codes, 16, rounding_mode="floor")
    return (c - 8) * scales.double()[..., None]


def _exact_read(s):
    case, parts = s["case"], {"k": [], "v": []}
    offsets, starts = s["offsets"].tolist(), s["starts"].tolist()
    for b in range(case["batch"]):
        end = starts[b] + offsets[b + 1] - offsets[b]
        pages = s["page_table"][b, starts[b] // case["page"]:-(-end // case["page"])].long()
        low = starts[b] % case["page"]
        for n, rows in parts.items():
            x = _unpacked(s[n + "_codes"][pages], s[n + "_scales"][pages])
            x = x.transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])
            rows.append(x[low:low + end - starts[b]])
    return {n: torch.cat(rows) for n, rows in parts.items()}


def _exact_attend(s):
    case = s["case"]
    heads, dim, window = case["kv_heads"], case["dim"], case["window"]
    group = case["heads"] // heads
    offsets, lengths, table = s["offsets"].tolist(), s["lengths"].tolist(), s["page_table"].long()
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["query"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        first, count, length = offsets[b], offsets[b + 1] - offsets[b], lengths[b]
        position = torch.arange(length - count, length, device="cuda")
        q = s["query"][first:first + count].double()
        if s["rope"] is not None:
            q = _turn(q, position, s["rope"])
        pages = table[b, :-(-length // case["page"])]
        low = max(0, length - count - window + 1) if window else 0
        key = torch.arange(low, length, device="cuda")
        hidden = key[None] > position[:, None]
        if window:
            hidden |= key[None] <= position[:, None] - window
        for h in range(heads):
            k, v = (_unpacked(s[n + "_codes"][pages, h], s[n + "_scales"][pages, h]).reshape(-1, dim)[low:length]
                    for n in ("k", "v"))
            for i in range(h * group, (h + 1) * group):
                x = (q[:, i] @ k.T / math.sqrt(dim)).masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                out[first:first + count, i] = (x - z[:, None]).exp_() @ v
                lse[first:first + count, i] = z
    return {"out": out, "lse": lse}


def exact(case, seed):
    return {"norm": _exact_norm, "gradient": _exact_gradient, "append": _exact_append,
            "read": _exact_read, "attend": _exact_attend}[case["op"]](prepare(case, seed))

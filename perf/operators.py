"""The operators around the 4-bit linears of a decoder, as they are measured: what goes
into each, what comes out, and the same results from elementary torch operations.

  append     keys and values appended to a paged 8-bit cache, the keys rotated on the way
  attend     attention over that cache: one token a sequence, a few, or a prompt's chunk
  logprobs   log probability of a given token, entropy and the top alternatives per row
  gradient   the gradient of those two for the logits

With `own` false, run() computes them in plain torch, in 32 bits; with `own` true it calls
the framework.  A cache holds, for each page of `page` tokens and each key-value head,
keys [page, dim] and values [dim, page] as bytes, and a scale for each: a byte c stands
for (c - 128) * scale.  The bytes are whole numbers that the definition fixes (every
step rounds once, in a given order), so they come back as they are and have to be equal.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROPE_BASE = 500000.0
_handles = []


def _append(name, batch, start, tokens, kv_heads, dim, page, dtype, rotated=None):
    return {"name": name, "op": "append", "batch": batch, "start": start, "tokens": tokens,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "rotated": dim if rotated is None else rotated}


def _attend(name, batch, length, tokens, heads, kv_heads, dim, page, dtype, window=0):
    return {"name": name, "op": "attend", "batch": batch, "length": length, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "window": window}


def listed():
    return [
        # One conversation, one token: the 1B shape's key and value projections (512 wide).
        _append("append_one", 1, 700, 1, 8, 64, 16, "f32"),
        # A decode step of 64 conversations of different lengths, the 8B shape.
        _append("append_step", 64, 4095, 1, 8, 128, 64, "bf16"),
        # Seven prompts of odd lengths written in one call, as q4lin_run gives them (fp32).
        _append("append_prompts", 7, 0, 2047, 8, 128, 64, "f32"),
        # One token over a short conversation, the 1B shape: latency.
        _attend("attend_one", 1, 701, 1, 32, 8, 64, 16, "f32"),
        # One token over one very long document, the 8B shape: the long axis is all there is.
        _attend("attend_long", 1, 131071, 1, 32, 8, 128, 64, "bf16"),
        # A decode step of 64 conversations of up to 8192 tokens, the 8B shape.
        _attend("attend_batch", 64, 8192, 1, 32, 8, 128, 64, "f32"),
        # One to five draft tokens a sequence, seven heads to a key head, a sliding window.
        _attend("attend_draft", 9, 5003, 5, 28, 4, 128, 32, "f16", window=1024),
        # The last 2048 tokens of an 8192-token prompt that is read in chunks, the 8B shape.
        _attend("attend_prompt", 1, 8192, 2048, 32, 8, 128, 64, "bf16"),
        # The sampled token of one conversation, with five alternatives.
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "vocabulary": 128256, "top": 5,
         "dtype": "f32"},
        # Scoring 1000 tokens of a text, with twenty alternatives; a vocabulary of odd size.
        {"name": "logprobs_rows", "op": "logprobs", "rows": 1000, "vocabulary": 128257,
         "top": 20, "dtype": "f32"},
        # The gradient for a few tokens, logits in 16 bits.
        {"name": "gradient_few", "op": "gradient", "rows": 8, "vocabulary": 128256,
         "dtype": "bf16"},
        # The gradient for a batch of texts, a vocabulary of odd size.
        {"name": "gradient_rows", "op": "gradient", "rows": 1000, "vocabulary": 128257,
         "dtype": "f32"},
    ]


def _between(rng, low, high):
    """A whole number spread evenly over the logarithm of [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs", "gradient"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("append", "attend"):
        kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 256])
        page = rng.choice([16, 32, 64])
    if op == "append":
        batch = _between(rng, 1, 64)
        tokens = rng.choice([1, _between(rng, 1, 8), _between(rng, 1, max(1, 8192 // batch))])
        c = _append("", batch, rng.choice([0, _between(rng, 1, 8191)]), tokens, kv_heads, dim, page,
                    dtype, rng.choice([dim, dim // 2]))
    elif op == "attend":
        group = rng.choice([1, 2, 3, 4, 7, 8])
        batch = _between(rng, 1, 64)
        length = _between(rng, 1, min(131072, 524288 * 1024 // (batch * kv_heads * dim)))
        # Chunks stay below the work of the largest listed one.
        most = int(2.2e11 / (4.0 * dim * kv_heads * group * batch * length))
        tokens = rng.choice([1, 1, _between(rng, 1, 8), _between(rng, 1, 2048)])
        tokens = max(1, min(tokens, length, most))
        c = _attend("", batch, length, tokens, kv_heads * group, kv_heads, dim, page, dtype,
                    rng.choice([0, 0, 0, _between(rng, 16, 8192)]))
    else:
        vocabulary = _between(rng, 1000, 131072)
        rows = _between(rng, 1, max(1, min(4096, 128000000 // vocabulary)))
        c = {"op": op, "rows": rows, "vocabulary": vocabulary, "dtype": dtype}
        if op == "logprobs":
            c["top"] = rng.choice([0, 1, 5, 20, 32])
    c.pop("name", None)
    return c


def _spread(n, low, high):
    """n whole numbers over [low, high], the first one `high`; the same in every run."""
    return [high - (high - low) * (i * 7919 % 997) // 997 for i in range(n)]


def _counts(case):
    """New tokens of each sequence, and the length before (append) or after (attend) them."""
    n = case["batch"]
    tokens = _spread(n, 1, case["tokens"])
    if case["op"] == "append":
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
    if case["op"] == "append":
        tokens, starts = _counts(case)
        rows, heads, dim, page = sum(tokens), case["kv_heads"], case["dim"], case["page"]
        pages = sum(-(-(s + t) // page) - s // page for s, t in zip(starts, tokens))
        return {"bytes": rows * heads * dim * 2 * (size + 1) + rows * case["rotated"] * 4
                + pages * heads * 2 * 8 + pages * 4, "flops": rows * heads * dim * 8}
    if case["op"] == "attend":
        tokens, lengths = _counts(case)
        heads, dim, window = case["heads"], case["dim"], case["window"]
        read = sum(min(n, window + t - 1) if window else n for t, n in zip(tokens, lengths))
        pages = sum(-(-n // case["page"]) for n in lengths)
        return {"bytes": read * case["kv_heads"] * dim * 2 + pages * case["kv_heads"] * 8
                + sum(tokens) * heads * (dim * 2 * size + 4) + sum(tokens) * dim * 4,
                "flops": 4 * dim * heads * _pairs(case)}
    rows, vocabulary = case["rows"], case["vocabulary"]
    if case["op"] == "logprobs":
        return {"bytes": rows * (vocabulary * size + 16 + 8 * case["top"]),
                "flops": 5 * rows * vocabulary}
    return {"bytes": rows * (2 * vocabulary * size + 20), "flops": 7 * rows * vocabulary}


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
    """A cache in use: its pages in no order, and bytes and scales as attention leaves them."""
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table, at = torch.full((len(lengths), max(need) + 1), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    codes = [(_randn(g, *shape, dtype=torch.float16) * 36 + 128).round_().clamp_(1, 255).to(torch.uint8)
             for shape in ((total, heads, page, dim), (total, heads, dim, page))]
    scales = [(torch.rand(total, heads, generator=g, device="cuda") + 1.5) * c for c in (0.02, 0.008)]
    return {"k_codes": codes[0], "k_scales": scales[0], "v_codes": codes[1], "v_scales": scales[1],
            "page_table": table.cuda()}


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("append", "attend"):
        tokens, counts = _counts(case)
        offsets = [0]
        for t in tokens:
            offsets.append(offsets[-1] + t)
        ends = [c + t for c, t in zip(counts, tokens)] if case["op"] == "append" else counts
        s.update(_cache(g, case, ends))
        s.update(offsets=_index(offsets), most=max(tokens))
        heads = case["kv_heads"] if case["op"] == "append" else case["heads"]
        # Some channels of keys and queries are larger than the others in every model.
        gain = _randn(g, heads, case["dim"]).mul(0.4).exp()
        x = (_randn(g, offsets[-1], heads, case["dim"]) * gain).to(dtype)
        if case["op"] == "append":
            v = (_randn(g, offsets[-1], heads, case["dim"]) * 0.4).to(dtype)
            s.update(k=x, v=v, starts=_index(counts))
            s["rope"] = _rope_table(max(ends), case["rotated"])
        else:
            s.update(query=x, lengths=_index(counts), rope=_rope_table(max(ends), case["dim"]))
    else:
        rows, vocabulary = case["rows"], case["vocabulary"]
        # Most words are unlikely, a few are not.
        x = _randn(g, rows, vocabulary) * 2.0
        likely = torch.randint(0, vocabulary, (rows, 8), generator=g, device="cuda")
        x.scatter_add_(1, likely, _randn(g, rows, 8) * 2.0 + 9.0)
        s["logits"] = x.to(dtype)
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, likely[:, 0],
                                  torch.randint(0, vocabulary, (rows,), generator=g, device="cuda")).int()
        if case["op"] == "gradient":
            y = s["logits"].float()
            lse = torch.logsumexp(y, 1)
            s["lse"] = lse
            s["entropy"] = lse - ((y - lse[:, None]).exp() * y).sum(1)
            s["d_logprob"] = -torch.rand(rows, generator=g, device="cuda")
            s["d_entropy"] = _randn(g, rows) * 0.1
    if own:
        from bit_weight_quantized_int4_gb300 import q4lin
        if not _handles:
            _handles.append(q4lin.Handle(0))
        s["handle"] = _handles[0]
        if "k_codes" in s:
            s["cache"] = q4lin.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                       s["page_table"])
    return s


# --------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin):
    """Channel i of the first half with channel i of the second; the rest as it is."""
    half = cos.shape[-1]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _places(offsets, count):
    """Of each token: its sequence, and its place among the sequence's new tokens."""
    token = torch.arange(count, device="cuda")
    sequence = torch.searchsorted(offsets[1:].contiguous(), token.int(), right=True)
    return sequence, token - offsets[sequence].long()


def _open_pages(codes, scales, grown, pages, keep):
    """Bytes of the open pages [batch, heads, a, b], rounded again where the scale grew."""
    old, new = scales[pages], grown[pages]
    c = codes[pages]
    ratio = torch.where(new > 0, old / new, torch.zeros_like(new))[..., None, None]
    again = torch.round((c.float() - 128) * ratio) + 128
    c = torch.where(keep & (new > old)[..., None, None], again.to(torch.uint8), c)
    codes[pages] = c


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    sequence, place = _places(s["offsets"], s["k"].shape[0])
    starts = s["starts"].long()
    position = starts[sequence] + place
    cos, sin = s["rope"]
    k = _rotate(s["k"].float(), cos[position][:, None], sin[position][:, None])
    v = s["v"].float()
    table = s["page_table"].long()
    pages, slot = table[sequence, position // page], position % page
    first = table[torch.arange(case["batch"], device="cuda"), starts // page]
    held = starts % page  # tokens that the open page of each sequence holds already
    older = torch.arange(page, device="cuda")[None] < held[:, None]
    for x, name, keep in ((k, "k", older[:, None, :, None]), (v, "v", older[:, None, None, :])):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        most = torch.full_like(scales, -1.0)
        most.scatter_reduce_(0, pages[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        kept = torch.zeros_like(scales)
        kept[first] = torch.where(held[:, None] > 0, scales[first], torch.zeros_like(scales[first]))
        grown = torch.where(most >= 0, torch.maximum(kept, most * (1.0 / 127.0)), scales)
        _open_pages(codes, scales, grown, first, keep)
        scales.copy_(grown)
        inverse = torch.where(grown > 0, 1.0 / grown, torch.zeros_like(grown))[pages]
        c = (torch.round(x * inverse[..., None]).clamp(-127, 127) + 128).to(torch.uint8)
        if name == "k":
            codes[pages, :, slot] = c
        else:
            codes[pages, :, :, slot] = c
    return _buffers(s)


def _buffers(s):
    return {n: s[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def _plain_attend(s):
    case = s["case"]
    batch, page, heads, dim = case["batch"], case["page"], case["kv_heads"], case["dim"]
    group, most, window = case["heads"] // heads, s["most"], case["window"]
    sequence, place = _places(s["offsets"], s["query"].shape[0])
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    counts = offsets[1:] - offsets[:-1]
    position = (lengths - counts)[sequence] + place
    cos, sin = s["rope"]
    q = _rotate(s["query"].float(), cos[position][:, None], sin[position][:, None])
    dense = torch.zeros(batch, most, heads, group, dim, device="cuda")
    dense[sequence, place] = q.view(-1, heads, group, dim)
    dense = dense.permute(0, 2, 1, 3, 4).reshape(batch, heads, most * group, dim)
    pages = s["page_table"].long().clamp(min=0)
    span = pages.shape[1] * page
    k = (s["k_codes"][pages].float() - 128) * s["k_scales"][pages][..., None, None]
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
    v = (s["v_codes"][pages].float() - 128) * s["v_scales"][pages][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, heads, span, dim)
    o = torch.matmul(p.view(batch, heads, most * group, span), v).view(batch, heads, most, group, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    out = o.permute(0, 2, 1, 3, 4).reshape(batch, most, heads * group, dim)[sequence, place]
    lse = lse.permute(0, 2, 1, 3).reshape(batch, most, heads * group)[sequence, place]
    return {"out": out.to(s["query"].dtype), "lse": lse}


def _plain_logprobs(s):
    x, top = s["logits"].float(), s["case"]["top"]
    most = x.amax(1, keepdim=True)
    e = (x - most).exp()
    total = e.sum(1, keepdim=True)
    lse = most + total.log()
    entropy = total.log()[:, 0] - (e * (x - most)).sum(1) / total[:, 0]
    result = {"logprob": x.gather(1, s["tokens"].long()[:, None])[:, 0] - lse[:, 0],
              "entropy": entropy, "lse": lse[:, 0]}
    if top:
        best, token = torch.sort(x, dim=1, descending=True, stable=True)
        result["top_tokens"] = token[:, :top].int()
        result["top_logprobs"] = best[:, :top] - lse
    return result


def _plain_gradient(s):
    x = s["logits"].float() - s["lse"][:, None]
    p = x.exp()
    d = p * -(s["d_logprob"][:, None] + s["d_entropy"][:, None] * (x + s["entropy"][:, None]))
    d.scatter_add_(1, s["tokens"].long()[:, None], s["d_logprob"][:, None])
    return {"d_logits": d.to(s["logits"].dtype)}


_PLAIN = {"append": _plain_append, "attend": _plain_attend, "logprobs": _plain_logprobs,
          "gradient": _plain_gradient}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    from bit_weight_quantized_int4_gb300 import q4lin
    if op == "append":
        q4lin.kv_append(s["handle"], s["cache"], s["k"], s["v"], s["offsets"], s["starts"],
                        rope=s["rope"])
        return _buffers(s)
    if op == "attend":
        out, lse = q4lin.attention(s["handle"], s["cache"], s["query"], s["offsets"], s["lengths"],
                                   1.0 / math.sqrt(s["case"]["dim"]), max_query=s["most"],
                                   rope=s["rope"], window=s["case"]["window"])
        return {"out": out, "lse": lse}
    if op == "logprobs":
        r = q4lin.logprobs(s["handle"], s["logits"], s["tokens"], top=s["case"]["top"])
        result = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if s["case"]["top"]:
            result.update(top_tokens=r.top_tokens, top_logprobs=r.top_logprobs)
        return result
    return {"d_logits": q4lin.logprobs_backward(s["handle"], s["logits"], s["tokens"], s["lse"],
                                                s["entropy"], s["d_logprob"], s["d_entropy"])}


# ----------------------------------------------------------------- the definitions, 64 bits
def _turn(x, position, rope):
    """Rotation of x [tokens, heads, dim] as the product of complex numbers, in 64 bits."""
    half = rope[0].shape[1]
    turn = torch.complex(rope[0].double(), rope[1].double())[position][:, None]
    z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
    return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)


def _exact_append(s):
    case, page = s["case"], s["case"]["page"]
    offsets, starts, table = s["offsets"].tolist(), s["starts"].tolist(), s["page_table"].tolist()
    scales = {n: s[n + "_scales"].double() for n in ("k", "v")}
    for b in range(case["batch"]):
        first, count = offsets[b], offsets[b + 1] - offsets[b]
        position = torch.arange(starts[b], starts[b] + count, device="cuda")
        new = {"k": _turn(s["k"][first:first + count].double(), position, s["rope"]),
               "v": s["v"][first:first + count].double()}
        for p in range(starts[b] // page, (starts[b] + count - 1) // page + 1):
            low, high = max(p * page, starts[b]) - starts[b], min((p + 1) * page, starts[b] + count) - starts[b]
            for n, x in new.items():
                most = x[low:high].abs().amax((0, 2)) / 127.0
                if p * page < starts[b]:
                    most = torch.maximum(most, scales[n][table[b][p]])
                scales[n][table[b][p]] = most
    return {"k_codes": None, "k_scales": scales["k"], "v_codes": None, "v_scales": scales["v"]}


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
        q = _turn(s["query"][first:first + count].double(), position, s["rope"])
        pages = table[b, :-(-length // case["page"])]
        low = max(0, length - count - window + 1) if window else 0
        key = torch.arange(low, length, device="cuda")
        hidden = key[None] > position[:, None]
        if window:
            hidden |= key[None] <= position[:, None] - window
        for h in range(heads):
            k = (s["k_codes"][pages, h].double() - 128) * s["k_scales"][pages, h].double()[:, None, None]
            v = (s["v_codes"][pages, h].double() - 128) * s["v_scales"][pages, h].double()[:, None, None]
            k = k.reshape(-1, dim)[low:length]
            v = v.transpose(1, 2).reshape(-1, dim)[low:length]
            for i in range(h * group, (h + 1) * group):
                x = (q[:, i] @ k.T / math.sqrt(dim)).masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                out[first:first + count, i] = (x - z[:, None]).exp_() @ v
                lse[first:first + count, i] = z
    return {"out": out, "lse": lse}


def _exact_logprobs(s):
    top, parts = s["case"]["top"], []
    for x, token in zip(s["logits"].split(64), s["tokens"].long().split(64)):
        x = torch.log_softmax(x.double(), 1)
        r = {"logprob": x.gather(1, token[:, None])[:, 0], "entropy": -(x.exp() * x).sum(1)}
        if top:
            r["top_logprobs"] = torch.topk(x, top, 1).values
        parts.append(r)
    lse = torch.cat([torch.logsumexp(x.double(), 1) for x in s["logits"].split(64)])
    result = {n: torch.cat([r[n] for r in parts]) for n in parts[0]}
    result["lse"] = lse
    if top:
        result["top_tokens"] = None
    return result


def _exact_gradient(s):
    # The gradient as defined for the normalisation and the entropy that the call is given.
    parts = []
    for i in range(0, s["logits"].shape[0], 64):
        x = s["logits"][i:i + 64].double() - s["lse"][i:i + 64, None].double()
        a, b = s["d_logprob"][i:i + 64, None].double(), s["d_entropy"][i:i + 64, None].double()
        d = torch.nn.functional.one_hot(s["tokens"][i:i + 64].long(), x.shape[1]) * a
        parts.append(d - x.exp() * (a + b * (x + s["entropy"][i:i + 64, None].double())))
    return {"d_logits": torch.cat(parts)}


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs,
            "gradient": _exact_gradient}[case["op"]](prepare(case, seed))

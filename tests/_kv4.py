"""Plain float64 (numpy) forms of the 4-bit cache's operators and of the norms with rotation,
written from their definitions."""
import numpy as np

from tests import _operators as ops


class Cache(ops.Cache):
    """A 4-bit cache on the host: codes [page, head, slot, dim] unpacked, scales [page, head, slot]."""

    def __init__(self, rng, lengths, kv_heads, page, dim, spare=2, filled=True):
        super().__init__(rng, lengths, kv_heads, page, dim, spare, False)
        shape = self.total, kv_heads, page, dim
        if filled:
            draw = lambda: np.clip(np.rint(rng.standard_normal(shape) * 3 + 8), 0, 15).astype(np.uint8)
            self.k, self.v = draw(), draw()
            self.ks = rng.uniform(0.1, 0.7, shape[:3]).astype(np.float32)
            self.vs = rng.uniform(0.05, 0.3, shape[:3]).astype(np.float32)
        else:
            self.k, self.v = np.full(shape, 8, np.uint8), np.full(shape, 8, np.uint8)
            self.ks, self.vs = np.zeros(shape[:3], np.float32), np.zeros(shape[:3], np.float32)

    def device(self):
        from bit_weight_quantized_int4_gb300 import q4lin
        pack = lambda c: ops.to_device(c[..., ::2] + 16 * c[..., 1::2])
        return q4lin.KVCache4(pack(self.k), ops.to_device(self.ks), pack(self.v), ops.to_device(self.vs),
                              ops.to_device(self.table))

    def _rows(self, codes, scales, b, n, h):
        p = self.table[b, :-(-n // self.page)]
        with np.errstate(all="ignore"):
            x = (codes[p, h].astype(np.float64) - 8) * scales[p, h].astype(np.float64)[..., None]
        return x.reshape(-1, self.dim)[:n]

    def keys(self, b, n, h):
        return self._rows(self.k, self.ks, b, n, h)

    def values(self, b, n, h):
        return self._rows(self.v, self.vs, b, n, h)


class DeviceCache(Cache):
    """A device cache's contents after a call."""

    def __init__(self, cache):
        unpack = lambda t: np.stack([t.cpu().numpy() & 15, t.cpu().numpy() >> 4], -1).reshape(*t.shape[:3], -1)
        self.k, self.v = unpack(cache.k_codes), unpack(cache.v_codes)
        self.ks, self.vs = cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()
        self.table = cache.page_table.cpu().numpy()
        self.total, self.heads, self.page, self.dim = self.k.shape


def quantise(x):
    """(codes, scales) of float32 rows, in the fp32 steps that fix them."""
    f = np.float32
    with np.errstate(all="ignore"):
        size = np.abs(x)
        amax = np.where(np.isfinite(size), size, f(0)).max(-1)
        scale = amax * f(1.0 / 7.5)
        scale = np.where(scale >= f(2.0**-126), scale, f(0)).astype(f)
        inverse = np.where(scale > 0, f(1) / scale, f(0)).astype(f)
        c = np.rint(x * inverse[..., None])
        c = np.where(np.isnan(c), 0, np.clip(c, -8, 7)) + 8
    return c.astype(np.uint8), scale


def append(cache, k, v, offsets, starts, rope=None, interleaved=False):
    """The append's definition on the host cache."""
    for b in range(len(starts)):
        for i in range(offsets[b + 1] - offsets[b]):
            position = starts[b] + i
            row = slice(offsets[b] + i, offsets[b] + i + 1)
            page, slot = cache.table[b, position // cache.page], position % cache.page
            with np.errstate(all="ignore"):
                x = ops.rotate(k[row], np.array([position]), rope, interleaved, np.float32)[0]
            cache.k[page, :, slot], cache.ks[page, :, slot] = quantise(x)
            cache.v[page, :, slot], cache.vs[page, :, slot] = quantise(v[row][0].astype(np.float32))


def rotate_back(x, position, rope, interleaved):
    return ops.rotate(x, position, None if rope is None else (rope[0], -rope[1]), interleaved)


def norm_rope(x, weight, position, rope, eps, interleaved):
    """(y, the size of the two terms behind each element of it) of x [tokens, heads, dim]."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r * weight
    size = u if rope is None else ops.rotate(np.abs(u), position, (np.abs(rope[0]), -np.abs(rope[1])), interleaved)
    other = np.abs(u) if rope is None else ops.rotate(np.abs(u), position, (np.abs(rope[0]), np.abs(rope[1])), interleaved)
    return ops.rotate(u, position, rope, interleaved), np.maximum(np.abs(size), np.abs(other))


def norm_rope_backward(x, weight, position, rope, eps, interleaved, d):
    """(d_x, d_weight, bounds of what their terms add up to)."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r
    g = rotate_back(d, position, rope, interleaved)
    back = lambda sign: np.abs(ops.rotate(np.abs(d), position, None if rope is None else
                                          (np.abs(rope[0]), sign * np.abs(rope[1])), interleaved))
    size = np.maximum(back(1), back(-1))
    gw = g * weight
    d_x = r * (gw - u * (gw * u).mean(-1, keepdims=True))
    d_x_size = r * (size * np.abs(weight) + np.abs(u) * (size * np.abs(weight * u)).mean(-1, keepdims=True))
    return d_x, (g * u).sum((0, 1)), d_x_size, (size * np.abs(u)).sum((0, 1))

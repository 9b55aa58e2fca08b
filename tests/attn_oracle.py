"""Plain forms of the attention operators: rotations and attention in 64 bits, the cache's codes bit for bit in FP32, and
the error bounds that the kernels are held to.

U is half a step of FP32.  FP16's half step is 2^-11, E4M3's 2^-4 relative (2^-10 below 2^-6).
"""
import math

import torch

from ffn_oracle import HALF, TINY, U, assert_within  # noqa: F401

LARGEST = {"int8": 127.0, "e4m3": 448.0}
PLACE = [(t >> 2 & 1) * 16 + (t >> 4) * 8 + (t >> 3 & 1) * 4 + (t & 3) for t in range(32)]


# ---- rotary ------------------------------------------------------------------------
def rotate(x, positions, table, interleaved=False, amplitude=1.0, way=1):
    """x [tokens, heads, dim] turned by way * 2 pi positions table, 64 bits."""
    x, half = x.double(), table.numel()
    t = positions.double()[:, None] * table.double()
    t = (t - t.round())[:, None] * (2 * math.pi)
    c, s = torch.cos(t) * amplitude, torch.sin(t) * amplitude * way
    y = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def rotate_bound(x, table, interleaved=False, amplitude=1.0):
    """The reduced angle is off by half a step of FP32 at half a turn (2^-25 turns, 2 pi 2^-25 = 3.2 U radians) and its
    cosine and sine by two steps (4 U); times the amplitude, a product and a sum: 3 U more."""
    x, half = x.double().abs(), table.numel()
    e = torch.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    e[..., a] = e[..., b] = (x[..., a] + x[..., b]) * abs(amplitude) * 10.2 * U + TINY
    return e


# ---- the cache -----------------------------------------------------------------------
def value_of(codes, fmt):
    return codes.contiguous().view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def code_of(y, fmt):
    y = torch.nan_to_num(y, nan=0.0, posinf=LARGEST[fmt], neginf=-LARGEST[fmt]).clamp(-LARGEST[fmt], LARGEST[fmt])
    return y.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else y.round().to(torch.int8).view(torch.uint8)


class Cache:
    """The cache as include/iq.h describes it, on the CPU: codes and scales in their layout."""

    def __init__(self, codes, scales, fmt, heads, dim, page):
        self.codes, self.scales, self.fmt, self.heads, self.dim, self.page = codes.cpu().clone(), scales.cpu().clone(), fmt, heads, dim, page

    def block(self, page, head, block, which):
        """Codes [32, dim] of a block, a copy."""
        c = self.codes[page, head, block, which]
        return (c.view(self.dim // 16, 32, 16).transpose(0, 1).reshape(32, self.dim) if which == 0
                else c.view(self.dim, 32)[:, PLACE].t()).contiguous()

    def store(self, page, head, block, which, codes):
        if which == 0:
            c = codes.view(32, self.dim // 16, 16).transpose(0, 1)
        else:
            c = torch.empty(self.dim, 32, dtype=torch.uint8)
            c[:, PLACE] = codes.t()
        self.codes[page, head, block, which] = c.reshape(-1)

    def page_of(self, row, position):
        entry = position // self.page
        page = int(row[entry]) if entry < len(row) else -1
        return page if 0 <= page < self.codes.shape[0] else None

    def append(self, k, v, page_table, lengths, starts=None):
        """k and v FP32 [tokens, heads, dim], already turned."""
        for b, length in enumerate(lengths):
            length = max(length, 0)
            lo, hi = (starts[b], min(starts[b + 1], k.shape[0])) if starts is not None else (b, b + 1)
            first = length - (hi - lo)
            for block in range(max(first, 0) // 32, -(-length // 32) if hi > lo else 0):
                page = self.page_of(page_table[b], 32 * block)
                if page is None:
                    continue
                inside = block % (self.page // 32)
                at, to = max(first - 32 * block, 0), min(length - 32 * block, 32)
                rows = slice(lo + 32 * block + at - first, lo + 32 * block + to - first)
                for head in range(self.heads):
                    for which, x in enumerate((k, v)):
                        self._append(page, head, inside, which, x[rows, head].float(), at, to)

    def _append(self, page, head, block, which, x, at, to):
        codes, had = self.block(page, head, block, which), self.scales[page, head, block, which].item() if at > 0 else 0.0
        finite = torch.where(torch.isfinite(x), x.abs(), torch.zeros(()))
        scale, up = finite.amax() / torch.tensor(LARGEST[self.fmt]), 0
        if had > 0:
            if scale.item() > had:
                up = 0
                while math.ldexp(had, up) < scale.item():
                    up += 1
            scale = torch.tensor(math.ldexp(had, up), dtype=torch.float32)
            codes[:at] = code_of(torch.ldexp(value_of(codes[:at], self.fmt), torch.tensor(-up)), self.fmt)
        codes[at:to] = code_of(x / scale, self.fmt) if scale > 0 else 0
        self.store(page, head, block, which, codes)
        self.scales[page, head, block, which] = scale

    def values(self, row, count):
        """Keys and values [count, heads, dim] of a sequence's first tokens, FP32; tokens of absent pages NaN."""
        out = torch.full((2, count, self.heads, self.dim), float("nan"))
        for block in range(-(-count // 32)):
            page, n = self.page_of(row, 32 * block), min(32, count - 32 * block)
            if page is None:
                continue
            inside = block % (self.page // 32)
            for head in range(self.heads):
                for which in range(2):
                    c = self.block(page, head, inside, which)[:n]
                    out[which, 32 * block:32 * block + n, head] = value_of(c, self.fmt) * self.scales[page, head, inside, which]
        return out[0], out[1]


def fill(cache, seed, spread=1.0, garbage=False):
    """Fills a cache of the binding with random finite codes and scales; garbage: bytes of any value and NaN scales."""
    g = torch.Generator(device=cache.codes.device).manual_seed(seed)
    cache.codes.random_(0, 256, generator=g)
    if garbage:
        cache.scales.fill_(float("nan"))
        return
    bad = 0x7F if cache.fmt == "e4m3" else 0x80               # NaN codes; -128, which no quantizer writes
    hide = (cache.codes & 0x7F) == 0x7F if cache.fmt == "e4m3" else cache.codes == bad
    cache.codes[hide] = 0x35
    size = torch.randn(cache.scales.shape, generator=g, device=cache.codes.device) * 0.7 * spread
    cache.scales.copy_(torch.exp(size) / LARGEST[cache.fmt])


# ---- attention -------------------------------------------------------------------------
def attention(q, k, v, first, length, scale, causal=True, window=0):
    """Rows q [n, q_heads, dim], the first at position `first`, over k and v [keys, heads, dim] (NaN: an absent token): o in
    64 bits and its bound before rounding.

    A score is a sum of dim exact products in FP32, off by (dim + 4) U sum |q k|, and rounded once more; its exponent is
    rounded as often as the running maximum changes, at sizes up to |score| + |maximum| + 15 ln 2.  A probability is rounded
    to FP16 (2^-11; held times 2^9 of a maximum that is at most the row's, so small ones are off by half of 2^-24 over 2^9 =
    2^-34 of the largest), its scale and exponential add 4 U, and every sum, rescaling and join of N tokens N U."""
    q, k, v = q.double(), k.double(), v.double()
    n, heads, dim = q.shape
    group, keys = heads // k.shape[1], k.shape[0]
    there = ~torch.isnan(k[:, 0, 0]) if keys else torch.zeros(0, dtype=torch.bool)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    position, key = first + torch.arange(n), torch.arange(keys)
    seen = there[None, :] & (key[None, :] < length) & (position[:, None] >= 0)
    if causal:
        seen = seen & (key[None, :] <= position[:, None])
    if window:
        seen = seen & (key[None, :] > position[:, None] - window)
    o, e = torch.zeros(n, heads, dim, dtype=torch.float64), torch.zeros(n, heads, dim, dtype=torch.float64)
    some = seen.any(1)
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        s = (q[:, h] @ kh.t().contiguous()) * scale
        size = (q[:, h].abs() @ kh.abs().t().contiguous()) * scale
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(1, keepdim=True) if keys else torch.zeros(n, 1, dtype=torch.float64)
        top = torch.where(some[:, None], top, torch.zeros_like(top))
        p = torch.exp(s - top)
        total = p.sum(1, keepdim=True).clamp_min(TINY)
        p = p / total
        far = torch.where(seen, s.abs(), torch.zeros_like(s)).amax(1) + 15 * math.log(2) if keys else torch.zeros(n, dtype=torch.float64)
        delta = torch.where(seen, size, torch.zeros_like(s)).amax(1) * (dim + 4) * U + 8 * U * far if keys else torch.zeros(n, dtype=torch.float64)
        each = 2.0 ** -11 + 2 * delta + (2 * keys + 64) * U
        o[:, h] = p @ vh
        e[:, h] = (p @ vh.abs()) * (2 * each)[:, None] + vh.abs().amax(0, keepdim=True) * keys * 2.0 ** -34 + TINY if keys else TINY
        bad = torch.isnan(q[:, h]).any(1) | torch.isinf(q[:, h]).any(1)
        o[:, h][bad & some] = math.nan
    o[~some], e[~some] = 0, 0
    return o, e


def check_attention(iq, cache, q, page_table, lengths, starts=None, *, scale=None, causal=True, window=0, got=None, what=""):
    """Runs cache_attention (unless its result is given) and holds it to the plain form."""
    if got is None:
        got = iq.cache_attention(cache, q, page_table, lengths, starts, scale=scale, causal=causal, window=window)
    model = Cache(cache.codes, cache.scales, cache.fmt, cache.heads, cache.dim, cache.page)
    scale = cache.dim ** -0.5 if scale is None else scale
    at = [0] * 0 if starts is None else starts.tolist()
    limit = page_table.shape[1] * cache.page
    for b, length in enumerate(lengths.tolist()):
        lo, hi = (at[b], at[b + 1]) if starts is not None else (b, b + 1)
        if hi <= lo:
            continue
        length = max(length, 0)
        k, v = model.values(page_table[b].tolist(), min(length, limit))
        o, e = attention(q[lo:hi].cpu(), k, v, length - (hi - lo), length, scale, causal, window)
        assert_within(got[lo:hi].cpu(), o, e, f"{what} sequence {b}")
    return got

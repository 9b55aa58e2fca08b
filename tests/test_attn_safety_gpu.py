"""The attention operators on the GPU where numbers lie far apart and where a query's answer must not hang on what it does not see.

Errors are bounded by what each row sees alone.  U is half a step of FP32."""
import math

import pytest
import torch

import attn_oracle as ao
from attn_oracle import TINY, U
from test_attn_gpu import FORMATS, I32, ends, gen, iq, model_of, rand, same_memory, scene, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def parts_of(model, row, count):
    """Code values and scales [count, heads, dim] and [count, heads] of keys and of values, 64 bits, of a sequence's first
    tokens; and which of them lie in pages that are there."""
    codes = torch.zeros(2, count, model.heads, model.dim, dtype=torch.float64)
    scales, there = torch.zeros(2, count, model.heads, dtype=torch.float64), torch.zeros(count, dtype=torch.bool)
    for block in range(-(-count // 32)):
        page, n = model.page_of(row, 32 * block), min(32, count - 32 * block)
        if page is None:
            continue
        at = slice(32 * block, 32 * block + n)
        there[at] = True
        for head in range(model.heads):
            for which in range(2):
                inside = block % (model.page // 32)
                codes[which, at, head] = ao.value_of(model.block(page, head, inside, which)[:n], model.fmt).double()
                scales[which, at, head] = model.scales[page, head, inside, which].double()
    return codes, scales, there


def answer(q, codes, scales, there, first, length, scale, causal, window):
    """Rows q [n, q_heads, dim] as attn_oracle.attention has them, and a bound before rounding that goes by seen tokens alone.

    A score is a sum of dim exact products, off by (dim + 4) U of their magnitudes, and its exponent is formed from it, the
    running maximum and offsets of up to 75, each rounded (8 U of those sizes in all): delta.  A probability times its values
    scale is rounded to FP16: 2^-11 of it, or, held times 2^9 of the largest such product so far, 2^-25 - 9 = 2^-34 of that
    where it is small; the codes that it meets are exact.  A weight of FP32 below its smallest normal number is 0, so that a
    probability below 2^-126 may be.  Sums over N tokens with their rescalings: (2 N + 64) U."""
    q = q.double()
    n, heads, dim = q.shape
    group, keys = heads // codes.shape[2], codes.shape[1]
    position, key = first + torch.arange(n), torch.arange(keys)
    seen = there[None, :] & (key[None, :] < length) & (position[:, None] >= 0)
    if causal:
        seen = seen & (key[None, :] <= position[:, None])
    if window:
        seen = seen & (key[None, :] > position[:, None] - window)
    o, e = torch.zeros(n, heads, dim, dtype=torch.float64), torch.zeros(n, heads, dim, dtype=torch.float64)
    some, zero = seen.any(1), torch.zeros((), dtype=torch.float64)
    for h in range(heads):
        (ck, cv), (sk, sv) = codes[:, :, h // group], scales[:, :, h // group]
        s = torch.where(seen, (q[:, h] @ ck.t().contiguous()) * sk * scale, zero)
        size = torch.where(seen, (q[:, h].abs() @ ck.abs().t().contiguous()) * sk * scale, zero).amax(1)
        p = torch.softmax(s.masked_fill(~seen, -math.inf), 1)
        z = torch.where(seen, p * sv, zero)
        delta = size * (dim + 4) * U + 8 * U * (s.abs().amax(1) + 75)
        each = 2.0 ** -11 + 2 * delta + (2 * seen.sum(1) + 64) * U
        o[:, h] = z @ cv
        e[:, h] = 2 * each[:, None] * (z @ cv.abs()) + 2.0 ** -34 * z.amax(1)[:, None] * (seen.double() @ cv.abs())
        e[:, h] += TINY * (torch.where(seen, sv, zero) @ cv.abs()) + TINY
    o[~some], e[~some] = 0, 0
    return o, e


def check(iq, cache, q, table, lengths, starts, *, causal=True, window=0, scale=None, rows=None, got=None, what="", **kw):  # noqa: F811
    """Runs cache_attention (unless its result is given) and holds its rows (those where `rows` is true) to `answer`."""
    got = got if got is not None else iq.cache_attention(cache, q, table, lengths, starts, causal=causal, window=window, scale=scale, **kw)
    model, scale = model_of(cache), cache.dim ** -0.5 if scale is None else scale
    for b, length in enumerate(lengths.tolist()):
        lo, hi = (int(starts[b]), int(starts[b + 1])) if starts is not None else (b, b + 1)
        if lo >= hi or length <= 0:
            continue
        codes, scales, there = parts_of(model, table[b].tolist(), min(length, table.shape[1] * cache.page))
        o, e = answer(q[lo:hi].cpu(), codes, scales, there, length - (hi - lo), length, scale, causal, window)
        keep = slice(None) if rows is None else rows[lo:hi].cpu()
        ao.assert_within(got[lo:hi].cpu()[keep], o[keep], e[keep], f"{what} sequence {b}")
    return got


def widened(table, width):
    wide = torch.full((table.shape[0], width), -1, dtype=I32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


# ---- values of very different sizes ---------------------------------------------------------
KINDS = (([300], [1]), ([200, 77], [5, 3]), ([70], [150]), ([0, 190], [140, 33]))     # new tokens behind cached ones


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_values_scales_far_apart(iq, fmt, dim):  # noqa: F811
    """Blocks whose value scales are 2^-60 to 2^60, some 0: each row is as exact as the largest product of a probability and a
    scale that it sees allows, with a window, without, and in tables that share rows out."""
    for k, (had, new) in enumerate(KINDS):
        cache, q, table, lengths, starts = scene(iq, fmt, 1, 2, dim, 32, had, new, dim + k, garbage=False)
        power = torch.randint(-60, 61, cache.scales[..., 1].shape, generator=gen(k), device="cuda")
        cache.scales[..., 1] = torch.exp2(power) * (power % 7 != 0)
        for t in (table, widened(table, 400)):
            for kw in (dict(), dict(window=20), dict(window=100), dict(causal=False)):
                check(iq, cache, q, t, lengths, starts, what=f"{had} {new} {t.shape[1]} {kw}", **kw)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ratio", [-30, -50, -110])
def test_values_behind_a_large_block(iq, fmt, ratio):  # noqa: F811
    """One block of large values that a window has left, that is not yet seen, or that is seen with next to no probability."""
    for had, new in KINDS:
        for spot in (0, 2, 5):
            cache, q, table, lengths, starts = scene(iq, fmt, 1, 3, 128, 32, had, new, 5, garbage=False)
            cache.scales[..., 1] = 2.0 ** ratio
            for b in range(len(had)):
                if table[b, min(spot, table.shape[1] - 1)] >= 0:
                    cache.scales[table[b, min(spot, table.shape[1] - 1)].long(), ..., 1] = 1.0
            for kw in (dict(window=33), dict(window=70), dict(), dict(scale=3.0)):
                check(iq, cache, q, table, lengths, starts, what=f"{had} {new} {spot} {kw}", **kw)


@pytest.mark.parametrize("fmt", FORMATS)
def test_scales_of_blocks_that_a_query_does_not_see(iq, fmt):  # noqa: F811
    """Whatever the scales of a block hold: queries that do not see it, of the same call, answer without it."""
    for had, new in KINDS[1:]:
        for bad in (math.nan, math.inf, -math.inf, 3e38):
            for window in (0, 12, 40):
                cache, q, table, lengths, starts = scene(iq, fmt, 1, 2, 64, 32, had, new, 9, garbage=False)
                rows = torch.ones(sum(new), dtype=torch.bool)
                for b, (h, n) in enumerate(zip(had, new)):
                    spot = (h + n // 2) // 32                       # the block that the sequence's middle new token lies in
                    cache.scales[table[b, spot].long()] = bad
                    at = torch.arange(h, h + n)
                    least = (at - window + 1).clamp_min(0) if window else torch.zeros_like(at)
                    rows[int(starts[b]):int(starts[b + 1])] = (at < 32 * spot) | (least >= 32 * spot + 32)
                check(iq, cache, q, table, lengths, starts, window=window, rows=rows, what=f"{had} {new} {bad} {window}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_queries_that_see_nothing(iq, bad):  # noqa: F811
    """A query that is not finite answers NaN where it sees a token, and zeros where it sees none, whatever the others of its
    tile see: rows before a sequence's first token, and rows of absent pages, in calls of few and of many columns."""
    for new, length, table in ((5, 3, [[1, 2]]), (150, 60, [[1, 2]]), (7, 40, [[-1, 2]]), (160, 160, [[1, -1, 2, 3, 4]]), (150, 160, [[-1, -1, 2, 3, 9]])):
        cache = iq.make_cache(6, 1, 64, "e4m3", 32)
        ao.fill(cache, 4)
        table, starts = torch.tensor(table, dtype=I32, device="cuda"), torch.tensor([0, new], dtype=I32, device="cuda")
        lengths = torch.tensor([length], dtype=I32, device="cuda")
        q = rand(gen(2), new, 3, 64)
        want = iq.cache_attention(cache, q, table, lengths, starts, window=50)
        hurt = torch.arange(new, device="cuda") % 3 == 1
        q[hurt, 1, 7] = bad
        position = torch.arange(length - new, length)
        there = torch.tensor([0 <= p < len(table[0]) * 32 and 0 <= int(table[0, p // 32]) < 6 for p in range(max(length, 1))])
        sees = torch.tensor([bool(there[max(0, p - 49):p + 1].any()) if p >= 0 else False for p in position.tolist()]).cuda()
        got = iq.cache_attention(cache, q, table, lengths, starts, window=50)
        assert torch.isnan(got[hurt & sees, 1]).all() and not got[~sees].any()
        want[hurt & sees, 1] = got[hurt & sees, 1] = 0
        assert torch.equal(got, want), (new, length)


# ---- scores at the ends of their range ------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100, 2.0 ** 124])
def test_scores_far_from_zero(iq, fmt, size):  # noqa: F811
    """Scores of one sign, up to the ends of FP32: the query takes the token of the largest, and the mean of those that are equal
    to it.  Keys are one code times a power of two, so scores are exact, differ by their own size where they differ, and
    roundings of exponents do not show."""
    dim, heads = 64, 2
    for had, new in (([0], [1]), ([70], [3]), ([300], [40]), ([20], [170]), ([5000], [1])):
        n = had[0] + new[0]
        pages = -(-n // 32)
        cache = iq.make_cache(pages, heads, dim, fmt, 32)
        ao.fill(cache, 3)
        one = 0x38 if fmt == "e4m3" else 1
        cache.codes[:, :, :, 0] = one
        cache.scales[..., 1] = 1.0
        power = torch.randint(0, 3, (pages, heads, 1), generator=gen(n), device="cuda")
        cache.scales[..., 0] = torch.exp2(-4.0 * power)
        table = torch.arange(pages, dtype=I32, device="cuda")[None]
        starts, lengths = torch.tensor([0, new[0]], dtype=I32, device="cuda"), torch.tensor([n], dtype=I32, device="cuda")
        for t in (table, widened(table, 400)):
            for sign in (1.0, -1.0):
                q = torch.zeros(new[0], heads, dim, dtype=torch.bfloat16, device="cuda")
                q[..., 9], q[..., 10] = sign * size, sign * size * 2.0 ** -9 * (2 - 2.0 ** -7)      # more digits than BF16 has
                for kw in (dict(), dict(window=45)):
                    got = iq.cache_attention(cache, q, t, lengths, starts, scale=1.0, **kw).cpu().double()
                    codes, scales, _ = parts_of(model_of(cache), table[0].tolist(), n)
                    at, key = torch.arange(had[0], n)[:, None], torch.arange(n)[None]
                    seen = (key <= at) & (key > at - kw.get("window", 1 << 30))
                    for h in range(heads):
                        score = torch.where(seen, sign * scales[0, :, h], torch.tensor(-math.inf, dtype=torch.float64))
                        p = (score == score.amax(1, keepdim=True)).double()
                        p = p / p.sum(1, keepdim=True)
                        want = p @ codes[1, :, h]
                        # FP16 holds the equal probabilities alike to 2^-11, and sums of them in FP32
                        e = (p @ codes[1, :, h].abs()) * (2.0 ** -10 + (2 * n + 64) * U) + TINY
                        ao.assert_within(got[:, h].to(torch.float32), want, e + 2.0 ** -8 * (want.abs() + e), f"{had} {new} {sign} {kw}")


# ---- angles -----------------------------------------------------------------------------------
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_angles_keep_their_digits(iq, inter):  # noqa: F811
    """Cosines and sines of angles that FP32 does not hold, read off pairs (1, 0): off by one step of the largest below 1 (the
    functions' own, U in all) and half a step for what the rest of the angle adds.  An angle rounded to FP32 alone is off
    by up to 2^-25 half turns, 1.57 U."""
    g = gen(70)
    x = torch.zeros(3, 2, 1024, device="cuda")
    x[..., 0::2 if inter else 1][..., :512] = 1
    a, b = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, 512), slice(512, None))
    at = torch.tensor([1, -1, 3], dtype=I32, device="cuda")
    for _ in range(100):
        table = torch.rand(512, generator=g, device="cuda", dtype=torch.float64) - 0.5
        for call, way in ((iq.rotary, 1), (iq.rotary_backward, -1)):
            y = call(x, at, table, interleaved=inter).double()
            t = at.double()[:, None] * table
            t = ((t - t.round()) * (2 * math.pi * way))[:, None]
            assert max((y[..., a] - torch.cos(t)).abs().max(), (y[..., b] - torch.sin(t)).abs().max()) <= 1.5 * U


# ---- strides ------------------------------------------------------------------------------------
def test_strides_of_single_tokens_and_heads(iq):  # noqa: F811
    """A row of a buffer whose rows do not lie on 16 bytes, and one head of it: the stride that leads nowhere is not looked at."""
    g = gen(71)
    cache, q, table, lengths, starts = scene(iq, "int8", 1, 3, 64, 32, [70], [1], 7)
    want = iq.cache_attention(cache, q, table, lengths)
    odd = torch.as_strided(q, (1, 3, 64), (2051, 64, 1))
    for t in (None, torch.empty_like(q)):
        assert torch.equal(iq.cache_attention(cache, odd, table, lengths, out=t), want)
    cache, q, table, lengths, starts = scene(iq, "int8", 1, 1, 64, 32, [70], [5], 7)
    want = iq.cache_attention(cache, q, table, lengths, starts)
    assert torch.equal(iq.cache_attention(cache, torch.as_strided(q, (5, 1, 64), (64, 67, 1)), table, lengths, starts), want)
    turns, at = iq.rotary_table(64), torch.tensor([9], dtype=I32, device="cuda")
    x = rand(g, 1, 3, 64)
    want = iq.rotary(x, at, turns)
    y = x.clone()
    assert torch.equal(iq.rotary(y, at, turns, out=torch.as_strided(y, (1, 3, 64), (2051, 64, 1))), want) and torch.equal(y, want)


# ---- arrays of any content ------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
def test_starts_and_lengths_of_any_content(iq, fmt):  # noqa: F811
    """Starts that descend, are negative or point behind the rows, lengths past the table: nothing outside the operands changes,
    and sequences whose entries are sound beside others answer as alone."""
    g, heads, dim, n, guard = gen(80), 2, 64, 90, 64
    odd = [-(1 << 31), (1 << 31) - 1, -1, 0, 40, 91, 1 << 30]
    for width in (3, 300):
        cache = iq.make_cache(40, heads, dim, fmt, 32)
        ao.fill(cache, 6)
        table = torch.full((5, width), -1, dtype=I32, device="cuda")
        table[:, :3] = torch.randperm(36, generator=torch.Generator().manual_seed(2))[:15].view(5, 3).to(I32)
        for k in range(len(odd)):
            print("case", width, k, flush=True)
            # sequence 0 has rows 0 to 29; the others' starts are anything
            starts = torch.tensor([0, 30] + [odd[(k + 3 * i) % len(odd)] for i in range(4)], dtype=torch.int64).to(I32).cuda()
            lengths = torch.tensor([77] + [odd[(2 * k + i) % len(odd)] for i in range(4)], dtype=torch.int64).to(I32).cuda()
            q, k_, v = rand(g, n, 8, dim), rand(g, n, heads, dim), rand(g, n, heads, dim)
            around = torch.full((2 * guard + n, 8, dim), 7.0, dtype=torch.bfloat16, device="cuda")
            out = around[guard:guard + n]
            before = model_of(cache)
            iq.cache_attention(cache, q, table, lengths, starts, out=out)
            assert (around[:guard] == 7).all() and (around[guard + n:] == 7).all()
            if not any(int(starts[i]) < 30 and int(starts[i + 1]) > int(starts[i]) for i in range(1, 5)):
                check(iq, cache, q[:30], table[:1], lengths[:1], starts[:2], got=out[:30], what=f"{k}")
            keys = torch.full((2 * guard + n, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
            values = keys.clone()
            iq.cache_read(cache, table, lengths, starts, n, out=(keys[guard:guard + n], values[guard:guard + n]))
            for t in (keys, values):
                assert (t[:guard] == 7).all() and (t[guard + n:] == 7).all()
            after = model_of(cache)
            assert torch.equal(before.codes, after.codes) and torch.equal(before.scales, after.scales)
            iq.cache_append(cache, k_, v, table, lengths, starts, q=q)
            free = torch.ones(40, dtype=torch.bool)
            free[table[:, :3].cpu().long().flatten()] = False
            after = model_of(cache)
            assert torch.equal(before.codes[free], after.codes[free]) and torch.equal(before.scales[free], after.scales[free])
            ao.fill(cache, 6)


# ---- far offsets, calls at once, calls again -----------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
def test_cache_past_32_bits(iq, fmt):  # noqa: F811
    """Pages that lie 5 GB into the memory, with scales to match: the bits of a small cache."""
    heads, dim, page = 8, 128, 256
    pages = 5 * 2 ** 30 // (heads * page * 2 * dim) + 40
    g, had, new = gen(90), [700, 0, 90], [1, 300, 20]
    total = [a + b for a, b in zip(had, new)]
    whole = lambda t: torch.tensor(t, dtype=I32, device="cuda")  # noqa: E731
    small, large = iq.make_cache(9, heads, dim, fmt, page), iq.make_cache(pages, heads, dim, fmt, page)
    assert large.codes.numel() > 5 * 2 ** 30
    near = whole([[0, 1, 2, -1], [3, 4, -1, -1], [5, -1, -1, -1]])
    far = torch.where(near >= 0, pages - 9 + near, near)
    n = sum(total)
    k, v, q = rand(g, n, heads, dim), rand(g, n, heads, dim), rand(g, sum(new), 32, dim)
    every, starts = whole([0, total[0], total[0] + total[1], n]), whole([0, 1, 301, 321])
    turns, outs = iq.rotary_table(dim), []
    for cache, table in ((small, near), (large, far)):
        cache.codes.zero_()                                         # what no token writes is compared too
        cache.scales.zero_()
        iq.cache_append(cache, k, v, table, whole(total), every, rotary=turns)
        outs.append([iq.cache_attention(cache, q, table, whole(total), starts), iq.cache_attention(cache, q[:3], table, whole(total)),
                     *iq.cache_read(cache, table, whole(total), every, n)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(small.codes[:6], large.codes[pages - 9:pages - 3]) and torch.equal(small.scales[:6], large.scales[pages - 9:pages - 3])


def test_strides_past_32_bits(iq):  # noqa: F811
    """Rows 2^31 elements apart."""
    g, far = gen(91), (1 << 31) + 8
    at, turns = torch.tensor([5, 70000], dtype=I32, device="cuda"), iq.rotary_table(64)
    memory = torch.empty(far + 4 * 64, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(memory, (2, 4, 64), (far, 64, 1))
    x.copy_(rand(g, 2, 4, 64))
    near = x.contiguous()
    want = iq.rotary(near, at, turns)
    assert torch.equal(iq.rotary(x, at, turns), want)
    cache, _, table, lengths, starts = scene(iq, "e4m3", 2, 2, 64, 32, [40, 90], [1, 1], 3)
    assert torch.equal(iq.cache_attention(cache, x, table, lengths), iq.cache_attention(cache, near, table, lengths))
    before = model_of(cache)
    q = iq.cache_append(cache, x[:, :2], x[:, 2:], table, lengths, q=x, rotary=turns)
    after = model_of(cache)
    cache.codes.copy_(before.codes)
    cache.scales.copy_(before.scales)
    assert torch.equal(iq.cache_append(cache, near[:, :2], near[:, 2:], table, lengths, q=near, rotary=turns), q)
    same_memory(cache, after)
    assert iq.rotary(x, at, turns, out=x) is x and torch.equal(x.contiguous(), want)


def test_calls_at_once(iq):  # noqa: F811
    """Two streams in one cache: attention of some sequences while others are appended to, again and again."""
    cache, q, table, lengths, starts = scene(iq, "int8", 2, 4, 128, 32, [3000, 200, 10, 64], [1, 130, 1, 40], 12)
    k, v, turns = rand(gen(1), 172, 2, 128), rand(gen(2), 172, 2, 128), iq.rotary_table(128)
    mine, yours = slice(0, 2), slice(2, 4)
    first, rest = starts[:3].clone(), starts[2:] - starts[2]
    want = iq.cache_attention(cache, q[:131], table[mine], lengths[mine], first)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(30):
        iq.cache_append(cache, k[131:], v[131:], table[yours], lengths[yours], rest, rotary=turns, stream=streams[0])
        outs.append(iq.cache_attention(cache, q[:131], table[mine], lengths[mine], first, stream=streams[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    # appended thirty times over, the sequences hold what one append leaves
    again = model_of(cache)
    iq.cache_append(cache, k[131:], v[131:], table[yours], lengths[yours], rest, rotary=turns)
    same_memory(cache, again)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_repeats_its_bits(iq, fmt):  # noqa: F811
    g, had, new = gen(93), [5, 64, 0], [70, 3, 400]
    total = [a + b for a, b in zip(had, new)]
    table, pages = tables(total, 64, 1)
    k, v, q = (rand(g, sum(new), h, 96) for h in (3, 3, 6))
    turns, seen = iq.rotary_table(40), []
    for _ in range(4):
        cache = iq.make_cache(pages, 3, 96, fmt, 64)
        ao.fill(cache, 1)
        out = iq.cache_append(cache, k, v, table, torch.tensor(total, dtype=I32, device="cuda"), ends(new), q=q, rotary=turns)
        seen.append((out, cache.codes, cache.scales))
    assert all(torch.equal(a, b) for s in seen[1:] for a, b in zip(seen[0], s))

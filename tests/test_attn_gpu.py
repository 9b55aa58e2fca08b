"""The attention operators on the GPU against their plain forms: rotations and attention in 64 bits, the cache's codes bit for bit."""
import math

import pytest
import torch

import attn_oracle as ao

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FORMATS = ("e4m3", "int8")


@pytest.fixture(scope="module")
def iq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int_quantization_amd as m
    m.load_library()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def whole(values):
    return torch.tensor(values, dtype=I32, device="cuda")


def ends(counts):
    return whole([0] + torch.tensor(counts).cumsum(0).tolist())


def tables(lengths, page, seed, spare=2, width=None):
    """A page table of pages in random order for these lengths, unused entries -1; and the number of pages."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max([1] + need) if width is None else width
    rows = [[order.pop() for _ in range(n)][:width] + [-1] * (width - n) for n in need]
    return whole(rows), pages


# ---- rotary ---------------------------------------------------------------------------
def check_rotary(iq, x, at, table, inter, amplitude=1.0, out=None, what=""):
    for call, way in ((iq.rotary, 1), (iq.rotary_backward, -1)):
        want = ao.rotate(x, at, table, inter, amplitude, way)
        got = call(x, at, table, interleaved=inter, amplitude=amplitude, out=out)
        ao.assert_within(got, want, ao.rotate_bound(x, table, inter, amplitude), what)
        rot = 2 * table.numel()
        assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_sizes(iq, dtype, inter):
    g = gen(1)
    for dim, rots in ((1, (0,)), (2, (0, 2)), (7, (2, 6)), (64, (0, 2, 8, 16, 30, 32, 64)), (96, (40, 96)), (128, (64, 128)), (256, (256,)), (1024, (1024,))):
        for tokens, heads in ((1, 1), (1, 5), (3, 32), (130, 3)):
            for rot in rots:
                x = rand(g, tokens, heads, dim, dtype=dtype)
                at = torch.randint(-5000, 200000, (tokens,), generator=g, device="cuda", dtype=I32)
                check_rotary(iq, x, at, iq.rotary_table(rot), inter, 1.25, what=f"{tokens} x {heads} x {dim}, {rot}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_of_few_elements(iq, dtype, inter):
    """Ends of what turns inside 16 bytes, whole rows and rows that start anywhere, into a new result and in place."""
    g = gen(40)
    for dim, rots in ((192, (0, 2, 4, 10, 186, 190)), (40, (2, 6, 34, 38)), (8, (2, 6, 8)), (44, (2, 4, 42))):
        for rot in rots:
            table, at = iq.rotary_table(rot), whole([3, 70000, -5, 0, 11])
            wide = rand(g, 5, 3, dim + 3, dtype=dtype)
            for x in (rand(g, 5, 3, dim, dtype=dtype), wide[..., :dim], wide[..., 3:]):
                check_rotary(iq, x, at, table, inter, what=f"{dim} {rot}")
                want, here = iq.rotary(x, at, table, interleaved=inter), x.clone(memory_format=torch.contiguous_format)
                assert torch.equal(iq.rotary(here, at, table, interleaved=inter, out=here), want)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_strides_and_in_place(iq, inter):
    g = gen(2)
    for dtype in (BF, F32):
        for dim, heads in ((64, 4), (48, 3), (9, 5)):
            table = iq.rotary_table(dim // 4 * 2)
            fused = rand(g, 21, 3 * heads + 1, dim, dtype=dtype)       # queries, keys and values of one product
            at = torch.arange(21, device="cuda", dtype=I32)
            x = fused[:, heads:2 * heads]
            check_rotary(iq, x, at, table, inter, what="a slice")
            swapped = rand(g, heads, 21, dim, dtype=dtype).transpose(0, 1)
            check_rotary(iq, swapped, at, table, inter, out=rand(g, heads, 21, dim, dtype=dtype).transpose(0, 1), what="heads first")
            odd = rand(g, 21 * heads * dim + 1, dtype=dtype)[1:].view(21, heads, dim)      # not on 16 bytes
            check_rotary(iq, odd, at, table, inter, what="odd address")
            one = rand(g, 1, 1, dim, dtype=dtype).expand(21, heads, dim)
            check_rotary(iq, one, at, table, inter, what="broadcast")
            want, around = iq.rotary(x, at, table, interleaved=inter), fused.clone()
            assert iq.rotary(x, at, table, interleaved=inter, out=x) is x and torch.equal(x, want)
            around[:, heads:2 * heads] = want
            assert torch.equal(fused, around)
    with pytest.raises(iq.IQError):
        iq.rotary(x, at, table, out=rand(g, 1, heads, dim, dtype=F32).expand(21, heads, dim))


def test_rotary_far_positions(iq):
    """Up to the ends of 32 bits, where an FP32 angle has no digits left."""
    at = whole([0, 1, -1, 1 << 20, (1 << 24) + 1, 2147483647, -2147483648, 123456789])
    for inter in (False, True):
        for dtype in (F32, BF):
            for table in (iq.rotary_table(128), iq.rotary_table(128, 5e5, "parts", 16.0, 8192), iq.rotary_table(128, 1e4, "base", 8.0)):
                check_rotary(iq, rand(gen(3), 8, 4, 128, dtype=dtype), at, table, inter)


def test_rotary_turns_back(iq):
    g = gen(4)
    x, at, table = rand(g, 50, 6, 64, dtype=F32), torch.arange(50, device="cuda", dtype=I32), iq.rotary_table(64)
    back = iq.rotary_backward(iq.rotary(x, at, table), at, table)
    ao.assert_within(back, x.double(), 3 * ao.rotate_bound(x, table), "x")


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient_against_differences(iq, inter):
    """The map is linear, so <dy, R(x)> - <R'(dy), x> is rounding alone."""
    g = gen(5)
    x, dy = rand(g, 40, 5, 96, dtype=F32), rand(g, 40, 5, 96, dtype=F32)
    at, table = torch.randint(0, 100000, (40,), generator=g, device="cuda", dtype=I32), iq.rotary_table(64)
    y, dx = (f(t, at, table, interleaved=inter, amplitude=1.5) for f, t in ((iq.rotary, x), (iq.rotary_backward, dy)))
    off = (dy.double() * y.double()).sum() - (dx.double() * x.double()).sum()
    most = sum(((ao.rotate_bound(a, table, inter, 1.5) + ao.U * b.double().abs()) * c.double().abs()).sum() for a, b, c in ((x, y, dy), (dy, dx, x)))
    assert off.abs() <= most


def test_rotary_not_finite(iq):
    """An infinity or a NaN stays in its pair."""
    x, at, table = rand(gen(6), 3, 2, 64), whole([5, 6, 7]), iq.rotary_table(64)
    want = iq.rotary(x, at, table)
    x[1, 1, 3], x[2, 0, 40] = math.nan, math.inf
    got = iq.rotary(x, at, table)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, 1, 3] = hit[1, 1, 35] = hit[2, 0, 40] = hit[2, 0, 8] = True
    assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()


# ---- append and read -----------------------------------------------------------------------
def model_of(cache):
    return ao.Cache(cache.codes, cache.scales, cache.fmt, cache.heads, cache.dim, cache.page)


def same_memory(cache, model):
    """Codes and scales of the whole memory, bytes that are no sequence's among them."""
    assert torch.equal(cache.codes.cpu(), model.codes)
    assert torch.equal(cache.scales.cpu().view(I32), model.scales.view(I32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,page,dtype", [(64, 1, 32, F32), (64, 3, 64, BF), (96, 2, 128, BF), (128, 2, 32, F32), (192, 1, 64, F32), (256, 2, 32, BF)])
def test_append_codes_are_exact(iq, fmt, dim, heads, page, dtype):
    """Pieces of many lengths into a memory of any content: codes, scales and everything that is left alone, bit for bit."""
    g = gen(dim + page)
    for k, (had, new) in enumerate((([0], [1]), ([0], [200]), ([31, 32, 33, 1], [1, 1, 1, 1]), ([0, 17, 64, 5, 95], [70, 3, 0, 27, 66]),
                                    ([63, 0, 2], [0, 97, 0]))):
        total = [a + b for a, b in zip(had, new)]
        table, pages = tables(total, page, k)
        cache = iq.make_cache(pages, heads, dim, fmt, page)
        ao.fill(cache, k)
        model = model_of(cache)
        size = torch.exp2(torch.randint(-3, 4, (sum(new), heads, 1), generator=g, device="cuda"))
        x, y = ((torch.randn(sum(new), heads, dim, generator=g, device="cuda") * size).to(dtype) for _ in range(2))
        starts = ends(new)
        assert iq.cache_append(cache, x, y, table, whole(total), None if set(new) == {1} else starts) is None
        model.append(x.cpu().float(), y.cpu().float(), table.tolist(), total, starts.tolist())
        same_memory(cache, model)
        read = ends(total)
        for out in (F32, BF):
            got = iq.cache_read(cache, table, whole(total), read, sum(total), out)
            for which in range(2):
                want = torch.cat([model.values(table[b].tolist(), n)[which] for b, n in enumerate(total)])
                assert torch.equal(got[which].cpu(), want.to(out))


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_token_by_token(iq, fmt):
    """Blocks whose scale grows, stays, and starts at zero; rows of zeros, and of sizes from the least to the most that FP32 holds."""
    g, heads, dim, batch = gen(9), 2, 64, 5
    cache = iq.make_cache(16, heads, dim, fmt, 32)
    ao.fill(cache, 1, garbage=True)
    model = model_of(cache)
    table = torch.randperm(15, generator=torch.Generator().manual_seed(1)).view(batch, 3).to(I32).cuda()
    for t in range(70):
        x, y = (torch.randn(batch, heads, dim, generator=g, device="cuda") for _ in range(2))
        x[1] *= 2.0 ** t                                    # grows at every token
        x[2] *= 0 if t % 5 else 1                           # zeros first and in between
        if t < 3:
            x[2] = y[2] = 0
        x[3] *= 2.0 ** (-149 + 3 * t)                       # from subnormal
        y[3] *= 2.0 ** (120 if t == 20 else -100)
        y[4] *= 2.0 ** -t                                   # the first is the largest
        iq.cache_append(cache, x, y, table, whole([t + 1] * batch))
        model.append(x.cpu(), y.cpu(), table.tolist(), [t + 1] * batch)
        same_memory(cache, model)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_not_finite(iq, fmt):
    cache = iq.make_cache(2, 1, 64, fmt, 32)
    ao.fill(cache, 2, garbage=True)
    model = model_of(cache)
    x = torch.randn(40, 1, 64, device="cuda", generator=gen(3))
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7], x[33] = math.nan, math.inf, -math.inf, math.nan
    y = torch.full_like(x, math.inf)
    table, n = whole([[1, 0]]), ends([40])
    iq.cache_append(cache, x, y, table, whole([40]), n)
    model.append(x.cpu(), y.cpu(), [[1, 0]], [40], [0, 40])
    same_memory(cache, model)
    k, v = iq.cache_read(cache, table, whole([40]), n, 40, F32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all() and not k[3, 0, 5] and not k[33].any()
    # an infinite x is the block's largest value; where nothing is finite there is no largest, and all are zeros
    assert k[4, 0, 6] == k[:32].max() and k[5, 0, 7] == k[:32].min() and not v.any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_turns_keys_and_queries(iq, fmt, inter, dtype):
    g = gen(11)
    for dim, rot, q_heads in ((64, 64, 4), (128, 40, 16), (96, 2, 6), (64, 0, 2), (256, 256, 2), (64, 6, 2)):
        had, new, heads = [0, 1000, 4090, 7], [33, 1, 40, 0], 2
        total = [a + b for a, b in zip(had, new)]
        table, pages = tables(total, 64, dim)
        cache = iq.make_cache(pages, heads, dim, fmt, 64)
        ao.fill(cache, dim)
        freqs, n, starts = iq.rotary_table(rot), sum(new), ends(new)
        fused = rand(g, n, q_heads + 2 * heads, dim, dtype=dtype)
        q, k, v = fused[:, :q_heads], fused[:, q_heads:q_heads + heads], fused[:, q_heads + heads:]
        before = model_of(cache)
        got = iq.cache_append(cache, k, v, table, whole(total), starts, q=q, rotary=freqs, interleaved=inter, amplitude=1.1)
        at = torch.cat([torch.arange(a, a + b) for a, b in zip(had, new)]).to(I32).cuda()
        ao.assert_within(got, ao.rotate(q, at, freqs, inter, 1.1), ao.rotate_bound(q, freqs, inter, 1.1), "q")
        # values bit for bit; keys within half a step of the turned key, whose own error may move it to the next code
        after = model_of(cache)
        before.append(k.cpu().float(), v.cpu().float(), table.tolist(), total, starts.tolist())
        assert torch.equal(after.codes[:, :, :, 1], before.codes[:, :, :, 1])
        want, e = ao.rotate(k, at, freqs, inter, 1.1).cpu(), ao.rotate_bound(k, freqs, inter, 1.1).cpu()
        for b, (a, m) in enumerate(zip(had, new)):
            if not m:
                continue
            keys = after.values(table[b].tolist(), a + m)[0][a:].double()
            scale = torch.stack([after.scales[after.page_of(table[b].tolist(), p), :, p % 64 // 32, 0] for p in range(a, a + m)])[..., None].double()
            rows = slice(int(starts[b]), int(starts[b]) + m)
            step = scale / 2 if fmt == "int8" else torch.maximum(want[rows].abs() * 2.0 ** -4, scale * 2.0 ** -10)
            assert ((keys - want[rows]).abs() <= step + e[rows] + want[rows].abs() * 2 * ao.U).all(), (dim, b)


def test_append_leaves_the_rest(iq):
    """Rows behind the last sequence, rows before a sequence's first token, absent pages, and pages past the table."""
    g, dim, heads = gen(12), 64, 2
    for fmt in FORMATS:
        cache = iq.make_cache(8, heads, dim, fmt, 32)
        ao.fill(cache, 5)
        table = whole([[3, -1, 5], [8, 1, 2], [-7, 2147483647, 6], [7, 4, 0]])
        new, total = [90, 40, 20, 50], [90, 60, 80, 45]                       # the last has more rows than tokens
        n = sum(new) + 6
        k, v, q = (rand(g, n, h, dim, dtype=F32) for h in (heads, heads, 4))
        starts = ends(new)
        model = model_of(cache)
        got = iq.cache_append(cache, k, v, table, whole(total), starts, q=q)
        model.append(k.cpu(), v.cpu(), table.tolist(), total, starts.tolist())
        same_memory(cache, model)
        rows = torch.ones(n, dtype=torch.bool)
        rows[150:155] = rows[200:] = False
        assert torch.equal(got.cpu()[rows], q.cpu()[rows])
        # read: zeros for absent pages, rows that are no token's left alone
        out = (torch.full_like(k, 7.0), torch.full_like(v, 7.0))
        a, b = iq.cache_read(cache, table, whole(total), starts, n, out=out)
        assert a is out[0] and b is out[1]
        for i, (m, length) in enumerate(zip(new, total)):
            want = model.values(table[i].tolist(), length)
            for which, t in enumerate((a, b)):
                lo = int(starts[i]) + max(0, m - length)
                assert torch.equal(t[lo:int(starts[i + 1])].cpu(), torch.nan_to_num(want[which][max(0, length - m):]))
        for t in (a, b):
            assert (t[150:155] == 7).all() and (t[200:] == 7).all()


# ---- attention -------------------------------------------------------------------------------
def scene(iq, fmt, heads, group, dim, page, had, new, seed, garbage=True, scale=1.0):
    """A cache whose memory held anything, with sequences of had + new tokens appended to it; queries of the new ones."""
    g = gen(seed)
    total = [a + b for a, b in zip(had, new)]
    table, pages = tables(total, page, seed)
    cache = iq.make_cache(pages, heads, dim, fmt, page)
    ao.fill(cache, seed, garbage=garbage)
    if garbage:
        n = sum(total)
        iq.cache_append(cache, rand(g, n, heads, dim), rand(g, n, heads, dim), table, whole(total), ends(total))
    q = rand(g, sum(new), heads * group, dim, scale=scale)
    return cache, q, table, whole(total), ends(new)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 32), (1, 40)])
def test_attention_single_tokens(iq, fmt, dim, heads, group):
    for k, had in enumerate(([0], [31], [32, 0, 200], [63, 64, 65, 1, 640])):
        new = [1] * len(had)
        cache, q, table, lengths, starts = scene(iq, fmt, heads, group, dim, (32, 64, 128, 256)[k], had, new, dim + k)
        a = ao.check_attention(iq, cache, q, table, lengths, what=f"{had}")
        ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{had}, starts")
        assert torch.equal(a, iq.cache_attention(cache, q, table, lengths))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 1), (96, 1, 3), (128, 2, 4), (192, 1, 2), (256, 1, 8)])
def test_attention_prompts(iq, fmt, dim, heads, group):
    for k, (had, new) in enumerate((([0], [97]), ([0, 0, 0, 0], [33, 1, 0, 64]), ([100, 0, 7], [31, 130, 2]), ([500, 3], [70, 290]))):
        cache, q, table, lengths, starts = scene(iq, fmt, heads, group, dim, (32, 64, 128, 64)[k], had, new, dim + k)
        for kw in (dict(), dict(causal=False), dict(window=1), dict(window=20), dict(window=100), dict(window=10 ** 9)):
            ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{had} {new} {kw}", **kw)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_scales_and_sizes(iq, fmt):
    """Scores from none to far apart, values and blocks of very different sizes."""
    for dim in (64, 128):
        for scale in (0.0, 1e-3, 1.0, 30.0):
            cache, q, table, lengths, starts = scene(iq, fmt, 2, 3, dim, 64, [200, 30], [5, 40], dim)
            ao.check_attention(iq, cache, q, table, lengths, starts, scale=scale, what=f"scale {scale}")
        for spread in (1.0, 6.0, 20.0):
            cache, q, table, lengths, starts = scene(iq, fmt, 2, 3, dim, 64, [200, 300], [5, 40], dim, garbage=False)
            ao.fill(cache, 7, spread)
            cache.scales[..., 0].clamp_(max=0.02)
            ao.check_attention(iq, cache, q, table, lengths, starts, what=f"spread {spread}")
        for size in (2.0 ** -126, 2.0 ** -60, 2.0 ** 40):
            cache, q, table, lengths, starts = scene(iq, fmt, 2, 3, dim, 64, [100], [40], dim)
            ao.check_attention(iq, cache, (q.float() * size).to(BF), table, lengths, starts, scale=0.1 / size if size > 1e-30 else 1.0, what=f"queries of {size}")
        cache.scales[..., 1] = 0                                                  # values of zeros
        assert not iq.cache_attention(cache, q, table, lengths, starts).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_rows_that_see_nothing(iq, fmt):
    """Empty sequences, rows before the first token, absent pages, pages past the table: zeros, or what is left to see."""
    g, dim, heads, group = gen(20), 64, 2, 3
    cache = iq.make_cache(9, heads, dim, fmt, 32)
    ao.fill(cache, 3)
    cache.scales[0], cache.codes[0] = math.nan, 0x7F                              # a page that nobody has
    table = whole([[1, 2, 3], [-1, 4, 9], [2147483647, -2147483648, -1], [5, -1, 6], [7, 8, 1], [2, 3, 4]])
    lengths, new = whole([96, 80, 70, 96, 10, 500]), [3, 70, 5, 96, 30, 40]
    starts = ends(new)
    q = rand(g, sum(new) + 4, heads * group, dim)
    for kw in (dict(), dict(window=40), dict(window=1), dict(causal=False)):
        out = torch.full((sum(new) + 4, heads * group, dim), 7.0, dtype=BF, device="cuda")
        got = iq.cache_attention(cache, q, table, lengths, starts, out=out, **kw)
        assert got is out and (out[sum(new):] == 7).all()
        ao.check_attention(iq, cache, q, table, lengths, starts, got=got, what=str(kw), **kw)
        assert not got[73:78].any() and not got[174:194].any()
    got = iq.cache_attention(cache, q[:2], table[:2], whole([0, -5]))
    assert not got.any()
    got = iq.cache_attention(cache, q[:0], table[:0], lengths[:0])
    assert got.shape == (0, heads * group, dim)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_takes_nothing_from_hidden_tokens(iq, fmt):
    """The same bits whatever codes lie behind a sequence and whatever scales lie in blocks that nobody sees."""
    for had, new, window in (([70, 0, 31], [1, 1, 1], 0), ([3, 90], [50, 7], 0), ([300, 200], [9, 40], 30)):
        cache, q, table, lengths, starts = scene(iq, fmt, 2, 4, 128, 32, had, new, 5)
        want = iq.cache_attention(cache, q, table, lengths, starts, window=window)
        model, keep = model_of(cache), torch.zeros(cache.codes.shape[:3], dtype=torch.bool)
        for b, length in enumerate(lengths.tolist()):
            least = max(0, length - new[b] - window + 1) if window else 0
            for block in range(least // 32, -(-length // 32)):
                page = model.page_of(table[b].tolist(), 32 * block)
                keep[page, :, block % 1] = True
                n = length - 32 * block
                for head in range(2):
                    for which in range(2) if n < 32 else ():
                        c = model.block(page, head, 0, which)
                        c[n:] = 0x7F
                        model.store(page, head, 0, which, c)
        model.codes[~keep], model.scales[~keep] = 0xFF, math.nan
        other = iq.KVCache(model.codes.cuda(), model.scales.cuda(), fmt, 2, 128, 32)
        assert torch.equal(iq.cache_attention(other, q, table, lengths, starts, window=window), want)


def test_attention_bad_queries(iq):
    """A NaN or an infinity in a query is its own row's and head's affair."""
    cache, q, table, lengths, starts = scene(iq, "e4m3", 2, 3, 64, 64, [40, 0], [30, 20], 8)
    want = iq.cache_attention(cache, q, table, lengths, starts)
    q[3, 2, 5], q[31, 4, 0], q[45, 0, 63] = math.nan, math.inf, -math.inf
    got = iq.cache_attention(cache, q, table, lengths, starts)
    bad = torch.zeros(50, 6, dtype=torch.bool, device="cuda")
    bad[3, 2] = bad[31, 4] = bad[45, 0] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_long(iq, fmt):
    """Sums split over the cache: thousands of tokens, lengths far apart, a table much wider than the sequences."""
    for had, new in (([4999], [1]), ([20000, 3, 700], [1, 1, 1]), ([6001], [40]), ([2900, 0], [3, 300])):
        cache, q, table, lengths, starts = scene(iq, fmt, 2, 4, 64, 64, had, new, 13)
        wide = torch.full((len(had), 2000), -1, dtype=I32, device="cuda")
        wide[:, :table.shape[1]] = table
        a = ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{had}")
        ao.check_attention(iq, cache, q, wide, lengths, starts, what=f"{had}, wide")
        ao.check_attention(iq, cache, q, table, lengths, starts, window=1500, what=f"{had}, window")
        assert torch.equal(a, iq.cache_attention(cache, q, table, lengths, starts))


def test_attention_one_large_score(iq):
    """The running maximum jumps late, and early."""
    for spot in (0, 40, 777, 1500):
        for causal in (True, False):
            cache, q, table, lengths, starts = scene(iq, "int8", 1, 4, 64, 64, [1400], [101], 3)
            k, v = iq.cache_read(cache, table, lengths, ends([1501]), 1501)
            k[spot] = 40.0
            iq.cache_append(cache, k, v, table, lengths, ends([1501]))
            q.abs_()
            ao.check_attention(iq, cache, q, table, lengths, starts, causal=causal, what=f"at {spot}")


def test_attention_strides(iq):
    cache, q, table, lengths, starts = scene(iq, "e4m3", 2, 4, 128, 64, [100, 5], [33, 60], 4)
    want = iq.cache_attention(cache, q, table, lengths, starts)
    fused = torch.zeros(93, 14, 128, dtype=BF, device="cuda")
    fused[:, 3:11] = q
    assert torch.equal(iq.cache_attention(cache, fused[:, 3:11], table, lengths, starts), want)
    assert torch.equal(iq.cache_attention(cache, q.transpose(0, 1).contiguous().transpose(0, 1), table, lengths, starts), want)
    odd = torch.zeros(q.numel() + 4, dtype=BF, device="cuda")[4:].view_as(q)
    with pytest.raises(iq.IQError):
        iq.cache_attention(cache, odd, table, lengths, starts)
    with pytest.raises(ValueError):
        iq.cache_attention(cache, q, table, lengths, starts, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ---- together ---------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("inter", [False, True])
def test_answers(iq, fmt, inter):
    """Prompts of three sequences in two pieces, then tokens one by one: rotation, append and attention as a server calls
    them, every output held to 64 bits on the cache's own values."""
    g, heads, group, dim, page = gen(30), 2, 3, 64, 32
    freqs = iq.rotary_table(dim, 1e4, "parts", 4.0, 64)
    table, pages = tables([90, 60, 120], page, 3)
    cache = iq.make_cache(pages, heads, dim, fmt, page)
    ao.fill(cache, 1, garbage=True)
    have = [0, 0, 0]
    for new in ([40, 1, 33], [7, 20, 50], *[[1, 1, 1]] * 12, [0, 1, 0], [3, 1, 2]):
        have = [a + b for a, b in zip(have, new)]
        n, single = sum(new), set(new) == {1}
        fused = rand(g, n, heads * (group + 2), dim)
        q, k, v = fused[:, :heads * group], fused[:, heads * group:-heads], fused[:, -heads:]
        lengths, starts = whole(have), None if single else ends(new)
        q = iq.cache_append(cache, k, v, table, lengths, starts, q=q, rotary=freqs, interleaved=inter, amplitude=1.05)
        ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{have}")


def test_captured_steps(iq):
    """A decoding step captured once and replayed with new inputs, between eager work of the same kind; two graphs by turns."""
    g, heads, group, dim, batch = gen(31), 2, 4, 128, 6
    table, pages = tables([200] * batch, 64, 5)
    freqs = iq.rotary_table(dim)

    def make():
        c = iq.make_cache(pages, heads, dim, "e4m3", 64)
        c.codes.zero_()
        c.scales.zero_()
        return c

    def step(cache, x, lengths):
        q = iq.cache_append(cache, x[:, 8:10], x[:, 10:], table, lengths, q=x[:, :8], rotary=freqs)
        return iq.cache_attention(cache, q, table, lengths)

    x, lengths = rand(g, batch, 12, dim), whole([1] * batch)
    caches, graphs, outs = [make(), make()], [], []
    step(make(), x, lengths)
    torch.cuda.synchronize()
    for c in caches:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(c, x, lengths))
    eager = [make(), make()]
    for t in range(40):
        for which in range(2):
            x.copy_(rand(g, batch, 12, dim))
            lengths.fill_(t + 1)
            graphs[which].replay()
            got = outs[which].clone()
            want = step(eager[which], x, lengths)
            assert torch.equal(got, want), (t, which)
        torch.cuda.synchronize()
    assert all(torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) for a, b in zip(caches, eager))


def test_calls_on_a_named_stream_keep_their_buffers(iq):
    """Calls on a stream that is still busy, while the current stream takes and overwrites blocks of their sizes."""
    cache, q, table, lengths, starts = scene(iq, "int8", 2, 4, 128, 64, [3000, 100], [1, 90], 6)
    k, v = rand(gen(1), 91, 2, 128), rand(gen(2), 91, 2, 128)
    freqs, at = iq.rotary_table(128), torch.arange(91, device="cuda", dtype=I32)
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    calls = [lambda s: [iq.rotary(q, at, freqs, stream=s)], lambda s: [iq.rotary_backward(q, at, freqs, stream=s)],
             lambda s: [iq.cache_append(cache, k, v, table, lengths, starts, q=q, rotary=freqs, stream=s)],
             lambda s: iq.cache_read(cache, table, lengths, starts, 91, stream=s),
             lambda s: [iq.cache_attention(cache, q, table, lengths, starts, stream=s)]]
    for i, call in enumerate(calls):
        print("call", i, flush=True)
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            keep = [busy @ busy for _ in range(4)]
        got = call(side)
        for _ in range(3):
            blocks = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (256, 4096, 46592, 186368, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
            del blocks
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        torch.cuda.synchronize()
        del keep


def test_tensors_that_require_gradients(iq):
    cache, q, table, lengths, starts = scene(iq, "e4m3", 2, 2, 64, 64, [10], [5], 6)
    k, at, freqs = rand(gen(1), 5, 2, 64), torch.arange(5, device="cuda", dtype=I32), iq.rotary_table(64)
    leaf = q.clone().requires_grad_()
    calls = [lambda q: iq.rotary(q, at, freqs), lambda q: iq.rotary_backward(q, at, freqs),
             lambda q: iq.cache_append(cache, k, k, table, lengths, starts, q=q, rotary=freqs),
             lambda q: iq.cache_attention(cache, q, table, lengths, starts)]
    for call in calls:
        with pytest.raises(RuntimeError, match="no gradient passes"):
            call(leaf)
        want, got = call(q), torch.no_grad()(call)(leaf)
        assert torch.equal(got, want) and not got.requires_grad


# ---- calls of many kinds of sequences ---------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 8), (96, 3, 2), (128, 1, 6), (192, 2, 3), (256, 1, 4)])
def test_attention_mixed(iq, fmt, dim, heads, group):
    """Prompts, pieces behind a long cache, single tokens and sequences without new tokens in one call: rows split among
    workgroups and whole ones, of both kinds of kernels."""
    cases = (([0, 3000, 500, 17, 900], [700, 1, 90, 1, 0]), ([2000, 0], [64 // group, 64 // group + 1]), ([1, 1, 4000], [1, 300, 33]))
    for had, new in cases:
        cache, q, table, lengths, starts = scene(iq, fmt, heads, group, dim, 64, had, new, dim)
        for kw in (dict(), dict(causal=False), dict(window=333), dict(window=2500)):
            a = ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{had} {new} {kw}", **kw)
            assert torch.equal(a, iq.cache_attention(cache, q, table, lengths, starts, **kw))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,group", [(64, 2, 8), (96, 3, 3), (128, 1, 4), (192, 2, 4)])
def test_attention_short_pieces(iq, fmt, dim, heads, group):
    """Calls of short pieces only, up to and past 64 and 128 columns, behind short and long caches."""
    for had in (0, 600, 5000):
        for columns in ([128], [129], [65, 128, 40], [70] * 5, [128, 129, 1]):
            new = [max(1, n // group) for n in columns]
            cache, q, table, lengths, starts = scene(iq, fmt, heads, group, dim, 64, [had] * len(new), new, dim)
            for kw in (dict(), dict(window=100)):
                ao.check_attention(iq, cache, q, table, lengths, starts, what=f"{had} {new} {kw}", **kw)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_many_short_sequences(iq, fmt):
    """More sequences than a workgroup has threads, in a wide table: single tokens, and prompts of all short lengths."""
    n = 600
    for had, new in (([k % 37 for k in range(n)], [1] * n), ([0] * 90, [k % 45 for k in range(90)])):
        cache, q, table, lengths, starts = scene(iq, fmt, 2, 4, 64, 32, had, new, 9)
        wide = torch.full((len(had), 64), -1, dtype=I32, device="cuda")
        wide[:, :table.shape[1]] = table
        for t in (wide, table):
            ao.check_attention(iq, cache, q, t, lengths, starts, what=f"{len(had)}, {t.shape[1]}")
        if max(new) == 1:
            ao.check_attention(iq, cache, q, wide, lengths, what="without starts")


@pytest.mark.parametrize("width", [8, 200])
def test_attention_writes_its_rows_only(iq, width):
    """Rows behind the last sequence stay as they were, in all kernels; sequences whose table is too narrow see what it holds."""
    for had, new in (([100, 30, 0], [1, 5, 0]), ([400, 90, 0], [150, 1, 40]), ([0], [130])):
        cache, q, table, lengths, starts = scene(iq, "e4m3", 2, 4, 64, 64, had, new, 5)
        n = sum(new)
        t = torch.full((len(had), width), -1, dtype=I32, device="cuda")
        t[:, :min(width, table.shape[1])] = table[:, :width]
        long = torch.cat([q, rand(gen(3), 70, 8, 64)])
        out = torch.full_like(long, 7.0)
        got = iq.cache_attention(cache, long, t, lengths, starts, out=out)
        assert got is out and (out[n:] == 7).all()
        ao.check_attention(iq, cache, q, t, lengths, starts, got=out[:n], what=f"{had}")


def test_attention_without_pages(iq):
    """No pages, no table entries, no tokens, no sequences."""
    q, one = rand(gen(1), 90, 8, 128), whole([90])
    empty, some = iq.make_cache(0, 2, 128), iq.make_cache(3, 2, 128)
    some.scales.fill_(math.nan)
    for cache, table in ((empty, whole([[0, 1]])), (some, whole([[]]).view(1, 0)), (some, whole([[-1, 3]]))):
        for rows, starts in ((90, whole([0, 90])), (3, whole([0, 3])), (1, None)):
            out = torch.full_like(q[:rows], 7.0)
            assert not iq.cache_attention(cache, q[:rows], table, one, starts, out=out).any()
            k, v = iq.cache_read(cache, table, one, starts, rows)
            assert not k.any() and not v.any()
            iq.cache_append(cache, q[:rows, :2], q[:rows, 2:4], table, one, starts)
    assert torch.isnan(some.scales).all()
    assert iq.cache_attention(some, q[:0], whole([[0]]), whole([5]), whole([0, 0])).shape == (0, 8, 128)
    none = whole([]).view(0, 4)
    assert iq.cache_attention(some, q[:0], none, whole([])).shape == (0, 8, 128)
    out = torch.full_like(q, 7.0)
    assert (iq.cache_attention(some, q, none, whole([]), whole([0]), out=out) == 7).all()


def test_results_in_place_of_queries(iq):
    """Dense queries may be overwritten by their turned form and by their outputs, in all kernels."""
    freqs = iq.rotary_table(128)
    for had, new in (([5000, 90], [1, 1]), ([1000], [3]), ([3000, 5], [200, 1])):
        cache, q, table, lengths, starts = scene(iq, "e4m3", 2, 4, 128, 64, had, new, 8)
        want = iq.cache_attention(cache, q, table, lengths, starts)
        here = q.clone()
        assert iq.cache_attention(cache, here, table, lengths, starts, out=here) is here
        assert torch.equal(here, want)
        k = rand(gen(2), sum(new), 2, 128)
        want = iq.cache_append(cache, k, k, table, lengths, starts, q=q, rotary=freqs)
        d = iq._cache_desc(cache, table, lengths, starts, sum(new), q)
        a = iq.IQAppendDesc(iq.IQ_BF16, 0, sum(new), 8, 256, 128, 256, 128, 1024, 128, 128, 1.0, 0, 0)
        here = q.clone()
        assert iq.iq_cache_append(d, a, k.data_ptr(), k.data_ptr(), table.data_ptr(), lengths.data_ptr(), starts.data_ptr(), freqs.data_ptr(),
                                  here.data_ptr(), here.data_ptr(), cache.codes.data_ptr(), cache.scales.data_ptr(),
                                  torch.cuda.current_stream().cuda_stream) == iq.IQ_OK
        assert torch.equal(here, want)


def test_captured_prompts(iq):
    """A call with both kinds of sequences captured, in two graphs that share a workspace and are replayed by turns with other
    lengths, between eager calls."""
    cache, q, table, lengths, starts = scene(iq, "int8", 2, 4, 64, 64, [1500, 700, 40], [120, 1, 30], 21)
    need = iq.iq_cache_attention_workspace_bytes(iq._cache_desc(cache, table, lengths, starts, 151, q),
                                                 iq.IQAttentionDesc(iq.IQ_BF16, 1, 151, 8, 512, 64, 0, 0.125, 0))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    x, at, outs, graphs = [q.clone(), q.clone()], [lengths.clone(), lengths.clone()], [], []
    iq.cache_attention(cache, q, table, lengths, starts, workspace=ws)
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(iq.cache_attention(cache, x[i], table, at[i], starts, workspace=ws))
    full = lengths.tolist()
    for t in range(12):
        i = t % 2
        x[i].copy_(rand(gen(100 + t), 151, 8, 64))
        at[i].copy_(whole([n - (17 * t) % 30 for n in full]))
        graphs[i].replay()
        got = outs[i].clone()
        want = iq.cache_attention(cache, x[i], table, at[i], starts)
        assert torch.equal(got, want), t
        torch.cuda.synchronize()

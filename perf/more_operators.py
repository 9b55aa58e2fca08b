"""Measured cases of the attention half of a layer around an 8-bit cache: rotary positions, the paged cache's append and read, and attention over it.

`run` computes one pass either in plain torch operations (`own` false) or through the library (`own` true):

  rotary  a training step's rotation of queries or keys: y from x, and dx from dy
  append  keys rotated, keys and values quantized into the pages of their sequences, queries rotated on the way; then
          the sequences' keys and values read back
  attend  attention of the newest tokens of every sequence over what its pages hold

The cache: `codes` uint8 [pages, heads, page / 32, 2, 32 * dim] (INT8 or E4M3, keys then values of 32 tokens) and
`scales` float32 [pages, heads, page / 32, 2].  Keys of a block lie as [dim / 16, 32 tokens, 16], values as
[dim, 32 places], token t of the block at place PLACE[t].
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
BASE = 10000.0
CONTEXT = 4096                      # the context that scaled rotations were made for
LARGEST = {"e4m3": 448.0, "int8": 127.0}
PLACE = [(t >> 2 & 1) * 16 + (t >> 4) * 8 + (t >> 3 & 1) * 4 + (t & 3) for t in range(32)]


def listed():
    return [
        # the queries of a training batch, rotated forward and backward
        dict(name="rotary step", op="rotary", tokens=8192, heads=32, dim=128, rot=128, layout="half", scaling="none", far=8192, dtype="bf16"),
        # part of every head, neighbouring pairs, positions far past the trained context, full precision
        dict(name="rotary partial f32", op="rotary", tokens=1531, heads=12, dim=96, rot=40, layout="interleaved", scaling="parts", far=120000,
             dtype="f32"),
        # one sequence decoding, where only latency counts
        dict(name="append one token", op="append", fmt="e4m3", batch=1, least=1, most=1, shortest=700, longest=700, heads=32, kv=8, dim=128,
             rot=128, layout="half", page=64, dtype="bf16"),
        # a prompt written into an empty cache
        dict(name="append prompt", op="append", fmt="int8", batch=1, least=8192, most=8192, shortest=0, longest=0, heads=32, kv=8, dim=128,
             rot=128, layout="half", page=128, dtype="bf16"),
        # pieces of several prompts, every length odd, blocks that begin and end inside
        dict(name="append ragged f32", op="append", fmt="e4m3", batch=7, least=1, most=397, shortest=3, longest=1021, heads=10, kv=2, dim=64,
             rot=32, layout="interleaved", page=32, dtype="f32"),
        # one sequence decoding early in its answer
        dict(name="attend one token short", op="attend", fmt="e4m3", batch=1, least=1, most=1, shortest=500, longest=500, heads=32, kv=8, dim=128,
             page=64, window=0),
        # a batch decoding, contexts of every length
        dict(name="attend batch", op="attend", fmt="e4m3", batch=64, least=1, most=1, shortest=1024, longest=16384, heads=32, kv=8, dim=128,
             page=64, window=0),
        # one sequence decoding behind a very long context
        dict(name="attend long", op="attend", fmt="int8", batch=1, least=1, most=1, shortest=131072, longest=131072, heads=64, kv=8, dim=128,
             page=256, window=0),
        # several tokens a sequence, as when proposed tokens are checked
        dict(name="attend few tokens", op="attend", fmt="int8", batch=9, least=2, most=6, shortest=201, longest=4999, heads=16, kv=4, dim=256,
             page=32, window=0),
        # a whole prompt
        dict(name="attend prompt", op="attend", fmt="e4m3", batch=1, least=8192, most=8192, shortest=0, longest=0, heads=32, kv=8, dim=128,
             page=128, window=0),
        # pieces of prompts behind what the cache already holds, a sliding window, odd sizes
        dict(name="attend pieces window", op="attend", fmt="int8", batch=5, least=129, most=1501, shortest=0, longest=6001, heads=15, kv=3,
             dim=96, page=64, window=1000),
        # a small model's prompts
        dict(name="attend prompts narrow", op="attend", fmt="e4m3", batch=6, least=77, most=2047, shortest=0, longest=0, heads=12, kv=12, dim=64,
             page=32, window=0),
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        lo = max(lo, step)
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))) / step) * step))

    op = rng.choice(["rotary", "append", "attend", "attend"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    layout = rng.choice(["half", "interleaved"])
    if op == "rotary":
        heads = spread(1, 64)
        return dict(op=op, tokens=spread(1, max(1, min(16384, 8192 * 4096 // (heads * dim)))), heads=heads, dim=dim, rot=spread(2, dim, 2),
                    layout=layout, scaling=rng.choice(["none", "linear", "parts"]), far=spread(64, 1000000), dtype=rng.choice(["bf16", "bf16", "f32"]))
    kv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    case = dict(op=op, fmt=rng.choice(["e4m3", "int8"]), heads=kv * group, kv=kv, dim=dim, page=rng.choice([32, 64, 128, 256]))
    wide = kv * dim                                     # elements of a token's keys
    if op == "append":
        batch = rng.choice([1, spread(2, 48)])
        most = rng.choice([1, spread(1, max(1, 4000000 // (wide * batch)))])
        longest = spread(1, max(1, min(8192, 4000000 // (wide * batch))))
        return dict(case, batch=batch, least=rng.randint(1, most), most=most, shortest=rng.randint(0, longest), longest=longest,
                    rot=spread(2, dim, 2), layout=layout, dtype=rng.choice(["bf16", "bf16", "f32"]))
    window = rng.choice([0, 0, spread(16, 4096)])
    if rng.random() < 0.6:                              # single tokens, or a few
        batch = spread(1, 64)
        longest = spread(1, max(1, min(131072, 400000000 // (wide * batch))))
        most = rng.choice([1, 1, spread(2, 9)])
        return dict(case, batch=batch, least=1, most=most, shortest=rng.randint(1, longest), longest=longest, window=window)
    batch = spread(1, 8)
    cost = 4 * batch * kv * group * dim                 # operations for each pair of a query and a key
    most = spread(16, min(8192 // batch, math.isqrt(10 ** 12 // cost)))
    longest = rng.choice([0, spread(1, max(1, min(8192 - most, 5 * 10 ** 11 // (cost * most) - most // 2)))])
    return dict(case, batch=batch, least=rng.randint(1, most), most=most, shortest=rng.randint(0, longest), longest=longest, window=window)


def _sizes(case):
    """New tokens and cached tokens of every sequence."""
    def between(a, b, i):
        return a + (b - a) * i // max(1, case["batch"] - 1)

    n = case["batch"]
    return ([between(case["least"], case["most"], i) for i in range(n)],
            [between(case["shortest"], case["longest"], n - 1 - i) for i in range(n)])


def work(case):
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        return dict(bytes=4 * n * case["dim"] * e + 4 * case["tokens"], flops=6 * n * case["rot"])
    new, old = _sizes(case)
    wide = case["kv"] * case["dim"]
    if case["op"] == "append":
        t, whole = sum(new), sum(new) + sum(old)
        return dict(bytes=2 * t * (case["heads"] + case["kv"]) * case["dim"] * e + 2 * t * wide + whole * wide * (2 + 4),
                    flops=t * (3 * case["rot"] * (case["heads"] + case["kv"]) + 6 * wide) + 2 * whole * wide)
    seen = rows = 0
    for n, o in zip(new, old):
        w = case["window"] or n + o
        full = max(0, min(n, n + o - w))               # queries that the window cuts
        seen += full * w + (n - full) * o + (n - full) * (n - full + 1) // 2
        rows += min(n + o, w + n - 1)                  # tokens that some query sees
    return dict(bytes=4 * sum(new) * case["heads"] * case["dim"] + 2 * rows * wide + 8 * (rows // 32) * case["kv"],
                flops=4 * seen * case["heads"] * case["dim"])


# ---- inputs -----------------------------------------------------------------------
def _turns(rot, scaling):
    """Turns per position of every pair, and the amplitude."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    turns = BASE ** (-2 * i / rot) / (2 * math.pi)
    if scaling == "linear":
        return turns / 4, 1.0
    if scaling == "parts":                              # slow pairs stretched eight times, fast ones kept
        keep = ((CONTEXT * turns - 1) / (32 - 1)).clamp(0, 1)
        return turns / 8 * (1 - keep) + turns * keep, 0.1 * math.log(8) + 1
    return turns, 1.0


def _cache(case, pages, gen):
    """Pages full of quantized keys and values, as appended prompts leave them."""
    kv, dim, blocks = case["kv"], case["dim"], case["page"] // 32
    codes = torch.empty(pages, kv, blocks, 2, 32 * dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, kv, blocks, 2, device="cuda")
    at = torch.tensor(PLACE, device="cuda")
    many = max(1, (1 << 26) // (kv * blocks * 32 * dim))
    for p in range(0, pages, many):
        n = min(many, pages - p)
        for which in range(2):
            x = torch.randn(n, kv, blocks, 32, dim, generator=gen, device="cuda")
            if which == 0:
                x[..., :: max(1, dim // 4)] *= 6.0      # keys have channels that stand out
            s = x.abs().amax((3, 4)) / LARGEST[case["fmt"]]
            x = x / s[..., None, None]
            x = x.to(torch.float8_e4m3fn).view(torch.uint8) if case["fmt"] == "e4m3" else x.round().to(torch.int8).view(torch.uint8)
            if which == 0:
                x = x.view(n, kv, blocks, 32, dim // 16, 16).transpose(3, 4)
            else:
                x = torch.empty_like(x.transpose(3, 4)).index_copy_(4, at, x.transpose(3, 4))
            codes[p:p + n, :, :, which], scales[p:p + n, :, :, which] = x.reshape(n, kv, blocks, 32 * dim), s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s, op, dim = dict(case), case["op"], case["dim"]
    dt = DTYPE[case.get("dtype", "bf16")]
    if op == "rotary":
        turns, s["amplitude"] = _turns(case["rot"], case["scaling"])
        s["turns"] = turns.cuda()
        s["x"], s["dy"] = normal(case["tokens"], case["heads"], dim, dtype=dt), normal(case["tokens"], case["heads"], dim, dtype=dt)
        s["positions"] = torch.randint(case["far"], (case["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
        return s
    new, old = _sizes(case)
    lengths = [n + o for n, o in zip(new, old)]
    need = [-(-n // case["page"]) for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    s["page_table"] = torch.full((case["batch"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        s["page_table"][i, :n] = order[at:at + n]
        at += n
    s["codes"], s["scales"] = _cache(case, pages, gen)
    starts = [sum(new[:i]) for i in range(case["batch"] + 1)]
    s["lengths"], s["starts"] = whole(lengths), whole(starts)
    s["single"] = max(new) == 1                         # a token a sequence: no starts are needed
    s["q"] = normal(starts[-1], case["heads"], dim, dtype=dt)
    if op == "append":
        s["turns"] = _turns(case["rot"], "none")[0].cuda()
        s["k"], s["v"] = normal(starts[-1], case["kv"], dim, dtype=dt), normal(starts[-1], case["kv"], dim, dtype=dt)
        s["k"][..., :: dim // 4] *= 6.0
        s["total"] = sum(lengths)
        s["whole"] = whole([sum(lengths[:i]) for i in range(case["batch"] + 1)])
    else:
        s["q"] *= 1.5                                   # some keys stand out for a query
    return s


# ---- the plain form ---------------------------------------------------------------
def _rotate(x, positions, turns, layout, amplitude, way):
    """The first 2 * len(turns) elements of every head turned by `way` times the position's angles, FP32."""
    rot = 2 * turns.numel()
    t = positions.double()[:, None] * turns
    angle = (t - t.round()) * (2 * math.pi)
    cos, sin = (torch.cos(angle) * amplitude).float()[:, None], (torch.sin(angle) * amplitude * way).float()[:, None]
    x = x.float()
    first, second = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = first * cos - second * sin, second * cos + first * sin
    turned = torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _decode(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _blocks(s, ids):
    """Keys and values [..., heads, 32, dim] of the blocks `ids` (page * blocks a page + block) as code values."""
    kv, dim, blocks = s["kv"], s["dim"], s["page"] // 32
    got = s["codes"][ids // blocks, :, ids % blocks]                              # [..., heads, 2, 32 * dim]
    lead = got.shape[:-2]
    k = got[..., 0, :].reshape(*lead, dim // 16, 32, 16).transpose(-2, -3).reshape(*lead, 32, dim)
    v = got[..., 1, :].reshape(*lead, dim, 32)[..., torch.tensor(PLACE, device="cuda")].transpose(-1, -2)
    return _decode(k.contiguous(), s["fmt"]), _decode(v.contiguous(), s["fmt"])


def _rows_of(starts, total):
    """Sequence and number within it of `total` tokens."""
    i = torch.arange(total, device="cuda")
    b = torch.searchsorted(starts.long(), i, right=True) - 1
    return b, i - starts.long()[b]


def _plain_append(s):
    kv, dim, blocks, fmt = s["kv"], s["dim"], s["page"] // 32, s["fmt"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    tokens, batch = s["q"].shape[0], s["batch"]
    b, i = _rows_of(starts, tokens)
    n = starts[1:] - starts[:-1]
    first = lengths - n                                                           # position of each sequence's first new token
    position = first[b] + i
    q = _rotate(s["q"], position, s["turns"], s["layout"], 1.0, 1)
    fresh = [_rotate(s["k"], position, s["turns"], s["layout"], 1.0, 1), s["v"].float()]
    many = (s["most"] + 62) // 32                                                 # blocks that a sequence may touch
    block = torch.minimum((first // 32)[:, None] + torch.arange(many, device="cuda"), ((lengths - 1) // 32)[:, None])
    ids = s["page_table"].long().gather(1, block // blocks) * blocks + block % blocks          # [batch, many]
    place = block[:, :, None] * 32 + torch.arange(32, device="cuda")              # positions of the blocks' tokens
    is_new = ((place >= first[:, None, None]) & (place < lengths[:, None, None]))[:, :, None, :, None]
    is_old = (place < first[:, None, None])[:, :, None, :, None]
    row = (place - first[:, None, None]).clamp_min(0) + starts[:-1, None, None]
    row = row.clamp_max(tokens - 1)
    old_codes = _blocks(s, ids)
    scales = s["scales"][ids // blocks, :, ids % blocks]                          # [batch, many, heads, 2]
    kept = is_old.any(3).squeeze(-1)                                              # [batch, many, 1]
    new_codes, new_scales = [], []
    for which in range(2):
        x = fresh[which][row].transpose(2, 3)                                     # [batch, many, heads, 32, dim]
        amax = torch.where(is_new, x.abs(), 0).amax((3, 4))
        want, had = amax / LARGEST[fmt], scales[..., which]
        mw, ew = torch.frexp(want)
        mh, eh = torch.frexp(had)
        up = torch.where(kept & (had > 0) & (want > had), ew - eh + (mw > mh).int(), 0)        # doublings of the old scale
        scale = torch.where(kept & (had > 0), torch.ldexp(had, up), want)
        y = x / torch.where(scale > 0, scale, 1)[..., None, None]
        z = torch.ldexp(old_codes[which], -up[..., None, None])
        y = torch.where(is_new, y, z).clamp(-LARGEST[fmt], LARGEST[fmt])
        y = y.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else y.round().to(torch.int8).view(torch.uint8)
        new_codes.append(y)
        new_scales.append(scale)
    there = s["codes"][ids // blocks, :, ids % blocks]                            # what lies behind the sequence stays
    written = (is_new | is_old).expand(batch, many, kv, 32, dim)
    k = new_codes[0].view(batch, many, kv, 32, dim // 16, 16).transpose(3, 4).flatten(3)
    mk = written.reshape(batch, many, kv, 32, dim // 16, 16).transpose(3, 4).flatten(3)
    token = torch.tensor([PLACE.index(p) for p in range(32)], device="cuda")
    v = new_codes[1].transpose(3, 4)[..., token].flatten(3)
    mv = written.transpose(3, 4)[..., token].flatten(3)
    there = torch.stack((torch.where(mk, k, there[..., 0, :]), torch.where(mv, v, there[..., 1, :])), 3)
    s["codes"][ids // blocks, :, ids % blocks] = there
    s["scales"][ids // blocks, :, ids % blocks] = torch.stack(new_scales, 3)
    # the sequences' keys and values, read back
    b, i = _rows_of(s["whole"], s["total"])
    page = s["page_table"].long()[b, i // s["page"]]
    inside = (i % s["page"]) // 32
    got, at, scale = s["codes"], i % 32, s["scales"][page, :, inside]
    k = got[:, :, :, 0].view(-1, kv, blocks, dim // 16, 32, 16)[page, :, inside, :, at].flatten(2)
    v = got[:, :, :, 1].view(-1, kv, blocks, dim, 32)[page, :, inside, :, torch.tensor(PLACE, device="cuda")[at]]
    out = [(_decode(c.contiguous(), fmt) * scale[:, :, w, None]).to(torch.bfloat16) for w, c in enumerate((k, v))]
    return {"q": q.to(s["q"].dtype), "k": out[0], "v": out[1]}


def _plain_attend(s):
    kv, dim, group = s["kv"], s["dim"], s["heads"] // s["kv"]
    starts, lengths, batch = s["starts"].long(), s["lengths"].long(), s["batch"]
    blocks, width = s["page"] // 32, s["page_table"].shape[1]
    block = torch.arange(width * blocks, device="cuda")
    ids = s["page_table"].long()[:, block // blocks].clamp_min(0) * blocks + block % blocks    # [batch, blocks]
    scale = s["scales"][ids // blocks, :, ids % blocks].permute(3, 0, 2, 1)       # [2, batch, heads, blocks]
    k, v = ((x * y[..., None, None]).flatten(2, 3) for x, y in zip((y.transpose(1, 2) for y in _blocks(s, ids)), scale))
    tokens, most = s["q"].shape[0], s["most"]
    i = torch.arange(most, device="cuda")
    q = s["q"].float()[(starts[:-1, None] + i).clamp_max(tokens - 1)]             # [batch, most, heads, dim]
    q = q.view(batch, most, kv, group, dim).transpose(1, 2).reshape(batch, kv, most * group, dim)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * dim ** -0.5
    key = torch.arange(width * s["page"], device="cuda")
    n = starts[1:] - starts[:-1]
    position = (lengths - n)[:, None] + i                                         # [batch, most]
    seen = (key <= position[..., None]) & (key < lengths[:, None, None])
    if s["window"]:
        seen = seen & (key > position[..., None] - s["window"])
    hidden = ~seen[:, None, :, None]                                              # [batch, 1, most, 1, keys]
    score = score.view(batch, kv, most, group, -1).masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, kv, most * group, -1), v).view(batch, kv, most, group, dim)
    o = (o / total.clamp_min(1e-38)).transpose(1, 2).reshape(batch, most, kv * group, dim)
    b, i = _rows_of(starts, tokens)
    return {"o": o[b, i].to(s["q"].dtype)}


def _plain(s):
    if s["op"] == "rotary":
        turn = (s["positions"], s["turns"], s["layout"], s["amplitude"])
        return {"y": _rotate(s["x"], *turn, 1).to(s["x"].dtype), "dx": _rotate(s["dy"], *turn, -1).to(s["x"].dtype)}
    return _plain_append(s) if s["op"] == "append" else _plain_attend(s)


# ---- the library's form -----------------------------------------------------------
def _library(s):
    import int_quantization_amd as iq

    inter = s.get("layout") == "interleaved"
    if s["op"] == "rotary":
        turn = dict(interleaved=inter, amplitude=s["amplitude"])
        return {"y": iq.rotary(s["x"], s["positions"], s["turns"], **turn), "dx": iq.rotary_backward(s["dy"], s["positions"], s["turns"], **turn)}
    cache = iq.KVCache(s["codes"], s["scales"], s["fmt"], s["kv"], s["dim"], s["page"])
    starts = None if s["single"] else s["starts"]
    if s["op"] == "append":
        q = iq.cache_append(cache, s["k"], s["v"], s["page_table"], s["lengths"], starts, q=s["q"], rotary=s["turns"], interleaved=inter)
        k, v = iq.cache_read(cache, s["page_table"], s["lengths"], s["whole"], s["total"])
        return {"q": q, "k": k, "v": v}
    return {"o": iq.cache_attention(cache, s["q"], s["page_table"], s["lengths"], starts, window=s["window"])}


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# ---- 64 bits, from the definitions ------------------------------------------------
def _turned64(x, positions, turns, layout, amplitude, way):
    """Pairs as complex numbers times amplitude * e^(i angle)."""
    rot, x = 2 * turns.numel(), x.double()
    t = torch.remainder(positions.double()[:, None] * turns, 1.0) * (2 * math.pi * way)
    unit = torch.polar(torch.full_like(t, amplitude), t)[:, None]
    y = x.clone()
    if layout == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * unit
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _value64(codes, fmt):
    c = codes.long()
    if fmt == "int8":
        return torch.where(c > 127, c - 256, c).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10)) * torch.where(c > 127, -1.0, 1.0)


def _round64(y, fmt):
    """The nearest value that a code stands for, ties to even."""
    y = y.clamp(-LARGEST[fmt], LARGEST[fmt])
    if fmt == "int8":
        return torch.round(y)
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _sequence64(s, i):
    """Keys and values [heads, tokens, dim] of sequence i's pages as code values, and the scales [heads, tokens]."""
    kv, dim = s["kv"], s["dim"]
    pages = s["page_table"][i].long()
    pages = pages[pages >= 0]
    codes, scales = s["codes"][pages].transpose(0, 1).flatten(1, 2), s["scales"][pages].transpose(0, 1).flatten(1, 2)
    keys = codes[:, :, 0].view(kv, -1, dim // 16, 32, 16)
    values = codes[:, :, 1].view(kv, -1, dim, 32)
    k = torch.stack([keys[:, :, :, t].flatten(2) for t in range(32)], 2).flatten(1, 2)
    v = torch.stack([values[..., PLACE[t]] for t in range(32)], 2).flatten(1, 2)
    return [_value64(x, s["fmt"]) for x in (k, v)], [scales[:, :, w].double().repeat_interleave(32, 1) for w in range(2)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        turn = (s["positions"], s["turns"], case["layout"], s["amplitude"])
        return {"y": _turned64(s["x"], *turn, 1), "dx": _turned64(s["dy"], *turn, -1)}
    new, old = _sizes(case)
    outs = {"q": [], "k": [], "v": [], "o": []}
    at = 0
    for i, (n, o) in enumerate(zip(new, old)):
        values, scales = _sequence64(s, i)
        q = s["q"][at:at + n]
        if case["op"] == "append":
            positions = torch.arange(o, o + n, device="cuda")
            outs["q"].append(_turned64(q, positions, s["turns"], case["layout"], 1.0, 1))
            fresh = [_turned64(s["k"][at:at + n], positions, s["turns"], case["layout"], 1.0, 1), s["v"][at:at + n].double()]
            for name, x, c, sc in zip("kv", fresh, values, scales):
                x, c, sc = x.transpose(0, 1), c[:, :o + n].clone(), sc[:, :o + n].clone()
                first = o // 32 * 32                   # the block that both old and new tokens share
                if first < o:
                    had = sc[:, first].clone()
                    want = x[:, : 32 - (o - first)].abs().amax((1, 2)) / LARGEST[case["fmt"]]
                    up = torch.exp2(torch.ceil(torch.log2(want / had)).clamp_min(0))
                    c[:, first:o] = _round64(c[:, first:o] / up[:, None, None], case["fmt"])
                    end = min(o + n, first + 32)
                    sc[:, first:end] = (had * up)[:, None]
                    c[:, o:end] = _round64(x[:, :end - o] / (had * up)[:, None, None], case["fmt"])
                for b in range(-(-o // 32) * 32, o + n, 32):
                    part = x[:, b - o:b - o + 32]
                    want = part.abs().amax((1, 2)) / LARGEST[case["fmt"]]
                    sc[:, b:b + 32] = want[:, None]
                    c[:, b:min(b + 32, o + n)] = _round64(part / want[:, None, None], case["fmt"])
                outs[name].append((c * sc[..., None]).transpose(0, 1))
        else:
            (k, v), (sk, sv) = values, scales
            k, v = k[:, :o + n] * sk[:, :o + n, None], v[:, :o + n] * sv[:, :o + n, None]
            group = case["heads"] // case["kv"]
            key, position = torch.arange(o + n, device="cuda"), torch.arange(o, o + n, device="cuda")
            seen = key <= position[:, None]
            if case["window"]:
                seen &= key > position[:, None] - case["window"]
            o_ = torch.empty(n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
            for h in range(case["heads"]):
                z = torch.matmul(q[:, h].double(), k[h // group].t().contiguous()) / math.sqrt(case["dim"])
                o_[:, h] = torch.matmul(torch.softmax(z.masked_fill(~seen, -math.inf), 1), v[h // group])
            outs["o"].append(o_)
        at += n
    return {name: torch.cat(parts) for name, parts in outs.items() if parts}

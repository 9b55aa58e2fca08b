"""Plain 64-bit forms of the feed-forward operators and the error bounds their FP32 kernels are held to.

U is half a step of FP32, HALF[t] half a step of an output type, both relative
to the value.  A sum of n terms in FP32, in any order of at most `depth`
additions per term, is off by at most depth * U * sum |terms|.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -126            # below the smallest normal number nothing is relative
BLOCK = {"int4": 128, "nvfp4": 16, "mxfp4": 32}
ACTS = ("silu", "gelu", "gelu_tanh")


def act_parts(g, kind):
    """act(g) and act'(g) in 64 bits."""
    g = g.double()
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if kind == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def act_error(g, kind):
    """What FP32 evaluation of act(g) may be off by: a few roundings, the exponential's argument (rounded, so off by
    |argument| U) and erf's cancellation against 1."""
    g = g.double()
    if kind == "gelu":
        return 8 * U * g.abs()
    arg = g.abs() if kind == "silu" else 1.6 * (g.abs() + 0.044715 * g.abs() ** 3)
    return (16 + 8 * torch.clamp(arg, max=100.0)) * U * act_parts(g, kind)[0].abs() + TINY


# ---- layer norm -----------------------------------------------------------------
def norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if w is not None:
        y = y * w.double()
    return (y if b is None else y + b.double()), mean, rstd


def norm_bounds(x, w, b, eps):
    """Bounds of y (before its rounding), mean and rstd.  A thread adds cols / 256 terms at most before the tree."""
    y, mean, rstd = norm(x, w, b, eps)
    x = x.double()
    cols = x.shape[1]
    depth = math.ceil(cols / 256) * 8 + 24
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if w is None else w.double().abs()
    b = torch.zeros(cols, dtype=torch.float64, device=x.device) if b is None else b.double().abs()
    e_mean = depth * U * x.abs().mean(1) + TINY
    d = (x - mean[:, None]).abs()
    e_d = e_mean[:, None] + U * d
    var = (d * d).mean(1)
    e_var = (depth + 4) * U * var + (2 * d * e_d + e_d * e_d).mean(1)
    e_rel = 0.5 * e_var * rstd * rstd + 4 * U              # of rstd
    e_y = (d * rstd[:, None] * w) * (e_rel[:, None] + 4 * U) + e_d * rstd[:, None] * w * (1 + e_rel[:, None]) + 2 * U * (y.abs() + b)
    return (y, mean, rstd), (e_y, e_mean, e_rel * rstd)


def norm_grad(dy, x, w, mean, rstd):
    """dx, dweight, dbias from the mean and rstd that the kernel is given, and their bounds before rounding."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, cols = x.shape
    n = (x - mean) * rstd
    a = dy if w is None else dy * w.double()
    s1, s2 = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    dx = rstd * (a - s1 - n * s2)
    depth = math.ceil(cols / 256) * 8 + 24
    e_n = 3 * U * n.abs()
    e_s1 = (depth + 2) * U * a.abs().mean(1, keepdim=True)
    e_s2 = (depth + 6) * U * (a * n).abs().mean(1, keepdim=True)
    e_dx = rstd.abs() * (U * a.abs() + e_s1 + n.abs() * e_s2 + s2.abs() * e_n + 4 * U * (a.abs() + s1.abs() + (n * s2).abs()))
    deep = math.ceil(rows / 64) + 96
    dw, db = (dy * n).sum(0), dy.sum(0)
    e_dw = (deep + 4) * U * (dy * n).abs().sum(0)
    e_db = deep * U * dy.abs().sum(0)
    return (dx, dw, db), (e_dx, e_dw, e_db)


# ---- gated block ------------------------------------------------------------------
def product(x, w):
    """x w^T in 64 bits and the bound of its FP32 sum over exact products."""
    x, wt = x.double(), w.double().t().contiguous()
    return x @ wt, (x.shape[1] + 2) * U * (x.abs() @ wt.abs()) + TINY


def gate(g, u, e_g, e_u, kind):
    """h = act(g) u and its bound, from g and u and theirs."""
    a = act_parts(g, kind)[0]
    e_a = 1.2 * e_g + act_error(g, kind)
    return a * u, u.abs() * e_a + a.abs() * e_u + e_a * e_u + 2 * U * (a * u).abs()


def gated(x, wg, wu, kind):
    (g, e_g), (u, e_u) = product(x, wg), product(x, wu)
    return gate(g, u, e_g, e_u, kind)


def gated_grad(dh, x, wg, wu, kind):
    """dx, dwg, dwu and their bounds: dg and du are rounded to BF16 once, then summed in FP32."""
    (g, e_g), (u, e_u) = product(x, wg), product(x, wu)
    dh, x, wg, wu = dh.double(), x.double(), wg.double(), wu.double()
    a, s = act_parts(g, kind)
    dg, du = dh * u * s, dh * a
    h = HALF[torch.bfloat16]
    # act'' is at most 1.2 in magnitude and act' 1.2
    e_dg = h * dg.abs() + dh.abs() * (s.abs() * e_u + u.abs() * (1.2 * e_g + 48 * U * (1 + g.abs()))) * (1 + h) + TINY
    e_du = h * du.abs() + dh.abs() * (1.2 * e_g + act_error(g, kind)) * (1 + h) + TINY

    def out(parts):
        value = sum(p @ q for p, _, q in parts)
        size = sum(p.abs() @ q.abs() for p, _, q in parts)
        terms = sum(p.shape[1] for p, _, _ in parts)
        return value, sum(e @ q.abs() for _, e, q in parts) * 1.01 + (terms + 20) * U * size + TINY

    dx = out([(dg, e_dg, wg), (du, e_du, wu)])
    dwg = out([(dg.t().contiguous(), e_dg.t().contiguous(), x)])
    dwu = out([(du.t().contiguous(), e_du.t().contiguous(), x)])
    return (dx[0], dwg[0], dwu[0]), (dx[1], dwg[1], dwu[1])


# ---- packed weights ------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def unpack(fmt, codes, scales, global_scale=None):
    """Values of packed weights in 64 bits, and the size the product's bound counts each with."""
    rows, half = codes.shape
    nib = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, 2 * half).long()
    if fmt == "int4":
        v = torch.where(nib > 7, nib - 16, nib).double()
        s = scales.view(torch.float16).double()
    else:
        v = torch.tensor(E2M1 + tuple(-e for e in E2M1), dtype=torch.float64, device=codes.device)[nib]
        if fmt == "mxfp4":
            s = torch.exp2(scales.double() - 127)
            s[scales == 255] = float("nan")
        else:
            s = scales.view(torch.float8_e4m3fn).double() * global_scale.double()
    s = s.repeat_interleave(BLOCK[fmt], 1)
    return v * s, (v.abs() + (6 if fmt == "int4" else 0)) * s.abs()


def packed(x, weights):
    """x w^T for unpacked weights (value, size) and its bound."""
    w, m = weights
    x = x.double()
    return x @ w.t().contiguous(), (2 * x.shape[1] + 8) * U * (x.abs() @ m.t().contiguous()) + TINY


# ---- comparison ----------------------------------------------------------------------
def assert_within(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type, and the same places not finite."""
    g = got.double()
    assert g.shape == want.shape, f"{what}: shape {tuple(g.shape)} and {tuple(want.shape)}"
    if not g.numel():
        return
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(g[inf], want[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    off = (g - want).abs()[fine]
    most = (bound + HALF[got.dtype] * (want.abs() + bound))[fine]
    if off.numel():
        worst = (off / most.clamp_min(TINY)).max().item()
        assert worst <= 1, f"{what}: {worst:.3g} times its bound"

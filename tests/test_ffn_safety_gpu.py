"""The feed-forward operators on the GPU where operands are short or uncommon and where streams meet."""
import pytest
import torch

import ffn_oracle as fo
from test_ffn_gpu import BF, F32, any_weights, gen, iq, rand, values  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- packed weights: a workgroup's rows shorter than a step ---------------------------
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows", [1, 2, 3, 17, 33])
def test_packed_lone_short_rows(iq, fmt, rows):  # noqa: F811
    """One to three rows, or one in the last workgroup, of fewer codes than a step of 128."""
    for cols in range(32, 289, 32):
        q = any_weights(iq, rows, cols, fmt, cols)
        for n1 in (1, 5, 16, 33):
            x = rand(gen(n1), n1, cols)
            want = fo.packed(x, values(q))
            fo.assert_within(iq.packed_gemv(q, x, F32), *want, f"{cols} columns, {n1} tokens")
            h = iq.packed_gated(q, q, torch.zeros_like(x), "silu", BF)
            assert not h.any()


# ---- a named stream -----------------------------------------------------------------------
def test_calls_on_a_named_stream_keep_their_buffers(iq):  # noqa: F811
    """Every call on a stream of its own that is still busy, while the current stream takes blocks of the sizes of the calls'
    results and workspaces and overwrites them: the same bits as without."""
    g = gen(60)
    x, wg, wu = rand(g, 300, 256), rand(g, 512, 256, scale=0.06), rand(g, 512, 256, scale=0.06)
    dh, dy, few = rand(g, 300, 512, scale=0.1), rand(g, 300, 256), x[:7].contiguous()
    y, mean, rstd = iq.layer_norm(x)
    h, saved = iq.gated(x, wg, wu, save=True)
    q, zp = iq.quantize(wg, "nvfp4", "block", stats=False), iq.quantize(wg, "int4zp", "block", stats=False)
    mx, mxa = iq.quantize(wg, "mxfp4", "block", stats=False), iq.quantize(x, "mxfp4", "block", stats=False)

    def outputs(t):
        if isinstance(t, iq.Quantized):
            return [u for u in (t.codes, t.scales, t.global_scale, t.xhat, t.shifts) if u is not None]
        return [t] if torch.is_tensor(t) else list(t)

    calls = [lambda s: iq.layer_norm(x, stream=s), lambda s: iq.layer_norm_backward(dy, x, None, mean, rstd, stream=s),
             lambda s: iq.gated(x, wg, wu, save=True, stream=s), lambda s: iq.gated_backward(dh, x, wg, wu, saved, stream=s),
             lambda s: iq.packed_gemv(q, few, F32, stream=s), lambda s: iq.packed_gated(q, q, few, stream=s),
             lambda s: iq.quantize(x, "nvfp4", "block", xhat_dtype=F32, stream=s), lambda s: iq.quantize(x, "int8", "tensor", stream=s),
             lambda s: iq.quantize(x, "int4zp", "block", stream=s), lambda s: iq.amax(x, stream=s), lambda s: iq.dequantize(q, stream=s),
             lambda s: iq.zp_gemm(zp, few, stream=s), lambda s: iq.mx_gemm(mx, mxa, stream=s), lambda s: iq.mxw_gemm(mx, few, stream=s)]
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, generator=g, device="cuda")
    sizes = [n for n in (256, 512, 1024, 4096, 65536, 153600, 307100, 614400, 921600, 1228800) for _ in range(4)]
    for k, call in enumerate(calls):
        print("call", k, flush=True)
        want = [t.clone() for t in outputs(call(None))]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            keep = [busy @ busy for _ in range(4)]         # a few milliseconds before the call's kernels
        got = outputs(call(side))
        for _ in range(3):
            blocks = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
            del blocks
        side.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), k
        torch.cuda.synchronize()
        del keep


def test_gated_save_by_truth(iq):  # noqa: F811
    x, w = torch.zeros(3, 64, dtype=BF, device="cuda"), torch.zeros(8, 64, dtype=BF, device="cuda")
    h, saved = iq.gated(x, w, w, save=1)
    assert h.shape == (3, 8) and saved.shape == (2, 3, 8) and torch.is_tensor(iq.gated(x, w, w, save=0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 5, 3000])
def test_layer_norm_rows_without_elements(iq, dtype, rows):  # noqa: F811
    """Sums of nothing: mean 0 and rstd 1 / sqrt(eps), on both ways through the binding."""
    x = torch.empty((rows, 0), dtype=dtype, device="cuda")
    for stream in (None, torch.cuda.current_stream()):
        for _ in range(3):
            old = [torch.full((rows,), float("nan"), device="cuda") for _ in range(8)]
            old += [torch.full((2, rows), float("nan"), device="cuda") for _ in range(8)]
            del old                                    # what the allocator hands out next
            y, mean, rstd = iq.layer_norm(x, eps=0.25, stream=stream)
            assert y.shape == x.shape and torch.equal(mean, torch.zeros(rows, device="cuda"))
            assert torch.equal(rstd, torch.full((rows,), 2.0, device="cuda"))
        dx, dw, db = iq.layer_norm_backward(x, x, None, mean, rstd, stream=stream)
        assert dx.shape == x.shape and dw.shape == db.shape == (0,)


def test_tensors_that_require_gradients_on_the_gpu(iq):  # noqa: F811
    """Refused on the short path too, and taken under no_grad()."""
    g = gen(70)
    x, w, p = rand(g, 5, 128), rand(g, 32, 128), rand(g, 128, offset=1.0)
    q = iq.quantize(w, "int4", "block", stats=False)
    y, mean, rstd = iq.layer_norm(x, p)
    h, saved = iq.gated(x, w, w, save=True)
    z = iq.packed_gemv(q, x)
    calls = [(lambda x, w, p: iq.layer_norm(x, p), (y, mean, rstd)), (lambda x, w, p: (iq.gated(x, w, w),), (h,)),
             (lambda x, w, p: iq.layer_norm_backward(y, x, p, mean, rstd), iq.layer_norm_backward(y, x, p, mean, rstd)),
             (lambda x, w, p: iq.gated_backward(h, x, w, w, saved), iq.gated_backward(h, x, w, w, saved)),
             (lambda x, w, p: (iq.packed_gemv(q, x),), (z,))]
    leaf = [t.clone().requires_grad_() for t in (x, w, p)]
    for call, want in calls:
        with pytest.raises(RuntimeError, match="no gradient passes"):
            call(*leaf)
        for got in (call(x, w, p), torch.no_grad()(call)(*leaf)):
            assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,tokens", [(6128, (1, 8, 16)), (6144, (1, 4, 5, 8, 9, 16)), (6161, (3, 7, 16, 17)), (3056, (17, 32)), (3089, (20, 33)),
                                         (1537, (49, 64))])
def test_packed_workgroups_around_the_choice_of_rows(iq, fmt, rows, tokens):  # noqa: F811
    """16 or 32 rows to a workgroup, chosen by the number of workgroups, with every way of staging tokens."""
    q = any_weights(iq, rows, 384 if fmt == "int4" else 352, fmt, rows)
    for n1 in tokens:
        x = rand(gen(n1), n1, q.cols)
        fo.assert_within(iq.packed_gemv(q, x, F32), *fo.packed(x, values(q)), f"{n1} tokens")


# ---- packed weights: both ends of the MXFP4 scales ------------------------------------------
def mx_weights(iq, rows, cols, low, high, seed):  # noqa: F811
    q = any_weights(iq, rows, cols, "mxfp4", seed)
    q.scales.random_(low, high + 1, generator=gen(seed))
    return q


@pytest.mark.parametrize("n1", [1, 5, 16, 33])
@pytest.mark.parametrize("low,high,exponent", [(0, 0, 100), (1, 1, 100), (0, 3, 100), (0, 40, 90), (140, 200, -60), (200, 252, -100),
                                               (252, 252, -120)])
def test_packed_mx_scales_of_every_size(iq, n1, low, high, exponent):  # noqa: F811
    """Scale bytes 0 and 1, whose weights are subnormal BF16, to 252, the last whose weights BF16 holds all of, with
    activations that bring the products back to ordinary numbers."""
    for rows, cols in ((40, 96), (33, 1184), (4133, 256)):
        q = mx_weights(iq, rows, cols, low, high, low + n1)
        x = (rand(gen(high), n1, cols, dtype=F32) * 2.0 ** exponent).to(BF)
        g, e = fo.packed(x, values(q))
        fo.assert_within(iq.packed_gemv(q, x, F32), g, e, f"{rows} rows")
        if high < 64:                                  # products near 1, where act has something to say
            fo.assert_within(iq.packed_gated(q, q, x, "silu", F32), *fo.gate(g, g, e, e, "silu"), f"gated, {rows} rows")


@pytest.mark.parametrize("n1", [1, 20])
@pytest.mark.parametrize("byte", [253, 254])
def test_packed_mx_weights_past_bf16_are_infinite(iq, n1, byte):  # noqa: F811
    """Of scale bytes 253 and 254 the largest codes' weights are 2^128 and more, infinite as iq_dequantize gives them."""
    q = mx_weights(iq, 48, 256, byte, byte, byte)
    q.codes[0] = 0x11                                  # the smallest code alone: all finite
    q.codes[1, :] = 0x99
    x = torch.full((n1, 256), 2.0 ** -130, dtype=BF, device="cuda")
    w, m = values(q)
    past = w.abs() >= 2.0 ** 128
    assert torch.equal(torch.isinf(iq.dequantize(q)), past) and torch.equal(torch.isinf(iq.dequantize(q, BF)), past)
    w = torch.where(past, w.sign() * float("inf"), w)
    z = iq.packed_gemv(q, x, F32)
    want, e = fo.packed(x, (w, torch.where(past, torch.zeros_like(m), m)))
    fo.assert_within(z, want, e, "z")
    assert torch.isfinite(z[:, :2]).all() and not torch.isfinite(z[:, 2:]).any()


# ---- activations far out and in their tails ---------------------------------------------------
@pytest.mark.parametrize("act", fo.ACTS)
def test_gated_very_far_arguments(iq, act):  # noqa: F811
    """g of either sign from 1 to 2^119, whose square is infinite: no product of 0 and infinity, forward or backward."""
    tokens, cols, features = 240, 64, 64
    x = torch.zeros(tokens, cols, dtype=BF, device="cuda")
    x[:120, 0] = torch.exp2(torch.arange(120, device="cuda").float()).to(BF)
    x[120:, 0] = -x[:120, 0]
    x[:, 1] = 1
    wg, wu = torch.zeros(features, cols, dtype=BF, device="cuda"), torch.zeros(features, cols, dtype=BF, device="cuda")
    wg[:, 0], wu[:, 1] = 1, 2
    dh = torch.full((tokens, features), 2.0 ** -100, dtype=BF, device="cuda")
    h, saved = iq.gated(x, wg, wu, act, save=True)
    fo.assert_within(h, *fo.gated(x, wg, wu, act), "h")
    want, bound = fo.gated_grad(dh, x, wg, wu, act)
    for got, r, e, what in zip(iq.gated_backward(dh, x, wg, wu, saved, act), want, bound, ("dx", "dwg", "dwu")):
        r = torch.where(r.abs() >= 2.0 ** 128, r.sign() * float("inf"), r)     # x act(x) of the farthest: more than FP32 holds
        fo.assert_within(got, r, e, what)


def tail_inputs():
    """g from -9 to 9 in steps of 1/16 as BF16, in the first column of x; u is 1."""
    g = torch.arange(-144, 145, device="cuda").div(16).to(BF)
    x = torch.zeros(g.numel(), 128, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = g, 1
    return x, g


def tail_error(g, act, value):
    """What FP32 may be off by, relative: a function of g rounded a few times within takes the relative error of e^(-g^2 / 2)
    for GELU and of e^-arg for the others, |exponent| roundings, and 16 more."""
    g = g.double().abs()
    exponent = g if act == "silu" else 0.5 * g * g if act == "gelu" else 1.6 * (g + 0.044715 * g ** 3)
    return (16 + 4 * exponent) * fo.U * value.abs() + fo.TINY


@pytest.mark.parametrize("act", fo.ACTS)
def test_gated_tails_keep_their_digits(iq, act):  # noqa: F811
    """The activations' left tails, 10^-6 and less, to the last digit of the output's type: nothing is taken off 1."""
    x, g = tail_inputs()
    a = fo.act_parts(g, act)[0]
    if act == "gelu_tanh":                              # 1 + tanh loses the tail in 64 bits too: (1 + tanh z) / 2 = 1 / (1 + e^-2z)
        a = g.double() * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g.double() + 0.044715 * g.double() ** 3))
    w = torch.zeros(2, 8, 128, dtype=BF, device="cuda")
    w[0, :, 0], w[1, :, 1] = 1, 1
    h, saved = iq.gated(x, w[0], w[1], act, save=True)
    fo.assert_within(h[:, 0], a, tail_error(g, act, a), "h of 289 tokens")
    fo.assert_within(iq.gated(x[:40], w[0], w[1], act)[:, 0], a[:40], tail_error(g, act, a)[:40], "h of 40 tokens")
    q = iq.Quantized(torch.zeros(8, 64, dtype=torch.uint8, device="cuda"), torch.full((8, 1), 0x3C00, dtype=torch.int16, device="cuda"),
                     None, None, None, "int4", "block", 8, 128)
    q.codes[:, 0] = 0x01                                # code 1 in column 0, scale 1
    up = iq.Quantized(q.codes.clone(), q.scales, None, None, None, "int4", "block", 8, 128)
    up.codes[:, 0] = 0x10
    for at in range(0, 289, 64):
        z = iq.packed_gated(q, up, x[at:at + 64].contiguous(), act, F32)
        fo.assert_within(z[:, 0], a[at:at + 64], tail_error(g, act, a)[at:at + 64], "packed, FP32")
    # du = dh act(g) through dw_up's first tokens: one token at a time has a weight gradient of its own
    dh = torch.ones(1, 8, dtype=BF, device="cuda")
    for t in (8, 40, 72, 100, 144, 180, 250):
        kept = saved[:, t:t + 1].contiguous()
        dwu = iq.gated_backward(dh, x[t:t + 1].contiguous(), w[0], w[1], kept, act)[2]
        e = tail_error(g, act, a)[t] + fo.HALF[BF] * a[t].abs()          # du is rounded to BF16, and dw_up again
        fo.assert_within(dwu[:1, 1], a[t:t + 1], e[None], f"dw_up at {t}")


# ---- layer norm: what lies past a row's end -------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [7, 8, 9, 1001, 2049, 4099, 8191, 16389])
def test_layer_norm_backward_takes_nothing_from_past_the_row(iq, dtype, cols):  # noqa: F811
    """A row of equal large values has n = 0 throughout; the elements that fill its last vector up would have
    n = -mean rstd, infinite here, and make the sum of a n NaN."""
    g = gen(cols)
    for rows in (1, 3, 300):
        x, dy = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, dtype=dtype)
        mean, rstd = x.float().mean(1), torch.ones(rows, device="cuda")
        x[rows // 2], mean[rows // 2], rstd[rows // 2] = 2.0 ** 110, 2.0 ** 110, 2.0 ** 20
        for w in (None, rand(g, cols, dtype=dtype, offset=1.0)):
            want, bound = fo.norm_grad(dy, x, w, mean, rstd)
            for got, r, e, what in zip(iq.layer_norm_backward(dy, x, w, mean, rstd), want, bound, ("dx", "dweight", "dbias")):
                fo.assert_within(got, r, e, f"{what}, {rows} rows")

"""The feed-forward operators on the GPU against their plain forms in 64 bits."""
import pytest
import torch

import ffn_oracle as fo

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def iq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int_quantization_amd as m
    m.load_library()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=BF, scale=1.0, offset=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + offset).to(dtype)


# ---- layer norm -----------------------------------------------------------------
# widths around the vector and register limits: single elements, 8 to a load,
# one to four vectors a thread, rows longer than the registers hold
WIDTHS = (1, 2, 7, 8, 33, 64, 255, 256, 1000, 1001, 2047, 2048, 2049, 2056, 4096, 4104, 5003, 8192, 16384, 16392, 20001)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype,param", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_layer_norm_widths(iq, cols, dtype, param):
    g = gen(cols)
    for rows in (1, 5):
        x = rand(g, rows, cols, dtype=dtype, scale=2.0, offset=0.5)
        w, b = rand(g, cols, dtype=param, offset=1.0), rand(g, cols, dtype=param)
        dy = rand(g, rows, cols, dtype=dtype)
        check_norm(iq, x, w, b, dy, 1e-5)


def check_norm(iq, x, w, b, dy, eps):
    y, mean, rstd = iq.layer_norm(x, w, b, eps)
    (ry, rm, rr), (ey, em, er) = fo.norm_bounds(x, w, b, eps)
    fo.assert_within(mean, rm, em, "mean")
    fo.assert_within(rstd, rr, er, "rstd")
    fo.assert_within(y, ry, ey, "y")
    dx, dw, db = iq.layer_norm_backward(dy, x, w, mean, rstd, param_dtype=None if b is None else b.dtype)
    want, bound = fo.norm_grad(dy, x, w, mean, rstd)
    for got, r, e, what in zip((dx, dw, db), want, bound, ("dx", "dweight", "dbias")):
        fo.assert_within(got, r, e, what)


@pytest.mark.parametrize("rows,cols", [(255, 264), (256, 100), (257, 4096), (700, 96), (1031, 1001), (300, 16392)])
def test_layer_norm_many_rows(iq, rows, cols):
    g = gen(rows)
    for dtype in (BF, F32):
        check_norm(iq, rand(g, rows, cols, dtype=dtype), rand(g, cols, dtype=F32), rand(g, cols, dtype=F32),
                   rand(g, rows, cols, dtype=dtype), 1e-6)


@pytest.mark.parametrize("cols,ld", [(64, 72), (64, 65), (1001, 1008), (4096, 4099), (8, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_norm_strided_rows_and_no_parameters(iq, cols, ld, dtype):
    g = gen(ld)
    whole = torch.full((9, ld), float("nan"), dtype=dtype, device="cuda")
    x = whole[:, :cols]
    x.copy_(rand(g, 9, cols, dtype=dtype))
    check_norm(iq, x, None, None, rand(g, 9, cols, dtype=dtype), 1e-5)
    off = whole.view(-1)[1: 1 + 8 * ld].view(8, ld)[:, :cols]      # rows that no 16-byte word starts
    off.copy_(rand(g, 8, cols, dtype=dtype))
    check_norm(iq, off, rand(g, cols, dtype=dtype), None, rand(g, 8, cols, dtype=dtype), 1e-5)


def test_layer_norm_large_offset_keeps_its_digits(iq):
    """A mean 4096 times the spread: the variance is taken about the mean."""
    g = gen(3)
    x = rand(g, 17, 2048, dtype=F32, offset=4096.0)
    check_norm(iq, x, rand(g, 2048, dtype=F32), rand(g, 2048, dtype=F32), rand(g, 17, 2048, dtype=F32), 1e-5)


def test_layer_norm_constant_rows_and_eps(iq):
    x = torch.full((4, 100), 3.0, device="cuda")
    x[2] = 0
    y, mean, rstd = iq.layer_norm(x, None, None, 0.25)
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(rstd, torch.full_like(rstd, 2.0))
    assert mean.tolist() == [3.0, 3.0, 0.0, 3.0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cols", [50, 64, 20001])
def test_layer_norm_non_finite_rows_stay_apart(iq, bad, cols):
    g = gen(5)
    x, dy = rand(g, 6, cols), rand(g, 6, cols)
    clean = iq.layer_norm(x)
    x2 = x.clone()
    x2[3, cols // 2] = bad
    y, mean, rstd = iq.layer_norm(x2)
    assert torch.isnan(y[3]).all()
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(mean[keep], clean[1][keep])
    dx = iq.layer_norm_backward(dy, x2, None, mean, rstd)[0]
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 6])
def test_layer_norm_few_rows(iq, rows):
    """Around the number of rows whose sums one workgroup writes itself."""
    g = gen(rows)
    for cols in (96, 1001, 8192, 16384, 20008):
        check_norm(iq, rand(g, rows, cols), rand(g, cols), rand(g, cols), rand(g, rows, cols), 1e-5)


def test_layer_norm_rows_beyond_the_grid(iq):
    """More rows than workgroups, so that each goes over several with the next in flight."""
    g = gen(9)
    for rows, cols, dtype in ((5000, 64, BF), (2100, 2560, F32), (1030, 4104, BF), (1030, 9000, F32), (520, 12288, BF)):
        check_norm(iq, rand(g, rows, cols, dtype=dtype), rand(g, cols, dtype=F32), rand(g, cols, dtype=F32),
                   rand(g, rows, cols, dtype=dtype), 1e-5)


def test_layer_norm_empty(iq):
    x = torch.empty((0, 40), dtype=BF, device="cuda")
    y, mean, rstd = iq.layer_norm(x)
    dx, dw, db = iq.layer_norm_backward(x, x, None, mean, rstd)
    assert y.shape == (0, 40) and dx.shape == (0, 40)
    assert torch.equal(dw, torch.zeros(40, device="cuda")) and torch.equal(db, dw)


def test_layer_norm_offsets_past_32_bits(iq):
    """Rows 2^31 + 8 elements apart."""
    ld, cols = (1 << 31) + 8, 1024
    whole = torch.empty(2 * ld + cols, dtype=BF, device="cuda")
    x = torch.as_strided(whole, (3, cols), (ld, 1))
    g = gen(6)
    x.copy_(rand(g, 3, cols))
    check_norm(iq, x, rand(g, cols), rand(g, cols), rand(g, 3, cols), 1e-5)


# ---- gated block ------------------------------------------------------------------
def gated_inputs(tokens, cols, features, seed, ld=None):
    g = gen(seed)
    x = rand(g, tokens, cols)
    if ld:
        whole = torch.full((tokens, ld), float("nan"), dtype=BF, device="cuda")
        whole[:, :cols] = x
        x = whole[:, :cols]
    s = max(cols, 1) ** -0.5
    return x, rand(g, features, cols, scale=s), rand(g, features, cols, scale=s), rand(g, tokens, features, scale=0.1)


def check_gated(iq, x, wg, wu, dh, act):
    h, saved = iq.gated(x, wg, wu, act, save=True)
    want, bound = fo.gated(x, wg, wu, act)
    fo.assert_within(h, want, bound, "h")
    assert torch.equal(h, iq.gated(x, wg, wu, act)), "h without saving differs"
    for k, w in enumerate((wg, wu)):
        r, e = fo.product(x, w)
        fo.assert_within(saved[k], r, e, "saved")
    got = iq.gated_backward(dh, x, wg, wu, saved, act)
    want, bound = fo.gated_grad(dh, x, wg, wu, act)
    for o, r, e, what in zip(got, want, bound, ("dx", "dwg", "dwu")):
        fo.assert_within(o, r, e, what)


# tokens around the few-token limit and the tiles' 128 and 256; widths around
# the k step of 64 and the tiles' 64, 128 and 256
GATED = [(1, 8, 8), (1, 64, 128), (3, 136, 40), (16, 512, 264), (17, 256, 64), (33, 1032, 520), (64, 128, 136),
         (65, 64, 64), (65, 72, 200), (127, 256, 128), (128, 128, 256), (129, 200, 264), (200, 1032, 72),
         (255, 320, 256), (257, 264, 1000), (513, 520, 392), (771, 1032, 2824)]


@pytest.mark.parametrize("act", fo.ACTS)
@pytest.mark.parametrize("tokens,cols,features", GATED)
def test_gated_shapes(iq, tokens, cols, features, act):
    check_gated(iq, *gated_inputs(tokens, cols, features, tokens + cols), act)


@pytest.mark.parametrize("tokens,cols,features", [(512, 2048, 4096), (1100, 1024, 2600), (2048, 2112, 2304)])
def test_gated_large(iq, tokens, cols, features):
    check_gated(iq, *gated_inputs(tokens, cols, features, 1), "silu")


@pytest.mark.parametrize("tokens,cols,features,act", [(2050, 328, 3336, "silu"), (2050, 6408, 264, "gelu"), (70, 1096, 5640, "silu"),
                                                      (300, 2056, 3592, "gelu_tanh"), (1793, 8, 4096, "silu"), (1800, 6408, 8, "silu"),
                                                      (2048, 4096, 3592, "silu"),
                                                      # a last round of tiles that smaller ones take: forward, x's gradient, the weights'
                                                      (2050, 200, 3752, "gelu"), (2050, 7496, 136, "silu"), (200, 1096, 6952, "gelu_tanh"),
                                                      # few tiles and a long sum: x's gradient and the weights' in parts
                                                      (3000, 264, 392, "silu"), (72, 136, 5000, "gelu"), (5001, 24, 16, "silu")])
def test_gated_wide_tiles(iq, tokens, cols, features, act):
    """Products large enough for 256 x 256 tiles, forward or in one of the gradients, with ragged edges and odd numbers of steps."""
    check_gated(iq, *gated_inputs(tokens, cols, features, 6), act)


@pytest.mark.parametrize("tokens,features", [(2050, 3336), (300, 15000)])
def test_gated_wide_tiles_strided_x_and_a_bad_token(iq, tokens, features):
    """The space between rows of x and one token hold NaN: neither reaches another token."""
    x, wg, wu, dh = gated_inputs(tokens, 328, features, 7, ld=344)
    check_gated(iq, x, wg, wu, dh, "silu")
    h0, s0 = iq.gated(x, wg, wu, save=True)
    dx0 = iq.gated_backward(dh, x, wg, wu, s0)[0]
    x[tokens - 1, 327] = float("nan")
    h, saved = iq.gated(x, wg, wu, save=True)
    assert torch.equal(h[:-1], h0[:-1]) and torch.isnan(h[-1]).all()
    assert torch.equal(iq.gated_backward(dh, x, wg, wu, saved)[0][:-1], dx0[:-1])


@pytest.mark.parametrize("tokens", [5, 40, 200, 600])
def test_gated_strided_x(iq, tokens):
    """Rows of x further apart than its columns; the space between holds NaN."""
    check_gated(iq, *gated_inputs(tokens, 328, 184, 2, ld=344), "gelu_tanh")


def test_gated_empty(iq):
    for tokens, cols, features in ((0, 64, 32), (7, 0, 32), (70, 0, 32), (5, 64, 0), (0, 0, 0)):
        x, wg, wu, dh = gated_inputs(tokens, cols, features, 3)
        h, saved = iq.gated(x, wg, wu, save=True)
        assert h.shape == (tokens, features) and not h.any()
        for out, shape in zip(iq.gated_backward(dh, x, wg, wu, saved), ((tokens, cols), (features, cols), (features, cols))):
            assert out.shape == shape and not out.any()


@pytest.mark.parametrize("tokens", [4, 130, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gated_non_finite_tokens_stay_apart(iq, tokens, bad):
    """A token that is not finite spoils its own rows and the weights' gradients only."""
    x, wg, wu, dh = gated_inputs(tokens, 136, 264, 4)
    h0, s0 = iq.gated(x, wg, wu, save=True)
    x2 = x.clone()
    x2[2, 130] = bad
    h, saved = iq.gated(x2, wg, wu, save=True)
    keep = [t for t in range(tokens) if t != 2]
    assert torch.equal(h[keep], h0[keep]) and not torch.isfinite(h[2]).all()
    dx = iq.gated_backward(dh, x2, wg, wu, saved)[0]
    assert torch.equal(dx[keep], iq.gated_backward(dh, x, wg, wu, s0)[0][keep])


@pytest.mark.parametrize("act", fo.ACTS)
def test_gated_far_arguments(iq, act):
    """g from -400 to 400: no overflow turns into NaN, forward or backward."""
    tokens, cols, features = 130, 64, 64
    x = torch.zeros(tokens, cols, dtype=BF, device="cuda")
    x[:, 0] = torch.linspace(-400, 400, tokens, device="cuda").to(BF)
    x[:, 1] = 1
    wg, wu = torch.zeros(features, cols, dtype=BF, device="cuda"), torch.zeros(features, cols, dtype=BF, device="cuda")
    wg[:, 0], wu[:, 1] = 1, 2
    dh = torch.ones(tokens, features, dtype=BF, device="cuda")
    check_gated(iq, x, wg, wu, dh, act)
    check_gated(iq, x[:50], wg, wu, dh[:50], act)


def test_gated_offsets_past_32_bits(iq):
    """140000 tokens by 16384 features: the saved values pass 2^32 elements, the outputs 2^31."""
    tokens, cols, features = 140000, 64, 16384
    x, wg, wu, _ = gated_inputs(8, cols, features, 5)
    x = x.repeat(tokens // 8, 1)
    h, saved = iq.gated(x, wg, wu, save=True)
    first = h[:8].clone()
    fo.assert_within(first, *fo.gated(x[:8], wg, wu, "silu"), "h")
    assert torch.equal(h[-8:], first) and torch.equal(saved[1, -8:], saved[1, :8])
    dx = iq.gated_backward(h, x, wg, wu, saved)[0]
    assert torch.equal(dx[-8:], dx[:8]) and dx[:8].abs().sum() > 0


# ---- packed weights ------------------------------------------------------------------
def random_weights(iq, rows, cols, fmt, seed, scale=0.02):
    """Weights quantized by the library."""
    w = rand(gen(seed), rows, cols, dtype=F32, scale=scale)
    w[rows // 3] *= 30
    return iq.quantize(w, fmt, "block", stats=False)


def any_weights(iq, rows, cols, fmt, seed):
    """Every code and many scales, which quantize itself does not all produce."""
    g = gen(seed)
    q = random_weights(iq, rows, cols, fmt, seed)
    q.codes.random_(0, 256, generator=g)
    if fmt == "nvfp4":
        q.scales.random_(0, 127, generator=g)
    if fmt == "mxfp4":
        q.scales.random_(100, 140, generator=g)
    if fmt == "int4":
        q.scales.copy_(rand(g, *q.scales.shape, dtype=torch.float16).view(torch.int16))
    return q


def values(q):
    return fo.unpack(q.fmt, q.codes, q.scales, q.global_scale)


PACKED = [(1, 1, 128), (1, 17, 256), (2, 32, 128), (3, 33, 384), (8, 100, 1024), (15, 48, 640), (16, 96, 4096),
          (17, 130, 1792), (31, 16, 8192), (32, 64, 4224), (33, 65, 512), (37, 1501, 1792), (64, 200, 2176), (1, 300, 8320)]


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("n1,rows,cols", PACKED)
def test_packed_shapes(iq, fmt, n1, rows, cols):
    for make, narrow in ((random_weights, 0), (any_weights, 0 if fmt == "int4" else 32)):
        c = cols - narrow if cols > 128 else cols                # 32 columns fewer end inside a step
        x = rand(gen(n1), n1, c)
        qg, qu = make(iq, rows, c, fmt, 1), make(iq, rows, c, fmt, 2)
        vg, vu = values(qg), values(qu)
        for dt in (BF, F32):
            z, e = fo.packed(x, vg)
            fo.assert_within(iq.packed_gemv(qg, x, dt), z, e, "z")
            act = fo.ACTS[(n1 + rows) % 3]
            u, eu = fo.packed(x, vu)
            if make is random_weights:                            # others reach 10^6, where act says nothing
                fo.assert_within(iq.packed_gated(qg, qu, x, act, dt), *fo.gate(z, u, e, eu, act), "h")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("cols", [32, 64, 96, 160, 288])
def test_packed_short_rows(iq, fmt, cols):
    for n1 in (1, 5, 20, 50):
        x = rand(gen(n1), n1, cols)
        q = any_weights(iq, 19, cols, fmt, 4)
        fo.assert_within(iq.packed_gemv(q, x, F32), *fo.packed(x, values(q)), "z")


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("n1", [1, 4, 5, 8, 9, 16, 17, 48, 49, 64])
def test_packed_token_counts(iq, fmt, n1):
    """Every way the tokens are staged, in wide and narrow matrices and over more k than one round of scales."""
    for rows, cols in ((130, 768), (4133, 512), (40, 8832 if fmt == "int4" else 8864)):
        cols -= cols % (128 if fmt == "int4" else 32)
        x = rand(gen(n1), n1, cols)
        q, q2 = any_weights(iq, rows, cols, fmt, 5), random_weights(iq, rows, cols, fmt, 6)
        fo.assert_within(iq.packed_gemv(q, x, F32), *fo.packed(x, values(q)), "z")
        (g, eg), h = fo.packed(x, values(q2)), iq.packed_gated(q2, q2, x, "silu", F32)
        fo.assert_within(h, *fo.gate(g, g, eg, eg, "silu"), "h")


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
def test_packed_infinities_stay_infinite(iq, fmt):
    """An infinite activation gives infinities of its weights' signs, whichever step of k it is in."""
    rows, cols = 33, 896
    q = random_weights(iq, rows, cols, fmt, 12)
    w = values(q)[0]
    for n1, k in ((1, 0), (3, 895), (6, 500), (20, 130), (64, 640)):
        x = rand(gen(k), n1, cols)
        x[n1 - 1, k] = float("inf")
        z = iq.packed_gemv(q, x, F32)[n1 - 1].double()
        want = w[:, k] * float("inf")                  # NaN where the weight is zero
        assert torch.equal(torch.isnan(z), torch.isnan(want)) or fmt == "int4"
        there = w[:, k] != 0
        if fmt != "int4":                              # INT4's two parts of a weight may both be infinite, with either sign
            assert torch.equal(z[there], want[there])
        assert not torch.isfinite(z[there]).any()


def test_packed_empty(iq):
    q = random_weights(iq, 64, 128, "nvfp4", 1)
    x = rand(gen(1), 0, 128)
    assert iq.packed_gemv(q, x).shape == (0, 64)
    none = iq.Quantized(q.codes[:0], q.scales[:0], q.global_scale, None, None, "nvfp4", "block", 0, 128)
    assert iq.packed_gemv(none, rand(gen(1), 3, 128)).shape == (3, 0)
    flat = iq.Quantized(q.codes[:, :0], q.scales[:, :0], q.global_scale, None, None, "nvfp4", "block", 64, 0)
    assert not iq.packed_gemv(flat, torch.empty((3, 0), dtype=BF, device="cuda")).any()


@pytest.mark.parametrize("fmt,byte", [("mxfp4", 255), ("nvfp4", 0x7F), ("nvfp4", 0xFF)])
def test_packed_nan_scales_stay_in_their_rows(iq, fmt, byte):
    for n1 in (1, 20):
        x = rand(gen(7), n1, 512)
        q = random_weights(iq, 40, 512, fmt, 3)
        clean = iq.packed_gemv(q, x)
        q.scales[11, 5] = byte
        z = iq.packed_gemv(q, x)
        keep = [j for j in range(40) if j != 11]
        assert torch.isnan(z[:, 11]).all() and torch.equal(z[:, keep], clean[:, keep])


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
def test_packed_non_finite_tokens_stay_apart(iq, fmt):
    q = random_weights(iq, 40, 512, fmt, 3)
    for n1 in (4, 20, 40):
        x = rand(gen(8), n1, 512)
        clean = iq.packed_gemv(q, x)
        x[1, 77] = float("nan")
        z = iq.packed_gemv(q, x)
        keep = [t for t in range(n1) if t != 1]
        assert torch.isnan(z[1]).all() and torch.equal(z[keep], clean[keep])


def test_packed_subnormal_scales_and_values(iq):
    """E8M0 0 and E4M3 subnormals with activations that bring the products back."""
    x = torch.full((2, 128), 2.0 ** 100, dtype=BF, device="cuda")
    q = any_weights(iq, 16, 128, "mxfp4", 9)
    q.scales.random_(2, 12, generator=gen(9))
    fo.assert_within(iq.packed_gemv(q, x, F32), *fo.packed(x, values(q)), "mxfp4")
    q = any_weights(iq, 16, 128, "nvfp4", 9)
    q.scales.random_(0, 9, generator=gen(9))
    fo.assert_within(iq.packed_gemv(q, x, F32), *fo.packed(x, values(q)), "nvfp4")


def test_packed_codes_past_32_bits(iq):
    """1050624 rows of 8192 columns: 4.3 GB of codes."""
    rows, cols = (1 << 20) + 2048, 8192
    q = iq.Quantized(torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda"),
                     torch.full((rows, cols // 128), 0x2C00, dtype=torch.int16, device="cuda"), None, None, None, "int4",
                     "block", rows, cols)
    q.codes.random_(0, 256, generator=gen(10))
    x = rand(gen(11), 3, cols)
    z = iq.packed_gemv(q, x, F32)
    for at in (0, rows // 2 + 5, rows - 33):
        part = fo.unpack("int4", q.codes[at: at + 33], q.scales[at: at + 33])
        want, e = fo.packed(x, part)
        fo.assert_within(z[:, at: at + 33].contiguous(), want, e, f"rows from {at}")


# ---- one after another, on other streams, in graphs --------------------------------------
def block(iq, x, w, b, wg, wu, dh, qg, qu, qd):
    """Every operator once, one feeding the next."""
    y, mean, rstd = iq.layer_norm(x, w, b)
    h, saved = iq.gated(y, wg, wu, save=True)
    dy, dwg, dwu = iq.gated_backward(dh, y, wg, wu, saved)
    dx, dw, db = iq.layer_norm_backward(dy, x, w, mean, rstd)
    few = y[:7].contiguous()
    hp = iq.packed_gated(qg, qu, few)
    z = iq.packed_gemv(qd, hp, F32)
    return y, mean, rstd, h, dy, dwg, dwu, dx, dw, db, hp, z


def block_inputs(iq):
    g = gen(20)
    x, wg, wu, dh = gated_inputs(300, 256, 512, 21)
    qs = [iq.quantize(t, "nvfp4", "block", stats=False) for t in (wg, wu, rand(g, 256, 512, scale=0.05))]
    return (x, rand(g, 256, offset=1.0), rand(g, 256), wg, wu, dh, *qs)


def test_calls_repeat_bit_for_bit(iq):
    args = block_inputs(iq)
    first = block(iq, *args)
    for a, b in zip(first, block(iq, *args)):
        assert torch.equal(a, b)


def test_short_calls_and_checked_calls_agree(iq):
    """With a stream named every call goes through the checks in Python; without, dense tensors do not."""
    x, w, b, wg, wu, dh, qg, qu, qd = block_inputs(iq)
    s = torch.cuda.current_stream()
    y, mean, rstd = iq.layer_norm(x, w, b)
    h, saved = iq.gated(y, wg, wu, "gelu", save=True)
    few = y[:7].contiguous()
    for p in (w, None):
        pairs = [(iq.layer_norm(x, p, b), iq.layer_norm(x, p, b, stream=s)),
                 (iq.layer_norm_backward(y, x, p, mean, rstd), iq.layer_norm_backward(y, x, p, mean, rstd, stream=s)),
                 (iq.gated(y, wg, wu, "gelu", save=True), iq.gated(y, wg, wu, "gelu", save=True, stream=s)),
                 ([iq.gated(y, wg, wu)], [iq.gated(y, wg, wu, stream=s)]),
                 (iq.gated_backward(dh, y, wg, wu, saved, "gelu"), iq.gated_backward(dh, y, wg, wu, saved, "gelu", stream=s)),
                 ([iq.packed_gated(qg, qu, few, "gelu_tanh", F32)], [iq.packed_gated(qg, qu, few, "gelu_tanh", F32, stream=s)]),
                 ([iq.packed_gemv(qg, few)], [iq.packed_gemv(qg, few, stream=s)])]
        for a, c in pairs:
            assert len(a) == len(c)
            for t, u in zip(a, c):
                assert t.dtype == u.dtype and t.shape == u.shape and torch.equal(t, u)
    assert iq._bind_fast().layer_norm(x, w, b, 1e-5) is not None and iq._bind_fast().layer_norm(x.t(), w, b, 1e-5) is None


def test_refusals_on_the_gpu(iq):
    """What is wrong is still said, whichever way a call goes first."""
    x, w, b, wg, wu, dh, qg, qu, qd = block_inputs(iq)
    y, mean, rstd = iq.layer_norm(x, w, b)
    h, saved = iq.gated(y, wg, wu, save=True)
    for error, call in ((ValueError, lambda: iq.layer_norm(x, w[:-1], b)), (TypeError, lambda: iq.layer_norm(x, w, b.float())),
                        (TypeError, lambda: iq.layer_norm(x.half())), (iq.IQError, lambda: iq.layer_norm(x, w, b, -1.0)),
                        (ValueError, lambda: iq.layer_norm(x, w.cpu(), b)), (ValueError, lambda: iq.layer_norm_backward(y[1:], x, w, mean, rstd)),
                        (ValueError, lambda: iq.gated(y, wg, wu, "relu")), (ValueError, lambda: iq.gated(y, wg[:, 1:], wu)),
                        (iq.IQError, lambda: iq.gated(y[:, :4].contiguous(), wg[:, :4].contiguous(), wu[:, :4].contiguous())),
                        (TypeError, lambda: iq.gated_backward(dh, y, wg, wu, saved.half())), (ValueError, lambda: iq.packed_gemv(qg, y.float())),
                        (iq.IQError, lambda: iq.packed_gemv(qg, y)), (TypeError, lambda: iq.packed_gemv(qg, y[:3].contiguous(), torch.float16)),
                        (ValueError, lambda: iq.packed_gated(qg, qd, y[:3].contiguous())), (ValueError, lambda: iq.packed_gemv(qg, y[:3].cpu()))):
        with pytest.raises(error):
            call()


def test_another_stream(iq):
    args = block_inputs(iq)
    first = block(iq, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(iq, *args)
    side.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)


def test_graph_replays_equal_eager_calls(iq):
    args = block_inputs(iq)
    block(iq, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = block(iq, *args)
    for k in range(4):
        args[0].copy_(rand(gen(30 + k), *args[0].shape))
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, block(iq, *args)):
            assert torch.equal(a, b), f"replay {k}"
        torch.cuda.synchronize()


# ---- the operators together, as the example has them ----------------------------------------
@pytest.fixture(scope="module")
def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_gradients(iq, example):
    """The layer's gradients against those of its formula in 64 bits.  Six values between input and gradient are rounded
    to BF16 (the norm, h, dh, dg or du, dn and the gradient itself), each by half a step at most, and so are the weights
    in both; the errors of one tensor's elements point every way, so its norm is off by at most the sum of the six."""
    layer = example.FeedForward(264, 712, act="gelu", seed=4)
    g = gen(50)
    x, dy = rand(g, 300, 264), rand(g, 300, 264)
    y, kept = layer.forward(x)
    got = layer.backward(dy, kept)
    got = (y, got[0], *got[1])
    leaves = [t.double().requires_grad_() for t in (x, layer.weight, layer.bias, layer.gate.to(BF), layer.up.to(BF), layer.down.to(BF))]
    xd, w, b, wg, wu, wd = leaves
    c = xd - xd.mean(1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w + b
    pre = n @ wg.t()
    out = xd + (pre * 0.5 * torch.erfc(-pre / 2 ** 0.5) * (n @ wu.t())) @ wd.t()
    out.backward(dy.double())
    for o, r in zip(got, (out, *(t.grad for t in leaves))):
        assert ((o.double() - r).norm() / r.norm()).item() <= 6 * fo.HALF[BF]


def test_example_learns(iq, example):
    losses = example.train(cols=256, features=704, tokens=512, steps=12)[1]
    assert losses[-1] < losses[0], losses


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "int4"])
def test_example_answers_from_packed_weights(iq, example, fmt):
    layer = example.FeedForward(256, 768, seed=3)
    packed = layer.packed(fmt)
    x = rand(gen(40), 5, 256)
    n = iq.layer_norm(x, layer.weight, layer.bias)[0]
    (wg, mg), (wu, mu), (wd, md) = (values(q) for q in packed)
    (g, eg), (u, eu) = fo.packed(n, (wg, mg)), fo.packed(n, (wu, mu))
    h, eh = fo.gate(g, u, eg, eu, "silu")
    eh = eh + fo.HALF[BF] * (h.abs() + eh)                        # h is rounded to BF16
    z = h @ wd.t().contiguous()
    ez = eh @ md.t().contiguous() + (2 * 768 + 8) * fo.U * ((h.abs() + eh) @ md.t().contiguous()) + fo.TINY
    ez = ez + fo.HALF[BF] * (z.abs() + ez)                        # and so is z, and then its sum with x
    fo.assert_within(layer.answer(x, packed), x.double() + z, ez, fmt)

"""The feed-forward operators without a GPU: their 64-bit plain forms against
differences, and what the C ABI and the binding refuse before any launch."""
import pytest
import torch

import ffn_oracle as fo

FAKE = 0x10000          # a 256-byte aligned address that validation never dereferences


@pytest.fixture(scope="module")
def iq():
    import os

    import int_quantization_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int_quantization_amd import build
        build.build()
    m.load_library()
    return m


def slope(f, at, along, step=1e-5):
    """Derivative of the scalar f at the tensors `at` along `along`, by differences."""
    ahead = f(*(a + step * d for a, d in zip(at, along)))
    behind = f(*(a - step * d for a, d in zip(at, along)))
    return (ahead - behind).item() / (2 * step)


@pytest.mark.parametrize("rows,cols", [(1, 9), (5, 16), (13, 33)])
def test_layer_norm_gradient_against_differences(rows, cols):
    torch.manual_seed(rows)
    x, w, b, dy = (torch.randn(*s, dtype=torch.float64) for s in ((rows, cols), (cols,), (cols,), (rows, cols)))
    along = [torch.randn_like(t) for t in (x, w, b)]
    got = slope(lambda x, w, b: (fo.norm(x, w, b, 1e-5)[0] * dy).sum(), (x, w, b), along)
    _, mean, rstd = fo.norm(x, w, b, 1e-5)
    grads = fo.norm_grad(dy, x, w, mean, rstd)[0]
    assert abs(got - sum((g * d).sum().item() for g, d in zip(grads, along))) < 1e-6 * (1 + abs(got))


@pytest.mark.parametrize("act", fo.ACTS)
def test_gated_gradient_against_differences(act):
    torch.manual_seed(7)
    x, wg, wu, dh = (torch.randn(*s, dtype=torch.float64) for s in ((5, 12), (9, 12), (9, 12), (5, 9)))
    along = [torch.randn_like(t) for t in (x, wg, wu)]
    got = slope(lambda x, wg, wu: (fo.gated(x, wg, wu, act)[0] * dh).sum(), (x, wg, wu), along)
    grads = fo.gated_grad(dh, x, wg, wu, act)[0]
    assert abs(got - sum((g * d).sum().item() for g, d in zip(grads, along))) < 1e-6 * (1 + abs(got))


def test_packed_values_are_the_formats():
    """One byte of each format, by hand."""
    codes = torch.tensor([[0x7F] + [0] * 63], dtype=torch.uint8)        # nibbles 15 and 7, then zeros
    s = torch.tensor([[0.5]], dtype=torch.float16).view(torch.int16)
    assert fo.unpack("int4", codes, s)[0][0, :3].tolist() == [-0.5, 3.5, 0.0]
    s = torch.tensor([[0x38] * 8], dtype=torch.uint8)                    # E4M3 1.0
    assert fo.unpack("nvfp4", codes, s, torch.tensor([2.0]))[0][0, :3].tolist() == [-12.0, 12.0, 0.0]
    s = torch.tensor([[128] * 4], dtype=torch.uint8)                     # 2^1
    assert fo.unpack("mxfp4", codes, s)[0][0, :3].tolist() == [-12.0, 12.0, 0.0]


# ---- refusals ---------------------------------------------------------------------------
def norm_desc(iq, rows=4, cols=24, ld=None, dtype=1):
    return iq.IQDesc(0, 0, dtype, 0, rows, cols, cols if ld is None else ld, 0, 0)


def test_layer_norm_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def fwd(d, x=FAKE, w=FAKE, b=FAKE, pt=1, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE):
        return iq.iq_layer_norm(d, x, w, b, pt, eps, y, mean, rstd, None)
    d = norm_desc(iq)
    assert fwd(norm_desc(iq, dtype=5)) == E
    assert fwd(norm_desc(iq, rows=-1)) == E
    assert fwd(norm_desc(iq, ld=23)) == E
    assert fwd(d, pt=9) == E
    for eps in (-1e-9, float("nan"), float("inf")):
        assert fwd(d, eps=eps) == E
    assert fwd(d, x=None) == E
    assert fwd(d, y=None) == E
    assert fwd(d, x=FAKE + 1) == A
    assert fwd(norm_desc(iq, dtype=0), y=FAKE + 2) == A
    assert fwd(d, pt=0, w=FAKE + 2) == A
    assert fwd(d, b=FAKE + 1) == A
    assert fwd(d, mean=FAKE + 2) == A
    assert fwd(norm_desc(iq, rows=1 << 31)) == U
    assert fwd(norm_desc(iq, ld=(1 << 40) + 1)) == U
    assert fwd(norm_desc(iq, rows=0), x=None, y=None) == iq.IQ_OK

    def bwd(d, x=FAKE, dy=FAKE, w=FAKE, pt=1, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE):
        return iq.iq_layer_norm_backward(d, x, dy, w, pt, mean, rstd, dx, dw, db, ws, None)
    for kw in ("x", "dy", "mean", "rstd", "ws"):
        assert bwd(d, **{kw: None}) == E, kw
    assert bwd(d, pt=2) == E
    assert bwd(norm_desc(iq, cols=-3)) == E
    assert bwd(d, ws=FAKE + 128) == A
    assert bwd(d, dx=FAKE + 1) == A
    assert bwd(d, pt=0, dw=FAKE + 2) == A
    assert bwd(d, rstd=FAKE + 2) == A
    assert bwd(d, dx=None, dw=None, db=None, ws=None) == iq.IQ_OK        # nothing asked for
    assert iq.iq_layer_norm_workspace_bytes(norm_desc(iq, rows=1000, cols=512)) == 256 * 2 * 512 * 4
    assert iq.iq_layer_norm_workspace_bytes(norm_desc(iq, rows=-1)) == 0


def gated_desc(iq, act=0, dtype=1, tokens=4, cols=64, features=32, ld=None, flags=0):
    return iq.IQGatedDesc(act, dtype, tokens, cols, features, cols if ld is None else ld, flags, 0)


def test_gated_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def fwd(d, x=FAKE, wg=FAKE, wu=FAKE, h=FAKE, saved=FAKE):
        return iq.iq_gated_forward(d, x, wg, wu, h, saved, None)
    d = gated_desc(iq)
    assert fwd(gated_desc(iq, act=3)) == E
    assert fwd(gated_desc(iq, dtype=4)) == E
    assert fwd(gated_desc(iq, dtype=0)) == U
    assert fwd(gated_desc(iq, flags=1)) == U
    assert fwd(gated_desc(iq, tokens=-1)) == E
    assert fwd(gated_desc(iq, cols=60)) == E
    assert fwd(gated_desc(iq, features=20)) == E
    assert fwd(gated_desc(iq, ld=56)) == E
    assert fwd(gated_desc(iq, ld=68)) == A
    assert fwd(gated_desc(iq, cols=(1 << 20) + 8)) == U
    assert fwd(gated_desc(iq, tokens=1 << 31)) == U
    for kw in ("x", "wg", "wu", "h"):
        assert fwd(d, **{kw: None}) == E, kw
        assert fwd(d, **{kw: FAKE + 8}) == A, kw
    assert fwd(d, saved=FAKE + 4) == A
    assert fwd(gated_desc(iq, tokens=0), x=None, h=None) == iq.IQ_OK

    def bwd(d, dh=FAKE, x=FAKE, wg=FAKE, wu=FAKE, saved=FAKE, dx=FAKE, dwg=FAKE, dwu=FAKE, ws=FAKE):
        return iq.iq_gated_backward(d, dh, x, wg, wu, saved, dx, dwg, dwu, ws, None)
    for kw in ("dh", "x", "wg", "wu", "saved", "dwg", "dwu", "ws"):
        assert bwd(d, **{kw: None}) == E, kw
        assert bwd(d, **{kw: FAKE + 8}) == A, kw
    assert bwd(d, dx=FAKE + 8) == A
    assert bwd(gated_desc(iq, act=-1)) == E
    assert bwd(gated_desc(iq, dtype=0)) == U
    assert iq.iq_gated_saved_bytes(d) == 2 * 4 * 32 * 4
    assert iq.iq_gated_saved_bytes(gated_desc(iq, cols=60)) == 0
    assert iq.iq_gated_workspace_bytes(d) >= 2 * 4 * 32 * 2


def test_packed_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def gemv(d, codes=FAKE, scales=FAKE, gs=FAKE, x=FAKE, xt=1, n1=2, z=FAKE, zt=1):
        return iq.iq_packed_gemv(d, codes, scales, gs, x, xt, n1, z, zt, None)

    def gated(d, codes=FAKE, scales=FAKE, gs=FAKE, x=FAKE, xt=1, n1=2, z=FAKE, zt=1, act=0, up=FAKE):
        return iq.iq_packed_gated(d, act, codes, scales, gs, up, scales, gs, x, xt, n1, z, zt, None)
    d = iq.make_desc("nvfp4", "block", 16, 256)
    for call in (gemv, gated):
        assert call(iq.make_desc("int4zp", "block", 16, 256)) == E
        assert call(iq.make_desc("e4m3", "row", 16, 256)) == E
        assert call(iq.make_desc("int4", "tensor", 16, 256)) == E
        assert call(iq.make_desc("int4", "block", 16, 192)) == E
        assert call(iq.make_desc("nvfp4", "block", 16, 48)) == E
        assert call(iq.make_desc("nvfp4", "block", -1, 64)) == E
        assert call(iq.make_desc("int4", "block", 16, 256, flags=4)) == U
        assert call(d, n1=-1) == E
        assert call(d, n1=65) == U
        assert call(d, xt=0) == U
        assert call(d, xt=3) == E
        assert call(d, zt=2) == E
        for kw in ("codes", "scales", "gs", "x", "z"):
            assert call(d, **{kw: None}) == E, kw
        assert call(d, codes=FAKE + 8) == A
        assert call(d, scales=FAKE + 2) == A
        assert call(d, gs=FAKE + 2) == A
        assert call(d, x=FAKE + 8) == A
        assert call(d, z=FAKE + 1) == A
        assert call(d, n1=0, x=None, z=None) == iq.IQ_OK
        assert call(iq.make_desc("nvfp4", "block", 0, 256), z=None) == iq.IQ_OK
        assert call(iq.make_desc("int4", "block", (1 << 31) - 1, 256)) == U
    assert gated(d, act=3) == E
    assert gated(d, up=None) == E


def test_binding_refusals(iq):
    """The binding's own checks, on CPU tensors, before the library is called."""
    bf = torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf)
    w = torch.zeros(32, 64, dtype=bf)
    with pytest.raises(ValueError):
        iq.layer_norm(torch.zeros(4))
    with pytest.raises(ValueError):
        iq.layer_norm(torch.zeros(64, 4).t())
    with pytest.raises(TypeError):
        iq.layer_norm(x.half())
    with pytest.raises(ValueError):
        iq.layer_norm(x, torch.zeros(63))
    with pytest.raises(TypeError):
        iq.layer_norm(x, torch.zeros(64), torch.zeros(64, dtype=bf))
    with pytest.raises(ValueError):
        iq.layer_norm(x, out=torch.zeros(4, 63, dtype=bf))
    stat = torch.zeros(4)
    with pytest.raises(ValueError):
        iq.layer_norm_backward(x[:3], x, None, stat, stat)
    with pytest.raises(TypeError):
        iq.layer_norm_backward(x.float(), x, None, stat, stat)
    with pytest.raises(ValueError):
        iq.gated(x, w, w, act="relu")
    with pytest.raises(ValueError):
        iq.gated(x.float(), w, w)
    with pytest.raises(ValueError):
        iq.gated(x, w, w[:16])
    with pytest.raises(ValueError):
        iq.gated(x, w[:, :32], w)
    with pytest.raises(ValueError):
        iq.gated_backward(torch.zeros(4, 31, dtype=bf), x, w, w, torch.zeros(2, 4, 32))
    with pytest.raises(TypeError):
        iq.gated_backward(torch.zeros(4, 32, dtype=bf), x, w, w, torch.zeros(2, 4, 32, dtype=bf))
    q = iq.Quantized(torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 2, dtype=torch.uint8), None, None, None,
                     "mxfp4", "block", 32, 64)
    with pytest.raises(ValueError):
        iq.packed_gemv(q, x[:, :32].contiguous())
    with pytest.raises(ValueError):
        iq.packed_gemv(q, x.float())
    with pytest.raises(TypeError):
        iq.packed_gemv(q, x, torch.float16)
    for call in (lambda: iq.packed_gemv(q, x), lambda: iq.gated(x, w, w), lambda: iq.layer_norm(x)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    with pytest.raises(ValueError):
        iq.packed_gemv(iq.Quantized(q.codes[:8], q.scales, None, None, None, "mxfp4", "block", 32, 64), x)
    with pytest.raises(ValueError):
        iq.packed_gated(q, iq.Quantized(q.codes, q.scales, None, None, None, "mxfp4", "block", 16, 64), x)
    with pytest.raises(ValueError):
        iq.packed_gated(q, q, x, act="tanh")


# ---- what the compiler makes of the products written out -----------------------------------
def test_products_read_only_operands_that_lds_reads_wrote(tmp_path):
    """The tiles' products are written out, so the compiler keeps no wait states before them: no vector instruction may
    write one of their operands within the two states before, none may use scratch memory between them, and 18 states
    lie between the last product and the first read of a result."""
    import os
    import re
    import subprocess

    from int_quantization_amd import build
    out = tmp_path / "gated.s"
    subprocess.run(["/opt/rocm/bin/hipcc", *build.HIPCC_FLAGS, "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only", "-S",
                    "-o", str(out), os.path.join(build.ROOT, "int_quantization_amd", "csrc", "iq_gated.hip")], check=True,
                   capture_output=True)

    def registers(operand):
        m = re.match(r"v\[(\d+):(\d+)\]$|v(\d+)$", operand)
        return set() if not m else set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}

    kernels, products = 0, 0
    code = None
    for line in out.read_text().splitlines():
        if re.match(r"_Z\S*k_gemm\S*:", line):
            code, kernels = [], kernels + 1
        elif line.startswith(".Lfunc_end") and code is not None:
            at = [i for i, c in enumerate(code) if c.startswith("v_mfma")]
            assert not any(c.startswith("scratch") for c in code)
            for i in at:
                name, *args = re.split(r"[ ,]+", code[i])
                assert args[0].startswith("a[") and args[0] == args[3], code[i]
                reads = registers(args[1]) | registers(args[2])
                for c in code[max(0, i - 2): i]:
                    if c.startswith("v_") and not c.startswith("v_mfma"):
                        assert not registers(re.split(r"[ ,]+", c)[1]) & reads, (c, code[i])
            after, states = code[at[-1] + 1:], 0
            for c in after:
                if c.startswith("v_accvgpr_read"):
                    break
                states += int(c.split()[1]) + 1 if c.startswith("s_nop") else 1
            assert states >= 18, states
            products, code = products + len(at), None
        elif code is not None:
            c = line.split(";")[0].strip()
            if c and not c.startswith(".") and not c.endswith(":"):
                code.append(c)
    assert kernels == 15 and products == 5 * (128 + 2 * 32)

"""What the feed-forward operators must not do, shown without a GPU: reads past
their operands, buffers that another stream may take, results cut from a graph."""
import os
import re
import subprocess
from functools import partial
from types import SimpleNamespace

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode


@pytest.fixture(scope="module")
def iq():
    import int_quantization_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int_quantization_amd import build
        build.build()
    m.load_library()
    return m


def kernels(source, name, tmp_path):
    """{mangled name: [instructions]} of the kernels of csrc/`source` whose name holds `name`, as the compiler writes them."""
    from int_quantization_amd import build
    out = tmp_path / "device.s"
    subprocess.run(["/opt/rocm/bin/hipcc", *build.HIPCC_FLAGS, "-I", os.path.join(build.ROOT, "include"), "--cuda-device-only", "-S",
                    "-o", str(out), os.path.join(build.ROOT, "int_quantization_amd", "csrc", source)], check=True, capture_output=True)
    found, code = {}, None
    for line in out.read_text().splitlines():
        label = re.match(r"(_Z\S*%s\S*):" % name, line)
        if label:
            code = found[label[1]] = []
        elif line.startswith(".Lfunc_end"):
            code = None
        elif code is not None:
            c = line.split(";")[0].strip()
            if c and not c.startswith(".") and not c.endswith(":"):
                code.append(c)
    return found


# ---- reads of packed codes ------------------------------------------------------------
def test_packed_code_loads_carry_their_whole_offset_in_the_range_check(tmp_path):
    """A buffer load compares its vector offset with the buffer's size less its scalar offset, as unsigned numbers, so a
    scalar offset past the buffer's end lets every load through.  Loads of weights past a row's last step are ordinary
    (the batch ahead), and a workgroup may hold a single row shorter than a step: their scalar offset has to be zero."""
    loads = 0
    for name, code in kernels("iq_packed.hip", "k_packed", tmp_path).items():
        for c in code:
            m = re.match(r"buffer_load_dwordx4 \S+ \S+ \S+ (\S+) offen(.*)", c)
            if m and " lds" not in m[2]:
                assert m[1] == "0", f"{name}: {c}"
                loads += 1
    assert loads > 100


@pytest.mark.parametrize("cols", range(32, 289, 32))
def test_packed_code_offsets_stay_in_their_rows(cols):
    """The kernel's offsets in numbers: lane (row, quarter h) of a step reads 16 bytes from row * K / 2 + 16 h + 64 step, steps
    past the matrix standing for its end; what the range check lets through lies in the workgroup's rows."""
    row_bytes, steps = cols // 2, -(-cols // 128)
    for rows in (1, 2, 3, 15, 16, 17, 32):
        size = rows * row_bytes
        for step in range(steps + 4):
            for row in range(rows):
                for h in range(4):
                    at = row * row_bytes + 16 * h + 64 * min(step, steps)
                    if at < size:
                        assert at + 16 <= size


# ---- the register of the copies written out ----------------------------------------------
def test_copies_set_m0_and_nothing_else_uses_it(tmp_path):
    """The tiles' copies write m0, which the compiler reserves and does not let them name: a use of its own would not see
    the change, and a copy that relied on an earlier one's value could be moved from behind it."""
    copies = 0
    for name, code in kernels("iq_gated.hip", "k_gemm", tmp_path).items():
        used = [i for i, c in enumerate(code) if re.search(r"\bm0\b", c)]
        sets = [i for i in used if re.match(r"s_mov_b32 m0, |s_add_u32 m0, ", code[i])]
        loads = [i for i, c in enumerate(code) if c.startswith("buffer_load") and c.endswith(" lds")]
        assert used == sets, name
        assert [i + 2 for i in sets] == loads, name        # one instruction between: the wait state
        copies += len(loads)
    assert copies > 300


# ---- buffers of a named stream -----------------------------------------------------------
class Allocations(TorchDispatchMode):
    """Notes for every tensor made whether `place` was entered."""

    def __init__(self, place):
        super().__init__()
        self.place, self.seen = place, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket.__name__ in ("empty", "empty_like", "new_empty", "empty_strided", "zeros", "full"):
            self.seen.append(self.place.inside)
        return func(*args, **(kwargs or {}))


class Place:
    """Stands for torch.cuda.stream: the streams named, and whether one is current."""

    def __init__(self):
        self.named, self.inside = [], False

    def __call__(self, stream):
        self.named.append(stream)
        return self

    def __enter__(self):
        self.inside = True

    def __exit__(self, *error):
        self.inside = False


class FakeStream:
    cuda_stream, device = 0, torch.device("cpu")


BF, F32 = torch.bfloat16, torch.float32


def packed(iq, fmt, rows=32, cols=256):
    d = iq.make_desc(fmt, "block", rows, cols)
    codes, scales, g = iq.empty_outputs(d, "cpu", fmt, "block")
    shifts = torch.zeros(rows, cols // 256, dtype=torch.uint8) if fmt == "int4zp" else None
    return iq.Quantized(codes, scales, g, None, None, fmt, "block", rows, cols, shifts)


X, W, STAT = torch.zeros(4, 256, dtype=BF), torch.zeros(32, 256, dtype=BF), torch.zeros(4)
DH, SAVED = torch.zeros(4, 32, dtype=BF), torch.zeros(2, 4, 32)
CALLS = {                          # each makes its operands and returns the call
    "quantize": lambda iq: partial(iq.quantize, X, "nvfp4", "block", xhat_dtype=F32),
    "quantize static": lambda iq: partial(iq.quantize, X, "nvfp4", "block", static_amax=STAT[:1]),
    "quantize int4zp": lambda iq: partial(iq.quantize, X, "int4zp", "block"),
    "dequantize": lambda iq: partial(iq.dequantize, packed(iq, "nvfp4")),
    "dequantize int4zp": lambda iq: partial(iq.dequantize, packed(iq, "int4zp")),
    "amax": lambda iq: partial(iq.amax, X),
    "zp_gemm": lambda iq: partial(iq.zp_gemm, packed(iq, "int4zp"), X),
    "mx_gemm": lambda iq: partial(iq.mx_gemm, packed(iq, "mxfp4"), packed(iq, "mxfp4", 4)),
    "mxw_gemm": lambda iq: partial(iq.mxw_gemm, packed(iq, "mxfp4"), X),
    "layer_norm": lambda iq: partial(iq.layer_norm, X),
    "layer_norm_backward": lambda iq: partial(iq.layer_norm_backward, X, X, None, STAT, STAT),
    "gated": lambda iq: partial(iq.gated, X, W, W, save=True),
    "gated_backward": lambda iq: partial(iq.gated_backward, DH, X, W, W, SAVED),
    "packed_gemv": lambda iq: partial(iq.packed_gemv, packed(iq, "int4"), X),
    "packed_gated": lambda iq: partial(iq.packed_gated, packed(iq, "mxfp4"), packed(iq, "mxfp4"), X),
}
LAUNCHES = ("iq_quantize", "iq_quantize_static", "iq_quantize_zp", "iq_dequantize", "iq_dequantize_zp", "iq_amax", "iq_zp_gemm",
            "iq_mx_gemm", "iq_mxw_gemm", "iq_layer_norm", "iq_layer_norm_backward", "iq_gated_forward", "iq_gated_backward",
            "iq_packed_gemv", "iq_packed_gated")


@pytest.mark.parametrize("name", CALLS)
def test_a_named_streams_call_allocates_under_that_stream(iq, monkeypatch, name):
    """Results and workspace taken from another stream's memory could be handed out again there while the call runs."""
    place, launched, call = Place(), [], CALLS[name](iq)
    monkeypatch.setattr(torch.cuda, "stream", place)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    for of in ("_stream", "_stream_for"):
        monkeypatch.setattr(iq, of, lambda *a: 0, raising=False)
    for launch in LAUNCHES:
        monkeypatch.setattr(iq, launch, lambda *a: launched.append(place.inside) or iq.IQ_OK)
    stream = FakeStream()
    with Allocations(place) as made:
        call(stream=stream)
    assert launched == [True] and place.named == [stream]
    assert made.seen and all(made.seen)


# ---- tensors elsewhere than on the current device ---------------------------------------------
def test_calls_run_on_their_tensors_device(iq, monkeypatch):
    """A launch on another device's stream would run where the tensor's memory is not."""
    entered = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered.append(d) or Place())
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    here, there = (SimpleNamespace(is_cuda=True, device=torch.device("cuda", k), get_device=lambda k=k: k) for k in (0, 1))
    with iq._place(None, here):
        assert not entered and iq._stream_for(here) == 100
    with iq._place(None, there):
        assert entered == [there.device] and iq._stream_for(there) == 101
    with pytest.raises(ValueError, match="the stream on"):
        iq._place(FakeStream(), there)


@pytest.mark.parametrize("name", CALLS)
def test_host_memory_is_refused(iq, name):
    with pytest.raises(ValueError, match="not on a GPU"):
        CALLS[name](iq)()


# ---- arguments of the short calls ----------------------------------------------------------
@pytest.mark.parametrize("save", [1, "yes", 0, ""])
def test_save_is_taken_for_its_truth(iq, monkeypatch, save):
    """The short calls compare with True itself, so 1 would return h alone where the caller unpacks two results."""
    given = []
    monkeypatch.setattr(iq, "_fast_calls", SimpleNamespace(gated=lambda *a: given.append(a[4]) or "done"))
    assert iq.gated(X, W, W, save=save) == "done" and given == [bool(save)]


# ---- rows without elements --------------------------------------------------------------
def test_layer_norm_without_columns_does_not_end_before_its_statistics(iq):
    """Returning early left mean and rstd as the allocator gave them; what is checked late shows that the call goes on."""
    d, fake = iq.IQDesc(0, 0, iq.IQ_BF16, 0, 5, 0, 0, 0, 0), 0x10000
    assert iq.iq_layer_norm(d, None, None, None, 1, 1e-5, None, fake + 2, fake, None) == iq.IQ_EALIGN
    assert iq.iq_layer_norm(d, None, None, None, 1, 1e-5, None, fake, fake + 2, None) == iq.IQ_EALIGN
    assert iq.iq_layer_norm(d, None, None, None, 1, 1e-5, None, None, None, None) == iq.IQ_OK


# ---- tensors that a graph follows ------------------------------------------------------------
GRAD = {                           # every tensor that may ask for a gradient, one at a time
    "layer_norm": (lambda iq, x, w, b: iq.layer_norm(x, w, b), (X, W[0], W[0])),
    "layer_norm_backward": (lambda iq, *a: iq.layer_norm_backward(*a), (X, X, W[0], STAT, STAT)),
    "gated": (lambda iq, *a: iq.gated(*a), (X, W, W)),
    "gated_backward": (lambda iq, *a: iq.gated_backward(*a), (DH, X, W, W, SAVED)),
    "packed_gemv": (lambda iq, x: iq.packed_gemv(packed(iq, "int4"), x), (X,)),
    "packed_gated": (lambda iq, x: iq.packed_gated(packed(iq, "int4"), packed(iq, "int4"), x), (X,)),
}


@pytest.mark.parametrize("name", GRAD)
def test_tensors_that_require_gradients_are_refused(iq, name):
    """The results would be cut from the graph without a word."""
    call, operands = GRAD[name]
    for k in range(len(operands)):
        given = [t.clone().requires_grad_(i == k) for i, t in enumerate(operands)]
        with pytest.raises(RuntimeError, match="no gradient passes"):
            call(iq, *given)
        with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):
            call(iq, *given)

"""The attention operators without a GPU: tables and layouts against their definitions, the gradient against differences,
the kernels' indexing compiled for the host, and what the C ABI and the binding refuse before any launch."""
import math
import os
import subprocess

import pytest
import torch

import attn_oracle as ao
from conftest import ROOT

FAKE = 0x10000          # a 256-byte aligned address that validation never dereferences


@pytest.fixture(scope="module")
def iq():
    import int_quantization_amd as m
    if not os.path.exists(m.LIB_PATH):
        from int_quantization_amd import build
        build.build()
    m.load_library()
    return m


def test_struct_layouts_match_header(iq, tmp_path):
    import ctypes
    names = {"iq_rotary_desc": iq.IQRotaryDesc, "iq_cache_desc": iq.IQCacheDesc, "iq_append_desc": iq.IQAppendDesc,
             "iq_attention_desc": iq.IQAttentionDesc}
    lines = [f'printf("%zu{" %zu" * len(c._fields_)}\\n", sizeof({n}), {", ".join(f"offsetof({n}, {f})" for f, _ in c._fields_)});'
             for n, c in names.items()]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "iq.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, c in zip(out, names.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(c)] + [getattr(c, f).offset for f, _ in c._fields_]


def test_indexing_stays_in_range(tmp_path):
    """The kernels' own index functions under any lengths, starts and page tables: bad pages, overlong sequences, starts out of order."""
    exe = tmp_path / "check"
    subprocess.run(["/opt/rocm/bin/hipcc", "-O1", "-Xarch_host", "-fsanitize=undefined", "-std=c++17", "--offload-arch=gfx950", "-x", "hip",
                    os.path.join(ROOT, "tests", "cache_index_check.cpp"), "-I", os.path.join(ROOT, "include"), "-o", str(exe)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok" and not r.stderr, r.stdout + r.stderr


def test_places_are_a_permutation():
    assert sorted(ao.PLACE) == list(range(32))
    assert [ao.PLACE[t] for t in (0, 1, 4, 8, 16, 31)] == [0, 1, 16, 4, 8, 31]


# ---- tables ---------------------------------------------------------------------------
def test_rotary_table(iq):
    tau = 2 * math.pi
    for rot in (0, 2, 6, 64, 128):
        for base in (10000.0, 500000.0):
            plain = [base ** (-2 * i / rot) / tau for i in range(rot // 2)]

            def close(got, want):
                assert got.dtype == torch.float64 and got.shape == (rot // 2,)
                assert all(abs(a - b) <= 4e-16 * b * 8 for a, b in zip(got.tolist(), want))
            close(iq.rotary_table(rot, base, device="cpu"), plain)
            close(iq.rotary_table(rot, base, "linear", 4.0, device="cpu"), [t / 4 for t in plain])
            larger = base * 8.0 ** (rot / (rot - 2)) if rot > 2 else base
            close(iq.rotary_table(rot, base, "base", 8.0, device="cpu"), [larger ** (-2 * i / rot) / tau for i in range(rot // 2)])
            keep = [min(1, max(0, (t * 4096 - 1) / 31)) for t in plain]
            parts = iq.rotary_table(rot, base, "parts", 8.0, 4096, device="cpu")
            close(parts, [t / 8 * (1 - w) + t * w for t, w in zip(plain, keep)])
    slow = iq.rotary_table(128, 1e4, "base", 8.0, device="cpu")[-1] / iq.rotary_table(128, 1e4, device="cpu")[-1]
    assert abs(slow.item() * 8 - 1) < 1e-12                              # the slowest pair's angle is divided by the factor


def test_rotary_table_refusals(iq):
    for args in ((-2, 1e4), (3, 1e4), (8, 0.0), (8, -1.0), (8, math.inf), (8, math.nan), (8, 1e4, "linear", 0.0), (8, 1e4, "linear", math.nan),
                 (8, 1e4, "parts", 2.0, 0.0), (8, 1e4, "parts", 2.0, 4096.0, 4.0, 4.0)):
        with pytest.raises(iq.IQError):
            iq.rotary_table(*args, device="cpu")
    with pytest.raises(ValueError):
        iq.rotary_table(8, scaling="other")
    assert iq.iq_rotary_table(8, 1e4, 4, 1.0, 0.0, 0.0, 0.0, FAKE) == iq.IQ_EINVAL
    assert iq.iq_rotary_table(8, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == iq.IQ_EINVAL


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_against_differences(interleaved):
    torch.manual_seed(3)
    table = 1000.0 ** (-torch.arange(5, dtype=torch.float64) / 5) / (2 * math.pi)
    x, dy, along = (torch.randn(7, 3, 16, dtype=torch.float64) for _ in range(3))
    at = torch.randint(-100, 10000, (7,))

    def f(x):
        return (ao.rotate(x, at, table, interleaved, 1.25) * dy).sum()
    step = 1e-5
    got = (f(x + step * along) - f(x - step * along)).item() / (2 * step)
    assert abs(got - (ao.rotate(dy, at, table, interleaved, 1.25, -1) * along).sum().item()) < 1e-8 * (1 + abs(got))


def test_codes_move_by_powers_of_two(iq):
    """The model's append, one token at a time: a block's scale only doubles, and INT8 codes end less than a step away."""
    for fmt in ("int8", "e4m3"):
        torch.manual_seed(1)
        cache = ao.Cache(torch.randint(0, 256, (2, 1, 1, 2, 32 * 64), dtype=torch.uint8), torch.full((2, 1, 1, 2), float("nan")), fmt, 1, 64, 32)
        x = torch.randn(40, 1, 64) * torch.exp2(torch.arange(40).div(8))[:, None, None]
        last = 0.0
        for t in range(40):
            cache.append(x[t:t + 1], x[t:t + 1], [[1, 0]], [t + 1])
            now = cache.scales[1, 0, 0, 0].item() if t < 32 else last
            assert t in (0, 32) or last == 0 or math.log2(now / last) == round(math.log2(now / last))
            last = now
        k, v = cache.values([1, 0], 40)
        assert torch.equal(k, v)
        step = cache.scales[1, 0, 0, 0].item()
        off = (k[:32] - x[:32]).abs()
        if fmt == "int8":
            assert off.max() < step
        else:
            assert (off <= torch.maximum(x[:32].abs() * 2 ** -4 * (1 + 2 ** -20), torch.tensor(step * 2 ** -9))).all()


# ---- refusals -----------------------------------------------------------------------------
def rotary_desc(iq, dtype=1, layout=0, tokens=4, heads=3, dim=64, strides=None, rot=32, amplitude=1.0, flags=0):
    s = strides or (heads * dim, dim, heads * dim, dim)
    return iq.IQRotaryDesc(dtype, layout, tokens, heads, dim, *s, rot, amplitude, flags, 0)


def test_rotary_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED
    for call in (iq.iq_rotary, iq.iq_rotary_backward):
        def run(d, x=FAKE, p=FAKE, t=FAKE, y=2 * FAKE):
            return call(d, x, p, t, y, None)
        d = rotary_desc(iq)
        for kw in (dict(dtype=2), dict(layout=2), dict(tokens=-1), dict(heads=-1), dict(dim=-1), dict(rot=-2), dict(rot=3), dict(rot=66),
                   dict(amplitude=float("nan")), dict(amplitude=float("inf")), dict(strides=(-192, 64, 192, 64)), dict(strides=(192, 64, 192, -64)),
                   dict(strides=(192, 64, 128, 64)), dict(strides=(192, 64, 0, 64)), dict(strides=(192, 64, 192, 0)),
                   dict(strides=(192, 64, 64, 192))):
            assert run(rotary_desc(iq, **kw)) == E, kw
        for kw in (dict(flags=1), dict(tokens=1 << 24), dict(heads=4097), dict(dim=1026), dict(heads=2048, dim=1024), dict(strides=((1 << 40) + 8, 64, 192, 64))):
            assert run(rotary_desc(iq, **kw)) == U, kw
        for kw in ("x", "p", "t", "y"):
            assert run(d, **{kw: None}) == E, kw
            assert run(d, **{kw: FAKE + 1}) == A, kw
        assert run(rotary_desc(iq, dtype=0), x=FAKE + 2) == A
        assert run(d, t=FAKE + 4) == A
        assert run(rotary_desc(iq, strides=(192, 64, 256, 64)), x=FAKE, y=FAKE) == E            # in place, other strides
        for kw in (dict(tokens=0), dict(heads=0), dict(dim=0, rot=0)):
            assert run(rotary_desc(iq, **kw), x=None, y=None) == iq.IQ_OK


def cache_desc(iq, fmt=1, heads=2, dim=64, page=64, pages=8, batch=3, width=4, flags=0):
    return iq.IQCacheDesc(fmt, heads, dim, page, pages, batch, width, flags, 0)


BAD_CACHE = (dict(fmt=2), dict(fmt=-1), dict(heads=0), dict(dim=0), dict(pages=-1), dict(page=16), dict(page=48), dict(page=0), dict(batch=-1),
             dict(width=-1))
TOO_MUCH = (dict(dim=80), dict(dim=512), dict(heads=1025), dict(page=8192), dict(pages=1 << 31), dict(width=(1 << 24) + 1), dict(flags=1),
            dict(batch=(1 << 20) + 1))


def test_cache_sizes(iq):
    assert iq.iq_cache_codes_bytes(cache_desc(iq)) == 8 * 2 * 64 * 2 * 64
    assert iq.iq_cache_scales_bytes(cache_desc(iq)) == 8 * 2 * 2 * 2 * 4
    for kw in BAD_CACHE[:-2] + TOO_MUCH[:5]:
        assert iq.iq_cache_codes_bytes(cache_desc(iq, **kw)) == iq.iq_cache_scales_bytes(cache_desc(iq, **kw)) == 0
    c = iq.make_cache(3, 2, 96, "int8", 128, device="cpu")
    assert c.codes.shape == (3, 2, 4, 2, 32 * 96) and c.scales.shape == (3, 2, 4, 2)
    for args in ((3, 2, 80), (3, 2, 64, "e4m3", 48), (-1, 2, 64), (3, 0, 64)):
        with pytest.raises(ValueError):
            iq.make_cache(*args, device="cpu")
    with pytest.raises(ValueError):
        iq.make_cache(3, 2, 64, "e5m2", device="cpu")


def append_desc(iq, dtype=1, layout=0, tokens=3, q_heads=4, strides=None, rot=32, amplitude=1.0, flags=0):
    return iq.IQAppendDesc(dtype, layout, tokens, q_heads, *(strides or (128, 64, 128, 64, 256, 64)), rot, amplitude, flags, 0)


def test_append_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def run(d, a, k=FAKE, v=FAKE, pages=FAKE, lengths=FAKE, starts=FAKE, table=FAKE, q=FAKE, out=FAKE, codes=FAKE, scales=FAKE):
        return iq.iq_cache_append(d, a, k, v, pages, lengths, starts, table, q, out, codes, scales, None)
    d, a = cache_desc(iq), append_desc(iq)
    for kw in BAD_CACHE:
        assert run(cache_desc(iq, **kw), a) == E, kw
    for kw in TOO_MUCH:
        assert run(cache_desc(iq, **kw), a) == U, kw
    for kw in (dict(dtype=3), dict(layout=-1), dict(tokens=-1), dict(q_heads=-1), dict(rot=5), dict(rot=66), dict(rot=-2), dict(amplitude=float("inf")),
               dict(strides=(128, -64, 128, 64, 256, 64))):
        assert run(d, append_desc(iq, **kw)) == E, kw
    for kw in (dict(flags=2), dict(q_heads=4097), dict(tokens=1 << 24), dict(tokens=8000000, q_heads=0)):
        assert run(d, append_desc(iq, **kw)) == U, kw
    assert run(d, append_desc(iq, tokens=4), starts=None) == E            # a token a sequence, and there are three
    for kw in ("k", "v", "pages", "lengths", "table", "q", "out", "codes", "scales"):
        assert run(d, a, **{kw: None}) == E, kw
        assert run(d, a, **{kw: FAKE + 1}) == A, kw
    assert run(d, a, codes=FAKE + 8) == A
    assert run(d, a, scales=FAKE + 4) == A
    assert run(d, append_desc(iq, dtype=0), k=FAKE + 2) == A
    assert run(d, append_desc(iq, tokens=0), k=None) == iq.IQ_OK
    assert run(cache_desc(iq, batch=0), a, k=None) == iq.IQ_OK


def test_read_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def run(d, codes=FAKE, scales=FAKE, pages=FAKE, lengths=FAKE, starts=FAKE, tokens=3, k=FAKE, v=FAKE, dtype=1):
        return iq.iq_cache_read(d, codes, scales, pages, lengths, starts, tokens, k, v, dtype, None)
    d = cache_desc(iq)
    for kw in BAD_CACHE:
        assert run(cache_desc(iq, **kw)) == E, kw
    for kw in TOO_MUCH:
        assert run(cache_desc(iq, **kw)) == U, kw
    assert run(d, tokens=-1) == E and run(d, tokens=2, starts=None) == E and run(d, dtype=2) == E
    assert run(d, tokens=1 << 24) == U
    assert run(cache_desc(iq, heads=1024), tokens=1 << 23) == U
    for kw in ("codes", "scales", "pages", "lengths"):
        assert run(d, **{kw: None}) == E, kw
        assert run(d, **{kw: FAKE + 1}) == A, kw
    assert run(d, starts=FAKE + 2) == A
    assert run(d, k=FAKE + 8) == A and run(d, v=FAKE + 8) == A
    assert run(d, k=None, v=None, codes=None) == iq.IQ_OK and run(d, tokens=0, codes=None) == iq.IQ_OK


def attention_desc(iq, dtype=1, causal=1, tokens=3, q_heads=4, strides=(256, 64), window=0, scale=0.125, flags=0):
    return iq.IQAttentionDesc(dtype, causal, tokens, q_heads, *strides, window, scale, flags)


def test_attention_refusals(iq):
    E, A, U = iq.IQ_EINVAL, iq.IQ_EALIGN, iq.IQ_EUNSUPPORTED

    def run(d, a, codes=FAKE, scales=FAKE, pages=FAKE, lengths=FAKE, starts=FAKE, q=FAKE, o=FAKE, ws=FAKE):
        return iq.iq_cache_attention(d, a, codes, scales, pages, lengths, starts, q, o, ws, None)
    d, a = cache_desc(iq), attention_desc(iq)
    for kw in BAD_CACHE:
        assert run(cache_desc(iq, **kw), a) == E, kw
        assert iq.iq_cache_attention_workspace_bytes(cache_desc(iq, **kw), a) == 0
    for kw in TOO_MUCH:
        assert run(cache_desc(iq, **kw), a) == U, kw
    for kw in (dict(dtype=2), dict(causal=2), dict(causal=-1), dict(tokens=-1), dict(q_heads=0), dict(q_heads=3), dict(window=-1),
               dict(causal=0, window=5), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(strides=(-256, 64))):
        assert run(d, attention_desc(iq, **kw)) == E, kw
        assert iq.iq_cache_attention_workspace_bytes(d, attention_desc(iq, **kw)) == 0
    for kw in (dict(dtype=0), dict(flags=1), dict(q_heads=4098), dict(tokens=1 << 24), dict(tokens=(1 << 20) + 1, q_heads=256)):
        assert run(d, attention_desc(iq, **kw)) == U, kw
    assert run(d, attention_desc(iq, tokens=4), starts=None) == E
    assert run(d, attention_desc(iq, strides=(252, 64))) == A and run(d, attention_desc(iq, strides=(256, 68))) == A
    for kw in ("codes", "scales", "pages", "lengths", "q", "o", "ws"):
        assert run(d, a, **{kw: None}) == E, kw
        assert run(d, a, **{kw: FAKE + 1}) == A, kw
    assert run(d, a, q=FAKE + 8) == A and run(d, a, o=FAKE + 8) == A and run(d, a, ws=FAKE + 128) == A
    assert run(d, attention_desc(iq, tokens=0), q=None) == iq.IQ_OK
    assert iq.iq_cache_attention_workspace_bytes(d, a) >= 256


def test_binding_refusals(iq):
    """The binding's own checks, on CPU tensors, before the library is called."""
    bf = torch.bfloat16
    x, at, table = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, dtype=torch.int32), torch.zeros(16, dtype=torch.float64)
    for call in (iq.rotary, iq.rotary_backward):
        for bad, kind in (((x[0], at, table), ValueError), ((x.transpose(1, 2), at, table), ValueError), ((x.half(), at, table), TypeError),
                          ((x, at.long(), table), TypeError), ((x, at[:3], table), ValueError), ((x, at, table.float()), TypeError),
                          ((x, at, torch.zeros(33, dtype=torch.float64)), ValueError)):
            with pytest.raises(kind):
                call(*bad)
        with pytest.raises(ValueError):
            call(x, at, table, out=torch.zeros(4, 2, 32, dtype=bf))
        with pytest.raises(ValueError, match="not on a GPU"):
            call(x, at, table)
        with pytest.raises(RuntimeError, match="no gradient passes"):
            call(x.float().requires_grad_(), at, table)
    cache = iq.make_cache(6, 2, 64, device="cpu")
    pages, lengths = torch.zeros(4, 3, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    starts, q = torch.zeros(5, dtype=torch.int32), torch.zeros(4, 6, 64, dtype=bf)

    def append(**kw):
        p = dict(dict(cache=cache, k=x, v=x, page_table=pages, lengths=lengths, starts=starts, q=q, rotary=table), **kw)
        return iq.cache_append(p.pop("cache"), p.pop("k"), p.pop("v"), p.pop("page_table"), p.pop("lengths"), p.pop("starts"), **p)

    def attend(**kw):
        p = dict(dict(cache=cache, q=q, page_table=pages, lengths=lengths, starts=starts), **kw)
        return iq.cache_attention(p.pop("cache"), p.pop("q"), p.pop("page_table"), p.pop("lengths"), p.pop("starts"), **p)

    def read(**kw):
        p = dict(dict(cache=cache, page_table=pages, lengths=lengths, starts=starts, tokens=4), **kw)
        return iq.cache_read(p.pop("cache"), p.pop("page_table"), p.pop("lengths"), p.pop("starts"), p.pop("tokens"), **p)

    other = [(dict(page_table=pages.long()), TypeError), (dict(page_table=pages[0]), ValueError), (dict(lengths=lengths[:3]), ValueError),
             (dict(lengths=lengths.long()), TypeError), (dict(starts=starts[:4]), ValueError), (dict(page_table=pages.t()), ValueError),
             (dict(cache=iq.KVCache(cache.codes, cache.scales[:5], "e4m3", 2, 64, 64)), ValueError),
             (dict(cache=iq.KVCache(cache.codes, cache.scales, "e5m2", 2, 64, 64)), ValueError),
             (dict(cache=iq.KVCache(cache.codes.view(torch.int8), cache.scales, "e4m3", 2, 64, 64)), TypeError)]
    for call in (append, attend, read):
        for kw, kind in other:
            with pytest.raises(kind):
                call(**kw)
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    for kw, kind in ((dict(k=x[:3]), ValueError), (dict(v=x[:, :1]), ValueError), (dict(v=x.float()), TypeError), (dict(q=q.float()), TypeError),
                     (dict(q=q[..., :32]), ValueError), (dict(rotary=table.float()), TypeError), (dict(k=x[:3], v=x[:3], q=q[:3], starts=None), ValueError),
                     (dict(rotary=torch.zeros(33, dtype=torch.float64)), ValueError)):
        with pytest.raises(kind):
            append(**kw)
    for kw, kind in ((dict(q=q.float()), TypeError), (dict(q=q[:, :5]), ValueError), (dict(q=q[:, :0]), ValueError), (dict(q=q[0]), ValueError),
                     (dict(q=q[:3], starts=None), ValueError), (dict(out=torch.zeros(4, 6, 64)), TypeError)):
        with pytest.raises(kind):
            attend(**kw)
    for kw, kind in ((dict(tokens=3, starts=None), ValueError), (dict(out_dtype=torch.float16), TypeError),
                     (dict(out=(torch.zeros(4, 2, 64), torch.zeros(4, 2, 32))), ValueError)):
        with pytest.raises(kind):
            read(**kw)
    with pytest.raises(RuntimeError, match="no gradient passes"):
        append(k=x.float().requires_grad_(), v=x.float(), q=None)


def test_results_that_lie_on_operands(iq):
    """q_out and o may be q where that is dense; k and v of a read are apart."""
    E, d, p = iq.IQ_EINVAL, cache_desc(iq), FAKE
    for strides in ((512, 64), (256, 128), (64, 192), (0, 64)):
        a = append_desc(iq, strides=(128, 64, 128, 64, *strides))
        assert iq.iq_cache_append(d, a, p, p, p, p, p, p, p, p, p, p, None) == E, strides
        assert iq.iq_cache_attention(d, attention_desc(iq, strides=strides), p, p, p, p, p, p, p, p, None) == E, strides
    assert iq.iq_cache_read(d, p, p, p, p, p, 3, p, p, 1, None) == E

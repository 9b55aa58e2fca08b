"""What the attention operators accept and refuse at the ends of their arguments, shown without a GPU."""
import os
import subprocess
from types import SimpleNamespace

import pytest
import torch

from conftest import ROOT
from test_attn_cpu import FAKE, attention_desc, cache_desc, iq, rotary_desc  # noqa: F401


def test_strides_that_are_not_used(iq):  # noqa: F811
    """A stride of one token or of one head leads nowhere: nothing is asked of it."""
    d = cache_desc(iq, batch=1)
    for strides in ((2051, 64), (-1, 64), (1 << 50, 64)):
        assert iq.iq_cache_attention_workspace_bytes(d, attention_desc(iq, tokens=1, strides=strides)) >= 256, strides
        assert iq.iq_cache_attention_workspace_bytes(d, attention_desc(iq, tokens=2, strides=strides)) == 0, strides
    one = cache_desc(iq, heads=1, batch=1)
    for strides in ((256, 67), (256, -1), (256, 1 << 50)):
        assert iq.iq_cache_attention_workspace_bytes(one, attention_desc(iq, tokens=2, q_heads=1, strides=strides)) >= 256, strides
        assert iq.iq_cache_attention_workspace_bytes(one, attention_desc(iq, tokens=2, q_heads=2, strides=strides)) == 0, strides
    # in place, strides that differ where they are used
    for tokens, heads, s in ((1, 3, (192, 64, 192, 72)), (4, 1, (64, 64, 72, 64))):
        assert iq.iq_rotary(rotary_desc(iq, tokens=tokens, heads=heads, strides=s), FAKE, FAKE, FAKE, FAKE, None) == iq.IQ_EINVAL


def test_rotary_tables_that_leave_the_range(iq):  # noqa: F811
    """Finite arguments whose turns would not be are refused, and the table is left as it was."""
    for args in ((64, 1e-300, "linear", 1e-300, 0.0), (64, 1e-200, "base", 1e-200, 0.0), (64, 1e4, "linear", 1e-310, 0.0), (64, 1e4, "parts", 1e-310, 4096.0)):
        rot, base, scaling, factor, context = args
        with pytest.raises(iq.IQError):
            iq.rotary_table(rot, base, scaling, factor, context, device="cpu")
        host = torch.full((rot // 2,), 7.0, dtype=torch.float64)
        assert iq.iq_rotary_table(rot, base, iq.ROTARY_SCALINGS[scaling], factor, context, 1.0, 32.0, host.data_ptr()) == iq.IQ_EINVAL
        assert (host == 7).all()
    for args in ((64, 1e300), (64, 1e-3), (64, 1e308, "base", 1e300), (64, 1e4, "linear", 1e300), (64, 1e4, "parts", 1e3, 1e-300)):
        table = iq.rotary_table(*args, device="cpu")
        assert torch.isfinite(table).all() and table[0] > 0 and (table >= 0).all()


# ---- the binding ------------------------------------------------------------------------------
def operands():
    bf, i32 = torch.bfloat16, torch.int32
    return SimpleNamespace(x=torch.zeros(4, 2, 64, dtype=bf), q=torch.zeros(4, 6, 64, dtype=bf), at=torch.zeros(4, dtype=i32),
                           turns=torch.zeros(16, dtype=torch.float64), pages=torch.zeros(4, 3, dtype=i32), lengths=torch.ones(4, dtype=i32),
                           starts=torch.zeros(5, dtype=i32))


def test_tables_scales_and_results_that_require_gradients(iq):  # noqa: F811
    """No graph is recorded for any operand, the table of a rotation, a cache's scales and given results among them."""
    o, cache = operands(), iq.make_cache(6, 2, 64, device="cpu")
    asks = iq.KVCache(cache.codes, cache.scales.zero_().clone().requires_grad_(), "e4m3", 2, 64, 64)
    turns, leaf = o.turns.clone().requires_grad_(), o.x.clone().requires_grad_()
    where = (o.pages, o.lengths, o.starts)
    for call in (lambda: iq.rotary(o.x, o.at, turns), lambda: iq.rotary_backward(o.x, o.at, turns), lambda: iq.rotary(o.x, o.at, o.turns, out=leaf),
                 lambda: iq.cache_append(cache, o.x, o.x, *where, q=o.q, rotary=turns), lambda: iq.cache_append(asks, o.x, o.x, *where),
                 lambda: iq.cache_attention(asks, o.q, *where), lambda: iq.cache_read(asks, *where, 4),
                 lambda: iq.cache_read(cache, *where, 4, out=(o.x.clone(), leaf))):
        with pytest.raises(RuntimeError, match="no gradient passes"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_one_given_result_of_a_read(iq):  # noqa: F811
    """Either result of a read may be given alone; both are of its type."""
    o, cache = operands(), iq.make_cache(6, 2, 64, device="cpu")
    for out in ((o.x.clone(), None), (None, o.x.clone()), (None, o.x.float()), (None, None)):
        with pytest.raises(ValueError, match="not on a GPU"):
            iq.cache_read(cache, o.pages, o.lengths, o.starts, 4, out=out)
    with pytest.raises(TypeError):
        iq.cache_read(cache, o.pages, o.lengths, o.starts, 4, out=(o.x.float(), o.x.clone()))


def test_shares_stay_in_range(tmp_path):
    """What columns see, rows, shares and their places in the workspace, by the kernels' own functions, under any lengths and starts."""
    exe = tmp_path / "check"
    subprocess.run(["/opt/rocm/bin/hipcc", "-O1", "-Xarch_host", "-fsanitize=undefined", "-std=c++17", "--offload-arch=gfx950", "-x", "hip",
                    os.path.join(ROOT, "tests", "attend_index_check.cpp"), "-I", os.path.join(ROOT, "include"), "-o", str(exe)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok" and not r.stderr, r.stdout + r.stderr

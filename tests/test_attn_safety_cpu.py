"""What the attention operators accept and refuse at the ends of their arguments, shown without a GPU."""
import pytest
import torch

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

"""What the attention operators accept and refuse at the ends of their arguments, shown without a GPU."""
import math

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

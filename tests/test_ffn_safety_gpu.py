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

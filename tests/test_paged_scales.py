"""Attention over an 8-bit cache whose value scales lie at the two ends of their range."""
import numpy as np
import pytest

import paged_ref as R
from test_paged import BF, FP, _i32, _scaled_pages
from transformer_attention_02_gb300 import attn as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,then", [(256, 96), (128, 128), (304, 1200)], ids=["one_warp", "warps", "ctas"])
def test_weights_that_count_beside_scales_far_above(first, then):
    """Keys with all the weight over values of scale 2^-72, then keys of weight 2^-20 over values of scale 2^120, the ends
    of what the header allows: the reference rises by 172 log2 units, more than a factor in FP32 holds, and the row
    sum has to keep what came before. In one warp's stages, between warps and between CTAs."""
    page = 16
    c, q, n = _scaled_pages([-72] * (first // page) + [120] * (then // page), [20] * (first // page) + [0] * (then // page), 5)
    o, lse = A.attention_paged(q, c.k, c.v, c.table, _i32([n]), **c.scales)
    k, v = (R.tokens(x, s, c.table_np[0], n, page) for x, s in ((c.k, c.ks), (c.v, c.vs)))
    want = R.attend(R.f64(q[0]), k, v, np.array([n - 1]), 64 ** -0.5, 0, 0)
    # the largest contribution: a weight of 2^-20 / first on values of 448 * 2^120 (as in test_value_scales_far_apart)
    R.check_rows(R.f64(o[0]), R.f64(lse[0]), want, R.step(BF), R.step(FP), 64, n, 2.0 ** 100 / first * 448, f"{first} {then}")

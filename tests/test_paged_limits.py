"""Paged cache and the attention over it: limits of sizes and scales, checked on the host."""
import ctypes

import pytest

from test_paged import _attn, _c, _t, lib  # noqa: F401


def test_scales_up_to_the_largest_the_kernels_can_weigh_with(lib):  # noqa: F811
    """Scores are weighed by powers of two: a scale whose product with log2(e) is beyond fp32 is refused."""
    from chunkwise_causal_linear_la_b200 import binding as b

    for scale in (2.4e38, 3.4e38):
        assert _attn(lib, scale=scale) == b.LA_ERR_INVALID_ARG and b"scale" in lib.la_last_error()
    for scale in (2.35e38, 1e-45):  # taken: the next check speaks
        assert _attn(lib, scale=scale) == b.LA_ERR_WORKSPACE

"""Paged cache and the attention over it: limits of sizes and scales, checked on the host."""
import ctypes

from test_paged import _attn, _c, _t, lib  # noqa: F401


def test_scales_up_to_the_largest_the_kernels_can_weigh_with(lib):  # noqa: F811
    """Scores are weighed by powers of two: a scale whose product with log2(e) is beyond fp32 is refused."""
    from chunkwise_causal_linear_la_b200 import binding as b

    for scale in (2.4e38, 3.4e38):
        assert _attn(lib, scale=scale) == b.LA_ERR_INVALID_ARG and b"scale" in lib.la_last_error()
    for scale in (2.35e38, 1e-45):  # taken: the next check speaks
        assert _attn(lib, scale=scale) == b.LA_ERR_WORKSPACE


def test_more_entries_than_the_plan_can_number_are_refused(lib):  # noqa: F811
    """An entry is one or two query tiles of a sequence.  The plan's searches add two entry numbers in 32 bits and its
    borders multiply the entries' costs by the cache heads in 64."""
    from chunkwise_causal_linear_la_b200 import binding as b

    size = lambda n, H: lib.la_paged_attn_workspace_size(1, 1, H, 64, n, 1, H, 16, 0, 1, 0)  # noqa: E731
    none = ctypes.c_size_t(-1).value
    assert size(1 << 30, 4) != none and size((1 << 30) + 1, 4) == none and size(0x7FFFFFE0, 4) == none
    assert size(1 << 21, 65536) != none and size((1 << 21) + 1, 65536) == none
    q, out = _t(T=1), _t(T=1)
    c = _c(fmt=0, k_scale=0, v_scale=0)
    assert lib.la_paged_attn(ctypes.byref(q), ctypes.byref(c), 0x100, 1, 0x200, 0x300, 0x7FFFFFE0, 0.1, 0,
                             ctypes.byref(out), None, 0, 0x100000, 1 << 62, None) == b.LA_ERR_UNSUPPORTED


def test_the_failure_path_has_its_flag(lib):  # noqa: F811
    from chunkwise_causal_linear_la_b200 import binding as b

    t = b.LA_FLAG_TEST_WAIT_TIMEOUT
    assert _attn(lib, flags=t) == b.LA_ERR_WORKSPACE  # taken: the next check speaks
    assert b.paged_attn_path(16, 64, 4, 16, flags=t) == b.LA_PATH_TENSOR_CORE
    assert b.paged_attn_path(16, 64, 4, 16, flags=t | b.LA_FLAG_SIMT) == b.LA_PATH_CUDA_CORE
    assert b.paged_attn_path(16, 64, 4, 16, flags=t | 2) == -1 and _attn(lib, flags=t | 2) == b.LA_ERR_INVALID_ARG
    assert b.paged_attn_workspace_size(1, 4, 4, 64, 1, False, 2, 16, flags=t) == b.paged_attn_workspace_size(
        1, 4, 4, 64, 1, False, 2, 16)

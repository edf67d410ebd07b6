"""Paged cache and attention over it: argument checks of the C ABI and of the binding, and the
plain 64-bit forms the GPU tests compare with.  No compute call is made here."""
import ctypes
import math

import pytest
import torch

from paged_util import attend, quantise


@pytest.fixture(scope="module")
def lib():
    from chunkwise_causal_linear_la_b200 import build, binding

    build.build()
    return binding.load_library()


def _t(B=1, T=4, H=4, D=64, dtype=1, ptr=0x1000, **kw):
    from chunkwise_causal_linear_la_b200.binding import LaTensor

    t = LaTensor(ptr, dtype, B, T, H, D, T * H * D, H * D, D)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _c(fmt=1, n=10, page=16, H=2, D=64, **kw):
    from chunkwise_causal_linear_la_b200.binding import LaKvCache

    c = LaKvCache(0x4000, 0x5000, 0x6000, 0x7000, fmt, n, page, H, D, page * H * D, H * D, D)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _attn(lib, q=None, out=None, c=None, table=0x100, max_pages=3, kv_len=0x200, cu=None, n=1, scale=0.125, window=0,
          lse=None, flags=0, ws=None, wsb=0):
    q, out, c = q or _t(), out or _t(), c or _c()
    return lib.la_paged_attn(ctypes.byref(q), ctypes.byref(c), table, max_pages, kv_len, cu, n, scale, window,
                             ctypes.byref(out), lse, flags, ws, wsb, None)


def test_attention_refuses_bad_arguments(lib):
    from chunkwise_causal_linear_la_b200 import binding as b

    bad = b.LA_ERR_INVALID_ARG
    assert lib.la_paged_attn(None, ctypes.byref(_c()), 0x100, 3, 0x200, None, 1, 0.1, 0, ctypes.byref(_t()), None, 0,
                             None, 0, None) == bad
    assert lib.la_paged_attn(ctypes.byref(_t()), None, 0x100, 3, 0x200, None, 1, 0.1, 0, ctypes.byref(_t()), None, 0,
                             None, 0, None) == bad
    assert _attn(lib, q=_t(dtype=0)) == bad                       # out has another dtype
    assert _attn(lib, q=_t(dtype=7), out=_t(dtype=7)) == bad
    assert _attn(lib, q=_t(T=5)) == bad                           # shapes disagree
    assert _attn(lib, q=_t(H=3), out=_t(H=3)) == bad              # 3 heads over 2
    assert _attn(lib, q=_t(ptr=0x1004)) == bad
    assert _attn(lib, q=_t(ptr=0)) == bad
    assert _attn(lib, q=_t(stride_t=-256)) == bad
    assert _attn(lib, q=_t(stride_t=257)) == bad
    assert _attn(lib, out=_t(stride_h=0)) == bad                  # rows that are written overlap
    assert _attn(lib, c=_c(D=128, stride_head=128, stride_token=256, stride_page=4096)) == bad
    assert _attn(lib, c=_c(fmt=3)) == bad
    assert _attn(lib, c=_c(page=0)) == bad
    assert _attn(lib, c=_c(n=-1)) == bad
    assert _attn(lib, c=_c(k=0)) == bad
    assert _attn(lib, c=_c(k=0x4008)) == bad
    assert _attn(lib, c=_c(k_scale=0)) == bad
    assert _attn(lib, c=_c(v_scale=0x7004)) == bad
    assert _attn(lib, c=_c(stride_head=0)) == bad
    assert _attn(lib, c=_c(stride_token=-128)) == bad
    assert _attn(lib, c=_c(stride_page=2049)) == bad
    assert _attn(lib, table=None) == bad
    assert _attn(lib, table=0x102) == bad
    assert _attn(lib, max_pages=-1) == bad
    assert _attn(lib, kv_len=None) == bad
    assert _attn(lib, kv_len=0x201) == bad
    assert _attn(lib, lse=0x301) == bad
    assert _attn(lib, n=2) == bad                                 # n_seqs is not B
    assert _attn(lib, n=-1) == bad
    assert _attn(lib, q=_t(B=2), out=_t(B=2), cu=0x300, n=2) == bad
    assert _attn(lib, cu=0x302, n=2) == bad
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert _attn(lib, scale=scale) == bad
    assert _attn(lib, window=-1) == bad
    assert _attn(lib, flags=2) == bad and b"flags" in lib.la_last_error()
    assert _attn(lib, ws=0x1001, wsb=1 << 30) == bad
    assert _attn(lib, q=_t(D=96), out=_t(D=96)) == b.LA_ERR_UNSUPPORTED
    assert _attn(lib, c=_c(page=70000)) == b.LA_ERR_UNSUPPORTED
    big = dict(T=1 << 20, H=1 << 10, D=64)
    assert _attn(lib, q=_t(**big), out=_t(**big)) == b.LA_ERR_UNSUPPORTED
    assert _attn(lib, max_pages=1 << 50) == b.LA_ERR_UNSUPPORTED
    # nothing to do: no pointer is needed
    none = dict(T=0, ptr=0)
    assert _attn(lib, q=_t(**none), out=_t(**none), table=None, max_pages=0, kv_len=None) == b.LA_OK


def test_writes_and_reads_refuse_bad_arguments(lib):
    from chunkwise_causal_linear_la_b200 import binding as b

    bad = b.LA_ERR_INVALID_ARG

    def both(k=None, v=None, c=None, table=0x100, pos=0x200, cu=None, n=1):
        k, v, c = k or _t(H=2), v or _t(H=2), c or _c()
        w = lib.la_kv_write(ctypes.byref(k), ctypes.byref(v), cu, n, ctypes.byref(c), table, 3, pos, None)
        r = lib.la_kv_read(ctypes.byref(c), table, 3, pos, cu, n, ctypes.byref(k), ctypes.byref(v), None)
        return w, r
    assert both(v=_t(H=2, dtype=0)) == (bad, bad)
    assert both(v=_t(H=2, T=5)) == (bad, bad)
    assert both(k=_t(H=4), v=_t(H=4)) == (bad, bad)               # other heads than the cache's
    assert both(c=_c(fmt=9)) == (bad, bad)
    assert both(c=_c(k_scale=0)) == (bad, bad)
    assert both(table=None) == (bad, bad)
    assert both(pos=0x202) == (bad, bad)
    assert both(n=3) == (bad, bad)
    assert both(k=_t(H=2, D=80), v=_t(H=2, D=80)) == (b.LA_ERR_UNSUPPORTED,) * 2
    k = _t(H=2)
    assert lib.la_kv_write(ctypes.byref(k), ctypes.byref(k), None, 1, ctypes.byref(_c()), 0x100, 3, None, None) == bad
    z = _t(H=2, stride_t=0)
    assert lib.la_kv_read(ctypes.byref(_c()), 0x100, 3, None, None, 1, ctypes.byref(z), ctypes.byref(k), None) == bad
    none = _t(H=2, T=0, ptr=0)
    assert lib.la_kv_write(ctypes.byref(none), ctypes.byref(none), None, 1, ctypes.byref(_c()), 0x100, 3, None,
                           None) == b.LA_OK


def test_paths_and_workspace(lib):
    from chunkwise_causal_linear_la_b200 import binding as b

    assert b.paged_attn_path(16, 96, 4, 16) == -1
    assert b.paged_attn_path(15, 64, 4, 16) == -1
    assert b.paged_attn_path(16, 64, 4, 0) == -1
    assert b.paged_attn_path(16, 64, 4, 16, flags=4) == -1
    for kw in (dict(dtype=torch.float32), dict(flags=b.LA_FLAG_SIMT)):
        assert b.paged_attn_path(16, 128, 4, 16, **kw) == b.LA_PATH_CUDA_CORE
        assert b.paged_attn_workspace_size(1, 64, 16, 128, 1, False, 4, 16, **kw) == 0
    for H, D, Hkv, page in ((16, 32, 4, 16), (16, 256, 4, 16), (16, 128, 4, 20), (258, 64, 2, 16)):
        assert b.paged_attn_path(H, D, Hkv, page) == b.LA_PATH_CUDA_CORE
    for H, D, Hkv, page in ((16, 64, 4, 16), (16, 128, 16, 8), (256, 128, 2, 200), (5, 64, 5, 48)):
        for fmt in (torch.bfloat16, torch.float8_e4m3fn, torch.int8):
            assert b.paged_attn_path(H, D, Hkv, page, fmt) == b.LA_PATH_TENSOR_CORE
    with pytest.raises(b.LaError):
        b.paged_attn_workspace_size(1, 64, 15, 128, 1, False, 4, 16)
    assert b.paged_attn_path(16, 64, 4, 16, torch.uint8) == -1 == b.paged_attn_path(16, 64, 4, 16, dtype=torch.float16)
    with pytest.raises(b.LaError):
        b.paged_attn_workspace_size(1, 64, 16, 128, 1, False, 4, 16, torch.float16)
    # entries (32 bytes and two 8-byte prefixes each) grow with the batch, the parts of 148 CTAs do not
    small = b.paged_attn_workspace_size(1, 1, 16, 128, 1, False, 4, 16)
    assert small >= 148 * 4 * 128 * (128 + 2) * 4
    assert b.paged_attn_workspace_size(1, 1, 16, 64, 1, False, 4, 16) < small
    many = b.paged_attn_workspace_size(1, 1 << 20, 16, 128, 1000, True, 4, 16)
    assert many - small >= ((1 << 20) // 64 + 1000 - 1) * 48
    assert b.paged_attn_workspace_size(1, 0, 16, 128, 1, False, 4, 16) == 0


def test_attention_needs_its_workspace(lib):
    from chunkwise_causal_linear_la_b200 import binding as b

    need = b.paged_attn_workspace_size(1, 4, 4, 64, 1, False, 2, 16, torch.float8_e4m3fn)
    assert _attn(lib) == b.LA_ERR_WORKSPACE and str(need).encode() in lib.la_last_error()
    assert _attn(lib, ws=0x100000, wsb=need - 1) == b.LA_ERR_WORKSPACE


def test_binding_refuses_what_it_cannot_describe():
    from chunkwise_causal_linear_la_b200 import binding as b

    k = torch.zeros(4, 16, 2, 64, dtype=torch.int8)
    s = torch.zeros(4, 2, 16)
    q = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16)
    table, kl = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(TypeError):  # an 8-bit cache without scales
        b.la_paged_attn(q, k, k, table, kl)
    with pytest.raises(TypeError):  # a workspace with fewer bytes than elements
        b.la_paged_attn(q, k, k, table, kl, k_scale=s, v_scale=s, workspace=torch.zeros(1).expand(1 << 26))
    with pytest.raises(TypeError):  # scales of another layout
        b.la_paged_attn(q, k, k, table, kl, k_scale=s.transpose(1, 2), v_scale=s)
    with pytest.raises(TypeError):
        b.la_paged_attn(q, k.bfloat16(), k.bfloat16(), table, kl, k_scale=s)
    with pytest.raises(ValueError):
        b.la_paged_attn(q, k, k.transpose(1, 2).contiguous().transpose(1, 2), table, kl, k_scale=s, v_scale=s)
    with pytest.raises(TypeError):
        b.la_paged_attn(q, k, k, table.long(), kl, k_scale=s, v_scale=s)
    with pytest.raises(TypeError):
        b.la_paged_attn(q, k, k, table.repeat(2, 1), kl, k_scale=s, v_scale=s)
    with pytest.raises(TypeError):
        b.la_paged_attn(q, k, k, table, kl.long(), k_scale=s, v_scale=s)
    with pytest.raises(TypeError):
        b.la_paged_attn(q, k, k, table, kl, k_scale=s, v_scale=s, lse=torch.zeros(1, 3, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="current CUDA device"):  # host tensors, or another device's
        b.la_paged_attn(q, k, k, table, kl, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="current CUDA device"):
        b.la_kv_write(q[:, :, :2], q[:, :, :2], k, k, table, kl, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="current CUDA device"):
        b.la_kv_read(k, k, table, 3, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="shape"):
        b.la_kv_read(k, k, table, 3, k_scale=s, v_scale=s, k_out=q)
    with pytest.raises(TypeError):
        b.kv_cache(4, 16, 2, 64, torch.float16, device="cpu")
    kc, vc, ks, vs = b.kv_cache(4, 16, 2, 64, torch.float8_e4m3fn, device="cpu")
    assert kc.shape == vc.shape == (4, 16, 2, 64) and ks.shape == vs.shape == (4, 2, 16)
    assert b.kv_cache(4, 16, 2, 64, device="cpu")[2:] == (None, None)


@pytest.mark.parametrize("dtype,qmax", [(torch.float8_e4m3fn, 448.0), (torch.int8, 127.0)])
def test_plain_quantiser(dtype, qmax):
    """Known rows: the largest code at the edge of a scale, the next scale just past it, ties to even, zero
    rows, and torch's own e4m3 grid."""
    rows = torch.zeros(6, 16, dtype=torch.float64)
    rows[0, 0] = qmax            # scale 1
    rows[1, 0] = qmax * 1.0001   # scale 2
    rows[2, 0] = qmax / 2        # scale 1/2
    rows[3, :2] = torch.tensor([qmax, 2.5])
    rows[4, 0] = 2.0 ** -140     # scale clamped
    c, s = quantise(rows, dtype)
    assert s.flatten().tolist() == [1.0, 2.0, 0.5, 1.0, 2.0 ** -126, 2.0 ** -126]
    assert c[0, 0] == qmax and c[2, 0] == qmax and c[3, 1] == (2.0 if dtype == torch.int8 else 2.5)
    assert c[4, 0] == 0 and c[5].abs().sum() == 0
    x = torch.randn(64, 32, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 37
    c, s = quantise(x, dtype)
    if dtype == torch.float8_e4m3fn:  # x / s is exact in fp32 for fp32 rows
        x = x.float()
        c, s = quantise(x.double(), dtype)
        assert torch.equal((x / s.float()).to(dtype).double(), c)
    assert float(c.abs().max()) <= qmax and bool((c.abs().amax(-1) > qmax / 2 - 1).all())


def test_plain_attention_against_torch_softmax():
    """The plain form against a dense softmax, its windows, and a row that sees nothing."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 4, 8), (9, 2, 8), (9, 2, 8)))
    for window in (0, 3):
        out, lse, a, big = attend(q, k, v, 4, window, 0.3)
        kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
        s = torch.einsum("ihd,jhd->hij", q, kk) * 0.3
        i, j = torch.arange(5)[:, None] + 4, torch.arange(9)[None]
        s = s.masked_fill((j > i) | ((j <= i - window) if window else False), -math.inf)
        assert torch.allclose(out, torch.einsum("hij,jhd->ihd", s.softmax(-1), vv))
        assert torch.allclose(lse, torch.logsumexp(s, -1).T)
        assert bool((a >= out.abs() - 1e-12).all()) and bool((big > 0).all())
    out, lse, _, _ = attend(q, k, v, -2, 0, 0.3)
    assert bool((out[:2] == 0).all()) and bool(torch.isinf(lse[:2]).all()) and torch.isfinite(lse[2:]).all()

"""Paged cache and the attention over it at the ends of the number ranges, and what repeated calls return."""
import math

import pytest
import torch

from paged_util import Case, attend, bounds, quantise

pytestmark = pytest.mark.gpu
E4, I8, BF = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_causal_linear_la_b200 as la

    la.load_library()
    return la


def attn(la, c, cache, **kw):
    dev = torch.device("cuda")
    k, v, ks, vs = cache
    return la.la_paged_attn(c.q.to(dev)[None], k, v, c.table.to(dev),
                            torch.tensor(c.kv_len, dtype=torch.int32, device=dev), cu_seqlens=c.cu.to(dev),
                            k_scale=ks, v_scale=vs, return_lse=True, **kw)


# ------------------------------------------- values whose code times scale leaves the range
@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("window", [0, 7])
@pytest.mark.parametrize("L,D", [(9, 64), (9, 128), (40, 64), (40, 128), (200, 128)])
@pytest.mark.parametrize("fmt", [E4, I8])
def test_values_past_the_range_reach_only_the_queries_that_see_them(la, fmt, L, D, window, simt):
    """Rows of values under a finite scale whose products with some codes are infinite: a query that does not see
    such a row returns what it returns without it, and one that does gets an infinity of the code's sign where the
    product is one.  Entries of one query tile (9 tokens) and of two."""
    c = Case([L], [100], 4, 2, D, 16, fmt, seed=L + D)
    k, v, ks, vs = c.fill(la, "cuda")
    flags = la.LA_FLAG_SIMT if simt else 0
    clean = attn(la, c, (k, v, ks, vs), window=window, flags=flags)[0][0].cpu()
    spots = [(104, 0), (107, 1)] + ([(250, 0)] if L > 150 else [])
    past = {}
    for p, h in spots:
        pg, sl = int(c.table[0, p // 16]), p % 16
        vs[pg, h, sl] = 2.0 ** 125
        code = v[pg, sl, h].float().cpu()
        past[p, h] = torch.sign(code) * (code.abs() >= 8)  # 8 * 2^125 = 2^128
        assert int((past[p, h] != 0).sum()) > 0
    out = attn(la, c, (k, v, ks, vs), window=window, flags=flags)[0][0].cpu()
    for i in range(L):
        at = 100 + i
        for h in range(2):
            seen = [past[p, g] for p, g in spots if g == h and p <= at and (not window or p > at - window)]
            o = out[i, 2 * h:2 * h + 2]
            if not seen:
                assert torch.equal(o, clean[i, 2 * h:2 * h + 2]), (i, h)
            elif not simt and len(seen) == 1:  # (in fp32, as the CUDA cores hold values, a weight times 2^133 may be finite)
                for d in torch.nonzero(seen[0]).flatten().tolist():
                    assert bool((o[:, d] == seen[0][d] * math.inf).all()), (i, h, d)


# ------------------------------------------------------------- the largest finite rows
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("fmt", [E4, I8])
def test_the_largest_rows_read_back_finite(la, fmt, dtype):
    """Rows up to the type's largest number: codes and scales of keys and of values are the formula's, but for a code whose
    product with the scale would be infinite, which is one step of the grid nearer to zero."""
    dev = torch.device("cuda")
    top = torch.finfo(dtype).max
    gen = torch.Generator().manual_seed(5)
    x = (torch.rand((2, 1, 12, 2, 64), generator=gen, dtype=torch.float64) * 2 - 1) * top
    x[:, 0, 1] = top
    x[:, 0, 2] = -top
    x[:, 0, 3] = top * (248 / 256)           # half way between e4m3's 240 and 256: to even is up
    x[:, 0, 4] = 63.5 * 2.0 ** 122           # half way between int8's 63 and 64
    x[:, 0, 5] = 127.0 * 2.0 ** 120
    x[:, 0, 6] = 0
    x[0, 0, 7, :, ::3] = -top                # keys and values have rows of their own
    x[1, 0, 8, :, ::3] = top
    x = x.to(dtype)
    k, v, ks, vs = la.kv_cache(1, 16, 2, 64, fmt)
    table, kl = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.tensor([12], dtype=torch.int32, device=dev)
    la.la_kv_write(x[0].to(dev), x[1].to(dev), k, v, table, kl, k_scale=ks, v_scale=vs)
    changed = 0
    for cache, scale, rows in ((k, ks, x[0, 0]), (v, vs, x[1, 0])):
        code, s = quantise(rows.double(), fmt)
        over = (code * s).abs() >= 2.0 ** 128
        changed += int(over.sum())
        code = torch.where(over, code.sign() * (240.0 if fmt == E4 else 63.0), code)
        assert torch.equal(scale[0, :, :12].T.cpu().double(), s[..., 0])
        assert torch.equal(cache[0, :12].float().cpu().double(), code)
        assert bool(((code * s - rows.double()).abs() <= 2.0 ** -4 * rows.double().abs() + s).all())
    assert changed > 200
    for odt in (BF, torch.float32):
        for r in la.la_kv_read(k, v, table, 12, k_scale=ks, v_scale=vs, dtype=odt):
            assert bool(torch.isfinite(r).all())


@pytest.mark.parametrize("fmt", [BF, E4, I8])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_codes_and_scales_of_values_as_of_keys(la, fmt, dtype):
    """Keys and values of rows of every size, each with rows of its own that hold an infinity, a NaN, zeros, subnormal
    numbers and ties: stored codes and scales are the formula's for both."""
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((2, 1, 40, 3, 32), generator=gen, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-140, 120, (2, 1, 40, 3, 1), generator=gen).double())
    x[0, 0, 3], x[1, 0, 4] = 0, 0
    x[0, 0, 5] = torch.arange(32) / 2.0
    x[1, 0, 6] = -torch.arange(32) / 2.0
    x = x.to(dtype)
    x[0, 0, 7, 1, 9], x[1, 0, 8, 2, 0], x[0, 0, 9, 0, 31], x[1, 0, 10, 0, 5] = math.inf, math.nan, math.nan, -math.inf
    k, v, ks, vs = la.kv_cache(3, 16, 3, 32, fmt)
    table, kl = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=dev), torch.tensor([40], dtype=torch.int32, device=dev)
    la.la_kv_write(x[0].to(dev), x[1].to(dev), k, v, table, kl, k_scale=ks, v_scale=vs)
    for cache, scale, rows in ((k, ks, x[0, 0]), (v, vs, x[1, 0])):
        got = cache[table[0].long()].reshape(48, 3, 32)[:40].cpu() if fmt != E4 else (
            cache.view(torch.int8)[table[0].long()].reshape(48, 3, 32)[:40].cpu().view(E4))
        if fmt == BF:
            want = rows.to(BF)
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
            continue
        s = scale[table[0].long()].transpose(1, 2).reshape(48, 3)[:40].cpu().double()
        bad = ~torch.isfinite(rows).all(-1)
        assert int(bad.sum()) == 2 and torch.equal(torch.isnan(s), bad)
        code, want = quantise(torch.where(bad[..., None], 0.0, rows.double()), fmt)
        assert torch.equal(got.float().double(), code)
        assert torch.equal(s[~bad], want[..., 0][~bad])


# ----------------------------------------------------------- scores that are all -infinity
@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("L,ctx", [(1, 20), (9, 100), (70, 300), (1, 20000)])
def test_scores_that_are_all_minus_infinity(la, L, ctx, simt):
    """Keys of +infinity in one element, under a query of -1 there: every score it sees is -infinity, the sum of the
    weights is 0, and the output is the formula's 0 / 0; its log-sum-exp is -infinity.  Queries of +1 there give NaN for
    both.  A query before position 0 still gives zeros.  One entry, two query tiles, keys split over CTAs."""
    c = Case([L, 3], [ctx, -2], 4, 2, 64, 16, BF, seed=L)
    c.k_rows[0][:, :, 5] = math.inf
    c.q[:L, :2, 5], c.q[:L, 2:, 5] = -1.0, 1.0
    out, lse = attn(la, c, c.fill(la, "cuda"), flags=la.LA_FLAG_SIMT if simt else 0)
    assert bool(torch.isnan(out[0, :L]).all())
    assert bool((lse[0, :L, :2] == -math.inf).all()) and bool(torch.isnan(lse[0, :L, 2:]).all())
    assert bool((out[0, L:L + 2] == 0).all()) and bool((lse[0, L:L + 2] == -math.inf).all())
    assert bool(torch.isfinite(out[0, L + 2:]).all()) and bool(torch.isfinite(lse[0, L + 2:]).all())


# --------------------------------------------------------------------- scales of the scores
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("simt", [False, True])
def test_a_large_scale_and_large_queries(la, simt, dtype):
    """A query element whose product with the scale is beyond fp32, on keys that are zero there, has no part."""
    from test_paged_gpu import hold

    c = Case([5], [60], 2, 2, 64, 16, BF, dtype=dtype, seed=3)
    c.q = (c.q.double() * 2.0 ** -100).to(dtype)
    c.q[:, :, 9] = 2.0 ** 50
    c.k_rows[0][:, :, 9] = 0
    scale = 2.0 ** 97
    out, lse = attn(la, c, c.fill(la, "cuda"), scale=scale, flags=la.LA_FLAG_SIMT if simt else 0)
    hold(c, out, lse, scale=scale, simt=simt or dtype != BF)


# ------------------------------------------------------------------------------ long items
def test_a_call_of_seconds(la):
    """28 sequences of 2^31 - 2^16 positions each, all in one page: a CTA works more than three seconds on one entry, and its
    warps without a row wait that long for its end.  The sum of the weights is the page's, once for each time it is
    seen.  (A lane's own sum takes 3.2 million additions: off by 3.2e6 2^-24 = 0.19 at most, a logarithm by 0.21.)"""
    n, page, pages = 28, 2 ** 16, 2 ** 15 - 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v, ks, vs = la.kv_cache(1, page, 1, 64, I8)
    rows = torch.randn((1, page, 1, 64), generator=gen, device="cuda").to(BF)
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    la.la_kv_write(rows, torch.zeros_like(rows), k, v, one, torch.tensor([page], dtype=torch.int32, device="cuda"),
                   k_scale=ks, v_scale=vs)
    q = torch.randn((n, 1, 1, 64), generator=gen, device="cuda").to(BF)
    out, lse = torch.full_like(q, math.nan), torch.full((n, 1, 1), math.nan, device="cuda")
    table = torch.zeros((n, pages), dtype=torch.int32, device="cuda")
    kl = torch.full((n,), page * pages, dtype=torch.int32, device="cuda")
    assert la.device_error(reset=True) == (0, 0)
    la.la_paged_attn(q, k, v, table, kl, k_scale=ks, v_scale=vs, out=out, lse=lse)
    torch.cuda.synchronize()
    assert la.device_error(reset=True) == (0, 0)
    stored = la.la_kv_read(k, v, one, page, k_scale=ks, v_scale=vs, dtype=torch.float32)[0][0, :, 0].double()
    want = torch.logsumexp(stored @ q[:, 0, 0].double().T / 8, 0) + math.log(pages)
    assert bool(((lse[:, 0, 0].double() - want).abs() <= 0.21 + 1e-3).all())
    assert bool((out == 0).all())


# ---------------------------------------------------------------------------- failure path
@pytest.mark.parametrize("fmt,lens,ctx,D", [(BF, [1, 1], [3000, 200], 128), (E4, [1, 1], [3000, 200], 128),
                                            (BF, [150, 40], [900, 0], 64), (I8, [150, 40], [900, 0], 128)])
def test_waits_that_run_out_are_reported(la, fmt, lens, ctx, D):
    """Failure detection without a GPU fault: with LA_FLAG_TEST_WAIT_TIMEOUT no CTA loads values, so its waits for them run
    out after about two seconds; it lets its copies land, frees its tensor memory and returns.  la_device_error tells
    of it, with no copy left under way, and the next calls are right.  One query tile and two, bf16 and 8 bits."""
    from test_paged_gpu import hold

    c = Case(lens, ctx, 8, 2, D, 16, fmt, seed=D)
    cache = c.fill(la, "cuda")
    assert la.device_error(reset=True) == (0, 0)
    attn(la, c, cache, flags=la.LA_FLAG_TEST_WAIT_TIMEOUT)
    torch.cuda.synchronize()
    flags, where = la.device_error(reset=True)
    assert flags == 1 and where >> 31 == 1, (flags, hex(where))
    assert la.device_error(reset=True) == (0, 0)
    for _ in range(2):
        hold(c, *attn(la, c, cache))
    assert la.device_error(reset=True) == (0, 0)


# --------------------------------------------------------------------------- repeated calls
@pytest.mark.parametrize("fmt", [BF, E4, I8])
@pytest.mark.parametrize("lens,ctx,H,Hkv,D,page,window", [
    ([1] * 33, [131 * (i % 9) + 29 * i for i in range(33)], 8, 2, 128, 16, 0),
    ([1], [30000], 8, 2, 128, 64, 0),
    ([5] * 7, [300 * i for i in range(7)], 16, 16, 64, 16, 0),
    ([1, 200, 1, 77], [4000, 700, 127, 2500], 10, 2, 128, 32, 0),
    ([300, 140], [1800, 900], 8, 2, 64, 48, 300),
])
def test_the_same_call_gives_the_same_bits(la, lens, ctx, H, Hkv, D, page, window, fmt):
    """Nothing of a result depends on the order in which CTAs or warps come: thirty calls agree bit by bit, with
    workspaces of different content and other calls in between."""
    c = Case(lens, ctx, H, Hkv, D, page, fmt, seed=D + len(lens))
    cache = c.fill(la, "cuda")
    other = Case([1, 60], [700, 40], 8, 2, 64, 16, I8, seed=2)
    other_cache = other.fill(la, "cuda")
    first = attn(la, c, cache, window=window)
    need = la.paged_attn_workspace_size(1, sum(lens), H, D, len(lens), True, Hkv, page, fmt)
    for i in range(30):
        if i % 3 == 0:
            attn(la, other, other_cache)
        ws = torch.full((need,), 37 * i % 256, dtype=torch.uint8, device="cuda")
        out, lse = attn(la, c, cache, window=window, workspace=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), i


def test_two_streams_agree_with_themselves(la):
    """Every one of many calls on two streams at once gives what the same call gives by itself."""
    cases = [Case([1, 60], [700, 40], 8, 2, 64, 16, BF, seed=1), Case([1, 60, 1], [2700, 40, 9], 8, 2, 128, 16, I8, seed=2)]
    caches = [c.fill(la, "cuda") for c in cases]
    alone = [attn(la, c, cache) for c, cache in zip(cases, caches)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attn(la, cases[i], caches[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])


@pytest.mark.parametrize("fmt", [BF, I8])
def test_a_cache_without_pages(la, fmt):
    """Every page is missing: rows of zeros, so zeros with the logarithm of the number of positions; writes go nowhere."""
    dev = torch.device("cuda")
    k, v, ks, vs = la.kv_cache(0, 16, 2, 64, fmt)
    table, kl = torch.full((1, 4), 3, dtype=torch.int32, device=dev), torch.tensor([40], dtype=torch.int32, device=dev)
    q = torch.randn(1, 5, 4, 64, device=dev).to(BF)
    la.la_kv_write(q[:, :, :2], q[:, :, 2:], k, v, table, kl, k_scale=ks, v_scale=vs)
    out, lse = la.la_paged_attn(q, k, v, table, kl, k_scale=ks, v_scale=vs, return_lse=True)
    assert bool((out == 0).all())
    want = torch.log(torch.arange(36, 41).double())[:, None].expand(5, 4)
    assert bool(((lse[0].double().cpu() - want).abs() <= 40 * 2.0 ** -23 + 2.0 ** -20).all())
    r = la.la_kv_read(k, v, table, 8, k_scale=ks, v_scale=vs)
    assert bool((r[0] == 0).all()) and bool((r[1] == 0).all())


# ---------------------------------------------------------------------- beside a linear layer
@pytest.mark.parametrize("fmt", [BF, E4, I8])
def test_a_linear_layer_and_a_softmax_layer_over_one_batch(la, oracle_mod, fmt):
    """As a hybrid stack runs: a linear-attention layer's outputs are the next layer's queries, keys and values, first for two
    packed prompts (la_fwd_chunk, then la_kv_write and la_paged_attn), then token by token (la_step on the first
    layer's states).  The first layer against the oracle, the second against the formula over the rows that the first
    one gave."""
    from parity_util import TOL, slice_rel_err, to_np

    dev, gen = torch.device("cuda"), torch.Generator().manual_seed(9)
    lens, steps, H, D, page = [150, 70], 6, 4, 64, 16
    gamma = torch.tensor([0.9, 0.95, 0.99, 0.999])
    x = [[(torch.randn((1, n + steps, H, D), generator=gen) * s).to(BF) for s in (D ** -0.5, 1.0, 0.3)] for n in lens]
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=dev)
    k, v, ks, vs = la.kv_cache(32, page, 2, D, fmt)
    table = torch.randperm(32, generator=gen).to(torch.int32).reshape(2, 16)[:, :12].contiguous().to(dev)
    sc = dict(k_scale=ks, v_scale=vs)

    def softmax_layer(o, kv_len, cu_seqlens):
        kl = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        la.la_kv_write(o[:, :, :2], o[:, :, 2:], k, v, table, kl, cu_seqlens=cu_seqlens, **sc)
        return la.la_paged_attn(o, k, v, table, kl, cu_seqlens=cu_seqlens, return_lse=True, **sc)
    q0, k0, v0 = (torch.cat([x[n][i][:, :lens[n]] for n in range(2)], 1).to(dev) for i in range(3))
    o, state = la.la_fwd_chunk(q0, k0, v0, gamma.to(dev), cu_seqlens=cu)
    p, lse = softmax_layer(o, lens, cu)
    first = [[o[0, :lens[0]]], [o[0, lens[0]:]]]
    second = [[(p[0, :lens[0]], lse[0, :lens[0]])], [(p[0, lens[0]:], lse[0, lens[0]:])]]
    for t in range(steps):
        one = [torch.cat([x[n][i][:, lens[n] + t] for n in range(2)]).to(dev) for i in range(3)]  # [2, H, D]
        o = la.la_step(one[0], one[1], one[2], gamma.to(dev), state)
        p, lse = softmax_layer(o[:, None], [n + t + 1 for n in lens], None)
        for n in range(2):
            first[n].append(o[n][None])
            second[n].append((p[n], lse[n]))
    for n in range(2):
        S = lens[n] + steps
        o = torch.cat(first[n])
        ref, _ = oracle_mod.recurrent(*x[n], gamma.tolist())
        assert slice_rel_err(to_np(o[None]), ref, [(0, 0, S)]) < TOL[BF]
        rows = o.cpu().double()
        stored = [rows[:, :2], rows[:, 2:]]
        if fmt != BF:
            stored = [c * s for c, s in (quantise(r, fmt) for r in stored)]
        want, wl, a, big = attend(rows, *stored, 0, 0, D ** -0.5)
        tol, ltol = bounds(want, wl, a, big, S, D, BF, True)
        got, gl = (torch.cat([y[i] for y in second[n]]).double().cpu() for i in range(2))
        assert bool(((got - want).abs() <= tol).all()) and bool(((gl - wl).abs() <= ltol).all())
    assert la.device_error(reset=True) == (0, 0)

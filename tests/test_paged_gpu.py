"""Paged cache and the attention over it on the GPU, against plain 64-bit forms, element by element."""
import math

import pytest
import torch

from paged_util import QMAX, Case, attend, bounds, quantise

pytestmark = pytest.mark.gpu
E4, I8, BF = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_causal_linear_la_b200 as la

    la.load_library()
    return la


def hold(c, out, lse, window=0, scale=None, simt=False, rows=None):
    """out [.., H, D] and lse against the case's 64-bit form, element by element."""
    want, wl, a, big = c.expect(window, scale)
    keys = max(max(c.kv_len), 1)
    tol, ltol = bounds(want, wl, a, big, keys, c.D, c.dtype, not simt and c.dtype == BF)
    T = int(c.cu[-1])
    o = out.reshape(-1, c.H, c.D)[:T].double().cpu()
    d = (o - want[:T]).abs()
    assert bool((d <= tol[:T]).all()), "out: worst %.3g of its bound" % float((d / tol[:T].clamp_min(1e-30)).max())
    if lse is not None:
        l = lse.reshape(-1, c.H)[:T].double().cpu()
        seen = torch.isfinite(wl[:T])
        assert torch.equal(torch.isfinite(l), seen) and bool((l[~seen] == -math.inf).all())
        assert bool(((l - wl[:T])[seen].abs() <= ltol[:T][seen]).all())


def attn(la, c, cache, window=0, scale=None, simt=False, **kw):
    dev = torch.device("cuda")
    k, v, ks, vs = cache
    q = c.q.to(dev)[None]
    return la.la_paged_attn(q, k, v, c.table.to(dev), torch.tensor(c.kv_len, dtype=torch.int32, device=dev),
                            cu_seqlens=c.cu.to(dev), k_scale=ks, v_scale=vs, window=window, scale=scale,
                            return_lse=True, flags=la.LA_FLAG_SIMT if simt else 0, **kw)


# ------------------------------------------------------------------- the cache
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("fmt", [BF, E4, I8])
@pytest.mark.parametrize("H,D,page,layout", [(3, 64, 16, "token"), (2, 128, 7, "head"), (1, 16, 1, "token"),
                                             (4, 256, 48, "token"), (5, 32, 64, "head")])
def test_write_then_read(la, dtype, fmt, H, D, page, layout):
    """Codes and scales are exactly the formula's; what was not written stays; reading gives code * scale."""
    dev = torch.device("cuda")
    c = Case([1, 0, 19, 5, 33], [0, 4, 30, 0, 77], H, H, D, page, fmt, dtype, seed=D + page, layout=layout)
    # rows of every size: an all-zero one, tiny, subnormal and huge ones, ties, an infinity, a NaN
    c.k_rows[2][30] = 0
    c.k_rows[2][31] *= 2.0 ** -120
    c.k_rows[2][32] = torch.full_like(c.k_rows[2][32], 2.0 ** -130)
    c.k_rows[2][33] *= 2.0 ** 120
    c.k_rows[2][34] = torch.arange(H * D).reshape(H, D).to(dtype) / 2
    k, v, ks, vs = c.pages(dev)
    before = k.clone(), v.clone()
    new = [torch.cat([r[s - x:] for r, s, x in zip(rows, c.kv_len, c.lens)])[None].to(dev)
           for rows in (c.k_rows, c.v_rows)]
    table, kl, cu = c.table.to(dev), torch.tensor(c.kv_len, dtype=torch.int32, device=dev), c.cu.to(dev)
    la.la_kv_write(new[0], new[1], k, v, table, kl, cu_seqlens=cu, k_scale=ks, v_scale=vs)
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for n, (x, s) in enumerate(zip(c.lens, c.kv_len)):
        for i in range(x):
            p = s - x + i
            touched[c.table[n, p // page], p % page] = True
    raw = lambda t: t.contiguous().view(torch.int16 if fmt == BF else torch.int8).cpu()  # noqa: E731
    for got, was in ((k, before[0]), (v, before[1])):
        assert torch.equal(raw(got)[~touched], raw(was)[~touched])
    start = kl - torch.tensor(c.lens, dtype=torch.int32, device=dev)
    for odt in (torch.float32, BF):
        rk, rv = la.la_kv_read(k, v, table, int(c.cu[-1]), start=start, cu_seqlens=cu, k_scale=ks, v_scale=vs,
                               dtype=odt)
        for got, rows in ((rk, c.k_rows), (rv, c.v_rows)):
            want = torch.cat([r[s - x:] for r, s, x in zip(rows, c.kv_len, c.lens)]).double()
            if fmt == BF:
                want = want.to(BF).double()
            else:
                code, s = quantise(want, fmt)
                want = code * s
            assert torch.equal(got[0].cpu(), want.to(torch.float32).to(odt))
    if fmt != BF:
        code, s = quantise(new[0][0].double().cpu(), fmt)
        at = 0
        for n, (x, ln) in enumerate(zip(c.lens, c.kv_len)):
            for i in range(x):
                p = ln - x + i
                pg, sl = c.table[n, p // page], p % page
                assert torch.equal(k[pg, sl].cpu().double(), code[at])
                assert torch.equal(ks[pg, :, sl].cpu().double(), s[at, :, 0])
                at += 1


@pytest.mark.parametrize("fmt", [E4, I8])
def test_rows_that_are_not_finite_read_back_as_nan(la, fmt):
    dev = torch.device("cuda")
    x = torch.randn(1, 4, 2, 64, device=dev)
    x[0, 1, 0, 5], x[0, 2, 1, 63], x[0, 3, 1, 0] = math.inf, math.nan, -math.inf
    k, v, ks, vs = la.kv_cache(3, 8, 2, 64, fmt)
    table, kl = torch.tensor([[2]], dtype=torch.int32, device=dev), torch.tensor([4], dtype=torch.int32, device=dev)
    la.la_kv_write(x, x, k, v, table, kl, k_scale=ks, v_scale=vs)
    r = la.la_kv_read(k, v, table, 4, k_scale=ks, v_scale=vs)[0][0]
    bad = torch.isnan(r).all(-1).cpu()
    assert bad.tolist() == [[False, False], [True, False], [False, True], [False, True]]
    assert torch.equal(torch.isnan(r).any(-1).cpu(), bad)


def test_dense_batch_strides_and_what_is_skipped(la):
    """A dense batch from a wider buffer; positions that are negative, past the table or in a missing page
    are skipped by the write and read as zeros; rows behind the packed batch stay."""
    dev = torch.device("cuda")
    wide = torch.randn(2, 6, 5, 2, 64, device=dev).to(BF)
    kx, vx = wide[:, :, 1], wide[:, :, 3]
    for fmt in (BF, E4):
        k, v, ks, vs = la.kv_cache(4, 4, 2, 64, fmt)
        for t in (k, v):
            t.view(torch.int8).zero_()
        if ks is not None:
            ks.zero_(), vs.zero_()
        # sequence 0: positions -2..3 in page 1; sequence 1: positions 4..9, pages (7: missing), 3, (past the table)
        table = torch.tensor([[1, -1], [7, 3]], dtype=torch.int32, device=dev)
        kl = torch.tensor([4, 10], dtype=torch.int32, device=dev)
        la.la_kv_write(kx, vx, k, v, table, kl, k_scale=ks, v_scale=vs)
        out = [torch.full((2, 6, 2, 64), 9.0, device=dev, dtype=BF) for _ in range(2)]
        start = torch.tensor([-2, 4], dtype=torch.int32, device=dev)
        la.la_kv_read(k, v, table, 6, start=start, k_scale=ks, v_scale=vs, k_out=out[0], v_out=out[1])
        for got, x in zip(out, (kx, vx)):
            want = x.cpu().double()
            if fmt != BF:
                code, s = quantise(want, fmt)
                want = code * s
            want[0, :2] = 0
            want[1, 4:] = 0
            assert torch.equal(got.cpu().double(), want)
        assert k[0].view(torch.int8).abs().sum() == 0 and k[2].view(torch.int8).abs().sum() == 0
        cu = torch.tensor([0, 2, 2], dtype=torch.int32, device=dev)
        o = torch.full((1, 6, 2, 64), 9.0, device=dev, dtype=BF)
        la.la_kv_read(k, v, table, 6, cu_seqlens=cu, k_scale=ks, v_scale=vs, k_out=o, v_out=torch.empty_like(o))
        assert bool((o[0, 2:] == 9).all()) and not bool((o[0, :2] == 9).any())


# --------------------------------------------------------------- the attention
SHAPES = [
    # lens, ctx, H, Hkv, D, page, layout
    ([1, 1, 1], [0, 62, 300], 4, 4, 64, 16, "token"),
    ([1, 1, 1, 1], [127, 128, 129, 511], 16, 2, 128, 64, "head"),
    ([1], [2000], 8, 1, 128, 16, "token"),
    ([3, 0, 1, 17], [5, 9, 0, 130], 6, 2, 64, 8, "token"),
    ([130, 1, 64], [0, 200, 64], 4, 4, 128, 32, "token"),
    ([70, 33], [63, 500], 10, 2, 128, 48, "head"),
    ([257], [0], 3, 1, 64, 128, "token"),
    ([40, 2], [100, 3], 12, 1, 64, 200, "token"),
    ([9], [250], 128, 1, 128, 256, "token"),
    ([5, 1], [1000, 700], 7, 7, 64, 24, "head"),
]


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("fmt", [BF, E4, I8])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-%d/%d-%d-p%d" % (len(s[0]), s[2], s[3], s[4], s[5]))
def test_attention_matches_the_formula(la, shape, fmt, simt):
    lens, ctx, H, Hkv, D, page, layout = shape
    c = Case(lens, ctx, H, Hkv, D, page, fmt, seed=page + D + H, layout=layout)
    cache = c.fill(la, "cuda")
    hold(c, *attn(la, c, cache, simt=simt), simt=simt)
    assert la.device_error(reset=True) == (0, 0)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("window", [1, 2, 31, 128, 129, 1000])
def test_windows(la, window, simt):
    c = Case([1, 150, 7], [600, 0, 250], 4, 2, 64, 16, I8, seed=window)
    cache = c.fill(la, "cuda")
    hold(c, *attn(la, c, cache, window=window, simt=simt), window=window, simt=simt)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("fmt", [BF, I8])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31, 2 ** 40])
def test_windows_past_every_position(la, window, fmt, simt):
    """The widest windows hide nothing, from queries before position 0 either."""
    c = Case([60, 3], [-20, 200], 4, 2, 64, 16, fmt, seed=31)
    hold(c, *attn(la, c, c.fill(la, "cuda"), window=window, simt=simt), window=window, simt=simt)


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("H,D,page", [(4, 16, 16), (4, 32, 5), (2, 256, 16), (4, 128, 20)])
def test_shapes_off_the_tensor_cores(la, H, D, page, fmt):
    c = Case([3, 1], [40, 7], H, 2, D, page, fmt, seed=D)
    assert la.paged_attn_path(H, D, 2, page, fmt) == la.LA_PATH_CUDA_CORE
    hold(c, *attn(la, c, c.fill(la, "cuda")), simt=True)


@pytest.mark.parametrize("fmt", [BF, E4, I8])
def test_f32_queries(la, fmt):
    c = Case([2, 40, 1], [300, 0, 5], 4, 2, 64, 16, fmt, dtype=torch.float32, seed=5)
    out, lse = attn(la, c, c.fill(la, "cuda"))
    assert out.dtype == torch.float32
    hold(c, out, lse, simt=True)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_and_rows_behind_the_batch(la, D, simt):
    """Sequences with fewer cached than new tokens (their first queries stand before position 0), an empty
    one, and tokens behind the last sequence: zeros with lse -inf, and left as they were."""
    c = Case([4, 3, 0, 200], [-4, -2, 5, -150], 4, 2, D, 16, BF, seed=2, extra_rows=3)
    c.kv_len = [max(0, s) for s in c.kv_len]
    c.ctx = [s - x for s, x in zip(c.kv_len, c.lens)]
    cache = c.fill(la, "cuda")
    T = c.q.shape[0]
    out = torch.full((1, T, 4, D), 7.0, dtype=BF, device="cuda")
    lse = torch.full((1, T, 4), 7.0, device="cuda")
    attn(la, c, cache, simt=simt, out=out, lse=lse)
    hold(c, out, lse, simt=simt)
    assert bool((out[0, -3:] == 7).all()) and bool((lse[0, -3:] == 7).all())
    assert bool((out[0, :4] == 0).all()) and bool((out[0, 4:6] == 0).all())


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("fmt", [BF, I8])
def test_missing_pages_and_short_tables(la, fmt, simt):
    """Entries outside the cache read as rows of zeros; positions past the table are not seen."""
    c = Case([5, 2], [200, 90], 4, 2, 64, 16, fmt, seed=11)
    cache = c.fill(la, "cuda")
    c.table[0, 3], c.table[0, 12], c.table[1, 0] = c.n_pages, 2 ** 31 - 1, -2 ** 31
    stored = [c.stored(0), c.stored(1)]
    for n, pages in ((0, (3, 12)), (1, (0,))):
        for x in stored[n]:
            for pg in pages:
                x[pg * 16:(pg + 1) * 16] = 0
    c.stored = lambda n: stored[n]
    hold(c, *attn(la, c, cache, simt=simt), simt=simt)
    # a table of 8 pages: positions from 128 on are not seen
    c.table = c.table[:, :8].contiguous()
    stored = [[x[:128] for x in s] for s in stored]
    c.stored = lambda n: stored[n]
    hold(c, *attn(la, c, cache, simt=simt), simt=simt)


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("fmt", [E4, I8, BF])
def test_not_finite_rows_reach_only_the_queries_that_see_them(la, fmt, simt):
    """A NaN key (and value, in the 8-bit caches) at a late position leaves earlier queries alone; the
    later ones get NaN."""
    c = Case([40], [100], 4, 2, 64, 16, fmt, seed=4)
    c.k_rows[0][120, 0, 3] = math.nan
    if fmt != BF:
        c.v_rows[0][125, 1, 3] = math.inf
    cache = c.fill(la, "cuda")
    out, lse = attn(la, c, cache, simt=simt)
    o = out[0].cpu()
    assert torch.isfinite(o[:20, :2]).all() and torch.isnan(o[20:, :2]).all()
    assert torch.isnan(lse[0, 20:, :2]).all()
    if fmt != BF:
        assert torch.isfinite(o[:25, 2:]).all() and torch.isnan(o[25:, 2:]).all()
    else:
        assert torch.isfinite(o[:, 2:]).all()


@pytest.mark.parametrize("simt", [False, True])
def test_scores_of_every_size(la, simt):
    """Scores of tens of thousands (one key takes all), and equal ones (a plain mean)."""
    c = Case([30], [300], 2, 2, 64, 16, BF, seed=8)
    cache = c.fill(la, "cuda")
    hold(c, *attn(la, c, cache, scale=20.0, simt=simt), scale=20.0, simt=simt)
    hold(c, *attn(la, c, cache, scale=1e-12, simt=simt), scale=1e-12, simt=simt)
    # rising scores: each block of keys beats the last, so the running maximum moves every time
    k = torch.arange(330).float()[:, None, None].expand(330, 2, 64) / 40
    c.k_rows[0] = k.to(BF)
    c.q = torch.ones_like(c.q)
    cache = c.fill(la, "cuda")
    hold(c, *attn(la, c, cache, scale=1.0, simt=simt), scale=1.0, simt=simt)


@pytest.mark.parametrize("fmt", [BF, E4])
def test_dense_batch_with_strides(la, fmt):
    """Queries and outputs in the middle of wider rows, a dense batch."""
    c = Case([6, 6, 6], [100, 0, 31], 8, 2, 64, 16, fmt, seed=21)
    cache = c.fill(la, "cuda")
    dev = torch.device("cuda")
    wide = torch.randn(3, 6, 24, 64, device=dev).to(BF)
    wide[:, :, 8:16] = c.q.reshape(3, 6, 8, 64).to(dev)
    owide = torch.full((3, 6, 24, 64), 5.0, dtype=BF, device=dev)
    k, v, ks, vs = cache
    out, lse = la.la_paged_attn(wide[:, :, 8:16], k, v, c.table.to(dev),
                                torch.tensor(c.kv_len, dtype=torch.int32, device=dev), k_scale=ks, v_scale=vs,
                                out=owide[:, :, 16:], return_lse=True)
    hold(c, out, lse)
    assert bool((owide[:, :, :16] == 5).all())


def test_broadcast_queries(la):
    """One query for every head (a zero head stride) takes the CUDA cores and gives the same."""
    c = Case([3], [50], 4, 2, 64, 16, BF, seed=3)
    one = c.q[:, :1].cuda()
    c.q = c.q[:, :1].expand(-1, 4, -1)
    k, v, _, _ = c.fill(la, "cuda")
    out, lse = la.la_paged_attn(one.expand(-1, 4, -1)[None], k, v, c.table.cuda(),
                                torch.tensor(c.kv_len, dtype=torch.int32, device="cuda"), cu_seqlens=c.cu.cuda(),
                                return_lse=True)
    hold(c, out, lse, simt=True)


@pytest.mark.parametrize("fmt", [BF, E4, I8])
def test_a_prompt_in_pieces_then_token_by_token(la, fmt):
    """As a server runs it: pieces of prompts of two sequences are written and attended to, then single
    tokens; every output equals the formula over the whole stored sequence."""
    dev = torch.device("cuda")
    c = Case([400, 260], [0, 0], 8, 2, 64, 16, fmt, seed=17)
    k, v, ks, vs = c.pages(dev)
    table = c.table.to(dev)
    want, wl, a, big = c.expect()
    tol, ltol = bounds(want, wl, a, big, 400, 64, BF, True)
    done = [0, 0]
    for step in ([128, 100], [1, 130], [200, 1], [64, 20]) + ([1, 1],) * 7:
        ln = [min(x, s - d) for x, s, d in zip(step, c.kv_len, done)]
        rows = [torch.cat([r[d:d + x] for r, d, x in zip(rs, done, ln)])[None].to(dev) for rs in (c.k_rows, c.v_rows)]
        q = torch.cat([c.q[int(c.cu[n]) + d:int(c.cu[n]) + d + x] for n, (d, x) in enumerate(zip(done, ln))])[None]
        done = [d + x for d, x in zip(done, ln)]
        cu = torch.tensor([0, ln[0], sum(ln)], dtype=torch.int32, device=dev)
        kl = torch.tensor(done, dtype=torch.int32, device=dev)
        la.la_kv_write(rows[0], rows[1], k, v, table, kl, cu_seqlens=cu, k_scale=ks, v_scale=vs)
        out, lse = la.la_paged_attn(q.to(dev), k, v, table, kl, cu_seqlens=cu, k_scale=ks, v_scale=vs,
                                    return_lse=True)
        at = torch.cat([torch.arange(int(c.cu[n]) + d - x, int(c.cu[n]) + d) for n, (d, x) in enumerate(zip(done, ln))])
        assert bool(((out[0].double().cpu() - want[at]).abs() <= tol[at]).all())
        assert bool(((lse[0].double().cpu() - wl[at]).abs() <= ltol[at]).all())
    assert done == [400, 258]  # the sum of the pieces


def test_replayed_graph_follows_its_inputs(la):
    """Write and attention captured once and replayed with other rows, lengths and tables; another call
    with a workspace of its own runs in between."""
    dev = torch.device("cuda")
    a, b = (Case([1, 1, 1], ctx, 8, 2, 128, 16, E4, seed=s) for s, ctx in ((1, [300, 5, 77]), (2, [129, 400, 0])))
    pages = max(a.n_pages, b.n_pages)
    k, v, ks, vs = la.kv_cache(pages, 16, 2, 128, E4)
    table = torch.full((3, max(a.max_pages, b.max_pages)), -1, dtype=torch.int32, device=dev)
    kl = torch.zeros(3, dtype=torch.int32, device=dev)
    q, kx, vx = (torch.zeros(3, 1, h, 128, dtype=BF, device=dev) for h in (8, 2, 2))
    ws = torch.empty(max(256, la.paged_attn_workspace_size(3, 1, 8, 128, 3, False, 2, 16, E4)), dtype=torch.uint8, device=dev)

    def load(c):
        cache = c.fill(la, dev, upto=[s - 1 for s in c.kv_len])
        for mine, theirs in zip((k, v, ks, vs), cache):
            mine[: c.n_pages].view(torch.int8).copy_(theirs.view(torch.int8))
        table.fill_(-1)
        table[:, : c.max_pages] = c.table.to(dev)
        kl.copy_(torch.tensor(c.kv_len, dtype=torch.int32))
        q.copy_(c.q[:, None].to(dev))
        kx.copy_(torch.stack([r[-1:] for r in c.k_rows]).to(dev))
        vx.copy_(torch.stack([r[-1:] for r in c.v_rows]).to(dev))

    def step():
        la.la_kv_write(kx, vx, k, v, table, kl, k_scale=ks, v_scale=vs)
        return la.la_paged_attn(q, k, v, table, kl, k_scale=ks, v_scale=vs, return_lse=True, workspace=ws)
    load(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for c in (a, b, a, b):
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        hold(c, out, lse)
        hold(c, *attn(la, c, c.fill(la, dev)))


def test_two_streams_with_a_workspace_each(la):
    dev = torch.device("cuda")
    cases = [Case([1, 60], [700, 40], 8, 2, 64, 16, f, seed=s) for s, f in ((1, BF), (2, I8))]
    caches = [c.fill(la, dev) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for c, cache, s in zip(cases, caches, streams):
            with torch.cuda.stream(s):
                got.append((c, attn(la, c, cache)))
    torch.cuda.synchronize()
    for c, r in got[-4:]:
        hold(c, *r)
    # the stream argument: outputs and workspace belong to that stream
    o = attn(la, cases[0], caches[0], stream=streams[1])
    streams[1].synchronize()
    hold(cases[0], *o)


def test_a_fresh_thread(la):
    import threading

    c = Case([20], [100], 4, 2, 64, 16, BF, seed=6)
    cache = c.fill(la, "cuda")
    torch.cuda.synchronize()
    got = []
    t = threading.Thread(target=lambda: got.append(attn(la, c, cache)))
    t.start()
    t.join()
    hold(c, *got[0])


def test_offsets_past_32_bits(la):
    """Pages far behind the first 2^32 bytes of a cache, and 2^31 elements."""
    dev = torch.device("cuda")
    page, H, D = 64, 4, 128
    n_pages = 2 ** 31 // (page * H * D) + 4096  # over 2^31 elements; 4.5 GB of bf16 keys
    for fmt in (BF, I8):
        k, v, ks, vs = la.kv_cache(n_pages, page, H, D, fmt)
        c = Case([70], [200], 8, H, D, page, fmt, seed=9)
        far = n_pages - 1 - torch.arange(c.max_pages, dtype=torch.int32)[None] * 3
        c.table = far.contiguous()
        rows = [r[0][None].to(dev) for r in (c.k_rows, c.v_rows)]
        kl = torch.tensor(c.kv_len, dtype=torch.int32, device=dev)
        la.la_kv_write(rows[0], rows[1], k, v, far.to(dev), kl, k_scale=ks, v_scale=vs)
        rk, _ = la.la_kv_read(k, v, far.to(dev), c.kv_len[0], k_scale=ks, v_scale=vs)
        assert torch.equal(rk[0].cpu().double(), c.stored(0)[0])
        hold(c, *attn(la, c, (k, v, ks, vs)))
        del k, v, ks, vs
        torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt,H,Hkv,D,n,ctx", [(BF, 16, 4, 128, 2, 20000), (I8, 8, 8, 64, 1, 33333),
                                               (E4, 8, 1, 128, 3, 9000)])
def test_long_contexts_of_single_tokens(la, fmt, H, Hkv, D, n, ctx):
    """Keys of one token split over many CTAs; ragged lengths beside each other."""
    ctxs = [ctx, 3, 700][:n]
    c = Case([1] * n, ctxs, H, Hkv, D, 64, fmt, seed=13)
    hold(c, *attn(la, c, c.fill(la, "cuda")))


@pytest.mark.parametrize("fmt", [BF, E4, I8])
@pytest.mark.parametrize("lens,ctx,H,Hkv,D,page,window", [
    ([1] * 40, [128 * (i % 7) + 37 * i for i in range(40)], 8, 8, 64, 16, 0),      # many short items a CTA
    ([1, 90, 1, 33, 2], [4000, 700, 127, 3000, 2500], 16, 8, 128, 32, 0),          # both kinds of items, mixed
    ([150, 70], [2100, 900], 6, 6, 64, 64, 0),                                      # two query tiles, cut items
    ([140, 1, 9], [1500, 4000, 2048], 16, 16, 64, 16, 700),                         # under a window
    ([300], [1800], 10, 2, 128, 128, 0),
])
def test_several_items_and_cut_ones_a_cta(la, lens, ctx, H, Hkv, D, page, window, fmt):
    """More key tiles than CTAs: a CTA walks several entries, and entries are cut between CTAs anywhere."""
    c = Case(lens, ctx, H, Hkv, D, page, fmt, seed=len(lens) + D, layout="head" if D == 64 else "token")
    hold(c, *attn(la, c, c.fill(la, "cuda"), window=window), window=window)
    assert la.device_error(reset=True) == (0, 0)


@pytest.mark.parametrize("packed", [True, False])
def test_more_sequences_than_the_plan_takes_at_once(la, packed):
    """1500 sequences: the plan's searches leave shared memory.  Every tenth is empty in the packed batch."""
    n = 1500
    lens = [0 if packed and i % 10 == 3 else 1 + (i % 3 if packed else 0) for i in range(n)]
    c = Case(lens, [(7 * i) % 150 for i in range(n)], 2, 2, 64, 16, I8, seed=30)
    k, v, ks, vs = c.fill(la, "cuda")
    q, cu = (c.q[None], c.cu.cuda()) if packed else (c.q[:, None], None)
    out, lse = la.la_paged_attn(q.cuda(), k, v, c.table.cuda(), torch.tensor(c.kv_len, dtype=torch.int32, device="cuda"),
                                cu_seqlens=cu, k_scale=ks, v_scale=vs, return_lse=True)
    hold(c, out, lse)


@pytest.mark.parametrize("H,D,lens", [(65, 64, [3, 1]), (100, 128, [2]), (128, 64, [1, 5]), (33, 64, [4])])
def test_many_heads_on_one_cache_head(la, H, D, lens):
    """Groups of heads that leave rows of a query tile unused, or more of them than a 64-row tile holds."""
    c = Case(lens, [300] * len(lens), H, 1, D, 16, BF, seed=H)
    hold(c, *attn(la, c, c.fill(la, "cuda")))


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("fmt", [BF, E4])
def test_values_that_are_not_numbers_element_by_element(la, fmt, window, simt):
    """An infinity (bf16) or a NaN code (e4m3) in one element of a value row reaches that column of the queries
    that see the row, and nothing else: 200 queries over two key tiles, rows seen by some of a query tile."""
    c = Case([200], [60], 4, 2, 64, 16, fmt, seed=14)
    k, v, ks, vs = c.fill(la, "cuda")
    clean = attn(la, c, (k, v, ks, vs), window=window, simt=simt)[0][0].cpu()
    for p, h, d in ((150, 0, 7), (250, 1, 63), (61, 0, 32)):
        row = v[c.table[0, p // 16], p % 16, h]
        (row.view(torch.int8) if fmt == E4 else row)[d] = 0x7F if fmt == E4 else -math.inf
    out = attn(la, c, (k, v, ks, vs), window=window, simt=simt)[0][0].cpu()
    want = clean.clone()
    for p, h, d in ((150, 0, 7), (250, 1, 63), (61, 0, 32)):
        for i in range(200):
            if p <= 60 + i and (not window or p > 60 + i - window):
                want[i, 2 * h:2 * h + 2, d] = math.nan if fmt == E4 else -math.inf
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isfinite(out), ~bad)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[~bad], clean[~bad])


def test_scales_of_every_size_and_other_ones(la):
    """Rows whose scales reach from 2^-100 to 2^100 in one cache, and scales that are not powers of two (rounded to
    the nearest bf16 product)."""
    for fmt in (E4, I8):
        c = Case([3], [200], 2, 2, 64, 16, fmt, seed=19)
        c.v_rows[0] = (c.v_rows[0].double() * torch.exp2(torch.randint(-100, 100, (203, 1, 1)).double())).to(BF)
        hold(c, *attn(la, c, c.fill(la, "cuda")))
        c = Case([3], [200], 2, 2, 64, 16, fmt, seed=20)
        k, v, ks, vs = c.fill(la, "cuda")
        ks *= 1.25  # 5 significant bits with e4m3's codes: exact; int8's round to bf16
        stored = c.stored(0)
        c.stored = lambda n: [(stored[0] * 1.25).to(torch.float32).to(BF).double(), stored[1]]
        hold(c, *attn(la, c, (k, v, ks, vs)))


def test_a_workspace_may_hold_anything_and_is_checked(la):
    c = Case([1, 70], [3000, 100], 8, 2, 128, 16, E4, seed=23)
    cache = c.fill(la, "cuda")
    need = la.paged_attn_workspace_size(1, 71, 8, 128, 2, True, 2, 16, E4)
    for byte in (0, 0xFF, 0x7F):
        ws = torch.full((need,), byte, dtype=torch.uint8, device="cuda")
        hold(c, *attn(la, c, cache, workspace=ws))
    with pytest.raises(la.LaError):
        attn(la, c, cache, workspace=ws[: need - 1])

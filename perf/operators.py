"""Cases, plain forms and 64-bit forms of the paged-cache attention operators.

Three operators of a serving stack that runs softmax attention layers beside
linear attention ones:

* ``la_kv_write``: new tokens' keys and values are quantised (8 bits with one
  power-of-two scale for each token and head, or bf16 as they are) and stored in
  the pages of a cache;
* ``la_kv_read``: a range of positions is read back from the pages;
* ``la_paged_attn``: a chunk of new tokens of each sequence (a prompt, a piece of
  one, a few drafted tokens, or a single one) attends causally to everything
  its sequence has in the cache, with an optional sliding window.

``own`` False computes them with elementary torch operations in 32 bits, ``own``
True through the package's entry points.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
# qmax = M * 2^E with M in [0.5, 1): the smallest power of two s with amax <= qmax * s follows
# from amax's own mantissa and exponent by one comparison
QMAX_ME = {"e4m3": (0.875, 9), "int8": (0.9921875, 7)}
CODE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
CODE_BYTES = {"bf16": 2, "e4m3": 1, "int8": 1}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of each of 64 running sequences is stored and read back: latency
        dict(name="cache step int8", kind="cache", write=True, n=64, steps=0, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=2047, Hkv=8, D=128, page=16, fmt="int8", layout="token"),
        # the packed batch of 64 prompts of 128 to 2048 tokens is stored, then read back for a dense kernel
        dict(name="cache prompts e4m3", kind="cache", write=True, n=64, steps=0, new_lo=128, new_hi=2048, ctx_lo=0,
             ctx_hi=0, Hkv=8, D=128, page=64, fmt="e4m3", layout="head"),
        # a long shared prefix is read back from an 8-bit cache (exporting it, or moving it to another worker)
        dict(name="cache read int8", kind="cache", write=False, n=16, steps=0, new_lo=4097, new_hi=16384, ctx_lo=0,
             ctx_hi=500, Hkv=8, D=128, page=16, fmt="int8", layout="token"),
        # a handful of short conversations, one token each: the smallest attention call
        dict(name="step short bf16", kind="attn", n=4, steps=4, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=511, H=16,
             Hkv=4, D=128, page=16, fmt="bf16", layout="token", window=0, lse=False),
        # the decode batch of 256 sequences, ragged lengths, bf16 cache: bound by memory
        dict(name="step batch bf16", kind="attn", n=256, steps=256, new_lo=1, new_hi=1, ctx_lo=127, ctx_hi=8191,
             H=16, Hkv=4, D=128, page=64, fmt="bf16", layout="token", window=0, lse=False),
        # a decode batch with 8 query heads a key head over an int8 cache in small pages
        dict(name="step batch int8", kind="attn", n=64, steps=64, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=16383, H=16,
             Hkv=2, D=128, page=16, fmt="int8", layout="head", window=0, lse=False),
        # one token over the 1,048,576 tokens of a single sequence: the key axis has to be split
        dict(name="step 1M e4m3", kind="attn", n=1, steps=1, new_lo=1, new_hi=1, ctx_lo=1048575, ctx_hi=1048575,
             H=16, Hkv=4, D=128, page=256, fmt="e4m3", layout="token", window=0, lse=False),
        # five drafted tokens of each of 32 sequences are verified; heads are not shared; with log-sum-exps
        dict(name="draft bf16 d64", kind="attn", n=32, steps=0, new_lo=5, new_hi=5, ctx_lo=0, ctx_hi=2990, H=16,
             Hkv=16, D=64, page=16, fmt="bf16", layout="token", window=0, lse=True),
        # a serving step that mixes single tokens with pieces of prompts; 5 query heads a key head
        dict(name="mixed e4m3", kind="attn", n=48, steps=44, new_lo=200, new_hi=512, ctx_lo=0, ctx_hi=4000, H=20,
             Hkv=4, D=128, page=32, fmt="e4m3", layout="token", window=0, lse=False),
        # pieces of prompts through sliding-window layers, int8 cache, 64-wide heads
        dict(name="window int8 d64", kind="attn", n=16, steps=0, new_lo=64, new_hi=1024, ctx_lo=0, ctx_hi=7000, H=16,
             Hkv=2, D=64, page=48, fmt="int8", layout="head", window=1024, lse=True),
        # the last 2048 tokens of a 16384-token prompt taken in chunks
        dict(name="chunk bf16", kind="attn", n=1, steps=0, new_lo=2048, new_hi=2048, ctx_lo=14336, ctx_hi=14336, H=16,
             Hkv=4, D=128, page=64, fmt="bf16", layout="token", window=0, lse=False),
        # two whole prompts of 8192 tokens: the largest work
        dict(name="prompt bf16", kind="attn", n=2, steps=0, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0, H=16,
             Hkv=4, D=128, page=128, fmt="bf16", layout="token", window=0, lse=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    fmt = rng.choice(["bf16", "e4m3", "int8"])
    base = dict(fmt=fmt, layout=rng.choice(["token", "head"]), D=rng.choice([64, 128]),
                page=rng.choice([8, 16, 32, 48, 64, 128, 200, 256]), Hkv=rng.choice([1, 2, 3, 4, 8]))
    if rng.random() < 0.3:
        write = rng.random() < 0.6
        hi = _log_int(rng, 1, 16384)
        c = dict(kind="cache", write=write, n=_log_int(rng, 1, 256), steps=0, new_lo=rng.randint(0, hi), new_hi=hi,
                 ctx_lo=0, ctx_hi=_log_int(rng, 1, 2048), **base)
        while _cache_cost(c) > 0.8e9:
            c["n"] = (c["n"] + 1) // 2
            c["new_hi"] = max(1, c["new_hi"] * 3 // 4)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
        return c
    mode = rng.choice(["step", "step", "draft", "chunk", "chunk", "mixed"])
    n = _log_int(rng, 1, 256 if mode in ("step", "draft") else 48)
    hi = {"step": 1, "draft": rng.randint(2, 16)}.get(mode) or _log_int(rng, 17, 4096)
    lo = hi if mode in ("step", "draft") else rng.randint(1, hi)
    c = dict(kind="attn", n=n, steps=n if mode == "step" else rng.randint(0, n) if mode == "mixed" else 0, new_lo=lo,
             new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 16, 32768),
             H=base["Hkv"] * rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]),
             window=0 if rng.random() < 0.6 else _log_int(rng, 1, 4096), lse=rng.random() < 0.5, **base)
    while True:
        lens, kv = _lengths(c)
        w = work(c)
        plain = c["n"] * max(lens) * c["H"] * max(kv)
        if w["flops"] <= 5e11 and w["bytes"] <= 2e9 and plain <= 8e8 and c["n"] * max(kv) * c["Hkv"] * c["D"] <= 1e9:
            return c
        c["n"] = (c["n"] + 1) // 2
        c["steps"] = min(c["steps"], c["n"])
        if mode == "step":
            c["steps"] = c["n"]
        c["ctx_hi"] = max(16, c["ctx_hi"] * 3 // 4)
        c["new_hi"] = c["new_hi"] if mode in ("step", "draft") else max(17, c["new_hi"] * 3 // 4)
        c["new_lo"] = min(c["new_lo"], c["new_hi"])


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence: they belong to the
    case, so that its work is known; the first `steps` sequences have one new token."""
    r = random.Random("%d %d %d %d %d" % (c["n"], c["new_lo"], c["new_hi"], c["ctx_lo"], c["ctx_hi"]))
    lens = [1 if i < c["steps"] else r.randint(c["new_lo"], c["new_hi"]) for i in range(c["n"])]
    if c["n"] > 0 and max(lens) == 0:
        lens[0] = 1
    return lens, [r.randint(c["ctx_lo"], c["ctx_hi"]) + x for x in lens]


def _cache_cost(c):
    return work(c)["bytes"]


def work(case):
    lens, kv = _lengths(case)
    D, Hkv, cb = case["D"], case["Hkv"], CODE_BYTES[case["fmt"]]
    row = Hkv * (D * cb + (4 if cb == 1 else 0))  # one token's codes and scales, keys or values
    if case["kind"] == "cache":
        t = sum(lens)
        # codes are written (or read) once, bf16 rows read and written once
        return {"bytes": 2.0 * t * (row + Hkv * D * 2 * (2 if case["write"] else 1)), "flops": 4.0 * t * Hkv * D}
    w, pairs, keys = case["window"], 0, 0
    for x, s in zip(lens, kv):
        first = s - x
        if w:
            # positions p = first .. s-1 see min(p + 1, w) keys
            full = max(0, s - max(first, w - 1))
            part = x - full
            pairs += full * w + part * (first + 1) + part * (part - 1) // 2
            keys += min(s, x + w - 1)
        else:
            pairs += x * (first + 1) + x * (x - 1) // 2
            keys += s
    t, H = sum(lens), case["H"]
    return {"bytes": float(2 * keys * row + 2 * t * H * D * 2 + (t * H * 4 if case["lse"] else 0)),
            "flops": 4.0 * D * H * pairs}


# ------------------------------------------------------------------------ inputs
def _rows(gen, shape, outliers):
    """Rows as a projection gives them: normal, with a few channels that are much larger (keys)."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if outliers:
        x *= torch.exp(0.5 * torch.randn((1,) * (len(shape) - 1) + shape[-1:], generator=gen, device="cuda"))
    return x


def _scale_of(x, fmt):
    """The smallest power of two s >= 2^-126 with max |x| <= qmax s, for each row of x."""
    m, e = torch.frexp(x.abs().amax(-1))
    qm, qe = QMAX_ME[fmt]
    e = (e - qe + (m > qm).to(e.dtype)).clamp_min(-126)
    return torch.ldexp(torch.ones_like(m), e)


def _codes_of(x, s, fmt):
    y = x / s.unsqueeze(-1)
    return torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)


def _in_layout(pages, layout):
    """[pages, slots, heads, D], stored token by token or head by head."""
    return pages if layout == "token" else pages.transpose(1, 2).contiguous().transpose(1, 2)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, kv = _lengths(c)
    N, Hkv, D, P, fmt = c["n"], c["Hkv"], c["D"], c["page"], c["fmt"]
    dev = dict(device="cuda")
    need = [-(-s // P) for s in kv]
    max_pages = max(1, max(need))
    n_pages = sum(need) + 3
    # pages are handed out in no order; entries of the table that no token needs are -1
    perm = torch.randperm(n_pages, generator=gen, **dev).to(torch.int32)
    kvt, lent = (torch.tensor(x, dtype=torch.int32, **dev) for x in (kv, lens))
    needt = (kvt + (P - 1)) // P
    slot = torch.arange(max_pages, **dev)
    used = slot[None, :] < needt[:, None]
    table = torch.full((N, max_pages), -1, dtype=torch.int32, **dev)
    table[used] = perm[: sum(need)]
    cu = torch.zeros(N + 1, dtype=torch.int32, **dev)
    cu[1:] = torch.cumsum(lent, 0)
    T = int(sum(lens))
    dense = min(lens) == max(lens)
    st = dict(case=c, table=table, kv_len=kvt, cu=None if dense else cu, T=T, N=N, lens=lent,
              L=max(lens), S=max(kv))
    lead = (N, lens[0]) if dense else (1, T)
    # which (page, slot) holds a token that was stored before this call
    have = kvt - lent if c["kind"] == "cache" and c["write"] else kvt
    pos = torch.full((n_pages, P), -1, dtype=torch.int64, **dev)
    owner = torch.zeros(n_pages, dtype=torch.int64, **dev)
    n_of, i_of = torch.nonzero(used, as_tuple=True)
    pg = table[used].long()
    owner[pg] = n_of
    pos[pg] = i_of[:, None] * P + torch.arange(P, **dev)[None, :]
    live = (pos >= 0) & (pos < have.long()[owner][:, None])
    # what was never stored is whatever the memory held: NaN in bf16 pages, any code and NaN scales in 8-bit ones
    for name, outliers in (("k", True), ("v", False)):
        x = _rows(gen, (n_pages, P, Hkv, D), outliers)
        if fmt == "bf16":
            x = torch.where(live[:, :, None, None], x, float("nan"))
            st[name + "_cache"] = _in_layout(x.to(torch.bfloat16), c["layout"])
            st[name + "_scale"] = None
        else:
            s = _scale_of(x, fmt)
            st[name + "_cache"] = _in_layout(_codes_of(x, s, fmt), c["layout"])
            s = torch.where(live[:, :, None], s, float("nan"))
            st[name + "_scale"] = s.transpose(1, 2).contiguous()  # [pages, heads, slots]
        del x
    if c["kind"] == "cache":
        st["start"] = (kvt - lent).to(torch.int32)
        if c["write"]:
            st["k"] = _rows(gen, lead + (Hkv, D), True).to(torch.bfloat16)
            st["v"] = _rows(gen, lead + (Hkv, D), False).to(torch.bfloat16)
        st["lead"] = lead
    else:
        # queries with logits of a spread that a trained layer shows
        st["q"] = (1.5 * _rows(gen, lead + (c["H"], D), False)).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------------ the pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["kind"] == "cache":
        return _cache_plain(state, c)
    return _attn_plain(state, c)


def _run_own(st, c):
    import chunkwise_causal_linear_la_b200 as la

    scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
    if c["kind"] == "cache":
        if c["write"]:
            la.la_kv_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                           cu_seqlens=st["cu"], **scales)
        k, v = la.la_kv_read(st["k_cache"], st["v_cache"], st["table"], st["lead"][1], start=st["start"],
                             cu_seqlens=st["cu"], **scales)
        return {"k": k, "v": v}
    out, lse = la.la_paged_attn(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"], cu_seqlens=st["cu"],
                                window=c["window"], return_lse=c["lse"], **scales)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _tokens(st):
    """Sequence and place in it of each new token, in the order of the packed rows."""
    n = torch.repeat_interleave(torch.arange(st["N"], device="cuda"), st["lens"].long(), output_size=st["T"])
    first = torch.cumsum(st["lens"].long(), 0) - st["lens"]
    return n, torch.arange(st["T"], device="cuda") - first[n]


def _cache_plain(st, c):
    n, i = _tokens(st)
    p = (st["kv_len"] - st["lens"]).long()[n] + i
    page, slot = st["table"].long()[n, p // c["page"]], p % c["page"]
    got = {}
    for name in ("k", "v"):
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        if c["write"]:
            x = st[name].reshape(st["T"], c["Hkv"], c["D"]).float()
            if scale is None:
                cache[page, slot] = x.to(torch.bfloat16)
            else:
                s = _scale_of(x, c["fmt"])
                # float8 tensors take no index assignment: as bytes
                cache.view(torch.int8)[page, slot] = _codes_of(x, s, c["fmt"]).view(torch.int8)
                scale[page, :, slot] = s
        raw = cache[page, slot] if scale is None else cache.view(torch.int8)[page, slot].view(cache.dtype)
        y = raw.float()
        if scale is not None:
            y = y * scale[page, :, slot].unsqueeze(-1)
        got[name] = y.to(torch.bfloat16).reshape(st["lead"] + (c["Hkv"], c["D"]))
    return got


def _attn_plain(st, c):
    N, L, S, H, Hkv, D, P = st["N"], st["L"], st["S"], c["H"], c["Hkv"], c["D"], c["page"]
    g = H // Hkv
    n, i = _tokens(st)
    q = torch.zeros((N, L, H, D), device="cuda")
    q[n, i] = st["q"].reshape(st["T"], H, D).float()
    kv_len, lens = st["kv_len"].long(), st["lens"].long()
    # the cache of each sequence as one padded block; rows behind its length are zeros
    p = torch.arange(S, device="cuda")
    page = st["table"].long()[:, p // P].clamp_min(0)
    slot = (p % P)[None, :].expand(N, S)
    live = p[None, :] < kv_len[:, None]
    kv = []
    for name in ("k", "v"):
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        if scale is None:
            x = cache[page, slot].float()
        else:
            x = cache.view(torch.int8)[page, slot].view(cache.dtype).float() * scale[page, :, slot].unsqueeze(-1)
        kv.append(x.masked_fill_(~live[:, :, None, None], 0.0).transpose(1, 2))  # [N, Hkv, S, D]
    qh = q.reshape(N, L, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, g * L, D)
    s = torch.matmul(qh, kv[0].transpose(2, 3)).mul_(D ** -0.5).reshape(N, Hkv, g, L, S)
    at = (kv_len - lens)[:, None] + torch.arange(L, device="cuda")[None, :]  # position of each query
    seen = p[None, None, :] <= at[:, :, None]
    if c["window"]:
        seen = seen & (p[None, None, :] > at[:, :, None] - c["window"])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = s.sub_(m).exp_()
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.reshape(N, Hkv, g * L, S), kv[1]).reshape(N, Hkv, g, L, D)
    o = o / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 3, 1, 2, 4).reshape(N, L, H, D)[n, i].to(torch.bfloat16).reshape(st["q"].shape)
    if not c["lse"]:
        return {"out": o}
    lse = (m + torch.log(z)).squeeze(-1).permute(0, 3, 1, 2).reshape(N, L, H)[n, i]
    return {"out": o, "lse": lse.reshape(st["q"].shape[:3])}


# ------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and key head by key head."""
    st = prepare(case, seed)
    c = st["case"]
    lens, kv = _lengths(c)
    P, Hkv, D = c["page"], c["Hkv"], c["D"]
    table = st["table"].cpu().long()

    def cached(name, n, lo, hi, h):
        p = torch.arange(lo, hi)
        page, slot = table[n][p // P].cuda(), (p % P).cuda()
        cache, scale = st[name + "_cache"], st[name + "_scale"]
        if scale is None:
            return cache[page, slot, h].double()
        x = cache[:, :, h].view(torch.int8)[page, slot].view(cache.dtype).double()
        return x * scale[page, h, slot].double()[:, None]

    if c["kind"] == "cache":
        if c["write"]:
            return {x: _stored(st[x].double(), c["fmt"]) for x in ("k", "v")}
        rows = {x: [torch.stack([cached(x, n, s - y, s, h) for h in range(Hkv)], 1)
                    for n, (y, s) in enumerate(zip(lens, kv))] for x in ("k", "v")}
        return {x: torch.cat(rows[x]).reshape(st["lead"] + (Hkv, D)) for x in rows}
    H, w = c["H"], c["window"]
    g = H // Hkv
    q = st["q"].reshape(st["T"], H, D)
    out = torch.zeros((st["T"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for n, (x, s) in enumerate(zip(lens, kv)):
        for a in range(0, x, 1024):
            b = min(x, a + 1024)
            at = torch.arange(s - x + a, s - x + b, device="cuda")
            lo, hi = max(0, s - x + a - w + 1) if w else 0, s - x + b
            p = torch.arange(lo, hi, device="cuda")
            hide = p[None, :] > at[:, None]
            if w:
                hide = hide | (p[None, :] <= at[:, None] - w)
            for h in range(Hkv):
                k, v = cached("k", n, lo, hi, h), cached("v", n, lo, hi, h)
                for j in range(h * g, (h + 1) * g):
                    z = (q[t0 + a:t0 + b, j].double() @ k.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
                    l = torch.logsumexp(z, -1)
                    lse[t0 + a:t0 + b, j] = l
                    out[t0 + a:t0 + b, j] = torch.exp(z - l[:, None]) @ v
        t0 += x
    out = out.reshape(st["q"].shape)
    return {"out": out, "lse": lse.reshape(out.shape[:3])} if c["lse"] else {"out": out}


def _stored(x, fmt):
    """What a row reads back as: its values on the 8-bit grid of its scale."""
    if fmt == "bf16":
        return x
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / QMAX[fmt]))
    s = torch.exp2(torch.where(top > QMAX[fmt] * torch.exp2(e), e + 1, torch.where(top <= QMAX[fmt] * torch.exp2(e - 1),
                                                                                 e - 1, e)).clamp_min(-126))
    y = x / s
    if fmt == "int8":
        return torch.round(y) * s
    # e4m3: steps of 2^-3 of the value's own power of two, at least 2^-9; ties to even
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step * s

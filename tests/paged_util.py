"""A paged cache and softmax attention over it in plain 64-bit steps, and the bounds
the kernels' results are held to.  Shares no code with the kernels."""
import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def quantise(x, dtype):
    """Codes (as float64 numbers) and scale of each row of x (float64 [..., D])."""
    top = x.abs().amax(-1, keepdim=True)
    s = torch.full_like(top, 2.0 ** -126)
    while bool((top > QMAX[dtype] * s).any()):  # doubling is exact: the smallest power of two that holds the row
        s = torch.where(top > QMAX[dtype] * s, 2 * s, s)
    y = x / s
    if dtype == torch.int8:
        return torch.round(y), s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, s


def attend(q, k, v, first, window, scale):
    """q [L, H, D] at positions first .. first + L - 1 over k, v [S, Hkv, D] (all float64).  Returns out,
    lse, a = sum softmax |v| (the size of the terms) and the largest |score| term sum sum |q_d k_d| scale."""
    L, H, D = q.shape
    S, Hkv = k.shape[:2]
    g = H // Hkv
    out, a = torch.zeros(L, H, D, dtype=torch.float64), torch.zeros(L, H, D, dtype=torch.float64)
    lse, big = torch.full((L, H), -math.inf, dtype=torch.float64), torch.zeros(L, H, dtype=torch.float64)
    for i in range(L):
        p = first + i
        lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, S)
        if hi <= lo:
            continue
        for h in range(H):
            kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
            s = kk @ q[i, h] * scale
            lse[i, h] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[i, h])
            out[i, h], a[i, h] = w @ vv, w @ vv.abs()
            big[i, h] = (kk.abs() @ q[i, h].abs()).max() * scale
    return out, lse, a, big


def bounds(out, lse, a, big, keys, D, dtype, weights_bf16):
    """Element-wise bounds on the kernels' error.

    A score is a sum of D products in fp32: off by at most (D + 2) 2^-23 of the sum of its terms' sizes
    (2^-23 a step: the tensor cores' accumulation may truncate); the exponential by 2^-21 (ex2.approx,
    its scaled argument |x| <= about 2^5 rounded at 2^-24) on top.  Numerator and denominator each carry
    that relative error and a sum of `keys` terms (keys 2^-23), so out is off by twice it of a = sum w |v|.
    On the tensor cores the weights are rounded to bf16: 2^-8 of each term.  The result is rounded
    once: half a step, 2^-8 (bf16) or 2^-24 (f32) of the value."""
    d = (D + 2) * 2.0 ** -23 * big + 2.0 ** -19
    rel = 2 * (d + keys * 2.0 ** -23)
    tol = (rel[..., None] + (2.0 ** -8 if weights_bf16 else 0.0)) * a
    tol = tol + torch.finfo(dtype).eps / 2 * (out.abs() + tol)
    return tol, d + keys * 2.0 ** -23 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


class Case:
    """Sequences of new tokens with a context, their cache in shuffled pages, all on the CPU."""

    def __init__(self, lens, ctx, H, Hkv, D, page, cache_dtype, dtype=torch.bfloat16, seed=0, layout="token",
                 extra_rows=0, garbage=True, packed=True):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.ctx, self.H, self.Hkv, self.D, self.page = lens, ctx, H, Hkv, D, page
        self.cache_dtype, self.dtype, self.packed = cache_dtype, dtype, packed
        N = len(lens)
        self.kv_len = [c + x for c, x in zip(ctx, lens)]
        need = [max(0, -(-s // page)) for s in self.kv_len]
        self.max_pages = max(1, max(need, default=1))
        self.n_pages = sum(need) + 2
        perm = torch.randperm(self.n_pages, generator=gen)
        self.table = torch.full((N, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for n in range(N):
            self.table[n, : need[n]] = perm[at : at + need[n]].to(torch.int32)
            at += need[n]
        T = sum(lens) + extra_rows
        self.q = torch.randn((T, H, D), generator=gen).mul_(1.5).to(dtype)
        self.k_rows, self.v_rows = [], []  # per sequence: float64 rows [kv_len, Hkv, D] as inputs
        for n in range(N):
            s = max(0, self.kv_len[n])
            self.k_rows.append(torch.randn((s, Hkv, D), generator=gen).to(dtype))
            self.v_rows.append(torch.randn((s, Hkv, D), generator=gen).to(dtype))
        shape = (self.n_pages, page, Hkv, D)
        self.layout, self.garbage = layout, garbage
        if cache_dtype == torch.bfloat16:
            self.blank = torch.full(shape, math.nan if garbage else 0.0, dtype=cache_dtype)
        else:
            b = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8) if garbage else torch.zeros(
                shape, dtype=torch.uint8)
            self.blank = b.view(cache_dtype)
        self.cu = torch.zeros(N + 1, dtype=torch.int32)
        self.cu[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int32), 0)

    def stored(self, n):
        """float64 keys and values that sequence n's cache stands for."""
        if self.cache_dtype == torch.bfloat16:
            return self.k_rows[n].to(torch.bfloat16).double(), self.v_rows[n].to(torch.bfloat16).double()
        got = []
        for x in (self.k_rows[n], self.v_rows[n]):
            if x.shape[0] == 0:
                got.append(x.double())
                continue
            c, s = quantise(x.double(), self.cache_dtype)
            got.append(c * s)
        return got

    def pages(self, device):
        """Caches holding every row but the new ones' when `new` is to be written, laid out as asked."""
        def lay(x):
            x = x.to(device)
            return x.transpose(1, 2).contiguous().transpose(1, 2) if self.layout == "head" else x
        k, v = lay(self.blank.clone()), lay(self.blank.clone())
        if self.cache_dtype == torch.bfloat16:
            return k, v, None, None
        ks, vs = (torch.full((self.n_pages, self.Hkv, self.page), math.nan, device=device) for _ in range(2))
        return k, v, ks, vs

    def fill(self, la, device, upto=None):
        """The cache after writing each sequence's rows [0, upto[n]) (default: all) with la_kv_write."""
        k, v, ks, vs = self.pages(device)
        ln = [max(0, s) for s in (self.kv_len if upto is None else upto)]
        if sum(ln):
            rows = [torch.cat([r[:x] for r, x in zip(rs, ln)])[None].to(device) for rs in (self.k_rows, self.v_rows)]
            cu = torch.zeros(len(ln) + 1, dtype=torch.int32, device=device)
            cu[1:] = torch.cumsum(torch.tensor(ln, dtype=torch.int32), 0).to(device)
            la.la_kv_write(rows[0], rows[1], k, v, self.table.to(device),
                           torch.tensor(ln, dtype=torch.int32, device=device), cu_seqlens=cu, k_scale=ks, v_scale=vs)
        return k, v, ks, vs

    def expect(self, window=0, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        T = self.q.shape[0]
        out = torch.zeros((T, self.H, self.D), dtype=torch.float64)
        a, lse = torch.zeros_like(out), torch.full((T, self.H), -math.inf, dtype=torch.float64)
        big = torch.zeros_like(lse)
        for n, x in enumerate(self.lens):
            t = int(self.cu[n])
            k, v = self.stored(n)
            out[t:t + x], lse[t:t + x], a[t:t + x], big[t:t + x] = attend(
                self.q[t:t + x].double(), k, v, self.kv_len[n] - x, window, scale)
        return out, lse, a, big

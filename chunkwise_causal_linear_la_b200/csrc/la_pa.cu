// la_pa.cu -- attention of new tokens over a paged cache on the sm_100a tensor
// cores (la_paged_attn for bf16, D = 64 or 128; tcgen05 + TMA + TMEM).
//
// The mathematics.  With s_j = scale q . k_j over the positions j a query sees,
//     o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  lse = m + ln sum_j e^(s_j - m)
// for any m.  Keys are taken in tiles of 128; m is a running maximum that only
// follows a tile's maximum when that is more than 8 (in powers of two) above it, so
// that the accumulator in tensor memory is rescaled rarely (weights stay below 2^8);
// two runs over disjoint keys join by their weights 2^(m_a - m), 2^(m_b - m).
//
// Rows.  The g query heads that share a cache head are rows of one product: row
// r of a 128-row tile is token r / g, head r % g of floor(128 / g) tokens.  An entry
// of work is one or two such tiles of a sequence and one cache head.  With two
// tiles the two softmax warpgroups take a tile each over the same keys; with one
// (single tokens, short chunks, the end of a prompt) they take the even and the odd
// key tiles of it, with an accumulator each, joined at the end.  Either way one
// group's exponentials run beside the other group's products.
//
// Work.  The key tiles of all entries and heads stand in one row; CTA c of G (one
// per SM) takes the c-th of G equal parts of it.  An entry cut by a border leaves
// partial results (unnormalised o, m, l) in the workspace, and the warp that brings
// the last part of a row joins them.  A small kernel lays out the row first:
// lengths are known to the device only.
//
// Roles (warps): 0 TMA producer (the tile's boxes on as many lanes; a box is a
// power-of-two piece of a page), 1 MMA issuer (one thread), 2-3 values fix-up
// (bf16), 4-7 and 8-11 softmax, 12-15 conversion (8-bit caches: codes become bf16
// operands, exact for power-of-two scales).
//   QK:  S[w] = Q K^T     (M = 128, N = 128 keys, K = D)        S in TMEM
//   PV:  O[w] += P V      (M = 128, N = D, K = 128 keys)        P (bf16) over S in TMEM
// Tensor-core instructions of one thread run in order, so PV(i) has read P before
// QK(i + 2) overwrites it, and the commit that announces S(i + 2) also says that O
// holds PV(i): the softmax group may rescale O then without another barrier.
//
// What a query does not see must not reach it even where it is an infinity or a NaN:
// scores are masked by selection, but 0 * inf in PV would be NaN.  Rows that no query
// of the entry sees are zeroed; in rows that some see, values that are not finite
// are taken out of the operand and added at the end for the queries that see them.
//
// Every wait is bounded (la_tc_sync.cuh): on a timeout the CTA records it, drains and
// returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_common.cuh"
#include "la_internal.h"
#include "la_kv.cuh"
#include "la_sm100.cuh"
#include "la_tc_sync.cuh"

namespace la {

__device__ unsigned int g_pa_error = 0;
__device__ unsigned int g_pa_where = 0;

namespace {

using namespace sm100;
using namespace tcsync;

constexpr int kTile = 128;  // keys of a tile, rows of a query tile

// One or two query tiles of a sequence: the same for every cache head.
struct alignas(16) Entry {
  int32_t seq, b, tok, ntok;     // sequence; batch row; first token (T axis) and tokens
  int32_t pos, kv_end, lo, cnt;  // position of the first token; positions in reach; first key tile, key tiles
};
struct alignas(16) CtaWork {
  int32_t head, entry, off;  // where this CTA's part starts: key tile `off` of an entry
  int32_t parts;             // CTAs that have a part (every CTA the same)
  int64_t count;             // key tiles
  int64_t total;             // key tiles of one head (every CTA the same)
};

struct PaArgs {
  const int32_t *cu, *kv_len, *table;
  int64_t T, max_pages, n_pages, n_seqs;
  int32_t page_size, box, g, tpt, Hkv, H, window;
  int32_t e_max, G;
  int64_t cap;  // max_pages * page_size
  float c;      // scale * log2(e)
  void *out;
  int64_t o_sb, o_st, o_sh;
  float *lse;
  const float *ks, *vs;  // 8-bit scales [n_pages][Hkv][page_size]
  const uint8_t *v;      // values (for what is not finite)
  int64_t s_page, s_tok, s_head;
  int32_t *seq_ent;    // [n_seqs + 1]
  Entry *ent;          // [e_max]
  int64_t *pre;        // [e_max + 1]
  CtaWork *work;       // [G]
  uint32_t *arrived;   // [G][2][4]
  float *po;           // [G][2][2][128][D]
  float2 *pml;         // [G][2][2][128]
};

// ------------------------------------------------------------------ schedule
constexpr int kPlanThreads = 1024;

// Exclusive prefix of v over the block, plus the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int64_t before = w ? warp_sums[w - 1] : 0;
  sum = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

__device__ __forceinline__ void seq_span(const PaArgs &a, int64_t n, int64_t &start, int64_t &len) {
  if (!a.cu) {
    start = 0;
    len = a.T;
    return;
  }
  start = min(max((int64_t)a.cu[n], (int64_t)0), a.T);
  len = min(max((int64_t)a.cu[n + 1], start), a.T) - start;
}

__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(const PaArgs a) {
  __shared__ int64_t ws[32];
  const int tid = threadIdx.x;
  const int64_t per = 2 * a.tpt;  // tokens of an entry
  int64_t sum, carry = 0;
  for (int64_t n0 = 0; n0 < a.n_seqs; n0 += kPlanThreads) {
    const int64_t n = n0 + tid;
    int64_t st = 0, len = 0;
    if (n < a.n_seqs) seq_span(a, n, st, len);
    const int64_t k = (len + per - 1) / per;
    const int64_t x = block_scan(k, ws, sum);
    if (n < a.n_seqs) a.seq_ent[n + 1] = (int32_t)min(carry + x + k, (int64_t)a.e_max);
    carry += sum;
  }
  if (tid == 0) a.seq_ent[0] = 0;
  __syncthreads();
  // overlapping sequences (an invalid cu_seqlens) could ask for more entries than there is room for
  const int E = (int)min(carry, (int64_t)a.e_max);
  carry = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int64_t cnt = 0;
    if (e < E) {
      int64_t lo = 0, hi = a.n_seqs;  // the last sequence whose first entry is <= e
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.seq_ent[mid] <= e) lo = mid; else hi = mid;
      }
      int64_t st, len;
      seq_span(a, lo, st, len);
      const int64_t t0 = (int64_t)(e - a.seq_ent[lo]) * per;
      const int64_t kv = max((int64_t)a.kv_len[lo], (int64_t)0);
      Entry x;
      x.seq = (int)lo;
      x.b = a.cu ? 0 : (int)lo;
      x.tok = (int)(st + t0);
      x.ntok = (int)max((int64_t)0, min(per, len - t0));
      const int64_t pos = kv - len + t0;
      x.pos = (int)max(pos, -((int64_t)1 << 31));
      x.kv_end = (int)min(kv, a.cap);
      const int64_t end = min(pos + x.ntok, (int64_t)x.kv_end);
      const int64_t beg = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
      x.lo = (int)(min(beg, max(end, (int64_t)0)) / kTile);
      cnt = end > beg ? (end + kTile - 1) / kTile - x.lo : 1;  // nothing seen: one tile, all masked
      x.cnt = (int)cnt;
      a.ent[e] = x;
    }
    const int64_t x = block_scan(cnt, ws, sum);
    if (e < E) a.pre[e] = carry + x;
    carry += sum;
  }
  __syncthreads();
  const int64_t P = carry, W = P * a.Hkv;
  const int64_t parts = min((int64_t)a.G, W);  // none of them empty: parts are counted by their numbers
  for (int c = tid; c < a.G; c += kPlanThreads) {
    const int64_t s0 = c < parts ? W * c / parts : 0, s1 = c < parts ? W * (c + 1) / parts : 0;
    CtaWork w;
    w.head = w.entry = w.off = 0;
    w.parts = (int)parts;
    w.count = s1 - s0;
    w.total = P;
    if (s1 > s0) {
      const int64_t r = s0 % P;
      int lo = 0, hi = E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.pre[mid] <= r) lo = mid; else hi = mid;
      }
      w.head = (int)(s0 / P);
      w.entry = lo;
      w.off = (int)(r - a.pre[lo]);
    }
    a.work[c] = w;
    for (int i = 0; i < 8; ++i) a.arrived[8 * c + i] = 0;
  }
  if (tid == 0) a.seq_ent[0] = E;  // the main kernel wraps to the next head after entry E - 1
}

// ------------------------------------------------------------------ main kernel
template <int D, int FMT>
struct PaCfg {
  static constexpr bool Q8 = FMT != LA_KV_BF16;
  static constexpr int THREADS = Q8 ? 512 : 384;
  static constexpr int SLABS = D / 64;               // 64-column slabs of a bf16 tile
  static constexpr int SLAB = kTile * 128;           // bytes of one
  static constexpr int TILE = SLABS * SLAB;          // a bf16 operand tile
  static constexpr int RAW = kTile * D;              // a tile of codes
  static constexpr int NS = Q8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);  // operand slots (keys and values in turn)
  static constexpr int NR = Q8 ? (D == 128 ? 3 : 8) : 0;                    // stages of codes
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_OP = 2 * TILE;
  static constexpr int OFF_RAW = OFF_OP + NS * TILE;
  static constexpr int OFF_SC = OFF_RAW + NR * RAW;  // scales of a stage, 128 floats
  static constexpr int OFF_ML = OFF_SC + NR * kTile * 4;
  static constexpr int OFF_BAR = OFF_ML + kTile * 8;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_RFULL = 2 * NS, B_REMPTY = B_RFULL + NR, B_QFULL = B_REMPTY + NR,
                       B_QEMPTY = B_QFULL + 1, B_SFULL = B_QFULL + 2, B_PFULL = B_QFULL + 4, B_OFULL = B_QFULL + 6,
                       B_OEMPTY = B_QFULL + 8, B_MERGE = B_QFULL + 10, B_DRAIN = B_QFULL + 11,
                       B_READY = B_QFULL + 12,  // bf16, per slot: fixed up
                       NBAR = B_READY + (Q8 ? 0 : NS);
  // per item (mod 16) and fix-up or conversion warp: values that are not finite were taken out.  (A flag left
  // from 16 items before only costs a look for such values.)
  static constexpr int OFF_BAD = OFF_BAR + (NBAR * 8 + 15) / 16 * 16;
  static constexpr int OFF_MISC = OFF_BAD + 16 * 16;
  static constexpr int SMEM_USED = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = SMEM_USED + 1024;
  // tensor memory columns
  static constexpr int T_S = 0, T_O = 2 * kTile, T_COLS = 512;
  static_assert(T_O + 2 * D <= 512, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  // register split (per thread; shares add up to the launch's)
  static constexpr int R_AUX = Q8 ? 56 : 104, R_SOFT = Q8 ? 192 : 200, R_CONV = 72;
};

// A piece of an entry: `n` key tiles from tile t0 on, of one cache head.
struct Item {
  Entry e;
  int head, entry, t0, n;
  bool first, last;  // the entry's first / last key tile is in this piece
};

// Walks a CTA's part of the row of work.  Every role runs it by itself.
struct Walk {
  int head, entry, off, E;
  int64_t left;
  __device__ __forceinline__ Walk(const PaArgs &a) {
    const CtaWork w = a.work[blockIdx.x];
    head = w.head;
    entry = w.entry;
    off = w.off;
    left = w.count;
    E = a.seq_ent[0];
  }
  __device__ __forceinline__ bool next(const PaArgs &a, Item &it) {
    if (left <= 0) return false;
    it.e = a.ent[entry];
    it.head = head;
    it.entry = entry;
    it.t0 = it.e.lo + off;
    it.n = (int)min((int64_t)(it.e.cnt - off), left);
    it.first = off == 0;
    it.last = off + it.n == it.e.cnt;
    left -= it.n;
    off = 0;
    if (++entry == E) {
      entry = 0;
      ++head;
    }
    return true;
  }
};

// Positions that token `tk` of an entry sees: [lo, hi).
__device__ __forceinline__ void sees(const PaArgs &a, const Entry &e, int tk, int64_t &lo, int64_t &hi) {
  const int64_t p = (int64_t)e.pos + tk;
  hi = min(p + 1, (int64_t)e.kv_end);
  lo = a.window > 0 ? max((int64_t)0, p - a.window + 1) : 0;
}

// Of the keys of tile t: all tokens of the entry see those in [b, c); some those in
// [a, d); none the rest (tile-relative, clamped).
struct Reach {
  int a, b, c, d;
};
__device__ __forceinline__ Reach reach(const PaArgs &a, const Entry &e, int t) {
  int64_t lo0, hi0, lo1, hi1;
  sees(a, e, 0, lo0, hi0);
  sees(a, e, max(e.ntok, 1) - 1, lo1, hi1);
  const int64_t ts = (int64_t)t * kTile;
  Reach r;
  r.a = (int)min(max(lo0 - ts, (int64_t)0), (int64_t)kTile);
  r.b = (int)min(max(lo1 - ts, (int64_t)0), (int64_t)kTile);
  r.c = (int)min(max(hi0 - ts, (int64_t)0), (int64_t)kTile);
  r.d = (int)min(max(hi1 - ts, (int64_t)0), (int64_t)kTile);
  return r;
}
__device__ __forceinline__ bool partly(const Reach &r) { return r.b > 0 || r.c < kTile; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two codes (byte positions picked by SEL) as bf16x2, times s2.
//   e4m3: exponent and mantissa bits moved to bf16's places, value 2^-120 of the code's; the product with
//         2^120 is exact (bf16 keeps subnormals), and so is the one with a power-of-two scale.
//   int8: with the low 7 bits L and the sign bit S, (128 + L) - (128 + 128 S) by bit patterns of bf16.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(uint32_t w, int hi, __nv_bfloat162 s2) {
  uint32_t v;
  __nv_bfloat162 r;
  if (FMT == LA_KV_E4M3) {
    const uint32_t x = __byte_perm(w, 0, hi ? 0x3424 : 0x1404);
    v = ((x >> 4) & 0x07F007F0u) | (x & 0x80008000u);
    const uint32_t big = 0x7B807B80u;
    r = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&big));
  } else {
    const uint32_t x = __byte_perm(w, 0, hi ? 0x4342 : 0x4140);
    v = (x & 0x007F007Fu) | 0x43004300u;
    const uint32_t b = (x & 0x00800080u) | 0x43004300u;
    r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  }
  r = __hmul2(r, s2);
  return *reinterpret_cast<uint32_t *>(&r);
}

__device__ __forceinline__ bool finite_f(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ uint32_t keep_finite(uint32_t w) {  // bf16x2
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

template <int D, int FMT>
__global__ void __launch_bounds__((PaCfg<D, FMT>::THREADS), 1)
pa_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
          const __grid_constant__ CUtensorMap tm_v, const PaArgs a) {
  using G = PaCfg<D, FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::OFF_BAR);
  float *sc = reinterpret_cast<float *>(sm + G::OFF_SC);
  float2 *ml = reinterpret_cast<float2 *>(sm + G::OFF_ML);
  volatile int *bad = reinterpret_cast<volatile int *>(sm + G::OFF_BAD);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + G::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + G::OFF_MISC + 4);
  const Sync sy{bars, abort_flag, &g_pa_error, &g_pa_where};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < G::NBAR; ++i) {
      uint32_t cnt = 1;
      if (G::Q8 && i < G::NS) cnt = 4;                                  // FULL: conversion warps
      if (!G::Q8 && i >= G::B_EMPTY && i < G::B_EMPTY + G::NS) cnt = 3;  // products done, seen by the fix-up warps
      if (i >= G::B_REMPTY && i < G::B_REMPTY + G::NR) cnt = 4;         // codes read
      if (i >= G::B_PFULL && i < G::B_PFULL + 2) cnt = 4;               // softmax warps
      if (i >= G::B_OEMPTY && i < G::B_OEMPTY + 2) cnt = 4;
      if (i == G::B_MERGE) cnt = 4;
      if (i >= G::B_READY) cnt = 2;  // fix-up warps
      mbar_init(bars + i, cnt);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) tmem_alloc(tmem_slot, G::T_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  auto op_slot = [&](int s) { return sm + G::OFF_OP + s * G::TILE; };
  auto raw_stage = [&](int s) { return sm + G::OFF_RAW + s * G::RAW; };

  Walk walk(a);
  Item it;
  if (warp < 4) {
    reg_dealloc<G::R_AUX>();
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      const int nb = kTile / a.box;
      const uint32_t q_bytes = (uint32_t)(a.g * a.tpt) * 128u * G::SLABS;
      uint32_t seq = 0, items = 0;  // operand tiles and items started
      bool ok = true;
      while (ok && walk.next(a, it)) {
        const bool two = it.e.ntok > a.tpt;
        // page of this lane's box in tile t
        auto page_at = [&](int t, int &slot) -> int {
          const int64_t p = (int64_t)t * kTile + lane * a.box;
          slot = 0;
          if (lane >= nb || p >= it.e.kv_end) return -1;
          const uint32_t idx = (uint32_t)p / (uint32_t)a.page_size;
          slot = (int)((uint32_t)p - idx * (uint32_t)a.page_size);
          const int pg = a.table[(int64_t)it.e.seq * a.max_pages + idx];
          return pg >= 0 && pg < a.n_pages ? pg : -1;
        };
        int slot, nslot = 0;
        int pg = page_at(it.t0, slot), npg = -1;
        for (int i = 0; i < it.n && ok; ++i) {
          if (i + 1 < it.n) npg = page_at(it.t0 + i + 1, nslot);
          // a missing page is read past the end of the page axis: zeros
          const int pc = pg >= 0 ? pg : (int)a.n_pages;
#pragma unroll
          for (int kvi = 0; kvi < 2; ++kvi, ++seq) {
            const CUtensorMap *tm = kvi ? &tm_v : &tm_k;
            if (!G::Q8) {
              const int s = seq % G::NS;
              if (!(ok = wait_bar_warp(sy, G::B_EMPTY + s, ((seq / G::NS) & 1) ^ 1, it.t0 + i))) break;
              if (lane == 0) mbar_arrive_expect_tx(bars + G::B_FULL + s, G::TILE);
              __syncwarp();
              if (lane < nb) {
#pragma unroll
                for (int sl = 0; sl < G::SLABS; ++sl)
                  tma_load_4d(op_slot(s) + sl * G::SLAB + lane * a.box * 128, tm, bars + G::B_FULL + s, sl * 64,
                              it.head, slot, pc);
              }
            } else {
              const int s = seq % (G::NR > 0 ? G::NR : 1);
              if (!(ok = wait_bar_warp(sy, G::B_REMPTY + s, ((seq / (G::NR > 0 ? G::NR : 1)) & 1) ^ 1, it.t0 + i))) break;
              const uint32_t have = __popc(__ballot_sync(0xffffffffu, pg >= 0));
              if (lane < nb && pg < 0)
                for (int r = 0; r < a.box; ++r) sc[s * kTile + lane * a.box + r] = 0.f;
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(bars + G::B_RFULL + s, G::RAW + have * a.box * 4);
              __syncwarp();
              if (lane < nb) {
                tma_load_4d(raw_stage(s) + lane * a.box * D, tm, bars + G::B_RFULL + s, 0, it.head, slot, pc);
                if (pg >= 0)
                  bulk_load(sc + s * kTile + lane * a.box,
                            (kvi ? a.vs : a.ks) + ((int64_t)pg * a.Hkv + it.head) * a.page_size + slot, a.box * 4,
                            bars + G::B_RFULL + s);
              }
            }
            if (i == 0 && kvi == 0) {  // the item's queries, after its first keys are on their way
              if (!(ok = wait_bar_warp(sy, G::B_QEMPTY, (items & 1) ^ 1, it.t0))) {
                ++seq;
                break;
              }
              if (lane == 0) {
                mbar_arrive_expect_tx(bars + G::B_QFULL, two ? 2 * q_bytes : q_bytes);
                for (int w = 0; w < (two ? 2 : 1); ++w)
                  for (int sl = 0; sl < G::SLABS; ++sl)
                    tma_load_4d(sm + G::OFF_Q + w * G::TILE + sl * G::SLAB, &tm_q, bars + G::B_QFULL, sl * 64,
                                it.head * a.g, it.e.tok + w * a.tpt, it.e.b);
              }
              ++items;
            }
          }
          pg = npg;
          slot = nslot;
        }
      }
      if (*abort_flag) {  // let every copy under way land before the CTA ends
        if (lane == 0) {
          constexpr uint32_t N = G::Q8 ? (G::NR > 0 ? G::NR : 1) : G::NS;
          const int b = G::Q8 ? G::B_RFULL : G::B_FULL;
          for (uint32_t s = seq > N ? seq - N : 0; s < seq; ++s) drain_bar(sy, b + s % N, (s / N) & 1);
          if (items) drain_bar(sy, G::B_QFULL, (items - 1) & 1);
        }
        __syncwarp();
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t ID_QK = idesc_bf16_f32(kTile, kTile, 0, 0);
        constexpr uint32_t ID_PV = idesc_bf16_f32(kTile, D, 0, 1);
        const uint64_t dq0 = smem_desc_sw128(smem_u32(sm + G::OFF_Q), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(op_slot(0)), 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(op_slot(0)), G::SLAB, 1024);
        uint32_t seq = 0, items = 0, used[2] = {0, 0}, pcnt[2] = {0, 0};
        bool ok = true;
        while (ok && walk.next(a, it)) {
          const bool two = it.e.ntok > a.tpt;
          const int ns = two ? 2 * it.n : it.n;
          auto qk = [&](int s) -> bool {
            const int w = s & 1, i = two ? s >> 1 : s;
            const uint32_t k = seq + 2 * i, sl = k % G::NS;
            if (!two || w == 0)
              if (!wait_bar(sy, G::B_FULL + sl, (k / G::NS) & 1, it.t0 + i)) return false;
            tc_fence_after();
            const uint64_t dq = dq0 + (uint64_t)((two ? w : 0) * (G::TILE >> 4));
            const uint64_t dk = dk0 + (uint64_t)(sl * (G::TILE >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * G::SLAB + (kk & 3) * 32) >> 4;
              umma_bf16(tbase + G::T_S + w * kTile, dq + off, dk + off, ID_QK, kk > 0);
            }
            umma_commit(bars + G::B_SFULL + w);
            if (!two || w == 1) umma_commit(bars + G::B_EMPTY + sl);
            if (s == ns - 1) umma_commit(bars + G::B_QEMPTY);
            return true;
          };
          ok = wait_bar(sy, G::B_QFULL, items & 1, it.t0);
          ++items;
          ok = ok && qk(0) && (ns < 2 || qk(1));
          for (int s = 0; s < ns && ok; ++s) {
            const int w = s & 1, i = two ? s >> 1 : s;
            const uint32_t k = seq + 2 * i + 1, sl = k % G::NS;
            if (!two || w == 0) {
              const bool fix = !G::Q8 && partly(reach(a, it.e, it.t0 + i));
              if (!(ok = wait_bar(sy, (fix ? G::B_READY : G::B_FULL) + sl, (k / G::NS) & 1, it.t0 + i))) break;
            }
            if (!(ok = wait_bar(sy, G::B_PFULL + w, pcnt[w] & 1, it.t0 + i))) break;
            ++pcnt[w];
            const bool fresh = s < 2;  // the group's first product of the item
            if (fresh) {
              if (used[w] && !(ok = wait_bar(sy, G::B_OEMPTY + w, (used[w] - 1) & 1, it.t0 + i))) break;
              ++used[w];
            }
            tc_fence_after();
            const uint64_t dv = dv0 + (uint64_t)(sl * (G::TILE >> 4));
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_bf16_ts(tbase + G::T_O + w * D, tbase + G::T_S + w * kTile + kk * 8, dv + ((kk * 2048) >> 4), ID_PV,
                           (!fresh || kk > 0) ? 1u : 0u);
            if (!two || w == 1) umma_commit(bars + G::B_EMPTY + sl);
            if (s >= ns - 2) umma_commit(bars + G::B_OFULL + w);  // the group's last product
            if (s + 2 < ns) ok = qk(s + 2);
          }
          seq += 2 * it.n;
        }
        umma_commit(bars + G::B_DRAIN);  // products under way end before tensor memory is freed
        drain_bar(sy, G::B_DRAIN, 0);
      }
      __syncwarp();
    } else if (!G::Q8) {
      // -------------------------------------------------------------- values fix-up
      // These warps see every tile and take part in its release: a slot is not filled again before they have
      // noted its phase, so they cannot fall behind the ring or run ahead of it.
      uint32_t seq = 0, items = 0;
      bool ok = true;
      const int t = tid - 64;
      while (ok && walk.next(a, it)) {
        if (lane == 0) bad[(items & 15) * 4 + warp - 2] = 0;
        __syncwarp();
        for (int i = 0; i < 2 * it.n; ++i, ++seq) {
          const uint32_t sl = seq % G::NS;
          if (!(ok = wait_bar_warp(sy, G::B_FULL + sl, (seq / G::NS) & 1, it.t0 + (i >> 1)))) break;
          Reach r;
          if ((i & 1) && partly(r = reach(a, it.e, it.t0 + (i >> 1)))) {
            uint8_t *v = op_slot(sl);
            int found = 0;
            // 16-byte pieces of the rows that not every token sees
            for (int x = t; x < kTile * 8 * G::SLABS; x += 64) {
              const int row = (x >> 3) & (kTile - 1);
              if (row >= r.b && row < r.c) continue;
              uint4 *p = reinterpret_cast<uint4 *>(v) + x;
              if (row < r.a || row >= r.d) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 u = *p;
                const uint4 f = make_uint4(keep_finite(u.x), keep_finite(u.y), keep_finite(u.z), keep_finite(u.w));
                if (f.x != u.x || f.y != u.y || f.z != u.z || f.w != u.w) {
                  *p = f;
                  found = 1;
                }
              }
            }
            if (found) bad[(items & 15) * 4 + warp - 2] = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive(bars + G::B_READY + sl);
            mbar_arrive(bars + G::B_EMPTY + sl);
          }
        }
        ++items;
      }
    }
  } else if (warp < 12) {
    reg_alloc<G::R_SOFT>();
    // ---------------------------------------------------------------- softmax groups
    const int w = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t ts_addr = tbase + G::T_S + w * kTile + lane_off;
    const uint32_t to_addr = tbase + G::T_O + lane_off;
    const float c = a.c, thr = 8.f / c;
    uint32_t scnt = 0, ocnt[2] = {0, 0}, mcnt = 0, items = 0;
    bool ok = true;
    while (ok && walk.next(a, it)) {
      const bool two = it.e.ntok > a.tpt;
      const int tk = (two ? w * a.tpt : 0) + r / a.g;
      const bool valid = r < a.g * a.tpt && tk < it.e.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      int64_t lo, hi;
      sees(a, it.e, tk, lo, hi);
      if (!valid) lo = hi = 0;
      float m = -INFINITY, l = 0.f;
      for (int i = two ? 0 : w; i < it.n; i += two ? 1 : 2) {
        if (!(ok = wait_bar_warp(sy, G::B_SFULL + w, scnt & 1, it.t0 + i))) break;
        ++scnt;
        if (active) {
          tc_fence_after();
          uint32_t s[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(ts_addr + 32 * q, s[q]);
          tmem_wait_ld();
          const int64_t ts = (int64_t)(it.t0 + i) * kTile;
          const int va = (int)min(max(lo - ts, (int64_t)0), (int64_t)kTile);
          const int vb = (int)min(max(hi - ts, (int64_t)0), (int64_t)kTile);
          if (__any_sync(0xffffffffu, va > 0 || vb < kTile)) {
            const uint32_t width = (uint32_t)max(vb - va, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if ((uint32_t)(32 * q + j - va) >= width) s[q][j] = 0xFF800000u;
          }
          float mx4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mx4[q] = __uint_as_float(s[q][0]);
#pragma unroll
            for (int j = 1; j < 32; ++j) mx4[q] = fmaxf(mx4[q], __uint_as_float(s[q][j]));
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          if (m == -INFINITY) m = mx;  // nothing summed yet: O's row is not there, or zero
          const bool up = mx > m + thr;
          if (__any_sync(0xffffffffu, up)) {
            const float f = up ? ex2((m - mx) * c) : 1.f;
            if (up) m = mx;
            l *= f;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to_addr + w * D + 32 * q, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_32x32b_x32(to_addr + w * D + 32 * q, o);
            }
          }
          const float mc = m == -INFINITY ? 0.f : m * c;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int q = 2 * hf + (j >> 4), k = 2 * (j & 15);
              const float x = ex2(fmaf(__uint_as_float(s[q][k]), c, -mc));
              const float y = ex2(fmaf(__uint_as_float(s[q][k + 1]), c, -mc));
              l4[j & 1] += x;
              l4[2 + (j & 1)] += y;
              p[j] = pack2(x, y);
            }
            tmem_st_32x32b_x32(ts_addr + 32 * hf, p);
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + G::B_PFULL + w);
      }
      if (!ok) break;
      // ------------------------------------------------------------------ epilogue
      const float mc = m * c;
      const bool mine = two || w == 0;
      const int n1 = two ? it.n : it.n / 2;          // steps of group 1
      if (!mine) {
        if (n1 > 0) {  // O[1] complete: the previous item's statistics have been read
          if (!(ok = wait_bar_warp(sy, G::B_OFULL + 1, ocnt[1] & 1, it.t0))) break;
          ++ocnt[1];
          ml[r] = make_float2(mc, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + G::B_MERGE);
        }
        ++items;
        continue;
      }
      const bool join = !two && n1 > 0;
      if (!(ok = wait_bar_warp(sy, G::B_OFULL + w, ocnt[w] & 1, it.t0))) break;
      ++ocnt[w];
      float M = mc, L = l, w0 = 1.f, w1 = 0.f;
      if (join) {
        if (!(ok = wait_bar_warp(sy, G::B_OFULL + 1, ocnt[1] & 1, it.t0))) break;
        if (!(ok = wait_bar_warp(sy, G::B_MERGE, mcnt & 1, it.t0))) break;
        ++mcnt;
        const float2 o = ml[r];
        M = fmaxf(mc, o.x);
        const float base = M == -INFINITY ? 0.f : M;
        w0 = ex2(mc - base);
        w1 = ex2(o.x - base);
        L = w0 * l + w1 * o.y;
      }
      if (w == 0 && n1 > 0) ++ocnt[1];  // group 0 follows group 1's phases
      tc_fence_after();
      const bool whole = it.first && it.last;
      int any_bad = 0;
#pragma unroll
      for (int x = 0; x < (G::Q8 ? 4 : 2); ++x) any_bad |= bad[(items & 15) * 4 + x];
      const int64_t tok = it.e.tok + tk;
      const int head = it.head * a.g + r % a.g;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int tile = two ? w : 0;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (it.first ? 1 : 0);
      float *po = a.po + ((slot * 2 + tile) * kTile + r) * D;
      if (active) {
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(to_addr + w * D + 32 * q, x);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(x[j]);
          if (join) {
            tmem_ld_32x32b_x32(to_addr + D + 32 * q, x);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = w0 * o[j] + w1 * __uint_as_float(x[j]);
          }
          if (any_bad) {  // values that are not finite, for the queries that see them
            for (int t = it.t0; t < it.t0 + it.n; ++t) {
              const Reach rc = reach(a, it.e, t);
              if (!partly(rc)) continue;
              for (int j = rc.a; j < rc.d; ++j) {
                if (j >= rc.b && j < rc.c) continue;
                const int64_t p = (int64_t)t * kTile + j;
                const int64_t idx = p / a.page_size;
                const int pg = a.table[(int64_t)it.e.seq * a.max_pages + idx];
                if (pg < 0 || pg >= a.n_pages || p < lo || p >= hi) continue;
                const int sl = (int)(p % a.page_size);
                const int64_t off = (int64_t)pg * a.s_page + (int64_t)sl * a.s_tok + (int64_t)it.head * a.s_head + 32 * q;
                const float vs = G::Q8 ? a.vs[((int64_t)pg * a.Hkv + it.head) * a.page_size + sl] : 0.f;
                if (G::Q8 && finite_f(vs)) continue;
#pragma unroll
                for (int u = 0; u < 32; ++u) {
                  float v = vs * 0.f;  // a scale that is not finite: NaN
                  if (!G::Q8) v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.v)[off + u]);
                  if (!finite_f(v)) o[u] += v;
                }
              }
            }
          }
          if (valid) {
            if (whole) {
              uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + (int64_t)it.e.b * a.o_sb +
                                                     tok * a.o_st + (int64_t)head * a.o_sh + 32 * q);
#pragma unroll
              for (int u = 0; u < 4; ++u)
                dst[u] = make_uint4(pack2(o[8 * u] * inv, o[8 * u + 1] * inv), pack2(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                    pack2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                    pack2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
            } else {
              float4 *dst = reinterpret_cast<float4 *>(po + 32 * q);
#pragma unroll
              for (int u = 0; u < 8; ++u) dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + G::B_OEMPTY + w);
        if (join) mbar_arrive(bars + G::B_OEMPTY + 1);
      }
      if (valid && whole && a.lse)
        a.lse[((int64_t)it.e.b * a.T + tok) * a.H + head] = (M + log2f(L)) * 0.6931471805599453f;
      if (active && !whole) {
        // leave the part, and join the entry's parts if this warp's rows are complete with it
        if (valid) a.pml[(slot * 2 + tile) * kTile + r] = make_float2(M, L);
        // tile s of the row of W tiles belongs to the last CTA c with floor(W c / parts) <= s
        const int64_t total = a.work[blockIdx.x].total, W = total * a.Hkv, parts = a.work[blockIdx.x].parts;
        const int64_t s0 = it.head * total + a.pre[it.entry], s1 = s0 + it.e.cnt - 1;
        const int c0 = (int)(((s0 + 1) * parts - 1) / W), c1 = (int)(((s1 + 1) * parts - 1) / W);
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) before = atomicAdd(a.arrived + (c0 * 2 + tile) * 4 + quad, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == (uint32_t)(c1 - c0)) {
          __threadfence();
          for (int rr = 0; rr < 32; ++rr) {
            const int row = quad * 32 + rr;
            if (!__shfl_sync(0xffffffffu, (int)valid, rr)) continue;
            auto part = [&](int cc) -> int64_t { return ((2 * (int64_t)cc + (cc == c0 ? 1 : 0)) * 2 + tile) * kTile + row; };
            float mm = -INFINITY;
            for (int cc = c0 + lane; cc <= c1; cc += 32) mm = fmaxf(mm, __ldcg(&a.pml[part(cc)]).x);
#pragma unroll
            for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
            const float base = mm == -INFINITY ? 0.f : mm;
            float acc[D / 32], ls = 0.f;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) acc[u] = 0.f;
#pragma unroll 4
            for (int cc = c0; cc <= c1; ++cc) {
              const float2 x = __ldcg(&a.pml[part(cc)]);
              const float wt = ex2(x.x - base);
              ls = fmaf(wt, x.y, ls);
              const float *src = a.po + part(cc) * D + lane;
#pragma unroll
              for (int u = 0; u < D / 32; ++u) acc[u] = fmaf(wt, __ldcg(src + 32 * u), acc[u]);
            }
            const float iv = ls == 0.f ? 0.f : 1.f / ls;
            const int64_t rt = it.e.tok + (two ? w * a.tpt : 0) + row / a.g;
            const int rh = it.head * a.g + row % a.g;
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(a.out) + (int64_t)it.e.b * a.o_sb + rt * a.o_st +
                                 (int64_t)rh * a.o_sh + lane;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) dst[32 * u] = __float2bfloat16_rn(acc[u] * iv);
            if (a.lse && lane == 0)
              a.lse[((int64_t)it.e.b * a.T + rt) * a.H + rh] = (mm + log2f(ls)) * 0.6931471805599453f;
          }
        }
      }
      ++items;
    }
  } else if (G::Q8) {
    reg_dealloc<G::R_CONV>();
    // ---------------------------------------------------------------- conversion
    const int t = tid - 384;
    constexpr int NRr = G::NR > 0 ? G::NR : 1;
    // D = 128 (codes under the 128-byte swizzle): eight lanes take half a row of rows a and a ^ 5 of an 8-row
    // group, which spreads both their 16-byte reads and their 16-byte writes over all banks.  D = 64 (plain rows of
    // 64 bytes): eight lanes take two rows.
    const int q4 = t & 3, slab = D == 128 ? (t >> 3) & 1 : 0;
    const int pair = (t >> 2) & 1;
    const int r8 = D == 128 ? (pair ? ((t >> 4) & 3) ^ 5 : (t >> 4) & 3) : ((t >> 3) & 3) * 2 + pair;
    constexpr int GROUPS = D == 128 ? 2 : 4;  // 8-row groups the 128 threads cover at once
    const int grp = D == 128 ? t >> 6 : t >> 5;
    uint32_t seq = 0, items = 0;
    bool ok = true;
    while (ok && walk.next(a, it)) {
      if (lane == 0) bad[(items & 15) * 4 + warp - 12] = 0;
      __syncwarp();
      for (int i = 0; i < it.n && ok; ++i) {
        const Reach rc = reach(a, it.e, it.t0 + i);
        for (int kvi = 0; kvi < 2; ++kvi, ++seq) {
          const int rs = seq % NRr, os = seq % G::NS;
          if (!(ok = wait_bar_warp(sy, G::B_RFULL + rs, (seq / NRr) & 1, it.t0 + i))) break;
          if (!(ok = wait_bar_warp(sy, G::B_EMPTY + os, ((seq / G::NS) & 1) ^ 1, it.t0 + i))) break;
          const uint8_t *src = raw_stage(rs);
          uint8_t *dst = op_slot(os) + slab * G::SLAB;
          int found = 0;
#pragma unroll
          for (int k = 0; k < 16 / GROUPS; ++k) {
            const int row = (k * GROUPS + grp) * 8 + r8;
            float s = sc[rs * kTile + row];
            if (row < rc.a || row >= rc.d) s = 0.f;  // seen by none (codes are finite by construction)
            if (kvi && !finite_f(s) && (row < rc.b || row >= rc.c)) {
              s = 0.f;
              found = 1;
            }
            const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
            const int cc = D == 128 ? ((slab * 4 + q4) ^ r8) : q4;
            const uint4 u = *reinterpret_cast<const uint4 *>(src + row * D + cc * 16);
            uint4 o0, o1;
            o0.x = codes2<FMT>(u.x, 0, s2), o0.y = codes2<FMT>(u.x, 1, s2);
            o0.z = codes2<FMT>(u.y, 0, s2), o0.w = codes2<FMT>(u.y, 1, s2);
            o1.x = codes2<FMT>(u.z, 0, s2), o1.y = codes2<FMT>(u.z, 1, s2);
            o1.z = codes2<FMT>(u.w, 0, s2), o1.w = codes2<FMT>(u.w, 1, s2);
            *reinterpret_cast<uint4 *>(dst + row * 128 + (((2 * q4) ^ r8) << 4)) = o0;
            *reinterpret_cast<uint4 *>(dst + row * 128 + (((2 * q4 + 1) ^ r8) << 4)) = o1;
          }
          if (found) bad[(items & 15) * 4 + warp - 12] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bars + G::B_FULL + os);
            mbar_arrive(bars + G::B_REMPTY + rs);
          }
        }
      }
      ++items;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tbase, G::T_COLS);
  }
}

// ------------------------------------------------------------------ host side
int tokens_per_tile(int g) { return kTile / g; }

int box_rows(int64_t page_size) {  // largest power of two that divides the page, up to a tile
  int b = 1;
  while (b < kTile && page_size % (2 * b) == 0) b *= 2;
  return b;
}

int64_t max_entries(int64_t B, int64_t T, int64_t n_seqs, bool packed, int g) {
  const int64_t per = 2 * tokens_per_tile(g);
  return packed ? T / per + n_seqs : B * ((T + per - 1) / per);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  size_t seq_ent, ent, pre, work, arrived, po, pml, bytes;
};
Plan plan(int64_t e_max, int64_t n_seqs, int D, int G) {
  Plan p;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += up256(n);
    return r;
  };
  p.seq_ent = take((size_t)(n_seqs + 1) * 4);
  p.ent = take((size_t)e_max * sizeof(Entry));
  p.pre = take((size_t)e_max * 8);
  p.work = take((size_t)G * sizeof(CtaWork));
  p.arrived = take((size_t)G * 32);
  p.pml = take((size_t)G * 4 * kTile * 8);
  p.po = take((size_t)G * 4 * kTile * D * 4);
  p.bytes = at;
  return p;
}

template <int D, int FMT>
cudaError_t launch_one(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const PaArgs &a,
                       cudaStream_t stream) {
  using G = PaCfg<D, FMT>;
  auto kern = pa_kernel<D, FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  pa_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  kern<<<a.G, G::THREADS, G::SMEM_BYTES, stream>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

bool pa_tc_shape(int64_t H, int64_t D, int64_t H_kv, int64_t page_size) {
  return (D == 64 || D == 128) && page_size % 8 == 0 && H / H_kv <= kTile;
}

bool pa_tc_supported(const PagedArgs &a) {
  // TMA steps along the axes of q: a zero stride (a broadcast) is not given to it
  return a.dtype == LA_BF16 && a.c.n_pages > 0 && pa_tc_shape(a.H, a.c.D, a.c.H, a.c.page_size) &&
         !((a.B > 1 && a.q.sb == 0) || (a.T > 1 && a.q.st == 0) || (a.H > 1 && a.q.sh == 0));
}

// (size_t)-1 where the problem is too large for 32-bit entry numbers.
size_t pa_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t D, int64_t n_seqs, bool packed, int64_t H_kv, int G) {
  const int64_t e = max_entries(B, T, n_seqs, packed, (int)(H / H_kv));
  if (e > 0x7FFFFFF0) return (size_t)-1;
  return plan(e, n_seqs, (int)D, G).bytes;
}

cudaError_t launch_paged_tc(const PagedArgs &a, int G, void *workspace, cudaStream_t stream, const char **why) {
  const int D = a.c.D, g = a.H / a.c.H;
  const bool q8 = a.c.format != LA_KV_BF16;
  PaArgs p;
  p.cu = a.cu_seqlens;
  p.kv_len = a.kv_len;
  p.table = a.c.table;
  p.T = a.T;
  p.max_pages = a.c.max_pages;
  p.n_pages = a.c.n_pages;
  p.n_seqs = a.n_seqs;
  p.page_size = a.c.page_size;
  p.box = box_rows(a.c.page_size);
  p.g = g;
  p.tpt = tokens_per_tile(g);
  p.Hkv = a.c.H;
  p.H = a.H;
  p.window = a.window;
  p.e_max = (int)max_entries(a.B, a.T, a.n_seqs, a.cu_seqlens != nullptr, g);
  p.G = G;
  p.cap = a.c.max_pages * (int64_t)a.c.page_size;
  p.c = a.scale * 1.4426950408889634f;
  p.out = a.out;
  p.o_sb = a.o_sb;
  p.o_st = a.o_st;
  p.o_sh = a.o_sh;
  p.lse = a.lse;
  p.ks = a.c.ks;
  p.vs = a.c.vs;
  p.v = a.c.v;
  p.s_page = a.c.s_page;
  p.s_tok = a.c.s_tok;
  p.s_head = a.c.s_head;
  const Plan pl = plan(p.e_max, a.n_seqs, D, G);
  uint8_t *ws = (uint8_t *)workspace;
  p.seq_ent = (int32_t *)(ws + pl.seq_ent);
  p.ent = (Entry *)(ws + pl.ent);
  p.pre = (int64_t *)(ws + pl.pre);
  p.work = (CtaWork *)(ws + pl.work);
  p.arrived = (uint32_t *)(ws + pl.arrived);
  p.pml = (float2 *)(ws + pl.pml);
  p.po = (float *)(ws + pl.po);

  // an axis of one entry is never stepped along: any legal stride will do
  auto stride = [](int64_t n, int64_t s, int es) -> uint64_t { return n > 1 ? (uint64_t)s * es : 16; };
  CUtensorMap mq, mk, mv;
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.T, (uint64_t)a.B};
    const uint64_t st[3] = {stride(a.H, a.q.sh, 2), stride(a.T, a.q.st, 2), stride(a.B, a.q.sb, 2)};
    const uint32_t box[4] = {64, (uint32_t)g, (uint32_t)p.tpt, 1};
    if (!encode_map4(&mq, false, a.q.data, dims, st, box, true)) {
      *why = "the tensor map of q was rejected";
      return cudaErrorInvalidValue;
    }
  }
  const uint64_t pages = (uint64_t)a.c.n_pages;
  for (int i = 0; i < 2; ++i) {
    const int es = q8 ? 1 : 2;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.c.H, (uint64_t)a.c.page_size, pages};
    const uint64_t st[3] = {stride(a.c.H, a.c.s_head, es), stride(a.c.page_size, a.c.s_tok, es),
                            stride((int64_t)pages, a.c.s_page, es)};
    const uint32_t box[4] = {q8 ? (uint32_t)D : 64u, 1, (uint32_t)p.box, 1};
    if (!encode_map4(i ? &mv : &mk, q8, i ? a.c.v : a.c.k, dims, st, box, !q8 || D == 128)) {
      *why = "the tensor map of the cache was rejected";
      return cudaErrorInvalidValue;
    }
  }
  if (D == 64) {
    if (a.c.format == LA_KV_E4M3) return launch_one<64, LA_KV_E4M3>(mq, mk, mv, p, stream);
    if (a.c.format == LA_KV_INT8) return launch_one<64, LA_KV_INT8>(mq, mk, mv, p, stream);
    return launch_one<64, LA_KV_BF16>(mq, mk, mv, p, stream);
  }
  if (a.c.format == LA_KV_E4M3) return launch_one<128, LA_KV_E4M3>(mq, mk, mv, p, stream);
  if (a.c.format == LA_KV_INT8) return launch_one<128, LA_KV_INT8>(mq, mk, mv, p, stream);
  return launch_one<128, LA_KV_BF16>(mq, mk, mv, p, stream);
}

cudaError_t pa_device_error(unsigned int *flags, unsigned int *where, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_pa_error, sizeof *flags);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(where, g_pa_where, sizeof *where);
  if (e == cudaSuccess && reset) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_pa_error, &zero, sizeof zero);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_pa_where, &zero, sizeof zero);
  }
  return e;
}

}  // namespace la

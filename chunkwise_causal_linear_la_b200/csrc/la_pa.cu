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
// r of a tile of 128 (or 64) is token r / g, head r % g of floor(128 / g) tokens.  An
// entry of work is one or two such tiles of a sequence and one cache head.  With two
// tiles the two softmax warpgroups take a tile each over the same keys; with one
// (single tokens, short chunks, the end of a prompt) they take the first and the
// second half of each key tile, with an accumulator each, joined at the end.  Either
// way one group's exponentials run beside the other group's products.
//
// Work.  The key tiles of all entries and heads stand in one row; CTA c of G (one
// per SM) takes the c-th of G parts of equal cost of it.  An entry cut by a border leaves
// partial results (unnormalised o, m, l) in the workspace, which a last kernel joins
// (joining inside, by whichever CTA came last, kept single CTAs busy for 12 us).  A
// first one lays out the row: lengths are known to the device only.  Each kernel sets
// itself up while the one before it ends.
//
// Roles (warps): 0 TMA producer (the tile's boxes on as many lanes; a box is a
// power-of-two piece of a page), 1 MMA issuer, 2-3 values fix-up (bf16) or scales
// (8-bit caches, one query tile), 4-7 and 8-11 softmax, from 12 on conversion (8-bit
// caches: codes become bf16 operands, exact for power-of-two scales).
//   QK:  S[w] = Q K^T     (M = 128 or 64, N = 128 keys, K = D)   S in TMEM
//   PV:  O[w] += P V      (N = D, K = 128 keys; 64 a group)      P (bf16) over S in TMEM
// Tensor-core instructions of one thread run in order, so the product that reads P is
// done before the next scores overwrite it.  With two tiles the commit that announces
// S[w] of the next key tile also says that O[w] holds the one before; where a group
// has to rescale O between the halves of a tile, or with one query tile (whose
// scores run two key tiles ahead), it waits for the product itself.
//
// What a query does not see must not reach it even where it is an infinity or a NaN:
// scores are masked by selection, but 0 * inf in PV would be NaN.  Rows that no query
// of the entry sees are zeroed; in rows that some see, values that are not finite
// are taken out of the operand and added at the end for the queries that see them.
// (8-bit caches: by the converted values, since a code times a finite scale may be
// infinite too.)
//
// Every wait is bounded: on a timeout the CTA records it, drains and returns.
//
// What bounds it, measured on one B200 (bf16 unless said, 16 query heads over 4 cache heads of 128):
//   2048 tokens over 16384               247 us (275 back to back, at the power limit), 1.04 PFLOP/s (63% of the
//                                        library's matrix product): a softmax group's chain (scores in, exponentials,
//                                        P out) beside its products; tensor pipe 53%
//   the same, e4m3 and int8              350 and 367 us: 3.4 and 3.5 us a key tile of a CTA where bf16 takes 2.3 (one
//                                        stage of codes each for keys and values, eight conversion warps, spills)
//   256 single tokens over up to 8192    342 us (353 back to back), 6.3 TB/s (97% of a copy): memory
//   one token over 1,048,576, e4m3       334 us (343 back to back), 3.3 TB/s: conversion of codes (244 us without it, 240
//                                        without the softmax's work too)
//   44 tokens and 4 pieces, e4m3,        179 us: 43 key tiles a CTA as above; its two entries cost it 4 - 6 us each
//   20 query heads                       beside them
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
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
using tcsync::drain_bar;
using tcsync::pack2;
using tcsync::Sync;

// Bounded wait on a barrier: true once the phase has completed, false when the CTA has given up or this wait does (2^19
// probes; one that fails sleeps for 7800 cycles: about two seconds), which is recorded.  It is kept short: it stands in
// some thirty places, by warps that would share the instruction cache with the ones that work.
constexpr uint32_t kProbes = 1u << 19;
__device__ __forceinline__ bool wait_on(const Sync &sy, int idx, uint32_t parity, int tile, uint32_t probes = kProbes) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n, f;\n\t"
      "mov.u32 n, %4;\n"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
      "ld.volatile.shared.u32 f, [%3];\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.eq.u32 q, f, 0;\n\t"
      "setp.ne.and.u32 q, n, 0, q;\n\t@q bra AGAIN;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(sy.bar + idx)), "r"(parity), "r"(smem_u32(const_cast<int *>(sy.abort))), "r"(probes)
      : "memory");
  if (!ok && !*sy.abort) {
    *sy.abort = 1;
    atomicOr(sy.err, 1u);
    atomicCAS(sy.where, 0u, 0x80000000u | ((uint32_t)(tile & 0x7FFFFF) << 8) | (uint32_t)idx);
  }
  return ok != 0;
}
__device__ __forceinline__ void arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ bool wait_on_warp(const Sync &sy, int idx, uint32_t parity, int tile,
                                             uint32_t probes = kProbes) {
  return __all_sync(0xffffffffu, wait_on(sy, idx, parity, tile, probes));
}

constexpr int kTile = 128;  // keys of a tile, rows of a query tile

// One or two query tiles of a sequence: the same for every cache head.
struct alignas(16) Entry {
  int32_t seq, b, tok, ntok;     // sequence; batch row; first token (T axis) and tokens
  int32_t pos, kv_end, lo, cnt;  // position of the first token; positions in reach; first key tile, key tiles
};
struct alignas(16) CtaWork {
  int32_t head, entry, off, pad;  // where this CTA's part starts: key tile `off` of an entry
  int64_t start, count;           // that place in the row of tiles; key tiles
};

struct PaArgs {
  const int32_t *cu, *kv_len, *table;
  int64_t T, max_pages, n_pages, n_seqs;
  int32_t page_size, box, g, tpt, per, Hkv, H, window;  // tokens of a query tile, of an entry
  int32_t e_max, G, test_stop;  // test_stop: LA_FLAG_TEST_WAIT_TIMEOUT
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
  int64_t *pre;        // [e_max][2]: cost and key tiles of the entries before
  CtaWork *work;       // [G]
  float *po;           // [G][2][2][D / 4][128][4]: four columns of all rows side by side
  float2 *pml;         // [G][2][2][128]
};

// ------------------------------------------------------------------ schedule
constexpr int kPlanThreads = 1024;

// Exclusive prefixes of u and v over the block, and its sums.
struct Pair {
  int64_t u, v;
};
__device__ __forceinline__ Pair block_scan(Pair x, Pair *warp_sums, Pair &sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto warp_scan = [&](Pair p) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, p.u, o), b = __shfl_up_sync(0xffffffffu, p.v, o);
      if (lane >= o) p.u += a, p.v += b;
    }
    return p;
  };
  const Pair p = warp_scan(x);
  if (lane == 31) warp_sums[w] = p;
  __syncthreads();
  if (w == 0) warp_sums[lane] = warp_scan(warp_sums[lane]);
  __syncthreads();
  const Pair before = w ? warp_sums[w - 1] : Pair{0, 0};
  sum = warp_sums[31];
  __syncthreads();
  return Pair{before.u + p.u - x.u, before.v + p.v - x.v};
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

// What a key tile and an entry cost a CTA, in thirds of a tile of two query tiles (about 2 us; one query tile: 1.4 us).
// An entry costs about two tiles besides its own: its queries' way in, the first weights, its results.  (As bf16 with
// heads of 128 measured; used for every form.  In 8 bits a two-tile one takes 3.4 us.)
__device__ __forceinline__ int tile_cost(const PaArgs &a, const Entry &e) { return e.ntok > a.tpt ? 3 : 2; }
__device__ __forceinline__ int64_t entry_cost(const PaArgs &a, const Entry &e) {
  return (int64_t)tile_cost(a, e) * e.cnt + (e.ntok > a.tpt ? 6 : 3);
}

// First entry of each sequence and first tile of each entry: searched in shared memory while there are at most
// kPlanThreads of them (the usual call), else where they lie in the workspace.
__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(const PaArgs a) {
  __shared__ Pair ws[32];
  __shared__ int64_t first_cost[kPlanThreads], begin[kPlanThreads + 1];
  __shared__ int32_t first_entry[kPlanThreads];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the main kernel's CTAs set themselves up meanwhile
  const int64_t per = a.per;
  Pair sum;
  int64_t carry = 0;
  const int64_t dense_k = (a.T + per - 1) / per;  // entries of a sequence of a dense batch
  if (a.cu) {
    for (int64_t n0 = 0; n0 < a.n_seqs; n0 += kPlanThreads) {
      const int64_t n = n0 + tid;
      int64_t st = 0, len = 0;
      if (n < a.n_seqs) seq_span(a, n, st, len);
      const int64_t k = (len + per - 1) / per;
      const int64_t x = block_scan(Pair{k, 0}, ws, sum).u;
      if (n < a.n_seqs) {
        a.seq_ent[n + 1] = (int32_t)min(carry + x + k, (int64_t)a.e_max);
        if (n0 == 0) first_entry[tid] = (int32_t)min(x, (int64_t)a.e_max);
      }
      carry += sum.u;
    }
    if (tid == 0) a.seq_ent[0] = 0;
    __syncthreads();
  } else {
    carry = dense_k * a.n_seqs;
  }
  // overlapping sequences (an invalid cu_seqlens) could ask for more entries than there is room for
  const int E = (int)min(carry, (int64_t)a.e_max);
  const int32_t *se = a.n_seqs <= kPlanThreads ? first_entry : a.seq_ent;
  carry = 0;
  int64_t tiles = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int64_t cnt = 0, cost = 0;
    if (e < E) {
      int64_t lo = 0, t0;  // the last sequence whose first entry is <= e
      if (a.cu) {
        int64_t hi = a.n_seqs;
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (se[mid] <= e) lo = mid; else hi = mid;
        }
        t0 = (int64_t)(e - se[lo]) * per;
      } else {
        lo = e / dense_k;
        t0 = (e - lo * dense_k) * per;
      }
      int64_t st, len;
      seq_span(a, lo, st, len);
      const int64_t kv = max((int64_t)a.kv_len[lo], (int64_t)0);
      Entry x;
      x.seq = (int)lo;
      x.b = a.cu ? 0 : (int)lo;
      x.tok = (int)(st + t0);
      x.ntok = (int)max((int64_t)0, min(per, len - t0));
      const int64_t pos = kv - len + t0;
      x.pos = (int)max(pos, -((int64_t)1 << 30));  // below 0 all the same
      x.kv_end = (int)min(kv, a.cap);
      const int64_t end = min(pos + x.ntok, (int64_t)x.kv_end);
      const int64_t beg = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
      x.lo = (int)(min(beg, max(end, (int64_t)0)) / kTile);
      cnt = end > beg ? (end + kTile - 1) / kTile - x.lo : 1;  // nothing seen: one tile, all masked
      x.cnt = (int)cnt;
      a.ent[e] = x;
      cost = entry_cost(a, x);
    }
    const Pair x = block_scan(Pair{cost, cnt}, ws, sum);
    if (e < E) {
      a.pre[2 * (int64_t)e] = carry + x.u;
      a.pre[2 * (int64_t)e + 1] = tiles + x.v;
      if (e0 == 0) first_cost[tid] = x.u;
    }
    carry += sum.u;
    tiles += sum.v;
  }
  __syncthreads();
  // Border c of G: where c G-ths of the cost are reached, at a tile (or an entry's start: what an entry costs besides its
  // tiles comes first).  Its place in the row of tiles; a CTA between two equal borders has nothing.
  const int64_t W = tiles * a.Hkv;
  for (int c = tid; c <= a.G; c += kPlanThreads) {
    CtaWork w;
    w.head = w.entry = w.off = w.pad = 0;
    w.start = W;
    w.count = 0;
    if (c < a.G && E > 0) {
      const int64_t s = carry * a.Hkv / a.G * c + carry * a.Hkv % a.G * c / a.G;
      w.head = (int)(s / carry);
      const int64_t r = s - w.head * carry;
      int lo = 0, hi = E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((E <= kPlanThreads ? first_cost[mid] : a.pre[2 * (int64_t)mid]) <= r) lo = mid; else hi = mid;
      }
      const Entry x = a.ent[lo];
      const int64_t in = r - a.pre[2 * (int64_t)lo] - entry_cost(a, x) + tile_cost(a, x) * (int64_t)x.cnt;
      w.entry = lo;
      w.off = in > 0 ? (int)(in / tile_cost(a, x)) : 0;
      w.start = w.head * tiles + a.pre[2 * (int64_t)lo + 1] + w.off;
    }
    begin[c] = w.start;
    if (c < a.G) a.work[c] = w;
  }
  __syncthreads();
  for (int c = tid; c < a.G; c += kPlanThreads) a.work[c].count = begin[c + 1] - begin[c];
  if (tid == 0) a.seq_ent[0] = E;  // the main kernel wraps to the next head after entry E - 1
}

// ------------------------------------------------------------------ main kernel
template <int D, int FMT, int NQ>
struct PaCfg {
  static constexpr bool Q8 = FMT != LA_KV_BF16;
  static constexpr int CONV = Q8 ? (NQ == 1 ? 16 : 8) : 0;  // conversion warps
  static constexpr int THREADS = 384 + 32 * CONV;
  // With one query tile and 8-bit codes a tile is short beside the issuing warp's waits and commits: what ends together is
  // announced together (scores with the keys' slot, a product with the values'), P with the values, and scales have
  // warps of their own (one token over 1M, e4m3: 369 -> 357 us).
  static constexpr bool LEAN = Q8 && NQ == 1;
  static constexpr int ROWS = NQ == 1 ? 64 : 128;    // rows of a query tile
  static constexpr int WROWS = ROWS / 4;             // of them, a softmax warp's
  static constexpr int SLABS = D / 64;               // 64-column slabs of a bf16 tile
  static constexpr int SLAB = kTile * 128;           // bytes of one
  static constexpr int TILE = SLABS * SLAB;          // a bf16 operand tile
  static constexpr int QSLAB = ROWS * 128;
  static constexpr int QTILE = SLABS * QSLAB;
  static constexpr int RAW = kTile * D;              // a tile of codes
  // operand slots and stages of codes, keys and values in turn: even numbers, so that the conversion warps of keys and
  // those of values have slots and stages of their own
  static constexpr int NS = (Q8 ? 4 : NQ == 1 ? 6 : 5) * (128 / D);
  static constexpr int NR = Q8 ? (D == 128 ? (NQ == 1 ? 4 : 2) : NQ == 1 ? 8 : 6) : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_OP = NQ * QTILE;
  static constexpr int OFF_RAW = OFF_OP + NS * TILE;
  static constexpr int OFF_SC = OFF_RAW + NR * RAW;  // scales of a stage, 128 floats
  static constexpr int OFF_ML = OFF_SC + NR * kTile * 4;
  static constexpr int OFF_BAR = OFF_ML + kTile * 8;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_RFULL = 2 * NS, B_REMPTY = B_RFULL + NR, B_QFULL = B_REMPTY + NR,
                       B_QEMPTY = B_QFULL + 1, B_SFULL = B_QFULL + 2, B_PFULL = B_QFULL + 4, B_OFULL = B_QFULL + 6,
                       B_OEMPTY = B_QFULL + 8, B_MERGE = B_QFULL + 10, B_DRAIN = B_QFULL + 11,
                       B_PSPLIT = B_QFULL + 12, B_ODONE = B_QFULL + 14,  // one query tile: P of both groups; PV done
                       B_PHALF = B_QFULL + 15,  // two query tiles: P's second half (PFULL: the first)
                       B_HDONE = B_QFULL + 17,  // ... PV of the first half done
                       B_READY = B_QFULL + 19,  // bf16, per slot: fixed up
                       NBAR = B_READY + (Q8 ? 0 : NS);
  // per item (mod 16) and fix-up or conversion warp: values that are not finite were taken out.  (A flag left
  // from 16 items before only costs a look for such values.)
  static constexpr int OFF_BAD = OFF_BAR + (NBAR * 8 + 15) / 16 * 16;
  static constexpr int OFF_MISC = OFF_BAD + 16 * 16;
  static constexpr int SMEM_USED = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = SMEM_USED;
  // tensor memory columns
  static constexpr int T_S = 0, T_O = 2 * kTile, T_COLS = 512;
  static_assert(T_O + 2 * D <= 512, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
  // register split (per thread; shares add up to the launch's)
  static constexpr int R_LAUNCH = 65536 / THREADS / 8 * 8;
  static constexpr int R_AUX = Q8 ? (NQ == 1 ? 72 : 80) : 104, R_SOFT = Q8 ? (NQ == 1 ? 112 : 136) : 200,
                       R_CONV = NQ == 1 ? 48 : 64;
  static_assert(R_AUX <= R_LAUNCH && R_CONV <= R_LAUNCH && R_SOFT >= R_LAUNCH, "setmaxnreg .dec and .inc");
  static_assert(128 * R_AUX + 256 * R_SOFT + 32 * CONV * R_CONV <= THREADS * R_LAUNCH, "register split");
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

// Positions that token `tk` of an entry sees: [lo, hi).  (32 bits hold a position: kv_len is an int32.)
__device__ __forceinline__ void sees(const PaArgs &a, const Entry &e, int tk, int &lo, int &hi) {
  const int p = e.pos + tk;
  hi = min(p + 1, e.kv_end);
  lo = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;  // (p may be far below 0, the window near 2^31)
}

// What the sum of weighted values is multiplied with.  The largest weight is 1 or more, so a sum of zero means a row that
// sees nothing (zeros), or one whose scores are all -infinity (NaN, the formula's 0 / 0).
__device__ __forceinline__ float factor(float l, bool sees_any) {
  return l != 0.f ? 1.f / l : sees_any ? __uint_as_float(0x7FC00000u) : 0.f;
}

// Of the keys of tile t: all tokens of the entry see those in [b, c); some those in
// [a, d); none the rest (tile-relative, clamped).
struct Reach {
  int a, b, c, d;
};
__device__ __forceinline__ int in_tile(int p, int ts) { return min(max(p - ts, 0), kTile); }
__device__ __forceinline__ Reach reach(const PaArgs &a, const Entry &e, int t) {
  int lo0, hi0, lo1, hi1;
  sees(a, e, 0, lo0, hi0);
  sees(a, e, max(e.ntok, 1) - 1, lo1, hi1);
  const int ts = t * kTile;
  return Reach{in_tile(lo0, ts), in_tile(lo1, ts), in_tile(hi0, ts), in_tile(hi1, ts)};
}
__device__ __forceinline__ bool partly(const Reach &r) { return r.b > 0 || r.c < kTile; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(s c + b) of two scores, and pairwise sums: two products or sums an instruction.
__device__ __forceinline__ float2 weight2(float s0, float s1, float c, float b) {
  float2 x;
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmov.b64 w, {%5, %5};\n\t"
      "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(x.x), "=f"(x.y)
      : "f"(s0), "f"(s1), "f"(c), "f"(b));
  x.x = ex2(x.x);
  x.y = ex2(x.y);
  return x;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tadd.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Sixteen codes times the scale f as bf16 (exact for the powers of two that la_kv_write stores).
//   e4m3: the hardware's conversion of pairs to fp16 (exact).
//   int8: the byte with its sign bit flipped, under the exponent of 2^10: 1152 plus the code in fp16.
// Then fp32 products and one rounding.  Instructions on bits and conversions run at half rate, which bounds this: two and
// a half a pair of codes before the two to fp32 (moving bits into bf16's places would take four and more).
template <int FMT>
__device__ __forceinline__ void convert16(const uint4 &w, float f, uint4 &o0, uint4 &o1) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t v[8];
  if (FMT == LA_KV_E4M3) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t pair = k & 1 ? in[k >> 1] >> 16 : in[k >> 1] & 0xFFFFu;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3);
      const float2 g = __half22float2(__half2(h));
      v[k] = pack2(g.x * f, g.y * f);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __byte_perm(in[k >> 1] ^ 0x80808080u, 0x64646464u, k & 1 ? 0x4342 : 0x4140);
      const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&b));
      v[k] = pack2((g.x - 1152.f) * f, (g.y - 1152.f) * f);
    }
  }
  o0 = make_uint4(v[0], v[1], v[2], v[3]);
  o1 = make_uint4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
  return u;
}
__device__ __forceinline__ void sts16(uint32_t at, const uint4 &u) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}

__device__ __forceinline__ bool finite_f(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ uint32_t keep_finite(uint32_t w) {  // bf16x2
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}
// Eight values: those that are not finite become zeros.  1 where there was one.
__device__ __forceinline__ int take_out(uint4 &u) {
  const uint4 f = make_uint4(keep_finite(u.x), keep_finite(u.y), keep_finite(u.z), keep_finite(u.w));
  const int found = f.x != u.x || f.y != u.y || f.z != u.z || f.w != u.w;
  u = f;
  return found;
}

template <int D, int FMT, int NQ>
__global__ void __launch_bounds__((PaCfg<D, FMT, NQ>::THREADS), 1)
pa_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
          const __grid_constant__ CUtensorMap tm_v, const PaArgs a) {
  using G = PaCfg<D, FMT, NQ>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + G::OFF_BAR);
  float *sc = reinterpret_cast<float *>(sm + G::OFF_SC);
  float2 *ml = reinterpret_cast<float2 *>(sm + G::OFF_ML);
  volatile uint8_t *bad = sm + G::OFF_BAD;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + G::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + G::OFF_MISC + 4);
  const Sync sy{bars, abort_flag, &g_pa_error, &g_pa_where};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (smem_u32(sm) & 1023) {  // the swizzled tiles need it (no static shared memory lies in front)
    if (tid == 0) atomicOr(&g_pa_error, 4u);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < G::NBAR; ++i) {
      uint32_t cnt = 1;
      if (G::Q8 && i < G::NS) cnt = G::CONV / 2 + (G::LEAN && (i & 1) ? 8 : 0);  // FULL: conversion (and softmax) warps
      if (!G::Q8 && i >= G::B_EMPTY && i < G::B_EMPTY + G::NS) cnt = 3;  // products done, seen by the fix-up warps
      if (i >= G::B_RFULL && i < G::B_RFULL + G::NR) cnt = G::LEAN ? 2 : 1;  // codes on their way, scales there
      if (i >= G::B_REMPTY && i < G::B_REMPTY + G::NR) cnt = G::CONV / 2;  // codes read
      if (i >= G::B_PFULL && i < G::B_PFULL + 2) cnt = 4;               // softmax warps
      if (i >= G::B_OEMPTY && i < G::B_OEMPTY + 2) cnt = 4;
      if (i == G::B_MERGE) cnt = 4;
      if (i >= G::B_PSPLIT && i < G::B_PSPLIT + 2) cnt = 8;
      if (i >= G::B_PHALF && i < G::B_PHALF + 2) cnt = 4;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan (and what came before it) is there
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
        const bool two = NQ == 2 && it.e.ntok > a.tpt;
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
        // 8 bits: the scales of this lane's four keys (and values) of the tile after, by plain loads: as many bulk
        // copies as there are boxes would cost more than the codes'
        float4 nsk = make_float4(0.f, 0.f, 0.f, 0.f), nsv = nsk;
        auto scales_at = [&](int t) {
          const int64_t p = (int64_t)t * kTile + 4 * lane;
          nsk = nsv = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p >= it.e.kv_end) return;
          const uint32_t idx = (uint32_t)p / (uint32_t)a.page_size;
          const int pg = a.table[(int64_t)it.e.seq * a.max_pages + idx];
          if (pg < 0 || pg >= a.n_pages) return;
          const int64_t at = ((int64_t)pg * a.Hkv + it.head) * a.page_size + (p - (int64_t)idx * a.page_size);
          nsk = *reinterpret_cast<const float4 *>(a.ks + at);
          nsv = *reinterpret_cast<const float4 *>(a.vs + at);
        };
        if (G::Q8 && !G::LEAN) scales_at(it.t0);
        for (int i = 0; i < it.n && ok; ++i) {
          if (i + 1 < it.n) npg = page_at(it.t0 + i + 1, nslot);
          const float4 sk = nsk, sv = nsv;
          if (G::Q8 && !G::LEAN && i + 1 < it.n) scales_at(it.t0 + i + 1);
          // a missing page is read past the end of the page axis: zeros
          const int pc = pg >= 0 ? pg : (int)a.n_pages;
#pragma unroll
          for (int kvi = 0; kvi < 2; ++kvi, ++seq) {
            if (kvi && a.test_stop) {  // no values: every role waits for them
              ok = false;
              break;
            }
            const CUtensorMap *tm = kvi ? &tm_v : &tm_k;
            if (!G::Q8) {
              const int s = seq % G::NS;
              if (!(ok = wait_on_warp(sy, G::B_EMPTY + s, ((seq / G::NS) & 1) ^ 1, it.t0 + i))) break;
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
              if (!(ok = wait_on_warp(sy, G::B_REMPTY + s, ((seq / (G::NR > 0 ? G::NR : 1)) & 1) ^ 1, it.t0 + i))) break;
              if (!G::LEAN) reinterpret_cast<float4 *>(sc + s * kTile)[lane] = kvi ? sv : sk;
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(bars + G::B_RFULL + s, G::RAW);
              __syncwarp();
              if (lane < nb)
                tma_load_4d(raw_stage(s) + lane * a.box * D, tm, bars + G::B_RFULL + s, 0, it.head, slot, pc);
            }
            if (i == 0 && kvi == 0) {  // the item's queries, after its first keys are on their way
              if (!(ok = wait_on_warp(sy, G::B_QEMPTY, (items & 1) ^ 1, it.t0))) {
                ++seq;
                break;
              }
              if (lane == 0) {
                mbar_arrive_expect_tx(bars + G::B_QFULL, two ? 2 * q_bytes : q_bytes);
                for (int w = 0; w < (two ? 2 : 1); ++w)
                  for (int sl = 0; sl < G::SLABS; ++sl)
                    tma_load_4d(sm + G::OFF_Q + w * G::QTILE + sl * G::QSLAB, &tm_q, bars + G::B_QFULL, sl * 64,
                                it.head * a.g, it.e.tok + w * a.tpt, it.e.b);
              }
              ++items;
            }
          }
          pg = npg;
          slot = nslot;
        }
      }
      // Every copy under way lands before the CTA ends.  (Asked whether or not the CTA has given up yet: it may do so
      // after this warp's last copies.)
      if (lane == 0) {
        constexpr uint32_t N = G::Q8 ? (G::NR > 0 ? G::NR : 1) : G::NS;
        const int b = G::Q8 ? G::B_RFULL : G::B_FULL;
        for (uint32_t s = seq > N ? seq - N : 0; s < seq; ++s) drain_bar(sy, b + s % N, (s / N) & 1);
        if (items) drain_bar(sy, G::B_QFULL, (items - 1) & 1);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp walks and waits, so that descriptors and addresses are uniform; one lane issues.
      constexpr uint32_t ID_QK = idesc_bf16_f32(G::ROWS, kTile, 0, 0);
      constexpr uint32_t ID_PV = idesc_bf16_f32(G::ROWS, D, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(sm + G::OFF_Q), 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(op_slot(0)), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(op_slot(0)), G::SLAB, 1024);
      uint32_t seq = 0, items = 0, used[2] = {0, 0}, pcnt[2] = {0, 0}, bcnt[2] = {0, 0};
      bool ok = true;
      // S[w] = Q[qt] K^T for the keys in slot sl
      auto qk = [&](int w, int qt, uint32_t sl) {
        tc_fence_after();
        const uint64_t dq = dq0 + (uint64_t)(qt * (G::QTILE >> 4));
        const uint64_t dk = dk0 + (uint64_t)(sl * (G::TILE >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tbase + G::T_S + w * kTile, dq + (((kk >> 2) * G::QSLAB + (kk & 3) * 32) >> 4),
                      dk + (((kk >> 2) * G::SLAB + (kk & 3) * 32) >> 4), ID_QK, kk > 0);
          if (!G::LEAN) umma_commit(bars + G::B_SFULL + w);
        }
        __syncwarp();
      };
      auto commit = [&](int bar) {
        if (elect_one()) umma_commit(bars + bar);
        __syncwarp();
      };
      auto keys = [&](int i) -> bool {  // tile i's keys are in their slot
        const uint32_t k = seq + 2 * i;
        return wait_on_warp(sy, G::B_FULL + k % G::NS, (k / G::NS) & 1, it.t0 + i);
      };
      auto values = [&](int i) -> bool {
        const uint32_t k = seq + 2 * i + 1;
        const bool fix = !G::Q8 && partly(reach(a, it.e, it.t0 + i));
        return wait_on_warp(sy, (fix ? G::B_READY : G::B_FULL) + k % G::NS, (k / G::NS) & 1, it.t0 + i);
      };
      auto o_free = [&](int w) -> bool {  // O[w] of the item before has been read
        if (used[w] && !wait_on_warp(sy, G::B_OEMPTY + w, (used[w] - 1) & 1, it.t0)) return false;
        ++used[w];
        return true;
      };
      while (ok && walk.next(a, it)) {
        const bool two = NQ == 2 && it.e.ntok > a.tpt;
        ok = wait_on_warp(sy, G::B_QFULL, items & 1, it.t0);
        ++items;
        if (two) {
          // QK(0, K0) QK(1, K0), then for each tile and group w: PV(w, Vi), QK(w, Ki+1)
          if (ok && (ok = keys(0))) {
            qk(0, 0, seq % G::NS);
            qk(1, 1, seq % G::NS);
            commit(G::B_EMPTY + seq % G::NS);
            if (it.n == 1) commit(G::B_QEMPTY);
          }
          for (int i = 0; i < it.n && ok; ++i) {
            const uint32_t vs = (seq + 2 * i + 1) % G::NS, ks = (seq + 2 * i + 2) % G::NS;
            if (!(ok = values(i))) break;
            for (int w = 0; w < 2 && ok; ++w) {
              if (i == 0 && !(ok = o_free(w))) break;
              const uint64_t dv = dv0 + (uint64_t)(vs * (G::TILE >> 4));
              // the first half of P's keys is multiplied while the second is worked out
              for (int hf = 0; hf < 2 && ok; ++hf) {
                if (!(ok = wait_on_warp(sy, (hf ? G::B_PHALF : G::B_PFULL) + w, pcnt[w] & 1, it.t0 + i))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                  for (int kk = 0; kk < kTile / 32; ++kk)
                    umma_bf16_ts(tbase + G::T_O + w * D, tbase + G::T_S + w * kTile + hf * 32 + kk * 8,
                                 dv + (((hf * 4 + kk) * 2048) >> 4), ID_PV, (i > 0 || hf > 0 || kk > 0) ? 1u : 0u);
                  if (hf == 0) umma_commit(bars + G::B_HDONE + w);
                }
                __syncwarp();
              }
              if (!ok) break;
              ++pcnt[w];
              if (w == 1) commit(G::B_EMPTY + vs);
              if (i + 1 == it.n) {
                commit(G::B_OFULL + w);
              } else {
                if (w == 0 && !(ok = keys(i + 1))) break;
                qk(w, w, ks);
                if (w == 1) {
                  commit(G::B_EMPTY + ks);
                  if (i + 2 == it.n) commit(G::B_QEMPTY);
                }
              }
            }
          }
        } else {
          // QK(0) QK(1), then for each tile: PV of the two groups' halves of its keys, QK two tiles ahead
          auto step = [&](int i) -> bool {
            if (!keys(i)) return false;
            const uint32_t ks = (seq + 2 * i) % G::NS;
            qk(i & 1, 0, ks);
            commit(G::B_EMPTY + ks);
            if (i + 1 == it.n) commit(G::B_QEMPTY);
            return true;
          };
          ok = ok && step(0) && (it.n < 2 || step(1));
          for (int i = 0; i < it.n && ok; ++i) {
            const int b = i & 1;
            const uint32_t vs = (seq + 2 * i + 1) % G::NS;
            if (!(ok = values(i))) break;
            if (i == 0 && !(ok = o_free(0) && o_free(1))) break;
            if (!G::LEAN && !(ok = wait_on_warp(sy, G::B_PSPLIT + b, bcnt[b] & 1, it.t0 + i))) break;
            ++bcnt[b];
            tc_fence_after();
            const uint64_t dv = dv0 + (uint64_t)(vs * (G::TILE >> 4));
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_bf16_ts(tbase + G::T_O + (kk >> 2) * D, tbase + G::T_S + b * kTile + (kk >> 2) * 64 + (kk & 3) * 8,
                             dv + ((kk * 2048) >> 4), ID_PV, (i > 0 || (kk & 3) > 0) ? 1u : 0u);
            }
            __syncwarp();
            if (!G::LEAN) commit(G::B_ODONE);
            commit(G::B_EMPTY + vs);
            if (i + 1 == it.n) {
              commit(G::B_OFULL);
              commit(G::B_OFULL + 1);
            }
            if (i + 2 < it.n) ok = step(i + 2);
          }
        }
        seq += 2 * it.n;
      }
      commit(G::B_DRAIN);  // products under way end before tensor memory is freed
      drain_bar(sy, G::B_DRAIN, 0);
      __syncwarp();
    } else if (G::LEAN) {
      // -------------------------------------------------------------- scales: of keys (warp 2) and values (warp 3)
      // (With two query tiles the producer does this.  With one it would be late with the codes: 64 sequences up to
      // 16384 in int8, pages of 16, 141 us so and 126 with warps of their own; two query tiles, mixed batch, 197 and 230.)
      constexpr int NRr = G::NR > 0 ? G::NR : 1;
      const int kvi = warp - 2;
      const float *from = kvi ? a.vs : a.ks;
      int rs = kvi;
      uint32_t rph = 1;
      bool ok = true;
      while (ok && walk.next(a, it)) {
        auto scales_at = [&](int i) -> float4 {
          const int64_t p = (int64_t)(it.t0 + i) * kTile + 4 * lane;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i >= it.n || p >= it.e.kv_end) return x;
          const uint32_t idx = (uint32_t)p / (uint32_t)a.page_size;
          const int pg = a.table[(int64_t)it.e.seq * a.max_pages + idx];
          if (pg >= 0 && pg < a.n_pages)
            x = *reinterpret_cast<const float4 *>(from + ((int64_t)pg * a.Hkv + it.head) * a.page_size +
                                                  ((uint32_t)p - idx * (uint32_t)a.page_size));
          return x;
        };
        float4 next = scales_at(0);
        for (int i = 0; i < it.n; ++i) {
          const float4 x = next;
          next = scales_at(i + 1);
          if (!(ok = wait_on_warp(sy, G::B_REMPTY + rs, rph, it.t0 + i))) break;
          reinterpret_cast<float4 *>(sc + rs * kTile)[lane] = x;
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + G::B_RFULL + rs);
          if ((rs += 2) >= NRr) rs = kvi, rph ^= 1;
        }
      }
    } else if (!G::Q8) {
      // -------------------------------------------------------------- values fix-up
      // These warps see every tile and take part in its release: a slot is not filled again before they have
      // noted its phase, so they cannot fall behind the ring or run ahead of it.
      uint32_t seq = 0, items = 0;
      bool ok = true;
      const int t = tid - 64;
      while (ok && walk.next(a, it)) {
        if (lane == 0) bad[(items & 15) * 16 + warp - 2] = 0;
        __syncwarp();
        for (int i = 0; i < 2 * it.n; ++i, ++seq) {
          const uint32_t sl = seq % G::NS;
          if (!(ok = wait_on_warp(sy, G::B_FULL + sl, (seq / G::NS) & 1, it.t0 + (i >> 1)))) break;
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
                uint4 u = *p;
                if (take_out(u)) {
                  *p = u;
                  found = 1;
                }
              }
            }
            if (found) bad[(items & 15) * 16 + warp - 2] = 1;
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
    const int w = (warp - 4) >> 2, quad = warp & 3;
    // rows lie in tensor memory lanes 32 q + l: 32 a quarter, or with 64-row tiles 16 (l < 16)
    const int r = quad * G::WROWS + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t ts_addr = tbase + G::T_S + lane_off;
    const uint32_t to_addr = tbase + G::T_O + lane_off;
    const float c = a.c;
    uint32_t scnt[2] = {0, 0}, ocnt[2] = {0, 0}, mcnt = 0, dcnt = 0, hcnt = 0, items = 0;
    bool ok = true;
    while (ok && walk.next(a, it)) {
      const bool two = NQ == 2 && it.e.ntok > a.tpt;
      const int tk = (two ? w * a.tpt : 0) + r / a.g;
      const bool valid = lane < G::WROWS && r < a.g * a.tpt && tk < it.e.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      // Warps without a row take no part in the tiles: rows fill them in order, the first arrives for them too.
      const int rows = min(a.g * a.tpt, max(0, (it.e.ntok - (two ? w * a.tpt : 0)) * a.g));
      const int idle = 4 - max(1, (rows + G::WROWS - 1) / G::WROWS);
      const bool part_of = active || quad == 0;
      int lo, hi;
      sees(a, it.e, tk, lo, hi);
      if (!valid) lo = hi = 0;
      // tiles [full0, full1) of the piece: every token of the entry sees all of their keys
      int full0, full1;
      {
        int x, lo1, hi0, y;
        sees(a, it.e, 0, x, hi0);
        sees(a, it.e, max(it.e.ntok, 1) - 1, lo1, y);
        full0 = (int)(((uint32_t)lo1 + kTile - 1) / kTile) - it.t0;
        full1 = max(hi0, 0) / kTile - it.t0;
      }
      float m = -INFINITY, l = 0.f;  // the maximum in powers of two: scale log2(e) times the score
      if (two) {
        // ---- this group's query tile: a lane is a row.  64 keys at a time; P's columns [32 h, 32 h + 32) lie over S's,
        // which are read by then.  The weights are worked out with the maximum as it stands while the keys' own is
        // found; where that is more than 8 above it (seldom after the first keys) O and l are rescaled and they are
        // worked out anew.
        const uint32_t sw = ts_addr + w * kTile, ow = to_addr + w * D;
        for (int i = 0; i < it.n && part_of; ++i) {
          if (!(ok = wait_on_warp(sy, G::B_SFULL + w, (scnt[w] + i) & 1, it.t0 + i))) break;
          if (active) {
            tc_fence_after();
            const bool masked = i < full0 || i >= full1;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t s[2][32];
              tmem_ld_32x32b_x32(sw + 64 * hf, s[0]);
              tmem_ld_32x32b_x32(sw + 64 * hf + 32, s[1]);
              tmem_wait_ld();
              if (masked) {
                const int ts = (it.t0 + i) * kTile + 64 * hf;
                const int va = min(max(lo - ts, 0), 64), vb = min(max(hi - ts, 0), 64);
                const uint32_t width = (uint32_t)max(vb - va, 0);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if ((uint32_t)(32 * q + j - va) >= width) s[q][j] = 0xFF800000u;
              }
              uint32_t p[32];
              float sum;
              while (true) {
                const float base = m == -INFINITY ? 0.f : m;
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float s0 = __uint_as_float(s[j >> 4][2 * (j & 15)]), s1 = __uint_as_float(s[j >> 4][2 * (j & 15) + 1]);
                  const float2 x = weight2(s0, s1, c, -base);
                  l2[j & 1] = add2(l2[j & 1], x);
                  m4[2 * (j & 1)] = fmaxf(m4[2 * (j & 1)], s0);
                  m4[2 * (j & 1) + 1] = fmaxf(m4[2 * (j & 1) + 1], s1);
                  p[j] = pack2(x.x, x.y);
                }
                sum = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
                const bool up = mx > m + 8.f;
                if (!__any_sync(0xffffffffu, up)) break;
                const float f = up ? ex2(m - mx) : 1.f;
                if (up) m = mx;
                l *= f;
                if (i > 0 || hf > 0) {  // O has all but this half's keys (the tile's first half: wait for its product)
                  if (hf > 0 && !wait_on_warp(sy, G::B_HDONE + w, (hcnt + i) & 1, it.t0 + i)) {
                    ok = false;
                    break;
                  }
                  tc_fence_after();
#pragma unroll 1
                  for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(ow + 32 * q, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st_32x32b_x32(ow + 32 * q, o);
                  }
                }
              }
              l += sum;
              tmem_st_32x32b_x32(sw + 32 * hf, p);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_n(bars + (hf ? G::B_PHALF : G::B_PFULL) + w, quad == 0 ? 1 + idle : 1);
            }
          } else if (lane == 0) {
            arrive_n(bars + G::B_PFULL + w, 4);
            arrive_n(bars + G::B_PHALF + w, 4);
          }
          __syncwarp();
          if (!ok) break;
        }
        hcnt += it.n;
        scnt[0] += it.n;
        scnt[1] += it.n;
      } else {
        // ---- one query tile: this group's 64 keys of each tile.  The warp's 32 rows are two halves of 16 in the
        // layout of 16 x 256-bit accesses: four lanes share a row, a lane has rows l / 4 and l / 4 + 8 of a half and
        // 16 of its 64 columns.  (With 16 rows or fewer, as single tokens have, one half is taken and all lanes
        // work.)  l is a lane's own sum until the end.
        constexpr int XH = G::WROWS / 16;
        float hm[XH][2], hl[XH][2];
        int rlo[XH][2], rhi[XH][2];
        bool act[XH];
#pragma unroll
        for (int x = 0; x < XH; ++x) {
          act[x] = __any_sync(0xffffffffu, valid && (lane >> 4) == x);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            hm[x][y] = -INFINITY;
            hl[x][y] = 0.f;
            rlo[x][y] = __shfl_sync(0xffffffffu, lo, 16 * x + 8 * y + (lane >> 2)) - 64 * w;
            rhi[x][y] = __shfl_sync(0xffffffffu, hi, 16 * x + 8 * y + (lane >> 2)) - 64 * w;
          }
        }
        if (!part_of) {
          scnt[0] += (it.n + 1) >> 1;
          scnt[1] += it.n >> 1;
          dcnt += it.n;
        }
        for (int i = 0; i < it.n && part_of; ++i, ++dcnt) {
          const int b = i & 1;
          const uint32_t seq = 2 * dcnt;  // (LEAN) this tile's keys in the ring of slots; its values come next
          if (!(ok = G::LEAN ? wait_on_warp(sy, G::B_EMPTY + seq % G::NS, (seq / G::NS) & 1, it.t0 + i)
                             : wait_on_warp(sy, G::B_SFULL + b, scnt[b] & 1, it.t0 + i))) break;
          ++scnt[b];
          if (active) {
            tc_fence_after();
            const int ts = (it.t0 + i) * kTile;
            const bool masked = i < full0 || i >= full1;
#pragma unroll
            for (int x = 0; x < XH; ++x) {
              if (!act[x]) continue;
              uint32_t s[32];
              const uint32_t at = ts_addr + b * kTile + 64 * w + ((uint32_t)(16 * x) << 16);
              tmem_ld_16x256b_x8(at, s);
              tmem_wait_ld();
              if (masked) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int va = min(max(rlo[x][y] - ts, 0), 64), vb = min(max(rhi[x][y] - ts, 0), 64);
                  const int base = 2 * (lane & 3) - va;
                  const uint32_t width = (uint32_t)max(vb - va, 0);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    if ((uint32_t)(base + 8 * (k >> 1) + (k & 1)) >= width) s[4 * (k >> 1) + 2 * y + (k & 1)] = 0xFF800000u;
                }
              }
              uint32_t p[16];
              float sum[2];
              while (true) {  // as above; a row's maximum is its four lanes' where it has to be known
                float mx[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const float base = hm[x][y] == -INFINITY ? 0.f : hm[x][y];
                  float2 l2 = make_float2(0.f, 0.f);
                  float e0 = -INFINITY, e1 = -INFINITY;
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const float s0 = __uint_as_float(s[4 * k + 2 * y]), s1 = __uint_as_float(s[4 * k + 2 * y + 1]);
                    const float2 v = weight2(s0, s1, c, -base);
                    l2 = add2(l2, v);
                    e0 = fmaxf(e0, s0);
                    e1 = fmaxf(e1, s1);
                    p[2 * k + y] = pack2(v.x, v.y);
                  }
                  sum[y] = l2.x + l2.y;
                  mx[y] = fmaxf(e0, e1) * c;
                }
                if (!__any_sync(0xffffffffu, mx[0] > hm[x][0] + 8.f || mx[1] > hm[x][1] + 8.f)) break;
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 1));
                  mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 2));
                  const bool up = mx[y] > hm[x][y] + 8.f;
                  f[y] = up ? ex2(hm[x][y] - mx[y]) : 1.f;
                  if (up) hm[x][y] = mx[y];
                  hl[x][y] *= f[y];
                }
                if (i > 0) {  // O must hold the tile before
                  if (!(G::LEAN ? wait_on_warp(sy, G::B_EMPTY + (seq - 1) % G::NS, ((seq - 1) / G::NS) & 1, it.t0 + i)
                                : wait_on_warp(sy, G::B_ODONE, (dcnt - 1) & 1, it.t0 + i))) {
                    ok = false;
                    break;
                  }
                  tc_fence_after();
#pragma unroll 1
                  for (int q = 0; q < D / 64; ++q) {
                    uint32_t o[32];
                    const uint32_t oa = to_addr + ((uint32_t)(16 * x) << 16) + w * D + 64 * q;
                    tmem_ld_16x256b_x8(oa, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f[(j >> 1) & 1]);
                    tmem_st_16x256b_x8(oa, o);
                  }
                }
              }
              hl[x][0] += sum[0];
              hl[x][1] += sum[1];
              tmem_st_16x128b_x8(at, p);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0)
            arrive_n(bars + (G::LEAN ? G::B_FULL + (seq + 1) % G::NS : G::B_PSPLIT + b), quad == 0 ? 1 + idle : 1);
          if (!ok) break;
        }
        // statistics of row `lane`
#pragma unroll
        for (int x = 0; x < 2 * XH; ++x) {
          float v = hl[x >> 1][x & 1];
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          v = __shfl_sync(0xffffffffu, v, (lane & 7) * 4);
          const float u = __shfl_sync(0xffffffffu, hm[x >> 1][x & 1], (lane & 7) * 4);
          if ((lane >> 3) == x) m = u, l = v;
        }
      }
      if (!ok) break;
      // ------------------------------------------------------------------ epilogue
      const float mc = m;
      const bool mine = two || w == 0;
      // Warps without a row come here at once and wait for the whole item: 16 probes a key tile (60 us; one takes about
      // two) on top.  (Where the CTA has stopped, the warps that wait for one tile give up first and end this one.)
      const uint32_t probes = kProbes + 16 * it.n;
      if (!mine) {  // O[1] complete: the previous item's statistics have been read
        if (!(ok = wait_on_warp(sy, G::B_OFULL + 1, ocnt[1] & 1, it.t0, probes))) break;
        ++ocnt[1];
        if (lane < G::WROWS) ml[r] = make_float2(mc, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + G::B_MERGE);
        ++items;
        continue;
      }
      const bool join = !two;
      if (!(ok = wait_on_warp(sy, G::B_OFULL + w, ocnt[w] & 1, it.t0, probes))) break;
      ++ocnt[w];
      float M = mc, L = l, w0 = 1.f, w1 = 0.f;
      if (join) {
        if (!(ok = wait_on_warp(sy, G::B_OFULL + 1, ocnt[1] & 1, it.t0, probes))) break;
        if (!(ok = wait_on_warp(sy, G::B_MERGE, mcnt & 1, it.t0))) break;
        ++mcnt;
        const float2 o = ml[r];
        M = fmaxf(mc, o.x);
        const float base = M == -INFINITY ? 0.f : M;
        w0 = ex2(mc - base);
        w1 = ex2(o.x - base);
        L = w0 * l + w1 * o.y;
      }
      if (w == 0) ++ocnt[1];  // group 0 follows group 1's phases
      tc_fence_after();
      const bool whole = it.first && it.last;
      int any_bad = 0;
#pragma unroll
      for (int x = 0; x < (G::Q8 ? G::CONV : 2); ++x) any_bad |= bad[(items & 15) * 16 + x];
      const int64_t tok = it.e.tok + tk;
      const int head = it.head * a.g + r % a.g;
      const float inv = factor(L, lo < hi);
      const int tile = two ? w : 0;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (it.first ? 1 : 0);
      float4 *po = reinterpret_cast<float4 *>(a.po) + (slot * 2 + tile) * (D / 4) * kTile + r;
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
            // One bit a column: + and - infinity, both for NaN.  (A loop that is not unrolled, for its size: 32 conversions
            // in a row here cost a call of many entries 7%, though they are not reached.)
            uint32_t up = 0, down = 0;
            for (int t = it.t0; t < it.t0 + it.n; ++t) {
              const Reach rc = reach(a, it.e, t);
              if (!partly(rc)) continue;
              for (int j = rc.a; j < rc.d; ++j) {
                if (j >= rc.b && j < rc.c) continue;
                const int64_t p = (int64_t)t * kTile + j;
                const uint32_t idx = (uint32_t)p / (uint32_t)a.page_size;
                const int pg = a.table[(int64_t)it.e.seq * a.max_pages + idx];
                if (pg < 0 || pg >= a.n_pages || p < lo || p >= hi) continue;
                const int sl = (int)((uint32_t)p - idx * (uint32_t)a.page_size);
                const int64_t off = (int64_t)pg * a.s_page + (int64_t)sl * a.s_tok + (int64_t)it.head * a.s_head + 32 * q;
                const float vs = G::Q8 ? a.vs[((int64_t)pg * a.Hkv + it.head) * a.page_size + sl] : 1.f;
#pragma unroll 1
                for (int u = 0; u < 32; ++u) {
                  float v;
                  if (FMT == LA_KV_BF16) v = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.v)[off + u]);
                  else if (FMT == LA_KV_INT8) v = (float)(int8_t)a.v[off + u];
                  else v = __half2float(__half(__nv_cvt_fp8_to_halfraw(a.v[off + u], __NV_E4M3)));
                  if (G::Q8) v = __bfloat162float(__float2bfloat16_rn(v * vs));  // as the operand had it
                  if (finite_f(v)) continue;
                  if (!(v < 0.f)) up |= 1u << u;
                  if (!(v > 0.f)) down |= 1u << u;
                }
              }
            }
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              if (up >> u & 1) o[u] += INFINITY;
              if (down >> u & 1) o[u] -= INFINITY;
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
#pragma unroll
              for (int u = 0; u < 8; ++u)
                po[(8 * q + u) * kTile] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
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
      if (valid && !whole) a.pml[(slot * 2 + tile) * kTile + r] = make_float2(M, L);
      ++items;
    }
  } else if (G::Q8) {
    reg_dealloc<G::R_CONV>();
    // ---------------------------------------------------------------- conversion
    constexpr int NRr = G::NR > 0 ? G::NR : 1;
    // Work is cut into turns of two times 16 codes a lane.  D = 128 (codes under the 128-byte swizzle), an 8-row group: two
    // pairs of rows a, a ^ 5 and the other four rows, a ^ 2; eight lanes take half a row of each of a pair, which
    // spreads both their 16-byte reads and their 16-byte writes over all banks.  D = 64 (plain rows of 64 bytes): two
    // 8-row groups.  Every other four warps take the keys, the others the values: a set's waits and fences pass while
    // the other works.
    constexpr int TURNS = D == 128 ? 16 : 8, SET = G::Q8 ? G::CONV / 2 : 8;
    const int q4 = lane & 3, slab = D == 128 ? (lane >> 3) & 1 : 0, cw = warp - 12;
    const int kvi = (cw >> 2) & 1, ci = (cw & 3) + 4 * (cw >> 3);
    const int r8 = D == 128 ? (lane >> 4) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    const int soff = r8 * D + (D == 128 ? ((slab * 4 + q4) ^ r8) : q4) * 16;
    const int doff = slab * G::SLAB + r8 * 128 + ((2 * q4) ^ r8) * 16;  // the second 16 bytes: at ^ 16
    int rs = kvi, os = kvi;
    uint32_t rph = 0, oph = 1, items = 0;
    bool ok = true;
    while (ok && walk.next(a, it)) {
      if (lane == 0) bad[(items & 15) * 16 + cw] = 0;
      __syncwarp();
      // Even shares beside two full softmax groups.  When the rows are few all of the softmax runs on the first quarter
      // of the SM (the first rows belong to its warps): the conversion warps there take an eighth together.  (Even
      // shares for few rows too: no slower in pages of 64, slower in pages of 16, where the producer lives there too.)
      const bool even = D == 64 || it.e.ntok * a.g > G::WROWS;
      const int first = even ? ci * (TURNS / SET) : ((SET == 8 ? 0xDB917520u : 0xC720u) >> (4 * ci)) & 15;
      const int last = first + (even ? TURNS / SET : ((SET == 8 ? 0x32212231u : 0x4552u) >> (4 * ci)) & 15);
      for (int i = 0; i < it.n && ok; ++i) {
        {
          if (!(ok = wait_on_warp(sy, G::B_RFULL + rs, rph, it.t0 + i))) break;
          if (!(ok = wait_on_warp(sy, G::B_EMPTY + os, oph, it.t0 + i))) break;
          const uint32_t src = smem_u32(raw_stage(rs)) + soff, dst = smem_u32(op_slot(os)) + doff;
          const float *ss = sc + rs * kTile + r8;
          int found = 0;
#pragma unroll 1
          for (int u = first; u < last; ++u) {
            uint4 w[2];
            float f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              w[x] = lds16(D == 128 ? (src + u * 1024) ^ (x * 0x120) : src + u * 1024 + x * 512);
              f[x] = D == 128 ? *reinterpret_cast<const float *>(reinterpret_cast<uintptr_t>(ss + u * 8) ^ (x * 8))
                              : ss[u * 16 + x * 8];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint4 o0, o1;
              convert16<FMT>(w[x], f[x], o0, o1);
              const uint32_t at = D == 128 ? (dst + u * 1024) ^ (x * 0x120) : dst + u * 2048 + x * 1024;
              sts16(at, o0);
              sts16(at ^ 16, o1);
            }
          }
          // Values in rows that not every token sees (keys there are masked as scores): rows that none sees become zeros, and
          // what is not finite in the others is taken out, products of codes and scales past the range too.  A second pass
          // over what this lane has written: in the loop above it costs the tiles that need nothing of it.
          if (kvi) {
            const Reach rc = reach(a, it.e, it.t0 + i);
            if (partly(rc)) {
#pragma unroll 1
              for (int u = 2 * first; u < 2 * last; ++u) {
                const int x = u & 1, row = D == 128 ? (u >> 1) * 8 + (r8 ^ (x * 2)) : u * 8 + r8;
                if (row >= rc.b && row < rc.c) continue;
                const uint32_t at = D == 128 ? (dst + (u >> 1) * 1024) ^ (x * 0x120) : dst + u * 1024;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  uint4 o = make_uint4(0, 0, 0, 0);
                  if (row >= rc.a && row < rc.d) {
                    o = lds16(at ^ (16 * y));
                    found |= take_out(o);
                  }
                  sts16(at ^ (16 * y), o);
                }
              }
            }
          }
          if (found) bad[(items & 15) * 16 + cw] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bars + G::B_FULL + os);
            mbar_arrive(bars + G::B_REMPTY + rs);
          }
          if ((rs += 2) >= NRr) rs = kvi, rph ^= 1;
          if ((os += 2) >= G::NS) os = kvi, oph ^= 1;
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

// ------------------------------------------------------------------ joining
// Blocks (c, .) join the entry that the border before CTA c cuts, if that is its first cut.  A thread takes eight
// columns of a row; a warp's rows lie side by side.
constexpr int kJoinThreads = 512;
static_assert(kPagedCtas <= kJoinThreads, "a thread looks a part up");
template <int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) pa_join_kernel(const PaArgs a) {
  __shared__ int parts[kJoinThreads], members[kJoinThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, tid = threadIdx.x;
  const CtaWork cw = a.work[c];
  if (c == 0 || cw.count <= 0 || cw.off == 0) return;
  const Entry e = a.ent[cw.entry];
  const int64_t t0 = cw.start - cw.off, t1 = t0 + e.cnt;  // the entry's tiles
  CtaWork x;
  x.count = 0;
  if (tid < a.G) x = a.work[tid];
  const bool in = x.count > 0 && x.start < t1 && x.start + x.count > t0;
  const uint32_t mask = __ballot_sync(0xffffffffu, in);
  if ((tid & 31) == 0) members[tid >> 5] = __popc(mask);
  __syncthreads();
  int rank = __popc(mask & ((1u << (tid & 31)) - 1)), nparts = 0;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < tid >> 5) rank += members[i];
    nparts += members[i];
  }
  if (in) parts[rank] = tid;
  __syncthreads();
  if (parts[1] != c) return;  // cut before
  constexpr int ROWS = NQ == 1 ? 64 : 128, CG = D / 8;
  const bool two = NQ == 2 && e.ntok > a.tpt;
  for (int task = blockIdx.y * kJoinThreads + tid; task < (two ? 2 : 1) * ROWS * CG; task += gridDim.y * kJoinThreads) {
    const int r = task % ROWS, cg = (task / ROWS) % CG, tile = task / (ROWS * CG);
    const int tk = tile * a.tpt + r / a.g;
    if (r >= a.g * a.tpt || tk >= e.ntok) continue;
    auto part = [&](int x) -> int64_t { return (2 * (int64_t)parts[x] + (x == 0 ? 1 : 0)) * 2 + tile; };
    float m = -INFINITY;
#pragma unroll 8
    for (int x = 0; x < nparts; ++x) m = fmaxf(m, a.pml[part(x) * kTile + r].x);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int x = 0; x < nparts; ++x) {
      const int64_t at = part(x);
      const float2 st = a.pml[at * kTile + r];
      const float4 *src = reinterpret_cast<const float4 *>(a.po) + (at * (D / 4) + 2 * cg) * kTile + r;
      const float4 u = src[0], v = src[kTile];
      const float wt = ex2(st.x - base);
      l = fmaf(wt, st.y, l);
      o[0] = fmaf(wt, u.x, o[0]), o[1] = fmaf(wt, u.y, o[1]), o[2] = fmaf(wt, u.z, o[2]), o[3] = fmaf(wt, u.w, o[3]);
      o[4] = fmaf(wt, v.x, o[4]), o[5] = fmaf(wt, v.y, o[5]), o[6] = fmaf(wt, v.z, o[6]), o[7] = fmaf(wt, v.w, o[7]);
    }
    int lo, hi;
    sees(a, e, tk, lo, hi);
    const float inv = factor(l, lo < hi);
    const int64_t tok = e.tok + tk;
    const int head = cw.head * a.g + r % a.g;
    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + (int64_t)e.b * a.o_sb + tok * a.o_st +
                               (int64_t)head * a.o_sh + 8 * cg) =
        make_uint4(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv), pack2(o[4] * inv, o[5] * inv),
                   pack2(o[6] * inv, o[7] * inv));
    if (a.lse && cg == 0) a.lse[((int64_t)e.b * a.T + tok) * a.H + head] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------ host side
int tokens_per_tile(int g, int tiles) { return (tiles == 1 ? 64 : kTile) / g; }

int box_rows(int64_t page_size) {  // largest power of two that divides the page, up to a tile
  int b = 1;
  while (b < kTile && page_size % (2 * b) == 0) b *= 2;
  return b;
}

// Query tiles of an entry: one of 64 rows where the sequences have no more rows each on average (single tokens, drafts:
// the two softmax groups take half of each key tile, and shared memory goes to more of those), else two of 128 (they
// share the keys).  Measured with 64 rows and with 128, 16 heads over 4 of 128:
//   256 single tokens over up to 8192    bf16 334 and 360 us, e4m3 349 and 475, int8 394 and 524
//   2048 tokens over 16384               bf16 456 and 247 us, e4m3 569 and 350, int8 668 and 367: a CTA that reads 64
//                                        rows' worth of keys does a quarter of the products for them
// The average decides for a whole call, since lengths are known to the device only.  Calls of both kinds:
//   256 single tokens, a piece of 2048   (64 is taken) bf16 434 and 454 us, e4m3 547 and 606, int8 625 and 646; as two
//                                        calls 444, 498 and 547
//   44 single tokens, 4 pieces           (128 is taken) bf16 174 and 138 us, e4m3 203 and 182, int8 223 and 193; as two
//   of 200 to 512, 20 heads over 4       calls 147, 175 and 191
int query_tiles(int64_t B, int64_t T, int64_t n_seqs, bool packed, int g) {
  const int64_t tokens = packed ? T : B * T;
  return g <= 64 && tokens <= n_seqs * tokens_per_tile(g, 1) ? 1 : 2;
}

int64_t max_entries(int64_t B, int64_t T, int64_t n_seqs, bool packed, int g) {
  const int tiles = query_tiles(B, T, n_seqs, packed, g);
  const int64_t per = (int64_t)tiles * tokens_per_tile(g, tiles);
  return packed ? T / per + n_seqs : B * ((T + per - 1) / per);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  size_t seq_ent, ent, pre, work, po, pml, bytes;
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
  p.pre = take((size_t)e_max * 16);
  p.work = take((size_t)G * sizeof(CtaWork));
  p.pml = take((size_t)G * 4 * kTile * 8);
  p.po = take((size_t)G * 4 * kTile * D * 4);
  p.bytes = at;
  return p;
}

template <int D, int FMT, int NQ>
cudaError_t launch_one(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const PaArgs &a,
                       cudaStream_t stream) {
  using G = PaCfg<D, FMT, NQ>;
  auto kern = pa_kernel<D, FMT, NQ>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  pa_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.G);
  cfg.blockDim = dim3(G::THREADS);
  cfg.dynamicSmemBytes = G::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3(a.G, NQ * (NQ == 1 ? 64 : 128) * (D / 8) / kJoinThreads);  // a task a thread
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, pa_join_kernel<D, NQ>, a);
}

template <int D, int NQ>
cudaError_t launch_format(int format, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                          const PaArgs &a, cudaStream_t stream) {
  if (format == LA_KV_E4M3) return launch_one<D, LA_KV_E4M3, NQ>(mq, mk, mv, a, stream);
  if (format == LA_KV_INT8) return launch_one<D, LA_KV_INT8, NQ>(mq, mk, mv, a, stream);
  return launch_one<D, LA_KV_BF16, NQ>(mq, mk, mv, a, stream);
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

// (size_t)-1 where the problem is too large: the plan adds two entry numbers in 32 bits, and multiplies the cost of all
// entries (below 2^26 each: 2^24 key tiles, three for each) by the cache heads in 64.
size_t pa_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t D, int64_t n_seqs, bool packed, int64_t H_kv, int G) {
  const int64_t e = max_entries(B, T, n_seqs, packed, (int)(H / H_kv));
  if (e > (int64_t)1 << 30 || e > ((int64_t)1 << 37) / H_kv) return (size_t)-1;
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
  const int tiles = query_tiles(a.B, a.T, a.n_seqs, a.cu_seqlens != nullptr, g);
  p.tpt = tokens_per_tile(g, tiles);
  p.per = p.tpt * tiles;
  p.Hkv = a.c.H;
  p.H = a.H;
  p.window = a.window;
  p.e_max = (int)max_entries(a.B, a.T, a.n_seqs, a.cu_seqlens != nullptr, g);
  p.G = G;
  p.test_stop = a.test_wait_timeout;
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
  if (tiles == 1)
    return D == 64 ? launch_format<64, 1>(a.c.format, mq, mk, mv, p, stream)
                   : launch_format<128, 1>(a.c.format, mq, mk, mv, p, stream);
  return D == 64 ? launch_format<64, 2>(a.c.format, mq, mk, mv, p, stream)
                 : launch_format<128, 2>(a.c.format, mq, mk, mv, p, stream);
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

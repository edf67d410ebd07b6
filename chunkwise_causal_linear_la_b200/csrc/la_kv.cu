// la_kv.cu -- rows into and out of a paged cache (la_kv_write, la_kv_read).
//
// A row is the D values of one token and head.  In the 8-bit formats it is kept
// as codes with one power-of-two scale s = 2^e, the smallest with
// max |x| <= qmax s and e >= -126.  With max |x| = m 2^E and qmax = m_q 2^E_q
// (m, m_q in [1, 2)) that is e = E - E_q + (m > m_q): one comparison of mantissa
// fields, no logarithm.  x / s is a product with 2^-e, exact but for subnormal
// results (which round to code 0 or the grid's smallest steps as the exact
// quotient would), so a code is the correctly rounded quotient.
//
// Both kernels move every byte once and are bound by memory: D / 8 threads share a
// row, each with 16 bytes of its dense side, keys and values of one row in one
// thread so that two loads are in flight, and the row's maximum goes through
// shuffles.  Measured for 16 sequences of up to 16384 tokens, 8 heads of 128, against
// the rate of a plain copy (one call by itself; an 8-bit read among others 176 us):
//   bf16 rows: bf16 written 203 us (94%), read 206 (93%); e4m3 212 (68%), 179 (81%); int8 212 (68%), 173 (84%)
//   f32 rows:  bf16 written 302 us (95%), read 322 (89%); e4m3 260 (93%), 281 (86%); int8 260 (92%), 282 (85%)
// 8-bit reads and writes of bf16 rows leave both memory (49% in a read of 64 prompts,
// under the profiler) and issue slots (65%) free: a block's turns follow one another,
// loads, maxima, stores.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "la_common.cuh"
#include "la_kv.cuh"

namespace la {
namespace {

using namespace kv;

constexpr int kKvThreads = 256;

template <typename T>
__device__ __forceinline__ void load_row8(const T *p, float (&f)[8]) {
  if (sizeof(T) == 2) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&p);
}

template <typename T>
__device__ __forceinline__ void store_row8(T *p, const float (&f)[8]) {
  if (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7])));
  } else {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
}

// Exponent e of the row's scale from the bits of max |x| (a finite, non-negative
// float).  Subnormal maxima (exponent field 0) land below the clamp either way.
template <int FMT>
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  constexpr uint32_t kQmax = FMT == LA_KV_E4M3 ? 0x43E00000u /* 448 */ : 0x42FE0000u /* 127 */;
  const int e = (int)(amax_bits >> 23) - (int)(kQmax >> 23) + ((amax_bits & 0x7FFFFFu) > (kQmax & 0x7FFFFFu));
  return max(e, -126);
}

// Eight codes of x * 2^-e.  2^-e lies in [2^-122, 2^126]: normal numbers.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FMT == LA_KV_E4M3) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h] * inv, f[4 * h + 1] * inv), __NV_SATFINITE,
                                                   __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h + 2] * inv, f[4 * h + 3] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | hi << 16;
    } else {
      // x 2^-e is exact, so adding 1.5 2^23 rounds it once, to nearest even, into the sum's low byte (|x 2^-e| <= 127).
      // (A conversion instruction would run at an eighth of the rate.)
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(fmaf(f[4 * h + i], inv, 12582912.f));
      const uint32_t b = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
      w[h] = b;
    }
  }
  return make_uint2(w[0], w[1]);
}

// Rows whose max |x| rounds to a code whose value is 2^128, beyond fp32 (from 248 2^120 on, and above 127 2^121; in bits),
// have the scale 2^kTopExp: there e4m3's 256 becomes 240, int8's 64 becomes 63.
template <int FMT>
constexpr uint32_t kTopBits = FMT == LA_KV_E4M3 ? 0x7F780000u : 0x7F7E0001u;
template <int FMT>
constexpr int kTopExp = FMT == LA_KV_E4M3 ? 120 : 122;
template <int FMT>
__device__ __forceinline__ uint32_t keep_in_range(uint32_t w) {
  if (FMT == LA_KV_E4M3) return w - (__vcmpeq4(w & 0x7F7F7F7Fu, 0x78787878u) & 0x01010101u);
  return __vmins4(__vmaxs4(w, 0xC1C1C1C1u /* -63 */), 0x3F3F3F3Fu);
}

// Where a token of the batch stands.  A block's threads look its few tokens up once (a search among the sequences and
// a table entry, each a chain of loads) and leave them in shared memory for its rows.
struct Place {
  int64_t k, v;   // element offsets of its first head's dense rows
  int64_t slot;   // page * page_size + slot in it, or -1: no slot
  int32_t in;     // belongs to a sequence
};

template <bool WRITE>
__device__ __forceinline__ void places(const KvMoveArgs &a, uint32_t first, uint32_t last, Place *tab) {
  for (uint32_t t = first + threadIdx.x; t <= last; t += kKvThreads) {
    Place p;
    int64_t n, i, L;
    p.slot = -1;
    p.k = p.v = 0;
    p.in = locate(a.cu_seqlens, a.n_seqs, a.T, t, n, i, L);
    if (p.in) {
      const int64_t tb = a.cu_seqlens ? 0 : n, tt = a.cu_seqlens ? (int64_t)t : i;
      p.k = tb * a.k.sb + tt * a.k.st;
      p.v = tb * a.v.sb + tt * a.v.st;
      const int64_t at = WRITE ? (int64_t)a.pos[n] - L + i : (a.pos ? (int64_t)a.pos[n] : 0) + i;
      const int64_t page = page_of(a.c, n, at);
      if (page >= 0) p.slot = page * a.c.page_size + slot_of(a.c, at);
    }
    tab[t - first] = p;
  }
  __syncthreads();
}

// A row of a block: its token's place, head, cache offset and scale index.
struct Row {
  int64_t k, v, off, scale;
  bool in, live;
};
__device__ __forceinline__ Row row_at(const KvMoveArgs &a, const Place *tab, uint32_t first, uint32_t row, uint32_t rows) {
  Row r;
  r.k = r.v = r.off = r.scale = 0;
  r.in = r.live = false;
  if (row >= rows) return r;
  const uint32_t t = row / (uint32_t)a.c.H, h = row - t * (uint32_t)a.c.H;
  const Place p = tab[t - first];
  r.in = p.in != 0;
  r.k = p.k + (int64_t)h * a.k.sh;
  r.v = p.v + (int64_t)h * a.v.sh;
  if (p.slot >= 0) {
    const int64_t page = (uint64_t)p.slot >> 32 ? p.slot / a.c.page_size : (int64_t)((uint32_t)p.slot / (uint32_t)a.c.page_size);
    const int64_t slot = p.slot - page * a.c.page_size;
    r.live = true;
    r.off = page * a.c.s_page + slot * a.c.s_tok + (int64_t)h * a.c.s_head;
    r.scale = (page * a.c.H + h) * (int64_t)a.c.page_size + slot;
  }
  return r;
}

// A block takes `turns` times its rows, one after the other; eight blocks share an SM and keep its loads under way.
template <typename T, int FMT>
__global__ void __launch_bounds__(kKvThreads, 8) kv_write_kernel(const KvMoveArgs a, int turns) {
  extern __shared__ Place tab[];
  const int lpr = a.c.D >> 3;  // threads of a row: a power of two <= 32
  const int part = (int)(threadIdx.x % lpr);
  const uint32_t rpb = kKvThreads / lpr, rows = (uint32_t)(a.B * a.T * a.c.H);
  const uint32_t begin = blockIdx.x * rpb * turns, end = min(begin + rpb * turns, rows);
  const uint32_t first = begin / (uint32_t)a.c.H;
  places<true>(a, first, (end - 1) / (uint32_t)a.c.H, tab);
#pragma unroll 1
  for (uint32_t row = begin + threadIdx.x / lpr; row - threadIdx.x / lpr < end; row += rpb) {
    const Row p = row_at(a, tab, first, row, end);
    float x[2][8];
    if (p.live) {
      load_row8((const T *)a.k.data + p.k + 8 * part, x[0]);
      load_row8((const T *)a.v.data + p.v + 8 * part, x[1]);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) x[0][u] = x[1][u] = 0.f;
    }
    if (FMT == LA_KV_BF16) {
      if (p.live) {
#pragma unroll
        for (int kvi = 0; kvi < 2; ++kvi)
          *reinterpret_cast<uint4 *>((kvi ? a.c.v : a.c.k) + 2 * (p.off + 8 * part)) =
              make_uint4(bf2(x[kvi][0], x[kvi][1]), bf2(x[kvi][2], x[kvi][3]), bf2(x[kvi][4], x[kvi][5]),
                         bf2(x[kvi][6], x[kvi][7]));
      }
      continue;
    }
    // magnitudes compare as unsigned bit patterns; infinities and NaN come out on top
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int kvi = 0; kvi < 2; ++kvi)
#pragma unroll
      for (int u = 0; u < 8; ++u) m[kvi] = max(m[kvi], __float_as_uint(x[kvi][u]) & 0x7FFFFFFFu);
    if (sizeof(T) == 2) {  // bf16 magnitudes fill 16 bits: both rows' maxima in one word
      uint32_t both = (m[1] & 0xFFFF0000u) | (m[0] >> 16);
      for (int o = 1; o < lpr; o <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o));
      m[0] = both << 16;
      m[1] = both & 0xFFFF0000u;
    } else {
      for (int o = 1; o < lpr; o <<= 1) {
        m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        m[1] = max(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
      }
    }
    if (p.live) {
#pragma unroll
      for (int kvi = 0; kvi < 2; ++kvi) {
        uint2 code;
        float scale;
        if (m[kvi] < kTopBits<FMT>) {
          const int e = scale_exp<FMT>(m[kvi]);
          code = encode8<FMT>(x[kvi], __uint_as_float((uint32_t)(127 - e) << 23));
          scale = __uint_as_float((uint32_t)(127 + e) << 23);
        } else if (m[kvi] < 0x7F800000u) {
          code = encode8<FMT>(x[kvi], __uint_as_float((uint32_t)(127 - kTopExp<FMT>) << 23));
          code = make_uint2(keep_in_range<FMT>(code.x), keep_in_range<FMT>(code.y));
          scale = __uint_as_float((uint32_t)(127 + kTopExp<FMT>) << 23);
        } else {  // an infinity or a NaN in the row
          code = make_uint2(0, 0);
          scale = __uint_as_float(0x7FC00000u);
        }
        *reinterpret_cast<uint2 *>((kvi ? a.c.v : a.c.k) + p.off + 8 * part) = code;
        if (part == 0) (kvi ? a.c.vs : a.c.ks)[p.scale] = scale;
      }
    }
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kKvThreads, 8) kv_read_kernel(const KvMoveArgs a, int turns) {
  extern __shared__ Place tab[];
  const int lpr = a.c.D >> 3;
  const int part = (int)(threadIdx.x % lpr);
  const uint32_t rpb = kKvThreads / lpr, rows = (uint32_t)(a.B * a.T * a.c.H);
  const uint32_t begin = blockIdx.x * rpb * turns, end = min(begin + rpb * turns, rows);
  const uint32_t first = begin / (uint32_t)a.c.H;
  places<false>(a, first, (end - 1) / (uint32_t)a.c.H, tab);
#pragma unroll 1
  for (uint32_t row = begin + threadIdx.x / lpr; row < end; row += rpb) {
    const Row p = row_at(a, tab, first, row, end);
    if (!p.in) continue;
    float x[2][8];
    if (p.live) {
      load8<FMT>(a.c.k + elem_bytes(FMT) * (p.off + 8 * part), x[0]);
      load8<FMT>(a.c.v + elem_bytes(FMT) * (p.off + 8 * part), x[1]);
      if (FMT != LA_KV_BF16) {
        const float ks = a.c.ks[p.scale], vs = a.c.vs[p.scale];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[0][u] *= ks, x[1][u] *= vs;
      }
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) x[0][u] = x[1][u] = 0.f;
    }
    store_row8((T *)a.k.data + p.k + 8 * part, x[0]);
    store_row8((T *)a.v.data + p.v + 8 * part, x[1]);
  }
}

// Eight turns a block where that still leaves eight blocks an SM, else one: a block's look-ups are a chain of loads
// (with one turn large calls reach 55% of the copy rate, with eight 67 - 94%), and small calls need all SMs.
template <template <typename, int> class K>
cudaError_t launch(const KvMoveArgs &a, cudaStream_t stream) {
  const int64_t rows = a.B * a.T * a.c.H;
  const int64_t rpb = kKvThreads / (a.c.D / 8);
  const int turns = rows >= rpb * 8 * 8 * 148 ? 8 : 1;
  const unsigned grid = (unsigned)((rows + rpb * turns - 1) / (rpb * turns));
  const size_t smem = (size_t)((rpb * turns - 1) / a.c.H + 2) * sizeof(Place);
  const bool bf = a.dtype == LA_BF16;
  switch (a.c.format) {
    case LA_KV_E4M3:
      bf ? K<__nv_bfloat16, LA_KV_E4M3>::go(a, grid, turns, smem, stream) : K<float, LA_KV_E4M3>::go(a, grid, turns, smem, stream);
      break;
    case LA_KV_INT8:
      bf ? K<__nv_bfloat16, LA_KV_INT8>::go(a, grid, turns, smem, stream) : K<float, LA_KV_INT8>::go(a, grid, turns, smem, stream);
      break;
    default:
      bf ? K<__nv_bfloat16, LA_KV_BF16>::go(a, grid, turns, smem, stream) : K<float, LA_KV_BF16>::go(a, grid, turns, smem, stream);
  }
  return cudaGetLastError();
}
template <typename T, int FMT>
struct Write {
  static void go(const KvMoveArgs &a, unsigned grid, int turns, size_t smem, cudaStream_t st) {
    kv_write_kernel<T, FMT><<<grid, kKvThreads, smem, st>>>(a, turns);
  }
};
template <typename T, int FMT>
struct Read {
  static void go(const KvMoveArgs &a, unsigned grid, int turns, size_t smem, cudaStream_t st) {
    kv_read_kernel<T, FMT><<<grid, kKvThreads, smem, st>>>(a, turns);
  }
};

}  // namespace

cudaError_t launch_kv_write(const KvMoveArgs &a, cudaStream_t stream) { return launch<Write>(a, stream); }
cudaError_t launch_kv_read(const KvMoveArgs &a, cudaStream_t stream) { return launch<Read>(a, stream); }

}  // namespace la

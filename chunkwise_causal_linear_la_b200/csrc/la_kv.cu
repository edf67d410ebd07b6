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
// shuffles.
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
      uint32_t b = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) b |= ((uint32_t)__float2int_rn(f[4 * h + i] * inv) & 0xFFu) << (8 * i);
      w[h] = b;
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvMoveArgs a) {
  const int lpr = a.c.D >> 3;  // threads of a row: a power of two <= 32
  const uint32_t gid = blockIdx.x * (uint32_t)kKvThreads + threadIdx.x;
  const uint32_t row = gid / lpr;
  const int part = (int)(gid % lpr);
  const uint32_t rows = (uint32_t)(a.B * a.T * a.c.H);
  const bool in = row < rows;
  const int64_t t = in ? row / (uint32_t)a.c.H : 0;
  const int h = in ? (int)(row % (uint32_t)a.c.H) : 0;
  int64_t n = 0, i = 0, L = 0;
  bool live = in && locate(a.cu_seqlens, a.n_seqs, a.T, t, n, i, L);
  const int64_t p = live ? (int64_t)a.pos[n] - L + i : -1;
  const int64_t page = live ? page_of(a.c, n, p) : -1;
  live = page >= 0;
  float x[2][8];
  if (live) {
    const int64_t tb = a.cu_seqlens ? 0 : n, tt = a.cu_seqlens ? t : i;
    load_row8((const T *)a.k.data + tb * a.k.sb + tt * a.k.st + h * a.k.sh + 8 * part, x[0]);
    load_row8((const T *)a.v.data + tb * a.v.sb + tt * a.v.st + h * a.v.sh + 8 * part, x[1]);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) x[0][u] = x[1][u] = 0.f;
  }
  const int slot = live ? slot_of(a.c, p) : 0;
  const int64_t off = live ? page * a.c.s_page + (int64_t)slot * a.c.s_tok + (int64_t)h * a.c.s_head + 8 * part : 0;
#pragma unroll
  for (int kvi = 0; kvi < 2; ++kvi) {
    uint8_t *dst = kvi ? a.c.v : a.c.k;
    if (FMT == LA_KV_BF16) {
      if (live)
        *reinterpret_cast<uint4 *>(dst + 2 * off) =
            make_uint4(bf2(x[kvi][0], x[kvi][1]), bf2(x[kvi][2], x[kvi][3]), bf2(x[kvi][4], x[kvi][5]),
                       bf2(x[kvi][6], x[kvi][7]));
      continue;
    }
    // magnitudes compare as unsigned bit patterns; infinities and NaN come out on top
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(x[kvi][u]) & 0x7FFFFFFFu);
    for (int o = 1; o < lpr; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (live) {
      const bool finite = m < 0x7F800000u;
      const int e = finite ? scale_exp<FMT>(m) : 0;
      const uint2 code = finite ? encode8<FMT>(x[kvi], __uint_as_float((uint32_t)(127 - e) << 23)) : make_uint2(0, 0);
      *reinterpret_cast<uint2 *>(dst + off) = code;
      if (part == 0)
        (kvi ? a.c.vs : a.c.ks)[(page * a.c.H + h) * (int64_t)a.c.page_size + slot] =
            finite ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x7FC00000u);
    }
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvMoveArgs a) {
  const int lpr = a.c.D >> 3;
  const uint32_t gid = blockIdx.x * (uint32_t)kKvThreads + threadIdx.x;
  const uint32_t row = gid / lpr;
  const int part = (int)(gid % lpr);
  if (row >= (uint32_t)(a.B * a.T * a.c.H)) return;
  const int64_t t = row / (uint32_t)a.c.H;
  const int h = (int)(row % (uint32_t)a.c.H);
  int64_t n = 0, i = 0, L = 0;
  if (!locate(a.cu_seqlens, a.n_seqs, a.T, t, n, i, L)) return;
  const int64_t p = (a.pos ? (int64_t)a.pos[n] : 0) + i;
  const int64_t page = page_of(a.c, n, p);
  const int64_t tb = a.cu_seqlens ? 0 : n, tt = a.cu_seqlens ? t : i;
  float x[2][8];
#pragma unroll
  for (int kvi = 0; kvi < 2; ++kvi)
#pragma unroll
    for (int u = 0; u < 8; ++u) x[kvi][u] = 0.f;
  if (page >= 0) {
    const int slot = slot_of(a.c, p);
    const int64_t off = page * a.c.s_page + (int64_t)slot * a.c.s_tok + (int64_t)h * a.c.s_head + 8 * part;
    load8<FMT>(a.c.k + elem_bytes(FMT) * off, x[0]);
    load8<FMT>(a.c.v + elem_bytes(FMT) * off, x[1]);
    if (FMT != LA_KV_BF16) {
      const int64_t so = (page * a.c.H + h) * (int64_t)a.c.page_size + slot;
      const float ks = a.c.ks[so], vs = a.c.vs[so];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[0][u] *= ks, x[1][u] *= vs;
    }
  }
  store_row8((T *)a.k.data + tb * a.k.sb + tt * a.k.st + h * a.k.sh + 8 * part, x[0]);
  store_row8((T *)a.v.data + tb * a.v.sb + tt * a.v.st + h * a.v.sh + 8 * part, x[1]);
}

unsigned kv_blocks(const KvMoveArgs &a) {
  const int64_t threads = a.B * a.T * a.c.H * (a.c.D / 8);
  return (unsigned)((threads + kKvThreads - 1) / kKvThreads);
}

}  // namespace

cudaError_t launch_kv_write(const KvMoveArgs &a, cudaStream_t stream) {
  const unsigned grid = kv_blocks(a);
#define LA_KV_LAUNCH(K, FMT)                                                       \
  do {                                                                             \
    if (a.dtype == LA_BF16) K<__nv_bfloat16, FMT><<<grid, kKvThreads, 0, stream>>>(a); \
    else K<float, FMT><<<grid, kKvThreads, 0, stream>>>(a);                        \
  } while (0)
  if (a.c.format == LA_KV_E4M3) LA_KV_LAUNCH(kv_write_kernel, LA_KV_E4M3);
  else if (a.c.format == LA_KV_INT8) LA_KV_LAUNCH(kv_write_kernel, LA_KV_INT8);
  else LA_KV_LAUNCH(kv_write_kernel, LA_KV_BF16);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvMoveArgs &a, cudaStream_t stream) {
  const unsigned grid = kv_blocks(a);
  if (a.c.format == LA_KV_E4M3) LA_KV_LAUNCH(kv_read_kernel, LA_KV_E4M3);
  else if (a.c.format == LA_KV_INT8) LA_KV_LAUNCH(kv_read_kernel, LA_KV_INT8);
  else LA_KV_LAUNCH(kv_read_kernel, LA_KV_BF16);
#undef LA_KV_LAUNCH
  return cudaGetLastError();
}

}  // namespace la

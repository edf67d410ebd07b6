// la_kv.cuh -- what the paged-cache kernels share: where a token of the batch
// belongs, where a position lives, and how eight values of a row are read.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "la_internal.h"

namespace la {
namespace kv {

// Sequence n and index i (of L) of global token t of the batch: dense batches by
// division, packed ones by a search for the last cu[n] <= t.  False for a token that
// belongs to no sequence.  Whatever cu holds, n stays inside [0, n_seqs).
__device__ __forceinline__ bool locate(const int32_t *cu, int64_t n_seqs, int64_t T, int64_t t, int64_t &n,
                                       int64_t &i, int64_t &L) {
  if (!cu) {
    n = t / T;
    i = t - n * T;
    L = T;
    return true;
  }
  int64_t lo = 0, hi = n_seqs;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if ((int64_t)cu[mid] <= t) lo = mid; else hi = mid;
  }
  const int64_t a = cu[lo], b = cu[lo + 1];
  n = lo;
  i = t - a;
  L = b - a;
  return t >= a && t < b;
}

// Page of position p of sequence n, or -1 where there is none.
__device__ __forceinline__ int64_t page_of(const KvView &c, int64_t n, int64_t p) {
  if (p < 0) return -1;
  const int64_t at = p < (int64_t)1 << 31 ? (int64_t)((uint32_t)p / (uint32_t)c.page_size) : p / c.page_size;
  if (at >= c.max_pages) return -1;
  const int64_t pg = c.table[n * c.max_pages + at];
  return pg >= 0 && pg < c.n_pages ? pg : -1;
}

__device__ __forceinline__ int slot_of(const KvView &c, int64_t p) {
  return p < (int64_t)1 << 31 ? (int)((uint32_t)p % (uint32_t)c.page_size) : (int)(p % c.page_size);
}

// Eight consecutive values of a row in its format, as fp32, without the scale.
template <int FMT>
__device__ __forceinline__ void load8(const uint8_t *p, float (&f)[8]) {
  if (FMT == LA_KV_BF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xFF;
      if (FMT == LA_KV_INT8)
        f[i] = (float)(int8_t)b;
      else
        f[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
    }
  }
}

__host__ __device__ constexpr int elem_bytes(int fmt) { return fmt == LA_KV_BF16 ? 2 : 1; }

}  // namespace kv
}  // namespace la

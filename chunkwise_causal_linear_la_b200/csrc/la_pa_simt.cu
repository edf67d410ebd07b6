// la_pa_simt.cu -- attention of new tokens over a paged cache on the CUDA cores
// (la_paged_attn for f32, head dims and pages off the tensor cores, LA_FLAG_SIMT).
//
// One CTA of four warps per (token, query head).  With s_j = scale q . k_j over the
// positions the query sees, each warp takes every fourth block of 32 keys and keeps
// a running maximum m, the sum l of e^(s_j - m) and o = sum_j e^(s_j - m) v_j; the
// four are joined at the end by the weights e^(m_w - max m).  A lane scores a key of
// its own (the row is one or a few 32-byte sectors), then the lanes turn to the
// value columns and each key's weight goes round by a shuffle.  Positions that are
// not seen are not read.  All arithmetic is fp32; the keys' reads are not
// coalesced, which bounds it (2048 tokens over 16384, 16 heads of 128 over 4: 86 ms,
// 3 TFLOP/s; the tensor cores' form takes 0.25): it is the form that is right for every
// shape, not the one that serves.
#include <cuda_bf16.h>
#include <math.h>

#include "la_common.cuh"
#include "la_kv.cuh"

namespace la {
namespace {

using namespace kv;

constexpr int kWarps = 4;

template <typename T, int FMT>
__global__ void __launch_bounds__(32 * kWarps) paged_simt_kernel(const PagedArgs a) {
  __shared__ float sq[256];
  __shared__ float so[kWarps][256];
  __shared__ float sm[kWarps], sl[kWarps];
  const int D = a.c.D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x / (unsigned)a.H;
  const int h = (int)(blockIdx.x % (unsigned)a.H);
  const int hk = h / (a.H / a.c.H);
  int64_t n, i, L;
  if (!locate(a.cu_seqlens, a.n_seqs, a.T, t, n, i, L)) return;
  const int64_t tb = a.cu_seqlens ? 0 : n, tt = a.cu_seqlens ? t : i;
  const T *q = (const T *)a.q.data + tb * a.q.sb + tt * a.q.st + h * a.q.sh;
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) sq[d] = to_f32<T>(q[d]);
  __syncthreads();
  const int64_t p = (int64_t)a.kv_len[n] - L + i;
  const int64_t cap = a.c.max_pages * (int64_t)a.c.page_size;
  const int64_t j1 = min(p + 1, cap), j0 = a.window > 0 ? max((int64_t)0, p - a.window + 1) : 0;

  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) o[u] = 0.f;
  for (int64_t jb = j0 + 32 * warp; jb < j1; jb += 32 * kWarps) {
    const int64_t j = jb + lane;
    float s = -INFINITY, vs = 0.f;
    int64_t off = -1;  // a missing page: a row of zeros
    if (j < j1) {
      const int64_t page = page_of(a.c, n, j);
      s = 0.f;
      if (page >= 0) {
        const int slot = slot_of(a.c, j);
        off = page * a.c.s_page + (int64_t)slot * a.c.s_tok + (int64_t)hk * a.c.s_head;
        float ks = 1.f;
        vs = 1.f;
        if (FMT != LA_KV_BF16) {
          const int64_t at = (page * a.c.H + hk) * (int64_t)a.c.page_size + slot;
          ks = a.c.ks[at];
          vs = a.c.vs[at];
        }
        for (int d = 0; d < D; d += 8) {
          float f[8];
          load8<FMT>(a.c.k + elem_bytes(FMT) * (off + d), f);
#pragma unroll
          for (int u = 0; u < 8; ++u) s = fmaf(f[u], sq[d + u], s);
        }
        s = s * ks * a.scale;  // last: a query times a large scale may leave fp32 where its score does not
      }
    }
    float mx = s;
#pragma unroll
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
    const float e = j < j1 ? expf(s - base) : 0.f, f = expf(m - base);
    m = mn;
    float ls = e;
#pragma unroll
    for (int w = 16; w; w >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, w);
    l = l * f + ls;
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] *= f;
    const int nk = (int)min((int64_t)32, j1 - jb);
    for (int kk = 0; kk < nk; ++kk) {
      const float ek = __shfl_sync(0xffffffffu, e, kk) * (FMT != LA_KV_BF16 ? __shfl_sync(0xffffffffu, vs, kk) : 1.f);
      const int64_t ok = __shfl_sync(0xffffffffu, off, kk);
      if (ok < 0) continue;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int d = lane + 32 * u;
        if (d >= D) break;
        const uint8_t *vp = a.c.v + elem_bytes(FMT) * (ok + d);
        float x;
        if (FMT == LA_KV_BF16) x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(vp));
        else if (FMT == LA_KV_INT8) x = (float)*reinterpret_cast<const int8_t *>(vp);
        else x = __half2float(__half(__nv_cvt_fp8_to_halfraw(*vp, __NV_E4M3)));
        o[u] = fmaf(ek, x, o[u]);
      }
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (lane + 32 * u < D) so[warp][lane + 32 * u] = o[u];
  __syncthreads();
  float M = sm[0];
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  const float base = M == -INFINITY ? 0.f : M;
  float wt[kWarps], Ls = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    wt[w] = expf(sm[w] - base);
    Ls += wt[w] * sl[w];
  }
  T *out = (T *)a.out + tb * a.o_sb + tt * a.o_st + h * a.o_sh;
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x = fmaf(wt[w], so[w][d], x);
    out[d] = from_f32<T>(j1 > j0 ? x / Ls : 0.f);  // nothing seen: zeros; all scores -infinity: 0 / 0
  }
  if (a.lse && threadIdx.x == 0) a.lse[t * a.H + h] = M + logf(Ls);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedArgs &a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(a.B * a.T * a.H);
#define LA_PA_LAUNCH(FMT)                                                                           \
  do {                                                                                              \
    if (a.dtype == LA_BF16) paged_simt_kernel<__nv_bfloat16, FMT><<<grid, 32 * kWarps, 0, stream>>>(a); \
    else paged_simt_kernel<float, FMT><<<grid, 32 * kWarps, 0, stream>>>(a);                        \
  } while (0)
  if (a.c.format == LA_KV_E4M3) LA_PA_LAUNCH(LA_KV_E4M3);
  else if (a.c.format == LA_KV_INT8) LA_PA_LAUNCH(LA_KV_INT8);
  else LA_PA_LAUNCH(LA_KV_BF16);
#undef LA_PA_LAUNCH
  return cudaGetLastError();
}

}  // namespace la

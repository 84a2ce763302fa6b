// Attention of one new token per sequence over a paged key/value cache.
//
// Mathematics. The new token of sequence b sits at position L - 1 (L = cache_lens[b]) and
// attends a set of positions: all of [0, L); or the last `window` and the first `sinks`; or
// routed positions, with the window and the first tokens where they are asked for. With
// x_j = scale * q.k_j, m = max x_j and l = sum e^{x_j - m}:
//   out = sum e^{x_j - m} v_j / l,   lse = m + ln l   (no position: out = 0, lse = -inf)
// Position j lives in row (page_table[b, j / page_size], j % page_size) of the pool.
#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kPagedThreads = 128;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One warp per (sequence, query head).
__global__ void __launch_bounds__(kPagedThreads) paged_decode_rows_kernel(PagedArgs a) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kPagedThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.B * a.Hq) return;
  const int b = row / a.Hq, h = row % a.Hq, g = h / a.G;
  const int L = a.cache_lens[b];
  const PagedSet set = paged_set(a, L);
  if (L != set.L && lane == 0) record_error(a.err, IRS_DEVERR_PAGE);
  bool bad = false;
  const int nq = a.Dqk >> 6, nv = a.Dv >> 6;
  float2 q[4], o[4];
  for (int i = 0; i < nq; ++i)
    q[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.q + (int64_t)b * a.q_sb + (int64_t)h * a.q_sh + 64 * i + 2 * lane));
  for (int i = 0; i < 4; ++i) o[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < set.n; ++j) {
    const int pos = paged_position(a, set, b, j, &bad);
    if (pos < 0) continue;
    const int pg = pos / a.page_size, off = pos - pg * a.page_size;
    const int page = a.page_table[(int64_t)b * a.table_stride + pg];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) record_error(a.err, IRS_DEVERR_PAGE);
      continue;
    }
    const __nv_bfloat16* k = a.k + (int64_t)page * a.k_sp + (int64_t)off * a.k_st + (int64_t)g * a.k_sh;
    const __nv_bfloat16* v = a.v + (int64_t)page * a.v_sp + (int64_t)off * a.v_st + (int64_t)g * a.v_sh;
    float s = 0.f;
    for (int i = 0; i < nq; ++i) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(k + 64 * i + 2 * lane));
      s = fmaf(q[i].x, x.x, fmaf(q[i].y, x.y, s));
    }
    s = warp_sum(s) * a.scale_log2;
    const float mn = fmaxf(m, s), c = ex2_approx(m - mn), p = ex2_approx(s - mn);
    m = mn;
    l = fmaf(l, c, p);
    for (int i = 0; i < nv; ++i) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(v + 64 * i + 2 * lane));
      o[i].x = fmaf(p, x.x, o[i].x * c);
      o[i].y = fmaf(p, x.y, o[i].y * c);
    }
  }
  if (bad && lane == 0) record_error(a.err, IRS_DEVERR_ROUTE_ID);
  const float f = l > 0.f ? 1.f / l : l;   // an empty row gives 0; a NaN sum stays NaN
  for (int i = 0; i < nv; ++i)
    *reinterpret_cast<__nv_bfloat162*>(a.out + (int64_t)row * a.Dv + 64 * i + 2 * lane) =
        __floats2bfloat162_rn(o[i].x * f, o[i].y * f);
  if (a.lse != nullptr && lane == 0) a.lse[row] = fmaf(m, 0.6931471805599453f, logf(l));
}

}  // namespace

size_t paged_workspace_bytes(int) { return 256; }

cudaError_t launch_paged_decode(const PagedArgs& a, int, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.Hq;
  paged_decode_rows_kernel<<<(unsigned)((rows + kPagedThreads / 32 - 1) / (kPagedThreads / 32)), kPagedThreads, 0,
                             stream>>>(a);
  return cudaGetLastError();
}

}  // namespace irs

// Attention over a prefix that many rows share, in a paged cache.
//
// Mathematics. Group g's tokens cu[g] .. cu[g+1] all attend the positions [0, n_g) of its prefix;
// decoding, the token of a sequence of length L attends its own positions [n_g, L) too. With
// x_j = scale * q.k_j, m = max x_j and l = sum e^{x_j - m}:
//   out = sum e^{x_j - m} v_j / l,   lse = m + ln l   (no position: out = 0, lse = -inf)
// and a part (o', lse') over other keys joins exactly: with M = max(lse, lse'),
//   out = (e^{lse - M} out + e^{lse' - M} o') / (e^{lse - M} + e^{lse' - M}).
#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kRowThreads = 256;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void prefix_check(const PrefixArgs& a) {
  int errors = 0;
  if (threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.P] > a.T)) errors |= IRS_DEVERR_CU_SEQLENS;
  for (int g = threadIdx.x; g < a.P; g += blockDim.x) {
    if (a.cu[g + 1] < a.cu[g]) errors |= IRS_DEVERR_CU_SEQLENS;
    const int n = a.prefix_lens[g];
    if (n < 0 || n > a.max_pages * a.page_size) errors |= IRS_DEVERR_PAGE;
  }
  if (errors) record_error(a.err, errors);
}

// One warp a row. Lane l holds the element pairs 2l, 2l + 1 of every 64 elements.
template <int NQ, int NV>
__global__ void __launch_bounds__(kRowThreads) prefix_rows_kernel(PrefixArgs a) {
  if (blockIdx.x == 0) prefix_check(a);
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.T * a.Hq) return;
  const int t = (int)(row / a.Hq), h = (int)(row % a.Hq), kv = h / a.G;
  const int g = prefix_group_of(a, t);
  if (g < 0 && a.cache_lens == nullptr) return;
  PrefixGroup grp{0, 0, 0};
  if (g >= 0) grp = prefix_group(a, g);
  int L = grp.n;
  if (a.cache_lens != nullptr) {
    L = prefix_length(a, t, grp.n);
    if (L == 0 && a.cache_lens[t] != 0 && h == 0 && lane == 0) record_error(a.err, IRS_DEVERR_PAGE);
  }
  float2 q[NQ], o[NV];
  const __nv_bfloat16* qr = a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh;
#pragma unroll
  for (int i = 0; i < NQ; ++i) q[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(qr + 64 * i + 2 * lane));
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  const int64_t shared_row = (int64_t)(a.cache_lens != nullptr ? grp.first : g) * a.table_stride;
  for (int p = 0; p < L; ++p) {
    const int pg = p / a.page_size;
    const int page = __ldg(a.page_table + (p < grp.n ? shared_row : (int64_t)t * a.table_stride) + pg);
    if (page < 0 || page >= a.num_pages) { bad = true; continue; }
    const __nv_bfloat16* kr = a.k + (int64_t)page * a.k_sp + (int64_t)(p - pg * a.page_size) * a.k_st + (int64_t)kv * a.k_sh;
    const __nv_bfloat16* vr = a.v + (int64_t)page * a.v_sp + (int64_t)(p - pg * a.page_size) * a.v_st + (int64_t)kv * a.v_sh;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(kr + 64 * i + 2 * lane));
      s = fmaf(q[i].x, x.x, fmaf(q[i].y, x.y, s));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float was = m;
    m = fmaxf(m, s);
    const float off = m == -INFINITY ? 0.f : m;
    const float c = ex2_approx(was - off), w = ex2_approx(s - off);
    l = fmaf(l, c, w);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(vr + 64 * i + 2 * lane));
      o[i].x = fmaf(w, y.x, o[i].x * c);
      o[i].y = fmaf(w, y.y, o[i].y * c);
    }
  }
  if (bad && lane == 0) record_error(a.err, IRS_DEVERR_PAGE);
  if (L > 0 && l == 0.f) l = NAN;   // no score above -inf: 0 / 0
  float lse = l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));
  float mine = l == 0.f ? 0.f : 1.f / l, theirs = 0.f;
  if (a.own_out != nullptr) {
    const float other = a.own_lse[row];
    if (other != -INFINITY) {
      const float M = fmaxf(lse, other), x = lse == -INFINITY ? 0.f : expf(lse - M), y = expf(other - M);
      mine *= x / (x + y);
      theirs = y / (x + y);
      lse = M + logf(x + y);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float2 y = make_float2(o[i].x * mine, o[i].y * mine);
    if (theirs != 0.f) {
      const float2 z = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.own_out + row * (64 * NV) + 64 * i + 2 * lane));
      y.x = fmaf(theirs, z.x, y.x);
      y.y = fmaf(theirs, z.y, y.y);
    }
    *reinterpret_cast<__nv_bfloat162*>(a.out + row * (64 * NV) + 64 * i + 2 * lane) = __floats2bfloat162_rn(y.x, y.y);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[row] = lse;
}

template <int NQ, int NV>
cudaError_t launch_rows(const PrefixArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * a.Hq;
  const unsigned grid = (unsigned)((rows + kRowThreads / 32 - 1) / (kRowThreads / 32));
  prefix_rows_kernel<NQ, NV><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_workspace_bytes(int, int, int, int, int, bool) { return 256; }

cudaError_t launch_prefix_rows(const PrefixArgs& a, cudaStream_t stream) {
  switch (a.Dqk / 64 * 4 + a.Dv / 64) {
    case 5: return launch_rows<1, 1>(a, stream);
    case 6: return launch_rows<1, 2>(a, stream);
    case 9: return launch_rows<2, 1>(a, stream);
    case 10: return launch_rows<2, 2>(a, stream);
    case 13: return launch_rows<3, 1>(a, stream);
    default: return launch_rows<3, 2>(a, stream);
  }
}

}  // namespace irs

// Attention over a prefix that many rows share, in a paged cache: what its kernels have in common.
//
// Mathematics. Group g's tokens cu[g] .. cu[g+1] all attend the positions [0, n_g) of its prefix;
// decoding, the token of a sequence of length L attends its own positions [n_g, L) too. With
// x_j = scale * q.k_j, m = max x_j and l = sum e^{x_j - m}:
//   out = sum e^{x_j - m} v_j / l,   lse = m + ln l   (no position: out = 0, lse = -inf)
// and parts over other keys join exactly: with M = max m_i, out = sum e^{m_i - M} o_i / sum e^{m_i - M} l_i.
#pragma once

#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

// Positions a block: 128 columns of scores a product where shared memory has room for the stages; beside queries
// of 192 dims it has for 96.
__host__ __device__ constexpr int prefix_block(int Dqk) { return Dqk == 192 ? 96 : 128; }
constexpr int kPrefixRows = 256;      // rows an item (two tiles)
constexpr int kMaxPrefixCtas = 160;
// A run has at least this many blocks: fewer leave more parts to join than they save. 77 tokens over 4099
// positions, and a step of 8 sequences behind 2000: 2 blocks 22.7 and 22.6 us, 1 block 22.7 and 25.0, 4 blocks 26.7 and 22.8.
constexpr int kMinBlocks = 2;

__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: sums of the groups' blocks; two parts a CTA (the item its run starts in, the one it ends
// in); decoding, the same a row for rows that no border cuts. Sums of n rows lie as [Dv / 4][n][4], then
// [n] pairs of maximum and sum: a warp's 32 rows are 512 bytes a store, where rows of Dv columns made
// a store touch 32 lines and an item's end take 8,000 cycles.
__host__ __device__ inline size_t prefix_pre_bytes(int P) { return align256(((size_t)P + 1) * 8); }
__host__ __device__ inline size_t prefix_part_floats(int Dv) { return (size_t)kPrefixRows * (Dv + 2); }
__host__ __device__ inline size_t prefix_parts_bytes(int Dv) { return (size_t)kMaxPrefixCtas * 2 * prefix_part_floats(Dv) * 4; }
__host__ __device__ inline size_t prefix_rows_bytes(int T, int Hq, int Dv) { return align256((size_t)T * Hq * (Dv + 2) * 4); }

__device__ __forceinline__ float* prefix_part(const PrefixArgs& a, int run, int head, int which) {
  return reinterpret_cast<float*>(a.ws + prefix_pre_bytes(a.P)) + (((size_t)run * a.Hkv + head) * 2 + which) * prefix_part_floats(a.Dv);
}
__device__ __forceinline__ float* prefix_rows(const PrefixArgs& a) {
  return reinterpret_cast<float*>(a.ws + prefix_pre_bytes(a.P) + prefix_parts_bytes(a.Dv));
}

__device__ __forceinline__ float4& prefix_sums4(float* sums, int64_t n, int64_t row, int d) {
  return *reinterpret_cast<float4*>(sums + ((int64_t)(d / 4) * n + row) * 4);
}
__device__ __forceinline__ float2& prefix_sums_ml(float* sums, int64_t n, int64_t row, int Dv) {
  return *reinterpret_cast<float2*>(sums + n * Dv + 2 * row);
}
__device__ __forceinline__ void prefix_sums8(float (&o)[8], float* sums, int64_t n, int64_t row, int d) {
  const float4 x = prefix_sums4(sums, n, row, d), y = prefix_sums4(sums, n, row, d + 4);
  o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
  o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
}

// Blocks of a group in a head's list: its pairs of tiles (qt tokens each), each over the whole prefix.
__device__ __forceinline__ int64_t prefix_units(const PrefixGroup& g, int qt, int blk) {
  return (int64_t)((g.last - g.first + 2 * qt - 1) / (2 * qt)) * ((g.n + blk - 1) / blk);
}
__device__ __forceinline__ int prefix_blocks(const PrefixArgs& a, int n) {
  const int blk = prefix_block(a.Dqk);
  return (n + blk - 1) / blk;
}
// Blocks of a run.
__device__ __forceinline__ int64_t prefix_share(int64_t total, int runs) {
  const int64_t q = total >> 30 == 0 ? (int64_t)(((uint32_t)total + (uint32_t)runs - 1u) / (uint32_t)runs) : (total + runs - 1) / runs;
  return q < kMinBlocks ? kMinBlocks : q;
}
// The run that holds unit f. (Divisions of 64 bits take a thread 100 instructions.)
__device__ __forceinline__ int prefix_run(int64_t f, int64_t share) {
  return ((f | share) >> 31) == 0 ? (int)((uint32_t)f / (uint32_t)share) : (int)(f / share);
}
// The group that holds unit f of a head's list.
__device__ __forceinline__ int prefix_find(const int64_t* pre, int P, int64_t f) {
  int lo = 0, hi = P;   // pre[lo] <= f < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= f) lo = mid; else hi = mid;
  }
  return lo;
}

// Malformed borders and prefix lengths, by threads 0 .. n - 1.
__device__ __forceinline__ void prefix_check(const PrefixArgs& a, int i, int n) {
  int errors = 0;
  if (i == 0 && (a.cu[0] != 0 || a.cu[a.P] > a.T)) errors |= IRS_DEVERR_CU_SEQLENS;
  for (int g = i; g < a.P; g += n) {
    if (a.cu[g + 1] < a.cu[g]) errors |= IRS_DEVERR_CU_SEQLENS;
    const int len = a.prefix_lens[g];
    if (len < 0 || len > a.max_pages * a.page_size) errors |= IRS_DEVERR_PAGE;
  }
  if (errors) record_error(a.err, errors);
}

// Sums N columns of parts with their own maxima. A part's sum of -1 says that it had positions and every
// score was -inf: any finite maximum wipes it out, and alone it is 0 / 0.
template <int N>
struct PrefixSum {
  float m, l, o[N];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
  }
  __device__ __forceinline__ void add(float pm, float pl, const float (&x)[N]) {
    const float n = fmaxf(m, pm);
    const float u = n == -INFINITY ? 0.f : ex2_approx(m - n), v = n == -INFINITY ? 0.f : ex2_approx(pm - n);
    m = n;
    l = n == -INFINITY ? l + pl : fmaf(l, u, pl * v);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], u, x[i] * v);
  }
};

__device__ __forceinline__ void prefix_load8(float (&o)[8], const float* p) {
  const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
  o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
  o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
}

// What a row's own sums and its other part count in the result, and its lse.
struct PrefixJoin {
  float mine, theirs, lse;
};
__device__ __forceinline__ PrefixJoin prefix_join_own(const PrefixArgs& a, int64_t row, float m, float l) {
  const float other = a.own_lse != nullptr ? a.own_lse[row] : -INFINITY;
  if (l < 0.f) l = other != -INFINITY ? 0.f : NAN;   // beside a part that counts a weight of 0, alone 0 / 0
  PrefixJoin j;
  j.lse = l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
  j.mine = l == 0.f ? 0.f : 1.f / l;
  j.theirs = 0.f;
  if (other != -INFINITY) {
    const float M = fmaxf(j.lse, other), x = j.lse == -INFINITY ? 0.f : expf(j.lse - M), y = expf(other - M);
    j.mine *= x / (x + y);
    j.theirs = y / (x + y);
    j.lse = M + logf(x + y);
  }
  return j;
}
// Eight columns of the result as bf16 pairs; z: those of the other part (not looked at where it does not count).
__device__ __forceinline__ void prefix_mix8(uint32_t* w, const PrefixJoin& j, const float* o, const uint4& z) {
  const __nv_bfloat162* zz = reinterpret_cast<const __nv_bfloat162*>(&z);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = j.mine == 0.f ? 0.f : o[2 * i] * j.mine, y = j.mine == 0.f ? 0.f : o[2 * i + 1] * j.mine;
    if (j.theirs != 0.f) {
      const float2 f = __bfloat1622float2(zz[i]);
      x = fmaf(j.theirs, f.x, x);
      y = fmaf(j.theirs, f.y, y);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}
// ... to element `at` of out on.
__device__ __forceinline__ void prefix_store8(const PrefixArgs& a, int64_t at, const PrefixJoin& j, const float* o) {
  uint4 z = make_uint4(0u, 0u, 0u, 0u), y;
  if (j.theirs != 0.f) z = *reinterpret_cast<const uint4*>(a.own_out + at);
  prefix_mix8(reinterpret_cast<uint32_t*>(&y), j, o, z);
  *reinterpret_cast<uint4*>(a.out + at) = y;
}

}  // namespace

}  // namespace irs

// Rotary positions of attention heads, on their own or on the way into a paged cache.
//
// Mathematics. Pair i of a rotated part (x_a, x_b) at position p turns by the angle p * f_i:
//   y_a = amp * (x_a cos - x_b sin),   y_b = amp * (x_b cos + x_a sin)
// (transpose: the sine's sign flips, which is the gradient). "Half" layout pairs dims i and
// i + rope_dims/2 of the part, "interleaved" 2i and 2i + 1.
//
// Angles. At position 10^6 an FP32 product p * f is off by 0.06 radians. The frequency is
// therefore held as a 64-bit binary fraction of a turn, F = (f / 2 pi mod 1) * 2^64, and
// p * F mod 2^64 is the exact fraction of a turn that remains: whole turns wrap away in the
// integer multiply. Its top 32 bits become the FP32 argument of sincospif. The only errors
// are F's (2^-53 of f, times p) and one rounding to FP32. FP64 work is one product and one
// rounding per pair and thread; a thread keeps its pairs for all its tokens and heads.
#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeSmemSeqs = 4096;   // cu_new of up to this many sequences is searched in shared memory

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(__nv_bfloat16* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf2(float x, float y) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Frequency (radians per token) as a fraction of a turn in units of 2^-64, whole turns dropped.
__device__ __forceinline__ int64_t turn_fraction(double f) {
  double turns = f * 0.15915494309189533577;   // 1 / (2 pi)
  turns -= rint(turns);
  return 2 * __double2ll_rn(turns * 9223372036854775808.0);   // 2^63; |turns| <= 1/2 keeps the product in range
}

// Rotate 8 pairs: `half` pairs a's elements with b's; otherwise a and b are two runs of
// adjacent pairs.
template <bool HALF>
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t* aw = reinterpret_cast<uint32_t*>(&a);
  uint32_t* bw = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (HALF) {
      const float2 u = bf2(aw[i]), w = bf2(bw[i]);
      aw[i] = pack_bf2(u.x * cs[2 * i] - w.x * sn[2 * i], u.y * cs[2 * i + 1] - w.y * sn[2 * i + 1]);
      bw[i] = pack_bf2(w.x * cs[2 * i] + u.x * sn[2 * i], w.y * cs[2 * i + 1] + u.y * sn[2 * i + 1]);
    } else {
      const float2 u = bf2(aw[i]), w = bf2(bw[i]);
      aw[i] = pack_bf2(u.x * cs[i] - u.y * sn[i], u.y * cs[i] + u.x * sn[i]);
      bw[i] = pack_bf2(w.x * cs[4 + i] - w.y * sn[4 + i], w.y * cs[4 + i] + w.x * sn[4 + i]);
    }
  }
}

// The sequence of token t: the last b with cu[b] <= t (sequences may be empty).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;   // cu[lo] <= t < cu[hi] where cu is well formed
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One thread: 16 elements of the rotated part (8 pairs), or 16 elements that are copied, of
// the heads hg, hg + groups, ... of the tokens t0, t0 + stride, ...
template <bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  extern __shared__ int32_t cu_s[];
  const bool paged = a.k_cache != nullptr;
  const int32_t* cu = a.cu_new;
  if (cu != nullptr && a.B <= kRopeSmemSeqs) {
    for (int i = threadIdx.x; i <= a.B; i += kRopeThreads) cu_s[i] = a.cu_new[i];
    __syncthreads();
    cu = cu_s;
  }
  int T = a.T;
  if (cu != nullptr) {
    if (blockIdx.x == 0) {
      bool bad = threadIdx.x == 0 && (cu[0] != 0 || cu[a.B] > a.T);
      for (int i = threadIdx.x; i < a.B; i += kRopeThreads) bad |= cu[i + 1] < cu[i];
      if (bad) record_error(a.err, IRS_DEVERR_CU_SEQLENS);
    }
    T = min(T, cu[a.B]);   // rows behind the last sequence are left as they were
  }
  const int64_t lane = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const int u = (int)(lane % a.units);
  const int hg = (int)((lane / a.units) % a.groups);
  const int64_t t0 = lane / ((int64_t)a.units * a.groups);
  const int64_t tstep = (int64_t)gridDim.x * kRopeThreads / ((int64_t)a.units * a.groups);
  if (t0 >= tstep) return;   // threads past the last whole (units x groups) set

  const int n_rot = a.rope_dims >> 4;
  const int n_copy = (a.D - a.rope_dims + 15) >> 4;
  const bool rot = u < n_rot;
  const bool is_v = u >= n_rot + n_copy;
  int d0, d1;          // the two 8-element chunks; d1 < 0: none
  int64_t F[8];
  if (rot) {
    d0 = a.start + (HALF ? 8 * u : 16 * u);
    d1 = HALF ? d0 + (a.rope_dims >> 1) : d0 + 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) F[i] = turn_fraction(a.inv_freq[8 * u + i]);
  } else if (!is_v) {
    // copied chunks: those before the part, then those behind it
    const int c0 = 2 * (u - n_rot), before = a.start >> 3, all = (a.D - a.rope_dims) >> 3;
    d0 = (c0 < before ? c0 : c0 + (a.rope_dims >> 3)) * 8;
    d1 = c0 + 1 >= all ? -1 : (c0 + 1 < before ? c0 + 1 : c0 + 1 + (a.rope_dims >> 3)) * 8;
  } else {
    d0 = 16 * (u - n_rot - n_copy);
    d1 = d0 + 8 < a.Dv ? d0 + 8 : -1;
  }
  if (!rot && !is_v && a.in_place) return;

  for (int64_t t = t0; t < T; t += tstep) {
    int pos;
    int64_t kslot = -1, vslot = -1;   // element offsets of the token's cache rows
    if (paged) {
      const int b = cu != nullptr ? sequence_of(cu, a.B, (int)t) : (int)t;
      const int len = a.cache_lens[b];
      pos = len + (cu != nullptr ? (int)t - cu[b] : 0);
      const int pg = pos / a.page_size;
      int page = -1;
      if (len >= 0 && pos >= 0 && pg < a.max_pages) page = a.page_table[(int64_t)b * a.table_stride + pg];
      if (page >= 0 && page < a.num_pages) {
        const int off = pos - pg * a.page_size;
        kslot = (int64_t)page * a.kc_sp + (int64_t)off * a.kc_st;
        vslot = (int64_t)page * a.vc_sp + (int64_t)off * a.vc_st;
      } else if (u == 0 && hg == 0) {
        record_error(a.err, IRS_DEVERR_PAGE);
      }
    } else {
      pos = a.positions[t];
    }
    if (is_v) {
      if (vslot < 0) continue;
      for (int h = hg; h < a.Hkv; h += a.groups) {
        const __nv_bfloat16* src = a.v + t * a.v_st + (int64_t)h * a.v_sh;
        __nv_bfloat16* dst = a.v_cache + vslot + (int64_t)h * a.vc_sh;
        st16(dst + d0, ld16(src + d0));
        if (d1 >= 0) st16(dst + d1, ld16(src + d1));
      }
      continue;
    }
    float cs[8], sn[8];
    if (rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t frac = (int32_t)(uint32_t)(((uint64_t)((int64_t)pos) * (uint64_t)F[i]) >> 32);
        sincospif((float)frac * 4.656612873077392578125e-10f, &sn[i], &cs[i]);   // 2^-31: half turns
        cs[i] *= a.amplitude;
        sn[i] *= a.transpose ? -a.amplitude : a.amplitude;
      }
    }
    const int H = a.Hq + a.Hkv;
    constexpr int kUnroll = 4;
    for (int hb = hg; hb < H; hb += kUnroll * a.groups) {
      uint4 x[kUnroll], y[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = hb + j * a.groups;
        if (h < H) {
          const __nv_bfloat16* src = h < a.Hq ? a.q + t * a.q_st + (int64_t)h * a.q_sh
                                              : a.k + t * a.k_st + (int64_t)(h - a.Hq) * a.k_sh;
          x[j] = ld16(src + d0);
          if (d1 >= 0) y[j] = ld16(src + d1);
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = hb + j * a.groups;
        if (h < H) {
          if (rot) rotate8<HALF>(x[j], y[j], cs, sn);
          if (h < a.Hq) {
            __nv_bfloat16* dst = a.q_out + t * a.qo_st + (int64_t)h * a.qo_sh;
            st16(dst + d0, x[j]);
            if (d1 >= 0) st16(dst + d1, y[j]);
          } else {
            const int g = h - a.Hq;
            if (kslot >= 0) {
              __nv_bfloat16* dst = a.k_cache + kslot + (int64_t)g * a.kc_sh;
              st16(dst + d0, x[j]);
              if (d1 >= 0) st16(dst + d1, y[j]);
            }
            if (a.k_out != nullptr) {
              __nv_bfloat16* dst = a.k_out + t * a.ko_st + (int64_t)g * a.ko_sh;
              st16(dst + d0, x[j]);
              if (d1 >= 0) st16(dst + d1, y[j]);
            }
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, bool half, int num_sms, cudaStream_t stream) {
  const int n_rot = a.rope_dims >> 4, n_copy = (a.D - a.rope_dims + 15) >> 4, n_v = a.k_cache ? (a.Dv + 15) >> 4 : 0;
  a.units = n_rot + n_copy + n_v;
  // Threads first: as many head groups as it takes to give every SM its 2048 threads; with
  // more tokens than that, a thread keeps its angles over several heads and tokens.
  const int H = a.Hq + a.Hkv;
  const int64_t full = (int64_t)num_sms * 2048;
  int64_t groups = full / ((int64_t)a.T * a.units);
  a.groups = (int)(groups < 1 ? 1 : groups > H ? H : groups);
  const int64_t per_token = (int64_t)a.units * a.groups;
  int64_t threads = (int64_t)a.T * per_token;
  if (threads > full) threads = full;
  if (threads < per_token) threads = per_token;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const size_t smem = a.cu_new != nullptr && a.B <= kRopeSmemSeqs ? (size_t)(a.B + 1) * 4 : 0;
  if (half) rope_kernel<true><<<(unsigned)blocks, kRopeThreads, smem, stream>>>(a);
  else rope_kernel<false><<<(unsigned)blocks, kRopeThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace irs

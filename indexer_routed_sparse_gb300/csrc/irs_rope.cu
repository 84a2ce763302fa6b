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
// are F's (2^-53 of f, times p) and one rounding to FP32. FP64 work, slow on this GPU (two
// operations a clock and SM), is one product and one rounding per frequency and block.
//
// What bounds it. Every element is read and written once, with a dozen operations: HBM. So
// the design keeps bytes in flight: a thread loads eight heads' chunks before it turns them,
// and 512 of them an SM have 128 KB on the way. Measured at 16384 tokens of 64 heads of 128:
// 86 us, 6.3 TB/s (eight heads ahead, 4096 threads an SM in the launch; four heads 93 us,
// two 97; 2048 threads 87, 8192 103, as the angles are then worked out for few heads each);
// 14,000 new tokens of 64 / 4 heads of 192 / 128, a third rotated, into pages of 16: 125 us.
#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 8;            // heads a thread has in flight
constexpr int kRopeFull = 4096;       // threads an SM that a launch aims at
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

// The sequence of token t: the last b with cu[b] <= t (sequences may be empty), or 0.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;   // cu[lo] <= t < cu[hi] where cu is well formed
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One thread: two 16-byte chunks of a head, of the heads hg, hg + groups, ... of the tokens
// t0, t0 + stride, ... In both layouts the chunks of a rotated unit stand half a part apart
// (the partners of "half"; two runs of whole pairs of "interleaved"), and neighbouring threads
// take neighbouring chunks. Heads in order: queries, keys, and into a cache the values.
template <bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(RopeArgs a) {
  extern __shared__ int64_t turn_s[];   // [rope_dims / 2] frequencies, then cu_new
  const bool paged = a.k_cache != nullptr;
  const int32_t* cu = a.cu_new;
  for (int i = threadIdx.x; i < a.rope_dims >> 1; i += kRopeThreads) turn_s[i] = turn_fraction(a.inv_freq[i]);
  if (cu != nullptr && a.B <= kRopeSmemSeqs) {
    int32_t* cu_s = reinterpret_cast<int32_t*>(turn_s + (a.rope_dims >> 1));
    for (int i = threadIdx.x; i <= a.B; i += kRopeThreads) cu_s[i] = a.cu_new[i];
    cu = cu_s;
  }
  __syncthreads();
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
  const bool rot = u < n_rot;
  int d0, d1;          // the two chunks; d1 < 0: none
  if (rot) {
    d0 = a.start + 8 * u;
    d1 = d0 + (a.rope_dims >> 1);
  } else {             // copied: chunks before the part, then those behind it
    const int c0 = u - n_rot, all = (a.D - a.rope_dims) >> 3, c1 = c0 + ((all + 1) >> 1), before = a.start >> 3;
    d0 = (c0 < before ? c0 : c0 + (a.rope_dims >> 3)) * 8;
    d1 = c1 >= all ? -1 : (c1 < before ? c1 : c1 + (a.rope_dims >> 3)) * 8;
  }
  if (!rot && a.in_place) return;
  const int H = a.Hq + a.Hkv, all_heads = paged ? H + a.Hkv : H;
  const int v_chunks = a.Dv >> 3, v_half = (v_chunks + 1) >> 1;
  const int v0 = u < v_half ? 8 * u : -1, v1 = u < v_half && u + v_half < v_chunks ? 8 * (u + v_half) : -1;

  for (int64_t t = t0; t < T; t += tstep) {
    int pos;
    int64_t kslot = -1, vslot = -1;   // element offsets of the token's cache rows
    if (paged) {
      const int b = cu != nullptr ? sequence_of(cu, a.B, (int)t) : (int)t;
      const int row0 = cu != nullptr ? cu[b] : (int)t;
      if (row0 < 0 || row0 > t) continue;   // a cu_new that does not start at 0: the row is no sequence's
      const int len = a.cache_lens[b];
      pos = len + ((int)t - row0);
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
    float cs[8], sn[8];
    if (rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // pairs of the first chunk and of the second ("half": they share their pairs)
        const int pair = HALF ? 8 * u + i : 4 * u + (i & 3) + (i >> 2) * (a.rope_dims >> 2);
        const int32_t frac = (int32_t)(uint32_t)(((uint64_t)((int64_t)pos) * (uint64_t)turn_s[pair]) >> 32);
        sincospif((float)frac * 4.656612873077392578125e-10f, &sn[i], &cs[i]);   // 2^-31: half turns
        cs[i] *= a.amplitude;
        sn[i] *= a.transpose ? -a.amplitude : a.amplitude;
      }
    }
    for (int hb = hg; hb < all_heads; hb += kUnroll * a.groups) {
      uint4 x[kUnroll], y[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = hb + j * a.groups;
        if (h < all_heads) {
          const __nv_bfloat16* src = h < a.Hq ? a.q + t * a.q_st + (int64_t)h * a.q_sh
                                     : h < H  ? a.k + t * a.k_st + (int64_t)(h - a.Hq) * a.k_sh
                                              : a.v + t * a.v_st + (int64_t)(h - H) * a.v_sh;
          const int e0 = h < H ? d0 : v0, e1 = h < H ? d1 : v1;
          if (e0 >= 0) x[j] = ld16(src + e0);
          if (e1 >= 0) y[j] = ld16(src + e1);
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = hb + j * a.groups;
        if (h >= all_heads) break;
        if (rot && h < H) rotate8<HALF>(x[j], y[j], cs, sn);
        if (h < a.Hq) {
          __nv_bfloat16* dst = a.q_out + t * a.qo_st + (int64_t)h * a.qo_sh;
          st16(dst + d0, x[j]);
          if (d1 >= 0) st16(dst + d1, y[j]);
        } else if (h < H) {
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
        } else if (vslot >= 0) {
          const __nv_bfloat16* src = a.v + t * a.v_st + (int64_t)(h - H) * a.v_sh;
          __nv_bfloat16* dst = a.v_cache + vslot + (int64_t)(h - H) * a.vc_sh;
          if (v0 >= 0) st16(dst + v0, x[j]);
          if (v1 >= 0) st16(dst + v1, y[j]);
          for (int c = u + a.units; c < v_half; c += a.units) {   // values wider than keys
            st16(dst + 8 * c, ld16(src + 8 * c));
            if (c + v_half < v_chunks) st16(dst + 8 * (c + v_half), ld16(src + 8 * (c + v_half)));
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, bool half, int num_sms, cudaStream_t stream) {
  a.units = (a.rope_dims >> 4) + ((a.D - a.rope_dims + 15) >> 4);
  // Threads first: as many head groups as it takes to give every SM its threads; with more
  // tokens than that, a thread keeps its angles over several heads and tokens.
  const int heads = a.Hq + a.Hkv + (a.k_cache != nullptr ? a.Hkv : 0);
  const int64_t full = (int64_t)num_sms * kRopeFull;
  int64_t groups = full / ((int64_t)a.T * a.units);
  a.groups = (int)(groups < 1 ? 1 : groups > heads ? heads : groups);
  const int64_t per_token = (int64_t)a.units * a.groups;
  int64_t threads = (int64_t)a.T * per_token;
  if (threads > full) threads = full;
  if (threads < per_token) threads = per_token;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const size_t smem = (size_t)(a.rope_dims >> 1) * 8 + (a.cu_new != nullptr && a.B <= kRopeSmemSeqs ? (size_t)(a.B + 1) * 4 : 0);
  if (half) rope_kernel<true><<<(unsigned)blocks, kRopeThreads, smem, stream>>>(a);
  else rope_kernel<false><<<(unsigned)blocks, kRopeThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace irs

// Attention of one new token per sequence over a paged key/value cache.
//
// Mathematics. The new token of sequence b sits at position L - 1 (L = cache_lens[b]) and
// attends a set of positions: all of [0, L); or the last `window` and the first `sinks`; or
// routed positions, with the window and the first tokens where they are asked for. With
// x_j = scale * q.k_j, m = max x_j and l = sum e^{x_j - m}:
//   out = sum e^{x_j - m} v_j / l,   lse = m + ln l   (no position: out = 0, lse = -inf)
// Position j lives in row (page_table[b, j / page_size], j % page_size) of the pool. Parts
// of a sequence join exactly: with M = max m_i, out = sum e^{m_i - M} o_i / sum e^{m_i - M} l_i.
//
// What bounds it. 2 (Dqk + Dv) bytes a position and KV head against 2 G (Dqk + Dv) flops: G
// flops a byte, so HBM; the tensor cores are used (mma.sync, 16 query heads a tile) because
// at G = 8 and above FP32 cores would be the bound.
//
// Design.
// * A tile is 16 positions of one KV head. The tiles of the batch, sequence by sequence, form
//   one list per head, and the lists are cut into runs of equal length, one a warp, so ragged
//   lengths load the SMs equally and one long sequence spreads over all of them. The list's
//   shape comes from the lengths on the device; nothing is read back. The warps of a CTA take
//   the same run for different heads: a token's heads lie next to one another in the pool,
//   and fetching them together is what keeps DRAM pages open (routed positions).
// * A warp works alone: its own ring of cp.async stages, its own running maximum, sum and
//   output in registers, no barrier anywhere in the loop, and its copies run on into the
//   next sequence. Positions, routes and page numbers are looked up two tiles ahead.
// * A run that holds a whole (sequence, head) writes the result. One that a warp border cuts
//   leaves its part in the workspace, and a second kernel (launched early, waiting for the
//   first) joins the parts in list order. No atomics: every run gives the same bits.
//   Joining the eight warps of a CTA in shared memory at every sequence's end instead cost
//   18 us a sequence.
// * The maximum is raised, and the output rescaled, only where a score passes it by 2^8:
//   weights then stay below 2^8 and sums below 2^8 n, harmless in FP32, and the rescaling of
//   Dv/2 registers a thread leaves the loop almost entirely.
// * A weight enters the second product as two bf16 terms (its first eight bits and the rest),
//   which keeps 16 bits of it; the extra product costs tensor time that HBM-bound code has.
// * Measured: 64 sequences of 20,000 to 50,000 positions, 64 / 8 heads of 128: 1.31 ms, 7.0
//   TB/s; 2051 routes of 96 sequences, 32 / 8 heads of 128: 132 us, 6.1 TB/s; 512 + 4
//   positions of 128 sequences, 64 / 4 heads of 192 / 128: 36 us for 120 MB, where the start
//   (lengths, pages, first copies) and the join count.
#include <type_traits>

#include "irs_internal.h"
#include "irs_paged.cuh"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr float kRaise = 8.f;          // raise the maximum only where a score passes it by 2^8
constexpr uint32_t kRingBytes = 223u * 1024u;

// How a launch lays out its warps: `groups` groups of CTAs take `heads` heads each; `per_head`
// warps of a CTA share a head's list.
struct PagedGrid {
  int groups, heads, per_head, warps, stages, ctas, workers;   // workers: runs of a head's list
  uint32_t mask_off, smem;
};

inline PagedGrid paged_grid(int Dqk, int Dv, int HK, int num_sms) {
  PagedGrid g{};
  const uint32_t stage = (uint32_t)(kTile * (Dqk + Dv) * 2);
  // As many warps (up to 8) as can have two stages each: a warp alone issues an instruction in
  // four cycles, so two a scheduler count for more than a third stage (192/128 with 4 KV heads,
  // 450k positions: 183 us with 8 warps of 2 stages, 198 us with 4 warps of 5).
  int most = (int)(kRingBytes / (2u * stage));
  most = most > kMaxWarps ? kMaxWarps : most;
  g.groups = (HK + most - 1) / most;
  g.heads = (HK + g.groups - 1) / g.groups;
  g.groups = (HK + g.heads - 1) / g.heads;
  g.per_head = most / g.heads;
  g.warps = g.heads * g.per_head;
  const int fit = (int)(kRingBytes / (stage * (uint32_t)g.warps));
  g.stages = fit > 6 ? 6 : fit;
  g.mask_off = stage * (uint32_t)(g.warps * g.stages);
  g.smem = g.mask_off + 4u * (uint32_t)(g.warps * g.stages);
  int c = (num_sms < kMaxPagedCtas ? num_sms : kMaxPagedCtas) / g.groups;   // CTAs a group
  c = c < 1 ? 1 : c;
  g.ctas = c * g.groups;
  g.workers = c * g.per_head;
  return g;
}

// The positions that the new token of a sequence of length L attends here; SHARED: those behind the n that its group shares.
template <bool SHARED>
__device__ __forceinline__ PagedSet set_of(const PagedArgs& a, int L, int n) {
  if constexpr (SHARED) {
    PagedSet s{};
    s.L = L < n || L > a.max_pages * a.page_size ? 0 : L;
    s.first = s.L > 0 ? n : 0;
    s.recent = s.n = s.L - s.first;
    return s;
  } else {
    return paged_set(a, L);
  }
}
__device__ __forceinline__ int tiles_of(const PagedSet& s) { return (s.n + kTile - 1) / kTile; }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Weights x and y (>= 0) as two bf16 pairs: cut to eight bits, and what the cut left, rounded: 2^-16
// of the weight is lost at most. Neither term is negative, and the second is never 0 (2^-126 where
// nothing is left, which no sum notices): times an infinite value both give that infinity, where a
// rest of 0 or of the other sign would make it NaN. Masked rows are 0 in shared memory.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint32_t xi = __float_as_uint(x), yi = __float_as_uint(y);
  hi = __byte_perm(xi, yi, 0x7632);
  const __nv_bfloat162 l = __hmax2(__floats2bfloat162_rn(x - __uint_as_float(xi & 0xffff0000u), y - __uint_as_float(yi & 0xffff0000u)),
                                   __halves2bfloat162(__ushort_as_bfloat16(0x0080), __ushort_as_bfloat16(0x0080)));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// One place in the list of tiles.
struct Cursor {
  int b, tile, nt;   // sequence, tile of it, its tile count
  PagedSet set;
};
// shared: how many positions sequence b shares with its group (kept for the first 32 kMaxWarps, else looked up).
template <bool SHARED>
using PagedOthers = std::conditional_t<SHARED, PagedShared, PagedAlone>;
template <bool SHARED>
__device__ __forceinline__ int shared_of(const PagedOthers<SHARED>& sh, const int* shared, int b) {
  if constexpr (SHARED) return b < 32 * kMaxWarps ? shared[b] : prefix_positions(sh.groups, b);
  else return 0;
}
template <bool SHARED>
__device__ __forceinline__ void cursor_open(const PagedArgs& a, const PagedOthers<SHARED>& sh, const int* shared, Cursor& c) {
  c.set = set_of<SHARED>(a, __ldg(a.cache_lens + c.b), shared_of<SHARED>(sh, shared, c.b));
  c.nt = tiles_of(c.set);
}
// Move on to the sequence that holds c.tile; the list must go on that far.
template <bool SHARED>
__device__ __forceinline__ void cursor_settle(const PagedArgs& a, const PagedOthers<SHARED>& sh, const int* shared, Cursor& c) {
  while (c.tile >= c.nt) {
    c.tile -= c.nt;
    if (++c.b >= a.B) { c.b = a.B - 1; c.tile = 0; return; }   // not reached on a list of the right length
    cursor_open<SHARED>(a, sh, shared, c);
  }
}

// SHARED: the own positions of sequences that share prefixes. Nothing is written but FP32 sums: parts as
// ever, and rows of a sequence that no border cuts, for the join with the prefixes' (irs_prefix_tc.cu).
template <int DQK, int DV, bool SHARED>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) paged_decode_kernel(PagedArgs a, PagedGrid pg, int nhb, PagedOthers<SHARED> sh) {
  constexpr int KS = DQK / 16, NV = DV / 8;
  constexpr uint32_t kStage = kTile * (DQK + DV) * 2;
  const int NW = pg.warps, S = pg.stages;
  constexpr bool QREG = DQK + DV <= 384;              // the queries stay in registers
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + pg.mask_off);
  __shared__ int64_t scan[32 * kMaxWarps + 1];
  __shared__ int64_t start_pre[kMaxWarps];
  __shared__ int start_b[kMaxWarps];
  __shared__ int shared[SHARED ? 32 * kMaxWarps : 1];

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HK = a.Hkv * nhb;
  const int hk = (int)(blockIdx.x % (unsigned)pg.groups) * pg.heads + warp / pg.per_head;   // KV head and block of query heads
  const int worker0 = (int)(blockIdx.x / (unsigned)pg.groups) * pg.per_head;   // the CTA's first run of each head's list

  // ---- the list of tiles: its length and where this CTA's runs start ----
  const int per = (a.B + 32 * NW - 1) / (32 * NW);
  const int bs = min(a.B, tid * per), be = min(a.B, bs + per);
  {
    int64_t n = 0;
    for (int b = bs; b < be; ++b) {
      const int L = __ldg(a.cache_lens + b);
      int prefix = 0;
      if constexpr (SHARED) {
        prefix = prefix_positions(sh.groups, b);
        if (b < 32 * kMaxWarps) shared[b] = prefix;
      }
      if (blockIdx.x == 0 && (L < prefix || L > a.max_pages * a.page_size) && (!SHARED || L != 0)) record_error(a.err, IRS_DEVERR_PAGE);
      n += tiles_of(set_of<SHARED>(a, L, prefix));
    }
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int64_t base = 0, total = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) base += scan[w];
      total += scan[w];
    }
    __syncthreads();
    scan[tid] = base + x - n;
    if (tid == 0) scan[32 * kMaxWarps] = total;
    if (tid < NW) start_b[tid] = -1;
    __syncthreads();
  }
  const int64_t total = scan[32 * kMaxWarps];
  const int64_t share = paged_share(total, pg.workers);
  {
    int64_t* pre = reinterpret_cast<int64_t*>(a.ws);
    int64_t n = scan[tid];
    for (int b = bs; b < be; ++b) {
      const int64_t next = n + tiles_of(set_of<SHARED>(a, __ldg(a.cache_lens + b), shared_of<SHARED>(sh, shared, b)));
      if (blockIdx.x == 0) pre[b] = n;
      for (int w = 0; w < pg.per_head; ++w) {
        const int64_t f = (worker0 + w) * share;
        if (f >= n && f < next) { start_b[w] = b; start_pre[w] = n; }
      }
      n = next;
    }
    if (blockIdx.x == 0 && tid == 0) pre[a.B] = total;
  }
  __syncthreads();
  const int sub = warp % pg.per_head, worker = worker0 + sub;
  const int64_t f0 = worker * share, f1 = min(total, f0 + share);
  // SHARED: launched early and waited for by the join, which then may rely on the kernel before this one
  if (f0 >= f1 || start_b[sub] < 0 || hk >= HK) {
    if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int g = hk / nhb, hb = hk % nhb;
  const int h0 = g * a.G + hb * kHeads, nh = min(kHeads, a.G - hb * kHeads);

  Cursor cc;                                            // the tile being computed
  cc.b = start_b[sub];
  cursor_open<SHARED>(a, sh, shared, cc);
  cc.tile = (int)(f0 - start_pre[sub]);

  // ---- loads: A looks up positions or routes, B pages, C issues the copies ----
  Cursor lc = cc;
  int64_t lf = f0;
  bool a_route = false;
  int a_pos = -1, a_b = 0, a_lo = 0, a_hi = 0, a_L = 0;
  int b_pos = -1, b_page = -1, b_off = 0;
  bool a_live = false, b_live = false, bad_route = false, bad_page = false;
  const int key = lane & 15;
  auto step_a = [&]() {
    a_live = lf < f1;
    a_pos = -1;
    a_route = false;
    if (a_live) {
      cursor_settle<SHARED>(a, sh, shared, lc);
      a_b = lc.b;
      int j = lc.tile * kTile + key;
      if (j < lc.set.n) {
        if (j < lc.set.early) a_pos = j;
        else if ((j -= lc.set.early) < lc.set.recent) a_pos = lc.set.first + j;
        else {
          a_route = true;
          a_pos = __ldg(a.route + (int64_t)a_b * a.route_stride + (j - lc.set.recent));
          a_lo = lc.set.early;
          a_hi = lc.set.first;
          a_L = lc.set.L;
        }
      }
      ++lf;
      ++lc.tile;
    }
  };
  auto step_b = [&]() {
    b_live = a_live;
    b_pos = a_pos;
    if (a_route) {
      if (b_pos < 0 || b_pos >= a_L) {
        bad_route |= b_pos != -1;
        b_pos = -1;
      } else if (b_pos < a_lo || b_pos >= a_hi) {
        b_pos = -1;
      }
    }
    b_page = -1;
    if (b_pos >= 0) {
      const int pg = b_pos / a.page_size;
      b_off = b_pos - pg * a.page_size;
      b_page = __ldg(a.page_table + (int64_t)a_b * a.table_stride + pg);
    }
  };
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * S * kStage;
  auto step_c = [&](int slot) {
    if (b_live) {
      bool ok = b_pos >= 0;
      if (ok && (b_page < 0 || b_page >= a.num_pages)) { bad_page = true; ok = false; }
      const int64_t ko = ok ? (int64_t)b_page * a.k_sp + (int64_t)b_off * a.k_st + (int64_t)g * a.k_sh : 0;
      const int64_t vo = ok ? (int64_t)b_page * a.v_sp + (int64_t)b_off * a.v_st + (int64_t)g * a.v_sh : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      if (lane == 0) masks[warp * S + slot] = m;
      // eight lanes a row: lane l takes the 16-byte chunks l % 8 + 8 j of the rows l / 8 + 4 i,
      // so that an address is worked out once a row and the chunks are constant offsets
      const int c8 = lane & 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + (lane >> 3);
        const __nv_bfloat16* ks = a.k + __shfl_sync(0xffffffffu, ko, row) + c8 * 8;
        const __nv_bfloat16* vs = a.v + __shfl_sync(0xffffffffu, vo, row) + c8 * 8;
        const uint32_t n = (m >> row) & 1u ? 16u : 0u;
        const uint32_t sw = (uint32_t)((c8 ^ (row & 7)) << 4);
        const uint32_t kd = ring + (uint32_t)slot * kStage + (uint32_t)row * (DQK * 2) + sw;
        const uint32_t vd = ring + (uint32_t)slot * kStage + kTile * DQK * 2 + (uint32_t)row * (DV * 2) + sw;
#pragma unroll
        for (int j = 0; j < DQK / 64; ++j) cp_async_16(kd + 128 * j, ks + 64 * j, n);
#pragma unroll
        for (int j = 0; j < DV / 64; ++j) cp_async_16(vd + 128 * j, vs + 64 * j, n);
      }
    }
    cp_async_commit();
  };

  step_a();
  step_b();
  step_a();
  for (int s = 0; s < S - 1; ++s) {
    step_c(s);
    step_b();
    step_a();
  }

  // ---- the run, a sequence at a time ----
  const int g4 = lane >> 2, t4 = lane & 3;
  int slot = 0;
  int64_t f = f0;
  while (f < f1) {
    cursor_settle<SHARED>(a, sh, shared, cc);
    const int tiles = (int)min(f1 - f, (int64_t)(cc.nt - cc.tile));
    const __nv_bfloat16* qrow = a.q + (int64_t)cc.b * a.q_sb;
    auto load_q = [&](uint32_t (&f)[4], int ks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = g4 + (i & 1) * 8, d = ks * 16 + 2 * t4 + (i >> 1) * 8;
        f[i] = r < nh ? *reinterpret_cast<const uint32_t*>(qrow + (int64_t)(h0 + r) * a.q_sh + d) : 0u;
      }
    };
    uint32_t qf[QREG ? KS : 1][4];
    if (QREG) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) load_q(qf[QREG ? ks : 0], ks);
    }
    float o[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows g4 and g4 + 8
    uint32_t seen = 0u;                                        // whether any position was attended

    for (int it = 0; it < tiles; ++it) {
      cp_async_wait_pending(S - 2);
      __syncwarp();
      step_c(slot == 0 ? S - 1 : slot - 1);
      step_b();
      step_a();
      const uint32_t kd = ring + (uint32_t)slot * kStage, vd = kd + kTile * DQK * 2;
      const uint32_t mask = masks[warp * S + slot];
      seen |= mask;
      slot = slot + 1 == S ? 0 : slot + 1;
      // S = Q K^T: two halves of 8 positions
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int mtx = lane >> 3, r = (mtx >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t kf[4];
          ldsm4(kf, kd + (uint32_t)(r * DQK * 2 + (((2 * ks + (mtx & 1)) ^ (r & 7)) << 4)));
          if (QREG) {
            mma16816(s[0], qf[QREG ? ks : 0], kf[0], kf[1]);
            mma16816(s[1], qf[QREG ? ks : 0], kf[2], kf[3]);
          } else {
            uint32_t f[4];
            load_q(f, ks);
            mma16816(s[0], f, kf[0], kf[1]);
            mma16816(s[1], f, kf[2], kf[3]);
          }
        }
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * j + 2 * t4 + (i & 1);
          s[j][i] = (mask >> c) & 1u ? s[j][i] * a.scale_log2 : -INFINITY;
          top[i >> 1] = fmaxf(top[i >> 1], s[j][i]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > mx[0] + kRaise || top[1] > mx[1] + kRaise)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float nm = fmaxf(mx[i], top[i]);
          const float c = nm == -INFINITY ? 1.f : ex2_approx(mx[i] - nm);
          mx[i] = nm;
          l[i] *= c;
#pragma unroll
          for (int n = 0; n < NV; ++n) { o[n][2 * i] *= c; o[n][2 * i + 1] *= c; }
        }
      }
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = mx[i] == -INFINITY ? 0.f : mx[i];
          const float p0 = ex2_approx(s[j][2 * i] - m), p1 = ex2_approx(s[j][2 * i + 1] - m);
          l[i] += p0 + p1;
          split2(p0, p1, ph[2 * j + i], pl[2 * j + i]);
        }
      {
        const int mtx = lane >> 3, r = (mtx & 1) * 8 + (lane & 7);
#pragma unroll
        for (int n = 0; n < NV; n += 2) {
          uint32_t vf[4];
          ldsm4_t(vf, vd + (uint32_t)(r * DV * 2 + (((n + (mtx >> 1)) ^ (r & 7)) << 4)));
          mma16816(o[n], ph, vf[0], vf[1]);
          mma16816(o[n + 1], ph, vf[2], vf[3]);
          mma16816(o[n], pl, vf[0], vf[1]);
          mma16816(o[n + 1], pl, vf[2], vf[3]);
        }
      }
    }

    // ---- the pair's result, or this run's part of it ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      // attended, and every score -inf: 0 / 0; in a part -1, which a finite maximum wipes out
      if (l[i] == 0.f && seen != 0u) l[i] = !SHARED && tiles == cc.nt ? NAN : -1.f;
    }
    if (tiles == cc.nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = g4 + 8 * i;
        if (row < nh) {
          const int64_t r = (int64_t)cc.b * a.Hq + h0 + row;
          if constexpr (SHARED) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
              *reinterpret_cast<float2*>(sh.rows + r * DV + n * 8 + 2 * t4) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
            if (t4 == 0) *reinterpret_cast<float2*>(sh.rows + (int64_t)a.B * a.Hq * DV + 2 * r) = make_float2(mx[i], l[i]);
          } else {
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];   // no position: 0; a NaN sum stays NaN
#pragma unroll
            for (int n = 0; n < NV; ++n)
              *reinterpret_cast<__nv_bfloat162*>(a.out + r * DV + n * 8 + 2 * t4) =
                  __floats2bfloat162_rn(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
            if (t4 == 0 && a.lse != nullptr) a.lse[r] = fmaf(mx[i], 0.6931471805599453f, logf(l[i]));
          }
        }
      }
    } else {
      float* part = reinterpret_cast<float*>(a.ws + paged_prefix_bytes(a.B)) +
                    (((size_t)worker * HK + hk) * 2 + (f == f0 ? 0 : 1)) * paged_part_floats(DV);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = g4 + 8 * i;
        if (row < nh) {
#pragma unroll
          for (int n = 0; n < NV; ++n)
            *reinterpret_cast<float2*>(part + row * DV + n * 8 + 2 * t4) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
          if (t4 == 0) {
            part[kHeads * DV + row] = mx[i];
            part[kHeads * DV + kHeads + row] = l[i];
          }
        }
      }
    }
    cc.tile += tiles;
    f += tiles;
  }
  cp_async_wait_pending(0);
  if (bad_route) record_error(a.err, IRS_DEVERR_ROUTE_ID);
  if (bad_page) record_error(a.err, IRS_DEVERR_PAGE);
  if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the parts of the (sequence, head) pairs that warp borders cut, and writes the empty
// ones. A block has Dv/4 column lanes and groups of them: `pg` groups share a row, each taking
// every pg-th part with its own running maximum; they are then joined in order. A thread gets
// four parts, all in flight together, where there are groups enough.
template <int DV>
__global__ void __launch_bounds__(1024) paged_join_kernel(PagedArgs a, int nhb, int workers) {
  constexpr int CL = DV / 4;
  __shared__ float4 sm_o[1024];
  __shared__ float2 sm_ml[1024 / CL];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int HK = a.Hkv * nhb;
  const int b = blockIdx.x / HK, hk = blockIdx.x % HK;
  const int64_t* pre = reinterpret_cast<const int64_t*>(a.ws);
  const int64_t p0 = pre[b], nt = pre[b + 1] - p0;
  const int64_t share = paged_share(pre[a.B], workers);
  const int64_t F0 = p0, F1 = p0 + nt;
  const int g = hk / nhb, hb = hk % nhb;
  const int h0 = g * a.G + hb * kHeads, nh = min(kHeads, a.G - hb * kHeads);
  const int cl = threadIdx.x % CL, grp = threadIdx.x / CL, groups = (int)blockDim.x / CL;
  int c0 = 0, c1 = -1;
  if (nt > 0) {
    c0 = (int)(F0 / share);
    c1 = (int)((F1 - 1) / share);
    if (c0 == c1) return;
  }
  int pg = 1;
  while (2 * pg <= groups && 4 * pg < c1 - c0 + 1) pg *= 2;
  const int part_grp = grp % pg, row_grp = grp / pg, rows = groups / pg;
  const float* parts = reinterpret_cast<const float*>(a.ws + paged_prefix_bytes(a.B));
  for (int rb = blockIdx.y * rows; rb < nh; rb += gridDim.y * rows) {
    const int row = row_grp < rows ? rb + row_grp : nh;
    float M = -INFINITY, ls = 0.f;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m, float l, const float4& x) {   // a part with its own maximum
      const float n = fmaxf(M, m);
      const float u = n == -INFINITY ? 0.f : ex2_approx(M - n), v = n == -INFINITY ? 0.f : ex2_approx(m - n);
      M = n;
      ls = n == -INFINITY ? ls + l : fmaf(ls, u, l * v);
      s.x = fmaf(s.x, u, x.x * v);
      s.y = fmaf(s.y, u, x.y * v);
      s.z = fmaf(s.z, u, x.z * v);
      s.w = fmaf(s.w, u, x.w * v);
    };
    if (row < nh) {
      constexpr int U = 4;
      for (int c = c0 + part_grp; c <= c1; c += U * pg) {
        float m[U], l[U];
        float4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int ci = c + i * pg;
          m[i] = -INFINITY;
          l[i] = 0.f;
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (ci <= c1) {
            // the sequence's first part is its run's second, unless the run starts with it
            const float* p = parts + (((size_t)ci * HK + hk) * 2 + (ci == c0 && F0 != (int64_t)c0 * share ? 1 : 0)) * paged_part_floats(DV);
            m[i] = p[kHeads * DV + row];
            l[i] = p[kHeads * DV + kHeads + row];
            x[i] = *reinterpret_cast<const float4*>(p + row * DV + 4 * cl);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) add(m[i], l[i], x[i]);
      }
    }
    if (pg > 1) {
      sm_o[threadIdx.x] = s;
      if (cl == 0) sm_ml[grp] = make_float2(M, ls);
      __syncthreads();
      if (part_grp == 0)
        for (int i = 1; i < pg; ++i) add(sm_ml[grp + i].x, sm_ml[grp + i].y, sm_o[threadIdx.x + i * CL]);
      __syncthreads();
    }
    if (part_grp == 0 && row < nh) {
      if (ls < 0.f) ls = NAN;
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      const int64_t r = (int64_t)b * a.Hq + h0 + row;
      __nv_bfloat162 y[2] = {__floats2bfloat162_rn(s.x * inv, s.y * inv), __floats2bfloat162_rn(s.z * inv, s.w * inv)};
      *reinterpret_cast<uint2*>(a.out + r * DV + 4 * cl) = *reinterpret_cast<const uint2*>(y);
      if (cl == 0 && a.lse != nullptr) a.lse[r] = fmaf(M, 0.6931471805599453f, logf(ls));
    }
  }
}

template <int DQK, int DV>
cudaError_t launch_decode(const PagedArgs& a, int num_sms, bool* configured, cudaStream_t stream) {
  if (!*configured) {
    const cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<DQK, DV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(kRingBytes + 256));
    if (e != cudaSuccess) return e;
    *configured = true;
  }
  const int nhb = (a.G + kHeads - 1) / kHeads;
  const PagedGrid pg = paged_grid(DQK, DV, a.Hkv * nhb, num_sms);
  paged_decode_kernel<DQK, DV, false><<<pg.ctas, 32 * pg.warps, pg.smem, stream>>>(a, pg, nhb, PagedAlone{});
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // About four parts a thread: a sequence has workers / B of them when the lengths are alike.
  // (One long sequence: 32 groups a row, a row a block. 16 sequences of 8000 with 8 heads, 10
  // parts each: 28 us when every row had 32 groups all the same.)
  const int pairs = a.B * a.Hkv * nhb, rows = a.G < kHeads ? a.G : kHeads;
  int per_row = 1;
  while (per_row < 32 && 4 * per_row < pg.workers / a.B) per_row *= 2;
  const int most = per_row == 32 ? 1024 : 512;
  int threads = (rows * per_row * (DV / 4) + 31) / 32 * 32;
  if (threads > most) threads = most;
  const int in_block = threads / (DV / 4);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)pairs, (unsigned)((rows * per_row + in_block - 1) / in_block));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<DV>, a, nhb, pg.workers);
}

// The own positions of sequences that share prefixes: the next kernel of the stream may start before
// the kernel before this one ends, and so may this one.
template <int DQK, int DV>
cudaError_t launch_shared(const PagedArgs& a, const PagedShared& sh, int num_sms, bool* configured, int* workers, cudaStream_t stream) {
  if (!*configured) {
    const cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<DQK, DV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(kRingBytes + 256));
    if (e != cudaSuccess) return e;
    *configured = true;
  }
  const int nhb = (a.G + kHeads - 1) / kHeads;
  const PagedGrid pg = paged_grid(DQK, DV, a.Hkv * nhb, num_sms);
  *workers = pg.workers;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)pg.ctas);
  cfg.blockDim = dim3((unsigned)(32 * pg.warps));
  cfg.dynamicSmemBytes = pg.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_kernel<DQK, DV, true>, a, pg, nhb, sh);
}

}  // namespace

size_t paged_workspace_bytes(int B, int Dv) {
  return paged_prefix_bytes(B) + (size_t)kMaxPagedCtas * kMaxWarps * 2 * paged_part_floats(Dv) * 4;
}

cudaError_t launch_paged_decode(const PagedArgs& a, int num_sms, bool* configured, cudaStream_t stream) {
  const int i = (a.Dqk / 64 - 1) * 3 + (a.Dv == 64 ? 0 : a.Dv == 128 ? 1 : 2);
  switch (i) {
    case 0: return launch_decode<64, 64>(a, num_sms, configured + i, stream);
    case 1: return launch_decode<64, 128>(a, num_sms, configured + i, stream);
    case 2: return launch_decode<64, 256>(a, num_sms, configured + i, stream);
    case 3: return launch_decode<128, 64>(a, num_sms, configured + i, stream);
    case 4: return launch_decode<128, 128>(a, num_sms, configured + i, stream);
    case 5: return launch_decode<128, 256>(a, num_sms, configured + i, stream);
    case 6: return launch_decode<192, 64>(a, num_sms, configured + i, stream);
    case 7: return launch_decode<192, 128>(a, num_sms, configured + i, stream);
    case 8: return launch_decode<192, 256>(a, num_sms, configured + i, stream);
    case 9: return launch_decode<256, 64>(a, num_sms, configured + i, stream);
    case 10: return launch_decode<256, 128>(a, num_sms, configured + i, stream);
    default: return launch_decode<256, 256>(a, num_sms, configured + i, stream);
  }
}

cudaError_t launch_paged_shared(const PagedArgs& a, const PagedShared& sh, int num_sms, bool* configured, int* workers, cudaStream_t stream) {
  const int i = (a.Dqk / 64 - 1) * 2 + (a.Dv / 64 - 1);
  switch (i) {
    case 0: return launch_shared<64, 64>(a, sh, num_sms, configured + i, workers, stream);
    case 1: return launch_shared<64, 128>(a, sh, num_sms, configured + i, workers, stream);
    case 2: return launch_shared<128, 64>(a, sh, num_sms, configured + i, workers, stream);
    case 3: return launch_shared<128, 128>(a, sh, num_sms, configured + i, workers, stream);
    case 4: return launch_shared<192, 64>(a, sh, num_sms, configured + i, workers, stream);
    default: return launch_shared<192, 128>(a, sh, num_sms, configured + i, workers, stream);
  }
}

}  // namespace irs

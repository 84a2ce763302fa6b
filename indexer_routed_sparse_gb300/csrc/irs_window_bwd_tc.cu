// Window attention on the tensor cores (tcgen05 + TMEM + TMA): the backward.
//
// Mathematics as in irs_window.cu, from the saved out and lse:
//   p = e^{scale q.k - lse},  ds = p (dout.v - D),  D = dout.out
//   dq = scale sum_s ds k,    dk = scale sum ds q,    dv = sum p dout
//
// Two kernels, each with its own sums in TMEM, so that nothing is added in memory and every
// run gives the same bits; the price is computing the scores and dout.v twice (7 products
// for 5). Adding dq tiles in memory instead would move an FP32 dq once for every key tile of
// the window: at window 512 about 8 GB against 1.6 GB of other traffic (T 32768, 64 heads of
// 192), four times the cost of the two products.
//
// * dq (also D): rows of a product are the query heads of 128 / G queries, as in the forward.
//   S = Q K^T and dP = dO V^T for a block of 96 keys; two warpgroups (48 keys each, one row a
//   thread) form dS and leave it in TMEM as bf16, the first operand of dQ += dS K (K read
//   MN-major). S and dP are read out at once, so the next block's products run
//   meanwhile. Four helper warps form D for the next item and store the last item's dq: done
//   by the score warps these took 13,000 of an item's 34,000 cycles (192/128, window 512).
// * dk, dv: rows are 128 keys, columns the rows (query, head) that see them, 64 at a time:
//   S^T = K Q^T, dP^T = V dO^T; P^T and dS^T return to TMEM as bf16, first operands of
//   dV += P^T dO and dK += dS^T Q. With Dqk = 192 and Dv = 128 the TMEM is full to the last
//   column: 64 + 64 scores, 32 + 32 weights, 128 + 192 sums. One warp issues the scores,
//   another the sums: a wait that succeeds at once still costs the issuer 115 cycles, and so
//   one's waits lie under the other's products. Copies, and the loads of lse and D, have a
//   warp each: together in one warp the loads' 1,300 cycles a block held the copies up.
//   Each tile starts at another of its query blocks (dkv_item). At T 32768, 64 / 4 heads of
//   192 / 128, window 512, 4 first tokens: one issuer and one loading warp 1.63 ms, split
//   1.56, tiles in step 1.46 (4.1 GB from DRAM); the products alone, at the rates measured
//   for these shapes, take 1.14.
// * First tokens are seen by every later query of their document, so their sums are long.
//   Queries beyond the window are cut into stretches, each an item of its own (one tile of
//   first-token keys) with FP32 partial sums in the workspace; a small kernel adds a first
//   token's window part and its stretches in order. Documents with one stretch's queries or
//   fewer beyond the window leave them to the window's tile: partial sums then grow with the
//   tokens, not with the documents (4000 documents of 16 tokens, window 8, 64 first tokens, 8
//   heads of 192 / 128 would have 5.4 GB of them).
// * Roundings: P and dS are bf16 as first operands (half a step, 2^-8, of each, on products
//   whose sums are FP32); D comes from the bf16 output the caller kept, as in the routed
//   attention's backward: half a step of the output, which tells only where a row sees a few
//   keys (the exact D = sum p dP would need a pass over the scores before dS).
// * 0 times an infinity or NaN of a masked row is NaN: rows and keys whose result is not
//   finite are computed again from what they see alone, outside the pipelines, whose waits have
//   a limit: a row or key takes as long as its window. Rows of dq are marked (a NaN in the
//   first column, the item in shared memory) and done when the CTA is through with its items.
//   A bad query reaches all 128 keys of every tile that loads it, so marked keys (a bit each in
//   the workspace) are spread over the GPU by a last small kernel, a block a key.
// * Measured at the size above: dq 1.03 ms (of its issuing warp's 1.98 million cycles, 1.28
//   are products on their way, 1.09 by the rates of their shapes; 64 / 4 heads: tiles of 8
//   queries), dk and dv 1.47 ms; looking for marked keys 2 us where there are none.
#include <climits>

#include "irs_internal.h"
#include "irs_ptx.cuh"
#include "irs_window_rows.cuh"

namespace irs {

namespace {

constexpr int kBlk = 128;               // keys a tile (dk, dv)
constexpr int kCols = 64;               // (query, head) rows a block (dk, dv)
constexpr uint32_t kAtom = 128 * 128;   // 128 rows x 64 bf16
constexpr uint32_t kAtom64 = 64 * 128;  // 64 rows x 64 bf16
constexpr int kDqThreads = 448;         // warps 0-7: score warps; 8: TMA; 9: MMA; 10-13: helpers
constexpr int kDkvThreads = 640;        // warps 0-15: score warps; 16: lse and D; 17, 18: MMA; 19: TMA

// A word that says whether any key is marked, then a bit a key.
__host__ __device__ inline int64_t redo_words(int T, int Hkv) { return 1 + ((int64_t)T * Hkv + 31) / 32; }
// (out of line: inlined into the dq kernel it costs that eight spilled registers)
__device__ __noinline__ void redo_clear(const WinArgs& a) {
  const int64_t words = redo_words(a.T, a.Hkv);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) a.redo[i] = 0u;
}
__device__ __forceinline__ void redo_mark(const WinArgs& a, int64_t row) {
  atomicOr(a.redo + 1 + (row >> 5), 1u << (row & 31));   // a set: the order does not matter
  a.redo[0] = 1u;
}

__device__ __forceinline__ void wait_landed(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kWaitLimitNs) {}
}

// D (+)= A . B with A (bf16, one row a lane) in TMEM and B a [row][dim] tile read MN-major:
// NK steps of 16 rows, 64-dim atoms `atom` bytes apart.
template <int NK>
__device__ __forceinline__ void ts_run(uint32_t d, uint32_t at, uint32_t bb, uint32_t atom, uint32_t idesc, bool accumulate) {
  const uint64_t b0 = sdesc_sw128(bb, atom, 1024);
#pragma unroll
  for (int ks = 0; ks < NK; ++ks)
    umma_bf16_ts_warp(d, at + 8 * ks, b0 + (uint64_t)((ks * 2048) >> 4), idesc, (accumulate || ks > 0) ? 1u : 0u);
}
// D = A . B^T, both K-major over NA 64-dim atoms.
template <int NA>
__device__ __forceinline__ void ss_run(uint32_t d, uint32_t ab, uint32_t a_atom, uint32_t bb, uint32_t b_atom, uint32_t idesc) {
  const uint64_t a0 = sdesc_sw128(ab, 16, 1024), b0 = sdesc_sw128(bb, 16, 1024);
#pragma unroll
  for (int ks = 0; ks < 4 * NA; ++ks)
    umma_bf16_warp(d, a0 + (uint64_t)(((ks >> 2) * a_atom + (ks & 3) * 32) >> 4),
              b0 + (uint64_t)(((ks >> 2) * b_atom + (ks & 3) * 32) >> 4), idesc, ks > 0);
}

// ---------------------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------------------
template <int DQK, int DV>
struct DqCfg {
  static constexpr int QA = DQK / 64, VA = DV / 64;
  static constexpr uint32_t q_bytes = QA * kAtom, do_bytes = VA * kAtom;
  // Three stages of keys (a block's keys stay until its dS K, two blocks' products later) and as
  // many of values as fit beside a tile's queries and dout.
  static constexpr bool fits(int blk, int vs) {
    return q_bytes + do_bytes + (3 * QA + vs * VA) * blk * 128 <= 212u * 1024u;
  }
  static constexpr int BLK = 96;                                // three pieces of 16 keys for each score warp
  static constexpr int KS = 3, VS = fits(BLK, 2) ? 2 : 1;
  static constexpr uint32_t kv_atom = BLK * 128, k_bytes = QA * kv_atom, v_bytes = VA * kv_atom;
  static constexpr uint32_t do_off = q_bytes, k_off = q_bytes + do_bytes, v_off = k_off + KS * k_bytes;
  static constexpr uint32_t row_off = v_off + VS * v_bytes;     // [2][128] of an item's rows: D, lse (base 2), window, document
  static constexpr uint32_t hdr_off = row_off + 2 * 128 * 16;   // [2][8] of an item: range and borders
  static constexpr uint32_t plan_off = hdr_off + 2 * 32;        // [2][4] its blocks, for the MMA warp
  static constexpr uint32_t bar_off = plan_off + 2 * 16;
  static constexpr uint32_t redo_off = bar_off + 24 * 8 + 16;   // [4][2] first and last item of a helper warp with marked rows
  static constexpr uint32_t cu_off = redo_off + 4 * 8;
  static constexpr int cu_cap = 2048;
  static constexpr uint32_t total = cu_off + 4 * cu_cap + 1024;
  static constexpr uint32_t S0 = 0, P0 = 128, DS0 = 256, DQ0 = 320;   // TMEM columns
};

// The keys of one tile of `qt` queries from t0 on: the first `sb` blocks hold the first tokens
// before the range, where there are any.
struct DqItem {
  int t0, last, ds0, klo, ns, sb, nbt;
};
template <int kBlk>
__device__ __forceinline__ DqItem dq_item(const WinArgs& a, const int32_t* cu, int t0, int qt) {
  DqItem m;
  m.t0 = t0;
  m.last = min(t0 + qt, a.T) - 1;
  m.ds0 = window_doc(cu, a.ndocs, a.T, t0).start;
  m.klo = max(m.ds0, t0 - a.window + 1);
  m.ns = max(0, min(m.ds0 + a.sinks, m.klo) - m.ds0);
  m.sb = (m.ns + kBlk - 1) / kBlk;
  m.nbt = (m.last - m.klo) / kBlk + 1 + m.sb;
  return m;
}
template <int kBlk>
__device__ __forceinline__ int dq_key(const DqItem& m, int j) {
  return j < m.sb ? m.ds0 + kBlk * j : m.klo + kBlk * (j - m.sb);
}
template <int kBlk>
__device__ __forceinline__ int dq_cols(const DqItem& m, int j) {
  const int n = min(kBlk, j < m.sb ? m.ns - kBlk * j : m.last - dq_key<kBlk>(m, j) + 1);
  return (n + 31) & ~31;
}

template <int DQK, int DV>
__global__ void __launch_bounds__(kDqThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, WinArgs a, int qt,
                     int tiles) {
  using C = DqCfg<DQK, DV>;
  constexpr int KS = C::KS, VS = C::VS, BLK = C::BLK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  volatile float* rows = reinterpret_cast<volatile float*>(smem + C::row_off);
  volatile int* head = reinterpret_cast<volatile int*>(smem + C::hdr_off);
  volatile int* plan = reinterpret_cast<volatile int*>(smem + C::plan_off);
  int* redo = reinterpret_cast<int*>(smem + C::redo_off);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::bar_off);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;    // [3]
  uint64_t* k_empty = k_full + 3;
  uint64_t* v_full = k_empty + 3;    // [2]
  uint64_t* v_empty = v_full + 2;
  uint64_t* sp_full = v_empty + 2;   // scores and dP of a block
  uint64_t* sp_empty = sp_full + 1;  // ... have been read
  uint64_t* ds_full = sp_empty + 1;
  uint64_t* ds_empty = ds_full + 1;  // dS has been read by its product
  uint64_t* dq_full = ds_empty + 1;
  uint64_t* dq_empty = dq_full + 1;
  uint64_t* d_full = dq_empty + 1;   // [2] an item's rows and head
  uint64_t* d_empty = d_full + 2;
  uint64_t* drain = d_empty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 1);
    for (int i = 0; i < KS; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1);
      mbar_init(&d_full[i], 4); mbar_init(&d_empty[i], 8);
    }
    mbar_init(sp_full, 1); mbar_init(sp_empty, 8);
    mbar_init(ds_full, 8); mbar_init(ds_empty, 1);
    mbar_init(dq_full, 1); mbar_init(dq_empty, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  if (tid < 4) {
    redo[2 * tid] = INT_MAX;
    redo[2 * tid + 1] = -1;
  }
  check_documents(a);
  const int32_t* cu = a.cu;
  if (a.ndocs < C::cu_cap) {   // searched for every item by every row
    int32_t* near = reinterpret_cast<int32_t*>(smem + C::cu_off);
    for (int i = tid; i <= a.ndocs; i += kDqThreads) near[i] = a.cu[i];
    cu = near;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int items = tiles * a.Hkv;

  if (warp == 8) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_do);
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      const uint32_t box = (uint32_t)(qt * a.G) * 128u;
      uint32_t nq = 0, nk = 0, nv = 0, ks = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const int tile = item / a.Hkv, g = item - tile * a.Hkv;
        const DqItem m = dq_item<BLK>(a, cu, tile * qt, qt);
        volatile int* pl = plan + 4 * (nq & 1);   // read before the last scores of two items ago
        pl[0] = m.nbt;
        pl[1] = (m.sb > 0 ? dq_cols<BLK>(m, m.sb - 1) : 0) | dq_cols<BLK>(m, m.nbt - 1) << 8 | m.sb << 16;
        if (nq > 0 && !mbar_wait(q_empty, (nq - 1) & 1, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(q_full, box * (C::QA + C::VA));
        for (int c = 0; c < C::QA; ++c) tma_load_3d(smem + c * kAtom, &tm_q, c * 64, g * a.G, m.t0, q_full);
        for (int c = 0; c < C::VA; ++c) tma_load_3d(smem + C::do_off + c * kAtom, &tm_do, c * 64, g * a.G, m.t0, q_full);
        ++nq;
        for (int j = 0; j < m.nbt; ++j) {
          const int kb = dq_key<BLK>(m, j);
          const uint32_t vs = nv % VS;
          if (nk >= KS && !mbar_wait(&k_empty[ks], (nk / KS - 1) & 1, abort_flag, a.err)) { ok = false; break; }
          mbar_arrive_expect_tx(&k_full[ks], C::k_bytes);
          for (int c = 0; c < C::QA; ++c)
            tma_load_3d(smem + C::k_off + ks * C::k_bytes + c * C::kv_atom, &tm_k, c * 64, g, kb, &k_full[ks]);
          ++nk;
          if (++ks == KS) ks = 0;
          if (nv >= VS && !mbar_wait(&v_empty[vs], (nv / VS - 1) & 1, abort_flag, a.err)) { ok = false; break; }
          mbar_arrive_expect_tx(&v_full[vs], C::v_bytes);
          for (int c = 0; c < C::VA; ++c)
            tma_load_3d(smem + C::v_off + vs * C::v_bytes + c * C::kv_atom, &tm_v, c * 64, g, kb, &v_full[vs]);
          ++nv;
        }
      }
      if (*abort_flag) {
        if (nq > 0) wait_landed(q_full, (nq - 1) & 1);
        for (uint32_t i = nk > KS ? nk - KS : 0; i < nk; ++i) wait_landed(&k_full[i % KS], (i / KS) & 1);
        for (uint32_t i = nv > VS ? nv - VS : 0; i < nv; ++i) wait_landed(&v_full[i % VS], (i / VS) & 1);
      }
    }
  } else if (warp == 9) {
    // ---------------- MMA issuer (the whole warp; one elected lane issues) ----------------
    constexpr uint32_t DQ_IDESC = idesc_bf16(128, DQK, false, true);
    const uint32_t sb = smem_u32(smem), tb = (uint32_t)uniform((int)tbase);
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)); };
    uint32_t nv = 0, nsp = 0, nds = 0, ni = 0, ks = 0, kph = 0, kd = 0;   // kd: stage of the block whose dS comes next
    bool alive = true;
    auto scores = [&](int cols) {
      const uint32_t vs = nv % VS;
      if (!wait(&k_full[ks], kph)) return false;
      if (nsp > 0 && !wait(sp_empty, (nsp - 1) & 1)) return false;
      tc_fence_after();
      const uint32_t idesc = idesc_bf16(128, cols, false, false);
      ss_run<C::QA>(tb + C::S0, sb, kAtom, sb + C::k_off + ks * C::k_bytes, C::kv_atom, idesc);
      if (!wait(&v_full[vs], (nv / VS) & 1)) return false;
      tc_fence_after();
      ss_run<C::VA>(tb + C::P0, sb + C::do_off, kAtom, sb + C::v_off + vs * C::v_bytes, C::kv_atom, idesc);
      umma_commit_warp(sp_full);
      umma_commit_warp(&v_empty[vs]);
      ++nv; ++nsp;
      if (++ks == KS) { ks = 0; kph ^= 1u; }
      return true;
    };
    for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
      if (!wait(q_full, ni & 1)) break;
      const volatile int* pl = plan + 4 * (ni & 1);
      const int nbt = uniform(pl[0]), pc = uniform(pl[1]);
      const int colsS = pc & 0xff, colsL = pc >> 8 & 0xff, sb1 = (pc >> 16) - 1;
      auto cols_of = [&](int j) { return j == sb1 ? colsS : j == nbt - 1 ? colsL : BLK; };
      if (!scores(cols_of(0))) break;
      if (nbt == 1) umma_commit_warp(q_empty);
      for (int j = 0; j < nbt; ++j) {
        if (j + 1 < nbt) {
          if (!scores(cols_of(j + 1))) { alive = false; break; }
          if (j + 2 == nbt) umma_commit_warp(q_empty);
        }
        if (!wait(ds_full, nds & 1)) { alive = false; break; }
        ++nds;
        if (j == 0 && ni > 0 && !wait(dq_empty, (ni - 1) & 1)) { alive = false; break; }
        tc_fence_after();
        const uint32_t kb = sb + C::k_off + kd * C::k_bytes;
        switch (cols_of(j) >> 5) {
          case 1: ts_run<2>(tb + C::DQ0, tb + C::DS0, kb, C::kv_atom, DQ_IDESC, j > 0); break;
          case 2: ts_run<4>(tb + C::DQ0, tb + C::DS0, kb, C::kv_atom, DQ_IDESC, j > 0); break;
          default: ts_run<6>(tb + C::DQ0, tb + C::DS0, kb, C::kv_atom, DQ_IDESC, j > 0); break;
        }
        umma_commit_warp(ds_empty);
        umma_commit_warp(&k_empty[kd]);
        if (++kd == KS) kd = 0;
      }
      if (!alive) break;
      umma_commit_warp(dq_full);
    }
    umma_commit_warp(drain);
    wait_landed(drain, 0);
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- helpers: the next item's D, lse and borders; the last item's dq ----------------
    constexpr int LR = DV / 8, RW = 32 / LR, U = 8;   // lanes a row; rows a step; steps in flight together
    const uint32_t lanes = tmem_lane_base(warp);
    const int rb = (warp - 10) * 32;                  // D: the warp's rows
    const int orq = (rb + lane) / a.G;                // the lane's own one
    const int orow = orq * a.Hq + (rb + lane) - orq * a.G;
    uint32_t ni = 0;
    int prev = -1;
    for (int item = blockIdx.x;; item += gridDim.x, ++ni) {
      if (item < items) {
        const int tile = item / a.Hkv, g = item - tile * a.Hkv;
        const uint32_t slot = ni & 1;
        if (ni >= 2 && !__all_sync(0xffffffffu, mbar_wait(&d_empty[slot], (ni / 2 - 1) & 1, abort_flag, a.err))) break;
        const DqItem m = dq_item<BLK>(a, cu, tile * qt, qt);
        const int64_t base = (int64_t)m.t0 * a.Hq + g * a.G;
        const int t = m.t0 + orq;
        const bool in = orq < qt && t < a.T;
        const int mine = in ? orow : -1;
        const float l = in ? a.lse_in[base + orow] : 0.f;
        volatile float* dst = rows + slot * 512;
        // eight steps' loads in flight; their sums over a row's lanes are folded together, each
        // exchange halving what a lane still holds (8 shuffles for 8 steps)
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += U * RW) {
          uint4 u[U], w[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int o = __shfl_sync(0xffffffffu, mine, r0 + i * RW + lane / LR);
            u[i] = w[i] = make_uint4(0, 0, 0, 0);
            if (o >= 0) {
              u[i] = *reinterpret_cast<const uint4*>(a.dout + (base + o) * DV + 8 * (lane % LR));
              w[i] = *reinterpret_cast<const uint4*>(a.out + (base + o) * DV + 8 * (lane % LR));
            }
          }
          float s[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const uint32_t uu[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x = fmaf(__uint_as_float(uu[k] << 16), __uint_as_float(ww[k] << 16), x);
              y = fmaf(__uint_as_float(uu[k] & 0xffff0000u), __uint_as_float(ww[k] & 0xffff0000u), y);
            }
            s[i] = x + y;
          }
          int step = 0;
#pragma unroll
          for (int n = U / 2, o = LR / 2; n > 0; n >>= 1, o >>= 1) {
            const bool hi = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const float keep = hi ? s[i + n] : s[i], send = hi ? s[i] : s[i + n];
              s[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            if (hi) step += n;
          }
          if (LR == 16) s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);   // two lanes hold the same step
          dst[4 * (rb + r0 + step * RW + lane / LR)] = s[0];
        }
        const int ds = window_doc(cu, a.ndocs, a.T, min(t, a.T - 1)).start;
        dst[4 * (rb + lane) + 1] = l * kLog2e;
        dst[4 * (rb + lane) + 2] = __int_as_float(max(ds, t - a.window + 1));
        dst[4 * (rb + lane) + 3] = __int_as_float(ds);
        if (warp == 10 && lane == 0) {
          volatile int* h = head + 8 * slot;
          h[0] = m.klo;
          h[1] = m.ns;
          h[2] = m.nbt;
          h[3] = max(window_doc(cu, a.ndocs, a.T, m.last).start, m.last - a.window + 1);
          h[4] = m.ds0;
          h[5] = m.last;
        }
        __syncwarp();
        if (in) a.delta[base + orow] = dst[4 * (rb + lane)];   // for later kernels, and this one's end
        if (lane == 0) mbar_arrive(&d_full[slot]);
      }
      if (prev >= 0) {
        const int tile = prev / a.Hkv, g = prev - tile * a.Hkv;
        const int r = (warp & 3) * 32 + lane, rq = r / a.G, t = tile * qt + rq, h = g * a.G + (r - rq * a.G);
        const bool live = rq < qt && t < a.T;
        if (!__all_sync(0xffffffffu, mbar_wait(dq_full, (ni - 1) & 1, abort_flag, a.err))) break;
        tc_fence_after();
        float odd = 0.f;
#pragma unroll 1
        for (int d = 0; d < DQK; d += 32) {
          float o[32];
          tmem_ld32(tbase + C::DQ0 + lanes + d, o);
          tmem_ld_wait_regs(o);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            odd = fmaf(o[i], 0.f, fmaf(o[i + 1], 0.f, odd));
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[i] * a.scale, o[i + 1] * a.scale);
            w[i >> 1] = *reinterpret_cast<const uint32_t*>(&b);
          }
          store_rows32(w, a.dq + ((int64_t)tile * qt * a.Hq + g * a.G) * DQK + d, live ? rq * a.Hq + r - rq * a.G : -1, DQK, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dq_empty);
        // rows to do again (NaN compares unequal): a NaN in the first column marks them (the lane
        // that stored the column did so before the __syncwarp)
        const bool bad = live && odd != 0.f;
        if (bad) a.dq[((int64_t)t * a.Hq + h) * DQK] = __ushort_as_bfloat16(0x7fff);
        if (__any_sync(0xffffffffu, bad) && lane == 0) {
          if (redo[2 * (warp & 3) + 1] < 0) redo[2 * (warp & 3)] = prev;
          redo[2 * (warp & 3) + 1] = prev;
        }
      }
      if (item >= items) break;
      prev = item;
    }
  } else {
    // ---------------- score warps: row = TMEM lane, half of the block's keys each ----------------
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int rq = r / a.G;
    const uint32_t lanes = tmem_lane_base(warp);
    uint32_t nsp = 0, ni = 0;
    bool alive = true;
    for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
      const uint32_t slot = ni & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&d_full[slot], (ni / 2) & 1, abort_flag, a.err))) break;
      const float4 mine = *reinterpret_cast<const float4*>(smem + C::row_off + (slot * 128 + r) * 16);
      const volatile int* hd = head + 8 * slot;
      DqItem m;
      m.klo = hd[0];
      m.ns = hd[1];
      m.nbt = hd[2];
      m.sb = (m.ns + BLK - 1) / BLK;
      const int lo_last = hd[3];
      m.ds0 = hd[4];
      m.last = hd[5];
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[slot]);
      m.t0 = item / a.Hkv * qt;
      const float D = mine.x, l2 = mine.y;
      const int lo = __float_as_int(mine.z), ds = __float_as_int(mine.w), t = m.t0 + rq;
      const int early = min(ds + a.sinks, lo);
      const bool live = rq < qt && t < a.T;
      for (int j = 0; j < m.nbt; ++j, ++nsp) {
        const int cols = dq_cols<BLK>(m, j), pieces = cols >> 5, c0 = half * (cols >> 1);   // 16-key pieces, first key
        const int kb = dq_key<BLK>(m, j) + c0;
        const bool sink_blk = j < m.sb;
        const bool border = sink_blk || kb < lo_last || kb + (cols >> 1) - 1 > m.t0;
        uint64_t seen = ~0ull;
        if (border) {
          seen = bit_range(lo - kb, t + 1 - kb) | bit_range(ds - kb, early - kb);
          if (sink_blk) seen = ds == m.ds0 ? bit_range(0, m.ns - BLK * j - c0) : 0ull;
          if (!live) seen = 0ull;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(sp_full, nsp & 1, abort_flag, a.err))) { alive = false; break; }
        tc_fence_after();
        // 16 keys at a time: a spilled register costs a trip to L2 (the tiles leave L1 nothing)
        float w[3][8];
        const uint64_t sc2 = pack2(a.scale_log2, a.scale_log2), l22 = pack2(-l2, -l2), d2 = pack2(-D, -D);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c < pieces) {
            float s[16], p[16];
            tmem_ld16(tbase + C::S0 + lanes + c0 + 16 * c, s);
            tmem_ld16(tbase + C::P0 + lanes + c0 + 16 * c, p);
            tmem_ld_wait_regs(s);
            tmem_ld_wait_regs(p);
            if (c + 1 == pieces) {   // the next block's products can start
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(sp_empty);
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 e = unpack2(ffma2(pack2(s[i], s[i + 1]), sc2, l22));
              const float2 y = unpack2(fadd2(pack2(p[i], p[i + 1]), d2));
              s[i] = ex2_approx(e.x) * y.x;
              s[i + 1] = ex2_approx(e.y) * y.y;
            }
            if (border) {
              const uint32_t bits = (uint32_t)(seen >> (16 * c));
#pragma unroll
              for (int i = 0; i < 16; ++i) s[i] = (bits >> i) & 1u ? s[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(s[i], s[i + 1]);
              w[c][i >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&b));
            }
          }
        }
        // dS of the block before must have been read by its product before it is replaced
        if (nsp > 0 && !__all_sync(0xffffffffu, mbar_wait(ds_empty, (nsp - 1) & 1, abort_flag, a.err))) { alive = false; break; }
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < pieces) tmem_st8(tbase + C::DS0 + lanes + ((c0 + 16 * c) >> 1), w[c]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  redo_clear(a);   // for the kernel behind this one
  // ---- marked rows, by all warps in turn: nothing waits for them any more ----
  if (*abort_flag) return;
  const int first = __reduce_min_sync(0xffffffffu, lane < 4 ? redo[2 * lane] : INT_MAX);
  const int last = __reduce_max_sync(0xffffffffu, lane < 4 ? redo[2 * lane + 1] : -1);
  int turn = 0;
  for (int item = first; item <= last; item += gridDim.x) {
    const int tile = item / a.Hkv, g = item - tile * a.Hkv, t0 = tile * qt;
    if (warp < 4) {   // which of 32 rows are marked; the plans' words are free by now
      const int r = warp * 32 + lane, rq = r / a.G, t = t0 + rq;
      const bool bad = rq < qt && t < a.T && __hisnan(a.dq[((int64_t)t * a.Hq + g * a.G + r - rq * a.G) * DQK]);
      const unsigned marks = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) plan[warp] = (int)marks;
    }
    __syncthreads();
    for (int i = 0; i < 4; ++i) {
      for (unsigned m = (unsigned)plan[i]; m; m &= m - 1) {
        const int r = i * 32 + __ffs((int)m) - 1, rq = r / a.G;
        if (turn == warp) dq_row<DQK / 64, DV / 64>(a, t0 + rq, g * a.G + r - rq * a.G, lane);
        if (++turn == kDqThreads / 32) turn = 0;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
// dk, dv
// ---------------------------------------------------------------------------------------
template <int DQK, int DV>
struct DkvCfg {
  static constexpr int QA = DQK / 64, VA = DV / 64;
  static constexpr uint32_t k_bytes = QA * kAtom, v_bytes = VA * kAtom;
  static constexpr uint32_t q_bytes = QA * kAtom64, do_bytes = VA * kAtom64, st_bytes = q_bytes + do_bytes;
  static constexpr uint32_t st_off = k_bytes + v_bytes;
  static constexpr int ST = st_off + 4 * st_bytes <= 220u * 1024u ? 4 : 3;
  static constexpr uint32_t ld_off = st_off + ST * st_bytes;              // lse (base 2) and D of each stage's rows
  static constexpr uint32_t bar_off = ld_off + ST * 2 * kCols * 4;
  static constexpr uint32_t total = bar_off + 32 * 8 + 16 + 1024;
  static constexpr uint32_t S0 = 0, P0 = 64, PW0 = 128, DS0 = 160, DV0 = 192, DK0 = 192 + DV;
};

struct DkvItem {
  int s0, keys;     // first key, number of keys
  int t0, t1;       // queries
  int g, chunk;     // KV head; stretch of far queries of first tokens, or -1
  int nblk;
  int off;          // the block of queries to start with
};

// The blocks of an item in turn: `tb` its first query, `hb` its first head of the group. From
// query block `off` on, around the end: key tiles in flight stand at the same place of a period
// as long as their range, so that the tiles that see a query load it at about the same time.
struct DkvWalk {
  int tb, hb;
  __device__ __forceinline__ DkvWalk(const DkvItem& m, int qt) : tb(m.t0 + m.off * qt), hb(0) {}
  __device__ __forceinline__ void next(const DkvItem& m, int qt, int hc, int G) {
    hb += hc;
    if (hb < G) return;
    hb = 0;
    tb += qt;
    if (tb >= m.t1) tb = m.t0;
  }
};

// Queries of one stretch beyond the window. At least eight a first token, so that the stretches' FP32
// rows stay a small part of the batch's (3 / 8 of one a key at most).
__host__ __device__ inline int sink_stretch(int window, int sinks) {
  const int n = window > 8 * sinks ? window : 8 * sinks;
  return n < 256 ? 256 : n > 4096 ? 4096 : n;
}
// Whether a document of `len` tokens has stretches of its own. With no more than one stretch's
// queries beyond the window, its first tokens' window tile takes those as well: as many blocks,
// and no partial sums.
__device__ __forceinline__ bool sink_far(const WinArgs& a, int len) {
  return a.sinks > 0 && len - a.window > sink_stretch(a.window, a.sinks);
}

__device__ __forceinline__ DkvItem dkv_item(const WinArgs& a, const WinSinks& sk, int item, int tiles, int qt, int nhc) {
  DkvItem m;
  const int u = item / a.Hkv;
  m.g = item - u * a.Hkv;
  if (u < tiles) {
    m.chunk = -1;
    m.s0 = u * kBlk;
    m.keys = min(kBlk, a.T - m.s0);
    m.t0 = m.s0;
    const int sl = m.s0 + m.keys - 1;
    const WinDoc d = window_doc(a.cu, a.ndocs, a.T, sl);
    m.t1 = max(m.s0 - d.start, 0) < a.sinks && !sink_far(a, d.end - d.start) ? d.end : (int)min((int64_t)sl + a.window, (int64_t)d.end);
  } else {
    m.chunk = u - tiles;
    int lo = 0, hi = a.ndocs;   // chunk0[lo] <= chunk < chunk0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sk.chunk0[mid] <= m.chunk) lo = mid; else hi = mid;
    }
    const int start = min(max(a.cu[lo], 0), a.T - 1), end = max(min(a.cu[lo + 1], a.T), start + 1);
    m.s0 = start;
    m.keys = min(a.sinks, end - start);
    const int n = sink_stretch(a.window, a.sinks);
    m.t0 = (int)min((int64_t)end, (int64_t)start + a.window + (int64_t)(m.chunk - sk.chunk0[lo]) * n);
    m.t1 = min(end, m.t0 + n);
  }
  m.t1 = max(m.t1, m.t0 + 1);   // only where cu_seqlens is malformed
  const int nq = (m.t1 - m.t0 + qt - 1) / qt;
  m.nblk = nq * nhc;
  const int period = (int)min((int64_t)a.window + kBlk - 1, (int64_t)a.T) / qt + 1;
  const int at = m.t0 / qt % period;
  m.off = m.chunk < 0 && at > 0 && period - at < nq ? period - at : 0;
  return m;
}

template <int DQK, int DV>
__global__ void __launch_bounds__(kDkvThreads, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, WinArgs a,
                      WinSinks sk, int tiles) {
  using C = DkvCfg<DQK, DV>;
  constexpr int ST = C::ST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* ld = reinterpret_cast<float*>(smem + C::ld_off);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::bar_off);
  uint64_t* kv_empty = kv_full + 1;
  uint64_t* st_full = kv_empty + 1;    // [4]
  uint64_t* st_empty = st_full + 4;    // [4]
  uint64_t* sp_full = st_empty + 4;
  uint64_t* sp_empty = sp_full + 1;
  uint64_t* pd_full = sp_empty + 1;    // weights and dS of a block
  uint64_t* pd_empty = pd_full + 1;    // ... have been read by the products
  uint64_t* acc_full = pd_empty + 1;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;     // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hc = a.G < kCols ? a.G : kCols;      // heads a block
  const int qt = kCols / hc;                     // queries a block
  const int nhc = (a.G + kCols - 1) / kCols;     // blocks that share their queries
  // stage rows that no copy writes (64 not a multiple of the heads) meet weights of 0
  if (qt * hc < kCols) {
    for (uint32_t i = tid; i < ST * C::st_bytes / 16u; i += kDkvThreads)
      reinterpret_cast<uint4*>(smem + C::st_off)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (tid == 0) {
    mbar_init(kv_full, 1); mbar_init(kv_empty, 1);
    for (int i = 0; i < 4; ++i) { mbar_init(&st_full[i], 33); mbar_init(&st_empty[i], 1); }
    mbar_init(sp_full, 1); mbar_init(sp_empty, 16);
    mbar_init(pd_full, 16); mbar_init(pd_empty, 1);
    mbar_init(acc_full, 1); mbar_init(acc_empty, 16);
    mbar_init(&drain[0], 1); mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int units = tiles + (a.sinks > 0 && sk.slots > 0 ? min(sk.chunk0[a.ndocs], sk.chunks) : 0);
  const int items = units * a.Hkv;

  if (warp == 16) {
    // ---------------- lse and D of each stage's rows ----------------
    // (a warp of its own: the copies below need not wait for what these loads take)
    uint32_t ns = 0, st = 0, ph = 0;
    // the lane's two rows of a block: query, head, and row of lse relative to the block's first (-1: none)
    int cq[2], ch[2], crow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = lane + 32 * i;
      cq[i] = c / hc;
      ch[i] = c - cq[i] * hc;
      crow[i] = c < qt * hc ? cq[i] * a.Hq + ch[i] : -1;
    }
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DkvItem m = dkv_item(a, sk, item, tiles, qt, nhc);
      DkvWalk at(m, qt);
      for (int b = 0; b < m.nblk; ++b, ++ns, at.next(m, qt, hc, a.G)) {
        const int64_t base = (int64_t)at.tb * a.Hq + m.g * a.G + at.hb;
        float v[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool in = crow[i] >= 0 && at.tb + cq[i] < a.T && at.hb + ch[i] < a.G;
          v[2 * i] = in ? a.lse_in[base + crow[i]] : 0.f;   // scaled where it is stored: nothing waits for it here
          v[2 * i + 1] = in ? a.delta[base + crow[i]] : 0.f;
        }
        if (ns >= ST && !__all_sync(0xffffffffu, mbar_wait(&st_empty[st], ph ^ 1u, abort_flag, a.err))) { ok = false; break; }
        float* l = ld + st * 2 * kCols;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[lane + 32 * i] = v[2 * i] * kLog2e;
          l[kCols + lane + 32 * i] = v[2 * i + 1];
        }
        mbar_arrive(&st_full[st]);
        if (++st == ST) { st = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 19) {
    // ---------------- copies, by lane 0 ----------------
    if (lane == 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_do);
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      const uint32_t box = (uint32_t)(qt * hc) * 128u * (C::QA + C::VA);
      uint32_t ni = 0, ns = 0, st = 0, ph = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x, ++ni) {
        const DkvItem m = dkv_item(a, sk, item, tiles, qt, nhc);
        if (ni > 0 && !mbar_wait(kv_empty, (ni - 1) & 1, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(kv_full, C::k_bytes + C::v_bytes);
        for (int c = 0; c < C::QA; ++c) tma_load_3d(smem + c * kAtom, &tm_k, c * 64, m.g, m.s0, kv_full);
        for (int c = 0; c < C::VA; ++c) tma_load_3d(smem + C::k_bytes + c * kAtom, &tm_v, c * 64, m.g, m.s0, kv_full);
        DkvWalk at(m, qt);
        for (int b = 0; b < m.nblk; ++b, ++ns, at.next(m, qt, hc, a.G)) {
          if (ns >= ST && !mbar_wait(&st_empty[st], ph ^ 1u, abort_flag, a.err)) { ok = false; break; }
          mbar_arrive_expect_tx(&st_full[st], box);
          uint8_t* dst = smem + C::st_off + st * C::st_bytes;
          for (int c = 0; c < C::QA; ++c) tma_load_3d(dst + c * kAtom64, &tm_q, c * 64, m.g * a.G + at.hb, at.tb, &st_full[st]);
          for (int c = 0; c < C::VA; ++c)
            tma_load_3d(dst + C::q_bytes + c * kAtom64, &tm_do, c * 64, m.g * a.G + at.hb, at.tb, &st_full[st]);
          if (++st == ST) { st = 0; ph ^= 1u; }
        }
      }
      if (*abort_flag) {
        if (ni > 0) wait_landed(kv_full, (ni - 1) & 1);
        for (uint32_t i = ns > ST ? ns - ST : 0; i < ns; ++i) wait_landed(&st_full[i % ST], (i / ST) & 1);
      }
    }
  } else if (warp > 16) {
    // ---------------- MMA issuers (a whole warp each; one elected lane issues) ----------------
    // One warp issues the scores and dP, another dv and dk: each one's waits (115 cycles even
    // where nothing is waited for) lie under the other's products.
    const uint32_t sb = smem_u32(smem), tb = (uint32_t)uniform((int)tbase);
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)); };
    uint32_t n = 0, ni = 0, st = 0, ph = 0;   // blocks, items; ring
    bool alive = true;
    if (warp == 17) {
      constexpr uint32_t S_IDESC = idesc_bf16(128, kCols, false, false);
      for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
        const int nblk = uniform(dkv_item(a, sk, item, tiles, qt, nhc).nblk);
        if (!wait(kv_full, ni & 1)) break;
        for (int b = 0; b < nblk; ++b, ++n) {
          if (!wait(&st_full[st], ph) || (n > 0 && !wait(sp_empty, (n - 1) & 1))) { alive = false; break; }
          tc_fence_after();
          const uint32_t q = sb + C::st_off + st * C::st_bytes;
          ss_run<C::QA>(tb + C::S0, sb, kAtom, q, kAtom64, S_IDESC);
          ss_run<C::VA>(tb + C::P0, sb + C::k_bytes, kAtom, q + C::q_bytes, kAtom64, S_IDESC);
          umma_commit_warp(sp_full);
          if (++st == ST) { st = 0; ph ^= 1u; }
        }
        umma_commit_warp(kv_empty);
      }
    } else {
      constexpr uint32_t DV_IDESC = idesc_bf16(128, DV, false, true), DK_IDESC = idesc_bf16(128, DQK, false, true);
      for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
        const int nblk = uniform(dkv_item(a, sk, item, tiles, qt, nhc).nblk);
        for (int b = 0; b < nblk; ++b, ++n) {
          if (!wait(pd_full, n & 1) || (b == 0 && ni > 0 && !wait(acc_empty, (ni - 1) & 1))) { alive = false; break; }
          tc_fence_after();
          const uint32_t q = sb + C::st_off + st * C::st_bytes;
          ts_run<4>(tb + C::DV0, tb + C::PW0, q + C::q_bytes, kAtom64, DV_IDESC, b > 0);
          ts_run<4>(tb + C::DK0, tb + C::DS0, q, kAtom64, DK_IDESC, b > 0);
          umma_commit_warp(pd_empty);
          umma_commit_warp(&st_empty[st]);
          if (++st == ST) st = 0;
        }
        if (!alive) break;
        umma_commit_warp(acc_full);
      }
    }
    umma_commit_warp(&drain[warp - 17]);
    wait_landed(&drain[warp - 17], 0);
    __syncwarp();
  } else {
    // ---------------- score warps: key = TMEM lane, 16 of a block's 64 rows each ----------------
    const int quart = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem_lane_base(warp);
    uint32_t nb = 0, ni = 0;
    bool alive = true;
    for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
      const DkvItem m = dkv_item(a, sk, item, tiles, qt, nhc);
      const int s = m.s0 + r;
      const bool live = r < m.keys;
      int di = 0;
      const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, min(s, a.T - 1), &di);
      // this key's queries of the item: [from, to)
      const int past = s - doc.start < a.sinks && !sink_far(a, doc.end - doc.start)
                           ? doc.end : (int)min((int64_t)s + a.window, (int64_t)(m.chunk < 0 ? doc.end : m.t1));
      const int from = m.chunk < 0 ? s : past;
      const int to = m.chunk < 0 ? past : m.t1;
      // a block is whole when every key of the tile sees every row
      int all0, all1;
      if (m.chunk < 0) {
        const WinDoc d0 = window_doc(a.cu, a.ndocs, a.T, m.s0);
        all0 = m.s0 + m.keys - 1;
        all1 = (int)min((int64_t)m.s0 + a.window, (int64_t)d0.end) - qt;
      } else {
        all0 = (int)min((int64_t)m.s0 + m.keys - 1 + a.window, (int64_t)m.t1);
        all1 = m.t1 - qt;
      }
      DkvWalk at(m, qt);
      for (int b = 0; b < m.nblk; ++b, ++nb, at.next(m, qt, hc, a.G)) {
        const uint32_t st = nb % ST;
        const int tb = at.tb, valid = a.G - at.hb < hc ? a.G - at.hb : qt * hc;
        uint32_t in = 0xffffu;   // which of this warp's rows the key sees
        if (!(tb >= all0 && tb <= all1 && valid == kCols))
          in = bit_range32(max(from - tb, 0) * hc - 16 * quart, min(min(valid, max(min(to - tb, qt), 0) * hc) - 16 * quart, 16));
        if (!__all_sync(0xffffffffu, mbar_wait(&st_full[st], (nb / ST) & 1, abort_flag, a.err) &&
                                         mbar_wait(sp_full, nb & 1, abort_flag, a.err))) {
          alive = false;
          break;
        }
        tc_fence_after();
        float sc[16], dp[16];
        tmem_ld16(tbase + C::S0 + lanes + 16 * quart, sc);
        tmem_ld16(tbase + C::P0 + lanes + 16 * quart, dp);
        tmem_ld_wait_regs(sc);
        tmem_ld_wait_regs(dp);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sp_empty);
        const float4* l4 = reinterpret_cast<const float4*>(ld + st * 2 * kCols + 16 * quart);
        const float4* d4 = reinterpret_cast<const float4*>(ld + st * 2 * kCols + kCols + 16 * quart);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 l = l4[i], d = d4[i];
          const float lv[4] = {l.x, l.y, l.z, l.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = 4 * i + k;
            sc[c] = ex2_approx(fmaf(sc[c], a.scale_log2, -lv[k]));
            dp[c] = sc[c] * (dp[c] - dv[k]);
          }
        }
        if (in != 0xffffu) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            sc[c] = (in >> c) & 1u ? sc[c] : 0.f;
            dp[c] = (in >> c) & 1u ? dp[c] : 0.f;
          }
        }
        float w[8], x[8];
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(sc[c], sc[c + 1]), q = __floats2bfloat162_rn(dp[c], dp[c + 1]);
          w[c >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&p));
          x[c >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&q));
        }
        if (nb > 0 && !__all_sync(0xffffffffu, mbar_wait(pd_empty, (nb - 1) & 1, abort_flag, a.err))) { alive = false; break; }
        tmem_st8(tbase + C::PW0 + lanes + 8 * quart, w);
        tmem_st8(tbase + C::DS0 + lanes + 8 * quart, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pd_full);
      }
      if (!alive) break;
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full, ni & 1, abort_flag, a.err))) break;
      tc_fence_after();
      // ---- this key's sums [dk | dv], pieces of 32 columns in turn ----
      const bool far = m.chunk >= 0 || (s - doc.start < a.sinks && sink_far(a, doc.end - doc.start) && sk.slots > 0);
      float* part = nullptr;   // FP32 rows of first tokens
      if (m.chunk >= 0) part = sk.part + (((int64_t)m.chunk * a.Hkv + m.g) * a.sinks + r) * (DQK + DV);
      else if (live && far) part = sk.base + (((int64_t)sk.slot[di] * a.Hkv + m.g) * a.sinks + (s - doc.start)) * (DQK + DV);
      const int64_t row = (int64_t)s * a.Hkv + m.g;
      float odd_k = 0.f, odd_v = 0.f;
#pragma unroll 1
      for (int d = 32 * quart; d < DQK + DV; d += 128) {
        const bool is_k = d < DQK;
        float o[32];
        tmem_ld32(tbase + (is_k ? C::DK0 + d : C::DV0 + (d - DQK)) + lanes, o);
        tmem_ld_wait_regs(o);
        const float f = is_k ? a.scale : 1.f;
        if (live && far) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(part + d + i) = make_float4(o[i] * f, o[i + 1] * f, o[i + 2] * f, o[i + 3] * f);
        } else {
          uint32_t w[16];
          float odd = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            odd = fmaf(o[i], 0.f, fmaf(o[i + 1], 0.f, odd));
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[i] * f, o[i + 1] * f);
            w[i >> 1] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (is_k) odd_k += odd; else odd_v += odd;
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(is_k ? a.dk + row * DQK + d : a.dv + row * DV + (d - DQK));
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      // keys whose sums are not finite (NaN compares unequal) are done again
      if (live && !far && (odd_k != 0.f || odd_v != 0.f)) redo_mark(a, row);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------------------------------
// First tokens: which documents have far queries, and the joining of their sums
// ---------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// slot[d]: the document's place among those with stretches; chunk0[d]: its first
// stretch; doc[slot]. One block.
__global__ void __launch_bounds__(kPlanThreads) window_plan_kernel(WinArgs a, WinSinks sk) {
  __shared__ int s_slot[kPlanThreads], s_chunk[kPlanThreads];
  const int tid = threadIdx.x;
  const int per = (a.ndocs + kPlanThreads - 1) / kPlanThreads;
  const int b = min(a.ndocs, tid * per), e = min(a.ndocs, b + per);
  const int n = sink_stretch(a.window, a.sinks);
  auto chunks_of = [&](int d) {
    const int start = min(max(a.cu[d], 0), a.T - 1), end = max(min(a.cu[d + 1], a.T), start + 1);
    return sink_far(a, end - start) ? (end - start - a.window + n - 1) / n : 0;
  };
  int slots = 0, chunks = 0;
  for (int d = b; d < e; ++d) {
    const int c = chunks_of(d);
    slots += c > 0;
    chunks += c;
  }
  s_slot[tid] = slots;
  s_chunk[tid] = chunks;
  __syncthreads();
  for (int o = 1; o < kPlanThreads; o <<= 1) {
    const int x = tid >= o ? s_slot[tid - o] : 0, y = tid >= o ? s_chunk[tid - o] : 0;
    __syncthreads();
    s_slot[tid] += x;
    s_chunk[tid] += y;
    __syncthreads();
  }
  int slot = s_slot[tid] - slots, chunk = s_chunk[tid] - chunks;
  for (int d = b; d < e; ++d) {
    const int c = chunks_of(d);
    // the clamps only matter where cu_seqlens is malformed
    sk.slot[d] = min(slot, sk.slots - 1);
    sk.chunk0[d] = min(chunk, sk.chunks);
    if (c > 0 && slot < sk.slots) sk.doc[slot] = d;
    slot += c > 0;
    chunk += c;
  }
  if (tid == kPlanThreads - 1) {
    sk.chunk0[a.ndocs] = min(s_chunk[tid], sk.chunks);
    sk.doc[sk.slots] = min(s_slot[tid], sk.slots);   // how many slots are used
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(128) window_join_kernel(WinArgs a, WinSinks sk) {
  const int slot = blockIdx.x / (a.Hkv * a.sinks), gi = blockIdx.x % (a.Hkv * a.sinks), g = gi / a.sinks, i = gi % a.sinks;
  if (slot >= sk.doc[sk.slots]) return;
  const int d = sk.doc[slot];
  const int start = min(max(a.cu[d], 0), a.T - 1), end = max(min(a.cu[d + 1], a.T), start + 1);
  if (i >= end - start) return;
  constexpr int D = DQK + DV;
  const int c0 = sk.chunk0[d], c1 = sk.chunk0[d + 1];
  const int64_t row = (int64_t)(start + i) * a.Hkv + g;
  const float* base = sk.base + (((int64_t)slot * a.Hkv + g) * a.sinks + i) * D;
  const float* part = sk.part + ((int64_t)g * a.sinks + i) * D;
  const int64_t step = (int64_t)a.Hkv * a.sinks * D;
  float odd = 0.f;
  for (int x = threadIdx.x; x < D; x += 128) {
    float s = base[x];
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += part[c * step + x];
    odd = fmaf(s, 0.f, odd);
    if (x < DQK) a.dk[row * DQK + x] = __float2bfloat16_rn(s);
    else a.dv[row * DV + x - DQK] = __float2bfloat16_rn(s);
  }
  if (odd != 0.f) redo_mark(a, row);
}

// dk and dv of the marked keys. Block b looks at every gridDim-th key; its warps share a marked
// key's queries and join their sums in order. With no key marked it costs its launch.
constexpr int kRedoThreads = 512;
template <int DQK, int DV>
__global__ void __launch_bounds__(kRedoThreads, 2) window_redo_kernel(WinArgs a) {
  constexpr int W = kRedoThreads / 32, D = DQK + DV;
  __shared__ float sums[W][D];
  __shared__ unsigned marks[W];
  __shared__ volatile int nan;
  if (a.redo[0] == 0u) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rows = (int64_t)a.T * a.Hkv;
  for (int64_t c0 = blockIdx.x; c0 < rows; c0 += (int64_t)kRedoThreads * gridDim.x) {
    const int64_t mine = c0 + (int64_t)tid * gridDim.x;
    const unsigned m = __ballot_sync(0xffffffffu, mine < rows && (a.redo[1 + (mine >> 5)] >> (mine & 31) & 1u));
    if (lane == 0) marks[warp] = m;
    __syncthreads();
    for (int w = 0; w < W; ++w) {
      for (unsigned left = marks[w]; left; left &= left - 1) {
        const int64_t row = c0 + (int64_t)(w * 32 + __ffs((int)left) - 1) * gridDim.x;
        const int s = (int)(row / a.Hkv), g = (int)(row % a.Hkv), end = key_end(a, s);
        // a NaN in lse makes every column NaN: looked for first, a lane a row
        bool bad = false;
        for (int64_t i = tid; i < (int64_t)(end - s) * a.G && !bad; i += kRedoThreads) {
          const float l = a.lse_in[(s + i / a.G) * a.Hq + g * a.G + i % a.G];
          bad = l != l;
        }
        if (tid == 0) nan = 0;
        bad = __syncthreads_or(bad);
        if (bad) {
          for (int d = tid; d < D; d += kRedoThreads) sums[0][d] = __int_as_float(0x7fffffff);
        } else {
          float2 dk[DQK / 64], dv[DV / 64];
          dkv_sums<DQK / 64, DV / 64>(a, s, g, lane, warp, W, &nan, dk, dv);
#pragma unroll
          for (int i = 0; i < DQK / 64; ++i) *reinterpret_cast<float2*>(&sums[warp][64 * i + 2 * lane]) = dk[i];
#pragma unroll
          for (int i = 0; i < DV / 64; ++i) *reinterpret_cast<float2*>(&sums[warp][DQK + 64 * i + 2 * lane]) = dv[i];
        }
        __syncthreads();
        for (int d = tid; d < D; d += kRedoThreads) {
          float x = sums[0][d];
          for (int i = 1; i < W && !bad; ++i) x += sums[i][d];
          if (d < DQK) a.dk[row * DQK + d] = __float2bfloat16_rn(x * a.scale);
          else a.dv[row * DV + d - DQK] = __float2bfloat16_rn(x);
        }
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

}  // namespace

// Keys a block of the dq kernel: the box of its k and v maps.
int window_dq_block() { return DqCfg<128, 128>::BLK; }

namespace {

template <int DQK, int DV>
cudaError_t launch_bwd(const WinBwdMaps& m, const WinArgs& a, const WinSinks& sk, int num_sms, bool* configured,
                       cudaStream_t stream) {
  using Q = DqCfg<DQK, DV>;
  using K = DkvCfg<DQK, DV>;
  cudaError_t e;
  if (!*configured) {
    if ((e = cudaFuncSetAttribute(window_dq_kernel<DQK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Q::total)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(window_dkv_kernel<DQK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::total)) != cudaSuccess)
      return e;
    *configured = true;
  }
  const int qt = 128 / a.G, tiles = (a.T + qt - 1) / qt, ktiles = (a.T + kBlk - 1) / kBlk;
  const int64_t items = (int64_t)tiles * a.Hkv;
  window_dq_kernel<DQK, DV><<<items < num_sms ? (int)items : num_sms, kDqThreads, Q::total, stream>>>(m.q, m.dout, m.kq, m.vq, a, qt, tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (sk.slots > 0) {
    window_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, sk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int64_t kitems = ((int64_t)ktiles + sk.chunks) * a.Hkv;
  window_dkv_kernel<DQK, DV><<<kitems < num_sms ? (int)kitems : num_sms, kDkvThreads, K::total, stream>>>(m.q2, m.dout2, m.k, m.v, a, sk, ktiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (sk.slots > 0) {
    window_join_kernel<DQK, DV><<<(unsigned)(sk.slots * a.Hkv * a.sinks), 128, 0, stream>>>(a, sk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  window_redo_kernel<DQK, DV><<<2 * num_sms, kRedoThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Workspace: D of every row and the marks of keys; then, with first tokens, the plan and the FP32 sums.
size_t window_bwd_workspace_bytes(int T, int Hq, int Hkv, int Dqk, int Dv, int ndocs, int window, int sinks) {
  WinArgs a;
  WinSinks s;
  return window_bwd_layout(nullptr, T, Hq, Hkv, Dqk, Dv, ndocs, window, sinks, &a, &s);
}

size_t window_bwd_layout(uint8_t* ws, int T, int Hq, int Hkv, int Dqk, int Dv, int ndocs, int window, int sinks, WinArgs* a,
                         WinSinks* s) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws + off;
    off += (bytes + 255) & ~size_t(255);
    return p;
  };
  a->delta = reinterpret_cast<float*>(take((size_t)T * Hq * 4));
  a->redo = reinterpret_cast<uint32_t*>(take((size_t)redo_words(T, Hkv) * 4));
  *s = WinSinks{};
  const int64_t longer = (int64_t)T / ((int64_t)window + sink_stretch(window, sinks) + 1);   // documents that can have stretches
  s->slots = sinks > 0 ? (int)(longer < ndocs ? longer : ndocs) : 0;
  if (s->slots > 0) {
    s->chunks = T / sink_stretch(window, sinks) + s->slots;
    s->slot = reinterpret_cast<int*>(take((size_t)ndocs * 4));
    s->chunk0 = reinterpret_cast<int*>(take((size_t)(ndocs + 1) * 4));
    s->doc = reinterpret_cast<int*>(take((size_t)(s->slots + 1) * 4));
    const size_t rows = (size_t)Hkv * sinks * (Dqk + Dv) * 4;
    s->base = reinterpret_cast<float*>(take((size_t)s->slots * rows));
    s->part = reinterpret_cast<float*>(take((size_t)s->chunks * rows));
  }
  return off + 256;
}

cudaError_t launch_window_bwd_tc(const WinBwdMaps& m, const WinArgs& a, const WinSinks& sk, int num_sms, bool* configured,
                                 cudaStream_t stream) {
  const int i = (a.Dqk / 64 - 1) * 2 + (a.Dv / 64 - 1);
  switch (i) {
    case 0: return launch_bwd<64, 64>(m, a, sk, num_sms, configured + i, stream);
    case 1: return launch_bwd<64, 128>(m, a, sk, num_sms, configured + i, stream);
    case 2: return launch_bwd<128, 64>(m, a, sk, num_sms, configured + i, stream);
    case 3: return launch_bwd<128, 128>(m, a, sk, num_sms, configured + i, stream);
    case 4: return launch_bwd<192, 64>(m, a, sk, num_sms, configured + i, stream);
    default: return launch_bwd<192, 128>(m, a, sk, num_sms, configured + i, stream);
  }
}

}  // namespace irs

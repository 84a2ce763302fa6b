// Window attention on the tensor cores (tcgen05 + TMEM + TMA): the forward.
//
// Mathematics as in irs_window.cu: query t of document [s_d, e_d) sees lo <= s <= t, lo =
// max(s_d, t - window + 1), and the first tokens s_d <= s < min(s_d + sinks, lo).
//
// What bounds it. 2 (Dqk + Dv) flops a (query, head, key) pair on operands that stay in L2:
// the tensor cores by count. As it runs no unit is full (tensor pipe 41% active, issue 47%, the
// exponential unit 17% at T 8192): the softmax's and the products' turns are.
//
// Design.
// * The 128 rows of a product are the G query heads of a KV head for 128 / G queries, so a
//   tile spans few queries and the keys it needs beyond one window are few: window 512 and
//   G = 16 give tiles of 8 queries over 519 keys.
// * An item is two such tiles of neighbouring queries over the same key blocks (64 keys, by
//   TMA), each with an issuing warp of its own that runs two blocks' scores ahead of the
//   weights' products: the softmax finds its scores ready. One issuing warp for both tiles
//   left the tensor cores idle for a third of its time (1.77 ms at T 65536, 64 / 4 heads of
//   192 / 128, window 512; two warps 1.72). A persistent CTA an SM walks the items; the next
//   item's queries and keys load while the last one drains.
// * One ring holds block t's keys with block t - 2's values, so a step of a tile has one wait
//   for both operands (two rings 1.72 ms, one 1.55).
// * Two threads share a row, 32 keys of a block each (16 softmax warps). With one thread a
//   row (8 warps) a warp's own latency was the bound: 4 to 5 cycles an instruction, 2.72 ms
//   against 2.45. They hold the same maximum; one barrier of the two warps a block carries
//   their vote whether to raise it.
// * S[128 x 64] = Q K^T lies in TMEM, two blocks a tile; the weights return over it as bf16
//   and are the first operand of O += P V straight from TMEM (V read MN-major from its
//   [key][dim] tile). No register may be spilled: shared memory leaves no L1, and a spilled
//   word is a trip to L2 (12 words in the loop: 1.53 -> 1.73 ms).
// * The running maximum is raised only where a half row's weights under it sum past 2^8 (sums
//   are FP32), so that after a tile's first block the scores are read once and O in TMEM is
//   hardly ever rescaled.
// * Documents are not aligned to tiles: a tile's keys are one range of the packed sequence,
//   and each row masks by its own document's start. Only blocks at a border of the range are
//   masked element by element. First tokens before the range are one more (narrow) block.
// * A masked weight is 0, but 0 times an infinity or NaN in a masked value row is NaN. Rows
//   whose sum or output is not finite are marked (a NaN in the output, the item in shared memory)
//   and computed again from their visible keys alone when the CTA is through with its items: a
//   row takes as long as its window, and the pipeline's waits have a limit.
// * Measured: 1.51 ms at the size above (890 TFLOP/s of the pairs that are seen). Of a softmax
//   warp's 29,300 cycles an item (ten blocks) 17,000 are its work on them, 5,600 its waits for
//   scores (115 cycles each where nothing is waited for) and 6,500 the item's output; the
//   products at the rates of their shapes (64 columns read at the limit of shared memory:
//   48.6 cycles for 16 dims, 32 if it were not) would take 17,000.
#include <climits>

#include "irs_internal.h"
#include "irs_ptx.cuh"
#include "irs_window_rows.cuh"

namespace irs {

namespace {

constexpr int kRows = 128;           // rows a tile
constexpr uint32_t kAtom = 128 * 128;   // 128 rows x 64 bf16
constexpr int kFwdThreads = 608;     // warps 0-7, 8-15: softmax of the two tiles; 16: TMA; 17, 18: MMA of the two tiles
constexpr float kRaise = 256.f;      // a half row's weights of a block with a sum past this raise the maximum

template <int DQK, int DV>
struct FwdCfg {
  static constexpr int QA = DQK / 64, VA = DV / 64;
  static constexpr uint32_t q_bytes = QA * kAtom;          // one tile's queries
  // 64 keys a block: two blocks' scores of both tiles (4 x 64 columns) lie in TMEM beside both
  // outputs, so a block's scores are there when the block before has its weights.
  static constexpr int BLK = 64;
  static constexpr uint32_t kv_atom = BLK * 128;           // BLK rows x 64 bf16
  static constexpr uint32_t k_bytes = QA * kv_atom, v_bytes = VA * kv_atom, st_bytes = k_bytes + v_bytes;
  static constexpr int ST = 3;                             // stages: block t's keys and block t - 2's values
  static constexpr uint32_t st_off = 2 * q_bytes, x_off = st_off + ST * st_bytes;
  // Two words a row, half and tile, by which the two threads of a row exchange maxima and sums. A
  // maximum's word is written again behind the barrier that ends its block's slow path; the sum's,
  // read last in an item, behind those of the next item's first block, which is always slow.
  static constexpr uint32_t x_bytes = 2 * 2 * kRows * 4;
  static constexpr uint32_t bar_off = x_off + 2 * x_bytes;
  static constexpr uint32_t plan_off = bar_off + 32 * 8 + 16;   // [4][8] an item's blocks and borders
  static constexpr uint32_t redo_off = plan_off + 4 * 32;       // [16][2] first and last item of a softmax warp with marked rows
  static constexpr uint32_t cu_off = redo_off + 16 * 8;
  static constexpr int cu_cap = (int)((232448u - cu_off) / 4u) < 2048 ? (int)((232448u - cu_off) / 4u) : 2048;
  static constexpr uint32_t total = cu_off + 4u * cu_cap;   // all of 227 KB at 192/128: none to spare for aligning
  static constexpr uint32_t S0 = 0, O0 = 256;              // TMEM: S of tile x, buffer b at 128 x + 64 b; O at 256 + x DV
};

// The keys of one item: two tiles of `qt` queries from t0 on. The first `sb` blocks hold the
// first tokens before the range, where there are any; the first tile takes blocks [0, l0],
// the second [f1, nbt).
struct Item {
  int t0, last, lastA;   // first query; last query of the item and of its first tile
  int ds0, de0, klo, ns; // document of the first query; first key of the range; first tokens before it
  int sb, nbt, l0, f1;
  bool hasB;
};
template <int kBlk>
__device__ __forceinline__ Item window_item(const WinArgs& a, const int32_t* cu, int t0, int qt) {
  Item m;
  m.t0 = t0;
  m.last = min(t0 + 2 * qt, a.T) - 1;
  m.lastA = min(t0 + qt, a.T) - 1;
  m.hasB = t0 + qt < a.T;
  const WinDoc d0 = window_doc(cu, a.ndocs, a.T, t0);
  m.ds0 = d0.start;
  m.de0 = d0.end;
  m.klo = max(m.ds0, t0 - a.window + 1);
  m.ns = max(0, min(m.ds0 + a.sinks, m.klo) - m.ds0);
  m.sb = (m.ns + kBlk - 1) / kBlk;
  m.nbt = (m.last - m.klo) / kBlk + 1 + m.sb;
  m.l0 = (m.lastA - m.klo) / kBlk + m.sb;
  m.f1 = 0;
  if (m.hasB) {
    const int tb = t0 + qt, dsB = tb < m.de0 ? m.ds0 : window_doc(cu, a.ndocs, a.T, tb).start;
    // blocks before the second tile's window are left out; with first tokens, only theirs
    if (a.sinks == 0) m.f1 = (max(dsB, tb - a.window + 1) - m.klo) / kBlk;
    else m.f1 = dsB != m.ds0 ? m.sb : 0;
  }
  return m;
}
template <int kBlk>
__device__ __forceinline__ int item_key(const Item& m, int j) {   // first key of block j
  return j < m.sb ? m.ds0 + kBlk * j : m.klo + kBlk * (j - m.sb);
}
template <int kBlk>
__device__ __forceinline__ int item_cols(const Item& m, int j) {  // its keys, up to a multiple of 32
  const int n = min(kBlk, j < m.sb ? m.ns - kBlk * j : m.last - item_key<kBlk>(m, j) + 1);
  return (n + 31) & ~31;
}

__device__ __forceinline__ void mask16(float (&v)[16], uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = (bits >> i) & 1u ? v[i] : -INFINITY;
}

// D[128 x DV] (+)= P . V: P bf16 in TMEM, V a [key][dim] tile read MN-major; NK steps of 16
// keys. Each half of the keys has its weights at the first of its own score columns.
template <int NK>
__device__ __forceinline__ void pv_run(uint32_t d, uint32_t p, uint32_t vb, uint32_t atom, uint32_t idesc, bool accumulate) {
  const uint64_t b0 = sdesc_sw128(vb, atom, 1024);
#pragma unroll
  for (int ks = 0; ks < NK; ++ks)
    umma_bf16_ts_warp(d, p + (ks < NK / 2 ? 8 * ks : 8 * NK + 8 * (ks - NK / 2)), b0 + (uint64_t)((ks * 2048) >> 4), idesc,
                 (accumulate || ks > 0) ? 1u : 0u);
}
__device__ __forceinline__ void pv_any(int cols, uint32_t d, uint32_t p, uint32_t vb, uint32_t atom, uint32_t idesc,
                                       bool accumulate) {
  switch (cols >> 5) {
    case 1: pv_run<2>(d, p, vb, atom, idesc, accumulate); break;
    default: pv_run<4>(d, p, vb, atom, idesc, accumulate); break;
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(kFwdThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, WinArgs a, int qt, int pairs) {
  using C = FwdCfg<DQK, DV>;
  constexpr int ST = C::ST;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {   // the attribute asks for it; the tiles need it
    record_error(a.err, IRS_DEVERR_TIMEOUT);
    return;
  }
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::bar_off);   // [2]
  uint64_t* q_empty = q_full + 2;     // [2]
  uint64_t* st_full = q_empty + 2;    // [ST]
  uint64_t* st_empty = st_full + ST;
  uint64_t* s_full = st_empty + ST;    // [2][2] scores of a tile's next block, by buffer
  uint64_t* p_full = s_full + 4;      // [2][2] the block's weights
  uint64_t* pv_done = p_full + 4;     // [2] ... have been multiplied
  uint64_t* o_full = pv_done + 2;     // [2] the tile's output
  uint64_t* o_empty = o_full + 2;     // [2]
  uint64_t* drain = o_empty + 2;      // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(smem + C::plan_off);
  int* redo = reinterpret_cast<int*>(smem + C::redo_off);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) { mbar_init(&st_full[i], 1); mbar_init(&st_empty[i], 2); }
    for (int i = 0; i < 4; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 8); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1); mbar_init(&o_empty[i], 8);
      mbar_init(&drain[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  if (tid < 16) {
    redo[2 * tid] = INT_MAX;
    redo[2 * tid + 1] = -1;
  }
  check_documents(a);
  // document borders are searched for every item by every row: in shared memory where they fit
  // (from L2 the searches took 9,000 of an item's 40,000 cycles)
  const int32_t* cu = a.cu;
  if (a.ndocs < C::cu_cap) {
    int32_t* near = reinterpret_cast<int32_t*>(smem + C::cu_off);
    for (int i = tid; i <= a.ndocs; i += kFwdThreads) near[i] = a.cu[i];
    cu = near;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int items = pairs * a.Hkv;

  if (warp == 16) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      const uint32_t q_box = (uint32_t)(qt * a.G) * 128u * C::QA;
      uint32_t nq[2] = {0, 0}, ns = 0, st = 0, ph = 0;
      bool ok = true;
      auto load_q = [&](int x, const Item& m, int g) {
        if (nq[x] > 0 && !mbar_wait(&q_empty[x], (nq[x] - 1) & 1, abort_flag, a.err)) return false;
        ++nq[x];
        if (x == 1 && !m.hasB) {   // the second tile's warp still learns of the item
          mbar_arrive(&q_full[1]);
          return true;
        }
        mbar_arrive_expect_tx(&q_full[x], q_box);
        for (int c = 0; c < C::QA; ++c)
          tma_load_3d(smem + x * C::q_bytes + c * kAtom, &tm_q, c * 64, g * a.G, m.t0 + x * qt, &q_full[x]);
        return true;
      };
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        const int pair = item / a.Hkv, g = item - pair * a.Hkv;
        const Item m = window_item<C::BLK>(a, cu, pair * 2 * qt, qt);
        // four slots: this one's reader, three items behind at most, is done with it
        volatile int* pl = plan + 8 * (nq[0] & 3);
        pl[0] = m.nbt;
        pl[1] = m.l0;
        pl[2] = m.hasB ? m.f1 : m.nbt;
        pl[3] = (m.sb > 0 ? item_cols<C::BLK>(m, m.sb - 1) : 0) | item_cols<C::BLK>(m, m.nbt - 1) << 8 | m.sb << 16;
        pl[4] = m.klo;
        pl[5] = m.ns;
        pl[6] = m.ds0;
        pl[7] = m.de0;
        if (!(ok = load_q(0, m, g))) break;
        for (int j = 0; j < m.nbt + 2; ++j) {   // block j's keys, block j - 2's values
          if (ns >= (uint32_t)ST && !mbar_wait(&st_empty[st], ph ^ 1u, abort_flag, a.err)) { ok = false; break; }
          mbar_arrive_expect_tx(&st_full[st], (j < m.nbt ? C::k_bytes : 0u) + (j >= 2 ? C::v_bytes : 0u));
          uint8_t* dst = smem + C::st_off + st * C::st_bytes;
          if (j < m.nbt)
            for (int c = 0; c < C::QA; ++c)
              tma_load_3d(dst + c * C::kv_atom, &tm_k, c * 64, g, item_key<C::BLK>(m, j), &st_full[st]);
          if (j >= 2)
            for (int c = 0; c < C::VA; ++c)
              tma_load_3d(dst + C::k_bytes + c * C::kv_atom, &tm_v, c * 64, g, item_key<C::BLK>(m, j - 2), &st_full[st]);
          ++ns;
          if (++st == (uint32_t)ST) { st = 0; ph ^= 1u; }
          if (j == 0 && !(ok = load_q(1, m, g))) break;
        }
      }
      if (*abort_flag) {
        // copies still in flight land before the CTA leaves
        auto landed = [&](uint64_t* bar, uint32_t parity) {
          const unsigned long long w0 = globaltimer_ns();
          while (!mbar_try_wait(bar, parity) && globaltimer_ns() - w0 < kWaitLimitNs) {}
        };
        for (int x = 0; x < 2; ++x) if (nq[x] > 0) landed(&q_full[x], (nq[x] - 1) & 1);
        for (uint32_t i = ns > (uint32_t)ST ? ns - ST : 0; i < ns; ++i) landed(&st_full[i % ST], (i / ST) & 1);
      }
    }
  } else if (warp >= 17) {
    // ---------------- MMA issuer of a tile (the whole warp; one elected lane issues) ----------------
    // One warp for both tiles left the tensor cores idle for a third of its time: a wait that
    // succeeds costs 115 cycles, and one tile's softmax held up the other tile's products.
    constexpr uint32_t PV_IDESC = idesc_bf16(kRows, DV, false, true);
    // A step is block t's scores and block t - 2's weights times its values: scores are two
    // blocks ahead of the softmax, and one wait covers both operands. The loop is kept this
    // plain because a lone warp takes ten cycles an instruction where the flow is not straight.
    const int x = uniform(warp - 17);
    const uint32_t tb = (uint32_t)uniform((int)tbase), sb = smem_u32(smem);
    const uint32_t s_tm = tb + C::S0 + 128 * x, o_tm = tb + C::O0 + x * DV;
    const uint64_t a0 = sdesc_sw128(sb + x * C::q_bytes, 16, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err)); };
    uint32_t ni = 0, no = 0, st = 0, ph = 0, ns = 0, nw = 0;   // items, outputs; ring; blocks scored, weighted
    bool alive = true;
    for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
      if (!wait(&q_full[x], ni & 1)) break;
      const volatile int* pl = plan + 8 * (ni & 3);
      const int nbt = uniform(pl[0]), pc = uniform(pl[3]);
      const int fx = x == 0 ? 0 : uniform(pl[2]), lx = x == 0 ? uniform(pl[1]) : nbt - 1;
      const int colsS = pc & 0xff, colsL = pc >> 8 & 0xff, sb1 = (pc >> 16) - 1;   // columns of the last first-token block (sb1) and of the last
      for (int t = 0; t < nbt + 2; ++t) {
        if (!wait(&st_full[st], ph)) { alive = false; break; }
        const uint32_t kv = sb + C::st_off + st * C::st_bytes;
        const int b = t - 2;
        if (b >= fx && b <= lx) {
          if (!wait(&p_full[2 * x + (nw & 1)], (nw >> 1) & 1)) { alive = false; break; }
          if (b == fx && no > 0 && !wait(&o_empty[x], (no - 1) & 1)) { alive = false; break; }
          tc_fence_after();
          pv_any(b == sb1 ? colsS : b == nbt - 1 ? colsL : C::BLK, o_tm, s_tm + 64 * (nw & 1), kv + C::k_bytes, C::kv_atom,
                 PV_IDESC, b > fx);
          if (b == lx) { umma_commit_warp(&o_full[x]); ++no; }
          umma_commit_warp(&pv_done[x]);
          ++nw;
        }
        if (t >= fx && t <= lx) {
          tc_fence_after();
          const uint32_t d = s_tm + 64 * (ns & 1);
          const uint32_t idesc = idesc_bf16(kRows, t == sb1 ? colsS : t == nbt - 1 ? colsL : C::BLK, false, false);
          const uint64_t b0 = sdesc_sw128(kv, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < 4 * C::QA; ++ks)
            umma_bf16_warp(d, a0 + (uint64_t)(((ks >> 2) * kAtom + (ks & 3) * 32) >> 4),
                           b0 + (uint64_t)(((ks >> 2) * C::kv_atom + (ks & 3) * 32) >> 4), idesc, ks > 0);
          umma_commit_warp(&s_full[2 * x + (ns & 1)]);
          if (t == lx) umma_commit_warp(&q_empty[x]);
          ++ns;
        }
        umma_commit_warp(&st_empty[st]);   // arrives at once where the tile had nothing to do
        if (++st == (uint32_t)ST) { st = 0; ph ^= 1u; }
      }
      if (alive && fx > lx && lane == 0) mbar_arrive(&q_empty[x]);   // an item without this tile
    }
    // every issued product completes before the CTA releases its tensor memory
    umma_commit_warp(&drain[x]);
    const unsigned long long w0 = globaltimer_ns();
    while (!mbar_try_wait(&drain[x], 0) && globaltimer_ns() - w0 < kWaitLimitNs) {}
    __syncwarp();
  } else {
    // ---------------- softmax: warps 0-7 the first tile, 8-15 the second ----------------
    const int x = warp >> 3, half = (warp >> 2) & 1;
    const int bar_id = 1 + x * 4 + (warp & 3);            // the two warps of these rows
    const int r = (warp & 3) * 32 + lane;                 // row of the tile = TMEM lane
    const int rq = r / a.G;                               // its query
    // its row of out, relative to the tile's first
    const int rel = rq < qt ? rq * a.Hq + r - rq * a.G : -1;
    const uint32_t s_base = tbase + C::S0 + 128 * x + tmem_lane_base(warp);
    const uint32_t o_addr = tbase + C::O0 + x * DV + tmem_lane_base(warp);
    const uint32_t mine = smem_u32(smem) + C::x_off + (uint32_t)((x * 2 + half) * kRows + r) * 4u;
    const uint32_t other = smem_u32(smem) + C::x_off + (uint32_t)((x * 2 + (half ^ 1)) * kRows + r) * 4u;
    uint32_t nsf = 0, nof = 0, ni = 0;
    bool alive = true;
    for (int item = blockIdx.x; item < items && alive; item += gridDim.x, ++ni) {
      const int pair = item / a.Hkv, g = item - pair * a.Hkv, t0 = pair * 2 * qt;
      const int t_first = t0 + x * qt, t_last = min(t_first + qt, a.T) - 1, t = t_first + rq;
      if (t_first >= a.T) continue;
      const bool live = rq < qt && t < a.T;
      // the first block's scores come after the item's plan
      alive = __all_sync(0xffffffffu, mbar_wait(&s_full[2 * x + (nsf & 1)], (nsf >> 1) & 1, abort_flag, a.err));
      const volatile int* pl = plan + 8 * (ni & 3);
      Item m;
      m.nbt = pl[0];
      m.klo = pl[4];
      m.ns = pl[5];
      m.sb = pl[3] >> 16;
      m.ds0 = pl[6];
      m.last = min(t0 + 2 * qt, a.T) - 1;
      const int jf = x == 0 ? 0 : pl[2], jl = x == 0 ? pl[1] : m.nbt - 1, de0 = pl[7];
      const int ds = t < de0 ? m.ds0 : window_doc(cu, a.ndocs, a.T, min(t, a.T - 1)).start;
      const int lo = max(ds, t - a.window + 1);
      const int early = min(ds + a.sinks, lo);            // first tokens: [ds, early)
      const int lo_last = max(t_last < de0 ? m.ds0 : window_doc(cu, a.ndocs, a.T, t_last).start, t_last - a.window + 1);
      float mx = -INFINITY, l = 0.f;
      bool settled = false;                               // every row of the warps has a maximum
      for (int j = jf; j <= jl && alive; ++j) {
        const int kb = item_key<C::BLK>(m, j), cols = item_cols<C::BLK>(m, j);
        const bool sink_blk = j < m.sb;
        const int pieces = cols >> 5, c0 = half * (cols >> 1);   // 16-key pieces of this half, its first column
        if (j > jf) alive = __all_sync(0xffffffffu, mbar_wait(&s_full[2 * x + (nsf & 1)], (nsf >> 1) & 1, abort_flag, a.err));
        const uint32_t s_addr = s_base + 64 * (nsf & 1);
        ++nsf;
        tc_fence_after();
        // border: key k0 + i is seen for i in [w0, w1) (the window) or [e0, e1) (first tokens)
        const bool border = sink_blk || kb < lo_last || kb + cols - 1 > t_first;
        uint32_t seen = ~0u;
        if (border) {
          const int k0 = kb + c0;
          seen = bit_range32(lo - k0, t + 1 - k0) | bit_range32(ds - k0, early - k0);
          if (sink_blk) seen = ds == m.ds0 ? bit_range32(0, m.ns - C::BLK * j - c0) : 0u;
          if (!live) seen = 0u;
        }
        // One pass: the weights under the present maximum, and whether their sum passes 2^8. They
        // wait in registers for the two halves' vote; where it asks for it (and for the first
        // blocks, before every row has a maximum) the scores are read again.
        uint32_t w[2][8];
        float ln = 0.f;
        auto weights = [&]() {
          const float off = mx == -INFINITY ? 0.f : -mx;
          const uint64_t sc2 = pack2(a.scale_log2, a.scale_log2), off2 = pack2(off, off);
          uint64_t sum0 = 0ull, sum1 = 0ull;   // FP32 pairs
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c < pieces) {
              float v[16];
              tmem_ld16(s_addr + c0 + 16 * c, v);
              tmem_ld_wait_regs(v);
              if (border) mask16(v, seen >> (16 * c));
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float2 x0 = unpack2(ffma2(pack2(v[i], v[i + 1]), sc2, off2));
                const float2 x1 = unpack2(ffma2(pack2(v[i + 2], v[i + 3]), sc2, off2));
                const float p0 = ex2_approx(x0.x), p1 = ex2_approx(x0.y), p2 = ex2_approx(x1.x), p3 = ex2_approx(x1.y);
                sum0 = fadd2(sum0, pack2(p0, p1));
                sum1 = fadd2(sum1, pack2(p2, p3));
                const __nv_bfloat162 b0 = __floats2bfloat162_rn(p0, p1), b1 = __floats2bfloat162_rn(p2, p3);
                w[c][i >> 1] = *reinterpret_cast<const uint32_t*>(&b0);
                w[c][(i >> 1) + 1] = *reinterpret_cast<const uint32_t*>(&b1);
              }
            }
          }
          const float2 s2 = unpack2(fadd2(sum0, sum1));
          ln = s2.x + s2.y;
        };
        bool slow = !settled;
        if (!slow) {
          weights();
          // a row that is none (its queries were never loaded) has no vote
          slow = named_bar_or(bar_id, 64, (live && ln > kRaise) || !alive);
        }
        if (slow) {
          float top = -INFINITY;
          for (int c = 0; c < pieces; ++c) {
            float v[16];
            tmem_ld16(s_addr + c0 + 16 * c, v);
            tmem_ld_wait_regs(v);
            if (border) mask16(v, seen >> (16 * c));
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, v[i]);
          }
          top *= a.scale_log2;
          st_shared(mine, top);
          alive = named_bar_and(bar_id, 64, alive);   // both halves leave together after a wait that gave up
          const float nm = fmaxf(mx, fmaxf(top, ld_shared(other)));
          const float c = nm == -INFINITY ? 1.f : ex2_approx(mx - nm);
          mx = nm;
          l *= c;
          // O has the products of the block before (these scores came after those of two before)
          if (j > jf && alive) alive = __all_sync(0xffffffffu, mbar_wait(&pv_done[x], (nsf - 2) & 1, abort_flag, a.err));
          if (j > jf && alive) {
            tc_fence_after();
#pragma unroll 1
            for (int d = half * (DV / 2); d < (half + 1) * (DV / 2); d += 16) {
              float o[16];
              tmem_ld16(o_addr + d, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= c;
              tmem_st16(o_addr + d, o);
            }
          }
          weights();
          settled = named_bar_and(bar_id, 64, !live || mx > -INFINITY);
        }
        l += ln;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (c < pieces) tmem_st8(s_addr + c0 + 8 * c, reinterpret_cast<const float(&)[8]>(w[c]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + ((nsf - 1) & 1)]);
      }
      // ---- the tile's rows, half the dims a thread ----
      if (alive) alive = __all_sync(0xffffffffu, mbar_wait(&o_full[x], nof & 1, abort_flag, a.err));
      ++nof;
      tc_fence_after();
      st_shared(mine + C::x_bytes, l);
      alive = named_bar_and(bar_id, 64, alive);
      if (!alive) break;
      l += ld_shared(other + C::x_bytes);
      const float inv = 1.f / l;
      const int64_t row0 = (int64_t)t_first * a.Hq + g * a.G;
      float odd = fmaf(mx, 0.f, l * 0.f);                 // NaN where anything is not finite
#pragma unroll 1
      for (int d = half * (DV / 2); d < (half + 1) * (DV / 2); d += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float o[16];
          tmem_ld16(o_addr + d + 16 * e, o);
          tmem_ld_wait_regs(o);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            odd = fmaf(o[i], 0.f, odd);
            odd = fmaf(o[i + 1], 0.f, odd);
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[i] * inv, o[i + 1] * inv);
            w[8 * e + (i >> 1)] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + (row0 + rel) * DV + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[x]);
      if (half == 0 && live && a.lse != nullptr) a.lse[row0 + rel] = fmaf(mx, 0.6931471805599453f, logf(l));
      // rows to do again (NaN compares unequal): a NaN over the half's first column marks them
      const bool bad = live && odd != 0.f;
      if (bad) a.out[(row0 + rel) * DV + half * (DV / 2)] = __ushort_as_bfloat16(0x7fff);
      if (__any_sync(0xffffffffu, bad) && lane == 0) {
        if (redo[2 * warp + 1] < 0) redo[2 * warp] = item;
        redo[2 * warp + 1] = item;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  // ---- marked rows, by all warps in turn: nothing waits for them any more ----
  if (*abort_flag) return;
  const int first = __reduce_min_sync(0xffffffffu, lane < 16 ? redo[2 * lane] : INT_MAX);
  const int last = __reduce_max_sync(0xffffffffu, lane < 16 ? redo[2 * lane + 1] : -1);
  int turn = 0;
  for (int item = first; item <= last; item += gridDim.x) {
    const int pair = item / a.Hkv, g = item - pair * a.Hkv, t0 = pair * 2 * qt;
    if (warp < 8) {   // which of 32 rows of a tile are marked; the plans' words are free by now
      const int r = (warp & 3) * 32 + lane, rq = r / a.G, t = t0 + (warp >> 2) * qt + rq;
      bool bad = false;
      if (rq < qt && t < a.T) {
        const __nv_bfloat16* o = a.out + ((int64_t)t * a.Hq + g * a.G + r - rq * a.G) * DV;
        bad = __hisnan(o[0]) || __hisnan(o[DV / 2]);
      }
      const unsigned marks = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) plan[warp] = (int)marks;
    }
    __syncthreads();
    for (int i = 0; i < 8; ++i) {
      for (unsigned m = (unsigned)plan[i]; m; m &= m - 1) {
        const int r = (i & 3) * 32 + __ffs((int)m) - 1, rq = r / a.G;
        if (turn == warp) fwd_row<DQK / 64, DV / 64>(a, t0 + (i >> 2) * qt + rq, g * a.G + r - rq * a.G, lane);
        if (++turn == kFwdThreads / 32) turn = 0;
      }
    }
    __syncthreads();
  }
}

}  // namespace

// Keys a block of the forward: the box of its k and v maps.
int window_fwd_block() { return FwdCfg<128, 128>::BLK; }

namespace {

template <int DQK, int DV>
cudaError_t launch_fwd(const WinMaps& m, const WinArgs& a, int num_sms, bool* configured, cudaStream_t stream) {
  using C = FwdCfg<DQK, DV>;
  if (!*configured) {
    const cudaError_t e =
        cudaFuncSetAttribute(window_fwd_kernel<DQK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
    if (e != cudaSuccess) return e;
    *configured = true;
  }
  const int qt = kRows / a.G;
  const int pairs = (a.T + 2 * qt - 1) / (2 * qt);
  const int64_t items = (int64_t)pairs * a.Hkv;
  const int grid = items < num_sms ? (int)items : num_sms;
  window_fwd_kernel<DQK, DV><<<grid, kFwdThreads, C::total, stream>>>(m.q, m.k, m.v, a, qt, pairs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd_tc(const WinMaps& m, const WinArgs& a, int num_sms, bool* configured, cudaStream_t stream) {
  const int i = (a.Dqk / 64 - 1) * 2 + (a.Dv / 64 - 1);
  switch (i) {
    case 0: return launch_fwd<64, 64>(m, a, num_sms, configured + i, stream);
    case 1: return launch_fwd<64, 128>(m, a, num_sms, configured + i, stream);
    case 2: return launch_fwd<128, 64>(m, a, num_sms, configured + i, stream);
    case 3: return launch_fwd<128, 128>(m, a, num_sms, configured + i, stream);
    case 4: return launch_fwd<192, 64>(m, a, num_sms, configured + i, stream);
    default: return launch_fwd<192, 128>(m, a, num_sms, configured + i, stream);
  }
}

}  // namespace irs

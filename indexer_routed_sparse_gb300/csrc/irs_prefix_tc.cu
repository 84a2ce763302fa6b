// Attention over shared prefixes on the tensor cores (tcgen05 + TMEM + TMA).
//
// Mathematics as in irs_prefix.cuh. A prefix has no mask: every row of a group attends every
// position, so this is two dense products with a softmax between them.
//
// What bounds it. 2 (Dqk + Dv) flops a (row, position) pair, and the prefix's keys and values once
// for every 256 rows of a KV head: the tensor cores for prompts, HBM for a few rows.
//
// Design.
// * A tile is 128 rows: the G query heads of a KV head for 128 / G tokens of one group. Two tiles
//   of neighbouring tokens are one item over the same key blocks, so that the tensor cores work on
//   one tile while the other's softmax runs.
// * The items of a KV head, each as many blocks long as its prefix, form one list; it is cut into
//   runs of equal length, one a CTA, so ragged prefixes and few rows load the SMs equally. The list
//   comes from the lengths on the device; nothing is read back. The CTAs of neighbouring numbers
//   take the same run for different heads, whose rows lie next to one another in the pool. An item
//   that a border cuts leaves parts (running maximum, sum, FP32 output) that a second kernel joins
//   in list order: every run gives the same bits.
// * Keys and values come through the page table by TMA, a chunk that lies in one page at a time;
//   where pages are not multiples of 8 positions, and for the positions behind the last whole
//   chunk of a prefix, by 16-byte copies with zeros behind the end: no position past it is read,
//   and 0 times whatever its value holds is never formed.
// * S[128 x block] = Q K^T lies in TMEM; the weights return over it as bf16 and are the first operand
//   of O += P V straight from TMEM. A thread has a row.
// * The tiles' products take turns: what a tile waits for is its own softmax, which the other's
//   products fill. Left to themselves both tiles' products ran at once, and then both softmaxes.
//   Blocks of 80 positions, whose weights find room beside the scores so that the next scores need
//   not wait for them, were slower (128 / 128: 2450 cycles a block of 80 for 3440 a block of 128): what
//   a softmax warp spends on a block of any size, its waits, loads and votes, is 1000 cycles.
// * The running maximum is raised only where a score passes it by 2^8 (weights stay below 2^8 and sums,
//   in FP32, far from their limits), so O is hardly ever rescaled in TMEM.
// * A weight is rounded once to bf16, as the operand that the tensor cores take.
// * Decoding, three kernels, each launched before the one before it ends: this one over the prefixes, the paged
//   decode over the own positions (irs_paged.cu), and the join of a row's parts from both.
//
// Measured (device time, replayed from a graph; of the measured 1932 TFLOP/s or 6678 GB/s):
//   8192 tokens, 64 / 4 heads of 192 / 128, over 16,384 positions: 3.55 ms, 1550 TFLOP/s, 0.80
//   4100 tokens, 32 / 8 heads of 128, over prefixes of 8000, 2051 and 5003: 296 us, 1330 TFLOP/s, 0.69; the main
//     loop takes 2900 to 3300 cycles a block of an item, of which the operands' reads and the copies' writes of
//     shared memory (128 bytes a cycle) take 2050 at least
//   1351 tokens over prefixes kept by tokens (16-byte copies): 215 us, 890 TFLOP/s, 0.46: a warp's
//     copies of 512 bytes take it 40 cycles
//   decoding, 128 sequences behind 8192 positions, 2000 own ones each: 140 us (592 MB), 0.63: the prefix 27, the
//     own positions until 122, then the join; 32 sequences behind 120,011 (64 / 8 heads): 129 us, 0.60
#include <climits>

#include "irs_internal.h"
#include "irs_paged.cuh"
#include "irs_prefix.cuh"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kRows = 128;              // rows a tile
constexpr uint32_t kAtom = 128 * 128;   // 128 rows x 64 bf16
// warps 0-3, 4-7: softmax of the two tiles, a thread a row; 8: list, queries and keys; 9: values; 10, 11: products
// of the two tiles. Registers: 384 x 168 at launch, of which the softmax's threads take 208
// and the others keep 88: 256 x 208 + 128 x 88 = 384 x 168. At 64 and 128 dims 28 to 36 bytes a thread are spilled all the same.
constexpr int kThreads = 384;
constexpr float kRaise = 256.f;         // half a block's weights of a row with a sum past this raise its maximum
constexpr int kPlanReaders = 11;        // warps that read an item's plan

template <int DQK, int DV>
struct Cfg {
  static constexpr int QA = DQK / 64, VA = DV / 64;
  static constexpr int BLK = prefix_block(DQK);            // positions a block
  static constexpr uint32_t q_bytes = QA * kAtom;          // one tile's queries
  static constexpr uint32_t atom = BLK * 128;              // BLK rows x 64 bf16
  static constexpr uint32_t k_bytes = QA * atom, v_bytes = VA * atom;
  static constexpr int KS = DQK == 64 ? 4 : DQK == 128 ? 3 : 2;                    // stages of keys
  static constexpr int VS = DQK == 64 ? (DV == 64 ? 4 : 3) : (DV == 64 ? 3 : 2);   // and values
  static constexpr uint32_t k_off = 2 * q_bytes, v_off = k_off + KS * k_bytes;
  static constexpr uint32_t bar_off = v_off + VS * v_bytes;
  static constexpr uint32_t plan_off = bar_off + 44 * 8 + 16;   // [4][8] the items' plans
  static constexpr uint32_t offsets_off = plan_off + 4 * 32;    // [2][BLK] where rows of keys and values lie
  static constexpr uint32_t total = offsets_off + 2 * BLK * 8;
  static_assert(total <= 232448, "227 KB");
  static constexpr uint32_t S0 = 0, O0 = 256;              // TMEM: scores (and weights) at 128 x, outputs at 256 + x DV
};

// D[128 x DV] (+)= P . V: P bf16 in TMEM, V a [position][dim] tile read MN-major; NK steps of 16 positions.
template <int NK>
__device__ __forceinline__ void pv_run(uint32_t d, uint32_t p, uint32_t vb, uint32_t atom, uint32_t idesc, bool accumulate) {
  const uint64_t b0 = sdesc_sw128(vb, atom, 1024);
#pragma unroll
  for (int ks = 0; ks < NK; ++ks)
    umma_bf16_ts_warp(d, p + 8 * ks, b0 + (uint64_t)((ks * 2048) >> 4), idesc, (accumulate || ks > 0) ? 1u : 0u);
}

// A row's weights of N pieces of a block, 2^(score * scale + off), as bf16 pairs, and their sum. Written in the
// order of issue: a piece's exponentials, then the sums and roundings of the piece before, so that a lone warp
// does not wait for each result in turn (pair by pair a block of 128 took 2300 cycles, so 770).
template <int N>
__device__ __forceinline__ float row_weights(const float (*v)[16], float scale, float off, uint32_t (&w)[N][8]) {
  const uint64_t sc2 = pack2(scale, scale), off2 = pack2(off, off);
  uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};   // FP32 pairs
  float p[2][16];
  auto finish = [&](int c) {
    float(&q)[16] = p[c & 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i & 3] = fadd2(sum[i & 3], pack2(q[2 * i], q[2 * i + 1]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(q[2 * i], q[2 * i + 1]);
      w[c][i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  };
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float z[16];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 f = unpack2(ffma2(pack2(v[c][i], v[c][i + 1]), sc2, off2));
      z[i] = f.x;
      z[i + 1] = f.y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(p[c & 1][i]) : "f"(z[i]));
    if (c > 0) finish(c - 1);
  }
  finish(N - 1);
  const float2 s2 = unpack2(fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3])));
  return s2.x + s2.y;
}
// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Copies blocks of a prefix's keys or values into a ring; a whole warp.
template <int ATOMS, int BLK, int ST>
struct Loader {
  const CUtensorMap* map;
  const __nv_bfloat16* base;
  int64_t sp, stt;            // strides: page, position in page
  const int32_t* row;         // the prefix's page table row
  int page_size, num_pages, chunk, head;   // chunk: positions a TMA copy (0: 16-byte copies)
  uint64_t* full;
  uint64_t* empty;
  uint32_t smem;              // of the first stage
  uint8_t* smem_p;
  int64_t* offsets;           // [BLK] in shared memory: where rows lie, or -1
  volatile int* abort_flag;
  int32_t* err;
  int lane;
  uint32_t st, ph, ns;
  bool bad;

  static constexpr uint32_t atom = BLK * 128, bytes = ATOMS * atom;

  // The page of position p, or num_pages where it is none.
  __device__ __forceinline__ int page_of(int p, int& off) {
    const int pg = p / page_size;
    off = p - pg * page_size;
    const int page = __ldg(row + pg);
    if (page >= 0 && page < num_pages) return page;
    bad = true;
    return num_pages;
  }
  // The pages of the lane's rows (lane + 32 i) of the block at position kb; the lookups run side by side.
  static constexpr int R = BLK / 32;
  __device__ __forceinline__ void look_rows(int kb, int valid, int (&page)[R], int (&off)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int p = kb + min(lane + 32 * i, valid - 1), pg = p / page_size;
      off[i] = p - pg * page_size;
      page[i] = __ldg(row + pg);
    }
  }
  // Copies the rows [r0, valid) of a block, and zeros behind them up to its end: eight lanes a row, four rows at a
  // time, by offsets that the lanes leave in shared memory. (Offsets by shuffles, and a test of each row, made a
  // copy of 512 bytes take 108 cycles of its warp, this loop 40.)
  __device__ __forceinline__ void copy_rows(int r0, int valid, const int (&page)[R], const int (&off)[R], uint32_t dst) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = page[i] >= 0 && page[i] < num_pages;
      bad |= !in;
      offsets[lane + 32 * i] = in && lane + 32 * i < valid ? (int64_t)page[i] * sp + (int64_t)off[i] * stt : -1;
    }
    __syncwarp();
    const int c8 = lane & 7;
    const __nv_bfloat16* src0 = base + c8 * 8;
#pragma unroll 8
    for (int r = r0 + (lane >> 3); r < BLK; r += 4) {
      const int64_t o = offsets[r];
      const __nv_bfloat16* src = src0 + (o < 0 ? 0 : o);
      const uint32_t d = dst + (uint32_t)r * 128u + (uint32_t)((c8 ^ (r & 7)) << 4);
#pragma unroll
      for (int c = 0; c < ATOMS; ++c) cp_async_16(d + c * atom, src + 64 * c, o < 0 ? 0u : 16u);
    }
    __syncwarp();
  }
  // Waits for the next stage.
  __device__ __forceinline__ bool stage() {
    return ns < (uint32_t)ST || __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1u, abort_flag, err));
  }
  __device__ __forceinline__ void advance() {
    ++ns;
    if (++st == (uint32_t)ST) { st = 0; ph ^= 1u; }
  }
  // The blocks [b0, b0 + nb) of a prefix of n positions. Pages are looked up a block ahead of the copies.
  __device__ __forceinline__ bool run(const int32_t* table_row, int b0, int nb, int n) {
    row = table_row;
    return chunk > 0 ? run_chunks(b0, nb, n) : run_rows(b0, nb, n);
  }
  __device__ __forceinline__ bool run_chunks(int b0, int nb, int n) {
    int page = 0, off = 0;
    auto look = [&](int b) {   // the lane's chunk of block b
      const int p = b * BLK + lane * chunk;
      if (lane * chunk < BLK && p + chunk <= n) page = page_of(p, off);
    };
    look(b0);
    for (int b = b0; b < b0 + nb; ++b) {
      const int valid = min(BLK, n - b * BLK), cols = (valid + 15) & ~15, p = page, o = off;
      if (b + 1 < b0 + nb) look(b + 1);
      if (!stage()) return false;
      const int whole = valid / chunk;
      if (whole > 0) {
        if (lane == 0) mbar_expect_tx(&full[st], (uint32_t)(whole * chunk) * 128u * ATOMS);
        __syncwarp();
        if (lane < whole) {
          uint8_t* d = smem_p + st * bytes + (uint32_t)(lane * chunk) * 128u;
#pragma unroll
          for (int c = 0; c < ATOMS; ++c) tma_load_4d(d + c * atom, map, c * 64, o, head, p, &full[st]);
        }
      }
      if (whole * chunk < cols) {
        int pages[R], offs[R];
        look_rows(b * BLK, valid, pages, offs);
        copy_rows(whole * chunk, valid, pages, offs, smem + st * bytes);
        cp_async_commit();
        cp_async_wait_pending(0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
      advance();
    }
    return true;
  }
  // Every lane's copies arrive on the stage's barrier when they have landed.
  __device__ __forceinline__ bool run_rows(int b0, int nb, int n) {
    int page[R], off[R];
    look_rows(b0 * BLK, min(BLK, n - b0 * BLK), page, off);
    for (int b = b0; b < b0 + nb; ++b) {
      if (!stage()) return false;
      copy_rows(0, min(BLK, n - b * BLK), page, off, smem + st * bytes);
      cp_async_mbar_arrive_noinc(&full[st]);
      advance();
      if (b + 1 < b0 + nb) look_rows((b + 1) * BLK, min(BLK, n - (b + 1) * BLK), page, off);
    }
    return true;
  }
  // Copies that are still in flight land before the CTA leaves.
  __device__ __forceinline__ void drain() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (*abort_flag) {
      for (uint32_t i = ns > (uint32_t)ST ? ns - ST : 0; i < ns; ++i) {
        const unsigned long long w0 = globaltimer_ns();
        while (!mbar_try_wait(&full[i % ST], (i / ST) & 1) && globaltimer_ns() - w0 < kWaitLimitNs) {}
      }
    }
    if (bad) record_error(err, IRS_DEVERR_PAGE);
  }
};

template <int DQK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, PrefixArgs a, int runs, int chunk, int q_map) {
  using C = Cfg<DQK, DV>;
  constexpr int KS = C::KS, VS = C::VS, BLK = C::BLK;
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((smem_u32(smem) & 1023u) != 0) {   // the attribute asks for it; the tiles need it
    record_error(a.err, IRS_DEVERR_TIMEOUT);
    return;
  }
  uint64_t* plan_full = reinterpret_cast<uint64_t*>(smem + C::bar_off);   // [4]
  uint64_t* plan_empty = plan_full + 4;   // [4]
  uint64_t* q_full = plan_empty + 4;      // [2]
  uint64_t* q_empty = q_full + 2;         // [2]
  uint64_t* k_full = q_empty + 2;         // [KS]
  uint64_t* k_empty = k_full + 4;
  uint64_t* v_full = k_empty + 4;         // [VS]
  uint64_t* v_empty = v_full + 4;
  uint64_t* s_full = v_empty + 4;         // [2] a tile's scores; all its earlier products are done too
  uint64_t* p_full = s_full + 2;          // [2] its weights
  uint64_t* o_full = p_full + 2;          // [2] its output
  uint64_t* o_empty = o_full + 2;         // [2]
  uint64_t* turn = o_empty + 2;           // [2] its products may be issued
  uint64_t* drain = turn + 2;             // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::bar_off + 44 * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(smem + C::plan_off);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = (int)(blockIdx.x % (unsigned)a.Hkv), run = (int)(blockIdx.x / (unsigned)a.Hkv);
  const int qt = kRows / a.G;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) { mbar_init(&plan_full[i], 1); mbar_init(&plan_empty[i], kPlanReaders); }
    for (int i = 0; i < KS; ++i) { mbar_init(&k_full[i], chunk > 0 ? 1 : 32); mbar_init(&k_empty[i], 2); }
    for (int i = 0; i < VS; ++i) { mbar_init(&v_full[i], chunk > 0 ? 1 : 32); mbar_init(&v_empty[i], 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1); mbar_init(&o_empty[i], 4);
      mbar_init(&turn[i], 1); mbar_init(&drain[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  // ---- the list of a head's blocks: its length, and where this CTA's run starts (one warp) ----
  PrefixGroup mine{0, 0, 0};              // the lane's group of the 32 from g0 on
  int64_t units = 0, pre = 0, f0 = 0, f1 = 0;   // its blocks, the blocks before it; the run
  int g0 = 0;
  auto look = [&](int base, int64_t before) {   // groups base .. base + 31; returns the blocks up to their end
    g0 = base;
    mine = PrefixGroup{0, 0, 0};
    if (base + lane < a.P) mine = prefix_group(a, base + lane);
    units = prefix_units(mine, qt, BLK);
    int64_t x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    pre = before + x - units;
    return before + __shfl_sync(0xffffffffu, x, 31);
  };
  if (warp == 8) {
    int64_t* sums = reinterpret_cast<int64_t*>(a.ws);
    int64_t total = 0;
    for (int base = 0; base < a.P; base += 32) {
      total = look(base, total);
      if (blockIdx.x == 0 && base + lane < a.P) sums[base + lane] = pre;
    }
    if (blockIdx.x == 0 && lane == 0) sums[a.P] = total;
    const int64_t share = prefix_share(total, runs);
    f0 = run * share;
    f1 = min(total, f0 + share);
    if (a.P > 32) {
      int64_t before = 0;
      for (int base = 0; base < a.P && before <= f0; base += 32) before = look(base, before);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;

  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.err));
  };
  // An item as its readers take it from its plan.
  struct Item {
    int nb, t0, t1, part, b0, n, row;   // part: 0 the whole item, 1 or 2 the run's first or second part
  };
  uint32_t items = 0;                     // read so far
  auto next_item = [&](Item& m) {
    if (!wait_all(&plan_full[items & 3], (items >> 2) & 1)) return false;
    const volatile int* pl = plan + 8 * (items & 3);
    m.nb = pl[0];
    m.t0 = pl[1];
    m.t1 = pl[2];
    m.part = pl[3];
    m.b0 = pl[4];
    m.n = pl[5];
    m.row = pl[6];
    __syncwarp();
    if (lane == 0) mbar_arrive(&plan_empty[items & 3]);
    ++items;
    return m.nb > 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ---------------- the list, queries and keys ----------------
      Loader<C::QA, BLK, KS> ld{};
      ld.map = &tm_k; ld.base = a.k + (int64_t)head * a.k_sh; ld.sp = a.k_sp; ld.stt = a.k_st;
      ld.page_size = a.page_size; ld.num_pages = a.num_pages; ld.chunk = chunk; ld.head = head;
      ld.offsets = reinterpret_cast<int64_t*>(smem + C::offsets_off);
      ld.full = k_full; ld.empty = k_empty; ld.smem_p = smem + C::k_off; ld.smem = smem_u32(smem) + C::k_off;
      ld.abort_flag = abort_flag; ld.err = a.err; ld.lane = lane;
      uint32_t np = 0, nq[2] = {0, 0};
      bool ok = true;
      auto publish = [&](const Item& m) {
        if (np >= 4 && !wait_all(&plan_empty[np & 3], ((np >> 2) - 1) & 1)) return false;
        if (lane == 0) {
          volatile int* pl = plan + 8 * (np & 3);
          pl[0] = m.nb;
          pl[1] = m.t0;
          pl[2] = m.t1;
          pl[3] = m.part;
          pl[4] = m.b0;
          pl[5] = m.n;
          pl[6] = m.row;
          mbar_arrive(&plan_full[np & 3]);
        }
        __syncwarp();
        ++np;
        return true;
      };
      auto load_q = [&](int x, const Item& m) {
        if (nq[x] > 0 && !wait_all(&q_empty[x], (nq[x] - 1) & 1)) return false;
        ++nq[x];
        const int t = m.t0 + x * qt;
        if (q_map) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[x], (uint32_t)(qt * a.G) * 128u * C::QA);
            for (int c = 0; c < C::QA; ++c)
              tma_load_3d(smem + x * C::q_bytes + c * kAtom, &tm_q, c * 64, head * a.G, t, &q_full[x]);
          }
        } else {
          // rows by address: strides that no map can have
          const uint32_t dst = smem_u32(smem) + x * C::q_bytes;
          const int c8 = lane & 7;
          for (int r = lane >> 3; r < kRows; r += 4) {
            const int tq = t + r / a.G;
            const bool live = r < qt * a.G && tq < a.T;
            const __nv_bfloat16* src = a.q + (live ? (int64_t)tq * a.q_st + (int64_t)(head * a.G + r % a.G) * a.q_sh : 0) + c8 * 8;
            const uint32_t d = dst + (uint32_t)r * 128u + (uint32_t)((c8 ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < C::QA; ++c) cp_async_16(d + c * kAtom, src + 64 * c, live ? 16u : 0u);
          }
          cp_async_commit();
          cp_async_wait_pending(0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[x]);
        }
        __syncwarp();
        return true;
      };
      int64_t f = f0;
      while (ok && f < f1) {
        const unsigned has = __ballot_sync(0xffffffffu, f >= pre && f < pre + units);
        if (has == 0) {                       // a later group
          if (g0 + 32 >= a.P) break;          // not reached on a list of the right length
          const int64_t end = __shfl_sync(0xffffffffu, pre + units, 31);
          look(g0 + 32, end);
          continue;
        }
        const int src = __ffs((int)has) - 1;
        const int first = __shfl_sync(0xffffffffu, mine.first, src), last = __shfl_sync(0xffffffffu, mine.last, src);
        const int n = __shfl_sync(0xffffffffu, mine.n, src);
        const int64_t before = __shfl_sync(0xffffffffu, pre, src);
        const int nbg = (n + BLK - 1) / BLK;
        const int pair = (int)((f - before) / nbg);
        Item m;
        m.b0 = (int)((f - before) - (int64_t)pair * nbg);
        m.nb = (int)min(f1 - f, (int64_t)(nbg - m.b0));
        m.t0 = first + pair * 2 * qt;
        m.t1 = last;
        m.part = m.nb == nbg ? 0 : f == f0 ? 1 : 2;
        m.n = n;
        m.row = a.cache_lens != nullptr ? first : g0 + src;
        ok = publish(m) && load_q(0, m) && (m.t0 + qt >= m.t1 || load_q(1, m)) &&
             ld.run(a.page_table + (int64_t)m.row * a.table_stride, m.b0, m.nb, m.n);
        f += m.nb;
      }
      if (ok) {
        Item end{};
        publish(end);
      }
      ld.drain();
      if (*abort_flag && q_map) {
        for (int x = 0; x < 2; ++x)
          if (nq[x] > 0) {
            const unsigned long long w0 = globaltimer_ns();
            while (!mbar_try_wait(&q_full[x], (nq[x] - 1) & 1) && globaltimer_ns() - w0 < kWaitLimitNs) {}
          }
      }
    } else if (warp == 9) {
      // ---------------- values ----------------
      Loader<C::VA, BLK, VS> ld{};
      ld.map = &tm_v; ld.base = a.v + (int64_t)head * a.v_sh; ld.sp = a.v_sp; ld.stt = a.v_st;
      ld.page_size = a.page_size; ld.num_pages = a.num_pages; ld.chunk = chunk; ld.head = head;
      ld.offsets = reinterpret_cast<int64_t*>(smem + C::offsets_off) + BLK;
      ld.full = v_full; ld.empty = v_empty; ld.smem_p = smem + C::v_off; ld.smem = smem_u32(smem) + C::v_off;
      ld.abort_flag = abort_flag; ld.err = a.err; ld.lane = lane;
      Item m;
      while (next_item(m))
        if (!ld.run(a.page_table + (int64_t)m.row * a.table_stride, m.b0, m.nb, m.n)) break;
      ld.drain();
    } else {
      // ---------------- the products of a tile (the whole warp; one elected lane issues) ----------------
      // A turn is a tile's weights of the block before times their values, then its scores of the next block. A
      // warp a tile, because waits and commits cost the issuing warp 100 to 300 cycles apiece, which the other's
      // products fill; and one commit a turn, whose readers release the operands.
      constexpr uint32_t PV_IDESC = idesc_bf16(kRows, DV, false, true);
      const int x = uniform(warp - 10);
      const uint32_t tb = (uint32_t)uniform((int)tbase), sb = smem_u32(smem);
      const uint32_t s_tm = tb + C::S0 + 128 * x, o_tm = tb + C::O0 + x * DV;
      const uint64_t q0 = sdesc_sw128(sb + x * C::q_bytes, 16, 1024);
      uint32_t nq = 0, no = 0, np = 0, nt = 0, ks = 0, kph = 0, vs = 0, vph = 0;
      bool alive = true;
      Item m;
      while (alive && next_item(m)) {
        const int nb = uniform(m.nb), b0 = uniform(m.b0), n = uniform(m.n);
        const bool two = m.t0 + qt < m.t1;
        if (x == 1 && !two) {                    // an item of one tile: its blocks pass by, every phase in turn
          for (int j = 0; j < nb && alive; ++j) {
            alive = wait_all(&k_full[ks], kph) && wait_all(&v_full[vs], vph);
            if (lane == 0) { mbar_arrive(&k_empty[ks]); mbar_arrive(&v_empty[vs]); }
            __syncwarp();
            if (++ks == (uint32_t)KS) { ks = 0; kph ^= 1u; }
            if (++vs == (uint32_t)VS) { vs = 0; vph ^= 1u; }
          }
          continue;
        }
        if (!wait_all(&q_full[x], nq & 1)) break;
        ++nq;
        for (int j = 0; j <= nb; ++j) {
          if (j < nb && !wait_all(&k_full[ks], kph)) { alive = false; break; }
          if (j > 0 && !(wait_all(&v_full[vs], vph) && (j > 1 || no == 0 || wait_all(&o_empty[x], (no - 1) & 1)))) { alive = false; break; }
          // A wait costs 100 to 250 cycles even where nothing is waited for, so what comes last is waited for last:
          // the weights, but at 192 dims, whose turns are longer than a softmax, the turn (294 against 306 us for
          // three prefixes at 128 / 128; 3.53 against 3.59 ms for 8192 tokens over 16,384 positions at 192 / 128).
          auto weights = [&]() { return j == 0 || wait_all(&p_full[x], np & 1); };
          if (DQK == 192 && !weights()) { alive = false; break; }
          if (two) {
            if ((x == 1 || nt > 0) && !wait_all(&turn[x], (x == 1 ? nt : nt - 1) & 1)) { alive = false; break; }
            ++nt;
          }
          if (DQK < 192 && !weights()) { alive = false; break; }
          if (chunk == 0) fence_proxy_async_smem();   // rows copied through the generic proxy
          tc_fence_after();
          if (j > 0) {
            const uint32_t vb = sb + C::v_off + vs * C::v_bytes;
            const int steps = (min(BLK, n - (b0 + j - 1) * BLK) + 15) >> 4;
            if (steps == BLK / 16) {
              pv_run<BLK / 16>(o_tm, s_tm, vb, C::atom, PV_IDESC, j > 1);
            } else {
              for (int k = 0; k < steps; ++k) pv_run<1>(o_tm, s_tm + 8 * k, vb + 2048 * k, C::atom, PV_IDESC, j > 1 || k > 0);
            }
            ++np;
            if (++vs == (uint32_t)VS) { vs = 0; vph ^= 1u; }
          }
          if (j < nb) {
            const uint32_t idesc = idesc_bf16(kRows, min(BLK, (n - (b0 + j) * BLK + 15) & ~15), false, false);
            const uint64_t b = sdesc_sw128(sb + C::k_off + ks * C::k_bytes, 16, 1024);
#pragma unroll
            for (int i = 0; i < 4 * C::QA; ++i)
              umma_bf16_warp(s_tm, q0 + (uint64_t)(((i >> 2) * kAtom + (i & 3) * 32) >> 4),
                             b + (uint64_t)(((i >> 2) * C::atom + (i & 3) * 32) >> 4), idesc, i > 0);
            if (++ks == (uint32_t)KS) { ks = 0; kph ^= 1u; }
          }
          if (two && lane == 0) mbar_arrive(&turn[x ^ 1]);
          __syncwarp();
          umma_commit_warp(j < nb ? &s_full[x] : &o_full[x]);
        }
        ++no;
      }
      // every issued product completes before the CTA releases its tensor memory
      umma_commit_warp(&drain[x]);
      const unsigned long long w0 = globaltimer_ns();
      while (!mbar_try_wait(&drain[x], 0) && globaltimer_ns() - w0 < kWaitLimitNs) {}
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------- softmax: warps 0-3 the first tile, 4-7 the second, a thread a row ----------------
    if (blockIdx.x == 0 && warp == 7) prefix_check(a, lane, 32);
    constexpr int NP = BLK / 16, HP = NP / 2;             // pieces of 16 columns; in half a block
    const int x = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                 // row of the tile = TMEM lane
    const int rq = r / a.G;                               // its token
    const int rel = rq * a.Hq + head * a.G + r - rq * a.G;   // its row of out, relative to the tile's first token's
    const uint32_t s_addr = tbase + C::S0 + 128 * x + tmem_lane_base(warp);
    const uint32_t o_addr = tbase + C::O0 + x * DV + tmem_lane_base(warp);
    const bool release = (warp & 3) == 0 && lane == 0;    // says for the tile that operands are free
    uint32_t ns = 0, no = 0, ks = 0, vs = 0;              // blocks, items; stages to release next
    bool alive = true;
    Item m;
    while (alive && next_item(m)) {
      const int t0 = m.t0 + x * qt, t = t0 + rq;
      if (t0 >= m.t1) {                                   // an item of one tile
        ks = (ks + m.nb) % KS;
        vs = (vs + m.nb) % VS;
        continue;
      }
      const bool live = rq < qt && t < m.t1;
      auto free_values = [&]() {                          // the products before the scores (or output) that came are done
        mbar_arrive(&v_empty[vs]);
        if (++vs == (uint32_t)VS) vs = 0;
      };
      float mx = -INFINITY, l = 0.f;
      bool settled = false;                               // every row of the warp has a maximum
      for (int j = 0; j < m.nb; ++j) {
        const int left = m.n - (m.b0 + j) * BLK;          // positions from the block's first on
        if (!(alive = wait_all(&s_full[x], ns & 1))) break;
        ++ns;
        tc_fence_after();
        // The common case: the first half's weights under the present maximum, while the second half loads. Where
        // a half's sum passes 2^8 both are done again.
        bool slow = !settled || left < BLK;
        float lo[HP][16], hi[HP][16];
        uint32_t w[HP][8];
        const float off = -mx;
        if (!slow) {
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_ld16(s_addr + 16 * c, lo[c]);
        }
        if (release) {
          mbar_arrive(&k_empty[ks]);
          if (++ks == (uint32_t)KS) ks = 0;
          if (j > 0) free_values();
          if (j == m.nb - 1) mbar_arrive(&q_empty[x]);
        }
        __syncwarp();
        if (!slow) {
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < HP; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(lo[c][i]));   // no use before the wait
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_ld16(s_addr + 16 * (HP + c), hi[c]);
          const float ln = row_weights<HP>(lo, a.scale_log2, off, w);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < HP; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(hi[c][i]));
          uint32_t u[HP][8];
          const float hn = row_weights<HP>(hi, a.scale_log2, off, u);
          // a row that is none has no vote; NaN goes on
          slow = __any_sync(0xffffffffu, live && (ln > kRaise || hn > kRaise));
          if (!slow) {
            l += ln + hn;
#pragma unroll
            for (int c = 0; c < HP; ++c) tmem_st8(s_addr + 8 * c, reinterpret_cast<const float(&)[8]>(w[c]));
#pragma unroll
            for (int c = 0; c < HP; ++c) tmem_st8(s_addr + 8 * (HP + c), reinterpret_cast<const float(&)[8]>(u[c]));
          }
        }
        // An item's first block (no row has a maximum yet), a prefix's last (it may end inside) and blocks that
        // raise a maximum: all scores at once, the maximum, then the weights.
        if (slow) {
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_ld16(s_addr + 16 * c, lo[c]);
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_ld16(s_addr + 16 * (HP + c), hi[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < HP; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              asm volatile("" : "+f"(lo[c][i]));
              asm volatile("" : "+f"(hi[c][i]));
            }
          if (left < BLK) {                               // columns behind the end are left from before
#pragma unroll
            for (int c = 0; c < HP; ++c)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                lo[c][i] = 16 * c + i < left ? lo[c][i] : -INFINITY;
                hi[c][i] = 16 * (HP + c) + i < left ? hi[c][i] : -INFINITY;
              }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < HP; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) top[i & 3] = max3(top[i & 3], lo[c][i], hi[c][i]);
          const float nm = fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2);
          const float f = nm == -INFINITY ? 1.f : ex2_approx(mx - nm);
          mx = nm;
          l *= f;
          if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {   // O has every earlier product: these scores were issued behind them
#pragma unroll 1
            for (int d = 0; d < DV; d += 16) {
              float o[16];
              tmem_ld16(o_addr + d, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tmem_st16(o_addr + d, o);
            }
          }
          const float now = mx == -INFINITY ? 0.f : -mx;
          l += row_weights<HP>(lo, a.scale_log2, now, w);
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_st8(s_addr + 8 * c, reinterpret_cast<const float(&)[8]>(w[c]));
          l += row_weights<HP>(hi, a.scale_log2, now, w);
#pragma unroll
          for (int c = 0; c < HP; ++c) tmem_st8(s_addr + 8 * (HP + c), reinterpret_cast<const float(&)[8]>(w[c]));
          settled = __all_sync(0xffffffffu, !live || mx > -INFINITY);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!alive) break;
      // ---- the tile's rows ----
      const bool sums = m.part != 0 || a.cache_lens != nullptr;   // FP32 sums, joined by the next kernel
      const bool joined = !sums && live && a.own_out != nullptr;
      const int64_t row = (int64_t)t0 * a.Hq + rel;
      uint4 own[2][4];                                    // 32 columns of the row's other part, fetched ahead
      auto fetch = [&](uint4 (&o)[4], int d) {
        if (joined) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint4*>(a.own_out + row * DV + d + 8 * i);
        }
      };
      fetch(own[0], 0);
      if (!(alive = wait_all(&o_full[x], no & 1))) break;
      ++no;
      if (release) free_values();
      __syncwarp();
      tc_fence_after();
      if (l == 0.f) l = -1.f;                             // attended, and every score -inf: in a part, a finite maximum wipes it out
      if (sums) {
        float* part = m.part != 0 ? prefix_part(a, run, head, m.part - 1) : prefix_rows(a);
        const int64_t rows = m.part != 0 ? kPrefixRows : (int64_t)a.T * a.Hq, at = m.part != 0 ? x * kRows + r : row;
#pragma unroll 1
        for (int d = 0; d < DV; d += 32) {
          float o[32];
          tmem_ld32(o_addr + d, o);
          tmem_ld_wait_regs(o);
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) prefix_sums4(part, rows, at, d + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (live) prefix_sums_ml(part, rows, at, DV) = make_float2(mx, l);
      } else {
        const PrefixJoin jn = live ? prefix_join_own(a, row, mx, l) : PrefixJoin{0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < DV; d += 32) {
          float o[32];
          tmem_ld32(o_addr + d, o);
          if (d + 32 < DV) fetch(own[(d / 32 + 1) & 1], d + 32);
          tmem_ld_wait_regs(o);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) prefix_mix8(w + 4 * i, jn, o + 8 * i, own[(d / 32) & 1][i]);
          store_rows32(w, a.out + (int64_t)t0 * a.Hq * DV + d, live ? rel : -1, DV, lane);
        }
        if (live && a.lse != nullptr) a.lse[row] = jn.lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[x]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Prompts: joins the parts of the items that runs' borders cut, with the rows' other parts too, and
// writes the rows of empty prefixes. The borders that cut one item share its rows, kJoinBlocks blocks a border;
// where a block has fewer than 32 rows, several groups of threads take a row's parts in turn and are then
// joined in order. Neighbouring threads have neighbouring rows, as the sums lie.
constexpr int kJoinThreads = 512, kJoinBlocks = 2;
template <int DV>
__global__ void __launch_bounds__(kJoinThreads, 2) prefix_join_kernel(PrefixArgs a, int runs) {
  constexpr int CL = DV / 8;                          // threads a row, eight columns each
  __shared__ float sm[kJoinThreads][9];
  __shared__ float2 sm_ml[kJoinThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int head = blockIdx.y, qt = kRows / a.G;
  const int64_t* pre = reinterpret_cast<const int64_t*>(a.ws);
  const int64_t total = pre[a.P], share = prefix_share(total, runs);
  const int64_t f = (int64_t)(blockIdx.x + 1) * share;
  if (f < total) {
    const int g = prefix_find(pre, a.P, f);
    const PrefixGroup grp = prefix_group(a, g);
    const int nbg = prefix_blocks(a, grp.n);
    const int pair = (int)((f - pre[g]) / nbg);
    const int64_t s = pre[g] + (int64_t)pair * nbg;
    if (s != f) {                                     // an item is cut here
      const int c0 = (int)(s / share), c1 = (int)((s + nbg - 1) / share);   // its runs: borders c0 .. c1 - 1
      const int blocks = (c1 - c0) * kJoinBlocks, me = ((int)blockIdx.x - c0) * kJoinBlocks + (int)blockIdx.z;
      int rpb = kPrefixRows / kJoinBlocks;            // rows a block
      while (rpb > 1 && rpb / 2 * blocks >= kPrefixRows) rpb /= 2;
      const int chunk = min(rpb, 32), pg = kJoinThreads / (chunk * CL);
      const int row_in = threadIdx.x % chunk, cl = threadIdx.x / chunk % CL, part_grp = threadIdx.x / (chunk * CL);
      const int64_t row0 = (int64_t)(grp.first + pair * 2 * qt) * a.Hq + head * a.G;
      const int tokens = grp.last - grp.first - pair * 2 * qt;
      const int slot0 = s != (int64_t)c0 * share ? 1 : 0;   // the item's first part is its run's second, unless the run starts with it
      for (int r = me * rpb + row_in; r - row_in < (me + 1) * rpb; r += chunk) {
        const int x = r / kRows, rr = r % kRows, rq = rr / a.G;
        const bool live = r < kPrefixRows && rq < qt && x * qt + rq < tokens;
        PrefixSum<8> sum;
        sum.clear();
        if (live) {
          constexpr int U = 2;
          for (int c = c0 + part_grp; c <= c1; c += U * pg) {
            float2 ml[U];
            float o[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int ci = c + u * pg;
              ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[u][k] = 0.f;
              if (ci <= c1) {
                float* part = prefix_part(a, ci, head, ci == c0 ? slot0 : 0);
                ml[u] = prefix_sums_ml(part, kPrefixRows, r, DV);
                prefix_sums8(o[u], part, kPrefixRows, r, 8 * cl);
              }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) sum.add(ml[u].x, ml[u].y, o[u]);
          }
        }
        if (pg > 1) {
#pragma unroll
          for (int k = 0; k < 8; ++k) sm[threadIdx.x][k] = sum.o[k];
          sm_ml[threadIdx.x] = make_float2(sum.m, sum.l);
          __syncthreads();
          if (part_grp == 0)
            for (int i = threadIdx.x + chunk * CL; i < kJoinThreads; i += chunk * CL) {
              float o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = sm[i][k];
              sum.add(sm_ml[i].x, sm_ml[i].y, o);
            }
        }
        const int64_t row = row0 + (int64_t)(x * qt + rq) * a.Hq + rr - rq * a.G;
        const bool mine = live && part_grp == 0;
        const PrefixJoin jn = mine ? prefix_join_own(a, row, sum.m, sum.l) : PrefixJoin{0.f, 0.f, 0.f};
        __syncthreads();                              // lse may be own_lse: the row's threads have read it; and the sums
        if (mine) {
          if (cl == 0 && a.lse != nullptr) a.lse[row] = jn.lse;
          prefix_store8(a, row * DV + 8 * cl, jn, sum.o);
        }
      }
    }
  }
  bool none = false;
  for (int g = threadIdx.x; g < a.P; g += kJoinThreads) none |= prefix_group(a, g).n == 0;
  if (!__syncthreads_or(none)) return;
  const float zero[8] = {};
  constexpr int R = kJoinThreads / CL;
  const int cl = threadIdx.x % CL;
  const int64_t blocks = (int64_t)gridDim.x * gridDim.z, me = (int64_t)blockIdx.x * gridDim.z + blockIdx.z;
  for (int g = 0; g < a.P; ++g) {
    const PrefixGroup grp = prefix_group(a, g);
    if (grp.n != 0) continue;
    const int64_t rows = (int64_t)(grp.last - grp.first) * a.G;
    for (int64_t base = me * R; base < rows; base += blocks * R) {
      const int64_t i = base + threadIdx.x / CL;
      const int64_t row = (grp.first + i / a.G) * a.Hq + head * a.G + i % a.G;
      const PrefixJoin jn = i < rows ? prefix_join_own(a, row, -INFINITY, 0.f) : PrefixJoin{0.f, 0.f, 0.f};
      __syncthreads();
      if (i < rows) {
        if (cl == 0 && a.lse != nullptr) a.lse[row] = jn.lse;
        prefix_store8(a, row * DV + 8 * cl, jn, zero);
      }
    }
  }
}

// Decoding: a row's parts over its group's prefix, then those over its own positions, joined in the
// order of the two lists. Eight columns a thread, neighbouring threads neighbouring rows; where the rows
// are few, pg groups of threads share a row, each taking every pg-th part, and are then joined in order.
constexpr int kStepThreads = 256, kStepBlocks = 4;   // blocks an SM
template <int DV>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks)
    prefix_step_join_kernel(PrefixArgs a, const uint8_t* own_ws, const float* own_rows, int runs, int workers, int pg) {
  constexpr int CL = DV / 8;
  __shared__ float sm[kStepThreads][9];
  __shared__ float2 sm_ml[kStepThreads];
  const int R = kStepThreads / (CL * pg);              // rows a block
  const int row_in = threadIdx.x % R, cl = threadIdx.x / R % CL, part_grp = threadIdx.x / (R * CL);
  const int64_t row = (int64_t)blockIdx.x * R + row_in;
  const bool there = row < (int64_t)a.T * a.Hq;
  // what no kernel before this one writes is looked up before these have ended
  const int t = there ? (int)(row / a.Hq) : 0, hq = (int)(row - (int64_t)t * a.Hq), head = there ? hq / a.G : 0, h = hq - head * a.G;
  const int g = prefix_group_of(a, t);
  PrefixGroup gr{0, 0, 0};
  if (g >= 0) gr = prefix_group(a, g);
  const bool live = there && prefix_length(a, t, gr.n) > 0;
  const int qt = kRows / a.G, nhb = (a.G + kHeads - 1) / kHeads, HK = a.Hkv * nhb;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int c0 = 0, np = 0, first_slot = 0, r = 0;            // the prefix's parts: runs c0 .. of the head's list, or one row
  int d0 = 0, no = 0, own_slot = 0;                     // the own positions' parts, by blocks of 16 query heads
  if (live) {
    const int64_t* pre = reinterpret_cast<const int64_t*>(a.ws);
    const int64_t* own_pre = reinterpret_cast<const int64_t*>(own_ws);
    const int64_t total = pre[a.P], before = g >= 0 ? pre[g] : 0, F0 = own_pre[t], F1 = own_pre[t + 1], own_total = own_pre[a.T];
    if (gr.n > 0) {
      const int64_t share = prefix_share(total, runs);
      const int nbg = prefix_blocks(a, gr.n), tt = t - gr.first;
      const int64_t s = before + (int64_t)(tt / (2 * qt)) * nbg;
      c0 = prefix_run(s, share);
      np = prefix_run(s + nbg - 1, share) - c0 + 1;
      first_slot = s != (int64_t)c0 * share ? 1 : 0;
      r = tt / qt % 2 * kRows + tt % qt * a.G + h;
    }
    if (F1 > F0) {
      const int64_t share = paged_share(own_total, workers);
      d0 = prefix_run(F0, share);
      no = prefix_run(F1 - 1, share) - d0 + 1;
      own_slot = F0 != (int64_t)d0 * share ? 1 : 0;
    }
  }
  const float* own_parts = reinterpret_cast<const float*>(own_ws + paged_prefix_bytes(a.T));
  const int parts = np + no;
  PrefixSum<8> sum;
  sum.clear();
  constexpr int U = 2;
  for (int p = part_grp; p < parts; p += U * pg) {
    float2 ml[U];
    float o[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = p + u * pg;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[u][k] = 0.f;
      if (i < np) {
        float* part = np == 1 ? prefix_rows(a) : prefix_part(a, c0 + i, head, i == 0 ? first_slot : 0);
        const int64_t n = np == 1 ? (int64_t)a.T * a.Hq : kPrefixRows, at = np == 1 ? row : r;
        ml[u] = prefix_sums_ml(part, n, at, DV);
        prefix_sums8(o[u], part, n, at, 8 * cl);
      } else if (i < parts && no == 1) {
        ml[u] = *reinterpret_cast<const float2*>(own_rows + (size_t)a.T * a.Hq * DV + 2 * row);
        prefix_load8(o[u], own_rows + row * DV + 8 * cl);
      } else if (i < parts) {
        const int j = i - np, hk = head * nhb + h / kHeads, hr = h % kHeads;
        const float* part = own_parts + (((size_t)(d0 + j) * HK + hk) * 2 + (j == 0 ? own_slot : 0)) * paged_part_floats(DV);
        ml[u] = make_float2(part[kHeads * DV + hr], part[kHeads * DV + kHeads + hr]);
        prefix_load8(o[u], part + hr * DV + 8 * cl);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) sum.add(ml[u].x, ml[u].y, o[u]);
  }
  if (pg > 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sm[threadIdx.x][k] = sum.o[k];
    sm_ml[threadIdx.x] = make_float2(sum.m, sum.l);
    __syncthreads();
    if (part_grp > 0) return;
    for (int i = threadIdx.x + R * CL; i < kStepThreads; i += R * CL) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = sm[i][k];
      sum.add(sm_ml[i].x, sm_ml[i].y, o);
    }
  }
  if (there) {
    const PrefixJoin jn = prefix_join_own(a, row, sum.m, sum.l);
    if (cl == 0 && a.lse != nullptr) a.lse[row] = jn.lse;
    prefix_store8(a, row * DV + 8 * cl, jn, sum.o);
  }
}

template <int DQK, int DV>
cudaError_t launch_prefix(const PrefixMaps& m, const PrefixArgs& a, int runs, bool* configured, cudaStream_t stream) {
  using C = Cfg<DQK, DV>;
  if (!*configured) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_kernel<DQK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::total);
    if (e != cudaSuccess) return e;
    *configured = true;
  }
  prefix_kernel<DQK, DV><<<runs * a.Hkv, kThreads, C::total, stream>>>(m.q, m.k, m.v, a, runs, m.chunk, m.has_q ? 1 : 0);
  return cudaGetLastError();
}

cudaError_t launch_prefix_any(const PrefixMaps& m, const PrefixArgs& a, int runs, bool* configured, cudaStream_t stream) {
  const int i = (a.Dqk / 64 - 1) * 2 + (a.Dv / 64 - 1);
  switch (i) {
    case 0: return launch_prefix<64, 64>(m, a, runs, configured + i, stream);
    case 1: return launch_prefix<64, 128>(m, a, runs, configured + i, stream);
    case 2: return launch_prefix<128, 64>(m, a, runs, configured + i, stream);
    case 3: return launch_prefix<128, 128>(m, a, runs, configured + i, stream);
    case 4: return launch_prefix<192, 64>(m, a, runs, configured + i, stream);
    default: return launch_prefix<192, 128>(m, a, runs, configured + i, stream);
  }
}

// A launch that may start before the kernel before it in the stream ends.
cudaLaunchConfig_t early(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

// Runs of a head's list: a CTA each, as many as there are SMs for all heads.
int prefix_runs(int Hkv, int num_sms) {
  const int ctas = num_sms < kMaxPrefixCtas ? num_sms : kMaxPrefixCtas;
  return ctas / Hkv > 1 ? ctas / Hkv : 1;
}

}  // namespace

int prefix_chunk(int Dqk, int page_size) {
  int c = Dqk == 192 ? 32 : 128;   // a divisor of prefix_block(Dqk)
  while (page_size % c != 0) c /= 2;
  return c < 8 ? 0 : c;
}

size_t prefix_workspace_bytes(int T, int P, int Hq, int Hkv, int Dv, bool decode) {
  size_t n = prefix_pre_bytes(P) + prefix_parts_bytes(Dv);
  if (decode) n += 2 * prefix_rows_bytes(T, Hq, Dv) + paged_workspace_bytes(T, Dv);
  return n;
}

cudaError_t launch_prefix_fwd(const PrefixMaps& m, const PrefixArgs& a, int num_sms, bool* configured, cudaStream_t stream) {
  const int runs = prefix_runs(a.Hkv, num_sms);
  const cudaError_t e = launch_prefix_any(m, a, runs, configured, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = early(dim3((unsigned)runs, (unsigned)a.Hkv, kJoinBlocks), kJoinThreads, stream, at);
  return a.Dv == 64 ? cudaLaunchKernelEx(&cfg, prefix_join_kernel<64>, a, runs)
                    : cudaLaunchKernelEx(&cfg, prefix_join_kernel<128>, a, runs);
}

cudaError_t launch_prefix_decode(const PrefixMaps& m, const PrefixArgs& a, int num_sms, bool* configured, bool* own_configured,
                                 cudaStream_t stream) {
  const int runs = prefix_runs(a.Hkv, num_sms);
  cudaError_t e = launch_prefix_any(m, a, runs, configured, stream);
  if (e != cudaSuccess) return e;
  uint8_t* ws = a.ws + prefix_pre_bytes(a.P) + prefix_parts_bytes(a.Dv) + prefix_rows_bytes(a.T, a.Hq, a.Dv);
  PagedArgs o{};
  o.q = a.q; o.q_sb = a.q_st; o.q_sh = a.q_sh;
  o.k = a.k; o.k_sp = a.k_sp; o.k_st = a.k_st; o.k_sh = a.k_sh;
  o.v = a.v; o.v_sp = a.v_sp; o.v_st = a.v_st; o.v_sh = a.v_sh;
  o.page_table = a.page_table; o.table_stride = a.table_stride;
  o.cache_lens = a.cache_lens;
  o.ws = ws + prefix_rows_bytes(a.T, a.Hq, a.Dv);
  o.err = a.err;
  o.B = a.T; o.Hq = a.Hq; o.Hkv = a.Hkv; o.G = a.G; o.Dqk = a.Dqk; o.Dv = a.Dv;
  o.max_pages = a.max_pages; o.num_pages = a.num_pages; o.page_size = a.page_size;
  o.scale_log2 = a.scale_log2;
  const PagedShared sh{a, reinterpret_cast<float*>(ws)};
  int workers = 0;
  if ((e = launch_paged_shared(o, sh, num_sms, own_configured, &workers, stream)) != cudaSuccess) return e;
  const int64_t threads = (int64_t)a.T * a.Hq * (a.Dv / 8);
  int pg = 1;   // as many threads as run at once
  while (pg < 8 && 2 * pg * threads <= (int64_t)num_sms * kStepBlocks * kStepThreads) pg *= 2;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = early(dim3((unsigned)((threads * pg + kStepThreads - 1) / kStepThreads)), kStepThreads, stream, at);
  const uint8_t* own_ws = o.ws;
  const float* own_rows = sh.rows;
  return a.Dv == 64 ? cudaLaunchKernelEx(&cfg, prefix_step_join_kernel<64>, a, own_ws, own_rows, runs, workers, pg)
                    : cudaLaunchKernelEx(&cfg, prefix_step_join_kernel<128>, a, own_ws, own_rows, runs, workers, pg);
}

}  // namespace irs

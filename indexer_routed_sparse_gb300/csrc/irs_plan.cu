// A serving step's page tables, token positions and slots, from the requests' lengths.
//
// Mathematics. Sequence b holds n_b tokens and takes m_b more; pages hold p tokens:
//   held_b = ceil(n_b / p),  need_b = ceil((n_b + m_b) / p) - held_b
//   b is given its pages where need_b <= count - at_b, at_b the sum of need_i over those i < b that are given theirs
//   page_table[b, held_b + i] = free[count - 1 - at_b - i]   for 0 <= i < need_b
//   token t = cu_b + i (cu the exclusive sums of m): position n_b + i, slot page * p + position % p
// and the sequences behind a group's first take its entries of the pages that the prefix fills.
//
// What bounds it. A step of decoding is a few hundred numbers: latency, one launch of dependent
// loads (lengths, sums, page, slot). Prompts write 12 bytes a token: HBM.
//
// Design. Every CTA sums over all sequences (a thread a run of them), so that nothing is handed from
// one CTA to another and one launch does; a token finds its sequence among the 256 runs' sums in
// shared memory and then inside the run. An entry that this call makes is worked out from the list of
// free pages wherever it is needed, never read back from the table, so CTAs need no order. A thread
// has four items in hand, so that their searches and loads run side by side. Where all together need more pages
// than are free, a warp goes through the sequences in order, to know what is given before each run. What is known of the first
// 1024 sequences stays in shared memory (480 sequences that share 7 prompts: 23 us without, 12 with).
//
// Measured (device time, replayed from a graph): 64 sequences, one token each, 6.2 us; 480 that share 7
// prompts 12.3; 48 prompts of 2000 to 60,000 tokens (16 MB) 14.3 us, 1.1 TB/s behind the
// same chain of lengths, sums, search and page that is all of the first. Launched alone, the host's 30 us. 480
// sequences of 40 tokens each 10.3 us, and 14.5 where pages run out.
#include <climits>

#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanItems = 4;        // items a thread has in hand
constexpr int kPlanCtas = 4;         // CTAs an SM
constexpr int kPlanCached = 1024;    // sequences, and borders of groups, that a CTA keeps in shared memory; others are worked out again

// What one sequence takes.
struct PlanSeq {
  int n, m, held, need, shared;   // tokens, new ones; pages; entries that its group's first sequence gives
};

// The group of sequence b, or -1; *first its first sequence. Borders that fall or pass B are cut.
__device__ __forceinline__ int plan_group(const int32_t* cu, int P, int b, int* first) {
  if (P == 0 || b < cu[0] || b >= cu[P]) return -1;
  int lo = 0, hi = P;   // cu[lo] <= b < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= b) lo = mid; else hi = mid;
  }
  *first = min(max(cu[lo], 0), b);
  return lo;
}
__device__ __forceinline__ int plan_page(const PlanArgs& a, int pos) { return a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size; }

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, const int32_t* cu, int b, bool* bad) {
  PlanSeq s;
  const int reach = a.max_pages * a.page_size;   // at most 2^30
  s.n = __ldg(a.cache_lens + b);
  s.m = __ldg(a.new_lens + b);
  s.held = s.need = s.shared = 0;
  if (s.n < 0 || s.n > reach) {   // holds nothing that is known
    *bad = true;
    s.m = 0;
    return s;
  }
  if (s.m < 0 || s.m > reach - s.n) {
    *bad = true;
    s.m = 0;
  }
  s.held = plan_page(a, s.n + a.page_size - 1);
  s.need = plan_page(a, s.n + s.m + a.page_size - 1) - s.held;
  int first = 0;
  const int g = plan_group(cu, a.P, b, &first);
  if (g >= 0 && b > first) {
    const int n = __ldg(a.prefix_lens + g);
    if (n > 0 && n <= s.n) s.shared = plan_page(a, n);
  }
  return s;
}

// Pages that the sequences before a place need, and that they are given; their tokens and shared entries.
struct PlanSum {
  int64_t pages, tokens, shared;
  int given;
};

__global__ void __launch_bounds__(kPlanThreads, kPlanCtas) plan_kernel(PlanArgs a) {
  __shared__ PlanSum sums[kPlanThreads];       // before each thread's run of sequences
  __shared__ PlanSum warp_sums[kPlanThreads / 32];
  __shared__ PlanSeq cached[kPlanCached];
  __shared__ int32_t cached_cu[kPlanCached];
  __shared__ int sm_granted;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int count = min(max(__ldg(a.free_count), 0), a.free_size);
  const int32_t* cu = a.cu_groups;
  if (a.P > 0 && a.P < kPlanCached) {
    for (int i = tid; i <= a.P; i += kPlanThreads) cached_cu[i] = a.cu_groups[i];
    cu = cached_cu;
    __syncthreads();
  }
  bool bad = false;
  auto seq = [&](int b) { return b < kPlanCached ? cached[b] : plan_seq(a, cu, b, &bad); };

  PlanSum n{};
  for (int b = b0; b < b1; ++b) {
    const PlanSeq s = plan_seq(a, cu, b, &bad);
    if (b < kPlanCached) cached[b] = s;
    n.pages += s.need;
    n.tokens += s.m;
    n.shared += s.shared;
  }
  int errors = bad ? IRS_DEVERR_PAGE : 0;
  PlanSum x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t p = __shfl_up_sync(0xffffffffu, x.pages, o), t = __shfl_up_sync(0xffffffffu, x.tokens, o),
                  h = __shfl_up_sync(0xffffffffu, x.shared, o);
    if (lane >= o) { x.pages += p; x.tokens += t; x.shared += h; }
  }
  if (lane == 31) warp_sums[warp] = x;
  if (tid == 0) sm_granted = 0;
  __syncthreads();
  PlanSum base{x.pages - n.pages, x.tokens - n.tokens, x.shared - n.shared, 0}, all{};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const PlanSum s = warp_sums[w];
    if (w < warp) { base.pages += s.pages; base.tokens += s.tokens; base.shared += s.shared; }
    all.pages += s.pages;
    all.tokens += s.tokens;
    all.shared += s.shared;
  }
  base.given = (int)min(base.pages, (int64_t)count);
  sums[tid] = base;
  __syncthreads();
  if (all.pages > count) {   // too few pages: what is given before each run of sequences, one after the other
    if (warp == 0) {
      int given = 0;
      auto need_of = [&](int b) { return b < a.B ? seq(b).need : 0; };
      int next = need_of(lane);
      for (int c = 0; c < a.B; c += 32) {   // 32 sequences at a time; next: of the following ones, looked up ahead
        const int need = next, b = c + lane;
        next = need_of(b + 32);
        int before = 0;
        for (int from = 0; from < 32;) {    // those from `from` on up to the first that finds too few
          const int left = count - given;
          const int want = lane >= from && need <= left ? need : 0;
          int64_t sum = want;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
          }
          if (lane >= from) before = given + (int)min(sum - want, (int64_t)left);
          const unsigned over = __ballot_sync(0xffffffffu, sum > left && want > 0);
          const int stop = over != 0 ? __ffs((int)over) - 1 : 31;
          given += (int)__shfl_sync(0xffffffffu, over != 0 ? sum - want : sum, stop);
          from = stop + 1;
        }
        if (b < a.B && b % per == 0) sums[b / per].given = before;
      }
    }
    __syncthreads();
    base.given = sums[tid].given;
  }

  // ---- the small results, by the first CTA ----
  if (blockIdx.x == 0) {
    PlanSum at = base;
    int granted = 0;
    for (int b = b0; b < b1; ++b) {
      const PlanSeq s = seq(b);
      a.cu_new[b] = (int)min(at.tokens, (int64_t)INT_MAX);
      const bool fits = s.need <= count - at.given;
      if (!fits) errors |= IRS_DEVERR_PAGE;
      a.lens_out[b] = fits ? s.n + s.m : s.n;
      at.tokens += s.m;
      if (fits) granted = at.given += s.need;
    }
    if (granted > 0) atomicMax(&sm_granted, granted);
    if (tid == 0) {
      a.cu_new[a.B] = (int)min(all.tokens, (int64_t)INT_MAX);
      if (all.tokens > a.tokens) errors |= IRS_DEVERR_CU_SEQLENS;
      if (count != *a.free_count) errors |= IRS_DEVERR_PAGE;
      if (a.P > 0 && (cu[0] != 0 || cu[a.P] > a.B)) errors |= IRS_DEVERR_CU_SEQLENS;
    }
    for (int g = tid; g < a.P; g += kPlanThreads) {
      if (cu[g + 1] < cu[g]) errors |= IRS_DEVERR_CU_SEQLENS;
      if (a.prefix_lens[g] < 0) errors |= IRS_DEVERR_PAGE;
    }
    if (errors) record_error(a.err, errors);
    __syncthreads();
    if (tid == 0) *a.free_left = count - sm_granted;
  }

  // The sequence that holds item i of the pages, tokens or shared entries, and the sums before it.
  auto find = [&](int64_t i, int64_t PlanSum::*of, int PlanSeq::*own, PlanSeq& s, PlanSum& at) {
    int lo = 0;   // the last run that starts at i or before
#pragma unroll
    for (int d = kPlanThreads / 2; d > 0; d >>= 1)
      if (sums[lo + d].*of <= i) lo += d;
    at = sums[lo];
    int b = min(lo * per, a.B - 1);
    s = seq(b);
    while (i >= at.*of + s.*own && b < a.B - 1) {
      at.pages += s.need;
      at.tokens += s.m;
      at.shared += s.shared;
      at.given += s.need <= count - at.given ? s.need : 0;
      s = seq(++b);
    }
    return b;
  };
  // Entry j of sequence b's table after this call.
  auto entry = [&](int b, const PlanSeq& s, int given_before, int j) {
    if (j < s.held) return a.page_table[(int64_t)b * a.table_stride + j];
    if (s.need > count - given_before) return -1;
    return a.free_pages[count - 1 - given_before - (j - s.held)];
  };
  auto given_before = [&](int b) {
    int p = sums[b / per].given;
    for (int i = b / per * per; i < b; ++i) {
      const int need = seq(i).need;
      p += need <= count - p ? need : 0;
    }
    return p;
  };

  // A CTA takes kPlanItems x kPlanThreads items at a time, neighbouring threads neighbouring items.
  constexpr int64_t kChunk = (int64_t)kPlanItems * kPlanThreads;
  const int64_t step = gridDim.x * kChunk, me = blockIdx.x * kChunk + tid;
  for (int64_t i0 = me; i0 < all.pages; i0 += step) {
    int32_t* dst[kPlanItems];
    int page[kPlanItems];
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      const int64_t i = i0 + u * kPlanThreads;
      dst[u] = nullptr;
      page[u] = -1;
      if (i < all.pages) {
        PlanSeq s;
        PlanSum at;
        const int b = find(i, &PlanSum::pages, &PlanSeq::need, s, at);
        const int j = s.held + (int)(i - at.pages);
        dst[u] = a.page_table + (int64_t)b * a.table_stride + j;
        page[u] = entry(b, s, at.given, j);
      }
    }
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u)
      if (dst[u] != nullptr) *dst[u] = page[u];
  }
  for (int64_t i0 = me; i0 < all.shared; i0 += step) {
    int32_t* dst[kPlanItems];
    const int32_t* src[kPlanItems];   // the first sequence's entry, in its row or in the list of free pages
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      const int64_t i = i0 + u * kPlanThreads;
      src[u] = nullptr;
      dst[u] = nullptr;
      if (i < all.shared) {
        PlanSeq s;
        PlanSum at;
        const int b = find(i, &PlanSum::shared, &PlanSeq::shared, s, at);
        const int j = (int)(i - at.shared);
        int first = 0;
        plan_group(cu, a.P, b, &first);
        const PlanSeq f = seq(first);
        const int32_t* row = a.page_table + (int64_t)first * a.table_stride + j;
        dst[u] = a.page_table + (int64_t)b * a.table_stride + j;
        // A page that the first sequence has not, finds none for or does not fill in this step it does not give; an
        // idle one gives what its row names, as the decode reads it.
        const int end = (j + 1) * a.page_size;   // at most the prefix's length
        if ((j < f.held && end <= f.n) || (f.n == 0 && f.m == 0)) {
          src[u] = row;
        } else if (j < f.held + f.need && end <= f.n + f.m) {
          const int before = given_before(first);
          if (f.need <= count - before) src[u] = j < f.held ? row : a.free_pages + count - 1 - before - (j - f.held);
        }
      }
    }
    int page[kPlanItems];
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) page[u] = src[u] != nullptr ? *src[u] : -1;
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u)
      if (page[u] >= 0) *dst[u] = page[u];   // an entry below 0 is no page
  }
  for (int64_t i0 = me; i0 < a.tokens; i0 += step) {
    int pos[kPlanItems], page[kPlanItems];
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      const int64_t i = i0 + u * kPlanThreads;
      pos[u] = page[u] = -1;
      if (i < all.tokens && i < a.tokens) {
        PlanSeq s;
        PlanSum at;
        const int b = find(i, &PlanSum::tokens, &PlanSeq::m, s, at);
        pos[u] = s.n + (int)(i - at.tokens);
        if (s.need <= count - at.given) page[u] = entry(b, s, at.given, plan_page(a, pos[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < kPlanItems; ++u) {
      const int64_t i = i0 + u * kPlanThreads;
      if (i < a.tokens) {
        a.positions[i] = pos[u];
        a.slots[i] = page[u] < 0 ? -1 : (int64_t)page[u] * a.page_size + pos[u] - plan_page(a, pos[u]) * a.page_size;
      }
    }
  }
}

}  // namespace

cudaError_t launch_plan(PlanArgs a, int num_sms, cudaStream_t stream) {
  a.page_shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (a.page_shift = 0; (1 << a.page_shift) < a.page_size; ++a.page_shift) {}
  // tables that are shared may have as many entries as they have places
  const int64_t items = (int64_t)a.tokens + (a.P > 0 ? (int64_t)a.B * a.max_pages / 4 : 0);
  int64_t grid = (items + kPlanItems * kPlanThreads - 1) / (kPlanItems * kPlanThreads);
  grid = grid < 1 ? 1 : grid > kPlanCtas * num_sms ? kPlanCtas * num_sms : grid;
  plan_kernel<<<(unsigned)grid, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace irs

// A serving step's page tables, token positions and slots, from the requests' lengths.
//
// Mathematics. Sequence b holds n_b tokens and takes m_b more; pages hold p tokens:
//   held_b = ceil(n_b / p),  need_b = ceil((n_b + m_b) / p) - held_b,  at_b = sum_{i<b} need_i
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
// free pages wherever it is needed, never read back from the table, so CTAs need no order.
#include <climits>

#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kPlanThreads = 256;

// What one sequence takes.
struct PlanSeq {
  int n, m, held, need, shared;   // tokens, new ones; pages; entries that its group's first sequence gives
  bool bad;
};

// The group of sequence b, or -1; *first its first sequence. Borders that fall or pass B are cut.
__device__ __forceinline__ int plan_group(const PlanArgs& a, int b, int* first) {
  int lo = 0, hi = a.P;   // cu[lo] <= b < cu[hi]
  if (a.P == 0 || b < a.cu_groups[0] || b >= a.cu_groups[a.P]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_groups[mid] <= b) lo = mid; else hi = mid;
  }
  *first = min(max(a.cu_groups[lo], 0), b);
  return lo;
}

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int b) {
  PlanSeq s;
  const int reach = a.max_pages * a.page_size;   // at most 2^30
  s.n = __ldg(a.cache_lens + b);
  s.m = __ldg(a.new_lens + b);
  s.bad = s.n < 0 || s.m < 0 || s.n > reach || s.m > reach - s.n;
  s.held = s.need = s.shared = 0;
  if (s.bad) {
    s.m = 0;
    return s;
  }
  s.held = (s.n + a.page_size - 1) / a.page_size;
  s.need = (s.n + s.m + a.page_size - 1) / a.page_size - s.held;
  int first = 0;
  const int g = plan_group(a, b, &first);
  if (g >= 0 && b > first) {
    const int n = __ldg(a.prefix_lens + g);
    if (n > 0 && n <= s.n) s.shared = n / a.page_size;
  }
  return s;
}

// Pages, tokens and shared entries of the sequences before a place.
struct PlanSum {
  int64_t pages, tokens, shared;
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ PlanSum sums[kPlanThreads + 1];   // before each thread's run of sequences, and the whole
  __shared__ PlanSum warp_sums[kPlanThreads / 32];
  __shared__ int sm_granted;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int count = min(max(__ldg(a.free_count), 0), a.free_size);
  int errors = 0;

  PlanSum n{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const PlanSeq s = plan_seq(a, b);
    n.pages += s.need;
    n.tokens += s.m;
    n.shared += s.shared;
    if (s.bad) errors |= IRS_DEVERR_PAGE;
  }
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
  PlanSum base{x.pages - n.pages, x.tokens - n.tokens, x.shared - n.shared};
  for (int w = 0; w < warp; ++w) {
    base.pages += warp_sums[w].pages;
    base.tokens += warp_sums[w].tokens;
    base.shared += warp_sums[w].shared;
  }
  sums[tid] = base;
  if (tid == kPlanThreads - 1) sums[kPlanThreads] = PlanSum{base.pages + n.pages, base.tokens + n.tokens, base.shared + n.shared};
  __syncthreads();
  const PlanSum all = sums[kPlanThreads];

  // ---- the small results, by the first CTA ----
  if (blockIdx.x == 0) {
    PlanSum at = base;
    int granted = 0;
    for (int b = b0; b < b1; ++b) {
      const PlanSeq s = plan_seq(a, b);
      a.cu_new[b] = (int)min(at.tokens, (int64_t)INT_MAX);
      const bool fits = s.need == 0 || at.pages + s.need <= count;
      if (!fits) errors |= IRS_DEVERR_PAGE;
      a.lens_out[b] = fits ? s.n + s.m : s.n;
      at.pages += s.need;
      at.tokens += s.m;
      if (fits && s.need > 0) granted = (int)at.pages;
    }
    if (granted > 0) atomicMax(&sm_granted, granted);
    if (tid == 0) {
      a.cu_new[a.B] = (int)min(all.tokens, (int64_t)INT_MAX);
      if (all.tokens > a.tokens) errors |= IRS_DEVERR_CU_SEQLENS;
      if (count != *a.free_count) errors |= IRS_DEVERR_PAGE;
      if (a.P > 0 && (a.cu_groups[0] != 0 || a.cu_groups[a.P] > a.B)) errors |= IRS_DEVERR_CU_SEQLENS;
    }
    for (int g = tid; g < a.P; g += kPlanThreads) {
      if (a.cu_groups[g + 1] < a.cu_groups[g]) errors |= IRS_DEVERR_CU_SEQLENS;
      if (a.prefix_lens[g] < 0) errors |= IRS_DEVERR_PAGE;
    }
    if (errors) record_error(a.err, errors);
    __syncthreads();
    if (tid == 0) *a.free_left = count - sm_granted;
  }

  // The sequence that holds item i of the pages, tokens or shared entries, and the sums before it.
  auto find = [&](int64_t i, int64_t PlanSum::*of, int PlanSeq::*own, PlanSeq& s, PlanSum& at) {
    int lo = 0, hi = kPlanThreads;   // sums[lo] <= i < sums[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid].*of <= i) lo = mid; else hi = mid;
    }
    at = sums[lo];
    int b = lo * per;
    s = plan_seq(a, b);
    while (i >= at.*of + s.*own && b < a.B - 1) {
      at.pages += s.need;
      at.tokens += s.m;
      at.shared += s.shared;
      s = plan_seq(a, ++b);
    }
    return b;
  };
  // Entry j of sequence b's table after this call.
  auto entry = [&](int b, const PlanSeq& s, int64_t pages_before, int j) {
    if (j < s.held) return a.page_table[(int64_t)b * a.table_stride + j];
    if (pages_before + s.need > count) return -1;
    return a.free_pages[count - 1 - (pages_before + j - s.held)];
  };
  auto pages_before = [&](int b) {
    int64_t p = sums[b / per].pages;
    for (int i = b / per * per; i < b; ++i) p += plan_seq(a, i).need;
    return p;
  };

  const int64_t step = (int64_t)gridDim.x * kPlanThreads, me = (int64_t)blockIdx.x * kPlanThreads + tid;
  for (int64_t i = me; i < all.pages; i += step) {
    PlanSeq s;
    PlanSum at;
    const int b = find(i, &PlanSum::pages, &PlanSeq::need, s, at);
    const int j = s.held + (int)(i - at.pages);
    a.page_table[(int64_t)b * a.table_stride + j] = entry(b, s, at.pages, j);
  }
  for (int64_t i = me; i < all.shared; i += step) {
    PlanSeq s;
    PlanSum at;
    const int b = find(i, &PlanSum::shared, &PlanSeq::shared, s, at);
    const int j = (int)(i - at.shared);
    int first = 0;
    plan_group(a, b, &first);
    const PlanSeq f = plan_seq(a, first);
    // entries that the first sequence has not, it does not give
    if (j < f.held + f.need) a.page_table[(int64_t)b * a.table_stride + j] = entry(first, f, pages_before(first), j);
  }
  for (int64_t i = me; i < a.tokens; i += step) {
    int pos = -1;
    int64_t slot = -1;
    if (i < all.tokens) {
      PlanSeq s;
      PlanSum at;
      const int b = find(i, &PlanSum::tokens, &PlanSeq::m, s, at);
      pos = s.n + (int)(i - at.tokens);
      const int j = pos / a.page_size;
      const int page = s.need > 0 && at.pages + s.need > count ? -1 : entry(b, s, at.pages, j);
      if (page >= 0) slot = (int64_t)page * a.page_size + pos - j * a.page_size;
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream) {
  // a thread eight items; tables that are shared may have as many entries as they have places
  const int64_t items = (int64_t)a.tokens + (a.P > 0 ? (int64_t)a.B * a.max_pages / 4 : 0);
  int64_t grid = (items + 8 * kPlanThreads - 1) / (8 * kPlanThreads);
  grid = grid < 1 ? 1 : grid > 4 * num_sms ? 4 * num_sms : grid;
  plan_kernel<<<(unsigned)grid, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace irs

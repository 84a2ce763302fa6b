// C ABI of libirs.so: argument validation (by the pages' error categories), device
// checks, TMA descriptor encoding and kernel launches. See include/irs.h for the
// contract of every entry point.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace {

thread_local char g_msg[512] = "";

irs_status fail(irs_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

struct DeviceInfo {
  bool checked = false;
  bool ok = false;
  int num_sms = 0;
  size_t l2_bytes = 0;
  size_t score_smem = 0, topk_smem = 0, attn_smem = 0, mla_smem = 0, bwd_smem = 0;   // largest configured so far
  bool proj_configured = false;
  bool paged_configured[irs::kPagedKinds] = {};
  bool prefix_configured[irs::kPrefixKinds] = {}, prefix_own_configured[irs::kPrefixKinds] = {};
  bool window_fwd_configured[irs::kWindowKinds] = {}, window_bwd_configured[irs::kWindowKinds] = {};
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// The current device must be an sm_103 GPU; returns its slot.
irs_status current_device(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(IRS_ERR_RUNTIME, "no CUDA device: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(IRS_ERR_RUNTIME, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.checked) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int l2 = 0;
    cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev);
    d.l2_bytes = (size_t)(l2 > 0 ? l2 : 0);
    d.checked = true;
    d.ok = (major == 10 && minor == 3);
    d.num_sms = sms;
  }
  if (!d.ok) return fail(IRS_ERR_RUNTIME, "libirs needs an sm_103 (GB300) device; device %d is not one", dev);
  *out = &d;
  return IRS_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D bf16 tensor map [rows][inner] (inner contiguous), SW128 boxes of {64, box_rows}.
irs_status make_tmap(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {inner * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return IRS_OK;
}

// 2-D bf16 row-tile map: rows of `inner` elements `row_stride` elements apart, box {64, 64}
// (one SW128 atom of 64 consecutive rows).
irs_status make_row_tile_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t row_stride) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {row_stride * 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (row tiles) failed (%d)", (int)r);
  return IRS_OK;
}

// 3-D bf16 map of index queries [T][rows_per_token][Di] (contiguous), box {64, Hi, 256/Hi}:
// the (query, head) rows of one score tile, for any head group of the token.
irs_status make_query_tiles_map(CUtensorMap* m, const void* base, uint64_t Di, uint64_t rows_per_token, uint64_t T,
                                uint32_t Hi) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {Di, rows_per_token, T};
  cuuint64_t strides[2] = {Di * 2, rows_per_token * Di * 2};
  cuuint32_t box[3] = {64, Hi, 256 / Hi};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (query tiles) failed (%d)", (int)r);
  return IRS_OK;
}

// Byte maps for E4M3 operands (128-byte SW128 rows of 128 elements): the queries as
// [T][rows_per_token][Di] with box {128, Hi, 256/Hi} (rows_per_token = G*Hi), the pooled keys
// as [krows][Di] with box {128, 128}.
irs_status make_e4m3_maps(CUtensorMap* tq, CUtensorMap* tk, const void* q8, const void* k8, uint64_t Di, uint64_t Hi,
                          uint64_t rows_per_token, uint64_t T, uint64_t krows) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  {
    cuuint64_t dims[3] = {Di, rows_per_token, T};
    cuuint64_t strides[2] = {Di, rows_per_token * Di};
    cuuint32_t box[3] = {128, (cuuint32_t)Hi, (cuuint32_t)(256 / Hi)};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = fn(tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(q8), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (E4M3 queries) failed (%d)", (int)r);
  }
  cuuint64_t dims[2] = {Di, krows};
  cuuint64_t strides[1] = {Di};
  cuuint32_t box[2] = {128, 128};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(k8), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (E4M3 keys) failed (%d)", (int)r);
  return IRS_OK;
}

irs_status launch_status(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(IRS_ERR_RUNTIME, "%s: %s", what, cudaGetErrorString(e));
  return IRS_OK;
}

constexpr size_t kMaxSmem = 227 * 1024;

irs_status check_index_sizes(int T, int Hi, int Di, int c, int budget, int ndocs, int max_doc_len) {
  if (T < 1) return fail(IRS_ERR_VALUE, "T must be >= 1 (got %d)", T);
  if (ndocs < 1 || ndocs > T) return fail(IRS_ERR_VALUE, "ndocs must be in [1, T] (got %d)", ndocs);
  if (max_doc_len < 1 || max_doc_len > T) return fail(IRS_ERR_VALUE, "max_doc_len must be in [1, T]");
  if (!pow2(Hi) || Hi > 256) return fail(IRS_ERR_VALUE, "Hi must be a power of two in [1, 256] (got %d)", Hi);
  if (Di != 64 && Di != 128) return fail(IRS_ERR_VALUE, "Di must be 64 or 128 (got %d)", Di);
  if (c < 1) return fail(IRS_ERR_VALUE, "c must be >= 1 (got %d)", c);
  if (budget < c || budget % c != 0) return fail(IRS_ERR_VALUE, "budget must be a positive multiple of c");
  if ((long long)T * Hi >= (1LL << 31)) return fail(IRS_ERR_VALUE, "T*Hi too large");
  if ((long long)budget + c - 1 >= (1LL << 24)) return fail(IRS_ERR_VALUE, "route width too large");
  if (irs::topk_smem_bytes(max_doc_len / c > 0 ? max_doc_len / c : 1, budget / c) > kMaxSmem)
    return fail(IRS_ERR_VALUE, "max_doc_len / c too large for the on-chip top-k (max about 48k blocks)");
  return IRS_OK;
}

// Raise the dynamic shared-memory limits of the indexer kernels to what this call needs.
irs_status configure_index(DeviceInfo* dev, const irs::IndexPlan& p) {
  if (p.score_smem > kMaxSmem) return fail(IRS_ERR_VALUE, "score tile does not fit in shared memory");
  std::lock_guard<std::mutex> lk(g_dev_mu);
  irs_status s = IRS_OK;
  if (dev->score_smem < p.score_smem) {
    if ((s = launch_status(irs::configure_score_kernels(p.score_smem), "configuring scoring")) != IRS_OK) return s;
    dev->score_smem = p.score_smem;
  }
  if (dev->topk_smem < p.topk_smem) {
    if ((s = launch_status(irs::configure_topk_kernel(p.topk_smem), "configuring top-k")) != IRS_OK) return s;
    dev->topk_smem = p.topk_smem;
  }
  return IRS_OK;
}

}  // namespace

extern "C" {

int irs_abi_version(void) { return 1; }

const char* irs_last_error(void) { return g_msg; }

size_t irs_index_workspace_bytes(int T, int Hi, int Di, int c, int budget, int ndocs, int max_doc_len,
                                 int with_score_buffer) {
  if (check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len) != IRS_OK) return 0;
  return irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, with_score_buffer != 0).ws_bytes;
}

}  // extern "C"

namespace {

irs_status check_front(const float* q_weight, const float* k_weight, float eps, const float* rope, int rope_dims,
                       int Di) {
  if (!q_weight || !k_weight) return fail(IRS_ERR_VALUE, "NULL RMSNorm weights");
  if (!aligned16(q_weight) || !aligned16(k_weight) || (rope != nullptr && !aligned16(rope)))
    return fail(IRS_ERR_VALUE, "RMSNorm weights and the rotary table must be 16-byte aligned");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(IRS_ERR_VALUE, "eps must be finite and >= 0");
  if (rope_dims < 0 || rope_dims > Di || rope_dims % 16 != 0)
    return fail(IRS_ERR_VALUE, "rope_dims must be a multiple of 16 in [0, Di] (got %d)", rope_dims);
  if (rope_dims > 0 && rope == nullptr) return fail(IRS_ERR_VALUE, "NULL rotary table");
  return IRS_OK;
}

// The indexer with or without its front half (front == nullptr).
irs_status index_impl(const void* qI, const void* kI, const float* w, const int32_t* cu_seqlens, int ndocs,
                      int max_doc_len, int T, int Hi, int Di, int c, int budget, const irs::FrontHalf* front,
                      int32_t* route_ids, float* scores_dbg, int64_t ld_scores, void* workspace,
                      size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream, int G = 1,
                      bool e4m3 = false, const void* z = nullptr) {
  irs_status s = check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len);
  if (s != IRS_OK) return s;
  if (e4m3 && (Di != 128 || front != nullptr))
    return fail(IRS_ERR_VALUE, "E4M3 scoring needs Di = 128 (no front half)");
  if (z != nullptr && !aligned16(z)) return fail(IRS_ERR_VALUE, "the compression logits must be 16-byte aligned");
  if (G < 1 || (long long)T * G * Hi >= (1LL << 31)) return fail(IRS_ERR_VALUE, "bad group count %d", G);
  if (!qI || !kI || !w || !cu_seqlens || !route_ids || !workspace)
    return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(qI) || !aligned16(kI)) return fail(IRS_ERR_VALUE, "qI and kI must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  const irs::IndexPlan p =
      irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, scores_dbg == nullptr, front != nullptr, e4m3, G);
  if (scores_dbg != nullptr && ld_scores < p.ldS)
    return fail(IRS_ERR_VALUE, "ld_scores must be >= max_doc_len / c (%lld)", (long long)p.ldS);
  if (workspace_bytes < p.ws_bytes)
    return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, p.ws_bytes);
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  if ((s = configure_index(dev, p)) != IRS_OK) return s;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // score rows: the caller's [T, G, ld_scores] (group g of token t at (t*G + g) * ld_scores),
  // or the workspace's [T, ldS], reused group after group
  float* scores = scores_dbg != nullptr ? scores_dbg : reinterpret_cast<float*>(ws + p.off_scores);
  const int64_t ldS = scores_dbg != nullptr ? ld_scores * G : p.ldS;
  const int64_t group_stride = scores_dbg != nullptr ? ld_scores : 0;
  CUtensorMap tm_q, tm_k;
  // with the front half the scores read the transformed queries from the workspace (unless
  // the caller's queries are already transformed)
  const void* qsrc =
      (front != nullptr && front->q_weight != nullptr) ? static_cast<const void*>(ws + p.off_qfront) : qI;
  if (e4m3) {
    if ((s = make_e4m3_maps(&tm_q, &tm_k, ws + p.off_q8, ws + p.off_k8, (uint64_t)Di, (uint64_t)Hi,
                            (uint64_t)G * Hi, (uint64_t)T, (uint64_t)p.nblk_cap)) != IRS_OK)
      return s;
  } else {
    if ((s = make_query_tiles_map(&tm_q, qsrc, (uint64_t)Di, (uint64_t)G * Hi, (uint64_t)T, (uint32_t)Hi)) != IRS_OK)
      return s;
    if ((s = make_tmap(&tm_k, ws + p.off_kbar, (uint64_t)Di, (uint64_t)p.nblk_cap, 128)) != IRS_OK) return s;
  }
  return launch_status(irs::launch_index(p, static_cast<const __nv_bfloat16*>(qI),
                                         static_cast<const __nv_bfloat16*>(kI), w, cu_seqlens, ndocs, max_doc_len, T,
                                         Hi, Di, c, budget, route_ids, scores, ldS, ws, err_flag, tm_q, tm_k,
                                         dev->num_sms, reinterpret_cast<cudaStream_t>(stream), front, G,
                                         group_stride, e4m3, static_cast<const __nv_bfloat16*>(z)),
                       "launching the indexer");
}

}  // namespace

extern "C" {

irs_status irs_sparse_index_score_topk(const void* qI, const void* kI, const float* w, const int32_t* cu_seqlens,
                                       int ndocs, int max_doc_len, int T, int Hi, int Di, int c, int budget,
                                       int32_t* route_ids, float* scores_dbg, int64_t ld_scores, void* workspace,
                                       size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, nullptr, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream);
}

size_t irs_index_front_workspace_bytes(int T, int Hi, int Di, int c, int budget, int ndocs, int max_doc_len,
                                       int with_score_buffer) {
  if (check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len) != IRS_OK) return 0;
  return irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, with_score_buffer != 0, true).ws_bytes;
}

irs_status irs_sparse_index_score_topk_front(const void* qI, const void* kI, const float* w,
                                             const int32_t* cu_seqlens, int ndocs, int max_doc_len, int T, int Hi,
                                             int Di, int c, int budget, const float* q_weight, const float* k_weight,
                                             float eps, const float* rope, int rope_dims, int32_t* route_ids,
                                             float* scores_dbg, int64_t ld_scores, void* workspace,
                                             size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  irs_status s = check_front(q_weight, k_weight, eps, rope, rope_dims, Di);
  if (s != IRS_OK) return s;
  const irs::FrontHalf f{q_weight, k_weight, eps, rope, rope_dims};
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, &f, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream);
}

irs_status irs_sparse_index_score_topk_grouped(const void* qI, const void* kI, const float* w,
                                               const int32_t* cu_seqlens, int ndocs, int max_doc_len, int T, int G,
                                               int Hi, int Di, int c, int budget, int32_t* route_ids,
                                               float* scores_dbg, int64_t ld_scores, void* workspace,
                                               size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, nullptr, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream, G);
}

size_t irs_index_e4m3_workspace_bytes(int T, int Hi, int Di, int c, int budget, int ndocs, int max_doc_len,
                                      int with_score_buffer) {
  if (check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len) != IRS_OK || Di != 128) return 0;
  return irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, with_score_buffer != 0, false, true).ws_bytes;
}

irs_status irs_sparse_index_score_topk_e4m3(const void* qI, const void* kI, const float* w, const int32_t* cu_seqlens,
                                            int ndocs, int max_doc_len, int T, int Hi, int Di, int c, int budget,
                                            int32_t* route_ids, float* scores_dbg, int64_t ld_scores, void* workspace,
                                            size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, nullptr, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream, 1, true);
}

size_t irs_index_summaries_workspace_bytes(int T, int G, int Hi, int Di, int c, int budget, int ndocs,
                                           int max_doc_len, int e4m3_queries, int with_score_buffer) {
  if (check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len) != IRS_OK || G < 1) return 0;
  if (e4m3_queries != 0 && Di != 128) return 0;
  return irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, with_score_buffer != 0, false, e4m3_queries != 0,
                         G)
      .ws_bytes;
}

irs_status irs_sparse_index_score_topk_summaries(const void* qI, const void* kI, const void* z, const float* w,
                                                 const int32_t* cu_seqlens, int ndocs, int max_doc_len, int T, int G,
                                                 int Hi, int Di, int c, int budget, int e4m3_queries,
                                                 int32_t* route_ids, float* scores_dbg, int64_t ld_scores,
                                                 void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                                 irs_stream_t stream) {
  if (z == nullptr) return fail(IRS_ERR_VALUE, "NULL compression logits");
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, nullptr, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream, G, e4m3_queries != 0, z);
}

size_t irs_region_summaries_workspace_bytes(int T, int Di, int c, int ndocs, int max_doc_len) {
  if (check_index_sizes(T, 1, Di, c, c, ndocs, max_doc_len) != IRS_OK) return 0;
  return irs::plan_index(T, 1, Di, c, c, ndocs, max_doc_len, false).ws_bytes;
}

irs_status irs_region_summaries(const void* kI, const void* z, const int32_t* cu_seqlens, int ndocs, int max_doc_len,
                                int T, int Di, int c, void* out, void* workspace, size_t workspace_bytes,
                                int32_t* err_flag, irs_stream_t stream) {
  irs_status s = check_index_sizes(T, 1, Di, c, c, ndocs, max_doc_len);
  if (s != IRS_OK) return s;
  if (!kI || !z || !cu_seqlens || !out || !workspace) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(kI) || !aligned16(z) || !aligned16(out))
    return fail(IRS_ERR_VALUE, "kI, z and out must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  const irs::IndexPlan p = irs::plan_index(T, 1, Di, c, c, ndocs, max_doc_len, false);
  if (workspace_bytes < p.ws_bytes)
    return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, p.ws_bytes);
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  return launch_status(irs::launch_summaries(p, static_cast<const __nv_bfloat16*>(kI),
                                             static_cast<const __nv_bfloat16*>(z), cu_seqlens, ndocs, max_doc_len, T,
                                             Di, c, static_cast<uint8_t*>(workspace), err_flag,
                                             static_cast<__nv_bfloat16*>(out), reinterpret_cast<cudaStream_t>(stream)),
                       "launching the region summaries");
}

}  // extern "C"

namespace {

irs_status projection_impl(const void* hidden, const void* weight, int T, int H, int Hi, int Di, void* qI, void* kI,
                           float* w, int32_t* err_flag, irs_stream_t stream, const float* q_weight, float eps,
                           const float* rope, int rope_dims) {
  if (T < 1 || H < 8 || H % 8 != 0) return fail(IRS_ERR_VALUE, "need T >= 1 and H a positive multiple of 8");
  if (Hi < 1 || Di < 8 || Di % 8 != 0) return fail(IRS_ERR_VALUE, "need Hi >= 1 and Di a positive multiple of 8");
  const long long N = (long long)(Hi + 1) * Di + Hi;
  if (N >= (1LL << 24) || (long long)T * N >= (1LL << 40)) return fail(IRS_ERR_VALUE, "projection too large");
  if (!hidden || !weight || !qI || !kI || !w) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(qI) || !aligned16(kI))
    return fail(IRS_ERR_VALUE, "hidden, weight, qI and kI must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(w) & 3u) != 0) return fail(IRS_ERR_VALUE, "w must be 4-byte aligned");
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!dev->proj_configured) {
      if ((s = launch_status(irs::configure_proj_kernel(), "configuring the projection")) != IRS_OK) return s;
      dev->proj_configured = true;
    }
  }
  CUtensorMap tm_x, tm_w;
  if ((s = make_tmap(&tm_x, hidden, (uint64_t)H, (uint64_t)T, 128)) != IRS_OK) return s;
  if ((s = make_tmap(&tm_w, weight, (uint64_t)H, (uint64_t)N, 256)) != IRS_OK) return s;
  irs::ProjArgs a{T, H, (int)N, Hi, Di, static_cast<__nv_bfloat16*>(qI), static_cast<__nv_bfloat16*>(kI), w,
                  err_flag, (T + 127) / 128, (int)((N + 255) / 256), q_weight, eps, rope, rope_dims};
  return launch_status(irs::launch_proj(tm_x, tm_w, a, dev->num_sms, reinterpret_cast<cudaStream_t>(stream)),
                       "launching the projection");
}

}  // namespace

extern "C" {

irs_status irs_indexer_projection(const void* hidden, const void* weight, int T, int H, int Hi, int Di, void* qI,
                                  void* kI, float* w, int32_t* err_flag, irs_stream_t stream) {
  return projection_impl(hidden, weight, T, H, Hi, Di, qI, kI, w, err_flag, stream, nullptr, 0.f, nullptr, 0);
}

irs_status irs_sparse_index_score_topk_front_keys(const void* qI, const void* kI, const float* w,
                                                  const int32_t* cu_seqlens, int ndocs, int max_doc_len, int T, int Hi,
                                                  int Di, int c, int budget, const float* k_weight, float eps,
                                                  const float* rope, int rope_dims, int32_t* route_ids,
                                                  float* scores_dbg, int64_t ld_scores, void* workspace,
                                                  size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  irs_status s = check_front(k_weight, k_weight, eps, rope, rope_dims, Di);
  if (s != IRS_OK) return s;
  const irs::FrontHalf f{nullptr, k_weight, eps, rope, rope_dims};
  return index_impl(qI, kI, w, cu_seqlens, ndocs, max_doc_len, T, Hi, Di, c, budget, &f, route_ids, scores_dbg,
                    ld_scores, workspace, workspace_bytes, err_flag, stream);
}

irs_status irs_indexer_projection_front(const void* hidden, const void* weight, int T, int H, int Hi, int Di,
                                        const float* q_weight, float eps, const float* rope, int rope_dims, void* qI,
                                        void* kI, float* w, int32_t* err_flag, irs_stream_t stream) {
  if (Di != 64 && Di != 128) return fail(IRS_ERR_VALUE, "the fused front half needs Di = 64 or 128 (got %d)", Di);
  irs_status s = check_front(q_weight, q_weight, eps, rope, rope_dims, Di);
  if (s != IRS_OK) return s;
  return projection_impl(hidden, weight, T, H, Hi, Di, qI, kI, w, err_flag, stream, q_weight, eps, rope, rope_dims);
}

irs_status irs_index_front_operands(const void* qI, const void* kI, const int32_t* cu_seqlens, int ndocs,
                                    int max_doc_len, int T, int Hi, int Di, int c, int budget, const float* q_weight,
                                    const float* k_weight, float eps, const float* rope, int rope_dims, void* q_out,
                                    void* k_out, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                    irs_stream_t stream) {
  irs_status s = check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len);
  if (s != IRS_OK) return s;
  if ((s = check_front(q_weight, k_weight, eps, rope, rope_dims, Di)) != IRS_OK) return s;
  if (!qI || !kI || !cu_seqlens || !q_out || !k_out || !workspace) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(qI) || !aligned16(kI) || !aligned16(q_out) || !aligned16(k_out))
    return fail(IRS_ERR_VALUE, "qI, kI, q_out and k_out must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  const irs::IndexPlan p = irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, false, true);
  if (workspace_bytes < p.ws_bytes)
    return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, p.ws_bytes);
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  const irs::FrontHalf f{q_weight, k_weight, eps, rope, rope_dims};
  return launch_status(irs::launch_front_operands(p, static_cast<const __nv_bfloat16*>(qI),
                                                  static_cast<const __nv_bfloat16*>(kI), cu_seqlens, ndocs,
                                                  max_doc_len, T, Hi, Di, c, static_cast<uint8_t*>(workspace),
                                                  err_flag, f, static_cast<__nv_bfloat16*>(q_out),
                                                  static_cast<__nv_bfloat16*>(k_out),
                                                  reinterpret_cast<cudaStream_t>(stream)),
                       "launching the indexer front half");
}

irs_status irs_topk_from_scores(const float* scores, int64_t ld_scores, const int32_t* cu_seqlens, int ndocs,
                                int max_doc_len, int T, int c, int budget, int32_t* route_ids, int32_t* err_flag,
                                irs_stream_t stream) {
  irs_status s = check_index_sizes(T, 1, 64, c, budget, ndocs, max_doc_len);
  if (s != IRS_OK) return s;
  if (!scores || !cu_seqlens || !route_ids) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (ld_scores < max_doc_len / c) return fail(IRS_ERR_VALUE, "ld_scores must be >= max_doc_len / c");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  const size_t smem = irs::topk_smem_bytes(max_doc_len / c > 0 ? max_doc_len / c : 1, budget / c);
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (dev->topk_smem < smem) {
      if ((s = launch_status(irs::configure_topk_kernel(smem), "configuring top-k")) != IRS_OK) return s;
      dev->topk_smem = smem;
    }
  }
  return launch_status(irs::launch_topk_from_scores(scores, ld_scores, cu_seqlens, ndocs, max_doc_len, T, c, budget,
                                                    route_ids, err_flag, reinterpret_cast<cudaStream_t>(stream)),
                       "launching top-k");
}

irs_status irs_compose_window_routes(const int32_t* route_ids, int W, const int32_t* cu_seqlens, int ndocs,
                                     int T, int window, int32_t* out, int32_t* err_flag, irs_stream_t stream) {
  if (T < 1 || W < 1 || window < 1 || ndocs < 1 || ndocs > T)
    return fail(IRS_ERR_VALUE, "bad sizes (T=%d W=%d window=%d ndocs=%d)", T, W, window, ndocs);
  if ((long long)W + window >= (1LL << 24)) return fail(IRS_ERR_VALUE, "composed width too large");
  if (!route_ids || !cu_seqlens || !out) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;
  return launch_status(irs::launch_compose_window(route_ids, W, cu_seqlens, ndocs, T, window, out, err_flag,
                                                  reinterpret_cast<cudaStream_t>(stream)),
                       "launching window composition");
}

}  // extern "C"

namespace {

// Forward attention over routes, optionally with a sliding window in front of each route
// (window > 0: cu_seqlens / ndocs give the documents the window stays inside).
irs_status attn_fwd_impl(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k, int64_t k_stride_t,
                         int64_t k_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h,
                         const int32_t* route_ids, int64_t route_stride, int T, int Tk, int Hq, int Hkv, int Dqk,
                         int Dv, int W, float scale, const int32_t* cu_seqlens, int ndocs, int window, void* out,
                         float* lse, int32_t* err_flag, irs_stream_t stream, int64_t route_group_stride = 0) {
  if (T < 0 || Tk < 1 || Hq < 1 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d Tk=%d Hq=%d Hkv=%d)", T, Tk, Hq, Hkv);
  if (Hq % Hkv != 0) return fail(IRS_ERR_VALUE, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (Dqk < 64 || Dqk > 576 || Dqk % 64 != 0) return fail(IRS_ERR_VALUE, "Dqk must be a multiple of 64 in [64, 576]");
  if (Dv < 128 || Dv > 512 || Dv % 128 != 0) return fail(IRS_ERR_VALUE, "Dv must be a multiple of 128 in [128, 512]");
  if (W < 1 || W > 4096) return fail(IRS_ERR_VALUE, "route width W must be in [1, 4096] (got %d)", W);
  if (route_stride < W) return fail(IRS_ERR_VALUE, "route_stride must be >= W");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(IRS_ERR_VALUE, "scale must be positive and finite");
  if (T == 0) return IRS_OK;
  if (!q || !k || !v || !route_ids || !out) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(IRS_ERR_VALUE, "q, k, v and out must be 16-byte aligned");
  if (q_stride_t % 8 || q_stride_h % 8 || k_stride_t % 8 || k_stride_h % 8 || v_stride_t % 8 || v_stride_h % 8)
    return fail(IRS_ERR_VALUE, "q/k/v strides must be multiples of 8 elements (16 bytes)");
  if (q_stride_t < 0 || q_stride_h < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0)
    return fail(IRS_ERR_VALUE, "negative strides are not supported");
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;

  irs::AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_st = q_stride_t; a.q_sh = q_stride_h;
  a.k_st = k_stride_t; a.k_sh = k_stride_h;
  a.v_st = v_stride_t; a.v_sh = v_stride_h;
  a.route = route_ids;
  a.route_stride = route_stride;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = err_flag;
  a.T = T; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.Dqk = Dqk; a.Dv = Dv; a.W = W;
  a.G = Hq / Hkv;
  a.HB = a.G < 16 ? a.G : 16;
  a.nhb = (a.G + a.HB - 1) / a.HB;
  a.v_alias = (v == k && v_stride_t == k_stride_t && v_stride_h == k_stride_h && Dv <= Dqk) ? 1 : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.cu = cu_seqlens;
  a.ndocs = ndocs;
  a.window = window;
  a.flag_routes = 1;
  if (window == 0 && route_group_stride == 0 && irs::mla_supported(a)) {
    const size_t smem = irs::mla_smem_bytes(a);
    {
      std::lock_guard<std::mutex> lk(g_dev_mu);
      if (dev->mla_smem < smem) {
        if ((s = launch_status(irs::configure_mla_kernel(smem), "configuring latent attention")) != IRS_OK) return s;
        dev->mla_smem = smem;
      }
    }
    return launch_status(irs::launch_mla(a, dev->num_sms, reinterpret_cast<cudaStream_t>(stream)),
                         "launching latent attention");
  }
  const irs::AttnPlan p = irs::plan_attn(a, dev->num_sms);
  if (p.smem > kMaxSmem) return fail(IRS_ERR_VALUE, "attention tile does not fit in shared memory");
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (dev->attn_smem < p.smem) {
      if ((s = launch_status(irs::configure_attn_kernel(p.smem), "configuring attention")) != IRS_OK) return s;
      dev->attn_smem = p.smem;
    }
  }
  // one launch per group of up to kMaxKvMaps KV heads (one row-tile map per head and operand)
  // per-group routes: one launch per KV head, on that head's route rows
  const int gstep = route_group_stride != 0 ? 1 : irs::kMaxKvMaps;
  for (int g0 = 0; g0 < Hkv; g0 += gstep) {
    const int ng = Hkv - g0 < gstep ? Hkv - g0 : gstep;
    a.route = route_ids + (int64_t)g0 * route_group_stride;
    a.flag_routes = (route_group_stride != 0 || g0 == 0) ? 1 : 0;
    irs::AttnMaps maps;
    memset(&maps, 0, sizeof(maps));
    // Runs of 64 consecutive routed rows load as TMA row tiles when the key/value rows cannot
    // stay L2-resident (more than half the L2): the tiles keep many more bytes in flight for
    // DRAM latency than 16-byte copies. Rows that do stay in L2 are served faster by the copies.
    const double kv_bytes = (double)Tk * Hkv * (Dqk + (a.v_alias ? 0 : Dv)) * 2.0;
    a.tile_runs = (Tk >= 64 && kv_bytes > 0.5 * (double)dev->l2_bytes) ? 1 : 0;
    for (int i = 0; i < ng && a.tile_runs; ++i) {
      const __nv_bfloat16* kb = a.k + (int64_t)(g0 + i) * k_stride_h;
      if ((s = make_row_tile_map(&maps.k[i], kb, (uint64_t)Dqk, (uint64_t)Tk, (uint64_t)k_stride_t)) != IRS_OK)
        return s;
      if (!a.v_alias) {
        const __nv_bfloat16* vb = a.v + (int64_t)(g0 + i) * v_stride_h;
        if ((s = make_row_tile_map(&maps.v[i], vb, (uint64_t)Dv, (uint64_t)Tk, (uint64_t)v_stride_t)) != IRS_OK)
          return s;
      }
    }
    a.g0 = g0;
    a.ng = ng;
    if ((s = launch_status(irs::launch_attn(maps, a, p, reinterpret_cast<cudaStream_t>(stream)),
                           "launching attention")) != IRS_OK)
      return s;
  }
  return IRS_OK;
}

}  // namespace

extern "C" {

irs_status irs_sparse_gqa_attn_fwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                   int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                   int64_t v_stride_h, const int32_t* route_ids, int64_t route_stride, int T,
                                   int Tk, int Hq, int Hkv, int Dqk, int Dv, int W, float scale, void* out,
                                   float* lse, int32_t* err_flag, irs_stream_t stream) {
  return attn_fwd_impl(q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, route_ids,
                       route_stride, T, Tk, Hq, Hkv, Dqk, Dv, W, scale, nullptr, 0, 0, out, lse, err_flag, stream);
}

irs_status irs_sparse_gqa_attn_fwd_grouped(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                           int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                           int64_t v_stride_h, const int32_t* route_ids, int64_t route_stride,
                                           int64_t route_group_stride, int T, int Tk, int Hq, int Hkv, int Dqk,
                                           int Dv, int W, float scale, void* out, float* lse, int32_t* err_flag,
                                           irs_stream_t stream) {
  if (route_group_stride < W) return fail(IRS_ERR_VALUE, "route_group_stride must be >= W");
  return attn_fwd_impl(q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, route_ids,
                       route_stride, T, Tk, Hq, Hkv, Dqk, Dv, W, scale, nullptr, 0, 0, out, lse, err_flag, stream,
                       route_group_stride);
}

irs_status irs_sparse_gqa_attn_fwd_windowed(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                            int64_t k_stride_t, int64_t k_stride_h, const void* v,
                                            int64_t v_stride_t, int64_t v_stride_h, const int32_t* route_ids,
                                            int64_t route_stride, const int32_t* cu_seqlens, int ndocs, int window,
                                            int T, int Tk, int Hq, int Hkv, int Dqk, int Dv, int W, float scale,
                                            void* out, float* lse, int32_t* err_flag, irs_stream_t stream) {
  if (window < 1) return fail(IRS_ERR_VALUE, "window must be >= 1 (got %d)", window);
  if (W < 1 || (long long)W + window > 4096)
    return fail(IRS_ERR_VALUE, "route width plus window must be in [2, 4096] (W=%d, window=%d)", W, window);
  if (ndocs < 1 || ndocs > T) return fail(IRS_ERR_VALUE, "ndocs must be in [1, T] (got %d)", ndocs);
  if (Tk < T) return fail(IRS_ERR_VALUE, "the window needs key positions for every query (Tk >= T)");
  if (cu_seqlens == nullptr) return fail(IRS_ERR_VALUE, "NULL cu_seqlens");
  return attn_fwd_impl(q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, route_ids,
                       route_stride, T, Tk, Hq, Hkv, Dqk, Dv, W, scale, cu_seqlens, ndocs, window, out, lse, err_flag,
                       stream);
}


irs_status irs_sparse_gqa_attn_bwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                   int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                   int64_t v_stride_h, const int32_t* route_ids, int64_t route_stride,
                                   const void* out, const float* lse, const void* dout, int T, int Tk, int Hq,
                                   int Hkv, int Dqk, int Dv, int W, float scale, float* dq, float* dk, float* dv,
                                   int32_t* err_flag, irs_stream_t stream) {
  if (T < 0 || Tk < 1 || Hq < 1 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d Tk=%d Hq=%d Hkv=%d)", T, Tk, Hq, Hkv);
  if (Hq % Hkv != 0) return fail(IRS_ERR_VALUE, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (Dqk < 64 || Dqk > 576 || Dqk % 64 != 0) return fail(IRS_ERR_VALUE, "Dqk must be a multiple of 64 in [64, 576]");
  if (Dv < 128 || Dv > 512 || Dv % 128 != 0) return fail(IRS_ERR_VALUE, "Dv must be a multiple of 128 in [128, 512]");
  if (W < 1 || W > 4096) return fail(IRS_ERR_VALUE, "route width W must be in [1, 4096] (got %d)", W);
  if (route_stride < W) return fail(IRS_ERR_VALUE, "route_stride must be >= W");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(IRS_ERR_VALUE, "scale must be positive and finite");
  if (T == 0) return IRS_OK;
  if (!q || !k || !v || !route_ids || !out || !lse || !dout || !dq || !dk || !dv)
    return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dk) || !aligned16(dv))
    return fail(IRS_ERR_VALUE, "q, k, v, dk and dv must be 16-byte aligned");
  if (q_stride_t % 8 || q_stride_h % 8 || k_stride_t % 8 || k_stride_h % 8 || v_stride_t % 8 || v_stride_h % 8)
    return fail(IRS_ERR_VALUE, "q/k/v strides must be multiples of 8 elements (16 bytes)");
  if (q_stride_t < 0 || q_stride_h < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0)
    return fail(IRS_ERR_VALUE, "negative strides are not supported");
  if (dv == dk) {
    // one gradient buffer for keys and values is the gradient of latent rows used as both;
    // for separate value rows it would silently add the value gradient into the key gradient
    if (Dv > Dqk) return fail(IRS_ERR_VALUE, "dv may share dk's buffer only when Dv <= Dqk");
    if (!(v == k && v_stride_t == k_stride_t && v_stride_h == k_stride_h))
      return fail(IRS_ERR_VALUE, "dv may share dk's buffer only when v is a view of k's first Dv dims");
  }
  if ((long long)T * Hkv * ((Hq / Hkv + irs::bwd_max_heads() - 1) / irs::bwd_max_heads()) > 0x7fffffffLL)
    return fail(IRS_ERR_VALUE, "too many work items");
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;

  irs::BwdArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_st = q_stride_t; a.q_sh = q_stride_h;
  a.k_st = k_stride_t; a.k_sh = k_stride_h;
  a.v_st = v_stride_t; a.v_sh = v_stride_h;
  a.route = route_ids;
  a.route_stride = route_stride;
  a.out = static_cast<const __nv_bfloat16*>(out);
  a.lse = lse;
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.err = err_flag;
  a.T = T; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.Dqk = Dqk; a.Dv = Dv; a.W = W;
  a.G = Hq / Hkv;
  a.HB = a.G < irs::bwd_max_heads() ? a.G : irs::bwd_max_heads();
  a.nhb = (a.G + a.HB - 1) / a.HB;
  a.v_alias = (v == k && v_stride_t == k_stride_t && v_stride_h == k_stride_h && Dv <= Dqk) ? 1 : 0;
  a.dv_alias = dv == dk ? 1 : 0;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.nkc = irs::bwd_pick_rows(a, kMaxSmem);
  if (a.nkc == 0) return fail(IRS_ERR_VALUE, "backward tile does not fit in shared memory");
  const size_t smem = irs::bwd_smem_bytes(a);
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (dev->bwd_smem < smem) {
      if ((s = launch_status(irs::configure_bwd_kernel(smem), "configuring the backward")) != IRS_OK) return s;
      dev->bwd_smem = smem;
    }
  }
  return launch_status(irs::launch_bwd(a, reinterpret_cast<cudaStream_t>(stream)), "launching the backward");
}

}  // extern "C"

// =====================================================================================
// Indexer without allocation: the scratch lives in one fixed device array.
//
// For callers that cannot hand the library a workspace: code that runs where cudaMalloc
// is not allowed or not wanted, e.g. plugin interfaces of inference runtimes that give a
// plugin no allocator, or latency-critical loops that must not risk the device-wide
// synchronisation an allocation can cause. The array is a file-scope __device__ object,
// so every GPU that loads this library holds it until the process exits.
// =====================================================================================
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;   // 16 MiB
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];
void* g_noalloc_addr[kMaxDevices] = {};
std::mutex g_noalloc_mu;

}  // namespace

extern "C" irs_status irs_sparse_index_score_topk_noalloc(const void* qI, const void* kI, const float* w,
                                                          const int32_t* cu_seqlens, int ndocs, int max_doc_len, int T,
                                                          int Hi, int Di, int c, int budget, int32_t* route_ids,
                                                          float* scores_dbg, int64_t ld_scores, int32_t* err_flag,
                                                          irs_stream_t stream) {
  irs_status s = check_index_sizes(T, Hi, Di, c, budget, ndocs, max_doc_len);
  if (s != IRS_OK) return s;
  if (!qI || !kI || !w || !cu_seqlens || !route_ids) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(qI) || !aligned16(kI)) return fail(IRS_ERR_VALUE, "qI and kI must be 16-byte aligned");
  const irs::IndexPlan p = irs::plan_index(T, Hi, Di, c, budget, ndocs, max_doc_len, scores_dbg == nullptr);
  if (scores_dbg != nullptr && ld_scores < p.ldS)
    return fail(IRS_ERR_VALUE, "ld_scores must be >= max_doc_len / c (%lld)", (long long)p.ldS);
  if (p.ws_bytes > kNoAllocScratchBytes)
    return fail(IRS_ERR_VALUE,
                "these sizes need %zu bytes of scratch but the fixed array holds %zu: pass a score buffer "
                "(scores_dbg) to drop the score rows from the scratch, or use irs_sparse_index_score_topk",
                p.ws_bytes, kNoAllocScratchBytes);
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  int ordinal = 0;
  if (cudaGetDevice(&ordinal) != cudaSuccess) return fail(IRS_ERR_RUNTIME, "cudaGetDevice failed");
  uint8_t* ws = nullptr;
  {
    // once per device, with that device current: the array's device address
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    if (g_noalloc_addr[ordinal] == nullptr) {
      void* addr = nullptr;
      const cudaError_t e = cudaGetSymbolAddress(&addr, g_noalloc_scratch);
      if (e != cudaSuccess)
        return fail(IRS_ERR_RUNTIME, "cudaGetSymbolAddress of the fixed scratch failed: %s", cudaGetErrorString(e));
      g_noalloc_addr[ordinal] = addr;
    }
    ws = static_cast<uint8_t*>(g_noalloc_addr[ordinal]);
  }
  if ((s = configure_index(dev, p)) != IRS_OK) return s;
  float* scores = scores_dbg != nullptr ? scores_dbg : reinterpret_cast<float*>(ws + p.off_scores);
  const int64_t ldS = scores_dbg != nullptr ? ld_scores : p.ldS;
  CUtensorMap tm_q, tm_k;
  if ((s = make_query_tiles_map(&tm_q, qI, (uint64_t)Di, (uint64_t)Hi, (uint64_t)T, (uint32_t)Hi)) != IRS_OK) return s;
  if ((s = make_tmap(&tm_k, ws + p.off_kbar, (uint64_t)Di, (uint64_t)p.nblk_cap, 128)) != IRS_OK) return s;
  return launch_status(irs::launch_index(p, static_cast<const __nv_bfloat16*>(qI),
                                         static_cast<const __nv_bfloat16*>(kI), w, cu_seqlens, ndocs, max_doc_len, T,
                                         Hi, Di, c, budget, route_ids, scores, ldS, ws, err_flag, tm_q, tm_k,
                                         dev->num_sms, reinterpret_cast<cudaStream_t>(stream)),
                       "launching the indexer (fixed scratch)");
}

// =====================================================================================
// Failure-detection self-test: one bounded wait on an mbarrier phase that nothing
// completes. The wait gives up after limit_ns, records IRS_DEVERR_TIMEOUT and the kernel
// returns, so the context stays usable (no trap, no fault, no endless loop).
// =====================================================================================
namespace {

__global__ void bounded_wait_probe_kernel(int32_t* err, unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_word;
  if (threadIdx.x != 0) return;
  irs::mbar_init(&bar, 1);
  abort_word = 0;
  irs::fence_mbar_init();
  volatile int* abort_flag = &abort_word;
  (void)irs::mbar_wait(&bar, 0, abort_flag, err, limit_ns);   // nobody arrives: gives up
}

}  // namespace

extern "C" irs_status irs_check_bounded_wait(uint64_t limit_ns, int32_t* err_flag, irs_stream_t stream) {
  if (err_flag == nullptr) return fail(IRS_ERR_VALUE, "err_flag must be a device int32");
  if (limit_ns < 1000000ull || limit_ns > 2000000000ull)
    return fail(IRS_ERR_VALUE, "limit_ns must be in [1e6, 2e9] (got %llu)", (unsigned long long)limit_ns);
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;
  bounded_wait_probe_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(err_flag, limit_ns);
  return launch_status(cudaGetLastError(), "launching the bounded-wait check");
}

// =====================================================================================
// Rotary positions, the paged cache and window attention.
// =====================================================================================
namespace {

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(void* p) { return static_cast<__nv_bfloat16*>(p); }

// The stride of a dim with one entry is never used: 0, whatever the caller's says.
void one_entry(int n, int64_t& stride) {
  if (n <= 1) stride = 0;
}

bool bad_stride(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if (s < 0 || s % 8 != 0) return true;
  return false;
}

// Whether rows of `row` elements `stride` apart along a dim of n entries are written over one another.
bool rows_meet(int n, int64_t stride, int row) { return n > 1 && stride < row; }

irs_status check_rope(const double* inv_freq, int D, int rope_dims, int start, int layout, float amplitude) {
  if (D < 8 || D % 8 != 0 || D > 4096) return fail(IRS_ERR_VALUE, "the head dim must be a multiple of 8 in [8, 4096] (got %d)", D);
  if (rope_dims < 0 || rope_dims % 16 != 0) return fail(IRS_ERR_VALUE, "rope_dims must be a multiple of 16 (got %d)", rope_dims);
  if (start < 0 || start % 8 != 0 || rope_dims > D - start)
    return fail(IRS_ERR_VALUE, "the rotated part [%d, %d + %d) must start at a multiple of 8 inside the head", start, start, rope_dims);
  if (layout != IRS_ROPE_HALF && layout != IRS_ROPE_INTERLEAVED) return fail(IRS_ERR_VALUE, "unknown rotary layout %d", layout);
  if (!std::isfinite(amplitude)) return fail(IRS_ERR_VALUE, "amplitude must be finite");
  if (rope_dims > 0 && (inv_freq == nullptr || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0))
    return fail(IRS_ERR_VALUE, "inv_freq must be an 8-byte aligned device table");
  return IRS_OK;
}

irs_status check_pool(const void* k_cache, const void* v_cache, const int32_t* page_table, const int32_t* cache_lens,
                      int64_t table_stride, int max_pages, int num_pages, int page_size) {
  if (max_pages < 1 || num_pages < 1 || page_size < 1)
    return fail(IRS_ERR_VALUE, "bad pool sizes (max_pages=%d num_pages=%d page_size=%d)", max_pages, num_pages, page_size);
  if ((long long)max_pages * page_size > (1LL << 30)) return fail(IRS_ERR_VALUE, "max_pages * page_size must be at most 2^30");
  if (table_stride < max_pages) return fail(IRS_ERR_VALUE, "table_stride must be >= max_pages");
  if (!k_cache || !v_cache || !page_table || !cache_lens) return fail(IRS_ERR_VALUE, "NULL cache pointer");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(IRS_ERR_VALUE, "the caches must be 16-byte aligned");
  return IRS_OK;
}

}  // namespace

extern "C" {

irs_status irs_rope(const void* x, int64_t x_stride_t, int64_t x_stride_h, const int32_t* positions,
                    const double* inv_freq, int T, int H, int D, int rope_dims, int start, int layout,
                    float amplitude, int transpose, void* out, int64_t out_stride_t, int64_t out_stride_h,
                    irs_stream_t stream) {
  if (T < 0 || H < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d H=%d)", T, H);
  irs_status s = check_rope(inv_freq, D, rope_dims, start, layout, amplitude);
  if (s != IRS_OK || T == 0) return s;
  if (!x || !positions || !out) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  one_entry(T, x_stride_t); one_entry(H, x_stride_h);
  one_entry(T, out_stride_t); one_entry(H, out_stride_h);
  if (!aligned16(x) || !aligned16(out)) return fail(IRS_ERR_VALUE, "x and out must be 16-byte aligned");
  if (bad_stride({x_stride_t, x_stride_h, out_stride_t, out_stride_h}))
    return fail(IRS_ERR_VALUE, "strides must be non-negative multiples of 8 elements (16 bytes)");
  if (x == out && (x_stride_t != out_stride_t || x_stride_h != out_stride_h))
    return fail(IRS_ERR_VALUE, "out may be x only with x's strides");
  if (rows_meet(T, out_stride_t, D) || rows_meet(H, out_stride_h, D))
    return fail(IRS_ERR_VALUE, "rows of out overlap: strides of at least D are needed");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  irs::RopeArgs a{};
  a.q = bf(x); a.q_st = x_stride_t; a.q_sh = x_stride_h;
  a.q_out = bf(out); a.qo_st = out_stride_t; a.qo_sh = out_stride_h;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.T = T; a.Hq = H; a.D = D; a.rope_dims = rope_dims; a.start = start;
  a.amplitude = amplitude;
  a.transpose = transpose != 0;
  a.in_place = x == out;
  return launch_status(irs::launch_rope(a, layout == IRS_ROPE_HALF, dev->num_sms, reinterpret_cast<cudaStream_t>(stream)),
                       "launching the rotation");
}

irs_status irs_paged_rope_append(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                 int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                 int64_t v_stride_h, const int32_t* cu_new, int T, int B, int Hq, int Hkv, int Dqk,
                                 int Dv, const int32_t* page_table, int64_t table_stride, int max_pages,
                                 int num_pages, int page_size, const int32_t* cache_lens, const double* inv_freq,
                                 int rope_dims, int start, int layout, float amplitude, void* k_cache,
                                 int64_t kc_stride_p, int64_t kc_stride_t, int64_t kc_stride_h, void* v_cache,
                                 int64_t vc_stride_p, int64_t vc_stride_t, int64_t vc_stride_h, void* q_out,
                                 int64_t qo_stride_t, int64_t qo_stride_h, void* k_out, int64_t ko_stride_t,
                                 int64_t ko_stride_h, int32_t* err_flag, irs_stream_t stream) {
  if (T < 0 || B < 1 || Hq < 0 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d B=%d Hq=%d Hkv=%d)", T, B, Hq, Hkv);
  if (cu_new == nullptr && T != B) return fail(IRS_ERR_VALUE, "without cu_new every sequence has one row: T (%d) must be B (%d)", T, B);
  irs_status s = check_rope(inv_freq, Dqk, rope_dims, start, layout, amplitude);
  if (s != IRS_OK) return s;
  if (Dv < 8 || Dv % 8 != 0 || Dv > 4096) return fail(IRS_ERR_VALUE, "Dv must be a multiple of 8 in [8, 4096] (got %d)", Dv);
  if (T == 0) return IRS_OK;
  if ((s = check_pool(k_cache, v_cache, page_table, cache_lens, table_stride, max_pages, num_pages, page_size)) != IRS_OK)
    return s;
  if (!k || !v || (Hq > 0 && (!q || !q_out))) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  for (int64_t* st : {&q_stride_t, &k_stride_t, &v_stride_t, &qo_stride_t, &ko_stride_t}) one_entry(T, *st);
  for (int64_t* st : {&k_stride_h, &v_stride_h, &ko_stride_h, &kc_stride_h, &vc_stride_h}) one_entry(Hkv, *st);
  one_entry(Hq, q_stride_h); one_entry(Hq, qo_stride_h);
  one_entry(num_pages, kc_stride_p); one_entry(num_pages, vc_stride_p);
  one_entry(page_size, kc_stride_t); one_entry(page_size, vc_stride_t);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out))
    return fail(IRS_ERR_VALUE, "q, k, v, q_out and k_out must be 16-byte aligned");
  if (bad_stride({q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h, kc_stride_p, kc_stride_t,
                  kc_stride_h, vc_stride_p, vc_stride_t, vc_stride_h, qo_stride_t, qo_stride_h, ko_stride_t, ko_stride_h}))
    return fail(IRS_ERR_VALUE, "strides must be non-negative multiples of 8 elements (16 bytes)");
  if (Hq > 0 && q == q_out && (q_stride_t != qo_stride_t || q_stride_h != qo_stride_h))
    return fail(IRS_ERR_VALUE, "q_out may be q only with q's strides");
  if (k == k_out && (k_stride_t != ko_stride_t || k_stride_h != ko_stride_h))
    return fail(IRS_ERR_VALUE, "k_out may be k only with k's strides");
  if (rows_meet(num_pages, kc_stride_p, Dqk) || rows_meet(page_size, kc_stride_t, Dqk) || rows_meet(Hkv, kc_stride_h, Dqk) ||
      rows_meet(num_pages, vc_stride_p, Dv) || rows_meet(page_size, vc_stride_t, Dv) || rows_meet(Hkv, vc_stride_h, Dv))
    return fail(IRS_ERR_VALUE, "rows of a cache overlap: strides of at least the head dim are needed");
  if ((Hq > 0 && (rows_meet(T, qo_stride_t, Dqk) || rows_meet(Hq, qo_stride_h, Dqk))) ||
      (k_out != nullptr && (rows_meet(T, ko_stride_t, Dqk) || rows_meet(Hkv, ko_stride_h, Dqk))))
    return fail(IRS_ERR_VALUE, "rows of q_out or k_out overlap: strides of at least Dqk are needed");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  irs::RopeArgs a{};
  a.q = bf(q); a.q_st = q_stride_t; a.q_sh = q_stride_h;
  a.k = bf(k); a.k_st = k_stride_t; a.k_sh = k_stride_h;
  a.v = bf(v); a.v_st = v_stride_t; a.v_sh = v_stride_h;
  a.inv_freq = inv_freq;
  a.cu_new = cu_new;
  a.cache_lens = cache_lens;
  a.page_table = page_table; a.table_stride = table_stride;
  a.q_out = bf(q_out); a.qo_st = qo_stride_t; a.qo_sh = qo_stride_h;
  a.k_out = bf(k_out); a.ko_st = ko_stride_t; a.ko_sh = ko_stride_h;
  a.k_cache = bf(k_cache); a.kc_sp = kc_stride_p; a.kc_st = kc_stride_t; a.kc_sh = kc_stride_h;
  a.v_cache = bf(v_cache); a.vc_sp = vc_stride_p; a.vc_st = vc_stride_t; a.vc_sh = vc_stride_h;
  a.err = err_flag;
  a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = Dqk; a.Dv = Dv;
  a.rope_dims = rope_dims; a.start = start;
  a.max_pages = max_pages; a.num_pages = num_pages; a.page_size = page_size;
  a.amplitude = amplitude;
  return launch_status(irs::launch_rope(a, layout == IRS_ROPE_HALF, dev->num_sms, reinterpret_cast<cudaStream_t>(stream)),
                       "launching the cache append");
}

size_t irs_paged_gqa_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int Dv) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Dv < 64) return 0;
  return irs::paged_workspace_bytes(B, Dv);
}

irs_status irs_paged_gqa_attn_decode(const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache,
                                     int64_t kc_stride_p, int64_t kc_stride_t, int64_t kc_stride_h,
                                     const void* v_cache, int64_t vc_stride_p, int64_t vc_stride_t,
                                     int64_t vc_stride_h, const int32_t* page_table, int64_t table_stride,
                                     int max_pages, int num_pages, int page_size, const int32_t* cache_lens,
                                     const int32_t* route_ids, int64_t route_stride, int W, int window, int sinks,
                                     int B, int Hq, int Hkv, int Dqk, int Dv, float scale, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                     irs_stream_t stream) {
  if (B < 0 || Hq < 1 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (B=%d Hq=%d Hkv=%d)", B, Hq, Hkv);
  if (Hq % Hkv != 0) return fail(IRS_ERR_VALUE, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (Dqk != 64 && Dqk != 128 && Dqk != 192 && Dqk != 256) return fail(IRS_ERR_VALUE, "Dqk must be 64, 128, 192 or 256 (got %d)", Dqk);
  if (Dv != 64 && Dv != 128 && Dv != 256) return fail(IRS_ERR_VALUE, "Dv must be 64, 128 or 256 (got %d)", Dv);
  if ((long long)B * Hq >= (1LL << 24)) return fail(IRS_ERR_VALUE, "B * Hq must be below 2^24");
  if ((long long)Hkv * ((Hq / Hkv + 15) / 16) > 1024) return fail(IRS_ERR_VALUE, "at most 1024 KV heads times blocks of 16 query heads");
  if (window < 0 || sinks < 0 || window > (1 << 30) || sinks > (1 << 30)) return fail(IRS_ERR_VALUE, "window and sinks must be in [0, 2^30]");
  if (route_ids == nullptr && W != 0) return fail(IRS_ERR_VALUE, "W must be 0 without routes");
  if (route_ids != nullptr && (W < 1 || W > (1 << 24) || route_stride < W))
    return fail(IRS_ERR_VALUE, "routes need 1 <= W <= 2^24 and route_stride >= W");
  if (sinks > 0 && window == 0 && route_ids == nullptr) return fail(IRS_ERR_VALUE, "sinks need a window or routes");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(IRS_ERR_VALUE, "scale must be positive and finite");
  if (B == 0) return IRS_OK;
  irs_status s = check_pool(k_cache, v_cache, page_table, cache_lens, table_stride, max_pages, num_pages, page_size);
  if (s != IRS_OK) return s;
  if (!q || !out || !workspace) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(out)) return fail(IRS_ERR_VALUE, "q and out must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  if (workspace_bytes < irs::paged_workspace_bytes(B, Dv))
    return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, irs::paged_workspace_bytes(B, Dv));
  one_entry(B, q_stride_b); one_entry(Hq, q_stride_h);
  one_entry(num_pages, kc_stride_p); one_entry(num_pages, vc_stride_p);
  one_entry(page_size, kc_stride_t); one_entry(page_size, vc_stride_t);
  one_entry(Hkv, kc_stride_h); one_entry(Hkv, vc_stride_h);
  if (bad_stride({q_stride_b, q_stride_h, kc_stride_p, kc_stride_t, kc_stride_h, vc_stride_p, vc_stride_t, vc_stride_h}))
    return fail(IRS_ERR_VALUE, "strides must be non-negative multiples of 8 elements (16 bytes)");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  irs::PagedArgs a{};
  a.q = bf(q); a.q_sb = q_stride_b; a.q_sh = q_stride_h;
  a.k = bf(k_cache); a.k_sp = kc_stride_p; a.k_st = kc_stride_t; a.k_sh = kc_stride_h;
  a.v = bf(v_cache); a.v_sp = vc_stride_p; a.v_st = vc_stride_t; a.v_sh = vc_stride_h;
  a.page_table = page_table; a.table_stride = table_stride;
  a.cache_lens = cache_lens;
  a.route = route_ids; a.route_stride = route_stride;
  a.out = bf(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.err = err_flag;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.Dqk = Dqk; a.Dv = Dv;
  a.W = W; a.window = window; a.sinks = sinks;
  a.max_pages = max_pages; a.num_pages = num_pages; a.page_size = page_size;
  a.scale_log2 = scale * 1.4426950408889634f;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return launch_status(irs::launch_paged_decode(a, dev->num_sms, dev->paged_configured, reinterpret_cast<cudaStream_t>(stream)),
                       "launching paged attention");
}

}  // extern "C"

namespace {

// 3-D bf16 map of a packed tensor [T][heads][D] by strides (elements), boxes of 64 dims x
// box_heads x box_tokens.
irs_status make_packed_map(CUtensorMap* m, const void* base, int D, int heads, int T, int64_t stride_h, int64_t stride_t,
                           int box_heads, int box_tokens) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  // the stride of a dim with one entry is never used, but has to be a valid one
  cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? stride_h : D) * 2, (cuuint64_t)(T > 1 ? stride_t : (int64_t)D * heads) * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (packed heads) failed (%d)", (int)r);
  return IRS_OK;
}

// Tensors with a stride of 0 over tokens or heads (broadcast) have no tensor map; they take
// the kernels that read rows by address.
bool window_has_maps(const irs::WinArgs& a) {
  auto ok = [&](int64_t st, int64_t sh, int heads) {
    return (a.T == 1 || (st > 0 && st < (1LL << 38))) && (heads == 1 || (sh > 0 && sh < (1LL << 38)));
  };
  return ok(a.q_st, a.q_sh, a.Hq) && ok(a.k_st, a.k_sh, a.Hkv) && ok(a.v_st, a.v_sh, a.Hkv);
}

// The bytes that a [T, heads, row] bf16 tensor reaches over.
struct Span {
  uintptr_t from, to;
};
Span span_of(const void* p, int T, int64_t stride_t, int heads, int64_t stride_h, int row) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + 2 * (uintptr_t)((T - 1) * stride_t + (heads - 1) * stride_h + row)};
}
Span bytes_of(const void* p, int64_t n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + (uintptr_t)n};
}
Span span_of(const void* p, int T, int heads, int row) { return span_of(p, T, (int64_t)heads * row, heads, row, row); }
// Kernels read their inputs again after the first outputs are written.
bool meets(const Span& out, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (out.from < out.to && o.from < o.to && out.from < o.to && o.from < out.to) return true;   // an empty one meets none
  return false;
}

// Checks shared by the window forward and backward; fills the arguments both need.
irs_status window_args(irs::WinArgs* a, const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                       int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h,
                       const int32_t* cu_seqlens, int ndocs, int window, int sinks, int T, int Hq, int Hkv, int Dqk,
                       int Dv, float scale, int32_t* err_flag) {
  if (T < 0 || Hq < 1 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d Hq=%d Hkv=%d)", T, Hq, Hkv);
  if (Hq % Hkv != 0) return fail(IRS_ERR_VALUE, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (Hq / Hkv > 128) return fail(IRS_ERR_VALUE, "at most 128 query heads share a KV head (got %d)", Hq / Hkv);
  if (Dqk != 64 && Dqk != 128 && Dqk != 192) return fail(IRS_ERR_VALUE, "Dqk must be 64, 128 or 192 (got %d)", Dqk);
  if (Dv != 64 && Dv != 128) return fail(IRS_ERR_VALUE, "Dv must be 64 or 128 (got %d)", Dv);
  if (window < 1 || window > (1 << 30)) return fail(IRS_ERR_VALUE, "window must be in [1, 2^30] (got %d)", window);
  if (sinks < 0 || sinks > 128) return fail(IRS_ERR_VALUE, "sinks must be in [0, 128] (got %d)", sinks);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(IRS_ERR_VALUE, "scale must be positive and finite");
  if (T > (1 << 30) || (long long)T * Hq >= (1LL << 31)) return fail(IRS_ERR_VALUE, "T * Hq must be below 2^31");
  if (T == 0) return IRS_OK;
  if (ndocs < 1 || ndocs > T) return fail(IRS_ERR_VALUE, "ndocs must be in [1, T] (got %d)", ndocs);
  for (int64_t* st : {&q_stride_t, &k_stride_t, &v_stride_t}) one_entry(T, *st);
  for (int64_t* st : {&k_stride_h, &v_stride_h}) one_entry(Hkv, *st);
  one_entry(Hq, q_stride_h);
  if (!q || !k || !v || !cu_seqlens) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return fail(IRS_ERR_VALUE, "q, k and v must be 16-byte aligned");
  if (bad_stride({q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h}))
    return fail(IRS_ERR_VALUE, "strides must be non-negative multiples of 8 elements (16 bytes)");
  a->q = bf(q); a->q_st = q_stride_t; a->q_sh = q_stride_h;
  a->k = bf(k); a->k_st = k_stride_t; a->k_sh = k_stride_h;
  a->v = bf(v); a->v_st = v_stride_t; a->v_sh = v_stride_h;
  a->cu = cu_seqlens; a->ndocs = ndocs;
  a->T = T; a->Hq = Hq; a->Hkv = Hkv; a->G = Hq / Hkv; a->Dqk = Dqk; a->Dv = Dv;
  a->window = window; a->sinks = sinks;
  a->scale = scale;
  a->scale_log2 = scale * 1.4426950408889634f;
  a->err = err_flag;
  return IRS_OK;
}

}  // namespace

extern "C" {

irs_status irs_window_gqa_attn_fwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                   int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                   int64_t v_stride_h, const int32_t* cu_seqlens, int ndocs, int window, int sinks,
                                   int T, int Hq, int Hkv, int Dqk, int Dv, float scale, void* out, float* lse,
                                   int32_t* err_flag, irs_stream_t stream) {
  irs::WinArgs a{};
  irs_status s = window_args(&a, q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h,
                             cu_seqlens, ndocs, window, sinks, T, Hq, Hkv, Dqk, Dv, scale, err_flag);
  if (s != IRS_OK || T == 0) return s;
  if (!out || !aligned16(out)) return fail(IRS_ERR_VALUE, "out must be a 16-byte aligned buffer");
  const Span in[] = {span_of(q, T, a.q_st, Hq, a.q_sh, Dqk), span_of(k, T, a.k_st, Hkv, a.k_sh, Dqk), span_of(v, T, a.v_st, Hkv, a.v_sh, Dv)};
  if (meets(span_of(out, T, Hq, Dv), {in[0], in[1], in[2]})) return fail(IRS_ERR_VALUE, "out overlaps q, k or v");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  a.out = bf(out);
  a.lse = lse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!window_has_maps(a)) return launch_status(irs::launch_window_fwd_rows(a, st), "launching window attention (rows)");
  irs::WinMaps m;
  if ((s = make_packed_map(&m.q, q, Dqk, Hq, T, q_stride_h, q_stride_t, a.G, 128 / a.G)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.k, k, Dqk, Hkv, T, k_stride_h, k_stride_t, 1, irs::window_fwd_block())) != IRS_OK) return s;
  if ((s = make_packed_map(&m.v, v, Dv, Hkv, T, v_stride_h, v_stride_t, 1, irs::window_fwd_block())) != IRS_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return launch_status(irs::launch_window_fwd_tc(m, a, dev->num_sms, dev->window_fwd_configured, st),
                       "launching window attention");
}

size_t irs_window_gqa_attn_bwd_workspace_bytes(int T, int Hq, int Hkv, int Dqk, int Dv, int ndocs, int window,
                                               int sinks) {
  if (T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Dqk < 64 || Dv < 64 || ndocs < 0 || window < 1 || sinks < 0) return 0;
  return irs::window_bwd_workspace_bytes(T, Hq, Hkv, Dqk, Dv, ndocs, window, sinks);
}

irs_status irs_window_gqa_attn_bwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                   int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                   int64_t v_stride_h, const int32_t* cu_seqlens, int ndocs, int window, int sinks,
                                   const void* out, const float* lse, const void* dout, int T, int Hq, int Hkv,
                                   int Dqk, int Dv, float scale, void* dq, void* dk, void* dv, void* workspace,
                                   size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  irs::WinArgs a{};
  irs_status s = window_args(&a, q, q_stride_t, q_stride_h, k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h,
                             cu_seqlens, ndocs, window, sinks, T, Hq, Hkv, Dqk, Dv, scale, err_flag);
  if (s != IRS_OK || T == 0) return s;
  if (!out || !lse || !dout || !dq || !dk || !dv || !workspace) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(IRS_ERR_VALUE, "out, dout, dq, dk and dv must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  const size_t need = irs::window_bwd_workspace_bytes(T, Hq, Hkv, Dqk, Dv, ndocs, window, sinks);
  if (workspace_bytes < need) return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
  const Span in[] = {span_of(q, T, a.q_st, Hq, a.q_sh, Dqk), span_of(k, T, a.k_st, Hkv, a.k_sh, Dqk),
                     span_of(v, T, a.v_st, Hkv, a.v_sh, Dv), span_of(dout, T, Hq, Dv)};
  const Span grads[] = {span_of(dq, T, Hq, Dqk), span_of(dk, T, Hkv, Dqk), span_of(dv, T, Hkv, Dv)};
  for (const Span& g : grads)
    if (meets(g, {in[0], in[1], in[2], in[3]})) return fail(IRS_ERR_VALUE, "dq, dk or dv overlaps q, k, v or dout");
  // a row of out is read for the last time before its row of dq is written, and all before dk and dv
  if (!(dq == out && Dqk == Dv) && meets(grads[0], {span_of(out, T, Hq, Dv)})) return fail(IRS_ERR_VALUE, "dq overlaps out row by other row");
  if (meets(grads[0], {grads[1], grads[2]}) || meets(grads[1], {grads[2]})) return fail(IRS_ERR_VALUE, "dq, dk and dv overlap");
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  a.out = bf(const_cast<void*>(out));
  a.lse_in = lse;
  a.dout = bf(dout);
  a.dq = bf(dq); a.dk = bf(dk); a.dv = bf(dv);
  irs::WinSinks sk;
  irs::window_bwd_layout(static_cast<uint8_t*>(workspace), T, Hq, Hkv, Dqk, Dv, ndocs, window, sinks, &a, &sk);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!window_has_maps(a)) return launch_status(irs::launch_window_bwd_rows(a, st), "launching the window backward (rows)");
  const int hc = a.G < 64 ? a.G : 64;
  irs::WinBwdMaps m;
  if ((s = make_packed_map(&m.q, q, Dqk, Hq, T, q_stride_h, q_stride_t, a.G, 128 / a.G)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.q2, q, Dqk, Hq, T, q_stride_h, q_stride_t, hc, 64 / hc)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.dout, dout, Dv, Hq, T, Dv, (int64_t)Hq * Dv, a.G, 128 / a.G)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.dout2, dout, Dv, Hq, T, Dv, (int64_t)Hq * Dv, hc, 64 / hc)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.k, k, Dqk, Hkv, T, k_stride_h, k_stride_t, 1, 128)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.v, v, Dv, Hkv, T, v_stride_h, v_stride_t, 1, 128)) != IRS_OK) return s;
  const int blk = irs::window_dq_block();
  if ((s = make_packed_map(&m.kq, k, Dqk, Hkv, T, k_stride_h, k_stride_t, 1, blk)) != IRS_OK) return s;
  if ((s = make_packed_map(&m.vq, v, Dv, Hkv, T, v_stride_h, v_stride_t, 1, blk)) != IRS_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return launch_status(irs::launch_window_bwd_tc(m, a, sk, dev->num_sms, dev->window_bwd_configured, st),
                       "launching the window attention backward");
}

irs_status irs_paged_plan(const int32_t* cache_lens, const int32_t* new_lens, int B, int32_t* page_table,
                          int64_t table_stride, int max_pages, int page_size, const int32_t* free_pages, int free_size,
                          const int32_t* free_count, const int32_t* cu_groups, const int32_t* prefix_lens, int P,
                          int tokens, int32_t* cu_new, int32_t* positions, int64_t* slots, int32_t* lens_out,
                          int32_t* free_left, int32_t* err_flag, irs_stream_t stream) {
  if (B < 1 || P < 0 || tokens < 0 || free_size < 0) return fail(IRS_ERR_VALUE, "bad sizes (B=%d P=%d tokens=%d free_size=%d)", B, P, tokens, free_size);
  if (max_pages < 1 || page_size < 1) return fail(IRS_ERR_VALUE, "bad pool sizes (max_pages=%d page_size=%d)", max_pages, page_size);
  if ((long long)max_pages * page_size > (1LL << 30)) return fail(IRS_ERR_VALUE, "max_pages * page_size must be at most 2^30");
  if (B > 1 && table_stride < max_pages) return fail(IRS_ERR_VALUE, "table_stride must be >= max_pages");
  if (!cache_lens || !new_lens || !page_table || !free_count || !cu_new || !lens_out || !free_left)
    return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if ((tokens > 0 && (!positions || !slots)) || (free_size > 0 && !free_pages) || (P > 0 && (!cu_groups || !prefix_lens)))
    return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  const Span out[] = {bytes_of(cu_new, 4 * ((int64_t)B + 1)), bytes_of(positions, 4 * (int64_t)tokens), bytes_of(slots, 8 * (int64_t)tokens),
                      bytes_of(lens_out, 4 * (int64_t)B), bytes_of(free_left, 4),
                      bytes_of(page_table, 4 * ((B - 1) * (B > 1 ? table_stride : 0) + max_pages))};
  const Span in[] = {bytes_of(cache_lens, 4 * (int64_t)B), bytes_of(new_lens, 4 * (int64_t)B), bytes_of(free_pages, 4 * (int64_t)free_size),
                     bytes_of(free_count, 4), bytes_of(cu_groups, P > 0 ? 4 * ((int64_t)P + 1) : 0), bytes_of(prefix_lens, 4 * (int64_t)P)};
  // every CTA reads all inputs, some after others have written
  for (int i = 0; i < 6; ++i) {
    if (meets(out[i], {in[0], in[1], in[2], in[3], in[4], in[5]})) return fail(IRS_ERR_VALUE, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (meets(out[i], {out[j]})) return fail(IRS_ERR_VALUE, "outputs overlap");
  }
  DeviceInfo* dev = nullptr;
  irs_status s = current_device(&dev);
  if (s != IRS_OK) return s;
  irs::PlanArgs a{};
  a.cache_lens = cache_lens; a.new_lens = new_lens;
  a.page_table = page_table; a.table_stride = table_stride;
  a.free_pages = free_pages; a.free_count = free_count;
  a.cu_groups = cu_groups; a.prefix_lens = prefix_lens;
  a.cu_new = cu_new; a.positions = positions; a.slots = slots;
  a.lens_out = lens_out; a.free_left = free_left;
  a.err = err_flag;
  a.B = B; a.P = P; a.max_pages = max_pages; a.page_size = page_size; a.free_size = free_size; a.tokens = tokens;
  return launch_status(irs::launch_plan(a, dev->num_sms, reinterpret_cast<cudaStream_t>(stream)), "launching the page plan");
}

}  // extern "C"

namespace {

// Checks shared by the two forms of shared-prefix attention; fills the arguments both need.
irs_status prefix_args(irs::PrefixArgs* a, const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
                       int64_t kc_stride_p, int64_t kc_stride_t, int64_t kc_stride_h, const void* v_cache,
                       int64_t vc_stride_p, int64_t vc_stride_t, int64_t vc_stride_h, const int32_t* page_table,
                       int64_t table_stride, int max_pages, int num_pages, int page_size, const int32_t* cu,
                       const int32_t* prefix_lens, int P, int T, int Hq, int Hkv, int Dqk, int Dv, float scale, void* out,
                       float* lse, void* workspace, size_t workspace_bytes, size_t need, bool decode, int32_t* err_flag) {
  if (T < 0 || P < 0 || Hq < 1 || Hkv < 1) return fail(IRS_ERR_VALUE, "bad sizes (T=%d P=%d Hq=%d Hkv=%d)", T, P, Hq, Hkv);
  if (Hq % Hkv != 0) return fail(IRS_ERR_VALUE, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (Hq / Hkv > 128) return fail(IRS_ERR_VALUE, "at most 128 query heads a KV head (got %d)", Hq / Hkv);
  if (Hkv > 1024) return fail(IRS_ERR_VALUE, "at most 1024 KV heads (got %d)", Hkv);
  if (Dqk != 64 && Dqk != 128 && Dqk != 192) return fail(IRS_ERR_VALUE, "Dqk must be 64, 128 or 192 (got %d)", Dqk);
  if (Dv != 64 && Dv != 128) return fail(IRS_ERR_VALUE, "Dv must be 64 or 128 (got %d)", Dv);
  if ((long long)T * Hq >= (1LL << 31)) return fail(IRS_ERR_VALUE, "T * Hq must be below 2^31");
  if (decode && (long long)T * Hq >= (1LL << 24)) return fail(IRS_ERR_VALUE, "B * Hq must be below 2^24");
  if (decode && (long long)Hkv * ((Hq / Hkv + 15) / 16) > 1024)
    return fail(IRS_ERR_VALUE, "at most 1024 KV heads times blocks of 16 query heads");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(IRS_ERR_VALUE, "scale must be positive and finite");
  if (T == 0) return IRS_OK;
  if (P < 1) return fail(IRS_ERR_VALUE, "at least one group is needed");
  irs_status s = check_pool(k_cache, v_cache, page_table, page_table, table_stride, max_pages, num_pages, page_size);
  if (s != IRS_OK) return s;
  if (!q || !out || !workspace || !cu || !prefix_lens) return fail(IRS_ERR_VALUE, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(out)) return fail(IRS_ERR_VALUE, "q and out must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(IRS_ERR_VALUE, "workspace must be 256-byte aligned");
  if (workspace_bytes < need) return fail(IRS_ERR_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
  one_entry(T, q_stride_t); one_entry(Hq, q_stride_h);
  one_entry(num_pages, kc_stride_p); one_entry(num_pages, vc_stride_p);
  one_entry(page_size, kc_stride_t); one_entry(page_size, vc_stride_t);
  one_entry(Hkv, kc_stride_h); one_entry(Hkv, vc_stride_h);
  if (bad_stride({q_stride_t, q_stride_h, kc_stride_p, kc_stride_t, kc_stride_h, vc_stride_p, vc_stride_t, vc_stride_h}))
    return fail(IRS_ERR_VALUE, "strides must be non-negative multiples of 8 elements (16 bytes)");
  if (meets(span_of(out, T, Hq, Dv), {span_of(q, T, q_stride_t, Hq, q_stride_h, Dqk)})) return fail(IRS_ERR_VALUE, "out overlaps q");
  a->q = bf(q); a->q_st = q_stride_t; a->q_sh = q_stride_h;
  a->k = bf(k_cache); a->k_sp = kc_stride_p; a->k_st = kc_stride_t; a->k_sh = kc_stride_h;
  a->v = bf(v_cache); a->v_sp = vc_stride_p; a->v_st = vc_stride_t; a->v_sh = vc_stride_h;
  a->page_table = page_table; a->table_stride = table_stride;
  a->cu = cu; a->prefix_lens = prefix_lens;
  a->out = bf(out); a->lse = lse;
  a->ws = static_cast<uint8_t*>(workspace);
  a->err = err_flag;
  a->T = T; a->P = P; a->Hq = Hq; a->Hkv = Hkv; a->G = Hq / Hkv; a->Dqk = Dqk; a->Dv = Dv;
  a->max_pages = max_pages; a->num_pages = num_pages; a->page_size = page_size;
  a->scale_log2 = scale * 1.4426950408889634f;
  return IRS_OK;
}

// CTAs read inputs while others write, and a call's kernels overlap: outputs and the workspace (`need` bytes of it) lie over
// neither inputs nor one another. A row of own_out or own_lse is read by those who write that row, so out and lse may be these.
irs_status prefix_apart(const irs::PrefixArgs& a, size_t need) {
  struct Named {
    const char* name;
    Span span;
  };
  auto pool = [&](const void* p, int64_t sp, int64_t st, int64_t sh, int row) {
    return bytes_of(p, 2 * ((a.num_pages - 1) * sp + (a.page_size - 1) * st + (a.Hkv - 1) * sh + row));
  };
  const int rows = a.cache_lens != nullptr ? a.T : a.P;   // of the page table
  const int64_t n = (int64_t)a.T * a.Hq;
  const Named in[] = {{"q", span_of(a.q, a.T, a.q_st, a.Hq, a.q_sh, a.Dqk)},
                      {"k_cache", pool(a.k, a.k_sp, a.k_st, a.k_sh, a.Dqk)},
                      {"v_cache", pool(a.v, a.v_sp, a.v_st, a.v_sh, a.Dv)},
                      {"page_table", bytes_of(a.page_table, 4 * ((rows - 1) * a.table_stride + a.max_pages))},
                      {"cu", bytes_of(a.cu, 4 * ((int64_t)a.P + 1))},
                      {"prefix_lens", bytes_of(a.prefix_lens, 4 * (int64_t)a.P)},
                      {"cache_lens", bytes_of(a.cache_lens, a.cache_lens != nullptr ? 4 * (int64_t)a.T : 0)},
                      {"own_out", bytes_of(a.own_out, a.own_out != nullptr ? 2 * n * a.Dv : 0)},
                      {"own_lse", bytes_of(a.own_lse, a.own_lse != nullptr ? 4 * n : 0)}};
  const Named out[] = {{"out", bytes_of(a.out, 2 * n * a.Dv)},
                       {"lse", bytes_of(a.lse, a.lse != nullptr ? 4 * n : 0)},
                       {"workspace", bytes_of(a.ws, (int64_t)need)}};
  for (int i = 0; i < 3; ++i) {
    for (int k = 0; k < 9; ++k) {
      const bool same = (i == 0 && k == 7 && a.out == a.own_out) || (i == 1 && k == 8 && a.lse == a.own_lse);
      if (!same && meets(out[i].span, {in[k].span})) return fail(IRS_ERR_VALUE, "%s overlaps %s", out[i].name, in[k].name);
    }
    for (int j = 0; j < i; ++j)
      if (meets(out[i].span, {out[j].span})) return fail(IRS_ERR_VALUE, "%s overlaps %s", out[i].name, out[j].name);
  }
  return IRS_OK;
}

// 4-D bf16 map of a pool [pages][heads][positions][D], boxes of 64 dims x `chunk` positions; false where
// a stride cannot be a map's.
irs_status make_pool_map(CUtensorMap* m, const void* base, int D, const irs::PrefixArgs& a, int64_t sp, int64_t st, int64_t sh,
                         int chunk, bool* made) {
  auto ok = [](int n, int64_t s) { return n == 1 || (s > 0 && s < (1LL << 38)); };
  *made = ok(a.num_pages, sp) && ok(a.page_size, st) && ok(a.Hkv, sh);
  if (!*made) return IRS_OK;
  auto fn = encode_fn();
  if (fn == nullptr) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  // the stride of a dim with one entry is never used, but has to be a valid one
  cuuint64_t strides[3] = {(cuuint64_t)(a.page_size > 1 ? st : D) * 2, (cuuint64_t)(a.Hkv > 1 ? sh : D) * 2,
                           (cuuint64_t)(a.num_pages > 1 ? sp : D) * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)chunk, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(IRS_ERR_RUNTIME, "cuTensorMapEncodeTiled (pool) failed (%d)", (int)r);
  return IRS_OK;
}

irs_status prefix_maps(irs::PrefixMaps* m, const irs::PrefixArgs& a) {
  *m = irs::PrefixMaps{};
  irs_status s;
  m->has_q = (a.T == 1 || (a.q_st > 0 && a.q_st < (1LL << 38))) && (a.Hq == 1 || (a.q_sh > 0 && a.q_sh < (1LL << 38)));
  if (m->has_q && (s = make_packed_map(&m->q, a.q, a.Dqk, a.Hq, a.T, a.q_sh, a.q_st, a.G, 128 / a.G)) != IRS_OK) return s;
  m->chunk = irs::prefix_chunk(a.Dqk, a.page_size);
  if (m->chunk > 0) {
    bool k = false, v = false;
    if ((s = make_pool_map(&m->k, a.k, a.Dqk, a, a.k_sp, a.k_st, a.k_sh, m->chunk, &k)) != IRS_OK) return s;
    if ((s = make_pool_map(&m->v, a.v, a.Dv, a, a.v_sp, a.v_st, a.v_sh, m->chunk, &v)) != IRS_OK) return s;
    if (!k || !v) m->chunk = 0;
  }
  return IRS_OK;
}

}  // namespace

extern "C" {

size_t irs_shared_prefix_gqa_attn_fwd_workspace_bytes(int T, int P, int Hq, int Hkv, int Dv) {
  if (T < 0 || P < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Dv < 64) return 0;
  return irs::prefix_workspace_bytes(T, P, Hq, Hkv, Dv, false);
}

irs_status irs_shared_prefix_gqa_attn_fwd(const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
                                          int64_t kc_stride_p, int64_t kc_stride_t, int64_t kc_stride_h,
                                          const void* v_cache, int64_t vc_stride_p, int64_t vc_stride_t,
                                          int64_t vc_stride_h, const int32_t* page_table, int64_t table_stride,
                                          int max_pages, int num_pages, int page_size, const int32_t* cu_rows,
                                          const int32_t* prefix_lens, int P, const void* own_out, const float* own_lse,
                                          int T, int Hq, int Hkv, int Dqk, int Dv, float scale, void* out, float* lse,
                                          void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                          irs_stream_t stream) {
  irs::PrefixArgs a{};
  const size_t need = irs_shared_prefix_gqa_attn_fwd_workspace_bytes(T, P, Hq, Hkv, Dv);
  irs_status s = prefix_args(&a, q, q_stride_t, q_stride_h, k_cache, kc_stride_p, kc_stride_t, kc_stride_h, v_cache,
                             vc_stride_p, vc_stride_t, vc_stride_h, page_table, table_stride, max_pages, num_pages, page_size,
                             cu_rows, prefix_lens, P, T, Hq, Hkv, Dqk, Dv, scale, out, lse, workspace, workspace_bytes, need,
                             false, err_flag);
  if (s != IRS_OK || T == 0) return s;
  if ((own_out == nullptr) != (own_lse == nullptr)) return fail(IRS_ERR_VALUE, "own_out and own_lse come together");
  if (!aligned16(own_out)) return fail(IRS_ERR_VALUE, "own_out must be 16-byte aligned");
  // a row of own_out is read by the thread that writes that row of out, and nothing else reads it
  if (own_out != nullptr && own_out != out && meets(span_of(out, T, Hq, Dv), {span_of(own_out, T, Hq, Dv)}))
    return fail(IRS_ERR_VALUE, "out overlaps own_out row by other row");
  if (own_lse != nullptr && lse != nullptr && own_lse != lse &&
      meets(bytes_of(lse, 4LL * T * Hq), {bytes_of(own_lse, 4LL * T * Hq)}))
    return fail(IRS_ERR_VALUE, "lse overlaps own_lse row by other row");
  a.own_out = static_cast<const __nv_bfloat16*>(own_out);
  a.own_lse = own_lse;
  if ((s = prefix_apart(a, need)) != IRS_OK) return s;
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  irs::PrefixMaps m;
  if ((s = prefix_maps(&m, a)) != IRS_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return launch_status(irs::launch_prefix_fwd(m, a, dev->num_sms, dev->prefix_configured, reinterpret_cast<cudaStream_t>(stream)),
                       "launching shared-prefix attention");
}

size_t irs_shared_prefix_gqa_attn_decode_workspace_bytes(int B, int P, int Hq, int Hkv, int Dv) {
  if (B < 0 || P < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Dv < 64) return 0;
  return irs::prefix_workspace_bytes(B, P, Hq, Hkv, Dv, true);
}

irs_status irs_shared_prefix_gqa_attn_decode(const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache,
                                             int64_t kc_stride_p, int64_t kc_stride_t, int64_t kc_stride_h,
                                             const void* v_cache, int64_t vc_stride_p, int64_t vc_stride_t,
                                             int64_t vc_stride_h, const int32_t* page_table, int64_t table_stride,
                                             int max_pages, int num_pages, int page_size, const int32_t* cache_lens,
                                             const int32_t* cu_groups, const int32_t* prefix_lens, int P, int B, int Hq,
                                             int Hkv, int Dqk, int Dv, float scale, void* out, float* lse, void* workspace,
                                             size_t workspace_bytes, int32_t* err_flag, irs_stream_t stream) {
  irs::PrefixArgs a{};
  const size_t need = irs_shared_prefix_gqa_attn_decode_workspace_bytes(B, P, Hq, Hkv, Dv);
  irs_status s = prefix_args(&a, q, q_stride_b, q_stride_h, k_cache, kc_stride_p, kc_stride_t, kc_stride_h, v_cache,
                             vc_stride_p, vc_stride_t, vc_stride_h, page_table, table_stride, max_pages, num_pages, page_size,
                             cu_groups, prefix_lens, P, B, Hq, Hkv, Dqk, Dv, scale, out, lse, workspace, workspace_bytes,
                             need, true, err_flag);
  if (s != IRS_OK || B == 0) return s;
  if (!cache_lens) return fail(IRS_ERR_VALUE, "NULL cache pointer");
  a.cache_lens = cache_lens;
  if ((s = prefix_apart(a, need)) != IRS_OK) return s;
  DeviceInfo* dev = nullptr;
  if ((s = current_device(&dev)) != IRS_OK) return s;
  irs::PrefixMaps m;
  if ((s = prefix_maps(&m, a)) != IRS_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  return launch_status(irs::launch_prefix_decode(m, a, dev->num_sms, dev->prefix_configured, dev->prefix_own_configured,
                                                 reinterpret_cast<cudaStream_t>(stream)),
                       "launching shared-prefix decoding");
}

}  // extern "C"

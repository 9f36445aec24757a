// Host side of the libhs C ABI: argument validation, kernel choice, the
// device status word and error reporting.  See include/hs.h for the contract
// of every entry point.

#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "hs.h"
#include "hs_internal.h"

namespace {

// Device-side status word: kernels record the first device-detected problem
// here (one copy per device that loads the library).
__device__ int g_device_status;

constexpr int kMaxDevices = 64;
int* g_status_ptr[kMaxDevices];
std::mutex g_status_mu;

std::atomic<int> g_force_simt{0};
std::atomic<long long> g_wait_limit{0};  // 0 = the kernels' default bound

thread_local char g_last_error[512];
// Kernel family of the calling thread's most recent successful compute call
// (hs_last_path), -1 before the first one.
thread_local int g_last_path = -1;

hs_status fail(hs_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

hs_status cuda_fail(cudaError_t e, const char* what) {
  return fail(HS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Address of the status word on the current device (looked up once per
// device with that device current).
hs_status status_ptr(int** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(HS_ERR_UNSUPPORTED, "device id %d", dev);
  std::lock_guard<std::mutex> lk(g_status_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_device_status);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  *out = g_status_ptr[dev];
  return HS_OK;
}

bool valid_block(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

int nbmax_of(int max_seqlen, int block_size) {
  return (max_seqlen + block_size - 1) / block_size;
}

constexpr int kMaxHeads = 128;
constexpr int kMaxDim = 1024;

// Checks shared by the calls that read q and k; fills p (status excluded).
hs_status check_problem(hs::Problem& p, const void* q, int64_t qrs, int64_t qhs, const void* k,
                        int64_t krs, const int32_t* cu, int num_docs, int total_tokens,
                        int max_seqlen, int num_heads, int dk, int dv, hs_dtype dtype,
                        float scale) {
  if (total_tokens < 0) return fail(HS_ERR_INVALID_ARG, "total_tokens < 0");
  if (num_docs < 0) return fail(HS_ERR_INVALID_ARG, "num_docs < 0");
  if (total_tokens > 0 && num_docs < 1)
    return fail(HS_ERR_INVALID_ARG, "num_docs must be >= 1 when total_tokens > 0");
  if (total_tokens > 0 && max_seqlen < 1)
    return fail(HS_ERR_INVALID_ARG, "max_seqlen must be >= 1");
  if (!cu) return fail(HS_ERR_INVALID_ARG, "cu_seqlens is NULL");
  if (!q || !k) return fail(HS_ERR_INVALID_ARG, "q or k is NULL");
  if (dtype != HS_F32 && dtype != HS_BF16) return fail(HS_ERR_UNSUPPORTED, "dtype %d", (int)dtype);
  if (num_heads < 1 || num_heads > kMaxHeads)
    return fail(HS_ERR_UNSUPPORTED, "num_heads %d not in [1, %d]", num_heads, kMaxHeads);
  if (dk < 1 || dk > kMaxDim) return fail(HS_ERR_UNSUPPORTED, "dk %d not in [1, %d]", dk, kMaxDim);
  if (dv < 0 || dv > kMaxDim) return fail(HS_ERR_UNSUPPORTED, "dv %d not in [1, %d]", dv, kMaxDim);
  if (qhs < dk) return fail(HS_ERR_INVALID_ARG, "q_head_stride %lld < dk", (long long)qhs);
  if (qrs < (int64_t)num_heads * qhs)
    return fail(HS_ERR_INVALID_ARG, "q_row_stride %lld < num_heads * q_head_stride", (long long)qrs);
  if (krs < dk) return fail(HS_ERR_INVALID_ARG, "k_row_stride %lld < dk", (long long)krs);
  if (!(isfinite(scale))) return fail(HS_ERR_INVALID_ARG, "softmax_scale is not finite");
  p.q = q;
  p.q_row_stride = qrs;
  p.q_head_stride = qhs;
  p.k = k;
  p.k_row_stride = krs;
  p.v = nullptr;
  p.v_row_stride = 0;
  p.cu_seqlens = cu;
  p.num_docs = num_docs;
  p.total_tokens = total_tokens;
  p.max_seqlen = max_seqlen;
  p.num_heads = num_heads;
  p.dk = dk;
  p.dv = dv;
  p.dtype = dtype;
  p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)dk);
  p.status = nullptr;
  return HS_OK;
}

// The backward's workspace: the delta / sink terms of every path, then (for
// shapes the tensor-core passes take) the dk / dv pass's partial sums at a
// 256-byte boundary.
size_t bwd_simt_bytes(int total_tokens, int num_heads, bool with_first) {
  const size_t flags = with_first ? 2 * sizeof(int) * (size_t)total_tokens : 0;
  return (hs::simt_backward_workspace(total_tokens, num_heads) + flags + 255) & ~(size_t)255;
}
// span > 0: the window attention with first tokens, window + first keys.
size_t bwd_workspace(int total_tokens, int num_heads, int dk, int dv, hs_dtype dtype,
                     int num_docs = 0, int max_seqlen = 0, int span = 0) {
  size_t need = bwd_simt_bytes(total_tokens, num_heads, span > 0);
  if (!g_force_simt.load() && hs::tc_backward_shape_ok(dtype, num_heads, dk, dv)) {
    size_t tc = hs::tc_bwd_dkdv_workspace(total_tokens, dk, dv);
    if (span > 0)
      tc = std::max(tc, hs::tc_first_bwd_workspace(total_tokens, num_docs, max_seqlen, span, dk, dv));
    need += tc;
  }
  return need;
}

hs_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return cuda_fail(e, what);
  return HS_OK;
}

// launched(), and on success records `path` as the call's kernel family.
hs_status launched_on(cudaError_t e, const char* what, int path) {
  hs_status r = launched(e, what);
  if (r == HS_OK) g_last_path = path;
  return r;
}

}  // namespace

namespace hs {
// Lets other translation units of the library report a host-side failure
// through hs_last_error().
hs_status report_error(hs_status st, const char* msg) { return fail(st, "%s", msg); }

// Host checks of hs_block_score's arguments, without any device work.
hs_status check_score_args(const void* q, int64_t qrs, int64_t qhs, const void* k, int64_t krs,
                           const int32_t* cu, int num_docs, int total_tokens, int max_seqlen,
                           int num_heads, int dk, hs_dtype dtype, float scale, int block_size,
                           const float* lse, const float* block_score, int nb_stride) {
  Problem p{};
  hs_status r = check_problem(p, q, qrs, qhs, k, krs, cu, num_docs, total_tokens, max_seqlen,
                              num_heads, dk, 0, dtype, scale);
  if (r != HS_OK) return r;
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (!lse || !block_score) return fail(HS_ERR_INVALID_ARG, "lse or block_score is NULL");
  if (total_tokens > 0 && nb_stride < nbmax_of(max_seqlen, block_size))
    return fail(HS_ERR_INVALID_ARG, "nb_stride %d < ceil(max_seqlen / block_size) = %d", nb_stride,
                nbmax_of(max_seqlen, block_size));
  return HS_OK;
}
}  // namespace hs

extern "C" {

int hs_version(void) { return 400; }

const char* hs_status_string(hs_status s) {
  switch (s) {
    case HS_OK: return "HS_OK";
    case HS_ERR_INVALID_ARG: return "HS_ERR_INVALID_ARG";
    case HS_ERR_UNSUPPORTED: return "HS_ERR_UNSUPPORTED";
    case HS_ERR_CUDA: return "HS_ERR_CUDA";
    case HS_ERR_INVALID_INDEX: return "HS_ERR_INVALID_INDEX";
    case HS_ERR_TIMEOUT: return "HS_ERR_TIMEOUT";
    case HS_ERR_WORKSPACE: return "HS_ERR_WORKSPACE";
  }
  return "HS_ERR_UNKNOWN";
}

const char* hs_last_error(void) { return g_last_error; }

int hs_last_path(void) { return g_last_path; }

void hs_set_force_simt(int on) { g_force_simt.store(on ? 1 : 0); }

hs_status hs_selftest_wait(long long limit_ns, hs_stream_t stream) {
  if (limit_ns < 1 || limit_ns > 1000000000ll)
    return fail(HS_ERR_INVALID_ARG, "limit_ns %lld not in [1, 1e9]", limit_ns);
  int* st = nullptr;
  hs_status r = status_ptr(&st);
  if (r != HS_OK) return r;
  return launched(hs::launch_selftest_wait(limit_ns, st, stream), "self-test wait");
}

int hs_path(int op, hs_dtype dtype, int num_heads, int dk, int dv, int block_size) {
  if (dtype != HS_F32 && dtype != HS_BF16) return -1;
  switch (op) {
    case HS_OP_SELECT_TOPK: return HS_PATH_SIMT;
    case HS_OP_BLOCK_SCORE:
      if (dtype == HS_BF16 && !g_force_simt.load() &&
          hs::tc_block_score_supported(num_heads, dk, block_size, 0))
        return HS_PATH_TCGEN05;
      return HS_PATH_SIMT;
    case HS_OP_SWA_FIRST_MQA:
      return !g_force_simt.load() && hs::tc_first_shape_ok(dtype, num_heads, dk, dv)
                 ? HS_PATH_TCGEN05
                 : HS_PATH_SIMT;
    case HS_OP_KV4_MQA_DECODE:
      return !g_force_simt.load() && hs::tc_kv4_decode_shape_ok(num_heads, dk, dv, dtype)
                 ? HS_PATH_TCGEN05
                 : HS_PATH_SIMT;
    case HS_OP_SPARSE_MQA_BWD:
    case HS_OP_SWA_MQA_BWD:
    case HS_OP_SWA_FIRST_MQA_BWD:
      if (!g_force_simt.load() && hs::tc_backward_shape_ok(dtype, num_heads, dk, dv))
        return HS_PATH_MMA;
      return HS_PATH_SIMT;
    case HS_OP_SPARSE_MQA:
    case HS_OP_SWA_MQA:
    case HS_OP_BLOCK_SCORE_ATTN:  // fused, or the attention then the score kernel
    case HS_OP_SWA_LAYER:         // the sparse branch, then the window branch combining
      if (dtype == HS_BF16 && !g_force_simt.load() &&
          hs::tc_attention_supported(num_heads, dk, dv, block_size, op == HS_OP_SPARSE_MQA))
        return HS_PATH_TCGEN05;
      return HS_PATH_SIMT;
  }
  return -1;
}

size_t hs_workspace_size(int op, int total_tokens, int num_docs, int max_seqlen, int num_heads,
                         int dk, int dv, hs_dtype dtype, int block_size) {
  if (op == HS_OP_KV4_MQA_DECODE) {  // total_tokens = the number of sequences
    if (total_tokens <= 0 || num_heads <= 0 || dv <= 0) return 0;
    size_t need = hs::simt_kv4_decode_workspace(total_tokens, num_heads, max_seqlen, dv);
    if (!g_force_simt.load() && hs::tc_kv4_decode_shape_ok(num_heads, dk, dv, dtype))
      need = std::max(need, hs::tc_kv4_decode_workspace(total_tokens, num_heads, dv));
    return need;
  }
  if ((op == HS_OP_SPARSE_MQA_BWD || op == HS_OP_SWA_MQA_BWD || op == HS_OP_SWA_FIRST_MQA_BWD) &&
      total_tokens > 0 && num_heads > 0)
    return op == HS_OP_SWA_FIRST_MQA_BWD
               ? bwd_workspace(total_tokens, num_heads, dk, dv, dtype, std::max(num_docs, 1),
                               std::max(max_seqlen, 1), std::max(block_size, 1))
               : bwd_workspace(total_tokens, num_heads, dk, dv, dtype);
  if ((op != HS_OP_BLOCK_SCORE && op != HS_OP_BLOCK_SCORE_ATTN) || total_tokens <= 0 ||
      !valid_block(block_size))
    return 0;
  const int nbmax = nbmax_of(max_seqlen, block_size);
  size_t need = 0;
  if (dtype == HS_BF16 && !g_force_simt.load() &&
      hs::tc_block_score_supported(num_heads, dk, block_size, nbmax))
    need = hs::tc_block_score_workspace(total_tokens, num_docs, num_heads, nbmax);
  // the fused kernel's scratch (the call falls back to the score kernel when
  // pointer alignment rules the fused one out, so cover both)
  if (op == HS_OP_BLOCK_SCORE_ATTN && dtype == HS_BF16 && !g_force_simt.load() &&
      hs::tc_full_supported(num_heads, dk, dv, block_size)) {
    const size_t f = hs::tc_full_workspace(total_tokens, nbmax);
    if (f > need) need = f;
  }
  return need;
}

hs_status hs_poll_status(hs_stream_t stream) {
  int* st = nullptr;
  hs_status r = status_ptr(&st);
  if (r != HS_OK) return r;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int host = 0;
  e = cudaMemcpyFromSymbol(&host, g_device_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "read status");
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "clear status");
  if (host != 0)
    return fail((hs_status)host, "device reported %s", hs_status_string((hs_status)host));
  return HS_OK;
}

hs_status hs_block_score(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* k, int64_t k_row_stride, const int32_t* cu_seqlens,
                         int num_docs, int total_tokens, int max_seqlen, int num_heads, int dk,
                         hs_dtype dtype, float softmax_scale, int block_size, float* lse,
                         float* block_score, int nb_stride, float* block_lse, void* workspace,
                         size_t workspace_bytes, hs_stream_t stream) {
  hs::ScoreArgs a{};
  hs_status r = check_problem(a.p, q, q_row_stride, q_head_stride, k, k_row_stride, cu_seqlens,
                              num_docs, total_tokens, max_seqlen, num_heads, dk, 0, dtype,
                              softmax_scale);
  if (r != HS_OK) return r;
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (!lse || !block_score) return fail(HS_ERR_INVALID_ARG, "lse or block_score is NULL");
  if (total_tokens == 0) return HS_OK;
  const int nbmax = nbmax_of(max_seqlen, block_size);
  if (nb_stride < nbmax)
    return fail(HS_ERR_INVALID_ARG, "nb_stride %d < ceil(max_seqlen / block_size) = %d", nb_stride,
                nbmax);
  a.block_size = block_size;
  a.nbmax = nbmax;
  a.nb_stride = nb_stride;
  a.lse = lse;
  a.block_score = block_score;
  a.block_lse = block_lse;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  r = status_ptr(&a.p.status);
  if (r != HS_OK) return r;
  const bool tc = dtype == HS_BF16 && !g_force_simt.load() &&
                  hs::tc_block_score_supported(num_heads, dk, block_size, nbmax) &&
                  hs::tc_block_score_eligible(a);
  if (tc) {
    const size_t need = hs::tc_block_score_workspace(total_tokens, num_docs, num_heads, nbmax);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(HS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                  workspace ? workspace_bytes : (size_t)0);
    return launched_on(hs::launch_tc_block_score(a, g_wait_limit.load(), stream),
                       "tc block score", HS_PATH_TCGEN05);
  }
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (hs::simt_block_score_smem(num_heads, dk, nbmax) > (size_t)optin)
    return fail(HS_ERR_UNSUPPORTED, "num_heads * dk + blocks too large for the CUDA-core kernel");
  return launched_on(hs::launch_simt_block_score(a, stream), "simt block score", HS_PATH_SIMT);
}

hs_status hs_select_topk(const float* block_score, int nb_stride, const int32_t* cu_seqlens,
                         int num_docs, int total_tokens, int max_seqlen, int block_size, int topk,
                         int32_t* idx, hs_stream_t stream) {
  if (total_tokens < 0 || num_docs < 0) return fail(HS_ERR_INVALID_ARG, "negative size");
  if (total_tokens > 0 && (num_docs < 1 || max_seqlen < 1))
    return fail(HS_ERR_INVALID_ARG, "num_docs and max_seqlen must be >= 1");
  if (!block_score || !cu_seqlens || !idx) return fail(HS_ERR_INVALID_ARG, "NULL pointer");
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (topk < 1 || topk > 256) return fail(HS_ERR_UNSUPPORTED, "topk %d not in [1, 256]", topk);
  if (total_tokens == 0) return HS_OK;
  const int nbmax = nbmax_of(max_seqlen, block_size);
  if (nb_stride < nbmax)
    return fail(HS_ERR_INVALID_ARG, "nb_stride %d < ceil(max_seqlen / block_size) = %d", nb_stride,
                nbmax);
  if (nbmax > hs::kMaxSelectBlocks)
    return fail(HS_ERR_UNSUPPORTED, "ceil(max_seqlen / block_size) = %d blocks > %d", nbmax,
                hs::kMaxSelectBlocks);
  int* st = nullptr;
  hs_status r = status_ptr(&st);
  if (r != HS_OK) return r;
  return launched_on(hs::launch_select_topk(block_score, nb_stride, cu_seqlens, num_docs,
                                            total_tokens, max_seqlen, block_size, topk, idx, st,
                                            stream),
                     "select topk", HS_PATH_SIMT);
}

static hs_status attention_common(hs::AttnArgs& a, bool sparse, const void* q, int64_t qrs,
                                  int64_t qhs, const void* k, int64_t krs, const void* v,
                                  int64_t vrs, const int32_t* cu, int num_docs, int total_tokens,
                                  int max_seqlen, int num_heads, int dk, int dv, hs_dtype dtype,
                                  float scale, const float* sink, void* out, float* lse,
                                  hs_stream_t stream) {
  hs_status r = check_problem(a.p, q, qrs, qhs, k, krs, cu, num_docs, total_tokens, max_seqlen,
                              num_heads, dk, dv, dtype, scale);
  if (r != HS_OK) return r;
  if (dv < 1) return fail(HS_ERR_UNSUPPORTED, "dv must be >= 1");
  if (!v) return fail(HS_ERR_INVALID_ARG, "v is NULL");
  if (vrs < dv) return fail(HS_ERR_INVALID_ARG, "v_row_stride %lld < dv", (long long)vrs);
  if (!out || !lse) return fail(HS_ERR_INVALID_ARG, "out or lse is NULL");
  a.p.v = v;
  a.p.v_row_stride = vrs;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  if (total_tokens == 0) return HS_OK;
  r = status_ptr(&a.p.status);
  if (r != HS_OK) return r;
  if (a.with_first) {
    if (!g_force_simt.load() && hs::tc_first_eligible(a.p) &&
        (reinterpret_cast<uintptr_t>(out) & 15) == 0)
      return launched_on(hs::launch_tc_first_fwd(a, g_wait_limit.load(), stream),
                         "tc window attention with first tokens", HS_PATH_TCGEN05);
    return launched_on(hs::launch_simt_attention(a, false, stream),
                       "simt window attention with first tokens", HS_PATH_SIMT);
  }
  const bool tc = dtype == HS_BF16 && !g_force_simt.load() &&
                  hs::tc_attention_supported(num_heads, dk, dv, a.block_size, sparse) &&
                  hs::tc_attention_eligible(a);
  if (tc) return launched_on(hs::launch_tc_attention(a, sparse, g_wait_limit.load(), stream),
                             sparse ? "tc sparse attention" : "tc swa attention",
                             HS_PATH_TCGEN05);
  return launched_on(hs::launch_simt_attention(a, sparse, stream),
                     sparse ? "simt sparse attention" : "simt swa attention", HS_PATH_SIMT);
}

hs_status hs_sparse_mqa_fwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* k, int64_t k_row_stride, const void* v,
                            int64_t v_row_stride, const int32_t* cu_seqlens, int num_docs,
                            int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                            hs_dtype dtype, float softmax_scale, const int32_t* idx, int topk,
                            int block_size, const float* sink, void* out, float* lse,
                            hs_stream_t stream) {
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (topk < 1 || topk > 256) return fail(HS_ERR_UNSUPPORTED, "topk %d not in [1, 256]", topk);
  if (!idx) return fail(HS_ERR_INVALID_ARG, "idx is NULL");
  hs::AttnArgs a{};
  a.idx = idx;
  a.topk = topk;
  a.block_size = block_size;
  a.window = 0;
  return attention_common(a, true, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                          v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen,
                          num_heads, dk, dv, dtype, softmax_scale, sink, out, lse, stream);
}

hs_status hs_swa_mqa_fwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                         const int32_t* cu_seqlens, int num_docs, int total_tokens,
                         int max_seqlen, int num_heads, int dk, int dv, hs_dtype dtype,
                         float softmax_scale, int window, const float* sink, void* out,
                         float* lse, hs_stream_t stream) {
  if (window < 1) return fail(HS_ERR_INVALID_ARG, "window %d < 1", window);
  hs::AttnArgs a{};
  a.idx = nullptr;
  a.topk = 0;
  a.block_size = 64;  // block size plays no part in the window; any valid value
  a.window = window;
  return attention_common(a, false, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                          v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen,
                          num_heads, dk, dv, dtype, softmax_scale, sink, out, lse, stream);
}

hs_status hs_block_score_attn_fwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                  const void* k, int64_t k_row_stride, const void* v,
                                  int64_t v_row_stride, const int32_t* cu_seqlens, int num_docs,
                                  int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                                  hs_dtype dtype, float softmax_scale, int block_size, void* out,
                                  float* lse, float* block_score, int nb_stride, float* block_lse,
                                  void* workspace, size_t workspace_bytes, hs_stream_t stream) {
  hs::FullArgs f{};
  hs_status r = check_problem(f.p, q, q_row_stride, q_head_stride, k, k_row_stride, cu_seqlens,
                              num_docs, total_tokens, max_seqlen, num_heads, dk, dv, dtype,
                              softmax_scale);
  if (r != HS_OK) return r;
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (dv < 1) return fail(HS_ERR_UNSUPPORTED, "dv must be >= 1");
  if (!v) return fail(HS_ERR_INVALID_ARG, "v is NULL");
  if (v_row_stride < dv) return fail(HS_ERR_INVALID_ARG, "v_row_stride %lld < dv",
                                     (long long)v_row_stride);
  if (!out || !lse || !block_score) return fail(HS_ERR_INVALID_ARG, "out, lse or block_score is NULL");
  if (total_tokens == 0) return HS_OK;
  const int nbmax = nbmax_of(max_seqlen, block_size);
  if (nb_stride < nbmax)
    return fail(HS_ERR_INVALID_ARG, "nb_stride %d < ceil(max_seqlen / block_size) = %d", nb_stride,
                nbmax);
  f.p.v = v;
  f.p.v_row_stride = v_row_stride;
  f.block_size = block_size;
  f.nbmax = nbmax;
  f.nb_stride = nb_stride;
  f.out = out;
  f.lse = lse;
  f.block_score = block_score;
  f.block_lse = block_lse;
  f.workspace = workspace;
  r = status_ptr(&f.p.status);
  if (r != HS_OK) return r;
  hs::AttnArgs a{};  // the attention part, for the eligibility test and the two-kernel path
  a.p = f.p;
  a.block_size = block_size;
  a.window = max_seqlen;  // covers every document: dense causal
  a.sink = nullptr;
  a.out = out;
  a.lse = lse;
  const bool fused = dtype == HS_BF16 && !g_force_simt.load() &&
                     hs::tc_full_supported(num_heads, dk, dv, block_size) &&
                     hs::tc_attention_eligible(a);
  if (fused) {
    const size_t need = hs::tc_full_workspace(total_tokens, nbmax);
    if (!workspace || workspace_bytes < need)
      return fail(HS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                  workspace ? workspace_bytes : (size_t)0);
    return launched_on(hs::launch_tc_full(f, g_wait_limit.load(), stream), "tc full layer",
                       HS_PATH_TCGEN05);
  }
  // two kernels: the attention (its lse is the same quantity; the score
  // kernel then writes lse again), then step 1
  const bool tca = dtype == HS_BF16 && !g_force_simt.load() &&
                   hs::tc_attention_supported(num_heads, dk, dv, block_size, false) &&
                   hs::tc_attention_eligible(a);
  r = launched(tca ? hs::launch_tc_attention(a, false, g_wait_limit.load(), stream)
                   : hs::launch_simt_attention(a, false, stream),
               "full layer attention");
  if (r != HS_OK) return r;
  r = hs_block_score(q, q_row_stride, q_head_stride, k, k_row_stride, cu_seqlens, num_docs,
                     total_tokens, max_seqlen, num_heads, dk, dtype, softmax_scale, block_size,
                     lse, block_score, nb_stride, block_lse, workspace, workspace_bytes, stream);
  if (r == HS_OK && !tca) g_last_path = HS_PATH_SIMT;  // the attention ran on CUDA cores
  return r;
}

hs_status hs_swa_layer_fwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                           const void* k, int64_t k_row_stride, const void* v,
                           int64_t v_row_stride, const void* k_shared,
                           int64_t k_shared_row_stride, const void* v_shared,
                           int64_t v_shared_row_stride, const int32_t* cu_seqlens, int num_docs,
                           int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                           hs_dtype dtype, float softmax_scale, int window, const float* sink_swa,
                           const int32_t* idx, int topk, int block_size,
                           const float* sink_sparse, const float* gate_swa,
                           const float* gate_sparse, void* out, float* lse_swa,
                           float* lse_sparse, hs_stream_t stream) {
  if (window < 1) return fail(HS_ERR_INVALID_ARG, "window %d < 1", window);
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (topk < 1 || topk > 256) return fail(HS_ERR_UNSUPPORTED, "topk %d not in [1, 256]", topk);
  if (!idx) return fail(HS_ERR_INVALID_ARG, "idx is NULL");
  if (!k_shared || !v_shared) return fail(HS_ERR_INVALID_ARG, "k_shared or v_shared is NULL");
  if (k_shared_row_stride < dk)
    return fail(HS_ERR_INVALID_ARG, "k_shared_row_stride %lld < dk", (long long)k_shared_row_stride);
  if (v_shared_row_stride < dv)
    return fail(HS_ERR_INVALID_ARG, "v_shared_row_stride %lld < dv", (long long)v_shared_row_stride);
  if (!lse_sparse || !lse_swa) return fail(HS_ERR_INVALID_ARG, "lse_swa or lse_sparse is NULL");
  // the window branch's own arguments, checked before the first launch
  if (!k || !v) return fail(HS_ERR_INVALID_ARG, "k or v is NULL");
  if (k_row_stride < dk) return fail(HS_ERR_INVALID_ARG, "k_row_stride %lld < dk",
                                     (long long)k_row_stride);
  if (v_row_stride < dv) return fail(HS_ERR_INVALID_ARG, "v_row_stride %lld < dv",
                                     (long long)v_row_stride);
  // the sparse branch over the shared KV, written to out
  hs::AttnArgs sp{};
  sp.idx = idx;
  sp.topk = topk;
  sp.block_size = block_size;
  sp.window = 0;
  hs_status r = attention_common(sp, true, q, q_row_stride, q_head_stride, k_shared,
                                 k_shared_row_stride, v_shared, v_shared_row_stride, cu_seqlens,
                                 num_docs, total_tokens, max_seqlen, num_heads, dk, dv, dtype,
                                 softmax_scale, sink_sparse, out, lse_sparse, stream);
  if (r != HS_OK) return r;
  const int sparse_path = g_last_path;
  // the window branch, whose epilogue adds the gated sparse result from out
  hs::AttnArgs w{};
  w.idx = nullptr;
  w.topk = 0;
  w.block_size = 64;
  w.window = window;
  w.prev = out;
  w.gate_own = gate_swa;
  w.gate_prev = gate_sparse;
  r = attention_common(w, false, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                       v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen, num_heads,
                       dk, dv, dtype, softmax_scale, sink_swa, out, lse_swa, stream);
  if (r == HS_OK && sparse_path == HS_PATH_SIMT) g_last_path = HS_PATH_SIMT;
  return r;
}

static hs_status backward_common(hs::BwdArgs& a, bool sparse, const void* q, int64_t qrs,
                                 int64_t qhs, const void* k, int64_t krs, const void* v,
                                 int64_t vrs, const int32_t* cu, int num_docs, int total_tokens,
                                 int max_seqlen, int num_heads, int dk, int dv, hs_dtype dtype,
                                 float scale, const float* sink, const void* out,
                                 const float* lse, const void* dout, void* dq, void* dkey,
                                 void* dval, float* dsink, void* workspace,
                                 size_t workspace_bytes, hs_stream_t stream) {
  hs_status r = check_problem(a.p, q, qrs, qhs, k, krs, cu, num_docs, total_tokens, max_seqlen,
                              num_heads, dk, dv, dtype, scale);
  if (r != HS_OK) return r;
  if (dv < 1) return fail(HS_ERR_UNSUPPORTED, "dv must be >= 1");
  if (!v) return fail(HS_ERR_INVALID_ARG, "v is NULL");
  if (vrs < dv) return fail(HS_ERR_INVALID_ARG, "v_row_stride %lld < dv", (long long)vrs);
  if (!out || !lse || !dout) return fail(HS_ERR_INVALID_ARG, "out, lse or dout is NULL");
  if (!dq || !dkey || !dval) return fail(HS_ERR_INVALID_ARG, "dq, dk or dv is NULL");
  a.p.v = v;
  a.p.v_row_stride = vrs;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  a.dout = dout;
  a.dq = dq;
  a.dkey = dkey;
  a.dval = dval;
  a.dsink = dsink;
  if (total_tokens == 0) return HS_OK;
  int span = 0;  // of keys, none of them past a document
  if (a.with_first) {
    const int most = std::min(max_seqlen, total_tokens);
    span = std::min(a.window, most) + std::min(a.first, most);
  }
  const size_t need = bwd_workspace(total_tokens, num_heads, dk, dv, dtype, num_docs, max_seqlen, span);
  if (!workspace || workspace_bytes < need)
    return fail(HS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if ((reinterpret_cast<uintptr_t>(workspace) & 15) != 0)
    return fail(HS_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  a.workspace = workspace;
  const size_t own = bwd_simt_bytes(total_tokens, num_heads, a.with_first);
  a.dkdv_ws = need > own ? static_cast<char*>(workspace) + own : nullptr;
  a.dkdv_bytes = need - own;
  r = status_ptr(&a.p.status);
  if (r != HS_OK) return r;
  int path = HS_PATH_SIMT;
  const cudaError_t e = hs::launch_simt_backward(a, sparse, !g_force_simt.load(), &path, stream);
  return launched_on(e, sparse ? "sparse attention backward" : "swa attention backward", path);
}

hs_status hs_sparse_mqa_bwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* k, int64_t k_row_stride, const void* v,
                            int64_t v_row_stride, const int32_t* cu_seqlens, int num_docs,
                            int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                            hs_dtype dtype, float softmax_scale, const int32_t* idx, int topk,
                            int block_size, const float* sink, const void* out, const float* lse,
                            const void* dout, float* dq, float* dkey, float* dval, float* dsink,
                            void* workspace, size_t workspace_bytes, hs_stream_t stream) {
  if (!valid_block(block_size))
    return fail(HS_ERR_UNSUPPORTED, "block_size %d not in {16, 32, 64, 128}", block_size);
  if (topk < 1 || topk > 256) return fail(HS_ERR_UNSUPPORTED, "topk %d not in [1, 256]", topk);
  if (!idx) return fail(HS_ERR_INVALID_ARG, "idx is NULL");
  hs::BwdArgs a{};
  a.idx = idx;
  a.topk = topk;
  a.block_size = block_size;
  a.window = 0;
  return backward_common(a, true, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                         v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen, num_heads,
                         dk, dv, dtype, softmax_scale, sink, out, lse, dout, dq, dkey, dval,
                         dsink, workspace, workspace_bytes, stream);
}

hs_status hs_swa_mqa_bwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                         const int32_t* cu_seqlens, int num_docs, int total_tokens,
                         int max_seqlen, int num_heads, int dk, int dv, hs_dtype dtype,
                         float softmax_scale, int window, const float* sink, const void* out,
                         const float* lse, const void* dout, float* dq, float* dkey, float* dval,
                         float* dsink, void* workspace, size_t workspace_bytes,
                         hs_stream_t stream) {
  if (window < 1) return fail(HS_ERR_INVALID_ARG, "window %d < 1", window);
  hs::BwdArgs a{};
  a.idx = nullptr;
  a.topk = 0;
  a.block_size = 64;
  a.window = window;
  return backward_common(a, false, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                         v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen, num_heads,
                         dk, dv, dtype, softmax_scale, sink, out, lse, dout, dq, dkey, dval,
                         dsink, workspace, workspace_bytes, stream);
}

// Window and first tokens beyond every document change nothing; clamped so
// that sums of token indices stay far from the 32-bit limit.
static hs_status check_window_first(int& window, int& num_first, int total_tokens) {
  if (window < 1) return fail(HS_ERR_INVALID_ARG, "window %d < 1", window);
  if (num_first < 0) return fail(HS_ERR_INVALID_ARG, "num_first %d < 0", num_first);
  const int most = total_tokens > 1 ? total_tokens : 1;
  if (window > most) window = most;
  if (num_first > most) num_first = most;
  return HS_OK;
}

hs_status hs_swa_first_mqa_fwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                               const void* k, int64_t k_row_stride, const void* v,
                               int64_t v_row_stride, const int32_t* cu_seqlens, int num_docs,
                               int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                               hs_dtype dtype, float softmax_scale, int window, int num_first,
                               const float* sink, void* out, float* lse, hs_stream_t stream) {
  hs_status r = check_window_first(window, num_first, total_tokens);
  if (r != HS_OK) return r;
  hs::AttnArgs a{};
  a.block_size = 64;  // plays no part
  a.window = window;
  a.first = num_first;
  a.with_first = true;
  return attention_common(a, false, q, q_row_stride, q_head_stride, k, k_row_stride, v,
                          v_row_stride, cu_seqlens, num_docs, total_tokens, max_seqlen,
                          num_heads, dk, dv, dtype, softmax_scale, sink, out, lse, stream);
}

hs_status hs_swa_first_mqa_bwd(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                               const void* k, int64_t k_row_stride, const void* v,
                               int64_t v_row_stride, const int32_t* cu_seqlens, int num_docs,
                               int total_tokens, int max_seqlen, int num_heads, int dk, int dv,
                               hs_dtype dtype, float softmax_scale, int window, int num_first,
                               const float* sink, const void* out, const float* lse,
                               const void* dout, void* dq, void* dkey, void* dval, float* dsink,
                               void* workspace, size_t workspace_bytes, hs_stream_t stream) {
  hs_status r = check_window_first(window, num_first, total_tokens);
  if (r != HS_OK) return r;
  hs::BwdArgs a{};
  a.block_size = 64;
  a.window = window;
  a.first = num_first;
  a.with_first = true;
  a.grad_like_input = true;
  r = backward_common(a, false, q, q_row_stride, q_head_stride, k, k_row_stride, v, v_row_stride,
                      cu_seqlens, num_docs, total_tokens, max_seqlen, num_heads, dk, dv, dtype,
                      softmax_scale, sink, out, lse, dout, dq, dkey, dval, dsink, workspace,
                      workspace_bytes, stream);
  // no tokens: the sink's gradient is the one output that still has elements
  if (r == HS_OK && total_tokens == 0 && sink && dsink) {
    const cudaError_t e = cudaMemsetAsync(dsink, 0, sizeof(float) * num_heads, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  }
  return r;
}

// ------------------------------------------------------------ 4-bit cache

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static int log2_of(int v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

// Checks of the page geometry shared by the cache calls.
static hs_status check_pages(const int32_t* block_table, int64_t table_stride, int table_width,
                             int num_pages, int page_size, int num_seqs) {
  if (!valid_block(page_size))
    return fail(HS_ERR_UNSUPPORTED, "page_size %d not in {16, 32, 64, 128}", page_size);
  if (num_pages < 0 || num_seqs < 0) return fail(HS_ERR_INVALID_ARG, "negative size");
  if (!block_table) return fail(HS_ERR_INVALID_ARG, "block_table is NULL");
  if (table_width < 1) return fail(HS_ERR_INVALID_ARG, "table_width %d < 1", table_width);
  if (table_stride < table_width)
    return fail(HS_ERR_INVALID_ARG, "table_stride %lld < table_width", (long long)table_stride);
  return HS_OK;
}

static hs_status check_width(const char* name, int width) {
  if (width < 32 || width > kMaxDim || width % 32 != 0)
    return fail(HS_ERR_UNSUPPORTED, "%s %d is not a multiple of 32 in [32, %d]", name, width,
                kMaxDim);
  return HS_OK;
}

static hs_status check_dtype(hs_dtype dtype) {
  if (dtype != HS_F32 && dtype != HS_BF16) return fail(HS_ERR_UNSUPPORTED, "dtype %d", (int)dtype);
  return HS_OK;
}

size_t hs_kv4_page_bytes(int width, int page_size) {
  if (width < 32 || width > kMaxDim || width % 32 != 0 || !valid_block(page_size)) return 0;
  const int g = width / 32;
  return (size_t)page_size * (16 * g + 4 * ((g + 3) / 4));
}

static hs_status check_rows(hs::Kv4Rows& a, const int32_t* block_table, int64_t table_stride,
                            int table_width, int num_pages, int page_size,
                            const int32_t* cu_seqlens, const int32_t* seq_lens, int num_seqs,
                            int total_tokens) {
  hs_status r =
      check_pages(block_table, table_stride, table_width, num_pages, page_size, num_seqs);
  if (r != HS_OK) return r;
  if (total_tokens < 0) return fail(HS_ERR_INVALID_ARG, "total_tokens < 0");
  if (total_tokens > 0 && num_seqs < 1)
    return fail(HS_ERR_INVALID_ARG, "num_seqs must be >= 1 when total_tokens > 0");
  if (!cu_seqlens || !seq_lens) return fail(HS_ERR_INVALID_ARG, "cu_seqlens or seq_lens is NULL");
  a.table = block_table;
  a.table_stride = table_stride;
  a.table_width = table_width;
  a.num_pages = num_pages;
  a.ps_log2 = log2_of(page_size);
  a.cu = cu_seqlens;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.total_tokens = total_tokens;
  return HS_OK;
}

hs_status hs_kv4_append(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                        void* k_cache, void* v_cache, const int32_t* block_table,
                        int64_t table_stride, int table_width, int num_pages, int page_size,
                        const int32_t* cu_seqlens, const int32_t* seq_lens, int num_seqs,
                        int total_tokens, int dk, int dv, hs_dtype dtype, hs_stream_t stream) {
  hs::Kv4Rows a{};
  hs_status r = check_rows(a, block_table, table_stride, table_width, num_pages, page_size,
                           cu_seqlens, seq_lens, num_seqs, total_tokens);
  if (r != HS_OK) return r;
  if ((r = check_dtype(dtype)) != HS_OK) return r;
  if ((r = check_width("dk", dk)) != HS_OK) return r;
  if (dv != 0 && (r = check_width("dv", dv)) != HS_OK) return r;
  if (!k || !k_cache) return fail(HS_ERR_INVALID_ARG, "k or k_cache is NULL");
  if (dv == 0 ? (v || v_cache) : (!v || !v_cache))
    return fail(HS_ERR_INVALID_ARG, "v and v_cache go with dv > 0, and only with it");
  if (k_row_stride < dk)
    return fail(HS_ERR_INVALID_ARG, "k_row_stride %lld < dk", (long long)k_row_stride);
  if (v_row_stride < dv)
    return fail(HS_ERR_INVALID_ARG, "v_row_stride %lld < dv", (long long)v_row_stride);
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(HS_ERR_INVALID_ARG, "a cache is not 16-byte aligned");
  if (total_tokens == 0) return HS_OK;
  r = status_ptr(&a.status);
  if (r != HS_OK) return r;
  const hs::Kv4Append w{k, k_row_stride, v, v_row_stride, k_cache, v_cache, dk, dv, dtype};
  return launched_on(hs::launch_kv4_append(a, w, stream), "4-bit cache append", HS_PATH_SIMT);
}

hs_status hs_kv4_read(const void* cache, int width, const int32_t* block_table,
                      int64_t table_stride, int table_width, int num_pages, int page_size,
                      const int32_t* cu_seqlens, const int32_t* seq_lens, int num_seqs,
                      int total_tokens, void* out, int64_t out_row_stride, hs_dtype dtype,
                      hs_stream_t stream) {
  hs::Kv4Rows a{};
  hs_status r = check_rows(a, block_table, table_stride, table_width, num_pages, page_size,
                           cu_seqlens, seq_lens, num_seqs, total_tokens);
  if (r != HS_OK) return r;
  if ((r = check_dtype(dtype)) != HS_OK) return r;
  if ((r = check_width("width", width)) != HS_OK) return r;
  if (!cache || !out) return fail(HS_ERR_INVALID_ARG, "cache or out is NULL");
  if (out_row_stride < width)
    return fail(HS_ERR_INVALID_ARG, "out_row_stride %lld < width", (long long)out_row_stride);
  if (!aligned16(cache)) return fail(HS_ERR_INVALID_ARG, "the cache is not 16-byte aligned");
  if (total_tokens == 0) return HS_OK;
  r = status_ptr(&a.status);
  if (r != HS_OK) return r;
  return launched_on(hs::launch_kv4_read(a, cache, width, out, out_row_stride, dtype, stream),
                     "4-bit cache read", HS_PATH_SIMT);
}

hs_status hs_kv4_mqa_decode(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* k_cache, const void* v_cache, const int32_t* block_table,
                            int64_t table_stride, int table_width, int num_pages, int page_size,
                            const int32_t* seq_lens, int num_seqs, int max_seqlen, int num_heads,
                            int dk, int dv, hs_dtype dtype, float softmax_scale, int window,
                            int num_first, const float* sink, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, hs_stream_t stream) {
  hs_status r =
      check_pages(block_table, table_stride, table_width, num_pages, page_size, num_seqs);
  if (r != HS_OK) return r;
  if ((r = check_dtype(dtype)) != HS_OK) return r;
  if ((r = check_width("dk", dk)) != HS_OK) return r;
  if ((r = check_width("dv", dv)) != HS_OK) return r;
  if (num_heads < 1 || num_heads > kMaxHeads)
    return fail(HS_ERR_UNSUPPORTED, "num_heads %d not in [1, %d]", num_heads, kMaxHeads);
  if ((int64_t)num_seqs * num_heads > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "num_seqs * num_heads does not fit 31 bits");
  if (num_seqs > 0 && max_seqlen < 1)
    return fail(HS_ERR_INVALID_ARG, "max_seqlen must be >= 1");
  if (!q || !k_cache || !seq_lens)
    return fail(HS_ERR_INVALID_ARG, "q, k_cache or seq_lens is NULL");
  if (!out || !lse) return fail(HS_ERR_INVALID_ARG, "out or lse is NULL");
  if (!v_cache && dv > dk)
    return fail(HS_ERR_INVALID_ARG, "without a v_cache dv %d must not exceed dk %d", dv, dk);
  if (q_head_stride < dk)
    return fail(HS_ERR_INVALID_ARG, "q_head_stride %lld < dk", (long long)q_head_stride);
  if (q_row_stride < (int64_t)num_heads * q_head_stride)
    return fail(HS_ERR_INVALID_ARG, "q_row_stride %lld < num_heads * q_head_stride",
                (long long)q_row_stride);
  if (!isfinite(softmax_scale)) return fail(HS_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (window < 0 || num_first < 0)
    return fail(HS_ERR_INVALID_ARG, "window %d or num_first %d < 0", window, num_first);
  if (window == 0 && num_first != 0)
    return fail(HS_ERR_INVALID_ARG, "num_first without a window");
  // the kernels count the batch's tiles of 128 keys in 31 bits
  const int64_t keys = window > 0 ? std::min((int64_t)max_seqlen, (int64_t)window + num_first) : max_seqlen;
  if ((keys + 127) / 128 * num_seqs > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "num_seqs %d times %lld keys is more than one call takes", num_seqs,
                (long long)keys);
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(HS_ERR_INVALID_ARG, "a cache is not 16-byte aligned");
  if (num_seqs == 0) return HS_OK;
  const size_t need = hs_workspace_size(HS_OP_KV4_MQA_DECODE, num_seqs, num_seqs, max_seqlen,
                                        num_heads, dk, dv, dtype, page_size);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(HS_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(HS_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  hs::Kv4Decode a{};
  a.q = q;
  a.q_row_stride = q_row_stride;
  a.q_head_stride = q_head_stride;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.table = block_table;
  a.table_stride = table_stride;
  a.table_width = table_width;
  a.num_pages = num_pages;
  a.ps_log2 = log2_of(page_size);
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  // a longer one counts as out of range: the kernels add a tile's or a split's size
  // to key counts in 32 bits
  a.max_seqlen = std::min(max_seqlen, INT32_MAX - 4095);
  a.num_heads = num_heads;
  a.dk = dk;
  a.dv = dv;
  a.dtype = dtype;
  a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)dk);
  a.window = window < max_seqlen ? window : max_seqlen;  // beyond every sequence: the same
  a.first = num_first < max_seqlen ? num_first : max_seqlen;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  r = status_ptr(&a.status);
  if (r != HS_OK) return r;
  if (!g_force_simt.load() && hs::tc_kv4_decode_eligible(a))
    return launched_on(hs::launch_tc_kv4_decode(a, g_wait_limit.load(), stream),
                       "tc 4-bit cache decode", HS_PATH_TCGEN05);
  return launched_on(hs::launch_simt_kv4_decode(a, stream), "simt 4-bit cache decode",
                     HS_PATH_SIMT);
}

}  // extern "C"

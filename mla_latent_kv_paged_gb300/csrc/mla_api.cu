// C ABI entry points: argument validation on the host, then kernel launches on
// the caller's stream. Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>

#include "blocks.cuh"
#include "chunk.cuh"
#include "mla_internal.cuh"

using namespace mla;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

mla_status launch_status(cudaError_t e) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

bool heads_ok(int H) { return H >= 1 && H <= kMaxHeads; }

// The address a kernel uses for p: device or managed memory as it is, pinned
// host memory through its mapped device address; false for memory the device
// cannot address (pageable host memory) or when the runtime cannot tell.
bool device_address(const void* p, const void** out) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) {
    *out = p;
    return true;
  }
  if (a.type == cudaMemoryTypeHost && a.devicePointer) {
    // the same offset inside the allocation
    *out = static_cast<const char*>(a.devicePointer) +
           (static_cast<const char*>(p) - static_cast<const char*>(a.hostPointer));
    return true;
  }
  return false;
}

}  // namespace

extern "C" {

const char* mla_status_string(int status) {
  switch (status) {
    case MLA_OK: return "MLA_OK";
    case MLA_ERR_INVALID_ARG: return "MLA_ERR_INVALID_ARG";
    case MLA_ERR_UNSUPPORTED_SHAPE: return "MLA_ERR_UNSUPPORTED_SHAPE";
    case MLA_ERR_WORKSPACE_TOO_SMALL: return "MLA_ERR_WORKSPACE_TOO_SMALL";
    case MLA_ERR_CUDA: return "MLA_ERR_CUDA";
    case MLA_ERR_TIMEOUT: return "MLA_ERR_TIMEOUT";
    case MLA_ERR_BOUNDS: return "MLA_ERR_BOUNDS";
    case MLA_ERR_RANGE: return "MLA_ERR_RANGE";
    case MLA_ERR_NO_PAGES: return "MLA_ERR_NO_PAGES";
    default: return "MLA_ERR_UNKNOWN";
  }
}

int mla_abi_version(void) { return MLA_ABI_VERSION; }

size_t mla_cache_bytes_per_token(int d_c, int d_r) {
  if (d_c < 0 || d_r < 0) return 0;
  return (size_t)(d_c + d_r) * 2u;
}

size_t mla_page_bytes(int page_size, int d_c, int d_r) {
  if (page_size < 0) return 0;
  return (size_t)page_size * mla_cache_bytes_per_token(d_c, d_r);
}

mla_status mla_absorb_q(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w_uk,
                        uint16_t* q_abs, int T, int H, int d_nope, int d_r, int d_c, void* stream) {
  if (!q_nope || !q_rope || !w_uk || !q_abs) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_nope) || !aligned16(q_rope) || !aligned16(w_uk) || !aligned16(q_abs))
    return MLA_ERR_INVALID_ARG;
  if (T < 1) return MLA_ERR_INVALID_ARG;
  if (d_nope != kDNope || d_r != kDR || d_c != kDC || !heads_ok(H)) return MLA_ERR_UNSUPPORTED_SHAPE;
  return launch_status(launch_absorb_q(q_nope, q_rope, w_uk, q_abs, T, H, (cudaStream_t)stream));
}

mla_status mla_merge_w_kq(const uint16_t* w_uq, const uint16_t* w_uk, uint16_t* w_kq, int d_q, int H, int d_nope,
                          int d_c, void* stream) {
  if (!w_uq || !w_uk || !w_kq) return MLA_ERR_INVALID_ARG;
  if (!aligned16(w_uq) || !aligned16(w_uk) || !aligned16(w_kq)) return MLA_ERR_INVALID_ARG;
  if (d_q < 1) return MLA_ERR_INVALID_ARG;
  if (d_nope != kDNope || d_c != kDC || !heads_ok(H) || d_q % 64 != 0 || d_q > 16384)
    return MLA_ERR_UNSUPPORTED_SHAPE;
  return launch_status(launch_merge_w_kq(w_uq, w_uk, w_kq, d_q, H, (cudaStream_t)stream));
}

mla_status mla_absorb_q_latent(const uint16_t* c_q, const uint16_t* q_rope, const uint16_t* w_kq, uint16_t* q_abs,
                               int T, int H, int d_q, int d_r, int d_c, void* stream) {
  if (!c_q || !q_rope || !w_kq || !q_abs) return MLA_ERR_INVALID_ARG;
  if (!aligned16(c_q) || !aligned16(q_rope) || !aligned16(w_kq) || !aligned16(q_abs)) return MLA_ERR_INVALID_ARG;
  if (T < 1 || d_q < 1) return MLA_ERR_INVALID_ARG;
  if (d_r != kDR || d_c != kDC || !heads_ok(H) || d_q % 64 != 0 || d_q > 16384) return MLA_ERR_UNSUPPORTED_SHAPE;
  return launch_status(launch_absorb_latent(c_q, q_rope, w_kq, q_abs, T, H, d_q, (cudaStream_t)stream));
}

namespace {
bool comb_shape_ok(int H, int d_model) { return heads_ok(H) && d_model % 128 == 0 && d_model >= 128 && d_model <= 65536; }
}  // namespace

mla_status mla_merge_w_comb(const uint16_t* w_uv, const uint16_t* w_o, uint16_t* w_comb, int H, int d_v, int d_c,
                            int d_model, void* stream) {
  if (!w_uv || !w_o || !w_comb) return MLA_ERR_INVALID_ARG;
  if (!aligned16(w_uv) || !aligned16(w_o) || !aligned16(w_comb)) return MLA_ERR_INVALID_ARG;
  if (d_model < 1) return MLA_ERR_INVALID_ARG;
  if (d_v != kDV || d_c != kDC || !comb_shape_ok(H, d_model)) return MLA_ERR_UNSUPPORTED_SHAPE;
  // w_comb[n][h][c] = sum_v w_o[n][h][v] w_uv[h][v][c]: the absorption kernel with
  // the rows of w_o in place of query rows and w_uv in place of w_uk
  return launch_status(launch_merge_w_kq(w_o, w_uv, w_comb, d_model, H, (cudaStream_t)stream));
}

size_t mla_out_comb_workspace_bytes(int T, int H, int d_model) {
  if (T < 1 || T > 2 * MLA_MAX_BATCH || !comb_shape_ok(H, d_model)) return 0;
  return out_comb_workspace_bytes(T, H, d_model);
}

mla_status mla_out_comb(const uint16_t* u, const uint16_t* w_comb, uint16_t* out, int T, int H, int d_c, int d_model,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!u || !w_comb || !out || !workspace) return MLA_ERR_INVALID_ARG;
  if (!aligned16(u) || !aligned16(w_comb) || !aligned16(out) || !aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  if (T < 1 || d_model < 1) return MLA_ERR_INVALID_ARG;
  if (T > 2 * MLA_MAX_BATCH || d_c != kDC || !comb_shape_ok(H, d_model)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < out_comb_workspace_bytes(T, H, d_model)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  return launch_status(launch_out_comb(u, w_comb, out, T, H, d_model, workspace, (cudaStream_t)stream));
}

int mla_decode_default_splits(int n_q) {
  if (n_q < 1) return -1;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  // one wave of worker clusters, shared by the n_q query indices
  int workers = decode_max_workers();
  if (workers < 1) workers = sms / 2;
  int g = workers / n_q;
  return g < 1 ? 1 : g;
}

size_t mla_decode_workspace_bytes(int B, int n_q, int H, int num_splits) {
  if (B < 1 || B > MLA_MAX_BATCH || n_q < 1 || n_q > 2 || !heads_ok(H) || num_splits < 1) return 0;
  return plan_layout(nullptr, B, n_q, H, num_splits, nullptr);
}

namespace {
// the checks shared by the decode entry points; fills `plan` on success
mla_status decode_args(void* workspace, size_t workspace_bytes, int B, int n_q, int H, int num_pages,
                       int page_size, int max_pages_per_seq, int num_splits, Plan* plan) {
  if (!workspace || !aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  if (B < 1 || num_pages < 1 || max_pages_per_seq < 1 || num_splits < 1) return MLA_ERR_INVALID_ARG;
  if (B > MLA_MAX_BATCH || n_q < 1 || n_q > 2 || !heads_ok(H) || !page_size_ok(page_size))
    return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  const size_t need = plan_layout(nullptr, B, n_q, H, num_splits, nullptr);
  if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
  plan_layout(workspace, B, n_q, H, num_splits, plan);
  return MLA_OK;
}
}  // namespace

mla_status mla_decode_paged(const uint16_t* q_abs, const uint16_t* cache,
                            const int32_t* block_table, const int32_t* seq_lens,
                            int B, int n_q, int H, int num_pages, int page_size,
                            int max_pages_per_seq, float softmax_scale, int num_splits,
                            void* workspace, size_t workspace_bytes, int32_t* err_word,
                            void* stream) {
  if (!q_abs || !cache || !block_table || !seq_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(cache) || !aligned16(block_table) || !aligned16(seq_lens))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale != softmax_scale) return MLA_ERR_INVALID_ARG;
  Plan plan;
  mla_status st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                              num_splits, &plan);
  if (st != MLA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  st = launch_status(launch_plan(seq_lens, block_table, B, n_q, max_pages_per_seq, page_size, num_pages, num_splits,
                                 plan, err_word, s));
  if (st != MLA_OK) return st;
  return launch_status(launch_decode(q_abs, cache, block_table, B, n_q, H, num_pages, page_size,
                                     max_pages_per_seq, softmax_scale, num_splits, plan, err_word, s));
}

mla_status mla_quantize_fp8(const uint16_t* rows, const float* scales, uint8_t* codes, int64_t n_rows,
                            void* stream) {
  if (!rows || !scales || !codes) return MLA_ERR_INVALID_ARG;
  if (!aligned16(rows) || !aligned16(scales) || !aligned16(codes)) return MLA_ERR_INVALID_ARG;
  if (n_rows < 1 || n_rows > ((int64_t)1 << 40)) return MLA_ERR_INVALID_ARG;
  return launch_status(launch_quantize_fp8(rows, scales, codes, n_rows, (cudaStream_t)stream));
}

mla_status mla_decode_paged_fp8(const uint16_t* q_abs, const uint8_t* cache8, const float* scales,
                                const int32_t* block_table, const int32_t* seq_lens, int B, int n_q, int H,
                                int num_pages, int page_size, int max_pages_per_seq, float softmax_scale,
                                int num_splits, void* workspace, size_t workspace_bytes, int32_t* err_word,
                                void* stream) {
  if (!q_abs || !cache8 || !scales || !block_table || !seq_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(cache8) || !aligned16(scales) || !aligned16(block_table) ||
      !aligned16(seq_lens))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale != softmax_scale) return MLA_ERR_INVALID_ARG;
  Plan plan;
  mla_status st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                              num_splits, &plan);
  if (st != MLA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  st = launch_status(launch_plan(seq_lens, block_table, B, n_q, max_pages_per_seq, page_size, num_pages, num_splits,
                                 plan, err_word, s));
  if (st != MLA_OK) return st;
  return launch_status(launch_decode_fp8(q_abs, cache8, scales, block_table, B, n_q, H, num_pages, page_size,
                                         max_pages_per_seq, softmax_scale, num_splits, plan, err_word, s));
}

mla_status mla_decode_paged_planned_fp8(const uint16_t* q_abs, const uint8_t* cache8, const float* scales,
                                        const int32_t* block_table, int B, int n_q, int H, int num_pages,
                                        int page_size, int max_pages_per_seq, float softmax_scale, int num_splits,
                                        void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  if (!q_abs || !cache8 || !scales || !block_table) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(cache8) || !aligned16(scales) || !aligned16(block_table))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale != softmax_scale) return MLA_ERR_INVALID_ARG;
  Plan plan;
  mla_status st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                              num_splits, &plan);
  if (st != MLA_OK) return st;
  return launch_status(launch_decode_fp8(q_abs, cache8, scales, block_table, B, n_q, H, num_pages, page_size,
                                         max_pages_per_seq, softmax_scale, num_splits, plan, err_word,
                                         (cudaStream_t)stream));
}

mla_status mla_decode_plan(const int32_t* seq_lens, int B, int n_q, int H, int num_pages, int page_size,
                           int max_pages_per_seq, int num_splits, void* workspace, size_t workspace_bytes,
                           int32_t* err_word, void* stream) {
  if (!seq_lens || !aligned16(seq_lens)) return MLA_ERR_INVALID_ARG;
  Plan plan;
  mla_status st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                              num_splits, &plan);
  if (st != MLA_OK) return st;
  return launch_status(launch_plan(seq_lens, nullptr, B, n_q, max_pages_per_seq, page_size, num_pages, num_splits,
                                   plan, err_word, (cudaStream_t)stream));
}

mla_status mla_decode_paged_planned(const uint16_t* q_abs, const uint16_t* cache, const int32_t* block_table,
                                    int B, int n_q, int H, int num_pages, int page_size, int max_pages_per_seq,
                                    float softmax_scale, int num_splits, void* workspace, size_t workspace_bytes,
                                    int32_t* err_word, void* stream) {
  if (!q_abs || !cache || !block_table) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(cache) || !aligned16(block_table)) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale != softmax_scale) return MLA_ERR_INVALID_ARG;
  Plan plan;
  mla_status st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                              num_splits, &plan);
  if (st != MLA_OK) return st;
  return launch_status(launch_decode(q_abs, cache, block_table, B, n_q, H, num_pages, page_size, max_pages_per_seq,
                                     softmax_scale, num_splits, plan, err_word, (cudaStream_t)stream));
}

mla_status mla_combine(const void* workspace, int B, int n_q, int H, int num_splits, uint16_t* u,
                       float* lse, void* stream) {
  if (!workspace || !u) return MLA_ERR_INVALID_ARG;
  if (!aligned16(workspace) || !aligned16(u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || num_splits < 1) return MLA_ERR_INVALID_ARG;
  if (B > MLA_MAX_BATCH || n_q < 1 || n_q > 2 || !heads_ok(H)) return MLA_ERR_UNSUPPORTED_SHAPE;
  // lse may be pinned host memory, written over the host link
  const void* lse_dev = nullptr;
  if (lse && !device_address(lse, &lse_dev)) return MLA_ERR_INVALID_ARG;
  Plan plan;
  plan_layout(const_cast<void*>(workspace), B, n_q, H, num_splits, &plan);
  return launch_status(launch_combine(plan, B, n_q, H, u, static_cast<float*>(const_cast<void*>(lse_dev)),
                                      (cudaStream_t)stream));
}

mla_status mla_out_proj(const uint16_t* u, const uint16_t* w_uv, uint16_t* out, int T, int H,
                        int d_c, int d_v, void* stream) {
  if (!u || !w_uv || !out) return MLA_ERR_INVALID_ARG;
  if (!aligned16(u) || !aligned16(w_uv) || !aligned16(out)) return MLA_ERR_INVALID_ARG;
  if (T < 1) return MLA_ERR_INVALID_ARG;
  if (d_c != kDC || d_v != kDV || !heads_ok(H)) return MLA_ERR_UNSUPPORTED_SHAPE;
  // out may be pinned host memory, written over the host link
  const void* out_dev = nullptr;
  if (!device_address(out, &out_dev)) return MLA_ERR_INVALID_ARG;
  return launch_status(launch_out_proj(u, w_uv, static_cast<uint16_t*>(const_cast<void*>(out_dev)), T, H,
                                       (cudaStream_t)stream));
}

mla_status mla_copy16(const void* src, void* dst, size_t bytes, void* stream) {
  if (!src || !dst || bytes == 0 || bytes % 16 != 0) return MLA_ERR_INVALID_ARG;
  if (!aligned16(src) || !aligned16(dst)) return MLA_ERR_INVALID_ARG;
  const void* s_dev = nullptr;
  const void* d_dev = nullptr;
  if (!device_address(src, &s_dev) || !device_address(dst, &d_dev)) return MLA_ERR_INVALID_ARG;
  return launch_status(launch_copy16(s_dev, const_cast<void*>(d_dev), bytes, (cudaStream_t)stream));
}

size_t mla_append_workspace_bytes(int T, int d_model) {
  if (T < 1 || T > 2 * MLA_MAX_BATCH || d_model < 64 || d_model % 64 != 0 || d_model > 65536) return 0;
  return append_workspace_bytes(T, d_model);
}

mla_status mla_append_kv(const uint16_t* h, const uint16_t* w_dkr, uint16_t* cache, const int32_t* block_table,
                         const int32_t* seq_lens, int B, int n_q, int d_model, int num_pages, int page_size,
                         int max_pages_per_seq, float rope_theta, void* workspace, size_t workspace_bytes,
                         int32_t* err_word, void* stream) {
  if (!h || !w_dkr || !cache || !block_table || !seq_lens || !workspace) return MLA_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(w_dkr) || !aligned16(cache) || !aligned16(block_table) || !aligned16(seq_lens) ||
      !aligned16(workspace))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || num_pages < 1 || max_pages_per_seq < 1) return MLA_ERR_INVALID_ARG;
  if (!(rope_theta > 1.f) || rope_theta != rope_theta) return MLA_ERR_INVALID_ARG;
  if (B > MLA_MAX_BATCH || n_q < 1 || n_q > 2 || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (d_model < 64 || d_model % 64 != 0 || d_model > 65536) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < append_workspace_bytes(B * n_q, d_model)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  return launch_status(launch_append(h, w_dkr, cache, block_table, seq_lens, B, n_q, d_model, num_pages, page_size,
                                     max_pages_per_seq, (double)rope_theta, workspace, err_word,
                                     (cudaStream_t)stream));
}

// ------------------------------------------------------------------ block scales
namespace {
// the checks of the arguments that name a block-scaled cache; fills `out` on success
mla_status block_args(const void* cache8, const void* entries, int block_tokens, BlockScales* out) {
  if (!cache8 || !entries || !aligned16(cache8) || !aligned16(entries)) return MLA_ERR_INVALID_ARG;
  if (!block_tokens_ok(block_tokens)) return MLA_ERR_UNSUPPORTED_SHAPE;
  out->entries = static_cast<uint8_t*>(const_cast<void*>(entries));
  out->shift = block_shift(block_tokens);
  return MLA_OK;
}
}  // namespace

mla_status mla_decode_paged_blocks(const uint16_t* q_abs, int q_f16, const uint8_t* cache8, const uint8_t* entries,
                                   int block_tokens, const int32_t* block_table, const int32_t* seq_lens, int B,
                                   int n_q, int H, int num_pages, int page_size, int max_pages_per_seq,
                                   float softmax_scale, int num_splits, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  if (!q_abs || !block_table || !seq_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(block_table) || !aligned16(seq_lens)) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  BlockScales scales;
  mla_status st = block_args(cache8, entries, block_tokens, &scales);
  Plan plan;
  if (st == MLA_OK)
    st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq, num_splits, &plan);
  cudaStream_t s = (cudaStream_t)stream;
  if (st == MLA_OK)
    st = launch_status(launch_plan(seq_lens, block_table, B, n_q, max_pages_per_seq, page_size, num_pages, num_splits,
                                   plan, err_word, s));
  if (st == MLA_OK)
    st = launch_status(launch_decode_blocks(q_abs, q_f16 != 0, cache8, scales, block_table, B, n_q, H, num_pages,
                                            page_size, max_pages_per_seq, softmax_scale, num_splits, plan, err_word, s));
  return st;
}

mla_status mla_decode_paged_planned_blocks(const uint16_t* q_abs, int q_f16, const uint8_t* cache8,
                                           const uint8_t* entries, int block_tokens, const int32_t* block_table,
                                           int B, int n_q, int H, int num_pages, int page_size, int max_pages_per_seq,
                                           float softmax_scale,
                                           int num_splits, void* workspace, size_t workspace_bytes,
                                           int32_t* err_word, void* stream) {
  if (!q_abs || !block_table) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(block_table)) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  BlockScales scales;
  mla_status st = block_args(cache8, entries, block_tokens, &scales);
  Plan plan;
  if (st == MLA_OK)
    st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq, num_splits, &plan);
  if (st == MLA_OK)
    st = launch_status(launch_decode_blocks(q_abs, q_f16 != 0, cache8, scales, block_table, B, n_q, H, num_pages,
                                            page_size, max_pages_per_seq, softmax_scale, num_splits, plan, err_word,
                                            (cudaStream_t)stream));
  return st;
}

mla_status mla_decode_step_blocks(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w_uk,
                                  const uint16_t* w_uv, const uint8_t* cache8, const uint8_t* entries, int block_tokens,
                                  const int32_t* block_table, const int32_t* seq_lens, int B, int n_q, int H,
                                  int num_pages, int page_size, int max_pages_per_seq, float softmax_scale,
                                  int num_splits, uint16_t* q_abs, uint16_t* u, float* lse, uint16_t* out,
                                  void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  if (!q_nope || !q_rope || !w_uk || !w_uv || !block_table || !seq_lens || !q_abs || !u || !out)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_nope) || !aligned16(q_rope) || !aligned16(w_uk) || !aligned16(w_uv) || !aligned16(block_table) ||
      !aligned16(seq_lens) || !aligned16(q_abs) || !aligned16(u) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  BlockScales scales;
  mla_status st = block_args(cache8, entries, block_tokens, &scales);
  Plan plan;
  if (st == MLA_OK)
    st = decode_args(workspace, workspace_bytes, B, n_q, H, num_pages, page_size, max_pages_per_seq, num_splits, &plan);
  if (st != MLA_OK) return st;
  // lse and out may be pinned host memory, written over the host link
  const void *lse_dev = nullptr, *out_dev = nullptr;
  if ((lse && !device_address(lse, &lse_dev)) || !device_address(out, &out_dev)) return MLA_ERR_INVALID_ARG;
  const int T = B * n_q;
  cudaStream_t s = (cudaStream_t)stream;
  st = launch_status(launch_plan(seq_lens, nullptr, B, n_q, max_pages_per_seq, page_size, num_pages, num_splits, plan,
                                 err_word, s));
  if (st == MLA_OK)
    st = launch_status(launch_absorb_q(q_nope, q_rope, w_uk, q_abs, T, H, s, nullptr, nullptr, err_word, true));
  if (st == MLA_OK)
    st = launch_status(launch_decode_blocks(q_abs, true, cache8, scales, block_table, B, n_q, H, num_pages, page_size,
                                            max_pages_per_seq, softmax_scale, num_splits, plan, err_word, s));
  if (st == MLA_OK)
    st = launch_status(launch_combine(plan, B, n_q, H, u, static_cast<float*>(const_cast<void*>(lse_dev)), s));
  if (st == MLA_OK)
    st = launch_status(launch_out_proj(u, w_uv, static_cast<uint16_t*>(const_cast<void*>(out_dev)), T, H, s));
  return st;
}

// ------------------------------------------------------------------ chunks of new tokens
namespace {
bool chunk_counts_ok(int B, int T) { return B <= MLA_MAX_BATCH && T <= kMaxChunkRows; }
// heads whose keys and values are expanded at once: all of them while those fit
// kExpandBytes (the default workspace stays bounded on long contexts)
constexpr int64_t kExpandBytes = (int64_t)2 << 30;
int chunk_head_group(int H, int64_t cap) {
  int64_t g = kExpandBytes / (cap * (kDNope + kDV) * 2);
  if (g < 1) g = 1;
  if (g >= H) return H;
  const int64_t rounds = (H + g - 1) / g;
  return (int)((H + rounds - 1) / rounds);
}
// The form of MLA_CHUNK_AUTO, for n = T / B new tokens on contexts of L = max_tokens / B.
// Measured, in us: absorbed n (2.1e-4 L + 0.2) whatever H (its MMAs take 128 head rows
// always), expanded 2.9e-4 H L (n hardly counts), beside about 25 for either; an FP8
// cache costs the absorbed form 1.4 times as much. So absorbed up to
// n = c H L / (L + 950), c = 1.37 (bf16) or 1.0 (FP8). Both sides at H = 128, bf16
// (absorbed / expanded): L = 512: n = 32 35/44, 64 48/44; L = 4096: n = 128 162/184,
// 160 203/191; L = 16384: n = 160 603/655, 192 714/659; FP8, L = 4096: n = 96 172/195,
// 128 216/197; H = 16, L = 16384: n = 16 84/111, 32 139/112. With block scales c = 1.12,
// H = 128: L = 512: n = 48 38/39, 64 42/39; L = 4096: n = 112 161/166, 128 180/167; L = 16384:
// n = 128 566/576, 160 712/598; H = 16, L = 16384: n = 16 99/112, 24 126/103.
enum CacheKind { kBf16Cache, kColumnScales, kBlockScales };
int chunk_form(int form, int B, int T, int H, int64_t max_tokens, CacheKind kind) {
  if (form != MLA_CHUNK_AUTO) return form;
  const double L = (double)max_tokens / B, n = (double)T / B;
  const double c = kind == kBf16Cache ? 1.37 : kind == kColumnScales ? 1.0 : 1.12;
  return T <= MLA_MAX_BATCH && n * (L + 950.0) <= c * H * L ? MLA_CHUNK_ABSORBED : MLA_CHUNK_EXPANDED;
}
// bytes of workspace of a form that is not AUTO; 0 without a device
size_t chunk_form_bytes(int form, int B, int T, int H, int64_t max_tokens) {
  if (form == MLA_CHUNK_ABSORBED) {
    const int G = T > MLA_MAX_BATCH ? -1 : mla_decode_default_splits(1);
    return G < 1 ? 0 : chunk_rows_layout(nullptr, T, H, G, nullptr);
  }
  // (with the weight copies that an FP8 cache needs)
  return chunk_layout(nullptr, B, T, chunk_head_group(H, chunk_cap(max_tokens, B)), max_tokens, H, nullptr);
}
}  // namespace

namespace {
mla_status read_rows(const void* cache, const float* fp8_scales, const BlockScales* blocks, const int32_t* block_table,
                     const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* rows, int B,
                     int n_rows, int num_pages, int page_size, int max_pages_per_seq, int32_t* err_word,
                     cudaStream_t s) {
  if (!cache || !block_table || !seq_lens || !cu || !rows) return MLA_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(fp8_scales) || !aligned16(block_table) || !aligned16(seq_lens) ||
      !aligned16(first) || !aligned16(cu) || !aligned16(rows))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || n_rows < 1 || num_pages < 1 || max_pages_per_seq < 1) return MLA_ERR_INVALID_ARG;
  if (B > MLA_MAX_BATCH || n_rows > kMaxTokens || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (blocks)
    return launch_status(launch_read_blocks(static_cast<const uint8_t*>(cache), *blocks, block_table, seq_lens, first,
                                            cu, rows, B, n_rows, num_pages, page_size, max_pages_per_seq, err_word, s));
  return launch_status(launch_read_kv(cache, fp8_scales, block_table, seq_lens, first, cu, rows, B, n_rows, num_pages,
                                      page_size, max_pages_per_seq, err_word, s));
}
}  // namespace

mla_status mla_read_kv(const void* cache, const float* fp8_scales, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* rows, int B,
                       int n_rows, int num_pages, int page_size, int max_pages_per_seq, int32_t* err_word,
                       void* stream) {
  return read_rows(cache, fp8_scales, nullptr, block_table, seq_lens, first, cu, rows, B, n_rows, num_pages, page_size,
                   max_pages_per_seq, err_word, (cudaStream_t)stream);
}

mla_status mla_read_kv_blocks(const uint8_t* cache8, const uint8_t* entries, int block_tokens,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* first,
                              const int32_t* cu, uint16_t* rows, int B, int n_rows, int num_pages, int page_size,
                              int max_pages_per_seq, int32_t* err_word, void* stream) {
  BlockScales scales;
  const mla_status st = block_args(cache8, entries, block_tokens, &scales);
  if (st != MLA_OK) return st;
  return read_rows(cache8, nullptr, &scales, block_table, seq_lens, first, cu, rows, B, n_rows, num_pages, page_size,
                   max_pages_per_seq, err_word, (cudaStream_t)stream);
}

mla_status mla_write_kv(const uint16_t* rows, uint8_t* cache8, uint8_t* entries, int block_tokens,
                        const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                        int num_pages, int page_size, int max_pages_per_seq, int32_t* err_word, void* stream) {
  if (!rows || !block_table || !seq_lens || !cu) return MLA_ERR_INVALID_ARG;
  if (!aligned16(rows) || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(cu)) return MLA_ERR_INVALID_ARG;
  BlockScales scales;
  const mla_status st = block_args(cache8, entries, block_tokens, &scales);
  if (st != MLA_OK) return st;
  if (B < 1 || T < 1 || num_pages < 1 || max_pages_per_seq < 1) return MLA_ERR_INVALID_ARG;
  if (!chunk_counts_ok(B, T) || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  return launch_status(launch_write_kv(rows, cache8, scales, block_table, seq_lens, cu, B, T, num_pages, page_size,
                                       max_pages_per_seq, err_word, (cudaStream_t)stream));
}

mla_status mla_update_pages(int32_t* block_table, int32_t* held, const int32_t* seq_lens, int32_t* free_pages,
                            int32_t* free_count, const int32_t* cu, int64_t* slots, int B, int n_rows, int num_pages,
                            int page_size, int max_pages_per_seq, int32_t* err_word, void* stream) {
  if (!block_table || !held || !seq_lens || !free_pages || !free_count) return MLA_ERR_INVALID_ARG;
  if (!aligned16(block_table) || !aligned16(held) || !aligned16(seq_lens) || !aligned16(free_pages) ||
      !aligned16(free_count) || !aligned16(cu) || !aligned16(slots))
    return MLA_ERR_INVALID_ARG;
  if ((cu == nullptr) != (slots == nullptr)) return MLA_ERR_INVALID_ARG;
  if (B < 1 || num_pages < 1 || max_pages_per_seq < 1 || n_rows < (slots ? 1 : 0)) return MLA_ERR_INVALID_ARG;
  if (!chunk_counts_ok(B, n_rows) || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  Pages p = {block_table, held, seq_lens, free_pages, free_count, cu, slots, B, slots ? n_rows : 0, num_pages,
             page_size == 64 ? 6 : 7, max_pages_per_seq};
  return launch_status(launch_update_pages(p, err_word, (cudaStream_t)stream));
}

size_t mla_append_chunk_workspace_bytes(int T, int d_model) {
  if (T < 1 || T > kMaxChunkRows || d_model < 64 || d_model % 64 != 0 || d_model > 65536) return 0;
  return append_chunk_workspace_bytes(T, d_model);
}

size_t mla_append_chunk_blocks_workspace_bytes(int T, int d_model) {
  return mla_append_chunk_workspace_bytes(T, d_model) == 0 ? 0 : append_blocks_workspace_bytes(T, d_model);
}

namespace {
mla_status append_rows(const uint16_t* h, const uint16_t* w_dkr, void* cache, const float* fp8_scales,
                       const BlockScales* blocks, const int32_t* block_table, const int32_t* seq_lens,
                       const int32_t* cu, int B, int T, int d_model, int num_pages, int page_size,
                       int max_pages_per_seq, float rope_theta, void* workspace, size_t workspace_bytes,
                       int32_t* err_word, cudaStream_t s) {
  if (!h || !w_dkr || !cache || !block_table || !seq_lens || !cu || !workspace) return MLA_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(w_dkr) || !aligned16(cache) || !aligned16(fp8_scales) || !aligned16(block_table) ||
      !aligned16(seq_lens) || !aligned16(cu) || !aligned16(workspace))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || num_pages < 1 || max_pages_per_seq < 1) return MLA_ERR_INVALID_ARG;
  if (!(rope_theta > 1.f) || rope_theta > 3.0e38f) return MLA_ERR_INVALID_ARG;
  if (!chunk_counts_ok(B, T) || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (d_model < 64 || d_model % 64 != 0 || d_model > 65536) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < (blocks ? append_blocks_workspace_bytes(T, d_model) : append_chunk_workspace_bytes(T, d_model)))
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (blocks)
    return launch_status(launch_append_blocks(h, w_dkr, static_cast<uint8_t*>(cache), *blocks, block_table, seq_lens,
                                              cu, B, T, d_model, num_pages, page_size, max_pages_per_seq,
                                              (double)rope_theta, workspace, err_word, s));
  return launch_status(launch_append_chunk(h, w_dkr, cache, fp8_scales, block_table, seq_lens, cu, B, T, d_model,
                                           num_pages, page_size, max_pages_per_seq, (double)rope_theta, workspace,
                                           err_word, s));
}
}  // namespace

mla_status mla_append_chunk(const uint16_t* h, const uint16_t* w_dkr, void* cache, const float* fp8_scales,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                            int d_model, int num_pages, int page_size, int max_pages_per_seq, float rope_theta,
                            void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  return append_rows(h, w_dkr, cache, fp8_scales, nullptr, block_table, seq_lens, cu, B, T, d_model, num_pages,
                     page_size, max_pages_per_seq, rope_theta, workspace, workspace_bytes, err_word,
                     (cudaStream_t)stream);
}

mla_status mla_append_chunk_blocks(const uint16_t* h, const uint16_t* w_dkr, uint8_t* cache8, uint8_t* entries,
                                   int block_tokens, const int32_t* block_table, const int32_t* seq_lens,
                                   const int32_t* cu, int B, int T, int d_model, int num_pages, int page_size,
                                   int max_pages_per_seq, float rope_theta, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  BlockScales scales;
  const mla_status st = block_args(cache8, entries, block_tokens, &scales);
  if (st != MLA_OK) return st;
  return append_rows(h, w_dkr, cache8, nullptr, &scales, block_table, seq_lens, cu, B, T, d_model, num_pages, page_size,
                     max_pages_per_seq, rope_theta, workspace, workspace_bytes, err_word, (cudaStream_t)stream);
}

size_t mla_attend_chunk_workspace_bytes(int B, int T, int H, int64_t max_tokens, int form) {
  if (B < 1 || T < 1 || !chunk_counts_ok(B, T) || !heads_ok(H) || max_tokens < 1 || max_tokens > kMaxTokens ||
      form < MLA_CHUNK_AUTO || form > MLA_CHUNK_ABSORBED)
    return 0;
  // the largest of what the kinds of cache need
  size_t most = 0;
  for (const CacheKind kind : {kBf16Cache, kColumnScales, kBlockScales}) {
    const size_t n = chunk_form_bytes(chunk_form(form, B, T, H, max_tokens, kind), B, T, H, max_tokens);
    if (n == 0) return 0;
    if (n > most) most = n;
  }
  return most;
}

namespace {
mla_status attend_rows(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w_uk, const uint16_t* w_uv,
                       const void* cache, const float* fp8_scales, const BlockScales* blocks,
                       const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T, int H,
                       int num_pages, int page_size, int max_pages_per_seq, int64_t max_tokens, float softmax_scale,
                       int form, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                       int32_t* err_word, cudaStream_t s) {
  if (!q_nope || !q_rope || !w_uk || !w_uv || !cache || !block_table || !seq_lens || !cu || !out || !workspace)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_nope) || !aligned16(q_rope) || !aligned16(w_uk) || !aligned16(w_uv) || !aligned16(cache) ||
      !aligned16(fp8_scales) || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(cu) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u) || !aligned16(workspace))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || num_pages < 1 || max_pages_per_seq < 1 || max_tokens < 1) return MLA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || softmax_scale > 1.0e38f) return MLA_ERR_INVALID_ARG;
  if (form < MLA_CHUNK_AUTO || form > MLA_CHUNK_ABSORBED) return MLA_ERR_INVALID_ARG;
  if (!chunk_counts_ok(B, T) || !heads_ok(H) || !page_size_ok(page_size) || max_tokens > kMaxTokens)
    return MLA_ERR_UNSUPPORTED_SHAPE;
  if (!token_counts_ok(num_pages, page_size, max_pages_per_seq)) return MLA_ERR_UNSUPPORTED_SHAPE;
  const int max_tokens_seq = max_pages_per_seq * page_size;
  form = chunk_form(form, B, T, H, max_tokens, blocks ? kBlockScales : fp8_scales ? kColumnScales : kBf16Cache);
  if (form == MLA_CHUNK_ABSORBED) {
    if (T > MLA_MAX_BATCH) return MLA_ERR_UNSUPPORTED_SHAPE;
    // the plan counts the tiles of all rows' contexts, each row's by itself, in 32 bits
    if ((int64_t)T * ((max_tokens_seq + kTile - 1) / kTile) > INT32_MAX) return MLA_ERR_UNSUPPORTED_SHAPE;
    const int G = mla_decode_default_splits(1);
    if (G < 1) return MLA_ERR_CUDA;
    if (workspace_bytes < chunk_rows_layout(nullptr, T, H, G, nullptr)) return MLA_ERR_WORKSPACE_TOO_SMALL;
    ChunkRows r;
    chunk_rows_layout(workspace, T, H, G, &r);
    Plan plan;
    plan_layout(r.decode_ws, T, 1, H, G, &plan);
    plan.seq_row = r.seq_row;
    mla_status st = launch_status(launch_rows_plan(seq_lens, cu, B, T, H, max_pages_per_seq, page_size, num_pages,
                                                   G, plan, r, w_uv, err_word, s));
    if (st == MLA_OK)
      st = launch_status(launch_absorb_q(q_nope, q_rope, w_uk, r.q_abs, T, H, s, r.hdr, fp8_scales, err_word,
                                         fp8_scales || blocks));
    if (st == MLA_OK)
      st = launch_status(blocks ? launch_decode_blocks(r.q_abs, true, static_cast<const uint8_t*>(cache), *blocks,
                                                       block_table, T, 1, H, num_pages, page_size, max_pages_per_seq,
                                                       softmax_scale, G, plan, err_word, s)
                         : fp8_scales ? launch_decode_fp8(r.q_abs, static_cast<const uint8_t*>(cache), fp8_scales,
                                                        block_table, T, 1, H, num_pages, page_size,
                                                        max_pages_per_seq, softmax_scale, G, plan, err_word, s)
                                    : launch_decode(r.q_abs, static_cast<const uint16_t*>(cache), block_table, T, 1,
                                                    H, num_pages, page_size, max_pages_per_seq, softmax_scale, G,
                                                    plan, err_word, s));
    if (st == MLA_OK) st = launch_status(launch_combine(plan, T, 1, H, r.u, lse, s, r.hdr));
    if (st == MLA_OK) st = launch_status(launch_out_proj(r.u, r.w16, out, T, H, s, r.hdr));
    return st;
  }
  const int64_t cap = chunk_cap(max_tokens, B);
  const int group = chunk_head_group(H, cap), slots = chunk_slots(B, T, group, max_tokens);
  if (workspace_bytes < chunk_layout(nullptr, B, T, group, max_tokens, H, nullptr)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  ChunkPlan plan;
  chunk_layout(workspace, B, T, group, max_tokens, H, &plan);
  mla_status st = launch_status(launch_chunk_plan(seq_lens, cu, B, T, max_tokens_seq, max_tokens, group, plan, err_word, s));
  // the contexts' rows, each sequence from its own multiple of 128 on, zeros behind its end
  const bool f16 = fp8_scales != nullptr;
  if (f16) {
    if (st == MLA_OK)
      st = launch_status(launch_rows_f16(cache, fp8_scales, block_table, plan.len_eff, plan.pstart, plan.rows, B,
                                         (int)cap, num_pages, page_size, max_pages_per_seq, err_word, s));
    if (st == MLA_OK) st = launch_status(launch_weights_f16(w_uk, w_uv, plan.w16, H, err_word, s));
    w_uk = plan.w16;
    w_uv = plan.w16 + (size_t)H * kDNope * kDC;
  } else if (st == MLA_OK && blocks) {
    // (bf16 holds a code times a power of two exactly)
    st = launch_status(launch_read_blocks(static_cast<const uint8_t*>(cache), *blocks, block_table, plan.len_eff,
                                          nullptr, plan.pstart, plan.rows, B, (int)cap, num_pages, page_size,
                                          max_pages_per_seq, err_word, s));
  } else if (st == MLA_OK) {
    st = launch_status(launch_read_kv(cache, nullptr, block_table, plan.len_eff, nullptr, plan.pstart, plan.rows, B,
                                      (int)cap, num_pages, page_size, max_pages_per_seq, err_word, s));
  }
  for (int h0 = 0; h0 < H && st == MLA_OK; h0 += group) {
    const int heads = H - h0 < group ? H - h0 : group;
    st = launch_status(launch_expand(plan, w_uk, w_uv, H, h0, heads, cap, f16, err_word, s));
    if (st == MLA_OK)
      st = launch_status(launch_attend(plan, q_nope, q_rope, out, lse, B, T, H, h0, heads, cap, slots, h0 / group,
                                       softmax_scale, f16, err_word, s));
  }
  return st;
}
}  // namespace

mla_status mla_attend_chunk(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w_uk,
                            const uint16_t* w_uv, const void* cache, const float* fp8_scales,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                            int H, int num_pages, int page_size, int max_pages_per_seq, int64_t max_tokens,
                            float softmax_scale, int form, uint16_t* out, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* err_word, void* stream) {
  return attend_rows(q_nope, q_rope, w_uk, w_uv, cache, fp8_scales, nullptr, block_table, seq_lens, cu, B, T, H,
                     num_pages, page_size, max_pages_per_seq, max_tokens, softmax_scale, form, out, lse, workspace,
                     workspace_bytes, err_word, (cudaStream_t)stream);
}

mla_status mla_attend_chunk_blocks(const uint16_t* q_nope, const uint16_t* q_rope, const uint16_t* w_uk,
                                   const uint16_t* w_uv, const uint8_t* cache8, const uint8_t* entries,
                                   int block_tokens, const int32_t* block_table, const int32_t* seq_lens,
                                   const int32_t* cu, int B, int T, int H, int num_pages, int page_size,
                                   int max_pages_per_seq, int64_t max_tokens, float softmax_scale, int form,
                                   uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  BlockScales scales;
  const mla_status st = block_args(cache8, entries, block_tokens, &scales);
  if (st != MLA_OK) return st;
  return attend_rows(q_nope, q_rope, w_uk, w_uv, cache8, nullptr, &scales, block_table, seq_lens, cu, B, T, H,
                     num_pages, page_size, max_pages_per_seq, max_tokens, softmax_scale, form, out, lse, workspace,
                     workspace_bytes, err_word, (cudaStream_t)stream);
}

}  // extern "C"

// Declarations shared by the kernels that work on a ragged chunk of new tokens
// (append_chunk, read_kv, attend_chunk): sequence b owns rows cu[b] .. cu[b+1]
// of the row arrays; rows at and past cu[B] belong to no sequence.
#pragma once

#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {

constexpr int kMaxChunkRows = 1 << 20;  // rows of one call
constexpr int kQTile = 256;             // query rows of one attention work item (two MMA tiles of 128)
constexpr int kKvTile = 128;            // cached tokens of one attention step; padding of the expanded rows

// The sequence that owns row t, or -1. Safe for any contents of cu: the search
// stays inside [0, B) and its result is checked against its own bounds.
__device__ inline int row_sequence(const int32_t* __restrict__ cu, int B, int t) {
  int lo = 0, hi = B - 1;  // largest b with cu[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return __ldg(cu + lo) <= t && t < __ldg(cu + lo + 1) ? lo : -1;
}

// Reports a cu that does not start at 0, decreases or passes the T rows of the array:
// rows that no thread of one of their own would meet. Every `threads`-th sequence from
// `thread` on; for one block of the grid.
__device__ inline void report_rows(const int32_t* __restrict__ cu, int B, int T, int thread, int threads,
                                   int32_t* err_word) {
  bool bad = false;
  for (int b = thread; b < B; b += threads) {
    const int a = __ldg(cu + b), e = __ldg(cu + b + 1);
    bad |= (b == 0 && a != 0) || e < a || e > T;
  }
  if (bad) report_error(err_word, MLA_ERR_BOUNDS);
}

// New rows [*c0, *c0 + n) and context length of sequence b, clamped to the row
// array and the block table; anything out of range is reported.
__device__ inline int sequence_of_chunk(const int32_t* seq_lens, const int32_t* cu, int b, int T, int max_tokens, int* c0,
                                 int* len, int32_t* err_word) {
  const int a = cu[b], e = cu[b + 1];
  const int first = min(max(a, 0), T), end = min(max(e, first), T);
  const int n = min(end - first, max_tokens);
  int L = seq_lens[b];
  if (a != first || (b == 0 && a != 0) || e != first + n || ((L < n || L > max_tokens) && n > 0)) report_error(err_word, MLA_ERR_BOUNDS);
  L = min(max(L, n), max_tokens);
  *c0 = first;
  *len = n > 0 ? L : 0;  // a sequence without new rows takes no part
  return n;
}

// Eight bf16 values as fp16 (exact for values of normal fp16 size); *top: the largest
// |value| so far, as bits.
__device__ __forceinline__ uint4 bf16x8_to_f16(uint4 w, uint32_t* top) {
  const uint32_t e[4] = {w.x, w.y, w.z, w.w};
  uint32_t f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[k] = sm100::cvt_f16x2(bf16_lo(e[k]), bf16_hi(e[k]));
    *top = max(*top, max((e[k] << 16) & 0x7FFFFFFFu, e[k] & 0x7FFF0000u));
  }
  return make_uint4(f[0], f[1], f[2], f[3]);
}
constexpr uint32_t kF16Limit = 0x477FF000u;  // 65520.0f: from here on fp16 rounds to infinity

// The MMA issuer's last act: every MMA it issued is done (a wait that gave up
// elsewhere included) before the CTA gives its tensor memory back. Bounded.
__device__ __forceinline__ void wait_mmas(uint32_t bar) {
  const long long t0 = clock64();
  while (!sm100::mbar_try_wait(bar, 0) && clock64() - t0 < sm100::kWaitLimitCycles) {
  }
}

// ---------------------------------------------------------------- workspaces
// The arrays start at the first 256-byte boundary of the caller's workspace (the
// sizes below include the room for it).
inline char* workspace_base(void* p) {
  return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p) + 255) & ~(uintptr_t)255);
}
// Expanded form. cap: rows of the expanded cache (a multiple of kKvTile).
struct ChunkPlan {
  int32_t* hdr;      // [64] hdr[0] = pieces, hdr[1] = expanded rows in use, hdr[2] = items in several pieces
  int32_t* counter;  // [kMaxHeads] the next item of each round of heads, beyond one per CTA
  int32_t* pstart;   // [B + 1] first expanded row of each sequence, a multiple of kKvTile
  int32_t* len_eff;  // [B] context lengths in use (clamped; 0 without new rows)
  int4* item;        // [max_items] {sequence, first query row in it, rows of the sequence, its first row}
  int4* piece;       // [max_items + slots][2] {first query row, rows of the sequence, its first row, its context};
                     // {first step over the keys, end step, slot of the partial result or -1, first expanded
                     // row of the sequence}: all that a work item needs, in one read
  int4* join;        // [slots] {first slot, pieces, first row of the item, its rows}
  float* o_part;     // [slots * heads][256][128] sums of weighted values of a piece
  float2* ml_part;   // [slots * heads][256] {reference maximum of the scores, sum of weights}
  uint16_t* rows;    // [cap][576] the sequences' cache rows, bf16 (of an FP8 cache: fp16, see launch_rows_f16);
                     // zeros from a context's end to its padding
  uint16_t* w16;     // [2][H][128][512] fp16 copies of w_uk and w_uv (FP8 cache only)
  uint16_t* k;       // [heads][cap][128] fp16 keys without position
  uint16_t* v;       // [heads][cap][128] fp16 values
};

inline int64_t chunk_cap(int64_t max_tokens, int B) {
  const int64_t c = max_tokens + (int64_t)(kKvTile - 1) * B;
  return (c + kKvTile - 1) / kKvTile * kKvTile;
}
inline int chunk_max_items(int B, int T) { return T / kQTile + (B < T ? B : T); }

// Work items are split over the keys only while they number fewer than four per
// SM (the imbalance of the last of more waves is small), and into at most as many
// pieces; a piece has at least kMinPiece steps.
constexpr int kSplitCtas = 4 * 152;
constexpr int kMinPiece = 4;
// Room for partial results, in pieces; 0: no item is split.
inline int chunk_slots(int B, int T, int heads, int64_t max_tokens) {
  if ((int64_t)(T / kQTile) * heads >= kSplitCtas) return 0;
  const int64_t by_steps = (int64_t)chunk_max_items(B, T) * ((max_tokens + kKvTile - 1) / kKvTile / kMinPiece);
  const int64_t by_ctas = kSplitCtas / heads;
  const int64_t n = by_steps < by_ctas ? by_steps : by_ctas;
  return n < 2 ? 0 : (int)n;
}

// w_heads: heads of the weight copies (0: none)
inline size_t chunk_layout(void* base, int B, int T, int heads, int64_t max_tokens, int w_heads, ChunkPlan* p) {
  const int64_t cap = chunk_cap(max_tokens, B);
  const int slots = chunk_slots(B, T, heads, max_tokens);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  const size_t o_hdr = take(64 * 4), o_cn = take(kMaxHeads * 4), o_ps = take((size_t)(B + 1) * 4), o_le = take((size_t)B * 4);
  const size_t o_it = take((size_t)chunk_max_items(B, T) * 16);
  const size_t o_pc = take(((size_t)chunk_max_items(B, T) + slots) * 32), o_j = take((size_t)slots * 16);
  const size_t o_o = take((size_t)slots * heads * kQTile * kDV * 4), o_m = take((size_t)slots * heads * kQTile * 8);
  const size_t o_r = take((size_t)cap * kRow * 2);
  const size_t o_w = take((size_t)w_heads * (kDNope + kDV) * kDC * 2);
  const size_t o_k = take((size_t)heads * cap * kDNope * 2), o_v = take((size_t)heads * cap * kDV * 2);
  if (base && p) {
    char* c = workspace_base(base);
    p->hdr = reinterpret_cast<int32_t*>(c + o_hdr);
    p->counter = reinterpret_cast<int32_t*>(c + o_cn);
    p->pstart = reinterpret_cast<int32_t*>(c + o_ps);
    p->len_eff = reinterpret_cast<int32_t*>(c + o_le);
    p->item = reinterpret_cast<int4*>(c + o_it);
    p->piece = reinterpret_cast<int4*>(c + o_pc);
    p->join = reinterpret_cast<int4*>(c + o_j);
    p->o_part = reinterpret_cast<float*>(c + o_o);
    p->ml_part = reinterpret_cast<float2*>(c + o_m);
    p->rows = reinterpret_cast<uint16_t*>(c + o_r);
    p->w16 = reinterpret_cast<uint16_t*>(c + o_w);
    p->k = reinterpret_cast<uint16_t*>(c + o_k);
    p->v = reinterpret_cast<uint16_t*>(c + o_v);
  }
  return off + 256;
}

// Absorbed form: each new token is a decode sequence of its own.
struct ChunkRows {
  int32_t* hdr;      // [64] hdr[0] = rows that belong to a sequence
  int32_t* seq_row;  // [T] block-table row (-1 for rows of no sequence)
  uint16_t* q_abs;   // [T][H][576] bf16 (on an FP8 cache fp16, scaled by its columns)
  uint16_t* u;       // [T][H][512] fp16
  uint16_t* w16;     // [H][128][512] fp16 copy of w_uv
  void* decode_ws;   // workspace of the decode over T sequences
};

inline size_t chunk_rows_layout(void* base, int T, int H, int G, ChunkRows* p) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  const size_t o_hdr = take(64 * 4), o_s = take((size_t)T * 4);
  const size_t o_q = take((size_t)T * H * kRow * 2), o_u = take((size_t)T * H * kDC * 2);
  const size_t o_w = take((size_t)H * kDV * kDC * 2);
  const size_t o_d = take(plan_layout(nullptr, T, 1, H, G, nullptr));
  if (base && p) {
    char* c = workspace_base(base);
    p->hdr = reinterpret_cast<int32_t*>(c + o_hdr);
    p->seq_row = reinterpret_cast<int32_t*>(c + o_s);
    p->q_abs = reinterpret_cast<uint16_t*>(c + o_q);
    p->u = reinterpret_cast<uint16_t*>(c + o_u);
    p->w16 = reinterpret_cast<uint16_t*>(c + o_w);
    p->decode_ws = c + o_d;
  }
  return off + 256;
}

// ---------------------------------------------------------------- launchers
cudaError_t launch_read_kv(const void* cache, const float* fp8_scales, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* out, int B,
                           int n_rows, int num_pages, int page_size, int max_pages, int32_t* err_word,
                           cudaStream_t s);
// The same into an fp16 workspace, of an FP8 cache: scale * e4m3 rounded to fp16 (2^-11
// relative; to bf16 it would be 2^-8, as much as the output's own rounding).
// |value| >= 65520 is reported.
cudaError_t launch_rows_f16(const void* cache8, const float* fp8_scales, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu, uint16_t* out, int B, int n_rows,
                            int num_pages, int page_size, int max_pages, int32_t* err_word, cudaStream_t s);
// ... and the weights that multiply them (MMA operands have one type): exact for bf16
// values of normal fp16 size, |value| >= 65520 is reported. out [2][H][128][512].
cudaError_t launch_weights_f16(const uint16_t* w_uk, const uint16_t* w_uv, uint16_t* out, int H, int32_t* err_word,
                               cudaStream_t s);
size_t append_chunk_workspace_bytes(int T, int d_model);
cudaError_t launch_append_chunk(const uint16_t* h, const uint16_t* w_dkr, void* cache, const float* fp8_scales,
                                const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                                int d_model, int num_pages, int page_size, int max_pages, double theta,
                                void* workspace, int32_t* err_word, cudaStream_t s);
cudaError_t launch_chunk_plan(const int32_t* seq_lens, const int32_t* cu, int B, int T, int max_tokens,
                              int64_t max_total, int heads, const ChunkPlan& plan, int32_t* err_word,
                              cudaStream_t s);
// the decode plan of a chunk's T rows, each a sequence of its own, and beside it the
// fp16 copy of w_uv that out_proj takes (plan.cu)
cudaError_t launch_rows_plan(const int32_t* seq_lens, const int32_t* cu, int sequences, int T, int H, int max_pages,
                             int page_size, int num_pages, int G, const Plan& plan, const ChunkRows& rows,
                             const uint16_t* w_uv, int32_t* err_word, cudaStream_t s);
// keys and values of heads [h0, h0 + heads) of every expanded row; f16: rows and weights are fp16, not bf16
cudaError_t launch_expand(const ChunkPlan& plan, const uint16_t* w_uk, const uint16_t* w_uv, int H, int h0, int heads,
                          int64_t cap, bool f16, int32_t* err_word, cudaStream_t s);
cudaError_t launch_attend(const ChunkPlan& plan, const uint16_t* q_nope, const uint16_t* q_rope, uint16_t* out,
                          float* lse, int B, int T, int H, int h0, int heads, int64_t cap, int slots, int round,
                          float scale, bool f16, int32_t* err_word, cudaStream_t s);

#if MLA_DEBUG_CHECKS
// Test builds only: the wait limit and the loads left out (null: as they are) of the
// kernels of one file.
cudaError_t debug_append_chunk(const long long* limit, const int* skip);
cudaError_t debug_expand(const long long* limit, const int* skip);
cudaError_t debug_attend(const long long* limit, const int* skip);
#endif

}  // namespace mla

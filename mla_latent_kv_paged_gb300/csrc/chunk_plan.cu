// Plan of the expanded attention of a ragged chunk of new tokens, from seq_lens and
// cu on the device (so a captured graph follows their contents): where each
// sequence's expanded rows start (contexts padded to 128 rows) and the list of query
// items (256 rows of one sequence each, the longest work first), cut over the keys
// into pieces when the items alone would leave SMs idle.
// Integer work on a few thousand numbers, one block: bound by launch and barrier
// latency.
#include "chunk.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kFixed = 3;  // a piece's start and end, in steps (about 1.6 us each)
constexpr int kRanked = 512;
constexpr int kJoin = 4;   // the launch that joins the pieces, in steps

// Exclusive scan over the block's threads of a 64-bit value; *total = the sum.
__device__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads, 1)
chunk_plan_kernel(const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu, int B, int T, int max_tokens,
                  int64_t max_total, int max_items, int heads, int slots, ChunkPlan plan, int32_t* err_word) {
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x;
  if (tid < kMaxHeads) plan.counter[tid] = 0;
  int64_t row_base = 0, item_base = 0, token_base = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    int c0 = 0, L = 0, n = 0;
    if (b < B) n = sequence_of_chunk(seq_lens, cu, b, T, max_tokens, &c0, &L, err_word);
    int64_t rows = (int64_t)(L + kKvTile - 1) / kKvTile * kKvTile;
    int items = (n + kQTile - 1) / kQTile;
    int64_t row_sum, item_sum, token_sum;
    const int64_t t0 = token_base + block_scan(L, &token_sum);
    // a sequence that passes the tokens (or, with overlapping rows, the items) the
    // caller announced is left out: no expanded rows, no work
    const bool fits = t0 + L <= max_total;
    if (!fits) rows = 0;
    const int64_t r0 = row_base + block_scan(rows, &row_sum);
    const int64_t i0 = item_base + block_scan(items, &item_sum);
    if (b < B) {
      if (!fits || i0 + items > max_items) report_error(err_word, MLA_ERR_BOUNDS);
      plan.pstart[b] = (int)r0;
      plan.len_eff[b] = fits ? L : 0;
      for (int k = 0; k < items; ++k)
        if (i0 + k < max_items)
          plan.item[i0 + k] = make_int4(fits ? b : -1, (items - 1 - k) * kQTile, n, c0);
    }
    row_base += row_sum;
    token_base += token_sum;
    item_base += item_sum;
  }
  if (tid == 0) {
    plan.pstart[B] = (int)row_base;
    plan.hdr[1] = (int)row_base;
  }
  __syncthreads();  // the items and lengths are written
  const int items = (int)min(item_base, (int64_t)max_items);
  auto steps_of = [&](int i) {
    const int4 it = plan.item[i];
    return it.x < 0 ? 0 : (plan.len_eff[it.x] - it.z + min(it.y + kQTile, it.z) + kKvTile - 1) / kKvTile;
  };
  // The piece length: the longest item in 1, 2, 3, ... parts is tried by one thread
  // each. A length of p steps makes N(p) pieces per head that run in
  // ceil(N heads / SMs) waves of p steps and a fixed part worth kFixed steps; the
  // shortest total wins. N must fit the room for partial results.
  __shared__ unsigned long long best;
  __shared__ int longest, steps_s[kSplitCtas];
  if (tid == 0) {
    best = ~0ull;
    longest = 0;
  }
  __syncthreads();
  if (slots > 0 && items * (int64_t)heads < kSplitCtas) {
    int mx = 0;
    for (int i = tid; i < items; i += kThreads) {
      steps_s[i] = steps_of(i);
      mx = max(mx, steps_s[i]);
    }
    if (mx) atomicMax(&longest, mx);
    __syncthreads();
    const int p = (longest + tid) / (tid + 1);
    if (p >= kMinPiece || tid == 0) {
      int N = 0;
      for (int i = 0; i < items; ++i) N += (steps_s[i] + max(p, 1) - 1) / max(p, 1);
      if (N <= slots || tid == 0) {
        const int64_t waves = ((int64_t)N * heads + 151) / 152;
        const int64_t cost = waves * (p + kFixed) + (tid > 0 ? kJoin : 0);
        atomicMin(&best, (unsigned long long)cost << 8 | (unsigned)tid);
      }
    }
  }
  __syncthreads();
  const int parts = best == ~0ull ? 1 : (int)(best & 255) + 1;
  const int p = parts == 1 ? INT32_MAX / 2 : (longest + parts - 1) / parts;
  int64_t piece_base = 0, slot_base = 0, join_base = 0;
  // listed longest first where they are few enough to be ranked by comparison (the
  // items of a sequence come that way already)
  const bool ranked = items <= kRanked;
  if (ranked) {
    for (int i = tid; i < items; i += kThreads) steps_s[i] = steps_of(i);
    __syncthreads();
  }
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int i = i0 + tid;
    const int st = i < items ? steps_of(i) : 0;
    const int q = st > 0 ? (st + p - 1) / p : 0;
    int64_t piece_sum, slot_sum, join_sum;
    int64_t k0 = piece_base + block_scan(q, &piece_sum);
    const int64_t s0 = slot_base + block_scan(q > 1 ? q : 0, &slot_sum);
    const int64_t n0 = join_base + block_scan(q > 1 ? 1 : 0, &join_sum);
    if (ranked && q > 0) {  // the pieces of every item whose pieces are longer, then of those before it
      k0 = 0;
      for (int o = 0; o < items; ++o) {
        const int so = steps_s[o], qo = (so + p - 1) / p;
        // so / qo > st / q, in integers
        const int64_t d = (int64_t)so * q - (int64_t)st * qo;
        if (qo > 0 && (d > 0 || (d == 0 && o < i))) k0 += qo;
      }
    }
    if (q > 0) {
      const int4 it = plan.item[i];
      for (int k = 0; k < q; ++k) {
        plan.piece[2 * (k0 + k)] = make_int4(it.y, it.z, it.w, plan.len_eff[it.x]);
        plan.piece[2 * (k0 + k) + 1] = make_int4((int)((int64_t)k * st / q), (int)((int64_t)(k + 1) * st / q),
                                                 q > 1 ? (int)s0 + k : -1, plan.pstart[it.x]);
      }
      if (q > 1) plan.join[n0] = make_int4((int)s0, q, it.w + it.y, min(kQTile, it.z - it.y));
    }
    piece_base += piece_sum;
    slot_base += slot_sum;
    join_base += join_sum;
  }
  if (tid == 0) {
    plan.hdr[0] = (int)piece_base;
    plan.hdr[2] = (int)join_base;
  }
}

}  // namespace

cudaError_t launch_chunk_plan(const int32_t* seq_lens, const int32_t* cu, int B, int T, int max_tokens,
                              int64_t max_total, int heads, const ChunkPlan& plan, int32_t* err_word,
                              cudaStream_t s) {
  return launch_pdl(chunk_plan_kernel, dim3(1), dim3(kThreads), 0, s, seq_lens, cu, B, T, max_tokens, max_total,
                    chunk_max_items(B, T), heads, chunk_slots(B, T, heads, max_total), plan, err_word);
}

}  // namespace mla

// Rows of new tokens quantised into the pages of a block-scaled 8-bit cache
// (blocks.cuh): for every block of tokens that gets new rows and every group g of columns
//   e = max(the smallest power with max |x| <= 448 * 2^e over the new rows,
//           the block's power before, where it holds older tokens)
//   code = e4m3(x * 2^-e), nearest even
// and where a power grows, the codes of the block's older tokens are requantised by
// 2^(before - e). What is not finite becomes the NaN code and does not count in e.
//
// HBM-bound for prompts (1152 bytes read, 576 written a token), latency-bound for a
// decode step's one row a sequence. A CTA owns 64 positions of one sequence (a tile:
// whole blocks), so a power is decided in one place and no two CTAs write one entry: its
// rows are read once into registers, the magnitudes meet in shared memory, and the
// codes are written from the registers. CTA c belongs to the last sequence b with
// cu[b] / 64 + 2b <= c: a run of n rows touches at most n / 64 + 2 tiles, so every
// tile has a CTA without a plan on the device before (the CTAs left over end at once).
#include "blocks.cuh"
#include "chunk.cuh"

namespace mla {
namespace {

constexpr int kChunks = kRow / 8;              // 72 chunks of 8 columns per row
constexpr int kRowsAtOnce = 4;
constexpr int kThreads = kChunks * kRowsAtOnce;  // 288
constexpr int kPer = kTile / kRowsAtOnce;      // rows of a tile per thread
constexpr int kSub = kTile / 16;               // a block is at least 16 tokens: four rows of a thread

// the last sequence whose first CTA is at or before c, by all lanes of a warp: each
// round cuts the candidates by 32. Inside [0, B) whatever cu holds.
__device__ __forceinline__ int sequence_of_cta(const int32_t* __restrict__ cu, int B, int c) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool before = at < n && (__ldg(cu + lo + at) >> 6) + 2 * (lo + at) <= c;
    const int k = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
  return sm100::f16x2_to_f32(h);
}
// 0x8000 in each half that is infinite or NaN (bf16 pair)
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }

__global__ void __launch_bounds__(kThreads)
write_kv_kernel(const uint4* __restrict__ rows, uint8_t* __restrict__ cache, uint8_t* __restrict__ entries, int shift,
                const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
                const int32_t* __restrict__ cu, int B, int T, int num_pages, int page_size, int max_pages,
                int32_t* err_word) {
  __shared__ uint32_t top[kSub][kEntryBytes];    // largest magnitude of block j's new rows, bf16 bits
  __shared__ uint32_t power[kSub][kEntryBytes];  // the block's powers from now on
  __shared__ uint32_t before[kSub][kEntryBytes];  // ... and those of its older tokens' codes
  const int tid = threadIdx.x;
  if (tid < kSub * kEntryBytes) top[tid / kEntryBytes][tid % kEntryBytes] = 0;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  if (blockIdx.x == 0) report_rows(cu, B, T, tid, kThreads, err_word);
  const int b = sequence_of_cta(cu, B, blockIdx.x);
  const int first = __ldg(cu + b), end = __ldg(cu + b + 1), n = end - first, L = __ldg(seq_lens + b);
  const int tile = blockIdx.x - ((first >> 6) + 2 * b);  // of those of this sequence's new rows
  if (tile < 0 || n <= 0) return;
  if (first < 0 || end > T || L < n || L > max_pages * page_size) {  // nothing of it is written
    if (tile == 0 && tid == 0) report_error(err_word, MLA_ERR_BOUNDS);
    return;
  }
  const int p0 = L - n, t0 = (p0 / kTile + tile) * kTile;  // the first new position; the tile's first
  if (t0 >= L) return;
  const int lo = max(p0 - t0, 0), hi = min(L - t0, kTile);  // new rows of the tile
  const int page = __ldg(block_table + (int64_t)b * max_pages + t0 / page_size);
  if (page < 0 || page >= num_pages) {
    if (tid == 0) report_error(err_word, MLA_ERR_BOUNDS);
    return;
  }
  const int64_t row0 = (int64_t)page * page_size + t0 % page_size;  // of the pool
  uint8_t* entry = entries + ((row0 >> shift) << 3);

  const int g = tid % kChunks, r0 = tid / kChunks;
  const int group = g < 64 ? g >> 4 : 4;
  const uint4* src = rows + ((int64_t)first + t0 - p0) * kChunks + g;
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kRowsAtOnce * k + r0;
    v[k] = r >= lo && r < hi ? __ldg(src + (int64_t)r * kChunks) : make_uint4(0, 0, 0, 0);
  }
  uint32_t m[kSub];  // this thread's largest magnitudes of 16 positions (bf16 pairs)
#pragma unroll
  for (int j = 0; j < kSub; ++j) {
    m[j] = 0;
#pragma unroll
    for (int k = 4 * j; k < 4 * j + 4; ++k) {
      uint32_t* w = &v[k].x;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t bad = not_finite(w[q]);
        w[q] |= bad - (bad >> 15);  // 0x7FFF: infinities are stored as NaN
        m[j] = __vmaxu2(m[j], w[q] & 0x7FFF7FFFu & ~((bad >> 15) * 0xFFFFu));
      }
    }
    m[j] = max(m[j] & 0xFFFFu, m[j] >> 16);
  }
  // over the eight threads of 64 columns of a row (part of one group, and of one warp)
  uint32_t m01 = m[0] | m[1] << 16, m23 = m[2] | m[3] << 16;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    m01 = __vmaxu2(m01, __shfl_xor_sync(0xffffffffu, m01, d));
    m23 = __vmaxu2(m23, __shfl_xor_sync(0xffffffffu, m23, d));
  }
  __syncthreads();
  if ((tid & 7) == 0) {
    atomicMax(&top[0][group], m01 & 0xFFFFu);
    atomicMax(&top[16 >> shift][group], m01 >> 16);
    atomicMax(&top[32 >> shift][group], m23 & 0xFFFFu);
    atomicMax(&top[48 >> shift][group], m23 >> 16);
  }
  __syncthreads();
  if (tid < (kTile >> shift) * kEntryBytes) {
    const int j = tid / kEntryBytes, e = tid % kEntryBytes, at = j << shift;
    if (max(at, lo) < min(at + (1 << shift), hi)) {
      uint32_t p = e < kGroups ? power_of(top[j][e] << 16) : 0u, old = p;
      if (e < kGroups && at < lo && t0 + at < p0) {  // the block holds older tokens
        old = entry[tid];
        p = max(p, old);
      }
      power[j][e] = p;
      before[j][e] = old;
      entry[tid] = (uint8_t)p;
    }
  }
  __syncthreads();
  uint2* dst = reinterpret_cast<uint2*>(cache + row0 * kRow) + g;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kRowsAtOnce * k + r0;
    if (r >= lo && r < hi) {
      const float inv = inverse_step_of(power[r >> shift][group]);
      const uint32_t* w = &v[k].x;
      uint32_t c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] = e4m3x2(bf16_lo(w[q]) * inv, bf16_hi(w[q]) * inv);
      dst[(int64_t)r * kChunks] = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
  }
  // the older tokens of the block in which the new rows start
  const int start = lo >> shift << shift;
  if (t0 + lo == p0 && start < lo) {
    const uint32_t now = power[lo >> shift][group], old = before[lo >> shift][group];
    if (now != old) {  // now is the larger
      const float f = now - old < 127 ? step_of(127 + old - now) : 0.f;
      for (int r = start + r0; r < lo; r += kRowsAtOnce) {
        const uint2 w = dst[(int64_t)r * kChunks];
        const float2 a = from_e4m3x2(w.x & 0xFFFFu), b2 = from_e4m3x2(w.x >> 16), c = from_e4m3x2(w.y & 0xFFFFu),
                     d = from_e4m3x2(w.y >> 16);
        dst[(int64_t)r * kChunks] = make_uint2(e4m3x2(a.x * f, a.y * f) | e4m3x2(b2.x * f, b2.y * f) << 16,
                                               e4m3x2(c.x * f, c.y * f) | e4m3x2(d.x * f, d.y * f) << 16);
      }
    }
  }
}

}  // namespace

cudaError_t launch_write_kv(const uint16_t* rows, uint8_t* cache, const BlockScales& scales, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu, int B, int T, int num_pages, int page_size,
                            int max_pages, int32_t* err_word, cudaStream_t s) {
  return launch_pdl(write_kv_kernel, dim3(T / kTile + 2 * B), dim3(kThreads), 0, s, reinterpret_cast<const uint4*>(rows),
                    cache, scales.entries, scales.shift, block_table, seq_lens, cu, B, T, num_pages, page_size,
                    max_pages, err_word);
}

}  // namespace mla

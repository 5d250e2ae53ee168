// Rows of new tokens quantised into the pages of a block-scaled 8-bit cache
// (blocks.cuh): for every block of tokens that gets new rows and every group g of columns
//   e = max(the smallest power with max |x| <= 448 * 2^e over the new rows,
//           the block's power before, where it holds older tokens)
//   code = e4m3(x * 2^-e), nearest even
// and where a power grows, the codes of the block's older tokens are requantised by
// 2^(before - e). What is not finite becomes the NaN code and does not count in e.
//
// HBM-bound for prompts (1152 bytes read, 576 written a token), latency-bound for a
// decode step's one row a sequence. A CTA owns one group of columns at 64 positions of one
// sequence (a tile: whole blocks), so a power is decided in one place and no two CTAs write one
// byte: its values are read once into registers, the magnitudes meet in shared memory, and
// the codes are written from the registers. CTA c of a group belongs to the last sequence b with
// cu[b] / 64 + 2b <= c: a run of n rows touches at most n / 64 + 2 tiles, so every
// tile has a CTA without a plan on the device before (the CTAs left over end at once).
//
// Measured: 42026 rows of 24 prompt pieces 14.5 us (72.7 MB, 5.0 TB/s: the reads that come before a row's,
// of cu, length and page, are as long as the row's own, and over half of the issue slots are taken), one row for
// each of 128 sequences 4.0 us, a launch and five dependent reads. With magnitudes looked over two by two first and
// what is not finite only where there is some, and the products two by two in bf16 (exact: powers): 16.3 and
// 4.8 before. With 256 threads 15.2 and 4.9, held to 48 registers (ten CTAs an SM) 14.0 and 4.3; before that step
// all five groups in one CTA took 21.9 and 6.8.
#include "blocks.cuh"
#include "chunk.cuh"

namespace mla {
namespace {

constexpr int kChunks = kRow / 8;  // 72 chunks of 8 columns per row
constexpr int kThreads = 128;
constexpr int kSub = kTile / 16;   // a block is at least 16 tokens
static_assert(kGroups == 5, "four groups of 16 chunks, one of 8");

struct Rows {
  int b, first, end, L;  // the sequence, its rows of the array, its context
};
// The last sequence whose first CTA is at or before c, by all lanes of a warp: a round cuts the
// candidates by 32, the last one brings what is needed of the sequence along. Inside [0, B) whatever cu holds.
__device__ __forceinline__ Rows sequence_of_cta(const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                                                int B, int c) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 32) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool before = at < n && (__ldg(cu + lo + at) >> 6) + 2 * (lo + at) <= c;
    const int k = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  Rows r = {lo + min(lane, n - 1), 0, 0, 0};
  r.first = __ldg(cu + r.b);
  r.end = __ldg(cu + r.b + 1);
  r.L = __ldg(seq_lens + r.b);
  const int k = max(__popc(__ballot_sync(0xffffffffu, lane < n && (r.first >> 6) + 2 * r.b <= c)) - 1, 0);
  r.b = lo + k;
  r.first = __shfl_sync(0xffffffffu, r.first, k);
  r.end = __shfl_sync(0xffffffffu, r.end, k);
  r.L = __shfl_sync(0xffffffffu, r.L, k);
  return r;
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
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 0x8000 in each half that is infinite or NaN (bf16 pair)
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }

// What a CTA knows before it reads its rows.
struct Tile {
  const uint4* src;       // the group's first chunk at the tile's first position (rows before `lo` are not read)
  const int32_t* page;    // the tile's page, read beside the rows
  int64_t row;            // the tile's row in its page
  int lo, hi;             // the tile's new rows
  bool older;             // tokens older than the chunk lie in the block of row lo
};
struct Cache {
  uint8_t *codes, *entries;
  int shift, num_pages, page_size;
};

// kWide: chunks of the group in a row
template <int kWide>
__device__ __forceinline__ void write_tile(const Tile& tile, const Cache& cache, int group, uint32_t* top,
                                           uint32_t* power, uint32_t* before, int32_t* err_word) {
  constexpr int kAtOnce = kThreads / kWide, kPer = kTile / kAtOnce;  // rows of a pass, passes
  const int tid = threadIdx.x, r0 = tid / kWide, c = tid % kWide, shift = cache.shift;
  const uint4* src = tile.src + c;
  const int lo = tile.lo, hi = tile.hi;
  const int page = __ldg(tile.page);
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kAtOnce * k + r0;
    v[k] = r >= lo && r < hi ? __ldg(src + (int64_t)r * kChunks) : make_uint4(0, 0, 0, 0);
  }
  if (page < 0 || page >= cache.num_pages) {
    if (tid == 0) report_error(err_word, MLA_ERR_BOUNDS);
    return;
  }
  const int64_t row0 = (int64_t)page * cache.page_size + tile.row;  // of the pool
  uint2* dst = reinterpret_cast<uint2*>(cache.codes + row0 * kRow) + 16 * group + c;
  // thread j < blocks of a tile: its block's entry
  uint8_t* entry = cache.entries + ((row0 >> shift) + tid) * kEntryBytes + group;
  const int at = tid << shift;
  const bool owner = tid < kTile >> shift && max(at, lo) < min(at + (1 << shift), hi);
  uint32_t old = 0;
  if (owner && at < lo && tile.older) old = *entry;
  uint32_t m[kSub];  // this thread's largest magnitudes of 16 positions (bf16 pairs)
#pragma unroll
  for (int j = 0; j < kSub; ++j) m[j] = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t* w = &v[k].x;
    uint32_t& mj = m[k * kAtOnce / 16];
#pragma unroll
    for (int q = 0; q < 4; ++q) mj = __vmaxu2(mj, w[q] & 0x7FFF7FFFu);
  }
  if (not_finite(__vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3])))) {  // some value is: the maxima without those
#pragma unroll
    for (int j = 0; j < kSub; ++j) m[j] = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      uint32_t* w = &v[k].x;
      uint32_t& mj = m[k * kAtOnce / 16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t bad = not_finite(w[q]);
        w[q] |= bad - (bad >> 15);  // 0x7FFF: infinities are stored as NaN
        mj = __vmaxu2(mj, w[q] & 0x7FFF7FFFu & ~((bad >> 15) * 0xFFFFu));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kSub; ++j) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, max(m[j] & 0xFFFFu, m[j] >> 16));
    if ((tid & 31) == 0) atomicMax(top + (16 * j >> shift), most);
  }
  __syncthreads();
  if (owner) {
    const uint32_t p = max(power_of(top[tid] << 16), old);
    power[tid] = p;
    before[tid] = at < lo && tile.older ? old : p;
    *entry = (uint8_t)p;
    if (group == kGroups - 1)
      for (int k = 1; k <= kEntryBytes - kGroups; ++k) entry[k] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kAtOnce * k + r0;
    if (r >= lo && r < hi) {
      const uint32_t inv = (254u - power[r >> shift]) * 0x00800080u;  // 2^-e, a bf16 pair
      const uint32_t* w = &v[k].x;
      uint32_t e[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = mul_bf16x2(w[q], inv);  // exact wherever a code is not zero
        e[q] = e4m3x2(bf16_lo(x), bf16_hi(x));
      }
      dst[(int64_t)r * kChunks] = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
    }
  }
  // the older tokens of the block in which the new rows start, where its power grew
  const int start = lo >> shift << shift;
  if (tile.older && start < lo) {
    const uint32_t now = power[lo >> shift], old = before[lo >> shift];
    if (now != old) {
      const float f = now - old < 127 ? step_of(127 + old - now) : 0.f;
      for (int r = start + r0; r < lo; r += kAtOnce) {
        const uint2 w = dst[(int64_t)r * kChunks];
        const float2 e0 = from_e4m3x2(w.x & 0xFFFFu), e1 = from_e4m3x2(w.x >> 16), e2 = from_e4m3x2(w.y & 0xFFFFu),
                     e3 = from_e4m3x2(w.y >> 16);
        dst[(int64_t)r * kChunks] = make_uint2(e4m3x2(e0.x * f, e0.y * f) | e4m3x2(e1.x * f, e1.y * f) << 16,
                                               e4m3x2(e2.x * f, e2.y * f) | e4m3x2(e3.x * f, e3.y * f) << 16);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
write_kv_kernel(const uint4* __restrict__ rows, Cache cache, const int32_t* __restrict__ block_table,
                const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu, int B, int T, int max_pages,
                int32_t* err_word) {
  __shared__ uint32_t top[kSub];     // largest magnitude of block j's new rows, bf16 bits
  __shared__ uint32_t power[kSub];   // the block's power from now on
  __shared__ uint32_t before[kSub];  // ... and that of its older tokens' codes
  const int tid = threadIdx.x, cta = blockIdx.x / kGroups, group = blockIdx.x % kGroups;
  if (tid < kSub) top[tid] = 0;
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  if (blockIdx.x == 0) report_rows(cu, B, T, tid, kThreads, err_word);
  const Rows s = sequence_of_cta(cu, seq_lens, B, cta);
  const int n = s.end - s.first;
  const int number = cta - ((s.first >> 6) + 2 * s.b);  // of the tiles of this sequence's new rows
  if (number < 0 || n <= 0) return;
  if (s.first < 0 || s.end > T || s.L < n || s.L > max_pages * cache.page_size) {  // nothing of it is written
    if (number == 0 && tid == 0) report_error(err_word, MLA_ERR_BOUNDS);
    return;
  }
  const int p0 = s.L - n, t0 = (p0 / kTile + number) * kTile;  // the first new position; the tile's first
  if (t0 >= s.L) return;
  Tile tile;
  tile.src = rows + ((int64_t)s.first + t0 - p0) * kChunks + 16 * group;
  tile.page = block_table + (int64_t)s.b * max_pages + t0 / cache.page_size;
  tile.row = t0 % cache.page_size;
  tile.lo = max(p0 - t0, 0);
  tile.hi = min(s.L - t0, kTile);
  tile.older = p0 > t0;
  __syncthreads();  // top is cleared
  if (group < kGroups - 1)
    write_tile<16>(tile, cache, group, top, power, before, err_word);
  else
    write_tile<8>(tile, cache, group, top, power, before, err_word);
}

}  // namespace

cudaError_t launch_write_kv(const uint16_t* rows, uint8_t* cache, const BlockScales& scales, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu, int B, int T, int num_pages, int page_size,
                            int max_pages, int32_t* err_word, cudaStream_t s) {
  const Cache to = {cache, scales.entries, scales.shift, num_pages, page_size};
  return launch_pdl(write_kv_kernel, dim3(kGroups * (T / kTile + 2 * B)), dim3(kThreads), 0, s,
                    reinterpret_cast<const uint4*>(rows), to, block_table, seq_lens, cu, B, T, max_pages, err_word);
}

}  // namespace mla

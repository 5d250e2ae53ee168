// The block-scaled 8-bit latent cache: e4m3 codes as in the per-column FP8 cache,
// and for every block of 16, 32 or 64 tokens of a page an 8-byte entry with one
// power of two for each of five groups of columns (four of 128 latent columns, the
// 64 positional ones): value = code * 2^(entry[group] - 127). Bytes 5..7 are 0.
//
// Why powers of two: e4m3 is a floating format, so a scale only moves its window of
// 17 binades and a power of two loses no precision against amax / 448; requantising
// a block whose power grows then is exact but for values that fall into e4m3's
// subnormals; and a value is a bf16 number exactly (four significant bits), so rows read
// back and the keys' expansion are those of a bf16 cache, bit for bit. It is an fp16 number as well
// (below 2^-14 rounded to multiples of 2^-24), which the decode takes: codes widen to fp16 in two
// instructions for four, and weights in fp16 carry three bits more than in bf16.
#pragma once

#include "mla_internal.cuh"

namespace mla {

constexpr int kGroups = 5;
constexpr int kEntryBytes = 8;
// The least power is 2^(17 - 127): all products with codes then are normal fp32 and
// bf16 numbers. (Values below 2^-120 become zeros.)
constexpr int kLeastPower = 17;

// the powers of a cache; null: no block scales. shift: log2 of a block's tokens
struct BlockScales {
  uint8_t* entries;
  int shift;
};
inline bool block_tokens_ok(int n) { return n == 16 || n == 32 || n == 64; }
inline int block_shift(int n) { return n == 16 ? 4 : n == 32 ? 5 : 6; }

// 127 + the smallest power e with top <= 448 * 2^e (448 = 1.75 * 2^8), from the bits of
// a finite fp32 top >= 0; at least kLeastPower. (top at most bf16's largest: the byte is at most 247.)
__device__ __forceinline__ uint32_t power_of(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23) - 8 + ((top_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, kLeastPower);
}
// 2^(b - 127) of a power's byte, fp32 (b in [1, 254])
__device__ __forceinline__ float step_of(uint32_t b) { return __uint_as_float(b << 23); }

// Rows of a chunk (rows [T][576] bf16; chunk.cuh) quantised into their pages.
cudaError_t launch_write_kv(const uint16_t* rows, uint8_t* cache, const BlockScales& scales, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu, int B, int T, int num_pages, int page_size,
                            int max_pages, int32_t* err_word, cudaStream_t s);
// append_chunk into a block-scaled cache
size_t append_blocks_workspace_bytes(int T, int d_model);
cudaError_t launch_append_blocks(const uint16_t* h, const uint16_t* w_dkr, uint8_t* cache, const BlockScales& scales,
                                 const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                                 int d_model, int num_pages, int page_size, int max_pages, double theta,
                                 void* workspace, int32_t* err_word, cudaStream_t s);
// read_kv on a block-scaled cache
cudaError_t launch_read_blocks(const uint8_t* cache, const BlockScales& scales, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* out, int B,
                               int n_rows, int num_pages, int page_size, int max_pages, int32_t* err_word,
                               cudaStream_t s);
// decode on a block-scaled cache; q_abs bf16, or fp16 with q_f16 (a chunk's rows: fp16 always)
cudaError_t launch_decode_blocks(const uint16_t* q_abs, bool q_f16, const uint8_t* cache, const BlockScales& scales,
                                 const int32_t* block_table, int B, int n_q, int H, int num_pages, int page_size,
                                 int max_pages, float scale, int G, const Plan& plan, int32_t* err_word,
                                 cudaStream_t s);

#if MLA_DEBUG_CHECKS
// Test builds only: the wait limit, the producer switch and the counters (n < 0: set to zero) of the
// block-scaled decode (null: as they are).
cudaError_t debug_decode_blocks(const long long* limit, const int* skip_producer, unsigned long long* counters, int n);
#endif

// Page tables (update_pages.cu)
struct Pages {
  int32_t* block_table;   // [B][max_pages]
  int32_t* held;          // [B]
  const int32_t* lens;    // [B]
  int32_t* free_pages;    // [num_pages]
  int32_t* free_count;    // [1]
  const int32_t* cu;      // [B + 1] or null
  int64_t* slots;         // [n_rows] or null
  int B, n_rows, num_pages, page_shift, max_pages;  // page_shift: log2 of the tokens of a page
};
cudaError_t launch_update_pages(const Pages& p, int32_t* err_word, cudaStream_t s);

}  // namespace mla

// Rows of the sequences read back from their pages into one bf16 array: row
// cu[b] + i is token first[b] + i of sequence b (zeros at and past the context's
// end), an FP8 row as bf16(scales[d] * e4m3(code)), a row of a block-scaled cache as
// code * 2^power (exact in bf16).
//
// A copy: HBM-bound, each cached byte read once and each output byte written
// once. One thread owns one 8-value column group of every fourth row of its
// block's rows, so the FP8 scales of its columns stay in registers, a row's 72
// groups are contiguous across threads (16-byte accesses, 8-byte code reads)
// and eight rows' loads are in flight per thread. The block first finds the
// source of each of its rows (search in cu, one block-table entry).
// 4 x 131072 rows of a bf16 cache: 176 us, 6.86 TB/s, the measured copy rate; a few
// hundred rows: 3.2 us, the latency of one launch and three dependent reads.
// 4 x 65536 rows of a block-scaled cache: 69.7 us, 6.5 TB/s; 2000 rows of seven sequences 3.3 us.
#include "blocks.cuh"
#include "chunk.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kGroups = kRow / 8;             // 72 groups of 8 values per row
constexpr int kRowsAtOnce = 4;
constexpr int kThreads = kGroups * kRowsAtOnce;  // 288
constexpr int kInFlight = 8;

// kF16: fp16 rows instead of bf16 (the workspace of attend_chunk). kBlocks: codes with an
// 8-byte entry of powers for each block of 1 << shift rows (blocks.cuh) in place of scales.
template <bool kF8, bool kF16, bool kBlocks, int kRows>
__global__ void __launch_bounds__(kThreads)
read_kv_kernel(const void* __restrict__ cache, const float* __restrict__ scales, const int32_t* __restrict__ block_table,
               const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ first, const int32_t* __restrict__ cu,
               uint4* __restrict__ out, int B, int n_rows, int num_pages, int page_size, int max_pages,
               int32_t* err_word, const uint8_t* __restrict__ entries, int shift) {
  __shared__ int64_t src[kRows];  // row of the pool; -1 zeros, -2 not a sequence's row
  __shared__ uint2 entry[kBlocks ? kRows : 1];  // the row's block's
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int t0 = blockIdx.x * kRows;
  for (int i = threadIdx.x; i < kRows; i += kThreads) {
    int64_t r = -2;
    const int t = t0 + i;
    const int b = t < n_rows ? row_sequence(cu, B, t) : -1;
    if (b >= 0) {
      const int64_t pos = (int64_t)(t - cu[b]) + (first ? first[b] : 0);
      const int max_tokens = max_pages * page_size, raw = seq_lens[b];
      const int L = min(max(raw, 0), max_tokens);
      if (raw != L || pos < 0) report_error(err_word, MLA_ERR_BOUNDS);
      r = -1;
      if (pos >= 0 && pos < L) {
        const int page = block_table[(int64_t)b * max_pages + pos / page_size];
        if (page >= 0 && page < num_pages)
          r = (int64_t)page * page_size + pos % page_size;
        else
          report_error(err_word, MLA_ERR_BOUNDS);
      }
    }
    src[i] = r;
    if (kBlocks && r >= 0) entry[i] = __ldg(reinterpret_cast<const uint2*>(entries) + (r >> shift));
  }
  if (blockIdx.x == 0) report_rows(cu, B, n_rows, threadIdx.x, kThreads, err_word);
  const int g = threadIdx.x % kGroups, r0 = threadIdx.x / kGroups;
  float sc[8];
  if (kF8 && !kBlocks) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sc[i] = __ldg(scales + 8 * g + i);
  }
  __syncthreads();
  float top = 0.f;
  constexpr int kPer = kRows / kRowsAtOnce;
  constexpr int kStep = kPer < kInFlight ? kPer : kInFlight;
#pragma unroll 1
  for (int k0 = 0; k0 < kPer; k0 += kStep) {
    uint4 v[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const int64_t s = src[(k0 + k) * kRowsAtOnce + r0];
      v[k] = make_uint4(0, 0, 0, 0);
      if (s >= 0) {
        if (kF8) {
          const uint2 c = __ldg(static_cast<const uint2*>(cache) + s * kGroups + g);
          v[k].x = c.x;
          v[k].y = c.y;
        } else {
          v[k] = __ldg(static_cast<const uint4*>(cache) + s * kGroups + g);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const int i = (k0 + k) * kRowsAtOnce + r0;
      if (src[i] == -2) continue;
      uint4 o = v[k];
      if (kF8) {
        // e4m3 -> fp16 (exact) -> fp32, times the scale in fp32, rounded once to bf16
        const uint32_t w[2] = {v[k].x, v[k].y};
        uint32_t f[4], p[4];
        const float step =
            kBlocks ? step_of(reinterpret_cast<const uint8_t*>(entry)[8 * i + (g < 64 ? g >> 4 : 4)]) : 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
              "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
              : "=r"(f[2 * q]), "=r"(f[2 * q + 1])
              : "r"(w[q]));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 x = sm100::f16x2_to_f32(f[q]);
          const float s0 = kBlocks ? step : sc[2 * q], s1 = kBlocks ? s0 : sc[2 * q + 1];
          const float a = x.x * s0, b = x.y * s1;
          p[q] = kF16 ? sm100::cvt_f16x2(a, b) : sm100::cvt_bf16x2(a, b);
          if (kF16 && src[i] >= 0) top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
        }
        o = make_uint4(p[0], p[1], p[2], p[3]);
        if (src[i] == -1) o = make_uint4(0, 0, 0, 0);  // 0 x scale, whatever the scale
      }
      out[(int64_t)(t0 + i) * kGroups + g] = o;
    }
  }
  if (kF16 && top >= 65520.f && top < INFINITY) report_error(err_word, MLA_ERR_RANGE);
}

constexpr int kWThreads = 256;
__global__ void __launch_bounds__(kWThreads)
weights_f16_kernel(const uint4* __restrict__ w_uk, const uint4* __restrict__ w_uv, uint4* __restrict__ out, int n8,
                   int32_t* err_word) {
  sm100::grid_launch_dependents();  // the next kernel reads the copies after its own dependency wait
  sm100::grid_dependency_wait();    // the workspace may still be in use
  const int i = blockIdx.x * kWThreads + threadIdx.x;
  if (i >= 2 * n8) return;
  const uint4 w = i < n8 ? __ldg(w_uk + i) : __ldg(w_uv + (i - n8));
  uint32_t top = 0;
  out[i] = bf16x8_to_f16(w, &top);
  if (top >= kF16Limit && top < 0x7F800000u) report_error(err_word, MLA_ERR_RANGE);
}

template <bool kF8, bool kF16, bool kBlocks, int kRows>
cudaError_t launch(const void* cache, const float* scales, const int32_t* block_table, const int32_t* seq_lens,
                   const int32_t* first, const int32_t* cu, uint16_t* out, int B, int n_rows, int num_pages,
                   int page_size, int max_pages, int32_t* err_word, cudaStream_t s,
                   const BlockScales& blocks = BlockScales{nullptr, 0}) {
  return launch_pdl(read_kv_kernel<kF8, kF16, kBlocks, kRows>, dim3((n_rows + kRows - 1) / kRows), dim3(kThreads), 0,
                    s, cache,
                    scales, block_table, seq_lens, first, cu, reinterpret_cast<uint4*>(out), B, n_rows, num_pages,
                    page_size, max_pages, err_word, static_cast<const uint8_t*>(blocks.entries), blocks.shift);
}

}  // namespace

cudaError_t launch_read_kv(const void* cache, const float* fp8_scales, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* out, int B,
                           int n_rows, int num_pages, int page_size, int max_pages, int32_t* err_word,
                           cudaStream_t s) {
  return fp8_scales ? launch<true, false, false, 32>(cache, fp8_scales, block_table, seq_lens, first, cu, out, B,
                                                     n_rows, num_pages, page_size, max_pages, err_word, s)
                    : launch<false, false, false, 32>(cache, fp8_scales, block_table, seq_lens, first, cu, out, B,
                                                      n_rows, num_pages, page_size, max_pages, err_word, s);
}

cudaError_t launch_read_blocks(const uint8_t* cache, const BlockScales& scales, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* first, const int32_t* cu, uint16_t* out, int B,
                               int n_rows, int num_pages, int page_size, int max_pages, int32_t* err_word,
                               cudaStream_t s) {
  return launch<true, false, true, 32>(cache, nullptr, block_table, seq_lens, first, cu, out, B, n_rows, num_pages,
                                       page_size, max_pages, err_word, s, scales);
}

cudaError_t launch_rows_f16(const void* cache8, const float* fp8_scales, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* cu, uint16_t* out, int B, int n_rows,
                            int num_pages, int page_size, int max_pages, int32_t* err_word, cudaStream_t s) {
  return launch<true, true, false, 32>(cache8, fp8_scales, block_table, seq_lens, nullptr, cu, out, B, n_rows,
                                       num_pages, page_size, max_pages, err_word, s);
}

cudaError_t launch_weights_f16(const uint16_t* w_uk, const uint16_t* w_uv, uint16_t* out, int H, int32_t* err_word,
                               cudaStream_t s) {
  const int n8 = H * kDNope * kDC / 8;  // each of the two
  return launch_pdl(weights_f16_kernel, dim3((2 * n8 + kWThreads - 1) / kWThreads), dim3(kWThreads), 0, s,
                    reinterpret_cast<const uint4*>(w_uk), reinterpret_cast<const uint4*>(w_uv),
                    reinterpret_cast<uint4*>(out), n8, err_word);
}

}  // namespace mla

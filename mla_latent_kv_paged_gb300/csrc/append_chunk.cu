// Latent-cache rows of a ragged chunk of new tokens, written into their pages as
// bf16 or, quantised as they are written, as e4m3 codes with one scale per column.
//
// What it computes (Huny's Dev Blog "MLA 아키텍처 해부" section 1.2,
// c_t^KV = h_t W^DKV, and section 2.2, k^R_t = RoPE(h_t W^KR); section 6 item 4:
// FP8 on the latent needs per-channel scales): for row t of sequence b at
// position pos = L_b - n_b + (t - cu[b]),
//   row[i] = sum_k h[t][k] w_dkr[i][k], the pairs from column 512 on rotated
//   cache row = bf16(row[i])   or   e4m3(row[i] / scales[i]), saturating
// The quotient is taken from the fp32 sum: a row is rounded once.
//
// A GEMM [T x d_model] x [d_model x 576]: weight-streaming for a few rows,
// tensor-bound for a prompt. A pair of CTAs (M = 256 MMAs over two SMs) computes 256
// rows x 288 columns (two column tiles; the positional columns lie in the second)
// over a slice of d_model, each CTA loading its 128 rows of h and half of the
// tile's weights through a six-stage TMA ring: 34 KB per 64-wide block and CTA
// (one CTA on its own with 128 x 192 took 40 KB per third of that work and was
// bound by what L2 delivers, 11.6 TB/s: 88 us for 9700 rows of 7168). When the
// tiles alone do not fill the SMs the reduction over d_model is split: each split
// writes fp32 partials and a second kernel adds them in split order (results are
// bit-reproducible), rotates, quantises and scatters; with one split the GEMM's own
// epilogue does that.
#include <math.h>

#include "blocks.cuh"
#include "chunk.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kN = 288;               // output columns of a pair, as two MMAs of 144
constexpr int kHalfN = kN / 2;
constexpr int kColTiles = kRow / kN;  // 2
constexpr int kM = 128;               // rows per CTA, 256 per pair
constexpr int kStages = 6;
constexpr uint32_t kABytes = kM * 128;
constexpr uint32_t kBBox = kHalfN / 2 * 128;  // this CTA's 72 of an MMA's 144 columns
constexpr uint32_t kStageBytes = kABytes + 2 * kBBox;
constexpr uint32_t kOffBar = kStages * kStageBytes;
constexpr uint32_t kOffFreq = kOffBar + (2 * kStages + 2) * 8;  // 8-byte aligned
constexpr uint32_t kOffSlots = kOffFreq + 32 * 8;
constexpr uint32_t kSmem = kOffSlots + 16;
static_assert(kStageBytes % 1024 == 0 && kSmem <= 232448, "shared memory");
constexpr uint32_t kTmCols = 512;
constexpr int kThreads = 320;  // warps 0..7 epilogue, 8 producer, 9 MMA issuer
constexpr int kPairs = 76;     // one pair per two SMs

struct Shape {
  int tiles, KB, S;
};
// Splits of the d_model reduction: the cheapest by a count fitted to measured times, in
// 64-wide blocks of a pair (0.31 us): a wave's blocks, 16 for a further wave, and beside
// them 21 for one split, else 16 for the two launches, the partial sums' way out and
// back, 0.0187 a row and 0.0013 a row and split, and 0.12 a split. A function of
// (T, d_model) only. In us on the GPU, d_model 7168 (splits: time): 32 rows 1: 37.2,
// 8: 9.6, 24: 7.0, 38: 7.9; 512 rows 1: 40.4, 4: 17.1, 12: 12.2, 19: 14.9; 2048 rows
// 1: 40.9, 2: 36.4, 4: 29.8, 5 (a second wave): 42.8; 4096 rows 1: 41.2, 2: 50.4.
inline Shape shape_of(int T, int d_model) {
  Shape a;
  a.tiles = (T + 2 * kM - 1) / (2 * kM);
  a.KB = d_model / 64;
  double best = 0.;
  a.S = 1;
  for (int S = 1; S <= kPairs / kColTiles && 2 * S <= (a.KB > 1 ? a.KB : 2); ++S) {
    const int64_t waves = ((int64_t)a.tiles * kColTiles * S + kPairs - 1) / kPairs;
    const double cost = (double)waves * ((a.KB + S - 1) / S) + 16. * (double)(waves - 1) +
                        (S > 1 ? 16. + 0.0187 * T + 0.0013 * T * S + 0.12 * S : 21.);
    if (S == 1 || cost < best) {
      best = cost;
      a.S = S;
    }
  }
  return a;
}

// Fraction of a turn per position of positional pair i, in units of 2^-64 turns:
// theta^(-2i/64) / (2 pi). pos times it modulo 2^64 is the angle's fraction of a
// turn, exact to 2^-64 pos + the double's rounding, whatever the position.
__device__ __forceinline__ uint64_t turn_fraction(double theta, int i) {
  return __double2ull_rn(pow(theta, -2.0 * (double)i / kDR) * 0.15915494309189535 * 18446744073709551616.0);
}
// The turn is taken apart into the nearest quarter and the rest, so that a sine or cosine
// that is small keeps fp32's relative precision: within 2^-22 of itself, and 2^-32 of a
// turn in the angle. (With __sincosf, 2^-21 whatever the size, small ones were off by
// more than their bf16 rounding; it is no faster here.)
__device__ __forceinline__ void turn_of(uint64_t per_pos, int pos, float& sn, float& cs) {
  const uint32_t turn = (uint32_t)((per_pos * (uint64_t)(uint32_t)pos + 0x80000000u) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  sincospif((float)(int32_t)(turn - (quarter << 30)) * 0x1p-31f, &sn, &cs);
  if (quarter & 1u) {
    const float t = sn;
    sn = cs;
    cs = -t;
  }
  if (quarter & 2u) {
    sn = -sn;
    cs = -cs;
  }
}
__device__ __forceinline__ void rotate(float& x, float& y, float sn, float cs) {
  const float rx = x * cs - y * sn;
  y = x * sn + y * cs;
  x = rx;
}
// two values -> two e4m3 codes (lo in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The codes of fp32's quotients x / s, as mla_quantize_fp8's.
__device__ __forceinline__ uint32_t quantise2(float x, float y, float sx, float sy) {
  return e4m3x2(__fdiv_rn(x, sx), __fdiv_rn(y, sy));
}
// The codes of 16 columns. Approximate quotients first, where every scale of the tile is
// in [2^-126, 2^126] (`plain`): they are within two units in the last place then. One
// surely has the exact quotient's code if it is no e4m3 subnormal (below 2^-6) and is
// more than three units from the middle of two codes (half of the 2^20 units between
// them). If one of the 16 may not, all are divided again (one in fifteen groups of a warp
// at scales of five standard deviations). 9.7k rows of 7168: 50 us; with 144 divisions a
// thread 54, with none 49.
__device__ __forceinline__ uint4 quantise16(const uint32_t (&r)[16], const float* __restrict__ scales, bool plain) {
  uint32_t w[4], apart = ~0u;
  float low = INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 sc = __ldg(reinterpret_cast<const float4*>(scales) + q);
    const float s[4] = {sc.x, sc.y, sc.z, sc.w};
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __fdividef(__uint_as_float(r[4 * q + e]), s[e]);
      low = fminf(low, fabsf(v[e]));
      apart = min(apart, (__float_as_uint(v[e]) - 0x80000u + 3u) & 0xFFFFFu);
    }
    w[q] = e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16;
  }
  if (!plain || low < 0x1p-6f || apart <= 6u) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 sc = __ldg(reinterpret_cast<const float4*>(scales) + q);
      w[q] = quantise2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]), sc.x, sc.y) |
             quantise2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]), sc.z, sc.w) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Target {
  int64_t row;  // row of the pool, or -1
  int pos;
};
// Where row t goes. A row whose sequence's length does not hold the new rows or passes
// the block table, whose sequence has rows outside the array, or whose page id is out of
// range, is reported and not written (a clamped length would put it over another token's
// row); a row of no sequence is not written.
__device__ Target target_of(const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                            const int32_t* __restrict__ block_table, int B, int T, int t, int num_pages,
                            int page_size, int max_pages, bool report, int32_t* err_word) {
  Target r = {-1, 0};
  const int b = row_sequence(cu, B, t);
  if (b < 0) return r;
  const int first = cu[b], end = cu[b + 1], L = seq_lens[b];
  bool bad = first < 0 || end > T || L < end - first || L > max_pages * page_size;
  if (!bad) {
    const int pos = L - (end - t);
    const int page = block_table[(int64_t)b * max_pages + pos / page_size];
    if (page >= 0 && page < num_pages)
      r = {(int64_t)page * page_size + pos % page_size, pos};
    else
      bad = true;
  }
  if (bad && report) report_error(err_word, MLA_ERR_BOUNDS);
  return r;
}

struct Args {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu;
  const float* scales;  // null: bf16 cache
  void* cache;
  float* partials;
  int32_t* err_word;
  double theta;
  int B, T, KB, S, num_pages, page_size, max_pages;
  bool dense;  // row t goes to row t of `cache` (the rows of a block-scaled cache, quantised after)
};

template <bool kDirect, bool kF8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
append_chunk_gemm(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h, Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int nt = blockIdx.x >> 1, s = blockIdx.y, tile = blockIdx.z;
  const int t0 = (2 * tile + (int)rank) * kM;  // this CTA's first row
  const int kb0 = (int)((int64_t)s * a.KB / a.S), nkb = (int)((int64_t)(s + 1) * a.KB / a.S) - kb0;
  auto full = [&](int i) { return sbase + kOffBar + 8u * i; };
  auto empty = [&](int i) { return sbase + kOffBar + 8u * (kStages + i); };
  const uint32_t bar_d = sbase + kOffBar + 8u * 2 * kStages;
  uint64_t* freq = reinterpret_cast<uint64_t*>(smem + kOffFreq);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffSlots + 4);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) report_error(a.err_word, MLA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    mbar_init(bar_d, 1);
    mbar_init(bar_d + 8, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish_pair();
  }
  if (kDirect && warp == 0) freq[lane] = turn_fraction(a.theta, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any copy or arrive across the pair
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    if (elect()) {
      prefetch_tmap(&map_w);
      prefetch_tmap(&map_h);
      const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
      // the pair's copies complete on the even CTA's barriers, which it arms for both
      auto weights = [&](int st, int k) {
        if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * kStageBytes);
        for (int m = 0; m < 2; ++m)
          tma_load_2d_pair(sbase + st * kStageBytes + kABytes + m * kBBox, &map_w, mapa(full(st), 0), (kb0 + k) * 64,
                           nt * kN + m * kHalfN + (int)rank * (kHalfN / 2), keep);
      };
      // the first stages' weights while the kernel before is finishing (weights
      // are never its output); the hidden states after the wait
      const int skip = skip_loads(), loads = skip == 1 || (skip == 2 && rank == 1) ? 0 : nkb;
      const int early = loads < kStages ? loads : kStages;
      for (int k = 0; k < early; ++k) weights(k, k);
      grid_dependency_wait();
      int k = 0;
      for (; k < loads; ++k) {
        const int st = k % kStages;
        if (k >= kStages) {
          if (!wait_phase(empty(st), (uint32_t)((k / kStages - 1) & 1), abort_flag, a.err_word)) break;
          weights(st, k);
        }
        tma_load_2d_pair(sbase + st * kStageBytes, &map_h, mapa(full(st), 0), (kb0 + k) * 64, t0, stream);
      }
      if (rank == 0) {
        // let the pair's copies in flight land before the pair can exit, whoever gives up
        // and whenever (the odd CTA waits for this one below; where it issued fewer, the
        // limit ends the wait)
        const long long start = clock64();
        for (int i = k > kStages ? k - kStages : 0; i < k; ++i)
          while (!mbar_try_wait(full(i % kStages), (uint32_t)((i / kStages) & 1)) &&
                 clock64() - start < wait_limit()) {
          }
      }
    }
  } else if (warp == 9) {
    if (rank == 0 && elect()) {
      const uint32_t idesc = idesc_bf16(2 * kM, kHalfN, false, false);
      const uint64_t d0 = smem_desc(0, 16, 1024, kSwizzle128B);
      auto da = [](uint32_t addr) -> uint64_t { return (uint64_t)((addr >> 4) & 0x3FFFu); };
      for (int k = 0; k < nkb; ++k) {
        const int st = k % kStages;
        if (!wait_phase(full(st), (uint32_t)((k / kStages) & 1), abort_flag, a.err_word)) break;
        tc_fence_after();
        const uint64_t ad = d0 + da(sbase + st * kStageBytes), bd = d0 + da(sbase + st * kStageBytes + kABytes);
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            mma_ss_pair(tmem + m * 256, ad + 2 * k4, bd + (m * kBBox >> 4) + 2 * k4, idesc, (k > 0 || k4 > 0) ? 1u : 0u);
        mma_commit_pair(empty(st), 3);
      }
      mma_commit_pair(bar_d, 3);
      mma_commit_pair(bar_d + 8, 1);
      wait_mmas(bar_d + 8);
    }
  } else {
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x == 0 && s == 0 && tile == 0) report_rows(a.cu, a.B, a.T, threadIdx.x, 256, a.err_word);
    // a warp per 32 rows and every other 16 columns
    const int row = (warp & 3) * 32 + lane, t = t0 + row;
    Target to = {-1, 0};
    if (kDirect && t < a.T)
      to = target_of(a.cu, a.seq_lens, a.block_table, a.B, a.T, t, a.num_pages, a.page_size, a.max_pages,
                     nt == 0, a.err_word);
    if (a.dense && to.row >= 0) to.row = t;
    bool plain = true;  // the tile's scales, see quantise16
    for (int i = lane; kDirect && kF8 && i < kN; i += 32) {
      const float v = fabsf(__ldg(a.scales + nt * kN + i));
      plain = plain && v >= 0x1p-126f && v <= 0x1p126f;
    }
    plain = __all_sync(0xffffffffu, plain);
    if (__all_sync(0xffffffffu, wait_phase(bar_d, 0, abort_flag, a.err_word))) {
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      auto tcol = [&](int c) { return taddr + (c < kHalfN ? c : 256 + c - kHalfN); };
      if (!kDirect) {
        // fp32 partials, 128 bytes of a row at a time, transposed in quads so that a
        // store covers whole lines
        float* part = a.partials + ((size_t)(2 * tile + (int)rank) * a.S + s) * kM * kRow + nt * kN + 8 * (lane & 3);
#pragma unroll 1
        for (int c0 = 32 * (warp >> 2); c0 < kN; c0 += 64) {
          uint32_t r[32];
          tmem_ld16(tcol(c0), *reinterpret_cast<uint32_t(*)[16]>(r));
          tmem_ld16(tcol(c0 + 16), *reinterpret_cast<uint32_t(*)[16]>(r + 16));
          tmem_wait_ld();
          quad_transpose(r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rk = (row & ~3) + k;
            if (t0 + rk < a.T) st_global_32(part + (size_t)rk * kRow + c0, r + 8 * k);
          }
        }
      }
#pragma unroll 1
      for (int c0 = 16 * (warp >> 2); kDirect && c0 < kN; c0 += 32) {
        uint32_t r[16];
        tmem_ld16(tcol(c0), r);
        tmem_wait_ld();
        const int col = nt * kN + c0;
        if (to.row >= 0) {
          if (col >= kDC) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {  // the pairs pass through the first two registers
              float x = __uint_as_float(r[0]), y = __uint_as_float(r[1]);
              float sn, cs;
              turn_of(freq[(col - kDC) / 2 + i], to.pos, sn, cs);
              rotate(x, y, sn, cs);
#pragma unroll
              for (int q = 0; q < 14; ++q) r[q] = r[q + 2];
              r[14] = __float_as_uint(x);
              r[15] = __float_as_uint(y);
            }
          }
          if (kF8) {
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.cache) + to.row * kRow + col) =
                quantise16(r, a.scales + col, plain);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.cache) + to.row * kRow + col);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = cvt_bf16x2(__uint_as_float(r[8 * q + 2 * e]), __uint_as_float(r[8 * q + 2 * e + 1]));
              dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the pair is under way: MMAs, copies, arrives
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmCols);
  }
}

// Row t: the split partials added in order, the positional pairs rotated, the
// row written. Thread c handles columns 2c and 2c + 1.
template <bool kF8>
__global__ void __launch_bounds__(kRow / 2)
append_chunk_finalize(Args a) {
  const int t = blockIdx.x, c = threadIdx.x, col = 2 * c;
  const uint64_t per_pos = col >= kDC ? turn_fraction(a.theta, (col - kDC) / 2) : 0;
  // the GEMM before passed its own dependency wait before this kernel could
  // start, so the lengths and tables are final; the partials are not
  Target to = target_of(a.cu, a.seq_lens, a.block_table, a.B, a.T, t, a.num_pages, a.page_size, a.max_pages, c == 0,
                        a.err_word);
  if (a.dense && to.row >= 0) to.row = t;
  float sn = 0.f, cs = 1.f;
  if (col >= kDC) turn_of(per_pos, to.pos, sn, cs);
  grid_dependency_wait();
  grid_launch_dependents();
  if (to.row < 0) return;
  const float2* p =
      reinterpret_cast<const float2*>(a.partials + (((size_t)(t / kM) * a.S) * kM + t % kM) * kRow + col);
  constexpr size_t kStep = (size_t)kM * kRow / 2;
  float x = 0.f, y = 0.f;
  constexpr int kInFlight = 16;
  for (int s0 = 0; s0 < a.S; s0 += kInFlight) {
    float2 v[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (s0 + k < a.S) v[k] = __ldcg(p + (size_t)(s0 + k) * kStep);
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (s0 + k < a.S) {
        x += v[k].x;
        y += v[k].y;
      }
  }
  if (col >= kDC) rotate(x, y, sn, cs);
  if (kF8) {
    const float2 sc = __ldg(reinterpret_cast<const float2*>(a.scales) + c);
    reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.cache) + to.row * kRow)[c] =
        (uint16_t)quantise2(x, y, sc.x, sc.y);
  } else {
    reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.cache) + to.row * kRow)[c] = cvt_bf16x2(x, y);
  }
}

template <bool kDirect, bool kF8>
cudaError_t launch_gemm(const CUtensorMap& mw, const CUtensorMap& mh, const Shape& sh, const Args& a, cudaStream_t s) {
  cudaError_t e = smem_limit<append_chunk_gemm<kDirect, kF8>>(kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(append_chunk_gemm<kDirect, kF8>, dim3(2 * kColTiles, sh.S, sh.tiles), dim3(kThreads), kSmem, s, mw, mh,
                    a);
}

}  // namespace

size_t append_chunk_workspace_bytes(int T, int d_model) {
  const Shape sh = shape_of(T, d_model);
  return 256 + (sh.S > 1 ? (size_t)sh.tiles * 2 * sh.S * kM * kRow * 4 : 0);
}

size_t append_blocks_workspace_bytes(int T, int d_model) {
  return append_chunk_workspace_bytes(T, d_model) + (size_t)T * kRow * 2;
}

namespace {
cudaError_t launch_rows(const uint16_t* h, const uint16_t* w_dkr, void* cache, bool dense, const float* fp8_scales,
                        const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                        int d_model, int num_pages, int page_size, int max_pages, double theta, void* workspace,
                        int32_t* err_word, cudaStream_t s) {
  const Shape sh = shape_of(T, d_model);
  CUtensorMap mw, mh;
  const uint64_t dw[2] = {(uint64_t)d_model, (uint64_t)kRow}, dh[2] = {(uint64_t)d_model, (uint64_t)T};
  const uint64_t st[1] = {(uint64_t)d_model * 2};
  const uint32_t bw[2] = {64, kHalfN / 2}, bh[2] = {64, kM};
  if (!make_tmap(&mw, w_dkr, 2, dw, st, bw, 128) || !make_tmap(&mh, h, 2, dh, st, bh, 128))
    return cudaErrorInvalidValue;
  Args a = {};
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu = cu;
  a.scales = fp8_scales;
  a.cache = cache;
  a.partials = reinterpret_cast<float*>(workspace_base(workspace));
  a.err_word = err_word;
  a.theta = theta;
  a.B = B;
  a.T = T;
  a.KB = sh.KB;
  a.S = sh.S;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.dense = dense;
  if (sh.S == 1)
    return fp8_scales ? launch_gemm<true, true>(mw, mh, sh, a, s) : launch_gemm<true, false>(mw, mh, sh, a, s);
  cudaError_t e = launch_gemm<false, false>(mw, mh, sh, a, s);
  if (e != cudaSuccess) return e;
  return fp8_scales ? launch_pdl(append_chunk_finalize<true>, dim3(T), dim3(kRow / 2), 0, s, a)
                    : launch_pdl(append_chunk_finalize<false>, dim3(T), dim3(kRow / 2), 0, s, a);
}
}  // namespace

cudaError_t launch_append_chunk(const uint16_t* h, const uint16_t* w_dkr, void* cache, const float* fp8_scales,
                                const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                                int d_model, int num_pages, int page_size, int max_pages, double theta,
                                void* workspace, int32_t* err_word, cudaStream_t s) {
  return launch_rows(h, w_dkr, cache, false, fp8_scales, block_table, seq_lens, cu, B, T, d_model, num_pages, page_size,
                     max_pages, theta, workspace, err_word, s);
}

// The rows in bf16 first (a block's power needs all of its rows), then quantised.
cudaError_t launch_append_blocks(const uint16_t* h, const uint16_t* w_dkr, uint8_t* cache, const BlockScales& scales,
                                 const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu, int B, int T,
                                 int d_model, int num_pages, int page_size, int max_pages, double theta,
                                 void* workspace, int32_t* err_word, cudaStream_t s) {
  // behind the partial sums (a multiple of 256 bytes)
  uint16_t* rows =
      reinterpret_cast<uint16_t*>(workspace_base(workspace) + append_chunk_workspace_bytes(T, d_model) - 256);
  cudaError_t e = launch_rows(h, w_dkr, rows, true, nullptr, block_table, seq_lens, cu, B, T, d_model, num_pages,
                              page_size, max_pages, theta, workspace, err_word, s);
  if (e != cudaSuccess) return e;
  return launch_write_kv(rows, cache, scales, block_table, seq_lens, cu, B, T, num_pages, page_size, max_pages,
                         err_word, s);
}

#if MLA_DEBUG_CHECKS
cudaError_t debug_append_chunk(const long long* limit, const int* skip) { return sm100::debug_set(limit, skip); }
#endif

}  // namespace mla

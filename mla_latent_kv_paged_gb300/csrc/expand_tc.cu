// Keys and values of every head expanded from the cached latents, for the
// attention of a chunk of new tokens (attend_tc.cu):
//   k[h][s][i] = sum_c row_s[c] w_uk[h][i][c]      v[h][s][i] = sum_c row_s[c] w_uv[h][i][c]
// (Huny's Dev Blog "MLA 아키텍처 해부" section 1.2, k^C = c W^UK, v^C = c W^UV),
// bf16 operands (fp16 for an FP8 cache), fp32 sums, rounded once to fp16: three more
// mantissa bits than bf16 for the two products that follow, |value| < 65520 (beyond:
// MLA_ERR_RANGE).
//
// Tensor-bound: 2 x 512 x 256 flop per (token, head). A pair of CTAs (one
// M = 256, N = 256 MMA over two SMs) keeps 2 x 128 tokens' latents in shared
// memory (128 KB each) and streams the weights of consecutive heads past them:
// the even CTA holds the W_UK half of each ring slot, the odd one the W_UV half
// ([128 rows][64 columns]), so a CTA reads 128 KB of weights from L2 per 256
// tokens and head (one CTA on its own, 256 KB per 128 tokens, was bound by that
// stream: 500 us for 128 heads of 16384 tokens). Two accumulators in tensor
// memory let the write-out of one head run under the MMAs of the next. The units
// (pair of token tiles, head) are dealt out as equal contiguous runs.
//
// Half a value row that is not finite is written as zeros, with a NaN in its key row:
// the queries that see the token get NaN, those that do not are untouched (a
// zero weight times a NaN value would reach them).
//
// 16384 tokens x 128 heads: 362 us, 1520 TFLOP/s (as single CTAs 500; as pairs 403; with
// the accumulator given back before the stores 387; storing whole lines 362).
#include "chunk.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kStages = 6;
constexpr int kKB = kDC / 64;                       // 8 boxes of 64 latent columns
constexpr uint32_t kASlab = 128 * 128;              // [128 tokens][64 columns], 128B swizzle
constexpr uint32_t kABytes = 8 * kASlab;
constexpr uint32_t kBBytes = 128 * 128;             // this CTA's half of B: [128 rows][64 columns], 128B swizzle
constexpr uint32_t kOffB = kABytes, kOffBar = kOffB + kStages * kBBytes;
enum { FULL0 = 0, EMPTY0 = FULL0 + kStages, AF = EMPTY0 + kStages, AE, DF0, DE0 = DF0 + 2, MD = DE0 + 2, kBars };
constexpr uint32_t kOffSlots = kOffBar + 8 * kBars;
constexpr uint32_t kSmem = kOffSlots + 16;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kThreads = 320;  // warps 0..7 write-out, 8 producer, 9 MMA issuer

// 64 values of each lane's token as fp16 to a [32 tokens][128] tile at dst; the largest
// |value| of the lane's token as bits.
__device__ __forceinline__ uint32_t write_rows(const uint32_t (&r)[64], uint16_t* dst) {
  uint32_t top = 0, w[32];
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    top = max(top, max(r[2 * q] & 0x7FFFFFFFu, r[2 * q + 1] & 0x7FFFFFFFu));
    w[q] = cvt_f16x2(__uint_as_float(r[2 * q]), __uint_as_float(r[2 * q + 1]));
  }
  quad_transpose(w);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) st_global_32(dst + ((lane & ~3) + k) * 128 + 16 * (lane & 3), w + 8 * k);
  return top;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_kernel(const __grid_constant__ CUtensorMap map_rows, const __grid_constant__ CUtensorMap map_uk,
              const __grid_constant__ CUtensorMap map_uv, ChunkPlan plan, int h0, int heads, int64_t cap,
              uint32_t idesc, int32_t* err_word) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffSlots + 4);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) report_error(err_word, MLA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(FULL0 + i), 1);
      mbar_init(bar(EMPTY0 + i), 1);
    }
    mbar_init(bar(AF), 1);
    mbar_init(bar(AE), 1);
    mbar_init(bar(MD), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(DF0 + i), 1);
      mbar_init(bar(DE0 + i), 16);  // the write-out warps of both CTAs
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any copy or arrive across the pair
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();
  // token tiles in pairs; CTA `rank` has tile 2m + rank (past the last one: computed, not written)
  const int tiles = plan.hdr[1] / kKvTile;
  const int64_t units = (int64_t)((tiles + 1) / 2) * heads;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int64_t u0 = units * pair / pairs, u1 = units * (pair + 1) / pairs;

  if (warp == 8) {
    if (elect()) {
      prefetch_tmap(&map_rows);
      const CUtensorMap* map_w = rank == 0 ? &map_uk : &map_uv;
      prefetch_tmap(map_w);
      const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
      // the pair's copies complete on the even CTA's barriers, which it arms for both
      const uint32_t af = mapa(bar(AF), 0);
      bool ok = true;
      int it = 0, loads = 0;
      const int skip = skip_loads();
      for (int64_t u = skip == 1 || (skip == 2 && rank == 1) ? u1 : u0; u < u1 && ok; ++u) {
        const int m = (int)(u / heads), h = h0 + (int)(u % heads);
        if (skip != 3 && (u == u0 || u % heads == 0)) {  // the next tokens, once the MMAs on the last ones are done
          if (loads > 0 && !wait_phase(bar(AE), (uint32_t)((loads - 1) & 1), abort_flag, err_word)) break;
          if (rank == 0) mbar_arrive_expect_tx(bar(AF), 2 * kABytes);
          for (int c = 0; c < 8; ++c)
            tma_load_2d_pair(sbase + c * kASlab, &map_rows, af, 64 * c, (2 * m + (int)rank) * 128, stream);
          ++loads;
        }
        for (int kb = 0; kb < kKB; ++kb, ++it) {
          const int st = it % kStages;
          if (it >= kStages && !wait_phase(bar(EMPTY0 + st), (uint32_t)((it / kStages - 1) & 1), abort_flag, err_word)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(bar(FULL0 + st), 2 * kBBytes);
          tma_load_2d_pair(sbase + kOffB + st * kBBytes, map_w, mapa(bar(FULL0 + st), 0), 64 * kb, h * 128, keep);
        }
      }
      if (rank == 0) {
        // let the pair's copies in flight land before the pair can exit, whoever gives up
        // and whenever (the odd CTA waits for this one below; where it issued fewer, the
        // limit ends the wait)
        const long long t0 = clock64();
        auto land = [&](int b, int use) {
          while (!mbar_try_wait(bar(b), (uint32_t)(use & 1)) && clock64() - t0 < wait_limit()) {
          }
        };
        if (loads > 0) land(AF, loads - 1);
        for (int i = it > kStages ? it - kStages : 0; i < it; ++i) land(FULL0 + i % kStages, i / kStages);
      }
    }
  } else if (warp == 9) {
    if (rank == 0 && elect()) {
      auto da = [](uint32_t addr) -> uint64_t { return (uint64_t)((addr >> 4) & 0x3FFFu); };
      const uint64_t ad0 = smem_desc(0, 16, 1024, kSwizzle128B) + da(sbase);
      const uint64_t bd0 = smem_desc(0, 16, 1024, kSwizzle128B);
      bool ok = true;
      int it = 0, loads = 0, n = 0;
      for (int64_t u = u0; u < u1 && ok; ++u, ++n) {
        const int buf = n & 1;
        if (u == u0 || u % heads == 0) {
          if (!wait_phase(bar(AF), (uint32_t)(loads & 1), abort_flag, err_word)) break;
          ++loads;
        }
        if (n >= 2 && !wait_phase(bar(DE0 + buf), (uint32_t)(((n >> 1) - 1) & 1), abort_flag, err_word, true)) break;
        for (int kb = 0; kb < kKB; ++kb, ++it) {
          const int st = it % kStages;
          if (!wait_phase(bar(FULL0 + st), (uint32_t)((it / kStages) & 1), abort_flag, err_word)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = ad0 + (kb * kASlab >> 4), bd = bd0 + da(sbase + kOffB + st * kBBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss_pair(tmem + 256 * buf, ad + 2 * k, bd + 2 * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(bar(EMPTY0 + st), 3);
        }
        if (!ok) break;
        mma_commit_pair(bar(DF0 + buf), 3);
        if ((u + 1) % heads == 0 && u + 1 < u1) mma_commit_pair(bar(AE), 3);
      }
      mma_commit_pair(bar(MD), 1);
      wait_mmas(bar(MD));
    }
  } else {
    int n = 0;
    for (int64_t u = u0; u < u1; ++u, ++n) {
      const int m = (int)(u / heads), hh = (int)(u % heads), buf = n & 1;
      if (!__all_sync(0xffffffffu, wait_phase(bar(DF0 + buf), (uint32_t)((n >> 1) & 1), abort_flag, err_word))) break;
      tc_fence_after();
      // a warp per 32 tokens and half of the columns of keys and values; the
      // accumulator is given back before anything is stored (the remote arrive
      // releases, so it would wait for the stores)
      const int quad = warp & 3, half = warp >> 2, tile = 2 * m + (int)rank;
      const uint32_t taddr = tmem + 256 * buf + 64 * half + ((uint32_t)(quad * 32) << 16);
      const int64_t at = ((int64_t)hh * cap + (int64_t)tile * 128 + quad * 32) * 128 + 64 * half;
      uint16_t *kd = plan.k + at, *vd = plan.v + at;
      uint32_t kr[64], vr[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        tmem_ld32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(kr + c));
        tmem_ld32(taddr + 128 + c, *reinterpret_cast<uint32_t(*)[32]>(vr + c));
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa(bar(DE0 + buf), 0));
      if (tile >= tiles) continue;
      const uint32_t vtop = write_rows(vr, vd), ktop = write_rows(kr, kd);
      if (__any_sync(0xffffffffu, max(vtop, ktop) >= kF16Limit)) {
        __syncwarp();  // other lanes wrote this lane's row
        if ((vtop >= kF16Limit && vtop < 0x7F800000u) || (ktop >= kF16Limit && ktop < 0x7F800000u))
          report_error(err_word, MLA_ERR_RANGE);
        if (vtop >= kF16Limit) {
          for (int q = 0; q < 8; ++q) reinterpret_cast<uint4*>(vd + lane * 128)[q] = make_uint4(0, 0, 0, 0);
          kd[lane * 128] = 0x7FFF;  // NaN
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the pair is under way: MMAs, copies, arrives
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_expand(const ChunkPlan& plan, const uint16_t* w_uk, const uint16_t* w_uv, int H, int h0, int heads,
                          int64_t cap, bool f16, int32_t* err_word, cudaStream_t s) {
  CUtensorMap mr, mk, mv;
  const uint64_t dr[2] = {kRow, (uint64_t)cap}, sr[1] = {kRow * 2};
  const uint64_t dw[2] = {kDC, (uint64_t)H * 128}, sw[1] = {kDC * 2};
  const uint32_t br[2] = {64, 128};
  if (!make_tmap(&mr, plan.rows, 2, dr, sr, br, 128) || !make_tmap(&mk, w_uk, 2, dw, sw, br, 128) ||
      !make_tmap(&mv, w_uv, 2, dw, sw, br, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = smem_limit<expand_kernel>(kSmem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t units = (cap / kKvTile + 1) / 2 * heads;
  const int pairs = sms / 2;
  return launch_pdl(expand_kernel, dim3(2 * (unsigned)(units < pairs ? units : pairs)), dim3(kThreads), kSmem, s, mr, mk, mv,
                    plan, h0, heads, cap, f16 ? idesc_f16(256, 256, false, false) : idesc_bf16(256, 256, false, false),
                    err_word);
}

#if MLA_DEBUG_CHECKS
cudaError_t debug_expand(const long long* limit, const int* skip) { return sm100::debug_set(limit, skip); }
#endif

}  // namespace mla

// Attention of a ragged chunk of new tokens over expanded keys and values on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
// What it computes, per head and new token t at row j of a sequence with n new
// tokens and context L (Huny's Dev Blog "MLA 아키텍처 해부" section 2.2, the score
// as content plus position; section 1.2, the explicit keys and values):
//   z_s = scale (q_nope . k_s + q_rope . kr_s)     s = 0 .. L - n + j
//   out = sum_s exp(z_s - m) v_s / sum_s exp(z_s - m)
//
// A CTA takes 256 query rows of one sequence and one head as two MMA tiles of
// 128 rows and walks the keys in steps of 128, so that every key and value it
// loads serves 256 rows. Per step and tile: S = Q K^T (three 64-wide slabs: two
// of fp16 content, one of bf16 position, accumulated in one fp32 tile), the
// online softmax with a thread per row, P as fp16 into the tensor memory of S,
// O += P V. While one tile's softmax runs, the tensor cores work on the other
// tile: P0 V, the next S0, P1 V, the next S1, ...
//
// Shared memory (224 KB of slabs of 16 KB): Q 6, a ring of 5 for K and one of 3
// for V. A slab is freed by the last MMAs that read it, not a whole tile at a
// time, so the next tile's slabs have more than 1000 cycles to arrive. Tensor
// memory: S0, S1, O0, O1, 128 columns each.
//
// The running maximum is a reference that is only raised when a row exceeds it
// by 2^8 (O is then rescaled by the thread that owns the row); P is held times
// 2^7, so that fp16 keeps weights down to 2^-31 of the largest and never
// overflows (2^15). Sums are fp32, of the unrounded weights.
#include "chunk.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr uint32_t kSlab = 128 * 128;  // [128 rows][64 16-bit columns], 128B swizzle
constexpr uint32_t kVBox = 64 * 128;   // [64 keys][64 columns]
constexpr int kQSlabs = 6, kKStages = 5, kVStages = 3;
constexpr uint32_t kOffK = kQSlabs * kSlab, kOffV = kOffK + kKStages * kSlab, kOffBar = kOffV + kVStages * kSlab;
enum {
  KF0 = 0, KE0 = KF0 + kKStages, VF0 = KE0 + kKStages, VE0 = VF0 + kVStages, QF0 = VE0 + kVStages, SF0 = QF0 + 2,
  PF0 = SF0 + 2, OF0 = PF0 + 2, MD = OF0 + 2, kBars
};
constexpr uint32_t kOffX = kOffBar + 8 * kBars;  // [2 tiles][2 halves][128] half-row maxima, then sums
constexpr uint32_t kOffSlots = kOffX + 4 * 128 * 4;
constexpr uint32_t kSmem = kOffSlots + 16;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kThreads = 576;  // warps 0..15 softmax, 16 producer, 17 MMA issuer
constexpr uint32_t kTmS = 0, kTmO = 256;
constexpr float kBias = 7.0f;       // P = 2^7 exp(z - m)
constexpr float kRescale = 8.0f;    // log2 units
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// pairs of fp32 values
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_kr,
              const __grid_constant__ CUtensorMap map_v, const uint16_t* __restrict__ q_nope,
              const uint16_t* __restrict__ q_rope, uint16_t* __restrict__ out, float* __restrict__ lse, ChunkPlan plan,
              int H, int h0, int64_t cap, float sl2, int32_t* err_word) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_index();
  const int hh = blockIdx.y, h = h0 + hh;
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffSlots + 4);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) report_error(err_word, MLA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(bar(KF0 + i), 1);
      mbar_init(bar(KE0 + i), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(bar(VF0 + i), 1);
      mbar_init(bar(VE0 + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(QF0 + i), 256);
      mbar_init(bar(SF0 + i), 1);
      mbar_init(bar(PF0 + i), 256);
      mbar_init(bar(OF0 + i), 1);
    }
    mbar_init(bar(MD), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  // the piece: query rows [q0, q0 + 256) of n, steps [j0, j1) over the keys (read
  // beside the number of pieces; what lies past it is not used)
  const int4 qp = plan.piece[2 * blockIdx.x], kp = plan.piece[2 * blockIdx.x + 1];
  const bool work = (int)blockIdx.x < plan.hdr[0];
  const int q0 = qp.x, n = qp.y, c0 = qp.z, L = qp.w, j0 = kp.x, slot = kp.z;
  const int64_t k0 = kp.w + (int64_t)j0 * kKvTile;  // first expanded row of the piece
  const bool two = n - q0 > 128;
  auto steps = [&](int x) {  // of tile x in this piece: up to the last token that its last row sees
    if (!work || (x == 1 && !two)) return 0;
    return min((L - n + min(q0 + 128 * (x + 1), n) + kKvTile - 1) / kKvTile, kp.y) - j0;
  };
  const int n0 = steps(0), n1 = steps(1), nkv = max(n0, n1);

  if (warp == 16) {
    if (nkv > 0 && elect()) {
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_kr);
      prefetch_tmap(&map_v);
      const uint64_t keep = policy_evict_last();
      bool ok = true;
      int ki = 0, vi = 0;
      for (int j = 0; j < nkv && ok; ++j) {
        const int row = (int)(k0 + (int64_t)j * kKvTile), hrow = (int)((int64_t)hh * cap + row);
        for (int s = 0; s < 3; ++s, ++ki) {
          const int st = ki % kKStages;
          if (ki >= kKStages && !wait_phase(bar(KE0 + st), (uint32_t)((ki / kKStages - 1) & 1), abort_flag, err_word)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(KF0 + st), kSlab);
          if (s < 2)
            tma_load_2d(sbase + kOffK + st * kSlab, &map_k, bar(KF0 + st), 64 * s, hrow, keep);
          else
            tma_load_2d(sbase + kOffK + st * kSlab, &map_kr, bar(KF0 + st), kDC, row, keep);
        }
        for (int s = 0; s < 2 && ok; ++s, ++vi) {
          const int st = vi % kVStages;
          if (vi >= kVStages && !wait_phase(bar(VE0 + st), (uint32_t)((vi / kVStages - 1) & 1), abort_flag, err_word)) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + kOffV + st * kSlab;
          mbar_arrive_expect_tx(bar(VF0 + st), kSlab);
          tma_load_2d(dst, &map_v, bar(VF0 + st), 0, hrow + 64 * s, keep);
          tma_load_2d(dst + kVBox, &map_v, bar(VF0 + st), 64, hrow + 64 * s, keep);
        }
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA can exit
        const long long t0 = clock64();
        for (int i = ki > kKStages ? ki - kKStages : 0; i < ki; ++i)
          while (!mbar_try_wait(bar(KF0 + i % kKStages), (uint32_t)((i / kKStages) & 1)) &&
                 clock64() - t0 < kWaitLimitCycles) {
          }
        for (int i = vi > kVStages ? vi - kVStages : 0; i < vi; ++i)
          while (!mbar_try_wait(bar(VF0 + i % kVStages), (uint32_t)((i / kVStages) & 1)) &&
                 clock64() - t0 < kWaitLimitCycles) {
          }
      }
    }
  } else if (warp == 17) {
    if (nkv > 0 && elect()) {
      constexpr uint32_t kIdC = idesc_f16(128, 128, false, false), kIdR = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdV = idesc_f16(128, 128, false, true);
      auto da = [](uint32_t addr) -> uint64_t { return (uint64_t)((addr >> 4) & 0x3FFFu); };
      const uint64_t d0 = smem_desc(0, 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(0, kVBox, 1024, kSwizzle128B);
      bool ok = true;
      // S of tile x = Q K^T of step j; `last`: no other tile reads these slabs
      auto scores = [&](int x, int j, bool last) {
        for (int s = 0; s < 3 && ok; ++s) {
          const int i = 3 * j + s, st = i % kKStages;
          ok = wait_phase(bar(KF0 + st), (uint32_t)((i / kKStages) & 1), abort_flag, err_word);
          if (!ok) return;
          tc_fence_after();
          const uint64_t ad = d0 + da(sbase + (3 * x + s) * kSlab), bd = d0 + da(sbase + kOffK + st * kSlab);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + kTmS + 128 * x, ad + 2 * k, bd + 2 * k, s < 2 ? kIdC : kIdR, (s > 0 || k > 0) ? 1u : 0u);
          if (last) mma_commit(bar(KE0 + st));
        }
        mma_commit(bar(SF0 + x));
      };
      auto values = [&](int x, int j, bool last) {
        ok = wait_phase(bar(PF0 + x), (uint32_t)(j & 1), abort_flag, err_word);
        for (int s = 0; s < 2 && ok; ++s) {
          const int i = 2 * j + s, st = i % kVStages;
          ok = wait_phase(bar(VF0 + st), (uint32_t)((i / kVStages) & 1), abort_flag, err_word);
          if (!ok) return;
          tc_fence_after();
          const uint64_t bd = dv + da(sbase + kOffV + st * kSlab);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tmem + kTmO + 128 * x, tmem + kTmS + 128 * x + 32 * s + 8 * k, bd + (k * 2048 >> 4), kIdV,
                   (j > 0 || s > 0 || k > 0) ? 1u : 0u);
          if (last) mma_commit(bar(VE0 + st));
        }
      };
      ok = wait_phase(bar(QF0), 0, abort_flag, err_word);
      if (ok) scores(0, 0, !two);
      if (ok && two) {
        ok = wait_phase(bar(QF0 + 1), 0, abort_flag, err_word);
        if (ok) scores(1, 0, true);
      }
      // tile 1, when there is one, takes at least as many steps as tile 0
      for (int j = 0; j < nkv && ok; ++j) {
        if (j < n0) {
          values(0, j, !two);
          if (ok && j + 1 < n0) scores(0, j + 1, !two);
          if (ok && j + 1 == n0) mma_commit(bar(OF0));
        }
        if (ok && j < n1) {
          values(1, j, true);
          if (ok && j + 1 < n1) scores(1, j + 1, true);
          if (ok && j + 1 == n1) mma_commit(bar(OF0 + 1));
        }
      }
      mma_commit(bar(MD));
      wait_mmas(bar(MD));
    }
  } else if (nkv > 0) {
    // tile x, column half y; the row is the tensor-memory lane of this thread
    const int x = (warp >> 2) & 1, y = warp >> 3, row = threadIdx.x & 127, tid = row + 128 * y;
    const int nx = x ? n1 : n0, r0 = q0 + 128 * x;
    if (nx > 0) {
      // the tile's queries: content as fp16 (exact for bf16 values of normal fp16
      // size), position as it is, into the swizzled slabs
      // (all twelve loads of a thread in flight together)
      uint4 wn[8], wr[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = tid + 256 * k, r = i >> 4, ch = i & 15;
        wn[k] = make_uint4(0, 0, 0, 0);
        if (r0 + r < n) wn[k] = __ldg(reinterpret_cast<const uint4*>(q_nope + ((size_t)(c0 + r0 + r) * H + h) * kDNope) + ch);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = tid + 256 * k, r = i >> 3, ch = i & 7;
        wr[k] = make_uint4(0, 0, 0, 0);
        if (r0 + r < n) wr[k] = __ldg(reinterpret_cast<const uint4*>(q_rope + ((size_t)(c0 + r0 + r) * H + h) * kDR) + ch);
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = tid + 256 * k, r = i >> 4, ch = i & 15;
        const uint32_t e[4] = {wn[k].x, wn[k].y, wn[k].z, wn[k].w};
        uint32_t f[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f[q] = cvt_f16x2(bf16_lo(e[q]), bf16_hi(e[q]));
          top = max(top, max((e[q] << 16) & 0x7FFFFFFFu, e[q] & 0x7FFF0000u));
        }
        st_shared_v4(sbase + (3 * x + (ch >> 3)) * kSlab + r * 128 + (((ch & 7) ^ (r & 7)) << 4), f[0], f[1], f[2], f[3]);
      }
      if (top >= 0x477FF000u && top < 0x7F800000u) report_error(err_word, MLA_ERR_RANGE);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = tid + 256 * k, r = i >> 3, ch = i & 7;
        st_shared_v4(sbase + (3 * x + 2) * kSlab + r * 128 + ((ch ^ (r & 7)) << 4), wr[k].x, wr[k].y, wr[k].z, wr[k].w);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(QF0 + x));

      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + kTmS + 128 * x + lane_off, tO = tmem + kTmO + 128 * x + 64 * y + lane_off;
      const int first_seen = L - n + r0 + 1;                       // tokens that the tile's first row sees
      const int seen = L - n + min(r0 + row, n - 1) + 1;           // tokens that this row sees
      volatile float* mine = reinterpret_cast<float*>(smem + kOffX) + (2 * x + y) * 128 + row;
      volatile float* theirs = reinterpret_cast<float*>(smem + kOffX) + (2 * x + (y ^ 1)) * 128 + row;
      auto meet = [&] { asm volatile("bar.sync %0, 256;" ::"r"(1 + x) : "memory"); };  // the tile's 256 threads
      float ref = -INFINITY;
      uint64_t sum2[2] = {0, 0};
      bool ok = true;
      int j = 0;
      for (; j < nx; ++j) {
        // the warp leaves together: the tensor-memory loads below need every lane
        ok = __all_sync(0xffffffffu, wait_phase(bar(SF0 + x), (uint32_t)(j & 1), abort_flag, err_word));
        tc_fence_after();
        uint32_t z[64];
        tmem_ld32(tS + 64 * y, *reinterpret_cast<uint32_t(*)[32]>(z));
        tmem_ld32(tS + 64 * y + 32, *reinterpret_cast<uint32_t(*)[32]>(z + 32));
        tmem_wait_ld();
        if ((j0 + j + 1) * kKvTile > first_seen) {
          const int lim = seen - (j0 + j) * kKvTile - 64 * y;
#pragma unroll
          for (int c = 0; c < 64; ++c) z[c] = c < lim ? z[c] : 0xFF800000u;
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = __uint_as_float(z[c]);
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m4[q] = fmaxf(m4[q], fmaxf(__uint_as_float(z[c + 2 * q]), __uint_as_float(z[c + 2 * q + 1])));
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], __uint_as_float(z[60 + c]));
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        *mine = mx;
        meet();  // also: both halves of S are in registers, P may overwrite them
        // (the next step's maxima follow its scores, which follow every thread's P)
        mx = fmaxf(mx, *theirs);
        // all MMAs issued before this step's scores are done, the last P V among them
        if (__any_sync(0xffffffffu, mx * sl2 > ref * sl2 + kRescale)) {
          const float up = fmaxf(ref, mx);
          if (j > 0) {
            const float f = ref == up ? 1.f : ex2((ref - up) * sl2);
            const uint64_t f2 = pack2(f, f);
            sum2[0] = mul2(sum2[0], f2);
            sum2[1] = mul2(sum2[1], f2);
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              uint32_t o[16];
              tmem_ld16(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
              tmem_st16(tO + c, o);
            }
          }
          ref = up;
        }
        const float off = kBias - (ref == -INFINITY ? 0.f : ref * sl2);
        const uint64_t off2 = pack2(off, off), sl22 = pack2(sl2, sl2);
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const uint64_t t = fma2(pack2(__uint_as_float(z[c + 2 * q]), __uint_as_float(z[c + 2 * q + 1])), sl22, off2);
            float a, e;
            unpack2(t, a, e);
            a = ex2(a);
            e = ex2(e);
            sum2[q & 1] = add2(sum2[q & 1], pack2(a, e));
            p[q] = cvt_f16x2(a, e);
          }
          tmem_st16(tS + 32 * y + c / 2, p);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(PF0 + x));
        if (!ok) break;
      }
      // the two halves' sums
      float s0, s1, sum;
      unpack2(add2(sum2[0], sum2[1]), s0, s1);
      sum = s0 + s1;
      if (!ok) {  // gave up: the barriers of this tile stay matched, nothing is written
        for (++j; j < nx; ++j) meet();
      }
      meet();  // the last maxima are read
      *mine = sum;
      meet();
      sum += *theirs;  // the same in both halves
      if (ok && __all_sync(0xffffffffu, wait_phase(bar(OF0 + x), 0, abort_flag, err_word))) {
        tc_fence_after();
        const bool live = r0 + row < n;
        const size_t at = (size_t)(c0 + r0 + row) * H + h;
        // a whole item: the output row; a piece of one: its sums and reference, as they are
        const float inv = slot >= 0 ? 1.f : sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN stays NaN
        const size_t pr = slot >= 0 ? ((size_t)slot * gridDim.y + hh) * kQTile + 128 * x + row : 0;
        if (slot >= 0 && y == 0) plan.ml_part[pr] = make_float2(ref == -INFINITY ? ref : ref * sl2, sum);
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          uint32_t o[32], w[16];
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
          if (slot >= 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              reinterpret_cast<uint4*>(plan.o_part + pr * kDV + 64 * y + c)[q] =
                  make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            continue;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q)
            w[q] = cvt_bf16x2(__uint_as_float(o[2 * q]) * inv, __uint_as_float(o[2 * q + 1]) * inv);
          if (live) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              reinterpret_cast<uint4*>(out + at * kDV + 64 * y + c)[q] =
                  make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          }
        }
        if (lse && live && y == 0 && slot < 0)
          lse[at] = sum > 0.f ? (ref * sl2 - kBias + log2f(sum)) * kLn2 : (sum == 0.f ? -INFINITY : sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Items that were cut over the keys: out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k,
// added in the order of the pieces. A warp per row, 16 bytes a lane; the partials of
// a row are read once (HBM or L2-bound, 512 bytes a piece).
__global__ void __launch_bounds__(256)
join_kernel(ChunkPlan plan, uint16_t* __restrict__ out, float* __restrict__ lse, int H, int h0) {
  grid_dependency_wait();
  grid_launch_dependents();
  if ((int)blockIdx.x >= plan.hdr[2]) return;
  const int4 jn = plan.join[blockIdx.x];  // {first slot, pieces, first row, rows}
  const int hh = blockIdx.y, heads = gridDim.y, lane = threadIdx.x & 31;
  for (int r = blockIdx.z * 8 + (threadIdx.x >> 5); r < jn.w; r += 8 * gridDim.z) {
    auto at = [&](int k) { return ((size_t)(jn.x + k) * heads + hh) * kQTile + r; };
    float m = -INFINITY;
    for (int k = 0; k < jn.y; ++k) m = fmaxf(m, __ldcg(&plan.ml_part[at(k)].x));
    float l = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll 4
    for (int k = 0; k < jn.y; ++k) {
      const float2 ml = __ldcg(&plan.ml_part[at(k)]);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(plan.o_part + at(k) * kDV) + lane);
      const float w = ml.x == m ? 1.f : ex2(ml.x - m);
      l = fmaf(w, ml.y, l);
      a0 = fmaf(w, o.x, a0);
      a1 = fmaf(w, o.y, a1);
      a2 = fmaf(w, o.z, a2);
      a3 = fmaf(w, o.w, a3);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const size_t row = (size_t)(jn.z + r) * H + h0 + hh;
    reinterpret_cast<uint2*>(out + row * kDV)[lane] =
        make_uint2(cvt_bf16x2(a0 * inv, a1 * inv), cvt_bf16x2(a2 * inv, a3 * inv));
    if (lse && lane == 0) lse[row] = l > 0.f ? (m - kBias + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
  }
}

}  // namespace

cudaError_t launch_attend(const ChunkPlan& plan, const uint16_t* q_nope, const uint16_t* q_rope, uint16_t* out,
                          float* lse, int B, int T, int H, int h0, int heads, int64_t cap, int slots,
                          float scale, int32_t* err_word, cudaStream_t s) {
  CUtensorMap mk, mr, mv;
  const uint64_t dk[2] = {kDNope, (uint64_t)heads * cap}, sk[1] = {kDNope * 2};
  const uint64_t dr[2] = {kRow, (uint64_t)cap}, sr[1] = {kRow * 2};
  const uint32_t bk[2] = {64, 128}, bv[2] = {64, 64};
  if (!make_tmap(&mk, plan.k, 2, dk, sk, bk, 128) || !make_tmap(&mr, plan.rows, 2, dr, sr, bk, 128) ||
      !make_tmap(&mv, plan.v, 2, dk, sk, bv, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = smem_limit<attend_kernel>(kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attend_kernel, dim3(chunk_max_items(B, T) + slots, heads), dim3(kThreads), kSmem, s, mk, mr, mv,
                 q_nope, q_rope, out, lse, plan, H, h0, cap, scale * 1.4426950408889634f, err_word);
  if (e != cudaSuccess || slots == 0) return e;
  const int joins = chunk_max_items(B, T) < slots / 2 ? chunk_max_items(B, T) : slots / 2;  // two pieces at least
  return launch_pdl(join_kernel, dim3(joins, heads, 8), dim3(256), 0, s, plan, out, lse, H, h0);
}

}  // namespace mla

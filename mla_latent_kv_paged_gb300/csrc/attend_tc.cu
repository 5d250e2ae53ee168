// Attention of a ragged chunk of new tokens over expanded keys and values on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
// What it computes, per head and new token t at row j of a sequence with n new
// tokens and context L (Huny's Dev Blog "MLA 아키텍처 해부" section 2.2, the score
// as content plus position; section 1.2, the explicit keys and values):
//   z_s = scale (q_nope . k_s + q_rope . kr_s)     s = 0 .. L - n + j
//   out = sum_s exp(z_s - m) v_s / sum_s exp(z_s - m)
//
// A work item is 256 query rows of one sequence and one head, as two MMA tiles of
// 128 rows, and a run of steps of 128 keys, so that every key and value loaded
// serves 256 rows. Per step and tile: S = Q K^T (three 64-wide slabs: two of fp16
// content, one of bf16 position, accumulated in one fp32 tile), the online softmax
// with two threads per row (64 keys each), P as fp16 into the tensor memory of S,
// O += P V. The tensor cores alternate between the tiles: [P0 V, the next S0],
// [P1 V, the next S1], each while the other tile's softmax runs.
//
// Shared memory (224 KB of slabs of 16 KB): Q 6, rings of 4 for K and V. A slab is
// freed by the last MMAs that read it, not a whole step at a time. Tensor memory:
// S0, S1, O0, O1, 128 columns each.
//
// The CTAs are persistent, one per SM, and take (piece, head) items from a counter.
// The next item's queries, keys and values follow the current one's through the same
// buffers, and the softmax warps convert the next queries before they write the
// current rows out, so the tensor cores go on (as one CTA per item, 7.3 us of start
// and end stood beside 16 us of steps for a prompt of 2048: 249 -> 229 us a call).
//
// Bound by power where it runs long: at 2048 rows on 16384 tokens x 128 heads the
// card sits at its limit (1350 W, the SM clock down to 1.70 GHz) and the call does
// 1490 TFLOP/s, 87% of what cuBLAS sustains under the same cap (this kernel 1640 us).
// On short contexts it is bound by the chain S -> softmax -> P V -> next S of each tile
// (a prompt of 2048 x 128 heads: 146 us, the tensor pipe 65% active, the clock at 2.01
// GHz of 2.07).
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

constexpr int kItems = 4;      // item slots: the item after the current one is known to every warp early
constexpr uint32_t kSlab = 128 * 128;  // [128 rows][64 16-bit columns], 128B swizzle
constexpr uint32_t kVBox = 64 * 128;   // [64 keys][64 columns]
constexpr int kQSlabs = 6, kKStages = 4, kVStages = 4;
constexpr uint32_t kOffK = kQSlabs * kSlab, kOffV = kOffK + kKStages * kSlab, kOffBar = kOffV + kVStages * kSlab;
enum {
  KF0 = 0, KE0 = KF0 + kKStages, VF0 = KE0 + kKStages, VE0 = VF0 + kVStages,
  QL0 = VE0 + kVStages,  // a tile's queries have landed
  QF0 = QL0 + 2,         // ... are converted
  QE0 = QF0 + 2,         // ... are no longer read
  SF0 = QE0 + 2,
  PF0 = SF0 + 2,         // the weights of keys 0-31 and 64-95, of the others: [part][tile]
  OF0 = PF0 + 4,         // a tile's output is complete
  OE0 = OF0 + 2,         // ... has been read
  IF0 = OE0 + 2, IE0 = IF0 + kItems,  // the item slots
  TK0 = IE0 + kItems,            // the turn to issue MMAs
  MD0 = TK0 + 2, kBars = MD0 + 2
};
constexpr uint32_t kOffX = kOffBar + 8 * kBars;  // [2 tiles][2 halves][128] half-row maxima, then sums
constexpr uint32_t kOffItem = kOffX + 4 * 128 * 4;       // [kItems] items of 12 int32
constexpr uint32_t kOffSlots = kOffItem + kItems * 48;
constexpr uint32_t kSmem = kOffSlots + 16;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kThreads = 640;  // warps 0..15 softmax, 16 producer of keys and values, 17 and 18 MMA issuers of
                               // tiles 0 and 1, 19 producer of queries
constexpr uint32_t kTmS = 0, kTmO = 256;
constexpr int kEarly = 3;  // steps before an item's end at which the next one is taken
constexpr int64_t kTailBytes = 64 << 20;  // half of L2
constexpr float kBias = 7.0f;       // P = 2^7 exp(z - m)
constexpr float kRescale = 8.0f;    // log2 units
constexpr float kExactOff = 4096.f;  // log2 units
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

// A work item as the warps see it: its numbers from the plan, and each tile's steps.
struct Item {
  int q0, n, c0, L, j0, slot, hh, n0, n1;
  bool live;
};
__device__ __forceinline__ Item read_item(const int* s) {
  Item t;
  t.q0 = s[0], t.n = s[1], t.c0 = s[2], t.L = s[3], t.j0 = s[4], t.slot = s[6], t.hh = s[8];
  t.live = s[9] != 0;
  // tile x takes the steps up to the last token that its last row sees
  auto steps = [&](int x) {
    return min((t.L - t.n + min(t.q0 + 128 * (x + 1), t.n) + kKvTile - 1) / kKvTile, s[5]) - t.j0;
  };
  t.n0 = t.live ? steps(0) : 0;
  t.n1 = t.live && t.n - t.q0 > 128 ? steps(1) : 0;
  return t;
}

__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_qr,
              const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_kr,
              const __grid_constant__ CUtensorMap map_v, uint16_t* __restrict__ out, float* __restrict__ lse,
              ChunkPlan plan, int32_t* counter, int H, int h0, int heads, int64_t cap, float sl2, bool rope_f16,
              int32_t* err_word) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_index();
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };
  int* items = reinterpret_cast<int*>(smem + kOffItem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffSlots + 4);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) report_error(err_word, MLA_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool rows = (i >= QF0 && i < QE0) || (i >= OE0 && i < IF0);
      const bool both = (i >= KE0 && i < VF0) || (i >= VE0 && i < QL0);  // the two issuers
      mbar_init(bar(i), rows ? 256 : both ? 2 : i >= PF0 && i < OF0 ? 8 : i >= IE0 && i < TK0 ? 19 : 1);
    }
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

  if (warp == 16) {
    // ------------------------------------------------------------ items, keys and values
    if (elect()) {
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_kr);
      prefetch_tmap(&map_v);
      const uint64_t keep = policy_evict_last();
      const int pieces = plan.hdr[0];
      const int64_t total = (int64_t)pieces * heads;
      // The pieces are listed longest first. Head by head, so that a head's keys and
      // values are read by its pieces at about the same time (from L2); the last heads
      // piece by piece, so that the shortest end the run: as many as give three items
      // per SM, and as L2 holds the keys and values of (a context of 65536 tokens read
      // that way comes from HBM once per piece: 725 -> 771 us for 16 heads).
      const int64_t head_bytes = (int64_t)plan.hdr[1] * (kDNope + kDV) * 2;
      const int tail = pieces > 0 ? (int)min(min((long long)heads, (3ll * gridDim.x + pieces - 1) / pieces),
                                             (long long)(kTailBytes / head_bytes))
                                  : 0;
      const int64_t bulk = (int64_t)(heads - tail) * pieces;
      const int skip = skip_loads();
      bool ok = skip != 3;
      int ki = 0, vi = 0;
      int64_t idx = blockIdx.x;
      // item `it` into its slot: {q0, n, c0, L, j0, j1, slot, first expanded row, head, live}
      auto publish = [&](int it) {
        int* s = items + 12 * (it % kItems);
        if (it >= kItems)
          ok = wait_phase(bar(IE0 + it % kItems), (uint32_t)((it / kItems - 1) & 1), abort_flag, err_word);
        if (!ok) return;
        const bool live = idx < total;
        if (live) {
          const int pc = (int)(idx < bulk ? idx % pieces : (idx - bulk) / tail);
          const int4 a = __ldcg(plan.piece + 2 * pc), c = __ldcg(plan.piece + 2 * pc + 1);
          s[0] = a.x, s[1] = a.y, s[2] = a.z, s[3] = a.w, s[4] = c.x, s[5] = c.y, s[6] = c.z, s[7] = c.w;
          s[8] = (int)(idx < bulk ? idx / pieces : (heads - tail) + (idx - bulk) % tail);
          idx = gridDim.x + (int64_t)atomicAdd(counter, 1);
        }
        s[9] = live;
        mbar_arrive(bar(IF0 + it % kItems));
      };
      // a slot of a ring, once its last readers are done
      auto slab = [&](int full, int empty, int stages, int i) -> int {
        const int st = i % stages;
        ok = i < stages || wait_phase(bar(empty + st), (uint32_t)((i / stages - 1) & 1), abort_flag, err_word);
        if (ok) mbar_arrive_expect_tx(bar(full + st), kSlab);
        return st;
      };
      if (ok) publish(0);
      for (int it = 0; ok; ++it) {
        const int* s = items + 12 * (it % kItems);
        const Item t = read_item(s);
        if (!t.live) break;
        const int64_t k0 = s[7] + (int64_t)t.j0 * kKvTile;  // first expanded row of the piece
        const int nkv = max(t.n0, t.n1);
        for (int j = 0; j < nkv && ok; ++j) {
          // the next item is taken near this one's end, so that the CTAs stay in balance
          if (j == max(nkv - kEarly, 0)) publish(it + 1);
          if (!ok) break;
          if (skip == 1) continue;
          const int row = (int)(k0 + (int64_t)j * kKvTile), hrow = (int)((int64_t)t.hh * cap + row);
          for (int c = 0; c < 3 && ok; ++c) {
            const int st = slab(KF0, KE0, kKStages, ki);
            if (!ok) break;
            ++ki;
            if (c < 2)
              tma_load_2d(sbase + kOffK + st * kSlab, &map_k, bar(KF0 + st), 64 * c, hrow, keep);
            else
              tma_load_2d(sbase + kOffK + st * kSlab, &map_kr, bar(KF0 + st), kDC, row, keep);
          }
          for (int c = 0; c < 2 && ok; ++c) {
            const int st = slab(VF0, VE0, kVStages, vi);
            if (!ok) break;
            ++vi;
            const uint32_t dst = sbase + kOffV + st * kSlab;
            tma_load_2d(dst, &map_v, bar(VF0 + st), 0, hrow + 64 * c, keep);
            tma_load_2d(dst + kVBox, &map_v, bar(VF0 + st), 64, hrow + 64 * c, keep);
          }
        }
      }
      // let the copies in flight land before the CTA can exit, whoever gives up and whenever
      const long long t0 = clock64();
      auto drain = [&](int full, int stages, int i) {
        for (int k = i > stages ? i - stages : 0; k < i; ++k)
          while (!mbar_try_wait(bar(full + k % stages), (uint32_t)((k / stages) & 1)) &&
                 clock64() - t0 < wait_limit()) {
          }
      };
      drain(KF0, kKStages, ki);
      drain(VF0, kVStages, vi);
    }
  } else if (warp == 19) {
    // ------------------------------------------------------------ queries
    // A tile's queries as soon as the item before has computed its last scores
    if (elect()) {
      prefetch_tmap(&map_q);
      prefetch_tmap(&map_qr);
      const uint64_t once = policy_evict_first();
      bool ok = skip_loads() != 2;
      int qn[2] = {0, 0};
      for (int it = 0; ok; ++it) {
        ok = wait_phase(bar(IF0 + it % kItems), (uint32_t)((it / kItems) & 1), abort_flag, err_word);
        if (!ok) break;
        const Item t = read_item(items + 12 * (it % kItems));
        mbar_arrive(bar(IE0 + it % kItems));
        if (!t.live) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || (x ? t.n1 : t.n0) == 0) continue;
          ok = qn[x] == 0 || wait_phase(bar(QE0 + x), (uint32_t)((qn[x] - 1) & 1), abort_flag, err_word);
          if (!ok) continue;
          ++qn[x];
          // rows past the sequence's are loaded too (zeros past the array) and never written out
          mbar_arrive_expect_tx(bar(QL0 + x), 3 * kSlab);
          const uint32_t dst = sbase + 3 * x * kSlab;
          const int row = t.c0 + t.q0 + 128 * x;
          tma_load_3d(dst, &map_q, bar(QL0 + x), 0, h0 + t.hh, row, once);
          tma_load_3d(dst + kSlab, &map_q, bar(QL0 + x), 64, h0 + t.hh, row, once);
          tma_load_3d(dst + 2 * kSlab, &map_qr, bar(QL0 + x), 0, h0 + t.hh, row, once);
        }
      }
      const long long t0 = clock64();
      for (int x = 0; x < 2; ++x)
        while (qn[x] > 0 && !mbar_try_wait(bar(QL0 + x), (uint32_t)((qn[x] - 1) & 1)) &&
               clock64() - t0 < wait_limit()) {
        }
    }
  } else if (warp >= 17) {
    // ------------------------------------------------------------ MMA issuers
    // One per tile, in turns: [P V of a step, scores of the next] of tile 0, then of
    // tile 1. While one issues, the other does its waits, and takes over when the
    // last MMA is queued. (One thread for both left the pipe idle ~400 cycles a turn;
    // two without turns ran both tiles in step, all softmax and then all MMAs.)
    // A slab is free when both have committed; a tile that does not take a step
    // arrives in its place.
    const int x = warp - 17;
    if (elect()) {
      constexpr uint32_t kIdC = idesc_f16(128, 128, false, false);
      const uint32_t id_r = rope_f16 ? kIdC : idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdV = idesc_f16(128, 128, false, true);
      auto da = [](uint32_t addr) -> uint64_t { return (uint64_t)((addr >> 4) & 0x3FFFu); };
      const uint64_t dq = smem_desc(0, 16, 1024, kSwizzle128B) + da(sbase + 3 * x * kSlab);
      const uint64_t dk = smem_desc(0, 16, 1024, kSwizzle128B) + da(sbase + kOffK);
      const uint64_t dv = smem_desc(0, kVBox, 1024, kSwizzle128B) + da(sbase + kOffV);
      const uint32_t tS = tmem + kTmS + 128 * x, tO = tmem + kTmO + 128 * x;
      bool ok = true;
      int ks = 0, vs = 0;            // slots of the rings, and their uses' parity
      uint32_t kp = 0, vp = 0;
      uint32_t pn = 0, an = 0;       // steps and items of this tile so far
      auto key_slab = [&](bool use, int s) {
        ok = wait_phase(bar(KF0 + ks), kp, abort_flag, err_word) && ok;
        if (use && ok) {
          tc_fence_after();
          const uint64_t ad = dq + (s * kSlab >> 4), bd = dk + ((uint64_t)ks * kSlab >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss(tS, ad + 2 * k, bd + 2 * k, s < 2 ? kIdC : id_r, (s > 0 || k > 0) ? 1u : 0u);
          mma_commit(bar(KE0 + ks));
        } else {
          mbar_arrive(bar(KE0 + ks));
        }
        if (++ks == kKStages) ks = 0, kp ^= 1u;
      };
      uint32_t turn = 0;
      auto take = [&] {  // tile 0 starts; its turn n follows tile 1's turn n - 1
        if (x == 1 || turn > 0) ok = wait_phase(bar(TK0 + x), (x == 1 ? turn : turn - 1) & 1u, abort_flag, err_word) && ok;
        ++turn;
      };
      auto pass = [&] { mbar_arrive(bar(TK0 + (x ^ 1))); };
      // S = Q K^T of the next step
      // (the turn passes before the last slab: the other issuer sees it about 300
      // cycles later, when this slab's MMAs are under way)
      auto scores = [&](bool use) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          if (s == 2 && use) pass();
          key_slab(use, s);
        }
        if (use) mma_commit(bar(SF0 + x));
      };
      // O += P V, as the two parts of P come: 32 keys of each slab at a time
      auto values = [&](bool use, bool first) {
        const int v0 = vs, v1 = vs + 1 == kVStages ? 0 : vs + 1;
        const uint32_t p0 = vp, p1 = v1 == 0 ? vp ^ 1u : vp;
        if (use) {
          ok = wait_phase(bar(PF0 + x), pn & 1u, abort_flag, err_word) && ok;
          take();
        }
        ok = wait_phase(bar(VF0 + v0), p0, abort_flag, err_word) && ok;
        ok = wait_phase(bar(VF0 + v1), p1, abort_flag, err_word) && ok;
        if (use && ok) {
          const uint64_t b0 = dv + ((uint64_t)v0 * kSlab >> 4), b1 = dv + ((uint64_t)v1 * kSlab >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (part) ok = wait_phase(bar(PF0 + 2 + x), pn & 1u, abort_flag, err_word) && ok;
            tc_fence_after();
#pragma unroll
            for (int k = 2 * part; k < 2 * part + 2; ++k) {
              mma_ts(tO, tS + 8 * k, b0 + (k * 2048 >> 4), kIdV, (!first || k > 0) ? 1u : 0u);
              mma_ts(tO, tS + 32 + 8 * k, b1 + (k * 2048 >> 4), kIdV, 1u);
            }
          }
          mma_commit(bar(VE0 + v0));
          mma_commit(bar(VE0 + v1));
          ++pn;
        } else {
          mbar_arrive(bar(VE0 + v0));
          mbar_arrive(bar(VE0 + v1));
        }
        vs = v1 + 1 == kVStages ? 0 : v1 + 1;
        vp = vs == 0 ? p1 ^ 1u : p1;
      };
      for (int it = 0; ok; ++it) {
        ok = wait_phase(bar(IF0 + it % kItems), (uint32_t)((it / kItems) & 1), abort_flag, err_word);
        if (!ok) break;
        const Item t = read_item(items + 12 * (it % kItems));
        mbar_arrive(bar(IE0 + it % kItems));
        if (!t.live) break;
        const int nx = x ? t.n1 : t.n0, nkv = max(t.n0, t.n1);
        if (nx > 0) ok = wait_phase(bar(QF0 + x), an & 1u, abort_flag, err_word);
        take();
        if (nx == 0) pass();
        scores(nx > 0);
        if (nx == 1) mma_commit(bar(QE0 + x));
        for (int j = 0; j < nkv && ok; ++j) {
          // the rows of the item before have left the accumulator
          if (j == 0 && nx > 0 && an > 0) ok = wait_phase(bar(OE0 + x), (an - 1) & 1u, abort_flag, err_word) && ok;
          if (j >= nx) {  // (take() in values() otherwise, after P)
            take();
            pass();
          }
          values(j < nx, j == 0);
          if (j + 1 == nx) pass();
          if (j + 1 < nkv) scores(j + 1 < nx);
          if (j + 2 == nx) mma_commit(bar(QE0 + x));
          if (j + 1 == nx) mma_commit(bar(OF0 + x));
        }
        if (nx > 0) ++an;
      }
      mma_commit(bar(MD0 + x));
      wait_mmas(bar(MD0 + x));
    }
  } else {
    // ------------------------------------------------------------ softmax
    // tile x, column half y; the row is the tensor-memory lane of this thread
    const int x = (warp >> 2) & 1, y = warp >> 3, lane = threadIdx.x & 31, row = threadIdx.x & 127, tid = row + 128 * y;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tZ = tmem + kTmS + 128 * x + 64 * y + lane_off;  // this thread's half of S
    const uint32_t tP = tZ - 32 * y, tO = tZ + kTmO;                 // ... of P and of O
    // one float per thread for its other half-row (maxima, then sums)
    const uint32_t mine = sbase + kOffX + 512u * (2 * x + y) + 4u * row;
    auto put = [&](float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine), "f"(v) : "memory"); };
    auto get = [&] {
      float v;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(y ? mine - 512u : mine + 512u) : "memory");
      return v;
    };
    uint32_t sn = 0, an = 0;  // steps and items of this tile so far
    // waits of a warp: its lanes leave together (the tensor-memory loads need them all)
    auto wait = [&](int i, uint32_t phase) {
      return __all_sync(0xffffffffu, wait_phase(bar(i), phase & 1u, abort_flag, err_word)) != 0;
    };
    // The tile's eight warps meet at named barriers, which cannot give up. So a warp
    // whose wait gave up goes on through the item's steps (every later wait returns at
    // once, nothing is written out), and whether there is a next item is agreed on.
    auto meet = [&] { asm volatile("barrier.cta.sync.aligned %0, 256;" ::"r"(1 + x) : "memory"); };
    auto agree = [&](bool v) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred.aligned q, %2, 256, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"((uint32_t)v), "r"(1 + x)
          : "memory");
      return r != 0;
    };
    // an item's slot is given back once the item is written out: its numbers are read
    // again there instead of being kept in registers through the steps
    auto item_of = [&](int it) { return read_item(items + 12 * (it % kItems)); };
    auto release = [&](int it) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(IE0 + it % kItems));
    };
    // the tile's queries, in place: content from bf16 to fp16 (exact for values of
    // normal fp16 size), position as the cache's (fp16 for an FP8 cache, else as it is)
    auto convert = [&](int it, uint32_t uses) {
      const Item t = item_of(it);
      if (!t.live) return false;
      if ((x ? t.n1 : t.n0) == 0) return true;
      if (!wait(QL0 + x, uses)) return false;
      const int rows = t.n - t.q0 - 128 * x;
      bool beyond = false;  // of each row by itself: a NaN in one hides nothing in another
#pragma unroll 4
      for (int k = 0; k < (rope_f16 ? 12 : 8); ++k) {
        const int i = tid + 256 * k;  // 16 bytes of the two content slabs, then of the positional one
        const uint32_t at = sbase + 3 * x * kSlab + 16 * i;
        uint32_t e[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(e[0]), "=r"(e[1]), "=r"(e[2]), "=r"(e[3]) : "r"(at));
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          top = max(top, max((e[q] << 16) & 0x7FFFFFFFu, e[q] & 0x7FFF0000u));
          e[q] = cvt_f16x2(bf16_lo(e[q]), bf16_hi(e[q]));
        }
        st_shared_v4(at, e[0], e[1], e[2], e[3]);
        beyond |= top >= kF16Limit && top < 0x7F800000u && ((i >> 3) & 127) < rows;
      }
      if (beyond) report_error(err_word, MLA_ERR_RANGE);
      fence_proxy_async_smem();
      mbar_arrive(bar(QF0 + x));
      return true;
    };

    bool ok = true, more = agree(wait(IF0, 0) && convert(0, 0));
    for (int it = 0; more; ++it) {
      int nx, first_seen, seen;
      {
        const Item t = item_of(it);
        const int r0 = t.q0 + 128 * x, before = t.L - t.n + 1 - t.j0 * kKvTile;
        nx = x ? t.n1 : t.n0;
        first_seen = before + r0;                  // tokens of the piece that the tile's first row sees
        seen = before + min(r0 + row, t.n - 1);    // ... that this row sees
      }
      float ref = -INFINITY;
      uint64_t sum2[2] = {0, 0};
      for (int j = 0; j < nx; ++j) {
        ok = wait(SF0 + x, sn++) && ok;
        tc_fence_after();
        uint32_t z[64];
        tmem_ld32(tZ, *reinterpret_cast<uint32_t(*)[32]>(z));
        tmem_ld32(tZ + 32, *reinterpret_cast<uint32_t(*)[32]>(z + 32));
        tmem_wait_ld();
        if ((j + 1) * kKvTile > first_seen) {
          const int lim = seen - j * kKvTile - 64 * y;
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
        put(mx);
        // both halves of S are in registers then: P may overwrite them. (The next
        // step's maxima follow its scores, which follow every thread's P.)
        meet();
        mx = fmaxf(mx, get());
        // all MMAs issued before this step's scores are done, the last P V among them
        // (the difference first: it is exact where the products would round it away)
        if (__any_sync(0xffffffffu, (mx - ref) * sl2 > kRescale)) {
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
        const float base = ref == -INFINITY ? 0.f : ref;
        float off = kBias - base * sl2;
        // A product beyond 2^12 would bring its rounding (2^-13 and more) into the weights,
        // beyond 2^28 overflow or lose them all: the reference is taken off first there.
        if (__any_sync(0xffffffffu, fabsf(base) * sl2 > kExactOff)) {
#pragma unroll
          for (int c = 0; c < 64; ++c) z[c] = __float_as_uint(__uint_as_float(z[c]) - base);
          off = kBias;
        }
        const uint64_t off2 = pack2(off, off), sl22 = pack2(sl2, sl2);
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const uint64_t u = fma2(pack2(__uint_as_float(z[c + 2 * q]), __uint_as_float(z[c + 2 * q + 1])), sl22, off2);
            float a, e;
            unpack2(u, a, e);
            a = ex2(a);
            e = ex2(e);
            sum2[q & 1] = add2(sum2[q & 1], pack2(a, e));
            p[q] = cvt_f16x2(a, e);
          }
          tmem_st16(tP + c / 2, p);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(PF0 + (c / 32) * 2 + x));
        }
      }
      // the next item's queries first: its scores may run while this one is written out
      more = agree(wait(IF0 + (it + 1) % kItems, (uint32_t)((it + 1) / kItems)) &&
                   convert(it + 1, an + (nx > 0 ? 1 : 0)));  // (they have all read the last maxima, too)
      if (nx > 0) {
        // the two halves' sums
        float s0, s1;
        unpack2(add2(sum2[0], sum2[1]), s0, s1);
        float sum = s0 + s1;
        put(sum);
        meet();
        sum += get();  // the same in both halves
        ok = wait(OF0 + x, an++) && ok;
        tc_fence_after();
        const Item t = item_of(it);
        const int r0 = t.q0 + 128 * x;
        const bool live = ok && r0 + row < t.n;
        const size_t at = (size_t)(t.c0 + r0 + row) * H + h0 + t.hh;
        // a whole item: the output row; a piece of one: its sums and reference, as they are
        const bool part = t.slot >= 0;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN stays NaN
        const size_t pr = part ? ((size_t)t.slot * heads + t.hh) * kQTile + 128 * x + row : 0;
        if (part && y == 0) plan.ml_part[pr] = make_float2(ref, sum);
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
          if (c == 32) {
            tc_fence_before();
            mbar_arrive(bar(OE0 + x));
          }
          if (part && ok) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              reinterpret_cast<uint4*>(plan.o_part + pr * kDV + 64 * y + c)[q] =
                  make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else if (live && !part) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = cvt_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * inv, __uint_as_float(o[8 * q + 2 * e + 1]) * inv);
              reinterpret_cast<uint4*>(out + at * kDV + 64 * y + c)[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (lse && live && y == 0 && !part)
          lse[at] = sum > 0.f ? (ref * sl2 - kBias + log2f(sum)) * kLn2 : (sum == 0.f ? -INFINITY : sum);
        meet();  // the sums are read: the next item's maxima may take their place
      }
      release(it);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Items that were cut over the keys:
//   out = sum_k 2^((m_k - m) sl2) O_k / sum_k 2^((m_k - m) sl2) l_k,
// added in the order of the pieces. A warp per row, 16 bytes a lane; the partials of
// a row are read once (HBM or L2-bound, 512 bytes a piece).
__global__ void __launch_bounds__(256)
join_kernel(ChunkPlan plan, uint16_t* __restrict__ out, float* __restrict__ lse, int H, int h0, float sl2) {
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
      const float w = ml.x == m ? 1.f : ex2((ml.x - m) * sl2);
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
    if (lse && lane == 0) lse[row] = l > 0.f ? (m * sl2 - kBias + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
  }
}

}  // namespace

cudaError_t launch_attend(const ChunkPlan& plan, const uint16_t* q_nope, const uint16_t* q_rope, uint16_t* out,
                          float* lse, int B, int T, int H, int h0, int heads, int64_t cap, int slots, int round,
                          float scale, bool f16, int32_t* err_word, cudaStream_t s) {
  CUtensorMap mq, mqr, mk, mr, mv;
  const uint64_t dq[3] = {kDNope, (uint64_t)H, (uint64_t)T}, sq[2] = {kDNope * 2, (uint64_t)H * kDNope * 2};
  const uint64_t dqr[3] = {kDR, (uint64_t)H, (uint64_t)T}, sqr[2] = {kDR * 2, (uint64_t)H * kDR * 2};
  const uint64_t dk[2] = {kDNope, (uint64_t)heads * cap}, sk[1] = {kDNope * 2};
  const uint64_t dr[2] = {kRow, (uint64_t)cap}, sr[1] = {kRow * 2};
  const uint32_t bq[3] = {64, 1, 128}, bk[2] = {64, 128}, bv[2] = {64, 64};
  if (!make_tmap(&mq, q_nope, 3, dq, sq, bq, 128) || !make_tmap(&mqr, q_rope, 3, dqr, sqr, bq, 128) ||
      !make_tmap(&mk, plan.k, 2, dk, sk, bk, 128) || !make_tmap(&mr, plan.rows, 2, dr, sr, bk, 128) ||
      !make_tmap(&mv, plan.v, 2, dk, sk, bv, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = smem_limit<attend_kernel>(kSmem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const float sl2 = scale * 1.4426950408889634f;
  const int64_t most = ((int64_t)chunk_max_items(B, T) + slots) * heads;
  e = launch_pdl(attend_kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), kSmem, s, mq, mqr, mk, mr,
                 mv, out, lse, plan, plan.counter + round, H, h0, heads, cap, sl2, f16,
                 err_word);
  if (e != cudaSuccess || slots == 0) return e;
  const int joins = chunk_max_items(B, T) < slots / 2 ? chunk_max_items(B, T) : slots / 2;  // two pieces at least
  return launch_pdl(join_kernel, dim3(joins, heads, 8), dim3(256), 0, s, plan, out, lse, H, h0, sl2);
}

#if MLA_DEBUG_CHECKS
cudaError_t debug_attend(const long long* limit, const int* skip) { return sm100::debug_set(limit, skip); }
#endif

}  // namespace mla

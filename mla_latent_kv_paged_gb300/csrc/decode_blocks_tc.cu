// Split-KV MLA decode over a block-scaled 8-bit latent cache (blocks.cuh), tcgen05, sm_103a.
//
// What it computes, and how the work is laid out, is decode_tc.cu's: a cluster of two CTAs per range
// of tiles, CTA r with latent columns [256r, 256r + 256) and positional columns [512 + 32r, +32) of
// every 64-token tile; partial scores, page maxima and weights exchanged between the two; the head
// rows as the M = 128 rows of both products. It differs in
//   - the tile: e4m3 codes with a power of two for each block of tokens and group of columns, which
//     twelve warps of their own widen to the fp16 boxes that the MMAs read, powers applied
//     (exact from 2^-14 on). Column scales can be folded into the query and the output instead, as
//     decode_tc.cu does for its 8-bit cache; a block's cannot;
//   - the ring: four operand slots (queries and widened tiles, 36 KB) and two slots of codes (18 KB),
//     each free again as soon as its codes are widened;
//   - the operands: query, weights and tiles in fp16, fp32 sums;
//   - the roles: a warpgroup each, with registers dealt out by setmaxnreg (28 warps: producer, two
//     MMA issuers and an idle one; score readers; softmax 2 x 4; wideners 3 x 4).
// It is a kernel of its own because a change to the other's code, even one that its template
// folds away, costs it up to 2%.
//
// What bounds it: a tile's chain of work, as there (2400 cycles a tile at long contexts), and the wideners'
// share of the issue slots and of shared memory. More room does not help: five operand slots in place of
// four (with the positional columns in a ring of two, and P in two buffers) took the same time.
// 32 sequences of 4096 tokens, 128 heads (this kernel alone with cold caches / decode step, us): 8-bit with
// column scales 60 / 72; here 44 / 56; bf16 41 / 55. Four sequences of 131072: here 133 / 159; steps of the other two
// 215 and 148. (Steps: twelve in one graph, on three sets of inputs in turn.)
// Steps on the way (32 x 4096, a graph a step, some us of which are the gaps between them): widened by the score
// readers 102; by four warps of their own, to bf16 73 (83 instructions for 16 codes), to fp16 72; by eight 63; with the roles' code made
// short (packed fp32 pairs, maxima of three, waits of few instructions, loops left rolled) and the next
// codes read ahead 60: five roles share the SM's instruction caches, and every unrolled loop was
// slower; with registers dealt by need 58.5; by twelve, three chunks each, all read before the wait for the
// operand slot, 57.
// Measured and not taken: tiles prefetched into L2 (65), codes as 256-byte rows (60), the entries read ahead
// (60 to 63), score MMAs started on the first half of a widened tile (60), weights taken with an older reference
// while the maxima travel (58). A slot of codes is given back
// after the widened values are stored, not once its codes are read: given back right after the loads,
// the next copy overtook some of them, for 0.2% of the time.
//
// Tensor memory (512 columns x 128 lanes of 32 bits): O [0,256), S [256,320), this CTA's P half for three
// tiles [320,368), positional query half [368,384), latent query half [384,512).
#include "blocks.cuh"
#include "chunk.cuh"
#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kOpSlots = 4, kCodeSlots = 2;
constexpr int kAWarps = 4;  // score readers: one per TMEM lane quadrant
constexpr int kBWarps = 8;  // softmax: two groups of four (one per lane quadrant), alternate pages
constexpr int kAThreads = kAWarps * 32, kBThreads = kBWarps * 32;
constexpr int kGThreads = kBThreads / 2;  // one softmax group: a thread per head row
constexpr int kWThreads = 12 * 32;  // wideners: three 16-byte chunks of a tile each
constexpr int kRead0 = 4, kSoft0 = kRead0 + kAWarps, kWide0 = kSoft0 + kBWarps;  // first warps of the roles
constexpr int kThreads = 32 * kWide0 + kWThreads;
constexpr int kRegsIssue = 56, kRegsRead = 96, kRegsSoftmax = 104, kRegsWiden = 48;
static_assert(kRegsIssue + kRegsRead + 2 * kRegsSoftmax + 3 * kRegsWiden <= 7 * 72, "the launch's registers");
constexpr uint32_t kCBoxBytes = 64 * 128;   // [64 tokens][64 latent cols] fp16, 128B swizzle
constexpr uint32_t kKrBoxBytes = 64 * 64;   // [64 tokens][32 positional cols] fp16, 64B swizzle
constexpr uint32_t kOpBytes = 4 * kCBoxBytes + kKrBoxBytes;  // 36864: an operand slot
constexpr uint32_t kQrBoxBytes = 64 * 64;   // [64 heads][32 positional cols], 64B swizzle
constexpr uint32_t kQBoxBytes = 128 * 128;  // [128 heads][64 latent cols], 128B swizzle
constexpr int kQSlots = 2;                  // operand slots taken by a range's latent query half (4 boxes)
constexpr uint32_t kVecBytes = 128 * 4;     // one float per head
// peer partial scores: [4 groups of 8 tokens][128 heads] fp16 offsets from a per-head
// midpoint, then the midpoints [128 heads] fp32 (log2 units)
constexpr uint32_t kXDataBytes = 4 * 128 * 16;
constexpr uint32_t kXBytes = kXDataBytes + kVecBytes;
constexpr uint32_t kPPeerBytes = 128 * 64;  // the peer's half of P: [128 heads][32 tokens] fp16, 64B swizzle
constexpr uint32_t kPHalfBytes = kPPeerBytes;
constexpr int kPBufs = 3;  // P buffers: page g uses g % 3, so its writers wait for page g - 3
constexpr uint32_t kTokBytes = 4 * 4;       // "partial consumed" tokens: one per warp of a group
// codes of a CTA's half of a tile, unswizzled rows of 64 and 32 bytes
constexpr uint32_t kCodeBoxBytes = 64 * 64;   // [64 tokens][64 latent cols]
constexpr uint32_t kCodeKrBoxBytes = 16 * 32;  // [16 tokens][32 positional cols], four per tile
constexpr uint32_t kCodeBytes = 4 * kCodeBoxBytes + 4 * kCodeKrBoxBytes;  // 18432: a slot of codes
constexpr uint32_t kEntriesBytes = kTile / 16 * kEntryBytes;  // a tile's 8-byte entries (blocks of 16 tokens or more)

constexpr uint32_t kOffOp = 0;
constexpr uint32_t kOffCode = kOffOp + kOpSlots * kOpBytes;
constexpr uint32_t kOffX = kOffCode + kCodeSlots * kCodeBytes;  // peer partial scores, one buffer per group
constexpr uint32_t kOffP = kOffX + 2 * kXBytes;        // the peer's half of P, two pages
constexpr uint32_t kOffMX = kOffP + kPBufs * kPPeerBytes;  // peer page maxima [2 groups][128]
constexpr uint32_t kOffLX = kOffMX + 2 * kVecBytes;  // peer softmax sums [2 ranges][128]
constexpr uint32_t kOffMR = kOffLX + 2 * kVecBytes;    // reference maximum after the latest page [128]
constexpr uint32_t kOffLG = kOffMR + kVecBytes;        // handed-over group sums [2 ranges][sum, ref][128]
constexpr uint32_t kOffIV = kOffLG + 4 * kVecBytes;    // 1 / softmax sum of the range [128]
constexpr uint32_t kOffTok = kOffIV + kVecBytes;       // tokens from the peer
constexpr uint32_t kOffBar = kOffTok + kTokBytes;

// barrier indices. A barrier that completes once per page and is waited by
// only one of the two softmax groups exists once per group (index g % 2): a
// parity wait is only sound if the barrier's previous phase is one this
// waiter has already seen complete.
enum {
  // operand slots: filled (by the wideners, or with a query), and free; codes' slots: filled, and widened
  OPF0 = 0, EMPTY0 = OPF0 + kOpSlots, CF0 = EMPTY0 + kOpSlots, CE0 = CF0 + kCodeSlots, QCF = CE0 + kCodeSlots,
  SF0 = QCF + 1, SFREE = SF0 + 2, PF0 = SFREE + 1, PVD0 = PF0 + kPBufs, XF0 = PVD0 + kPBufs, XE0 = XF0 + 2,
  MXF0 = XE0 + 2, LXF0 = MXF0 + 2, MRF = LXF0 + 2, LGF0 = MRF + 1, IVF0 = LGF0 + 2, OFREE = IVF0 + 2,
  MMAD = OFREE + 1, kNumBars = MMAD + 1
};
constexpr uint32_t kOffSlots = kOffBar + kNumBars * 8;
constexpr uint32_t kOffEntries = (kOffSlots + 15) / 16 * 16 + 16;
constexpr uint32_t kSmemBytes = kOffEntries + kCodeSlots * kEntriesBytes;  // the base is checked to be 1024-byte aligned
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(2 * kQBoxBytes + kQrBoxBytes <= kOpBytes, "an operand slot holds half of a query half");

constexpr uint32_t kTmO = 0, kTmS = 256, kTmP = 320, kTmQr = 368, kTmQ = 384, kTmCols = 512;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: weights stay <= 2^8 of the reference
// P holds weights times 2^7 (at most 2^15 then, of fp16's 65504), so that one becomes zero below 2^-32 of the
// reference only, and not below 2^-25, where 131072 light tokens together are 2^-8 of a heavy one. (Of 131072 tokens
// of 2^-25.5 in one range, values of the heavy one zero: u off by all of itself before, by 0.6% now. The fp32 sums
// of the value MMAs cut each addend at 2^-24 of the sum, n 2^-24 of n tokens, whatever the type of the weights: a
// value that all tokens share is off by up to 0.3% in that case, before and now.)
constexpr float kWeightShift = 7.0f;

#if MLA_DEBUG_CHECKS
// Test builds only: the counters of decode_tc.cu, for this kernel, and its switch.
__device__ unsigned long long g_dbg_counters[4];
__device__ int g_dbg_skip_producer;
__device__ __noinline__ bool dbg_check(bool ok, int32_t* err_word) {
  if (!ok) {
    atomicAdd(&g_dbg_counters[1], 1ull);
    report_error(err_word, MLA_ERR_BOUNDS);
  }
  return ok;
}
// true when [addr, addr + bytes) lies inside this CTA's dynamic shared memory
// (for an address of the peer CTA: the same offset before mapa)
#define MLA_SMEM_OK(addr, bytes) \
  dbg_check((addr) >= sbase && (uint64_t)(addr) + (bytes) <= (uint64_t)sbase + kSmemBytes, err_word)
#define MLA_TMEM_OK(col, ncols) dbg_check((uint32_t)(col) + (ncols) <= (uint32_t)kTmCols, err_word)
#else
#define MLA_SMEM_OK(addr, bytes) true
#define MLA_TMEM_OK(col, ncols) true
#endif


__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr));
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Four e4m3 codes (byte i = value i) -> fp16 pairs: values 0,1 in lo, 2,3 in hi
// (exact: every e4m3 value is an fp16 value).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kLeastF16 = 127 - 24, kMostF16 = 127 + 15, kSafeF16 = 127 + 7;  // 448 * 2^7 < 65504
constexpr uint32_t kExactF16 = 127 - 15;  // codes are multiples of 2^-9: products with 2^-15 and more are exact
__device__ __forceinline__ uint32_t power_f16x2(uint32_t p) {
  const float step = step_of(min(p < kLeastF16 ? kExactF16 : p, kMostF16));
  return cvt_f16x2(step, step);
}
// 16 codes times 2^(p - 127), as fp16 pairs, by: power_f16x2(p). Exact but below fp16's normal range (2^-14),
// where a value is rounded once to 2^-24's multiples. fp16 holds the powers 2^-24 .. 2^15. One below takes two
// products, the first of them, with 2^-15, exact (the other factor underflows where every value is less than 2^-30,
// a zero either way); one above stands for values that fp16 does not hold. Returns whether one of the values
// became infinite.
__device__ __forceinline__ bool widen16(const uint32_t (&v)[4], uint32_t by, uint32_t p, uint32_t (&o)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    e4m3x4_to_f16(v[c], o[2 * c], o[2 * c + 1]);
    o[2 * c] = mul_f16x2(o[2 * c], by);
    o[2 * c + 1] = mul_f16x2(o[2 * c + 1], by);
  }
  bool beyond = false;
  if (__builtin_expect(p < kLeastF16 || p > kSafeF16, 0)) {
    // what is left of the power (at most 2^15 of it: every value but zero then is infinite)
    const float rest = step_of(p < kLeastF16 ? p + 127 - kExactF16 : p > kMostF16 ? min(p - 15, kMostF16) : 127);
    const uint32_t more = cvt_f16x2(rest, rest);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      o[c] = mul_f16x2(o[c], more);
      beyond |= (o[c] & 0x7FFFu) == 0x7C00u || (o[c] & 0x7FFF0000u) == 0x7C000000u;
    }
  }
  return beyond;
}
// Pairs of fp32 in one instruction, and the largest or smallest of three (the step of 32 x 4096 took
// 62.9 us with single ones, 61.3 with these).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// an fp16 pair's two values, each plus c
__device__ __forceinline__ uint64_t f16x2_plus(uint32_t w, float c) {
  float lo, hi;
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.f16 %0, l, %3;\n\tadd.rn.f32.f16 %1, h, %3;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w), "f"(c));
  return pair(lo, hi);
}
// A head's query, from bf16 to fp16; what fp16 does not hold is reported.
template <int kN>
__device__ __forceinline__ void query_f16(uint32_t (&r)[kN], bool live, int32_t* err_word) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    top = max(top, max((r[k] << 16) & 0x7FFFFFFFu, r[k] & 0x7FFF0000u));
    r[k] = cvt_f16x2(bf16_lo(r[k]), bf16_hi(r[k]));
  }
  if (live && top >= kF16Limit && top < 0x7F800000u) report_error(err_word, MLA_ERR_RANGE);
}
// kRows: the sequences are rows of a chunk (chunk.cuh): seq_row[b] is the block-table row of sequence b,
// -1 for a row of no sequence (it reads zeros and its result is not used); the query then is fp16.
template <bool kRows>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode_blocks_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_kr,
                     const __grid_constant__ CUtensorMap map_qkr, const __grid_constant__ CUtensorMap map_q,
                     const int32_t* __restrict__ block_table, int n_q, int H, int max_pages, int num_pages,
                     int tile_shift, int block_shift, int q_is_f16, float sl2, Plan plan,
                     const uint8_t* __restrict__ entries, int32_t* err_word, const int32_t* __restrict__ seq_row) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const bool q_f16 = kRows || q_is_f16;
  if (sbase & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) report_error(err_word, MLA_ERR_CUDA);
    return;
  }
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
  const int worker = blockIdx.x >> 1, j = blockIdx.y;
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffSlots + 4);

  // (as in decode_tc.cu, a warp's lanes wait in step: one try, one look at the flag and the clock for all
  // of them. A vote on the result in every wait cost 3%.)
  auto wait = [&](uint32_t b, uint32_t parity) -> bool { return wait_short(b, parity, abort_flag); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kOpSlots; ++i) {
      mbar_init(bar(OPF0 + i), kWThreads / 32);
      mbar_init(bar(EMPTY0 + i), 1);
    }
    for (int i = 0; i < kCodeSlots; ++i) {
      mbar_init(bar(CF0 + i), 1 + kTile / 16);  // the copies of the codes and of the entries
      mbar_init(bar(CE0 + i), kWThreads / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(LXF0 + i), 1);
      mbar_init(bar(LGF0 + i), kGThreads);  // a group's sums handed over
      mbar_init(bar(IVF0 + i), kGThreads);  // 1/l posted for helper group i
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(bar(PF0 + i), kGThreads + 1);  // a group's rows + the arming arrive for the peer's half
      mbar_init(bar(PVD0 + i), 2);             // the value MMAs of the page done in both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(SF0 + i), 1);
      mbar_init(bar(XF0 + i), 1);  // armed here, filled by the peer's st.async
      mbar_init(bar(XE0 + i), 1);  // armed here, completed by the peer's four 4-byte tokens
      mbar_init(bar(MXF0 + i), 1);
    }
    mbar_init(bar(SFREE), kAThreads + kGThreads);

    mbar_init(bar(MRF), kGThreads);  // the reference maximum of a page posted
    mbar_init(bar(QCF), kAThreads);  // the range's latent query half is in tensor memory
    mbar_init(bar(OFREE), 2 * kGThreads);        // both halves of O drained
    mbar_init(bar(MMAD), 2);  // both MMA issuers done
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < kPBufs; ++i) mbar_arrive_expect_tx(bar(PF0 + i), kPHalfBytes);
    for (int i = 0; i < 2; ++i) {
      mbar_arrive_expect_tx(bar(LXF0 + i), kVecBytes);
      mbar_arrive_expect_tx(bar(XF0 + i), kXBytes);
      mbar_arrive_expect_tx(bar(XE0 + i), kTokBytes);
      mbar_arrive_expect_tx(bar(MXF0 + i), kVecBytes);
    }
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_c);
    prefetch_tmap(&map_kr);
    prefetch_tmap(&map_qkr);
    prefetch_tmap(&map_q);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peer's barriers are initialised before any remote arrive
  const uint32_t tmem = *tmem_slot;
  // set-up above overlaps the plan kernel; the plan and q_abs are read below.
  // (The order of these two matters to a chunk's rows: out_proj, two launches on, loads the
  // fp16 copy of W^UV that their plan kernel writes before its own dependency wait, and
  // may do so because it starts after this wait.)
  grid_dependency_wait();
  grid_launch_dependents();
  const int it0 = plan.range_item[worker], it1 = plan.range_item[worker + 1];

  auto produce = [&]() {
    // ------------------------------------------------------------ TMA producer
    // Loads the codes and entries of this CTA's half of each tile.
    const uint64_t pol_stream = policy_evict_first();
    int stage = 0;
    uint32_t ph = 0;
    int last_ph[kCodeSlots];
#pragma unroll
    for (int i = 0; i < kCodeSlots; ++i) last_ph[i] = -1;
    bool ok = true;
    // tile cursors over (range, tile): lanes hold the page ids of 32 consecutive
    // tiles (a page holds 1 << tile_shift tiles of 64 tokens)
    const int tile_mask = (1 << tile_shift) - 1;
    struct Cursor {
      int it, pg, pg1, base, id_l, pg0, seq;  // pg0, seq: the piece's first tile and its sequence
      int64_t row;  // block-table row of the current range (its first entry), or < 0: none
    };
    auto table_row = [&](int seq) -> int64_t {
      return (int64_t)(kRows ? seq_row[seq] : seq) * max_pages;
    };
    auto cur_load = [&](Cursor& c) {
      const int mine = c.base + lane;
      // (a row of no sequence reads past the pool: zeros)
      if (kRows && c.row < 0)
        c.id_l = num_pages;
      else
        c.id_l = mine < c.pg1 ? block_table[c.row + (mine >> tile_shift)] : 0;
    };
    auto cur_init = [&](Cursor& c, int it) {
      c.it = it;
      if (it < it1) {
        c.seq = plan.item_seq[it];
        c.row = table_row(c.seq);
        c.pg = c.base = c.pg0 = plan.item_tile0[it];
        c.pg1 = plan.item_tile1[it];
        cur_load(c);
      }
    };
    auto cur_next = [&](Cursor& c) -> int {  // page id of the tile at the cursor, then advance
      const int id = __shfl_sync(0xffffffffu, c.id_l, c.pg - c.base);
      if (++c.pg == c.pg1) {
        cur_init(c, c.it + 1);
      } else if (c.pg - c.base == 32) {
        c.base = c.pg;
        cur_load(c);
      }
      return id;
    };
    Cursor ld;
    {  // the range's first piece from its 16-byte description
      const int4 d0 = plan.range_desc[worker];
      ld.it = d0.x;
      if (d0.x < it1) {
        ld.seq = d0.y;
        ld.row = table_row(d0.y);
        ld.pg = ld.base = ld.pg0 = d0.z;
        ld.pg1 = d0.w;
        cur_load(ld);
      }
    }
#if MLA_DEBUG_CHECKS
    if (*reinterpret_cast<volatile int*>(&g_dbg_skip_producer)) ld.it = it1;  // load nothing
#endif
    while (ok && ld.it < it1) {
      const int sub = ld.pg & tile_mask;  // the tile's place in its page
      const bool none = kRows && ld.row < 0;
      const int pid = cur_next(ld);
      // an id outside the pool loads zeros (TMA bounds) and is reported
      if (lane == 0 && !none && (pid < 0 || pid >= num_pages)) report_error(err_word, MLA_ERR_BOUNDS);
      if (!wait(bar(CE0 + stage), ph ^ 1u)) { ok = false; break; }
      const uint32_t fb = bar(CF0 + stage), dst = sbase + kOffCode + stage * kCodeBytes;
      if (lane == 0 && MLA_SMEM_OK(dst, kCodeBytes)) {
        const int y = ((pid << tile_shift) + sub) * kTile;
        mbar_arrive_expect_tx(fb, kCodeBytes);
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
          tma_load_2d(dst + cb * kCodeBoxBytes, &map_c, fb, 256 * (int)rank + 64 * cb, y, pol_stream);
        // (as four boxes of 16 rows, as in decode_tc.cu)
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          tma_load_2d(dst + 4 * kCodeBoxBytes + kb * kCodeKrBoxBytes, &map_kr, fb, kDC + 32 * (int)rank, y + 16 * kb,
                      pol_stream);
      }
      if (lane < kTile / 16) {
        // lane i copies block i's entry (of a page outside the pool: zeros) and arrives once it is there
        const uint32_t de = sbase + kOffEntries + stage * kEntriesBytes + 8 * lane;
        if (lane < kTile >> block_shift && MLA_SMEM_OK(de, 8)) {
          const int64_t tile = ((int64_t)pid << tile_shift) + sub;
          if (pid >= 0 && pid < num_pages)
            cp_async_8(de, entries + ((tile * kTile >> block_shift) + lane) * kEntryBytes);
          else
            asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(de), "r"(0u) : "memory");
        }
        cp_async_arrive(fb);
      }
      last_ph[stage] = (int)ph;
      __syncwarp();
      if (++stage == kCodeSlots) { stage = 0; ph ^= 1u; }
    }
    if (!ok) {
      // let every issued copy land before this CTA can exit
#pragma unroll
      for (int i = 0; i < kCodeSlots; ++i) {
        if (last_ph[i] >= 0) {
          const long long t0 = clock64();
          while (!mbar_try_wait(bar(CF0 + i), (uint32_t)last_ph[i]) && clock64() - t0 < wait_limit()) {
          }
        }
      }
    }
  };
  auto issue = [&]() {
    // ------------------------------------------------------------ MMA issuers
    // Two threads feed the tensor pipe: warp 1 the score MMAs, warp 2 the value
    // MMAs. An MMA issue stalls at the pipe's execution rate, so with one
    // issuer the pipe idled whenever that thread waited for P or for a tile;
    // with two, whichever has work ready keeps it busy. A value MMA of a page
    // follows that page's score MMAs through S -> P, so its commit (EMPTY)
    // also covers the page's score MMAs.
    if (elect()) {
      constexpr uint32_t kIdQK = idesc_f16(128, 64, false, false);
      constexpr uint32_t kIdPV = idesc_f16(128, 256, false, true);
      // descriptor templates; the start address is added per use
      const uint64_t dQK_c = smem_desc(0, 16, 1024, kSwizzle128B);
      const uint64_t dQK_r = smem_desc(0, 16, 512, kSwizzle64B);
      const uint64_t dPV_a = smem_desc(0, 16, 512, kSwizzle64B);  // the peer's half of P
      const uint64_t dPV_b = smem_desc(0, kCBoxBytes, 1024, kSwizzle128B);
      // start-address field: 14 bits of (shared address >> 4). Shared
      // addresses of the second CTA of a cluster carry high bits that must
      // not spill into the neighbouring descriptor fields.
      auto da = [](uint32_t addr) -> uint64_t { return (uint64_t)((addr >> 4) & 0x3FFFu); };
      bool ok = true;
      int g = 0, stage = 0;
      uint32_t ph = 0;
      if (warp == 1) {
        // ---- score MMAs: S = q_abs half . [c ; k^R] half of the page
        for (int it = it0; it < it1 && ok; ++it) {
          const int li = it - it0;
          const int ntiles = plan.item_tile1[it] - plan.item_tile0[it];
          // the range's query: the score readers have moved the latent and
          // positional halves from their two ring slots into tensor memory (and
          // read the slots: free them)
          if (!wait(bar(QCF), li & 1)) { ok = false; break; }
          for (int q = 0; q < kQSlots; ++q) {
            mbar_arrive(bar(EMPTY0 + stage));
            if (++stage == kOpSlots) { stage = 0; ph ^= 1u; }
          }
          for (int i = 0; i < ntiles; ++i, ++g) {
            if (!wait(bar(OPF0 + stage), ph) ||
                !wait(bar(SFREE), (g & 1) ^ 1)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d = tmem + kTmS;
            const uint64_t bc = dQK_c + da(sbase + kOffOp + stage * kOpBytes);
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
              mma_ts(d, tmem + kTmQ + ks * 8, bc + (((ks >> 2) * kCBoxBytes + (ks & 3) * 32) >> 4), kIdQK,
                     ks > 0 ? 1u : 0u);
            // positional part: A = the positional query half in tensor memory
            const uint64_t br = dQK_r + da(sbase + kOffOp + stage * kOpBytes + 4 * kCBoxBytes);
            mma_ts(d, tmem + kTmQr, br, kIdQK, 1u);
            mma_ts(d, tmem + kTmQr + 8, br + 2, kIdQK, 1u);
            mma_commit(bar(SF0 + (g & 1)));
            if (++stage == kOpSlots) { stage = 0; ph ^= 1u; }
          }
        }
      } else {
        // ---- value MMAs: O += P . C half, P from tensor memory (this CTA's
        // tokens) and from shared memory (the peer's tokens)
        for (int it = it0; it < it1 && ok; ++it) {
          const int li = it - it0;
          const int ntiles = plan.item_tile1[it] - plan.item_tile0[it];
          for (int q = 0; q < kQSlots; ++q)  // the range's query slots (released by the score issuer)
            if (++stage == kOpSlots) { stage = 0; ph ^= 1u; }
          for (int i = 0; i < ntiles; ++i, ++g) {
            const int pb = g % kPBufs;
            if (!wait(bar(PF0 + pb), (g / kPBufs) & 1)) { ok = false; break; }
            // the first value MMA of a range overwrites O: the previous range's
            // epilogue must have read it
            if (i == 0 && li > 0 && !wait(bar(OFREE), (li - 1) & 1)) { ok = false; break; }
            // arm the P buffer for page g+2; its peer half can only come after
            // this page's value MMAs (waited through PVD by the peer)
            mbar_arrive_expect_tx(bar(PF0 + pb), kPHalfBytes);
            tc_fence_after();
            const uint64_t ad = dPV_a + da(sbase + kOffP + pb * kPPeerBytes);
            const uint64_t bd = dPV_b + da(sbase + kOffOp + stage * kOpBytes);
            const uint32_t am = tmem + kTmP + 16 * pb;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint32_t acc = (i > 0 || ks > 0) ? 1u : 0u;
              if ((ks >> 1) == (int)rank)
                mma_ts(tmem + kTmO, am + 8 * (ks & 1), bd + (ks * 2048 >> 4), kIdPV, acc);
              else
                mma_ss(tmem + kTmO, ad + ((ks & 1) * 32 >> 4), bd + (ks * 2048 >> 4), kIdPV, acc);
            }
            mma_commit_multicast(bar(PVD0 + pb), 0x3);
            mma_commit(bar(EMPTY0 + stage));
            if (++stage == kOpSlots) { stage = 0; ph ^= 1u; }
          }
        }
      }
      (void)ph;
      mma_commit(bar(MMAD));
    }
    __syncwarp();
  };
  auto score = [&]() {
    // ------------------------------------------------------------ score readers and softmax
    const int quad = warp & 3;
    const int row = quad * 32 + lane;  // head row == TMEM lane
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + kTmS, tO = tmem + lane_off + kTmO;
    const uint32_t r_x = mapa(sbase + kOffX, peer), r_p = mapa(sbase + kOffP, peer);
    const uint32_t r_lx = mapa(sbase + kOffLX, peer), r_mx = mapa(sbase + kOffMX, peer);
    const uint32_t r_xf = mapa(bar(XF0), peer), r_xe = mapa(bar(XE0), peer), r_pf = mapa(bar(PF0), peer);
    const uint32_t r_lxf = mapa(bar(LXF0), peer), r_mxf = mapa(bar(MXF0), peer);
    const uint32_t r_tok = mapa(sbase + kOffTok, peer);

    if (warp < kSoft0) {
      reg_inc<kRegsRead>();
      // -------------------------------------------------------- A: score readers
      // Per page: read the peer's 32 tokens of this CTA's partial scores and send
      // them (log2 units, fp16) into the peer's shared memory.
      const int atid = threadIdx.x - 32 * kRead0;  // 0 .. 127
      const uint32_t tQ = tmem + lane_off + kTmQ;
      int g = 0;
      bool ok = true;
      for (int it = it0; it < it1 && ok; ++it) {
        const int li = it - it0;
        const int pg0 = plan.item_tile0[it];
        const int ntiles = plan.item_tile1[it] - pg0;
        const int n_att = plan.seq_len_eff[plan.item_seq[it]] - n_q + j + 1;  // tokens query j attends
        // the range's latent query half: this thread's head row from the two ring
        // slots (four [128][64] boxes, 128B-swizzled: 16-byte chunk c of row r at
        // c ^ (r % 8)) into tensor memory. The previous range's score MMAs are done
        // (this warp read the S of its last page), so Q may be overwritten.
        for (int q = 0; q < kQSlots && ok; ++q) {
          const int slot = g + kQSlots * li + q;
          if (!wait(bar(OPF0 + slot % kOpSlots), (slot / kOpSlots) & 1)) { ok = false; break; }
          const uint32_t sq = sbase + kOffOp + (slot % kOpSlots) * kOpBytes + (uint32_t)row * 128;
          (void)MLA_SMEM_OK(sq + kQBoxBytes, 128);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 8; ++c)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(r[4 * c]), "=r"(r[4 * c + 1]), "=r"(r[4 * c + 2]), "=r"(r[4 * c + 3])
                           : "r"(sq + m * kQBoxBytes + ((c ^ (row & 7)) * 16)));
            if (!q_f16) query_f16(r, row < H, err_word);
            tmem_st32(tQ + 64 * q + 32 * m, r);
          }
          if ((row >> 6) == q) {  // this row's positional half: 64 bytes, 64B-swizzled (warp-uniform)
            const uint32_t sr = sbase + kOffOp + (slot % kOpSlots) * kOpBytes + 2 * kQBoxBytes;
            const int rl = row & 63;
            uint32_t r[16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(r[4 * c]), "=r"(r[4 * c + 1]), "=r"(r[4 * c + 2]), "=r"(r[4 * c + 3])
                           : "r"(sr + rl * 64 + ((c ^ ((rl >> 1) & 3)) * 16)));
            if (!q_f16) query_f16(r, row < H, err_word);
            tmem_st16(tmem + lane_off + kTmQr, r);
          }
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(QCF));
        for (int i = 0; i < ntiles; ++i, ++g) {
          if (!wait(bar(SF0 + (g & 1)), (g >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          uint32_t r[32];
          tmem_ld32(tS + 32 * peer, r);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(bar(SFREE));
          // the peer has read this CTA's partial of page g-2 (same buffer)
          if (g >= 2) {
            if (!wait(bar(XE0 + (g & 1)), ((g >> 1) & 1) ^ 1)) { ok = false; break; }
            if (atid == 0) mbar_arrive_expect_tx(bar(XE0 + (g & 1)), kTokBytes);  // arm for this page
          }
          // The partial scores go out as fp16 offsets from the midpoint of this head's
          // values (sent in fp32): the rounding error then follows the spread of the
          // scores within the 32 tokens, not their size (a score shared by the tokens
          // costs no precision). Only tokens the query attends count toward the
          // midpoint; slack rows past the context may hold any bits.
          const int nvp = n_att - ((pg0 + i) * kTile + 32 * (int)peer);  // attended among the 32
          // (what is not attended is masked where it arrives: any of the others will do)
          if (nvp < 32) {
#pragma unroll
            for (int k = 1; k < 32; ++k)
              if (k >= nvp) r[k] = r[0];
          }
          float hi = __uint_as_float(r[0]), lo = hi;
#pragma unroll
          for (int k = 1; k < 31; k += 2) {
            hi = max3(hi, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
            lo = min3(lo, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
          }
          hi = fmaxf(hi, __uint_as_float(r[31])) * sl2;
          lo = fminf(lo, __uint_as_float(r[31])) * sl2;
          const float mid = 0.5f * lo + 0.5f * hi;
          if (kRows && row < H && 0.5f * hi - 0.5f * lo >= 65520.f && hi < INFINITY && lo > -INFINITY)
            report_error(err_word, MLA_ERR_RANGE);
          const uint32_t xoff = (uint32_t)(g & 1) * kXBytes;
          const uint32_t xa = r_x + xoff + (uint32_t)row * 16;
          const uint32_t xf = r_xf + 8u * (uint32_t)(g & 1);
          if (MLA_SMEM_OK(sbase + kOffX + xoff + (uint32_t)row * 16 + 3 * 128 * 16, 16) &&
              MLA_SMEM_OK(sbase + kOffX + xoff + kXDataBytes + (uint32_t)row * 4, 4)) {
            const uint64_t by = pair(sl2, sl2), off = pair(-mid, -mid);
            auto offset = [&](int k) -> uint32_t {  // tokens k and k + 1
              const float2 e = unpair(fma2(pair(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), by, off));
              return cvt_f16x2(e.x, e.y);
            };
#pragma unroll
            for (int q8 = 0; q8 < 4; ++q8) {
              uint4 w;
              w.x = offset(8 * q8);
              w.y = offset(8 * q8 + 2);
              w.z = offset(8 * q8 + 4);
              w.w = offset(8 * q8 + 6);
              st_async_v4(xa + q8 * 128 * 16, w, xf);
            }
            st_async_b32(r_x + xoff + kXDataBytes + (uint32_t)row * 4, __float_as_uint(mid), xf);
          }
        }
      }
    } else {
      reg_inc<kRegsSoftmax>();
      // -------------------------------------------------------- B: softmax + epilogue
      // Two groups of four warps (one per TMEM lane quadrant) take alternate
      // pages: group grp handles the pages g with g % 2 == grp, one thread per
      // head row and all 32 of this CTA's tokens of the page, so one group's
      // exchanges with the peer overlap the other group's arithmetic. Through
      // shared memory the groups pass the reference maximum of each head
      // (decided page by page, in page order) and, at the end of a range, the
      // softmax sum of the group that does not write the output.
      const int grp = (warp - kSoft0) >> 2;
      const int gwarp = (warp - kSoft0) & 3;
      const int gtid = gwarp * 32 + lane;  // 0 .. 127
      const uint32_t vec_off = (uint32_t)row * 4;
      float x[32];
      float l_g = 0.f, m_l = -INFINITY;  // this group's sum over the range so far, on reference m_l
      int g = 0, lg_n = 0, iv_n = 0;
      bool ok = true;
      // The group that does not handle a range's last page drains columns
      // [128, 256) of O at the range switch, once the other group has posted 1/l.
      // O columns [128 half, 128 half + 128) of this CTA's half, scaled by inv,
      // as fp16 into the head-minor partials o_part[item][j][column / 8][head][column % 8]
      // (each warp store is 512 contiguous bytes).
      auto drain_o = [&](int it, int half, float inv) {
        uint4* dst = reinterpret_cast<uint4*>(plan.o_part) +
                     ((size_t)(it * n_q + j) * (kDC / 8) + (256 * rank + 128 * half) / 8) * H + row;
        float amax = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + 128 * half + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = __uint_as_float(r[8 * v + e]) * inv;
              amax = fmaxf(amax, fabsf(f[e]));
            }
            if (row < H)
              dst[(size_t)(4 * c + v) * H] = make_uint4(cvt_f16x2(f[0], f[1]), cvt_f16x2(f[2], f[3]),
                                                       cvt_f16x2(f[4], f[5]), cvt_f16x2(f[6], f[7]));
          }
        }
        // a partial beyond the fp16 range would turn into infinity
        if (row < H && !(amax <= 65504.f)) report_error(err_word, MLA_ERR_RANGE);
      };
      for (int it = it0; it < it1 && ok; ++it) {
        const int li = it - it0;
        const int b = plan.item_seq[it], pg0 = plan.item_tile0[it], pg1 = plan.item_tile1[it];
        const int L = plan.seq_len_eff[b];
        const int n_att = L - n_q + j + 1;
        const int ntiles = pg1 - pg0;
        bool fresh = true;  // no page of this range handled by this group yet
        for (int i = 0; i < ntiles && ok; ++i, ++g) {
          if ((g & 1) != grp) {
            if (i == ntiles - 1) {
              // helper at the end of the range handled by the other group
              if (!wait(bar(IVF0 + grp), iv_n & 1)) { ok = false; break; }
              ++iv_n;
              float inv;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(inv) : "r"(sbase + kOffIV + vec_off));
              if (!wait(bar(PVD0 + g % kPBufs), (g / kPBufs) & 1)) { ok = false; break; }
              tc_fence_after();
              drain_o(it, 1, inv);
              tc_fence_before();
              mbar_arrive(bar(OFREE));
            }
            continue;
          }
          const int xb = g & 1;
          // this CTA's partial scores of its 32 tokens
          const int nv = n_att - ((pg0 + i) * kTile + 32 * (int)rank);  // valid tokens among these 32
          if (!wait(bar(SF0 + xb), (g >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          {
            uint32_t r[32];
            tmem_ld32(tS + 32 * rank, r);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 32; ++v) x[v] = __uint_as_float(r[v]);  // scaled below
          }
          tc_fence_before();
          mbar_arrive(bar(SFREE));
          // add the peer's partial for these tokens: its midpoint plus the fp16 offsets
          if (!wait(bar(XF0 + xb), (g >> 1) & 1)) { ok = false; break; }
          if (gtid == 0) mbar_arrive_expect_tx(bar(XF0 + xb), kXBytes);  // arm for page g+2
          float mid_p;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(mid_p) : "r"(sbase + kOffX + xb * kXBytes + kXDataBytes + vec_off));
#pragma unroll
          for (int q8 = 0; q8 < 4; ++q8) {
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(sbase + kOffX + xb * kXBytes + (uint32_t)((q8 * 128 + row) * 16)));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * q8 + 2 * k;
              const float2 f = unpair(fma2(pair(x[e], x[e + 1]), pair(sl2, sl2), f16x2_plus(ww[k], mid_p)));
              x[e] = f.x;
              x[e + 1] = f.y;
            }
          }
          __syncwarp();
          // tell the peer this warp has read its partial (a 4-byte token completes
          // the peer's barrier; the loads above have all returned by now)
          if (lane == 0) st_async_b32(r_tok + (uint32_t)gwarp * 4, 1u, r_xe + 8u * xb);
          if (nv < 32) {
#pragma unroll
            for (int jj = 0; jj < 32; ++jj)
              if (jj >= nv) x[jj] = -INFINITY;
          }
          // both CTAs' value MMAs of page g-3 are done: P buffer g % 3 is free. (Its
          // previous phase, page g-6, is complete: the value MMAs complete in page
          // order and this group waited for page g-5 at page g-2.)
          const int pb = g % kPBufs;
          if (g >= kPBufs && !wait(bar(PVD0 + pb), ((g / kPBufs) & 1) ^ 1)) { ok = false; break; }
          const int rows_valid = n_att - (pg0 + i) * kTile;
          if (rows_valid < kTile) {
            // rows past what the query sees may hold any bits: zero this CTA's latent
            // half so 0-weight x NaN cannot reach O. The score MMAs have read the
            // stage (SF); the value MMAs read it after this group's P-ready arrive.
            const int stage = (g + kQSlots * (li + 1)) % kOpSlots;  // operand slot of page g
            const uint32_t sa = sbase + kOffOp + stage * kOpBytes;
            (void)MLA_SMEM_OK(sa, 4 * kCBoxBytes);
            const int nz = (kTile - rows_valid) * 4 * 8;  // 16-byte chunks
            for (int z = gtid; z < nz; z += kGThreads) {
              const int rr = rows_valid + z / 32, cb = (z / 8) & 3, ch = z & 7;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sa + cb * kCBoxBytes + rr * 128 + ch * 16),
                           "r"(0u)
                           : "memory");
            }
            fence_proxy_async_smem();
          }
          float m = x[0];
#pragma unroll
          for (int jj = 1; jj < 31; jj += 2) m = max3(m, x[jj], x[jj + 1]);
          m = fmaxf(m, x[31]);
          st_async_b32(r_mx + xb * kVecBytes + vec_off, __float_as_uint(m), r_mxf + 8u * xb);
          if (!wait(bar(MXF0 + xb), (g >> 1) & 1)) { ok = false; break; }
          if (gtid == 0) mbar_arrive_expect_tx(bar(MXF0 + xb), kVecBytes);
          float m_p;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(m_p) : "r"(sbase + kOffMX + xb * kVecBytes + vec_off));
          const float mt = fmaxf(m, m_p);
          // the reference maximum: the previous page's decision (the other group's)
          // is raised lazily, only when this page exceeds it by the threshold
          if (g >= 1 && !wait(bar(MRF), (g - 1) & 1)) { ok = false; break; }
          float m_new = mt, alpha = 1.f;
          bool need = false;
          if (i > 0) {
            float m_prev;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(m_prev) : "r"(sbase + kOffMR + vec_off));
            m_new = m_prev;
            if (mt > m_prev + kRescaleThreshold) {
              alpha = ex2(m_prev - mt);
              m_new = mt;
              need = true;
            }
          }
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sbase + kOffMR + vec_off), "f"(m_new) : "memory");
          mbar_arrive(bar(MRF));
          if (__any_sync(0xffffffffu, need)) {
#if MLA_DEBUG_CHECKS
            if (lane == 0) atomicAdd(&g_dbg_counters[0], 1ull);
#endif
            // O must hold every earlier page before it is rescaled
            if (!wait(bar(PVD0 + (g - 1) % kPBufs), ((g - 1) / kPBufs) & 1)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t r[32];
              tmem_ld32(tO + 32 * c, r);
              tmem_wait_ld();
#pragma unroll
              for (int v = 0; v < 32; ++v) r[v] = __float_as_uint(__uint_as_float(r[v]) * alpha);
              tmem_st32(tO + 32 * c, r);
            }
          }
          // this group's running sum, on the new reference
          if (fresh) {
            l_g = 0.f;
            m_l = m_new;
            fresh = false;
          } else if (m_l != m_new) {
            if (l_g != 0.f) l_g *= ex2(m_l - m_new);
            m_l = m_new;
          }
          const float mref = m_new == -INFINITY ? 0.f : m_new;  // all masked so far: every p is 0
          // P: into tensor memory for this CTA's value MMAs and into the peer's
          // shared memory (64B-swizzled, K-major) for its own
          const uint32_t pr = r_p + pb * kPPeerBytes + (uint32_t)row * 64;
          const uint32_t pfr = r_pf + 8u * pb;
          (void)MLA_SMEM_OK(sbase + kOffP + pb * kPPeerBytes + (uint32_t)row * 64, 64);
          (void)MLA_TMEM_OK(kTmP + 16 * pb, 16);
          // (the sum of the weights before their rounding to fp16. A rounded weight is off by 2^-11 of itself at
          // most, and below 2^-21 of the reference by 2^-32 of that, which is at most the sum: of n tokens the
          // sum of the rounded ones is off by 2^-11 + n 2^-32 of itself. Summed after their rounding, the
          // same cases were off as much in u, up to 0.3% more in lse, and steps took 1 to 2% longer.)
          uint64_t sum = pair(0.f, 0.f);
          const uint64_t off = pair(kWeightShift - mref, kWeightShift - mref);
          uint32_t pw[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const float2 d = unpair(add2(pair(x[2 * v], x[2 * v + 1]), off));
            const float p0 = ex2(d.x), p1 = ex2(d.y);
            pw[v] = cvt_f16x2(p0, p1);
            sum = add2(sum, pair(p0, p1));
          }
          const float2 lsum = unpair(sum);
          tmem_st16(tmem + lane_off + kTmP + 16 * pb, pw);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_async_v4(pr + (uint32_t)((c ^ ((row >> 1) & 3)) * 16),
                        make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]), pfr);
          tmem_wait_st();
          l_g += lsum.x + lsum.y;
          tc_fence_before();
          mbar_arrive(bar(PF0 + pb));
          if (i == ntiles - 2) {
            // the other group handles the last page of the range: hand over this sum
            const uint32_t lg = sbase + kOffLG + (uint32_t)(lg_n & 1) * 2 * kVecBytes;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(lg + vec_off), "f"(l_g) : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(lg + kVecBytes + vec_off), "f"(m_l) : "memory");
            mbar_arrive(bar(LGF0 + (lg_n & 1)));
          }
          if (i == ntiles - 1) {
            // epilogue: the CTA's sum (both groups), the peer's, the normalised output
            float l_c = l_g;
            if (ntiles >= 2) {
              if (!wait(bar(LGF0 + (lg_n & 1)), (lg_n >> 1) & 1)) { ok = false; break; }
              const uint32_t lg = sbase + kOffLG + (uint32_t)(lg_n & 1) * 2 * kVecBytes;
              float l_o, m_o;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(l_o) : "r"(lg + vec_off));
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(m_o) : "r"(lg + kVecBytes + vec_off));
              if (l_o != 0.f) l_c += l_o * ex2(m_o - m_new);
            }
            const int lb = li & 1;
            st_async_b32(r_lx + lb * kVecBytes + vec_off, __float_as_uint(l_c), r_lxf + 8u * lb);
            if (!wait(bar(LXF0 + lb), (li >> 1) & 1)) { ok = false; break; }
            if (gtid == 0) mbar_arrive_expect_tx(bar(LXF0 + lb), kVecBytes);  // arm for range li+2
            float l_p;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(l_p) : "r"(sbase + kOffLX + lb * kVecBytes + vec_off));
            // the same addition in the same order in both CTAs: rank 0's sum first
            const float l_tot = rank == 0 ? l_c + l_p : l_p + l_c;
            const float inv = l_tot > 0.f ? 1.f / l_tot : 0.f;
            // 1/l for the helper group, which drains the other half of O
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sbase + kOffIV + vec_off), "f"(inv) : "memory");
            mbar_arrive(bar(IVF0 + (grp ^ 1)));
            if (!wait(bar(PVD0 + pb), (g / kPBufs) & 1)) { ok = false; break; }
            tc_fence_after();
            const size_t orow = ((size_t)it * n_q + j) * H + row;
            drain_o(it, 0, inv);
            tc_fence_before();
            mbar_arrive(bar(OFREE));
            if (rank == 0 && row < H)
              // a chunk's row keeps a sum that is not a number, so that the merge passes it on
              plan.lse_part[orow] =
                  l_tot > 0.f ? (m_new + log2f(l_tot * 0x1p-7f)) * kLn2 : (kRows && l_tot != l_tot ? l_tot : -INFINITY);
          }
        }
        if (ntiles >= 2) ++lg_n;
      }
    }
  };
  auto widen = [&]() {
    // ------------------------------------------------------------ wideners
    // They hand out the operand slots in ring order. A query's two slots are filled by TMA; a tile's codes become
    // the fp16 half that the MMAs read, in the swizzled layout of decode_tc.cu's boxes. The code stays short:
    // longer code kept the other roles waiting for their instructions.
    const int wtid = threadIdx.x - 32 * kWide0;  // 0 .. 383
    // 16-byte chunks q = wtid + 384 k of the 1152 of a tile's half: q < 1024: box q / 256, token q / 4 % 64, 16 of
    // its 64 columns; then the positional box: token (q - 1024) / 2, 16 of its 32 columns (64B swizzle)
    constexpr int kChunks = kCodeBytes / 16 / kWThreads;
    static_assert(kChunks * kWThreads * 16 == kCodeBytes, "the same number for every thread");
    // where a chunk's first eight values go (the other eight: 16 bytes on or back), and its power's place
    uint32_t to[kChunks], at[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const uint32_t q = wtid + kWThreads * k, latent = q < 1024;
      const uint32_t t = latent ? q >> 2 & 63 : (q - 1024) >> 1, kk = latent ? 2 * (q & 3) : 2 * (q & 1);
      to[k] = latent ? (q >> 8) * kCBoxBytes + t * 128 + (kk ^ (t & 7)) * 16
                     : 4 * kCBoxBytes + t * 64 + (kk ^ (t >> 1 & 3)) * 16;
      at[k] = (t >> block_shift) * kEntryBytes + (latent ? 2 * rank + (q >> 9) : 4u);
    }
    int slot = 0, page = 0;  // uses of operand slots, and of slots of codes
    int asked = 0;           // uses of operand slots up to the last query's
    bool ok = true;
    auto next_slot = [&]() -> bool {  // the next operand slot, once its last use is over
      const bool free = wait(bar(EMPTY0 + slot % kOpSlots), ((slot / kOpSlots) & 1) ^ 1);
      if (!free) ok = false;
      return free;
    };
    for (int it = it0; it < it1 && ok; ++it) {
      const int ntiles = plan.item_tile1[it] - plan.item_tile0[it];
      const int seq = plan.item_seq[it], qrow = (seq * n_q + j) * H;
      const int end = plan.seq_len_eff[seq] - plan.item_tile0[it] * kTile;  // of the context, from the first tile on
      for (int q = 0; q < kQSlots && next_slot(); ++q, ++slot) {
        // as the producer of the bf16 path: latent boxes [128 heads][64] for columns 256r + 128q + {0, 64}
        // and positional rows [64q, 64q + 64) of columns 512 + 32r
        const uint32_t fb = bar(OPF0 + slot % kOpSlots), dst = sbase + kOffOp + (slot % kOpSlots) * kOpBytes;
        if (wtid == 0 && MLA_SMEM_OK(dst, kOpBytes)) {
          const uint64_t keep = policy_evict_last();
          mbar_arrive_expect_tx(fb, 2 * kQBoxBytes + kQrBoxBytes);
          for (int m = 0; m < 2; ++m)
            tma_load_2d(dst + m * kQBoxBytes, &map_q, fb, 256 * (int)rank + 128 * q + 64 * m, qrow, keep);
          tma_load_2d(dst + 2 * kQBoxBytes, &map_qkr, fb, kDC + 32 * (int)rank, qrow + 64 * q, keep);
          asked = slot + 1;
        } else if ((wtid & 31) == 0) {
          mbar_arrive(fb);
        }
      }
      for (int i = 0; i < ntiles && ok; ++i, ++slot, ++page) {
        const int cs = page % kCodeSlots;
        if (!wait(bar(CF0 + cs), (page / kCodeSlots) & 1)) { ok = false; break; }
        const uint32_t sc = sbase + kOffCode + cs * kCodeBytes + wtid * 16;
        const uint32_t se = sbase + kOffEntries + cs * kEntriesBytes;
        const uint32_t dst = sbase + kOffOp + (slot % kOpSlots) * kOpBytes;
        uint32_t v[kChunks][4], p[kChunks], o[8] = {};
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          ld_shared_v4(sc + 16 * kWThreads * k, v[k][0], v[k][1], v[k][2], v[k][3]);
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(p[k]) : "r"(se + at[k]));
        }
        if (!next_slot()) break;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const bool beyond = widen16(v[k], power_f16x2(p[k]), p[k], o);
          const uint32_t a0 = dst + to[k], a1 = a0 ^ 16u;
          if (beyond) {
            const int q = wtid + kWThreads * k, t = q < 1024 ? q >> 2 & 63 : (q - 1024) >> 1;
            if (t < end - i * kTile) report_error(err_word, MLA_ERR_RANGE);  // a token of the context
          }
          if (MLA_SMEM_OK(a0, 16) && MLA_SMEM_OK(a1, 16)) {
            st_shared_v4(a0, o[0], o[1], o[2], o[3]);
            st_shared_v4(a1, o[4], o[5], o[6], o[7]);
          }
        }
        fence_proxy_async_smem();  // read by the MMAs (async proxy)
        __syncwarp();
        if ((wtid & 31) == 0) {
          mbar_arrive(bar(CE0 + cs));
          mbar_arrive(bar(OPF0 + slot % kOpSlots));
        }
      }
    }
    if (!ok && wtid == 0) {
      // let the last query's copies land before this CTA can exit (where another thread gave up before
      // it arrived, the limit ends the wait)
      const long long start = clock64();
      for (int u = asked > kQSlots ? asked - kQSlots : 0; u < asked; ++u)
        while (!mbar_try_wait(bar(OPF0 + u % kOpSlots), (u / kOpSlots) & 1) && clock64() - start < wait_limit()) {
        }
    }
  };
  // (whole warpgroups change their registers; the score part does so by role)
  if (warp < kRead0) {
    reg_dec<kRegsIssue>();
    if (warp == 0) produce();
    else if (warp < 3) issue();
  } else if (warp < kWide0) {
    score();
  } else {
    reg_dec<kRegsWiden>();
    widen();
  }

  // ------------------------------------------------------------ teardown
  if (warp == 1 && lane == 0) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar(MMAD), 0) && clock64() - t0 < kWaitLimitCycles) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) report_error(err_word, MLA_ERR_TIMEOUT);
  cluster_sync();  // the peer has finished writing into this CTA's shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

}  // namespace

// ---------------------------------------------------------------- host side
namespace {
template <bool kRows>
cudaError_t launch_as(const uint16_t* q_abs, bool q_f16, const uint8_t* cache8, const BlockScales& scales,
                      const int32_t* block_table, int B, int n_q, int H, int num_pages, int page_size, int max_pages,
                      float scale, int G, const Plan& plan, int32_t* err_word, cudaStream_t s) {
  CUtensorMap map_c, map_kr, map_qkr, map_q;
  const uint64_t cache_dims[2] = {kRow, (uint64_t)num_pages * page_size}, q_dims[2] = {kRow, (uint64_t)B * n_q * H};
  const uint64_t code_stride[1] = {kRow}, q_stride[1] = {kRow * 2};
  const uint32_t box_c[2] = {64, 64}, box_kr[2] = {32, 16}, box_qkr[2] = {32, 64}, box_q[2] = {64, 128};
  if (!make_tmap(&map_c, cache8, 2, cache_dims, code_stride, box_c, 0, true) ||
      !make_tmap(&map_kr, cache8, 2, cache_dims, code_stride, box_kr, 0, true) ||
      !make_tmap(&map_qkr, q_abs, 2, q_dims, q_stride, box_qkr, 64) ||
      !make_tmap(&map_q, q_abs, 2, q_dims, q_stride, box_q, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = smem_limit<decode_blocks_kernel<kRows>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  const float sl2 = scale * 1.4426950408889634f;
  return launch_pdl(decode_blocks_kernel<kRows>, dim3(2 * G, n_q, 1), dim3(kThreads), kSmemBytes, s, map_c, map_kr,
                    map_qkr, map_q, block_table, n_q, H, max_pages, num_pages, page_size == 2 * kTile ? 1 : 0,
                    scales.shift, q_f16 ? 1 : 0, sl2, plan, static_cast<const uint8_t*>(scales.entries), err_word,
                    plan.seq_row);
}
}  // namespace

cudaError_t launch_decode_blocks(const uint16_t* q_abs, bool q_f16, const uint8_t* cache8, const BlockScales& scales,
                                 const int32_t* block_table, int B, int n_q, int H, int num_pages, int page_size,
                                 int max_pages, float scale, int G, const Plan& plan, int32_t* err_word,
                                 cudaStream_t s) {
  return (plan.seq_row ? launch_as<true> : launch_as<false>)(q_abs, q_f16, cache8, scales, block_table, B, n_q, H,
                                                             num_pages, page_size, max_pages, scale, G, plan, err_word,
                                                             s);
}

#if MLA_DEBUG_CHECKS
cudaError_t debug_decode_blocks(const long long* limit, const int* skip_producer, unsigned long long* counters, int n) {
  cudaError_t e = sm100::debug_set(limit, nullptr);
  if (e == cudaSuccess && skip_producer)
    e = cudaMemcpyToSymbol(g_dbg_skip_producer, skip_producer, sizeof(*skip_producer));
  if (e == cudaSuccess && counters && n < 0) {  // set to zero
    const unsigned long long zero[4] = {0, 0, 0, 0};
    e = cudaMemcpyToSymbol(g_dbg_counters, zero, sizeof(zero));
  } else if (e == cudaSuccess && counters) {
    e = cudaMemcpyFromSymbol(counters, g_dbg_counters, sizeof(unsigned long long) * (size_t)n);
  }
  return e;
}
#endif

}  // namespace mla

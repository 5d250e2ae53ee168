// Block tables, the pages that sequences hold, a stack of free pages and the slots of
// new tokens, brought up to date from the sequences' lengths on the GPU:
//   need_b = ceil(lens_b / page_size); where held_b is larger the pages past need_b
//   go back to the stack, where it is smaller the missing ones are taken from it;
//   slots[cu_b + i] = table_b[pos / page_size] * page_size + pos % page_size,
//   pos = lens_b - n_b + i.
// Pages given back are numbered q = 0 .. R - 1 and pages taken k = 0 .. K - 1, both in
// order of the sequences and of the pages in each. The given back lie on the stack of F
// free pages with q = 0 on top (q at F + R - 1 - q), and k takes from the top: k < R is
// q = k, then the stack's own, k at F - 1 - (k - R). So a step and the step back leave
// stack and tables as they were, and the result does not depend on timing. Sequences
// are served whole and in order: one whose pages would pass F + R gets none, nor
// does one behind it.
//
// Latency-bound: a step of a few hundred sequences moves some kilobytes. One block
// counts and scans (three running sums over the sequences), then the pages are dealt out
// to groups of eight lanes (without slots: to lanes), a page with the slots in it to a group; no two
// groups touch one entry: a page that goes from one sequence to another in the same call is
// read and cleared by the group that takes it. While the slots are few one block does
// it all (one launch); else every block of a grid scans for itself, in its shared memory, and deals out its part,
// and a last block updates `held` and the count, which the grid's blocks have to read as they were.
// Measured: 32 sequences 3.9 us a call in a graph, about a launch; 2048 sequences, prompts of up to 4096 tokens
// started in an eighth of them, 11.6 us, and 11.6 a call from Python. One scan handed to the grid through a workspace:
// 9.8 in a graph but 15 from Python, which has to allocate it. One cluster of 8 or 16 CTAs: 23 and 16. Warp totals
// added by one reduction each save 0.4 us over five shuffles. The one block without slots, all
// pages taken or given back: 2048 pages 4.3 us, 8192 7.4, 65536 47 (a page to eight lanes, one read after another: 9.5,
// 28, 239).
#include "blocks.cuh"
#include "chunk.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
static_assert(MLA_MAX_BATCH == 4 * kThreads, "one, two or four sequences a thread");
constexpr int kLanesOfAPage = 8;  // with slots to fill
constexpr int kGridBlocks = 152;
// One launch up to these sizes.
constexpr int kSmallRows = 4096, kSmallBatch = 1024;
static_assert(kSmallBatch <= kThreads, "a sequence a thread");

struct alignas(32) Sequence {  // one read of what a page's group needs
  int32_t page0;   // its first page
  int32_t held;    // pages held before
  int32_t need;    // ... and after
  int32_t row0;    // row of its first new token
  int32_t pos0;    // ... and its position
  int32_t end;     // the context's length; its new tokens are pos0 .. end - 1
  int32_t refused;
  int32_t taken;   // pages taken by those before
};
__device__ __forceinline__ void put(Sequence* to, const Sequence& s) {
  reinterpret_cast<int4*>(to)[0] = make_int4(s.page0, s.held, s.need, s.row0);
  reinterpret_cast<int4*>(to)[1] = make_int4(s.pos0, s.end, s.refused, s.taken);
}
__device__ __forceinline__ Sequence get(const Sequence* from) {
  const int4 a = reinterpret_cast<const int4*>(from)[0], b = reinterpret_cast<const int4*>(from)[1];
  return Sequence{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
struct Work {  // in shared memory
  int32_t* give;   // [B] pages given back by the sequences before
  int32_t* unit;   // [B] pages worked on for those before
  Sequence* seq;   // [B]
  int32_t* total;  // [4] free pages before, given back, taken, units
};

// the last i in [0, n) with sum[i] <= x (sum[0] = 0 <= x)
__device__ __forceinline__ int last_at(const int32_t* sum, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The pages, each by one group of lanes; then the pages given back and not taken, each
// by a thread; then the rows behind the last sequence.
template <int kLanes>
__device__ __forceinline__ void deal_pages(const Pages& p, const Work& w, int thread, int threads, int32_t* err_word) {
  const int F = w.total[0], R = w.total[1], K = w.total[2], units = w.total[3];
  const int32_t *give = w.give, *unit = w.unit;
  const int lane = thread % kLanes, shift = p.page_shift;
  const uint32_t group = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) & ~(kLanes - 1));
  bool bad = false;
  for (int i = thread / kLanes; i < units; i += threads / kLanes) {
    const int b = last_at(unit, p.B, i);
    const Sequence s = get(w.seq + b);
    const int pi = s.page0 + i - unit[b];
    int32_t* place = p.block_table + (int64_t)b * p.max_pages + pi;
    int page = -1;
    if (pi < s.held) {
      page = *place;
    } else if (pi < s.need) {
      const int k = s.taken + pi - s.held;
      if (k < R) {
        const int from = last_at(give, p.B, k);
        int32_t* old = p.block_table + (int64_t)from * p.max_pages + w.seq[from].need + k - give[from];
        page = *old;
        __syncwarp(group);  // every lane has read it
        if (lane == 0) *old = -1;
      } else {
        page = p.free_pages[F - 1 - (k - R)];
      }
      if (lane == 0) *place = page;
    }
    const bool good = page >= 0 && page < p.num_pages && !s.refused;
    bad |= !good && !s.refused;
    const int a = max(s.pos0, pi << shift), e = min(s.end, (pi + 1) << shift);
    for (int pos = a + lane; pos < e; pos += kLanes)
      p.slots[s.row0 + pos - s.pos0] = good ? (int64_t)(page - pi) * (1 << shift) + pos : -1;
  }
  constexpr int kAtOnce = 4;  // one read after another cost 2 us for every 8192 pages
  for (int q0 = K + thread; q0 < R; q0 += kAtOnce * threads) {
    int32_t* old[kAtOnce];
    int page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int q = q0 + k * threads;
      if (q >= R) break;
      const int b = last_at(give, p.B, q);
      old[k] = p.block_table + (int64_t)b * p.max_pages + w.seq[b].need + q - give[b];
      page[k] = *old[k];
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int q = q0 + k * threads;
      if (q >= R) break;
      bad |= page[k] < 0 || page[k] >= p.num_pages;
      p.free_pages[F + R - 1 - q] = page[k];
      *old[k] = -1;
    }
  }
  if (p.slots)
    for (int t = max(p.cu[p.B], 0) + thread; t < p.n_rows; t += threads) p.slots[t] = -1;
  if (bad) report_error(err_word, MLA_ERR_BOUNDS);
}

// Sums that stay at kMany once they reach it: more pages than a pool can have (2^25).
constexpr int kMany = 1 << 26;
__device__ __forceinline__ int plus(int a, int b) { return min(a + b, kMany); }

// Exclusive sums over the block's threads of kN values each (at most kMany), in v; the totals in all.
// A warp's 32 values, and the 32 warps' sums, add up to 2^31 at most: they saturate once they are added.
template <int kN>
__device__ __forceinline__ void block_scan(int (&v)[kN], int (&all)[kN], int (*shared)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const uint32_t own = v[k];
    uint32_t x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) shared[warp][k] = min(x, (uint32_t)kMany);
    v[k] = min(x - own, (uint32_t)kMany);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kN; ++k) {  // every warp adds up the warps' sums for itself
    const uint32_t y = shared[lane][k];
    all[k] = min(__reduce_add_sync(0xffffffffu, y), (uint32_t)kMany);
    v[k] = plus(v[k], min(__reduce_add_sync(0xffffffffu, lane < warp ? y : 0u), (uint32_t)kMany));
  }
}

// Every block counts and scans all sequences for itself. kAlone: one block does everything; kDeal: a grid
// that deals out the pages and leaves `held` and the count as its other blocks still have to read them; kState:
// one block, after that grid, that updates these two.
enum Way { kAlone, kDeal, kState };
// kPer: sequences a thread
template <int kPer, Way kWay>
__global__ void __launch_bounds__(kThreads)
update_pages_kernel(Pages p, int32_t* err_word) {
  __shared__ int sums[32][2], unit_sums[32][1];
  __shared__ int served;  // pages taken in all
  __shared__ int refused;  // some sequence is short of pages
  __shared__ int32_t total[4];
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kMost = kPer * kThreads;
  const Work w = {reinterpret_cast<int32_t*>(smem + kMost * sizeof(Sequence)),
                  reinterpret_cast<int32_t*>(smem + kMost * (sizeof(Sequence) + 4)), reinterpret_cast<Sequence*>(smem),
                  total};
  sm100::grid_dependency_wait();
  sm100::grid_launch_dependents();
  const int tid = threadIdx.x, b0 = tid * kPer;
  const int shift = p.page_shift, round = (1 << shift) - 1, max_tokens = p.max_pages << shift;
  if (tid == 0) served = refused = 0;
  int F = *p.free_count;
  bool bad = false;
  Sequence s[kPer];
  int moved[2] = {0, 0}, all[2];  // pages given back, taken
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    s[i] = Sequence{};
    s[i].refused = 1;
    if (b >= p.B) continue;
    const int L = p.lens[b], h = p.held[b];
    int c0 = 0, n = 0;
    bool ok = L >= 0 && L <= max_tokens && h >= 0 && h <= p.max_pages;
    if (p.slots) {
      const int a = p.cu[b], e = p.cu[b + 1];
      c0 = min(max(a, 0), p.n_rows);
      n = min(max(e, c0), p.n_rows) - c0;
      ok = ok && a == c0 && e == c0 + n && (b > 0 || a == 0);
    }
    ok = ok && n <= L;
    bad |= !ok;
    // a sequence whose numbers are out of range is left as it is
    s[i].held = ok ? h : 0;
    s[i].need = ok ? (L + round) >> shift : 0;
    s[i].row0 = c0;
    s[i].end = ok ? L : n;
    s[i].pos0 = s[i].end - n;
    s[i].refused = !ok;
    moved[0] = plus(moved[0], max(s[i].held - s[i].need, 0));
    moved[1] = plus(moved[1], max(s[i].need - s[i].held, 0));
  }
  block_scan<2>(moved, all, sums);
  int g = moved[0], k = moved[1];
  if (F < 0 || F > p.num_pages) {
    bad = true;
    F = min(max(F, 0), p.num_pages);
  }
  // more pages than there are: some are held or free twice, and nothing is moved
  const bool broken = F + all[0] > p.num_pages;
  bad |= broken;
  const int R = broken ? 0 : all[0], room = broken ? 0 : F + R;
  int units[1] = {0}, all_units[1];
  int gives[kPer], count[kPer], most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int held = s[i].held, back = max(held - s[i].need, 0), more = max(s[i].need - held, 0);
    gives[i] = broken ? 0 : g;
    s[i].taken = k;
    g = plus(g, back);
    k = plus(k, more);
    if (more > 0 && !broken) {
      if (k > room) {
        s[i].refused = 1;
        refused = 1;
      } else {
        most = k;
      }
    }
    if (broken) s[i].refused = 1;
    if (s[i].refused) {
      s[i].need = held;
    } else if (s[i].need != held && kWay != kDeal) {
      p.held[b0 + i] = s[i].need;
    }
    const int n = s[i].end - s[i].pos0;
    int u0 = n > 0 ? s[i].pos0 >> shift : INT32_MAX, u1 = n > 0 ? (s[i].end + round) >> shift : 0;
    if (s[i].need > held) {
      u0 = min(u0, held);
      u1 = max(u1, s[i].need);
    }
    s[i].page0 = u0;
    count[i] = max(u1 - u0, 0);
    units[0] = plus(units[0], count[i]);
  }
  if (most > 0) atomicMax(&served, most);
  block_scan<1>(units, all_units, unit_sums);
  if (kWay != kDeal && tid == 0 && R != served) *p.free_count = F + R - served;
  // MLA_ERR_BOUNDS is told before MLA_ERR_NO_PAGES, whichever thread or block finds it: the latter by the last
  // block to run, once all of its threads have told the former.
  if (kWay != kDeal && bad) report_error(err_word, MLA_ERR_BOUNDS);
  auto tell_refused = [&]() {
    if (kWay == kDeal || !refused) return;
    __syncthreads();
    if (tid == 0) report_error(err_word, MLA_ERR_NO_PAGES);
  };
  if (kWay == kState) {
    tell_refused();
    return;
  }
  int u = units[0];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (b < p.B) {
      w.give[b] = gives[i];
      w.unit[b] = u;
      put(w.seq + b, s[i]);
    }
    u = plus(u, count[i]);
  }
  if (tid == 0) {
    w.total[0] = F;
    w.total[1] = R;
    w.total[2] = served;
    w.total[3] = all_units[0];
  }
  __syncthreads();
  const int thread = blockIdx.x * kThreads + tid, threads = gridDim.x * kThreads;
  if (p.slots) deal_pages<kLanesOfAPage>(p, w, thread, threads, err_word);
  else deal_pages<1>(p, w, thread, threads, err_word);
  tell_refused();
}

template <int kPer>
cudaError_t deal_and_update(const Pages& p, int32_t* err_word, cudaStream_t s) {
  constexpr size_t kSmem = (size_t)kPer * kThreads * (sizeof(Sequence) + 8);
  cudaError_t e = smem_limit<update_pages_kernel<kPer, kDeal>>(kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(update_pages_kernel<kPer, kDeal>, dim3(kGridBlocks), dim3(kThreads), kSmem, s, p, err_word);
  if (e == cudaSuccess) e = launch_pdl(update_pages_kernel<kPer, kState>, dim3(1), dim3(kThreads), 0, s, p, err_word);
  return e;
}

}  // namespace

cudaError_t launch_update_pages(const Pages& p, int32_t* err_word, cudaStream_t s) {
  if (p.n_rows <= kSmallRows && p.B <= kSmallBatch)
    return launch_pdl(update_pages_kernel<1, kAlone>, dim3(1), dim3(kThreads), kThreads * (sizeof(Sequence) + 8), s, p,
                      err_word);
  return (p.B <= kThreads       ? deal_and_update<1>
          : p.B <= 2 * kThreads ? deal_and_update<2>
                                : deal_and_update<4>)(p, err_word, s);
}

}  // namespace mla

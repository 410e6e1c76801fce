// sample.cu -- sampled decoding: a token of every position by temperature, min-p,
// top-k and top-p from a given random number, and the accepted prefix of a verify's
// drafts.
//
// A position belongs to a cluster of C CTAs, each with a slice of its logits, which are
// read once:
//   1. From its slice's first 16384 logits each CTA bounds what can matter: nothing
//      whose weight rounds to 0 or is below min_p, and, with top_k, nothing below a
//      value that the first k reach for sure (the least of as many lanes' maxima, or
//      groups of lanes', as are needed to have k of them).
//   2. Logits are counted by value in shared memory: 2048 magnitudes, the 16 binades
//      below the slice's largest, of either sign, in the order of the row.  Where a
//      warp's 256 logits have few above the bound, these one by one, else all of them,
//      two in a 32-bit register: what is below the bound is behind all that matters, so
//      it does no harm.  What was taken one by one is also listed, with its index.  What
//      lies between the two signs' magnitudes, near zero, is rare and goes to a list.
//   3. The CTAs add up their counts, each a part of the values, and form counts and
//      masses up to each value of a group of 32 for the first CTA, whose first warp
//      asks them where the first k end, where p of the mass ends, and where u falls.
//   4. It finds that value's logit in the slice that has it: among the listed ones, or,
//      where the list does not hold all, in the slice, from the nearer end.
// A logit above all of the 16 binades makes a CTA's counting begin again with others; an
// answer near zero is looked for in windows of 1024 values over the row.
//
// What bounds it.  Few rows: latency.  One row of 32000 takes 7.8 us: 1.4 to the first logits, 0.4 the bound, 0.9
// the counts, 1.2 the groups, 1.6 the questions (a share of the mass, three ballots, a weight and a quotient each),
// 1.1 the logit, 1.2 in three cluster barriers.  Sixteen of 151936, twelve of them live, 14.3: 1.8 between two
// kernels, 1.5 to the first logits, 0.3, 2.6 the counts (a slice is 14 % longer than what the first loads hold, so
// there is one more trip to memory), 0.8, 2.1, 1.3, 2.1 in barriers, and 1.8 that the slowest slice takes longer.
// Many unfiltered rows: instructions.  256 rows of 151936 (77.8 MB, 11.6 us of HBM) take 46.3 us and 29.2 million
// warp instructions, 0.60 an issue slot while an SM is active, 0.79 on the fullest: 1.4 million to the bound, 15.3 in
// the counts (6.3 loads with their bounds and maxima, 5.4 the bins' addresses and branches, 3.6 the atomics and
// what waits for them, 1.25 million atomics whose 32 random bins cost 3.4 cycles of the banks), 8.2 in the groups'
// weights, 0.8 in the questions, 3.5 in the search.  Ended after each of these the kernel takes 3.1, 27.6 (21.6
// without the atomics, 13.0 with loads and maxima alone), 39.7, 41.6 and 46.3 us.  256 rows leave 48 SMs with one
// row and 104 with two.  480 rows of 151936 with top-p: 90 us.
#include <cooperative_groups.h>

#include <atomic>

#include "sample.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kLoads = 4;                     // granules of a thread in flight
constexpr int kMagnitudes = 2048;             // of each sign: 16 binades
constexpr int kBins = 2 * kMagnitudes;        // in the order of the row
// Where the counts stand: a positive value's at its magnitude's number, a negative one's 32 KB
// behind, where its sign's bit points in 16 bits of address; behind each side 32 words, one
// a lane, for what has no bin; other arrays between the two.
constexpr int kSideWords = kMagnitudes + 32, kMinusWords = 8192, kWords = kMinusWords + kSideWords;
__device__ __forceinline__ int word_of(int bin) { return bin < kMagnitudes ? kMagnitudes - 1 - bin : kMinusWords + bin - kMagnitudes; }
constexpr int kGroups = kBins / 32;           // of 32 bins, a warp's
constexpr int kFewLanes = 12;                 // of a warp that have something to count: one by one
constexpr int kNear = 512;                    // places of the list of values near zero
constexpr int kWindow = 1024;                 // values of a window
constexpr int kListed = 480;                  // logits of the list of what passed
static_assert(kListed <= kThreads, "a thread each");
static_assert(kSideWords + kBins + kWindow + kNear / 2 + kListed + kListed / 2 <= kMinusWords, "they lie between the counts");
static_assert(kSideWords % 4 == 0, "in vectors");
static_assert(4 * kSideWords <= 0x8000 && 4 * kMinusWords == 0x8000, "offsets fit 16 bits, the sign's bit apart");

struct Found {
  int place;       // the value
  uint32_t n;      // logits of that value up to the one that was asked for, it included
  u64 w, mass;     // its weight; the mass before that value
  int hit;
};

// What a CTA tells the others of its cluster.
struct Told {
  float top, bound;  // its largest number; what matters is not below this
  int base;          // its least magnitude that has a bin
};

// A question about the values near zero: by count (0) or by mass; -1: there are no more.
struct Asked {
  int what;
  u64 target;
};

struct Shared {
  alignas(16) uint32_t hist[kWords];
  u64 mass[kBins];  // the cluster's masses, up to each bin of a group; first CTA
  // Between the counts of the two signs:
  // the cluster's counts, up to each bin of a group; then indices of one value; first CTA
  __device__ __forceinline__ uint32_t *sum() { return hist + kSideWords; }
  __device__ __forceinline__ uint32_t *window() { return sum() + kBins; }
  __device__ __forceinline__ uint16_t *near() { return reinterpret_cast<uint16_t *>(window() + kWindow); }
  // what passed the bound and has a bin: index and place, if no warp took all of its logits
  __device__ __forceinline__ uint32_t *index() { return window() + kWindow + kNear / 2; }
  __device__ __forceinline__ uint16_t *place() { return reinterpret_cast<uint16_t *>(index() + kListed); }

  u64 table[32];
  u64 group_mass[kGroups];
  uint32_t group_count[kGroups];
  u64 near_mass, warp_mass[32];
  uint32_t near_count, warp_count[32];  // near_count: of the cluster, first CTA
  // Written once each: of the first granules, behind the bound's barrier; of the whole slice, read behind
  // the counts' barrier, while others may still be at the bound's.
  float warp_top[32], warp_low[32], warp_bound[32], warp_largest[32];
  Told told[8];             // by rank
  uint32_t near_n, listed;  // of this CTA's lists
  int unlisted;             // some passed that are not listed
  int beyond, next, at, dust;
  uint32_t matches;
  u64 before_mass;
  uint32_t before_count;
  Found found;
  Asked asked;
};

// Inclusive sums over a warp of (count, mass).
__device__ __forceinline__ void sum_up_to(uint32_t &count, u64 &mass) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, count, o);
    const u64 b = __shfl_up_sync(0xffffffffu, mass, o);
    if (int(threadIdx.x & 31) >= o) count += a, mass += b;
  }
}

// The same over the CTA.
__device__ __forceinline__ void scan(uint32_t &count, u64 &mass, Shared &s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sum_up_to(count, mass);
  sync_cta();
  if (lane == 31) s.warp_count[warp] = count, s.warp_mass[warp] = mass;
  sync_cta();
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w)
    if (w < warp) count += s.warp_count[w], mass += s.warp_mass[w];
}

// Sum over a warp of numbers under 2^63.
__device__ __forceinline__ u64 warp_sum(u64 x) {
  const uint32_t a = uint32_t(x) & 0x7ffffffu, b = uint32_t(x >> 27) & 0x7ffffffu, c = uint32_t(x >> 54);
  return u64(__reduce_add_sync(0xffffffffu, a)) + (u64(__reduce_add_sync(0xffffffffu, b)) << 27) + (u64(__reduce_add_sync(0xffffffffu, c)) << 54);
}

// The answer among the values at places [from, end), in windows over the row, with count0 and
// mass0 before them.  Rare, and as slow as windows are many.
__device__ __noinline__ void find_in_windows(const SampleRow &row, int from, int end, int top, Scale scale, u64 least, uint32_t count0,
                                             u64 mass0, bool by_count, u64 target, Shared &s) {
  const int tid = threadIdx.x;
  constexpr int kPer = kWindow / kThreads;
  while (from < end) {
    sync_cta();
    for (int i = tid; i < kWindow; i += kThreads) s.window()[i] = 0;
    if (tid == 0) s.next = end, s.found.hit = 0;
    sync_cta();
    int next = end;
    for (int g = tid; g < row.granules; g += kThreads) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int place = place_of(half_of(q, j));
        if (place < from || place >= end) continue;
        if (place - from < kWindow) atomicAdd(&s.window()[place - from], 1u);
        else next = min(next, place);
      }
    }
    if (next < end) atomicMin(&s.next, next);
    sync_cta();
    uint32_t count = 0;
    u64 mass = 0;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const uint32_t n = s.window()[tid * kPer + i];
      const u64 w = n ? weight_of(from + tid * kPer + i, top, scale, s.table) : 0;
      if (w && w >= least) count += n, mass += n * w;
    }
    uint32_t count1 = count;
    u64 mass1 = mass;
    scan(count1, mass1, s);
    count1 += count0, mass1 += mass0;
    count = count1 - count, mass = mass1 - mass;  // before this thread's places
    const u64 lo = by_count ? u64(count) : mass, hi = by_count ? u64(count1) : mass1;
    if (lo < target && target <= hi) {
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        const int place = from + tid * kPer + i;
        uint32_t n = s.window()[tid * kPer + i];
        const u64 w = n ? weight_of(place, top, scale, s.table) : 0;
        if (!w || w < least) n = 0;
        if (n && target <= (by_count ? u64(count + n) : mass + n * w)) {
          s.found = Found{place, by_count ? uint32_t(target) - count : few_in(target - 1 - mass, w) + 1, w, mass, 1};
          break;
        }
        count += n, mass += n * w;
      }
    }
    if (tid == kThreads - 1) s.before_count = count1, s.before_mass = mass1;
    sync_cta();
    const bool hit = s.found.hit;
    count0 = s.before_count, mass0 = s.before_mass;
    from = s.next;
    sync_cta();  // everybody has read them
    if (hit) return;
  }
}

// Index of the n-th logit (from 1) with the given place among granules [g0, g1), tile after tile.
__device__ __noinline__ int locate_in_order(const SampleRow &row, int g0, int g1, int place, uint32_t n, Shared &s) {
  const int tid = threadIdx.x;
  uint32_t before = 0;
  for (; g0 < g1; g0 += kThreads) {
    const int g = g0 + tid;
    uint32_t mask = 0;
    if (g < g1) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) mask |= uint32_t(place_of(half_of(q, j)) == place) << j;
    }
    uint32_t end = __popc(mask);
    u64 none = 0;
    scan(end, none, s);
    end += before;
    if (end >= n && end - __popc(mask) < n) {
      uint32_t left = n - (end - __popc(mask)), j = 0;
      for (;; ++j)
        if ((mask >> j & 1) && --left == 0) break;
      s.at = row.first(g) + int(j);
    }
    sync_cta();
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += s.warp_count[w];
    before += all;
    if (before >= n) return s.at;
  }
  return 0;
}

// The n-th least of the first m of s.sum().
__device__ __forceinline__ int pick(uint32_t m, uint32_t n, Shared &s) {
  const int tid = threadIdx.x;
  if (tid < 4 && m + tid < uint32_t(kBins)) s.sum()[m + tid] = 0xffffffffu;
  sync_cta();
  for (uint32_t i = tid; i < m; i += kThreads) {
    const uint32_t x = s.sum()[i];
    uint32_t below = 0;
    for (uint32_t j = 0; j < m; j += 4) {
      const uint4 y = *reinterpret_cast<const uint4 *>(s.sum() + j);
      below += (y.x < x) + (y.y < x) + (y.z < x) + (y.w < x);
    }
    if (below + 1 == n) s.at = int(x);
  }
  sync_cta();
  return s.at;
}

// The same for a value that `all` logits have, few: they are listed, tile after tile until there are
// n, and counted against one another.  From the end, where it is nearer: a quarter of the slice
// on average.
__device__ int locate(const SampleRow &row, int g0, int g1, int place, uint32_t n, uint32_t all, Shared &s) {
  if (all > uint32_t(kBins)) return locate_in_order(row, g0, g1, place, n, s);
  const int tid = threadIdx.x;
  constexpr int kTile = kThreads * kLoads;
  const bool back = n > all - n;
  const uint32_t want = back ? all - n + 1 : n;
  const int tiles = (g1 - g0 + kTile - 1) / kTile;
  // equal as numbers: -0 as 0, NaN never
  const __nv_bfloat162 v = __float2bfloat162_rn(value_at(place));
  auto same = [&](uint32_t w) { return __heq2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&w), v); };
  auto start_of = [&](int tile) { return g0 + (back ? tiles - 1 - tile : tile) * kTile + tid; };
  uint4 next[kLoads];
  auto load = [&](int g) {
#pragma unroll
    for (int r = 0; r < kLoads; ++r)
      next[r] = g + r * kThreads < g1 ? row.load(g + r * kThreads) : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
  };
  load(start_of(0));
  uint32_t found = 0;
  for (int tile = 0; tile < tiles && found < want; ++tile) {  // the same for every thread
    const int g = start_of(tile);
    uint4 q[kLoads];
#pragma unroll
    for (int r = 0; r < kLoads; ++r) q[r] = next[r];
    if (tile + 1 < tiles) load(start_of(tile + 1));
#pragma unroll
    for (int r = 0; r < kLoads; ++r) {
      const uint32_t m0 = same(q[r].x), m1 = same(q[r].y), m2 = same(q[r].z), m3 = same(q[r].w);
      if (m0 | m1 | m2 | m3) {
        uint32_t bits = (m0 & 0x10001u) | (m1 & 0x10001u) << 2 | (m2 & 0x10001u) << 4 | (m3 & 0x10001u) << 6;
        bits = (bits | bits >> 15) & 0xffu;  // logit j at bit j
        uint32_t k = atomicAdd(&s.matches, uint32_t(__popc(bits)));
        const int at = row.first(g + r * kThreads);
        for (; bits && k < uint32_t(kBins); ++k, bits &= bits - 1) s.sum()[k] = uint32_t(at + __ffs(bits) - 1);
      }
    }
    sync_cta();
    found = s.matches;
    sync_cta();
  }
  const uint32_t m = min(found, uint32_t(kBins));
  return pick(m, back ? m - want + 1 : want, s);
}

__device__ __forceinline__ __nv_bfloat162 b2(const uint32_t &w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ __nv_bfloat162 max2_of(const uint4 &q) {
  return __hmax2(__hmax2(b2(q.x), b2(q.y)), __hmax2(b2(q.z), b2(q.w)));
}
__device__ __forceinline__ float max_of(const uint4 &q) {
  const __nv_bfloat162 m = max2_of(q);
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float min_of(const uint4 &q) {
  const __nv_bfloat162 m = __hmin2(__hmin2(b2(q.x), b2(q.y)), __hmin2(b2(q.z), b2(q.w)));
  return fminf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

constexpr uint32_t kNoNumbers = 0x7fff7fffu;

// One more in the bins of two logits, 16 bits each, where their magnitudes have one;
// returns their magnitudes' numbers, from kMagnitudes on where they have none.
// less_base: -base twice; most: the lane's word for what has no bin, twice.  The offsets fit 16
// bits; the counts' address does not (in a cluster it holds the CTA's rank) and is added in 32.
__device__ __forceinline__ uint32_t count_two(uint32_t w, uint32_t less_base, uint32_t most, uint32_t hist) {
  const uint32_t off = __viaddmin_u16x2(w & 0x7fff7fffu, less_base, most);
  const uint32_t at = off << 2 | (w & 0x80008000u);
  asm volatile("red.shared.add.u32 [%0], 1;\n red.shared.add.u32 [%1], 1;" ::"r"(hist + (at & 0xffffu)), "r"(hist + (at >> 16)) : "memory");
  return off;
}

// Which of a granule's logits reach the bound, logit j as bit j.
__device__ __forceinline__ uint32_t reaching(const uint4 &q, __nv_bfloat162 bound) {
  const uint32_t m = (__hge2_mask(b2(q.x), bound) & 0x10001u) | (__hge2_mask(b2(q.y), bound) & 0x10001u) << 2 |
                     (__hge2_mask(b2(q.z), bound) & 0x10001u) << 4 | (__hge2_mask(b2(q.w), bound) & 0x10001u) << 6;
  return (m | m >> 15) & 0xffu;
}

template <int C>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) unsigned char memory[];
  Shared &s = *reinterpret_cast<Shared *>(memory);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C > 1 ? int(cluster.block_rank()) : 0;
  const int bt = blockIdx.x / C, b = bt / p.T;
  auto together = [&] {
    __syncwarp();
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  const SampleRow row(p.logits + size_t(bt) * p.stride, p.V);
  const int each = (row.granules + C - 1) / C;
  const int g0 = min(row.granules, rank * each), g1 = min(row.granules, g0 + each);
  auto load = [&](int g) { return g < g1 ? row.load(g) : make_uint4(kNoNumbers, kNoNumbers, kNoNumbers, kNoNumbers); };
  uint4 ahead[kLoads];  // this thread's next granules, kThreads apart
  auto start = [&] {
#pragma unroll
    for (int r = 0; r < kLoads; ++r) ahead[r] = load(g0 + tid + r * kThreads);
  };
  start();
  float temperature = p.temperature ? p.temperature[b] : 1.f;
  float min_p = p.min_p ? p.min_p[b] : 0.f, top_p = p.top_p ? p.top_p[b] : 1.f;
  int top_k = p.top_k ? p.top_k[b] : 0;
  const float u = p.u[bt];
  const bool active = !p.active || p.active[b];  // the cluster agrees
  int token = -1;
  float logp = 0.f;
  if (active) {
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA runs
    auto clear = [&] {  // as many rounds for every thread
#pragma unroll
      for (int i = 4 * tid; i - 4 * tid < 2 * kSideWords; i += 4 * kThreads)
        if (i < 2 * kSideWords) *reinterpret_cast<uint4 *>(s.hist + (i < kSideWords ? i : i - kSideWords + kMinusWords)) = make_uint4(0, 0, 0, 0);
    };
    clear();
    if (tid < 32) s.table[tid] = kExp2Table[tid];
    if (tid == 0) s.near_n = 0, s.listed = 0, s.unlisted = 0, s.near_count = 0, s.near_mass = 0, s.beyond = 0, s.dust = 0;
    if (!(temperature > 0.f)) temperature = 0.f, min_p = 0.f, top_p = 1.f, top_k = 1;
    min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
    if (top_k <= 0 || top_k > p.V) top_k = p.V;

    // ---- what can matter ----------------------------------------------------------------
    float top = -INFINITY, low = INFINITY, bound = -INFINITY;
#pragma unroll
    for (int r = 0; r < kLoads; ++r) top = fmaxf(top, max_of(ahead[r])), low = fminf(low, min_of(ahead[r]));
    // so many lanes' maxima that the CTA has top_k groups or more; the least of the groups'
    const int lanes = top_k <= kWarps ? 32 : top_k <= kThreads ? 1 << (31 - __clz(kThreads / top_k)) : 0;
    bound = lanes == 1 ? top : bound;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      bound = lanes == 2 * o ? top : bound;
    }
    bound = warp_min(bound), low = warp_min(low);
    if (lane == 0) s.warp_top[warp] = top, s.warp_low[warp] = low, s.warp_bound[warp] = bound;
    sync_cta();
    top = s.warp_top[0], low = s.warp_low[0], bound = s.warp_bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s.warp_top[w]), low = fminf(low, s.warp_low[w]), bound = fminf(bound, s.warp_bound[w]);
    // Weights under 2^-44 round to 0 and are dust (below), those under 2^-53 are nothing: 54 ln 2
    // temperatures below the largest.  Rounding moves these bounds by far less than a step of bf16,
    // and never above the largest.
    if (top > -INFINITY && top < INFINITY) {
      bound = fmaxf(bound, top - 37.4f * temperature);
      if (min_p > 0.f) bound = fmaxf(bound, top + temperature * __logf(min_p) - (1e-3f * temperature + 1e-6f * fabsf(top)));
    } else if (top == INFINITY) {
      bound = INFINITY;
    }
    // the least number of bf16 that reaches it, and a finite one
    bound = __bfloat162float(__float2bfloat16_ru(fmaxf(bound, -3.3895314e38f)));
    // the largest magnitude that may come; where more is read than was looked at, of twice that
    uint32_t magnitude = (__float_as_uint(fmaxf(fabsf(top), fabsf(fmaxf(low, bound)))) >> 16);
    if (!(top > -INFINITY)) magnitude = 0;
    int binade = int(magnitude >> 7) + (each > kThreads * kLoads);
    // -infinity has no bin, so no weight either: only where +infinity is there, beside which nothing
    // has any, do the bins go up to the magnitude of infinity
    if (top < INFINITY) binade = min(binade, 254);

    // ---- counts by value ------------------------------------------------------------------
    int base;
    const __nv_bfloat162 bound2 = __float2bfloat162_rn(bound);
    const uint32_t hist = smem_u32(s.hist), most = (kMagnitudes + lane) * 0x10001u;
    for (;;) {
      base = max(0, min((binade + 1) << 7, 0x7f81) - kMagnitudes);  // +infinity is the last that has one
      const uint32_t less_base = (-uint32_t(base) & 0xffffu) * 0x10001u;
      __nv_bfloat162 largest2 = __float2bfloat162_rn(-INFINITY);
      auto count = [&](const uint4 &q, int g) {
        const __nv_bfloat162 x = max2_of(q);
        largest2 = __hmax2(largest2, x);
        // branches are the warp's, so that it stays together
        const uint32_t who = __ballot_sync(0xffffffffu, __hge2_mask(x, bound2) != 0);
        if (!who) return;
        uint32_t odd;  // logits to look at one by one, as bits
        bool counted = false;
        if (__popc(who) <= kFewLanes) {
          odd = reaching(q, bound2);
        } else {  // also what lies below the bound: it is behind all that matters
          const uint32_t off = count_two(q.x, less_base, most, hist) | count_two(q.y, less_base, most, hist) |
                               count_two(q.z, less_base, most, hist) | count_two(q.w, less_base, most, hist);
          const bool some = off & kMagnitudes * 0x10001u;
          if (lane == 0) s.unlisted = 1;
          if (!__any_sync(0xffffffffu, some)) return;
          odd = some ? reaching(q, bound2) : 0;
          counted = true;
        }
        for (; odd; odd &= odd - 1) {
          const int j = __ffs(odd) - 1;
          const uint32_t bits = half_of(q, j), a = bits & 0x7fffu, off = a - uint32_t(base);
          if (off < uint32_t(kMagnitudes)) {
            if (!counted) {
              atomicAdd(&s.hist[bits > 0x8000u ? kMinusWords + off : off], 1u);
              const uint32_t i = atomicAdd(&s.listed, 1u);
              if (i < uint32_t(kListed)) s.index()[i] = uint32_t(row.first(g) + j), s.place()[i] = uint16_t(place_of(bits));
            }
          } else if (a < uint32_t(base)) {
            const uint32_t i = atomicAdd(&s.near_n, 1u);
            if (i < uint32_t(kNear)) s.near()[i] = uint16_t(place_of(bits));
          } else {
            atomicMax(&s.beyond, int(a));
          }
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int g = g0 + tid; g - tid < g1; g += 2 * kThreads) {
        const uint4 q0 = ahead[0], q1 = ahead[1];
        ahead[0] = ahead[2], ahead[1] = ahead[3];
        ahead[2] = load(g + 4 * kThreads), ahead[3] = load(g + 5 * kThreads);
        count(q0, g);
        count(q1, g + kThreads);
      }
      const float largest = warp_max(fmaxf(__low2float(largest2), __high2float(largest2)));
      if (lane == 0) s.warp_largest[warp] = largest;
      sync_cta();
      const int beyond = s.beyond;
      __syncwarp();
      if (!__syncthreads_or(beyond)) break;
      // once more, with the bins that hold the largest of all
      binade = beyond >> 7;
      clear();
      if (tid == 0) s.near_n = 0, s.listed = 0, s.unlisted = 0, s.beyond = 0;
      start();
      sync_cta();
    }
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all of them run
    if (tid < C) {
      Told t{s.warp_largest[0], bound, base};
#pragma unroll
      for (int w = 1; w < kWarps; ++w) t.top = fmaxf(t.top, s.warp_largest[w]);
      (C > 1 ? cluster.map_shared_rank(s.told, tid) : s.told)[rank] = t;
    }
    if (tid == 32 && base == 0) s.hist[0] += s.hist[kMinusWords], s.hist[kMinusWords] = 0;  // -0 is 0
    together();
    const int own_base = base;
    const float own_bound = bound;
    top = s.told[0].top, bound = s.told[0].bound, base = s.told[0].base;
#pragma unroll
    for (int i = 1; i < C; ++i) top = fmaxf(top, s.told[i].top), bound = fmaxf(bound, s.told[i].bound), base = max(base, s.told[i].base);

    if (!(top > -INFINITY)) {  // nothing above -infinity: what greedy acceptance takes, and no probability
      if (rank == 0) token = locate_in_order(row, 0, row.granules, kPlaceEnd, 1, s);
      logp = -INFINITY;
    } else {
      const int best = place_of(__float_as_uint(top) >> 16);
      const Scale scale = temperature > 0.f ? scale_of(temperature) : Scale{0.f, 0.f, 1.f};
      const u64 least = __float2ull_ru(min_p * float(kWeightOne));  // exact before it is rounded up
      auto place_at = [&](int bin) { return bin < kMagnitudes ? kPlaceZero - base - (kMagnitudes - 1 - bin) : 0x8000 + base + bin - kMagnitudes; };
      Shared &s0 = C > 1 ? *cluster.map_shared_rank(&s, 0) : s;
      // a bin of the cluster's in a CTA with another base: nearer the middle, or none
      auto count_of = [&](int i, int bin) -> uint32_t {
        if (C == 1) return s.hist[word_of(bin)];
        const int shift = base - s.told[i].base, at = bin < kMagnitudes ? bin - shift : bin + shift;
        return at >= 0 && at < kBins ? cluster.map_shared_rank(s.hist, i)[word_of(at)] : 0;
      };

      // Dust: weights too small for the units of the masses.  It is told, because where the rest meets
      // a border exactly (two equal logits share the mass, top_p is 0.5) any more than nothing decides.
      // Only what min_p leaves is any: log(min_p) is as near here as 2^-22 of itself.  Halves of the logits, whose
      // differences are finite; 36.8 temperatures are 2^-53.1.
      const float half_top = 0.5f * top, dust_from = fmaxf(-18.4f * temperature, min_p > 0.f ? 0.5f * temperature * logf(min_p) : -INFINITY);
      auto is_dust = [&](int place, u64 w) { return !w && 0.5f * value_at(place) - half_top >= dust_from; };

      // ---- the cluster's counts, and its groups' counts and masses ---------------------------
      {
        constexpr int kMine = kGroups / (C * kWarps);  // groups of a warp
#pragma unroll 2
        for (int k = 0; k < kMine; ++k) {
          const int group = (rank + k * C) * kWarps + warp, bin = group * 32 + lane;
          uint32_t count = 0;
          u64 mass = 0;
          if (value_at(place_at(group * 32)) >= bound) {  // its largest; where it is not there, the rest does not matter
#pragma unroll
            for (int i = 0; i < C; ++i) count += count_of(i, bin);
            if (__any_sync(0xffffffffu, count != 0)) {
              const u64 w = weight_of(place_at(bin), best, scale, s.table);
              if (count && is_dust(place_at(bin), w)) s0.dust = 1;
              if (!w || w < least) count = 0;
              mass = count * w;
              sum_up_to(count, mass);
              s0.sum()[bin] = count, s0.mass[bin] = mass;
            }
          }
          if (lane == 31) s0.group_count[group] = count, s0.group_mass[group] = mass;
        }
      }
      // values near zero: from the list, or, where it was too short, from the slice once more,
      // and from the bins of this CTA that the cluster has none for
      const uint32_t near_n = s.near_n;
      if (near_n || base > own_base) {
        uint32_t count = 0;
        u64 mass = 0;
        auto add = [&](int place, uint32_t n) {
          const u64 w = weight_of(place, best, scale, s.table);
          if (is_dust(place, w)) s0.dust = 1;
          if (w && w >= least) count += n, mass += n * w;
        };
        if (near_n <= uint32_t(kNear)) {
          for (uint32_t i = tid; i < near_n; i += kThreads) add(s.near()[i], 1);
        } else {
          for (int g = g0 + tid; g < g1; g += kThreads) {
            const uint4 q = row.load(g);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              const uint32_t bits = half_of(q, j);
              if (int(bits & 0x7fffu) < own_base && bf2f(uint16_t(bits)) >= own_bound) add(place_of(bits), 1);
            }
          }
        }
        for (int i = tid; i < 2 * min(base - own_base, kMagnitudes); i += kThreads) {
          const int off = i >> 1;
          const uint32_t n = s.hist[i & 1 ? kMinusWords + off : off];
          if (n) add(i & 1 ? 0x8000 + own_base + off : kPlaceZero - own_base - off, n);
        }
        count = __reduce_add_sync(0xffffffffu, count), mass = warp_sum(mass);
        if (lane == 0 && count) atomicAdd(&s0.near_count, count), atomicAdd(&s0.near_mass, mass);
      }
      together();

      if (rank == 0) {
        // ---- three questions, asked by the first warp -------------------------------------------
        if (tid == 32) s.matches = 0, s.at = 0;
        if (warp == 0) {
          // group sums up to each group, the values near zero before the 65th; a lane has four
          constexpr int kMine = kGroups / 32;
          uint32_t count[kMine], counts = 0;
          u64 mass[kMine], masses = 0;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            count[i] = counts += s.group_count[lane * kMine + i];
            mass[i] = masses += s.group_mass[lane * kMine + i];
          }
          const uint32_t own_count = counts;
          const u64 own_mass = masses;
          sum_up_to(counts, masses);
          const uint32_t near_at = __shfl_sync(0xffffffffu, counts, 15), near_to = near_at + s.near_count;
          const u64 near_mass_at = __shfl_sync(0xffffffffu, masses, 15), near_mass_to = near_mass_at + s.near_mass;
          if (lane >= 16) counts += s.near_count, masses += s.near_mass;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            s.group_count[lane * kMine + i] = counts - own_count + count[i];
            s.group_mass[lane * kMine + i] = masses - own_mass + mass[i];
          }
          __syncwarp();
          const uint32_t total_count = __shfl_sync(0xffffffffu, counts, 31);
          u64 rest = __shfl_sync(0xffffffffu, masses, 31);
          Found f{best, 1, kWeightOne, 0, 0};
          // each question: the first value up to which there are `target` logits, or as much mass
#pragma unroll 1
          for (int step = 0; step < 3; ++step) {
            u64 target;
            if (step == 0) {
              if (uint32_t(top_k) >= total_count) continue;  // all that has weight
              target = u64(top_k);
            } else if (step == 1) {
              if (!(top_p < 1.f)) continue;
              const bool dust = s.dust && uint32_t(top_k) > total_count;
              target = dust ? share_of(fmaxf(top_p, 0.f), rest, false) + 1 : max(u64(1), share_of(fmaxf(top_p, 0.f), rest, true));
            } else {  // to pass a share is to reach one more
              target = u > 0.f ? share_of(fminf(u, 0x1.fffffep-1f), rest, false) + 1 : 1;
            }
            const bool by_count = step == 0;
            const uint32_t lead = __ffs(__ballot_sync(0xffffffffu, (by_count ? u64(counts) : masses) >= target)) - 1;
            if (lead == 16 && target <= (by_count ? u64(near_to) : near_mass_to)) {  // near zero: the whole CTA looks
              if (lane == 0) s.asked = Asked{step, target}, s.found = f, s.before_count = near_at, s.before_mass = near_mass_at;
              sync_cta();
              find_in_windows(row, kPlaceZero - base + 1, 0x8000 + base, best, scale, least, near_at, near_mass_at, step == 0, target, s);
              f = s.found;
            } else if (lead < 32) {
              const int mine = lead * kMine + (lane & (kMine - 1));
              const uint32_t c = s.group_count[mine];
              const u64 m = s.group_mass[mine];
              const int group = lead * kMine + __ffs(__ballot_sync(0xffffffffu, (by_count ? u64(c) : m) >= target)) - 1;
              const int bin = group * 32 + lane;
              // before the group: what is up to it less what it has
              const uint32_t c0 = s.group_count[group] - s.sum()[group * 32 + 31], c1 = c0 + s.sum()[bin];
              const u64 m0 = s.group_mass[group] - s.mass[group * 32 + 31], m1 = m0 + s.mass[bin];
              const int at = __ffs(__ballot_sync(0xffffffffu, (by_count ? u64(c1) : m1) >= target)) - 1;
              const uint32_t to = __shfl_sync(0xffffffffu, c1, at), up = __shfl_sync(0xffffffffu, c1, at - 1), n = to - (at ? up : c0);
              const u64 mass_to = __shfl_sync(0xffffffffu, m1, at), mass_up = __shfl_sync(0xffffffffu, m1, at - 1);
              f.place = place_at(group * 32 + at);
              f.mass = at ? mass_up : m0;
              f.w = mass_to - f.mass, f.n = 1;
              if (n > 1) {
                f.w = weight_of(f.place, best, scale, s.table);
                f.n = by_count ? uint32_t(target) - (to - n) : few_in(target - 1 - f.mass, f.w) + 1;
              }
            }
            if (step < 2) rest = f.mass + f.n * f.w;
          }
          // A weight under 2^24 units is off by more than 2^-25 of itself: its logarithm from the logits.
          if (f.w < (1u << 24)) {
            const float x = value_at(f.place), d = x - top;
            logp = (isinf(d) ? __fdiv_rn(.5f * x - .5f * top, .5f * temperature) : __fdiv_rn(d, temperature)) -
                   logf(float(rest) / float(kWeightOne));
          } else {
            logp = -log1pf(float(rest - f.w) / float(f.w));
          }
          if (lane == 0) s.asked.what = -1, s.found = f;
          sync_cta();
        } else {
          for (;;) {
            sync_cta();
            const Asked a = s.asked;
            if (a.what < 0) break;
            find_in_windows(row, kPlaceZero - base + 1, 0x8000 + base, best, scale, least, s.before_count, s.before_mass, a.what == 0, a.target, s);
          }
        }

        // ---- the logit ---------------------------------------------------------------------------
        const Found f = s.found;
        const int a = f.place <= kPlaceZero ? kPlaceZero - f.place : f.place - 0x8000;
        if (a < base) {
          token = locate_in_order(row, 0, row.granules, f.place, f.n, s);
        } else {
          const int bin = f.place <= kPlaceZero ? kMagnitudes - 1 - (a - base) : kMagnitudes + a - base;
          uint32_t n = f.n, has[C];
#pragma unroll
          for (int i = 0; i < C; ++i) has[i] = count_of(i, bin);
          int q = 0;
          uint32_t all = has[0];
#pragma unroll
          for (int i = 1; i < C; ++i)
            if (q == i - 1 && n > all) n -= all, q = i, all = has[i];
          Shared &sq = C > 1 ? *cluster.map_shared_rank(&s, q) : s;
          const uint32_t listed = sq.listed;
          if (!sq.unlisted && listed <= uint32_t(kListed)) {
            if (tid < int(listed) && sq.place()[tid] == f.place) s.sum()[atomicAdd(&s.matches, 1u)] = sq.index()[tid];
            sync_cta();
            token = pick(s.matches, n, s);
          } else {
            const int from = min(row.granules, q * each);
            token = locate(row, from, min(row.granules, from + each), f.place, n, all, s);
          }
        }
      }
    }
    __syncwarp();
    if (C > 1) cluster.sync();  // the first CTA has read what it needs of the others
  }
  if (rank != 0) return;
  if (tid == 0) {
    if (p.token) p.token[bt] = token;
    if (p.logp) p.logp[bt] = logp;
  }
  if (!p.draft) return;

  // ---- acceptance: the row's last position decides ------------------------------------------
  if (tid == 0) {
    p.ws_token[bt] = token;
    __threadfence();  // the token is visible before it is counted
    if (atomicAdd(&p.ws_count[b], 1u) + 1u == uint32_t(p.T)) {
      __threadfence();
      int k = 0;
      if (active) {
        k = 1;
        while (k < p.T && p.draft[size_t(b) * p.T + k] == __ldcg(p.ws_token + size_t(b) * p.T + k - 1)) ++k;
      }
      p.keep[b] = k;
      p.next[b] = k ? __ldcg(p.ws_token + size_t(b) * p.T + k - 1) : -1;
      // ready for the next call, also one of other sizes, whose counts lie elsewhere
      p.ws_count[b] = 0;
      for (int t = 0; t < p.T; ++t) p.ws_token[size_t(b) * p.T + t] = 0;
    }
  }
}

template <int C>
cudaError_t launch(const SampleParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.gridDim = dim3(unsigned(p.B) * unsigned(p.T) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<C>, p);
}

}  // namespace

size_t accept_sampled_workspace_bytes(int B, int T) {
  return align256(size_t(B) * T * sizeof(int32_t)) + align256(size_t(B) * sizeof(uint32_t));
}

// CTAs of a position: as many as the GPU holds at once (two an SM) for all of them, where
// each has 4096 logits at least.  Both sides, us of GPU time with 1, 2, 4, 8 CTAs:
//   1 row of 32000, top-k 40, top-p, min-p        8.0   8.3   7.8   7.9
//   7 of 100003, 0.9 forbidden, top-p            36.0  24.8  17.6  13.9
//   16 of 151936, top-k 20, top-p                30.4  21.6  14.8  14.2
//   64 of 151936, mixed                          34.3  25.2  21.4  29.1
//   256 of 151936, unfiltered                    46.1  57.9  79.2   123
//   480 of 151936, top-p                         89.8   108   148   242
cudaError_t launch_sample(const SampleParams &p, cudaStream_t s) {
  static std::atomic<int> cached[64];  // SMs by device, 0 until looked up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (!sms) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // more than the 48 KB of shared memory that need no asking
    const void *kernels[] = {reinterpret_cast<const void *>(sample_kernel<1>), reinterpret_cast<const void *>(sample_kernel<2>),
                             reinterpret_cast<const void *>(sample_kernel<4>), reinterpret_cast<const void *>(sample_kernel<8>)};
    for (const void *k : kernels)
      if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Shared)))) != cudaSuccess) return e;
    if (dev < 64) cached[dev].store(sms, std::memory_order_relaxed);
  }
  const long long rows = (long long)p.B * p.T;
  int C = 8;
  while (C > 1 && (rows * C > 2 * sms || p.V < 4096 * C)) C /= 2;
  switch (C) {
    case 8: return launch<8>(p, s);
    case 4: return launch<4>(p, s);
    case 2: return launch<2>(p, s);
    default: return launch<1>(p, s);
  }
}

}  // namespace gdn

// sample.cu -- sampled decoding: a token of every position by temperature, min-p,
// top-k and top-p from a given random number, and the accepted prefix of a verify's
// drafts.
//
// A position belongs to a cluster of C CTAs, each with a slice of its logits, which are
// read once:
//   1. From its slice's first 8192 logits each CTA bounds what can matter: nothing
//      whose weight rounds to 0 or is below min_p, and, with top_k, nothing below a
//      value that the first k reach for sure (each warp's ceil(k / warps)-th largest of
//      its granules' maxima, the least of them).
//   2. The logits that pass are counted by value in shared memory: 2048 magnitudes, the
//      16 binades below the largest, of either sign, in the order of the row.  What lies
//      between the two signs' magnitudes, near zero, is rare and goes to a list.
//   3. The CTAs add up their counts, each a part of the values, and form counts and
//      masses of groups of 16 values for the first CTA, which asks them where the first
//      k end, where p of the mass ends, and where u falls.
//   4. It finds that value's logit in the slice that has it.
// A logit above all of the 16 binades makes the counting begin again with others; an
// answer near zero is looked for in windows of 2048 values over the row.
#include <cooperative_groups.h>

#include "sample.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 4;                     // granules of a thread and tile
constexpr int kTile = kThreads * kLoads;      // granules of a tile
constexpr int kMagnitudes = 2048;             // of each sign: 16 binades
constexpr int kBins = 2 * kMagnitudes;        // in the order of the row
constexpr int kGroups = kBins / 32;           // of 32 bins, a warp's
constexpr int kFewGranules = 512;             // of a slice: counted without a bound of top_k
constexpr int kNear = 512;                    // places of the list of values near zero
constexpr int kWindow = 1024;                 // values of a window, and logits of one value found

struct Found {
  int place;       // the value
  uint32_t n;      // logits of that value up to the one that was asked for, it included
  u64 w, mass;     // its weight; the mass before that value
  int hit;
};

// What a CTA tells the others of its cluster.
struct Told {
  float top, low, bound;  // largest and least number, bound of what matters
  int beyond;             // largest magnitude that had no bin, 0 if none
};

// A question about the values near zero; what = -1: there are no more.
struct Asked {
  int what;
  u64 target;
};

struct Shared {
  alignas(16) uint32_t hist[kBins];
  uint32_t sum[kBins];      // the cluster's (where it has more than one CTA); first CTA
  uint32_t window[kWindow];
  uint16_t near[kNear];
  u64 table[32];
  u64 group_mass[kGroups];
  uint32_t group_count[kGroups];
  u64 near_mass, warp_mass[kWarps];
  uint32_t near_count, warp_count[kWarps];  // near_count: of the cluster, first CTA
  float warp_top[kWarps], warp_low[kWarps], warp_bound[kWarps];
  Told told[2][8];          // by rank: before and after the counts
  uint32_t near_n;          // of this CTA's list
  int beyond, next, at;
  uint32_t matches;
  u64 before_mass;
  uint32_t before_count;
  Found found;
  Asked asked;
};

enum Question { kCount, kMassReaches, kMassPasses };

__device__ __forceinline__ bool answers(Question what, u64 target, u64 count, u64 count1, u64 mass, u64 mass1) {
  return what == kCount ? count < target && target <= count1
                        : what == kMassReaches ? mass < target && target <= mass1 : mass <= target && target < mass1;
}
__device__ __forceinline__ uint32_t number_of(Question what, u64 target, u64 count, u64 mass, u64 w) {
  return what == kCount ? uint32_t(target - count) : few_in(target - mass - (what == kMassReaches), w) + 1;
}

// Inclusive sums over the CTA of (count, mass).
__device__ __forceinline__ void scan(uint32_t &count, u64 &mass, Shared &s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, count, o);
    const u64 b = __shfl_up_sync(0xffffffffu, mass, o);
    if (lane >= o) count += a, mass += b;
  }
  __syncthreads();
  if (lane == 31) s.warp_count[warp] = count, s.warp_mass[warp] = mass;
  __syncthreads();
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
                                             u64 mass0, Question what, u64 target, Shared &s) {
  const int tid = threadIdx.x;
  constexpr int kPer = kWindow / kThreads;
  while (from < end) {
    __syncthreads();
    for (int i = tid; i < kWindow; i += kThreads) s.window[i] = 0;
    if (tid == 0) s.next = end, s.found.hit = 0;
    __syncthreads();
    int next = end;
    for (int g = tid; g < row.granules; g += kThreads) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int place = place_of(half_of(q, j));
        if (place < from || place >= end) continue;
        if (place - from < kWindow) atomicAdd(&s.window[place - from], 1u);
        else next = min(next, place);
      }
    }
    if (next < end) atomicMin(&s.next, next);
    __syncthreads();
    uint32_t count = 0;
    u64 mass = 0;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const uint32_t n = s.window[tid * kPer + i];
      const u64 w = n ? weight_of(from + tid * kPer + i, top, scale, s.table) : 0;
      if (w >= least) count += n, mass += n * w;
    }
    uint32_t count1 = count;
    u64 mass1 = mass;
    scan(count1, mass1, s);
    count1 += count0, mass1 += mass0;
    count = count1 - count, mass = mass1 - mass;  // before this thread's places
    if (answers(what, target, count, count1, mass, mass1)) {
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        const int place = from + tid * kPer + i;
        uint32_t n = s.window[tid * kPer + i];
        const u64 w = n ? weight_of(place, top, scale, s.table) : 0;
        if (w < least) n = 0;
        if (n && answers(what, target, count, count + n, mass, mass + n * w)) {
          s.found = Found{place, number_of(what, target, count, mass, w), w, mass, 1};
          break;
        }
        count += n, mass += n * w;
      }
    }
    if (tid == kThreads - 1) s.before_count = count1, s.before_mass = mass1;
    __syncthreads();
    const bool hit = s.found.hit;
    count0 = s.before_count, mass0 = s.before_mass;
    from = s.next;
    __syncthreads();  // everybody has read them
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
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += s.warp_count[w];
    before += all;
    if (before >= n) return s.at;
  }
  return 0;
}

// The same for a value that few logits have: they are listed, and counted against one another.
__device__ int locate(const SampleRow &row, int g0, int g1, int place, uint32_t n, uint32_t all, Shared &s) {
  if (all > uint32_t(kWindow)) return locate_in_order(row, g0, g1, place, n, s);
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) s.matches = 0, s.at = 0;
  __syncthreads();
  // equal as numbers: -0 as 0, NaN never
  const __nv_bfloat162 v = __float2bfloat162_rn(value_at(place));
  auto same = [&](uint32_t w) { return __heq2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&w), v); };
  for (int g = g0 + tid; g - tid < g1; g += kTile) {  // the warp's lanes together
    uint4 q[kLoads];
#pragma unroll
    for (int r = 0; r < kLoads; ++r)
      q[r] = g + r * kThreads < g1 ? row.load(g + r * kThreads) : make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
#pragma unroll
    for (int r = 0; r < kLoads; ++r) {
      const uint32_t m0 = same(q[r].x), m1 = same(q[r].y), m2 = same(q[r].z), m3 = same(q[r].w);
      if (m0 | m1 | m2 | m3) {
        uint32_t bits = (m0 & 0x10001u) | (m1 & 0x10001u) << 2 | (m2 & 0x10001u) << 4 | (m3 & 0x10001u) << 6;
        bits = (bits | bits >> 15) & 0xffu;  // logit j at bit j
        const uint32_t i = atomicAdd(&s.matches, uint32_t(__popc(bits)));
        const int at = row.first(g + r * kThreads);
        for (uint32_t k = i; bits && k < uint32_t(kWindow); ++k, bits &= bits - 1) s.window[k] = uint32_t(at + __ffs(bits) - 1);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  const uint32_t m = min(s.matches, uint32_t(kWindow));
  if (tid < 4 && m + tid < uint32_t(kWindow)) s.window[m + tid] = 0xffffffffu;
  __syncthreads();
  for (uint32_t i = tid; i < m; i += kThreads) {
    const uint32_t x = s.window[i];
    uint32_t below = 0;
    for (uint32_t j = 0; j < m; j += 4) {
      const uint4 y = *reinterpret_cast<const uint4 *>(s.window + j);
      below += (y.x < x) + (y.y < x) + (y.z < x) + (y.w < x);
    }
    if (below + 1 == n) s.at = int(x);
  }
  __syncthreads();
  return s.at;
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ __nv_bfloat162 b2(const uint32_t &w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }
__device__ __forceinline__ float max_of(const uint4 &q) {
  const __nv_bfloat162 m = __hmax2(__hmax2(b2(q.x), b2(q.y)), __hmax2(b2(q.z), b2(q.w)));
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

// One more in the bin of f, if f >= bound and its magnitude has one.  Returns, where f >=
// bound, its magnitude beyond the least that has one, in the upper half, else 0.  `bins`
// is the address of the first bin of a negative value; positive ones lie before it, in
// the other direction.
__device__ __forceinline__ uint32_t count_value(float f, float bound, uint32_t least_magnitude, uint32_t bins) {
  const int x = __float_as_int(f + 0.f);  // -0 as 0
  const uint32_t off = (uint32_t(x) & 0x7fffffffu) - least_magnitude;
  const uint32_t at = bins + ((off >> 14) ^ (~uint32_t(x >> 31) & ~3u));
  uint32_t far;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ge.f32 p, %1, %2;\n setp.lt.and.u32 q, %3, %4, p;\n @q red.shared.add.u32 [%5], 1;\n"
      " selp.u32 %0, %3, 0, p;\n}"
      : "=r"(far)
      : "f"(f), "f"(bound), "r"(off), "r"(uint32_t(kMagnitudes) << 16), "r"(at)
      : "memory");
  return far;
}

template <int C>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleParams p) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C > 1 ? int(cluster.block_rank()) : 0;
  const int bt = blockIdx.x / C, b = bt / p.T;
  auto together = [&] {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  const bool active = !p.active || p.active[b];  // the cluster agrees
  int token = -1;
  float logp = 0.f;
  if (active) {
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA runs
    const SampleRow row(p.logits + size_t(bt) * p.stride, p.V);
    const int each = (row.granules + C - 1) / C;
    const int g0 = min(row.granules, rank * each), g1 = min(row.granules, g0 + each);
    auto load = [&](uint4(&q)[kLoads], int g) {
#pragma unroll
      for (int r = 0; r < kLoads; ++r)
        q[r] = g + r * kThreads < g1 ? row.load(g + r * kThreads) : make_uint4(kNoNumbers, kNoNumbers, kNoNumbers, kNoNumbers);
    };
    uint4 first[kLoads];
    load(first, g0 + tid);
    float temperature = p.temperature ? p.temperature[b] : 1.f;
    float min_p = p.min_p ? p.min_p[b] : 0.f, top_p = p.top_p ? p.top_p[b] : 1.f;
    int top_k = p.top_k ? p.top_k[b] : 0;
    for (int i = 4 * tid; i < kBins; i += 4 * kThreads) *reinterpret_cast<uint4 *>(s.hist + i) = make_uint4(0, 0, 0, 0);
    if (tid < 32) s.table[tid] = kExp2Table[tid];
    if (tid == 0) s.near_n = 0, s.near_count = 0, s.near_mass = 0, s.beyond = 0;
    if (!(temperature > 0.f)) temperature = 0.f, min_p = 0.f, top_p = 1.f, top_k = 1;
    min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
    if (top_k <= 0 || top_k > p.V) top_k = p.V;

    // ---- what can matter ----------------------------------------------------------------
    float top = -INFINITY, low = INFINITY, bound = -INFINITY;
    {
      int place[kLoads];
#pragma unroll
      for (int r = 0; r < kLoads; ++r) {
        const float x = max_of(first[r]);
        top = fmaxf(top, x), low = fminf(low, min_of(first[r]));
        place[r] = place_of(__float_as_uint(x) >> 16);
      }
      const int mine = (top_k + kWarps * C - 1) / (kWarps * C);
      if (each > kFewGranules && mine <= 32 * kLoads) {
        // a place that so many of the warp's granules reach, the least but for its last five bits
        int lo = 0, hi = kPlaceEnd >> 5;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          int n = 0;
#pragma unroll
          for (int r = 0; r < kLoads; ++r) n += place[r] < (mid + 1) << 5;
          if (int(__reduce_add_sync(0xffffffffu, unsigned(n))) >= mine) hi = mid;
          else lo = mid + 1;
        }
        if (lo < kPlaceEnd >> 5) bound = value_at((lo << 5) + 31);
      }
      top = warp_max(top), low = warp_min(low);
      if (lane == 0) s.warp_top[warp] = top, s.warp_low[warp] = low, s.warp_bound[warp] = bound;
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all of them do
    if (tid < C) {
      Told t{s.warp_top[0], s.warp_low[0], s.warp_bound[0], 0};
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
        t.top = fmaxf(t.top, s.warp_top[w]), t.low = fminf(t.low, s.warp_low[w]), t.bound = fminf(t.bound, s.warp_bound[w]);
      (C > 1 ? cluster.map_shared_rank(s.told[0], tid) : s.told[0])[rank] = t;
    }
    together();
    top = s.told[0][0].top, low = s.told[0][0].low, bound = s.told[0][0].bound;
#pragma unroll
    for (int i = 1; i < C; ++i) top = fmaxf(top, s.told[0][i].top), low = fminf(low, s.told[0][i].low), bound = fminf(bound, s.told[0][i].bound);
    // Weights under 2^-44 count as 0: 46 ln 2 temperatures below the largest.  Rounding moves these
    // bounds by far less than a step of bf16, and never above the largest.
    if (top > -INFINITY && top < INFINITY) {
      bound = fmaxf(bound, top - 31.9f * temperature);
      if (min_p > 0.f) bound = fmaxf(bound, top + temperature * __logf(min_p) - (1e-3f * temperature + 1e-6f * fabsf(top)));
    } else if (top == INFINITY) {
      bound = INFINITY;
    }
    bound = fmaxf(bound, -3.3895314e38f);  // the least finite number
    // the largest magnitude that may come; where more is read than was looked at, of twice that
    uint32_t magnitude = (__float_as_uint(fmaxf(fabsf(top), fabsf(fmaxf(low, bound)))) >> 16);
    if (!(top > -INFINITY)) magnitude = 0;
    int binade = int(magnitude >> 7) + (each > kTile);

    // ---- counts by value ------------------------------------------------------------------
    int base;
    const uint32_t bins = smem_u32(s.hist + kMagnitudes);
    for (;;) {
      base = max(0, ((min(binade, 255) + 1) << 7) - kMagnitudes);
      const uint32_t least_magnitude = uint32_t(base) << 16;
      float most = -INFINITY;
      auto look = [&](const uint4(&q)[kLoads]) {
#pragma unroll
        for (int r = 0; r < kLoads; ++r) {
          const float x = max_of(q[r]);
          most = fmaxf(most, x);
          // branches are the warp's, so that it stays together
          if (!__any_sync(0xffffffffu, x >= bound)) continue;
          const uint32_t w[4] = {q[r].x, q[r].y, q[r].z, q[r].w};
          uint32_t far = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            far = max(far, max(count_value(lo_of(w[j]), bound, least_magnitude, bins), count_value(hi_of(w[j]), bound, least_magnitude, bins)));
          if (!__any_sync(0xffffffffu, far >= uint32_t(kMagnitudes) << 16)) continue;
#pragma unroll 1
          for (int j = 0; j < 8; ++j) {  // some that matter have no bin
            const uint32_t bits = half_of(q[r], j), a = bits & 0x7fffu;
            if (bf2f(uint16_t(bits)) >= bound && a - uint32_t(base) >= uint32_t(kMagnitudes)) {
              if (a < uint32_t(base)) {
                const uint32_t i = atomicAdd(&s.near_n, 1u);
                if (i < uint32_t(kNear)) s.near[i] = uint16_t(place_of(bits));
              } else {
                atomicMax(&s.beyond, int(a));
              }
            }
            __syncwarp();
          }
        }
      };
      uint4 next[kLoads];
      int g = g0 + tid + kTile;
      if (g - tid < g1) load(next, g);
      look(first);
      for (; g - tid < g1; g += kTile) {
        uint4 q[kLoads];
#pragma unroll
        for (int r = 0; r < kLoads; ++r) q[r] = next[r];
        if (g - tid + kTile < g1) load(next, g + kTile);
        look(q);
      }
      most = warp_max(most);
      if (lane == 0) s.warp_top[warp] = most;
      __syncthreads();
      if (tid < C) {
        Told t{s.warp_top[0], 0.f, 0.f, s.beyond};
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t.top = fmaxf(t.top, s.warp_top[w]);
        (C > 1 ? cluster.map_shared_rank(s.told[1], tid) : s.told[1])[rank] = t;
      }
      together();
      top = s.told[1][0].top;
      int beyond = s.told[1][0].beyond;
#pragma unroll
      for (int i = 1; i < C; ++i) top = fmaxf(top, s.told[1][i].top), beyond = max(beyond, s.told[1][i].beyond);
      if (!beyond) break;
      // once more, with the bins that hold the largest of all
      binade = beyond >> 7;
      together();  // everybody has read what was told
      for (int i = 4 * tid; i < kBins; i += 4 * kThreads) *reinterpret_cast<uint4 *>(s.hist + i) = make_uint4(0, 0, 0, 0);
      if (tid == 0) s.near_n = 0, s.beyond = 0;
      __syncthreads();
    }

    if (!(top > -INFINITY)) {  // nothing above -infinity: what greedy acceptance takes, and no probability
      if (rank == 0) token = locate_in_order(row, 0, row.granules, kPlaceEnd, 1, s);
      logp = -INFINITY;
    } else {
      const int best = place_of(__float_as_uint(top) >> 16);
      const Scale scale = temperature > 0.f ? scale_of(temperature) : Scale{0.f, 0.f};
      const u64 least = __float2ull_ru(min_p * float(kWeightOne));  // exact before it is rounded up
      auto place_at = [&](int bin) { return bin < kMagnitudes ? kPlaceZero - base - (kMagnitudes - 1 - bin) : 0x8000 + base + bin - kMagnitudes; };
      Shared &s0 = C > 1 ? *cluster.map_shared_rank(&s, 0) : s;

      // ---- the cluster's counts, and its groups' counts and masses ---------------------------
      uint32_t *sum = C > 1 ? s.sum : s.hist;  // in the first CTA
#pragma unroll 2
      for (int group = rank * kWarps + warp; group < kGroups; group += C * kWarps) {
        const int bin = group * 32 + lane;
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) n += (C > 1 ? cluster.map_shared_rank(s.hist, i) : s.hist)[bin];
        uint32_t count = 0;
        u64 mass = 0;
        if (__any_sync(0xffffffffu, n != 0)) {
          const u64 w = weight_of(place_at(bin), best, scale, s.table);
          if (w < least) n = 0;
          count = __reduce_add_sync(0xffffffffu, n);
          mass = warp_sum(n * w);
        }
        if (C > 1) s0.sum[bin] = n;
        else if (least) s.hist[bin] = n;
        if (lane == 0) s0.group_count[group] = count, s0.group_mass[group] = mass;
      }
      // values near zero: from the list, or, where it was too short, from the slice once more
      const uint32_t near_n = s.near_n;
      if (near_n) {
        uint32_t count = 0;
        u64 mass = 0;
        auto add = [&](int place) {
          const u64 w = weight_of(place, best, scale, s.table);
          if (w >= least) ++count, mass += w;
        };
        if (near_n <= uint32_t(kNear)) {
          for (uint32_t i = tid; i < near_n; i += kThreads) add(s.near[i]);
        } else {
          for (int g = g0 + tid; g < g1; g += kThreads) {
            const uint4 q = row.load(g);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              const uint32_t bits = half_of(q, j);
              if (int(bits & 0x7fffu) < base && bf2f(uint16_t(bits)) >= bound) add(place_of(bits));
            }
          }
        }
        count = __reduce_add_sync(0xffffffffu, count), mass = warp_sum(mass);
        if (lane == 0 && count) atomicAdd(&s0.near_count, count), atomicAdd(&s0.near_mass, mass);
      }
      together();

      if (rank == 0) {
        // ---- three questions, asked by the first warp -------------------------------------------
        if (warp == 0) {
          constexpr int kMine = kGroups / 32;  // groups of a lane
          uint32_t count[kMine], before = 0;
          u64 mass[kMine], mass_before = 0;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            count[i] = s.group_count[lane * kMine + i], mass[i] = s.group_mass[lane * kMine + i];
            before += count[i], mass_before += mass[i];
          }
          const uint32_t own_count = before;
          const u64 own_mass = mass_before;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
            const u64 y = __shfl_up_sync(0xffffffffu, mass_before, o);
            if (lane >= o) before += x, mass_before += y;
          }
          const uint32_t near_at = __shfl_sync(0xffffffffu, before, 15);  // before the values near zero
          const u64 near_mass_at = __shfl_sync(0xffffffffu, mass_before, 15);
          if (lane >= 16) before += s.near_count, mass_before += s.near_mass;
          const uint32_t total_count = __shfl_sync(0xffffffffu, before, 31);
          const u64 total = __shfl_sync(0xffffffffu, mass_before, 31);
          before -= own_count, mass_before -= own_mass;
          auto find = [&](Question what, u64 target) -> Found {
            int group = -1;
            uint32_t c0 = before, c = 0;
            u64 m0 = mass_before, m = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
              if (answers(what, target, c0, c0 + count[i], m0, m0 + mass[i])) group = lane * kMine + i, c = c0, m = m0;
              c0 += count[i], m0 += mass[i];
            }
            const uint32_t who = __ballot_sync(0xffffffffu, group >= 0);
            Found f{best, 1, kWeightOne, 0, 0};
            if (!who) {  // among the values near zero: the whole CTA looks
              if (lane == 0) s.asked = Asked{what, target}, s.found = f, s.before_count = near_at, s.before_mass = near_mass_at;
              __syncthreads();
              find_in_windows(row, kPlaceZero - base + 1, 0x8000 + base, best, scale, least, near_at, near_mass_at, what, target, s);
              return s.found;
            }
            const int lead = __ffs(who) - 1;
            group = __shfl_sync(0xffffffffu, group, lead);
            c = __shfl_sync(0xffffffffu, c, lead), m = __shfl_sync(0xffffffffu, m, lead);
            const int bin = group * 32 + lane, place = place_at(bin);
            const uint32_t n = sum[bin];
            const u64 w = weight_of(place, best, scale, s.table);
            uint32_t c1 = n;
            u64 m1 = n * w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint32_t x = __shfl_up_sync(0xffffffffu, c1, o);
              const u64 y = __shfl_up_sync(0xffffffffu, m1, o);
              if (lane >= o) c1 += x, m1 += y;
            }
            c1 += c, m1 += m;
            const bool here = n && answers(what, target, c1 - n, c1, m1 - n * w, m1);
            if (here) f = Found{place, number_of(what, target, c1 - n, m1 - n * w, w), w, m1 - n * w, 1};
            const uint32_t whose = __ballot_sync(0xffffffffu, here);
            const int from = whose ? __ffs(whose) - 1 : 0;
            f.place = __shfl_sync(0xffffffffu, f.place, from), f.n = __shfl_sync(0xffffffffu, f.n, from);
            f.w = __shfl_sync(0xffffffffu, f.w, from), f.mass = __shfl_sync(0xffffffffu, f.mass, from);
            return f;
          };
          u64 rest = total;
          if (uint32_t(top_k) < total_count) {
            const Found f = find(kCount, u64(top_k));
            rest = f.mass + f.n * f.w;
          }
          if (top_p < 1.f) {
            const Found f = find(kMassReaches, max(u64(1), share_of(fmaxf(top_p, 0.f), rest, true)));
            rest = f.mass + f.n * f.w;
          }
          const float u = p.u[bt];
          const Found f = find(kMassPasses, u > 0.f ? (u < 1.f ? share_of(u, rest, false) : rest - 1) : 0);
          logp = -log1pf(float(rest - f.w) / float(f.w));
          if (lane == 0) s.asked.what = -1, s.found = f;
          __syncthreads();
        } else {
          for (;;) {
            __syncthreads();
            const Asked a = s.asked;
            if (a.what < 0) break;
            find_in_windows(row, kPlaceZero - base + 1, 0x8000 + base, best, scale, least, s.before_count, s.before_mass, Question(a.what), a.target, s);
          }
        }

        // ---- the logit ---------------------------------------------------------------------------
        const Found f = s.found;
        const int a = f.place <= kPlaceZero ? kPlaceZero - f.place : f.place - 0x8000;
        if (a < base) {
          token = locate_in_order(row, 0, row.granules, f.place, f.n, s);
        } else {
          const int bin = f.place <= kPlaceZero ? kMagnitudes - 1 - (a - base) : kMagnitudes + a - base;
          uint32_t n = f.n, all = s.hist[bin];
          int q = 0;
          if (C > 1) {
            while (q < C - 1 && n > all) n -= all, ++q, all = cluster.map_shared_rank(s.hist, q)[bin];
          }
          const int from = min(row.granules, q * each);
          token = locate(row, from, min(row.granules, from + each), f.place, n, all, s);
        }
      }
    }
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
      p.ws_count[b] = 0;  // ready for the next call
    }
  }
}

template <int C>
cudaError_t launch(const SampleParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.B) * unsigned(p.T) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<C>, p);
}

}  // namespace

size_t accept_sampled_workspace_bytes(int B, int T) {
  return align256(size_t(B) * T * sizeof(int32_t)) + align256(size_t(B) * sizeof(uint32_t));
}

cudaError_t launch_sample(const SampleParams &p, cudaStream_t s) {
  const int rows = p.B * p.T;
  int C = 8;
  while (C > 1 && (rows * C > (C > 2 ? 608 : 1216) || p.V < 2048 * C)) C /= 2;
  switch (C) {
    case 8: return launch<8>(p, s);
    case 4: return launch<4>(p, s);
    case 2: return launch<2>(p, s);
    default: return launch<1>(p, s);
  }
}

}  // namespace gdn

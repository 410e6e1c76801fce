// sample.cu -- sampled decoding: a token of every position by temperature, min-p,
// top-k and top-p from a given random number, and the accepted prefix of a verify's
// drafts.
//
// One CTA a position.  A row's values are taken in windows of 2048 places of the
// order, from the largest down: the CTA counts the row's logits in the window in
// shared memory, sums counts and masses over it, and stops where the question at hand
// is answered: which value ends the first k, which ends the first p of the mass, which
// one u falls on.  Windows begin at the next value that the row has.
#include "sample.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 2048;
constexpr int kPer = kWindow / kThreads;  // places of a thread

typedef unsigned long long u64;

struct Found {
  int place;       // the value
  uint32_t n;      // logits of that value up to the one that was asked for, it included
  uint32_t count;  // logits before that value
  u64 w, mass;     // its weight; the mass before that value
  int hit;         // 0: not within what the row has; count and mass are of all
};

struct Shared {
  uint32_t hist[kWindow];
  u64 table[32];
  u64 warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  int low;     // least place behind the window
  int place;   // least place of the row
  Found found;
  int last;
};

enum Question { kCount, kMassReaches, kMassPasses };

// Inclusive sums over the CTA of (count, mass).
__device__ __forceinline__ void scan(uint32_t &count, u64 &mass, Shared &s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, count, o);
    const u64 b = __shfl_up_sync(0xffffffffu, mass, o);
    if (lane >= o) count += a, mass += b;
  }
  if (lane == 31) s.warp_count[warp] = count, s.warp_mass[warp] = mass;
  __syncthreads();
  for (int w = 0; w < warp; ++w) count += s.warp_count[w], mass += s.warp_mass[w];
}

// The first value, among those with weight >= least, at which the number of logits (kCount) or
// their mass reaches the target, or their mass passes it.
__device__ Found find(const SampleRow &row, int top, Scale c, u64 least, Question what, u64 target, Shared &s) {
  const int tid = threadIdx.x;
  int from = top;
  uint32_t count0 = 0;
  u64 mass0 = 0;
  for (;;) {
    __syncthreads();
    for (int i = tid; i < kWindow; i += kThreads) s.hist[i] = 0;
    if (tid == 0) s.low = kPlaceEnd, s.found.hit = 0;
    __syncthreads();
    int low = kPlaceEnd;
    for (int g = tid; g < row.granules; g += kThreads) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = place_of(half_of(q, j)) - from;
        if (at >= 0 && at < kWindow) atomicAdd(&s.hist[at], 1u);
        else if (at >= kWindow) low = min(low, at + from);
      }
    }
    if (low < kPlaceEnd) atomicMin(&s.low, low);
    __syncthreads();
    u64 w[kPer];
    uint32_t n[kPer], count = 0;
    u64 mass = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int place = from + tid * kPer + i;
      n[i] = place < kPlaceEnd ? s.hist[tid * kPer + i] : 0;
      w[i] = n[i] ? weight_of(place, top, c, s.table) : 0;
      if (w[i] < least) n[i] = 0;
      count += n[i], mass += n[i] * w[i];
    }
    uint32_t count1 = count;
    u64 mass1 = mass;
    scan(count1, mass1, s);
    count1 += count0, mass1 += mass0;
    count = count1 - count, mass = mass1 - mass;  // before this thread's places
    const bool here = what == kCount ? count < target && target <= count1
                                     : what == kMassReaches ? mass < target && target <= mass1 : mass <= target && target < mass1;
    if (here) {
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        const u64 m = mass + n[i] * w[i];
        if (n[i] && (what == kCount ? target <= count + n[i] : what == kMassReaches ? target <= m : target < m)) {
          Found f;
          f.place = from + tid * kPer + i, f.count = count, f.w = w[i], f.mass = mass, f.hit = 1;
          f.n = what == kCount ? uint32_t(target - count)
                               : what == kMassReaches ? uint32_t((target - mass + w[i] - 1) / w[i]) : uint32_t((target - mass) / w[i]) + 1;
          s.found = f;
          break;
        }
        count += n[i], mass = m;
      }
    }
    if (tid == kThreads - 1) s.warp_count[0] = count1, s.warp_mass[0] = mass1;
    __syncthreads();
    count0 = s.warp_count[0], mass0 = s.warp_mass[0];
    from = s.low;
    if (s.found.hit) return s.found;
    // behind the least weight nothing counts any more
    const u64 next = from < kPlaceEnd ? weight_of(from, top, c, s.table) : 0;
    if (next < least || next == 0) {
      Found f{};
      f.count = count0, f.mass = mass0;
      return f;
    }
  }
}

// Index of the n-th logit (from 1) with the given place.
__device__ int locate(const SampleRow &row, int place, uint32_t n, Shared &s) {
  const int tid = threadIdx.x;
  uint32_t before = 0;
  for (int g0 = 0; g0 < row.granules; g0 += kThreads) {
    const int g = g0 + tid;
    uint32_t mask = 0;
    if (g < row.granules) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) mask |= uint32_t(place_of(half_of(q, j)) == place) << j;
    }
    __syncthreads();
    uint32_t end = __popc(mask);
    u64 none = 0;
    scan(end, none, s);
    end += before;
    if (end >= n && end - __popc(mask) < n) {
      uint32_t left = n - (end - __popc(mask)), j = 0;
      for (;; ++j)
        if ((mask >> j & 1) && --left == 0) break;
      s.last = row.first(g) + int(j);
    }
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += s.warp_count[w];
    before += all;
    if (before >= n) return s.last;
  }
  return 0;
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  __shared__ Shared s;
  const int tid = threadIdx.x;
  const int bt = blockIdx.x, b = bt / p.T;
  pdl_wait();
  pdl_trigger();
  if (tid < 32) s.table[tid] = kExp2Table[tid];
  if (tid == 0) s.place = 0xffff;
  __syncthreads();
  const bool active = !p.active || p.active[b];
  int token = -1;
  float logp = 0.f;
  if (active) {
    const SampleRow row(p.logits + size_t(bt) * p.stride, p.V);
    int top = 0xffff;
    for (int g = tid; g < row.granules; g += kThreads) {
      const uint4 q = row.load(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = min(top, place_of(half_of(q, j)));
    }
    atomicMin(&s.place, top);
    __syncthreads();
    top = s.place;
    __syncthreads();
    const float temperature = p.temperature ? p.temperature[b] : 1.f;
    if (top >= kPlaceEnd) {  // nothing above -infinity: what greedy acceptance takes, and no probability
      token = top == kPlaceEnd ? locate(row, top, 1, s) : 0;
      logp = -INFINITY;
    } else if (!(temperature > 0.f)) {
      token = locate(row, top, 1, s);
    } else {
      const Scale c = scale_of(temperature);
      const float min_p = p.min_p ? p.min_p[b] : 0.f, top_p = p.top_p ? p.top_p[b] : 1.f;
      const int top_k = p.top_k ? p.top_k[b] : 0;
      const u64 least = min_p > 0.f ? u64(ceil(fmin(double(min_p), 1.0) * double(kWeightOne))) : 0;
      Found f = find(row, top, c, least, kCount, top_k > 0 && top_k < p.V ? u64(top_k) : u64(p.V) + 1, s);
      u64 mass = f.hit ? f.mass + f.n * f.w : f.mass;
      if (top_p < 1.f) {
        const u64 want = max(u64(1), min(mass, u64(ceil(double(fmaxf(top_p, 0.f)) * double(mass)))));
        f = find(row, top, c, least, kMassReaches, want, s);
        mass = f.mass + f.n * f.w;
      }
      const float u = p.u[bt];
      const u64 at = u > 0.f ? min(mass - 1, u64(double(fminf(u, 1.f)) * double(mass))) : 0;
      f = find(row, top, c, least, kMassPasses, at, s);
      token = locate(row, f.place, f.n, s);
      logp = -log1pf(float(mass - f.w) / float(f.w));
    }
  }
  if (tid == 0) {
    if (p.token) p.token[bt] = token;
    if (p.logp) p.logp[bt] = logp;
  }
  if (!p.draft) return;

  // ---- acceptance: the row's last CTA decides -------------------------------------------
  if (tid == 0) {
    p.ws_token[bt] = token;
    __threadfence();  // the token is visible before it is counted
    s.last = atomicAdd(&p.ws_count[b], 1u) + 1u == uint32_t(p.T);
    if (s.last) {
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

}  // namespace

size_t accept_sampled_workspace_bytes(int B, int T) {
  return align256(size_t(B) * T * sizeof(int32_t)) + align256(size_t(B) * sizeof(uint32_t));
}

cudaError_t launch_sample(const SampleParams &p, cudaStream_t s) {
  return launch_pdl(sample_kernel, dim3(p.B * p.T), dim3(kThreads), s, p);
}

}  // namespace gdn

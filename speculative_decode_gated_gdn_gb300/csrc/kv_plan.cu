// kv_plan.cu -- block tables, slots and positions of a cycle's new tokens,
// from the rows' committed lengths, on the device.
//
// Per row b: a = active ? max(add, 0) : 0 new tokens, want = ceil((len + a) / P)
// pages.  Rows that hold more give the rest back (pushed on the free stack in
// row order); rows that hold less take pages from the stack's end, in row
// order.  Both places are prefix sums over the rows, so the result does not
// depend on the order in which threads run.
//
// The work is a few integers a row and a token: what bounds it is latency, so
// one CTA does the bookkeeping of all rows (scans in shared memory, pages
// moved one a thread by a search in the scan, whichever row they belong to),
// and, where the tokens are few, writes their slots too.
#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kPlanThreads = 1024;
// Tokens up to which the bookkeeping CTA writes the slots itself; a kernel of their own
// behind it costs 16 tokens 5.8 us for 4.7, and 2048 5.6 for 5.3, but 8192 take 5.5 for
// 7.3 and 65536 5.6 for 26.5.
constexpr int kPlanOneCta = 2048;

// Inclusive scan of v over the CTA; *total gets the sum of all threads.
__device__ __forceinline__ long long block_scan(long long v, long long *s_warp, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // s_warp may still be read by an earlier scan
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return v + (warp ? s_warp[warp - 1] : 0);
}

struct PlanRow {
  int len, a, held, want;
  bool bad;
};

__device__ __forceinline__ PlanRow plan_row(const KvPlanParams &p, int b) {
  PlanRow r;
  r.len = p.lens[b];
  r.held = p.held[b];
  const int add = p.add[b];
  r.a = p.active[b] && add > 0 ? add : 0;
  const long long P = 1ll << p.log2P;
  const long long want = ((long long)r.len + r.a + P - 1) >> p.log2P;
  r.bad = r.len < 0 || want > p.max_pages || (p.T > 0 && r.a > p.T) || r.held < 0 || r.held > p.max_pages;
  if (r.bad) r.a = 0;
  r.want = r.bad ? r.held : int(want);
  return r;
}

// First index i in [0, n) with ends[i] > x (ends ascending, ends[n - 1] > x).
__device__ __forceinline__ int find_row(const int *ends, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (ends[m] > x) hi = m;
    else lo = m + 1;
  }
  return lo;
}

// Slot and position of token i, -1 where no row has it.
__device__ __forceinline__ void plan_token(const KvPlanParams &p, int i) {
  const int b = p.T > 0 ? i / p.T : find_row(p.q_start + 1, p.B, i);
  int slot = -1, pos = -1;
  if (b < p.B) {
    const int k = i - p.q_start[b];
    if (k < p.q_count[b]) {
      pos = p.lens[b] + k;
      const int page = p.table[size_t(b) * p.max_pages + (pos >> p.log2P)];
      slot = page < 0 ? -1 : (page << p.log2P) + (pos & ((1 << p.log2P) - 1));
    }
  }
  p.slots[i] = slot;
  p.positions[i] = pos;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanParams p, const int write_slots) {
  __shared__ long long s_warp[32];
  __shared__ int s_ends[kPlanThreads];   // pages that the chunk's rows move, summed up to each row
  __shared__ int s_from[kPlanThreads];   // first table column that the row moves
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int n_pages = p.n_pages;
  const int count0 = min(max(*p.free_count, 0), n_pages);

  // ---- pages given back --------------------------------------------------------
  long long released = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid, rows = min(kPlanThreads, p.B - b0);
    PlanRow r{};
    if (b < p.B) r = plan_row(p, b);
    if (b < p.B && r.bad) atomicOr(p.status, GDN_STATUS_BAD_LEN);
    const int rel = max(r.held - r.want, 0);
    long long total;
    const long long end = block_scan(rel, s_warp, &total);
    if (total == 0) continue;  // the same for every thread
    s_ends[tid] = int(end);
    s_from[tid] = r.want;
    __syncthreads();
    for (int i = tid; i < int(total); i += kPlanThreads) {
      const int w = find_row(s_ends, rows, i);
      int32_t *cell = p.table + size_t(b0 + w) * p.max_pages + s_from[w] + i - (w ? s_ends[w - 1] : 0);
      const long long at = count0 + released + i;
      if (at < n_pages) p.free_list[at] = *cell;
      else atomicOr(p.status, GDN_STATUS_BAD_INDEX);
      *cell = -1;
    }
    released += total;
  }
  const long long avail = min((long long)n_pages, count0 + released);
  __syncthreads();  // the pushed pages are visible to the whole CTA

  // ---- pages taken, in row order -----------------------------------------------
  long long taken0 = 0, tokens0 = 0, granted = 0, got_sum = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid, rows = min(kPlanThreads, p.B - b0);
    PlanRow r{};
    if (b < p.B) r = plan_row(p, b);
    const int need = max(r.want - r.held, 0);
    long long need_total, tok_total;
    const long long need_end = taken0 + block_scan(need, s_warp, &need_total);
    const long long tok_end = tokens0 + block_scan(r.a, s_warp, &tok_total);
    const bool fits = need_end <= avail && (p.T > 0 || tok_end <= p.N);
    if (b < p.B && !fits && (need || r.a)) atomicOr(p.status, GDN_STATUS_NO_PAGES);
    const int got = fits ? need : 0, a = fits ? r.a : 0;
    // every row that got pages precedes every row that did not, so a row's
    // place among the pages taken is the plain prefix sum
    long long got_total;
    const long long got_end = block_scan(got, s_warp, &got_total);
    s_ends[tid] = int(got_end);
    s_from[tid] = r.held;
    // packed layout: a refused row has no tokens, and rows after it none either
    long long a_total;
    const long long a_end = block_scan(a, s_warp, &a_total);
    if (b < p.B) {
      p.q_count[b] = a;
      p.kv_len[b] = max(r.len, 0) + a;
      p.q_start[b] = p.T > 0 ? b * p.T : int(granted + a_end - a);
      if (b == p.B - 1) p.q_start[p.B] = p.T > 0 ? p.B * p.T : int(granted + a_end);
      p.held[b] = r.held - max(r.held - r.want, 0) + got;
    }
    __syncthreads();
    for (int i = tid; i < int(got_total); i += kPlanThreads) {
      const int w = find_row(s_ends, rows, i);
      const long long from = avail - 1 - (taken0 + i);
      p.table[size_t(b0 + w) * p.max_pages + s_from[w] + i - (w ? s_ends[w - 1] : 0)] = p.free_list[from];
    }
    taken0 += need_total;
    tokens0 += tok_total;
    granted += a_total;
    got_sum += got_total;
    __syncthreads();  // s_ends is free for the next chunk, and the rows' results are visible
  }
  if (tid == 0) *p.free_count = int(avail - got_sum);
  if (!write_slots) return;
  for (int i = tid; i < p.N; i += kPlanThreads) {
    plan_token(p, i);
  }
}

// The slots of many tokens, on the rows as kv_plan_kernel left them.
__global__ void __launch_bounds__(256) kv_slots_kernel(const KvPlanParams p) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.N) return;
  plan_token(p, i);
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t s) {
  const bool one = p.N <= kPlanOneCta;
  void *args[2];
  const int flag = one ? 1 : 0;
  args[0] = const_cast<KvPlanParams *>(&p), args[1] = const_cast<int *>(&flag);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kv_plan_kernel), args);
  if (e != cudaSuccess || one) return e;
  return launch_pdl(kv_slots_kernel, dim3((p.N + 255) / 256), dim3(256), s, p);
}

}  // namespace gdn

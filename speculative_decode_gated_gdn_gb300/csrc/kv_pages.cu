// kv_pages.cu -- pages of the attention cache between rows: forks that share them,
// compaction, and copies in all layers.
//
// A fork's row gets the source's full pages as they are (a holder more each) and a
// page of its own for the last, partly filled one.  Rows only write behind their own
// length, so nobody writes a shared page.
//
// The bookkeeping is a few dependent trips to L2, so it is latency that counts: one
// kernel of one cluster does it where it is small, whose CTAs wait for the first one's
// decisions and then share the cells; where it is large, a second kernel of many CTAs
// does the cells.  Behind other kernels eight forks of 207 pages take 4.9 us, 256 of 62
// 5.8; a compaction of 90 pages 4.8, of 11,818 pages and cells 10.7.  Copies are bound by
// HBM: 11,820 pages of 36,864 bytes in 133 us, 6.5 TB/s read and written, 0.97 of a plain
// copy.
#include <cooperative_groups.h>

#include <climits>

#include "kv4.cuh"
#include "scan.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;

// ---- forks --------------------------------------------------------------------------
struct ForkPair {
  int src, dst, len, want;
  bool rows;  // two rows of the cohort
};
enum { kAsks, kNothing, kBadRow, kBadLen, kBadPage };

__device__ __forceinline__ ForkPair fork_pair(const KvForkParams &p, int i) {
  ForkPair r;
  r.src = p.src_rows[i], r.dst = p.dst_rows[i], r.len = p.lens[i];
  const int P = 1 << p.log2P;
  r.want = int(((long long)r.len + P - 1) >> p.log2P);
  r.rows = r.src >= 0 && r.src < p.B && r.dst >= 0 && r.dst < p.B && r.src != r.dst;
  return r;
}

// What a pair leaves in the count of an empty row that it asks for: below what else stands there, the least for
// the first pair.
__device__ __forceinline__ int claim(int i) { return INT_MIN + i; }
__device__ __forceinline__ bool is_empty(int held) { return held == 0 || held < claim(kMaxForks); }

// Which pairs hold, and their last pages.  An empty row goes to the first pair that asks for it and, if that one
// gets no page, to the first later one that needs none.
__device__ void decide_forks(const KvForkParams &p, long long *s_warp) {
  const int tid = threadIdx.x;
  const int count0 = min(max(*p.free_count, 0), p.n_pages);
  auto held_of = [&](int row) { return *(volatile int32_t *)(p.held + row); };
  // a pair's verdict stands in copy_src until its page does; its thread is the same every time
  for (int i = tid; i < p.n; i += kScanThreads) {
    const ForkPair r = fork_pair(p, i);
    int verdict = kBadRow;
    if (r.len < 0 || r.want > p.max_pages) {
      verdict = kBadLen;
    } else if (r.rows) {
      const int held = held_of(r.src);
      const bool empty = is_empty(held_of(r.dst));
      const int whole = r.len >> p.log2P, last = r.want > whole ? p.table[size_t(r.src) * p.max_pages + whole] : 0;
      if (held < r.want || held > p.max_pages) {
        if (r.want > 0) verdict = kBadLen;
        else if (empty) verdict = kNothing;
      } else if (empty) {
        verdict = !r.len ? kNothing : last < 0 || last >= p.n_pages ? kBadPage : kAsks;
        if (verdict == kAsks) atomicMin(p.held + r.dst, claim(i));
      }
    }
    p.copy_src[i] = verdict;
  }
  sync_cta();
  constexpr int kLate = -3;  // in copy_dst: another pair asked first
  long long taken = 0, late = 0;
  for (int i0 = 0; i0 < p.n; i0 += kScanThreads) {
    const int i = i0 + tid;
    ForkPair r{};
    int verdict = kNothing;
    bool won = false;
    if (i < p.n) {
      r = fork_pair(p, i);
      verdict = p.copy_src[i];
      won = verdict == kAsks && held_of(r.dst) == claim(i);
    }
    const int whole = r.len >> p.log2P, need = won && r.want > whole;
    long long all;
    const long long end = taken + (block_scan(need | (long long)(verdict == kAsks && !won) << 32, s_warp, &all) & 0xffffffff);
    if (i < p.n) {
      int from = -2, to = -2;
      if (won) {
        bool made = !need || end <= count0;
        if (!made) atomicOr(p.status, GDN_STATUS_NO_PAGES);
        if (made && need) {
          const int page = p.free_list[count0 - end];
          made = page >= 0 && page < p.n_pages;
          if (made) {
            from = p.table[size_t(r.src) * p.max_pages + whole], to = page;
            p.table[size_t(r.dst) * p.max_pages + whole] = page;
            p.refs[page] = 1;
          } else {
            atomicOr(p.status, GDN_STATUS_BAD_INDEX);
          }
        } else if (made) {
          from = to = -1;
        }
        p.held[r.dst] = made ? r.want : 0;
      } else if (verdict == kAsks) {
        to = kLate;
      } else if (verdict == kNothing) {
        from = to = -1;
      } else {
        atomicOr(p.status, verdict == kBadLen ? GDN_STATUS_BAD_LEN : verdict == kBadPage ? GDN_STATUS_BAD_INDEX : GDN_STATUS_BAD_ROW);
      }
      p.copy_src[i] = from, p.copy_dst[i] = to;
    }
    taken += all & 0xffffffff, late += all >> 32;
    sync_cta();
  }
  if (tid == 0) *p.free_count = count0 - int(min(taken, (long long)count0));
  if (late == 0) return;  // the same for every thread

  // the pairs that came late, where the first one's page was missing
  for (int i = tid; i < p.n; i += kScanThreads) {
    const ForkPair r = fork_pair(p, i);
    if (p.copy_dst[i] == kLate && r.want == r.len >> p.log2P && is_empty(held_of(r.dst))) atomicMin(p.held + r.dst, claim(i));
  }
  sync_cta();
  for (int i = tid; i < p.n; i += kScanThreads) {
    if (p.copy_dst[i] != kLate) continue;
    const int held = held_of(p.dst_rows[i]);  // pages, or what the row's pair left, or 0
    const bool made = held == claim(i), before = held > 0 || (held < 0 && held < claim(i));
    if (!made) atomicOr(p.status, before || taken <= count0 ? GDN_STATUS_BAD_ROW : GDN_STATUS_NO_PAGES);
    p.copy_src[i] = p.copy_dst[i] = made ? -1 : -2;
  }
  sync_cta();
  for (int i = tid; i < p.n; i += kScanThreads) {
    const ForkPair r = fork_pair(p, i);
    if (p.copy_src[i] == -1 && r.len > 0 && held_of(r.dst) == claim(i)) p.held[r.dst] = r.want;
  }
}

// The shared pages' cells and counts of pair i, if it holds: cells first, first + step, ...
__device__ __forceinline__ void share_cells(const KvForkParams &p, int i, int first, int step) {
  if (__ldcg(p.copy_src + i) == -2) return;
  const ForkPair r = fork_pair(p, i);
  const int whole = r.len >> p.log2P;
  const int32_t *from = p.table + size_t(r.src) * p.max_pages;
  int32_t *to = p.table + size_t(r.dst) * p.max_pages;
  for (int c = first; c < whole; c += step) {
    const int page = from[c];
    to[c] = page;
    if (page >= 0 && page < p.n_pages) atomicAdd(p.refs + page, 1);
    else atomicOr(p.status, GDN_STATUS_BAD_INDEX);
  }
}

__global__ void __launch_bounds__(kScanThreads) kv_fork_kernel(const KvForkParams p) {
  __shared__ long long s_warp[32];
  pdl_wait();
  pdl_trigger();
  decide_forks(p, s_warp);
}

// Both in one cluster; a warp has a pair, or a part of one.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads) kv_fork_cluster_kernel(const KvForkParams p) {
  __shared__ long long s_warp[32];
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  if (cluster.block_rank() == 0) decide_forks(p, s_warp);
  __syncwarp();
  cluster.sync();
  constexpr int kWarps = kCluster * kScanThreads / 32;
  const int g = int(cluster.block_rank()) * (kScanThreads / 32) + int(threadIdx.x >> 5);
  const int parts = p.n < kWarps ? kWarps / p.n : 1;
  for (int i = g / parts; i < p.n; i += kWarps / parts) share_cells(p, i, (g % parts) * 32 + int(threadIdx.x & 31), parts * 32);
}

constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) kv_share_kernel(const KvForkParams p) {
  pdl_wait();
  pdl_trigger();
  share_cells(p, blockIdx.x, blockIdx.y * kForkThreads + threadIdx.x, gridDim.y * kForkThreads);
}

// ---- compaction ---------------------------------------------------------------------
// Counts in one cluster: each warp has a stretch of the pages, four a lane and step.
struct Stretch {
  int begin, end;
};
__device__ __forceinline__ Stretch stretch_of(int warp, int warps, int n) {
  const long long steps = (n + 127) / 128, each = (steps + warps - 1) / warps;
  return Stretch{int(min((long long)n, warp * each * 128)), int(min((long long)n, (warp + 1) * each * 128))};
}
// Which of the four pages from `at` on are in use, as bits.
__device__ __forceinline__ uint32_t used_of(const int32_t *refs, int at, int end) {
  if (at + 4 <= end && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
    const int4 x = *reinterpret_cast<const int4 *>(refs + at);
    return (x.x > 0) | (x.y > 0) << 1 | (x.z > 0) << 2 | (x.w > 0) << 3;
  }
  uint32_t m = 0;
  for (int j = 0; j < 4 && at + j < end; ++j) m |= uint32_t(refs[at + j] > 0) << j;
  return m;
}

// Tables, counts and the free stack by the map; item i of `step` threads.  Where an output
// is the input itself, each entry is read and written by one thread, or stands for the
// same either way.
__device__ __forceinline__ void remap(const KvCompactParams &p, int U, int moves, size_t first, size_t step) {
  const int n = p.n_pages;
  for (size_t i = first; i < size_t(p.B) * p.max_pages; i += step) {
    const int b = int(i / p.max_pages), c = int(i - size_t(b) * p.max_pages);
    int page = p.table[i];
    if (c < p.held[b]) {
      page = page >= 0 && page < n ? __ldcg(p.page_map + page) : -1;
      if (page < 0) atomicOr(p.status, GDN_STATUS_BAD_INDEX);
    }
    p.new_table[i] = page;
  }
  for (size_t i = first; i < size_t(n); i += step) {
    p.new_free_list[i] = i < size_t(n - U) ? n - 1 - int(i) : -1;
    const int r = p.refs[i];
    if ((r > 0) == (i < size_t(U))) p.new_refs[i] = max(r, 0);
  }
  for (size_t j = first; j < size_t(moves); j += step) {
    const int from = __ldcg(p.copy_src + j);
    const int r = p.refs[from];
    p.new_refs[__ldcg(p.copy_dst + j)] = r;
    p.new_refs[from] = 0;
  }
}

// In C CTAs; ALL: the tables too.
template <int C, bool ALL>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kScanThreads) kv_compact_kernel(const KvCompactParams p) {
  __shared__ long long s_warp[32];
  __shared__ int s_before[32], s_used[C], s_below;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = C > 1 ? int(cluster.block_rank()) : 0;
  auto together = [&] {
    __syncwarp();  // a warp that a loop has split would arrive more than once
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  const int n = p.n_pages;
  const Stretch s = stretch_of(rank * (kScanThreads / 32) + warp, C * (kScanThreads / 32), n);
  int count = 0;
#pragma unroll 4
  for (int at = s.begin + 4 * lane; at < s.end; at += 128) count += __popc(used_of(p.refs, at, s.end));
  long long used;
  const long long upto = block_scan(count, s_warp, &used);
  if (lane == 31) s_before[warp] = int(upto);
  __syncwarp();
  if (C > 1) cluster.sync();  // every CTA runs
  if (tid < C) (C > 1 ? cluster.map_shared_rank(s_used, tid) : s_used)[rank] = int(used);
  together();
  int U = 0, before = warp ? s_before[warp - 1] : 0;  // pages in use: all, before the stretch
  for (int q = 0; q < C; ++q) U += s_used[q], before += q < rank ? s_used[q] : 0;
  // pages in use below place U: those behind it move into the gaps
  if ((U >= s.begin && U < s.end) || (U == n && rank == 0 && warp == 0)) {
    int below = 0;
    if (U < n)
      for (int at = s.begin + 4 * lane; at < U; at += 128) below += __popc(used_of(p.refs, at, U));
    below = U < n ? before + __reduce_add_sync(0xffffffffu, below) : U;
    if (lane < C) *(C > 1 ? cluster.map_shared_rank(&s_below, lane) : &s_below) = below;
  }
  together();
  const int below = s_below;
  for (int base = s.begin; base < s.end; base += 128) {
    const int at = base + 4 * lane;
    const uint32_t m = at < s.end ? used_of(p.refs, at, s.end) : 0;
    int mine = __popc(m), sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    int k = before + sum - mine;  // pages in use before place at + j
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = at + j;
      if (i < s.end) {
        const bool in_use = m >> j & 1;
        if (!in_use || i < U) p.page_map[i] = in_use ? i : -1;  // the others' below
        if (in_use && i >= U) p.copy_src[k - below] = i;
        if (!in_use && i < U) p.copy_dst[i - k] = i;
        k += in_use;
      }
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  together();
  const int moves = U - below;
  for (int j = rank * kScanThreads + tid; j < moves; j += C * kScanThreads) p.page_map[__ldcg(p.copy_src + j)] = __ldcg(p.copy_dst + j);
  if (rank == 0 && tid == 0) *p.copy_count = moves, *p.new_free_count = n - U;
  if (!ALL) return;
  together();
  remap(p, U, moves, size_t(rank) * kScanThreads + tid, size_t(C) * kScanThreads);
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads) kv_remap_kernel(const KvCompactParams p) {
  pdl_wait();
  pdl_trigger();
  remap(p, p.n_pages - *p.new_free_count, *p.copy_count, size_t(blockIdx.x) * kRemapThreads + threadIdx.x, size_t(gridDim.x) * kRemapThreads);
}

// ---- copies -------------------------------------------------------------------------
constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int kCopyUnit = kCopyThreads * kCopyLoads * 16;  // bytes of a CTA's step

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ KvCopyParams p) {
  pdl_wait();
  pdl_trigger();
  const int n = p.count ? min(max(*p.count, 0), p.n) : p.n;
  const int units = (p.page_bytes + kCopyUnit - 1) / kCopyUnit;
  const size_t total = size_t(n) * p.n_layers * units;
  for (size_t u = blockIdx.x; u < total; u += gridDim.x) {
    const size_t q = u / units;
    const int part = int(u - q * units), layer = int(q / n), i = int(q - size_t(layer) * n);
    const int from = p.src[i], to = p.dst[i];
    if (from < 0 || to < 0) continue;
    if (from >= p.n_pages || to >= p.n_pages) {
      if (threadIdx.x == 0) atomicOr(p.status, GDN_STATUS_BAD_INDEX);
      continue;
    }
    const uint4 *s = reinterpret_cast<const uint4 *>(p.pages[layer] + size_t(from) * p.page_bytes);
    uint4 *d = reinterpret_cast<uint4 *>(p.pages[layer] + size_t(to) * p.page_bytes);
    const int words = p.page_bytes / 16, w0 = part * (kCopyUnit / 16) + threadIdx.x;
    uint4 x[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (w0 + j * kCopyThreads < words) x[j] = s[w0 + j * kCopyThreads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (w0 + j * kCopyThreads < words) d[w0 + j * kCopyThreads] = x[j];
  }
}

// Cells up to which one cluster does all: four a thread.  It saves a launch, 2 us of the caller's time, and on the GPU
// costs less than that, us behind other kernels in one cluster and in two kernels:
//   forks of 1,656 cells 4.9 / 4.2, 15,872 5.8 / 5.4, 32,768 6.2 / 5.1, 51,200 8.0 / 6.0, 131,072 10.9 / 8.6;
//   by the clock, with the caller, 13.0 / 14.7, 13.1 / 15.2, 13.0 / 14.2
//   compactions of 8,192 pages and cells 9.5 / 8.9, 32,768 11.4 / 9.5, 50,000 16.1 / 12.1
constexpr long long kOneClusterCells = 4ll * kCluster * kScanThreads;

// And one CTA: compactions of 1,000 pages and cells 5.0 us, in a cluster 7.3; 4,096 8.2 / 9.6; 6,000 10.3 / 9.1.
constexpr int kOneCtaCells = 4 * kScanThreads;

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 152;
}

}  // namespace

cudaError_t launch_kv_fork(const KvForkParams &p, cudaStream_t s) {
  if ((long long)p.n * p.max_pages <= kOneClusterCells) return launch_pdl(kv_fork_cluster_kernel, dim3(kCluster), dim3(kScanThreads), s, p);
  const cudaError_t e = launch_pdl(kv_fork_kernel, dim3(1), dim3(kScanThreads), s, p);
  if (e != cudaSuccess) return e;
  const int y = (p.max_pages + kForkThreads - 1) / kForkThreads;
  return launch_pdl(kv_share_kernel, dim3(p.n, y < 16 ? y : 16), dim3(kForkThreads), s, p);
}

cudaError_t launch_kv_compact(const KvCompactParams &p, cudaStream_t s) {
  const size_t cells = size_t(p.B) * p.max_pages, items = cells > size_t(p.n_pages) ? cells : size_t(p.n_pages);
  if (items <= size_t(kOneCtaCells)) return launch_pdl(kv_compact_kernel<1, true>, dim3(1), dim3(kScanThreads), s, p);
  if (items <= size_t(kOneClusterCells)) return launch_pdl(kv_compact_kernel<kCluster, true>, dim3(kCluster), dim3(kScanThreads), s, p);
  const cudaError_t e = launch_pdl(kv_compact_kernel<kCluster, false>, dim3(kCluster), dim3(kScanThreads), s, p);
  if (e != cudaSuccess) return e;
  size_t grid = (items + kRemapThreads - 1) / kRemapThreads;
  const size_t most = size_t(sm_count()) * 8;
  if (grid > most) grid = most;
  return launch_pdl(kv_remap_kernel, dim3(unsigned(grid)), dim3(kRemapThreads), s, p);
}

cudaError_t launch_kv_copy(const KvCopyParams &p, cudaStream_t s) {
  const size_t units = size_t(p.n) * p.n_layers * ((p.page_bytes + kCopyUnit - 1) / kCopyUnit);
  size_t grid = size_t(sm_count()) * 8;
  if (grid > units) grid = units;
  return launch_pdl(kv_copy_kernel, dim3(unsigned(grid)), dim3(kCopyThreads), s, p);
}

}  // namespace gdn

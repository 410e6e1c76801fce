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
//
// Shared pages (refs): a page given back loses a holder, and goes onto the stack when
// it has none left, at the place of the last of the cycle's releases of it.  Three
// passes over the releases in their order: the counts go down; where a count has
// reached zero, the releases of that page leave their least negative mark there, which
// is the last one's; the release that finds its own mark pushes the page.  Each pass
// is a few dependent trips to L2 a release, so where there may be many, a cluster of
// kPlanCluster CTAs shares them, and up to four of a thread stay in its registers from
// pass to pass: 24,400 releases of 122 rows take 66.8 us in one CTA, 20.2 in eight that look
// each up in every pass, 15.1 so.
//
// Whether a row writes into a shared page is two dependent reads a row more, 0.3 us of a plan's 5.
#include <cooperative_groups.h>

#include "kv4.cuh"
#include "scan.cuh"

namespace gdn {

namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = kScanThreads;
constexpr int kPlanCluster = 8, kBatch = 4;
// Cells of the table from which on shared releases go to a cluster.  One CTA keeps 4096 releases in registers:
// 4000 take 10.7 us there, 12.0 in the cluster; 4800 17.3 and 12.1; 16000 41.5 and 13.3.  A plan without releases
// takes 4.7 and 5.1.
constexpr long long kPlanCells = 4096;
// Tokens up to which the bookkeeping CTA writes the slots itself; a kernel of their own
// behind it costs 16 tokens 5.8 us for 4.7, and 2048 5.6 for 5.3, but 8192 take 5.5 for
// 7.3 and 65536 5.6 for 26.5.
constexpr int kPlanOneCta = 2048;

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

// Whether the row's first new token would stand in a page that another row holds too.  Where it
// does not, no later one does: rows share beginnings, and give pages back from their ends.
__device__ __forceinline__ bool writes_shared(const KvPlanParams &p, int b, const PlanRow &r) {
  const int c = r.len >> p.log2P;
  if (r.a == 0 || c >= r.held) return false;
  const int page = p.table[size_t(b) * p.max_pages + c];
  return page >= 0 && page < p.n_pages && __ldcg(p.refs + page) > 1;
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

// The releases of a chunk's rows: `total` of them, cell by cell.
struct PlanChunk {
  const int *ends, *from;  // releases up to each row of the chunk; its first column that goes
  int b0, rows;

  __device__ __forceinline__ int32_t *cell(const KvPlanParams &p, int i) const {
    const int w = find_row(ends, rows, i);
    return p.table + size_t(b0 + w) * p.max_pages + from[w] + i - (w ? ends[w - 1] : 0);
  }
};

// Pages given back where rows share them; how many went onto the stack.
template <int C>
__device__ __forceinline__ long long release_shared(const KvPlanParams &p, int count0, int *s_ends, int *s_from, long long *s_warp, int *s_pushed) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = C > 1 ? int(cluster.block_rank()) : 0, tid = threadIdx.x, n_pages = p.n_pages;
  auto together = [&] {
    __syncwarp();  // a warp that a loop has split would arrive more than once
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  long long released = 0, total = 0;
  // kBatch releases of a thread at a time, so that their trips to memory overlap; where that is
  // all, they stay from pass to pass
  int32_t *cell[kBatch];
  int page[kBatch];  // -1: none, or outside the cache
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    long long index0 = 0;  // releases of the rows before the chunk
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
      const int rows = min(kPlanThreads, p.B - b0);
      if (pass == 0 || p.B > kPlanThreads) {  // one chunk stays as it is
        const int b = b0 + tid;
        PlanRow r{};
        if (b < p.B) r = plan_row(p, b);
        if (pass == 0 && rank == 0 && b < p.B && r.bad) atomicOr(p.status, GDN_STATUS_BAD_LEN);
        const long long end = block_scan(max(r.held - r.want, 0), s_warp, &total);
        s_ends[tid] = int(end), s_from[tid] = r.want;
        sync_cta();
      }
      if (total == 0) continue;  // the same for every thread of the cluster
      const PlanChunk chunk{s_ends, s_from, b0, rows};
      const int lo = int(total * rank / C), hi = int(total * (rank + 1) / C);
      const bool again = pass > 0 && p.B <= kPlanThreads && total <= C * kBatch * kPlanThreads;
      auto gather = [&](int i0) {
        if (again) return;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * kPlanThreads + tid;
          cell[k] = i < hi ? chunk.cell(p, i) : nullptr;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) page[k] = cell[k] ? *cell[k] : -1;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (page[k] >= n_pages) page[k] = -1;
      };
      auto mark = [&](int i0, int k) { return -1 - int(index0 + i0 + k * kPlanThreads + tid); };
      auto counts = [&](int(&c)[kBatch]) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) c[k] = page[k] >= 0 ? *(volatile int32_t *)(p.refs + page[k]) : 1;
      };
      if (pass < 2) {
        for (int i0 = lo; i0 < hi; i0 += kBatch * kPlanThreads) {
          int c[kBatch];
          gather(i0);
          if (pass == 1) {
            counts(c);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
              if (c[k] <= 0) atomicMin(p.refs + page[k], mark(i0, k));
          } else {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) c[k] = page[k] >= 0 ? atomicSub(p.refs + page[k], 1) : 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
              if (cell[k] && c[k] <= 0) {  // no page, or nobody held it: not given back
                if (page[k] >= 0) atomicAdd(p.refs + page[k], 1);
                *cell[k] = -1, page[k] = -1;
                atomicOr(p.status, GDN_STATUS_BAD_INDEX);
              }
          }
        }
      } else {
        long long before = 0;
        if (C > 1) {  // pushed by the CTAs before this one
          int mine = 0;
          for (int i0 = lo; i0 < hi; i0 += kBatch * kPlanThreads) {
            int c[kBatch];
            gather(i0);
            counts(c);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              __syncwarp();
              mine += __syncthreads_count(page[k] >= 0 && c[k] == mark(i0, k));
            }
          }
          if (tid < C) cluster.map_shared_rank(s_pushed, tid)[rank] = mine;
          together();
          for (int q = 0; q < rank; ++q) before += s_pushed[q];
        }
        for (int i0 = lo; i0 < hi; i0 += kBatch * kPlanThreads) {
          int c[kBatch];
          gather(i0);
          counts(c);
          static_assert(kBatch * 16 <= 64 && kPlanThreads < (1 << 15), "a batch's counts in 16 bits each");
          long long pushes = 0, pushed;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) pushes |= (long long)(page[k] >= 0 && c[k] == mark(i0, k)) << (16 * k);
          const long long upto = block_scan(pushes, s_warp, &pushed);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (pushes >> (16 * k) & 1) {
              const long long place = count0 + released + before + (upto >> (16 * k) & 0xffff) - 1;
              if (place < n_pages) p.free_list[place] = page[k];
              else atomicOr(p.status, GDN_STATUS_BAD_INDEX);
              p.refs[page[k]] = 0;
            }
            if (cell[k]) *cell[k] = -1;
            before += pushed >> (16 * k) & 0xffff;
          }
        }
        if (C > 1) {
          for (int q = 0; q < C; ++q) released += s_pushed[q];
          together();  // everybody has read them
        } else {
          released += before;
        }
      }
      index0 += total;
    }
    if (index0 == 0) break;  // the same for every thread of the cluster
    together();
  }
  return released;
}

template <bool SHARED, int C>
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanParams p, const int write_slots) {
  __shared__ long long s_warp[32];
  __shared__ int s_ends[kPlanThreads];   // pages that the chunk's rows move, summed up to each row
  __shared__ int s_from[kPlanThreads];   // first table column that the row moves
  __shared__ int s_pushed[C];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int n_pages = p.n_pages;
  const int count0 = min(max(*p.free_count, 0), n_pages);

  // ---- pages given back --------------------------------------------------------
  long long released = 0;
  if (SHARED) {
    released = release_shared<C>(p, count0, s_ends, s_from, s_warp, s_pushed);
    if (C > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      __syncwarp();
      cluster.sync();  // the rows are read, the pushed pages visible
      if (cluster.block_rank() != 0) return;
    }
  } else {
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
      sync_cta();
      const PlanChunk chunk{s_ends, s_from, b0, rows};
      for (int i = tid; i < int(total); i += kPlanThreads) {
        int32_t *cell = chunk.cell(p, i);
        const long long at = count0 + released + i;
        if (at < n_pages) p.free_list[at] = *cell;
        else atomicOr(p.status, GDN_STATUS_BAD_INDEX);
        *cell = -1;
      }
      released += total;
    }
  }
  const long long avail = min((long long)n_pages, count0 + released);
  sync_cta();  // the pushed pages are visible to the whole CTA

  // ---- pages taken, in row order -----------------------------------------------
  long long taken0 = 0, tokens0 = 0, granted = 0, got_sum = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid, rows = min(kPlanThreads, p.B - b0);
    PlanRow r{};
    if (b < p.B) r = plan_row(p, b);
    if (SHARED && b < p.B && writes_shared(p, b, r)) {
      r.a = 0, r.want = min(r.want, r.held);
      atomicOr(p.status, GDN_STATUS_BAD_LEN);
    }
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
    sync_cta();
    for (int i = tid; i < int(got_total); i += kPlanThreads) {
      const int w = find_row(s_ends, rows, i);
      const long long from = avail - 1 - (taken0 + i);
      int page = SHARED ? __ldcg(p.free_list + from) : p.free_list[from];
      if (SHARED) {
        if (page >= 0 && page < n_pages) p.refs[page] = 1;
        else page = -1, atomicOr(p.status, GDN_STATUS_BAD_INDEX);
      }
      p.table[size_t(b0 + w) * p.max_pages + s_from[w] + i - (w ? s_ends[w - 1] : 0)] = page;
    }
    taken0 += need_total;
    tokens0 += tok_total;
    granted += a_total;
    got_sum += got_total;
    sync_cta();  // s_ends is free for the next chunk, and the rows' results are visible
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
  const int C = p.refs && (long long)p.B * p.max_pages >= kPlanCells ? kPlanCluster : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  const void *kernel = C > 1 ? reinterpret_cast<const void *>(kv_plan_kernel<true, kPlanCluster>)
                             : p.refs ? reinterpret_cast<const void *>(kv_plan_kernel<true, 1>) : reinterpret_cast<const void *>(kv_plan_kernel<false, 1>);
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess || one) return e;
  return launch_pdl(kv_slots_kernel, dim3((p.N + 255) / 256), dim3(256), s, p);
}

}  // namespace gdn

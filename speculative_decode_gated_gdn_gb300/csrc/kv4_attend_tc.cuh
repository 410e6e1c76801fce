// kv4_attend_tc.cuh -- causal attention of many query rows over the paged
// 4-bit cache on the tcgen05 tensor cores.
//
// A unit is (row b, kv head, tile of TT = floor(128 / G) whole tokens): up to
// 128 query rows share every key that is formed.  Per tile of NK keys:
//   dequant  4 warps form K [NK][D] and V^T [D][NK] in fp16 (each value rounded
//            once) in shared memory, K-major with the 128-byte swizzle;
//   scores   S = Q K^T, Q in tensor memory as the A operand;
//   softmax  4 warps, a thread a row: running maximum and sum in fp32; P goes
//            back to tensor memory in fp16 over S;
//   output   O += P V, P from tensor memory; O is rescaled only when a
//            probability passes 2^14.
// The channel order inside 8 channels is 0 4 1 5 2 6 3 7 in Q and K alike (a
// product does not see it): the order in which masks take codes out of a word.
//
// What bounds it: the tensor cores where rows are many (4 * 128 * NK * D
// operations a tile), the dequant's instructions where a tile's rows are few.
// With Q and P in tensor memory the products read only K and V from shared
// memory, so that a 64-key tile still feeds them at D = 256, where O takes half
// of the tensor memory.
//
// Units are laid on one line in tiles of keys and cut evenly over a persistent
// grid as in kv4_attend.cuh; causal tiles count as far as their last query sees.
#pragma once

#include "kv4_attend.cuh"

namespace gdn {

constexpr int kTcRows = 128;
constexpr int kTcThreads = 288;  // warps 0-3 softmax, 4-7 dequant, 8 products

template <int D>
struct TcShape {
  static constexpr int W = D / 64;
  static constexpr int NK = D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int kKBytes = NK * D * 2;      // K or V of a tile
  static constexpr int kSmem = 4 * kKBytes + 1024;
  // tensor memory columns: O [D], S two buffers [NK], Q [D / 2], P [NK / 2].
  // At D = 256 there is no room for P of its own: it lies over its S.
  static constexpr bool kOver = D == 256;
  static constexpr int kColS = D, kColQ = D + 2 * NK, kColP = kOver ? kColS : kColQ + D / 2;
  static constexpr int kCols = 512;
  static_assert(kColQ + D / 2 + (kOver ? 0 : NK / 2) <= kCols, "tensor memory");
  static __device__ __forceinline__ uint32_t col_p(uint32_t buf) { return kColP + (kOver ? buf * NK : 0); }
};

template <int D>
__host__ __device__ constexpr size_t tc_part_floats() { return size_t(kTcRows) * (D + 2); }

__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B^T for one K step of 16 fp16 elements; one thread.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}

// Loads of 32 columns without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// One row's part of the line.
struct TcRow {
  int start, span, count, len, tiles;
};

__device__ __forceinline__ TcRow tc_row(const Kv4AttendParams &p, int b, int TT, bool report) {
  TcRow r;
  r.start = p.q_start[b];
  int span = p.q_start[b + 1] - r.start;
  const int len = p.kv_len[b], cap = p.g.max_pages << p.g.log2P;
  int count = p.q_count[b];
  const bool bad = span < 0 || span > p.max_q || count < 0 || count > span || len < 0 || len > cap || r.start < 0 ||
                   r.start > p.N - max(span, 0);
  if (bad) {
    if (report) atomicOr(p.status, GDN_STATUS_BAD_LEN);
    r.start = min(max(r.start, 0), p.N);
    span = min(max(span, 0), min(p.max_q, p.N - r.start));
    count = min(max(count, 0), span);
  }
  r.span = span, r.count = count, r.len = min(max(len, 0), cap);
  r.tiles = (span + TT - 1) / TT;
  return r;
}

// Keys that the last query of tile t sees, and its tiles of keys (1 at least:
// a unit without keys still writes its zeros).
__device__ __forceinline__ int tc_limit(const TcRow &r, int t, int TT) {
  return r.count > t * TT ? max(0, r.len - r.count + min((t + 1) * TT, r.count)) : 0;
}
template <int NK>
__device__ __forceinline__ int tc_stages(const TcRow &r, int t, int TT) {
  return max(1, (tc_limit(r, t, TT) + NK - 1) / NK);
}

// sum over i < n of floor((a i + b) / m), a, b >= 0 (the Euclid-like descent of
// lattice points under a line).
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    s += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m, b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m, b = y % m;
    const long long t = m;
    m = a, a = t;
  }
  return s;
}

// Tiles of keys of all query tiles of a row (one head).
template <int NK>
__device__ inline long long tc_row_stages(const TcRow &r, int TT) {
  if (r.tiles <= 8) {
    long long s = 0;
    for (int t = 0; t < r.tiles; ++t) s += tc_stages<NK>(r, t, TT);
    return s;
  }
  const int live = (r.count + TT - 1) / TT;  // tiles with a query
  long long s = r.tiles - live;
  int first = 0;  // tiles whose queries see no key count as one
  const int base = r.len - r.count;
  while (first < live && base + min((first + 1) * TT, r.count) <= 0) {
    // jump: base + (t + 1) TT > 0
    const int t = min(live, max(first + 1, -base / TT));
    s += t - first;
    first = t;
  }
  if (first < live) {
    // full tiles first .. live - 2: ceil((base + (t + 1) TT) / NK), and the last
    const int n = live - 1 - first;
    if (n > 0) s += floor_sum(n, NK, TT, (long long)base + (long long)(first + 1) * TT + NK - 1);
    s += tc_stages<NK>(r, live - 1, TT);
  }
  return s;
}

// A thread's walk over its CTA's piece of the line.
template <int D>
struct TcWalk {
  static constexpr int NK = TcShape<D>::NK;
  const Kv4AttendParams &p;
  int TT;
  long long at, stop, unit_first;
  int b, hk, tile, st0, st1, stages;
  TcRow row;
  __device__ TcWalk(const Kv4AttendParams &q, int tt, long long at_, long long stop_, int b_, int hk_, int tile_, int st_)
      : p(q), TT(tt), at(at_), stop(stop_), b(b_), hk(hk_), tile(tile_), st0(st_), st1(0) {
    row = tc_row(p, b, TT, false);
    open();
  }
  __device__ void open() {
    stages = tc_stages<NK>(row, tile, TT);
    unit_first = at - st0;
    st1 = int(min((long long)stages, st0 + (stop - at)));
  }
  __device__ bool done() const { return at >= stop; }
  __device__ void next() {
    at += st1 - st0;
    if (at >= stop) return;
    st0 = 0;
    if (++tile == row.tiles) {
      tile = 0;
      if (++hk == p.g.H_kv) {
        hk = 0;
        do row = tc_row(p, ++b, TT, false);
        while (row.tiles == 0);
      }
    }
    open();
  }
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) kv4_attend_tc(const __grid_constant__ Kv4AttendParams p) {
  using S = TcShape<D>;
  constexpr int W = S::W, NK = S::NK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done, q_full, joined, drained;
  __shared__ uint32_t s_tmem;
  __shared__ long long s_warp[kTcThreads / 32];
  __shared__ long long s_place[5];
  __shared__ int s_flag, s_dead;
  __shared__ uint32_t s_bad[2][NK / 32][W];  // keys of a V tile with a value that is not finite, per group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int G = p.g.H_q / p.g.H_kv, Hkv = p.g.H_kv, TT = kTcRows / G;
  const int P = 1 << p.g.log2P;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128), mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1), mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 128);
    }
    mbar_init(&pv_done, 1), mbar_init(&q_full, 128), mbar_init(&joined, 128), mbar_init(&drained, 1);
    s_dead = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * (NK / 32) * W; i += kTcThreads) (&s_bad[0][0][0])[i] = 0;
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's piece of the line --------------------------------------------------
  auto block_sum = [&](long long v) -> long long {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    long long t = 0;
    for (int i = 0; i < kTcThreads / 32; ++i) t += s_warp[i];
    return t;
  };
  // exclusive prefix of v over the CTA
  auto block_before = [&](long long v) -> long long {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long t = x - v;
    for (int i = 0; i < warp; ++i) t += s_warp[i];
    return t;
  };
  long long mine = 0;
  for (int b = tid; b < p.g.B; b += kTcThreads) mine += tc_row_stages<NK>(tc_row(p, b, TT, blockIdx.x == 0), TT);
  const long long total = block_sum(mine) * Hkv;
  const long long ctas = min((long long)gridDim.x, total);
  const long long c = blockIdx.x;
  if (c >= ctas) return;
  const long long at = total * c / ctas, stop = total * (c + 1) / ctas;
  {
    long long before0 = 0;
    for (int b0 = 0; b0 < p.g.B; b0 += kTcThreads) {
      const long long v = b0 + tid < p.g.B ? tc_row_stages<NK>(tc_row(p, b0 + tid, TT, false), TT) * Hkv : 0;
      const long long before = before0 + block_before(v);
      if (tid == 0) s_place[0] = -1;
      __syncthreads();
      if (at >= before && at < before + v) s_place[0] = b0 + tid, s_place[1] = before;
      before0 += block_sum(v);
      if (s_place[0] >= 0) break;
    }
    const int b = int(s_place[0]);
    const TcRow row = tc_row(p, b, TT, false);
    const long long head = tc_row_stages<NK>(row, TT), in_row = at - s_place[1];
    const int hk = int(in_row / head);
    const long long x = in_row - hk * head;
    before0 = 0;
    for (int t0 = 0; t0 < row.tiles; t0 += kTcThreads) {
      const long long v = t0 + tid < row.tiles ? tc_stages<NK>(row, t0 + tid, TT) : 0;
      const long long before = before0 + block_before(v);
      __syncthreads();
      if (tid == 0) s_place[2] = -1;
      __syncthreads();
      if (x >= before && x < before + v) s_place[2] = t0 + tid, s_place[3] = x - before;
      before0 += block_sum(v);
      if (s_place[2] >= 0) break;
    }
    s_place[4] = hk;  // the same value from every thread
  }
  __syncthreads();
  TcWalk<D> walk(p, TT, at, stop, int(s_place[0]), int(s_place[4]), int(s_place[2]), int(s_place[3]));

  if (warp == 8) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *dead = &s_dead;
  // a bounded wait; false (for good) once any wait of the CTA has run out
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (*dead) return false;
    if (mbar_wait_spin(bar, parity, kWaitLimit)) return true;
    *dead = 1;
    atomicOr(p.status, GDN_STATUS_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (warp == 8) {
    // ---- products ---------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t idesc_s = umma_idesc_f16(kTcRows, NK), idesc_o = umma_idesc_f16(kTcRows, D);
      const uint32_t sb = smem_u32(smem);
      uint32_t it = 0, unit = 0;
      bool ok = true;
      auto scores = [&](uint32_t i) {
        const uint32_t buf = i & 1, ph = (i >> 1) & 1;
        ok = ok && wait(&k_full[buf], ph);
        if (!ok) return;
        tc_fence_after();
        const uint32_t kb = sb + buf * S::kKBytes;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_f16_ts(tmem + S::kColS + buf * NK, tmem + S::kColQ + ks * 8,
                      umma_desc_sw128(kb + (ks >> 2) * (NK * 128) + (ks & 3) * 32), idesc_s, ks > 0);
        umma_commit(&k_empty[buf]);
        umma_commit(&s_full[buf]);
      };
      for (; ok && !walk.done(); walk.next(), ++unit) {
        ok = wait(&q_full, unit & 1);
        tc_fence_after();
        const int n = walk.st1 - walk.st0;
        if (ok) scores(it);
        for (int i = 0; ok && i < n; ++i, ++it) {
          // the next tile's scores run while this tile's softmax does.  Their
          // buffer's scores were read before the last product was let go; a P
          // lying over them is used up only when that product is done
          if (i + 1 < n) {
            if (S::kOver && i > 0) ok = ok && wait(&pv_done, (it - 1) & 1);
            scores(it + 1);
          }
          const uint32_t buf = it & 1, ph = (it >> 1) & 1;
          ok = ok && wait(&v_full[buf], ph) && wait(&p_full[buf], ph);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vb = sb + 2 * S::kKBytes + buf * S::kKBytes;
#pragma unroll
          for (int ks = 0; ks < NK / 16; ++ks)
            umma_f16_ts(tmem, tmem + S::col_p(buf) + ks * 8, umma_desc_sw128(vb + (ks >> 2) * (D * 128) + (ks & 3) * 32),
                        idesc_o, i > 0 || ks > 0);
          umma_commit(&v_empty[buf]);
          umma_commit(&pv_done);
        }
      }
      if (!ok) {  // a wait ran out: the products in flight end before the CTA does
        umma_commit(&drained);
        mbar_wait_spin(&drained, 0, kWaitLimit);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---- dequant -------------------------------------------------------------------------
    const int dw = warp - 4;
    constexpr int KC = NK * D / 32 / 128;      // 16-byte chunks of K codes a thread
    constexpr int CB = D == 64 ? 1 : 2;        // words of V codes a thread and key
    constexpr int kChunks = D / 32;            // chunks of a key
    // K: row r = 8 * group + lane % 8, chunk; V: 8 keys, CB words
    uint32_t it = 0, had0[CB], had1[CB];  // what the thread noted in each buffer
#pragma unroll
    for (int x = 0; x < CB; ++x) had0[x] = had1[x] = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next()) {
      const int32_t *table = p.table + size_t(walk.b) * p.g.max_pages;
      const int lim = tc_limit(walk.row, walk.tile, TT);
      const size_t rec_bytes = kv4_record_bytes(D, P);
      const uint8_t *heads = p.pages + size_t(walk.hk) * rec_bytes;
      const size_t page_bytes = size_t(Hkv) * rec_bytes;
      // lane l holds the page of keys [16 l, 16 l + 16) of a tile
      auto pages_of = [&](int st) -> int {
        const int t = st * NK + 16 * lane;
        int pg = -1;
        if (lane < NK / 16 && st < walk.st1 && t < lim) {
          pg = table[t >> p.g.log2P];
          if (pg < 0 || pg >= p.g.n_pages) {
            pg = -1;
            atomicOr(p.status, GDN_STATUS_BAD_INDEX);
          }
        }
        return pg;
      };
      uint4 kr[KC];
      uint32_t ke[KC][W];
      uint32_t vr[8][CB], ve[8][CB];
      const int vkey = (dw & (NK / 64 - 1)) * 64 + (lane & 7) * 8;                       // first of the thread's 8 keys
      const int vword = ((dw / (NK / 64)) * 4 + (lane >> 3)) * CB;                       // first of its words
      auto load = [&](int st, int pg) {
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const int idx = (i * 4 + dw) * 4 + (lane >> 3);  // (8-row group, chunk)
          const int r = (idx / kChunks) * 8 + (lane & 7), chunk = idx % kChunks;
          const int page = __shfl_sync(0xffffffffu, pg, r >> 4);
          const int t = st * NK + r, off = t & (P - 1);
          kr[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int g = 0; g < W; ++g) ke[i][g] = 0;
          if (page >= 0 && t < lim) {
            const uint8_t *rec = heads + size_t(page) * page_bytes;
            kr[i] = __ldg(reinterpret_cast<const uint4 *>(rec + off * (D / 2) + chunk * 16));
            const uint8_t *e = rec + 2 * kv4_code_bytes(D, P) + off * (4 * W);
            if (W == 4) {
              const uint4 x = __ldg(reinterpret_cast<const uint4 *>(e));
              ke[i][0] = x.x, ke[i][1 % W] = x.y, ke[i][2 % W] = x.z, ke[i][3 % W] = x.w;
            } else if (W == 2) {
              const uint2 x = __ldg(reinterpret_cast<const uint2 *>(e));
              ke[i][0] = x.x, ke[i][1 % W] = x.y;
            } else {
              ke[i][0] = __ldg(reinterpret_cast<const uint32_t *>(e));
            }
          }
        }
        const int page = __shfl_sync(0xffffffffu, pg, vkey >> 4);
        const uint8_t *rec = heads + size_t(page < 0 ? 0 : page) * page_bytes;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int t = st * NK + vkey + k, off = t & (P - 1);
#pragma unroll
          for (int x = 0; x < CB; ++x) vr[k][x] = ve[k][x] = 0;
          if (page >= 0 && t < lim) {
            const uint8_t *cp = rec + kv4_code_bytes(D, P) + off * (D / 2) + vword * 4;
            const uint8_t *e = rec + 2 * kv4_code_bytes(D, P) + kv4_entry_bytes(D, P) + (off * W + vword % W) * 4;
            if (CB == 2) {
              const uint2 a = __ldg(reinterpret_cast<const uint2 *>(cp));
              const uint2 d = __ldg(reinterpret_cast<const uint2 *>(e));
              vr[k][0] = a.x, vr[k][CB - 1] = a.y, ve[k][0] = d.x, ve[k][CB - 1] = d.y;
            } else {
              vr[k][0] = __ldg(reinterpret_cast<const uint32_t *>(cp)), ve[k][0] = __ldg(reinterpret_cast<const uint32_t *>(e));
            }
          }
        }
      };
      __syncwarp();
      load(walk.st0, pages_of(walk.st0));
      int pg_next = pages_of(walk.st0 + 1);
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t buf = it & 1, ph = (it >> 1) & 1;
        // ---- K: the thread's 16-byte chunks as 4 rows of 16 bytes
        ok = wait_warp(&k_empty[buf], ph ^ 1);
        uint8_t *kb = smem + buf * S::kKBytes;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const int idx = (i * 4 + dw) * 4 + (lane >> 3);
          const int r = (idx / kChunks) * 8 + (lane & 7), chunk = idx % kChunks;
          const uint32_t wd[4] = {kr[i].x, kr[i].y, kr[i].z, kr[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t e = ke[i][q % W];
            const uint32_t step = __byte_perm(e, e, 0x1010), base = __byte_perm(e, e, 0x3232);
            const uint32_t x = wd[q], y = x >> 8;
            const uint4 o = make_uint4(att_even(x, step, base), att_odd(x, step, base), att_even(y, step, base), att_odd(y, step, base));
            const int u = chunk * 4 + q;  // 8-channel unit of the key
            *reinterpret_cast<uint4 *>(kb + (u >> 3) * (NK * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = o;
          }
        }
        fence_proxy_async_shared();
        mbar_arrive(&k_full[buf]);
        // ---- V^T: the thread's 8 keys as 16 bytes of each channel's row
        ok = ok && wait_warp(&v_empty[buf], ph ^ 1);
        uint8_t *vb = smem + 2 * S::kKBytes + buf * S::kKBytes;
        // values that are not finite are left out here and put back by the rows
        // that see their key: one thread notes each (key, group)
#pragma unroll
        for (int x = 0; x < CB; ++x) {
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (att_not_finite(ve[k][x])) bad |= 1u << k, ve[k][x] = 0;
          if (vword + x < W) {
            uint32_t &had = buf ? had1[x] : had0[x];
            if (had | bad) {
              uint32_t *flag = &s_bad[buf][vkey >> 5][(vword + x) % W];
              atomicAnd(flag, ~(0xffu << (vkey & 31)));
              if (bad) atomicOr(flag, bad << (vkey & 31));
            }
            had = bad;
          }
        }
#pragma unroll
        for (int x = 0; x < CB; ++x) {
          uint32_t es[4], eb[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            es[k] = __byte_perm(ve[2 * k][x], ve[2 * k + 1][x], 0x5410);
            eb[k] = __byte_perm(ve[2 * k][x], ve[2 * k + 1][x], 0x7632);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) lo[k] = __byte_perm(vr[2 * k][x], vr[2 * k + 1][x], half ? 0x7632 : 0x5410);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t y = e >= 2 ? lo[k] >> 8 : lo[k];
                o[k] = e & 1 ? att_odd(y, es[k], eb[k]) : att_even(y, es[k], eb[k]);
              }
              const int ch = (vword + x) * 8 + half * 4 + e;
              *reinterpret_cast<uint4 *>(vb + (vkey >> 6) * (D * 128) + ch * 128 + ((((vkey & 63) >> 3) ^ (ch & 7)) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_shared();
        mbar_arrive(&v_full[buf]);
        if (st + 1 < walk.st1) {
          load(st + 1, pg_next);
          pg_next = pages_of(st + 2);
        }
      }
    }
  } else {
    // ---- softmax: thread = query row ----------------------------------------------------------
    const uint32_t lane_base = tmem + (uint32_t(warp * 32) << 16);
    float *parts = reinterpret_cast<float *>(static_cast<char *>(p.ws) + 4096);
    uint32_t *counters = reinterpret_cast<uint32_t *>(p.ws);
    uint32_t it = 0, joins = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next()) {
      const TcRow &row = walk.row;
      const int r = tid, i = walk.tile * TT + r / G, head = walk.hk * G + r % G;
      const bool in = r < TT * G && i < row.span, live = in && i < row.count;
      const int tok = row.start + i;
      const int tile_lim = tc_limit(row, walk.tile, TT);
      const int lim = live ? max(0, row.len - row.count + i + 1) : in ? 0 : tile_lim;
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      // ---- Q: scaled by a power of two to [2^10, 2^11), fp16, into tensor memory
      float f;
      {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t(live ? tok : 0) * p.g.H_q + (live ? head : 0)) * D);
        uint32_t mx = 0;
#pragma unroll 4
        for (int u = 0; u < D / 8; ++u) {
          const uint4 x = live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        const int e = min(max(int(mx >> 7), 20), 240);
        const float up = __uint_as_float(uint32_t(264 - e) << 23);
        f = (1.f / up) * (p.scale * 1.4426950408889634f);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 x = live ? __ldg(src + 4 * u + k) : make_uint4(0, 0, 0, 0);
            const uint32_t a[4] = {x.x, x.y, x.z, x.w};
            float y[8];
#pragma unroll
            for (int h = 0; h < 4; ++h)
              y[2 * h] = __uint_as_float(a[h] << 16) * up, y[2 * h + 1] = __uint_as_float(a[h] & 0xffff0000u) * up;
#pragma unroll
            for (int h = 0; h < 4; ++h) w[4 * k + h] = pack_h2(y[h], y[h + 4]);
          }
          tmem_st16_async(lane_base + S::kColQ + 16 * u, w);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&q_full);
      }
      float m = -INFINITY, l = 0.f;
      uint32_t nan = 0;
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t buf = it & 1, ph = (it >> 1) & 1;
        ok = wait_warp(&s_full[buf], ph);
        if (!ok) break;
        tc_fence_after();
        uint32_t raw[NK / 32][32];
#pragma unroll
        for (int q = 0; q < NK / 32; ++q) tmem_ld32_async(lane_base + S::kColS + buf * NK + 32 * q, raw[q]);
        tmem_wait_ld();
        float x = -INFINITY;
        const int t0 = st * NK;
        if (t0 + NK > lim_min) {
#pragma unroll
          for (int q = 0; q < NK / 32; ++q)
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float s = t0 + 32 * q + k < lim ? __uint_as_float(raw[q][k]) * f : -INFINITY;
              raw[q][k] = __float_as_uint(s);
              x = fmaxf(x, s);
            }
        } else {
#pragma unroll
          for (int q = 0; q < NK / 32; ++q)
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float s = __uint_as_float(raw[q][k]) * f;
              raw[q][k] = __float_as_uint(s);
              x = fmaxf(x, s);
            }
        }
        float a = 1.f;
        const bool move = x > m + 14.f;
        if (move) {
          const float n = fmaxf(m, x - 6.f);
          a = m == -INFINITY ? 0.f : ex2(m - n);
          m = n;
          l *= a;
        }
        if (__any_sync(0xffffffffu, move) && st > walk.st0) {
          // the product that is still adding to O has to be done first
          ok = wait_warp(&pv_done, (it - 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32_async(lane_base + 32 * q, o);
            tmem_wait_ld();
            float y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * a;
            tmem_st32_async(lane_base + 32 * q, y);
          }
          tmem_wait_st();
        }
        const float r0 = m == -INFINITY ? 0.f : m;
        uint32_t w[NK / 32][16];
#pragma unroll
        for (int q = 0; q < NK / 32; ++q)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float pa = ex2(__uint_as_float(raw[q][2 * k]) - r0), pb = ex2(__uint_as_float(raw[q][2 * k + 1]) - r0);
            l += pa + pb;
            w[q][k] = pack_h2(pa, pb);
          }
        if (!S::kOver && st > walk.st0) {  // the last product has read its P
          ok = wait_warp(&pv_done, (it - 1) & 1);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int q = 0; q < NK / 32; ++q) tmem_st16_async(lane_base + S::col_p(buf) + 16 * q, w[q]);
        tmem_wait_st();
        tc_fence_before();
        // values that are not finite reach the rows that see their key
        ok = wait_warp(&v_full[buf], ph);
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < NK / 32; ++q)
#pragma unroll
          for (int g = 0; g < W; ++g) {
            const uint32_t bad = *reinterpret_cast<volatile uint32_t *>(&s_bad[buf][q][g]);
            if (bad) {
              const int n = lim - t0 - 32 * q;
              if (n > 0 && (bad & (n >= 32 ? 0xffffffffu : (1u << n) - 1))) nan |= 1u << g;
            }
          }
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // ---- the unit's rows, or a part of them ------------------------------------------
      ok = wait_warp(&pv_done, (it - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const bool whole = walk.st0 == 0 && walk.st1 == walk.stages;
      bool last = whole;
      long long c_first = 0, c_last = 0;
      if (!whole) {
        c_first = ((walk.unit_first + 1) * ctas - 1) / total;
        c_last = ((walk.unit_first + walk.stages) * ctas - 1) / total;
        float *part = parts + (size_t(c) * 2 + (c == c_first ? 1 : 0)) * tc_part_floats<D>();
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32_async(lane_base + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int g = ((32 * q + k) / 8) % W;
            part[size_t(32 * q + k) * kTcRows + r] = nan >> g & 1 ? __uint_as_float(0x7fc00000u) : __uint_as_float(o[k]);
          }
        }
        part[size_t(D) * kTcRows + r] = m, part[size_t(D + 1) * kTcRows + r] = l;
        __threadfence();
        mbar_arrive(&joined);
        ok = wait_warp(&joined, joins++ & 1);
        if (!ok) break;
        if (tid == 0) {
          const uint32_t need = uint32_t(c_last - c_first + 1);
          const uint32_t done = atomicAdd(&counters[c_first], 1u) + 1u;
          s_flag = done == need;
          if (done == need) counters[c_first] = 0;  // ready for the next call
          __threadfence();
        }
        __syncwarp();
        mbar_arrive(&joined);
        ok = wait_warp(&joined, joins++ & 1);
        if (!ok) break;
        last = *reinterpret_cast<volatile int *>(&s_flag) != 0;
      }
      if (last) {
        float M = m, Ls = l;
        if (!whole) {
          M = -INFINITY, Ls = 0.f;
          for (long long k = c_first; k <= c_last; ++k)
            M = fmaxf(M, __ldcg(parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * tc_part_floats<D>() + size_t(D) * kTcRows + r));
          for (long long k = c_first; k <= c_last; ++k) {
            const float *src = parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * tc_part_floats<D>() + r;
            const float mk = __ldcg(src + size_t(D) * kTcRows), lk = __ldcg(src + size_t(D + 1) * kTcRows);
            Ls = fmaf(lk, lk != lk ? 1.f : mk == -INFINITY ? 0.f : ex2(mk - M), Ls);
          }
        }
        const float v = Ls > 0.f ? 1.f / Ls : Ls;
        uint16_t *dst = p.out + (size_t(tok) * p.g.H_q + head) * D;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float y[32];
          if (whole) {
            uint32_t o[32];
            tmem_ld32_async(lane_base + 32 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              y[k] = nan >> (((32 * q + k) / 8) % W) & 1 ? __uint_as_float(0x7fc00000u) : __uint_as_float(o[k]);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = 0.f;
            for (long long kc = c_first; kc <= c_last; ++kc) {
              const float *src = parts + (size_t(kc) * 2 + (kc == c_first ? 1 : 0)) * tc_part_floats<D>() + r;
              const float mk = __ldcg(src + size_t(D) * kTcRows), lk = __ldcg(src + size_t(D + 1) * kTcRows);
              const float ck = lk != lk ? 1.f : mk == -INFINITY ? 0.f : ex2(mk - M);
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = fmaf(__ldcg(src + size_t(32 * q + k) * kTcRows), ck, y[k]);
            }
          }
          if (in) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[8 * k + 2 * e] * v, y[8 * k + 2 * e + 1] * v);
                w[e] = *reinterpret_cast<const uint32_t *>(&h);
              }
              *reinterpret_cast<uint4 *>(dst + 32 * q + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, S::kCols);
}

template <int D>
inline size_t att_tc_ws(int ctas) {
  return 4096 + sizeof(float) * 2 * size_t(ctas) * tc_part_floats<D>();
}

template <int D>
cudaError_t launch_att_tc(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv4_attend_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_smem(kv4_attend_tc<D>, dim3(ctas), dim3(kTcThreads), TcShape<D>::kSmem, s, p);
}

cudaError_t launch_att_tc_64(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_tc_128(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_tc_256(const Kv4AttendParams &p, int ctas, cudaStream_t s);

}  // namespace gdn

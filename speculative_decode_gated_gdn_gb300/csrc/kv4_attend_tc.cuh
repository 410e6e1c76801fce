// kv4_attend_tc.cuh -- causal attention of many query rows over the paged
// 4-bit cache on the tcgen05 tensor cores.
//
// A unit is (row b, kv head, tile of TT = floor(128 / G) whole tokens): up to
// 128 query rows share every key that is formed.  Per tile of NK keys:
//   copies   one warp brings the tile's codes and entries into a ring of four;
//   dequant  4 warps form K [NK][D] and 4 form V^T [D][NK] in fp16 (each value
//            rounded once) in shared memory, K-major with the 128-byte swizzle;
//   scores   S = Q K^T, Q in tensor memory as the A operand;
//   softmax  4 warps, a thread a row: running maximum and sum in fp32; P goes
//            back to tensor memory in fp16;
//   output   O += P V, P from tensor memory; O is rescaled only when a
//            probability passes 2^14.
// A product does not see the order of its inner dimension, nor O's columns the
// order they are kept in, so both follow what shared memory likes:
//  - inside 8 channels 0 4 1 5 2 6 3 7 (the order masks take codes out of a word);
//  - the words of a key as tc_unit() lays them, so that the threads that read a
//    key side by side store into different banks;
//  - channel 8 w + e of V in row e (D / 8) + w, for the same reason.
// The loops over a tile are kept short in code (a chunk of 32 scores, a word of
// codes at a time): unrolled whole, the roles' code passed what the SM's
// instruction caches hold, and every instruction waited for its fetch (5.5 us a
// tile of 64 keys at D = 256).
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
constexpr int kTcThreads = 448;  // warps 0-3 softmax, 4-7 K, 8-11 V, 12 products, 13 copies
constexpr int kTcRing = 4;       // tiles of codes in flight

template <int D>
struct TcShape {
  static constexpr int W = D / 64;
  static constexpr int NK = D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int kKBytes = NK * D * 2;      // K or V of a tile
  static constexpr int kCodes = NK * D / 2, kEntries = NK * W * 4;
  static constexpr int kRaw = 2 * (kCodes + kEntries);  // a tile as it comes
  static constexpr int kSmem = 4 * kKBytes + kTcRing * kRaw + 1024;
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// As mbar_wait_spin, kept small: the roles wait in many places.
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
  }
  return false;
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

__device__ __forceinline__ void tmem_ld4_async(uint32_t taddr, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_st4_async(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Where the word 4 c + q of a key (channels 8 (4 c + q) ..) stands among its
// 16-byte units: the 8 threads that store at a time hold 4 rows x 2 c (D = 64),
// 2 rows x 4 c or 1 row x 8 c, and the swizzle xors the row into the unit.
template <int D>
__host__ __device__ constexpr int tc_unit(int c, int q) {
  return D == 64 ? 4 * c + q : D == 128 ? (q >> 1) * 8 + 2 * c + (q & 1) : 8 * q + c;
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
  __shared__ uint64_t raw_full[kTcRing], raw_empty[kTcRing];
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done, q_full, joined, drained;
  __shared__ uint32_t s_tmem;
  __shared__ long long s_warp[kTcThreads / 32];
  __shared__ long long s_place[5];
  __shared__ int s_flag, s_dead;
  __shared__ uint32_t s_bad[2][NK / 32][W];  // keys of a V tile with a value that is not finite, per group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ring = smem + 4 * S::kKBytes;
  const int G = p.g.H_q / p.g.H_kv, Hkv = p.g.H_kv, TT = kTcRows / G;
  const int P = 1 << p.g.log2P;
  if (tid == 0) {
    for (int i = 0; i < kTcRing; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 8);
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

  if (warp == 12) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *dead = &s_dead;
  // a bounded wait; false (for good) once any wait of the CTA has run out
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (*dead) return false;
    if (tc_wait(bar, parity)) return true;
    *dead = 1;
    atomicOr(p.status, GDN_STATUS_TIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (warp == 13) {
    // ---- copies -------------------------------------------------------------------------
    const int pt = min(P, NK), n_sub = NK / pt;  // tokens of a copy, pages of a tile
    uint32_t it = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next()) {
      const int lim = tc_limit(walk.row, walk.tile, TT);
      const int32_t *table = p.table + size_t(walk.b) * p.g.max_pages;
      // lane l: piece l % 4 (K, V codes, K, V entries) of page l / 4
      const int piece = lane & 3, sub = lane >> 2;
      auto page_of = [&](int st) -> int {
        const int t = st * NK + sub * pt;
        return sub < n_sub && st < walk.st1 && t < lim ? table[t >> p.g.log2P] : -2;
      };
      int next = page_of(walk.st0);
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t slot = it % kTcRing;
        int page = next;
        next = page_of(st + 1);
        if (page != -2 && (page < 0 || page >= p.g.n_pages)) {
          page = -2;
          atomicOr(p.status, GDN_STATUS_BAD_INDEX);
        }
        ok = wait_warp(&raw_empty[slot], (it / kTcRing & 1) ^ 1);
        if (!ok) break;
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, page >= 0 && piece == 0));
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], pages * 2 * pt * (D / 2 + W * 4));
        __syncwarp();
        if (page >= 0) {
          const int off = (st * NK + sub * pt) & (P - 1);
          const uint8_t *rec = p.pages + (size_t(page) * Hkv + walk.hk) * kv4_record_bytes(D, P);
          const uint8_t *src = rec + (piece & 1) * (piece < 2 ? kv4_code_bytes(D, P) : kv4_entry_bytes(D, P)) +
                               (piece < 2 ? off * (D / 2) : 2 * kv4_code_bytes(D, P) + off * W * 4);
          uint8_t *dst = ring + slot * S::kRaw + (piece & 1) * (piece < 2 ? S::kCodes : S::kEntries) +
                         (piece < 2 ? sub * pt * (D / 2) : 2 * S::kCodes + sub * pt * W * 4);
          bulk_g2s(dst, src, piece < 2 ? pt * D / 2 : pt * W * 4, &raw_full[slot]);
        }
      }
    }
    // nothing is in flight when the CTA ends: every copy is waited for by its
    // readers, or here after a wait that ran out
    if (!ok)
      for (uint32_t k = it < kTcRing ? 0 : it - kTcRing; k < it; ++k)
        tc_wait(&raw_full[k % kTcRing], k / kTcRing & 1);
  } else if (warp == 12) {
    // ---- products -----------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t idesc_s = umma_idesc_f16(kTcRows, NK), idesc_o = umma_idesc_f16(kTcRows, D);
      const uint32_t sb = smem_u32(smem);
      uint32_t base = 0, unit = 0;  // tiles before this unit
      bool ok = true;
      for (; ok && !walk.done(); walk.next(), ++unit) {
        ok = wait(&q_full, unit & 1);
        const int n = walk.st1 - walk.st0;
        // scores of tile i, then the output of tile i - 1: a tile's scores run
        // while the softmax of the one before does
#pragma unroll 1
        for (int i = 0; ok && i <= n; ++i) {
          if (i < n) {
            const uint32_t it = base + i, buf = it & 1;
            // the buffer's scores were read before the product of two tiles ago
            // was let go; a P lying over them is used up only when it is done
            if (S::kOver && i > 1) ok = wait(&pv_done, (it - 2) & 1);
            ok = ok && wait(&k_full[buf], (it >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kb = umma_desc_sw128(sb + buf * S::kKBytes);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_f16_ts(tmem + S::kColS + buf * NK, tmem + S::kColQ + ks * 8,
                          kb + (((ks >> 2) * (NK * 128) + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
            umma_commit(&k_empty[buf]);
            umma_commit(&s_full[buf]);
          }
          if (i > 0) {
            const uint32_t it = base + i - 1, buf = it & 1, ph = (it >> 1) & 1;
            ok = wait(&v_full[buf], ph) && wait(&p_full[buf], ph);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vb = umma_desc_sw128(sb + (2 + buf) * S::kKBytes);
#pragma unroll
            for (int ks = 0; ks < NK / 16; ++ks)
              umma_f16_ts(tmem, tmem + S::col_p(buf) + ks * 8, vb + (((ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4), idesc_o,
                          i > 1 || ks > 0);
            umma_commit(&v_empty[buf]);
            umma_commit(&pv_done);
          }
        }
        base += n;
      }
      if (!ok) {  // a wait ran out: the products in flight end before the CTA does
        umma_commit(&drained);
        tc_wait(&drained, 0);
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- V^T: 8 keys of one word (8 channels) at a time, 16 bytes of 8 rows ------------------
    const int vt = tid - 256;
    constexpr int kWords = D / 8, kTasks = NK / 8 * kWords / 128;
    uint32_t had = 0;  // bit 16 buf + i: the thread noted keys of task i in the buffer
    uint32_t it = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next()) {
      const int lim = tc_limit(walk.row, walk.tile, TT);
#pragma unroll 1
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t buf = it & 1, slot = it % kTcRing;
        ok = wait_warp(&v_empty[buf], ((it >> 1) & 1) ^ 1) && wait_warp(&raw_full[slot], it / kTcRing & 1);
        if (!ok) break;
        const uint8_t *raw = ring + slot * S::kRaw;
        uint8_t *vb = smem + (2 + buf) * S::kKBytes;
        uint32_t noted = 0;
#pragma unroll 1
        for (int i = 0; i < kTasks; ++i) {
          const int id = i * 128 + vt, word = id % kWords, chunk = id / kWords;  // keys [8 chunk, 8 chunk + 8)
          // rows of two neighbouring chunks lie in the same banks: the odd ones
          // read their key pairs the other way round
          const int swap = D == 256 ? 0 : chunk & 1;
          const uint8_t *cp = raw + S::kCodes + chunk * 8 * (D / 2) + word * 4;
          const uint8_t *ep = raw + 2 * S::kCodes + S::kEntries + (chunk * 8 * W + word % W) * 4;
          uint32_t c[8], e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            c[k] = *reinterpret_cast<const uint32_t *>(cp + (k ^ swap) * (D / 2));
            e[k] = *reinterpret_cast<const uint32_t *>(ep + (k ^ swap) * (W * 4));
          }
          const int left = lim - st * NK - chunk * 8;  // keys that the row has
          if (left < 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if ((k ^ swap) >= left) e[k] = 0;
          }
          // values that are not finite are left out here and put back by the rows
          // that see their key: the thread of the group's first word notes them
          uint32_t odd = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) odd |= ((e[k] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
          const bool was = had >> (buf * 16 + i) & 1u;
          if (odd || was) {
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (att_not_finite(e[k])) bad |= 1u << (k ^ swap), e[k] = 0;
            if (word < W) {
              uint32_t *flag = &s_bad[buf][chunk >> 2][word];
              atomicAnd(flag, ~(0xffu << ((chunk & 3) * 8)));
              if (bad) atomicOr(flag, bad << ((chunk & 3) * 8)), noted |= 1u << i;
            }
          }
          const uint32_t sel0 = swap ? 0x1054u : 0x5410u, sel1 = swap ? 0x3276u : 0x7632u;
          uint32_t es[4], eb[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            es[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel0);
            eb[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel1);
          }
          uint8_t *dst = vb + (chunk >> 3) * (D * 128) + word * 128 + (((chunk ^ word) & 7) << 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __byte_perm(c[2 * k], c[2 * k + 1], half ? sel1 : sel0), y[k] = x[k] >> 8;
            *reinterpret_cast<uint4 *>(dst + (4 * half + 0) * (kWords * 128)) =
                make_uint4(att_even(x[0], es[0], eb[0]), att_even(x[1], es[1], eb[1]), att_even(x[2], es[2], eb[2]), att_even(x[3], es[3], eb[3]));
            *reinterpret_cast<uint4 *>(dst + (4 * half + 1) * (kWords * 128)) =
                make_uint4(att_odd(x[0], es[0], eb[0]), att_odd(x[1], es[1], eb[1]), att_odd(x[2], es[2], eb[2]), att_odd(x[3], es[3], eb[3]));
            *reinterpret_cast<uint4 *>(dst + (4 * half + 2) * (kWords * 128)) =
                make_uint4(att_even(y[0], es[0], eb[0]), att_even(y[1], es[1], eb[1]), att_even(y[2], es[2], eb[2]), att_even(y[3], es[3], eb[3]));
            *reinterpret_cast<uint4 *>(dst + (4 * half + 3) * (kWords * 128)) =
                make_uint4(att_odd(y[0], es[0], eb[0]), att_odd(y[1], es[1], eb[1]), att_odd(y[2], es[2], eb[2]), att_odd(y[3], es[3], eb[3]));
          }
        }
        had = (had & ~(0xffffu << (buf * 16))) | noted << (buf * 16);
        fence_proxy_async_shared();
        mbar_arrive(&v_full[buf]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[slot]);
      }
    }
  } else if (warp >= 4) {
    // ---- K: 4 words (32 channels) of a key at a time ----------------------------------------
    const int kt = tid - 128;
    constexpr int kChunks = D / 32, kTasks = NK * kChunks / 128;
    uint32_t it = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next()) {
#pragma unroll 1
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t buf = it & 1, slot = it % kTcRing;
        ok = wait_warp(&k_empty[buf], ((it >> 1) & 1) ^ 1) && wait_warp(&raw_full[slot], it / kTcRing & 1);
        if (!ok) break;
        const uint8_t *raw = ring + slot * S::kRaw;
        uint8_t *kb = smem + buf * S::kKBytes;
#pragma unroll 2
        for (int i = 0; i < kTasks; ++i) {
          const int id = i * 128 + kt, c = id % kChunks, r = id / kChunks;
          const uint4 x4 = *reinterpret_cast<const uint4 *>(raw + r * (D / 2) + c * 16);
          uint32_t e[W];
          att_words<W>(e, raw + 2 * S::kCodes + r * (W * 4));
          const uint32_t wd[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t step = __byte_perm(e[q % W], e[q % W], 0x1010), off = __byte_perm(e[q % W], e[q % W], 0x3232);
            const uint32_t x = wd[q], y = x >> 8;
            const int u = tc_unit<D>(c, q);
            *reinterpret_cast<uint4 *>(kb + (u >> 3) * (NK * 128) + r * 128 + (((u ^ r) & 7) << 4)) =
                make_uint4(att_even(x, step, off), att_odd(x, step, off), att_even(y, step, off), att_odd(y, step, off));
          }
        }
        fence_proxy_async_shared();
        mbar_arrive(&k_full[buf]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[slot]);
      }
    }
  } else {
    // ---- softmax: thread = query row --------------------------------------------------------
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
        float up = __uint_as_float(uint32_t(264 - e) << 23);
        // the factor of a score is kept positive: the maximum is taken before it
        f = p.scale != 0.f ? (1.f / up) * fabsf(p.scale * 1.4426950408889634f) : 1.f;
        up = p.scale > 0.f ? up : p.scale < 0.f ? -up : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 x = live ? __ldg(src + 4 * c + q) : make_uint4(0, 0, 0, 0);
            const uint32_t a[4] = {x.x, x.y, x.z, x.w};
            float y[8];
#pragma unroll
            for (int h = 0; h < 4; ++h)
              y[2 * h] = __uint_as_float(a[h] << 16) * up, y[2 * h + 1] = __uint_as_float(a[h] & 0xffff0000u) * up;
#pragma unroll
            for (int h = 0; h < 4; ++h) w[4 * q + h] = pack_h2(y[h], y[h + 4]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            tmem_st4_async(lane_base + S::kColQ + 4 * tc_unit<D>(c, q), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&q_full);
      }
      float m = -INFINITY, l = 0.f;
      uint32_t nan = 0;
#pragma unroll 1
      for (int st = walk.st0; ok && st < walk.st1; ++st, ++it) {
        const uint32_t buf = it & 1, ph = (it >> 1) & 1;
        ok = wait_warp(&s_full[buf], ph);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sc = lane_base + S::kColS + buf * NK;
        const int t0 = st * NK;
        const bool cut = t0 + NK > lim_min;
        float x = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < NK / 64; ++q) {
          uint32_t a[32], b[32];
          tmem_ld32_async(sc + 64 * q, a);
          tmem_ld32_async(sc + 64 * q + 32, b);
          tmem_wait_ld();
          if (cut) {
            const int left = lim - t0 - 64 * q;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (k >= left) a[k] = 0xff800000u;
              if (32 + k >= left) b[k] = 0xff800000u;
            }
          }
          float xs[4] = {x, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; ++k) xs[k & 3] = max3(xs[k & 3], __uint_as_float(a[k]), __uint_as_float(b[k]));
          x = fmaxf(max3(xs[0], xs[1], xs[2]), xs[3]);
        }
        x *= f;
        float a = 1.f;
        const bool move = x > m + 14.f;
        if (move) {
          const float n = fmaxf(m, x - 6.f);
          a = m == -INFINITY ? 0.f : ex2(m - n);
          m = n;
          l *= a;
        }
        if (st > walk.st0) {
          const bool any = __any_sync(0xffffffffu, move);
          // the last product has to be done before O is rescaled, or its P written over
          if (any || !S::kOver) {
            ok = wait_warp(&pv_done, (it - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          if (any) {
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
          }
        }
        const float r0 = m == -INFINITY ? 0.f : m;
        const F2 ff = f2(f, f), rr = f2(-r0, -r0);
        F2 ls[2] = {f2(l, 0.f), f2(0.f, 0.f)};
        // P's 16 columns of a chunk lie over scores that are read already
#pragma unroll 1
        for (int q = 0; q < NK / 32; ++q) {
          uint32_t b[32], w[16];
          tmem_ld32_async(sc + 32 * q, b);
          tmem_wait_ld();
          if (cut) {
            const int left = lim - t0 - 32 * q;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k >= left) b[k] = 0xff800000u;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float pa, pb;
            f2_get(f2_fma(f2(__uint_as_float(b[2 * k]), __uint_as_float(b[2 * k + 1])), ff, rr), pa, pb);
            pa = ex2(pa), pb = ex2(pb);
            ls[k & 1] = f2_add(ls[k & 1], f2(pa, pb));
            w[k] = pack_h2(pa, pb);
          }
          tmem_st16_async(lane_base + S::col_p(buf) + 16 * q, w);
        }
        {
          float la, lb;
          f2_get(f2_add(ls[0], ls[1]), la, lb);
          l = la + lb;
        }
        tmem_wait_st();
        tc_fence_before();
        // values that are not finite reach the rows that see their key
        ok = wait_warp(&v_full[buf], ph);
        if (!ok) break;
        {
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < NK / 32 * W; ++k) any |= *reinterpret_cast<volatile uint32_t *>(&s_bad[buf][0][0] + k);
          if (any) {
#pragma unroll 1
            for (int k = 0; k < NK / 32 * W; ++k) {
              const uint32_t bad = *reinterpret_cast<volatile uint32_t *>(&s_bad[buf][0][0] + k);
              const int n = lim - t0 - 32 * (k / W);
              if (n > 0 && (bad & (n >= 32 ? 0xffffffffu : (1u << n) - 1))) nan |= 1u << (k % W);
            }
          }
        }
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // ---- the unit's rows, or a part of them ------------------------------------------
      ok = wait_warp(&pv_done, (it - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      constexpr int kWords = D / 8;  // column e kWords + w of O is channel 8 w + e
      const bool whole = walk.st0 == 0 && walk.st1 == walk.stages;
      bool last = whole;
      long long c_first = 0, c_last = 0;
      auto part_of = [&](long long k) -> float * { return parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * tc_part_floats<D>() + r; };
      if (!whole) {
        c_first = ((walk.unit_first + 1) * ctas - 1) / total;
        c_last = ((walk.unit_first + walk.stages) * ctas - 1) / total;
        float *part = part_of(c);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32_async(lane_base + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            part[size_t(32 * q + k) * kTcRows] = nan >> ((32 * q + k) % kWords % W) & 1 ? __uint_as_float(0x7fc00000u) : __uint_as_float(o[k]);
        }
        part[size_t(D) * kTcRows] = m, part[size_t(D + 1) * kTcRows] = l;
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
          for (long long k = c_first; k <= c_last; ++k) M = fmaxf(M, __ldcg(part_of(k) + size_t(D) * kTcRows));
          for (long long k = c_first; k <= c_last; ++k) {
            const float mk = __ldcg(part_of(k) + size_t(D) * kTcRows), lk = __ldcg(part_of(k) + size_t(D + 1) * kTcRows);
            Ls = fmaf(lk, lk != lk ? 1.f : mk == -INFINITY ? 0.f : ex2(mk - M), Ls);
          }
        }
        const float v = Ls > 0.f ? 1.f / Ls : Ls;  // no key: 0; NaN stays
        uint16_t *dst = p.out + (size_t(tok) * p.g.H_q + head) * D;
#pragma unroll 1
        for (int w = 0; w < kWords; w += 4) {  // 4 words of 8 channels
          float y[8][4];
          if (whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) tmem_ld4_async(lane_base + e * kWords + w, y[e]);
            tmem_wait_ld();
            if (nan)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (nan >> (k % W) & 1)
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e][k] = __uint_as_float(0x7fc00000u);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e][0] = y[e][1] = y[e][2] = y[e][3] = 0.f;
#pragma unroll 1
            for (long long kc = c_first; kc <= c_last; ++kc) {
              const float *src = part_of(kc);
              const float mk = __ldcg(src + size_t(D) * kTcRows), lk = __ldcg(src + size_t(D + 1) * kTcRows);
              const float ck = lk != lk ? 1.f : mk == -INFINITY ? 0.f : ex2(mk - M);
#pragma unroll
              for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[e][k] = fmaf(__ldcg(src + size_t(e * kWords + w + k) * kTcRows), ck, y[e][k]);
            }
          }
          if (in) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * e][k] * v, y[2 * e + 1][k] * v);
                h[e] = *reinterpret_cast<const uint32_t *>(&b2);
              }
              *reinterpret_cast<uint4 *>(dst + 8 * (w + k)) = make_uint4(h[0], h[1], h[2], h[3]);
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
  if (warp == 12) tmem_dealloc(tmem, S::kCols);
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

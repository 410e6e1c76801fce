// kv4_attend_tc.cuh -- causal attention of many query rows over the paged
// 4-bit cache on the tcgen05 tensor cores.
//
// A unit is (row b, kv head, tile of TT = floor(128 / G) whole tokens): up to
// 128 query rows share every key that is formed.  Per tile of NK keys:
//   copies   one warp brings the tile's codes and entries into a ring of four;
//   dequant  4 warps form K [NK][D] and 4 form V^T [D][NK] in fp16 (each value
//            rounded once) in shared memory, K-major with the 128-byte swizzle;
//   scores   S = Q K^T, Q in tensor memory as the A operand;
//   softmax  two groups of 4 warps take half of the tile's keys each, a thread a
//            row: running maximum and sum in fp32, the maxima of both halves
//            exchanged; P goes back to tensor memory in fp16, over its scores (a
//            group a tile in turn cost the chunk 618 us for 615, deep drafts 51.6
//            for 50.6);
//   output   O += P V, P from tensor memory; O is rescaled only when a
//            probability passes 2^14.
// Entries whose levels pass fp16 (kv4_attend.cuh, "Wide groups") are noted by their key.
// In K they spoil the key's own column of scores, which is formed anew before the
// maximum; from V they are left out, and the rows that see the key add them to O when
// the unit's products are done.
// A product does not see the order of its inner dimension, nor O's columns the
// order they are kept in, so both follow what shared memory likes:
//  - inside 8 channels 0 4 1 5 2 6 3 7 (the order masks take codes out of a word);
//  - the words of a key as tc_unit() lays them, so that the threads that read a
//    key side by side store into different banks;
//  - channel 8 w + e of V in row e (D / 8) + w, for the same reason.
// The loops over a tile are kept short in code (a chunk of 32 scores, a word of
// codes at a time): unrolled whole, the roles' code passed what the SM's
// instruction caches hold, and every instruction waited for its fetch (5.5 us a
// tile of 64 keys at D = 256, for 1.4).
//
// What bounds it: a tile is a chain (scores, their maximum, exponentials, output)
// whose steps wait for one another, and the roles share the issue slots, which
// are 58 % busy; the tensor cores work 28 % of the time.  A tile of 128 keys at D =
// 128 takes 2740 cycles where its products alone take 1090; with the dequant, the
// exponentials and the maxima left out, 1790: what then is left is the products
// and the barriers between them.  Neither separate columns for P (no
// scores wait for the output of the tile before last, 3 % slower), nor loads of
// scores 16 at a time and one ahead (17 % slower), nor leaving out the softmax of
// warps without rows (2 % slower), nor the products' waits two at a time (the same)
// shortened it.
// With Q and P in tensor memory the products read only K and V from shared
// memory, so that a 64-key tile still feeds them at D = 256, where O takes half
// of the tensor memory.
// 2000 queries behind 16001 keys, 32 heads over 8 of 128: 624 us, 893 TFLOP/s of
// the products; a prompt of 4096, 16 heads over 2 of 256: 198 us, 690 TFLOP/s
// (back to back; 628 and 202 us with other work between the calls).
//
// Units are laid on one line in tiles of keys and cut evenly over a persistent
// grid as in kv4_attend.cuh; causal tiles count as far as their last query sees.
// A unit that is cut leaves parts in the workspace.
#pragma once

#include "kv4_attend.cuh"

namespace gdn {

constexpr int kTcRows = 128;
// Roles by `role` = (warp + 16) mod 20: 0-7 softmax, 8-11 K, 12-15 V, 16 products,
// 17 copies, 18 units, 19 wide keys.  The products' warp is the oldest of its
// scheduler, which seems to favour the oldest ready one (a prompt of 4096 at
// D = 256: 242 us with it as the youngest, 227 so).
constexpr int kTcThreads = 640;
constexpr int kTcRing = 4;       // tiles of codes in flight
constexpr int kTcUnits = 4;      // units handed out ahead
// What a unit costs besides its tiles of keys (queries in, outputs out), in
// tiles: its place on the line is that much longer, so that the pieces of the
// CTAs that have many short units are not the last to end.  The prompt of 4096
// above: 329 us with 1, 241 with 3, 189 with 6, 193 with 10; 24 rows of 8 drafts
// over 6001 keys, 32 heads over 4 of 128: 59.8, 49.8, 51.6, 55.1.
constexpr int kTcUnitCost = 6;
// Parts of a cut unit that are joined at a time: by one CTA, part after part, those of
// 32768 keys with 24 rows at D = 256 (76 parts) made the call take 240 us, 39 so.
constexpr int kTcJoin = 8;

template <int D>
struct TcShape {
  static constexpr int W = D / 64;
  static constexpr int NK = D == 256 ? 64 : 128;  // keys of a tile
  static constexpr int kKBytes = NK * D * 2;      // K or V of a tile
  static constexpr int kRaw = 2 * (NK * D / 2 + NK * W * 4);  // a tile as it comes: its pages' records
  static constexpr int kSmem = 4 * kKBytes + kTcRing * kRaw + 1024;
  // tensor memory columns: O [D], S two buffers [NK] with P over them, Q [D / 2]
  static constexpr int kColS = D, kColQ = D + 2 * NK;
  static constexpr int kCols = 512;
  static_assert(kColQ + D / 2 <= kCols, "tensor memory");
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

static __device__ __noinline__ TcRow tc_row(const Kv4AttendParams &p, int b, int TT, bool report) {
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
template <typename Row>
__device__ __forceinline__ int tc_limit(const Row &r, int t, int TT) {
  return r.count > t * TT ? max(0, r.len - r.count + min((t + 1) * TT, r.count)) : 0;
}
template <int NK, typename Row>
__device__ __forceinline__ int tc_stages(const Row &r, int t, int TT) {
  return max(1, (tc_limit(r, t, TT) + NK - 1) / NK);
}

// Places on the line of all query tiles of a row (one head): the tiles of keys,
// and kTcUnitCost each.  Query tile t of the full ones takes ceil((base + (t + 1) TT) / NK): with NK a power of two its
// fractions repeat every `per` tiles, so whole periods come from a formula.
template <int NK>
__device__ __noinline__ long long tc_row_stages(const TcRow r, int TT) {
  const int live = (r.count + TT - 1) / TT;  // tiles with a query
  const int base = r.len - r.count;
  long long s = (long long)r.tiles * kTcUnitCost + r.tiles - live;
  // tiles whose queries see no key count as one
  int first = 0;
  if (base < 0) first = min(live, -base / TT);
  s += first;
  const int n = live - first;
  if (n <= 0) return s;
  int per = NK;
  while (per > 1 && ((per >> 1) * TT) % NK == 0) per >>= 1;
  const int full = (n - 1) / per;  // the last tile may be short: left to the loop
  const int b0 = base + (first + 1) * TT + NK - 1, rise = per * TT / NK;
  long long one = 0;
#pragma unroll 1
  for (int j = 0; j < per && full; ++j) one += (b0 + j * TT) / NK;
  s += full * one + (long long)rise * per * ((long long)full * (full - 1) / 2);
#pragma unroll 1
  for (int t = first + full * per; t < live; ++t) s += tc_stages<NK>(r, t, TT);
  return s;
}

// A unit, or the part of one that a CTA has: tiles of keys [st0, st1) of stages.
struct TcUnit {
  int b, hk, tile, st0, st1, stages;  // st1 = 0: there are no more
  int start, span, count, len;
  long long first;                    // the unit's place in the line
};

// One thread of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// S[BUF] = Q K[BUF]^T; kv: the descriptor of the first K buffer.
template <int D, int BUF>
__device__ __forceinline__ void tc_scores(uint64_t kv) {
  using S = TcShape<D>;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    umma_f16_ts(S::kColS + BUF * S::NK, S::kColQ + ks * 8,
                kv + ((BUF * S::kKBytes + (ks >> 2) * (S::NK * 128) + (ks & 3) * 32) >> 4), umma_idesc_f16(kTcRows, S::NK), ks > 0);
}

// O (+)= P V[BUF].
template <int D, int BUF>
__device__ __forceinline__ void tc_output(uint64_t kv, bool acc) {
  using S = TcShape<D>;
#pragma unroll
  for (int ks = 0; ks < S::NK / 16; ++ks)
    umma_f16_ts(0, S::kColS + BUF * S::NK + (ks < S::NK / 32 ? 0 : S::NK / 4) + ks * 8,  // each half of P over its scores
                kv + (((2 + BUF) * S::kKBytes + (ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4), umma_idesc_f16(kTcRows, D),
                acc || ks > 0);
}

// The rest of a wait that did not end at once; out of line to keep the roles'
// code small.
static __device__ __noinline__ bool tc_wait_slow(uint64_t *bar, uint32_t parity, volatile int *dead, uint32_t *status, uint32_t limit) {
  bool ok = false;
  if (!*dead) {
    ok = att_wait(bar, parity, limit);
    if (!ok && !*dead) {
      *dead = 1;
      atomicOr(status, GDN_STATUS_TIMEOUT);
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Exclusive prefix of v over the CTA, and the sum.
static __device__ __noinline__ long long tc_scan(long long v, long long *s_warp, long long *sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = lane < warp ? s_warp[lane] : 0, all = lane < kTcThreads / 32 ? s_warp[lane] : 0;
#pragma unroll 1
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  *sum = all;
  return before + x - v;
}

__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  float v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr));
  tmem_wait_ld();
  return v;
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(v) : "memory");
  tmem_wait_st();
}

// A softmax thread's query row: its query (NULL: none) and the keys it sees.
struct TcQuery {
  const uint16_t *q;
  int lim;
};
template <int D>
static __device__ TcQuery tc_query(const Kv4AttendParams &p, const TcUnit &u) {
  const int G = p.g.H_q / p.g.H_kv, TT = kTcRows / G, r = (threadIdx.x - 128) & 127, i = u.tile * TT + r / G;
  if (r >= TT * G || i >= u.count) return TcQuery{nullptr, 0};
  return TcQuery{p.q + (size_t(u.start + i) * p.g.H_q + u.hk * G + r % G) * D, max(0, u.len - u.count + i + 1)};
}

// The scores of a tile's wide keys (bits), formed anew for a softmax warp's rows and half
// of the tile, which starts with key t0; in the columns from sc on, in units of f.
template <int D>
static __device__ __noinline__ void tc_new_scores(const Kv4AttendParams &p, const TcUnit &u, const uint32_t *keys, int t0, float f,
                                                  uint32_t sc) {
  const TcQuery row = tc_query<D>(p, u);
#pragma unroll 1
  for (int e = 0; e < TcShape<D>::NK / 2; ++e) {
    if (!(keys[e >> 5] >> (e & 31) & 1u)) continue;
    const float x = row.q && t0 + e < row.lim ? att_dot<D>(p, u.b, u.hk, t0 + e, row.q) * (p.scale * 1.4426950408889634f / f) : 0.f;
    __syncwarp();
    tmem_st1(sc + e, x);
  }
}

// The wide groups' part of O, of the unit's keys [t0, t1), weighted against a row's
// reference m, for a softmax warp's rows: its half of the words of O's columns, or
// (blocks) of the columns themselves.
template <int D>
static __device__ __noinline__ void tc_add_values(const Kv4AttendParams &p, const TcUnit &u, int t0, int t1, float m, bool blocks) {
  constexpr int W = D / 64, kWords = D / 8;
  const TcQuery row = tc_query<D>(p, u);
  const int lane = threadIdx.x & 31, P = 1 << p.g.log2P, half = (threadIdx.x - 128) >> 7, b = u.b, hk = u.hk;
  const uint32_t tmem = (threadIdx.x & 96) << 16;
#pragma unroll 1
  for (int t = t0; t < t1; t += 32) {
    uint32_t groups = 0;  // wide ones of the lane's key
    if (t + lane < t1) {
      const uint8_t *e = att_place(p, b, hk, t + lane, 2 * kv4_code_bytes(D, P) + kv4_entry_bytes(D, P), W * 4);
      for (int g = 0; e && g < W; ++g) groups |= uint32_t(att_wide(reinterpret_cast<const uint32_t *>(e)[g])) << g;
    }
    uint32_t keys = __ballot_sync(0xffffffffu, groups != 0);
#pragma unroll 1
    for (; keys; keys &= keys - 1) {
      const int k = __ffs(keys) - 1;
      const uint32_t of = __shfl_sync(0xffffffffu, groups, k);
      const uint8_t *codes = att_place(p, b, hk, t + k, kv4_code_bytes(D, P), D / 2);
      const uint8_t *entries = att_place(p, b, hk, t + k, 2 * kv4_code_bytes(D, P) + kv4_entry_bytes(D, P), W * 4);
      float weight = 0.f;
      if (row.q && t + k < row.lim && m != -INFINITY)
        weight = ex2(att_dot<D>(p, b, hk, t + k, row.q) * (p.scale * 1.4426950408889634f) - m);
      __syncwarp();
#pragma unroll 1
      for (int col = blocks ? half * (D / 2) : 0; col < (blocks ? (half + 1) * (D / 2) : D); ++col) {
        const int w = col % kWords, e = col / kWords;  // channel 8 w + e
        if (!(of >> (w % W) & 1u) || (!blocks && w / (kWords / 2) != half)) continue;
        const uint32_t entry = reinterpret_cast<const uint32_t *>(entries)[w % W];
        const float code = float(reinterpret_cast<const uint32_t *>(codes)[w] >> (4 * e) & 15u);
        tmem_st1(tmem + col, fmaf(weight, fmaf(half_lo(entry), code, half_hi(entry)), tmem_ld1(tmem + col)));
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) kv4_attend_tc(const __grid_constant__ Kv4AttendParams p) {
  using S = TcShape<D>;
  constexpr int W = S::W, NK = S::NK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t raw_full[kTcRing], raw_empty[kTcRing], unit_full[kTcUnits], unit_empty[kTcUnits];
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], x_full[4], pv_done[2];
  __shared__ uint64_t q_full, joined, drained;
  __shared__ TcUnit s_unit[kTcUnits];
  __shared__ uint32_t s_tmem;
  __shared__ long long s_warp[kTcThreads / 32];
  __shared__ struct {
    int b;
    TcRow row;
    long long in_row, len;
  } s_at;  // the row that holds the CTA's first place
  __shared__ float s_top[2][2][kTcRows], s_sum[2][kTcRows];
  __shared__ float s_w[(kAttMaxCtas + kTcJoin - 1) / kTcJoin][kTcRows];  // weights of the parts of a join
  __shared__ uint32_t s_nan[2 * kTcRows], s_mx[2][kTcRows];
  __shared__ int s_flag, s_dead;
  // keys of a V tile with a group that is not finite or wide, per group; of four tiles,
  // since the rows look two tiles later; and keys of a K tile with a wide group
  __shared__ __align__(16) uint32_t s_bad[4][NK / 32 * W];
  __shared__ uint32_t s_keys[4][NK / 32], s_some[4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int role = ((tid >> 5) + 16) % 20, rtid = role * 32 + lane;  // and the thread's place among the roles'
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ring = smem + 4 * S::kKBytes;
  const int G = p.g.H_q / p.g.H_kv, Hkv = p.g.H_kv, TT = kTcRows / G;
  const int P = 1 << p.g.log2P;
  if (tid == 0) {
    for (int i = 0; i < kTcRing; ++i) mbar_init(&raw_full[i], 1 + (blockIdx.x + i == 0 ? p.test_hold : 0u)), mbar_init(&raw_empty[i], 9);
    for (int i = 0; i < kTcUnits; ++i) mbar_init(&unit_full[i], 1), mbar_init(&unit_empty[i], 19);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 129), mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1), mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 256), mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&x_full[i], 64);
    mbar_init(&q_full, 256), mbar_init(&joined, 256), mbar_init(&drained, 1);
    s_dead = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 4 * (NK / 32) * W; i += kTcThreads) (&s_bad[0][0])[i] = 0;
  if (tid < 4) s_some[tid] = 0;
  pdl_wait();

  // ---- this CTA's piece of the line --------------------------------------------------
  // rows beyond the CTA's threads are summed first and looked at again below
  auto places = [&](const TcRow &r) -> long long { return tc_row_stages<NK>(r, TT) * Hkv; };
  long long total = 0, mine = 0, before, len = 0;
  TcRow own{};
#pragma unroll 1
  for (int b = tid; b < p.g.B; b += kTcThreads) {
    const TcRow r = tc_row(p, b, TT, blockIdx.x == 0);
    const long long x = places(r);
    if (b == tid) own = r, len = x;
    mine += x;
  }
  before = tc_scan(mine, s_warp, &total);
  // a piece is worth its fixed costs, or there are fewer
  const int ctas = int(min((long long)gridDim.x, (total + kTcUnitCost + 1) / (kTcUnitCost + 2)));
  const int c = blockIdx.x;
  if (c >= ctas) return;
  // pieces of `per` places, the first `more` of one more
  const long long per = total < (1ll << 31) ? int(total) / ctas : total / ctas;
  const int more = int(total - per * ctas);
  const long long at0 = per * c + min(c, more), stop = at0 + per + (c < more);
  auto cta_of = [&](long long x) -> int {
    const long long y = x - more * (per + 1);
    if (x < (1ll << 31)) return y < 0 ? int(x) / int(per + 1) : more + int(y) / int(per);
    return int(y < 0 ? x / (per + 1) : more + y / per);
  };
  // the row that holds at0, by its thread
  long long before0 = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.g.B; b0 += kTcThreads) {
    if (p.g.B > kTcThreads) {
      long long sum;
      len = 0;
      if (b0 + tid < p.g.B) own = tc_row(p, b0 + tid, TT, false), len = places(own);
      before = before0 + tc_scan(len, s_warp, &sum);
      before0 += sum;
    }
    if (at0 >= before && at0 < before + len) s_at.b = b0 + tid, s_at.row = own, s_at.in_row = at0 - before, s_at.len = len;
  }

  if (role == 16) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The next kernel starts only now: a flagged verify takes tensor memory before its wait,
  // and one that came before the allocation above would wait for this kernel and it for
  // the verify.
  pdl_trigger();
  // a bounded wait of the whole warp; false once any wait of the CTA has run out
  auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return tc_wait_slow(bar, parity, &s_dead, p.status, p.wait_limit);
  };
  uint32_t un = 0;  // units taken so far
  // the next unit, for a role's warp; false when there is none or a wait ran out
  auto next_unit = [&](bool ok) -> bool {
    const uint32_t i = un % kTcUnits;
    if (un > 0) {  // the last one is done with
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[(un - 1) % kTcUnits]);
    }
    if (!ok || !wait_warp(&unit_full[i], un / kTcUnits & 1)) return false;
    ++un;
    return s_unit[i].st1 > 0;
  };
  auto unit = [&]() -> const TcUnit & { return s_unit[(un - 1) % kTcUnits]; };

  if (role == 18) {
    // ---- units ------------------------------------------------------------------------------
    long long at = at0;
    int b = s_at.b, hk = 0, t = 0, place;  // place in the unit, of stages + kTcUnitCost
    TcRow row = s_at.row;
    {
      // the head, then the query tile: 32 at a time
      const long long head = s_at.len / Hkv;
      long long left = s_at.in_row;
      while (left >= head) left -= head, ++hk;
#pragma unroll 1
      for (;;) {
        const int v = t + lane < row.tiles ? tc_stages<NK>(row, t + lane, TT) + kTcUnitCost : 0;
        int sum = v;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += u;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, sum > left);
        if (past) {
          const int f = __ffs(past) - 1;
          t += f;
          place = int(left) - __shfl_sync(0xffffffffu, sum - v, f);
          break;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
        t += 32;
      }
    }
    bool ok = true;
    uint32_t k = 0;
#pragma unroll 1
    while (ok) {
      const bool more_units = at < stop;
      int stages = 0, end = 0;
      if (more_units) {
        stages = tc_stages<NK>(row, t, TT);
        end = int(min((long long)stages + kTcUnitCost, place + (stop - at)));
      }
      // a piece that ends in a unit's fixed part has none of its tiles
      if (!more_units || end > kTcUnitCost) {
        ok = wait_warp(&unit_empty[k % kTcUnits], (k / kTcUnits & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          TcUnit u{};
          if (more_units) {
            u.stages = stages, u.st0 = max(0, place - kTcUnitCost), u.st1 = end - kTcUnitCost;
            u.first = at - place;
            u.b = b, u.hk = hk, u.tile = t, u.start = row.start, u.span = row.span, u.count = row.count, u.len = row.len;
          }
          s_unit[k % kTcUnits] = u;
          mbar_arrive(&unit_full[k % kTcUnits]);
        }
        ++k;
      }
      if (!more_units) break;
      at += end - place;
      place = 0;
      if (at < stop && ++t == row.tiles) {
        t = 0;
        if (++hk == Hkv) {
          hk = 0;
          do row = tc_row(p, ++b, TT, false);
          while (row.tiles == 0);
        }
      }
    }
  } else if (role == 17) {
    // ---- copies -------------------------------------------------------------------------
    // A page is one copy, as it lies in memory: copies are taken one in about 70
    // cycles whatever their size, so 32 pieces of eight small pages took 2250
    // cycles a tile.
    const int n_sub = NK >> p.g.log2P;  // pages of a tile
    const uint32_t rec_bytes = kv4_record_bytes(D, P);
    uint32_t it = 0;
    bool ok = true;
    while (next_unit(ok)) {
      const int lim = tc_limit(unit(), unit().tile, TT), st1 = unit().st1;
      const int32_t *table = p.table + size_t(unit().b) * p.g.max_pages;
      const uint8_t *head = p.pages + size_t(unit().hk) * rec_bytes;
      auto page_of = [&](int st) -> int {  // lane l: page l of the tile, -2: none; a negative one is -1
        const int t = st * NK + (lane << p.g.log2P);
        return lane < n_sub && st < st1 && t < lim ? max(-1, table[t >> p.g.log2P]) : -2;
      };
      int next = page_of(unit().st0);
#pragma unroll 1
      for (int st = unit().st0; ok && st < st1; ++st, ++it) {
        const uint32_t slot = it % kTcRing;
        int page = next;
        next = page_of(st + 1);
        if (page != -2 && (page < 0 || page >= p.g.n_pages)) {
          page = -2;
          atomicOr(p.status, GDN_STATUS_BAD_INDEX);
        }
        ok = wait_warp(&raw_empty[slot], (it / kTcRing & 1) ^ 1);
        if (!ok) break;
        const uint32_t pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], pages * rec_bytes);
        __syncwarp();
        if (page >= 0)
          bulk_g2s(ring + slot * S::kRaw + lane * rec_bytes, head + size_t(page) * (Hkv * size_t(rec_bytes)), rec_bytes, &raw_full[slot]);
      }
    }
    // no copy is in flight when the CTA ends, whichever role's wait may have run out: its
    // readers have waited for it, or do no more
    for (uint32_t k = it < kTcRing ? 0 : it - kTcRing; k < it; ++k)
      att_wait(&raw_full[k % kTcRing], k / kTcRing & 1, p.wait_limit);
  } else if (role == 16) {
    // ---- products -----------------------------------------------------------------------
    // The whole warp waits, one elected thread issues; the operands'
    // addresses are constants of each buffer's own code, so that they stand in
    // uniform registers (moved there one by one, they made a product of 32
    // cycles take 90 to issue).
    const uint64_t kv = umma_desc_sw128(smem_u32(smem));
    uint32_t base = 0, units = 0;  // tiles and units before this one
    bool ok = true;
    while (next_unit(ok)) {
      ok = wait_warp(&q_full, units++ & 1);
      const int n = unit().st1 - unit().st0;
      // scores of tile i, then the output of tile i - 1
#pragma unroll 1
      for (int i = 0; ok && i <= n; ++i) {
        if (i < n) {
          const uint32_t it = base + i, buf = it & 1;
          // the P of two tiles ago that lies over them is used up
          if (i > 1) ok = wait_warp(&pv_done[buf], ((it - 2) >> 1) & 1);
          ok = ok && wait_warp(&k_full[buf], (it >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (buf) tc_scores<D, 1>(kv);
            else tc_scores<D, 0>(kv);
            umma_commit(&k_empty[buf]);
            umma_commit(&s_full[buf]);
          }
          __syncwarp();
        }
        if (i > 0) {
          const uint32_t it = base + i - 1, buf = it & 1, ph = (it >> 1) & 1;
          ok = wait_warp(&v_full[buf], ph) && wait_warp(&p_full[buf], ph);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (buf) tc_output<D, 1>(kv, i > 1);
            else tc_output<D, 0>(kv, i > 1);
            umma_commit(&v_empty[buf]);
            umma_commit(&pv_done[buf]);
          }
          __syncwarp();
        }
      }
      base += n;
    }
    // no product is in flight when the CTA ends, whichever role's wait may have run out
    if (elect_one()) umma_commit(&drained);
    __syncwarp();
    att_wait(&drained, 0, p.wait_limit);
  } else if (role >= 12 && role < 16) {
    // ---- V^T: 8 keys of one word (8 channels) at a time, 16 bytes of 8 rows ------------------
    const int vt = rtid - 384;
    constexpr int kWords = D / 8, kTasks = NK / 8 * kWords / 128, kChunkStep = 128 / kWords;
    uint32_t had = 0;  // bit kTasks * (tile % 4) + i: the thread noted keys of task i
    // what a thread's tasks read and write, the same in every tile
    const int word = vt % kWords, chunk0 = vt / kWords;  // task i has keys 8 (chunk0 + i kChunkStep) ..
    // rows of two neighbouring chunks lie in the same banks: the odd ones read
    // their key pairs the other way round
    static_assert(kTasks == 1 || kChunkStep % 2 == 0, "chunks of a thread share their order");
    const int swap = D == 256 ? 0 : chunk0 & 1;
    const uint32_t sel0 = swap ? 0x1054u : 0x5410u, sel1 = swap ? 0x3276u : 0x7632u;
    // (the second task's a fixed step behind the first's)
    int code_at = 0, entry_at = 0, to = 0, code_step = 0, entry_step = 0, to_step = 0;
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
      const int chunk = chunk0 + i * kChunkStep, off = (chunk * 8) & (P - 1);
      const int rec = (chunk >> (p.g.log2P - 3)) * kv4_record_bytes(D, P);
      const int code = rec + kv4_code_bytes(D, P) + off * (D / 2) + word * 4;
      const int entry = rec + 2 * kv4_code_bytes(D, P) + kv4_entry_bytes(D, P) + (off * W + word % W) * 4;
      const int at = (chunk >> 3) * (D * 128) + word * 128 + (((chunk ^ word) & 7) << 4);
      if (i == 0) code_at = code, entry_at = entry, to = at;
      else code_step = code - code_at, entry_step = entry - entry_at, to_step = at - to;
    }
    static_assert(kTasks <= 2, "two tasks at most");
    uint32_t it = 0;
    bool ok = true;
    while (next_unit(ok)) {
      const int lim = tc_limit(unit(), unit().tile, TT), st1 = unit().st1;
#pragma unroll 1
      for (int st = unit().st0; ok && st < st1; ++st, ++it) {
        const uint32_t buf = it & 1, slot = it % kTcRing;
        ok = wait_warp(&v_empty[buf], ((it >> 1) & 1) ^ 1) && wait_warp(&raw_full[slot], it / kTcRing & 1);
        if (!ok) break;
        const uint8_t *raw = ring + slot * S::kRaw;
        uint8_t *vb = smem + (2 + buf) * S::kKBytes;
        uint32_t noted = 0;
        const bool tail = st * NK + NK > lim;
#pragma unroll 1
        for (int i = 0; i < kTasks; ++i) {
          const int chunk = chunk0 + i * kChunkStep;  // keys [8 chunk, 8 chunk + 8)
          const uint8_t *codes = raw + code_at + i * code_step, *entries = raw + entry_at + i * entry_step;
          const uint8_t *ce = codes + swap * (D / 2), *co = codes - swap * (D / 2);
          const uint8_t *ee = entries + swap * (W * 4), *eo = entries - swap * (W * 4);
          uint32_t c[8], e[8];  // of key k ^ swap
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            c[k] = *reinterpret_cast<const uint32_t *>((k & 1 ? co : ce) + k * (D / 2));
            e[k] = *reinterpret_cast<const uint32_t *>((k & 1 ? eo : ee) + k * (W * 4));
          }
          if (tail) {  // keys that the row does not have
            const int left = lim - st * NK - chunk * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if ((k ^ swap) >= left) e[k] = 0;
          }
          uint32_t es[4], eb[4], nil = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            es[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel0);
            eb[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel1);
            nil = att_look(es[k], eb[k], nil);
          }
          // values that are not finite, or wide, are left out here and put back by the rows
          // that see their key: the thread of the group's first word notes them
          const bool was = had >> ((it & 3) * kTasks + i) & 1u;
          if (att_found(nil) || was) {
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (att_not_fp16(e[k])) bad |= 1u << (k ^ swap), e[k] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              es[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel0);
              eb[k] = __byte_perm(e[2 * k], e[2 * k + 1], sel1);
            }
            if (word < W) {
              uint32_t *flag = &s_bad[it & 3][(chunk >> 2) * W + word];
              atomicAnd(flag, ~(0xffu << ((chunk & 3) * 8)));
              if (bad) atomicOr(flag, bad << ((chunk & 3) * 8)), noted |= 1u << i;
            }
          }
          uint8_t *dst = vb + to + i * to_step;
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
        had = (had & ~(((1u << kTasks) - 1) << ((it & 3) * kTasks))) | noted << ((it & 3) * kTasks);
        fence_proxy_async_shared();
        mbar_arrive(&v_full[buf]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[slot]);
      }
    }
  } else if (role >= 8 && role < 12) {
    // ---- K: 4 words (32 channels) of a key at a time ----------------------------------------
    const int kt = rtid - 256;
    constexpr int kChunks = D / 32, kTasks = NK * kChunks / 128, kRowStep = 128 / kChunks;
    // what a thread's tasks read and write, the same in every tile
    const int c = kt % kChunks, r0 = kt / kChunks;  // chunk, first row; task i has row r0 + i kRowStep
    // (two at a time, the next two a fixed step behind: short code, above)
    int code_at[2], entry_at[2], code_step = 0, entry_step = 0, to[4];
#pragma unroll
    for (int i = 0; i < (kTasks > 2 ? 3 : 2); ++i) {
      const int r = r0 + i * kRowStep, off = r & (P - 1);
      const int rec = (r >> p.g.log2P) * kv4_record_bytes(D, P);
      const int code = rec + off * (D / 2) + c * 16, entry = rec + 2 * kv4_code_bytes(D, P) + off * (W * 4);
      if (i < 2) code_at[i % 2] = code, entry_at[i % 2] = entry;
      else code_step = code - code_at[0], entry_step = entry - entry_at[0];
    }
    static_assert(kTasks == 2 || kTasks == 4, "two pairs at most");
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int u = tc_unit<D>(c, q);
      to[q] = (u >> 3) * (NK * 128) + r0 * 128 + (((u ^ r0) & 7) << 4);  // kRowStep is a multiple of 8
    }
    static_assert(kRowStep % 8 == 0, "rows of a thread share their swizzle");
    uint32_t it = 0;
    bool ok = true;
    while (next_unit(ok)) {
      const int st1 = unit().st1;
#pragma unroll 1
      for (int st = unit().st0; ok && st < st1; ++st, ++it) {
        const uint32_t buf = it & 1, slot = it % kTcRing;
        ok = wait_warp(&k_empty[buf], ((it >> 1) & 1) ^ 1) && wait_warp(&raw_full[slot], it / kTcRing & 1);
        if (!ok) break;
        const uint8_t *raw = ring + slot * S::kRaw;
        uint8_t *kb = smem + buf * S::kKBytes;
#pragma unroll 1
        for (int h = 0; h < kTasks / 2; ++h, kb += 2 * kRowStep * 128) {
         const uint8_t *codes = raw + h * code_step, *entries = raw + h * entry_step;
#pragma unroll
         for (int i = 0; i < 2; ++i) {
          const uint4 x4 = *reinterpret_cast<const uint4 *>(codes + code_at[i]);
          uint32_t e[W], step[W], base[W];
          att_words<W>(e, entries + entry_at[i]);
#pragma unroll
          for (int g = 0; g < W; ++g) step[g] = __byte_perm(e[g], e[g], 0x1010), base[g] = __byte_perm(e[g], e[g], 0x3232);
          const uint32_t wd[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t x = wd[q], y = x >> 8, sw = step[q % W], bw = base[q % W];
            *reinterpret_cast<uint4 *>(kb + to[q] + i * (kRowStep * 128)) =
                make_uint4(att_even(x, sw, bw), att_odd(x, sw, bw), att_even(y, sw, bw), att_odd(y, sw, bw));
          }
         }
        }
        fence_proxy_async_shared();
        mbar_arrive(&k_full[buf]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[slot]);
      }
    }
  } else if (role == 19) {
    // ---- wide keys: the entries of NK / 32 keys a lane, noted as the tile's K is formed -------
    constexpr int kKeys = NK / 32, kOwn = kKeys * W;
    const int key = lane * kKeys, off = key & (P - 1);
    const int at = (key >> p.g.log2P) * kv4_record_bytes(D, P) + 2 * kv4_code_bytes(D, P) + off * (W * 4);
    uint32_t had = 0;  // bit tile % 4: some key is noted
    uint32_t it = 0;
    bool ok = true;
    while (next_unit(ok)) {
      const int st1 = unit().st1;
#pragma unroll 1
      for (int st = unit().st0; ok && st < st1; ++st, ++it) {
        const uint32_t buf = it & 1, slot = it % kTcRing, of = 1u << (it & 3);
        ok = wait_warp(&k_empty[buf], ((it >> 1) & 1) ^ 1) && wait_warp(&raw_full[slot], it / kTcRing & 1);
        if (!ok) break;
        const uint32_t *e = reinterpret_cast<const uint32_t *>(ring + slot * S::kRaw + at);
        uint32_t nil = 0;
#pragma unroll
        for (int i = 0; i < kOwn; i += 4) {
          uint32_t x[4];
          att_words<4>(x, reinterpret_cast<const uint8_t *>(e + i));
          nil = att_look(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632), nil);
          nil = att_look(__byte_perm(x[2], x[3], 0x5410), __byte_perm(x[2], x[3], 0x7632), nil);
        }
        if (__any_sync(0xffffffffu, att_found(nil)) || (had & of)) {
          uint32_t keys = 0, any = 0;
#pragma unroll 1
          for (int i = 0; i < kOwn; ++i) keys |= uint32_t(att_wide(e[i])) << (i / W);
#pragma unroll 1
          for (int w = 0; w < NK / 32; ++w) {
            const uint32_t note = __reduce_or_sync(0xffffffffu, key >> 5 == w ? keys << (key & 31) : 0u);
            if (lane == 0) s_keys[it & 3][w] = note;
            any |= note;
          }
          if (lane == 0) s_some[it & 3] = any;
          had = any ? had | of : had & ~of;
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(&k_full[buf]);
          mbar_arrive(&raw_empty[slot]);
        }
      }
    }
  } else if (role < 8) {
    // ---- softmax: two threads a query row, half of a tile's keys a group of 4 warps -------------
    const uint32_t wg = role >> 2;
    const int r = rtid & 127;
    const uint32_t lane_base = uint32_t((role & 3) * 32) << 16;
    constexpr int kWords = D / 8;  // column e kWords + w of O is channel 8 w + e
    constexpr int kHalf = NK / 2;  // keys of a tile that a group has
    float *parts = reinterpret_cast<float *>(static_cast<char *>(p.ws) + 4096);
    uint32_t *counters = reinterpret_cast<uint32_t *>(p.ws);
    uint32_t base = 0, joins = 0;
    bool ok = true;
    while (next_unit(ok)) {
      const int st0 = unit().st0, n = unit().st1 - st0;
      const int i = unit().tile * TT + r / G, head = unit().hk * G + r % G;
      const bool in = r < TT * G && i < unit().span, live = in && i < unit().count;
      const int tok = unit().start + i;
      const int tile_lim = tc_limit(unit(), unit().tile, TT);
      const int lim = live ? max(0, unit().len - unit().count + i + 1) : in ? 0 : tile_lim;
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      // ---- Q as fp16 into tensor memory, half of a row's words a group.  Rows whose
      // largest magnitude is far from 1 are scaled by a power of two (exactly).
      float f = fabsf(p.scale) * 1.4426950408889634f;
      {
        // the factor of a score is kept positive: the maximum is taken before it
        const float sign = p.scale > 0.f ? 1.f : p.scale < 0.f ? -1.f : 0.f;
        if (p.scale == 0.f) f = 1.f;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t(live ? tok : 0) * p.g.H_q + (live ? head : 0)) * D) + wg * (D / 16);
        uint4 x[D / 16];
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) x[k] = live ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // the largest of both halves of a word: as unsigned pairs, signs away
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu), __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu)));
        }
        mx = max(mx & 0xffffu, mx >> 16);
        s_mx[wg][r] = mx;
        mbar_arrive(&joined);
        ok = wait_warp(&joined, joins++ & 1);
        if (!ok) break;
        mx = max(mx, s_mx[wg ^ 1][r]);
        const int e = int(mx >> 7);
        float up = sign;
        if (mx != 0 && (e < 127 - 6 || e > 127 + 13)) {
          const int k = min(max(e, 20), 240);
          const float s2 = __uint_as_float(uint32_t(264 - k) << 23);
          up *= s2;
          f *= 1.f / s2;
        }
        f = fmaxf(f, kLeastFactor);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t a[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          float y[8];
#pragma unroll
          for (int h = 0; h < 4; ++h)
            y[2 * h] = __uint_as_float(a[h] << 16) * up, y[2 * h + 1] = __uint_as_float(a[h] & 0xffff0000u) * up;
          const int w = wg * (D / 16) + k;
          tmem_st4_async(lane_base + S::kColQ + 4 * tc_unit<D>(w >> 2, w & 3), pack_h2(y[0], y[4]), pack_h2(y[1], y[5]),
                         pack_h2(y[2], y[6]), pack_h2(y[3], y[7]));
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&q_full);
      }
      float m = -INFINITY, l = 0.f;
      uint32_t nan = 0;
      // values that are not finite reach the rows that see their key; wide ones (bit 31)
      // are added to what the products leave in O
      auto look = [&](int k) {  // tile k of the unit
        const uint32_t *bad = s_bad[(base + k) & 3];
        uint32_t any = 0;
#pragma unroll
        for (int g = 0; g < NK / 32 * W; g += 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(bad + g);
          any |= x.x | x.y | x.z | x.w;
        }
        if (any) {
#pragma unroll 1
          for (int g = 0; g < NK / 32 * W; ++g) {
            const int t = (st0 + k) * NK + 32 * (g / W), left = lim - t;
            uint32_t seen = left <= 0 ? 0u : bad[g] & (left >= 32 ? 0xffffffffu : (1u << left) - 1);
#pragma unroll 1
            for (; seen; seen &= seen - 1) {
              const uint8_t *e = att_place(p, unit().b, unit().hk, t + __ffs(seen) - 1, 2 * kv4_code_bytes(D, P) + kv4_entry_bytes(D, P), W * 4);
              if (e) nan |= att_not_finite(reinterpret_cast<const uint32_t *>(e)[g % W]) ? 1u << (g % W) : 1u << 31;
            }
          }
        }
      };
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const uint32_t it = base + k, buf = it & 1;
        ok = wait_warp(&s_full[buf], (it >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sc = lane_base + S::kColS + buf * NK + wg * kHalf;
        const int t0 = (st0 + k) * NK + wg * kHalf;
        const bool cut = t0 + kHalf > lim_min;
        if (__builtin_expect(s_some[it & 3] != 0, 0))
          tc_new_scores<D>(p, unit(), s_keys[it & 3] + wg * (kHalf / 32), t0, f, sc);
        float x = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < kHalf / 32; ++q) {
          uint32_t a[32];
          tmem_ld32_async(sc + 32 * q, a);
          tmem_wait_ld();
          if (cut) {
            const int left = lim - t0 - 32 * q;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) a[e] = 0xff800000u;
          }
          float xs[4] = {x, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2) xs[(e >> 1) & 3] = max3(xs[(e >> 1) & 3], __uint_as_float(a[e]), __uint_as_float(a[e + 1]));
          x = fmaxf(max3(xs[0], xs[1], xs[2]), xs[3]);
        }
        // the row's other half, by the warp of the other group with the same rows
        s_top[buf][wg][r] = x;
        mbar_arrive(&x_full[role & 3]);
        ok = wait_warp(&x_full[role & 3], it & 1);
        if (!ok) break;
        x = fmaxf(x, s_top[buf][wg ^ 1][r]) * f;
        const bool move = x > m + 14.f;
        float a = 1.f;
        if (move) {
          const float to = fmaxf(m, x - 6.f);
          a = m == -INFINITY ? 0.f : ex2(m - to);
          m = to;
          l *= a;
        }
        if (k > 0 && __any_sync(0xffffffffu, move)) {
          // every product before this tile's is in O, half of whose columns a group
          // rescales.  (A wait names a phase by its parity, so the one before has to be
          // over: this tile's scores were let go after the product of two tiles ago.)
          ok = wait_warp(&pv_done[buf ^ 1], ((it - 1) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = wg * (D / 64); q < (wg + 1) * (D / 64); ++q) {
            uint32_t o[32];
            tmem_ld32_async(lane_base + 32 * q, o);
            tmem_wait_ld();
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * a;
            tmem_st32_async(lane_base + 32 * q, y);
          }
          tmem_wait_st();
        }
        const float r0 = m == -INFINITY ? 0.f : m;
        const F2 ff = f2(f, f), rr = f2(-r0, -r0);
        F2 ls[2] = {f2(l, 0.f), f2(0.f, 0.f)};
        // P's 16 columns of a chunk lie over scores that are read already
#pragma unroll 1
        for (int q = 0; q < kHalf / 32; ++q) {
          uint32_t b[32], w[16];
          tmem_ld32_async(sc + 32 * q, b);
          tmem_wait_ld();
          if (cut) {
            const int left = lim - t0 - 32 * q;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) b[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float pa, pb;
            f2_get(f2_fma(f2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])), ff, rr), pa, pb);
            pa = ex2(pa), pb = ex2(pb);
            ls[e & 1] = f2_add(ls[e & 1], f2(pa, pb));
            w[e] = pack_h2(pa, pb);
          }
          tmem_st16_async(sc + 16 * q, w);
        }
        {
          float la, lb;
          f2_get(f2_add(ls[0], ls[1]), la, lb);
          l = la + lb;
        }
        // the scores of this tile were let go after the values of two tiles ago
        if (k > 1 && buf == wg) look(k - 2);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // ---- the unit's rows, or a part of them: half of the words a group -----------------
      const uint32_t last_it = base + n - 1;
      ok = wait_warp(&pv_done[last_it & 1], (last_it >> 1) & 1);  // ends after all others
      if (!ok) break;
      s_sum[wg][r] = l;
      s_nan[wg * kTcRows + r] = nan;
      mbar_arrive(&joined);
      ok = wait_warp(&joined, joins++ & 1);
      if (!ok) break;
      tc_fence_after();
      nan |= s_nan[(wg ^ 1) * kTcRows + r];
      if (n > 1) look(n - 2);  // neither group has looked at these two
      look(n - 1);
      l += s_sum[wg ^ 1][r];
      const bool whole = st0 == 0 && n == unit().stages;
      if (__any_sync(0xffffffffu, nan >> 31)) {
        tc_add_values<D>(p, unit(), st0 * NK, min(unit().st1 * NK, tile_lim), m, !whole);
        nan &= 0x7fffffffu;
      }
      if (whole) {
        const float v = l > 0.f ? 1.f / l : l;  // no key: 0; NaN stays
        uint16_t *dst = p.out + (size_t(tok) * p.g.H_q + head) * D;
#pragma unroll 1
        for (int w = wg * (kWords / 2); w < (wg + 1) * (kWords / 2); w += 4) {  // 4 words of 8 channels
          float y[8][4];
#pragma unroll
          for (int e = 0; e < 8; ++e) tmem_ld4_async(lane_base + e * kWords + w, y[e]);
          tmem_wait_ld();
          if (nan)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (nan >> (k % W) & 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e][k] = __uint_as_float(0x7fc00000u);
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
      } else {
        // A part of 32-row blocks that hold rows; then the parts are joined kTcJoin
        // at a time by the CTA that brings the last of them, and what comes of that,
        // in the place of the first, once more.  The order of a sum does not depend
        // on who joins.
        const int c_first = cta_of(unit().first + kTcUnitCost);
        const int c_last = cta_of(unit().first + unit().stages + kTcUnitCost - 1);
        const int rows = min(TT, unit().span - unit().tile * TT) * G, blocks = (rows + 31) >> 5;
        auto part_of = [&](int k) -> float * { return parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * tc_part_floats<D>(); };
        if (r < blocks * 32) {
          float *part = part_of(c) + r;
#pragma unroll 1
          for (int q = wg * (D / 64); q < (wg + 1) * (D / 64); ++q) {
            uint32_t o[32];
            tmem_ld32_async(lane_base + 32 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              part[size_t(32 * q + e) * kTcRows] = nan >> ((32 * q + e) % kWords % W) & 1 ? __uint_as_float(0x7fc00000u) : __uint_as_float(o[e]);
          }
          if (wg == 0) part[size_t(D) * kTcRows] = m, part[size_t(D + 1) * kTcRows] = l;
        }
        // a warp: one block of rows, the words from w0
        const int splits = blocks == 1 ? 8 : blocks == 2 ? 4 : 2, words = kWords / splits;
        const int jr = role / splits * 32 + lane, w0 = role % splits * words;
        const int ji = unit().tile * TT + jr / G;
        const bool there = jr < blocks * 32;
        uint16_t *dst = p.out + (size_t(unit().start + ji) * p.g.H_q + unit().hk * G + jr % G) * D;
        int from = c - (c - c_first) % kTcJoin, step = 1, some = min(kTcJoin, c_last + 1 - from);
        uint32_t *count = counters + 256 + 2 * from + (from == c_first);
        if (c_last - c_first < kTcJoin) count = counters + c_first;
#pragma unroll 1
        for (;;) {
          __threadfence();
          mbar_arrive(&joined);
          ok = wait_warp(&joined, joins++ & 1);
          if (!ok) break;
          if (rtid == 0) {
            const uint32_t done = atomicAdd(count, 1u) + 1u;
            s_flag = done == uint32_t(some);
            if (done == uint32_t(some)) *count = 0;  // ready for the next call
            __threadfence();
          }
          __syncwarp();
          mbar_arrive(&joined);
          ok = wait_warp(&joined, joins++ & 1);
          if (!ok || *reinterpret_cast<volatile int *>(&s_flag) == 0) break;
          const bool final = count == counters + c_first;
          // weights of the parts against the common maximum, by the block's first warp
          float M = -INFINITY, L = 0.f;
          if (there && w0 == 0) {
#pragma unroll 4
            for (int k = 0; k < some; ++k) M = fmaxf(M, __ldcg(part_of(from + k * step) + size_t(D) * kTcRows + jr));
#pragma unroll 4
            for (int k = 0; k < some; ++k) {
              const float *src = part_of(from + k * step) + size_t(D) * kTcRows + jr;
              const float mk = __ldcg(src), lk = __ldcg(src + kTcRows);
              const float ck = lk != lk ? 1.f : mk == -INFINITY ? 0.f : ex2(mk - M);
              s_w[k][jr] = ck;
              L = fmaf(lk, ck, L);
            }
            s_sum[0][jr] = L;
          }
          mbar_arrive(&joined);
          ok = wait_warp(&joined, joins++ & 1);
          if (!ok) break;
          if (there) {
            const float Ls = s_sum[0][jr], v = Ls > 0.f ? 1.f / Ls : Ls;  // no key: 0; NaN stays
#pragma unroll 1
            for (int w = w0; w < w0 + words; ++w) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll 1
              for (int k = 0; k < some; k += 4) {  // 4 parts' loads on their way
                float x[4][8];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                  const float *src = part_of(from + (k + f) * step) + jr;
#pragma unroll
                  for (int e = 0; e < 8; ++e) x[f][e] = k + f < some ? __ldcg(src + size_t(e * kWords + w) * kTcRows) : 0.f;
                }
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                  const float ck = k + f < some ? s_w[k + f][jr] : 0.f;
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = fmaf(x[f][e], ck, y[e]);
                }
              }
              if (!final) {
                float *part = part_of(from) + jr;
#pragma unroll
                for (int e = 0; e < 8; ++e) part[size_t(e * kWords + w) * kTcRows] = y[e];
              } else if (jr < rows) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * e] * v, y[2 * e + 1] * v);
                  h[e] = *reinterpret_cast<const uint32_t *>(&b2);
                }
                *reinterpret_cast<uint4 *>(dst + 8 * w) = make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
          }
          if (final) break;
          mbar_arrive(&joined);  // every warp has read the parts' maxima and sums
          ok = wait_warp(&joined, joins++ & 1);
          if (!ok) break;
          if (there && w0 == 0) {
            float *part = part_of(from) + jr;
            part[size_t(D) * kTcRows] = M, part[size_t(D + 1) * kTcRows] = L;
          }
          from = c_first, step = kTcJoin, some = (c_last - c_first) / kTcJoin + 1;
          count = counters + c_first;
        }
        if (!ok) break;
      }
      base += n;
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (role == 16) tmem_dealloc(s_tmem, S::kCols);
}

template <int D>
inline size_t att_tc_ws(int ctas) {
  return 4096 + sizeof(float) * 2 * size_t(ctas) * tc_part_floats<D>();
}

template <int D>
cudaError_t launch_att_tc(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  static std::atomic<bool> configured[64];
  const cudaError_t e = att_configure(reinterpret_cast<const void *>(kv4_attend_tc<D>), TcShape<D>::kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl_smem(kv4_attend_tc<D>, dim3(ctas), dim3(kTcThreads), TcShape<D>::kSmem, s, p);
}

cudaError_t launch_att_tc_64(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_tc_128(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_tc_256(const Kv4AttendParams &p, int ctas, cudaStream_t s);

}  // namespace gdn

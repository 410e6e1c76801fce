// kv4_attend.cuh -- causal attention of a few query rows over the paged 4-bit
// cache: one pass over the keys, the codes as matrix operands.
//
// A unit is (row b, kv head, tile of 8 query rows); a query row is one
// (token, head of the group), so the group's heads and a row's draft positions
// share every byte that is read.  A warp takes stages of ST keys:
//   scores   mma m16n8k16 (fp16, fp32 accumulators) of Q with the keys' codes.
//            A code is put into a 16-bit operand by one AND: the bits 0..15 of
//            the pattern 0x000f are the fp16 subnormal code * 2^-24, those of
//            0x00f0 are 16 * code * 2^-24 (q is divided by 16 there).  Nothing
//            is rounded.  Step and base enter in fp32 afterwards:
//            s = sum_g step_g (q_g . code_g) + base_g sum(q_g).
//   softmax  running maximum and sum in fp32; the reference only moves when a
//            probability passes 2^14, so the accumulators are rarely rescaled.
//   output   mma of P with the values in fp16, each rounded once: a code comes
//            out exactly (1024 + code, less 1024, or 1024 + 16 code, / 16 - 64),
//            then base + step * code in one fused multiply-add; P is rounded
//            once to fp16, at most 2^14 and exact to 2^-11 down to 2^-20 of
//            the largest.  The values are the first operand and P the second, so that
//            the eight rows fill a product.
// q is scaled per row by a power of two before fp16, exactly.
//
// What bounds it: the instructions that unpack 2 x D codes a token, before HBM (144
// bytes a token and head pair at D = 128): 1740 a warp and 64 keys, at 56 % of the
// issue slots, with the halved rate of the logic instructions behind most stalls;
// hence the AND-only unpacking of the keys, packed fp32 arithmetic and as many
// warps as the registers allow.  Where the keys are few it is latency: 3 us until
// the line is cut, 2 to the first keys, 5 to 8 for the joins.
// 59 ragged rows of up to 8192 keys, 32 heads over 8 of 128: 109 us, 3.3 TB/s of the
// cache's bytes; one row of 131001 keys: 54.5 us, 2.8 TB/s.
//
// The keys' stages of all units form one line, which the warps of a persistent
// grid (one CTA an SM) cut into equal pieces, each with its own ring of bulk
// copies that runs ahead into the next unit: a short unit costs its warp a load
// of queries and a store, and nobody else waits.  A unit cut between warps is
// joined at the end, in shared memory among the warps of a CTA, and by
// whichever CTA finishes last among several, in the order of the pieces, so the
// result does not depend on timing.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "kv4.cuh"

namespace gdn {

constexpr int kAttRows = 8;  // query rows of a unit

template <int D>
struct AttShape {
  static constexpr int W = D / 64;               // groups of a head
  static constexpr int ST = D == 256 ? 32 : 64;  // keys of a stage: what a copy brings
  // Keys, and key tiles, taken at a time.  64 at D = 128 spill heavily with 12 warps
  // (ragged rows below: 117 us for 106); 16 at D = 256: 95.8 us for 71.9.
  static constexpr int CK = D == 64 ? 64 : 32, NT = CK / 8;
  // Warps of a CTA, as the registers of a thread allow, and a multiple of 4 (the compiler
  // spills 96 bytes a thread at D = 256 with 8, 8 at D = 128 with 12, none at D = 64).  48
  // rows of 8000 keys at D = 256: 82.5 us with 12, which spill more, 100 with 9, 71.9 with
  // 8, 73.9 with 7; 64 ragged rows of 8192 at D = 128: 106 with 12, 119 with 10, 114 with
  // 8; at D = 64, 16 rows of 2000: 15.9 with 12, 17.6 with 16 (and 38.8, 39.1 for 48 rows
  // of 16000).
  static constexpr int NW = D == 256 ? 8 : 12;
  static constexpr int kThreads = 32 * NW;
  static constexpr int kCodes = ST * D / 2, kEntries = ST * W * 4;
  static constexpr int kStage = 2 * (kCodes + kEntries);
  static constexpr int kSlots = (224 * 1024 / kStage) / NW;  // stages of a warp's ring
  static constexpr int kRegs = D / 4;            // accumulators of a lane: channel tiles x 2 rows
  static constexpr int kPart = kRegs * 32;       // floats of a part: outputs [accumulator][lane]
  static constexpr int kPartAll = kPart + 2 * kAttRows;  // a CTA's part in the workspace: with the rows' maxima and sums
  static constexpr int kRing = kSlots * kStage;
  static constexpr int kSmem = NW * kRing + 128;
  static_assert(kSlots >= 2, "ring");
  // accumulator of channel tile t (channels 8 g + e: t = 8 g + e), row 2 j + x:
  // two tiles a product
  static __host__ __device__ constexpr int reg(int t, int x) { return (t >> 1) * 4 + 2 * (t & 1) + x; }
};

// CTAs of the persistent grids at most: the workspace has room for the parts of
// so many, on whichever device it is used.
constexpr int kAttMaxCtas = 160;

// Least factor of a score: 0 would make NaN of a masked key's -infinity; with this one
// every score that the products can give is as good as 0.
constexpr float kLeastFactor = 1.17549435e-38f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
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

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w))); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w >> 16))); }

// The key of column c of an 8-key tile: 0 1 3 2 4 5 7 6, so that the two keys
// of a lane differ in the parity of their place (shared-memory banks).
__device__ __forceinline__ int att_key(int c) { return c ^ ((c >> 1) & 1); }

// As mbar_wait_spin, kept small: the roles wait in many places.
__device__ __forceinline__ bool att_wait(uint64_t *bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i) {
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

// The rest of a wait that did not end at once.  One that runs out is reported and begun
// once more: what it waits for is a copy into memory that is given up afterwards.
static __device__ __noinline__ bool att_wait_slow(uint64_t *bar, uint32_t parity, uint32_t *status, uint32_t limit) {
  if (att_wait(bar, parity, limit)) return true;
  atomicOr(status, GDN_STATUS_TIMEOUT);
  att_wait(bar, parity, limit);
  return false;
}

// W consecutive 32-bit words of shared memory.
template <int W>
__device__ __forceinline__ void att_words(uint32_t (&w)[W], const uint8_t *p) {
  if (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x, w[1 % W] = x.y, w[2 % W] = x.z, w[3 % W] = x.w;
  } else if (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x, w[1 % W] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

__device__ __forceinline__ bool att_not_finite(uint32_t entry) {
  return (entry & 0x7c00u) == 0x7c00u || (entry & 0x7c000000u) == 0x7c000000u;
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// base + step * code of the codes in bits 0..3 (even) or 4..7 (odd) of both halves.
__device__ __forceinline__ uint32_t att_even(uint32_t x, uint32_t step, uint32_t base) {
  return h2_fma(h2_add((x & 0x000f000fu) | 0x64006400u, 0xe400e400u), step, base);
}
__device__ __forceinline__ uint32_t att_odd(uint32_t x, uint32_t step, uint32_t base) {
  return h2_fma(h2_fma((x & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd400d400u), step, base);
}

// Wide groups.  A step and a base are finite fp16 numbers, but the levels base + step *
// code lie anywhere up to 16 * 65504, and one that passes fp16 would enter a product as
// an infinity, which even a query that does not see the key would meet, as 0 * infinity.
// So every entry's top level is formed (one product and sum for two entries), and the
// groups that do not fit in fp16 go another way.  Ordinary caches pay 2 % for it on the
// tensor cores and 2 to 3 % with few rows (64 ragged rows of 8192 keys at D = 128: 105.3
// us without the look, 108.9 with it).
constexpr uint32_t kH2Fifteen = 0x4b804b80u, kH2Sixteenth = 0x2c002c00u;

// `nil` with the top levels of two entries looked at: what is not 0 (signs aside) in the
// end tells that one of them is wide, or not finite.
__device__ __forceinline__ uint32_t att_look(uint32_t steps, uint32_t bases, uint32_t nil) {
  return h2_fma(h2_fma(steps, kH2Fifteen, bases), 0u, nil);  // an infinity or NaN leaves a NaN
}
__device__ __forceinline__ bool att_found(uint32_t nil) { return (nil & 0x7fff7fffu) != 0; }

// The entry is wide, or not finite.
__device__ __forceinline__ bool att_not_fp16(uint32_t entry) {
  return att_found(att_look(__byte_perm(entry, entry, 0x1010), __byte_perm(entry, entry, 0x3232), 0u));
}
__device__ __forceinline__ bool att_wide(uint32_t entry) { return att_not_fp16(entry) && !att_not_finite(entry); }

// Where the cache holds token t of row b for head hk, the record's part `off` bytes from
// its start with `bytes` bytes a token; NULL where the page is outside the cache.  t is
// less than the row's length.
__device__ __forceinline__ const uint8_t *att_place(const Kv4AttendParams &p, int b, int hk, int t, int off, int bytes) {
  const int page = p.table[size_t(b) * p.g.max_pages + (t >> p.g.log2P)];
  if (page < 0 || page >= p.g.n_pages) return nullptr;
  return p.pages + (size_t(page) * p.g.H_kv + hk) * kv4_record_bytes(p.g.D, 1 << p.g.log2P) + off +
         (t & ((1 << p.g.log2P) - 1)) * bytes;
}

// q . k of token t in fp32.  Few tokens of few caches come here, so it is kept short, not
// fast.
template <int D>
static __device__ __noinline__ float att_dot(const Kv4AttendParams &p, int b, int hk, int t, const uint16_t *q) {
  constexpr int W = D / 64;
  const int P = 1 << p.g.log2P;
  const uint8_t *codes = att_place(p, b, hk, t, 0, D / 2), *entries = att_place(p, b, hk, t, 2 * kv4_code_bytes(D, P), W * 4);
  if (!codes) return 0.f;
  float sum = 0.f;
#pragma unroll 1
  for (int w = 0; w < D / 8; ++w) {
    const uint32_t e = reinterpret_cast<const uint32_t *>(entries)[w % W];
    const uint32_t c = reinterpret_cast<const uint32_t *>(codes)[w];
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      sum = fmaf(__uint_as_float(uint32_t(q[8 * w + i]) << 16), fmaf(half_lo(e), float(c >> (4 * i) & 15u), half_hi(e)), sum);
  }
  return sum;
}

// One row's part of the line of stages.
struct AttRow {
  int start, span, count, len;  // tokens of its span, queries, cached tokens
  int tiles, stages;            // query tiles; stages of each
};

template <int D>
__device__ __forceinline__ AttRow att_row(const Kv4AttendParams &p, int b, bool report) {
  AttRow r;
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
  const int G = p.g.H_q / p.g.H_kv;
  r.tiles = int(((long long)span * G + kAttRows - 1) / kAttRows);
  r.stages = count > 0 ? max(1, (r.len + AttShape<D>::ST - 1) / AttShape<D>::ST) : 1;
  return r;
}

// Exclusive prefix of v over a CTA of NW warps, and the sum.
template <int NW>
__device__ __forceinline__ long long att_scan(long long v, long long *s_warp, long long *sum) {
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
  long long before = lane < warp ? s_warp[lane] : 0, all = lane < NW ? s_warp[lane] : 0;
#pragma unroll 1
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  *sum = all;
  return before + x - v;
}

// A unit, or the part of one that a warp has: stages [st0, st1) of `stages`, of
// which those below st_hi hold keys that a query sees.  On the line a unit is
// one place (queries in, outputs out: about half a stage's time) and then two
// places a stage; a stage belongs to the piece that holds its first.  A unit of
// kAttUncut stages or fewer is not cut: it belongs to the piece that holds its
// first place, whole (40 rows of 100 keys at D = 64: 12.0 us, cut at every stage
// 16.2; 64 of 300: 17.7, uncut up to 8 stages 19.3).
constexpr int kAttUncut = 4;

struct AttPiece {
  int b, hk, tile, st0, st1, stages, st_hi, lim_max;
  int more;         // the warp has another piece
  long long first;  // the unit's first place
  AttRow row;
};

// What the join needs in shared memory; it lies in the first warp's ring, behind
// that warp's part.
template <int D>
struct AttJoin {
  static constexpr int NW = AttShape<D>::NW;
  const float *src[2 * NW];              // the warps' parts, those of entry e from at[e] on
  float c[2 * NW][kAttRows];             // their weights
  int at[NW + 2], whole[NW + 1], n;      // entries: parts, nothing of it elsewhere; how many
  const AttPiece *piece[NW + 1];
  float max[NW + 1][kAttRows], sum[NW + 1][kAttRows];
  float w[16][kAttRows], lw[16][kAttRows], old[kAttRows];  // weights, and weighted sums, of 16 CTAs' parts
};

template <int D>
__global__ void __launch_bounds__(AttShape<D>::kThreads, 1) kv4_attend_mma(const __grid_constant__ Kv4AttendParams p) {
  using S = AttShape<D>;
  constexpr int W = S::W, ST = S::ST, NT = S::NT, NW = S::NW;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[NW][S::kSlots];
  __shared__ AttPiece s_piece[NW][2], s_cut[2][NW];  // current and next pieces; cut pieces (0: begun before the warp's)
  __shared__ int s_has[2][NW];                       // 1: a cut piece's part is in the ring, 2: in the workspace
  __shared__ int s_none[NW];                         // the warp has no stage at all
  __shared__ float s_m[2][NW][kAttRows], s_l[2][NW][kAttRows];
  __shared__ long long s_warp[NW];
  __shared__ int s_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = lane >> 2, j = lane & 3;
  const int G = p.g.H_q / p.g.H_kv, Hkv = p.g.H_kv;
  const int P = 1 << p.g.log2P;
  if (lane == 0) {
    for (int i = 0; i < S::kSlots; ++i) mbar_init(&s_full[warp][i], 1 + (blockIdx.x + warp + i == 0 ? p.test_hold : 0u));
    s_has[0][warp] = s_has[1][warp] = 0;
  }
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();

  // ---- the line, and this CTA's pieces of it ------------------------------------------
  // rows beyond the CTA's threads are summed first and looked at again below
  auto places = [&](const AttRow &r) -> long long { return (long long)r.tiles * (2 * r.stages + 1) * Hkv; };
  long long mine = 0, total, before = 0;
  AttRow own{};
  for (int b = tid; b < p.g.B; b += S::kThreads) {
    const AttRow r = att_row<D>(p, b, blockIdx.x == 0);
    if (b == tid) own = r;
    mine += places(r);
  }
  before = att_scan<NW>(mine, s_warp, &total);
  if (total == 0) return;
  // a warp wants a stage at least (16 rows of 2000 keys at D = 128: 20.4 us, with two
  // stages 24.6)
  const int ctas = int(min((long long)gridDim.x, (total + 3 * NW - 1) / (3 * NW)));
  const int c = blockIdx.x;
  if (c >= ctas) return;
  // pieces of `per` places, the first `plus` of one more
  const long long per = total < (1ll << 31) ? int(total) / (ctas * NW) : total / (ctas * NW);
  const int plus = int(total - per * (ctas * NW));
  auto start_of = [&](int w) -> long long { return per * w + min(w, plus); };  // of a warp of the grid
  auto cta_of = [&](long long x) -> int {
    const long long y = x - plus * (per + 1);
    if (x < (1ll << 31)) return (y < 0 ? int(x) / int(per + 1) : plus + int(y) / int(per)) / NW;
    return int(y < 0 ? x / (per + 1) : plus + y / per) / NW;
  };
  const long long stop = start_of(c * NW + warp + 1);
  // a piece from place x on, x in the unit, of the warp whose places end at `to`
  auto close = [&](AttPiece &u, long long x, long long to) {
    u.stages = u.row.stages;
    u.st0 = int(min((long long)u.stages, (x - u.first) >> 1));
    u.st1 = int(min((long long)u.stages, (to - u.first) >> 1));
    if (u.stages <= kAttUncut) u.st0 = x > u.first ? u.stages : 0, u.st1 = u.stages;
    const int first = u.tile * kAttRows / G;
    const int last = min(((u.tile + 1) * kAttRows - 1) / G, u.row.count - 1);
    u.lim_max = last >= first ? max(0, u.row.len - u.row.count + last + 1) : 0;
    u.st_hi = min(u.st1, (u.lim_max + ST - 1) / ST);
  };
  // the row that holds each warp's first place, by that row's thread
  long long before0 = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.g.B; b0 += S::kThreads) {
    if (p.g.B > S::kThreads) {
      if (b0 + tid < p.g.B) own = att_row<D>(p, b0 + tid, false);
      else own.tiles = 0;
      long long sum;
      before = before0 + att_scan<NW>(places(own), s_warp, &sum);
      before0 += sum;
    }
    const long long end = before + places(own);
#pragma unroll 1
    for (int w = 0; w < NW; ++w) {
      const long long x = start_of(c * NW + w);
      if (x >= before && x < end) s_piece[w][0].b = b0 + tid, s_piece[w][0].first = before, s_piece[w][0].row = own;
    }
  }
  __syncthreads();

  uint8_t *ring = smem + warp * S::kRing;
  float *parts = reinterpret_cast<float *>(static_cast<char *>(p.ws) + 4096);
  float *stash = parts + 2 * size_t(gridDim.x) * S::kPartAll + (size_t(c) * NW) * S::kPart;
  uint32_t *counters = reinterpret_cast<uint32_t *>(p.ws);
  uint32_t phases = 0;      // parity of each ring slot
  int slot = 0, in = 0;     // next slot to read and to fill
  bool dead = false;        // a copy never came: nothing more is issued
  AttPiece *pieces = s_piece[warp];

  // the first piece with a stage from u on; without a stage if there is none
  auto seek = [&](AttPiece u) -> AttPiece {
    while (u.st0 >= u.st1) {
      const long long x = u.first + 2 * u.row.stages + 1;
      if (x >= stop) break;
      if (++u.tile == u.row.tiles) {
        u.tile = 0;
        if (++u.hk == Hkv) {
          u.hk = 0;
          do u.row = att_row<D>(p, ++u.b, false);
          while (u.row.tiles == 0);
        }
      }
      u.first = x;
      close(u, x, stop);
    }
    return u;
  };
  // the piece behind u, into `to`; marks u as followed
  auto follow = [&](AttPiece &u, AttPiece &to) {
    AttPiece v = u;
    v.st0 = v.st1;  // done with
    v = seek(v);
    u.more = v.st0 < v.st1;
    if (u.more) to = v;
  };
  if (lane == 0) {
    AttPiece u = pieces[0];
    const long long x = start_of(c * NW + warp);
    if (x < stop) {
      const int len = 2 * u.row.stages + 1;  // a unit's places
      const int k = x - u.first < (1ll << 31) ? int(x - u.first) / len : int((x - u.first) / len);
      u.first += (long long)k * len;
      u.hk = k / u.row.tiles, u.tile = k - u.hk * u.row.tiles;
      close(u, x, stop);
      u = seek(u);
    } else {
      u.st0 = u.st1 = u.st_hi = 0;  // no place at all
    }
    pieces[0] = u;
    s_none[warp] = u.st0 >= u.st1;
  }
  __syncwarp();

  // ---- copies: a page is one copy, as it lies in memory (copies are taken one in
  // about 70 cycles whatever their size); half of a page is four pieces ---------------
  const bool half_page = P > ST;
  const int n_sub = half_page ? 4 : ST >> p.g.log2P;
  const uint32_t rec_bytes = kv4_record_bytes(D, P);
  // Table cells of the stages ahead, a lane a cell: `look` loads those of kBatch
  // stages from `st` on, so that a stage costs no round trip to the table.
  const int n_cells = half_page ? 1 : n_sub;  // cells of a stage
  constexpr int kBatch = 32 * 16 / ST > 32 ? 32 : 32 * 16 / ST;  // stages whose cells 32 lanes hold at any page size
  int cells = -2, cells_st = 0;               // the lane's cell, the first stage they are of
  auto look = [&](const AttPiece &u, int st) {
    const int k = lane / n_cells, t = (st + k) * ST + ((lane - k * n_cells) << p.g.log2P);
    cells_st = st;
    // (-2: there is no such cell; a negative one of the table is -1)
    cells = k < kBatch && st + k < u.st_hi && t < u.lim_max ? max(-1, p.table[size_t(u.b) * p.g.max_pages + (t >> p.g.log2P)]) : -2;
  };
  auto issue = [&](const AttPiece &u, int st) {
    const int k = (st - cells_st) * n_cells + (half_page ? 0 : lane);
    int page = __shfl_sync(0xffffffffu, cells, k & 31);
    if (lane >= n_sub) page = -2;
    bool ok = page != -2;
    if (ok && (page < 0 || page >= p.g.n_pages)) {
      ok = false;
      atomicOr(p.status, GDN_STATUS_BAD_INDEX);
    }
    const uint32_t pages = __popc(__ballot_sync(0xffffffffu, ok));
    uint64_t *bar = &s_full[warp][in];
    if (lane == 0) mbar_arrive_expect_tx(bar, half_page ? (pages ? uint32_t(S::kStage) : 0u) : pages * rec_bytes);
    __syncwarp();
    if (ok) {
      const uint8_t *rec = p.pages + (size_t(page) * Hkv + u.hk) * rec_bytes;
      uint8_t *dst = ring + in * S::kStage;
      if (half_page) {  // K, V codes, K, V entries by lanes 0 .. 3
        const int off = (st * ST) & (P - 1);
        const bool codes = lane < 2, second = lane & 1;
        bulk_g2s(dst + (codes ? second * S::kCodes : 2 * S::kCodes + second * S::kEntries),
                 rec + (codes ? second * kv4_code_bytes(D, P) + off * (D / 2)
                              : 2 * kv4_code_bytes(D, P) + second * kv4_entry_bytes(D, P) + off * W * 4),
                 codes ? S::kCodes : S::kEntries, bar);
      } else {
        bulk_g2s(dst + lane * rec_bytes, rec, rec_bytes, bar);
      }
    }
    in = in + 1 == S::kSlots ? 0 : in + 1;
  };
  // places of a stage's keys: records of `pt` keys (a page, or the half of one);
  // 16 keys always lie in one
  const int log2pt = min(p.g.log2P, ST == 32 ? 5 : 6), pt = 1 << log2pt;
  const int rec_c = pt * (D / 2), rec_e = pt * (W * 4), rec_s = 2 * (rec_c + rec_e);
  const uint32_t lane_k = att_key(n) * (D / 2) + (D == 64 ? 8 : 16) * j;  // the lane's key of 8, its words
  const uint32_t lane_v0 = att_key(2 * j) * (D / 2) + n * (4 * W), lane_v1 = att_key(2 * j + 1) * (D / 2) + n * (4 * W);
  const uint32_t lane_e0 = att_key(2 * j) * (4 * W), lane_e1 = att_key(2 * j + 1) * (4 * W);

  // the piece whose stages are being issued: the current one or the one behind it
  int ahead = 0, issued = pieces[0].st0;
  int flight = 0;     // stages issued and not read yet
  uint32_t turn = 0;  // pieces[turn & 1] is the current piece
  look(pieces[0], issued);
  auto refill = [&](bool go_on) {
#pragma unroll 1
    while (flight < S::kSlots && !dead) {
      if (issued < pieces[ahead].st_hi) {
        if (issued - cells_st >= kBatch) look(pieces[ahead], issued);
        issue(pieces[ahead], issued);
        ++issued, ++flight;
      } else if (go_on && ahead == int(turn & 1) && pieces[ahead].more) {  // on into the next piece
        ahead ^= 1, issued = pieces[ahead].st0;
        look(pieces[ahead], issued);
      } else {
        break;
      }
    }
  };

#pragma unroll 1
  for (bool any = !s_none[warp]; any; any = pieces[turn & 1].more != 0, ++turn) {
    // (the loop's step reads `more` of the piece that is done)
    const AttPiece &cur = pieces[turn & 1];
    const int lim_max = cur.lim_max, st_hi = cur.st_hi, st_first = cur.st0;
    refill(false);
    // ---- the tile's queries: row n of a lane -------------------------------------------
    const AttRow row = cur.row;
    const int rn = cur.tile * kAttRows + n, at = rn / G;
    const bool inside = at < row.span, live = inside && at < row.count;
    // keys that the row's query sees; rows past the span follow the others
    const int lim = live ? max(0, row.len - row.count + at + 1) : inside ? 0 : lim_max;
    const int lim_min = __reduce_min_sync(0xffffffffu, lim);

    // ---- Q as fp16 fragments, scaled by a power of two per row -------------------------
    uint32_t qa[D / 16][2];  // columns 0-7, then 8-15
    float qs[W];
    float f = fabsf(p.scale) * 1.4426950408889634f * 16777216.f;  // 2^24 of the subnormal codes
    // the factor of a score is kept positive: the maximum is taken before it
    const float sign = p.scale > 0.f ? 1.f : p.scale < 0.f ? -1.f : 0.f;
    if (p.scale == 0.f) f = 1.f;
    {
      const uint16_t *src = p.q + (size_t(live ? row.start + at : 0) * p.g.H_q + (live ? cur.hk * G + rn - at * G : 0)) * D;
      uint4 raw[D / 32];
      uint32_t mx = 0;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // word w of the lane: the channels of the keys' words below
        const int ch = D == 64 ? 16 * j + 8 * w : 128 * (w >> 2) + 32 * j + 8 * (w & 3);
        raw[w] = live ? *reinterpret_cast<const uint4 *>(src + ch) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)  // the largest of both halves of a word: as unsigned pairs, signs away
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(raw[w].x & 0x7fff7fffu, raw[w].y & 0x7fff7fffu),
                                   __vmaxu2(raw[w].z & 0x7fff7fffu, raw[w].w & 0x7fff7fffu)));
      mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // the largest magnitude goes to [2^10, 2^11)
      const int e = min(max(int(mx >> 7), 20), 240);
      const float s2 = __uint_as_float(uint32_t(264 - e) << 23), up = s2 * sign;
      f = fmaxf(f * (1.f / s2), kLeastFactor);
#pragma unroll
      for (int g = 0; g < W; ++g) qs[g] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float x[8];
        const uint32_t a[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[2 * k] = __uint_as_float(a[k] << 16) * up, x[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u) * up;
#pragma unroll
        for (int k = 0; k < 8; ++k) qs[w % W] += x[k];
        // step 2w: columns (0, 4) and (1, 5) / 16; step 2w + 1: (2, 6) and (3, 7) / 16
        qa[2 * w][0] = pack_h2(x[0], x[4]), qa[2 * w][1] = pack_h2(x[1] * 0.0625f, x[5] * 0.0625f);
        qa[2 * w + 1][0] = pack_h2(x[2], x[6]), qa[2 * w + 1][1] = pack_h2(x[3] * 0.0625f, x[7] * 0.0625f);
      }
#pragma unroll
      for (int g = 0; g < W; ++g) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], o);
        qs[g] *= 5.9604644775390625e-08f;  // 2^-24, as the codes
      }
    }

    float o_acc[S::kRegs / 4][4];
#pragma unroll
    for (int i = 0; i < S::kRegs / 4; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.f;
    __syncwarp();  // every lane is done with the piece before
    if (lane == 0) follow(pieces[turn & 1], pieces[(turn & 1) ^ 1]);
    __syncwarp();
    uint32_t nan = 0;  // groups in which the row has seen a value that is not finite
    float m = -INFINITY;
    F2 l2 = f2(0.f, 0.f);

#pragma unroll 1
    for (int st = st_first; st < st_hi; ++st) {
      if (flight > 0) {  // once a wait has run out nothing more is issued, and what is in flight still waited for
        --flight;
        if (!mbar_try_wait(&s_full[warp][slot], (phases >> slot) & 1))
          dead = !att_wait_slow(&s_full[warp][slot], (phases >> slot) & 1, p.status, p.wait_limit) || dead;
        dead = __any_sync(0xffffffffu, dead);
        phases ^= 1u << slot;
      }
      // ---- wide groups among the stage's keys (1) and values (2): a lane has kOwn of the
      // entries of each -----------------------------------------------------------------
      uint32_t wide;
      {
        constexpr int kOwn = ST * W / 32;
        const int key = lane * kOwn / W, off = key & (pt - 1);
        const uint8_t *at = ring + slot * S::kStage + (key >> log2pt) * rec_s + 2 * rec_c + off * (W * 4);
        uint32_t ke[kOwn], ve[kOwn], kn = 0, vn = 0;
        att_words<kOwn>(ke, at), att_words<kOwn>(ve, at + rec_e);
        if (st * ST + ST > lim_max) {  // places behind the last key hold anything
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            if (st * ST + key + i / W >= lim_max) ke[i] = ve[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < kOwn; i += 2) {
          kn = att_look(__byte_perm(ke[i], ke[i + 1], 0x5410), __byte_perm(ke[i], ke[i + 1], 0x7632), kn);
          vn = att_look(__byte_perm(ve[i], ve[i + 1], 0x5410), __byte_perm(ve[i], ve[i + 1], 0x7632), vn);
        }
        wide = (__any_sync(0xffffffffu, att_found(kn)) ? 1u : 0u) | (__any_sync(0xffffffffu, att_found(vn)) ? 2u : 0u);
      }
#pragma unroll 1
     for (int ck = 0; ck < ST && st * ST + ck < lim_max; ck += S::CK) {
      const int t_base = st * ST + ck;
      // 16-key groups: K codes and K entries; the values' lie rec_c and rec_e behind
      const uint8_t *codes[NT / 2], *entries[NT / 2];
#pragma unroll
      for (int h = 0; h < NT / 2; ++h) {
        const int key = ck + 16 * h, off = key & (pt - 1);
        const uint8_t *rec = ring + slot * S::kStage + (key >> log2pt) * rec_s;
        codes[h] = rec + off * (D / 2), entries[h] = rec + 2 * rec_c + off * (W * 4);
      }
      const bool cut = t_base + S::CK > lim_min;  // some query does not see all of them
      const bool care = cut || wide != 0;

      // ---- scores, and their maximum ----------------------------------------------
      float s[NT][2], top = -INFINITY;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float acc[W][4];
#pragma unroll
        for (int g = 0; g < W; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
        const uint8_t *kr = codes[u / 2] + lane_k + (u & 1) * (8 * (D / 2));
        uint32_t word[D / 32];
        if (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2 *>(kr);
          word[0] = x.x, word[1] = x.y;
        } else {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kr + 64 * i);
            word[4 * i] = x.x, word[4 * i + 1] = x.y, word[4 * i + 2] = x.z, word[4 * i + 3] = x.w;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t x = word[w], y = x >> 8;
          mma16816(acc[w % W], qa[2 * w][0], 0u, qa[2 * w][1], 0u, x & 0x000f000fu, x & 0x00f000f0u);
          mma16816(acc[w % W], qa[2 * w + 1][0], 0u, qa[2 * w + 1][1], 0u, y & 0x000f000fu, y & 0x00f000f0u);
        }
        uint32_t ka[W], kb[W];
        att_words<W>(ka, entries[u / 2] + lane_e0 + (u & 1) * (32 * W));
        att_words<W>(kb, entries[u / 2] + lane_e1 + (u & 1) * (32 * W));
        F2 sum = f2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < W; ++g) {
          const F2 step = f2(half_lo(ka[g]), half_lo(kb[g])), base = f2(half_hi(ka[g]), half_hi(kb[g]));
          sum = f2_fma(base, f2(qs[g], qs[g]), f2_fma(step, f2(acc[g][0], acc[g][1]), sum));
        }
        f2_get(sum, s[u][0], s[u][1]);
        if (cut) {
          const int ta = t_base + 8 * u + att_key(2 * j), tb = t_base + 8 * u + att_key(2 * j + 1);
          if (ta >= lim) s[u][0] = -INFINITY;
          if (tb >= lim) s[u][1] = -INFINITY;
        }
        top = max3(top, s[u][0], s[u][1]);
      }
      if (__builtin_expect(wide & 1, 0)) {
        // of wide keys the two sums step * (q . code) and base * sum(q) may be so large that
        // nothing is left of their difference in fp32: those scores are formed anew
        const uint16_t *query = p.q + (size_t(row.start + at) * p.g.H_q + cur.hk * G + rn - at * G) * D;
#pragma unroll 1
        for (int i = 0; i < 2 * NT; ++i) {
          const int key = ck + 8 * (i >> 1) + att_key(2 * j + (i & 1)), t = st * ST + key;
          if (!live || t >= lim) continue;
          uint32_t e[W];
          att_words<W>(e, ring + slot * S::kStage + (key >> log2pt) * rec_s + 2 * rec_c + (key & (pt - 1)) * (W * 4));
          bool any = false;
#pragma unroll
          for (int g = 0; g < W; ++g) any = any || att_wide(e[g]);
          if (!any) continue;
          const float x = att_dot<D>(p, cur.b, cur.hk, t, query) * (p.scale * 1.4426950408889634f / f);
#pragma unroll
          for (int k = 0; k < 2 * NT; ++k)
            if (k == i) s[k >> 1][k & 1] = x;
        }
        top = -INFINITY;
#pragma unroll
        for (int u = 0; u < NT; ++u) top = max3(top, s[u][0], s[u][1]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      top *= f;
      if (__any_sync(0xffffffffu, top > m + (wide & 2 ? 10.f : 14.f))) {
        const float to = fmaxf(m, top - 6.f), a = to == m ? 1.f : ex2(m - to);
        m = to;
        l2 = f2_mul(l2, f2(a, a));
        // columns 2j, 2j + 1 are the rows
        const float ca = __shfl_sync(0xffffffffu, a, 8 * j), cb = __shfl_sync(0xffffffffu, a, 8 * j + 4);
#pragma unroll
        for (int i = 0; i < S::kRegs / 4; ++i) o_acc[i][0] *= ca, o_acc[i][1] *= cb, o_acc[i][2] *= ca, o_acc[i][3] *= cb;
      }
      float r0 = m == -INFINITY ? 0.f : -m;
      // wide values are formed as sixteenths, which always fit, and all values of their
      // stage with them (they keep 16 * 2^-25 of absolute precision): sixteen times the
      // probabilities, and the sums until the chunk's end
      if (wide & 2) r0 += 4.f, l2 = f2_mul(l2, f2(16.f, 16.f));

      // ---- probabilities and output, 16 keys at a time --------------------------------
#pragma unroll
      for (int h = 0; h < NT / 2; ++h) {
        uint32_t a[2], es[W][2], eb[W][2];  // P; (step, step), (base, base) of the key pairs
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int u = 2 * h + half;
          float pa, pb;
          f2_get(f2_fma(f2(s[u][0], s[u][1]), f2(f, f), f2(r0, r0)), pa, pb);
          pa = ex2(pa), pb = ex2(pb);
          l2 = f2_add(l2, f2(pa, pb));
          a[half] = pack_h2(pa, pb);
          const int ka = 8 * u + att_key(2 * j), kb = 8 * u + att_key(2 * j + 1);
          uint32_t wa[W], wb[W];
          att_words<W>(wa, entries[h] + rec_e + lane_e0 + half * (32 * W));
          att_words<W>(wb, entries[h] + rec_e + lane_e1 + half * (32 * W));
          if (care) {
            if (cut) {
              // a value that one query sees and another does not must not reach
              // the other as 0 * NaN: it is left out and remembered by the row
#pragma unroll
              for (int g = 0; g < W; ++g) {
                const int ta = t_base + ka, tb = t_base + kb;
                if (att_not_finite(wa[g])) nan |= uint32_t(ta < lim) << g, wa[g] = 0;
                if (att_not_finite(wb[g])) nan |= uint32_t(tb < lim) << g, wb[g] = 0;
                if (ta >= lim_max) wa[g] = 0;
                if (tb >= lim_max) wb[g] = 0;
              }
            }
            if (wide & 2) {
#pragma unroll
              for (int g = 0; g < W; ++g) wa[g] = h2_mul(wa[g], kH2Sixteenth), wb[g] = h2_mul(wb[g], kH2Sixteenth);
            }
          }
#pragma unroll
          for (int g = 0; g < W; ++g) {
            es[g][half] = __byte_perm(wa[g], wb[g], 0x5410);
            eb[g][half] = __byte_perm(wa[g], wb[g], 0x7632);
          }
        }
        uint32_t w0[W], w1[W], w2[W], w3[W];
        att_words<W>(w0, codes[h] + rec_c + lane_v0);
        att_words<W>(w1, codes[h] + rec_c + lane_v1);
        att_words<W>(w2, codes[h] + rec_c + lane_v0 + 8 * (D / 2));
        att_words<W>(w3, codes[h] + rec_c + lane_v1 + 8 * (D / 2));
#pragma unroll
        for (int g = 0; g < W; ++g) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = __byte_perm(w0[g], w1[g], half ? 0x7632 : 0x5410);
            const uint32_t y = __byte_perm(w2[g], w3[g], half ? 0x7632 : 0x5410);
            const uint32_t v00 = att_even(x, es[g][0], eb[g][0]), v01 = att_even(y, es[g][1], eb[g][1]);
            const uint32_t v10 = att_odd(x, es[g][0], eb[g][0]), v11 = att_odd(y, es[g][1], eb[g][1]);
            const uint32_t v20 = att_even(x >> 8, es[g][0], eb[g][0]), v21 = att_even(y >> 8, es[g][1], eb[g][1]);
            const uint32_t v30 = att_odd(x >> 8, es[g][0], eb[g][0]), v31 = att_odd(y >> 8, es[g][1], eb[g][1]);
            const int o = 8 * g + 4 * half;
            mma16816(o_acc[o / 2], v00, v10, v01, v11, a[0], a[1]);
            mma16816(o_acc[o / 2 + 1], v20, v30, v21, v31, a[0], a[1]);
          }
        }
      }
      if (wide & 2) l2 = f2_mul(l2, f2(0.0625f, 0.0625f));
     }
      __syncwarp();  // every lane is done with the slot
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
      refill(true);
    }
    refill(true);  // a piece without copies has not gone on yet

    // ---- the piece's outputs ---------------------------------------------------------
    float l;
    {
      float la, lb;
      f2_get(l2, la, lb);
      l = la + lb;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      nan |= __shfl_xor_sync(0xffffffffu, nan, o);
    }
    // of the rows of the lane's values: 2 j, 2 j + 1
    const uint32_t nans[2] = {__shfl_sync(0xffffffffu, nan, 8 * j), __shfl_sync(0xffffffffu, nan, 8 * j + 4)};
    const float sums[2] = {__shfl_sync(0xffffffffu, l, 8 * j), __shfl_sync(0xffffffffu, l, 8 * j + 4)};
    const bool starts = st_first == 0, ends = cur.st1 == cur.stages;
    const float none = __uint_as_float(0x7fc00000u);
    if (starts && ends) {  // the whole unit
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rr = cur.tile * kAttRows + 2 * j + x, i = rr / G;
        const float v = sums[x] > 0.f ? 1.f / sums[x] : sums[x];  // no key: 0; NaN stays
        uint16_t *dst = p.out + (size_t(cur.row.start + i) * p.g.H_q + cur.hk * G + rr - i * G) * D + n * W * 8;
        if (i < cur.row.span) {
#pragma unroll
          for (int g = 0; g < W; ++g) {
            const float w = nans[x] >> g & 1u ? none : v;
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int a = S::reg(8 * g + 2 * e, x), b = S::reg(8 * g + 2 * e + 1, x);
              const __nv_bfloat162 y = __floats2bfloat162_rn(o_acc[a / 4][a % 4] * w, o_acc[b / 4][b % 4] * w);
              h[e] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(dst + 8 * g) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
    } else {
      const int kind = starts ? 1 : 0;
      const bool stay = !cur.more;  // the ring is free after the last piece
      float *dst = stay ? reinterpret_cast<float *>(ring) : stash + size_t(warp) * S::kPart;
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = S::reg(t, x);
          dst[i * 32 + lane] = nans[x] >> (t / 8) & 1u ? none : o_acc[i / 4][i % 4];
        }
      if (j == 0) s_m[kind][warp][n] = m, s_l[kind][warp][n] = l;
      if (lane == 0) s_has[kind][warp] = stay ? 1 : 2, s_cut[kind][warp] = cur;
    }
  }

  // ---- join of the cut units: entry 0 is one begun before this CTA, the others those
  // that begin in it.  A lane is a piece, in the order of the line: of warp lane / 2,
  // the one begun before that warp and the one that begins in it. ---------------------
  AttJoin<D> &join = *reinterpret_cast<AttJoin<D> *>(smem + S::kPart * 4);
  __syncthreads();
  // a part's weight against the common maximum M; a NaN sum keeps its NaN
  auto weight = [](float m, float l, float M) { return l != l ? 1.f : m == -INFINITY ? 0.f : ex2(m - M); };
  if (warp < kAttRows) {  // a row a warp
    const int w = lane >> 1, kind = lane & 1, has = w < NW ? s_has[kind][w % NW] : 0;
    const uint32_t all = __ballot_sync(0xffffffffu, has != 0), heads = __ballot_sync(0xffffffffu, has != 0 && kind == 1);
    const uint32_t upto = 0xffffffffu >> (31 - lane), before_it = heads & upto, behind = heads & ~upto;
    const int e = __popc(before_it);  // the entry, and its lanes
    const int first = before_it ? 31 - __clz(before_it) : 0, last = behind ? __ffs(behind) - 2 : 31;
    const float m = has ? s_m[kind][w % NW][warp] : -INFINITY, l = has ? s_l[kind][w % NW][warp] : 0.f;
    float M = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, M, o);
      if (lane - o >= first) M = fmaxf(M, x);
    }
    M = __shfl_sync(0xffffffffu, M, last);
    const float cw = weight(m, l, M);
    float L = l * cw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, L, o);
      if (lane - o >= first) L += x;
    }
    const int pos = __popc(all & (upto >> 1));
    if (has) join.c[pos][warp] = cw;
    if (lane == last) join.max[e][warp] = M, join.sum[e][warp] = L;
    if (warp == 0) {
      if (has) {
        join.src[pos] = has == 1 ? reinterpret_cast<const float *>(smem + w * S::kRing) : stash + size_t(w) * S::kPart;
        if (lane == first || (e == 0 && pos == 0)) join.piece[e] = &s_cut[kind][w];
        const uint32_t rest = all & ~upto;
        if (!rest || __ffs(rest) - 1 > last)  // the entry's last piece
          join.whole[e] = e > 0 && kind == 0 && s_cut[0][w].st1 == s_cut[0][w].stages;
      }
      if (lane == last) join.at[e + 1] = pos + (has != 0);
      if (lane == 0) join.at[0] = 0, join.n = __popc(heads) + 1;
    }
  }
  __syncthreads();
  // items: the channels 8 g + e, 8 g + e + 1 of value x
  constexpr int kPairs = S::kPart / 2;
  auto place = [&](int item, int &ln, int &x, int &t, int &r, int &col) {
    ln = item & 31, x = (item >> 5) & 1, t = (item >> 6) * 2;
    r = 2 * (ln & 3) + x, col = ln >> 2;
  };
  auto put = [&](const AttPiece &u, float L, float y0, float y1, int t, int r, int col) {
    const int rr = u.tile * kAttRows + r, i = rr / G;
    if (i >= u.row.span) return;
    const float v = L > 0.f ? 1.f / L : L;
    uint16_t *dst = p.out + (size_t(u.row.start + i) * p.g.H_q + u.hk * G + rr - i * G) * D + (col * W + t / 8) * 8 + t % 8;
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(y0 * v, y1 * v);
  };
  auto part_of = [&](int k, int c_first) -> float * { return parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * S::kPartAll; };
  const int entries = join.n;
#pragma unroll 1
  for (int i = tid; i < entries * kPairs; i += S::kThreads) {
    const int e = i / kPairs, item = i % kPairs, k1 = join.at[e + 1];
    int k = join.at[e], ln, x, t, r, col;
    if (k == k1) continue;
    place(item, ln, x, t, r, col);
    const int at = S::reg(t, x) * 32 + ln;  // tile t + 1: two accumulators on
    float y0 = 0.f, y1 = 0.f;
#pragma unroll 1
    for (; k < k1; k += 4) {  // 4 parts' loads on their way
      float x0[4], x1[4], cw[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int q = k + f < k1 ? k + f : k;
        x0[f] = join.src[q][at], x1[f] = join.src[q][at + 64], cw[f] = join.c[q][r];
      }
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (k + f < k1) y0 = fmaf(x0[f], cw[f], y0), y1 = fmaf(x1[f], cw[f], y1);
    }
    if (join.whole[e]) put(*join.piece[e], join.sum[e][r], y0, y1, t, r, col);
    else *(reinterpret_cast<float2 *>(part_of(c, e > 0 ? c : -1)) + item) = make_float2(y0, y1);
  }
  // ---- units cut between CTAs: two at most -----------------------------------------------
#pragma unroll 1
  for (int e = 0; e < entries; ++e) {
    if (join.at[e] == join.at[e + 1] || join.whole[e]) continue;
    const AttPiece &u = *join.piece[e];
    if (tid < kAttRows) {
      float *part = part_of(c, e > 0 ? c : -1);
      part[S::kPart + tid] = join.max[e][tid], part[S::kPart + kAttRows + tid] = join.sum[e][tid];
    }
    const int c_first = cta_of(u.first + 1), c_last = cta_of(u.first + 2 * u.stages - 1);
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const uint32_t need = uint32_t(c_last - c_first + 1);
      const uint32_t done = atomicAdd(&counters[c_first], 1u) + 1u;
      s_flag = done == need;
      if (done == need) counters[c_first] = 0;  // ready for the next call
      __threadfence();
    }
    __syncthreads();
    if (!s_flag) continue;
    // 16 parts at a time: maxima and sums by 16 * 8 threads, then the items, whose
    // first loads are on their way meanwhile
    constexpr int kItems = (kPairs + S::kThreads - 1) / S::kThreads;
    float2 y[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) y[k] = make_float2(0.f, 0.f);
    if (tid < kAttRows) join.max[e][tid] = -INFINITY, join.sum[e][tid] = 0.f;
#pragma unroll 1
    for (int q0 = c_first; q0 <= c_last; q0 += 16) {
      const int some = min(16, c_last + 1 - q0);
      float2 v[4][kItems];
      auto load4 = [&](int q) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            const int item = k * S::kThreads + tid;
            v[f][k] = item < kPairs && q + f < some ? __ldcg(reinterpret_cast<const float2 *>(part_of(q0 + q + f, c_first)) + item)
                                                       : make_float2(0.f, 0.f);
          }
      };
      float m = -INFINITY, l = 0.f;
      if (tid < 16 * kAttRows && tid / kAttRows < some) {
        const float *src = part_of(q0 + tid / kAttRows, c_first) + S::kPart + tid % kAttRows;
        m = __ldcg(src), l = __ldcg(src + kAttRows);
      }
      load4(0);
      __syncthreads();
      if (tid < 16 * kAttRows) join.w[tid / kAttRows][tid % kAttRows] = m;
      __syncthreads();
      float M = -INFINITY;
      if (tid < 16 * kAttRows) {
        M = join.max[e][tid % kAttRows];
        for (int q = 0; q < 16; ++q) M = fmaxf(M, join.w[q][tid % kAttRows]);
      }
      __syncthreads();
      if (tid < 16 * kAttRows) {
        const float w = weight(m, l, M);
        join.w[tid / kAttRows][tid % kAttRows] = w, join.lw[tid / kAttRows][tid % kAttRows] = tid / kAttRows < some ? l * w : 0.f;
        if (tid < kAttRows) {
          const float old = join.max[e][tid];
          join.old[tid] = old == -INFINITY ? 0.f : ex2(old - M);  // of the batches before
          join.max[e][tid] = M;
        }
      }
      __syncthreads();
      if (tid < kAttRows) {
        float L = join.sum[e][tid];
        L = L != L ? L : L * join.old[tid];
        for (int q = 0; q < 16; ++q) L += join.lw[q][tid];
        join.sum[e][tid] = L;
      }
      if (q0 > c_first) {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          int ln, x, t, r, col;
          place(k * S::kThreads + tid, ln, x, t, r, col);
          const float w = join.old[r];
          y[k].x *= w, y[k].y *= w;
        }
      }
#pragma unroll 1
      for (int q = 0; q < some; q += 4) {
        if (q > 0) load4(q);
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            int ln, x, t, r, col;
            place(k * S::kThreads + tid, ln, x, t, r, col);
            const float w = q + f < some ? join.w[q + f][r] : 0.f;
            y[k].x = fmaf(v[f][k].x, w, y[k].x), y[k].y = fmaf(v[f][k].y, w, y[k].y);
          }
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int item = k * S::kThreads + tid;
      if (item < kPairs) {
        int ln, x, t, r, col;
        place(item, ln, x, t, r, col);
        put(u, join.sum[e][r], y[k].x, y[k].y, t, r, col);
      }
    }
  }
}

template <int D>
inline size_t att_mma_ws(int ctas) {
  // counters; two parts a CTA; what a warp puts aside while its ring goes on
  return 4096 + sizeof(float) * size_t(ctas) * (2 * AttShape<D>::kPartAll + AttShape<D>::NW * AttShape<D>::kPart);
}

// Raise a kernel's shared-memory limit, once per device.
inline cudaError_t att_configure(const void *kernel, int smem, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int D>
cudaError_t launch_att_mma(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  using S = AttShape<D>;
  static_assert(S::kPart * 4 + sizeof(AttJoin<D>) <= S::kRing, "join");
  static std::atomic<bool> configured[64];
  const cudaError_t e = att_configure(reinterpret_cast<const void *>(kv4_attend_mma<D>), S::kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl_smem(kv4_attend_mma<D>, dim3(ctas), dim3(S::kThreads), S::kSmem, s, p);
}

cudaError_t launch_att_mma_64(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_mma_128(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_mma_256(const Kv4AttendParams &p, int ctas, cudaStream_t s);

}  // namespace gdn

// kv4_attend.cuh -- causal attention of a few query rows over the paged 4-bit
// cache: one pass over the keys, the codes as matrix operands.
//
// A unit is (row b, kv head, tile of 16 query rows); a query row is one
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
//            the largest.
// q is scaled per row by a power of two before fp16, exactly.
//
// What bounds it: HBM for single tokens and drafts (144 bytes a token and
// head pair at D = 128), with the instructions that unpack 2 x D codes a token
// close behind; hence the AND-only unpacking of the keys and packed fp32
// arithmetic.
//
// The keys' stages of all units form one line, which the CTAs of a persistent
// grid cut into equal pieces; the warps of a CTA take its stages in turn, each
// with its own ring of bulk copies, and join in shared memory.  A unit cut
// between CTAs is joined by whichever of them finishes last, in the order of
// the pieces, so the result does not depend on timing.
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace gdn {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kAttRows = 16;

template <int D>
struct AttShape {
  static constexpr int W = D / 64;               // groups of a head
  static constexpr int ST = D == 256 ? 32 : 64;  // keys of a stage
  static constexpr int NT = ST / 8;              // key tiles of a stage
  static constexpr int kCodes = ST * D / 2, kEntries = ST * W * 4;
  static constexpr int kStage = 2 * (kCodes + kEntries);
  static constexpr int kSlots = 3;               // stages of a warp's ring
  static constexpr int kPart = 16 * D;           // floats of a partial output
  static constexpr int kRing = kSlots * kStage;
  static constexpr int kSmem = kAttWarps * kRing + 128;
  static_assert(kRing >= kPart * 4, "the join reuses the ring");
};

// Partial results in the workspace: two per CTA, [16 D] outputs then m, l [16].
template <int D>
__host__ __device__ constexpr size_t att_part_floats() { return AttShape<D>::kPart + 32; }

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
__device__ __forceinline__ bool att_wait(uint64_t *bar, uint32_t parity) {
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

template <int D>
__global__ void __launch_bounds__(kAttThreads, 2) kv4_attend_mma(const __grid_constant__ Kv4AttendParams p) {
  using S = AttShape<D>;
  constexpr int W = S::W, ST = S::ST, NT = S::NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[kAttWarps][S::kSlots];
  __shared__ float s_m[kAttWarps][kAttRows], s_l[kAttWarps][kAttRows];
  __shared__ long long s_scan[kAttThreads];
  __shared__ long long s_place[2];
  __shared__ int s_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = lane >> 2, j = lane & 3;
  const int G = p.g.H_q / p.g.H_kv, Hkv = p.g.H_kv;
  const int P = 1 << p.g.log2P;
  if (lane == 0)
    for (int i = 0; i < S::kSlots; ++i) mbar_init(&s_full[warp][i], 1);
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's piece of the line ----------------------------------------------
  long long mine = 0;
  for (int b = tid; b < p.g.B; b += kAttThreads) {
    const AttRow r = att_row<D>(p, b, blockIdx.x == 0);
    mine += (long long)r.tiles * r.stages;
  }
  s_scan[tid] = mine;
  __syncthreads();
  long long total = 0;
  for (int i = 0; i < min(kAttThreads, p.g.B); ++i) total += s_scan[i];
  total *= Hkv;
  if (total == 0) return;
  // a CTA wants a stage for each warp at least
  const long long ctas = min((long long)gridDim.x, (total + kAttWarps - 1) / kAttWarps);
  const long long c = blockIdx.x;
  if (c >= ctas) return;
  long long at = total * c / ctas;
  const long long stop = total * (c + 1) / ctas;
  // the row that holds `at`
  int b = 0;
  long long row0 = 0;
  for (int b0 = 0; b0 < p.g.B; b0 += kAttThreads) {
    __syncthreads();
    long long v = 0;
    if (b0 + tid < p.g.B) {
      const AttRow r = att_row<D>(p, b0 + tid, false);
      v = (long long)r.tiles * r.stages * Hkv;
    }
    s_scan[tid] = v;
    if (tid == 0) s_place[0] = -1;
    __syncthreads();
    long long before = row0, all = 0;
    for (int i = 0; i < min(kAttThreads, p.g.B - b0); ++i) {
      const long long x = s_scan[i];
      if (i < tid) before += x;
      all += x;
    }
    if (at >= before && at < before + v) s_place[0] = b0 + tid, s_place[1] = before;
    __syncthreads();
    if (s_place[0] >= 0) {
      b = int(s_place[0]), row0 = s_place[1];
      break;
    }
    row0 += all;
  }

  uint8_t *ring = smem + warp * S::kRing;
  float *join = reinterpret_cast<float *>(ring);
  float *parts = reinterpret_cast<float *>(static_cast<char *>(p.ws) + 4096);
  uint32_t *counters = reinterpret_cast<uint32_t *>(p.ws);
  uint32_t phases = 0;  // parity of each ring slot
  bool dead = false;    // a copy never came: nothing more is waited for
  AttRow row = att_row<D>(p, b, false);

  while (at < stop) {
    while (at >= row0 + (long long)row.tiles * row.stages * Hkv) {
      row0 += (long long)row.tiles * row.stages * Hkv;
      row = att_row<D>(p, ++b, false);
    }
    const long long in_row = at - row0;
    const int unit = int(in_row / row.stages), st0 = int(in_row - (long long)unit * row.stages);
    const int hk = unit / row.tiles, tile = unit - hk * row.tiles;
    const long long unit_first = at - st0, unit_end = unit_first + row.stages;
    const int st1 = int(min((long long)row.stages, st0 + (stop - at)));

    // ---- the tile's queries ----------------------------------------------------
    const int R0 = tile * kAttRows + n, R1 = R0 + 8;
    const int i0 = R0 / G, i1 = R1 / G;
    const int tok0 = row.start + i0, tok1 = row.start + i1;
    const bool in0 = i0 < row.span, in1 = i1 < row.span;
    const int head0 = hk * G + R0 - i0 * G, head1 = hk * G + R1 - i1 * G;
    // keys that the row's query sees; rows past the span follow the others
    const bool live0 = in0 && i0 < row.count, live1 = in1 && i1 < row.count;
    int lim0 = live0 ? max(0, row.len - row.count + i0 + 1) : 0, lim1 = live1 ? max(0, row.len - row.count + i1 + 1) : 0;
    const int lim_max = __reduce_max_sync(0xffffffffu, max(lim0, lim1));
    if (!in0) lim0 = lim_max;
    if (!in1) lim1 = lim_max;
    const int lim_min = __reduce_min_sync(0xffffffffu, min(lim0, lim1));
    const int st_hi = min(st1, (lim_max + ST - 1) / ST);

    // ---- copies: a page is one copy, as it lies in memory (copies are taken one in
    // about 70 cycles whatever their size); half of a page is four pieces ---------------
    const bool half_page = P > ST;
    const int n_sub = half_page ? 4 : ST >> p.g.log2P;
    const int32_t *table = p.table + size_t(b) * p.g.max_pages;
    const uint32_t rec_bytes = kv4_record_bytes(D, P);
    const uint8_t *head_pages = p.pages + size_t(hk) * rec_bytes;
    auto page_of = [&](int st) -> int {
      const int t = st * ST + (half_page ? 0 : lane << p.g.log2P);
      return lane < n_sub && t < lim_max && st < st_hi ? table[t >> p.g.log2P] : -2;
    };
    auto issue = [&](int st, int slot, int page) {
      bool ok = page != -2;
      if (ok && (page < 0 || page >= p.g.n_pages)) {
        ok = false;
        atomicOr(p.status, GDN_STATUS_BAD_INDEX);
      }
      const uint32_t pages = __popc(__ballot_sync(0xffffffffu, ok));
      if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][slot], half_page ? (pages ? uint32_t(S::kStage) : 0u) : pages * rec_bytes);
      __syncwarp();
      if (ok) {
        const uint8_t *rec = head_pages + size_t(page) * (Hkv * size_t(rec_bytes));
        uint8_t *dst = ring + slot * S::kStage;
        if (half_page) {  // K, V codes, K, V entries by lanes 0 .. 3
          const int off = (st * ST) & (P - 1);
          const bool codes = lane < 2, second = lane & 1;
          bulk_g2s(dst + (codes ? second * S::kCodes : 2 * S::kCodes + second * S::kEntries),
                   rec + (codes ? second * kv4_code_bytes(D, P) + off * (D / 2)
                                : 2 * kv4_code_bytes(D, P) + second * kv4_entry_bytes(D, P) + off * W * 4),
                   codes ? S::kCodes : S::kEntries, &s_full[warp][slot]);
        } else {
          bulk_g2s(dst + lane * rec_bytes, rec, rec_bytes, &s_full[warp][slot]);
        }
      }
    };
    // places of a stage's keys: `pt` keys (a page, or the half of one) a record
    const int log2pt = min(p.g.log2P, ST == 32 ? 5 : 6), pt = 1 << log2pt;
    const int rec_c = pt * (D / 2), rec_e = pt * (W * 4), rec_s = 2 * (rec_c + rec_e);
    auto code_at = [&](const uint8_t *stage, int which, int key) {
      return stage + (key >> log2pt) * rec_s + which * rec_c + (key & (pt - 1)) * (D / 2);
    };
    auto entry_at = [&](const uint8_t *stage, int which, int key) {
      return stage + (key >> log2pt) * rec_s + 2 * rec_c + which * rec_e + (key & (pt - 1)) * (W * 4);
    };
    int next = page_of(st0 + warp);
    int issued = st0 + warp;  // next stage to issue
    int slot_in = 0;
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i) {
      if (issued < st_hi && !dead) {
        const int page = next;
        next = page_of(issued + kAttWarps);
        issue(issued, slot_in, page);
        issued += kAttWarps;
        slot_in = slot_in + 1 == S::kSlots ? 0 : slot_in + 1;
      }
    }

    // ---- Q as fp16 fragments, scaled by a power of two per row -------------------------
    uint32_t qa[D / 16][4];
    float qs0[W], qs1[W];
    float f0, f1;
    {
      uint32_t mx0 = 0, mx1 = 0;
      uint4 raw0[D / 32], raw1[D / 32];
      const uint16_t *src0 = p.q + (size_t(tok0) * p.g.H_q + head0) * D;
      const uint16_t *src1 = p.q + (size_t(tok1) * p.g.H_q + head1) * D;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // word w of the lane: channels 8 * (4 * (w / WL) ... ) as the keys' words below
        const int ch = D == 64 ? 16 * j + 8 * w : 128 * (w >> 2) + 32 * j + 8 * (w & 3);
        raw0[w] = live0 ? *reinterpret_cast<const uint4 *>(src0 + ch) : make_uint4(0, 0, 0, 0);
        raw1[w] = live1 ? *reinterpret_cast<const uint4 *>(src1 + ch) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t a[4] = {raw0[w].x, raw0[w].y, raw0[w].z, raw0[w].w};
        const uint32_t d[4] = {raw1[w].x, raw1[w].y, raw1[w].z, raw1[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx0 = max(mx0, max(a[e] & 0x7fffu, (a[e] >> 16) & 0x7fffu));
          mx1 = max(mx1, max(d[e] & 0x7fffu, (d[e] >> 16) & 0x7fffu));
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx0 = max(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = max(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      // the largest magnitude goes to [2^10, 2^11); exponents kept where both
      // powers of two are normal numbers
      const int e0 = min(max(int(mx0 >> 7), 20), 240), e1 = min(max(int(mx1 >> 7), 20), 240);
      const float up0 = __uint_as_float(uint32_t(264 - e0) << 23), up1 = __uint_as_float(uint32_t(264 - e1) << 23);
      // back to the score in base 2: 1 / up, 2^24 of the subnormal codes, scale * log2(e)
      f0 = (1.f / up0) * (p.scale * 1.4426950408889634f) * 16777216.f;
      f1 = (1.f / up1) * (p.scale * 1.4426950408889634f) * 16777216.f;
#pragma unroll
      for (int g = 0; g < W; ++g) qs0[g] = qs1[g] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const int g = D == 64 ? 0 : w % W;
        float x[8], y[8];
        const uint32_t a[4] = {raw0[w].x, raw0[w].y, raw0[w].z, raw0[w].w};
        const uint32_t d[4] = {raw1[w].x, raw1[w].y, raw1[w].z, raw1[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(a[e] << 16) * up0, x[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u) * up0;
          y[2 * e] = __uint_as_float(d[e] << 16) * up1, y[2 * e + 1] = __uint_as_float(d[e] & 0xffff0000u) * up1;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) qs0[g] += x[e], qs1[g] += y[e];
        // step 2w: columns (0, 4) and (1, 5) / 16; step 2w + 1: (2, 6) and (3, 7) / 16
        qa[2 * w][0] = pack_h2(x[0], x[4]), qa[2 * w][1] = pack_h2(y[0], y[4]);
        qa[2 * w][2] = pack_h2(x[1] * 0.0625f, x[5] * 0.0625f), qa[2 * w][3] = pack_h2(y[1] * 0.0625f, y[5] * 0.0625f);
        qa[2 * w + 1][0] = pack_h2(x[2], x[6]), qa[2 * w + 1][1] = pack_h2(y[2], y[6]);
        qa[2 * w + 1][2] = pack_h2(x[3] * 0.0625f, x[7] * 0.0625f), qa[2 * w + 1][3] = pack_h2(y[3] * 0.0625f, y[7] * 0.0625f);
      }
#pragma unroll
      for (int g = 0; g < W; ++g) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          qs0[g] += __shfl_xor_sync(0xffffffffu, qs0[g], o);
          qs1[g] += __shfl_xor_sync(0xffffffffu, qs1[g], o);
        }
        qs0[g] *= 5.9604644775390625e-08f, qs1[g] *= 5.9604644775390625e-08f;  // 2^-24, as the codes
      }
    }

    float o_acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.f;
    uint32_t nan0 = 0, nan1 = 0;  // groups in which the row has seen a value that is not finite
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    int slot = 0;
    for (int st = st0 + warp; st < st_hi; st += kAttWarps) {
      if (st < issued) {  // once a wait has run out nothing more is issued, and what is in flight still waited for
        if (!att_wait(&s_full[warp][slot], (phases >> slot) & 1)) {
          dead = true;
          atomicOr(p.status, GDN_STATUS_TIMEOUT);
        }
        dead = __any_sync(0xffffffffu, dead);
        phases ^= 1u << slot;
      }
      const uint8_t *stage = ring + slot * S::kStage;
      const int t_base = st * ST;

      // ---- scores ------------------------------------------------------------------
      float s[NT][4];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float acc[W][4];
#pragma unroll
        for (int g = 0; g < W; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
        const uint8_t *kr = code_at(stage, 0, 8 * u + att_key(n));
        uint32_t word[D / 32];
        if (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2 *>(kr + 8 * j);
          word[0] = x.x, word[1] = x.y;
        } else {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kr + 64 * i + 16 * j);
            word[4 * i] = x.x, word[4 * i + 1] = x.y, word[4 * i + 2] = x.z, word[4 * i + 3] = x.w;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const int g = D == 64 ? 0 : w % W;
          const uint32_t x = word[w], y = x >> 8;
          mma16816(acc[g], qa[2 * w][0], qa[2 * w][1], qa[2 * w][2], qa[2 * w][3], x & 0x000f000fu, x & 0x00f000f0u);
          mma16816(acc[g], qa[2 * w + 1][0], qa[2 * w + 1][1], qa[2 * w + 1][2], qa[2 * w + 1][3], y & 0x000f000fu,
                   y & 0x00f000f0u);
        }
        uint32_t x0[W], x1[W];
        att_words<W>(x0, entry_at(stage, 0, 8 * u + att_key(2 * j)));
        att_words<W>(x1, entry_at(stage, 0, 8 * u + att_key(2 * j + 1)));
        F2 r0 = f2(0.f, 0.f), r1 = f2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < W; ++g) {
          const F2 step = f2(half_lo(x0[g]), half_lo(x1[g])), base = f2(half_hi(x0[g]), half_hi(x1[g]));
          r0 = f2_fma(step, f2(acc[g][0], acc[g][1]), r0);
          r1 = f2_fma(step, f2(acc[g][2], acc[g][3]), r1);
          r0 = f2_fma(base, f2(qs0[g], qs0[g]), r0);
          r1 = f2_fma(base, f2(qs1[g], qs1[g]), r1);
        }
        f2_get(r0, s[u][0], s[u][1]);
        f2_get(r1, s[u][2], s[u][3]);
      }
      const bool cut = t_base + ST > lim_min;  // some query does not see all of the stage
      if (cut) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const int ta = t_base + 8 * u + att_key(2 * j), tb = t_base + 8 * u + att_key(2 * j + 1);
          if (ta >= lim0) s[u][0] = -INFINITY;
          if (tb >= lim0) s[u][1] = -INFINITY;
          if (ta >= lim1) s[u][2] = -INFINITY;
          if (tb >= lim1) s[u][3] = -INFINITY;
        }
      }
      // ---- running maximum; the largest step of each group ----------------------------
      // f may be negative (a negative scale): the maximum is taken after it
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        if (cut) {
          s[u][0] = s[u][0] == -INFINITY ? -INFINITY : s[u][0] * f0;
          s[u][1] = s[u][1] == -INFINITY ? -INFINITY : s[u][1] * f0;
          s[u][2] = s[u][2] == -INFINITY ? -INFINITY : s[u][2] * f1;
          s[u][3] = s[u][3] == -INFINITY ? -INFINITY : s[u][3] * f1;
        } else {
          s[u][0] *= f0, s[u][1] *= f0, s[u][2] *= f1, s[u][3] *= f1;
        }
        x0 = fmaxf(x0, fmaxf(s[u][0], s[u][1]));
        x1 = fmaxf(x1, fmaxf(s[u][2], s[u][3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
      }
      if (__any_sync(0xffffffffu, x0 > m0 + 14.f || x1 > m1 + 14.f)) {
        const float n0 = fmaxf(m0, x0 - 6.f), n1 = fmaxf(m1, x1 - 6.f);
        const float a0 = n0 == m0 ? 1.f : ex2(m0 - n0), a1 = n1 == m1 ? 1.f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= a0, l1 *= a1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o_acc[i][0] *= a0, o_acc[i][1] *= a0, o_acc[i][2] *= a1, o_acc[i][3] *= a1;
      }
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;

      // ---- probabilities and output, 16 keys at a time --------------------------------
#pragma unroll
      for (int h = 0; h < NT / 2; ++h) {
        uint32_t a[4], es[W][2], eb[W][2];  // P; (step, step), (base, base) of the key pairs
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int u = 2 * h + half;
          const float p00 = ex2(s[u][0] - r0), p01 = ex2(s[u][1] - r0);
          const float p10 = ex2(s[u][2] - r1), p11 = ex2(s[u][3] - r1);
          l0 += p00 + p01, l1 += p10 + p11;
          a[2 * half] = pack_h2(p00, p01);
          a[2 * half + 1] = pack_h2(p10, p11);
          const int ka = 8 * u + att_key(2 * j), kb = 8 * u + att_key(2 * j + 1);
          uint32_t wa[W], wb[W];
          att_words<W>(wa, entry_at(stage, 1, ka));
          att_words<W>(wb, entry_at(stage, 1, kb));
          if (cut) {
            // a value that one query sees and another does not must not reach
            // the other as 0 * NaN: it is left out and remembered by the row
#pragma unroll
            for (int g = 0; g < W; ++g) {
              const int ta = t_base + ka, tb = t_base + kb;
              if (att_not_finite(wa[g])) nan0 |= uint32_t(ta < lim0) << g, nan1 |= uint32_t(ta < lim1) << g, wa[g] = 0;
              if (att_not_finite(wb[g])) nan0 |= uint32_t(tb < lim0) << g, nan1 |= uint32_t(tb < lim1) << g, wb[g] = 0;
              if (ta >= lim_max) wa[g] = 0;
              if (tb >= lim_max) wb[g] = 0;
            }
          }
#pragma unroll
          for (int g = 0; g < W; ++g) {
            es[g][half] = __byte_perm(wa[g], wb[g], 0x5410);
            eb[g][half] = __byte_perm(wa[g], wb[g], 0x7632);
          }
        }
        uint32_t w0[W], w1[W], w2[W], w3[W];
        att_words<W>(w0, code_at(stage, 1, 16 * h + att_key(2 * j)) + n * (4 * W));
        att_words<W>(w1, code_at(stage, 1, 16 * h + att_key(2 * j + 1)) + n * (4 * W));
        att_words<W>(w2, code_at(stage, 1, 16 * h + 8 + att_key(2 * j)) + n * (4 * W));
        att_words<W>(w3, code_at(stage, 1, 16 * h + 8 + att_key(2 * j + 1)) + n * (4 * W));
#pragma unroll
        for (int g = 0; g < W; ++g) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = __byte_perm(w0[g], w1[g], half ? 0x7632 : 0x5410);
            const uint32_t y = __byte_perm(w2[g], w3[g], half ? 0x7632 : 0x5410);
            const uint32_t xs = x >> 8, ys = y >> 8;
            const int o = 8 * g + 4 * half;
            mma16816(o_acc[o], a[0], a[1], a[2], a[3], att_even(x, es[g][0], eb[g][0]), att_even(y, es[g][1], eb[g][1]));
            mma16816(o_acc[o + 1], a[0], a[1], a[2], a[3], att_odd(x, es[g][0], eb[g][0]), att_odd(y, es[g][1], eb[g][1]));
            mma16816(o_acc[o + 2], a[0], a[1], a[2], a[3], att_even(xs, es[g][0], eb[g][0]), att_even(ys, es[g][1], eb[g][1]));
            mma16816(o_acc[o + 3], a[0], a[1], a[2], a[3], att_odd(xs, es[g][0], eb[g][0]), att_odd(ys, es[g][1], eb[g][1]));
          }
        }
      }
      __syncwarp();  // every lane is done with the slot
      if (issued < st_hi && !dead) {
        const int page = next;
        next = page_of(issued + kAttWarps);
        issue(issued, slot, page);
        issued += kAttWarps;
      }
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
    }
    // the ring starts again at slot 0: all its copies of this piece have been waited for
    // ---- this warp's part: outputs, maximum and sum of its keys -----------------------
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      nan0 |= __shfl_xor_sync(0xffffffffu, nan0, o);
      nan1 |= __shfl_xor_sync(0xffffffffu, nan1, o);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        join[(i * 4 + k) * 32 + lane] = ((k < 2 ? nan0 : nan1) >> (i / 8) & 1u) ? __uint_as_float(0x7fc00000u) : o_acc[i][k];
    if (j == 0) s_m[warp][n] = m0, s_m[warp][n + 8] = m1, s_l[warp][n] = l0, s_l[warp][n + 8] = l1;
    __syncthreads();

    // ---- join of the warps: warp w has the 8-channel tiles [w D / 32, (w + 1) D / 32) ------
    constexpr int TW = D / 8 / kAttWarps;
    float y[TW][4], M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int i = 0; i < TW; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
    {
      float c0[kAttWarps], c1[kAttWarps];
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) M0 = fmaxf(M0, s_m[w][n]), M1 = fmaxf(M1, s_m[w][n + 8]);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        c0[w] = s_m[w][n] == -INFINITY ? 0.f : ex2(s_m[w][n] - M0);
        c1[w] = s_m[w][n + 8] == -INFINITY ? 0.f : ex2(s_m[w][n + 8] - M1);
        // a NaN score leaves the maximum alone but not the sum
        if (s_l[w][n] != s_l[w][n]) c0[w] = 1.f;
        if (s_l[w][n + 8] != s_l[w][n + 8]) c1[w] = 1.f;
        L0 = fmaf(s_l[w][n], c0[w], L0), L1 = fmaf(s_l[w][n + 8], c1[w], L1);
      }
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float *src = reinterpret_cast<const float *>(smem + w * S::kRing);
#pragma unroll
        for (int i = 0; i < TW; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i][k] = fmaf(src[((warp * TW + i) * 4 + k) * 32 + lane], k < 2 ? c0[w] : c1[w], y[i][k]);
      }
    }

    // ---- the whole unit, or a part of it ------------------------------------------------
    bool whole = unit_first >= at && unit_end <= at + (st1 - st0);
    if (!whole) {
      const long long c_first = ((unit_first + 1) * ctas - 1) / total, c_last = (unit_end * ctas - 1) / total;
      float *part = parts + (size_t(c) * 2 + (c == c_first ? 1 : 0)) * att_part_floats<D>();
#pragma unroll
      for (int i = 0; i < TW; ++i)
        *reinterpret_cast<float4 *>(part + ((warp * TW + i) * 32 + lane) * 4) = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
      if (warp == 0 && j == 0) {
        part[S::kPart + n] = M0, part[S::kPart + n + 8] = M1;
        part[S::kPart + 16 + n] = L0, part[S::kPart + 16 + n + 8] = L1;
      }
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
      whole = s_flag != 0;
      if (whole) {
        M0 = M1 = -INFINITY;
        for (long long k = c_first; k <= c_last; ++k) {
          const float *src = parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * att_part_floats<D>();
          M0 = fmaxf(M0, __ldcg(src + S::kPart + n)), M1 = fmaxf(M1, __ldcg(src + S::kPart + n + 8));
        }
        L0 = L1 = 0.f;
#pragma unroll
        for (int i = 0; i < TW; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
        for (long long k = c_first; k <= c_last; ++k) {
          const float *src = parts + (size_t(k) * 2 + (k == c_first ? 1 : 0)) * att_part_floats<D>();
          const float ma = __ldcg(src + S::kPart + n), mb = __ldcg(src + S::kPart + n + 8);
          const float la = __ldcg(src + S::kPart + 16 + n), lb = __ldcg(src + S::kPart + 16 + n + 8);
          const float c0 = la != la ? 1.f : ma == -INFINITY ? 0.f : ex2(ma - M0);
          const float c1 = lb != lb ? 1.f : mb == -INFINITY ? 0.f : ex2(mb - M1);
          L0 = fmaf(la, c0, L0), L1 = fmaf(lb, c1, L1);
#pragma unroll
          for (int i = 0; i < TW; ++i) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + ((warp * TW + i) * 32 + lane) * 4));
            y[i][0] = fmaf(v.x, c0, y[i][0]), y[i][1] = fmaf(v.y, c0, y[i][1]);
            y[i][2] = fmaf(v.z, c1, y[i][2]), y[i][3] = fmaf(v.w, c1, y[i][3]);
          }
        }
      }
    }
    if (whole) {
      // tile 8 g + e, column c: channel (c W + g) 8 + e; a warp holds TW (a
      // multiple of 2) neighbouring channels of each column
      const float v0 = L0 > 0.f ? 1.f / L0 : L0, v1 = L1 > 0.f ? 1.f / L1 : L1;  // no key: 0; NaN stays
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c8 = 2 * j + (k & 1), tok = k < 2 ? tok0 : tok1, head = k < 2 ? head0 : head1;
        if (!(k < 2 ? in0 : in1)) continue;
        const float v = k < 2 ? v0 : v1;
        uint16_t *dst = p.out + (size_t(tok) * p.g.H_q + head) * D;
#pragma unroll
        for (int i = 0; i < TW; i += 2) {
          const int t = warp * TW + i, ch = (c8 * W + t / 8) * 8 + t % 8;
          const __nv_bfloat162 x = __floats2bfloat162_rn(y[i][k] * v, y[i + 1][k] * v);
          *reinterpret_cast<__nv_bfloat162 *>(dst + ch) = x;
        }
      }
    }
    at += st1 - st0;
    fence_proxy_async_shared();  // the join's writes before the next piece's copies
    __syncthreads();
  }
}

template <int D>
inline size_t att_mma_ws(int ctas) {
  return 4096 + sizeof(float) * 2 * size_t(ctas) * att_part_floats<D>();
}

template <int D>
cudaError_t launch_att_mma(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv4_attend_mma<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, AttShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_smem(kv4_attend_mma<D>, dim3(ctas), dim3(kAttThreads), AttShape<D>::kSmem, s, p);
}

cudaError_t launch_att_mma_64(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_mma_128(const Kv4AttendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_att_mma_256(const Kv4AttendParams &p, int ctas, cudaStream_t s);

}  // namespace gdn

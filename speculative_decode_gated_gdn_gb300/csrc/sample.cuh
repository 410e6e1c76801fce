// sample.cuh -- parameters and arithmetic of sampled decoding.
//
// A logit is bf16, so a row of any length has at most 65,280 different numbers.
// The order in which a row is taken (values descending, equal ones by index), the
// mass of its filters and the drawn token all follow from how many logits have
// each value: the mass is the sum over values of count * weight.  Weights are
// integers of 2^-43 (the largest logit's is 1), so sums are exact and do not depend
// on their order, and a row of up to 2^20 logits stays below 2^63.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

struct SampleParams {
  const uint16_t *logits;  // position i at i * stride
  long long stride;
  const int32_t *draft;    // [B][T]; NULL: no acceptance
  const uint8_t *active;   // [B] or NULL
  const float *temperature, *top_p, *min_p;  // [B] or NULL
  const int32_t *top_k;                      // [B] or NULL
  const float *u;          // [B][T]
  int32_t *token;          // [B][T] or NULL
  float *logp;             // [B][T] or NULL
  int32_t *keep, *next;    // [B] (acceptance)
  int32_t *ws_token;       // [B][T]
  uint32_t *ws_count;      // [B] positions of the row that are done
  int B, T, V;
};

constexpr int kMaxSampleV = 1 << 20;
size_t accept_sampled_workspace_bytes(int B, int T);
cudaError_t launch_sample(const SampleParams &p, cudaStream_t s);

// ---- a value's place in the order -------------------------------------------------
// 16 bits, ascending where values descend; -0 counts as 0.  Numbers above
// -infinity lie in [kPlaceInf, kPlaceEnd).
constexpr int kPlaceInf = 0x007f, kPlaceZero = 0x7fff, kPlaceEnd = 0xff80;

__device__ __forceinline__ int place_of(uint32_t bits) {
  const int a = int(bits & 0x7fffu);
  if (a > 0x7f80) return 0xffff;  // NaN: nowhere
  return (bits & 0x8000u) && a ? 0x8000 + a : kPlaceZero - a;
}
__device__ __forceinline__ float value_at(int place) {
  return place <= kPlaceZero ? bf2f(uint16_t(kPlaceZero - place)) : -bf2f(uint16_t(place - 0x8000));
}

// ---- weights ----------------------------------------------------------------------
constexpr int kWeightBits = 43;
constexpr unsigned long long kWeightOne = 1ull << kWeightBits;

// 2^(m / 32) in units of 2^-62
__device__ const unsigned long long kExp2Table[32] = {
    0x4000000000000000ull, 0x4166c34c5615d0ecull, 0x42d561b3e6243d8aull, 0x444c0740496d4294ull,
    0x45cae0f1f545eb73ull, 0x47521cc5a2e6a9e0ull, 0x48e1e9b9d588e19bull, 0x4a7a77d47f7b84b1ull,
    0x4c1bf828c6dc54b8ull, 0x4dc69cdceaa72a9cull, 0x4f7a993048d088d7ull, 0x513821818624b40cull,
    0x52ff6b54d8a89c75ull, 0x54d0ad5a753e077cull, 0x56ac1f752150a563ull, 0x5891fac0e95612c8ull,
    0x5a827999fcef3242ull, 0x5c7dd7a3b17dcf75ull, 0x5e8451cfac061b5full, 0x6096266533384a2bull,
    0x62b39508aa836d6full, 0x64dcdec3371793d1ull, 0x6712460a8fc24072ull, 0x69540ec8f895722dull,
    0x6ba27e656b4eb57aull, 0x6dfddbcbed791babull, 0x70666f76154a7089ull, 0x72dc8373be41a454ull,
    0x75606373ee921c97ull, 0x77f25ccdee6d7ae6ull, 0x7a92be8a92436616ull, 0x7d41d96db915019dull,
};

struct Scale {
  float hi, lo;  // 2 / (temperature * unit * ln 2); 0: every weight is 1
  float unit;    // a power of two that keeps the quotient and its remainder among the normal numbers
};

// The quotient's remainder is exact by fma, so hi + lo is within 2^-46 of it.
__device__ __forceinline__ Scale scale_of(float temperature) {
  constexpr float k = 2.88539004f, k_lo = 3.851926067e-8f;  // 2 / ln 2
  constexpr float large = 18446744073709551616.f;           // 2^64
  Scale s;
  s.unit = temperature >= large ? 1.f / large : temperature < 1.f / large ? large : 1.f;
  temperature *= s.unit;
  s.hi = __fdiv_rn(k, temperature);
  s.lo = __fdiv_rn(fmaf(-s.hi, temperature, k) + k_lo, temperature);
  return s;
}

// x * mass for 0 <= x < 1, rounded down or up, exactly.
__device__ __forceinline__ unsigned long long share_of(float x, unsigned long long mass, bool up) {
  const uint32_t bits = __float_as_uint(x);
  const uint32_t e = max(bits >> 23, 1u), m = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
  const unsigned long long lo = m * mass, hi = __umul64hi(m, mass);
  const uint32_t shift = 150 - e;  // 24 .. 149
  if (shift >= 128) return up && m && mass;
  unsigned long long q, rest;
  if (shift >= 64) q = hi >> (shift - 64), rest = lo | (shift > 64 ? hi << (128 - shift) : 0);
  else q = hi << (64 - shift) | lo >> shift, rest = lo << (64 - shift);
  return q + (up && rest);
}

// floor(a / b) where it is at most 2^20; 0 < b, a < 2^63.  The quotient of the rounded
// numbers is within 2^-21 of itself, so less than one off.
__device__ __forceinline__ uint32_t few_in(unsigned long long a, unsigned long long b) {
  uint32_t q = uint32_t(__fdividef(__ull2float_rn(a), __ull2float_rn(b)));
  if (q * b > a) --q;
  else if ((q + 1ull) * b <= a) ++q;
  return q;
}

// exp((value_at(place) - value_at(top)) / temperature) in units of 2^-43, rounded; top <= place.
// The exponent t (base 2) is a sum of two floats, 2^-46 exact; 2^t = 2^n 2^(m/32) 2^r with the middle
// factor from the table and the last, |r| <= 1/64, by its series: 2^-38 of the weight in all, half
// a unit aside.
static __device__ __noinline__ unsigned long long weight_of(int place, int top, Scale c, const unsigned long long *table) {
  if (place == top) return kWeightOne;
  if (top == kPlaceInf) return 0;
  if (c.hi == 0.f) return kWeightOne;
  const float z = 0.5f * value_at(place), z0 = 0.5f * value_at(top);  // halves: their difference is finite
  const float d = z - z0, back = d - z;
  const float s = d * c.unit, err = ((z - (d - back)) + (-z0 - back)) * c.unit;
  const float t = s * c.hi;
  if (!(t > -46.f)) return 0;
  const float t_lo = fmaf(s, c.hi, -t) + fmaf(s, c.lo, err * c.hi);
  const float kf = rintf(t * 32.f);
  const int k = int(kf);
  const float r = fmaf(kf, -0.03125f, t);
  constexpr float kLn2 = 0.693147182464599609f, kLn2Lo = -1.9046542121259336e-9f;
  const float y = r * kLn2, y_lo = fmaf(r, kLn2, -y) + fmaf(r, kLn2Lo, t_lo * kLn2);
  const float hi = y + y_lo, lo = y_lo - (hi - y);
  // 1 + hi + hi^2 / 2 + ..: the first two in a sum of two floats, the square with its remainder
  const float sq = hi * hi, half = 0.5f * sq, first = hi + half;
  const float rest = fmaf(0.5f, fmaf(hi, hi, -sq), fmaf(sq * hi, fmaf(hi, fmaf(hi, 1.f / 120, 1.f / 24), 1.f / 6), fmaf(lo, hi, lo) + (half - (first - hi))));
  const float unit = 1125899906842624.f;  // 2^50
  const unsigned long long f = (1ull << 50) + (unsigned long long)(__float2ll_rn(first * unit) + __float2ll_rn(rest * unit));
  const unsigned long long w = __umul64hi(table[k & 31], f << 13);  // in units of 2^(n - 61)
  const int shift = 61 - kWeightBits - (k >> 5);
  if (shift > 62) return 0;
  return (w + (1ull << (shift - 1))) >> shift;
}

// ---- a row in memory ----------------------------------------------------------------
// Taken in granules of eight logits that lie on 16-byte boundaries, whatever address
// the row begins at; places of a granule outside the row read as NaN.
struct SampleRow {
  const uint16_t *base;  // the first granule's address
  int skip, V, granules;

  __device__ __forceinline__ SampleRow(const uint16_t *p, int V_) : V(V_) {
    skip = int((reinterpret_cast<uintptr_t>(p) >> 1) & 7);
    base = p - skip;
    granules = (skip + V + 7) >> 3;
  }
  __device__ __forceinline__ int first(int g) const { return 8 * g - skip; }  // index of a granule's first logit
  __device__ __forceinline__ uint4 load(int g) const {
    const int i = first(g);
    if (i >= 0 && i + 8 <= V) return *reinterpret_cast<const uint4 *>(base + 8 * size_t(g));
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t x = i + j >= 0 && i + j < V ? base[8 * size_t(g) + j] : 0x7fffu;
      w[j >> 1] = (j & 1) ? (w[j >> 1] | x << 16) : x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint32_t half_of(const uint4 &q, int j) {
  const uint32_t w = j < 2 ? q.x : j < 4 ? q.y : j < 6 ? q.z : q.w;
  return (j & 1) ? w >> 16 : w & 0xffffu;
}

}  // namespace gdn

// kv4_append.cu -- rotary positions with several axes on q and k, and k and v
// into the paged 4-bit cache; and the cache's tokens back in bf16.
//
// Rotation: pair i of a token turns by the angle whose (cos, sin) the caller's
// fp32 table holds at [positions[axis[i]]][i].  The table, and not an angle
// formed here, keeps far positions exact: an fp32 product pos * frequency is
// off by 0.06 rad at a million.  Products and sums are rounded one by one
// (no fused multiply-add), so that a value next to a border between two codes
// falls on the side the plain formula puts it.
//
// Quantisation, per token, head and group of 64 channels (kv4.cuh):
//   base = fp16(min), step = fp16((max - min) / 15)
//   code = clamp(round_half_even((y - base) / step), 0, 15), 0 where step is 0
// from the fp32 rotated value; min, max and the step are exact or rounded once
// in fp32 before fp16.  A group that holds an infinity or NaN reads back as
// NaN; base and step are held within 65504 each, so that a level base + step *
// code may lie up to 16 * 65504 from zero.
//
// Both kernels move each byte once: 8 channels a lane (16 bytes of bf16, one
// 32-bit word of codes), a head on D / 8 lanes, the loads of the next heads on
// their way under a head's work.  The read is bound by HBM.  The append is
// bound by its instructions: rotation, the group's minimum and maximum, a
// quotient and its rounding for every channel of K and V keep the issue slots
// 71 % busy where HBM is at half its rate.  One launch over 4101 tokens of 32 + 8
// + 8 heads of 128, all rotated: 27.0 us, 3.3 TB/s; over 32768 of 16 + 2 + 2 heads
// of 256, a quarter rotated: 121.6 us, 5.1 TB/s; reading the latter back: 15.3 us.
// Tried and not kept: evict-first stores, CTAs of 128 threads, other numbers of
// loads ahead.
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kAppendThreads = 256;
constexpr float kHalfMax = 65504.f;

__device__ __forceinline__ uint4 ld_stream_u4(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Quantise the lane's 8 channels with the 8 lanes of its group (lanes equal
// modulo W within the head) and write codes and, from the group's first lane,
// the entry.
template <int D>
__device__ __forceinline__ void store_codes(const float (&y)[8], uint8_t *codes, uint8_t *entries, int chunk, bool store) {
  constexpr int W = D / 64;
  float mn = y[0], mx = y[0], nil = y[0] * 0.f;
#pragma unroll
  for (int e = 1; e < 8; ++e) mn = fminf(mn, y[e]), mx = fmaxf(mx, y[e]), nil = fmaf(y[e], 0.f, nil);
  int ok = nil == 0.f;  // an infinity or NaN leaves a NaN
#pragma unroll
  for (int o = W; o < 8 * W; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    ok &= __shfl_xor_sync(0xffffffffu, ok, o);
  }
  __half base = __float2half_rn(fminf(fmaxf(mn, -kHalfMax), kHalfMax));
  __half step = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(mx, mn), 15.f), kHalfMax));
  if (!ok) base = step = __ushort_as_half(0x7e00);
  const float b = __half2float(base), s = __half2float(step);
  uint32_t word = 0;
  if (ok && s > 0.f) {
    // (y - b) / s by a reciprocal, off by a few 2^-23 of at most 15: only next to
    // a border between two codes can that matter, and there the division decides
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the sum's last bits are the nearest integer
    const float inv = __fdividef(1.f, s);
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = fminf(fmaxf(__fsub_rn(y[e], b) * inv, 0.f), 15.f), u = __fadd_rn(t, kMagic);
      near = near || fabsf(t - __fsub_rn(u, kMagic)) > 0.4999f;
      word |= (__float_as_uint(u) & 15u) << (4 * e);
    }
    if (near) {
      word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y[e], b), s)), 0.f), 15.f);
        word |= uint32_t(c) << (4 * e);
      }
    }
  }
  if (!store) return;
  reinterpret_cast<uint32_t *>(codes)[chunk] = word;
  if (chunk < W)
    reinterpret_cast<uint32_t *>(entries)[chunk] = uint32_t(__half_as_ushort(step)) | uint32_t(__half_as_ushort(base)) << 16;
}

// One token a warp sub-group: D / 8 lanes hold a head, the warp's 32 / (D / 8)
// heads at a time; blockIdx.y splits the heads of a token where tokens are few.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) kv4_append_kernel(const Kv4AppendParams p, const int splits) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, W = D / 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = lane % LPH, sub = lane / LPH;
  const int n = blockIdx.x * (kAppendThreads / 32) + warp;
  pdl_wait();
  pdl_trigger();
  if (n >= p.N) return;  // whole warps
  const int heads = p.H_q + 2 * p.H_kv;
  const int per = (heads + splits - 1) / splits;
  const int h1 = min(heads, int(blockIdx.y + 1) * per);
  int h0 = blockIdx.y * per;
  // the loads of kAhead heads are on their way together, the next ones' and the
  // angles' while these are worked on
  constexpr int kAhead = 2;
  uint4 raws[kAhead];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * HPW + sub;
      raws[u] = make_uint4(0, 0, 0, 0);
      if (h < h1) {
        const uint16_t *src = h < p.H_q              ? p.q + n * p.q_stride + size_t(h) * D
                              : h < p.H_q + p.H_kv ? p.k + n * p.k_stride + size_t(h - p.H_q) * D
                                                   : p.v + n * p.v_stride + size_t(h - p.H_q - p.H_kv) * D;
        raws[u] = ld_stream_u4(src + 8 * chunk);
      }
    }
  };
  load(h0);
  const int P = 1 << p.log2P;
  const int slot = p.slots[n];
  bool write = slot >= 0;
  if (write && (slot >> p.log2P) >= p.n_pages) {
    write = false;
    if (lane == 0) atomicOr(p.status, GDN_STATUS_BAD_INDEX);
  }
  // the lane's angles: it holds channels [8 chunk, 8 chunk + 8)
  const int half = p.rot >> 1;
  const bool turned = 8 * chunk < p.rot;
  float cs[8], sn[8];
  uint32_t still = 0;  // channels whose position is outside the table: they do not turn
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f, sn[e] = 0.f;
    if (turned) {
      const int c = 8 * chunk + e;
      const int i = p.pairs ? c >> 1 : (c < half ? c : c - half);
      const int pos = p.positions[size_t(p.axis[i]) * p.N + n];
      if (pos >= 0 && pos < p.max_pos) {
        const float2 t = __ldg(p.rope + size_t(pos) * half + i);
        cs[e] = t.x, sn[e] = t.y;
      } else {
        still |= 1u << e;
        if (slot >= 0) {
          write = false;
          atomicOr(p.status, GDN_STATUS_BAD_INDEX);
        }
      }
    }
  }
  write = __all_sync(0xffffffffu, write);
  const int page = write ? slot >> p.log2P : 0, off = write ? slot & (P - 1) : 0;
  const int partner = lane + (p.pairs || !turned ? 0 : (8 * chunk < half ? half / 8 : -half / 8));
  if (!p.pairs && 8 * chunk < half) {  // the lower half takes the partner's product away
#pragma unroll
    for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
  }
  auto turn = [&](const uint4 raw, float (&y)[8], bool rotate) {  // the whole warp
    if (p.pairs) {
      if (rotate) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = y[e], b = y[e + 1];
          y[e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
          y[e + 1] = __fadd_rn(__fmul_rn(b, cs[e + 1]), __fmul_rn(a, sn[e + 1]));
        }
      }
    } else {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw.x, partner);
      o.y = __shfl_sync(0xffffffffu, raw.y, partner);
      o.z = __shfl_sync(0xffffffffu, raw.z, partner);
      o.w = __shfl_sync(0xffffffffu, raw.w, partner);
      if (rotate) {
        float z[8];
        unpack8(o, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fadd_rn(__fmul_rn(y[e], cs[e]), __fmul_rn(z[e], sn[e]));
      }
    }
  };
  // A token some of whose positions are outside the table: its queries one load at a time.
  // (Times 1 plus times 0 would not do: an infinity in the pair, a zero's sign.)
  if (__any_sync(0xffffffffu, still != 0)) {
#pragma unroll 1
    for (; h0 < min(h1, p.H_q); h0 += HPW) {
      const int h = h0 + sub;
      const bool in = h < min(h1, p.H_q);
      const uint4 raw = in ? ld_stream_u4(p.q + n * p.q_stride + size_t(h) * D + 8 * chunk) : make_uint4(0, 0, 0, 0);
      float x[8], y[8];
      unpack8(raw, x), unpack8(raw, y);
      turn(raw, y, turned);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (still >> e & 1u) y[e] = x[e];
      if (in) *reinterpret_cast<uint4 *>(p.q_out + (size_t(n) * p.H_q + h) * D + 8 * chunk) = turned ? pack8(y) : raw;
    }
    h0 = max(int(blockIdx.y) * per, min(h1, p.H_q));
    load(h0);
  }
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += kAhead * HPW) {
    uint4 now[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) now[u] = raws[u];
    load(hb + kAhead * HPW);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = hb + u * HPW + sub;
      if (hb + u * HPW >= h1) break;  // the whole warp
      const bool in = h < h1;
      const int kind = h < p.H_q ? 0 : h < p.H_q + p.H_kv ? 1 : 2;
      const uint4 raw = now[u];
      float y[8];
      unpack8(raw, y);
      if (p.rot) turn(raw, y, turned && kind < 2);
      if (in && kind == 0)
        *reinterpret_cast<uint4 *>(p.q_out + (size_t(n) * p.H_q + h) * D + 8 * chunk) = turned ? pack8(y) : raw;
      // the groups' exchanges need every lane of a head, so the whole warp goes in
      if (__any_sync(0xffffffffu, in && kind > 0)) {
        const int hk = kind == 1 ? h - p.H_q : h - p.H_q - p.H_kv;
        const bool store = in && kind > 0 && write;
        uint8_t *rec = p.pages + (size_t(page) * p.H_kv + (store ? hk : 0)) * kv4_record_bytes(D, P);
        const int w = kind == 2;
        store_codes<D>(y, rec + w * kv4_code_bytes(D, P) + off * (D / 2),
                       rec + 2 * kv4_code_bytes(D, P) + w * kv4_entry_bytes(D, P) + off * (W * 4), chunk, store);
      }
    }
  }
}

// Two words (16 channels) a thread.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_read_kernel(const Kv4ReadParams p) {
  constexpr int LPH = D / 16, W = D / 64;
  pdl_wait();
  pdl_trigger();
  const long long item = (blockIdx.x * (long long)kAppendThreads + threadIdx.x) / LPH;  // (token, head, K or V)
  const int pair = threadIdx.x % LPH;
  const long long th = item >> 1;
  if (th >= (long long)p.N * p.H_kv) return;
  const int w = int(item & 1), n = int(th / p.H_kv), h = int(th - (long long)n * p.H_kv);
  const int P = 1 << p.log2P;
  const int slot = p.slots[n];
  bool in = slot >= 0;
  if (in && (slot >> p.log2P) >= p.n_pages) {
    in = false;
    atomicOr(p.status, GDN_STATUS_BAD_INDEX);
  }
  uint2 word = make_uint2(0, 0), entry = make_uint2(0, 0);
  if (in) {
    const int off = slot & (P - 1);
    const uint8_t *rec = p.pages + (size_t(slot >> p.log2P) * p.H_kv + h) * kv4_record_bytes(D, P);
    word = *reinterpret_cast<const uint2 *>(rec + w * kv4_code_bytes(D, P) + off * (D / 2) + 8 * pair);
    const uint8_t *e = rec + 2 * kv4_code_bytes(D, P) + w * kv4_entry_bytes(D, P) + off * (W * 4);
    if (W == 1) {
      entry.x = entry.y = *reinterpret_cast<const uint32_t *>(e);
    } else {
      entry = *reinterpret_cast<const uint2 *>(e + (2 * pair % W) * 4);
    }
  }
  uint4 *dst = reinterpret_cast<uint4 *>((w ? p.v : p.k) + (size_t(n) * p.H_kv + h) * D + 16 * pair);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t c = k ? word.y : word.x, g = k ? entry.y : entry.x;
    const float s = __half2float(__ushort_as_half(uint16_t(g))), b = __half2float(__ushort_as_half(uint16_t(g >> 16)));
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(s, float((c >> (4 * e)) & 15u), b);  // s * code is exact in fp32
    dst[k] = pack8(y);
  }
}

template <int D>
cudaError_t launch_append(const Kv4AppendParams &p, cudaStream_t s) {
  // Heads split until a few thousand warps are there, while each keeps a load.  32 + 8
  // + 8 heads of 128: 16 tokens 11.9 us without a split, 3.7 so; 600 tokens 12.4
  // without, 9.4 up to 608 warps, 7.9 so, 14.8 up to 9728.
  const int heads = p.H_q + 2 * p.H_kv, at_a_time = 32 / (D / 8);
  int splits = 1;
  while (splits < (heads + at_a_time - 1) / at_a_time && (long long)p.N * splits < 2432) splits *= 2;
  if (splits > heads) splits = heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.N + kAppendThreads / 32 - 1) / (kAppendThreads / 32), splits);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_append_kernel<D>, p, splits);
}

template <int D>
cudaError_t launch_read(const Kv4ReadParams &p, cudaStream_t s) {
  const long long threads = (long long)p.N * p.H_kv * 2 * (D / 16);
  return launch_pdl(kv4_read_kernel<D>, dim3(unsigned((threads + kAppendThreads - 1) / kAppendThreads)), dim3(kAppendThreads), s, p);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams &p, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch_append<64>(p, s);
    case 128: return launch_append<128>(p, s);
    default: return launch_append<256>(p, s);
  }
}

cudaError_t launch_kv4_read(const Kv4ReadParams &p, int D, cudaStream_t s) {
  switch (D) {
    case 64: return launch_read<64>(p, s);
    case 128: return launch_read<128>(p, s);
    default: return launch_read<256>(p, s);
  }
}

}  // namespace gdn

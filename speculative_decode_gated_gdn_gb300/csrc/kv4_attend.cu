// kv4_attend.cu -- causal attention of the new tokens over the paged 4-bit
// cache.
//
// Query i of row b sits at place kv_len[b] - q_count[b] + i and sees every key
// at its own place or before it:
//   o = sum_t softmax_t(scale * q . k_t) v_t.
// One pass over the keys with the running maximum m and sum l of a softmax;
// m, l and the output are held in fp32, keys and values are the exact fp32
// values base + step * code.
//
// One warp per (query, head): each lane holds D / 32 channels of q and of the
// output, a key's product is summed over the warp.
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kAttendThreads = 128;

template <int D>
__device__ __forceinline__ void kv4_load(const uint8_t *rec, int which, int P, int off, int lane, float (&x)[D / 32]) {
  constexpr int C = D / 32, W = D / 64;
  const int c0 = C * lane;
  const uint8_t *codes = rec + which * kv4_code_bytes(D, P) + off * (D / 2) + c0 / 2;
  const uint32_t entry = *reinterpret_cast<const uint32_t *>(rec + 2 * kv4_code_bytes(D, P) + which * kv4_entry_bytes(D, P) +
                                                             (off * W + (c0 / 8) % W) * 4);
  const float s = __half2float(__ushort_as_half(uint16_t(entry))), b = __half2float(__ushort_as_half(uint16_t(entry >> 16)));
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    const uint32_t v = codes[i];
    x[2 * i] = fmaf(s, float(v & 15u), b);
    x[2 * i + 1] = fmaf(s, float(v >> 4), b);
  }
}

template <int D>
__global__ void __launch_bounds__(kAttendThreads) kv4_attend_kernel(const Kv4AttendParams p) {
  constexpr int C = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, i = blockIdx.x, h = blockIdx.y * (kAttendThreads / 32) + warp;
  pdl_wait();
  pdl_trigger();
  if (h >= p.g.H_q) return;
  const int start = p.q_start[b], span = p.q_start[b + 1] - start, n = start + i;
  if (i >= span || n < 0 || n >= p.N) return;
  const int P = 1 << p.g.log2P;
  int len = p.kv_len[b];
  if (len < 0 || len > p.g.max_pages * P) {
    if (lane == 0) atomicOr(p.status, GDN_STATUS_BAD_LEN);
    len = min(max(len, 0), p.g.max_pages * P);
  }
  const int count = p.q_count[b];
  const int last = i < count ? len - count + i : -1;  // the last key this query sees
  const int hk = h / (p.g.H_q / p.g.H_kv);
  float q[C], o[C];
  const uint16_t *src = p.q + (size_t(n) * p.g.H_q + h) * D + C * lane;
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = bf2f(src[c]) * p.scale, o[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t <= last; ++t) {
    const int page = p.table[size_t(b) * p.g.max_pages + (t >> p.g.log2P)];
    if (page < 0 || page >= p.g.n_pages) {
      if (lane == 0) atomicOr(p.status, GDN_STATUS_BAD_INDEX);
      continue;
    }
    const uint8_t *rec = p.pages + (size_t(page) * p.g.H_kv + hk) * kv4_record_bytes(D, P);
    float x[C], s = 0.f;
    kv4_load<D>(rec, 0, P, t & (P - 1), lane, x);
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(q[c], x[c], s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    kv4_load<D>(rec, 1, P, t & (P - 1), lane, x);
    const float mn = fmaxf(m, s);
    const float r = m == mn ? 1.f : __expf(m - mn), w = s == mn ? 1.f : __expf(s - mn);
    l = fmaf(l, r, w);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(o[c], r, w * x[c]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : l;
  uint16_t *dst = p.out + (size_t(n) * p.g.H_q + h) * D + C * lane;
#pragma unroll
  for (int c = 0; c < C; ++c) dst[c] = f2bf(o[c] * inv);
}

}  // namespace

size_t kv4_attend_workspace_bytes(const Kv4Geom &, int, int) { return 256; }

cudaError_t launch_kv4_attend(const Kv4AttendParams &p, cudaStream_t s) {
  const dim3 grid(p.max_q, (p.g.H_q + 3) / 4, p.g.B);
  switch (p.g.D) {
    case 64: return launch_pdl(kv4_attend_kernel<64>, grid, dim3(kAttendThreads), s, p);
    case 128: return launch_pdl(kv4_attend_kernel<128>, grid, dim3(kAttendThreads), s, p);
    default: return launch_pdl(kv4_attend_kernel<256>, grid, dim3(kAttendThreads), s, p);
  }
}

}  // namespace gdn

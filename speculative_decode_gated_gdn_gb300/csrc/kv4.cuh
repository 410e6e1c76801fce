// kv4.cuh -- layout and kernel parameter blocks of the paged 4-bit key/value
// cache that the attention layers of a cohort read next to its GDN layers.
//
// A page holds P tokens (P = 16, 32 or 64).  For each kv head it is one
// contiguous record, so that whatever part of a page a warp needs arrives by
// plain contiguous copies:
//   K codes [P][D/2] | V codes [P][D/2] | K entries [P][D/64] | V entries [P][D/64]
// Byte i of a token's codes holds channel 2i in its low and 2i+1 in its high
// four bits.  Channel c belongs to group (c / 8) mod (D / 64): groups of 64
// channels made of runs of 8, so that the 8 codes of any aligned 32-bit word
// share one entry and the words of a 16-byte load cover all groups in order.
// An entry is (fp16 step, fp16 base); a channel stands for base + step * code.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

struct Kv4Geom {
  int B, H_q, H_kv, D;
  int log2P;      // tokens per page, as a power of two
  int max_pages;  // columns of the block table
  int n_pages;    // pages of the cache
};

__host__ __device__ constexpr int kv4_code_bytes(int D, int P) { return P * D / 2; }        // K or V codes of a record
__host__ __device__ constexpr int kv4_entry_bytes(int D, int P) { return P * (D / 64) * 4; }  // K or V entries
__host__ __device__ constexpr int kv4_record_bytes(int D, int P) {
  return 2 * (kv4_code_bytes(D, P) + kv4_entry_bytes(D, P));
}

struct KvPlanParams {
  const int32_t *lens, *add;
  const uint8_t *active;
  int32_t *held, *table, *free_list, *free_count;
  int32_t *q_start, *q_count, *kv_len, *slots, *positions;
  uint32_t *status;
  int B, T, N;  // T > 0: row b's tokens at b * T; T == 0: packed
  int log2P, max_pages, n_pages;
};

constexpr int kMaxRopePairs = 128;  // rot / 2 <= D / 2

struct Kv4AppendParams {
  const uint16_t *q, *k, *v;  // token n at n * stride; heads densely packed
  long long q_stride, k_stride, v_stride;
  const int32_t *positions;  // [axes][N]
  const float2 *rope;        // [max_pos][rot / 2] (cos, sin)
  const int32_t *slots;
  uint8_t *pages;
  uint16_t *q_out;
  uint32_t *status;
  int N, H_q, H_kv, rot, max_pos, n_axes, pairs;  // pairs: 1 = channels (2i, 2i+1), 0 = (i, i + rot/2)
  int log2P, n_pages;
  uint8_t axis[kMaxRopePairs];
};

struct Kv4ReadParams {
  const int32_t *slots;
  const uint8_t *pages;
  uint16_t *k, *v;
  uint32_t *status;
  int N, H_kv, log2P, n_pages;
};

struct Kv4AttendParams {
  const uint16_t *q;  // [N][H_q][D]
  const uint8_t *pages;
  const int32_t *table, *q_start, *q_count, *kv_len;
  uint16_t *out;
  void *ws;
  uint32_t *status;
  float scale;
  int N, max_q;
  uint32_t wait_limit;  // polls of a bounded wait (kWaitLimit)
  uint32_t test_hold;   // 1: the first copies of CTA 0 never count as complete (a test hook)
  Kv4Geom g;
};

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t s);
cudaError_t launch_kv4_append(const Kv4AppendParams &p, int D, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4ReadParams &p, int D, cudaStream_t s);
size_t kv4_attend_workspace_bytes(const Kv4Geom &g, int N, int max_q);
cudaError_t launch_kv4_attend(const Kv4AttendParams &p, cudaStream_t s);

}  // namespace gdn

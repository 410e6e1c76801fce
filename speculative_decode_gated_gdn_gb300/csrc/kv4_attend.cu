// kv4_attend.cu -- choice of the cache attention's form, and its workspace.
#include <atomic>

#include "kv4_attend_tc.cuh"

namespace gdn {

namespace {

int att_sms() {
  static std::atomic<int> cached[64];  // per device, 0 until looked up
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  n = cached[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    n = n < kAttMaxCtas ? n : kAttMaxCtas;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// More query rows a kv head than one 16-row tile: the tensor-core form, which
// shares every formed key among up to 128 rows.
bool att_many_rows(const Kv4Geom &g, int max_q) { return (long long)max_q * (g.H_q / g.H_kv) > kAttMaxRows; }

}  // namespace

size_t kv4_attend_workspace_bytes(const Kv4Geom &g, int, int max_q) {
  if (att_many_rows(g, max_q)) {
    switch (g.D) {
      case 64: return att_tc_ws<64>(kAttMaxCtas);
      case 128: return att_tc_ws<128>(kAttMaxCtas);
      default: return att_tc_ws<256>(kAttMaxCtas);
    }
  }
  switch (g.D) {
    case 64: return att_mma_ws<64, 16>(kAttMaxCtas);
    case 128: return att_mma_ws<128, 16>(kAttMaxCtas);
    default: return att_mma_ws<256, 16>(kAttMaxCtas);
  }
}

cudaError_t launch_kv4_attend(const Kv4AttendParams &p, cudaStream_t s) {
  const int sms = att_sms();
  if (att_many_rows(p.g, p.max_q)) {
    switch (p.g.D) {
      case 64: return launch_att_tc_64(p, sms, s);
      case 128: return launch_att_tc_128(p, sms, s);
      default: return launch_att_tc_256(p, sms, s);
    }
  }
  const int rows = (long long)p.max_q * (p.g.H_q / p.g.H_kv) <= 8 ? 8 : 16;
  switch (p.g.D) {
    case 64: return launch_att_mma_64(p, rows, sms, s);
    case 128: return launch_att_mma_128(p, rows, sms, s);
    default: return launch_att_mma_256(p, rows, sms, s);
  }
}

}  // namespace gdn

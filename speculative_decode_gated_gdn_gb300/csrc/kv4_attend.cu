// kv4_attend.cu -- choice of the cache attention's form, and its workspace.
#include <atomic>

#include "kv4_attend.cuh"

namespace gdn {

namespace {

// CTAs of the persistent grid at most: the workspace has room for the parts of
// so many, on whichever device it is used.
constexpr int kAttMaxCtas = 320;

int att_ctas() {
  static std::atomic<int> cached[64];  // per device, 0 until looked up
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 2 * 152;
  n = cached[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    n = 2 * n < kAttMaxCtas ? 2 * n : kAttMaxCtas;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

size_t kv4_attend_workspace_bytes(const Kv4Geom &g, int, int) {
  switch (g.D) {
    case 64: return att_mma_ws<64>(kAttMaxCtas);
    case 128: return att_mma_ws<128>(kAttMaxCtas);
    default: return att_mma_ws<256>(kAttMaxCtas);
  }
}

cudaError_t launch_kv4_attend(const Kv4AttendParams &p, cudaStream_t s) {
  const int ctas = att_ctas();
  switch (p.g.D) {
    case 64: return launch_att_mma_64(p, ctas, s);
    case 128: return launch_att_mma_128(p, ctas, s);
    default: return launch_att_mma_256(p, ctas, s);
  }
}

}  // namespace gdn

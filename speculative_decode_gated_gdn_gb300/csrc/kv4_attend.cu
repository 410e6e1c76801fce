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

// More query rows a kv head than a few units of eight: the tensor-core form, which
// shares every formed key among up to 128 rows.  Both sides, us (units of eight,
// tensor cores), 2 kv heads:
//                       D = 64            D = 128           D = 256
//   rows                16      24        16      24        8       16
//   1 row  of 32768     20 26   20 26     23 31   26 30     33 38   38 38
//   2 rows of 100000    31 41   37 41     42 48   56 48     61 77   93 77
//   16 rows of 2000     18 21   18 20     21 23   22 24     26 27   31 27
//   48 rows of 4000     29 38   36 38     42 45   54 45     58 69   89 69
//   64 rows of 300      18 21   18 21     21 23   21 23     26 25   27 25
// The lengths are not known on the host, so the choice is by rows alone.
bool att_many_rows(const Kv4Geom &g, int max_q) {
  return (long long)max_q * (g.H_q / g.H_kv) > (g.D == 64 ? 3 * kAttRows : g.D == 128 ? 2 * kAttRows : kAttRows);
}

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
    case 64: return att_mma_ws<64>(kAttMaxCtas);
    case 128: return att_mma_ws<128>(kAttMaxCtas);
    default: return att_mma_ws<256>(kAttMaxCtas);
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
  switch (p.g.D) {
    case 64: return launch_att_mma_64(p, sms, s);
    case 128: return launch_att_mma_128(p, sms, s);
    default: return launch_att_mma_256(p, sms, s);
  }
}

}  // namespace gdn

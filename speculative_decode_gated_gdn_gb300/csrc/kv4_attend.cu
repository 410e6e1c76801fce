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

// More query rows a kv head than a unit of eight: the tensor-core form, which
// shares every formed key among up to 128 rows.  Both sides, us, 8 rows (few, many)
// and 16 (in units of 16 rows, which were taken out, many), 2 kv heads:
//                       D = 64                  D = 128                 D = 256
//   1 row  of 32768     25 26 | 28 26           26 31 | 32 31           36 39 | 47 39
//   2 rows of 100000    31 41 | 35 41           37 49 | 45 49           64 77 | 87 77
//   16 rows of 2000     26 21 | 28 21           25 24 | 31 24           30 27 | 37 27
//   48 rows of 4000     30 38 | 33 38           34 45 | 42 45           62 70 | 79 70
// The lengths are not known on the host, so the choice is by rows alone.
bool att_many_rows(const Kv4Geom &g, int max_q) { return (long long)max_q * (g.H_q / g.H_kv) > kAttRows; }

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

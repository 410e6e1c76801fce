// kv4_attend_d64.cu -- the cache attention at head size 64.
#include "kv4_attend.cuh"

namespace gdn {

cudaError_t launch_att_mma_64(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  return launch_att_mma<64>(p, ctas, s);
}

}  // namespace gdn

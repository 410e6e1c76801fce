// kv4_attend_d256.cu -- the cache attention at head size 256.
#include "kv4_attend.cuh"

namespace gdn {

cudaError_t launch_att_mma_256(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  return launch_att_mma<256>(p, ctas, s);
}

}  // namespace gdn

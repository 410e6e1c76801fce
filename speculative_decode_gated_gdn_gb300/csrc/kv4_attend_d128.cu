// kv4_attend_d128.cu -- the cache attention at head size 128.
#include "kv4_attend.cuh"

namespace gdn {

cudaError_t launch_att_mma_128(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  return launch_att_mma<128>(p, ctas, s);
}

}  // namespace gdn

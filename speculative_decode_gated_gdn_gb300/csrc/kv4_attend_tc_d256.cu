// kv4_attend_tc_d256.cu -- the tensor-core cache attention at head size 256.
#include "kv4_attend_tc.cuh"

namespace gdn {

cudaError_t launch_att_tc_256(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  return launch_att_tc<256>(p, ctas, s);
}

}  // namespace gdn

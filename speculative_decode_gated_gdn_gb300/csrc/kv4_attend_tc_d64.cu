// kv4_attend_tc_d64.cu -- the tensor-core cache attention at head size 64.
#include "kv4_attend_tc.cuh"

namespace gdn {

cudaError_t launch_att_tc_64(const Kv4AttendParams &p, int ctas, cudaStream_t s) {
  return launch_att_tc<64>(p, ctas, s);
}

}  // namespace gdn

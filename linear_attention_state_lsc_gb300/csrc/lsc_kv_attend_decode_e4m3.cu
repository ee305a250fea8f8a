// lsc_kv_attend_decode_e4m3.cu -- decode attention instantiations for e4m3 pools.
#include "lsc_kv_attend_decode.cuh"

namespace lsc {
cudaError_t launch_kv_attend_decode_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::decode::launch_type<false, 1>(p, plan, stream);
}
}  // namespace lsc

// lsc_kv_attend_decode_f16.cu -- decode attention instantiations for f16 pools.
#include "lsc_kv_attend_decode.cuh"

namespace lsc {
cudaError_t launch_kv_attend_decode_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::decode::launch_type<false, 2>(p, plan, stream);
}
}  // namespace lsc

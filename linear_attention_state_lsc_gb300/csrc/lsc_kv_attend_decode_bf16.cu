// lsc_kv_attend_decode_bf16.cu -- decode attention instantiations for bf16 pools.
#include "lsc_kv_attend_decode.cuh"

namespace lsc {
cudaError_t launch_kv_attend_decode_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::decode::launch_type<true, 2>(p, plan, stream);
}
}  // namespace lsc

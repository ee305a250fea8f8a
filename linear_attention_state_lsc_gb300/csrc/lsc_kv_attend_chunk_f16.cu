// lsc_kv_attend_chunk_f16.cu -- many-row attention instantiations for f16 pools.
#include "lsc_kv_attend_chunk.cuh"

namespace lsc {
cudaError_t launch_kv_attend_chunk_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::chunk::launch_type<false, false>(p, plan, stream);
}
}  // namespace lsc

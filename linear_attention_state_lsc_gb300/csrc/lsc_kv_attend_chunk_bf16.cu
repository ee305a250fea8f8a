// lsc_kv_attend_chunk_bf16.cu -- many-row attention instantiations for bf16 pools.
#include "lsc_kv_attend_chunk.cuh"

namespace lsc {
cudaError_t launch_kv_attend_chunk_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::chunk::launch_type<true, false>(p, plan, stream);
}
}  // namespace lsc

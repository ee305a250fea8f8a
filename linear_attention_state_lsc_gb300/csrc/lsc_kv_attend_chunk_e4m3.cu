// lsc_kv_attend_chunk_e4m3.cu -- many-row attention instantiations for e4m3 pools.
#include "lsc_kv_attend_chunk.cuh"

namespace lsc {
cudaError_t launch_kv_attend_chunk_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::chunk::launch_type<true, true>(p, plan, stream);
}
}  // namespace lsc

// lsc_kv_attend_chunk_e2m1.cu -- many-row attention instantiations for e2m1 pools (products in f16).
#include "lsc_kv_attend_chunk.cuh"

namespace lsc {
cudaError_t launch_kv_attend_chunk_e2m1(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::chunk::launch_type<false, false, true>(p, plan, stream);
}
}  // namespace lsc

// lsc_kv_attend_chunk_f16_q_bf16.cu -- many-row attention instantiations for f16 blocks and bf16 rows of q: the expanded
// rows of e2m1 pools.
#include "lsc_kv_attend_chunk.cuh"

namespace lsc {
cudaError_t launch_kv_attend_chunk_f16_q_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::chunk::launch_type<false, false, false, true>(p, plan, stream);
}
}  // namespace lsc

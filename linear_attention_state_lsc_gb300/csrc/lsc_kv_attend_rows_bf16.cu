// lsc_kv_attend_rows_bf16.cu -- few-row attention instantiations for bf16 pools.
#include "lsc_kv_attend_rows.cuh"

namespace lsc {
cudaError_t launch_kv_attend_rows_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::rows::launch_type<true, 2>(p, plan, stream);
}
}  // namespace lsc

// lsc_kv_attend_rows_f16.cu -- few-row attention instantiations for f16 pools.
#include "lsc_kv_attend_rows.cuh"

namespace lsc {
cudaError_t launch_kv_attend_rows_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::rows::launch_type<false, 2>(p, plan, stream);
}
}  // namespace lsc

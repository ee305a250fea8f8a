// lsc_kv_attend_rows_e4m3.cu -- few-row attention instantiations for e4m3 pools.
#include "lsc_kv_attend_rows.cuh"

namespace lsc {
cudaError_t launch_kv_attend_rows_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return kv::rows::launch_type<false, 1>(p, plan, stream);
}
}  // namespace lsc

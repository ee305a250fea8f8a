// lsc_kv_attend_decode_e2m1.cu -- decode attention instantiations for e2m1 pools.
#include "lsc_kv_attend_decode4.cuh"

namespace lsc {
cudaError_t launch_kv_attend_decode_e2m1(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  switch (p.L.head_dim) {
    case 64: return kv::decode4::launch_rows<64>(p, plan, stream);
    case 128: return kv::decode4::launch_rows<128>(p, plan, stream);
    default: return kv::decode4::launch_rows<256>(p, plan, stream);
  }
}
}  // namespace lsc

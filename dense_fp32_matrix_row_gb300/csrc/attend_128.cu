// attend_128.cu -- attend.cuh for heads of 112 and 128 elements.
#include "attend.cuh"

namespace sgemm_gb300 {
cudaError_t launch_attend_128(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    return attend_of_dim<128>(p, type, nt, sms, stream);
}
}  // namespace sgemm_gb300

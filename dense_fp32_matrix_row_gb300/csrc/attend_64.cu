// attend_64.cu -- attend.cuh for heads of up to 64 elements.
#include "attend.cuh"

namespace sgemm_gb300 {
cudaError_t launch_attend_64(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    return attend_of_dim<64>(p, type, nt, sms, stream);
}
}  // namespace sgemm_gb300

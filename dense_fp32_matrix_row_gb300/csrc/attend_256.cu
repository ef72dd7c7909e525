// attend_256.cu -- attend.cuh for heads of 208 to 256 elements.
#include "attend.cuh"

namespace sgemm_gb300 {
cudaError_t launch_attend_256(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    return attend_of_dim<256>(p, type, nt, sms, stream);
}
}  // namespace sgemm_gb300

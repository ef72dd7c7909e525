// attend_192.cu -- attend.cuh for heads of 144 to 192 elements.
#include "attend.cuh"

namespace sgemm_gb300 {
cudaError_t launch_attend_192(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    return attend_of_dim<192>(p, type, nt, sms, stream);
}
}  // namespace sgemm_gb300

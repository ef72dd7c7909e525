// attend_96.cu -- attend.cuh for heads of 80 and 96 elements.
#include "attend.cuh"

namespace sgemm_gb300 {
cudaError_t launch_attend_96(const AttendParams &p, int type, int nt, int sms, cudaStream_t stream) {
    return attend_of_dim<96>(p, type, nt, sms, stream);
}
}  // namespace sgemm_gb300

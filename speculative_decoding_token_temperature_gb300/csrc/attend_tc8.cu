// The tensor-memory attention kernel over 8-bit pages.
#include "attend_tc.cuh"

namespace specdec {

cudaError_t launch_attend_tc8(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? tc::launch_typed<__nv_bfloat16, 8>(P, mr, stream) : tc::launch_typed<__half, 8>(P, mr, stream);
}

}  // namespace specdec

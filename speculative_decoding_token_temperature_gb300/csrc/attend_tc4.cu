// The tensor-memory attention kernel over 4-bit pages.
#include "attend_tc.cuh"

namespace specdec {

cudaError_t launch_attend_tc4(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? tc::launch_typed<__nv_bfloat16, true>(P, mr, stream) : tc::launch_typed<__half, true>(P, mr, stream);
}

}  // namespace specdec

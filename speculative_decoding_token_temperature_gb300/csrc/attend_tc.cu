// The tensor-memory attention kernel over 16-bit pages.
#include "attend_tc.cuh"

namespace specdec {

int attend_tc_rows(int64_t rows) { return rows <= 32 ? 32 : rows <= 128 ? 128 : 256; }

cudaError_t launch_attend_tc(const AttendParams& P, specdec_dtype dt, int mr, cudaStream_t stream) {
  return dt == SPECDEC_BF16 ? tc::launch_typed<__nv_bfloat16, false>(P, mr, stream) : tc::launch_typed<__half, false>(P, mr, stream);
}

}  // namespace specdec

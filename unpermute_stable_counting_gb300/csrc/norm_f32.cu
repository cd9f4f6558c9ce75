// The kernels of rows8.cuh for fp32 rows.
#include "rows8.cuh"

namespace mr {

MR_ROWS_TO_8(MR_DTYPE_F32)
MR_CHECK_ACCESSOR(norm_f32)

}  // namespace mr

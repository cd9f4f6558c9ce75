// The kernels of rows8.cuh for f16 rows.
#include "rows8.cuh"

namespace mr {

MR_ROWS_TO_8(MR_DTYPE_F16)
MR_CHECK_ACCESSOR(norm_f16)

}  // namespace mr

// Host halves of moe_quantize_int8 and moe_add_rms_norm; the kernels (rows8.cuh) of
// bf16 rows. Those of f16 and fp32 rows are in norm_f16.cu and norm_f32.cu.
#include "rows8.cuh"

#include <algorithm>

namespace mr {

MR_ROWS_TO_8(MR_DTYPE_BF16)
template <> cudaError_t rows_to_8<MR_DTYPE_F16>(const RowArgs&, bool, bool, cudaStream_t);
template <> cudaError_t rows_to_8<MR_DTYPE_F32>(const RowArgs&, bool, bool, cudaStream_t);

namespace {

cudaError_t launch(const RowArgs& a, int dt, bool norm, bool loose, cudaStream_t s) {
    return dt == MR_DTYPE_F32   ? rows_to_8<MR_DTYPE_F32>(a, norm, loose, s)
           : dt == MR_DTYPE_F16 ? rows_to_8<MR_DTYPE_F16>(a, norm, loose, s)
                                : rows_to_8<MR_DTYPE_BF16>(a, norm, loose, s);
}

// The bytes that every row of a tensor starts on: 16, 8, 4 or 1 at most `most`.
int start_of(const void* p, int64_t row, int64_t batch, int most) {
    int n = most;
    while (n > 1 && (!aligned(p, (uintptr_t)n) || row % n || batch % n)) n = n > 4 ? n / 2 : 1;
    return n;
}

constexpr int64_t kTop = INT64_C(1) << 40;
bool float_type(int32_t dt) { return dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16 || dt == MR_DTYPE_F32; }

}  // namespace

MR_CHECK_ACCESSOR(norm_bf16)

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_quantize_int8(const void* x, int32_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                       const int64_t* xStrides, const int64_t* numRows, void* values,
                                       const int64_t* valueStrides, float* scales, const int64_t* scaleStrides,
                                       void* stream) {
    if (!float_type(dtype)) return MR_ERR_PARAM_INVALID;
    if (batch < 1 || rows < 0 || cols < 1 || rows > MR_MAX_EXPERT_ROWS || cols > MR_MAX_EXPERT_COLS ||
        batch > MR_MAX_EXPERT_ROWS || batch * rows > INT32_MAX)
        return MR_ERR_PARAM_INVALID;
    if (batch != 1 && numRows) return MR_ERR_PARAM_INVALID;
    int64_t xb = rows * cols, xr = cols, vb = rows * cols, vr = cols, sb = rows, sr = 1;
    if (xStrides) xb = xStrides[0], xr = xStrides[1];
    if (valueStrides) vb = valueStrides[0], vr = valueStrides[1];
    if (scaleStrides) sb = scaleStrides[0], sr = scaleStrides[1];
    if (xb < 0 || xr < 0 || xb > kTop || xr > kTop) return MR_ERR_PARAM_INVALID;
    if (vr < cols || vr > kTop || vb > kTop || (batch > 1 && vb < (rows - 1) * vr + cols)) return MR_ERR_PARAM_INVALID;
    if (sr < 1 || sr > kTop || sb > kTop || (batch > 1 && sb < (rows - 1) * sr + 1)) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    if (!x || !values || !scales) return MR_ERR_PARAM_NULLPTR;
    const int64_t elem = dtype == MR_DTYPE_F32 ? 4 : 2;
    if (!aligned(x, elem) || !aligned(scales, 4) || !aligned(numRows, 8)) return MR_ERR_PARAM_INVALID;
    RowArgs a{};
    a.x = reinterpret_cast<const char*>(x);
    a.x_row = xr * elem;
    a.x_batch = xb * elem;
    a.x_end = a.x + ((batch - 1) * xb + (rows - 1) * xr + cols) * elem;
    a.rows = batch * rows;
    a.per_batch = batch > 1 ? rows : 0;
    a.K = cols;
    a.num_rows = numRows;
    a.q = reinterpret_cast<uint8_t*>(values);
    a.q_row = vr;
    a.q_batch = vb;
    a.scales = scales;
    a.s_row = sr;
    a.s_batch = sb;
    a.quant = MR_DTYPE_INT8;
    a.q_vec = start_of(values, vr, batch > 1 ? vb : 0, 8);
    const bool loose = start_of(x, a.x_row, batch > 1 ? a.x_batch : 0, 16) < 16;
    MR_TRY_CUDA(launch(a, dtype, false, loose, reinterpret_cast<cudaStream_t>(stream)));
    return MR_OK;
}

extern "C" mr_status moe_add_rms_norm(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t xStride,
                                      const void* residual, int64_t residualStride, const void* weight,
                                      int32_t weightDtype, double eps, const int64_t* numRows, void* residualOut,
                                      int64_t residualOutStride, void* y, int64_t yStride, int32_t quantDtype,
                                      void* values, int64_t valueStride, float* scales, const int64_t* scaleStrides,
                                      void* stream) {
    if (!float_type(dtype) || (weightDtype != dtype && weightDtype != MR_DTYPE_F32)) return MR_ERR_PARAM_INVALID;
    const bool eight = quantDtype != -1;
    if (eight && quantDtype != MR_DTYPE_INT8 && quantDtype != MR_DTYPE_E4M3) return MR_ERR_PARAM_INVALID;
    if (rows < 0 || cols < 1 || rows > MR_MAX_EXPERT_ROWS || cols > MR_MAX_EXPERT_COLS) return MR_ERR_PARAM_INVALID;
    if (!(eps >= 0x1p-100) || !(eps <= 0x1p100)) return MR_ERR_PARAM_INVALID;
    if (xStride < 0 || xStride > kTop) return MR_ERR_PARAM_INVALID;
    if (residual && (residualStride < 0 || residualStride > kTop)) return MR_ERR_PARAM_INVALID;
    if (residualOut && (!residual || residualOutStride < cols || residualOutStride > kTop)) return MR_ERR_PARAM_INVALID;
    if (y && (yStride < cols || yStride > kTop)) return MR_ERR_PARAM_INVALID;
    if (eight && (valueStride < cols || valueStride > kTop)) return MR_ERR_PARAM_INVALID;
    int64_t sr = quantDtype == MR_DTYPE_E4M3 ? (cols + kScaleBlock - 1) / kScaleBlock : 1, sb = 1;
    if (scaleStrides) sr = scaleStrides[0], sb = scaleStrides[1];
    if (eight && (sr < 1 || sb < 1 || sr > kTop || sb > kTop)) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    if (!x || !weight || (!y && !eight && !residualOut) || (eight && (!values || !scales))) return MR_ERR_PARAM_NULLPTR;
    const int64_t elem = dtype == MR_DTYPE_F32 ? 4 : 2;
    if (!aligned(x, elem) || !aligned(residual, elem) || !aligned(residualOut, elem) || !aligned(y, elem) ||
        !aligned(weight, weightDtype == MR_DTYPE_F32 ? 4 : elem) || !aligned(numRows, 8) || (eight && !aligned(scales, 4)))
        return MR_ERR_PARAM_INVALID;
    RowArgs a{};
    a.x = reinterpret_cast<const char*>(x);
    a.x_row = xStride * elem;
    a.x_end = a.x + ((rows - 1) * xStride + cols) * elem;
    a.residual = reinterpret_cast<const char*>(residual);
    a.residual_row = residualStride * elem;
    a.residual_end = a.residual + (residual ? ((rows - 1) * residualStride + cols) * elem : 0);
    a.h = reinterpret_cast<char*>(residualOut);
    a.h_row = residualOutStride * elem;
    a.y = reinterpret_cast<char*>(y);
    a.y_row = yStride * elem;
    a.w = reinterpret_cast<const char*>(weight);
    a.w_f32 = weightDtype == MR_DTYPE_F32;
    a.w_vec = aligned(weight, 16);
    a.eps_hi = (float)eps;
    a.eps_lo = (float)(eps - (double)a.eps_hi);
    a.rows = rows;
    a.K = cols;
    a.num_rows = numRows;
    a.quant = quantDtype;
    if (eight) {
        a.q = reinterpret_cast<uint8_t*>(values);
        a.q_row = valueStride;
        a.scales = scales;
        a.s_row = sr;
        a.s_block = sb;
        a.q_vec = start_of(values, valueStride, 0, 8);
    }
    int start = start_of(x, a.x_row, 0, 16);
    if (residual) start = std::min(start, start_of(residual, a.residual_row, 0, 16));
    if (residualOut) start = std::min(start, start_of(residualOut, a.h_row, 0, 16));
    if (y) start = std::min(start, start_of(y, a.y_row, 0, 16));
    MR_TRY_CUDA(launch(a, dtype, true, start < 16, reinterpret_cast<cudaStream_t>(stream)));
    return MR_OK;
}

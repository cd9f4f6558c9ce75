// Block quantization to e4m3 (the operand of the expert products):
//   per row r (or 128 rows) and block b of 128 columns
//     s = the smallest power of two with max(max |x|, 2^-96) <= 448 s
//     q = e4m3(x / s), round to nearest even
//
// One pass: 8 threads hold a block's 128 values in registers (16 each), find
// the maximum with three shuffles, and write 16 bytes each. HBM bound.
#include "tensor.cuh"

namespace mr {

template <int DT> struct Wide;  // 16 consecutive values of a row as floats
template <> struct Wide<MR_DTYPE_F32> {
    static __device__ __forceinline__ void load(const void* p, float (&v)[16]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 w = ld_stream_v4(reinterpret_cast<const char*>(p) + 16 * j);
            v[4 * j] = __uint_as_float(w.x);
            v[4 * j + 1] = __uint_as_float(w.y);
            v[4 * j + 2] = __uint_as_float(w.z);
            v[4 * j + 3] = __uint_as_float(w.w);
        }
    }
};
template <int DT> struct Wide16 {
    static __device__ __forceinline__ void load(const void* p, float (&v)[16]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 w = ld_stream_v4(reinterpret_cast<const char*>(p) + 16 * j);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[8 * j + 2 * i] = Elem<DT>::to_f32((uint16_t)(u[i] & 0xFFFFu));
                v[8 * j + 2 * i + 1] = Elem<DT>::to_f32((uint16_t)(u[i] >> 16));
            }
        }
    }
};
template <> struct Wide<MR_DTYPE_F16> : Wide16<MR_DTYPE_F16> {};
template <> struct Wide<MR_DTYPE_BF16> : Wide16<MR_DTYPE_BF16> {};

struct QuantArgs {
    const void* x;
    int64_t rows, K, x_stride;
    const int64_t* num_rows;
    uint8_t* q;
    int64_t q_stride;
    float* scales;
    int64_t row_step, block_step;
    int blocks;    // ceil(K / 128)
    int vec_in;    // rows readable as 16-byte vectors
    int vec_out;   // q rows start on 16 bytes
};

template <int DT>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
    pdl_enter();
    int64_t rows = a.rows;
    if (a.num_rows) rows = max((int64_t)0, min(rows, *a.num_rows));
    const int64_t total = rows * a.blocks * 8;
    // a block's 8 threads are in one warp and leave together: total is a multiple of 8
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const unsigned group = 0xFFu << (threadIdx.x & 24);
        const int64_t rb = i >> 3;
        const int64_t r = rb / a.blocks;
        const int b = (int)(rb - r * a.blocks);
        const int64_t c0 = (int64_t)b * kScaleBlock + (i & 7) * 16;
        constexpr int kElem = DT == MR_DTYPE_F32 ? 4 : 2;
        float v[16];
        if (a.vec_in && c0 + 16 <= a.K) {
            Wide<DT>::load(reinterpret_cast<const char*>(a.x) + (r * a.x_stride + c0) * kElem, v);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = c0 + j < a.K ? load_f32(a.x, r * a.x_stride + c0 + j, DT) : 0.0f;
        }
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[j]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(group, m, o));
        float s, inv;
        block_scale(m, &s, &inv);
        if ((i & 7) == 0) a.scales[r * a.row_step + b * a.block_step] = s;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = e4m3x4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
        uint8_t* dst = a.q + r * a.q_stride + c0;
        if (c0 < a.K) {
            if (a.vec_out && c0 + 16 <= a.K) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                for (int j = 0; j < 16 && c0 + j < a.K; ++j) dst[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
}

// 128 x 128 blocks (weights, quantized once when a model is loaded): one block
// of threads per block of values, read twice.
__global__ void __launch_bounds__(256)
    quantize_tile_kernel(const void* x, int dt, int64_t rows, int64_t K, int64_t x_stride,
                         int64_t x_batch, uint8_t* q, int64_t q_stride, int64_t q_batch, float* scales,
                         int row_blocks, int blocks) {
    pdl_enter();
    __shared__ uint32_t warp_max[8];
    const int b = blockIdx.x % blocks;
    const int64_t rest = blockIdx.x / blocks;
    const int rb = (int)(rest % row_blocks);
    const int64_t e = rest / row_blocks;
    const int64_t r0 = (int64_t)rb * kScaleBlock, c = (int64_t)b * kScaleBlock + (threadIdx.x & 127);
    const int64_t r1 = min(r0 + kScaleBlock, rows);
    uint32_t m = 0u;
    if (c < K)
        for (int64_t r = r0 + (threadIdx.x >> 7); r < r1; r += 2)
            m = max(m, abs_bits(load_f32(x, e * x_batch + r * x_stride + c, dt)));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, warp_max[j]);
    float s, inv;
    block_scale(m, &s, &inv);
    if (threadIdx.x == 0) scales[(e * row_blocks + rb) * blocks + b] = s;
    if (c < K)
        for (int64_t r = r0 + (threadIdx.x >> 7); r < r1; r += 2)
            q[e * q_batch + r * q_stride + c] = (uint8_t)__nv_cvt_float_to_fp8(
                load_f32(x, e * x_batch + r * x_stride + c, dt) * inv, __NV_SATFINITE, __NV_E4M3);
}

cudaError_t enqueue_quantize(const void* x, int dt, int64_t rows, int64_t K, int64_t xStride,
                             const int64_t* numRows, void* q, int64_t qStride, float* scales,
                             int64_t rowStep, int64_t blockStep, cudaStream_t stream) {
    const int elem = dt == MR_DTYPE_F32 ? 4 : 2;
    QuantArgs a;
    a.x = x;
    a.rows = rows;
    a.K = K;
    a.x_stride = xStride;
    a.num_rows = numRows;
    a.q = reinterpret_cast<uint8_t*>(q);
    a.q_stride = qStride;
    a.scales = scales;
    a.row_step = rowStep;
    a.block_step = blockStep;
    a.blocks = (int)((K + kScaleBlock - 1) / kScaleBlock);
    a.vec_in = (reinterpret_cast<uintptr_t>(x) % 16 == 0) && (xStride * elem) % 16 == 0;
    a.vec_out = (reinterpret_cast<uintptr_t>(q) % 16 == 0) && qStride % 16 == 0;
    const int64_t total = rows * a.blocks * 8;
    const int64_t grid = (total + 255) / 256;
    auto kernel = dt == MR_DTYPE_F32   ? quantize_kernel<MR_DTYPE_F32>
                  : dt == MR_DTYPE_F16 ? quantize_kernel<MR_DTYPE_F16>
                                       : quantize_kernel<MR_DTYPE_BF16>;
    const int64_t most = (int64_t)device_sm_count() * 8 * 16;
    return launch_pdl(kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0, stream, a);
}

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_quantize(const void* x, int32_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                  const int64_t* xStrides, int32_t blockRows, const int64_t* numRows,
                                  void* values, const int64_t* valueStrides, float* scales,
                                  const int64_t* scaleStrides, void* stream) {
    if (dtype != MR_DTYPE_F16 && dtype != MR_DTYPE_BF16 && dtype != MR_DTYPE_F32) return MR_ERR_PARAM_INVALID;
    if (batch < 1 || rows < 0 || cols < 1 || (blockRows != 1 && blockRows != kScaleBlock))
        return MR_ERR_PARAM_INVALID;
    if (rows > MR_MAX_EXPERT_ROWS || cols > MR_MAX_EXPERT_ROWS || batch > MR_MAX_EXPERT_ROWS)
        return MR_ERR_PARAM_INVALID;
    if (blockRows == 1 && batch != 1) return MR_ERR_PARAM_INVALID;
    if (blockRows != 1 && numRows) return MR_ERR_PARAM_INVALID;
    const int64_t cb = (cols + kScaleBlock - 1) / kScaleBlock, rb = (rows + kScaleBlock - 1) / kScaleBlock;
    // contiguous unless strides say otherwise: {batch, row} of x and of values, {row, block} of scales
    int64_t xb = rows * cols, xr = cols, vb = rows * cols, vr = cols, sr = cb, sb = 1;
    if (xStrides) xb = xStrides[0], xr = xStrides[1];
    if (valueStrides) vb = valueStrides[0], vr = valueStrides[1];
    if (scaleStrides) sr = scaleStrides[0], sb = scaleStrides[1];
    const int64_t top = INT64_C(1) << 40;
    if (xb < 0 || xr < 0 || xb > top || xr > top || sr < 1 || sb < 1 || sr > top || sb > top)
        return MR_ERR_PARAM_INVALID;
    if (vr < cols || vr > top || vb > top || (batch > 1 && vb < (rows - 1) * vr + cols)) return MR_ERR_PARAM_INVALID;
    if (blockRows != 1 && scaleStrides) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    if (!x || !values || !scales) return MR_ERR_PARAM_NULLPTR;
    const uintptr_t elem = dtype == MR_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(x) % elem || reinterpret_cast<uintptr_t>(scales) % 4) return MR_ERR_PARAM_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (blockRows == 1) {
        MR_TRY_CUDA(enqueue_quantize(x, dtype, rows, cols, xr, numRows, values, vr, scales, sr, sb, s));
    } else {
        if (batch * rb * cb > INT32_MAX) return MR_ERR_PARAM_INVALID;
        MR_TRY_CUDA(launch_pdl(quantize_tile_kernel, dim3((unsigned)(batch * rb * cb)), dim3(256), 0, s, x,
                               (int)dtype, rows, cols, xr, xb, reinterpret_cast<uint8_t*>(values), vr, vb,
                               scales, (int)rb, (int)cb));
    }
    MR_TRY_CUDA(cudaGetLastError());
    return MR_OK;
}

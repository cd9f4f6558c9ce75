// Block quantization to e4m3 (the operand of the expert products):
//   per row r (or 128 rows) and block b of 128 columns
//     s = the smallest power of two with max(max |x|, 2^-96) <= 448 s
//     q = e4m3(x / s), round to nearest even
//
// One pass: 8 lanes hold a block's 128 values in registers, find the maximum with
// three shuffles, and write them.
#include "tensor.cuh"

namespace mr {

// max(m, |v|), NaN if either is (one instruction).
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(m), "f"(v));
    return r;
}

// A lane's 16 values of a block, as 16-byte pieces 128 bytes apart (8 lanes read
// whole lines).
template <int DT> struct Piece {
    static constexpr int kValues = DT == MR_DTYPE_F32 ? 4 : 8;  // of a piece
    static constexpr int kElem = 16 / kValues;
    static constexpr int kPieces = 16 / kValues;
    static constexpr int kStep = 8 * kValues;                   // values from piece to piece

    // A piece of a row that starts on 16 bytes, or its values one by one.
    static __device__ __forceinline__ uint4 load(const char* row, uint32_t col, int64_t K, bool vec) {
        if (vec && col + kValues <= K) return ld_stream_v4(row + col * kElem);
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < kValues; ++j) {
            if (col + j >= K) break;
            if (DT == MR_DTYPE_F32) u[j & 3] = reinterpret_cast<const uint32_t*>(row)[col + j];
            else u[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[col + j] << (16 * (j & 1));
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    // 16 bytes that start `off` bytes into two aligned words of 16: words by selection, halves by a shift.
    static __device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t off) {
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (off & 8u) {
#pragma unroll
            for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
        }
        if (off & 4u) {
#pragma unroll
            for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
        }
        if (DT != MR_DTYPE_F32) {
            const uint32_t bits = (off & 2u) * 8u;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], bits);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The pieces of a row that starts anywhere, from the aligned words that hold them; inside: the 16 bytes
    // on either side of the row belong to x too, otherwise words outside [lo, hi) are left alone.
    static __device__ __forceinline__ void load_loose(uint4 (&v)[kPieces], const char* row, uint32_t col, int64_t K,
                                                      bool inside, const char* lo, const char* hi) {
        const char* p = row + col * kElem;
        const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);  // the same for all pieces
        const char* q = p - off;
        const uint32_t next = off ? 16 : 0;
        if (inside && col + (kPieces - 1) * kStep + kValues <= K) {
            uint4 b[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                v[i] = __ldg(reinterpret_cast<const uint4*>(q + i * 128));
                b[i] = __ldg(reinterpret_cast<const uint4*>(q + i * 128 + next));
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) v[i] = shifted(v[i], b[i], off);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const char* w = q + i * 128;
            if (col + i * kStep + kValues <= K && w >= lo && w + next + 16 <= hi)
                v[i] = shifted(__ldg(reinterpret_cast<const uint4*>(w)), __ldg(reinterpret_cast<const uint4*>(w + next)), off);
            else v[i] = load(row, col + i * kStep, K, false);
        }
    }
    static __device__ __forceinline__ void widen(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MR_DTYPE_F32) {
                v[i] = __uint_as_float(u[i]);
            } else if constexpr (DT == MR_DTYPE_BF16) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(reinterpret_cast<const __half2&>(u[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

struct QuantArgs {
    const void* x;
    const char* x_end;  // past its last row's last value
    int64_t rows, K, x_stride;
    const int64_t* num_rows;
    uint8_t* q;
    int64_t q_stride;
    float* scales;
    int64_t row_step, block_step;
    uint32_t blocks;        // ceil(K / 128)
    uint32_t magic, shift;  // i / blocks = umulhi(i, magic) >> shift for i < 2^31 (magic 0: blocks is 1)
    int vec_out;            // q rows start on 16 bytes
};

// kItems blocks per 8 lanes, all loads before the first use. The instructions are
// what to keep low: 10 per value here, which fill 62 % of the issue slots, and
// 32768 x 4096 bf16 rows take 60 to 61 us, 0.98 of the copy rate; with 8 values per
// lane and 64-bit index arithmetic there were 19, and it took 75.6 us.
// LOOSE: rows that do not start on 16 bytes, by aligned words shifted into place
// (27285 x 5005 bf16: 104 us, fp32 136; rows of 5008 take 87 and 120; with bounds
// checks and a load-and-shift per piece it took 131 and 228).
template <int DT, int kItems, bool LOOSE>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
    pdl_enter();
    using P = Piece<DT>;
    int64_t rows = a.rows;
    if (a.num_rows) rows = max((int64_t)0, min(rows, *a.num_rows));
    const uint32_t total = (uint32_t)(rows * a.blocks);
    const uint32_t first = blockIdx.x * (32 * kItems) + (threadIdx.x >> 3);
    if (blockIdx.x * (32 * kItems) >= total) return;
    const int sub = threadIdx.x & 7;
    uint4 raw[kItems][P::kPieces];
    uint32_t row[kItems], col[kItems];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
        const uint32_t i = min(first + n * 32, total - 1);  // past the end: the last block again, not stored
        row[n] = a.magic ? __umulhi(i, a.magic) >> a.shift : i;
        col[n] = (i - row[n] * a.blocks) * kScaleBlock + sub * P::kValues;
        // (a row or block out of range: the first one again)
        if (!MR_IN_RANGE(row[n], rows, 971) || !MR_IN_RANGE(col[n] / kScaleBlock, a.blocks, 972))
            row[n] = 0u, col[n] = sub * P::kValues;
        const char* src = reinterpret_cast<const char*>(a.x) + row[n] * a.x_stride * P::kElem;
        if constexpr (LOOSE) {
            const bool inside = a.x_stride >= 8 && row[n] - 1u < (uint32_t)a.rows - 2u;
            P::load_loose(raw[n], src, col[n], a.K, inside, reinterpret_cast<const char*>(a.x), a.x_end);
        } else {
#pragma unroll
            for (int p = 0; p < P::kPieces; ++p) raw[n][p] = P::load(src, col[n] + p * P::kStep, a.K, true);
        }
    }
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
        float v[16], m = 0.0f;
#pragma unroll
        for (int p = 0; p < P::kPieces; ++p) P::widen(raw[n][p], v + p * P::kValues);
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max_abs(m, v[j]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (first + n * 32 >= total) continue;
        float s, inv;
        block_scale(__float_as_uint(m), &s, &inv);
        if (sub == 0) a.scales[row[n] * a.row_step + (col[n] / kScaleBlock) * a.block_step] = s;
        uint8_t* dst = a.q + row[n] * a.q_stride + col[n];
#pragma unroll
        for (int p = 0; p < P::kPieces; ++p) {
            uint32_t q[P::kValues / 4];
#pragma unroll
            for (int j = 0; j < P::kValues / 4; ++j) {
                const float* f = v + p * P::kValues + 4 * j;
                q[j] = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            }
            if (a.vec_out && col[n] + p * P::kStep + P::kValues <= a.K) {
                if constexpr (P::kValues == 8)
                    *reinterpret_cast<uint2*>(dst + p * P::kStep) = make_uint2(q[0], q[1]);
                else *reinterpret_cast<uint32_t*>(dst + p * P::kStep) = q[0];
            } else {
#pragma unroll
                for (int j = 0; j < P::kValues; ++j)
                    if (col[n] + p * P::kStep + j < a.K)
                        dst[p * P::kStep + j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
}

template <int DT, bool LOOSE>
cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t s) {
    // two blocks per 8 lanes once that still fills the SMs twice over
    const int64_t total = a.rows * a.blocks;
    if (total >= (int64_t)device_sm_count() * 8 * 64 * 2)
        return launch_pdl(quantize_kernel<DT, 2, LOOSE>, dim3((unsigned)((total + 63) / 64)), dim3(256), 0, s, a);
    return launch_pdl(quantize_kernel<DT, 1, LOOSE>, dim3((unsigned)((total + 31) / 32)), dim3(256), 0, s, a);
}

template <bool LOOSE> cudaError_t launch_quantize(const QuantArgs& a, int dt, cudaStream_t s) {
    return dt == MR_DTYPE_F32   ? launch_quantize<MR_DTYPE_F32, LOOSE>(a, s)
           : dt == MR_DTYPE_F16 ? launch_quantize<MR_DTYPE_F16, LOOSE>(a, s)
                                : launch_quantize<MR_DTYPE_BF16, LOOSE>(a, s);
}

// 128 x 128 blocks (weights, quantized once when a model is loaded): one block
// of threads per block of values, read twice, a value per thread and access. 128
// matrices of 2048 x 4096 bf16 take 1105 us, 2.3 times their bytes at the copy rate.
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
    if (!MR_IN_RANGE(r0, rows, 973) || !MR_IN_RANGE((int64_t)b * kScaleBlock, K, 974)) return;
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
    a.x_end = reinterpret_cast<const char*>(x) + ((rows - 1) * xStride + K) * elem;
    a.rows = rows;
    a.K = K;
    a.x_stride = xStride;
    a.num_rows = numRows;
    a.q = reinterpret_cast<uint8_t*>(q);
    a.q_stride = qStride;
    a.scales = scales;
    a.row_step = rowStep;
    a.block_step = blockStep;
    a.blocks = (uint32_t)((K + kScaleBlock - 1) / kScaleBlock);
    a.vec_out = (reinterpret_cast<uintptr_t>(q) % 16 == 0) && qStride % 16 == 0;
    // ceil(2^(31 + l) / blocks) for 2^(l - 1) < blocks <= 2^l: below 2^32, and exact for i < 2^31
    int l = 0;
    while ((1u << l) < a.blocks) ++l;
    a.magic = l ? (uint32_t)(((1ull << (31 + l)) + a.blocks - 1) / a.blocks) : 0u;
    a.shift = l ? l - 1 : 0;
    const bool loose = reinterpret_cast<uintptr_t>(x) % 16 != 0 || (xStride * elem) % 16 != 0;
    return loose ? launch_quantize<true>(a, dt, stream) : launch_quantize<false>(a, dt, stream);
}

MR_CHECK_ACCESSOR(quantize)

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_quantize(const void* x, int32_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                  const int64_t* xStrides, int32_t blockRows, const int64_t* numRows,
                                  void* values, const int64_t* valueStrides, float* scales,
                                  const int64_t* scaleStrides, void* stream) {
    if (dtype != MR_DTYPE_F16 && dtype != MR_DTYPE_BF16 && dtype != MR_DTYPE_F32) return MR_ERR_PARAM_INVALID;
    if (batch < 1 || rows < 0 || cols < 1 || (blockRows != 1 && blockRows != kScaleBlock))
        return MR_ERR_PARAM_INVALID;
    if (rows > MR_MAX_EXPERT_ROWS || cols > MR_MAX_EXPERT_COLS || batch > MR_MAX_EXPERT_ROWS)
        return MR_ERR_PARAM_INVALID;
    if (blockRows == 1 && rows * ((cols + kScaleBlock - 1) / kScaleBlock) > INT32_MAX) return MR_ERR_PARAM_INVALID;
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
    if (!aligned(x, elem) || !aligned(scales, 4) || !aligned(numRows, 8)) return MR_ERR_PARAM_INVALID;
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

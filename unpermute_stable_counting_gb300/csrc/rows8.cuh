// Rows to 8 bits in one pass over them: with a root-mean-square norm (and the
// residual's addition) before, or alone.
//   h = x + residual, rounded to x's type
//   r = 1 / sqrt(mean(h^2) + eps), rounded to fp32 once
//   y = (h r) w, each product rounded to fp32
//   out: y in x's type; int8 rows, q = round(y (127 / a)), s = a / 127 with
//   a = max(max |y|, 2^-96) of the row; or e4m3 blocks as moe_quantize makes them
//
// A row's values stay in registers (32 a thread, fewer of short rows and of fp32 ones; a warp, 128,
// 256 or 512 threads a row) from the load to the stores, so x and residual are read once. Rows of more
// than 16384 values (8192 of fp32 rows' norm) are read once more for every sweep that follows the first: the
// norm's sum is one, int8's maximum another, the stores the last.
//
// The mean of squares is kept in two fp32 numbers (two-sum steps, the squares'
// own rounding errors included), so that r is the correctly rounded value but for
// one row in a million: an 8-bit result does not depend on how the sum was cut into threads.
#pragma once

#include "rows.cuh"

namespace mr {

struct RowArgs {
    const char* x;
    int64_t x_row, x_batch;  // byte strides
    const char* x_end;       // past its last value
    const char* residual;
    int64_t residual_row;
    const char* residual_end;
    char* h;                 // the residual's successor
    int64_t h_row;
    char* y;
    int64_t y_row;
    const char* w;
    int w_f32, w_vec;        // w_vec: starts on 16 bytes
    float eps_hi, eps_lo;    // eps as a sum
    int64_t rows, per_batch, K;
    const int64_t* num_rows;
    uint8_t* q;
    int64_t q_row, q_batch;
    int q_vec;               // rows of q start on this many bytes: 8, 4 or 1
    float* scales;
    int64_t s_row, s_block, s_batch;
    int quant;               // MR_DTYPE_INT8, MR_DTYPE_E4M3, or -1
};

// (s, e) + v: s + e stays the sum, s is its fp32 value
__device__ __forceinline__ void two_add(float& s, float& e, float v, float v_low) {
    const float t = __fadd_rn(s, v), b = __fsub_rn(t, s);
    e = __fadd_rn(__fadd_rn(e, v_low), __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(v, b)));
    s = t;
}

// The same for v >= 0 and s >= 0: the smaller one's lost digits, with two instructions less (the norm's time is
// its instructions: it issues three quarters of what it could). A NaN is in s.
__device__ __forceinline__ void two_add_positive(float& s, float& e, float v) {
    const float t = __fadd_rn(s, v), hi = fmaxf(s, v), lo = fminf(s, v);
    e = __fadd_rn(e, __fsub_rn(lo, __fsub_rn(t, hi)));
    s = t;
}

// 1 / sqrt(v + v_low), v a normal number: a Newton step whose residual is formed without rounding
__device__ __forceinline__ float rsqrt_rn(float v, float v_low) {
    if (!(v < __int_as_float(0x7F800000))) return v > 0.0f ? 0.0f : v;  // infinity, NaN
    const float r = rsqrtf(v), p = __fmul_rn(r, r), p_low = __fmaf_rn(r, r, -p);
    float t = __fmaf_rn(-v, p, 1.0f);
    t = __fmaf_rn(-v, p_low, t);
    t = __fmaf_rn(-v_low, p, t);
    return __fmaf_rn(__fmul_rn(0.5f, r), t, r);
}

template <int DT> __device__ __forceinline__ void widen(const uint4& w, float* v) { Piece<DT>::widen(w, v); }
template <int DT> __device__ __forceinline__ uint4 narrow(const float* v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MR_DTYPE_F32) {
            u[i] = __float_as_uint(v[i]);
        } else if constexpr (DT == MR_DTYPE_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = reinterpret_cast<const uint32_t&>(b);
        } else {
            const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = reinterpret_cast<const uint32_t&>(b);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// 16 bytes of a row that starts anywhere, from the aligned words that hold them; inside:
// the 16 bytes on either side of the row belong to the tensor too, otherwise words
// outside [lo, hi) are left alone.
template <int DT>
__device__ __forceinline__ uint4 load_any(const char* row, uint32_t col, int64_t K, bool inside, const char* lo,
                                          const char* hi) {
    using P = Piece<DT>;
    const char* p = row + (int64_t)col * P::kElem;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* q = p - off;
    const uint32_t next = off ? 16 : 0;
    if (col + P::kValues <= K && (inside || (q >= lo && q + next + 16 <= hi))) {
        const uint4 a = ld_stream_v4(q), b = ld_stream_v4(q + next);
        return P::shifted(a, b, off);
    }
    return P::load(row, col, K, false);
}

template <int DT> __device__ __forceinline__ void store_one(char* p, const uint4& w, int j) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (DT == MR_DTYPE_F32) reinterpret_cast<uint32_t*>(p)[j] = u[j];
    else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(u[j >> 1] >> (16 * (j & 1)));
}

// The lanes' 16-byte pieces, side by side, to a row; all lanes of the warp call it.
// LOOSE: the row starts anywhere. Aligned words then leave, each made of a lane's
// piece and the end of its neighbour's, and what is left at either end goes one by one.
template <int DT, bool LOOSE>
__device__ __forceinline__ void store_piece(char* row, uint32_t col, int64_t K, const uint4& w) {
    using P = Piece<DT>;
    char* p = row + (int64_t)col * P::kElem;
    const int64_t left = K - (int64_t)col;
    const int n = left < 0 ? 0 : left < P::kValues ? (int)left : P::kValues;
    if constexpr (!LOOSE) {
        if (n == P::kValues) {
            *reinterpret_cast<uint4*>(p) = w;
        } else {
#pragma unroll
            for (int j = 0; j < P::kValues; ++j)
                if (j < n) store_one<DT>(p, w, j);
        }
        return;
    }
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u), head = off ? 16 - off : 16;  // the same for all lanes
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, w.x, 1);
    before.y = __shfl_up_sync(0xffffffffu, w.y, 1);
    before.z = __shfl_up_sync(0xffffffffu, w.z, 1);
    before.w = __shfl_up_sync(0xffffffffu, w.w, 1);
    const int lane = threadIdx.x & 31;
    const bool mine = (lane > 0 || !off) && n * P::kElem >= head;
    const bool next = off && lane < 31 && (left - P::kValues) * P::kElem >= head;  // the neighbour stores this piece's end
    if (mine) *reinterpret_cast<uint4*>(p - off) = off ? P::shifted(before, w, (uint32_t)head) : w;
#pragma unroll
    for (int j = 0; j < P::kValues; ++j) {
        const bool in_head = j * P::kElem < head;
        if (j < n && (in_head ? !mine : !next)) store_one<DT>(p, w, j);
    }
}

// A thread's 8-bit results of one piece, 4 to a word.
template <int DT> __device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t* q, int n, int vec) {
    constexpr int V = Piece<DT>::kValues;
    if (n >= V && vec >= V) {
        if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
        else *reinterpret_cast<uint32_t*>(p) = q[0];
    } else if (n >= V && vec >= 4) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) reinterpret_cast<uint32_t*>(p)[j] = q[j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < n) p[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
    }
}

// Four fp32 numbers of at most 127 to int8, to nearest even: 1.5 * 2^23 leaves the integer in the low byte.
__device__ __forceinline__ uint32_t int8x4(const float* v, float inv) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// TPR threads a row (32: eight rows a block), PER values each in pieces of 16 bytes TPR
// pieces apart. LONG: rows of more than PER TPR values. Blocks of as few registers as
// let an SM hold 1280 threads, 1024 with the norm or of fp32 rows: threads in flight are worth a few spilled
// words, but not many. (The norm of 16384 x 7168 bf16 rows with residual, bf16 and e4m3 results: 191 us, 64 registers
// that spill 80 bytes; with 768 threads, 80 registers and no spills, 207; with 1280, 48 registers and 360 bytes, 249. The
// same of fp32 rows: 410, with 768 threads 630. 65536 x 4096 bf16 rows to int8: 132, 48 registers that spill 20 bytes;
// with 1024 threads and no spills 142.) Persistent blocks whose next
// row comes to shared memory meanwhile were slower (251 and 146), and so were 16 values
// a thread (219 and 181); fp32 rows' norm has 16 (with 32 847 us instead of 415), alone they have 32.
template <int DT, int TPR, int PER, bool NORM, bool LOOSE, bool LONG>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR,
                                  (NORM || DT == MR_DTYPE_F32 ? 1024 : 1280) / (TPR == 32 ? 256 : TPR))
    rows_kernel(const RowArgs a) {
    using P = Piece<DT>;
    constexpr int V = P::kValues, kPieces = PER / V, kWarps = TPR / 32;
    __shared__ float2 part_sum[kWarps];
    __shared__ uint32_t part_max[kWarps];
    pdl_enter();
    int64_t rows = a.rows;
    if (a.num_rows) rows = max((int64_t)0, min(rows, *a.num_rows));
    const int lane = threadIdx.x & 31, t = TPR == 32 ? lane : (int)threadIdx.x, warp = t >> 5;
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (row >= rows || !MR_IN_RANGE(row, a.rows, 981)) return;
    const int64_t batch = a.per_batch ? row / a.per_batch : 0, r_in = row - batch * a.per_batch;
    const char* xr = a.x + batch * a.x_batch + r_in * a.x_row;
    const char* rr = NORM && a.residual ? a.residual + row * a.residual_row : nullptr;
    char* hr = NORM && a.h ? a.h + row * a.h_row : nullptr;
    char* yr = NORM && a.y ? a.y + row * a.y_row : nullptr;
    uint8_t* qr = a.q + batch * a.q_batch + r_in * a.q_row;
    float* sr = a.scales + batch * a.s_batch + r_in * a.s_row;

    float v[PER];
    auto column = [&](int64_t base, int i) { return (uint32_t)(base + (int64_t)(i * TPR + t) * V); };
    // (rows before and behind it, whose 16 bytes next to it are rows' too)
    const bool inside = LOOSE && !a.per_batch && row > 0 && row + 1 < a.rows && a.K * P::kElem >= 16 &&
                        a.x_row >= a.K * P::kElem && (!NORM || !rr || a.residual_row >= a.K * P::kElem);
    auto piece = [&](const char* p, uint32_t col, const char* lo, const char* hi) {
        if constexpr (LOOSE) return load_any<DT>(p, col, a.K, inside, lo, hi);
        return P::load(p, col, a.K, true);
    };
    // the values of h from `base` on; first: the first time, when h is also written
    auto fetch = [&](int64_t base, bool first) {
        uint4 x[kPieces], res[NORM ? kPieces : 1];
        const bool again = LONG && !first && rr && hr;
        const char* src = again ? hr : xr;
        const bool add = rr && !again;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t col = column(base, i);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (NORM) res[NORM ? i : 0] = x[i];
            if (col >= a.K) continue;
            if (again) x[i] = P::load(src, col, a.K, false);
            else x[i] = piece(src, col, a.x, a.x_end);
            if (NORM && add) res[NORM ? i : 0] = piece(rr, col, a.residual, a.residual_end);
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            widen<DT>(x[i], v + i * V);
            if (!NORM || !add) continue;
            float b[V];
            widen<DT>(res[NORM ? i : 0], b);
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] = __fadd_rn(v[i * V + j], b[j]);
            const uint4 h = narrow<DT>(b);
            widen<DT>(h, v + i * V);
            if (first && hr) store_piece<DT, LOOSE>(hr, column(base, i), a.K, h);
        }
    };
    const int64_t step = LONG ? PER * TPR : a.K;
    if (!LONG) fetch(0, true);

    float r = 1.0f;
    if constexpr (NORM) {
        // scale 1, or 2^-80 where the squares pass fp32's range
        auto sums = [&](float f, bool first, float& s, float& e) {
            // four sums side by side: a step's six additions follow one another
            float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, e4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int64_t base = 0; base < a.K; base += step) {
                if (LONG) fetch(base, first);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float u = f == 1.0f ? v[j] : v[j] * f, sq = __fmul_rn(u, u);
                    // (a square of 11 bits is exact)
                    two_add_positive(s4[j & 3], e4[j & 3], sq);
                    if (DT == MR_DTYPE_F32) e4[j & 3] = __fadd_rn(e4[j & 3], __fmaf_rn(u, u, -sq));
                }
            }
            two_add(s4[0], e4[0], s4[1], e4[1]);
            two_add(s4[2], e4[2], s4[3], e4[3]);
            two_add(s4[0], e4[0], s4[2], e4[2]);
            s = s4[0], e = e4[0];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
                two_add(s, e, s2, e2);
            }
            if (kWarps > 1) {
                if (lane == 0) part_sum[warp] = make_float2(s, e);
                __syncthreads();
                const float2 p = part_sum[lane % kWarps];
                s = p.x, e = p.y;
#pragma unroll
                for (int o = kWarps / 2; o > 0; o >>= 1) {
                    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
                    two_add(s, e, s2, e2);
                }
            }
        };
        const float count = (float)a.K;  // at most 2^24: exact
        float s, e;
        sums(1.0f, true, s, e);
        const bool small = s < __int_as_float(0x7F800000);
        float eps_hi = a.eps_hi, eps_lo = a.eps_lo;
        if (!small) {
            if (kWarps > 1) __syncthreads();
            sums(0x1p-80f, false, s, e);
            // (2^-160 is no fp32 number)
            eps_hi = __fmul_rn(__fmul_rn(eps_hi, 0x1p-80f), 0x1p-80f);
            eps_lo = __fmul_rn(__fmul_rn(eps_lo, 0x1p-80f), 0x1p-80f);
        }
        const bool finite = s < __int_as_float(0x7F800000);
        float m = __fdiv_rn(s, count), low = 0.0f;
        if (finite) {
            low = __fdividef(__fmaf_rn(-m, count, s) + e, count);
            two_add(m, low, eps_hi, eps_lo);
        }
        r = rsqrt_rn(m, low);
        if (!small && finite) r *= 0x1p-80f;
    }
    auto norm = [&](int64_t base) {
        if constexpr (NORM) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t col = column(base, i);
                if (col >= a.K) continue;
                float w[V];
                if (a.w_f32 && DT != MR_DTYPE_F32) {
                    const float* p = reinterpret_cast<const float*>(a.w) + col;
                    if (a.w_vec && col + V <= a.K) {
#pragma unroll
                        for (int j = 0; j < V / 4; ++j) {
                            const float4 f = __ldg(reinterpret_cast<const float4*>(p) + j);
                            w[4 * j] = f.x, w[4 * j + 1] = f.y, w[4 * j + 2] = f.z, w[4 * j + 3] = f.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < V; ++j) w[j] = col + j < a.K ? __ldg(p + j) : 0.0f;
                    }
                } else {
                    const uint4 u = a.w_vec && col + V <= a.K
                                        ? __ldg(reinterpret_cast<const uint4*>(a.w + (int64_t)col * P::kElem))
                                        : P::load(a.w, col, a.K, false);
                    widen<DT>(u, w);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) v[i * V + j] = __fmul_rn(__fmul_rn(v[i * V + j], r), w[j]);
            }
        }
    };

    float s8 = 0.0f, inv8 = 0.0f;
    if (a.quant == MR_DTYPE_INT8) {
        float m = 0.0f;
        for (int64_t base = 0; base < a.K; base += step) {
            if (LONG) fetch(base, false);
            norm(base);
#pragma unroll
            for (int j = 0; j < PER; ++j) m = max_abs(m, v[j]);
        }
        uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7FFFFFFFu);
        if (kWarps > 1) {
            if (lane == 0) part_max[warp] = bits;
            __syncthreads();
            bits = __reduce_max_sync(0xffffffffu, lane < kWarps ? part_max[lane] : 0u);
        }
        const bool ok = bits < 0x7F800000u;
        const float amax = __uint_as_float(max(bits, (127u - 96u) << 23));
        s8 = ok ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
        inv8 = ok ? __fdiv_rn(127.0f, amax) : 0.0f;
        if (t == 0) *sr = s8;
    }

    for (int64_t base = 0; base < a.K; base += step) {
        if (LONG) fetch(base, false);
        if (LONG || a.quant != MR_DTYPE_INT8) norm(base);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t col = column(base, i);
            if (yr) store_piece<DT, LOOSE>(yr, col, a.K, narrow<DT>(v + i * V));
            const int64_t left = a.K - (int64_t)col;
            if (a.quant == MR_DTYPE_INT8) {
                if (left <= 0) continue;
                uint32_t q[V / 4];
#pragma unroll
                for (int j = 0; j < V / 4; ++j) q[j] = inv8 > 0.0f ? int8x4(v + i * V + 4 * j, inv8) : 0u;
                store_bytes<DT>(qr + col, q, (int)min(left, (int64_t)V), a.q_vec);
            } else if (a.quant == MR_DTYPE_E4M3) {
                // a block is 16 (fp32: 32) neighbouring lanes' pieces
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) m = max_abs(m, v[i * V + j]);
#pragma unroll
                for (int o = 1; o < kScaleBlock / V; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (left <= 0) continue;
                float s, inv;
                block_scale(__float_as_uint(m), &s, &inv);
                if (t % (kScaleBlock / V) == 0) sr[col / kScaleBlock * a.s_block] = s;
                uint32_t q[V / 4];
#pragma unroll
                for (int j = 0; j < V / 4; ++j) {
                    const float* f = v + i * V + 4 * j;
                    q[j] = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                }
                store_bytes<DT>(qr + col, q, (int)min(left, (int64_t)V), a.q_vec);
            }
        }
    }
}

template <int DT, int TPR, int PER, bool NORM, bool LONG>
cudaError_t launch_rows(const RowArgs& a, bool loose, cudaStream_t s) {
    const int64_t blocks = TPR == 32 ? (a.rows + 7) / 8 : a.rows;
    const dim3 grid((unsigned)blocks), block(TPR == 32 ? 256 : TPR);
    return loose ? launch_pdl(rows_kernel<DT, TPR, PER, NORM, true, LONG>, grid, block, 0, s, a)
                 : launch_pdl(rows_kernel<DT, TPR, PER, NORM, false, LONG>, grid, block, 0, s, a);
}

// The fewest values a thread that hold a short row (32768 rows of 70 bf16 values, norm to int8: 48 us,
// with 32 a thread 91; of 512: 38 and 50).
template <int DT, bool NORM> cudaError_t launch_rows(const RowArgs& a, bool loose, cudaStream_t s) {
    constexpr int P = DT == MR_DTYPE_F32 && NORM ? 16 : 32;
    if (a.K <= 256) return launch_rows<DT, 32, 8, NORM, false>(a, loose, s);
    if (a.K <= 512) return launch_rows<DT, 32, 16, NORM, false>(a, loose, s);
    if (P == 32 && a.K <= 1024) return launch_rows<DT, 32, P, NORM, false>(a, loose, s);
    if (a.K <= 128 * P) return launch_rows<DT, 128, P, NORM, false>(a, loose, s);
    if (a.K <= 256 * P) return launch_rows<DT, 256, P, NORM, false>(a, loose, s);
    if (a.K <= 512 * P) return launch_rows<DT, 512, P, NORM, false>(a, loose, s);
    return launch_rows<DT, 512, P, NORM, true>(a, loose, s);
}

// Rows of one type, in a translation unit of their own (they compile side by side).
template <int DT> cudaError_t rows_to_8(const RowArgs& a, bool norm, bool loose, cudaStream_t s);
#define MR_ROWS_TO_8(dt)                                                                              \
    template <> cudaError_t rows_to_8<dt>(const RowArgs& a, bool norm, bool loose, cudaStream_t s) {  \
        return norm ? launch_rows<dt, true>(a, loose, s) : launch_rows<dt, false>(a, loose, s);       \
    }

}  // namespace mr

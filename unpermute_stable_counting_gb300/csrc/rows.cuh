// Rows of 16- or 32-bit values in registers: 16-byte pieces of rows that start
// anywhere, and their fp32 values.
#pragma once

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

}  // namespace mr

// Grouped product of 8-bit rows with 8-bit expert weights, a scale per 128
// values of a row and per 128 x 128 block of a weight:
//   y[r, n] = sum_b sx[r, b] sw[e, n / 128, b] sum_{k in block b} q[r, k] w[e, n, k]
// for the rows r of each group (expert e, count) of a list on the device, and
// the experts' network built on it (silu(x W1^T) * (x W3^T), quantized again,
// times W2^T), whose first product quantizes its result in its epilogue.
//
// Tiles of 128 rows x BN columns, 128 values of k per step, on tcgen05 with
// e4m3 operands. The scales change every step, so a step's product goes to its
// own columns of tensor memory (two to four such buffers), and two warpgroups
// add it to the fp32 sums that they keep in registers, times the scales:
//   warp 0     TMA loads of the tiles' operands (a ring of stages)
//   warp 1     matrix instructions
//   warps 2-3  products of row and weight scales, in shared memory, four
//              steps at a time
//   warps 4-11 sums; at the end of a tile the result
// One persistent block per SM takes tiles round robin; every warp walks the
// group list for itself (32 groups at a time, one per lane), so there is no
// scheduling traffic and the host never reads the list.
#include "tensor.cuh"

#include <algorithm>

namespace mr {

namespace {

__device__ unsigned g_waits_out;  // blocks that left early, see mbar_wait

constexpr int kTileM = 128, kTileK = 128, kScaleBatch = 4, kScaleRing = 3;
constexpr int kThreads = 384;

struct GroupArgs {
    const float* x_scales;     // [r * xs_row + b * xs_block]
    int64_t xs_row, xs_block;
    const float* w_scales;     // [expert (, 2)][scale rows][KB]
    const int64_t* groups;     // [G, 2], or NULL: one group of all rows, expert 0
    int G, rows, experts;
    int64_t expert_base;
    int N, KB, scale_rows;     // N: columns (the network's first product: inter)
    int n_tiles;
    void* y;
    int64_t y_stride;
    int y_dtype, y_vec;        // y_vec: rows can be stored as 16-byte vectors
    uint8_t* hq;               // quantized result of the network's first product
    int64_t hq_stride;
    float* hs;                 // its scales, [b * hs_block + r]
    int64_t hs_block;
};

struct Tile {
    int expert, row0, rows, n0;
};

// Walks the group list. Every lane of the warp calls next() with the same t,
// ascending over the calls.
struct Walk {
    int first, base_tile, total;      // window of 32 groups; tiles before it, tiles in it
    int64_t base_row, window_rows;
    int expert, count, row0, tiles;   // this lane's group
    int end;                          // inclusive sum of tiles over the window

    __device__ __forceinline__ void load(const GroupArgs& a, int lane) {
        const int g = first + lane;
        int64_t e = 0, c = 0;
        if (g < a.G) {
            if (a.groups) {
                const longlong2 v = reinterpret_cast<const longlong2*>(a.groups)[g];
                e = v.x - a.expert_base;
                c = min(max((int64_t)v.y, (int64_t)0), (int64_t)a.rows);
            } else {
                c = a.rows;
            }
        }
        int64_t sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        window_rows = __shfl_sync(0xffffffffu, sum, 31);
        const int64_t start = min(base_row + sum - c, (int64_t)a.rows);
        row0 = (int)start;
        count = (int)min(c, a.rows - start);
        expert = (int)e;
        const bool ok = e >= 0 && e < a.experts;
        tiles = ok ? (count + kTileM - 1) / kTileM * a.n_tiles : 0;
        end = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += up;
        }
        total = __shfl_sync(0xffffffffu, end, 31);
    }
    __device__ __forceinline__ void begin(const GroupArgs& a, int lane) {
        first = base_tile = 0;
        base_row = 0;
        load(a, lane);
    }
    __device__ __forceinline__ bool next(const GroupArgs& a, int lane, int t, int bn, Tile& out) {
        while (t >= base_tile + total) {
            if (first + 32 >= a.G) return false;
            base_tile += total;
            base_row = min(base_row + window_rows, (int64_t)a.rows);
            first += 32;
            load(a, lane);
        }
        const int in = t - base_tile;
        const int src = __ffs(__ballot_sync(0xffffffffu, in < end)) - 1;
        const int i = in - __shfl_sync(0xffffffffu, end - tiles, src);
        const int c = __shfl_sync(0xffffffffu, count, src);
        const int mt = (c + kTileM - 1) / kTileM;
        const int n = i / mt, m = i - n * mt;  // a weight tile's row tiles side by side: it is read once
        out.expert = __shfl_sync(0xffffffffu, expert, src);
        out.row0 = __shfl_sync(0xffffffffu, row0, src) + m * kTileM;
        out.rows = min(c - m * kTileM, kTileM);
        out.n0 = n * bn;
        return true;
    }
};

template <int BN> struct Cfg {
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int kBufs = BN == 256 ? 2 : 4;                  // tensor memory buffers
    static constexpr int kScaleCols = BN == 256 ? 2 : 1;             // scale products per row and step
    static constexpr int kChunks = BN == 256 ? 2 : 1;                // column chunks per warpgroup
    static constexpr int kChunk = BN == 256 ? 64 : BN / 2;           // columns of a chunk
    static constexpr int kStageBytes = (kTileM + BN) * kTileK;
    static constexpr int kRingFloats = kScaleRing * kScaleBatch * kScaleCols * kTileM;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kRingFloats * 4 + 2 * 2 * kTileM * 4;
};

// 16-bit or fp32 stores of one row's columns [0, CW) from `p`, `left` of them real.
template <int CW>
__device__ __forceinline__ void store_row(const float2 (&acc)[CW / 2], void* y, int64_t at, int dt, int vec,
                                          int left) {
    if (left <= 0) return;
    if (dt == MR_DTYPE_F32) {
        float* p = reinterpret_cast<float*>(y) + at;
        if (vec && left >= CW) {
#pragma unroll
            for (int j = 0; j < CW / 4; ++j)
                reinterpret_cast<float4*>(p)[j] =
                    make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
        } else {
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) {
                if (2 * j < left) p[2 * j] = acc[j].x;
                if (2 * j + 1 < left) p[2 * j + 1] = acc[j].y;
            }
        }
        return;
    }
    uint32_t w[CW / 2];
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) {
        uint32_t lo, hi;
        if (dt == MR_DTYPE_F16) {
            lo = Elem<MR_DTYPE_F16>::from_f32(acc[j].x), hi = Elem<MR_DTYPE_F16>::from_f32(acc[j].y);
        } else {
            lo = Elem<MR_DTYPE_BF16>::from_f32(acc[j].x), hi = Elem<MR_DTYPE_BF16>::from_f32(acc[j].y);
        }
        w[j] = lo | (hi << 16);
    }
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + at;
    if (vec && left >= CW) {
#pragma unroll
        for (int j = 0; j < CW / 8; ++j)
            reinterpret_cast<uint4*>(p)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < CW / 2; ++j) {
            if (2 * j < left) p[2 * j] = (uint16_t)(w[j] & 0xFFFFu);
            if (2 * j + 1 < left) p[2 * j + 1] = (uint16_t)(w[j] >> 16);
        }
    }
}

template <int BN, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_matmul_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const GroupArgs a) {
    using C = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages];
    __shared__ __align__(8) uint64_t t_full[C::kBufs], t_empty[C::kBufs];
    __shared__ __align__(8) uint64_t r_full[kScaleRing], r_empty[kScaleRing];
    __shared__ __align__(8) uint64_t max_bar, drain_bar;
    __shared__ uint32_t tmem_base, abort_word;

    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(C::kSmem + 512 <= 232448, "shared memory of a block");
    float* ring = reinterpret_cast<float*>(tiles + C::kStages * C::kStageBytes);
    uint32_t* row_max = reinterpret_cast<uint32_t*>(ring + C::kRingFloats);  // [tile parity][warpgroup][128]
    volatile uint32_t* abort = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(smem_u32(&s_full[i]), 1), mbar_init(smem_u32(&s_empty[i]), 1);
        for (int i = 0; i < C::kBufs; ++i) mbar_init(smem_u32(&t_full[i]), 1), mbar_init(smem_u32(&t_empty[i]), 8);
        for (int i = 0; i < kScaleRing; ++i) mbar_init(smem_u32(&r_full[i]), 2), mbar_init(smem_u32(&r_empty[i]), 8);
        mbar_init(smem_u32(&max_bar), 8);
        mbar_init(smem_u32(&drain_bar), 1);
        abort_word = 0u;
        mbar_init_fence();
        tma_prefetch(&map_x);
        tma_prefetch(&map_w);
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_base), BN * C::kBufs);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_enter();

    Walk walk;
    Tile tile;
    uint32_t it = 0;  // steps that this warp has taken, over all of its tiles

    if (warp < 4) {
        regs_dec<80>();
        if (warp == 0) {
            walk.begin(a, lane);
            bool ok = true;
            for (int t = blockIdx.x; ok && walk.next(a, lane, t, BN, tile); t += gridDim.x) {
                const int boxes = (tile.rows + 31) / 32;
                const uint32_t bytes = (uint32_t)(boxes * 32 + BN) * kTileK;
                for (int kb = 0; kb < a.KB; ++kb, ++it) {
                    const uint32_t st = it % C::kStages;
                    ok = mbar_wait(smem_u32(&s_empty[st]), ((it / C::kStages) & 1) ^ 1, abort);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&s_full[st]);
                        const uint32_t dst = smem_u32(tiles + st * C::kStageBytes);
                        mbar_expect(bar, bytes);
                        if (SWIGLU) {
                            tma_load_3d(dst + kTileM * kTileK, &map_w, bar, kb * kTileK, tile.n0 / 2, tile.expert * 2);
                            tma_load_3d(dst + 2 * kTileM * kTileK, &map_w, bar, kb * kTileK, tile.n0 / 2,
                                        tile.expert * 2 + 1);
                        } else {
                            tma_load_3d(dst + kTileM * kTileK, &map_w, bar, kb * kTileK, tile.n0, tile.expert);
                        }
                        for (int j = 0; j < boxes; ++j)
                            tma_load_2d(dst + j * 32 * kTileK, &map_x, bar, kb * kTileK, tile.row0 + 32 * j);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1) {
            walk.begin(a, lane);
            bool ok = true;
            for (int t = blockIdx.x; ok && walk.next(a, lane, t, BN, tile); t += gridDim.x) {
                for (int kb = 0; kb < a.KB; ++kb, ++it) {
                    const uint32_t st = it % C::kStages, buf = it % C::kBufs;
                    ok = mbar_wait(smem_u32(&t_empty[buf]), ((it / C::kBufs) & 1) ^ 1, abort) &&
                         mbar_wait(smem_u32(&s_full[st]), (it / C::kStages) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t at = smem_u32(tiles + st * C::kStageBytes);
                        const uint64_t da = smem_desc(at), db = smem_desc(at + kTileM * kTileK);
#pragma unroll
                        for (int k = 0; k < kTileK / 32; ++k)
                            mma_e4m3(tmem + buf * BN, da + 2 * k, db + 2 * k, idesc_e4m3(kTileM, BN), k > 0);
                        tc_commit(smem_u32(&s_empty[st]));
                        tc_commit(smem_u32(&t_full[buf]));
                    }
                    __syncwarp();
                }
            }
        } else {
            // Products of the scales: this warp's 64 rows, two per lane.
            walk.begin(a, lane);
            uint32_t batch = 0;
            bool ok = true;
            const int r0 = (warp - 2) * 64 + lane;
            for (int t = blockIdx.x; ok && walk.next(a, lane, t, BN, tile); t += gridDim.x) {
                const float* ws[C::kScaleCols];
                bool real[C::kScaleCols];
#pragma unroll
                for (int c = 0; c < C::kScaleCols; ++c) {
                    const int nb = (SWIGLU ? tile.n0 / 2 : tile.n0 + c * 128) / kScaleBlock;
                    real[c] = nb < a.scale_rows;
                    const int64_t row = SWIGLU ? ((int64_t)tile.expert * 2 + c) * a.scale_rows + nb
                                               : (int64_t)tile.expert * a.scale_rows + nb;
                    ws[c] = a.w_scales + row * a.KB;
                }
                const float* xs = a.x_scales + (int64_t)(tile.row0 + r0) * a.xs_row;
                const bool in0 = r0 < tile.rows, in1 = r0 + 32 < tile.rows;
                for (int kb = 0; kb < a.KB; kb += kScaleBatch, ++batch) {
                    float x0[kScaleBatch], x1[kScaleBatch], w[kScaleBatch][C::kScaleCols];
#pragma unroll
                    for (int j = 0; j < kScaleBatch; ++j) {
                        const bool k_in = kb + j < a.KB;
                        x0[j] = k_in && in0 ? xs[(kb + j) * a.xs_block] : 0.0f;
                        x1[j] = k_in && in1 ? xs[32 * a.xs_row + (kb + j) * a.xs_block] : 0.0f;
#pragma unroll
                        for (int c = 0; c < C::kScaleCols; ++c) w[j][c] = k_in && real[c] ? ws[c][kb + j] : 0.0f;
                    }
                    const uint32_t slot = batch % kScaleRing;
                    ok = mbar_wait(smem_u32(&r_empty[slot]), ((batch / kScaleRing) & 1) ^ 1, abort);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < kScaleBatch; ++j)
#pragma unroll
                        for (int c = 0; c < C::kScaleCols; ++c) {
                            float* dst = ring + ((slot * kScaleBatch + j) * C::kScaleCols + c) * kTileM;
                            dst[r0] = x0[j] * w[j][c];
                            dst[r0 + 32] = x1[j] * w[j][c];
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&r_full[slot]));
                }
            }
        }
    } else {
        regs_inc<208>();
        walk.begin(a, lane);
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // 32 lanes << 16
        // first column and scale of each chunk
        int col[C::kChunks], sc[C::kChunks];
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
            if (BN != 256) col[c] = group * C::kChunk, sc[c] = 0;
            else if (SWIGLU) col[c] = c * 128 + group * 64, sc[c] = c;
            else col[c] = group * 128 + c * 64, sc[c] = group;
        }
        uint32_t batch = 0, done = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && walk.next(a, lane, t, BN, tile); t += gridDim.x, ++done) {
            float2 acc[C::kChunks][C::kChunk / 2];
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                for (int j = 0; j < C::kChunk / 2; ++j) acc[c][j] = make_float2(0.0f, 0.0f);
            for (int kb = 0; kb < a.KB; ++kb, ++it) {
                const uint32_t buf = it % C::kBufs, slot = batch % kScaleRing;
                if (kb % kScaleBatch == 0) ok = mbar_wait(smem_u32(&r_full[slot]), (batch / kScaleRing) & 1, abort);
                ok = ok && mbar_wait(smem_u32(&t_full[buf]), (it / C::kBufs) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const float* rs = ring + (slot * kScaleBatch + kb % kScaleBatch) * C::kScaleCols * kTileM + row;
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) {
                    const float s = rs[sc[c] * kTileM];
                    const float2 s2 = make_float2(s, s);
#pragma unroll
                    for (int q = 0; q < C::kChunk / 16; ++q) {
                        uint32_t v[16];
                        tmem_ld16(v, lanes + buf * BN + col[c] + 16 * q);
                        tmem_ld_wait(v);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[c][8 * q + j] = fma2(
                                make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), s2,
                                acc[c][8 * q + j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                const bool last = kb % kScaleBatch == kScaleBatch - 1 || kb == a.KB - 1;
                if (lane == 0) {
                    mbar_arrive(smem_u32(&t_empty[buf]));
                    if (last) mbar_arrive(smem_u32(&r_empty[slot]));
                }
                batch += last;
            }
            if (!ok) break;
            const int64_t r = (int64_t)tile.row0 + row;
            if (SWIGLU) {
                // chunk 0 holds the gate's columns, chunk 1 the same columns of the other factor
                uint32_t m = 0u;
#pragma unroll
                for (int j = 0; j < C::kChunk / 2; ++j) {
                    acc[0][j].x = silu(acc[0][j].x) * acc[C::kChunks - 1][j].x;
                    acc[0][j].y = silu(acc[0][j].y) * acc[C::kChunks - 1][j].y;
                    m = max(m, max(abs_bits(acc[0][j].x), abs_bits(acc[0][j].y)));
                }
                // a block of 128 is half in each warpgroup
                uint32_t* mx = row_max + (done & 1) * 2 * kTileM;
                mx[group * kTileM + row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&max_bar));
                ok = mbar_wait(smem_u32(&max_bar), done & 1, abort);
                if (!ok) break;
                m = max(m, mx[(group ^ 1) * kTileM + row]);
                float s, inv;
                block_scale(m, &s, &inv);
                if (row < tile.rows) {
                    const int n = tile.n0 / 2 + group * 64;
                    if (group == 0) a.hs[(tile.n0 / 2 / kScaleBlock) * a.hs_block + r] = s;
                    uint4* dst = reinterpret_cast<uint4*>(a.hq + r * a.hq_stride + n);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 p = acc[0][8 * j + 2 * i], q = acc[0][8 * j + 2 * i + 1];
                            w[i] = e4m3x4(p.x * inv, p.y * inv, q.x * inv, q.y * inv);
                        }
                        dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else if (row < tile.rows && MR_IN_RANGE(r, a.rows, 901)) {
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                    store_row<C::kChunk>(acc[c], a.y, r * a.y_stride + tile.n0 + col[c], a.y_dtype, a.y_vec,
                                         a.N - tile.n0 - col[c]);
            }
        }
    }
    __syncthreads();
    if (abort_word) {  // let what is in flight land
        if (warp == 0)
            for (uint32_t k = it > C::kStages ? it - C::kStages : 0; k < it; ++k)
                mbar_drain(smem_u32(&s_full[k % C::kStages]), (k / C::kStages) & 1);
        if (warp == 1) {
            if (lane == 0) tc_commit(smem_u32(&drain_bar));
            mbar_drain(smem_u32(&drain_bar), 0);
        }
        if (threadIdx.x == 0) atomicAdd(&g_waits_out, 1u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem, BN * C::kBufs);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int BN, bool SWIGLU>
cudaError_t launch_grouped(const CUtensorMap& mx, const CUtensorMap& mw, const GroupArgs& a, int64_t tiles,
                           cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(grouped_matmul_kernel<BN, SWIGLU>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t sms = device_sm_count();
    return launch_pdl(grouped_matmul_kernel<BN, SWIGLU>, dim3((unsigned)(tiles < sms ? tiles : sms)),
                      dim3(kThreads), Cfg<BN>::kSmem, s, mx, mw, a);
}

// One product over the groups. x: e4m3 rows, w: e4m3 [experts][N][K]; the first
// product of the network (swiglu) has w [experts][2][N][K] and a quantized result.
struct Product {
    const void* x;
    int64_t x_stride, x_rows;
    const void* w;
    int64_t w_row, w_matrix;   // byte strides of a row and of a matrix [N, K]
    int64_t K;
    bool swiglu;
};

mr_status run_product(const Product& p, GroupArgs a, cudaStream_t s) {
    const int64_t m_tiles = std::min<int64_t>((int64_t)ceil_div(a.rows, kTileM) + a.G, a.rows);
    const int sms = device_sm_count();
    int bn = 256;
    if (!p.swiglu) {
        // the widest tile that still gives every SM one (narrower ones read the rows more often)
        while (bn > 32 && m_tiles * ceil_div(a.N, bn) < sms) bn /= 2;
    }
    a.n_tiles = p.swiglu ? ceil_div(a.N, 128) : ceil_div(a.N, bn);
    const int64_t tiles = m_tiles * a.n_tiles;
    if (tiles > INT32_MAX) return MR_ERR_PARAM_INVALID;
    CUtensorMap mx, mw;
    const uint64_t xd[2] = {(uint64_t)p.K, (uint64_t)p.x_rows}, xs[1] = {(uint64_t)p.x_stride};
    const uint32_t xb[2] = {kTileK, 32};
    const uint64_t wd[3] = {(uint64_t)p.K, (uint64_t)a.N, (uint64_t)a.experts * (p.swiglu ? 2 : 1)};
    const uint64_t ws[2] = {(uint64_t)p.w_row, (uint64_t)p.w_matrix};
    const uint32_t wb[3] = {kTileK, (uint32_t)(p.swiglu ? 128 : bn), 1};
    if (!make_tensor_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.x, 2, xd, xs, xb) ||
        !make_tensor_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.w, 3, wd, ws, wb))
        return MR_ERR_CUDA;
    cudaError_t e;
    if (p.swiglu) e = launch_grouped<256, true>(mx, mw, a, tiles, s);
    else if (bn == 256) e = launch_grouped<256, false>(mx, mw, a, tiles, s);
    else if (bn == 128) e = launch_grouped<128, false>(mx, mw, a, tiles, s);
    else if (bn == 64) e = launch_grouped<64, false>(mx, mw, a, tiles, s);
    else e = launch_grouped<32, false>(mx, mw, a, tiles, s);
    return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

bool float_dtype(int32_t dt) { return dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16 || dt == MR_DTYPE_F32; }
int64_t elem_bytes(int32_t dt) { return dt == MR_DTYPE_E4M3 ? 1 : dt == MR_DTYPE_F32 ? 4 : 2; }
int64_t blocks_of(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Workspace of rows quantized by the call: values with rows of whole blocks,
// scales block-major (a block's scales side by side: read by 32 rows at once).
struct Quantized {
    int64_t stride, step;
    uint64_t q_bytes, bytes;
    Quantized(int64_t rows, int64_t cols) {
        stride = blocks_of(cols) * kScaleBlock;
        step = (int64_t)align_up((uint64_t)rows, 32);
        q_bytes = align_up((uint64_t)rows * stride, 256);
        bytes = q_bytes + align_up((uint64_t)step * blocks_of(cols) * 4, 256);
    }
};

bool common_sizes(int64_t rows, int64_t experts, int64_t numGroups, int64_t a, int64_t b) {
    return rows >= 0 && rows <= MR_MAX_EXPERT_ROWS && experts >= 1 && experts <= MR_MAX_EXPERT_NUM &&
           numGroups >= -1 && numGroups <= MR_MAX_EXPERT_ROWS && a >= 1 && a <= MR_MAX_EXPERT_COLS && b >= 1 &&
           b <= MR_MAX_EXPERT_COLS;
}

}  // namespace

MR_CHECK_ACCESSOR(grouped_matmul)

cudaError_t waits_out_grouped_matmul(unsigned* out, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_waits_out, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0u;
        e = cudaMemcpyToSymbol(g_waits_out, &zero, sizeof(zero));
    }
    return e;
}

bool make_tensor_map(CUtensorMap* map, CUtensorMapDataType type, int elem_bytes, const void* base, int rank,
                     const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    (void)elem_bytes;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return encode(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_grouped_matmul_get_workspace_size(int64_t rows, int64_t cols, int32_t xDtype,
                                                           uint64_t* workspaceSize) {
    if (xDtype != MR_DTYPE_E4M3 && !float_dtype(xDtype)) return MR_ERR_PARAM_INVALID;
    if (!common_sizes(rows, 1, 0, cols, 1)) return MR_ERR_PARAM_INVALID;
    if (!workspaceSize) return MR_ERR_PARAM_NULLPTR;
    *workspaceSize = xDtype == MR_DTYPE_E4M3 ? 0 : Quantized(rows, cols).bytes;
    return MR_OK;
}

extern "C" mr_status moe_grouped_matmul(const void* x, int32_t xDtype, int64_t xStride, const float* xScales,
                                        const int64_t* xScaleStrides, const void* weights,
                                        const int64_t* weightStrides, const float* weightScales,
                                        const int64_t* groupList, int64_t numGroups, const int64_t* numRows,
                                        int64_t expertBase, int64_t rows, int64_t experts, int64_t outCols,
                                        int64_t cols, void* y, int32_t yDtype, int64_t yStride, void* workspace,
                                        uint64_t workspaceSize, void* stream) {
    const bool eight = xDtype == MR_DTYPE_E4M3;
    if ((!eight && !float_dtype(xDtype)) || !float_dtype(yDtype)) return MR_ERR_PARAM_INVALID;
    if (!common_sizes(rows, experts, numGroups, outCols, cols)) return MR_ERR_PARAM_INVALID;
    if (!groupList && numGroups > 0) return MR_ERR_PARAM_NULLPTR;
    const int64_t top = INT64_C(1) << 40;
    if (xStride < cols || xStride > top || yStride < outCols || yStride > top) return MR_ERR_PARAM_INVALID;
    int64_t wr = cols, wm = outCols * cols;
    if (weightStrides) wr = weightStrides[0], wm = weightStrides[1];
    if (wr < cols || wr % 16 || wm % 16 || wr > top || wm > top || (experts > 1 && wm < (outCols - 1) * wr + cols))
        return MR_ERR_PARAM_INVALID;
    int64_t sr = blocks_of(cols), sb = 1;
    if (xScaleStrides) sr = xScaleStrides[0], sb = xScaleStrides[1];
    if (eight && (xStride % 16 || sr < 0 || sb < 0 || sr > top || sb > top)) return MR_ERR_PARAM_INVALID;
    const Quantized ws(rows, cols);
    if (rows == 0) return MR_OK;
    if (!x || !weights || !weightScales || !y || (eight && !xScales)) return MR_ERR_PARAM_NULLPTR;
    if (!eight && !workspace) return MR_ERR_PARAM_NULLPTR;
    if (!eight && workspaceSize < ws.bytes) return MR_ERR_WORKSPACE;
    if (!aligned16(weights) || (eight && !aligned16(x)) || (numGroups > 0 && !aligned16(groupList)) ||
        (!eight && reinterpret_cast<uintptr_t>(workspace) % 256))
        return MR_ERR_PARAM_INVALID;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(xDtype) || reinterpret_cast<uintptr_t>(y) % elem_bytes(yDtype))
        return MR_ERR_PARAM_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Product p{x, xStride, rows, weights, wr, wm, cols, false};
    GroupArgs a{};
    a.x_scales = xScales;
    a.xs_row = sr;
    a.xs_block = sb;
    if (!eight) {
        float* scales = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + ws.q_bytes);
        MR_TRY_CUDA(enqueue_quantize(x, xDtype, rows, cols, xStride, numRows, workspace, ws.stride, scales, 1,
                                     ws.step, s));
        p.x = workspace;
        p.x_stride = ws.stride;
        a.x_scales = scales;
        a.xs_row = 1;
        a.xs_block = ws.step;
    }
    a.w_scales = weightScales;
    a.groups = numGroups < 0 ? nullptr : groupList;
    a.G = numGroups < 0 ? 1 : (int)numGroups;
    a.rows = (int)rows;
    a.experts = (int)experts;
    a.expert_base = expertBase;
    a.N = (int)outCols;
    a.KB = (int)blocks_of(cols);
    a.scale_rows = (int)blocks_of(outCols);
    a.y = y;
    a.y_stride = yStride;
    a.y_dtype = yDtype;
    a.y_vec = aligned16(y) && (yStride * elem_bytes(yDtype)) % 16 == 0;
    if (a.G == 0) return MR_OK;
    return run_product(p, a, s);
}

extern "C" mr_status moe_expert_ffn_get_workspace_size(int64_t rows, int64_t hidden, int64_t inter,
                                                       uint64_t* workspaceSize) {
    if (!common_sizes(rows, 1, 0, hidden, inter)) return MR_ERR_PARAM_INVALID;
    if (!workspaceSize) return MR_ERR_PARAM_NULLPTR;
    *workspaceSize = Quantized(rows, hidden).bytes + Quantized(rows, inter).bytes;
    return MR_OK;
}

extern "C" mr_status moe_expert_ffn(const void* x, int32_t xDtype, int64_t xStride, const float* xScales,
                                    const int64_t* xScaleStrides, const void* w13, const int64_t* w13Strides,
                                    const float* w13Scales, const void* w2, const int64_t* w2Strides,
                                    const float* w2Scales, const int64_t* groupList, int64_t numGroups,
                                    const int64_t* numRows, int64_t expertBase, int64_t rows, int64_t experts,
                                    int64_t hidden, int64_t inter, void* y, int32_t yDtype, int64_t yStride,
                                    void* workspace, uint64_t workspaceSize, void* stream) {
    const bool eight = xDtype == MR_DTYPE_E4M3;
    if ((!eight && !float_dtype(xDtype)) || !float_dtype(yDtype)) return MR_ERR_PARAM_INVALID;
    if (!common_sizes(rows, experts, numGroups, hidden, inter)) return MR_ERR_PARAM_INVALID;
    if (!groupList && numGroups > 0) return MR_ERR_PARAM_NULLPTR;
    const int64_t top = INT64_C(1) << 40;
    if (xStride < hidden || xStride > top || yStride < hidden || yStride > top) return MR_ERR_PARAM_INVALID;
    int64_t ar = hidden, am = inter * hidden, br = inter, bm = hidden * inter;
    if (w13Strides) ar = w13Strides[0], am = w13Strides[1];
    if (w2Strides) br = w2Strides[0], bm = w2Strides[1];
    if (ar < hidden || ar % 16 || am % 16 || ar > top || am > top || am < (inter - 1) * ar + hidden)
        return MR_ERR_PARAM_INVALID;
    if (br < inter || br % 16 || bm % 16 || br > top || bm > top || (experts > 1 && bm < (hidden - 1) * br + inter))
        return MR_ERR_PARAM_INVALID;
    int64_t sr = blocks_of(hidden), sb = 1;
    if (xScaleStrides) sr = xScaleStrides[0], sb = xScaleStrides[1];
    if (eight && (xStride % 16 || sr < 0 || sb < 0 || sr > top || sb > top)) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    if (!x || !w13 || !w13Scales || !w2 || !w2Scales || !y || !workspace || (eight && !xScales))
        return MR_ERR_PARAM_NULLPTR;
    const Quantized wx(rows, hidden), wh(rows, inter);
    if (workspaceSize < wx.bytes + wh.bytes) return MR_ERR_WORKSPACE;
    if (!aligned16(w13) || !aligned16(w2) || (eight && !aligned16(x)) || (numGroups > 0 && !aligned16(groupList)) ||
        reinterpret_cast<uintptr_t>(workspace) % 256)
        return MR_ERR_PARAM_INVALID;
    if (reinterpret_cast<uintptr_t>(x) % elem_bytes(xDtype) || reinterpret_cast<uintptr_t>(y) % elem_bytes(yDtype))
        return MR_ERR_PARAM_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* base = reinterpret_cast<char*>(workspace);
    char* h = base + wx.bytes;

    GroupArgs a{};
    a.groups = numGroups < 0 ? nullptr : groupList;
    a.G = numGroups < 0 ? 1 : (int)numGroups;
    a.rows = (int)rows;
    a.experts = (int)experts;
    a.expert_base = expertBase;
    if (a.G == 0) return MR_OK;
    Product p{x, xStride, rows, w13, ar, am, hidden, true};
    a.x_scales = xScales;
    a.xs_row = sr;
    a.xs_block = sb;
    if (!eight) {
        float* scales = reinterpret_cast<float*>(base + wx.q_bytes);
        MR_TRY_CUDA(enqueue_quantize(x, xDtype, rows, hidden, xStride, numRows, base, wx.stride, scales, 1, wx.step, s));
        p.x = base;
        p.x_stride = wx.stride;
        a.x_scales = scales;
        a.xs_row = 1;
        a.xs_block = wx.step;
    }
    a.w_scales = w13Scales;
    a.N = (int)inter;
    a.KB = (int)blocks_of(hidden);
    a.scale_rows = (int)blocks_of(inter);
    a.hq = reinterpret_cast<uint8_t*>(h);
    a.hq_stride = wh.stride;
    a.hs = reinterpret_cast<float*>(h + wh.q_bytes);
    a.hs_block = wh.step;
    mr_status st = run_product(p, a, s);
    if (st != MR_OK) return st;

    p = Product{h, wh.stride, rows, w2, br, bm, inter, false};
    a.x_scales = a.hs;
    a.xs_row = 1;
    a.xs_block = wh.step;
    a.w_scales = w2Scales;
    a.N = (int)hidden;
    a.KB = (int)blocks_of(inter);
    a.scale_rows = (int)blocks_of(hidden);
    a.y = y;
    a.y_stride = yStride;
    a.y_dtype = yDtype;
    a.y_vec = aligned16(y) && (yStride * elem_bytes(yDtype)) % 16 == 0;
    return run_product(p, a, s);
}

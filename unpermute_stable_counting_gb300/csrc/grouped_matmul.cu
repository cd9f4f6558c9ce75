// Grouped product of 8-bit rows with 8-bit expert weights, a scale per 128
// values of a row and per 128 x 128 block of a weight:
//   y[r, n] = sum_b sx[r, b] sw[e, n / 128, b] sum_{k in block b} q[r, k] w[e, n, k]
// for the rows r of each group (expert e, count) of a list on the device, and
// the experts' network built on it (silu(x W1^T) * (x W3^T), quantized again,
// times W2^T), whose first product quantizes its result in its epilogue.
//
// Tiles of 128 rows x BN columns, or of 256 rows on a pair of blocks (each loads
// its own rows and half of the weights, which halves what L2 and shared memory
// carry per product), 128 values of k per step, on tcgen05 with e4m3 operands. The
// scales change every step, so a step's product goes to its own columns of tensor
// memory (two to four such buffers), and two warpgroups add it to the fp32 sums
// that they keep in registers, times the scales:
//   warp 0      TMA loads of the tiles' operands (a ring of stages)
//   warp 1      matrix instructions
//   warp 2      hands the tiles to the sums
//   warps 4-11  sums; at the end of a tile the result
// One persistent block per SM takes tiles round robin; the loads, the instructions
// and the tiles' warp each walk the group list (32 groups at a time, one per
// lane), so the host never reads it.
//
// What bounds it: with many rows the sums. A step of a pair's tile is 512 cycles of
// the tensor cores, and 128 columns of loads from tensor memory and fp32 additions
// for each of two warps per scheduler take about 690; the tensor pipe is active
// 65 % of the time (4096 x 7168 x 7168). Sums of more warps with fewer columns, loads
// of 32 columns and a step unrolled twice were all slower: they spill. Without the
// additions the same kernel takes 516 us for 16384 x 7168 x 7168 (with them 572 us
// = 2.94 PFLOP/s). With few rows per group the weights' way from HBM: 576 rows over
// 64 experts, 7168 -> 4096, 275 to 287 us (from GPU to GPU), 0.97 to 1.01 of the
// measured copy rate.
#include "tensor.cuh"

#include <algorithm>
#include <atomic>

namespace mr {

namespace {

__device__ unsigned g_waits_out;  // blocks that left early, see mbar_wait

constexpr int kTileM = 128, kTileK = 128;
constexpr int kThreads = 384, kSumWarps = 8;

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
    int y_dtype, y_loose;  // y_loose: rows that cannot be stored as 16-byte vectors
    uint8_t* hq;               // quantized result of the network's first product
    int64_t hq_stride;
    float* hs;                 // its scales, [b * hs_block + r]
    int64_t hs_block;
};

struct Tile {
    int expert, row0, rows, n0;
};

// Walks the group list in tiles of TM rows. Every lane of the warp calls next()
// with the same t, ascending over the calls.
template <int TM> struct Walk {
    int first, base_tile, total;      // window of 32 groups; tiles before it, tiles in it
    uint32_t base_row, window_rows;   // rows before it, rows in it
    int expert, count, row0, tiles;   // this lane's group
    int end;                          // inclusive sum of tiles over the window

    __device__ __forceinline__ void load(const GroupArgs& a, int lane) {
        const int g = first + lane;
        int64_t e = 0;
        int c = 0;
        if (g < a.G) {
            if (a.groups) {
                const longlong2 v = reinterpret_cast<const longlong2*>(a.groups)[g];
                e = v.x - a.expert_base;
                c = (int)min(max((int64_t)v.y, (int64_t)0), (int64_t)a.rows);
            } else {
                c = a.rows;
            }
        }
        // rows up to and with this group, at most a.rows <= 2^30: the sum of two is 2^31, which an
        // unsigned number holds and a signed one does not
        const uint32_t most = (uint32_t)a.rows;
        uint32_t sum = (uint32_t)c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum = min(sum + up, most);
        }
        uint32_t before = __shfl_up_sync(0xffffffffu, sum, 1);
        if (lane == 0) before = 0u;
        window_rows = __shfl_sync(0xffffffffu, sum, 31);
        row0 = (int)min(base_row + before, most);
        count = min(c, a.rows - row0);
        const bool ok = e >= 0 && e < a.experts;
        expert = ok ? (int)e : 0;
        tiles = ok ? (count + TM - 1) / TM * a.n_tiles : 0;
        end = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += up;
        }
        total = __shfl_sync(0xffffffffu, end, 31);
    }
    // The first window from g on that has rows, or the list's last one: eight windows per round trip
    // to memory (a batching's list ends in a row of empty groups for every absent expert).
    static __device__ __forceinline__ int skip(const GroupArgs& a, int lane, int g) {
        while (g + 32 < a.G) {
            int64_t c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = g + 32 * j + lane;
                c[j] = i < a.G ? a.groups[2 * (int64_t)i + 1] : 0;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (g + 32 >= a.G || __ballot_sync(0xffffffffu, c[j] > 0)) return g;
                g += 32;
            }
        }
        return g;
    }
    __device__ __forceinline__ void begin(const GroupArgs& a, int lane) {
        first = base_tile = 0;
        base_row = 0u;
        load(a, lane);
    }
    __device__ __forceinline__ bool next(const GroupArgs& a, int lane, int t, int bn, Tile& out) {
        while (t >= base_tile + total) {
            if (first + 32 >= a.G) return false;
            base_tile += total;
            base_row = min(base_row + window_rows, (uint32_t)a.rows);
            first = skip(a, lane, first + 32);
            load(a, lane);
        }
        const int in = t - base_tile;
        const int src = __ffs(__ballot_sync(0xffffffffu, in < end)) - 1;
        const int i = in - __shfl_sync(0xffffffffu, end - tiles, src);
        const int c = __shfl_sync(0xffffffffu, count, src);
        const int mt = (c + TM - 1) / TM;
        // Bands of 8 row tiles, column tiles within a band, the band's row tiles side by side: the
        // tiles in flight share rows and weights through L2.
        const int band = i / (8 * a.n_tiles);
        const int bm = min(8, mt - 8 * band);
        const int j = i - band * 8 * a.n_tiles;
        const int n = j / bm, m = 8 * band + j - n * bm;
        out.expert = __shfl_sync(0xffffffffu, expert, src);
        out.row0 = __shfl_sync(0xffffffffu, row0, src) + m * TM;
        out.rows = min(c - m * TM, TM);
        out.n0 = n * bn;
        return true;
    }
};

// PAIR: two blocks share a tile of 256 rows. Each loads its own 128 rows and half
// of the weight columns, and the matrix instructions read both halves.
// LOOSE: rows of results that do not start on 16 bytes, in kernels of their own: in
// the others the code beside the sums cost aligned rows up to 14 percent (3026 rows
// x 3705 x 5396 fp32 out: 106 us without, 120 with it).
template <int BN, bool SWIGLU, bool PAIR, bool LOOSE> struct Cfg {
    static constexpr int kLoadN = PAIR ? BN / 2 : BN;                // weight columns this block loads
    static constexpr int kStages = PAIR ? (SWIGLU || LOOSE ? 6 : 5) : BN == 256 ? 4 : 6;
    static constexpr int kBufs = BN == 256 ? 2 : 4;                  // tensor memory buffers
    static constexpr int kHalves = BN == 256 ? 2 : 1;                // column halves with barriers of their own
    static constexpr int kHalf = BN / kHalves;
    static constexpr int kChunks = SWIGLU ? 2 : 1;                   // column chunks per warpgroup
    static constexpr int kChunk = BN / 2 / kChunks;                  // columns of a chunk
    static constexpr int kLoad = 16;                                 // columns per tensor memory load
    static constexpr int kLoads = kChunks * kChunk / kLoad;
    static constexpr int kStageBytes = (kTileM + kLoadN) * kTileK;
    // a summing warp's rows on their way out: a pair's results leave by 8 KB (send_columns), others
    // 64 bytes of a row at a time, which leaves a fourth stage for the weights of few rows
    // (decode batch: 294 against 306 us)
    static constexpr bool kSend = PAIR && !SWIGLU && !LOOSE;
    static constexpr int kOutBytes = kSend ? 8192 : 2048;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kSumWarps * kOutBytes;
};

// Rows of U 16-byte pieces from shared memory (store_rows' layout) to rows that
// start anywhere: 4-byte words side by side, a word between two of the source's
// where a row of 16-bit values starts in the middle of one, whose first and last
// value then go alone. Not inlined: one copy that stays in the instruction cache.
template <int U, int ELEM>
__device__ __noinline__ void store_words(const uint8_t* stage, uint8_t* row0, int64_t row_step, int rows, int left) {
    constexpr int kWords = 4 * U, kRows = 32 / kWords, kBatch = 4;
    const int lane = threadIdx.x & 31, j = lane % kWords, r = lane / kWords;
    uint8_t* to = row0 + r * row_step + 4 * j;
    // a lane's rows are an even number of rows apart, so all of them start alike
    const int mid = ELEM == 2 ? (int)(reinterpret_cast<uintptr_t>(to) & 2u) : 0;
    const bool first = mid != 0 && j == 0 && left > 0;
    left = min(left, 16 * U) - 4 * j - mid;  // bytes of this lane's word
    const bool word = left >= 4, half = ELEM == 2 && !word && left >= 2;
    to += mid;
    row_step *= kRows;
#pragma unroll
    for (int b = 0; b < 32 / (kBatch * kRows); ++b) {
        if (b * kBatch * kRows >= rows) break;
        uint32_t w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int q = r + (b * kBatch + i) * kRows;
            w[i] = *reinterpret_cast<const uint32_t*>(stage + q * 64 + (((j >> 2) ^ ((q >> 1) & 3)) << 4) + (j & 3) * 4);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i, to += row_step) {
            const bool mine = r + (b * kBatch + i) * kRows < rows;
            uint32_t v = w[i];
            if constexpr (ELEM == 2) {
                v = __funnelshift_r(v, __shfl_down_sync(0xffffffffu, v, 1), 8 * mid);
                if (mine && first) *reinterpret_cast<uint16_t*>(to - 2) = (uint16_t)w[i];
                if (mine && half) *reinterpret_cast<uint16_t*>(to) = (uint16_t)v;
            }
            if (mine && word) *reinterpret_cast<uint32_t*>(to) = v;
        }
    }
    __syncwarp();
}

// Stores a warp's 32 rows (lane: row) of U 16-byte pieces, U <= 4, so that the
// lanes of an instruction write whole segments of a few rows: straight from the
// registers every lane would write to a row of its own, 32 lines per
// instruction. `row0`: the first row's first piece; row_step: bytes from a row to
// the next. `whole`: every row and piece is real; otherwise `rows` rows and `left`
// bytes of each are. LOOSE: rows that do not start on 16 bytes.
template <int U, bool LOOSE>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint4 (&v)[U], uint8_t* row0, int64_t row_step,
                                           bool whole, int rows, int left, int elem, int lane) {
    // 64-byte rows, pieces permuted so that eight lanes hit different banks
    const int key = (lane >> 1) & 3;
#pragma unroll
    for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ key) << 4)) = v[u];
    __syncwarp();
    constexpr int kRows = 32 / U;  // rows per instruction
    if constexpr (LOOSE) {
        if (elem == 4) store_words<U, 4>(stage, row0, row_step, rows, left);
        else store_words<U, 2>(stage, row0, row_step, rows, left);
        return;
    }
    uint4 w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int r = i * kRows + lane / U, u = lane % U;
        w[i] = *reinterpret_cast<const uint4*>(stage + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
    }
    __syncwarp();
    uint8_t* to = row0 + lane / U * row_step + lane % U * 16;
    const int64_t step = kRows * row_step;
    if (whole) {
#pragma unroll
        for (int i = 0; i < U; ++i, to += step) *reinterpret_cast<uint4*>(to) = w[i];
        return;
    }
    left -= lane % U * 16;
#pragma unroll
    for (int i = 0; i < U; ++i, to += step) {
        if (i * kRows + lane / U >= rows || left <= 0) continue;
        if (left >= 16) {
            *reinterpret_cast<uint4*>(to) = w[i];
            continue;
        }
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (elem == 4) {
                if (4 * k < left) reinterpret_cast<uint32_t*>(to)[k] = x[k];
            } else {
                if (4 * k < left) reinterpret_cast<uint16_t*>(to)[2 * k] = (uint16_t)(x[k] & 0xFFFFu);
                if (4 * k + 2 < left) reinterpret_cast<uint16_t*>(to)[2 * k + 1] = (uint16_t)(x[k] >> 16);
            }
        }
    }
}

template <int DT> __device__ __forceinline__ uint32_t pack2(float2 v) {
    uint32_t r;
    if constexpr (DT == MR_DTYPE_F16) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        r = reinterpret_cast<const uint32_t&>(h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        r = reinterpret_cast<const uint32_t&>(h);
    }
    return r;
}

// CW columns of the warp's rows, from `row0` (first row, first column) on.
template <int DT, int CW, bool LOOSE>
__device__ __forceinline__ void store_columns(uint8_t* stage, const float2 (&acc)[CW / 2], uint8_t* row0,
                                              int64_t row_step, int rows, int cols, int lane) {
    constexpr int kElem = DT == MR_DTYPE_F32 ? 4 : 2;
    constexpr int kMost = 64 / kElem;                // columns per 64-byte segment
    constexpr int W = CW < kMost ? CW : kMost, U = W * kElem / 16;
    const bool whole = rows == 32 && cols >= CW;
#pragma unroll
    for (int c = 0; c < CW; c += W) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (DT == MR_DTYPE_F32) {
                    const float2 p = acc[c / 2 + 2 * u + k / 2];
                    x[k] = __float_as_uint(k % 2 ? p.y : p.x);
                } else {
                    x[k] = pack2<DT>(acc[c / 2 + 4 * u + k]);
                }
            }
            v[u] = make_uint4(x[0], x[1], x[2], x[3]);
        }
        store_rows<U, LOOSE>(stage, v, row0 + kElem * c, row_step, whole, rows, kElem * (cols - c), kElem, lane);
    }
}

// The same for 32 real rows and a map of y (whose columns that are real end on 16 bytes): the columns go to shared memory as
// tiles of 128-byte rows in the map's swizzle, two of them at a time (all of a
// warp's 16-bit columns, half of its fp32 ones), and from there by asynchronous
// copies beside the next tile's sums. (Stores from registers took 3400 cycles of a
// tile's 27500 at 32 steps, these take half.)
template <int DT, int CW>
__device__ __forceinline__ void send_columns(uint8_t* stage, const float2 (&acc)[CW / 2], const CUtensorMap* map,
                                             int row, int col, int cols, int lane) {
    constexpr int kCols = DT == MR_DTYPE_F32 ? 32 : 64;
#pragma unroll
    for (int b = 0; b < CW / kCols; ++b) {
        if (b % 2 == 0) {  // what was sent from here has left
            if (lane == 0) tma_store_read();
            __syncwarp();
        }
        uint8_t* tile = stage + b % 2 * 4096;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float2* p = &acc[(b * kCols + u * kCols / 8) / 2];
            uint4 v;
            if constexpr (DT == MR_DTYPE_F32)
                v = make_uint4(__float_as_uint(p[0].x), __float_as_uint(p[0].y), __float_as_uint(p[1].x),
                               __float_as_uint(p[1].y));
            else
                v = make_uint4(pack2<DT>(p[0]), pack2<DT>(p[1]), pack2<DT>(p[2]), pack2<DT>(p[3]));
            *reinterpret_cast<uint4*>(tile + lane * 128 + ((u ^ (lane & 7)) << 4)) = v;
        }
        smem_proxy_fence();
        __syncwarp();
        if (lane == 0 && b * kCols < cols) tma_store_2d(map, smem_u32(tile), col + b * kCols, row);
    }
}

template <int BN, bool SWIGLU, bool PAIR, bool LOOSE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_matmul_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ CUtensorMap map_y, const GroupArgs a) {
    using C = Cfg<BN, SWIGLU, PAIR, LOOSE>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages];
    __shared__ __align__(8) uint64_t t_full[C::kBufs * C::kHalves], t_empty[C::kBufs * C::kHalves];
    __shared__ __align__(8) uint64_t i_full[2], i_empty[2];
    __shared__ Tile info[2];
    __shared__ __align__(8) uint64_t max_bar, drain_bar;
    __shared__ uint32_t tmem_base, abort_word;
    __shared__ uint32_t row_max[SWIGLU ? 2 : 1][SWIGLU ? 2 : 1][SWIGLU ? kTileM : 1];  // [tile parity][warpgroup][row]

    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(C::kSmem + 512 + (SWIGLU ? 4 * kTileM * 4 : 0) <= 232448, "shared memory of a block");
    uint8_t* out_stage = tiles + C::kStages * C::kStageBytes;
    volatile uint32_t* abort = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(smem_u32(&s_full[i]), 1), mbar_init(smem_u32(&s_empty[i]), 1);
        for (int i = 0; i < C::kBufs * C::kHalves; ++i)
            mbar_init(smem_u32(&t_full[i]), 1), mbar_init(smem_u32(&t_empty[i]), (PAIR ? 2 : 1) * kSumWarps / C::kHalves);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&i_full[i]), 1), mbar_init(smem_u32(&i_empty[i]), kSumWarps);
        mbar_init(smem_u32(&max_bar), kSumWarps);
        mbar_init(smem_u32(&drain_bar), 1);
        abort_word = 0u;
        mbar_init_fence();
        tma_prefetch(&map_x);
        tma_prefetch(&map_w);
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(&tmem_base), BN * C::kBufs);
    tc_fence_before();
    if (PAIR) cluster_sync();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;
    const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
    pdl_enter();

    Walk<PAIR ? 2 * kTileM : kTileM> walk;
    Tile tile;
    uint32_t it = 0;  // steps that this warp has taken, over all of its tiles

    if (warp < 4) {
        regs_dec<104>();
        if (warp == 0) {
            walk.begin(a, lane);
            bool ok = true;
            for (int t = first; ok && walk.next(a, lane, t, BN, tile); t += step) {
                // every block's boxes of 32 rows; the first block of a pair expects the bytes of both
                const int all = (tile.rows + 31) / 32;
                const int boxes = PAIR ? max(0, min(4, all - 4 * (int)rank)) : all;
                const int row0 = tile.row0 + (int)rank * kTileM;
                const uint32_t bytes = (uint32_t)(all * 32 + BN) * kTileK;
                if (elect_one()) {  // one thread for all steps: issuing costs a third of what a branch per step does
                    for (int kb = 0; kb < a.KB; ++kb, ++it) {
                        const uint32_t st = it % C::kStages;
                        ok = mbar_wait<PAIR>(smem_u32(&s_empty[st]), ((it / C::kStages) & 1) ^ 1, abort);
                        if (!ok) break;
                        const uint32_t own = smem_u32(&s_full[st]);
                        const uint32_t bar = PAIR ? map_cluster(own, 0) : own;
                        const uint32_t dst = smem_u32(tiles + st * C::kStageBytes);
                        if (rank == 0) mbar_expect(own, bytes);
                        const uint32_t wdst = dst + kTileM * kTileK;
                        const int k = kb * kTileK, n = SWIGLU ? tile.n0 / 2 : tile.n0;
                        if (PAIR) {
                            // halves of 128 columns: 64 of each in this block; the network's: 64 columns
                            // of the gate in the first block, the same of the other factor in the second
                            const int plane = SWIGLU ? tile.expert * 2 + (int)rank : tile.expert;
                            const int n1 = SWIGLU ? n : n + 64 * (int)rank;
                            tma_load_3d<PAIR>(wdst, &map_w, bar, k, n1, plane);
                            tma_load_3d<PAIR>(wdst + 64 * kTileK, &map_w, bar, k, n1 + (SWIGLU ? 64 : 128), plane);
                        } else if (SWIGLU) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tma_load_3d(wdst + j * 64 * kTileK, &map_w, bar, k, n + (j >> 1) * 64,
                                            tile.expert * 2 + (j & 1));
                        } else {
                            tma_load_3d(wdst, &map_w, bar, k, n, tile.expert);
                        }
                        for (int j = 0; j < boxes; ++j)
                            tma_load_2d<PAIR>(dst + j * 32 * kTileK, &map_x, bar, kb * kTileK, row0 + 32 * j);
                    }
                }
                __syncwarp();
                it = __reduce_max_sync(0xffffffffu, it);
                ok = __all_sync(0xffffffffu, ok);
            }
        } else if (warp == 1) {
            walk.begin(a, lane);
            bool ok = rank == 0;
            for (int t = first; ok && walk.next(a, lane, t, BN, tile); t += step) {
                if (elect_one()) {
                    for (int kb = 0; kb < a.KB; ++kb, ++it) {
                        const uint32_t st = it % C::kStages, buf = it % C::kBufs;
                        const uint32_t at = smem_u32(tiles + st * C::kStageBytes);
                        const uint64_t da = smem_desc(at), db = smem_desc(at + kTileM * kTileK);
                        ok = mbar_wait<PAIR>(smem_u32(&s_full[st]), (it / C::kStages) & 1, abort);
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h) {
                            const uint32_t th = buf * C::kHalves + h;
                            ok = ok && mbar_wait<PAIR>(smem_u32(&t_empty[th]), ((it / C::kBufs) & 1) ^ 1, abort);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t dh = db + h * (C::kHalf / (PAIR ? 2 : 1) * kTileK / 16);
#pragma unroll
                            for (int k = 0; k < kTileK / 32; ++k)
                                mma_e4m3<PAIR>(tmem + buf * BN + h * C::kHalf, da + 2 * k, dh + 2 * k,
                                               idesc_e4m3(PAIR ? 2 * kTileM : kTileM, C::kHalf), k > 0);
                            if (h == C::kHalves - 1) tc_commit<PAIR>(smem_u32(&s_empty[st]));
                            tc_commit<PAIR>(smem_u32(&t_full[th]));
                        }
                        if (!ok) break;
                    }
                }
                __syncwarp();
                it = __reduce_max_sync(0xffffffffu, it);
                ok = __all_sync(0xffffffffu, ok);
            }
        } else if (warp == 2) {
            // tiles for the sums; one of no rows ends them
            walk.begin(a, lane);
            uint32_t n = 0;
            for (int t = first;; t += step, ++n) {
                const bool more = walk.next(a, lane, t, BN, tile);
                if (!mbar_wait<PAIR>(smem_u32(&i_empty[n & 1]), ((n >> 1) & 1) ^ 1, abort)) break;
                if (lane == 0) {
                    if (!more) tile = Tile{0, 0, 0, 0};
                    info[n & 1] = tile;
                    mbar_arrive(smem_u32(&i_full[n & 1]));
                }
                if (!more) break;
            }
        }
    } else {
        regs_inc<200>();
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // 32 lanes << 16
        // this warpgroup's half of the columns, of narrow tiles its chunk
        const int half = C::kHalves == 2 ? group : 0;
        const uint32_t from = lanes + (C::kHalves == 2 ? group * C::kHalf : group * C::kChunk);
        uint8_t* stage = out_stage + (warp - 4) * C::kOutBytes;
        uint32_t done = 0;
        // Scales come straight from memory, two steps ahead (through shared memory, whose bandwidth
        // the operands take, they cost the sums more than the loads do), and a tile's first ones
        // before the tile before it is stored. Rows and columns past the tile's take its last ones'
        // scales: their sums are not stored.
        const float *xp, *wp;
        float xs[2], ws[2][C::kChunks];  // of the next two steps
        const int64_t w_other = SWIGLU ? (int64_t)a.scale_rows * a.KB : 0;
        bool ok = true;
        auto take = [&](uint32_t n) {
            ok = mbar_wait<PAIR>(smem_u32(&i_full[n & 1]), (n >> 1) & 1, abort);
            if (!ok) return;
            tile = info[n & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&i_empty[n & 1]));
            int srow = tile.row0 + max(0, min((int)rank * kTileM + row, tile.rows - 1));
            if (tile.rows > 0 && !MR_IN_RANGE(srow, a.rows, 902)) srow = 0;
            if (!MR_IN_RANGE(tile.expert, a.experts, 903)) tile.expert = 0;
            xp = a.x_scales + (int64_t)srow * a.xs_row;
            const int nb = min(SWIGLU ? tile.n0 / 2 / kScaleBlock : tile.n0 / kScaleBlock + half, a.scale_rows - 1);
            wp = a.w_scales + ((int64_t)(SWIGLU ? tile.expert * 2 : tile.expert) * a.scale_rows + nb) * a.KB;
            xs[0] = *xp;
            ws[0][0] = *wp;
            if (SWIGLU) ws[0][C::kChunks - 1] = wp[w_other];
            if (a.KB > 1) xp += a.xs_block, ++wp;
            xs[1] = *xp;
            ws[1][0] = *wp;
            if (SWIGLU) ws[1][C::kChunks - 1] = wp[w_other];
        };
        take(0);
        while (ok && tile.rows != 0) {
            float2 acc[C::kChunks][C::kChunk / 2];
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                for (int j = 0; j < C::kChunk / 2; ++j) acc[c][j] = make_float2(0.0f, 0.0f);
            // (A wait that gives up does not leave this loop, whose sums would then have to be kept in
            // place at every way out; the tile is dropped after it.)
            for (int kb = 0; kb < a.KB; ++kb, ++it) {
                const uint32_t buf = it % C::kBufs, th = buf * C::kHalves + half;
                float s[C::kChunks];
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) s[c] = xs[0] * ws[0][c], ws[0][c] = ws[1][c];
                xs[0] = xs[1];
                if (kb + 2 < a.KB) xp += a.xs_block, ++wp;
                xs[1] = *xp;
                ws[1][0] = *wp;
                if (SWIGLU) ws[1][C::kChunks - 1] = wp[w_other];
                mbar_wait<PAIR>(smem_u32(&t_full[th]), (it / C::kBufs) & 1, abort);
                tc_fence_after();
                // a load in flight while the one before it is added
                uint32_t v[2][C::kLoad];
                tmem_load(v[0], from + buf * BN);
#pragma unroll
                for (int q = 0; q < C::kLoads; ++q) {
                    tmem_ld_wait(v[q & 1]);
                    if (q + 1 < C::kLoads) {
                        tmem_load(v[(q + 1) & 1], from + buf * BN + (q + 1) * C::kLoad);
                    } else {
                        // everything is in registers: hand the buffer back before the last additions
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR) mbar_arrive_cluster(map_cluster(smem_u32(&t_empty[th]), 0));
                            else mbar_arrive(smem_u32(&t_empty[th]));
                        }
                    }
                    const int c = q * C::kLoad / C::kChunk, base = q * C::kLoad % C::kChunk / 2;
                    const float2 s2 = make_float2(s[c], s[c]);
#pragma unroll
                    for (int j = 0; j < C::kLoad / 2; ++j)
                        acc[c][base + j] = fma2(make_float2(__uint_as_float(v[q & 1][2 * j]),
                                                            __uint_as_float(v[q & 1][2 * j + 1])),
                                                s2, acc[c][base + j]);
                }
            }
            if (*abort) break;
            // this warp's rows of the tile
            const int wrow = (int)rank * kTileM + (warp & 3) * 32;
            const int wrows = min(32, tile.rows - wrow);
            const int64_t r = (int64_t)tile.row0 + wrow;
            const int n0 = tile.n0;
            take(done + 1);
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
                uint32_t (*mx)[SWIGLU ? kTileM : 1] = row_max[done & 1];
                mx[group][row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&max_bar));
                if (!mbar_wait<PAIR>(smem_u32(&max_bar), done & 1, abort)) break;
                m = max(m, mx[group ^ 1][row]);
                float s, inv;
                block_scale(m, &s, &inv);
                const int n = n0 / 2 + group * 64;
                const bool mine = wrows <= 0 || (MR_IN_RANGE(r + wrows - 1, a.rows, 904) &&
                                                 MR_IN_RANGE(n + 63, a.hq_stride, 905));
                if (mine && group == 0 && lane < wrows) a.hs[(n0 / 2 / kScaleBlock) * a.hs_block + r + lane] = s;
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p = acc[0][8 * j + 2 * i], q = acc[0][8 * j + 2 * i + 1];
                        x[i] = e4m3x4(p.x * inv, p.y * inv, q.x * inv, q.y * inv);
                    }
                    w[j] = make_uint4(x[0], x[1], x[2], x[3]);
                }
                store_rows<4, false>(stage, w, a.hq + r * a.hq_stride + n, a.hq_stride,
                              mine && wrows == 32, mine ? wrows : 0, 64, 4, lane);
            } else if (wrows > 0 && MR_IN_RANGE(r + wrows - 1, a.rows, 901)) {
                const int elem = a.y_dtype == MR_DTYPE_F32 ? 4 : 2;
                const int n = n0 + group * C::kChunk;
                uint8_t* to = reinterpret_cast<uint8_t*>(a.y) + (r * a.y_stride + n) * elem;
                const int64_t step = a.y_stride * elem;
                bool sent = false;
                if constexpr (C::kSend) {
                    // A copy's last 16 bytes of a row are written whole: where the row ends inside them,
                    // what follows it is not the call's, and the warp with its end stores the values.
                    const bool cut = n + C::kChunk > a.N && (a.N * elem & 15) != 0;
                    if (wrows == 32 && !cut) {
                        sent = true;
                        if (n < a.N) {
                            if (a.y_dtype == MR_DTYPE_BF16)
                                send_columns<MR_DTYPE_BF16, C::kChunk>(stage, acc[0], &map_y, (int)r, n, a.N - n, lane);
                            else if (a.y_dtype == MR_DTYPE_F16)
                                send_columns<MR_DTYPE_F16, C::kChunk>(stage, acc[0], &map_y, (int)r, n, a.N - n, lane);
                            else
                                send_columns<MR_DTYPE_F32, C::kChunk>(stage, acc[0], &map_y, (int)r, n, a.N - n, lane);
                        }
                    } else {
                        if (lane == 0) tma_store_read();
                        __syncwarp();
                    }
                }
                if (!sent && n < a.N) {
                    if (a.y_dtype == MR_DTYPE_BF16)
                        store_columns<MR_DTYPE_BF16, C::kChunk, LOOSE>(stage, acc[0], to, step, wrows, a.N - n, lane);
                    else if (a.y_dtype == MR_DTYPE_F16)
                        store_columns<MR_DTYPE_F16, C::kChunk, LOOSE>(stage, acc[0], to, step, wrows, a.N - n, lane);
                    else
                        store_columns<MR_DTYPE_F32, C::kChunk, LOOSE>(stage, acc[0], to, step, wrows, a.N - n, lane);
                }
            }
            ++done;
        }
        if (C::kSend && lane == 0) tma_store_done();
    }
    __syncthreads();
    if (PAIR) cluster_sync();
    if (abort_word) {  // let what is in flight land
        if (warp == 0 && rank == 0)
            for (uint32_t k = it > C::kStages ? it - C::kStages : 0; k < it; ++k)
                mbar_drain(smem_u32(&s_full[k % C::kStages]), (k / C::kStages) & 1);
        if (warp == 1 && rank == 0) {
            if (elect_one()) tc_commit<PAIR>(smem_u32(&drain_bar));
            mbar_drain(smem_u32(&drain_bar), 0);
        }
        if (threadIdx.x == 0) atomicAdd(&g_waits_out, 1u);
    }
    tc_fence_before();
    if (PAIR) cluster_sync();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free<PAIR>(tmem, BN * C::kBufs);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

bool aligned16(const void* p) { return aligned(p, 16); }

template <int BN, bool SWIGLU, bool PAIR, bool LOOSE>
cudaError_t launch_grouped(const CUtensorMap (&m)[3], const GroupArgs& a, int64_t tiles,
                           cudaStream_t s) {
    auto kernel = grouped_matmul_kernel<BN, SWIGLU, PAIR, LOOSE>;
    constexpr int smem = Cfg<BN, SWIGLU, PAIR, LOOSE>::kSmem;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    // blocks (pairs) the device holds at once, found once per device
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    int n = resident[dev].load(std::memory_order_acquire);
    if (n == 0) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return e;
        n = device_sm_count();
        if (PAIR) {
            cfg.gridDim = dim3(n / 2 * 2);
            if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            n = std::min(n, device_sm_count() / 2);
        }
        resident[dev].store(n, std::memory_order_release);
    }
    cfg.gridDim = dim3((unsigned)(tiles < n ? tiles : n) * (PAIR ? 2 : 1));
    return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], a);
}

template <bool LOOSE>
cudaError_t launch_plain(const CUtensorMap (&m)[3], const GroupArgs& a, bool pair, int bn, int64_t tiles,
                         cudaStream_t s) {
    if (pair) return launch_grouped<256, false, true, LOOSE>(m, a, tiles, s);
    if (bn == 256) return launch_grouped<256, false, false, LOOSE>(m, a, tiles, s);
    return launch_grouped<128, false, false, LOOSE>(m, a, tiles, s);
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

// The tile whose rounds over the SMs cost least. A step of a tile of 128 x 128, of 128 x 256 and of a
// pair's 256 x 256 takes about 5 : 8 : 7 (in one round, of 56 steps: 25, 37 and 33 us; 64 columns
// take as long as 128, so there is no narrower tile). 512 rows x 7168 x 4096: 25 us in tiles of 128
// columns, 33 in pairs; 2048 x 4096 x 4096: 39 in pairs, 49 in tiles of 128, 43 of 256. The
// groups' sizes are not known here: half a tile of each row of the list is taken to be empty. What
// that costs full groups, and lists with many empty ones: four full groups of 256 rows went from 20 to
// 25 us when this rule replaced one by rows; 32768 rows of 64 full groups, 4096 -> 2048, 223 us with a list of 64 and 262 to
// 268 with one of 128 to 1024 rows, for which it takes single blocks.
struct TileChoice {
    bool pair;
    int bn;         // instruction columns of a tile (the network's: of both factors)
    int rows, cols;  // of the result
    int at_once;    // tiles
};
TileChoice choose_tile(int64_t all_rows, int64_t G, int64_t N, bool swiglu) {
    const int sms = device_sm_count();
    auto cost = [&](int rows, int cols, int units, int step) {
        const int64_t down =
            G == 1 ? ceil_div(all_rows, rows) : std::max(std::min(G, all_rows), all_rows / rows + G / 2);
        return (down * ceil_div(N, cols) + units - 1) / units * step;
    };
    const int cols = swiglu ? 128 : 256;
    const int64_t wide = cost(kTileM, cols, sms, 8);
    const int64_t narrow = swiglu ? INT64_MAX : cost(kTileM, 128, sms, 5);
    if (cost(2 * kTileM, cols, sms / 2, 7) <= std::min(wide, narrow)) return {true, 256, 2 * kTileM, cols, sms / 2};
    if (wide <= narrow) return {false, 256, kTileM, cols, sms};
    return {false, 128, kTileM, 128, sms};
}

mr_status run_product(const Product& p, GroupArgs a, cudaStream_t s) {
    const TileChoice tile = choose_tile(a.rows, a.G, a.N, p.swiglu);
    const bool pair = tile.pair;
    const int bn = tile.bn, tile_m = tile.rows;
    const int64_t m_tiles = std::min<int64_t>((int64_t)ceil_div(a.rows, tile_m) + a.G - 1, a.rows);  // or fewer
    a.n_tiles = ceil_div(a.N, tile.cols);
    const int64_t tiles = m_tiles * a.n_tiles;
    if (tiles > INT32_MAX) return MR_ERR_PARAM_INVALID;
    CUtensorMap m[3];
    const uint64_t xd[2] = {(uint64_t)p.K, (uint64_t)p.x_rows}, xs[1] = {(uint64_t)p.x_stride};
    const uint32_t xb[2] = {kTileK, 32};
    const uint64_t wd[3] = {(uint64_t)p.K, (uint64_t)a.N, (uint64_t)a.experts * (p.swiglu ? 2 : 1)};
    const uint64_t ws[2] = {(uint64_t)p.w_row, (uint64_t)p.w_matrix};
    const uint32_t wb[3] = {kTileK, (uint32_t)(p.swiglu || pair ? 64 : bn), 1};
    if (!make_tensor_map(&m[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.x, 2, xd, xs, xb) ||
        !make_tensor_map(&m[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.w, 3, wd, ws, wb))
        return MR_ERR_CUDA;
    m[2] = m[0];  // not read
    if (pair && !p.swiglu && !a.y_loose) {
        const bool wide = a.y_dtype == MR_DTYPE_F32;
        const int elem = wide ? 4 : 2;
        const uint64_t yd[2] = {(uint64_t)a.N, (uint64_t)a.rows}, ys[1] = {(uint64_t)a.y_stride * elem};
        const uint32_t yb[2] = {(uint32_t)(128 / elem), 32};
        if (!make_tensor_map(&m[2], wide ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, elem, a.y, 2,
                             yd, ys, yb))
            return MR_ERR_CUDA;
    }
    cudaError_t e;
    if (p.swiglu) e = pair ? launch_grouped<256, true, true, false>(m, a, tiles, s)
                           : launch_grouped<256, true, false, false>(m, a, tiles, s);
    else e = a.y_loose ? launch_plain<true>(m, a, pair, bn, tiles, s) : launch_plain<false>(m, a, pair, bn, tiles, s);
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
    const bool wide = box[0] * elem_bytes == 128;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return encode(map, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mr

using namespace mr;

extern "C" mr_status mr_expert_tile(int64_t rows, int64_t numGroups, int64_t outCols, int32_t network, int32_t* tile) {
    if (!common_sizes(rows, 1, numGroups, outCols, 1) || rows == 0 || numGroups == 0) return MR_ERR_PARAM_INVALID;
    if (!tile) return MR_ERR_PARAM_NULLPTR;
    const TileChoice t = choose_tile(rows, numGroups < 0 ? 1 : numGroups, outCols, network != 0);
    tile[0] = t.rows;
    tile[1] = t.cols;
    tile[2] = t.at_once;
    return MR_OK;
}

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
    if (eight) xStride = stride_of(rows, xStride, cols);
    if (xStride < cols || xStride > top || yStride < outCols || yStride > top) return MR_ERR_PARAM_INVALID;
    int64_t wr = cols, wm = outCols * cols;
    if (weightStrides) wr = weightStrides[0], wm = weightStrides[1];
    wr = stride_of(outCols, wr, cols);
    wm = stride_of(experts, wm, outCols * wr);
    if (wr < cols || wr % 16 || wm % 16 || wr > top || wm > top || (experts > 1 && wm < (outCols - 1) * wr + cols))
        return MR_ERR_PARAM_INVALID;
    int64_t sr = blocks_of(cols), sb = 1;
    if (xScaleStrides) sr = xScaleStrides[0], sb = xScaleStrides[1];
    if (eight && (xStride % 16 || sr < 0 || sb < 0 || sr > top || sb > top)) return MR_ERR_PARAM_INVALID;
    if (!eight && rows * blocks_of(cols) > INT32_MAX) return MR_ERR_PARAM_INVALID;  // moe_quantize's limit
    const Quantized ws(rows, cols);
    if (rows == 0) return MR_OK;
    if (!x || !weights || !weightScales || !y || (eight && !xScales)) return MR_ERR_PARAM_NULLPTR;
    if (!eight && !workspace) return MR_ERR_PARAM_NULLPTR;
    if (!eight && workspaceSize < ws.bytes) return MR_ERR_WORKSPACE;
    if (!aligned16(weights) || (eight && !aligned16(x)) || (numGroups > 0 && !aligned16(groupList)) ||
        (!eight && !aligned(workspace, 256)))
        return MR_ERR_PARAM_INVALID;
    if (!aligned(x, elem_bytes(xDtype)) || !aligned(y, elem_bytes(yDtype)) || !aligned(xScales, 4) ||
        !aligned(weightScales, 4) || !aligned(numRows, 8))
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
    a.y_loose = !aligned16(y) || (yStride * elem_bytes(yDtype)) % 16 != 0;
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
    if (eight) xStride = stride_of(rows, xStride, hidden);
    if (xStride < hidden || xStride > top || yStride < hidden || yStride > top) return MR_ERR_PARAM_INVALID;
    int64_t ar = hidden, am = inter * hidden, br = inter, bm = hidden * inter;
    if (w13Strides) ar = w13Strides[0], am = w13Strides[1];
    if (w2Strides) br = w2Strides[0], bm = w2Strides[1];
    ar = stride_of(inter, ar, hidden);
    br = stride_of(hidden, br, inter);
    bm = stride_of(experts, bm, hidden * br);
    if (ar < hidden || ar % 16 || am % 16 || ar > top || am > top || am < (inter - 1) * ar + hidden)
        return MR_ERR_PARAM_INVALID;
    if (br < inter || br % 16 || bm % 16 || br > top || bm > top || (experts > 1 && bm < (hidden - 1) * br + inter))
        return MR_ERR_PARAM_INVALID;
    int64_t sr = blocks_of(hidden), sb = 1;
    if (xScaleStrides) sr = xScaleStrides[0], sb = xScaleStrides[1];
    if (eight && (xStride % 16 || sr < 0 || sb < 0 || sr > top || sb > top)) return MR_ERR_PARAM_INVALID;
    if (!eight && rows * blocks_of(hidden) > INT32_MAX) return MR_ERR_PARAM_INVALID;  // moe_quantize's limit
    if (rows == 0) return MR_OK;
    if (!x || !w13 || !w13Scales || !w2 || !w2Scales || !y || !workspace || (eight && !xScales))
        return MR_ERR_PARAM_NULLPTR;
    const Quantized wx(rows, hidden), wh(rows, inter);
    if (workspaceSize < wx.bytes + wh.bytes) return MR_ERR_WORKSPACE;
    if (!aligned16(w13) || !aligned16(w2) || (eight && !aligned16(x)) || (numGroups > 0 && !aligned16(groupList)) ||
        !aligned(workspace, 256))
        return MR_ERR_PARAM_INVALID;
    if (!aligned(x, elem_bytes(xDtype)) || !aligned(y, elem_bytes(yDtype)) || !aligned(xScales, 4) ||
        !aligned(w13Scales, 4) || !aligned(w2Scales, 4) || !aligned(numRows, 8))
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
    a.y_loose = !aligned16(y) || (yStride * elem_bytes(yDtype)) % 16 != 0;
    return run_product(p, a, s);
}

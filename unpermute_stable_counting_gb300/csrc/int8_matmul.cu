// Grouped product of rows with 8-bit integer expert weights that have a scale per
// output channel, and the experts' network built on it:
//   y[r, n] = sx[r] sw[e, n] sum_k x[r, k] w[e, n, k]
// for the rows r of each group (expert e, count) of a list on the device. Rows are
// int8 with a scale each, or of 16 bits.
//
// The tensor cores of sm_103a have no 8-bit integer products. An int8 value is
// exact in f16 and in bf16, a product of two in the fp32 accumulators, and so is a
// sum while it stays below 2^24 (where results are fp32, or rows long, several sums make
// a value, see Int8Args). So the products run at the 16-bit rate, and the
// weights, which are the bulk of what is read, become 16 bits on their way to the
// tensor cores: W is the operand with 128 rows (A), and its values go from shared
// memory through registers to tensor memory, which costs shared memory neither the
// store nor the instructions' reads. The rows of a group are the other operand (B):
// an instruction has as many columns as the group has rows left, to the next 16.
//   warp 0       TMA loads of the weights (and of int8 rows): a ring of 128 values of k
//   warp 1       matrix instructions, 128 values of k a step
//   warp 2       hands tiles to the warps below
//   warp 3       TMA loads of 16-bit rows: a ring of steps
//   warps 4-11   weights to 16 bits; of a pair each warpgroup takes every other load, of a
//                single block one of a load's two operands
//   four warps   int8 rows, where there are any, to 16 bits, two on every other load
//   eight warps  results: scales, rounding, stores
// One persistent block per SM takes tiles round robin; a pair of blocks shares a tile
// of 256 channels, where each converts its own 128 and loads half of the rows. Where
// few rows leave SMs without a tile, single blocks take equal shares of all tiles' loads
// instead: a tile's sums may then come from several blocks, which leave them in the
// workspace, and the last one to arrive adds them up, in the order of k.
//
// What bounds it: with many rows the tensor cores and the power limit (4096 x 7168 ->
// 4096: tensor pipe active 71 % of 142 us; 16384 x 7168 -> 7168 takes 780 us, 2.16
// PFLOP/s, beside 53 to make the rows f16). With few rows per group the weights' way
// from HBM, and how long a load keeps its room: 576 rows over 64 experts, 7168 ->
// 4096, 298 us, 0.95 of the copy rate; a load of 32 KB takes a block's
// converters about 1150 cycles (waits 300, shared memory and conversion 450, the way
// to tensor memory 300), so that few tiles of long rows are bound by those. With few
// loads in all, the start (1.8 us up to the first load: list, descriptors), the results and
// their code's own way from memory.
#include "groups.cuh"
#include "tensor.cuh"

#include <algorithm>
#include <atomic>

namespace mr {

namespace {

__device__ unsigned g_waits_out;  // blocks that left early, see mbar_wait

constexpr int kConvertWarps = 8, kSumWarps = 8;
constexpr int kWRows = 128, kWBytes = kWRows * 128;  // a load: 128 channels x 128 values

struct Int8Args : Groups {
    const float* x_scales;  // [r * xs_row], or NULL
    int64_t xs_row;
    const float* w_scales;  // [expert (, 2)][N]
    int N, KB;              // channels (the network's first product: inter), loads of 128 values of k
    void* y;
    int64_t y_stride;
    int y_dtype;
    int many;               // blocks may have several tiles
    // Loads whose products one sum takes. The tensor cores cut what a sum has below fp32's digits at every addition:
    // f16 rows of 7168 values are off by 7e-6, of 1000 by 8e-7, and int8 rows of one sign, whose sums are exact up to
    // 2^24 (1024 values), of 7168 by 1.2e-5. Where the result is fp32, or rows are long, a tile is taken in several sums,
    // as `sums` says.
    int sum_loads, sums;
    // 16-bit results of several sums: kRows rows of 256 sums for each block (pair), of which a thread has the same words for
    // every tile, so that no tile's sums wait for another warp's
    float* room;
    // equal shares of the loads (NULL: whole tiles round robin)
    float* parts;           // two to a block, of part_rows rows of 256 sums
    int part_rows, part_loads;  // a share is this many loads at least
    unsigned* tickets;      // of each tile: blocks that have left their sums, 0 at the start
};

// Several sums to a value: each scaled and added to y (fp32 results of 16-bit rows), or put together before the scales, of
// fp32 results in y's place.
enum { kOneSum = 0, kScaledSums, kPlainSums };

constexpr int kMostShares = 256;  // groups of a list that is walked once more, for the number of its tiles

// The tiles, or parts of tiles, that a block (pair) takes: loads [kb0, kb1) of tile t.
// Every lane of the warp calls with the same values.
template <typename W, bool SHARES> struct Items {
    W walk;
    Tile tile;
    int t, kb0, kb1;
    bool again, more;             // of the block's sums of the tile: not the first, not the last
    int at, start, end, total, blocks;   // shares: loads of all tiles (2^17 of each, and fewer tiles than SMs)

    __device__ __forceinline__ void begin(const Int8Args& a, int lane, int first, int step) {
        walk.begin(a, lane);
        t = first - step;
        kb1 = a.KB;
        if (!SHARES || !a.parts) return;
        int tiles = walk.total;
        if (a.G > 32) {
            W all = walk;
            for (int g = 32; g < a.G; g += 32) {
                all.base_row = min(all.base_row + all.window_rows, (uint32_t)a.rows);
                all.first = g;
                all.load(a, lane);
                tiles += all.total;
            }
        }
        total = tiles * a.KB;
        blocks = min((int)gridDim.x, total / a.part_loads + 1);
        at = end = 0;
        if (first < blocks) at = (int)((int64_t)first * total / blocks), end = (int)((int64_t)(first + 1) * total / blocks);
        start = at;
    }
    __device__ __forceinline__ bool next(const Int8Args& a, int lane, int channels, int step) {
        if (SHARES && a.parts) {
            if (at >= end) return false;
            t = at / a.KB;
            kb0 = at - t * a.KB;
            again = kb0 > 0 && at > start;
            kb1 = min(a.KB, kb0 + min(end - at, a.sum_loads));
            at += kb1 - kb0;
            more = kb1 < a.KB && at < end;
        } else {
            if (kb1 == a.KB) t += step, kb1 = 0;
            kb0 = kb1;
            kb1 = min(a.KB, kb0 + a.sum_loads);
            again = kb0 > 0;
            more = kb1 < a.KB;
        }
        return walk.next(a, lane, t, channels, tile);
    }
    __device__ __forceinline__ int owner(int load) const { return (int)(((int64_t)(load + 1) * blocks - 1) / total); }
};

// Where a tile's sums lie: those of a single block's tiles of few rows in one half of
// their room or the other, in turn, so that the next tile's instructions need not wait
// for this one's results; others' in all of it. A half has barriers of its own.
template <bool PAIR, int HALF> struct SumRoom {
    uint32_t turn = 0, uses[2] = {0, 0};
    bool both = false;
    int half = 0;
    __device__ __forceinline__ void next(int columns) {
        both = !PAIR && columns > HALF;
        half = PAIR || both ? 0 : (int)(turn++ & 1);
    }
    __device__ __forceinline__ uint32_t parity(int h) const { return (h ? uses[1] : uses[0]) & 1; }
    __device__ __forceinline__ void used() {
        if (both || half == 0) ++uses[0];
        if (both || half == 1) ++uses[1];
    }
};

// A tile, or the part of one: for the warps that do not walk the list.
struct Item {
    Tile tile;
    int t, loads;
    bool again, more;        // of the block's sums of the tile: not the first, not the last
    int first, last, block;  // blocks that have a part of the tile; this one
};

enum { kInt8 = 0, kF16 = 1, kBf16 = 2 };  // rows

// XT: the rows' type. SWIGLU: the network's first product, with a gate's channels and
// the same ones of the other factor in a tile. A single block has two operands of 128
// channels a step, whose sums lie side by side: a plain product's 256 channels, or the
// two factors. Of a pair each block has one: its half of 256 channels, or 64 of the
// gate's above the same 64 of the other factor.
template <int XT, bool SWIGLU, bool PAIR> struct Cfg {
    static constexpr int kRows = PAIR ? 256 : 96;                   // rows of a tile
    static constexpr int kChannels = SWIGLU ? 128 : 256;            // and channels of the result
    static constexpr int kPlanes = PAIR ? 1 : 2;
    static constexpr int kLoadRows = PAIR ? kRows / 2 : kRows;      // of the rows, those this block loads
    static constexpr int kBox = PAIR ? 64 : 32;                     // rows of a TMA load
    // Steps of converted weights held, one for each operand and load, and of 16-bit rows. The way round (converted,
    // multiplied, free again) takes several steps' time: with three steps instead of four the dense 16384 x 7168 x
    // 7168 took pairs 851 us instead of 835. (A step of 64 values costs the thread that issues the instructions its
    // waits and commit twice: 884 instead of 848 us.) 16-bit rows of single blocks come from L2 only when a step is
    // free: with two of them 576 rows over 64 experts, 7168 -> 4096, take 328 us, with three 305.
    static constexpr int kSteps = PAIR ? 4 : 5, kRowSteps = PAIR ? 4 : XT == kInt8 ? 2 : 3;
    static constexpr int kRowWarps = XT == kInt8 ? 4 : 0;           // warps of int8 rows
    static constexpr int kWarps = 4 + kConvertWarps + kRowWarps + kSumWarps, kThreads = 32 * kWarps;
    static constexpr int kStepCols = 64;                            // tensor memory of a step's weights
    static constexpr int kACols = kRows * kPlanes;                  // tensor memory: sums, then weights
    static_assert(kACols + kSteps * kStepCols <= 512, "tensor memory");
    static constexpr int kLoads = PAIR && !SWIGLU ? 6 : 4;
    static constexpr int kLoadBytes = kPlanes * kWBytes + (XT == kInt8 ? kLoadRows * 128 : 0);
    static constexpr int kPartBytes = kLoadRows * 128, kStepBytes = kPartBytes * 2;  // 64 values, 128
    static constexpr int kHalf = kRows / 2;                         // rows of a warpgroup of results
    static constexpr int kChunk = PAIR ? 32 : 16;                   // of them, those read at once
    static constexpr bool kSwap = SWIGLU && PAIR;                   // the factors meet in shared memory
    static constexpr int kSwapBytes = kSwap ? 2 * kChunk / 2 * 128 : 0;  // of a warp of results
    // registers of a thread of the first four warps, of the converters, of int8 rows and of the results; blocks are
    // launched with as many for all as there are
    static constexpr int kRegs[4] = {PAIR ? 48 : 56, 80, 56, PAIR ? 136 : XT == kInt8 ? 104 : 128};
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static_assert(4 * kRegs[0] + kConvertWarps * kRegs[1] + kRowWarps * kRegs[2] + kSumWarps * kRegs[3] <=
                  kWarps * kLaunchRegs, "registers of a block");
    static constexpr int kSmem = 1024 + kLoads * kLoadBytes + kRowSteps * kStepBytes + kSumWarps * kSwapBytes;
};

// Matrix instruction with A in tensor memory.
template <bool PAIR>
__device__ __forceinline__ void mma_16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),
        "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),
        "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four int8 to four 16-bit values, without a conversion instruction: a byte below an
// exponent's byte is an offset value, and one subtraction, exact, takes the offset off.
//   f16   0x64xx is 1024 + xx; xx = x + 128 by flipping the sign bit
//   bf16  0x43xx is 128 + xx below 128 and 256 + 2 (xx - 128) above, 8 bits being all it
//         has: x = (128 + low 7 bits) - (256 if x < 0, else 128)
template <bool BF16> __device__ __forceinline__ void widen4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    if constexpr (BF16) {
        const uint32_t p = __byte_perm(x, 0x43434343u, 0x5140), q = __byte_perm(x, 0x43434343u, 0x5342);
        const uint32_t pa = p & 0xFF7FFF7Fu, pb = p & 0xFF80FF80u, qa = q & 0xFF7FFF7Fu, qb = q & 0xFF80FF80u;
        const __nv_bfloat162 l = __hsub2(reinterpret_cast<const __nv_bfloat162&>(pa), reinterpret_cast<const __nv_bfloat162&>(pb));
        const __nv_bfloat162 h = __hsub2(reinterpret_cast<const __nv_bfloat162&>(qa), reinterpret_cast<const __nv_bfloat162&>(qb));
        lo = reinterpret_cast<const uint32_t&>(l);
        hi = reinterpret_cast<const uint32_t&>(h);
    } else {
        x ^= 0x80808080u;
        const uint32_t p = __byte_perm(x, 0x64646464u, 0x5140), q = __byte_perm(x, 0x64646464u, 0x5342), off = 0x64806480u;
        const __half2 l = __hsub2(reinterpret_cast<const __half2&>(p), reinterpret_cast<const __half2&>(off));
        const __half2 h = __hsub2(reinterpret_cast<const __half2&>(q), reinterpret_cast<const __half2&>(off));
        lo = reinterpret_cast<const uint32_t&>(l);
        hi = reinterpret_cast<const uint32_t&>(h);
    }
}

// Pairs of 16-bit values. (The type is asked for once, not for each pair: 515 rows of 6 groups, 712 -> 1080: 32 rows
// of a warp's results took 3400 cycles so.)
template <int N> __device__ __forceinline__ void pack(bool f16, const float (&a)[N], const float (&b)[N], uint32_t (&w)[N]) {
    if (f16) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const __half2 h = __floats2half2_rn(a[j], b[j]);
            w[j] = reinterpret_cast<const uint32_t&>(h);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a[j], b[j]);
            w[j] = reinterpret_cast<const uint32_t&>(h);
        }
    }
}

// A value of y, or what is added to one that this thread has put there.
__device__ __forceinline__ void put(char* y, float v, bool add) {
    if (add) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(y), "f"(v) : "memory");
    else *reinterpret_cast<float*>(y) = v;
}

// One of several sums to where they are put together, by the same thread every time; past L1, which does not see what
// is added in L2.
__device__ __forceinline__ void put_sum(void* to, uint32_t sum, bool add) {
    if (add) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(to), "f"(__uint_as_float(sum)) : "memory");
    else asm volatile("st.global.cg.u32 [%0], %1;" ::"l"(to), "r"(sum) : "memory");
}
// The last one of them, and those before it.
__device__ __forceinline__ uint32_t take_sum(const void* from, uint32_t sum) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(from) : "memory");
    return __float_as_uint(__fadd_rn(v, __uint_as_float(sum)));
}

template <int XT, bool SWIGLU, bool PAIR>
__global__ void __launch_bounds__(Cfg<XT, SWIGLU, PAIR>::kThreads, 1)
    int8_matmul_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const Int8Args a) {
    using C = Cfg<XT, SWIGLU, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t l_full[C::kLoads], l_empty[C::kLoads];                   // loads
    __shared__ __align__(8) uint64_t a_full[C::kSteps], a_empty[C::kSteps];                   // steps of weights
    __shared__ __align__(8) uint64_t x_full[C::kRowSteps], x_empty[C::kRowSteps];             // and of rows
    __shared__ __align__(8) uint64_t t_full[2], t_empty[2], i_full[2], i_empty[2];
    __shared__ Item info[2];
    __shared__ __align__(8) uint64_t part_bar[2];
    __shared__ unsigned ticket;
    __shared__ __align__(8) uint64_t swap_bar[4], drain_bar;
    __shared__ uint32_t tmem_base, abort_word;

    uint8_t* loads = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(C::kSmem + 1024 <= 232448, "shared memory of a block");
    uint8_t* rows16 = loads + C::kLoads * C::kLoadBytes;
    float* swap = reinterpret_cast<float*>(rows16 + C::kRowSteps * C::kStepBytes);
    volatile uint32_t* abort = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kBlocks = PAIR ? 2 : 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kLoads; ++i)
            mbar_init(smem_u32(&l_full[i]), 1), mbar_init(smem_u32(&l_empty[i]), kConvertWarps / (PAIR ? 2 : 1) + C::kRowWarps / 2);
        for (int i = 0; i < C::kSteps; ++i) {
            mbar_init(smem_u32(&a_full[i]), kBlocks * kConvertWarps / 2);
            mbar_init(smem_u32(&a_empty[i]), 1);
        }
        for (int i = 0; i < C::kRowSteps; ++i)
            mbar_init(smem_u32(&x_full[i]), XT == kInt8 ? C::kRowWarps / 2 : 1), mbar_init(smem_u32(&x_empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&t_full[i]), 1);
            mbar_init(smem_u32(&t_empty[i]), kBlocks * kSumWarps);
            mbar_init(smem_u32(&i_full[i]), 1);
            mbar_init(smem_u32(&i_empty[i]), kConvertWarps + C::kRowWarps + kSumWarps);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&swap_bar[i]), 2);
        mbar_init(smem_u32(&part_bar[0]), kSumWarps);
        mbar_init(smem_u32(&part_bar[1]), 1);
        mbar_init(smem_u32(&drain_bar), 1);
        abort_word = 0u;
        mbar_init_fence();
        tma_prefetch(&map_x);
        tma_prefetch(&map_w);
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(&tmem_base), 512);
    tc_fence_before();
    if (PAIR) cluster_sync();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;
    const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, step = PAIR ? gridDim.x / 2 : gridDim.x;
    pdl_enter();

    Items<Walk<C::kRows, true>, !PAIR> items;
    const Tile& tile = items.tile;
    uint32_t it = 0;  // loads or steps that this warp has taken, over all of its tiles
    bool ok = true;
    // columns of a tile's instructions, and boxes of rows that this block loads
    auto columns = [](int rows) { return (rows + 15) / 16 * 16; };
    auto boxes_of = [&](int rows) { return (columns(rows) / kBlocks + C::kBox - 1) / C::kBox; };

    if (warp < 4) {
        regs_dec<C::kRegs[0]>();
        if (warp == 0) {
            items.begin(a, lane, first, step);
            while (ok && items.next(a, lane, C::kChannels, step)) {
                const int boxes = XT == kInt8 ? boxes_of(tile.rows) : 0;
                if (elect_one()) {
                    for (int kb = items.kb0; kb < items.kb1; ++kb, ++it) {
                        const uint32_t st = it % C::kLoads;
                        ok = mbar_wait<PAIR>(smem_u32(&l_empty[st]), ((it / C::kLoads) & 1) ^ 1, abort);
                        if (!ok) break;
                        const uint32_t bar = smem_u32(&l_full[st]), dst = smem_u32(loads + st * C::kLoadBytes);
                        mbar_expect(bar, (uint32_t)(C::kPlanes * kWBytes + boxes * C::kBox * 128));
                        const int k = kb * 128, e = tile.expert;
                        if (C::kSwap) {
                            tma_load_3d(dst, &map_w, bar, k, tile.n0 + (int)rank * 64, 2 * e);
                            tma_load_3d(dst + kWBytes / 2, &map_w, bar, k, tile.n0 + (int)rank * 64, 2 * e + 1);
                        } else if (PAIR) {
                            tma_load_3d(dst, &map_w, bar, k, tile.n0 + (int)rank * kWRows, e);
                        } else {
                            tma_load_3d(dst, &map_w, bar, k, tile.n0, SWIGLU ? 2 * e : e);
                            tma_load_3d(dst + kWBytes, &map_w, bar, k, SWIGLU ? tile.n0 : tile.n0 + kWRows,
                                        SWIGLU ? 2 * e + 1 : e);
                        }
                        if (XT == kInt8)
                            for (int j = 0; j < boxes; ++j)
                                tma_load_2d(dst + C::kPlanes * kWBytes + j * C::kBox * 128, &map_x, bar, k,
                                            tile.row0 + C::kBox * j);
                    }
                }
                __syncwarp();
                it = __reduce_max_sync(0xffffffffu, it);
                ok = __all_sync(0xffffffffu, ok);
            }
        } else if (warp == 1) {
            ok = rank == 0;
            items.begin(a, lane, first, step);
            SumRoom<PAIR, C::kRows / 2> room;
            while (ok && items.next(a, lane, C::kChannels, step)) {
                room.next(columns(tile.rows));
                const uint32_t d = tmem + room.half * (C::kRows / 2);
                const uint32_t idesc = idesc_16(kWRows * kBlocks, columns(tile.rows), XT == kBf16);
                if (elect_one()) {
                    ok = mbar_wait<PAIR>(smem_u32(&t_empty[room.half]), room.parity(room.half) ^ 1, abort);
                    if (room.both) ok = ok && mbar_wait<PAIR>(smem_u32(&t_empty[1]), room.parity(1) ^ 1, abort);
                    for (int k = items.kb0; ok && k < items.kb1; ++k, ++it) {
                        const uint32_t r = it % C::kRowSteps;
                        ok = mbar_wait<PAIR>(smem_u32(&x_full[r]), (it / C::kRowSteps) & 1, abort);
                        const uint64_t b = smem_desc(smem_u32(rows16 + r * C::kStepBytes));
#pragma unroll
                        for (int p = 0; p < C::kPlanes; ++p) {
                            const uint32_t i = it * C::kPlanes + p, s = i % C::kSteps;
                            ok = ok && mbar_wait<PAIR>(smem_u32(&a_full[s]), (i / C::kSteps) & 1, abort);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                mma_16_tmem<PAIR>(d + p * C::kRows, tmem + C::kACols + s * C::kStepCols + 8 * j,
                                                  b + j / 4 * (C::kPartBytes / 16) + 2 * (j % 4), idesc,
                                                  k > items.kb0 || j > 0);
                            tc_commit<PAIR>(smem_u32(&a_empty[s]));
                        }
                        if (!ok) break;
                        if (!PAIR) tc_commit(smem_u32(&x_empty[r]));
                    }
                    if (ok) tc_commit<PAIR>(smem_u32(&t_full[room.half]));
                    if (ok && room.both) tc_commit<PAIR>(smem_u32(&t_full[1]));
                }
                room.used();
                __syncwarp();
                it = __reduce_max_sync(0xffffffffu, it);
                ok = __all_sync(0xffffffffu, ok);
            }
        } else if (warp == 2) {
            // tiles for the warps below; one of no rows ends them
            items.begin(a, lane, first, step);
            for (uint32_t n = 0;; ++n) {
                const bool more = items.next(a, lane, C::kChannels, step);
                if (!mbar_wait<PAIR>(smem_u32(&i_empty[n & 1]), ((n >> 1) & 1) ^ 1, abort)) break;
                if (lane == 0) {
                    Item& i = info[n & 1];
                    i.tile = more ? tile : Tile{0, 0, 0, 0};
                    if (more) {
                        i.t = items.t;
                        i.loads = items.kb1 - items.kb0;
                        i.again = items.again;
                        i.more = items.more;
                        i.first = i.last = i.block = first;
                        if (!PAIR && a.parts) {
                            i.first = items.owner(items.t * a.KB);
                            i.last = items.owner(items.t * a.KB + a.KB - 1);
                        }
                    }
                    mbar_arrive(smem_u32(&i_full[n & 1]));
                }
                if (!more) break;
            }
        } else if (XT != kInt8) {
            items.begin(a, lane, first, step);
            while (ok && items.next(a, lane, C::kChannels, step)) {
                const int boxes = boxes_of(tile.rows);
                const int row0 = tile.row0 + (int)rank * columns(tile.rows) / 2;
                if (elect_one()) {
                    for (int k = items.kb0; k < items.kb1; ++k, ++it) {
                        // (pairs' rows and weights have the same steps, and one commit for both)
                        const uint32_t s = it % C::kRowSteps;
                        static_assert(!PAIR || C::kRowSteps == C::kSteps, "steps of pairs");
                        ok = mbar_wait<PAIR>(smem_u32(PAIR ? &a_empty[s] : &x_empty[s]), ((it / C::kRowSteps) & 1) ^ 1, abort);
                        if (!ok) break;
                        const uint32_t own = smem_u32(&x_full[s]), bar = PAIR ? map_cluster(own, 0) : own;
                        const uint32_t dst = smem_u32(rows16 + s * C::kStepBytes);
                        if (rank == 0) mbar_expect(own, (uint32_t)(kBlocks * 2 * boxes * C::kBox * 128));
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            for (int j = 0; j < boxes; ++j)
                                tma_load_2d<PAIR>(dst + h * C::kPartBytes + j * C::kBox * 128, &map_x, bar,
                                                  k * 128 + h * 64, row0 + C::kBox * j);
                    }
                }
                __syncwarp();
                it = __reduce_max_sync(0xffffffffu, it);
                ok = __all_sync(0xffffffffu, ok);
            }
        }
    } else if (warp < 4 + kConvertWarps) {
        static_assert(C::kRegs[1] <= C::kLaunchRegs, "registers of the converters");
        if constexpr (C::kRegs[1] < C::kLaunchRegs) regs_dec<C::kRegs[1]>();
        const uint32_t turn = (warp - 4) >> 2;
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)quarter << 21) + C::kACols;  // 32 lanes << 16
        for (uint32_t n = 0; ok; ++n) {
            ok = mbar_wait<PAIR>(smem_u32(&i_full[n & 1]), (n >> 1) & 1, abort);
            if (!ok) break;
            const int rows = info[n & 1].tile.rows, count = info[n & 1].loads;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&i_empty[n & 1]));
            if (rows == 0) break;
            for (int kb = 0; kb < count; ++kb, ++it) {
                if (PAIR && (it & 1) != turn) continue;
                const uint32_t st = it % C::kLoads, i = PAIR ? it : 2 * it + turn, s = i % C::kSteps;
                ok = mbar_wait<PAIR>(smem_u32(&l_full[st]), (it / C::kLoads) & 1, abort);
                if (!ok) break;
                const uint8_t* src = loads + st * C::kLoadBytes + (PAIR ? 0 : turn * kWBytes) + row * 128;
                uint4 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint4*>(src + ((j ^ (row & 7)) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&l_empty[st]));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        widen4<XT == kBf16>(w[4 * h + j].x, v[8 * j], v[8 * j + 1]);
                        widen4<XT == kBf16>(w[4 * h + j].y, v[8 * j + 2], v[8 * j + 3]);
                        widen4<XT == kBf16>(w[4 * h + j].z, v[8 * j + 4], v[8 * j + 5]);
                        widen4<XT == kBf16>(w[4 * h + j].w, v[8 * j + 6], v[8 * j + 7]);
                    }
                    if (h == 0) {  // (the first half is converted before the step is free)
                        ok = mbar_wait<PAIR>(smem_u32(&a_empty[s]), ((i / C::kSteps) & 1) ^ 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    tmem_st32(to + s * C::kStepCols + h * 32, v);
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(map_cluster(smem_u32(&a_full[s]), 0));
                    else mbar_arrive(smem_u32(&a_full[s]));
                }
            }
        }
    } else if (warp < 4 + kConvertWarps + C::kRowWarps) {
        regs_dec<C::kRegs[2]>();
        const uint32_t turn = (warp >> 1) & 1;
        const int h = warp & 1;  // half of a load's values
        for (uint32_t n = 0; ok && XT == kInt8; ++n) {
            ok = mbar_wait<PAIR>(smem_u32(&i_full[n & 1]), (n >> 1) & 1, abort);
            if (!ok) break;
            const int rows = info[n & 1].tile.rows, count = info[n & 1].loads;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&i_empty[n & 1]));
            if (rows == 0) break;
            for (int kb = 0; kb < count; ++kb, ++it) {
                if ((it & 1) != turn) continue;
                const uint32_t st = it % C::kLoads, s = it % C::kRowSteps;
                ok = mbar_wait<PAIR>(smem_u32(&l_full[st]), (it / C::kLoads) & 1, abort);
                if (!ok) break;
                const uint8_t* src = loads + st * C::kLoadBytes + C::kPlanes * kWBytes + lane * 128;
                uint8_t* dst = rows16 + s * C::kStepBytes + h * C::kPartBytes + lane * 128;
                ok = mbar_wait<PAIR>(smem_u32(&x_empty[s]), ((it / C::kRowSteps) & 1) ^ 1, abort);
                if (!ok) break;
                for (int i = 0; i < rows; i += 32) {
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = *reinterpret_cast<const uint4*>(src + i * 128 + (((h * 4 + j) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4 u, v;
                        widen4<false>(x[j].x, u.x, u.y);
                        widen4<false>(x[j].y, u.z, u.w);
                        widen4<false>(x[j].z, v.x, v.y);
                        widen4<false>(x[j].w, v.z, v.w);
                        *reinterpret_cast<uint4*>(dst + i * 128 + (((2 * j) ^ (lane & 7)) << 4)) = u;
                        *reinterpret_cast<uint4*>(dst + i * 128 + (((2 * j + 1) ^ (lane & 7)) << 4)) = v;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&l_empty[st]));
                smem_proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&x_full[s]));
            }
        }
    } else {
        regs_inc<C::kRegs[3]>();
        const int me = warp - (C::kWarps - kSumWarps), half = me >> 2, quarter = warp & 3;
        const uint32_t from = tmem + ((uint32_t)quarter << 21);
        SumRoom<PAIR, C::kRows / 2> room;
        uint32_t swaps = 0;  // of factors, or of tickets
        for (uint32_t n = 0;; ++n) {
            ok = mbar_wait<PAIR>(smem_u32(&i_full[n & 1]), (n >> 1) & 1, abort);
            if (!ok) break;
            const Item item = info[n & 1];
            Tile tile = item.tile;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&i_empty[n & 1]));
            if (tile.rows == 0) break;
            if (!MR_IN_RANGE(tile.expert, a.experts, 911)) tile.expert = 0;
            // this lane's channel; a pair's network: of the gate in the first two warps, of the other factor in the others
            const int factor = C::kSwap ? quarter >> 1 : 0;
            const int col = tile.n0 + (C::kSwap ? (int)rank * 64 + (quarter & 1) * 32 : (int)rank * kWRows + quarter * 32) + lane;
            const float* ws = a.w_scales + ((int64_t)tile.expert * (SWIGLU ? 2 : 1) + factor) * a.N;
            const bool real = col < a.N;
            // rows of this warp, may be none: those of half of the tile's columns
            const int cols = (columns(tile.rows) / 2 + 15) / 16 * 16;
            const int mine = min(cols, tile.rows - half * cols);
            const int64_t row0 = (int64_t)tile.row0 + half * cols;
            const bool inside = mine <= 0 || MR_IN_RANGE(row0 + mine - 1, a.rows, 912);
            constexpr int kGroups = (C::kHalf + 31) / 32;
            float xs[kGroups];  // lane i: those of rows i, 32 + i, ...
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                xs[i] = a.x_scales && inside && 32 * i + lane < mine ? a.x_scales[(row0 + 32 * i + lane) * a.xs_row] : 1.0f;
            constexpr int kLd = C::kChunk, kKeep = C::kSwap ? kLd / 2 : kLd;  // rows read at once, and of them this warp's
            const bool wide = !SWIGLU && a.y_dtype == MR_DTYPE_F32;
            const bool several = a.sums == kPlainSums && (item.again || item.more);
            const bool added = wide && a.sums == kScaledSums && item.again;
            const int elem = wide ? 4 : 2;
            char* y = reinterpret_cast<char*>(a.y) + (row0 * a.y_stride + col) * elem;
            const int64_t y_step = a.y_stride * elem;
            const float w_scale = ws[real ? col : 0];
            auto scaled = [&](const auto& v, float by, int c, auto& f) {
                constexpr int kCount = sizeof(f) / sizeof(f[0]);
#pragma unroll
                for (int j = 0; j < kCount; ++j) f[j] = __fmul_rn(__uint_as_float(v[j]), by);
                if (a.x_scales) {
                    float s = xs[0];
#pragma unroll
                    for (int i = 1; i < kGroups; ++i)
                        if (c / 32 == i) s = xs[i];
#pragma unroll
                    for (int j = 0; j < kCount; ++j) f[j] = __fmul_rn(f[j], __shfl_sync(0xffffffffu, s, c % 32 + j));
                }
            };
            room.next(columns(tile.rows));
            ok = mbar_wait<PAIR>(smem_u32(&t_full[room.half]), room.parity(room.half), abort);
            if (room.both) ok = ok && mbar_wait<PAIR>(smem_u32(&t_full[1]), room.parity(1), abort);
            if (!ok) break;
            room.used();
            tc_fence_after();
            const uint32_t sums = from + room.half * (C::kRows / 2) + half * cols;
            auto hand_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane != 0) return;
                if (PAIR) {
                    mbar_arrive_cluster(map_cluster(smem_u32(&t_empty[0]), 0));
                } else {
                    mbar_arrive(smem_u32(&t_empty[room.half]));
                    if (room.both) mbar_arrive(smem_u32(&t_empty[1]));
                }
            };
            if (mine <= 0) hand_back();
            if constexpr (!PAIR) {
                // the second operand's channels, or the same ones of the other factor
                const int col1 = SWIGLU ? col : col + kWRows;
                const bool real1 = col1 < a.N;
                const float w_scale1 = ws[SWIGLU ? (real ? a.N + col : 0) : (real1 ? col1 : 0)];
                // rows c .. of the result from their sums
                auto finish = [&](int c, const uint32_t (&v)[kLd], const uint32_t (&u)[kLd]) {
                    float f[kLd], g[kLd];
                    scaled(v, w_scale, c, f);
                    scaled(u, w_scale1, c, g);
                    if (SWIGLU) {
#pragma unroll
                        for (int j = 0; j < kLd; ++j) f[j] = silu(f[j]) * g[j];
                    }
                    if (!inside) return;
                    char* to = y + c * y_step;
                    if (wide) {
#pragma unroll
                        for (int j = 0; j < kLd; ++j, to += y_step) {
                            if (c + j < mine && real) put(to, f[j], added);
                            if (c + j < mine && real1) put(to + kWRows * 4, g[j], added);
                        }
                        return;
                    }
                    uint32_t w[kLd];
                    pack(!SWIGLU && a.y_dtype == MR_DTYPE_F16, f, g, w);
#pragma unroll
                    for (int j = 0; j < kLd; ++j, to += y_step) {
                        const bool in = c + j < mine;
                        if (in && real) *reinterpret_cast<uint16_t*>(to) = (uint16_t)w[j];
                        if (!SWIGLU && in && real1) *reinterpret_cast<uint16_t*>(to + kWRows * 2) = (uint16_t)(w[j] >> 16);
                    }
                };
                // where the block's sums of a tile in several parts go: its first part starts a tile, or is in one
                const bool whole = item.first == item.last;
                auto part_of = [&](int block) {
                    return a.parts + (((int64_t)(2 * block + (block == item.first)) * a.part_rows + half * cols) << 8) +
                           quarter * 32 + lane;
                };
                float* part = part_of(item.block);
#pragma unroll 1
                for (int c = 0; c < mine; c += kLd) {
                    uint32_t v[kLd], u[kLd];
                    tmem_load(v, sums + c);
                    tmem_load(u, sums + C::kRows + c);
                    tmem_ld_wait(v);
                    tmem_ld_wait(u);
                    if (c + kLd >= mine) hand_back();  // everything is in registers
                    if (whole) {
                        if (several) {
                            // (no whole tile is among those that blocks share: a share is at most 9 of 17 of a tile's loads)
                            float* room = a.room + (((int64_t)item.block * C::kRows + half * C::kHalf) << 8) + quarter * 32 + lane;
                            char* to = wide ? y + c * y_step : reinterpret_cast<char*>(room + c * 256);
                            const int64_t next = wide ? y_step : 1024;
#pragma unroll
                            for (int j = 0; j < kLd; ++j, to += next) {
                                if (c + j >= mine || !inside) continue;
                                if (item.more) {
                                    if (real) put_sum(to, v[j], item.again);
                                    if (real1) put_sum(to + kWRows * 4, u[j], item.again);
                                } else {
                                    if (real) v[j] = take_sum(to, v[j]);
                                    if (real1) u[j] = take_sum(to + kWRows * 4, u[j]);
                                }
                            }
                            if (item.more) continue;
                        }
                        finish(c, v, u);
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < kLd; ++j)
                        if (c + j < mine && MR_IN_RANGE(half * cols + c + j, a.part_rows, 913)) {
                            put_sum(part + (c + j) * 256, v[j], item.again);
                            put_sum(part + (c + j) * 256 + 128, u[j], item.again);
                        }
                }
                if (!whole && !item.more) {
                    // the warps' sums are out, one of them takes a ticket for all
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&part_bar[0]));
                    if (me == 0) {
                        ok = mbar_wait(smem_u32(&part_bar[0]), swaps & 1, abort);
                        if (!ok) break;
                        if (lane == 0) {
                            __threadfence();
                            ticket = atomicAdd(a.tickets + item.t, 1u);
                            __threadfence();
                            mbar_arrive(smem_u32(&part_bar[1]));
                        }
                    }
                    ok = mbar_wait(smem_u32(&part_bar[1]), swaps & 1, abort);
                    ++swaps;
                    if (!ok) break;
                    if (ticket == (unsigned)(item.last - item.first)) {
                        __threadfence();
#pragma unroll 1
                        for (int c = 0; c < mine; c += kLd) {
                            float f[kLd], g[kLd];
#pragma unroll
                            for (int j = 0; j < kLd; ++j) f[j] = g[j] = 0.0f;
                            for (int b = item.first; b <= item.last; ++b) {
                                const float* from_b = part_of(b) + c * 256;
#pragma unroll
                                for (int j = 0; j < kLd; ++j)
                                    if (c + j < mine) {
                                        f[j] = __fadd_rn(f[j], __ldcg(from_b + j * 256));
                                        g[j] = __fadd_rn(g[j], __ldcg(from_b + j * 256 + 128));
                                    }
                            }
                            uint32_t v[kLd], u[kLd];
#pragma unroll
                            for (int j = 0; j < kLd; ++j) v[j] = __float_as_uint(f[j]), u[j] = __float_as_uint(g[j]);
                            finish(c, v, u);
                        }
                    }
                }
            } else {
                if constexpr (!SWIGLU) {
                    // With tiles to come the sums are handed back before the stores of 16-bit results, which wait in
                    // registers (16384 x 7168 x 7168: 836 us, as below 869). In a launch of one tile a block what
                    // this code costs is its own way from memory (1003 rows of 12 groups, 1000 -> 1100: 15.9 us, as
                    // below 13.7).
                    if (a.many && !wide && !several) {
                        uint32_t packed[C::kHalf / 2];
#pragma unroll
                        for (int c = 0; c < C::kHalf; c += kLd) {
                            if (c >= mine) break;
                            uint32_t v[kLd];
                            tmem_load(v, sums + c);
                            tmem_ld_wait(v);
                            float f[kLd];
                            scaled(v, w_scale, c, f);
                            float even[kLd / 2], odd[kLd / 2];
                            uint32_t w[kLd / 2];
#pragma unroll
                            for (int j = 0; j < kLd / 2; ++j) even[j] = f[2 * j], odd[j] = f[2 * j + 1];
                            pack(a.y_dtype == MR_DTYPE_F16, even, odd, w);
#pragma unroll
                            for (int j = 0; j < kLd / 2; ++j) packed[c / 2 + j] = w[j];
                        }
                        if (mine > 0) hand_back();
                        if (real && inside) {
                            char* to = y;
#pragma unroll
                            for (int j = 0; j < C::kHalf; ++j, to += y_step)
                                if (j < mine) *reinterpret_cast<uint16_t*>(to) = (uint16_t)(packed[j / 2] >> (16 * (j & 1)));
                        }
                        continue;
                    }
                    if (several) {
                        // where row c's sums are put together. (Found anew for each chunk: 4096 x 7168 int8 -> 4096 fp32 275
                        // us, from an address held for the tile 447; one sum, which is not exact, 170.)
                        auto home = [&](int c) {
                            float* room = a.room + (((int64_t)first * C::kRows + half * C::kHalf + c) << 8) + (int)rank * kWRows +
                                          quarter * 32 + lane;
                            return wide ? y + c * y_step : reinterpret_cast<char*>(room);
                        };
                        if (item.more) {
#pragma unroll 1
                            for (int c = 0; c < mine; c += kLd) {
                                uint32_t v[kLd];
                                tmem_load(v, sums + c);
                                tmem_ld_wait(v);
                                if (c + kLd >= mine) hand_back();
                                char* to = home(c);
                                const int64_t next = wide ? y_step : 1024;
                                const bool out = real && inside;
                                if (out && item.again) {
#pragma unroll
                                    for (int j = 0; j < kLd; ++j, to += next)
                                        if (c + j < mine) put_sum(to, v[j], true);
                                } else if (out) {
#pragma unroll
                                    for (int j = 0; j < kLd; ++j, to += next)
                                        if (c + j < mine) put_sum(to, v[j], false);
                                }
                                __syncwarp();
                            }
                            continue;
                        }
                        constexpr int kFew = kLd / 2;  // (with kLd, whose earlier sums have registers, too, the kernel spills)
#pragma unroll 1
                        for (int c = 0; c < mine; c += kFew) {
                            uint32_t v[kFew];
                            tmem_load(v, sums + c);
                            tmem_ld_wait(v);
                            if (c + kFew >= mine) hand_back();
                            char* to = home(c);
                            const int64_t next = wide ? y_step : 1024;
                            const bool out = real && inside;
#pragma unroll
                            for (int j = 0; j < kFew; ++j, to += next)
                                if (out && c + j < mine) v[j] = take_sum(to, v[j]);
                            __syncwarp();
                            float f[kFew];
                            scaled(v, w_scale, c, f);
                            uint32_t w[kFew];
                            if (!wide) pack(a.y_dtype == MR_DTYPE_F16, f, f, w);
                            to = y + c * y_step;
#pragma unroll
                            for (int j = 0; j < kFew; ++j, to += y_step) {
                                if (!out || c + j >= mine) continue;
                                if (wide) put(to, f[j], false);
                                else *reinterpret_cast<uint16_t*>(to) = (uint16_t)w[j];
                            }
                            __syncwarp();
                        }
                        continue;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < mine; c += kLd) {
                    uint32_t v[kLd];
                    tmem_load(v, sums + c);
                    tmem_ld_wait(v);
                    if (c + kLd >= mine) hand_back();  // everything is in registers
                    float f[kLd];
                    scaled(v, w_scale, c, f);
                    int r = c;
                    if constexpr (C::kSwap) {
                        // Two warps have the two factors of the same channels: the first takes the chunk's first
                        // rows, the second the others, each from the other's half of `swap`, two of them in turn.
                        float* out = swap + ((me * 2 + (swaps & 1)) * kKeep) * 32 + lane;
                        const float* in = swap + (((me ^ 2) * 2 + (swaps & 1)) * kKeep) * 32 + lane;
                        const uint32_t bar = smem_u32(&swap_bar[half * 2 + (quarter & 1)]);
#pragma unroll
                        for (int j = 0; j < kKeep; ++j) out[j * 32] = factor ? f[j] : f[kKeep + j];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar);
                        ok = mbar_wait<PAIR>(bar, swaps & 1, abort);
                        ++swaps;
                        if (!ok) break;
#pragma unroll
                        for (int j = 0; j < kKeep; ++j) {
                            const float o = in[j * 32];
                            f[j] = factor ? silu(o) * f[kKeep + j] : silu(f[j]) * o;
                        }
                        r += factor * kKeep;
                    }
                    if (!real || !inside) continue;
                    char* to = y + r * y_step;
                    if (added) {
#pragma unroll
                        for (int j = 0; j < kKeep; ++j, to += y_step)
                            if (r + j < mine) put(to, f[j], true);
                    } else if (wide) {
#pragma unroll
                        for (int j = 0; j < kKeep; ++j, to += y_step)
                            if (r + j < mine) put(to, f[j], false);
                    } else {
                        float even[kKeep / 2], odd[kKeep / 2];
                        uint32_t w[kKeep / 2];
#pragma unroll
                        for (int j = 0; j < kKeep / 2; ++j) even[j] = f[2 * j], odd[j] = f[2 * j + 1];
                        pack(!SWIGLU && a.y_dtype == MR_DTYPE_F16, even, odd, w);
#pragma unroll
                        for (int j = 0; j < kKeep; ++j, to += y_step)
                            if (r + j < mine) *reinterpret_cast<uint16_t*>(to) = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
                    }
                }
                if (!ok) break;
            }
        }
    }
    __syncthreads();
    if (PAIR) cluster_sync();
    if (abort_word) {  // let what is in flight land
        if (warp == 0)
            for (uint32_t k = it > C::kLoads ? it - C::kLoads : 0; k < it; ++k)
                mbar_drain(smem_u32(&l_full[k % C::kLoads]), (k / C::kLoads) & 1);
        if (XT != kInt8 && warp == 3 && rank == 0)
            for (uint32_t k = it > C::kRowSteps ? it - C::kRowSteps : 0; k < it; ++k)
                mbar_drain(smem_u32(&x_full[k % C::kRowSteps]), (k / C::kRowSteps) & 1);
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
    if (warp == 1) tmem_free<PAIR>(tmem, 512);
}

// int8 rows to f16, whose sums the kernels above then take as they are: 16 values a thread.
__global__ void __launch_bounds__(256)
    widen_rows_kernel(const char* x, int64_t x_row, int64_t rows, int64_t K, const int64_t* num_rows, char* to,
                      int64_t to_row, uint32_t chunks) {
    pdl_enter();
    if (num_rows) rows = max((int64_t)0, min(rows, *num_rows));
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / chunks, c = i - row * chunks;
    if (row >= rows) return;
    const char* p = x + row * x_row + c * 16;
    uint4 w;
    if (c * 16 + 16 <= K) {
        w = ld_stream_v4(p);
    } else {
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c * 16 + j < K) u[j >> 2] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
        w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    uint4 a, b;
    widen4<false>(w.x, a.x, a.y);
    widen4<false>(w.y, a.z, a.w);
    widen4<false>(w.z, b.x, b.y);
    widen4<false>(w.w, b.z, b.w);
    uint4* q = reinterpret_cast<uint4*>(to + row * to_row + c * 32);
    q[0] = a;
    q[1] = b;
}

// Tickets to 0. (1 row, 4096 -> 2048: 14.8 us on the GPU, with a memset in front of the product 18.5.)
__global__ void __launch_bounds__(256) clear_kernel(uint4* tickets, int n) {
    pdl_enter();
    for (int i = threadIdx.x; i < n; i += 256) tickets[i] = make_uint4(0u, 0u, 0u, 0u);
}

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }
int ceil_div(int64_t a, int64_t b) { return (int)ceil_div64(a, b); }
bool aligned16(const void* p) { return aligned(p, 16); }

template <int XT, bool SWIGLU, bool PAIR>
cudaError_t launch_int8(const CUtensorMap (&m)[2], Int8Args a, int64_t tiles, cudaStream_t s) {
    if (a.parts) tiles = tiles * a.KB / a.part_loads + 1;
    auto kernel = int8_matmul_kernel<XT, SWIGLU, PAIR>;
    constexpr int smem = Cfg<XT, SWIGLU, PAIR>::kSmem;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Cfg<XT, SWIGLU, PAIR>::kThreads);
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
    a.many = tiles > n;
    return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], a);
}

// One product over the groups. x: rows of type xt; w: int8 [experts][N][K], or [experts][2][N][K]
// for the network's first product (swiglu).
struct Product {
    const void* x;
    int64_t x_stride;          // bytes
    int xt;
    const void* w;
    int64_t w_row, w_matrix;   // byte strides of a row and of a matrix [N, K]
    int64_t K;
    bool swiglu;
    bool exact;                // rows of int8 values (whatever type holds them)
};

// 16-bit results' values of k to a sum: what the tensor cores cut is 1e-4 of as many values of one sign (of 131072,
// 7.6e-4: more than f16's rounding).
constexpr int64_t kMostSum = 16384;

// The tiles of a product, or more.
int64_t most_tiles(int64_t rows, int64_t G, int64_t N, bool pair, bool swiglu) {
    const int64_t down = std::min<int64_t>((int64_t)ceil_div(rows, pair ? 256 : 96) + G - 1, rows);
    return down * ceil_div(N, swiglu ? 128 : 256);
}

// Pairs of blocks where the products count, single blocks where the weights' way from HBM does: a tile for
// each SM, of groups of few rows (int8 rows, 7168 -> 4096: 576 of 64 groups 310 us in single blocks, 365 in pairs;
// 4096 -> 4096: 1000 rows of 16 groups 71 and 79; 4096 -> 2048: 4000 rows of 64 groups 128 and 133, 8000 195 and 167;
// 515 rows of 6 groups through the network, 1080 / 712, 49 and 37). Up to 32 rows the blocks may share tiles (below).
// The network's rows of several sums go to single blocks, whose two factors are in one warp.
bool use_pairs(int64_t rows, int64_t G, int64_t N, int64_t K, bool swiglu) {
    if (rows <= 32 || (swiglu && K > kMostSum)) return false;
    return rows > 64 * std::min<int64_t>(G, rows) || most_tiles(rows, G, N, false, swiglu) < device_sm_count();
}

// Whether single blocks take equal shares of the loads: where few rows leave half of the SMs without a
// tile of their own (rows x cols -> channels, with and without: 1 x 4096 -> 2048 18 and 25 us, 1 x 7168 -> 7168
// 27 and 40, 32 x 7168 -> 4096 32 and 40). With a tile for each SM adding up costs more than it
// gives (8 rows of 8 groups, 7168 -> 4096: 63 and 59), and so it does for short rows (1 x 1024 -> 1024: 15 and 13) and with
// more sums to add up (1003 rows of 12 groups, 1000 -> 1100: 49 and 19).
bool use_shares(int64_t rows, int64_t G, int64_t N, int64_t K, bool swiglu) {
    return rows <= 32 && K > 15 * 128 && G <= kMostShares &&
           most_tiles(rows, G, N, false, swiglu) <= device_sm_count() / 2;
}
int64_t part_rows(int64_t rows) { return std::min<int64_t>(96, (rows + 15) / 16 * 16); }
uint64_t part_bytes(int64_t rows) { return (uint64_t)2 * device_sm_count() * part_rows(rows) * 1024; }
uint64_t ticket_bytes(int64_t rows, int64_t G, int64_t N, int64_t K, bool swiglu) {
    return use_shares(rows, G, N, K, swiglu) ? align_up((uint64_t)most_tiles(rows, G, N, false, swiglu) * 4, 256) : 0;
}

// The sums of a block's tile, where rows are long and blocks do not share tiles.
uint64_t sum_bytes(int64_t rows, int64_t G, int64_t N, int64_t K, bool swiglu) {
    if (K <= kMostSum || use_shares(rows, G, N, K, swiglu)) return 0;
    const bool pair = use_pairs(rows, G, N, K, swiglu);
    return (uint64_t)std::min<int64_t>(most_tiles(rows, G, N, pair, swiglu), device_sm_count() / (pair ? 2 : 1)) *
           (pair ? 256 : 96) * 1024;
}

// What counts a product's tiles, and the threads that widen its rows, holds them.
bool countable(int64_t rows, int64_t G, int64_t N, int64_t K, bool swiglu, bool eight) {
    const bool pair = use_pairs(rows, G, N, K, swiglu);
    return most_tiles(rows, G, N, pair, swiglu) <= INT32_MAX - 4096 &&  // (a block's count of them goes one round past)
           (!pair || !eight || ceil_div64(rows * ceil_div64(K, 16), 256) <= INT32_MAX);
}

mr_status run_product(const Product& p, Int8Args a, bool pair, cudaStream_t s) {
    a.n_tiles = ceil_div(a.N, p.swiglu ? 128 : 256);
    a.KB = ceil_div(p.K, 128);
    const bool wide = a.y_dtype == MR_DTYPE_F32 && !p.swiglu;
    const int sums = ceil_div(p.K, wide ? 1024 : kMostSum);
    a.sum_loads = ceil_div(a.KB, sums);
    a.sums = sums == 1 ? kOneSum : wide && !p.exact ? kScaledSums : kPlainSums;
    const int64_t tiles = most_tiles(a.rows, a.G, a.N, pair, p.swiglu);
    CUtensorMap m[2];
    const bool eight = p.xt == kInt8;
    const uint64_t xd[2] = {(uint64_t)p.K, (uint64_t)a.rows}, xs[1] = {(uint64_t)p.x_stride};
    const uint32_t xb[2] = {eight ? 128u : 64u, pair ? 64u : 32u};
    const uint64_t wd[3] = {(uint64_t)p.K, (uint64_t)a.N, (uint64_t)a.experts * (p.swiglu ? 2 : 1)};
    const uint64_t ws[2] = {(uint64_t)p.w_row, (uint64_t)p.w_matrix};
    const uint32_t wb[3] = {128, (uint32_t)(p.swiglu && pair ? kWRows / 2 : kWRows), 1};
    if (!make_tensor_map(&m[0], eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, eight ? 1 : 2, p.x, 2,
                         xd, xs, xb) ||
        !make_tensor_map(&m[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.w, 3, wd, ws, wb))
        return MR_ERR_CUDA;
    cudaError_t e;
    if (pair) {
        if (p.swiglu) e = p.xt == kBf16 ? launch_int8<kBf16, true, true>(m, a, tiles, s)
                                        : launch_int8<kF16, true, true>(m, a, tiles, s);
        else e = p.xt == kBf16 ? launch_int8<kBf16, false, true>(m, a, tiles, s)
                               : launch_int8<kF16, false, true>(m, a, tiles, s);
    } else if (p.swiglu) {
        e = p.xt == kBf16  ? launch_int8<kBf16, true, false>(m, a, tiles, s)
            : p.xt == kF16 ? launch_int8<kF16, true, false>(m, a, tiles, s)
                           : launch_int8<kInt8, true, false>(m, a, tiles, s);
    } else {
        e = p.xt == kBf16  ? launch_int8<kBf16, false, false>(m, a, tiles, s)
            : p.xt == kF16 ? launch_int8<kF16, false, false>(m, a, tiles, s)
                           : launch_int8<kInt8, false, false>(m, a, tiles, s);
    }
    return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

// Results that take several scaled sums (kScaledSums, where rows are as long as those of shared tiles): their tiles have
// no shares, although the size of the workspace, which does not go by y's type, has room for them.
bool scaled_sums(int32_t yDtype, bool eight) { return yDtype == MR_DTYPE_F32 && !eight; }

bool row_type(int32_t dt) { return dt == MR_DTYPE_INT8 || dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16; }
bool out_type(int32_t dt) { return dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16 || dt == MR_DTYPE_F32; }

bool common_sizes(int64_t rows, int64_t experts, int64_t numGroups, int64_t a, int64_t b) {
    return rows >= 0 && rows <= MR_MAX_EXPERT_ROWS && experts >= 1 && experts <= MR_MAX_EXPERT_NUM &&
           numGroups >= -1 && numGroups <= MR_MAX_EXPERT_ROWS && a >= 1 && a <= MR_MAX_EXPERT_COLS && b >= 1 &&
           b <= MR_MAX_EXPERT_COLS;
}

// 16-bit rows [rows, cols] in the workspace.
int64_t wide_stride(int64_t cols) { return (int64_t)align_up((uint64_t)cols, 64) * 2; }
uint64_t wide_bytes(int64_t rows, int64_t cols) { return align_up((uint64_t)rows * wide_stride(cols), 256); }

// x as the product takes it: int8 rows in front of a kernel of pairs become 16-bit rows in `room`.
cudaError_t prepare_rows(Product& p, const Int8Args& a, bool pair, const int64_t* numRows, void* room, cudaStream_t s) {
    if (!pair || p.xt != kInt8) return cudaSuccess;
    const uint32_t chunks = (uint32_t)((p.K + 15) / 16);
    const int64_t total = (int64_t)a.rows * chunks;
    cudaError_t e = launch_pdl(widen_rows_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s,
                               reinterpret_cast<const char*>(p.x), p.x_stride, (int64_t)a.rows, p.K, numRows,
                               reinterpret_cast<char*>(room), wide_stride(p.K), chunks);
    p.x = room;
    p.x_stride = wide_stride(p.K);
    p.xt = kF16;
    return e;
}

// A call's workspace: wide rows, the network's h, then tickets of each product, sums of parts of tiles and of long rows.
struct Room {
    uint64_t x, h, tickets[2], parts, sums;
    uint64_t total() const { return x + h + tickets[0] + tickets[1] + parts + sums; }
};
Room matmul_room(int64_t rows, int64_t G, int64_t N, int64_t K, int32_t dt) {
    Room r{dt == MR_DTYPE_INT8 && use_pairs(rows, G, N, K, false) ? wide_bytes(rows, K) : 0, 0,
           {ticket_bytes(rows, G, N, K, false), 0}, 0, sum_bytes(rows, G, N, K, false)};
    r.parts = r.tickets[0] ? part_bytes(rows) : 0;
    return r;
}
Room ffn_room(int64_t rows, int64_t G, int64_t hidden, int64_t inter, int32_t dt) {
    Room r{dt == MR_DTYPE_INT8 && use_pairs(rows, G, inter, hidden, true) ? wide_bytes(rows, hidden) : 0,
           wide_bytes(rows, inter),
           {ticket_bytes(rows, G, inter, hidden, true), ticket_bytes(rows, G, hidden, inter, false)}, 0,
           std::max(sum_bytes(rows, G, inter, hidden, true), sum_bytes(rows, G, hidden, inter, false))};
    r.parts = r.tickets[0] || r.tickets[1] ? part_bytes(rows) : 0;
    return r;
}
// Tickets at 0 (nothing keeps the workspace between calls), where products take some. scaled: the last product does not.
cudaError_t clear_tickets(const Room& r, bool scaled, bool network, char* workspace, cudaStream_t s) {
    const uint64_t n = (scaled && !network ? 0 : r.tickets[0]) + (scaled ? 0 : r.tickets[1]);
    return n ? launch_pdl(clear_kernel, dim3(1), dim3(256), 0, s, reinterpret_cast<uint4*>(workspace + r.x + r.h), (int)(n / 16))
             : cudaSuccess;
}
// The product's share of the room.
void take_room(Int8Args& a, const Room& r, bool scaled, char* workspace, int product) {
    char* tickets = workspace + r.x + r.h;
    a.parts = r.tickets[product] && !scaled ? reinterpret_cast<float*>(tickets + r.tickets[0] + r.tickets[1]) : nullptr;
    a.part_rows = (int)part_rows(a.rows);
    a.part_loads = a.rows > 8 ? 8 : 4;  // (16 x 4096 -> 4096: 21 us, with 4 loads 24; 1 x 4096 -> 2048: 18, with 8 19)
    a.tickets = reinterpret_cast<unsigned*>(tickets + (product ? r.tickets[0] : 0));
    a.room = reinterpret_cast<float*>(tickets + r.tickets[0] + r.tickets[1] + r.parts);
}

// Checks that both products make of their weights; wr, wm: byte strides.
bool weight_strides(const int64_t* strides, int64_t matrices, int64_t N, int64_t K, int64_t* wr, int64_t* wm) {
    const int64_t top = INT64_C(1) << 40;
    *wr = K, *wm = N * K;
    if (strides) *wr = strides[0], *wm = strides[1];
    *wr = stride_of(N, *wr, K);
    *wm = stride_of(matrices, *wm, N * *wr);
    return *wr >= K && *wr % 16 == 0 && *wm % 16 == 0 && *wr <= top && *wm <= top &&
           (matrices == 1 || *wm >= (N - 1) * *wr + K);
}

}  // namespace

MR_CHECK_ACCESSOR(int8_matmul)

cudaError_t waits_out_int8_matmul(unsigned* out, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_waits_out, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0u;
        e = cudaMemcpyToSymbol(g_waits_out, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_grouped_matmul_int8_get_workspace_size(int64_t rows, int64_t numGroups, int64_t outCols,
                                                                int64_t cols, int32_t xDtype, uint64_t* workspaceSize) {
    if (!row_type(xDtype) || !common_sizes(rows, 1, numGroups, outCols, cols)) return MR_ERR_PARAM_INVALID;
    if (!workspaceSize) return MR_ERR_PARAM_NULLPTR;
    *workspaceSize = rows && numGroups ? matmul_room(rows, numGroups < 0 ? 1 : numGroups, outCols, cols, xDtype).total() : 0;
    return MR_OK;
}

extern "C" mr_status moe_grouped_matmul_int8(const void* x, int32_t xDtype, int64_t xStride, const float* xScales,
                                             int64_t xScaleStride, const void* weights, const int64_t* weightStrides,
                                             const float* weightScales, const int64_t* groupList, int64_t numGroups,
                                             const int64_t* numRows, int64_t expertBase, int64_t rows, int64_t experts,
                                             int64_t outCols, int64_t cols, void* y, int32_t yDtype, int64_t yStride,
                                             void* workspace, uint64_t workspaceSize, void* stream) {
    const bool eight = xDtype == MR_DTYPE_INT8;
    const int64_t top = INT64_C(1) << 40, elem = eight ? 1 : 2;
    if (!row_type(xDtype) || !out_type(yDtype)) return MR_ERR_PARAM_INVALID;
    if (!common_sizes(rows, experts, numGroups, outCols, cols)) return MR_ERR_PARAM_INVALID;
    if (!groupList && numGroups > 0) return MR_ERR_PARAM_NULLPTR;
    if (xStride < 0 || xStride > top || yStride < outCols || yStride > top) return MR_ERR_PARAM_INVALID;
    xStride = stride_of(rows, xStride * elem, cols * elem);
    if (xStride < cols * elem || xStride % 16) return MR_ERR_PARAM_INVALID;
    int64_t wr, wm;
    if (!weight_strides(weightStrides, experts, outCols, cols, &wr, &wm)) return MR_ERR_PARAM_INVALID;
    if (xScales && (xScaleStride < 0 || xScaleStride > top)) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    const Room room = numGroups ? matmul_room(rows, numGroups < 0 ? 1 : numGroups, outCols, cols, xDtype) : Room{};
    if (!x || !weights || !weightScales || !y || (eight && !xScales) || (room.total() && !workspace))
        return MR_ERR_PARAM_NULLPTR;
    if (workspaceSize < room.total()) return MR_ERR_WORKSPACE;
    if (!aligned16(weights) || !aligned16(x) || (numGroups > 0 && !aligned16(groupList)) ||
        (room.total() && !aligned(workspace, 256)) || !aligned(y, yDtype == MR_DTYPE_F32 ? 4 : 2) || !aligned(xScales, 4) ||
        !aligned(weightScales, 4) || !aligned(numRows, 8))
        return MR_ERR_PARAM_INVALID;
    if (numGroups && !countable(rows, numGroups < 0 ? 1 : numGroups, outCols, cols, false, eight)) return MR_ERR_PARAM_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Int8Args a{};
    a.groups = numGroups < 0 ? nullptr : groupList;
    a.G = numGroups < 0 ? 1 : (int)numGroups;
    a.rows = (int)rows;
    a.experts = (int)experts;
    a.expert_base = expertBase;
    if (a.G == 0) return MR_OK;
    a.x_scales = xScales;
    a.xs_row = xScaleStride;
    a.w_scales = weightScales;
    a.N = (int)outCols;
    a.y = y;
    a.y_stride = yStride;
    a.y_dtype = yDtype;
    Product p{x, xStride, eight ? kInt8 : xDtype == MR_DTYPE_BF16 ? kBf16 : kF16, weights, wr, wm, cols, false, eight};
    const bool pair = use_pairs(rows, a.G, outCols, cols, false);
    char* base = reinterpret_cast<char*>(workspace);
    const bool scaled = scaled_sums(yDtype, eight);
    MR_TRY_CUDA(clear_tickets(room, scaled, false, base, s));
    MR_TRY_CUDA(prepare_rows(p, a, pair, numRows, base, s));
    take_room(a, room, scaled, base, 0);
    return run_product(p, a, pair, s);
}

extern "C" mr_status moe_expert_ffn_int8_get_workspace_size(int64_t rows, int64_t numGroups, int64_t hidden,
                                                            int64_t inter, int32_t xDtype, uint64_t* workspaceSize) {
    if (!row_type(xDtype) || !common_sizes(rows, 1, numGroups, hidden, inter)) return MR_ERR_PARAM_INVALID;
    if (!workspaceSize) return MR_ERR_PARAM_NULLPTR;
    *workspaceSize = rows && numGroups ? ffn_room(rows, numGroups < 0 ? 1 : numGroups, hidden, inter, xDtype).total() : 0;
    return MR_OK;
}

extern "C" mr_status moe_expert_ffn_int8(const void* x, int32_t xDtype, int64_t xStride, const float* xScales,
                                         int64_t xScaleStride, const void* w13, const int64_t* w13Strides,
                                         const float* w13Scales, const void* w2, const int64_t* w2Strides,
                                         const float* w2Scales, const int64_t* groupList, int64_t numGroups,
                                         const int64_t* numRows, int64_t expertBase, int64_t rows, int64_t experts,
                                         int64_t hidden, int64_t inter, void* y, int32_t yDtype, int64_t yStride,
                                         void* workspace, uint64_t workspaceSize, void* stream) {
    const bool eight = xDtype == MR_DTYPE_INT8;
    const int64_t top = INT64_C(1) << 40, elem = eight ? 1 : 2;
    if (!row_type(xDtype) || !out_type(yDtype)) return MR_ERR_PARAM_INVALID;
    if (!common_sizes(rows, experts, numGroups, hidden, inter)) return MR_ERR_PARAM_INVALID;
    if (!groupList && numGroups > 0) return MR_ERR_PARAM_NULLPTR;
    if (xStride < 0 || xStride > top || yStride < hidden || yStride > top) return MR_ERR_PARAM_INVALID;
    xStride = stride_of(rows, xStride * elem, hidden * elem);
    if (xStride < hidden * elem || xStride % 16) return MR_ERR_PARAM_INVALID;
    int64_t ar, am, br, bm;
    if (!weight_strides(w13Strides, 2 * experts, inter, hidden, &ar, &am) ||
        !weight_strides(w2Strides, experts, hidden, inter, &br, &bm))
        return MR_ERR_PARAM_INVALID;
    if (xScales && (xScaleStride < 0 || xScaleStride > top)) return MR_ERR_PARAM_INVALID;
    if (rows == 0) return MR_OK;
    const Room room = numGroups ? ffn_room(rows, numGroups < 0 ? 1 : numGroups, hidden, inter, xDtype) : Room{};
    if (!x || !w13 || !w13Scales || !w2 || !w2Scales || !y || (room.total() && !workspace) || (eight && !xScales))
        return MR_ERR_PARAM_NULLPTR;
    if (workspaceSize < room.total()) return MR_ERR_WORKSPACE;
    if (!aligned16(w13) || !aligned16(w2) || !aligned16(x) || (numGroups > 0 && !aligned16(groupList)) ||
        !aligned(workspace, 256) || !aligned(y, yDtype == MR_DTYPE_F32 ? 4 : 2) || !aligned(xScales, 4) ||
        !aligned(w13Scales, 4) || !aligned(w2Scales, 4) || !aligned(numRows, 8))
        return MR_ERR_PARAM_INVALID;
    const int64_t groups = numGroups < 0 ? 1 : numGroups;
    if (groups && (!countable(rows, groups, inter, hidden, true, eight) || !countable(rows, groups, hidden, inter, false, false)))
        return MR_ERR_PARAM_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Int8Args a{};
    a.groups = numGroups < 0 ? nullptr : groupList;
    a.G = numGroups < 0 ? 1 : (int)numGroups;
    a.rows = (int)rows;
    a.experts = (int)experts;
    a.expert_base = expertBase;
    if (a.G == 0) return MR_OK;
    char *base = reinterpret_cast<char*>(workspace), *h = base + room.x;
    a.x_scales = xScales;
    a.xs_row = xScaleStride;
    a.w_scales = w13Scales;
    a.N = (int)inter;
    a.y = h;
    a.y_stride = wide_stride(inter) / 2;
    a.y_dtype = MR_DTYPE_BF16;
    const bool pair = use_pairs(rows, a.G, inter, hidden, true);
    Product p{x, xStride, eight ? kInt8 : xDtype == MR_DTYPE_BF16 ? kBf16 : kF16, w13, ar, am, hidden, true, eight};
    const bool scaled = scaled_sums(yDtype, false);
    MR_TRY_CUDA(clear_tickets(room, scaled, true, base, s));
    MR_TRY_CUDA(prepare_rows(p, a, pair, numRows, base, s));
    take_room(a, room, false, base, 0);
    mr_status st = run_product(p, a, pair, s);
    if (st != MR_OK) return st;

    p = Product{h, wide_stride(inter), kBf16, w2, br, bm, inter, false, false};
    a.x_scales = nullptr;
    a.w_scales = w2Scales;
    a.N = (int)hidden;
    a.y = y;
    a.y_stride = yStride;
    a.y_dtype = yDtype;
    take_room(a, room, scaled, base, 1);
    return run_product(p, a, use_pairs(rows, a.G, hidden, inter, false), s);
}

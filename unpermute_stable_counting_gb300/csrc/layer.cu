// A whole mixture-of-experts layer for a few tokens in one launch:
//   logits = x R^T; the top-k experts of each token and their weights;
//   y[t] = sum over its experts e of weight * (silu(x W1e^T) * (x W3e^T)) W2e^T
// with e4m3 weights in blocks (rows quantized as moe_expert_ffn does) or
// 16-bit weights.
//
// With few tokens the time is that of reading the taken experts' weights once,
// so the weights are the wide operand: their rows fill the 128 lanes of the
// tcgen05 instructions, and the tokens are the columns (16 to 64). One
// cooperative grid of a block per SM runs three steps, a grid barrier between:
//   1. logits (a block per few experts and tokens, its warps along k), and the
//      rows of x as the second step's operand
//   2. every block finds all tokens' experts for itself, and takes an equal
//      share of the taken experts' W1/W3 rows, 8 rows at a time: rows of
//      several experts share an instruction, since all of them meet all tokens,
//      and a token keeps the products of its own experts
//   3. every block takes about 100 rows of y and a share of the taken experts'
//      W2 along k (lines of 128 bytes, over all experts); the shares' sums meet
//      in memory after a last barrier
// Equal shares matter more than whole tiles: with 8 experts of 2048 rows on
// 152 SMs, tiles of 128 rows would leave one SM in six idle.
// Copies run through a ring of TMA stages (one thread), instructions are
// issued by one thread, and two warpgroups take the results out of tensor
// memory. The first stages of step 3 are requested before its barrier.
//
// What bounds it: HBM in steps 2 and 3 (one token, 8 experts of 7168 x 2048 in 8
// bits: 235 MB in 39 us and 117 MB in 25 us with their starts and ends), and around
// them about 12 us of latency: the launch, the logits, three to four barriers of 1.3 us, and
// the choice, whose instructions come from L2. 76 us, 0.68 of the time that the copy
// rate gives the bytes; 64 tokens, 64 experts of 7168 x 1024 in 16 bits: 459 to 469 us
// (from GPU to GPU), 0.88 to 0.90. 8-bit weights with more tokens, 64 experts of 7168 x
// 2048: 8 tokens 344 us (0.79 of what their 42 experts' bytes take), 32 tokens 490 us
// (0.85), 64 tokens 528 us (0.79; the kernel for 33 to 64 tokens spills 48 bytes a thread).
#include "tensor.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

namespace mr {

namespace cg = cooperative_groups;

namespace {

__device__ unsigned g_waits_out;

constexpr int kThreads = 384, kWarps = kThreads / 32;
constexpr int kMaxTokens = MR_MAX_LAYER_TOKENS, kMaxExperts = MR_MAX_LAYER_EXPERTS;
constexpr int kLine = 128;            // bytes of a row per stage (the swizzle's width)
constexpr int kMaxStages = 24, kMaxSplits = 8;
constexpr int kBufs = 4, kBufCols = 128;  // tensor memory
constexpr float kLowScores = 7.8886091e-31f;  // 2^-100: sums of scores below it are taken anew
constexpr float kLowUp = 2048.0f;     // f16 weights: what the low parts of h are multiplied by
static_assert(kMaxTokens == 64, "a token set is a 64-bit mask");

struct LayerArgs {
    const void* x;
    int64_t x_stride;
    const void* router;
    int64_t router_stride;
    int x_dt, router_dt, vec_logits;
    const float* bias;
    int T, H, I, E, K;
    int sigmoid, keep;                // flags
    float scale;
    const float* s13;                 // [E][2][ceil(I/128)][ceil(H/128)]
    const float* s2;                  // [E][ceil(H/128)][ceil(I/128)]
    uint32_t bf16;                    // 16-bit weights: bf16 (1) or f16 (0)
    void* y;
    int64_t y_stride;
    int32_t* ids;
    float* weights;
    // workspace
    float* logits;                    // [T][E]
    uint8_t* xs;                      // staged rows, xs_stride bytes apart
    int64_t xs_stride;
    float* sx;                        // [ceil(H/128)][64]
    float* hf;                        // fp32 h, [slot][h_cols] (8-bit weights)
    uint8_t* hs;                      // staged h, hs_stride bytes apart; 16-bit: high parts, then low parts
    int64_t hs_stride;
    int h_cols, slots;                // slots: rows of a part
    float* sh;                        // [ceil(I/128)][slots]
    unsigned* count;                  // [E][ceil(I/128)] row groups of h done
    int rows2, splits;                // step 3: rows of y per block, blocks that share them
    float* part;                      // [splits][T][H] their sums
    int n1, stages1, stage1, stage2_a, ring_bytes;  // columns and stages of step 2, bytes
    int off_sx, off_acc, off_ring;    // dynamic shared memory, from its 1024-byte boundary
};

// Tables of the tokens' experts, at the start of dynamic shared memory.
struct Tables {
    unsigned long long mask[kMaxExperts];  // tokens that take the expert
    uint16_t start[kMaxExperts];           // its first slot: slots are sorted by expert, then token
    uint16_t active[kMaxTokens * MR_MAX_LAYER_TOPK];
    float weight[kMaxTokens * MR_MAX_LAYER_TOPK];  // by slot
    uint8_t token[kMaxTokens * MR_MAX_LAYER_TOPK];
};

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Step 1
// ---------------------------------------------------------------------------
__device__ __forceinline__ void widen8(uint4 w, int dt, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t lo = (uint16_t)(u[j] & 0xFFFFu), hi = (uint16_t)(u[j] >> 16);
        v[2 * j] = dt == MR_DTYPE_F16 ? Elem<MR_DTYPE_F16>::to_f32(lo) : Elem<MR_DTYPE_BF16>::to_f32(lo);
        v[2 * j + 1] = dt == MR_DTYPE_F16 ? Elem<MR_DTYPE_F16>::to_f32(hi) : Elem<MR_DTYPE_BF16>::to_f32(hi);
    }
}

// Logits of EB experts x TB tokens per block; its threads along k.
template <int EB, int TB>
__device__ __forceinline__ void logits_step(const LayerArgs& a, float (*part)[32]) {
    const int nt = (a.T + TB - 1) / TB, tasks = (a.E + EB - 1) / EB * nt;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int e0 = task / nt * EB, t0 = task % nt * TB;
        float acc[EB][TB] = {};
        // past the last expert or token: the last one again, not stored
        if (a.vec_logits) {
            // rows as 16-byte pieces, the next pieces requested before these are used
            const uint16_t* wp[EB];
            const uint16_t* xp[TB];
#pragma unroll
            for (int i = 0; i < EB; ++i)
                wp[i] = reinterpret_cast<const uint16_t*>(a.router) + min(e0 + i, a.E - 1) * a.router_stride;
#pragma unroll
            for (int j = 0; j < TB; ++j)
                xp[j] = reinterpret_cast<const uint16_t*>(a.x) + min(t0 + j, a.T - 1) * a.x_stride;
            uint4 wn[EB], xn[TB];
            int k = threadIdx.x * 8;
            auto fetch = [&](int at) {
                at = min(at, a.H - 8);
#pragma unroll
                for (int i = 0; i < EB; ++i) wn[i] = *reinterpret_cast<const uint4*>(wp[i] + at);
#pragma unroll
                for (int j = 0; j < TB; ++j) xn[j] = *reinterpret_cast<const uint4*>(xp[j] + at);
            };
            fetch(k);
            while (k < a.H) {
                float w[EB][8], x[TB][8];
#pragma unroll
                for (int i = 0; i < EB; ++i) widen8(wn[i], a.router_dt, w[i]);
#pragma unroll
                for (int j = 0; j < TB; ++j) widen8(xn[j], a.x_dt, x[j]);
                k += kThreads * 8;
                fetch(k);
#pragma unroll
                for (int i = 0; i < EB; ++i)
#pragma unroll
                    for (int j = 0; j < TB; ++j)
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc[i][j] = fmaf(w[i][q], x[j][q], acc[i][j]);
            }
        } else {
            for (int k = threadIdx.x; k < a.H; k += kThreads) {
                float w[EB];
#pragma unroll
                for (int i = 0; i < EB; ++i)
                    w[i] = load_f32(a.router, min(e0 + i, a.E - 1) * a.router_stride + k, a.router_dt);
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    const float x = load_f32(a.x, min(t0 + j, a.T - 1) * a.x_stride + k, a.x_dt);
#pragma unroll
                    for (int i = 0; i < EB; ++i) acc[i][j] = fmaf(w[i], x, acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < EB; ++i)
#pragma unroll
            for (int j = 0; j < TB; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
                if (lane == 0) part[warp][i * TB + j] = acc[i][j];
            }
        __syncthreads();
        if (threadIdx.x < EB * TB) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
            const int e = e0 + threadIdx.x / TB, t = t0 + threadIdx.x % TB;
            if (e < a.E && t < a.T) a.logits[t * a.E + e] = s;
        }
        __syncthreads();
    }
}

// Rows of x as the tensor operand: e4m3 blocks with scales, or the same 16 bits.
template <bool EIGHT>
__device__ __forceinline__ void stage_rows(const LayerArgs& a) {
    const int lane = threadIdx.x & 31;
    const int kb = (a.H + kScaleBlock - 1) / kScaleBlock;
    // blocks from the last one down: the first ones have logits to do
    for (int i = (gridDim.x - 1 - blockIdx.x) * kWarps + (threadIdx.x >> 5); i < a.T * kb; i += gridDim.x * kWarps) {
        const int t = i / kb, b = i - t * kb, c = b * kScaleBlock + lane * 4;
        if (EIGHT) {
            float v[4];
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = c + j < a.H ? load_f32(a.x, t * a.x_stride + c + j, a.x_dt) : 0.0f;
                m = max(m, abs_bits(v[j]));
            }
            m = __reduce_max_sync(0xffffffffu, m);
            float s, inv;
            block_scale(m, &s, &inv);
            if (lane == 0) a.sx[b * kMaxTokens + t] = s;
            *reinterpret_cast<uint32_t*>(a.xs + t * a.xs_stride + c) =
                e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        } else {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(a.x) + t * a.x_stride;
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.xs + t * a.xs_stride);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.H) dst[c + j] = src[c + j];
        }
    }
}

// ---------------------------------------------------------------------------
// Step 2: the tokens' experts
// ---------------------------------------------------------------------------
// Bits that order as the values do; NaN below everything.
__device__ __forceinline__ uint32_t order_bits(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The choice, in the ring's memory while it is free: a warp's logits as keys,
// and what was chosen, by token.
struct Choice {
    uint32_t key[kWarps][kMaxExperts];
    float weight[kMaxTokens][MR_MAX_LAYER_TOPK];
    uint16_t expert[kMaxTokens][MR_MAX_LAYER_TOPK];
};

// One token by a warp: the K experts of highest logit (or score + bias), ties to
// the lowest index. Rolled loops throughout: this runs once per launch, with the
// instructions not yet in the SM's cache, and takes the time of fetching them (3 us
// of the 5 us that an unrolled form with the logits in registers took).
__device__ __forceinline__ void choose(const LayerArgs& a, Choice& c, int t, bool write) {
    const int lane = threadIdx.x & 31;
    uint32_t* key = c.key[threadIdx.x >> 5];
    const float* logits = a.logits + t * a.E;
    float top = -INFINITY, sum = 1.0f;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, __ldcg(logits + e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        sum = 0.0f;
    }
    // softmax: exp(l - top) / sum; sigmoid: 1 / (1 + exp(-l))
    const float sign = a.sigmoid ? -1.0f : 1.0f, shift = a.sigmoid ? 0.0f : top;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
        const float l = __ldcg(logits + e);
        if (!a.sigmoid) sum += expf(l - shift);
        key[e] = __float_as_uint(l);
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    auto score = [&](float l) {
        const float x = expf(sign * (l - shift));
        return a.sigmoid ? 1.0f / (1.0f + x) : x / sum;
    };
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
        float v = __uint_as_float(key[e]);
        if (a.bias) v = score(v) + a.bias[e];
        key[e] = max(order_bits(v), 1u);  // 0: taken
    }
    int mine = 0;  // lane r: the r-th expert
#pragma unroll 1
    for (int r = 0; r < a.K; ++r) {
        uint32_t best = 0u, at = 0u;
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32)
            if (key[e] > best) best = key[e], at = e;
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const int e = (int)__reduce_min_sync(0xffffffffu, best == most ? at : 0xffffffffu);
        if ((e & 31) == lane) key[e] = 0u;
        if (lane == r) mine = e;
    }
    const float l = lane < a.K ? __ldcg(logits + mine) : -INFINITY;
    float s = lane < a.K ? score(l) : 0.0f, total = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (!a.keep && total < kLowScores) {
        // (chosen by a bias, or all of a token's sigmoids) fp32 loses digits of such scores, or all of
        // them: their ratios, those of exp(l) for a softmax and for sigmoids this small, are taken
        // with the largest one's exponent off
        float high = l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
        total = s = lane < a.K ? expf(l - high) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane < a.K) {
        const float w = (a.keep ? s : s / total) * a.scale;
        c.expert[t][lane] = (uint16_t)mine;
        c.weight[t][lane] = w;
        if (write) {
            a.ids[t * a.K + lane] = mine;
            a.weights[t * a.K + lane] = w;
        }
    }
}

__device__ __forceinline__ int rank_of(unsigned long long mask, int t) {
    return __popcll(mask & ((1ull << t) - 1ull));
}

// Fills the tables; returns the number of experts taken, *most the largest number of tokens of one.
// shared: the experts were chosen by other blocks and are in a.ids and a.weights.
__device__ __forceinline__ int make_tables(const LayerArgs& a, Tables& tb, Choice& c, bool shared,
                                           uint32_t* warp_sums, int* most_smem, int* most) {
    const int lane = threadIdx.x & 31;
    // pair i: token i / 16, its choice i % 16
    constexpr int kMine = (kMaxTokens * MR_MAX_LAYER_TOPK + kThreads - 1) / kThreads;
    static_assert(MR_MAX_LAYER_TOPK == 16, "pairs are numbered by shifts");
    if (shared) {
        int ex[kMine];
        float w[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int i = threadIdx.x + j * kThreads, at = min((i >> 4) * a.K + min(i & 15, a.K - 1), a.T * a.K - 1);
            ex[j] = __ldcg(a.ids + at);
            w[j] = __ldcg(a.weights + at);
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int i = threadIdx.x + j * kThreads;
            if ((i >> 4) < a.T && (i & 15) < a.K && !MR_IN_RANGE(ex[j], a.E, 951)) ex[j] = 0;
            if (i < kMaxTokens * 16) c.expert[i >> 4][i & 15] = (uint16_t)ex[j], c.weight[i >> 4][i & 15] = w[j];
        }
    }
    for (int e = threadIdx.x; e < a.E; e += kThreads) tb.mask[e] = 0ull;
    if (threadIdx.x == 0) *most_smem = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads)
        if ((i & 15) < a.K) atomicOr(&tb.mask[c.expert[i >> 4][i & 15]], 1ull << (i >> 4));
    __syncthreads();
    // experts of this thread: their slots, and their places among the taken ones
    constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * kPer, e1 = min(e0 + kPer, a.E);
    uint32_t sum = 0u;  // experts taken << 16 | slots
    int biggest = 0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        const int n = __popcll(tb.mask[e]);
        sum += (n ? 0x10000u : 0u) + n;
        biggest = max(biggest, n);
    }
    biggest = (int)__reduce_max_sync(0xffffffffu, (unsigned)biggest);
    if (lane == 0 && biggest) atomicMax(most_smem, biggest);
    uint32_t all = 0u;
    uint32_t before = block_exclusive_scan(sum, warp_sums, &all);
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        const int n = __popcll(tb.mask[e]);
        tb.start[e] = (uint16_t)(before & 0xFFFFu);
        if (n && MR_IN_RANGE(before >> 16, a.T * a.K, 952)) tb.active[before >> 16] = (uint16_t)e;
        before += (n ? 0x10000u : 0u) + n;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
        const int t = i >> 4, r = i & 15;
        if (r >= a.K) continue;
        const int e = c.expert[t][r], slot = tb.start[e] + rank_of(tb.mask[e], t);
        if (!MR_IN_RANGE(slot, a.T * a.K, 953)) continue;
        tb.weight[slot] = c.weight[t][r];
        tb.token[slot] = (uint8_t)t;
    }
    *most = *most_smem;
    return (int)(all >> 16);
}

// ---------------------------------------------------------------------------
// Barriers of the ring and of tensor memory
// ---------------------------------------------------------------------------
struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages], t_full[kBufs], t_empty[kBufs];
};
__device__ __forceinline__ void init_bars(Bars& b) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(smem_u32(&b.full[i]), 1), mbar_init(smem_u32(&b.empty[i]), 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(smem_u32(&b.t_full[i]), 1), mbar_init(smem_u32(&b.t_empty[i]), 8);
}

// ---------------------------------------------------------------------------
// Step 2: h. Row groups of 8 (of one expert) [g0, g1) of all taken experts.
// ---------------------------------------------------------------------------
// A place in a ring of n stages, and the parity of its current round.
struct Place {
    uint32_t at = 0, round = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++at == n) at = 0, round ^= 1;
    }
};

template <bool EIGHT, int COLS>
__device__ __forceinline__ void step_h(const LayerArgs& a, const Tables& tb, const CUtensorMap* map_x, const CUtensorMap* map_w8,
                       const CUtensorMap* map_w64, uint8_t* ring, const float* sx, Bars& bars, uint32_t tmem,
                       volatile uint32_t* abort, uint32_t* flag, int g0, int g1) {
    constexpr int kLineElems = EIGHT ? kLine : kLine / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (a.I + 7) / 8;  // row groups of an expert
    const int kbs = (a.H + kLineElems - 1) / kLineElems;
    // tiles of at most 16 groups, all alike: 17 groups as 16 and 1 would take the short one's steps,
    // bound by their latency, on top
    const int tiles = (g1 - g0 + 15) / 16;
    auto tile_end = [&](int n) { return g0 + (n + 1) * (g1 - g0) / tiles; };
    const int x_bytes = 2 * COLS * kLine;
    if (warp == 0) {
        if (elect_one()) {
            proxy_fence();
            const uint64_t policy = evict_first();
            Place p;
            for (int n = 0, f = g0; n < tiles; ++n) {
                const int l = tile_end(n);
                for (int kb = 0; kb < kbs; ++kb, p.next(a.stages1)) {
                    const uint32_t bar = smem_u32(&bars.full[p.at]);
                    if (!mbar_wait(smem_u32(&bars.empty[p.at]), p.round ^ 1, abort)) break;
                    const uint32_t dst = smem_u32(ring) + p.at * a.stage1;
                    mbar_expect(bar, (l - f) * 2048 + x_bytes);
                    for (int g = f; g < l;) {
                        const int j = g / per, r = g - j * per;
                        const int run = min(l - g, per - r);
                        const int plane = tb.active[j] * 2;
                        int done = 0;
                        for (; done + 8 <= run; done += 8) {
                            const uint32_t to = dst + (g - f + done) * 1024;
                            tma_load_3d_hint(to, map_w64, bar, kb * kLineElems, (r + done) * 8, plane, policy);
                            tma_load_3d_hint(to + 16384, map_w64, bar, kb * kLineElems, (r + done) * 8, plane + 1, policy);
                        }
                        for (; done < run; ++done) {
                            const uint32_t to = dst + (g - f + done) * 1024;
                            tma_load_3d_hint(to, map_w8, bar, kb * kLineElems, (r + done) * 8, plane, policy);
                            tma_load_3d_hint(to + 16384, map_w8, bar, kb * kLineElems, (r + done) * 8, plane + 1, policy);
                        }
                        g += run;
                    }
                    tma_load_2d(dst + 32768, map_x, bar, kb * kLineElems, 0);
                }
                f = l;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            Place p;
            uint32_t use = 0;  // tensor memory buffers used
            for (int n = 0; n < tiles; ++n) {
                for (int kb = 0; kb < kbs; ++kb, p.next(a.stages1)) {
                    const uint32_t buf = use % kBufs;
                    if (EIGHT || kb == 0) mbar_wait(smem_u32(&bars.t_empty[buf]), ((use / kBufs) & 1) ^ 1, abort);
                    if (!mbar_wait(smem_u32(&bars.full[p.at]), p.round, abort)) break;
                    tc_fence_after();
                    const uint32_t at = smem_u32(ring) + p.at * a.stage1;
                    const uint64_t dg = smem_desc(at), du = smem_desc(at + 16384), dx = smem_desc(at + 32768);
                    const uint32_t d = tmem + buf * kBufCols;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t add = EIGHT ? k > 0 : k > 0 || kb > 0;
                        if (EIGHT) {
                            mma_e4m3(d, dg + 2 * k, dx + 2 * k, idesc_e4m3(128, 2 * COLS), add);
                            mma_e4m3(d + 64, du + 2 * k, dx + 2 * k, idesc_e4m3(128, 2 * COLS), add);
                        } else {
                            mma_16(d, dg + 2 * k, dx + 2 * k, idesc_16(128, 2 * COLS, a.bf16), add);
                            mma_16(d + 64, du + 2 * k, dx + 2 * k, idesc_16(128, 2 * COLS, a.bf16), add);
                        }
                    }
                    tc_commit(smem_u32(&bars.empty[p.at]));
                    if (EIGHT || kb == kbs - 1) {
                        tc_commit(smem_u32(&bars.t_full[buf]));
                        ++use;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21) + half * COLS;
        const int hb = (a.H + kScaleBlock - 1) / kScaleBlock, ib = (a.I + kScaleBlock - 1) / kScaleBlock;
        uint32_t use = 0;
        for (int n = 0, f = g0; n < tiles; ++n) {
            const int l = tile_end(n);
            const int g = min(f + row / 8, l - 1);
            const int e = tb.active[g / per], i = g % per * 8 + (row & 7);
            const bool real = f + row / 8 < l && i < a.I;
            float hg[COLS], hu[COLS];
            if (EIGHT) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) hg[c] = hu[c] = 0.0f;
                const float* wg = a.s13 + ((int64_t)(2 * e) * ib + min(i, a.I - 1) / kScaleBlock) * hb;
                const float* wu = wg + (int64_t)ib * hb;
                float ng = wg[0], nu = wu[0];
                for (int kb = 0; kb < kbs; ++kb, ++use) {
                    const uint32_t buf = use % kBufs;
                    const float sg = ng, su = nu;
                    if (kb + 1 < kbs) ng = wg[kb + 1], nu = wu[kb + 1];
                    mbar_wait(smem_u32(&bars.t_full[buf]), (use / kBufs) & 1, abort);
                    tc_fence_after();
                    uint32_t vg[COLS], vu[COLS];
                    tmem_load(vg, from + buf * kBufCols);
                    tmem_load(vu, from + buf * kBufCols + 64);
                    tmem_ld_wait(vg);
                    tmem_ld_wait(vu);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[buf]));
                    const float4* s4 = reinterpret_cast<const float4*>(sx + kb * 2 * COLS + half * COLS);
#pragma unroll
                    for (int c = 0; c < COLS / 4; ++c) {
                        const float4 s = s4[c];
                        const float t[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            hg[4 * c + q] = fmaf(__uint_as_float(vg[4 * c + q]), sg * t[q], hg[4 * c + q]);
                            hu[4 * c + q] = fmaf(__uint_as_float(vu[4 * c + q]), su * t[q], hu[4 * c + q]);
                        }
                    }
                }
            } else {
                const uint32_t buf = use % kBufs;
                mbar_wait(smem_u32(&bars.t_full[buf]), (use / kBufs) & 1, abort);
                tc_fence_after();
                uint32_t vg[COLS], vu[COLS];
                tmem_load(vg, from + buf * kBufCols);
                tmem_load(vu, from + buf * kBufCols + 64);
                tmem_ld_wait(vg);
                tmem_ld_wait(vu);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[buf]));
                ++use;
#pragma unroll
                for (int c = 0; c < COLS; ++c) hg[c] = __uint_as_float(vg[c]), hu[c] = __uint_as_float(vu[c]);
            }
            // h of the tokens that take this row's expert
            const unsigned long long mask = real ? tb.mask[e] : 0ull;
            const int start = tb.start[e];
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const int t = half * COLS + c;
                if (t >= a.T || !((mask >> t) & 1ull)) continue;
                const int slot = start + rank_of(mask, t);
                if (!MR_IN_RANGE(slot, a.T * a.K, 950)) continue;
                const float h = silu(hg[c]) * hu[c];
                if (EIGHT) {
                    a.hf[(int64_t)slot * a.h_cols + i] = h;
                } else {
                    // the value in two 16-bit parts: 16 bits of it (bf16), 22 (f16; 16 down to 2^-20, and
                    // below that all but 2^-36)
                    uint16_t* p = reinterpret_cast<uint16_t*>(a.hs + (int64_t)slot * a.hs_stride) + i;
                    uint16_t* q = reinterpret_cast<uint16_t*>(a.hs + (int64_t)(a.slots + slot) * a.hs_stride) + i;
                    if (a.bf16) {
                        // the highest finite values round to an infinity: the high part is then the
                        // largest bf16 value, and what is above it the low part; an infinite h has none
                        uint16_t hi = Elem<MR_DTYPE_BF16>::from_f32(h);
                        const bool inf = abs_bits(h) == 0x7F800000u;
                        if ((hi & 0x7FFFu) == 0x7F80u && !inf) --hi;
                        *p = hi;
                        *q = inf ? 0 : Elem<MR_DTYPE_BF16>::from_f32(h - Elem<MR_DTYPE_BF16>::to_f32(hi));
                    } else {
                        const uint16_t hi = Elem<MR_DTYPE_F16>::from_f32(h);
                        *p = hi;
                        // past f16's range the high part is an infinity, and the whole value; the low part
                        // is held times 2^11, which keeps it out of f16's subnormal numbers
                        *q = (hi & 0x7FFFu) == 0x7C00u
                                 ? 0
                                 : Elem<MR_DTYPE_F16>::from_f32((h - Elem<MR_DTYPE_F16>::to_f32(hi)) * kLowUp);
                    }
                }
            }
            if (EIGHT) {
                // Blocks of 128 columns of h are quantized by whoever completes them.
                __threadfence();
                for (int g = f; g < l;) {
                    const int j = g / per, r = g - j * per, b = r / 16;
                    const int run = min(min(l - g, per - r), (b + 1) * 16 - r);
                    const int ex = tb.active[j], whole = min(16, per - b * 16);
                    named_barrier(1, 256);  // the tile's rows are stored; *flag is free
                    if (threadIdx.x == 128) {
                        *flag = MR_IN_RANGE(ex, a.E, 954) && MR_IN_RANGE(b, ib, 955) &&
                                atomicAdd(&a.count[ex * ib + b], (unsigned)run) + run == (unsigned)whole;
                        __threadfence();
                    }
                    named_barrier(1, 256);
                    if (*flag) {
                        const int tokens = __popcll(tb.mask[ex]), s0 = tb.start[ex];
                        for (int s = warp - 4; s < tokens; s += 8) {
                            if (!MR_IN_RANGE(s0 + s, a.T * a.K, 956)) break;
                            const int64_t at = (int64_t)(s0 + s) * a.h_cols + b * kScaleBlock + lane * 4;
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(a.hf + at));
                            // columns past I hold nothing
                            const int left = a.I - b * kScaleBlock - lane * 4;
                            const float x[4] = {left > 0 ? v.x : 0.0f, left > 1 ? v.y : 0.0f,
                                                left > 2 ? v.z : 0.0f, left > 3 ? v.w : 0.0f};
                            uint32_t m = max(max(abs_bits(x[0]), abs_bits(x[1])), max(abs_bits(x[2]), abs_bits(x[3])));
                            m = __reduce_max_sync(0xffffffffu, m);
                            float sc, inv;
                            block_scale(m, &sc, &inv);
                            *reinterpret_cast<uint32_t*>(a.hs + (int64_t)(s0 + s) * a.hs_stride + b * kScaleBlock +
                                                         lane * 4) =
                                e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                            if (lane == 0) a.sh[b * a.slots + s0 + s] = sc;
                        }
                    }
                    g += run;
                }
            }
            f = l;
        }
        proxy_fence();  // h is read by copies of the async proxy
    }
}

// ---------------------------------------------------------------------------
// Step 3: y. Rows [row0, row0 + rows2) of the taken experts' W2, lines [u0, u1)
// of k, counted over all of them. The second product's columns are an expert's
// slots; COLS of them per warpgroup, and (8-bit weights) 32 / COLS lines per
// tensor memory buffer.
// ---------------------------------------------------------------------------
template <bool EIGHT, int COLS>
__device__ __forceinline__ void step_y(const LayerArgs& a, const Tables& tb, const CUtensorMap* map_w2, const CUtensorMap* map_h,
                       uint8_t* ring, float* acc, Bars& bars, uint32_t tmem, volatile uint32_t* abort, int experts,
                       int row0, int split, cg::grid_group& grid) {
    constexpr int kLineElems = EIGHT ? kLine : kLine / 2;
    constexpr int kUnits = EIGHT ? 32 / COLS : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kbs = (a.I + kLineElems - 1) / kLineElems;
    const int stage = a.stage2_a + 2 * COLS * kLine * (EIGHT ? 1 : 2);
    // the instructions read 128 rows from a stage's start on, whatever rows2 is: 16 KB of slack
    const int stages = min(kMaxStages, (a.ring_bytes - 16384) / stage);
    const bool real = row0 < a.H && split < a.splits;
    const int u0 = real ? (int)((int64_t)experts * kbs * split / a.splits) : 0;
    const int u1 = real ? (int)((int64_t)experts * kbs * (split + 1) / a.splits) : 0;
    // experts with lines of this share (few lines: it may have none)
    const int j0 = u0 / kbs, j1 = u1 > u0 ? (u1 + kbs - 1) / kbs : j0;
    auto first_line = [&](int j) { return j == j0 ? u0 - j0 * kbs : 0; };
    auto last_line = [&](int j) { return min(kbs, u1 - j * kbs); };
    const uint32_t a_bytes = a.rows2 * kLine;
    const uint32_t base = smem_u32(ring);
    const uint64_t policy = evict_first();
    auto boxes = [&](int e) { return (__popcll(tb.mask[e]) + 15) / 16; };
    // the expert's weights of a stage, and its bytes of both operands announced
    auto request_w = [&](const Place& p, int e, int nb, int kb) {
        const uint32_t bar = smem_u32(&bars.full[p.at]);
        mbar_expect(bar, a_bytes + nb * 2048 * (EIGHT ? 1 : 2));
        tma_load_3d_hint(base + p.at * stage, map_w2, bar, kb * kLineElems, row0, e, policy);
    };
    auto request_h = [&](const Place& p, int nb, int s0, int kb) {
        const uint32_t dst = base + p.at * stage + a.stage2_a, bar = smem_u32(&bars.full[p.at]);
        for (int b = 0; b < nb; ++b) {
            tma_load_2d(dst + b * 2048, map_h, bar, kb * kLineElems, s0 + 16 * b);
            if (!EIGHT) tma_load_2d(dst + (nb + b) * 2048, map_h, bar, kb * kLineElems, a.slots + s0 + 16 * b);
        }
    };
    const int ahead = min(stages, u1 - u0);
    if (warp == 0) {
        if (elect_one()) {
            Place p;
            for (int j = j0, u = 0; u < ahead; ++j) {
                const int e = tb.active[j], nb = boxes(e), end = last_line(j);
                for (int kb = first_line(j); kb < end && u < ahead; ++kb, ++u, p.next(stages)) request_w(p, e, nb, kb);
            }
        }
        __syncwarp();
    }
    for (int i = threadIdx.x; i < 2 * a.T * a.rows2; i += kThreads) acc[i] = 0.0f;
    grid.sync();
    if (warp == 0) {
        if (elect_one()) {
            proxy_fence();
            Place p;
            for (int j = j0, u = 0; j < j1; ++j) {
                const int e = tb.active[j], nb = boxes(e), s0 = tb.start[e], end = last_line(j);
                for (int kb = first_line(j); kb < end; ++kb, ++u, p.next(stages)) {
                    if (u >= ahead) {
                        if (!mbar_wait(smem_u32(&bars.empty[p.at]), p.round ^ 1, abort)) continue;
                        request_w(p, e, nb, kb);
                    }
                    request_h(p, nb, s0, kb);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            Place p;
            uint32_t use = 0;
            for (int j = j0; j < j1; ++j) {
                const int nb = boxes(tb.active[j]), k0 = first_line(j), end = last_line(j);
                const uint32_t idesc = EIGHT ? idesc_e4m3(128, 16 * nb) : idesc_16(128, 32 * nb, a.bf16);
                for (int kb = k0; kb < end; ++kb, p.next(stages)) {
                    const uint32_t buf = use % kBufs;
                    const int part = (kb - k0) % kUnits;
                    if (EIGHT ? part == 0 : kb == k0)
                        mbar_wait(smem_u32(&bars.t_empty[buf]), ((use / kBufs) & 1) ^ 1, abort);
                    if (!mbar_wait(smem_u32(&bars.full[p.at]), p.round, abort)) break;
                    tc_fence_after();
                    const uint64_t dw = smem_desc(base + p.at * stage), dh = smem_desc(base + p.at * stage + a.stage2_a);
                    const uint32_t d = tmem + buf * kBufCols + (EIGHT ? part * 2 * COLS : 0);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (EIGHT) mma_e4m3(d, dw + 2 * k, dh + 2 * k, idesc, k > 0);
                        else mma_16(d, dw + 2 * k, dh + 2 * k, idesc, k > 0 || kb > k0);
                    }
                    tc_commit(smem_u32(&bars.empty[p.at]));
                    if (kb == end - 1 || (EIGHT && part == kUnits - 1)) {
                        tc_commit(smem_u32(&bars.t_full[buf]));
                        ++use;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21) + half * COLS;
        const int hb = (a.H + kScaleBlock - 1) / kScaleBlock, ib = (a.I + kScaleBlock - 1) / kScaleBlock;
        const int wrow = min(row0 + row, a.H - 1);
        float* mine = acc + half * a.T * a.rows2 + row;  // [token][row]
        uint32_t use = 0;
        for (int j = j0; j < j1; ++j) {
            const int e = tb.active[j], s0 = tb.start[e], tokens = __popcll(tb.mask[e]), end = last_line(j);
            float y[COLS];
            if (EIGHT) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) y[c] = 0.0f;
                const float* w = a.s2 + ((int64_t)e * hb + wrow / kScaleBlock) * ib;
                const int lc = half * COLS + lane % COLS;
                for (int kb = first_line(j); kb < end; kb += kUnits, ++use) {
                    const uint32_t buf = use % kBufs;
                    // lane: the scale of one column and line
                    const int lk = kb + lane / COLS;
                    const float sv = lk < end && lc < tokens ? __ldcg(a.sh + lk * a.slots + s0 + lc) : 0.0f;
                    float sw[kUnits];
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) sw[u] = kb + u < end ? w[kb + u] : 0.0f;
                    mbar_wait(smem_u32(&bars.t_full[buf]), (use / kBufs) & 1, abort);
                    tc_fence_after();
                    uint32_t v[kUnits][COLS];
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) tmem_load(v[u], from + buf * kBufCols + u * 2 * COLS);
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) tmem_ld_wait(v[u]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[buf]));
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        if (kb + u >= end) break;  // lines past the end: whatever the buffer held
#pragma unroll
                        for (int c = 0; c < COLS; ++c)
                            y[c] = fmaf(__uint_as_float(v[u][c]), sw[u] * __shfl_sync(0xffffffffu, sv, u * COLS + c),
                                        y[c]);
                    }
                }
            } else {
                const uint32_t buf = use % kBufs;
                mbar_wait(smem_u32(&bars.t_full[buf]), (use / kBufs) & 1, abort);
                tc_fence_after();
                uint32_t hi[COLS], lo[COLS];
                tmem_load(hi, from + buf * kBufCols);
                tmem_load(lo, from + buf * kBufCols + 16 * boxes(e));
                tmem_ld_wait(hi);
                tmem_ld_wait(lo);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[buf]));
                ++use;
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    y[c] = fmaf(__uint_as_float(lo[c]), a.bf16 ? 1.0f : 1.0f / kLowUp, __uint_as_float(hi[c]));
            }
            if (row < a.rows2) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    if (half * COLS + c >= tokens) break;
                    const int slot = s0 + half * COLS + c;
                    if (!MR_IN_RANGE(slot, a.T * a.K, 957) || !MR_IN_RANGE(tb.token[slot], a.T, 958)) break;
                    float* p = mine + tb.token[slot] * a.rows2;
                    *p = fmaf(tb.weight[slot], y[c], *p);
                }
            }
        }
    }
    __syncthreads();
    auto store = [&](int64_t at, float v) {
        if (a.x_dt == MR_DTYPE_F32) reinterpret_cast<float*>(a.y)[at] = v;
        else if (a.x_dt == MR_DTYPE_F16) reinterpret_cast<uint16_t*>(a.y)[at] = Elem<MR_DTYPE_F16>::from_f32(v);
        else reinterpret_cast<uint16_t*>(a.y)[at] = Elem<MR_DTYPE_BF16>::from_f32(v);
    };
    if (real)
        for (int i = threadIdx.x; i < a.T * a.rows2; i += kThreads) {
            const int t = i / a.rows2, r = row0 + i - t * a.rows2;
            if (r >= a.H) continue;
            const float v = acc[i] + acc[a.T * a.rows2 + i];
            if (a.splits == 1) store(t * a.y_stride + r, v);
            else a.part[((int64_t)split * a.T + t) * a.H + r] = v;
        }
    if (a.splits == 1) return;
    grid.sync();
    const int n = a.T * a.H;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
        float p[kMaxSplits], v = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxSplits; ++k) p[k] = k < a.splits ? __ldcg(a.part + (int64_t)k * n + i) : 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxSplits; ++k) v += p[k];
        const int t = i / a.H;
        store(t * a.y_stride + i - t * a.H, v);
    }
}

struct LayerMaps {
    CUtensorMap x, w8, w64, w2, h;
};

template <bool EIGHT, int COLS>
__global__ void __launch_bounds__(kThreads, 1)
    layer_kernel(const __grid_constant__ LayerMaps maps, const __grid_constant__ LayerArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars1, bars2;
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t tmem_base, abort_word, flag, warp_sums[32];
    __shared__ int most_smem;
    __shared__ float part[kWarps][32];
    cg::grid_group grid = cg::this_grid();
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Tables& tb = *reinterpret_cast<Tables*>(smem);
    float* sx = reinterpret_cast<float*>(smem + a.off_sx);
    float* acc = reinterpret_cast<float*>(smem + a.off_acc);
    uint8_t* ring = smem + a.off_ring;
    volatile uint32_t* abort = &abort_word;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        init_bars(bars1);
        init_bars(bars2);
        mbar_init(smem_u32(&drain_bar), 1);
        abort_word = 0u;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_base), kBufs * kBufCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_enter();

    // 1
    const int ib = (a.I + kScaleBlock - 1) / kScaleBlock, hb = (a.H + kScaleBlock - 1) / kScaleBlock;
    if (EIGHT)
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.E * ib; i += gridDim.x * kThreads) a.count[i] = 0u;
    stage_rows<EIGHT>(a);
    // few pairs: a block per pair; else the fewest rows read that still occupy every block once
    if (a.T * a.E <= 4 * (int)gridDim.x) logits_step<1, 1>(a, part);
    else if ((a.T + 3) / 4 * ((a.E + 3) / 4) <= (int)gridDim.x) logits_step<4, 4>(a, part);
    else logits_step<4, 8>(a, part);
    proxy_fence();
    grid.sync();

    // 2
    // Up to a token per warp every block chooses all tokens' experts for itself, which saves a
    // barrier (1.3 us); more tokens are a block's each (several, if there are fewer blocks than tokens).
    const bool shared_choice = a.T > kWarps;
    const int token = shared_choice ? (warp == 0 ? (int)blockIdx.x : a.T) : warp;
    Choice& choice = *reinterpret_cast<Choice*>(ring);
    for (int t = token; t < a.T; t += shared_choice ? (int)gridDim.x : kWarps)
        choose(a, choice, t, shared_choice || blockIdx.x == 0);
    if (shared_choice) grid.sync();
    else __syncthreads();
    int most = 0;
    if (EIGHT)  // the scales of x, on their way while the experts are chosen
        for (int i = threadIdx.x; i < hb * COLS / 2; i += kThreads) {
            const int b = i / (COLS / 2), t = i % (COLS / 2) * 4;
            copy_16(smem_u32(sx + b * 2 * COLS + t), a.sx + b * kMaxTokens + t);
        }
    const int experts = make_tables(a, tb, choice, shared_choice, warp_sums, &most_smem, &most);
    copy_wait();
    proxy_fence();  // the ring's memory goes to copies of the async proxy
    __syncthreads();
    const int groups = experts * ((a.I + 7) / 8);
    const int g0 = (int)((int64_t)groups * blockIdx.x / gridDim.x);
    const int g1 = (int)((int64_t)groups * (blockIdx.x + 1) / gridDim.x);
    step_h<EIGHT, COLS>(a, tb, &maps.x, &maps.w8, &maps.w64, ring, sx, bars1, tmem, abort, &flag, g0, g1);
    tc_fence_before();
    __syncthreads();  // the ring changes its layout, tensor memory its use
    tc_fence_after();

    // 3
    const int row0 = blockIdx.x / a.splits * a.rows2, split = blockIdx.x % a.splits;
    if (most <= 16)
        step_y<EIGHT, 8>(a, tb, &maps.w2, &maps.h, ring, acc, bars2, tmem, abort, experts, row0, split, grid);
    else if (most <= 32)
        step_y<EIGHT, 16>(a, tb, &maps.w2, &maps.h, ring, acc, bars2, tmem, abort, experts, row0, split, grid);
    else
        step_y<EIGHT, 32>(a, tb, &maps.w2, &maps.h, ring, acc, bars2, tmem, abort, experts, row0, split, grid);

    __syncthreads();
    if (abort_word) {
        // A wait gave up: let the instructions in flight end, and give the copies the time that
        // mbar_drain gives a barrier, before the block's memory goes.
        if (warp == 1) {
            if (elect_one()) tc_commit(smem_u32(&drain_bar));
            mbar_drain(smem_u32(&drain_bar), 0);
        }
        if (threadIdx.x == 0) {
            const uint64_t start = global_ns();
            while (global_ns() - start < 100000000ull) {
            }
            atomicAdd(&g_waits_out, 1u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem, kBufs * kBufCols);
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
bool float_dtype(int32_t dt) { return dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16 || dt == MR_DTYPE_F32; }
bool aligned16(const void* p) { return aligned(p, 16); }

// Workspace regions, 256-byte aligned.
struct LayerPlan {
    int64_t xs_stride, hs_stride, h_cols, slots;
    int rows2, splits;
    uint64_t logits, xs, sx, hf, hs, sh, count, part, bytes;
    LayerPlan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t K, bool eight) {
        const int64_t ib = ceil_div(I, kScaleBlock), hb = ceil_div(H, kScaleBlock);
        slots = ceil_div(T * K, 16) * 16 + 64;  // a box of 16 slots may start at any slot
        h_cols = ib * kScaleBlock;
        xs_stride = eight ? hb * kScaleBlock : (int64_t)align_up(2 * H, 128);
        hs_stride = eight ? h_cols : (int64_t)align_up(2 * I, 128);
        // Step 3: the most shares of k with at most 128 rows per block: a line of W2 then has about 100
        // rows, and the fixed cost of a line (waits, four instructions) stays below its time in HBM. With
        // one share and 48 rows (hidden 7168) step 3 of one token took 39 us, its bytes 17 us.
        const int grid = device_sm_count();
        splits = 1;
        while (splits < kMaxSplits && ceil_div(H, grid / (splits + 1)) <= 128) ++splits;
        rows2 = ceil_div(ceil_div(H, grid / splits), 8) * 8;
        uint64_t at = 0;
        auto take = [&](uint64_t n) {
            const uint64_t p = at;
            at += align_up(n, 256);
            return p;
        };
        logits = take(T * E * 4);
        xs = take(kMaxTokens * xs_stride);
        sx = take(hb * kMaxTokens * 4);
        hf = take(eight ? slots * h_cols * 4 : 0);
        hs = take((eight ? 1 : 2) * slots * hs_stride);
        sh = take(eight ? ib * slots * 4 : 0);
        count = take(eight ? E * ib * 4 : 0);
        part = take(splits > 1 ? splits * T * H * 4 : 0);
        bytes = at;
    }
};

template <bool EIGHT, int COLS>
cudaError_t launch_layer(const LayerMaps& maps, const LayerArgs& a, int smem, int grid, cudaStream_t s) {
    auto kernel = layer_kernel<EIGHT, COLS>;
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      232448 - (int)at.sharedSizeBytes)) != cudaSuccess)
            return e;
        ready[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

bool layer_sizes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t K, int32_t dt) {
    return T >= 0 && T <= MR_MAX_LAYER_TOKENS && H >= 1 && H <= MR_MAX_LAYER_COLS && I >= 1 &&
           I <= MR_MAX_LAYER_COLS && E >= 1 && E <= MR_MAX_LAYER_EXPERTS && K >= 1 && K <= MR_MAX_LAYER_TOPK &&
           K <= E && (dt == MR_DTYPE_E4M3 || dt == MR_DTYPE_F16 || dt == MR_DTYPE_BF16);
}

}  // namespace

MR_CHECK_ACCESSOR(layer)

cudaError_t waits_out_layer(unsigned* out, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_waits_out, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0u;
        e = cudaMemcpyToSymbol(g_waits_out, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace mr

using namespace mr;

extern "C" mr_status moe_layer_get_workspace_size(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts,
                                                  int64_t topK, int32_t weightDtype, uint64_t* workspaceSize) {
    if (!layer_sizes(tokens, hidden, inter, experts, topK, weightDtype)) return MR_ERR_PARAM_INVALID;
    if (!workspaceSize) return MR_ERR_PARAM_NULLPTR;
    *workspaceSize = LayerPlan(tokens, hidden, inter, experts, topK, weightDtype == MR_DTYPE_E4M3).bytes;
    return MR_OK;
}

extern "C" mr_status moe_layer(const void* x, int32_t xDtype, int64_t xStride, const void* router,
                               int32_t routerDtype, int64_t routerStride, const float* selectBias, const void* w13,
                               int32_t weightDtype, const int64_t* w13Strides, const float* w13Scales,
                               const void* w2, const int64_t* w2Strides, const float* w2Scales, int64_t tokens,
                               int64_t hidden, int64_t inter, int64_t experts, int64_t topK, uint32_t flags,
                               float routedScale, void* y, int64_t yStride, int32_t* expertIds, float* expertWeights,
                               void* workspace, uint64_t workspaceSize, void* stream) {
    const bool eight = weightDtype == MR_DTYPE_E4M3;
    if (!layer_sizes(tokens, hidden, inter, experts, topK, weightDtype)) return MR_ERR_PARAM_INVALID;
    if (!float_dtype(xDtype) || !float_dtype(routerDtype) || (!eight && xDtype != weightDtype))
        return MR_ERR_PARAM_INVALID;
    if (flags & ~(MR_LAYER_SIGMOID | MR_LAYER_KEEP_WEIGHTS)) return MR_ERR_PARAM_INVALID;
    const int64_t top = INT64_C(1) << 40;
    if (xStride < hidden || xStride > top || routerStride < hidden || routerStride > top || yStride < hidden ||
        yStride > top)
        return MR_ERR_PARAM_INVALID;
    const int64_t el = eight ? 1 : 2;
    int64_t ar = hidden * el, am = inter * ar, br = inter * el, bm = hidden * br;
    if (w13Strides) ar = w13Strides[0], am = w13Strides[1];
    if (w2Strides) br = w2Strides[0], bm = w2Strides[1];
    ar = stride_of(inter, ar, hidden * el);
    br = stride_of(hidden, br, inter * el);
    bm = stride_of(experts, bm, hidden * br);
    if (ar < hidden * el || ar % 16 || am % 16 || ar > top || am > top || am < (inter - 1) * ar + hidden * el)
        return MR_ERR_PARAM_INVALID;
    if (br < inter * el || br % 16 || bm % 16 || br > top || bm > top ||
        (experts > 1 && bm < (hidden - 1) * br + inter * el))
        return MR_ERR_PARAM_INVALID;
    if (tokens == 0) return MR_OK;
    if (!x || !router || !w13 || !w2 || !y || !expertIds || !expertWeights || !workspace) return MR_ERR_PARAM_NULLPTR;
    if (eight != (w13Scales != nullptr) || eight != (w2Scales != nullptr)) return MR_ERR_PARAM_NULLPTR;
    const LayerPlan p(tokens, hidden, inter, experts, topK, eight);
    if (workspaceSize < p.bytes) return MR_ERR_WORKSPACE;
    if (!aligned16(w13) || !aligned16(w2) || !aligned(workspace, 256)) return MR_ERR_PARAM_INVALID;
    const uintptr_t xe = xDtype == MR_DTYPE_F32 ? 4 : 2, re = routerDtype == MR_DTYPE_F32 ? 4 : 2;
    if (!aligned(x, xe) || !aligned(y, xe) || !aligned(router, re) || !aligned(selectBias, 4) ||
        !aligned(w13Scales, 4) || !aligned(w2Scales, 4) || !aligned(expertIds, 4) || !aligned(expertWeights, 4))
        return MR_ERR_PARAM_INVALID;

    const int grid = device_sm_count();
    LayerArgs a{};
    a.x = x;
    a.x_stride = xStride;
    a.router = router;
    a.router_stride = routerStride;
    a.x_dt = xDtype;
    a.router_dt = routerDtype;
    a.vec_logits = xe == 2 && re == 2 && aligned16(x) && aligned16(router) && xStride % 8 == 0 &&
                   routerStride % 8 == 0 && hidden % 8 == 0;
    a.bias = selectBias;
    a.T = (int)tokens;
    a.H = (int)hidden;
    a.I = (int)inter;
    a.E = (int)experts;
    a.K = (int)topK;
    a.sigmoid = (flags & MR_LAYER_SIGMOID) != 0;
    a.keep = (flags & MR_LAYER_KEEP_WEIGHTS) != 0;
    a.scale = routedScale;
    a.s13 = w13Scales;
    a.s2 = w2Scales;
    a.bf16 = weightDtype == MR_DTYPE_BF16;
    a.y = y;
    a.y_stride = yStride;
    a.ids = expertIds;
    a.weights = expertWeights;
    uint8_t* w = reinterpret_cast<uint8_t*>(workspace);
    a.logits = reinterpret_cast<float*>(w + p.logits);
    a.xs = w + p.xs;
    a.xs_stride = p.xs_stride;
    a.sx = reinterpret_cast<float*>(w + p.sx);
    a.hf = reinterpret_cast<float*>(w + p.hf);
    a.hs = w + p.hs;
    a.hs_stride = p.hs_stride;
    a.h_cols = (int)p.h_cols;
    a.slots = (int)p.slots;
    a.sh = reinterpret_cast<float*>(w + p.sh);
    a.count = reinterpret_cast<unsigned*>(w + p.count);
    a.rows2 = p.rows2;
    a.splits = p.splits;
    a.part = reinterpret_cast<float*>(w + p.part);
    if (a.rows2 > 128) return MR_ERR_UNSUPPORTED;  // a device with fewer SMs
    a.n1 = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;

    // shared memory: tables, scales of x, sums of y, then the ring
    a.off_sx = (int)align_up(sizeof(Tables), 128);
    a.off_acc = a.off_sx + (eight ? ceil_div(hidden, kScaleBlock) * a.n1 * 4 : 0);
    a.off_ring = (int)align_up(a.off_acc + 2 * tokens * a.rows2 * 4, 1024);
    constexpr int kStatic = 4096;  // at least the kernel's static shared memory and alignment
    const int room = 232448 - kStatic;
    a.ring_bytes = (room - a.off_ring) / 1024 * 1024;
    a.stage1 = 32768 + a.n1 * kLine;
    a.stages1 = std::min(kMaxStages, a.ring_bytes / a.stage1);
    a.stage2_a = (int)align_up(a.rows2 * kLine, 1024);
    // the widest stage of step 3: 64 columns, in two parts for 16-bit weights
    const int widest = a.stage2_a + 64 * kLine * (eight ? 1 : 2);
    static_assert(sizeof(Choice) <= 65536, "fits the ring");
    if (a.ring_bytes < 65536 || a.stages1 < 2 || (a.ring_bytes - 16384) / widest < 2) return MR_ERR_UNSUPPORTED;

    LayerMaps m;
    const CUtensorMapDataType type = eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const uint32_t line = (uint32_t)(kLine / el);
    const uint64_t xd[2] = {(uint64_t)hidden, (uint64_t)kMaxTokens}, xst[1] = {(uint64_t)p.xs_stride};
    const uint32_t xb[2] = {line, (uint32_t)a.n1};
    const uint64_t ad[3] = {(uint64_t)hidden, (uint64_t)inter, (uint64_t)experts * 2};
    const uint64_t ast[2] = {(uint64_t)ar, (uint64_t)am};
    const uint32_t a8[3] = {line, 8, 1}, a64[3] = {line, 64, 1};
    const uint64_t bd[3] = {(uint64_t)inter, (uint64_t)hidden, (uint64_t)experts};
    const uint64_t bst[2] = {(uint64_t)br, (uint64_t)bm};
    const uint32_t bb[3] = {line, (uint32_t)a.rows2, 1};
    const uint64_t hd[2] = {(uint64_t)inter, (uint64_t)(p.slots * (eight ? 1 : 2))}, hst[1] = {(uint64_t)p.hs_stride};
    const uint32_t hbx[2] = {line, 16};
    const int eb = (int)el;
    if (!make_tensor_map(&m.x, type, eb, a.xs, 2, xd, xst, xb) || !make_tensor_map(&m.w8, type, eb, w13, 3, ad, ast, a8) ||
        !make_tensor_map(&m.w64, type, eb, w13, 3, ad, ast, a64) ||
        !make_tensor_map(&m.w2, type, eb, w2, 3, bd, bst, bb) || !make_tensor_map(&m.h, type, eb, a.hs, 2, hd, hst, hbx))
        return MR_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int smem = 1024 + a.off_ring + a.ring_bytes;
    cudaError_t e;
    if (eight) {
        e = a.n1 == 16   ? launch_layer<true, 8>(m, a, smem, grid, s)
            : a.n1 == 32 ? launch_layer<true, 16>(m, a, smem, grid, s)
                         : launch_layer<true, 32>(m, a, smem, grid, s);
    } else {
        e = a.n1 == 16   ? launch_layer<false, 8>(m, a, smem, grid, s)
            : a.n1 == 32 ? launch_layer<false, 16>(m, a, smem, grid, s)
                         : launch_layer<false, 32>(m, a, smem, grid, s);
    }
    return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

// The group list of the expert products, and how a kernel's warps walk it.
#pragma once

#include "common.cuh"

namespace mr {

struct Groups {
    const int64_t* groups;     // [G, 2], or NULL: one group of all rows, expert 0
    int G, rows, experts;
    int64_t expert_base;
    int n_tiles;
};

struct Tile {
    int expert, row0, rows, n0;
};

// Walks the group list in tiles of TM rows. Every lane of the warp calls next()
// with the same t, ascending over the calls. EVEN: a group's tiles have as many rows
// each, to a multiple of 16, as its last one allows, so that tiles cost about the same.
template <int TM, bool EVEN = false> struct Walk {
    int first, base_tile, total;      // window of 32 groups; tiles before it, tiles in it
    uint32_t base_row, window_rows;   // rows before it, rows in it
    int expert, count, row0, tiles;   // this lane's group
    int end;                          // inclusive sum of tiles over the window

    __device__ __forceinline__ void load(const Groups& a, int lane) {
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
    static __device__ __forceinline__ int skip(const Groups& a, int lane, int g) {
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
    __device__ __forceinline__ void begin(const Groups& a, int lane) {
        first = base_tile = 0;
        base_row = 0u;
        load(a, lane);
    }
    __device__ __forceinline__ bool next(const Groups& a, int lane, int t, int bn, Tile& out) {
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
        const int rows = EVEN ? ((c + mt - 1) / mt + 15) / 16 * 16 : TM;
        out.row0 = __shfl_sync(0xffffffffu, row0, src) + m * rows;
        out.rows = min(c - m * rows, rows);
        out.n0 = n * bn;
        return true;
    }
};

}  // namespace mr

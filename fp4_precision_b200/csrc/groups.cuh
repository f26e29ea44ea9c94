// groups.cuh - groups of rows (the experts of a mixture) as a CTA sees them.
#pragma once

#include "qfp4_device.cuh"
#include "qfp4_internal.h"

namespace qfp4 {

// row[e]: the first row of group e; padded[e]: its first row in the padded
// layout, where groups start at multiples of 128; tiles[e]: the number of
// tile_rows-row tiles before it.
struct GroupTable {
    int row[kMaxGroups + 1];
    int padded[kMaxGroups + 1];
    int tiles[kMaxGroups + 1];
    __device__ __forceinline__ int size(int e) const { return row[e + 1] - row[e]; }
};

// Built by one warp from the device offsets. All loads are issued before the
// first use (one memory latency for 256 groups). Offsets that fall anywhere or
// leave [0, T] would lead out of the buffers: they raise the device error word
// and make every group empty.
__device__ __forceinline__ void build_groups(GroupTable& g, const int* offsets, int E, int T, int tile_rows, int lane) {
    constexpr int STEPS = kMaxGroups / 32 + 1;
    int o[STEPS + 1];  // o[i]: offset 32 i + lane
#pragma unroll
    for (int i = 0; i <= STEPS; ++i) o[i] = 32 * i + lane <= E ? offsets[32 * i + lane] : 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int e = 32 * i + lane;
        int next = __shfl_down_sync(0xffffffffu, o[i], 1);
        const int first = __shfl_sync(0xffffffffu, o[i + 1], 0);
        if (lane == 31) next = first;
        bad = bad || (e <= E && (o[i] < 0 || o[i] > T)) || (e < E && next < o[i]);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0 && blockIdx.x == 0) raise_device_error(DEV_ERR_OFFSETS);
    int padded = 0, tiles = 0;  // of the groups before this step's 32
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (32 * i > E) break;
        const int e = 32 * i + lane;
        int next = __shfl_down_sync(0xffffffffu, o[i], 1);
        const int first = __shfl_sync(0xffffffffu, o[i + 1], 0);
        if (lane == 31) next = first;
        const int m = e < E && !bad ? next - o[i] : 0;
        const int own_a = (m + 127) / 128, own_b = (m + tile_rows - 1) / tile_rows;
        int a = own_a, b = own_b;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int ua = __shfl_up_sync(0xffffffffu, a, s), ub = __shfl_up_sync(0xffffffffu, b, s);
            if (lane >= s) {
                a += ua;
                b += ub;
            }
        }
        if (e <= E) {
            g.row[e] = bad ? 0 : o[i];
            g.padded[e] = (padded + a - own_a) * 128;
            g.tiles[e] = tiles + b - own_b;
        }
        padded += __shfl_sync(0xffffffffu, a, 31);
        tiles += __shfl_sync(0xffffffffu, b, 31);
    }
}

// The group of position r in the prefix sums first[0 .. E], or -1 past the last.
__device__ __forceinline__ int group_of(const int* first, int E, int r) {
    if (r >= first[E]) return -1;
    int lo = 0, hi = E;  // first[lo] <= r < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace qfp4

// Row tiles of a grouped product, found on the device: the groups' sizes are
// in device memory and the host never reads them.  Internal linkage.
#pragma once

#include <hip/hip_runtime.h>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {
namespace {

struct RowRange {
    int row0, n;
};

// Sorted rows from offset a on, up to offset b.  Both are clamped to 0..n_rows
// (their difference fits 32 bits then, whatever they hold) and taken to not
// decrease, so a bad value reads and writes nothing out of bounds.
__device__ inline RowRange row_range(const GroupedCall& C, int a, int b) {
    RowRange r;
    r.row0 = min(max(a, 0), C.n_rows);
    r.n = max(min(max(b, 0), C.n_rows) - r.row0, 0);
    return r;
}

// Sorted rows of expert e.
__device__ inline RowRange group_rows(const GroupedCall& C, int e) {
    return row_range(C, C.offsets[e], C.offsets[e + 1]);
}

// The same for an expert that the whole wave shares, by scalar loads: these do
// not wait for the vector loads under way.  (Nothing writes the offsets while
// the kernel runs.)
__device__ inline RowRange group_rows_uniform(const GroupedCall& C, int e) {
    typedef const __attribute__((address_space(4))) int32_t* Constant;
    const Constant o = (Constant)(reinterpret_cast<uintptr_t>(C.offsets));
    return row_range(C, o[e], o[e + 1]);
}

// The number of row tiles of mt rows, no more than offsets that do not
// decrease can give, so that others end as soon.
__device__ inline int most_tiles(const GroupedCall& C, int mt, int total) {
    return min(max(total, 0), min(C.n_experts, C.n_rows) + C.n_rows / mt);
}

// The use of sorted row i (-1: left out).
__device__ inline int use_of(const GroupedCall& C, int i) {
    if (!C.order) return i;
    const int u = C.order[i];
    return u >= 0 && u < C.n_rows ? u : -1;
}

__device__ inline float silu_up(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Four adjacent outputs of row y + at, those below `left`.  Rows of y need no
// alignment beyond their element's: the hardware splits the stores that cross a
// line.
template <int YT>
__device__ inline void store4(void* y, int64_t at, int left, const float* v) {
    constexpr int B = YT == PM_F32 ? 4 : 2;
    if (left >= 4) {
        alignas(16) char o[4 * B];
#pragma unroll
        for (int r = 0; r < 4; ++r) store_f32<YT>(o, r, v[r]);
        __builtin_memcpy(static_cast<char*>(y) + at * B, o, 4 * B);
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (r < left) store_f32<YT>(y, at + r, v[r]);
}

// before[e] = row tiles of mt rows of the experts below e, e <= n_experts;
// returns their number, in every thread.  For all threads of the workgroup;
// the table may be read after a barrier.  Threads: a multiple of 64, 1024 at
// most.
__device__ inline int tile_table(const GroupedCall& C, int mt, int* before) {
    __shared__ int wave_tiles[16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int per = (C.n_experts + blockDim.x - 1) / blockDim.x;
    const int e0 = min(int(threadIdx.x) * per, C.n_experts), e1 = min(e0 + per, C.n_experts);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += (group_rows(C, e).n + mt - 1) / mt;
    int s = mine;
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    if (lane == 63) wave_tiles[wv] = s;
    __syncthreads();
    int at = s - mine, total = 0;
    for (int w = 0; w < waves; ++w) {
        if (w < wv) at += wave_tiles[w];
        total += wave_tiles[w];
    }
    for (int e = e0; e < e1; ++e) {
        before[e] = at;
        at += (group_rows(C, e).n + mt - 1) / mt;
    }
    if (threadIdx.x == 0) before[C.n_experts] = total;
    return uni(most_tiles(C, mt, total));
}

// The expert of row tile i < total: the last e with before[e] <= i.  Two
// rounds of 64 comparisons; every lane gets the result.
__device__ inline int tile_expert(const GroupedCall& C, const int* before, int i) {
    const int lane = threadIdx.x & 63;
    const int step = (C.n_experts + kWave - 1) / kWave;       // <= 64
    const int e = lane * step;
    const int lo = max(__popcll(__ballot(e < C.n_experts && before[e] <= i)) - 1, 0) * step;
    const int f = lo + lane;
    const int k = __popcll(__ballot(lane < step && f < C.n_experts && before[f] <= i)) - 1;
    return uni(lo + max(k, 0));
}

}  // namespace
}  // namespace pm

// Products grouped by expert.  The groups' sizes are on the device, so a
// workgroup finds its own tile: tile i counts the row tiles of the experts
// in order (find_tile).
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

namespace {

// Rows [row0, row0 + n) of the sorted order belong to expert e; e < 0: no
// such tile.
struct Tile {
    int e, row0, n;
};

// Row tile `i` of the call, tiles of `mt` rows.  Offsets are clamped to
// 0..n_rows and taken to not decrease, so a bad value reads and writes
// nothing out of bounds.  Every lane of the wave gets the result.
__device__ inline Tile find_tile(const GroupedCall& C, int mt, int i) {
    const int lane = threadIdx.x & 63;
    int seen = 0;
    for (int base = 0; base < C.n_experts; base += kWave) {
        const int e = base + lane;
        int a = 0, n = 0;
        if (e < C.n_experts) {
            a = min(max(C.offsets[e], 0), C.n_rows);
            n = max(min(C.offsets[e + 1], C.n_rows) - a, 0);
        }
        const int tiles = (n + mt - 1) / mt;
        int s = tiles;
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        const int before = seen + s - tiles;
        const uint64_t hit = __ballot(i >= before && i < before + tiles);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int k = i - __shfl(before, l);
            Tile t;
            t.e = base + l;
            t.row0 = __shfl(a, l) + k * mt;
            t.n = min(__shfl(n, l) - k * mt, mt);
            return t;
        }
        seen += __shfl(s, 63);
    }
    return Tile{-1, 0, 0};
}

template <int KIND, int WT>
__device__ inline float weight(const GroupedCall& C, int e, int o, int c) {
    const size_t row = size_t(e) * C.rows + o;
    if constexpr (KIND == kW16) return load_f32<WT>(C.w, row * C.cols + c);
    const uint8_t b = static_cast<const uint8_t*>(C.w)[(row * C.cols + c) / 2];
    const size_t g = row * (C.cols / C.group) + c / C.group;
    const int z = C.zeros ? C.zeros[g] : 8;
    return float(int(c & 1 ? b >> 4 : b & 15) - z) * load_f32<PM_F16>(C.scales, g);
}

// 16 rows x 16 outputs (x 2 with gate and up) per workgroup, one output per
// thread, 32 inputs at a time through LDS.
template <int KIND, int WT, int XT, int YT>
__global__ __launch_bounds__(256) void grouped_simple_kernel(const GroupedCall C) {
    __shared__ float xs[16][33], ws[2][16][33];
    const bool glu = C.flags & PM_GROUPED_SWIGLU;
    const int out = glu ? C.rows / 2 : C.rows;
    const Tile t = find_tile(C, 16, blockIdx.x);
    if (t.e < 0) return;
    const int o0 = blockIdx.y * 16;
    const int r = threadIdx.x / 16, c = threadIdx.x % 16;
    const int u = r < t.n ? use_of(C, t.row0 + r) : -1;
    const int64_t xr = C.flags & PM_GROUPED_GATHER ? u / C.top_k : t.row0 + r;
    float p0 = 0.0f, p1 = 0.0f;
    for (int k0 = 0; k0 < C.cols; k0 += 32) {
        __syncthreads();
        for (int h = 0; h < 2; ++h) {
            const int k = c + 16 * h;
            const bool in = k0 + k < C.cols;
            xs[r][k] = in && u >= 0 ? load_f32<XT>(C.x, xr * C.ldx + k0 + k) : 0.0f;
            const bool wr = in && o0 + r < out;
            ws[0][r][k] = wr ? weight<KIND, WT>(C, t.e, o0 + r, k0 + k) : 0.0f;
            if (glu) ws[1][r][k] = wr ? weight<KIND, WT>(C, t.e, out + o0 + r, k0 + k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < 32; ++k) {
            p0 = fmaf(xs[r][k], ws[0][c][k], p0);
            if (glu) p1 = fmaf(xs[r][k], ws[1][c][k], p1);
        }
    }
    if (u < 0 || o0 + c >= out) return;
    const int64_t yr = C.flags & PM_GROUPED_SCATTER ? u : t.row0 + r;
    store_f32<YT>(C.y, yr * C.ldy + o0 + c, glu ? silu_up(p0, p1) : p0);
}

template <int KIND, int WT, int XT, int YT>
hipError_t run_simple(const GroupedCall& C, hipStream_t st) {
    const int out = C.flags & PM_GROUPED_SWIGLU ? C.rows / 2 : C.rows;
    const unsigned tiles = unsigned(std::min(C.n_rows, C.n_experts) + C.n_rows / 16);
    hipLaunchKernelGGL((grouped_simple_kernel<KIND, WT, XT, YT>),
                       dim3(tiles, unsigned((out + 15) / 16)), dim3(256), 0, st, C);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedCall& C, int kind, hipStream_t st) {
    const bool f32 = C.y_type == PM_F32;
    if (kind == kW16) {
        const int64_t xrows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
        if (C.n_rows >= 48 * int64_t(std::min(C.n_experts, C.n_rows)) &&
            (xrows * C.ldx + C.cols) * 2 < 0xFFFFFFF0ll)
            return launch_grouped_tiles(C, st);
        if (C.w_type == PM_F16)
            return f32 ? run_simple<kW16, PM_F16, PM_F16, PM_F32>(C, st)
                       : run_simple<kW16, PM_F16, PM_F16, PM_F16>(C, st);
        return f32 ? run_simple<kW16, PM_BF16, PM_BF16, PM_F32>(C, st)
                   : run_simple<kW16, PM_BF16, PM_BF16, PM_BF16>(C, st);
    }
    switch (C.x_type) {
    case PM_F32: return run_simple<kW4, PM_F16, PM_F32, PM_F32>(C, st);
    case PM_F16:
        return f32 ? run_simple<kW4, PM_F16, PM_F16, PM_F32>(C, st)
                   : run_simple<kW4, PM_F16, PM_F16, PM_F16>(C, st);
    default:
        return f32 ? run_simple<kW4, PM_F16, PM_BF16, PM_F32>(C, st)
                   : run_simple<kW4, PM_F16, PM_BF16, PM_BF16>(C, st);
    }
}

}  // namespace pm

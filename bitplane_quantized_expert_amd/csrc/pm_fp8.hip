// Products grouped by expert of 8-bit weights and activations.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_fp8.h"
#include "pm_grouped_codes.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kRows8 = 16, kOut8 = 64;

// 16 rows of x by 64 outputs (32 of gate and up) per workgroup, 16 weight rows
// a wave.
template <int YT>
__global__ __launch_bounds__(256) void plain8_kernel(const GroupedCall C, int nt) {
#ifdef __HIP_DEVICE_COMPILE__
    extern __shared__ int before[];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const bool glu = C.flags & PM_GROUPED_SWIGLU;
    const int out = glu ? C.rows / 2 : C.rows;
    const int blocks = (C.cols + 127) / 128, row_blocks = (C.rows + 127) / 128;
    const int64_t n_tiles = int64_t(tile_table(C, kRows8, before)) * nt;
    __syncthreads();
    for (int64_t tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
        const int mt = int(tile / nt);
        const int e = tile_expert(C, before, mt);
        const RowRange g = group_rows(C, e);
        const int64_t skip = int64_t(mt - before[e]) * kRows8;
        if (skip < 0 || skip >= g.n) continue;            // (bad offsets only)
        const int row0 = g.row0 + int(skip), n = min(g.n - int(skip), kRows8);
        // the weight row of a lane: 16 outputs, or 8 of gate and 8 of up
        const int o0 = int(tile - int64_t(mt) * nt) * (glu ? kOut8 / 2 : kOut8) + wv * (glu ? 8 : 16);
        const int o = o0 + (glu ? i16 & 7 : i16);
        const int wr = o < out ? (glu && i16 >= 8 ? out + o : o) : -1;
        const int u = i16 < n ? use_of(C, row0 + i16) : -1;
        const int64_t xr = u < 0 ? 0 : C.flags & PM_GROUPED_GATHER ? u / C.top_k : row0 + i16;
        const uint8_t* wp = static_cast<const uint8_t*>(C.w) + (size_t(e) * C.rows + max(wr, 0)) * C.cols;
        const uint8_t* xp = static_cast<const uint8_t*>(C.x) + xr * C.ldx;
        // sums of weight rows 4q .. 4q + 3 of the wave
        const int first = 4 * q;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        int sr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int oo = o0 + (glu ? (first + r) & 7 : first + r);
            const int rr = glu && first >= 8 ? out + oo : oo;
            sr[r] = min(rr, C.rows - 1) / 128;
        }
        for (int b = 0; b < blocks; ++b) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = b * 128 + h * 64 + q * 16;
                u32x4 w = {0, 0, 0, 0}, x = w;
                if (c < C.cols && wr >= 0) w = *reinterpret_cast<const u32x4*>(wp + c);
                if (c < C.cols && u >= 0) x = *reinterpret_cast<const u32x4*>(xp + c);
                d = mfma_x_w<false>(codes_f16(w[0], w[1]), codes_f16(x[0], x[1]), d);
                d = mfma_x_w<false>(codes_f16(w[2], w[3]), codes_f16(x[2], x[3]), d);
            }
            const float sx = u >= 0 ? C.xscales8[xr * blocks + b] : 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float sw = C.wscales8[(size_t(e) * row_blocks + sr[r]) * blocks + b];
                acc[r] = fmaf(d[r], sw * sx, acc[r]);
            }
        }
        // gate and up rows of an output are 32 lanes apart
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float other = __shfl_xor(acc[r], 32);
            v[r] = glu ? silu_up(acc[r], other) : acc[r];
        }
        if (u < 0 || (glu && q >= 2)) continue;
        const int64_t yr = C.flags & PM_GROUPED_SCATTER ? u : row0 + i16;
        store4<YT>(C.y, yr * C.ldy + o0 + first, out - o0 - first, v);
    }
#endif
}

template <int YT>
hipError_t run_plain8(const GroupedCall& C, hipStream_t st) {
    const bool glu = C.flags & PM_GROUPED_SWIGLU;
    const int out = glu ? C.rows / 2 : C.rows, per = glu ? kOut8 / 2 : kOut8;
    const int nt = (out + per - 1) / per;
    const int64_t tiles = (int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / kRows8) * nt;
    const unsigned grid = unsigned(std::min<int64_t>(tiles, 8 * compute_units()));
    hipLaunchKernelGGL(plain8_kernel<YT>, dim3(grid), dim3(256), (C.n_experts + 1) * sizeof(int),
                       st, C, nt);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped8(const GroupedCall& C, hipStream_t st) {
    const int64_t groups = std::min(C.n_experts, C.n_rows);
    const int64_t x_rows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
    const bool far = x_rows * C.ldx + C.cols >= 0xFFFFFFF0ll;
    if (C.n_rows >= 8 * groups && !far && C.cols > 0) {
        const int64_t tiles256 = (C.n_rows / 256) * int64_t((C.rows + 255) / 256);
        const bool big =
            (C.n_rows >= 224 * groups && tiles256 >= 2 * compute_units()) || !fp8_tiles128_fit(C);
        return launch_fp8_tiles(C, big ? 256 : 128, st);
    }
    switch (C.y_type) {
    case PM_F32: return run_plain8<PM_F32>(C, st);
    case PM_F16: return run_plain8<PM_F16>(C, st);
    default: return run_plain8<PM_BF16>(C, st);
    }
}

}  // namespace pm

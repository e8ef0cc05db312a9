// The routing-weighted combine of a layer's uses, and the encoder of 4-bit
// weights.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

template <int ZT, int YT>
__global__ __launch_bounds__(256) void combine_uses_kernel(int n_tokens, int top_k, int hidden,
                                                           const void* z, int64_t ldz,
                                                           const float* w, void* y, int64_t ldy) {
    const size_t n = size_t(n_tokens) * hidden;
    const size_t i = size_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const size_t t = i / hidden, c = i % hidden;
    float s = 0.0f;
    for (int j = 0; j < top_k; ++j) {
        const float wj = w[t * top_k + j];
        if (wj != 0.0f) s = fmaf(wj, load_f32<ZT>(z, (t * top_k + j) * ldz + c), s);
    }
    store_f32<YT>(y, t * ldy + c, s);
}

// One thread per group of inputs of one row.
template <int TYPE>
__global__ __launch_bounds__(256) void encode_w4_kernel(size_t n_groups, int group, const void* w,
                                                        uint8_t* q, uint16_t* scales,
                                                        uint8_t* zeros) {
    const size_t g = size_t(blockIdx.x) * 256 + threadIdx.x;
    if (g >= n_groups) return;
    const size_t base = g * group;
    float lo = 0.0f, hi = 0.0f;
    for (int i = 0; i < group; ++i) {
        const float v = load_f32<TYPE>(w, base + i);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    const float range = zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
    const __half s = __float2half(range);
    const float sf = __half2float(s);
    float z = 8.0f;
    if (zeros) z = sf > 0.0f ? fminf(fmaxf(rintf(-lo / sf), 0.0f), 15.0f) : 0.0f;
    scales[g] = __half_as_ushort(s);
    if (zeros) zeros[g] = uint8_t(z);
    for (int i = 0; i < group; i += 2) {
        uint32_t b = 0;
        for (int h = 0; h < 2; ++h) {
            const float v = load_f32<TYPE>(w, base + i + h);
            float c = z;
            if (sf > 0.0f) c = fminf(fmaxf(rintf(v / sf) + z, 0.0f), 15.0f);
            b |= uint32_t(c) << (4 * h);
        }
        q[(base + i) / 2] = uint8_t(b);
    }
}

}  // namespace

hipError_t launch_encode_w4(size_t n_groups, int group, const void* w, int type, uint8_t* q,
                            uint16_t* scales, uint8_t* zeros, hipStream_t st) {
    const dim3 grid(grid_for(n_groups, 256)), block(256);
    switch (type) {
    case PM_F32:
        hipLaunchKernelGGL(encode_w4_kernel<PM_F32>, grid, block, 0, st, n_groups, group, w, q,
                           scales, zeros);
        break;
    case PM_F16:
        hipLaunchKernelGGL(encode_w4_kernel<PM_F16>, grid, block, 0, st, n_groups, group, w, q,
                           scales, zeros);
        break;
    default:
        hipLaunchKernelGGL(encode_w4_kernel<PM_BF16>, grid, block, 0, st, n_groups, group, w, q,
                           scales, zeros);
        break;
    }
    return hipGetLastError();
}

template <int ZT, int YT>
static hipError_t combine_typed(int n_tokens, int top_k, int hidden, const void* z, int64_t ldz,
                                const float* w, void* y, int64_t ldy, hipStream_t st) {
    const size_t n = size_t(n_tokens) * hidden;
    hipLaunchKernelGGL((combine_uses_kernel<ZT, YT>), dim3(grid_for(n, 256)), dim3(256), 0, st,
                       n_tokens, top_k, hidden, z, ldz, w, y, ldy);
    return hipGetLastError();
}

hipError_t launch_combine_uses(int n_tokens, int top_k, int hidden, const void* z, int z_type,
                               int64_t ldz, const float* w, void* y, int y_type, int64_t ldy,
                               hipStream_t st) {
    auto* f = &combine_typed<PM_F32, PM_F32>;
    if (z_type == PM_F16)
        f = y_type == PM_F32 ? &combine_typed<PM_F16, PM_F32> : &combine_typed<PM_F16, PM_F16>;
    if (z_type == PM_BF16)
        f = y_type == PM_F32 ? &combine_typed<PM_BF16, PM_F32> : &combine_typed<PM_BF16, PM_BF16>;
    return f(n_tokens, top_k, hidden, z, ldz, w, y, ldy, st);
}

}  // namespace pm

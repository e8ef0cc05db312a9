// The routing-weighted combine of a layer's uses, and the encoder of 4-bit
// weights.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

// y[t][c] = sum_j w[t][j] z[t * top_k + j][c]: bound by reading z once.  A
// wave takes 64 * V adjacent columns of one token, so that the weights are
// scalars; V elements are 16 bytes of z (rows need no alignment beyond their
// element's: the hardware splits the accesses that cross a line).  U rows are
// on their way together.  Measured: 8191 tokens, top-10, 4096 bf16 columns 136
// us, 5.4 TB/s (a large copy reaches 4.8); 8 tokens of fp32 3.0 us.
template <int ZT, int YT, int U>
__device__ __forceinline__ void combine_chunk(int64_t t, int chunk, int top_k, int hidden,
                                              const void* z, int64_t ldz, const float* w, void* y,
                                              int64_t ldy) {
    constexpr int V = ZT == PM_F32 ? 4 : 8, ZB = ZT == PM_F32 ? 4 : 2, YB = YT == PM_F32 ? 4 : 2;
    // (lanes past the row stay: each holds one weight)
    const int c = int(min((int64_t(chunk) * kWave + (threadIdx.x & 63)) * V, int64_t(hidden) - 1));
    // the last columns of a row are taken as a whole vector that ends there;
    // rows of fewer columns element by element
    const bool whole = hidden >= V;
    const int c0 = whole ? min(c, hidden - V) : c;
    const char* zp = static_cast<const char*>(z) + (t * top_k * ldz + c0) * ZB;
    const float* wp = w + t * top_k;
    float s[V] = {};
    if (whole) {
        for (int j0 = 0; j0 < top_k; j0 += U) {
            uint32_t d[U][4];
            const int jl = j0 + int(threadIdx.x & 63);
            const float wl = jl < top_k ? wp[jl] : 0.0f;
#pragma unroll
            for (int k = 0; k < U; ++k)
                __builtin_memcpy(d[k], zp + min(j0 + k, top_k - 1) * ldz * ZB, 16);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const float wj = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wl), k));
                if (wj != 0.0f) {
#pragma unroll
                    for (int i = 0; i < V; ++i) s[i] = fmaf(wj, load_f32<ZT>(d[k], i), s[i]);
                }
            }
        }
        alignas(16) char o[V * YB];
#pragma unroll
        for (int i = 0; i < V; ++i) store_f32<YT>(o, i, s[i]);
        __builtin_memcpy(static_cast<char*>(y) + (t * ldy + c0) * YB, o, V * YB);
        return;
    }
    for (int i = 0; i < hidden - c0; ++i) {
        float v = 0.0f;
        for (int j = 0; j < top_k; ++j)
            if (wp[j] != 0.0f) v = fmaf(wp[j], load_f32<ZT>(zp + j * ldz * ZB, i), v);
        store_f32<YT>(y, t * ldy + c0 + i, v);
    }
}

// A wave goes on by the waves of the grid, which is held below the 2^32 threads
// of a launch; up to 2^20 workgroups every wave has one chunk at most.
template <int ZT, int YT, int U>
__global__ __launch_bounds__(256) void combine_uses_kernel(int n_tokens, int top_k, int hidden,
                                                           int chunks, const void* z, int64_t ldz,
                                                           const float* w, void* y, int64_t ldy) {
    const int64_t all = int64_t(n_tokens) * chunks;
    for (int64_t id = int64_t(blockIdx.x) * 4 + uni(threadIdx.x >> 6); id < all;
         id += int64_t(gridDim.x) * 4) {
        const int64_t t = id / chunks;
        combine_chunk<ZT, YT, U>(t, int(id - t * chunks), top_k, hidden, z, ldz, w, y, ldy);
    }
}

// Offline, and simple: one thread per group of inputs of one row, so that no sum
// or maximum crosses threads.  Neighbouring lanes read a group apart, one element
// at a time, and a cache line is fetched again for most of its elements: 65536 x
// 4096 bf16 weights take 10 ms in groups of 128 (61 GB fetched for 0.54) and 1.2
// in groups of 32, fp32 ones 10 ms in both, where the bytes need 0.1 to 0.2.
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
    // (a scale beyond fp16 would be infinite, and zeros NaN)
    const __half s = __float2half(fminf(range, 65504.0f));
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
    const int per_wave = kWave * (ZT == PM_F32 ? 4 : 8);
    const int chunks = hidden / per_wave + (hidden % per_wave != 0);
    const dim3 grid(unsigned(std::min<int64_t>((int64_t(n_tokens) * chunks + 3) / 4, 1 << 20)));
    // all rows of a token together where they are 10 at most: 8 fp32 tokens of
    // top-10 3.2 us against 3.7 with 8 rows at a time, 512 bf16 tokens 10.7
    // against 11.3, from some thousands on equal within 1 %
    auto* f = &combine_uses_kernel<ZT, YT, 8>;
    if (top_k <= 2) f = &combine_uses_kernel<ZT, YT, 2>;
    else if (top_k <= 4) f = &combine_uses_kernel<ZT, YT, 4>;
    else if (top_k == 9 || top_k == 10) f = &combine_uses_kernel<ZT, YT, 10>;
    hipLaunchKernelGGL(f, grid, dim3(256), 0, st, n_tokens, top_k, hidden, chunks, z, ldz, w, y,
                       ldy);
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

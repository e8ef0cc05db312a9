// The encoder of 8-bit codes: per block of 128 inputs of 1 or 128 rows,
//   scale = max(max|x| / 448, 2^-126),   q = e4m3(x / scale)   (fp32).
// Bound by reading x and writing the codes once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

struct EncodeCall {
    const void* x;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldq;
    int32_t rows, cols, blocks;                     // of a matrix; blocks of 128 inputs
    int32_t row_blocks;                             // of a matrix
};

// The 8 inputs of a lane: 16 lanes hold 128.
struct Eight {
    float v[8];
};
template <int TYPE>
__device__ inline Eight load8(const void* x, int64_t at) {
    constexpr int B = TYPE == PM_F32 ? 4 : 2;
    uint32_t d[2 * B];
    __builtin_memcpy(d, __builtin_assume_aligned(static_cast<const char*>(x) + at * B, 16), 8 * B);
    Eight r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = load_f32<TYPE>(d, i);
    return r;
}

__device__ inline float largest8(const Eight& x) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fabsf(x.v[i]) < INFINITY ? fmaxf(m, fabsf(x.v[i])) : m;
    return m;
}
// Largest over each 16 lanes, in every lane.
__device__ inline float row16_max(float v) {
    v = fmaxf(v, dpp<0xB1, 0xF>(v));
    v = fmaxf(v, dpp<0x4E, 0xF>(v));
    v = fmaxf(v, dpp<0x141, 0xF>(v));
    return fmaxf(v, dpp<0x140, 0xF>(v));
}

__device__ inline float scale_of(float largest) {
    return fmaxf(largest / 448.0f, 1.17549435e-38f);
}

__device__ inline uint64_t codes8(const Eight& x, float scale) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * h] / scale, x.v[4 * h + 1] / scale, 0, false);
        w[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x.v[4 * h + 2] / scale,
                                                        x.v[4 * h + 3] / scale, p, true));
    }
    return uint64_t(w[1]) << 32 | w[0];
}

// One scale per row and 128 inputs: 16 lanes a block.
template <int TYPE>
__global__ __launch_bounds__(256) void encode_rows_kernel(const EncodeCall C, int64_t n) {
    const int64_t step = int64_t(gridDim.x) * 16;
    for (int64_t b = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4); b < n; b += step) {
        const int64_t row = b / C.blocks;
        const int col = int(b - row * C.blocks) * 128 + (threadIdx.x & 15) * 8;
        const bool in = col < C.cols;
        Eight x{};
        if (in) x = load8<TYPE>(C.x, row * C.ldx + col);
        const float scale = scale_of(row16_max(largest8(x)));
        if (in) *reinterpret_cast<uint64_t*>(C.q + row * C.ldq + col) = codes8(x, scale);
        if ((threadIdx.x & 15) == 0) C.scales[b] = scale;
    }
}

// One scale per 128 x 128: a workgroup a block, 8 rows of a thread's inputs in
// registers.
template <int TYPE>
__global__ __launch_bounds__(256) void encode_square_kernel(const EncodeCall C, int64_t n) {
    __shared__ float wave_max[2][4];
    int parity = 0;
    for (int64_t b = blockIdx.x; b < n; b += gridDim.x, parity ^= 1) {
        const int64_t rb = b / C.blocks, m = rb / C.row_blocks;
        const int col = int(b - rb * C.blocks) * 128 + (threadIdx.x & 15) * 8;
        const int row0 = int(rb - m * C.row_blocks) * 128 + (threadIdx.x >> 4);
        Eight x[8];
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = Eight{};
            if (col < C.cols && row0 + i * 16 < C.rows)
                x[i] = load8<TYPE>(C.x, (m * C.rows + row0 + i * 16) * C.ldx + col);
            big = fmaxf(big, largest8(x[i]));
        }
        big = row16_max(big);
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        if ((threadIdx.x & 63) == 0) wave_max[parity][threadIdx.x >> 6] = big;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) big = fmaxf(big, wave_max[parity][w]);
        const float scale = scale_of(big);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col < C.cols && row0 + i * 16 < C.rows)
                *reinterpret_cast<uint64_t*>(C.q + (m * C.rows + row0 + i * 16) * C.ldq + col) =
                    codes8(x[i], scale);
        if (threadIdx.x == 0) C.scales[b] = scale;
    }
}

template <int TYPE>
hipError_t run_encode8(const EncodeCall& C, int n, int block_rows, hipStream_t st) {
    const int64_t blocks = int64_t(n) * C.row_blocks * C.blocks;
    if (block_rows == 1) {
        const unsigned grid = unsigned(std::min<int64_t>((blocks + 15) / 16, 1 << 20));
        hipLaunchKernelGGL(encode_rows_kernel<TYPE>, dim3(grid), dim3(256), 0, st, C, blocks);
    } else {
        const unsigned grid = unsigned(std::min<int64_t>(blocks, 1 << 20));
        hipLaunchKernelGGL(encode_square_kernel<TYPE>, dim3(grid), dim3(256), 0, st, C, blocks);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_encode8(int n, int rows, int cols, int block_rows, const void* x, int type,
                          int64_t ldx, uint8_t* q, int64_t ldq, float* scales, hipStream_t st) {
    EncodeCall C{};
    C.x = x;
    C.q = q;
    C.scales = scales;
    C.ldx = ldx;
    C.ldq = ldq;
    C.rows = rows;
    C.cols = cols;
    C.blocks = int((int64_t(cols) + 127) / 128);
    C.row_blocks = int((int64_t(rows) + block_rows - 1) / block_rows);
    switch (type) {
    case PM_F32: return run_encode8<PM_F32>(C, n, block_rows, st);
    case PM_F16: return run_encode8<PM_F16>(C, n, block_rows, st);
    default: return run_encode8<PM_BF16>(C, n, block_rows, st);
    }
}

}  // namespace pm

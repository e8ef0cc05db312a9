// The encoder of 8-bit codes: per block of 128 inputs of 1 or 128 rows,
//   scale = max(max|x| / 448, 2^-126),   q = e4m3 of x / scale, rounded once.
// Bound by reading x and writing the codes once.  8 lanes take a row of a block,
// each of them a 16-byte piece of x in turn, so that every load and store of a
// wave covers whole lines.
//
// The quotient is not formed by a division: its own rounding would meet the
// border of two codes in some bf16 blocks in a hundred values, and a dozen
// instructions a value would bound the kernel (24 in all took 42 us for 16384 x 4096
// bf16 values, these 8 take 34.5).  With t = x / scale or up to 2^-20 of it more, and h = t cut off to
// 12 bits, which every border between two codes has, the sign of the remainder
// |x| - |h| scale says on which side of h the quotient lies, and h moved there by
// one ulp of fp32 rounds as the quotient does.  One fma gives that sign while the
// remainder is a multiple of fp32's smallest number, 2^-149: h counts from
// 2^-10 on (half the smallest code), so its last bit is 2^-21 or more, and that of
// a scale of 2^-105 or more is 2^-128 or more.  Below 2^-100 x and scale are both
// taken times 2^24, which changes no quotient: the last bits are 2^-125 and
// 2^-146 then.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct EncodeCall {
    const void* x;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldq;
    int32_t rows, cols, blocks;                     // of a matrix; blocks of 128 inputs
    int32_t row_blocks;                             // of a matrix
};

// The 16 inputs of lane l of 8: pieces l, l + 8, .. of 16 bytes of a block's row.
template <int TYPE>
struct Raw16 {
    static constexpr int kPieces = TYPE == PM_F32 ? 4 : 2, kPer = 16 / kPieces;
    u32x4 d[kPieces];
};
// The first input of piece k.
template <int TYPE>
__device__ inline int piece_at(int l, int k) {
    return (k * 8 + l) * Raw16<TYPE>::kPer;
}
// Input `col` of a row at p on; x is read once, past the caches.
template <int TYPE>
__device__ inline Raw16<TYPE> load16(const EncodeCall& C, int64_t row, int col, int l) {
    constexpr int B = TYPE == PM_F32 ? 4 : 2;
    const char* p = static_cast<const char*>(C.x) + row * C.ldx * B;
    Raw16<TYPE> r;
#pragma unroll
    for (int k = 0; k < Raw16<TYPE>::kPieces; ++k) {
        const int c = col + piece_at<TYPE>(l, k);
        r.d[k] = u32x4{0, 0, 0, 0};
        if (c < C.cols) {
            const u32x4* at = reinterpret_cast<const u32x4*>(p + int64_t(c) * B);
            r.d[k] = __builtin_nontemporal_load(at);
        }
    }
    return r;
}
template <int TYPE>
__device__ inline float value(const u32x4& d, int i) {
    if constexpr (TYPE == PM_F32) return __uint_as_float(d[i]);
    const uint32_t w = d[i >> 1];
    if constexpr (TYPE == PM_BF16) return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    return __half2float(__ushort_as_half(uint16_t(i & 1 ? w >> 16 : w)));
}

// The largest |x| of these, as a bit pattern of fp32 (which orders like the
// numbers): infinity or more where one is not finite, unless FINITE leaves these
// out.
template <int TYPE, bool FINITE>
__device__ inline uint32_t largest16(const Raw16<TYPE>& x) {
    uint32_t m = 0;
    if constexpr (FINITE || TYPE == PM_F32) {
#pragma unroll
        for (int k = 0; k < Raw16<TYPE>::kPieces; ++k)
#pragma unroll
            for (int i = 0; i < Raw16<TYPE>::kPer; ++i) {
                const uint32_t a = __float_as_uint(value<TYPE>(x.d[k], i)) & 0x7FFFFFFFu;
                m = !FINITE || a < 0x7F800000u ? max(m, a) : m;
            }
        return m;
    } else {
        // pairs of 16-bit patterns
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 p = {0, 0};
#pragma unroll
        for (int k = 0; k < Raw16<TYPE>::kPieces; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p = __builtin_elementwise_max(
                    p, __builtin_bit_cast(u16x2, uint32_t(x.d[k][i] & 0x7FFF7FFFu)));
        const uint32_t w = max(p[0], p[1]);
        if constexpr (TYPE == PM_BF16) return w << 16;
        return __float_as_uint(__half2float(__ushort_as_half(uint16_t(w))));
    }
}
template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
    return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false)));
}
// Largest over each 8 lanes, in every lane.
__device__ inline uint32_t row8_max(uint32_t v) {
    v = dpp_max<0xB1>(v);                           // quad_perm [1,0,3,2]
    v = dpp_max<0x4E>(v);                           // quad_perm [2,3,0,1]
    return dpp_max<0x141>(v);                       // row_half_mirror
}

// max(largest / 448, 2^-126), the quotient rounded to nearest: one correction by
// the exact remainder does that.
__device__ inline float scale_of(uint32_t largest) {
    const float a = __uint_as_float(largest), r = 1.0f / 448.0f;
    const float q = a * r;
    return fmaxf(fmaf(fmaf(-q, 448.0f, a), r, q), 1.17549435e-38f);
}

// A number that rounds to e4m3 as x / scale does; over = 1 / scale and a little.
__device__ inline float quotient(float x, float scale, float over) {
    const uint32_t h = __float_as_uint(x * over) & 0xFFFFF000u;
    const float rest = fmaf(-fabsf(__uint_as_float(h)), scale, fabsf(x));
    int side;                                       // (+0 where h is the quotient)
    asm("v_med3_i32 %0, %1, -1, 1" : "=v"(side) : "v"(rest));
    return __uint_as_float(h + uint32_t(side));
}

// Whether a block of this largest |x| is an ordinary one: no infinities or NaN,
// and its scale, largest / 448, is not below 2^-100 (or the block is all zeros).
__device__ inline bool ordinary(uint32_t largest) {
    constexpr uint32_t kLeast = (127u - 91u) << 23;      // of 2^-91 > 448 * 2^-100
    return largest == 0 || largest - kLeast < 0x7F800000u - kLeast;
}

// The codes of these.  ORDINARY: of an ordinary block.
template <int TYPE, bool ORDINARY>
__device__ inline void store16(const EncodeCall& C, int64_t row, int col, int l,
                               const Raw16<TYPE>& x, float scale) {
    constexpr int kPer = Raw16<TYPE>::kPer;
    const float lift = ORDINARY || scale >= 0x1p-100f ? 1.0f : 0x1p24f;
    scale *= lift;
    const float over = __builtin_amdgcn_rcpf(scale) * (1.0f + 0x1p-21f);
    uint8_t* p = C.q + row * C.ldq;
#pragma unroll
    for (int k = 0; k < Raw16<TYPE>::kPieces; ++k) {
        const int c = col + piece_at<TYPE>(l, k);
        uint32_t w[kPer / 4];
#pragma unroll
        for (int h = 0; h < kPer / 4; ++h) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float xi = value<TYPE>(x.d[k], 4 * h + i);
                if (!ORDINARY) xi *= lift;
                v[i] = quotient(xi, scale, over);
                if (!ORDINARY && !(fabsf(xi) < INFINITY)) v[i] = __uint_as_float(0x7FC00000u);
            }
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            w[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true));
        }
        if (c < C.cols)
            __builtin_memcpy(__builtin_assume_aligned(p + c, kPer), w, kPer);
    }
}

// One scale per row and 128 inputs.  A lane goes on by the blocks of the grid; its
// place is moved, not divided anew.  Measured: 16384 x 4096 bf16 34.5 us, 5.9 TB/s
// (6.2 is what an elementwise kernel of one read and one write reaches); with
// loads through the caches 36.7, with two blocks of a lane on their way together
// 34.8, with 8 workgroups per compute unit instead of 32 36.5.
template <int TYPE>
__global__ __launch_bounds__(256) void encode_rows_kernel(const EncodeCall C, int64_t n) {
    const uint32_t blocks = uint32_t(C.blocks);
    const uint32_t grid = gridDim.x * 32;
    const uint32_t step_rows = grid / blocks, step_cols = grid - step_rows * blocks;
    const uint32_t first = blockIdx.x * 32 + (threadIdx.x >> 3);
    uint32_t row = first / blocks, cb = first - row * blocks;
    const int l = threadIdx.x & 7;
    for (int64_t b = first; b < n; b += grid) {
        const int col = int(cb * 128);
        const Raw16<TYPE> x = load16<TYPE>(C, row, col, l);
        const uint32_t big = row8_max(largest16<TYPE, false>(x));
        float scale;
        if (__ballot(!ordinary(big)) == 0) {
            scale = scale_of(big);
            store16<TYPE, true>(C, row, col, l, x, scale);
        } else {
            scale = scale_of(row8_max(largest16<TYPE, true>(x)));
            store16<TYPE, false>(C, row, col, l, x, scale);
        }
        if (l == 0) C.scales[b] = scale;
        row += step_rows;
        cb += step_cols;
        if (cb >= blocks) {
            cb -= blocks;
            ++row;
        }
    }
}

// One scale per 128 x 128: a workgroup a block, R rows of a thread's inputs in
// registers.  Blocks that share rows go to one XCD, whose L2 then holds the lines
// that two of them share (rows need not begin at a line).  Measured: 64 matrices
// of 2048 x 4096 bf16 282 us, 5.7 TB/s (308 without regard to the XCDs, 298 with
// loads through the caches, 286 with 2 rows and twice the threads); 40 of 1426 x
// 1008 fp32 59.7 to 60.5 us, 4.8 TB/s (a twelfth of the workgroups has 18 rows); 80 of 1426
// x 1008 bf16 82 us (109 without regard to the XCDs; 75 through the caches: lines
// that two blocks share).
template <int TYPE, int R>
__global__ __launch_bounds__(1024 / R) void encode_square_kernel(const EncodeCall C, int64_t n) {
    __shared__ uint32_t wave_max[2][2][16 / R];          // of all, and of the finite
    constexpr int kStep = 128 / R;                  // rows apart of a thread
    int parity = 0;
    // workgroups go to the XCDs in turn: each of these has an eighth of the blocks
    const int64_t per = (n + 7) / 8, b0 = (blockIdx.x & 7) * per, end = min(b0 + per, n);
    for (int64_t b = b0 + (blockIdx.x >> 3); b < end; b += gridDim.x >> 3, parity ^= 1) {
        const int64_t rb = b / C.blocks, m = rb / C.row_blocks;
        const int col = int(b - rb * C.blocks) * 128, l = threadIdx.x & 7;
        const int row0 = int(rb - m * C.row_blocks) * 128 + (threadIdx.x >> 3);
        Raw16<TYPE> x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i] = Raw16<TYPE>{};
            if (row0 + i * kStep < C.rows) x[i] = load16<TYPE>(C, m * C.rows + row0 + i * kStep, col, l);
        }
        auto block_max = [&](uint32_t big, uint32_t* of) {
            big = row8_max(big);
#pragma unroll
            for (int d = 8; d < kWave; d <<= 1) big = max(big, uint32_t(__shfl_xor(int(big), d)));
            if ((threadIdx.x & 63) == 0) of[threadIdx.x >> 6] = big;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 16 / R; ++w) big = max(big, of[w]);
            return big;
        };
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) big = max(big, largest16<TYPE, false>(x[i]));
        big = block_max(big, wave_max[parity][0]);
        const bool plain = ordinary(big);           // the same in every thread
        if (!plain) {
            big = 0;
#pragma unroll
            for (int i = 0; i < R; ++i) big = max(big, largest16<TYPE, true>(x[i]));
            big = block_max(big, wave_max[parity][1]);
        }
        const float scale = scale_of(big);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (row0 + i * kStep >= C.rows) continue;
            const int64_t row = m * C.rows + row0 + i * kStep;
            if (plain)
                store16<TYPE, true>(C, row, col, l, x[i], scale);
            else
                store16<TYPE, false>(C, row, col, l, x[i], scale);
        }
        if (threadIdx.x == 0) C.scales[b] = scale;
    }
}

template <int TYPE>
hipError_t run_encode8(const EncodeCall& C, int n, int block_rows, hipStream_t st) {
    const int64_t blocks = int64_t(n) * C.row_blocks * C.blocks;
    if (block_rows == 1) {
        const unsigned grid =
            unsigned(std::min<int64_t>((blocks + 31) / 32, int64_t(compute_units()) * 32));
        hipLaunchKernelGGL((encode_rows_kernel<TYPE>), dim3(grid), dim3(256), 0, st, C, blocks);
    } else {
        const unsigned grid = unsigned(std::min<int64_t>((blocks + 7) / 8 * 8, 1 << 20));
        constexpr int R = 4;
        hipLaunchKernelGGL((encode_square_kernel<TYPE, R>), dim3(grid), dim3(1024 / R), 0, st, C, blocks);
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

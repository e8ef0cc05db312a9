// Pieces that the kernels of the 8-bit products share: operands of codes, and
// codes as halves.  Internal linkage.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "pm_device.h"
#include "pm_grouped_codes.h"
#include "pm_routed.h"

namespace pm {

// Whether the tiles of a call multiply codes as they are, in sums that are cut off.
inline bool fp8_cuts_off(const GroupedCall& C) {
    return C.y_type == PM_BF16 && !(C.flags & PM_GROUPED_FP32_SUMS);
}
// Tiles of 256 or 128 rows (where sums are not cut off: 128) x 256 (pm_fp8_tile.hip);
// the offsets of a tile's rows in x must fit 32 bits.
hipError_t launch_fp8_tiles(const GroupedCall& C, int rows, hipStream_t st);
// Whether the table of experts lies in LDS beside the three stages of 128-row
// tiles (beside those of 256 rows, and beside two stages, it always does).
bool fp8_tiles128_fit(const GroupedCall& C);
// Weights streamed past 16 rows of activations (pm_fp8_stream.hip); any sizes.
hipError_t launch_fp8_stream(const GroupedCall& C, hipStream_t st);

namespace {

// f(0), .., f(N - 1) with constant arguments.
template <int N, int I = 0, class F>
__device__ inline void for_each(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        for_each<N, I + 1>(f);
    }
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ inline i32x8 join(const u32x4& a, const u32x4& b) {
    return i32x8{int(a[0]), int(a[1]), int(a[2]), int(a[3]),
                 int(b[0]), int(b[1]), int(b[2]), int(b[3])};
}

// 128 inputs, 32 codes a lane: the lanes' pieces may hold any inputs that both
// operands share.
__device__ inline f32x4 mfma_codes(const i32x8& w, const i32x8& x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                            0, 0, 0, 0);
}

// 8 codes as halves, exactly (NaN stays NaN).
__device__ inline u32x4 codes_f16(uint32_t a, uint32_t b) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
    return r;
}

struct HalfOperand {
    u32x4 k[4];
};
__device__ inline HalfOperand halves_of(const i32x8& c) {
    HalfOperand h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h.k[i] = codes_f16(uint32_t(c[2 * i]), uint32_t(c[2 * i + 1]));
    return h;
}
__device__ inline f32x4 mfma_halves(const HalfOperand& w, const HalfOperand& x) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = mfma_x_w<false>(w.k[i], x.k[i], d);
    return d;
}

}  // namespace
}  // namespace pm

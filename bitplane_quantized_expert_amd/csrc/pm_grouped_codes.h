// Pieces that the kernels of the grouped products share: matrix products, 4-bit
// codes as halves, offsets beyond a buffer.  Internal linkage.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pm_device.h"
#include "pm_routed.h"

namespace pm {
namespace {

// An offset beyond any buffer of less than 2 GiB, with any immediate added, and
// one beyond any buffer.
constexpr uint32_t kNowhere = 0x80000000u, kOutside = 0xFFFFFFF0u;
constexpr int kRawBuffer = 0x00020000;          // raw buffer, 32-bit data format
// How scales are read and applied: groups of 32, 64 or 128 inputs in aligned
// vectors, or (kAnyGroup) one by one for every 32 inputs.
enum { kNoGroup = 0, kGroup32 = 32, kGroup64 = 64, kGroup128 = 128, kAnyGroup = 1 };
// Whether the scales of `blocks` blocks of 128 inputs can be read as aligned
// vectors of up to 4.
inline bool reads_scales_by(const GroupedCall& C, int group, int blocks) {
    const int n = std::min(4, blocks * 128 / group);
    return C.group == group && (C.cols / group) % n == 0 &&
           reinterpret_cast<uintptr_t>(C.scales) % (2 * n) == 0 &&
           reinterpret_cast<uintptr_t>(C.zeros) % n == 0;
}

// `at` or kNowhere, as a value: the compiler may not make branches of it with
// a load in each.
__device__ inline uint32_t chosen(bool ok, uint32_t at) {
    at = ok ? at : kNowhere;
    asm("" : "+v"(at));
    return at;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
__device__ inline f32x4 mfma_x_w(const u32x4& x, const u32x4& w, const f32x4& c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                       __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
}

// The constants of codes_to_f16 in registers, so that AND and OR are one
// instruction.
struct CodeBits {
    uint32_t even, odd, k1024, k64;
};
__device__ inline CodeBits code_bits() {
    CodeBits c{0x000F000Fu, 0x00F000F0u, 0x64006400u, 0x54005400u};
    asm("" : "+v"(c.even), "+v"(c.odd), "+s"(c.k1024), "+s"(c.k64));
    return c;
}

// The 8 codes of word w minus the zero point, as halves in the order
// 0 4 1 5 2 6 3 7; za = 1024 + z, zb = 64 + z, twice each.
__device__ inline u32x4 codes_to_f16(const CodeBits& k, uint32_t w, f16x2 za, f16x2 zb) {
    const uint32_t w8 = w >> 8;
    const f16x2 a = __builtin_bit_cast(f16x2, (w & k.even) | k.k1024) - za;
    const f16x2 b = __builtin_bit_cast(f16x2, (w & k.odd) | k.k64) - zb;
    const f16x2 c = __builtin_bit_cast(f16x2, (w8 & k.even) | k.k1024) - za;
    const f16x2 d = __builtin_bit_cast(f16x2, (w8 & k.odd) | k.k64) - zb;
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                 __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

// 4 x 4 transposition of the words of lanes i, i + 16, i + 32, i + 48.
__device__ inline u32x4 exchange(u32x4 w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{uint32_t(c[0]), uint32_t(c[1]), uint32_t(d[0]), uint32_t(d[1])};
}

__device__ inline float half_bits(uint32_t h) {
    return float(__builtin_bit_cast(_Float16, uint16_t(h)));
}

}  // namespace
}  // namespace pm

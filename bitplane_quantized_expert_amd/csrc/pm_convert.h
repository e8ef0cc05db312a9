// Element types of the routed-expert operators: loads to fp32 and stores
// rounded to nearest even.  Internal linkage.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pm.h"

namespace pm {
namespace {

template <int TYPE>
__device__ inline float load_f32(const void* p, int64_t i) {
    if constexpr (TYPE == PM_F32) return static_cast<const float*>(p)[i];
    if constexpr (TYPE == PM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
}

template <int TYPE>
__device__ inline void store_f32(void* p, int64_t i, float v) {
    if constexpr (TYPE == PM_F32)
        static_cast<float*>(p)[i] = v;
    else if constexpr (TYPE == PM_F16)
        static_cast<__half*>(p)[i] = __float2half(v);
    else
        static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

}  // namespace
}  // namespace pm

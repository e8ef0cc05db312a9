// The scored router's sigmoid in fp32, by which it ranks experts before it decides
// in fp64, and the bounds on what it is off by.  Internal linkage.
#pragma once

#include <hip/hip_runtime.h>

namespace pm {
namespace {

// Found by trying every fp32 logit: off by 1.108e-7 at most, and by 2^-17.9 of
// itself where it is kSigmoidSmall or more (below 2^-126 the reciprocal is 0).
// tests/native/device_facts.hip tries them again.
constexpr float kSigmoidError = 0x1p-23f, kSigmoidRelative = 0x1.2p-18f;
constexpr float kSigmoidSmall = 0x1p-125f;
__device__ inline float sigmoid_rank(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l * -1.44269504f));
}

}  // namespace
}  // namespace pm

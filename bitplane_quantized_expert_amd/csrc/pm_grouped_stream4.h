// Streamed grouped products with 4-bit weights: the choice of the kernel for
// one type of activations.  Instantiated for 16-bit activations in
// pm_grouped_stream4.hip and for fp32 in pm_grouped_stream4f.hip.
#pragma once

#include "pm_grouped_stream.h"

namespace pm {
namespace {

template <bool X32, int KB, int MT, bool ZEROS>
hipError_t run4_group(const GroupedCall& C, const StreamPlan& P, hipStream_t st) {
    // groups are read as aligned vectors of up to 4 scales
    auto vector_ok = [&](int group) {
        const int n = std::min(4, KB * 128 / group);
        return C.group == group && (C.cols / group) % n == 0 &&
               reinterpret_cast<uintptr_t>(C.scales) % (2 * n) == 0 &&
               reinterpret_cast<uintptr_t>(C.zeros) % n == 0;
    };
    if (vector_ok(128)) return run_stream<kW4, false, X32, KB, MT, kGroup128, ZEROS>(C, P, st);
    if (vector_ok(64)) return run_stream<kW4, false, X32, KB, MT, kGroup64, ZEROS>(C, P, st);
    if (vector_ok(32)) return run_stream<kW4, false, X32, KB, MT, kGroup32, ZEROS>(C, P, st);
    return run_stream<kW4, false, X32, KB, MT, kAnyGroup, ZEROS>(C, P, st);
}

template <bool X32, int MT, bool ZEROS>
hipError_t run4(const GroupedCall& C, hipStream_t st) {
    int kb;
    const StreamPlan P = plan_stream(C, MT, &kb);
    switch (kb) {
    case 1: return run4_group<X32, 1, MT, ZEROS>(C, P, st);
    case 2: return run4_group<X32, 2, MT, ZEROS>(C, P, st);
    default:
        if constexpr (MT == 1) return run4_group<X32, 4, 1, ZEROS>(C, P, st);
        return hipErrorInvalidValue;                      // plan_stream gives no such plan
    }
}

template <bool X32>
hipError_t run4_any(const GroupedCall& C, int mt, hipStream_t st) {
    if (C.zeros) return mt == 1 ? run4<X32, 1, true>(C, st) : run4<X32, 2, true>(C, st);
    return mt == 1 ? run4<X32, 1, false>(C, st) : run4<X32, 2, false>(C, st);
}

}  // namespace
}  // namespace pm

// Streamed grouped products with 4-bit weights: the choice of the kernel for
// one type of activations.  Instantiated for 16-bit activations in
// pm_grouped_stream4.hip and for fp32 in pm_grouped_stream4f.hip.
#pragma once

#include "pm_grouped_stream.h"

namespace pm {
namespace {

template <bool X32, int NW, int KB, bool ZEROS>
hipError_t run4_group(const GroupedCall& C, const StreamPlan& P, hipStream_t st) {
    if (reads_scales_by(C, 128, KB)) return run_stream<kW4, false, X32, NW, KB, kGroup128, ZEROS>(C, P, st);
    if (reads_scales_by(C, 64, KB)) return run_stream<kW4, false, X32, NW, KB, kGroup64, ZEROS>(C, P, st);
    if (reads_scales_by(C, 32, KB)) return run_stream<kW4, false, X32, NW, KB, kGroup32, ZEROS>(C, P, st);
    return run_stream<kW4, false, X32, NW, KB, kAnyGroup, ZEROS>(C, P, st);
}

template <bool X32, bool ZEROS>
hipError_t run4(const GroupedCall& C, hipStream_t st) {
    int nw, kb;
    const StreamPlan P = plan_stream(C, &nw, &kb);
    if (nw == 8) return run4_group<X32, 8, 4, ZEROS>(C, P, st);
    switch (kb) {
    case 1: return run4_group<X32, 4, 1, ZEROS>(C, P, st);
    case 2: return run4_group<X32, 4, 2, ZEROS>(C, P, st);
    default: return run4_group<X32, 4, 4, ZEROS>(C, P, st);
    }
}

}  // namespace
}  // namespace pm

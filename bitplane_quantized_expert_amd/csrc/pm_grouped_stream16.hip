// Streamed grouped products with 16-bit weights.
#include "pm_grouped_stream.h"

namespace pm {

namespace {

template <bool BF16, int MT>
hipError_t run16(const GroupedCall& C, hipStream_t st) {
    int kb;
    const StreamPlan P = plan_stream(C, MT, &kb);
    switch (kb) {
    case 1: return run_stream<kW16, BF16, false, 1, MT, kNoGroup, false>(C, P, st);
    case 2: return run_stream<kW16, BF16, false, 2, MT, kNoGroup, false>(C, P, st);
    default:
        if constexpr (MT == 1) return run_stream<kW16, BF16, false, 4, 1, kNoGroup, false>(C, P, st);
        return hipErrorInvalidValue;                      // plan_stream gives no such plan
    }
}

}  // namespace

hipError_t launch_grouped_stream16(const GroupedCall& C, int mt, hipStream_t st) {
    if (C.w_type == PM_BF16) return mt == 1 ? run16<true, 1>(C, st) : run16<true, 2>(C, st);
    return mt == 1 ? run16<false, 1>(C, st) : run16<false, 2>(C, st);
}

}  // namespace pm

// Streamed grouped products with 16-bit weights.
#include "pm_grouped_stream.h"

namespace pm {

namespace {

template <bool BF16>
hipError_t run16(const GroupedCall& C, hipStream_t st) {
    int nw, kb;
    const StreamPlan P = plan_stream(C, &nw, &kb);
    if (nw == 8) return run_stream<kW16, BF16, false, 8, 4, kNoGroup, false>(C, P, st);
    switch (kb) {
    case 1: return run_stream<kW16, BF16, false, 4, 1, kNoGroup, false>(C, P, st);
    case 2: return run_stream<kW16, BF16, false, 4, 2, kNoGroup, false>(C, P, st);
    default: return run_stream<kW16, BF16, false, 4, 4, kNoGroup, false>(C, P, st);
    }
}

}  // namespace

hipError_t launch_grouped_stream16(const GroupedCall& C, hipStream_t st) {
    return C.w_type == PM_BF16 ? run16<true>(C, st) : run16<false>(C, st);
}

}  // namespace pm

// Streamed grouped products with 4-bit weights and 16-bit activations.
#include "pm_grouped_stream4.h"

namespace pm {

hipError_t launch_grouped_stream4(const GroupedCall& C, hipStream_t st) {
    return C.zeros ? run4<false, true>(C, st) : run4<false, false>(C, st);
}

}  // namespace pm

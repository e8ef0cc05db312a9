// Streamed grouped products with 4-bit weights and fp32 activations.
#include "pm_grouped_stream4.h"

namespace pm {

hipError_t launch_grouped_stream4f(const GroupedCall& C, hipStream_t st) {
    return C.zeros ? run4<true, true>(C, st) : run4<true, false>(C, st);
}

}  // namespace pm

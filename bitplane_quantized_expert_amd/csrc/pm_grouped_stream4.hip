// Streamed grouped products with 4-bit weights and 16-bit activations.
#include "pm_grouped_stream4.h"

namespace pm {

hipError_t launch_grouped_stream4(const GroupedCall& C, int mt, hipStream_t st) {
    return run4_any<false>(C, mt, st);
}

}  // namespace pm

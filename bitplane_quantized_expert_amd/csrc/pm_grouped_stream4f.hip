// Streamed grouped products with 4-bit weights and fp32 activations.
#include "pm_grouped_stream4.h"

namespace pm {

hipError_t launch_grouped_stream4f(const GroupedCall& C, int mt, hipStream_t st) {
    return run4_any<true>(C, mt, st);
}

}  // namespace pm

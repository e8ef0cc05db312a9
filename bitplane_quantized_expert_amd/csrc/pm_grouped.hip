// Which kernel a grouped product takes.
#include <algorithm>

#include "pm_routed.h"

namespace pm {

hipError_t launch_grouped(const GroupedCall& C, int kind, hipStream_t st) {
    // rows per group if every expert had some: the groups' sizes are on the
    // device
    const int64_t groups = std::min(C.n_experts, C.n_rows);
    if (kind == kW16) {
        const int64_t xrows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
        if (C.n_rows >= 48 * groups && (xrows * C.ldx + C.cols) * 2 < 0xFFFFFFF0ll)
            return launch_grouped_tiles(C, C.n_rows < 160 * groups ? 128 : 256, st);
        return launch_grouped_stream16(C, C.n_rows <= 8 * groups ? 1 : 2, st);
    }
    // an fp32 row takes two columns
    if (C.x_type == PM_F32) return launch_grouped_stream4f(C, C.n_rows <= 4 * groups ? 1 : 2, st);
    return launch_grouped_stream4(C, C.n_rows <= 8 * groups ? 1 : 2, st);
}

}  // namespace pm

// Which kernel a grouped product of 8-bit weights and activations takes.
#include <algorithm>

#include "pm_fp8.h"

namespace pm {

hipError_t launch_grouped8(const GroupedCall& C, hipStream_t st) {
    const int64_t groups = std::min(C.n_experts, C.n_rows);
    const int64_t x_rows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
    const bool far = x_rows * C.ldx + C.cols >= 0xFFFFFFF0ll;
    if (C.n_rows >= 8 * groups && !far && C.cols > 0) {
        const int64_t tiles256 = (C.n_rows / 256) * int64_t((C.rows + 255) / 256);
        const bool big =
            (C.n_rows >= 224 * groups && tiles256 >= 2 * compute_units()) || !fp8_tiles128_fit(C);
        return launch_fp8_tiles(C, big ? 256 : 128, st);
    }
    return launch_fp8_stream(C, st);
}

}  // namespace pm

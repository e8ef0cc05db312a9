// Which kernel a grouped product takes.
#include <algorithm>

#include "pm_routed.h"

namespace pm {

// 16-bit weights are streamed while a group has few rows: measured on 128
// experts, us of the streamed kernel against 128-row tiles at 4, 8, 12 rows per
// group: 329/377, 406/413, 451/419 with 4096 inputs (2048 outputs); 16 experts,
// 2048 inputs, 1536 outputs: 28/34, 29/34, 33/34; with 1024 inputs (4096
// outputs) 160/148 already at 2 rows.  Tiles of 256 rows instead of 128 from 224
// rows per group on, where there are two for each compute unit: 353/359 us at
// 192 rows, 438/427 at 256, 760/726 at 512 (128 experts, 1024 inputs, 4096
// outputs), or where 128-row tiles' three stages leave no room in LDS for the
// table of experts (above some 3500).  The groups' sizes are on the device; these
// are rows per group if every expert had some.
//
// 4-bit weights: tiles decode them less often from 16 rows per group on: us of
// the streamed kernel against tiles at 12, 16, 32 rows, 16-bit activations:
// 193/228, 248/239, 403/276 (512 experts, 512 inputs, 4096 outputs); 92/107,
// 113/108, 178/119 (128 experts, 2048 x 2048); 74/63, 83/63, 113/66 (32 experts,
// 4096 inputs, 2048 outputs); 300/439, 387/449, 654/469 (256 of these); fp32:
// 288/328, 364/332, 661/404; 139/154, 170/164, 307/197; 87/85, 105/86, 162/97;
// 503/572, 622/619, 1128/692.  Where every workgroup has at most 4 blocks of 128
// inputs to do, tiles start sooner at any number of rows: 19/15 us at one row
// (128 experts, 256 inputs, 1024 outputs; fp32 19/18), 16/12 (16 experts, 512
// inputs, 1024 outputs; fp32 16/15); with 8 blocks (1024 inputs) 19/17, 17/23.
hipError_t launch_grouped(const GroupedCall& C, int kind, hipStream_t st) {
    const int64_t groups = std::min(C.n_experts, C.n_rows);
    const int64_t x_rows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
    const bool far = (x_rows * C.ldx + C.cols) * int64_t(type_bytes(C.x_type)) >= 0xFFFFFFF0ll;
    if (kind == kW4) {
        const int64_t blocks = (C.cols + 127) / 128, cus = compute_units();
        const int64_t rounds = (groups * ((C.rows + 255) / 256) + cus - 1) / cus;
        if (far || (C.n_rows < 16 * groups && blocks * rounds > 4))
            return C.x_type == PM_F32 ? launch_grouped_stream4f(C, st)
                                      : launch_grouped_stream4(C, st);
        return launch_grouped_tiles4(C, st);
    }
    if (int64_t(C.n_rows) * 512 <= C.cols * groups || far)
        return launch_grouped_stream16(C, st);
    const int64_t tiles256 = (C.n_rows / 256) * int64_t((C.rows + 255) / 256);
    const bool big =
        (C.n_rows >= 224 * groups && tiles256 >= 2 * compute_units()) || !tiles128_fit(C);
    return launch_grouped_tiles(C, big ? 256 : 128, st);
}

}  // namespace pm

// Which kernel a grouped product of 8-bit weights and activations takes.
#include <algorithm>

#include "pm_fp8.h"

namespace pm {

// Weights are streamed while a group has few rows.  Measured, us of the streamed
// kernel against 128-row tiles at 1, 2, 4, 8, 12, 16 rows per group; bf16 results
// (tiles of codes as they are), then fp32 (tiles of codes as halves, also those of
// bf16 results with fp32 sums):
//   128 experts, 256 inputs, 1024 outputs: 14/13 16/14 16/14 14/14 20/15 22/15;
//                                          14/16 16/16 17/17 15/17 20/18 22/19
//   64, 512, 4096:   21/21 28/26 30/27 33/28 40/28 52/29;  21/25 28/31 30/32 34/33 41/35 54/38
//   128, 1024, 4096: 66/64 90/87 104/101 110/105 136/108 174/110;
//                    66/71 90/96 107/112 119/116 144/121 183/125
//   16, 2048, 1536:  13/15 15/15 15/15 16/16 18/16 24/16;  13/24 15/24 15/24 16/24 18/24 24/25
//   128, 2048, 2048: 65/67 89/90 99/95 103/99 125/100 159/101;
//                    65/74 89/98 100/101 107/106 133/109 171/112
//   16, 4096, 2048:  24/25 27/25 31/25 32/29 36/29 46/29;  24/41 27/41 30/42 32/42 36/42 46/43
//   128, 4096, 2048: 116/146 165/199 184/227 192/237 223/238 280/239;
//                    116/158 164/212 185/234 196/244 234/246 296/249
//   32, 8192, 2048:  72/80 97/102 107/118 119/124 135/123 176/124;
//                    72/86 97/105 107/122 121/129 136/129 178/130
// Tiles from a 320th of the inputs (rows per group) on, at most 13; where no compute
// unit has a second tile, they take bf16 from 4 rows on.  Halves, converted
// anew for each tile, pay from 8 rows on, and from 16 where there is one tile
// each.  What the rule loses in the table: of bf16 calls 10 % at 4 rows of 8192 inputs
// (118 for 107, one tile each), 8 % at 2 rows of 16 experts of 4096 (27 for 25), 7 % at
// 12 rows of 128 experts of 4096 (238 for 223); of fp32 ones 13 % at 8 rows of 256
// inputs (17 for 15).
// Of bf16 results, tiles of 256 rows instead of 128 from 384 rows per group on,
// where there are two for each compute unit (128/256 us at 192, 256, 320, 384, 512,
// 1024 rows: 209/203 258/267 307/352 356/353 461/452 883/828, 128 experts of 4096 x
// 1024; 168/163 207/210 239/253 274/260 344/328 630/576, 64 of 2048 x 4096 with gate
// and up), or where 128-row tiles' three stages leave no room in LDS for the
// table of experts (above some 2000).  The rule counts tiles and not the rounds that
// the compute units take for them, and asking for two tiles each keeps 128 rows
// where 256 are faster by 10 to 19 %: 158/133 at 384 rows of 16 experts of 4096 x 4096
// (89/78 at 128), 133/120 127/109 139/113 at 256, 320, 384 of 8 of 4096 x 7168.  It
// loses less than 2 % where it takes 256 (370/375 at 512 rows of 256 of 1024 x 2048).
// The groups' sizes are on the device; these are rows per group if every expert had
// some.
hipError_t launch_grouped8(const GroupedCall& C, hipStream_t st) {
    const int64_t groups = std::min(C.n_experts, C.n_rows), cus = compute_units();
    const int64_t x_rows = C.flags & PM_GROUPED_GATHER ? (C.n_rows - 1) / C.top_k + 1 : 256;
    const bool far = x_rows * C.ldx + C.cols >= 0xFFFFFFF0ll;
    const bool glu = C.flags & PM_GROUPED_SWIGLU, bf16 = fp8_cuts_off(C);
    const int64_t out = glu ? C.rows / 2 : C.rows, per = glu ? 128 : 256;
    const bool one_each = groups * ((out + per - 1) / per) <= cus;
    int64_t from = std::min<int64_t>(C.cols / 320, 13);
    if (bf16)
        from = one_each ? std::min<int64_t>(from, 4) : from;
    else
        from = one_each ? 16 : std::max<int64_t>(from, 8);
    if (far || C.cols == 0 || C.n_rows < from * groups) return launch_fp8_stream(C, st);
    const int64_t tiles256 = (C.n_rows / 256) * int64_t((C.rows + 255) / 256);
    const bool big =
        (C.n_rows >= 384 * groups && tiles256 >= 2 * cus) || !fp8_tiles128_fit(C);
    return launch_fp8_tiles(C, big ? 256 : 128, st);
}

}  // namespace pm

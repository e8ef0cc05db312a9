// Which kernel a grouped product takes.
#include <algorithm>

#include "pm_routed.h"

namespace pm {

// 16-bit weights are streamed while a group has few rows.  Measured, us of the
// streamed kernel against 128-row tiles at 1, 2, 4, 8, 12, 16 rows per group, on
// more weights than the last cache holds where they are many:
//   128 experts, 256 inputs, 1024 outputs: 21/16 24/18 24/18 24/19 29/20 36/20
//   16, 512, 1024:    14/10 15/11 16/11 16/10 17/10 19/10
//   64, 512, 4096:    42/37 54/48 59/51 62/53 77/54 94/55
//   128, 1024, 4096:  137/125 178/162 204/180 210/190 240/193 332/196
//   16, 2048, 1536:   24/29 28/32 29/33 31/33 34/34 43/34
//   128, 2048, 2048:  132/154 171/200 188/221 192/232 214/234 289/237
//   16, 4096, 2048:   45/58 54/64 59/69 59/69 66/70 83/70
//   128, 4096, 2048:  262/265 315/356 362/407 376/426 406/430 562/432
// The rule (rows per group up to a 512th of the inputs) follows these from afar:
// at 512 and 1024 inputs it streams 1 and 2 rows that tiles do in 10 to 40 % less,
// and from 2048 inputs on it takes tiles at 8 to 12 rows that streaming does in 6
// to 20 % less.
// Tiles of 256 rows instead of 128 from 224 rows per group on, where there are two
// for each compute unit: 353/359 us at 192 rows, 438/427 at 256, 760/726 at 512
// (128 experts, 1024 inputs, 4096 outputs), or where 128-row tiles' three stages
// leave no room in LDS for the table of experts (above some 3500).  The groups'
// sizes are on the device; these are rows per group if every expert had some.
//
// 4-bit weights: tiles decode them less often, which pays from about 16 rows per
// group on: us of the streamed kernel against tiles at 12, 16, 20, 32 rows, zero
// points, bf16 activations, then fp32:
//   512 experts, 512 inputs, 4096 outputs: 189/231 239/244 289/257 395/284;
//                       286/300 359/319 398/339 590/384
//   512, 4096, 512:     196/222 244/225 298/228 406/239; 302/275 377/292 451/303 679/344
//   256, 4096, 2048:    313/433 393/438 477/440 663/455; 516/526 645/557 773/576 1169/654
//   128, 2048, 2048:    96/107 118/109 139/111 180/118; 137/151 169/154 199/161 292/177
//   64, 4096, 4096:     164/221 209/224 248/225 336/232; 261/270 322/283 381/293 575/329
//   32, 4096, 2048:     72/62 82/63 91/63 114/66; 85/80 103/79 119/81 170/95
//   16, 2048, 2048:     30/31 32/31 34/32 39/33; 30/41 35/43 38/43 58/48
//   8, 1024, 2048:      22/18 24/19 24/19 26/21; 21/23 22/25 23/25 27/28
// At 16 rows the rule loses 7 to 11 % on the largest bf16 products, and on small
// fp32 ones as much as 24 %, up to 20 rows.  Where every workgroup has at most 4
// blocks of 128 inputs to do, tiles start sooner: at 1, 8, 16 rows 19/14, 25/16,
// 38/17 us (128 experts, 256 inputs, 1024 outputs; fp32 18/16, 30/18, 35/20), 12/12,
// 18/13, 21/14 (16 experts, 512 inputs, 1024 outputs; fp32 12/14, 17/15, 19/17).
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

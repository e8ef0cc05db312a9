// Routed experts on the device: the router, the products grouped by expert,
// the combine and the 4-bit encoder (pm_route.hip, pm_grouped.hip,
// pm_combine.hip; entry points in pm_routed.cpp).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pm.h"

namespace pm {

inline size_t type_bytes(int t) { return t == PM_F32 ? 4 : 2; }

// ---------------------------------------------------------------- router
struct RouteCall {
    const void* logits;            // [n_tokens] rows of n_experts, ld apart
    int64_t ld;
    int32_t* ids;
    float* w;
    int32_t* offsets;              // null: no sorting
    int32_t* order;
    uint16_t* hist;                // workspace [blocks][hist_stride]
    int32_t hist_stride;           // n_experts, rounded up to 8
    int32_t n_tokens, n_experts, top_k, type;
    int32_t block_tokens, n_blocks;   // tokens per histogram block, blocks
};
// Tokens of one histogram block and the number of blocks.
void route_blocks(int n_tokens, int* block_tokens, int* n_blocks);
hipError_t launch_route(const RouteCall& C, hipStream_t st);

// ---------------------------------------------------------------- grouped products
enum { kW16 = 0, kW4 = 1 };
struct GroupedCall {
    const void* w;                 // 16-bit weights, or packed 4-bit codes
    const uint16_t* scales;        // 4-bit: fp16, one per group of inputs
    const uint8_t* zeros;          // 4-bit: zero points (null: 8)
    const void* x;
    void* y;
    const int32_t* offsets;
    const int32_t* order;
    int64_t ldx, ldy;
    int32_t n_experts, rows, cols, group;
    int32_t n_rows, top_k;
    int32_t w_type, x_type, y_type;   // w_type: PM_F16 / PM_BF16 (16-bit weights)
    uint32_t flags;
};
// Experts of one call (the kernels keep a table of them in LDS).
constexpr int kMaxGroupedExperts = PM_GROUPED_MAX_EXPERTS;
hipError_t launch_grouped(const GroupedCall& C, int kind, hipStream_t st);
// Tiles of `rows` (128 or 256) x 256 (pm_grouped_tile.hip), 16-bit weights; the
// offsets of a tile's rows in x must fit 32 bits.
hipError_t launch_grouped_tiles(const GroupedCall& C, int rows, hipStream_t st);
// Whether the table of experts lies in LDS beside the stages of 128-row tiles
// (beside those of 256 rows it always does).
bool tiles128_fit(const GroupedCall& C);
// Tiles of 128 (fp32 activations: 64) x 256 with 4-bit weights
// (pm_grouped_tile4.hip); the same limit.
hipError_t launch_grouped_tiles4(const GroupedCall& C, hipStream_t st);
// Weights streamed past 16 columns of activations (pm_grouped_stream.h): 16-bit
// weights, 4-bit weights with 16-bit and with fp32 activations; any sizes.
hipError_t launch_grouped_stream16(const GroupedCall& C, hipStream_t st);
hipError_t launch_grouped_stream4(const GroupedCall& C, hipStream_t st);
hipError_t launch_grouped_stream4f(const GroupedCall& C, hipStream_t st);

// Compute units of the current device.
int compute_units();
// Lets a kernel take up to `bytes` of dynamic LDS on the current device; `done`
// holds a bit for every device where it may, one word per kernel.
constexpr int kTileMaxLds = 160 * 1024 - 1024;
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>* done);

// ---------------------------------------------------------------- 4-bit encoder, combine
hipError_t launch_encode_w4(size_t n_groups, int group, const void* w, int type, uint8_t* q,
                            uint16_t* scales, uint8_t* zeros, hipStream_t st);
hipError_t launch_combine_uses(int n_tokens, int top_k, int hidden, const void* z, int z_type,
                               int64_t ldz, const float* w, void* y, int y_type, int64_t ldy,
                               hipStream_t st);

}  // namespace pm

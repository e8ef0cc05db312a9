// Products grouped by expert for groups of few rows: the kernel's template,
// instantiated for 16-bit weights in pm_grouped_stream16.hip and for 4-bit
// weights in pm_grouped_stream4.hip and pm_grouped_stream4f.hip.
//
//   D[v][o] = sum_k x[v][k] W[o][k]   (v_mfma_f32_16x16x32, fp32 sums)
//
// Bound by reading the weights, so they go from memory to the matrix cores
// through registers, once, and everything else stays out of the way.
//
// A workgroup of NW waves works on row tiles, 16 rows of one expert's matrix
// (8 gate and 8 up rows under PM_GROUPED_SWIGLU), for up to 16 columns v of
// activations.  KW waves split the inputs, the other factor of NW splits the
// row tiles.  A wave's share of the inputs, KB blocks of 128, stays in
// registers as matrix operands while the row tiles pass: a row tile costs the
// wave one 16-byte load per lane and 1 KiB, one product each (4-bit: 4) and
// nothing from LDS.  The loads of the next row tiles are in flight while one
// is multiplied.  The waves' sums meet in LDS after a chunk of 4 to 16 row
// tiles per wave, as many as LDS holds (one barrier), and are added in a fixed
// order.  The code that runs once per group of rows is kept small: a call that
// lasts 15 us fetches every instruction from memory once.
//
// The row tiles of all groups form one sequence, of which every workgroup
// takes an equal, contiguous part.
//
// 4-bit weights: a lane's 16 bytes are 32 adjacent inputs of one row.  Pairs
// of codes become pairs of halves by an AND and an OR with an exponent (1024
// + q and 64 + q), and q - z by one exact packed subtraction; the group's
// scale multiplies the fp32 sum of the group's products.  A product sums over
// the 4 x 8 inputs of 4 lanes; where a group is a multiple of 128 inputs these
// are 4 pieces of it, else a 4 x 4 exchange of words between the lanes (four
// v_permlane swaps) makes them 32 adjacent inputs.
//
// Activations meet 4-bit weights as fp16; bf16 and fp32 are scaled by a power
// of two per row and wave so that the largest lies in [2^14, 2^15): a bf16
// value loses at most 2^-39 of the largest, below fp16's normal range.  An fp32
// row takes two columns, its value rounded to fp16 and the rest (times 2^11)
// rounded again: off by 2^-23 of the value, or 2^-50 of the largest.  The waves convert a few columns at a time into LDS and
// take their operands from there.
//
// Measured: 80 rows over 512 experts, 2048 x 4096 fp16 with gate and up: 218 to
// 232 us, 5.4 to 5.7 TB/s (of 6.2 that a plain elementwise kernel reaches).  4-bit:
// 640 rows over 512 experts, 4096 x 1024 with zero points, bf16: 164 to 170 us,
// 4.9 TB/s; 10 rows of fp32, 2048 x 4096 with gate and up: 20 us for 43 MB, of
// which the stream takes 9 (a fifth more than equal shares: 128 row tiles of a
// group over 25 workgroups are up to 6 each, and 6 workgroups have none, where the
// mean is 5) and finding the groups, converting x and the last sums the rest.
// More than 4096 inputs take panels, and x is loaded (4-bit: converted) anew for
// every 4 row tiles of a wave.  256 experts, 2048 outputs, top-8, bf16, at 4096,
// 5120, 7168, 8192 inputs: 8 tokens 178, 290, 348, 351 us (5.4, 4.2, 4.8, 5.5 TB/s),
// 64 tokens 616, 1075, 1313, 1297; 4-bit 60, 132, 140, 146 (4.1, 2.4, 3.1, 3.4) and
// 190, 637, 661, 685; 4-bit with fp32 x 61, 146, 154, 161 and 203, 758, 777, 807.
// (5120 and 7168 inputs fill two panels of 4096 only in part.)
// The decoding, repeated for every 16 columns, bounds 4-bit calls of more rows:
// 64 experts of 4096 x 4096 with 32, 64, 128 bf16 rows each take 261, 500, 997
// us here, which is why tiles take over from some 16 rows on.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_grouped_codes.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

// How a call is split: waves over the inputs (KW = 1 << kw_log), panels of
// KW * KB * 128 inputs, row tiles of a matrix.
struct StreamPlan {
    int kw_log, panels, row_tiles;
};

namespace {

constexpr int kSteps = 4;                       // row tiles of an unrolled group
// Inclusive sum over the wave.
__device__ inline int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);    // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);    // row_shr 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);    // row_shr 4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);    // row_shr 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);    // row_bcast 15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);    // row_bcast 31
    return v;
}

// The tiles of MTILE (a power of two) sorted rows of all experts, by one wave without LDS: a
// lane holds the count of its run of `per` adjacent experts and of those
// before.
struct TileScan {
    int before, mine, total, per;
};

// 8 adjacent experts' offsets, loaded together.
struct Eight {
    int o[9];
};
__device__ inline Eight load_eight(const GroupedCall& C, int e) {
    Eight r;
#pragma unroll
    for (int k = 0; k < 9; ++k) r.o[k] = C.offsets[min(e + k, C.n_experts)];
    return r;
}
// First row and rows of expert e + k of them, none from `end` on.
__device__ inline RowRange range_of(const GroupedCall& C, const Eight& s, int e, int k, int end) {
    RowRange r = row_range(C, s.o[k], s.o[k + 1]);
    if (e + k >= end) r.n = 0;
    return r;
}

template <int MTILE>
__device__ inline TileScan scan_tiles(const GroupedCall& C, Eight* first) {
    const int lane = threadIdx.x & 63;
    TileScan s;
    s.per = (C.n_experts + kWave - 1) / kWave;
    const int e0 = lane * s.per, e1 = min(e0 + s.per, C.n_experts);
    s.mine = 0;
    for (int b = 0; b < s.per; b += 8) {
        const Eight o = load_eight(C, e0 + b);
        if (b == 0) *first = o;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s.mine += (range_of(C, o, e0 + b, k, e1).n + MTILE - 1) / MTILE;
    }
    const int incl = wave_scan(s.mine);
    s.before = incl - s.mine;
    s.total = most_tiles(C, MTILE, __builtin_amdgcn_readlane(incl, 63));
    return s;
}

// Row tile i < total: its expert, first row and rows, the same in every lane.
// `known`: the lanes' first 8 experts, where they are at hand.
struct TileRows {
    int e, row0, n;
};
template <int MTILE>
__device__ inline TileRows find_tile_rows(const GroupedCall& C, const TileScan& s, int i,
                                          const Eight* known) {
    const int lane = threadIdx.x & 63;
    const int e0 = lane * s.per, e1 = min(e0 + s.per, C.n_experts);
    const uint64_t hit = __ballot(i >= s.before && i < s.before + s.mine);
    TileRows r{0, 0, 0};
    if (!hit) return r;                                   // (bad offsets only)
    int at = s.before;
    for (int b = 0; b < s.per; b += 8) {
        const Eight o = known && b == 0 ? *known : load_eight(C, e0 + b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const RowRange g = range_of(C, o, e0 + b, k, e1);
            const int tiles = (g.n + MTILE - 1) / MTILE;
            if (i >= at && i < at + tiles) {
                const int skip = (i - at) * MTILE;
                r.e = e0 + b + k;
                r.row0 = g.row0 + skip;
                r.n = min(g.n - skip, MTILE);
            }
            at += tiles;
        }
    }
    const int l = __builtin_ctzll(hit);
    r.e = __builtin_amdgcn_readlane(r.e, l);
    r.row0 = __builtin_amdgcn_readlane(r.row0, l);
    r.n = __builtin_amdgcn_readlane(r.n, l);
    return r;
}

struct F8 {
    float v[8];
};
// Eight activations at p, and whether they count (p can be read in any case).
template <bool X32>
struct RawX {
    u32x4 d[X32 ? 2 : 1];
};
template <bool X32>
__device__ inline F8 widen(const RawX<X32>& x, bool bf16) {
    F8 r;
    if constexpr (X32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = __uint_as_float(x.d[i >> 2][i & 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = x.d[0][i];
            r.v[2 * i] = bf16 ? __uint_as_float(w << 16) : half_bits(w);
            r.v[2 * i + 1] = bf16 ? __uint_as_float(w & 0xFFFF0000u) : half_bits(w >> 16);
        }
    }
    return r;
}

template <int CTRL, int ROW_MASK>
__device__ inline float dpp_fmax(float v) {
    const int b = __builtin_bit_cast(int, v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, ROW_MASK, 0xF,
                                                                         false)));
}
__device__ inline float wave_fmax(float v) {
    v = dpp_fmax<0xB1, 0xF>(v);
    v = dpp_fmax<0x4E, 0xF>(v);
    v = dpp_fmax<0x141, 0xF>(v);
    v = dpp_fmax<0x140, 0xF>(v);
    v = dpp_fmax<0x142, 0xA>(v);
    v = dpp_fmax<0x143, 0xC>(v);
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Halves, rounded to nearest even, in the order of codes_to_f16.
__device__ inline u32x4 pack_codes(const _Float16* h) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = uint32_t(__builtin_bit_cast(uint16_t, h[i])) |
               uint32_t(__builtin_bit_cast(uint16_t, h[i + 4])) << 16;
    return r;
}

// Where the sum of column v lies in a row tile's [columns][16] of LDS: the 4
// columns that a lane holds are turned against those of its neighbours, so
// that a wave's writes fall in distinct banks.
__device__ inline int sum_at(int v) { return (v >> 2) * 64 + (((v & 3) + (v >> 2)) & 3) * 16; }

// f(0), .., f(N - 1) with constant arguments.
template <int N, int I = 0, class F>
__device__ inline void steps_to(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        steps_to<N, I + 1>(f);
    }
}

template <int KIND, bool BF16, bool X32, int NW, int KB, int GM, bool ZEROS>
__global__ __launch_bounds__(NW * kWave, 2) void stream_kernel(const GroupedCall C,
                                                               const StreamPlan P) {
#ifdef __HIP_DEVICE_COMPILE__
    // 16-byte loads of a row tile per lane, and scales: one per block where a
    // group covers it, else one per 32 inputs
    constexpr int kLoads = KIND == kW4 ? KB : KB * 4;
    constexpr int kUnits = KIND != kW4 ? 0 : GM == kGroup128 ? KB : GM == kGroup64 ? KB * 2 : KB * 4;
    constexpr bool kWhole = GM == kGroup128;
    // row tiles held in registers: one at work, the others on their way
    // (as many as 256 registers hold beside the activations)
    constexpr int kSlots = GM == kAnyGroup || (GM == kGroup32 && KB == 4) || kLoads > 8 ? 2 : 4;
    constexpr int kThreads = NW * kWave, kLogNW = NW == 8 ? 3 : 2;
    // sums of a chunk: [buffer][wave][row tile][column of x][16], room
    // for 4 row tiles of all columns; the buffer to be filled next holds the
    // converted activations before
    constexpr int kPart = kSteps * 256;
    __shared__ __attribute__((aligned(16))) float part[2][NW][kPart];
    __shared__ float xscale[16][NW];
    __shared__ int use_row[2][16];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const int kw = 1 << P.kw_log, rw = NW >> P.kw_log;
    const int ks = wv & (kw - 1), rg = wv >> P.kw_log;
    const bool glu = C.flags & PM_GROUPED_SWIGLU, gather = C.flags & PM_GROUPED_GATHER;
    const int out = glu ? C.rows / 2 : C.rows;
    const int per_tile = glu ? 8 : 16;

    // a short call's uses are loaded along with the offsets
    const bool few = C.n_rows <= kWave;
    const int u_few = few && lane < C.n_rows ? use_of(C, lane) : -1;
    Eight eight;
    // sorted rows of a tile: an fp32 row takes two columns
    constexpr int kTileRows = X32 ? 8 : 16;
    const TileScan scan = scan_tiles<kTileRows>(C, &eight);
    // Few groups: a whole number of workgroups each, which costs up to 1 part
    // in 8 of the workgroups but no workgroup prepares two groups' rows
    // (that takes as long as some 6 row tiles of 32 KiB).  Else equal parts of
    // the sequence.
    const int wps = scan.total > 0 ? int(gridDim.x) / scan.total : 0;
    const bool apart = wps >= 8;
    // row tiles of the sequence, this workgroup's first and their number: the
    // group mt, the row tile rt0 in it
    int mt, rt0, left;
    if (apart) {
        mt = int(blockIdx.x) / wps;
        const int k = int(blockIdx.x) - mt * wps;
        rt0 = int(int64_t(P.row_tiles) * k / wps);
        left = mt < scan.total ? int(int64_t(P.row_tiles) * (k + 1) / wps) - rt0 : 0;
    } else {
        const uint64_t all = uint64_t(scan.total) * P.row_tiles;
        const uint32_t b = blockIdx.x, n = gridDim.x;
        uint64_t pos;
        if (all >> 31 == 0) {                             // (64-bit divisions are long)
            const uint32_t q0 = uint32_t(all) / n, rest = uint32_t(all) - q0 * n;
            pos = q0 * b + min(b, rest);
            left = int(q0) + (b < rest ? 1 : 0);
            mt = int(uint32_t(pos) / uint32_t(P.row_tiles));
        } else {
            pos = all / n * b + min(uint64_t(b), all % n);
            left = int(all / n) + (b < all % n ? 1 : 0);
            mt = int(pos / P.row_tiles);
        }
        rt0 = int(pos - uint64_t(mt) * P.row_tiles);
    }
    if (left <= 0) return;
    TileRows g = find_tile_rows<kTileRows>(C, scan, mt, &eight);

    const uint32_t row_bytes = KIND == kW4 ? uint32_t(C.cols) / 2 : uint32_t(C.cols) * 2;
    const size_t w_bytes = size_t(C.rows) * row_bytes;
    const int ng = KIND == kW4 ? C.cols / C.group : 0;
    const CodeBits bits = code_bits();
    int buf = 0, seg = 0;
    for (;;) {
        const int rt1 = min(P.row_tiles, rt0 + left);
        left -= rt1 - rt0;
        // loads return in order: the uses come before any weights
        int u_lane = __shfl(u_few, (g.row0 + lane) & 63);
        if (!few && lane < g.n) u_lane = use_of(C, g.row0 + lane);
        u_lane = lane < g.n ? u_lane : -1;

        const auto wbuf = __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<char*>(static_cast<const char*>(C.w)) + size_t(g.e) * w_bytes), 0,
            int(uint32_t(w_bytes)), kRawBuffer);
        const auto sbuf = __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<uint16_t*>(C.scales) + size_t(g.e) * C.rows * ng), 0,
            int(uint32_t(C.rows) * uint32_t(ng) * 2), kRawBuffer);
        const auto zbuf = __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<uint8_t*>(C.zeros) + size_t(g.e) * C.rows * ng), 0,
            int(uint32_t(C.rows) * uint32_t(ng)), kRawBuffer);

        // ---- the stream of row tiles: chunk by chunk, panel by panel
        u32x4 w[kSlots][kLoads];
        uint32_t sc[kSlots][kUnits > 0 ? (kUnits + 1) / 2 : 1];
        uint32_t zp[kSlots][kUnits > 0 ? (kUnits + 3) / 4 : 1];
        auto weight_row = [&](int rt) {
            int o = rt * per_tile + (glu ? i16 & 7 : i16);
            const bool ok = rt < rt1 && o < out;
            if (glu && i16 >= 8) o += out;
            return ok ? o : -1;
        };
        auto first_block = [&](int panel) { return (panel * kw + ks) * KB; };
        // loads of a row tile, in one order on every path
        auto issue = [&](auto slot, int rt, int panel) {
            constexpr int S = decltype(slot)::value;
            const int row = weight_row(rt);
            const int kb = first_block(panel);
            const bool some = row >= 0 && kb * 128 < C.cols;
            const uint32_t at = chosen(
                some, uint32_t(row) * row_bytes + kb * (KIND == kW4 ? 64 : 256) + q * 16);
            // 16 bytes: the 32 inputs of a block's quarter q, or 8 inputs of
            // each quarter.  Past `cols` they are the next row's: see multiply
#pragma unroll
            for (int s = 0; s < kLoads; ++s)
                w[S][s] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(wbuf, at + s * 64, 0, 2));
            if constexpr (KIND == kW4) {
                constexpr int U = kUnits;
                if constexpr (GM == kAnyGroup) {
#pragma unroll
                    for (int s = 0; s < U; ++s) {
                        const int c = kb * 128 + s * 32;
                        const uint32_t g0 = uint32_t(row) * ng + c / C.group;
                        const bool in = row >= 0 && c < C.cols;
                        const uint32_t v = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(
                            sbuf, chosen(in, g0 * 2), 0, 0));
                        sc[S][s / 2] = s & 1 ? sc[S][s / 2] | v << 16 : v;
                        if constexpr (ZEROS) {
                            const uint32_t z = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(
                                zbuf, chosen(in, g0), 0, 0));
                            zp[S][s / 4] = s & 3 ? zp[S][s / 4] | z << (8 * (s & 3)) : z;
                        }
                    }
                } else {
                    const uint32_t g0 = uint32_t(row) * ng + uint32_t(kb) * (128 / GM);
                    const uint32_t so = chosen(some, g0 * 2), zo = chosen(some, g0);
                    if constexpr (U == 1) {
                        sc[S][0] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sbuf, so, 0, 0));
                        if constexpr (ZEROS)
                            zp[S][0] = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(zbuf, zo, 0, 0));
                    } else if constexpr (U == 2) {
                        sc[S][0] = __builtin_amdgcn_raw_buffer_load_b32(sbuf, so, 0, 0);
                        if constexpr (ZEROS)
                            zp[S][0] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(zbuf, zo, 0, 0));
                    } else {
#pragma unroll
                        for (int s = 0; s < U; s += 4) {
                            const u32x2 v = __builtin_bit_cast(
                                u32x2, __builtin_amdgcn_raw_buffer_load_b64(sbuf, so + s * 2, 0, 0));
                            sc[S][s / 2] = v[0];
                            sc[S][s / 2 + 1] = v[1];
                            if constexpr (ZEROS)
                                zp[S][s / 4] = __builtin_amdgcn_raw_buffer_load_b32(zbuf, zo + s, 0, 0);
                        }
                    }
                }
            }
        };

        auto issue_step = [&](auto slot, int c, int step, int panel) {
            // c row tiles on from row tile `step` of this wave in `panel`; past
            // the group, of the panel or group after it
            if (c >= kSteps) {
                c -= kSteps;
                if (++panel == P.panels) {
                    panel = 0;
                    step += kSteps;
                }
            }
            issue(slot, rt0 + (step + c) * rw + rg, panel);
        };
        issue(std::integral_constant<int, 0>{}, rt0 + rg, 0);

        // ---- activations of this wave's inputs, as matrix operands.  Column v
        // is row v, or the value (even v) or rest (odd v) of fp32 row v / 2
        const int nv = X32 ? 2 * g.n : g.n;
        int vlog = 2;
        while ((1 << vlog) < nv) ++vlog;
        if (wv == 0 && lane < g.n)
            use_row[seg][lane] =
                u_lane < 0 ? -1 : (C.flags & PM_GROUPED_SCATTER ? u_lane : g.row0 + lane);
        u32x4 xf[KB * 4];
        float xs[4];                                       // of columns 4q + r
        // row r of x (any row where r is not a row of the group)
        auto x_row = [&](int u, int r) {
            const int64_t xr = u < 0 ? 0 : gather ? u / C.top_k : g.row0 + r;
            return static_cast<const char*>(C.x) + xr * C.ldx * (X32 ? 4 : 2);
        };
        // kRaw rows of x from row rb on, this lane's 8 inputs of the panel
        constexpr int kRaw = KIND != kW4 ? 1 : X32 ? 2 : 4;
        RawX<X32> raw[kRaw];
        auto load_raw = [&](int panel, int rb) {
            const int c = first_block(panel) * 128 + lane * 8;
            const bool in = rg == 0 && lane < KB * 16 && c < C.cols;
#pragma unroll
            for (int k = 0; k < kRaw; ++k) {
                const int r = min(rb + k, g.n - 1);
                const int u = __builtin_amdgcn_readlane(u_lane, r);
                const char* p = x_row(u, r) + size_t(max(min(c, C.cols - 8), 0)) * (X32 ? 4 : 2);
#pragma unroll
                for (int h = 0; h < (X32 ? 2 : 1); ++h) {
                    const u32x4 d = *reinterpret_cast<const u32x4*>(p + 16 * h);
                    raw[k].d[h] = in && u >= 0 ? d : u32x4{0, 0, 0, 0};
                }
            }
        };
        // (first: the first rows of panel 0 are in `raw` already)
        auto load_x = [&](int panel, bool first) {
            const int c0 = first_block(panel) * 128;       // the wave's inputs
            if constexpr (KIND != kW4) {
                const int u = __shfl(u_lane, i16);
                const char* p = x_row(u, i16);
                int c = c0 + q * 8;
                asm volatile("" : "+v"(c));                // (addresses are not kept)
#pragma unroll
                for (int f = 0; f < KB * 4; ++f) {
                    const bool ok = u >= 0 && c + f * 32 < C.cols;
                    const u32x4 d = *reinterpret_cast<const u32x4*>(
                        p + size_t(max(min(c + f * 32, C.cols - 8), 0)) * 2);
                    xf[f] = ok ? d : u32x4{0, 0, 0, 0};
                }
            } else {
                // vper columns at a time: halves [column][inputs of the panel]
                char* const stage = reinterpret_cast<char*>(&part[buf][0][0]);
                const int width = KB * 128 << P.kw_log;
                const int vper = min(1 << vlog, NW * kPart * 2 / width);
                const int rper = X32 ? vper >> 1 : vper;
                const bool bf16 = C.x_type == PM_BF16;
                const bool scaled = X32 || bf16;
                for (int v0 = 0; v0 < nv; v0 += vper) {
                    const int r0 = X32 ? v0 >> 1 : v0, r1 = min(r0 + rper, g.n);
#pragma unroll 1
                    for (int rb = r0; rg == 0 && rb < r1; rb += kRaw) {
                        if (!(first && rb == 0)) load_raw(panel, rb);
#pragma unroll 1
                        for (int r = rb; r < min(rb + kRaw, r1); ++r) {
                            const F8 x = widen<X32>(raw[0], bf16);
#pragma unroll
                            for (int k = 0; k + 1 < kRaw; ++k) raw[k] = raw[k + 1];
                            const int v = X32 ? 2 * r : r;
                            float up = 1.0f, down = 1.0f;
                            if (scaled) {
                                float big = 0.0f;
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    big = fabsf(x.v[i]) < INFINITY ? fmaxf(big, fabsf(x.v[i])) : big;
                                big = wave_fmax(big);
                                // 2^e brings the largest to [2^14, 2^15)
                                const int e = min(
                                    max(14 - (int(__float_as_uint(big) >> 23) - 127), -113), 126);
                                up = __uint_as_float(uint32_t(127 + e) << 23);
                                down = __uint_as_float(uint32_t(127 - e) << 23);
                            }
                            _Float16 hi[8], lo[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float s = x.v[i] * up;
                                hi[i] = _Float16(s);
                                const float back = float(hi[i]);
                                lo[i] = fabsf(back) < INFINITY ? _Float16((s - back) * 2048.0f)
                                                               : _Float16(0.0f);
                            }
                            char* at = stage + (size_t(v - v0) * width + (ks * KB * 128) + lane * 8) * 2;
                            if (lane < KB * 16) {
                                *reinterpret_cast<u32x4*>(at) = pack_codes(hi);
                                if constexpr (X32)
                                    *reinterpret_cast<u32x4*>(at + size_t(width) * 2) = pack_codes(lo);
                            }
                            if (lane == 0) {
                                xscale[v][ks] = down;
                                if constexpr (X32) xscale[v + 1][ks] = down * (1.0f / 2048.0f);
                            }
                        }
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    // (a column without a row takes another's operands; its sums
                    // are not used)
                    const int v = i16 - v0;
                    const char* p = stage + (size_t(v & (vper - 1)) * width + ks * KB * 128 +
                                             (kWhole ? q * 32 : q * 8)) * 2;
                    if (v0 == 0 || (v >= 0 && v < vper)) {
#pragma unroll
                        for (int f = 0; f < KB * 4; ++f)
                            xf[f] = *reinterpret_cast<const u32x4*>(
                                p + ((f >> 2) * 128 + (f & 3) * (kWhole ? 8 : 32)) * 2);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) xs[r] = xscale[4 * q + r][ks];
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                }
            }
        };
        if constexpr (KIND == kW4) {
            if (C.cols > 0) load_raw(0, 0);
        }
        steps_to<kSlots - 2>([&](auto c) {
            issue(std::integral_constant<int, c + 1>{}, rt0 + (c + 1) * rw + rg, 0);
        });

        auto multiply = [&](auto slot, int panel, f32x4& a) {
            constexpr int S = decltype(slot)::value;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            if constexpr (KIND == kW4) {
                const int c0 = first_block(panel) * 128;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    __builtin_amdgcn_sched_barrier(0);
                    const u32x4 c = kWhole ? w[S][b] : exchange(w[S][b]);
                    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        constexpr int kPer = kWhole ? 4 : GM == kGroup64 ? 2 : 1;
                        const int unit = (b * 4 + j) / kPer;
                        f16x2 za = {_Float16(1032.0f), _Float16(1032.0f)};
                        f16x2 zb = {_Float16(72.0f), _Float16(72.0f)};
                        if constexpr (ZEROS) {
                            const uint32_t z = zp[S][unit / 4] >> (8 * (unit & 3)) & 255u;
                            za = __builtin_bit_cast(f16x2, 0x64006400u | z | z << 16);
                            zb = za - f16x2{_Float16(960.0f), _Float16(960.0f)};
                        }
                        const u32x4 wf = codes_to_f16(bits, c[j], za, zb);
                        d = mfma_x_w<false>(xf[b * 4 + j], wf,
                                            j % kPer == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : d);
                        if (j % kPer == kPer - 1) {
                            // past the last input there is no scale of this row
                            const bool in = c0 + b * 128 + (kWhole ? 0 : j / kPer * kPer * 32) < C.cols;
                            const float sf =
                                in ? half_bits(sc[S][unit / 2] >> (16 * (unit & 1))) : 0.0f;
#pragma unroll
                            for (int r = 0; r < 4; ++r) sum[r] = fmaf(d[r], sf, sum[r]);
                        }
                    }
                }
            } else {
                // weights past the last input are of another row, and may be
                // infinite: 0 in their place
                const int c0 = first_block(panel) * 128;
                if (c0 + KB * 128 > C.cols) {
#pragma unroll
                    for (int f = 0; f < kLoads; ++f)
                        if (c0 + f * 32 + q * 8 >= C.cols) w[S][f] = u32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int f = 0; f < kLoads; ++f) sum = mfma_x_w<BF16>(xf[f], w[S][f], sum);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                a[r] = KIND == kW4 ? fmaf(sum[r], xs[r], a[r]) : a[r] + sum[r];
        };

        f32x4 acc[kSteps];
        int nlog = 0;
        while ((1 << nlog) < g.n) ++nlog;
        const int plog = glu ? 3 : 4;
        // row tiles of a wave per chunk, and floats of one
        const int clog = P.panels > 1 ? 2 : min(4, 6 - vlog);
        const int tile_floats = 16 << vlog;
        if (C.cols > 0) load_x(0, true);
        bool first = true;
        for (int rtb = rt0, step = 0; rtb < rt1; rtb += rw << clog) {
            int here = 0;                                  // row tiles of the chunk so far
            do {
#pragma unroll
                for (int c = 0; c < kSteps; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
                for (int panel = 0; panel < P.panels; ++panel) {
                    if (P.panels > 1 && !first) load_x(panel, false);
                    first = false;
                    steps_to<kSteps>([&](auto c) {
                        constexpr int kNext = (c + kSlots - 1) % kSlots;
                        issue_step(std::integral_constant<int, kNext>{}, c + kSlots - 1, step, panel);
                        __builtin_amdgcn_sched_barrier(0);
                        if (C.cols > 0 && rt0 + (step + c) * rw + rg < rt1)
                            multiply(std::integral_constant<int, c % kSlots>{}, panel, acc[c]);
                        // registers: a row tile's decoded weights live in its own step
                        __builtin_amdgcn_sched_barrier(0);
                    });
                }
                if (4 * q < 1 << vlog) {
#pragma unroll
                    for (int c = 0; c < kSteps; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            part[buf][wv][(here + c) * tile_floats + sum_at(4 * q + r) + i16] =
                                acc[c][r];
                }
                here += kSteps;
                step += kSteps;
            } while (here < 1 << clog && rtb + here * rw < rt1);
            // LDS only: the weights under way are not waited for
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // 4 adjacent outputs of a row per thread
            const int items = (rw << clog) << (nlog + plog - 2);
#pragma unroll 1
            for (int it = threadIdx.x; it < items; it += kThreads) {
                const int col = (it & ((1 << plog) / 4 - 1)) * 4;
                const int r = (it >> (plog - 2)) & ((1 << nlog) - 1), t = it >> (plog - 2 + nlog);
                const int rt = rtb + t, o = rt * per_tile + col;
                if (r >= g.n || rt >= rt1 || o >= out) continue;
                const int yr = use_row[seg][r];
                if (yr < 0) continue;
                const int v = X32 ? 2 * r : r;
                const float* p = &part[buf][(t & (rw - 1)) << P.kw_log]
                                      [(t >> (kLogNW - P.kw_log)) * tile_floats + col];
                const int a0 = sum_at(v), a1 = sum_at(v + 1);
                f32x4 p0 = {0.f, 0.f, 0.f, 0.f}, p1 = p0;
#pragma unroll 2
                for (int k = 0; k < kw; ++k, p += kPart) {
                    p0 += *reinterpret_cast<const f32x4*>(p + a0);
                    if constexpr (X32) p0 += *reinterpret_cast<const f32x4*>(p + a1);
                    if (glu) {
                        p1 += *reinterpret_cast<const f32x4*>(p + a0 + 8);
                        if constexpr (X32) p1 += *reinterpret_cast<const f32x4*>(p + a1 + 8);
                    }
                }
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = glu ? silu_up(p0[i], p1[i]) : p0[i];
                const int64_t at = int64_t(yr) * C.ldy + o;
                if (C.y_type == PM_F32) store4<PM_F32>(C.y, at, out - o, y);
                else if (C.y_type == PM_F16) store4<PM_F16>(C.y, at, out - o, y);
                else store4<PM_BF16>(C.y, at, out - o, y);
            }
            buf ^= 1;
        }
        seg ^= 1;
        if (left <= 0) break;
        rt0 = 0;
        g = find_tile_rows<kTileRows>(C, scan, ++mt, nullptr);
    }
#endif
}

template <int KIND, bool BF16, bool X32, int NW, int KB, int GM, bool ZEROS>
hipError_t run_stream(const GroupedCall& C, const StreamPlan& P, hipStream_t st) {
    const int64_t tiles = int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / (X32 ? 8 : 16);
    const int64_t most = int64_t(compute_units()) * (8 / NW);
    hipLaunchKernelGGL((stream_kernel<KIND, BF16, X32, NW, KB, GM, ZEROS>),
                       dim3(unsigned(std::min<int64_t>(tiles * P.row_tiles, most))),
                       dim3(NW * kWave), 0, st, C, P);
    return hipGetLastError();
}

// The split of the inputs: 4 blocks of 128 per wave where there are as many.
// Up to 4 waves cover 2048 inputs: then workgroups have 4 waves and a compute
// unit holds two, of which one streams while the other prepares a group's
// rows.  Else 8 waves, and panels past 4096 inputs.
inline StreamPlan plan_stream(const GroupedCall& C, int* nw, int* kb) {
    StreamPlan P{};
    const int blocks = std::max(1, (C.cols + 127) / 128);
    while (P.kw_log < 3 && (4 << P.kw_log) < blocks) ++P.kw_log;
    *nw = P.kw_log == 3 ? 8 : 4;
    const int per = (blocks + (1 << P.kw_log) - 1) >> P.kw_log;
    *kb = per >= 3 ? 4 : per;
    P.panels = (blocks + (*kb << P.kw_log) - 1) / (*kb << P.kw_log);
    const int out = C.flags & PM_GROUPED_SWIGLU ? C.rows / 2 : C.rows;
    const int per_tile = C.flags & PM_GROUPED_SWIGLU ? 8 : 16;
    P.row_tiles = (out + per_tile - 1) / per_tile;
    return P;
}

}  // namespace
}  // namespace pm

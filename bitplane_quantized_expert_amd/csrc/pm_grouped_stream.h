// Products grouped by expert for groups of few rows: the kernel's template,
// instantiated for 16-bit weights in pm_grouped_stream16.hip and for 4-bit
// weights in pm_grouped_stream4.hip.
//
//   D[v][o] = sum_k x[v][k] W[o][k]   (v_mfma_f32_16x16x32, fp32 sums)
//
// Bound by reading the weights, so they go from memory to the matrix cores
// through registers, once, and everything else stays out of the way.
//
// A workgroup of 8 waves works on row tiles, 16 rows of one expert's matrix
// (8 gate and 8 up rows under PM_GROUPED_SWIGLU), for up to 16 * MT columns v
// of activations.  KW waves split the inputs, the other factor of 8 splits the
// row tiles.  A wave's share of the inputs, KB blocks of 128, stays in
// registers as matrix operands while the row tiles pass: a row tile costs the
// wave one 16-byte load per lane and 1 KiB, MT products each (4-bit: 4 MT) and
// nothing from LDS.  The loads of the next row tile are in flight while one is
// multiplied.  After kChunk row tiles the waves' sums meet in LDS (one
// barrier) and are added in the order of the waves.
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
// Activations meet 4-bit weights as fp16, scaled by a power of two per row
// and wave so that the largest lies in [2^14, 2^15): what is lost is below
// 2^-39 of the largest.  An fp32 row takes two columns, its value rounded to
// fp16 and the rest (times 2^11) rounded again, together 2^-24 of the value.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

// How a call is split: waves over the inputs (KW = 1 << kw_log), panels of
// KW * KB * 128 inputs, row tiles of a matrix.
struct StreamPlan {
    int kw_log, panels, row_tiles;
    int rows_per_tile;             // sorted rows of a tile: 16 * MT, halved for fp32 x
};

namespace {

constexpr int kStreamThreads = 512, kStreamWaves = 8, kChunk = 4;
// An offset beyond any buffer (all are below 2 GiB), with any immediate added.
constexpr uint32_t kNowhere = 0x80000000u;
constexpr int kRawBuffer = 0x00020000;
// How scales are read and applied: groups of 32, 64 or 128 inputs in aligned
// vectors, or (kAnyGroup) one by one for every 32 inputs.
enum { kNoGroup = 0, kGroup32 = 32, kGroup64 = 64, kGroup128 = 128, kAnyGroup = 1 };

// `at` or kNowhere, as a value: the compiler may not make branches of it with
// a load in each.
__device__ inline uint32_t chosen(bool ok, uint32_t at) {
    at = ok ? at : kNowhere;
    asm("" : "+v"(at));
    return at;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
__device__ inline f32x4 mfma_x_w(const u32x4& x, const u32x4& w, const f32x4& c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                       __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
}

// The constants of codes_to_f16 in registers, so that AND and OR are one
// instruction.
struct CodeBits {
    uint32_t even, odd, k1024, k64;
};
__device__ inline CodeBits code_bits() {
    CodeBits c{0x000F000Fu, 0x00F000F0u, 0x64006400u, 0x54005400u};
    asm("" : "+v"(c.even), "+v"(c.odd), "+s"(c.k1024), "+s"(c.k64));
    return c;
}

// The 8 codes of word w minus the zero point, as halves in the order
// 0 4 1 5 2 6 3 7; za = 1024 + z, zb = 64 + z, twice each.
__device__ inline u32x4 codes_to_f16(const CodeBits& k, uint32_t w, f16x2 za, f16x2 zb) {
    const uint32_t w8 = w >> 8;
    const f16x2 a = __builtin_bit_cast(f16x2, (w & k.even) | k.k1024) - za;
    const f16x2 b = __builtin_bit_cast(f16x2, (w & k.odd) | k.k64) - zb;
    const f16x2 c = __builtin_bit_cast(f16x2, (w8 & k.even) | k.k1024) - za;
    const f16x2 d = __builtin_bit_cast(f16x2, (w8 & k.odd) | k.k64) - zb;
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                 __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

// 8 halves in the order of codes_to_f16.
__device__ inline u32x4 code_order(u32x4 d) {
    return u32x4{__builtin_amdgcn_perm(d[2], d[0], 0x05040100u),
                 __builtin_amdgcn_perm(d[2], d[0], 0x07060302u),
                 __builtin_amdgcn_perm(d[3], d[1], 0x05040100u),
                 __builtin_amdgcn_perm(d[3], d[1], 0x07060302u)};
}

// 4 x 4 transposition of the words of lanes i, i + 16, i + 32, i + 48.
__device__ inline u32x4 exchange(u32x4 w) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{uint32_t(c[0]), uint32_t(c[1]), uint32_t(d[0]), uint32_t(d[1])};
}

__device__ inline float half_bits(uint32_t h) {
    return float(__builtin_bit_cast(_Float16, uint16_t(h)));
}

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

// The tiles of `mt` sorted rows of all experts, by one wave without LDS: a
// lane holds the count of its run of adjacent experts and of those before.
struct TileScan {
    int before, mine, total;
};

// Tiles of experts e .. e + 7 below `end`, their offsets loaded together.
__device__ inline void tiles_of_8(const GroupedCall& C, int mt, int e, int end, int* tiles,
                                  int* row0, int* n) {
    int o[9];
#pragma unroll
    for (int k = 0; k < 9; ++k) o[k] = C.offsets[min(e + k, C.n_experts)];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        row0[k] = min(max(o[k], 0), C.n_rows);
        n[k] = e + k < end ? max(min(o[k + 1], C.n_rows) - row0[k], 0) : 0;
        tiles[k] = (n[k] + mt - 1) / mt;
    }
}

__device__ inline TileScan scan_tiles(const GroupedCall& C, int mt) {
    const int lane = threadIdx.x & 63;
    const int per = (C.n_experts + kWave - 1) / kWave;
    const int e0 = min(lane * per, C.n_experts), e1 = min(e0 + per, C.n_experts);
    TileScan s;
    s.mine = 0;
    for (int b = 0; b < per; b += 8) {
        int tiles[8], row0[8], n[8];
        tiles_of_8(C, mt, e0 + b, e1, tiles, row0, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) s.mine += tiles[k];
    }
    const int incl = wave_scan(s.mine);
    s.before = incl - s.mine;
    s.total = __builtin_amdgcn_readlane(incl, 63);
    return s;
}

// Row tile i < total: its expert, first row and rows, the same in every lane.
struct TileRows {
    int e, row0, n;
};
__device__ inline TileRows find_tile_rows(const GroupedCall& C, int mt, const TileScan& s, int i) {
    const int lane = threadIdx.x & 63;
    const int per = (C.n_experts + kWave - 1) / kWave;
    const int e0 = min(lane * per, C.n_experts), e1 = min(e0 + per, C.n_experts);
    const uint64_t hit = __ballot(i >= s.before && i < s.before + s.mine);
    TileRows r{0, 0, 0};
    if (!hit) return r;                                   // (bad offsets only)
    int at = s.before;
    for (int b = 0; b < per; b += 8) {
        int tiles[8], row0[8], n[8];
        tiles_of_8(C, mt, e0 + b, e1, tiles, row0, n);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i >= at && i < at + tiles[k]) {
                const int skip = (i - at) * mt;
                r.e = e0 + b + k;
                r.row0 = row0[k] + skip;
                r.n = min(n[k] - skip, mt);
            }
            at += tiles[k];
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
// Eight activations at `p`, or zeros: `ok` says whether they count (p can be
// read in any case).
__device__ inline u32x4 load_x16(const char* p, bool ok) {
    const u32x4 d = *reinterpret_cast<const u32x4*>(p);
    return ok ? d : u32x4{0, 0, 0, 0};
}
__device__ inline F8 load_x32(const char* p, bool ok) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[i] = ok ? a[i] : 0.0f;
        r.v[4 + i] = ok ? b[i] : 0.0f;
    }
    return r;
}
__device__ inline F8 widen_bf16(u32x4 d) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = __uint_as_float(d[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
    return r;
}
__device__ inline float max_finite(const F8& x, float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x.v[i]);
        m = a < INFINITY ? fmaxf(m, a) : m;
    }
    return m;
}
// For a row of which the wave's largest finite value is `big` (a lane's part
// of it): 2^k that brings it to [2^14, 2^15), and 2^-k.
struct RowScale {
    float up, down;
};
__device__ inline RowScale row_scale(float big) {
    big = fmaxf(big, __shfl_xor(big, 16));
    big = fmaxf(big, __shfl_xor(big, 32));
    const int k = min(max(14 - (int(__float_as_uint(big) >> 23) - 127), -113), 126);
    return RowScale{__uint_as_float(uint32_t(127 + k) << 23), __uint_as_float(uint32_t(127 - k) << 23)};
}
// x * up as halves (lo: what that rounding leaves, times 2^11).
__device__ inline u32x4 to_f16(const F8& x, float up, bool lo) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = x.v[i] * up;
        _Float16 f = _Float16(s);
        if (lo) {
            const float hi = float(f);
            f = fabsf(hi) < INFINITY ? _Float16((s - hi) * 2048.0f) : _Float16(0.0f);
        }
        h[i] = __builtin_bit_cast(uint16_t, f);
    }
    return u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

// f(0), .., f(N - 1) with constant arguments.
template <int N, int I = 0, class F>
__device__ inline void steps_to(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        steps_to<N, I + 1>(f);
    }
}

template <int KIND, bool BF16, bool X32, int KB, int MT, int GM, bool ZEROS>
__global__ __launch_bounds__(kStreamThreads, 2) void stream_kernel(const GroupedCall C,
                                                                   const StreamPlan P) {
#ifdef __HIP_DEVICE_COMPILE__
    // 16-byte loads of a row tile per lane, and scales: one per block where a
    // group covers it, else one per 32 inputs
    constexpr int kLoads = KIND == kW4 ? KB : KB * 4;
    constexpr int kUnits = KIND != kW4 ? 0 : GM == kGroup128 ? KB : GM == kGroup64 ? KB * 2 : KB * 4;
    constexpr bool kWhole = GM == kGroup128;
    // row tiles held in registers: one at work, the others on their way
    // (as many as 256 registers hold beside the activations)
    constexpr int kSlots =
        GM == kAnyGroup || (GM == kGroup32 && KB == 4) || kLoads * MT > 8 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) float part[2][kStreamWaves][kChunk][MT * 256];
    __shared__ int use_row[2][16 * MT];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const int kw = 1 << P.kw_log, rw = kStreamWaves >> P.kw_log;
    const int ks = wv & (kw - 1), rg = wv >> P.kw_log;
    const bool glu = C.flags & PM_GROUPED_SWIGLU, gather = C.flags & PM_GROUPED_GATHER;
    const int out = glu ? C.rows / 2 : C.rows;
    const int per_tile = glu ? 8 : 16;

    const TileScan scan = scan_tiles(C, P.rows_per_tile);
    const int64_t all = int64_t(scan.total) * P.row_tiles;
    int64_t pos = all * blockIdx.x / gridDim.x;
    const int64_t end = all * (blockIdx.x + 1) / gridDim.x;

    const uint32_t row_bytes = KIND == kW4 ? uint32_t(C.cols) / 2 : uint32_t(C.cols) * 2;
    const size_t w_bytes = size_t(C.rows) * row_bytes;
    const int ng = KIND == kW4 ? C.cols / C.group : 0;
    const CodeBits bits = code_bits();
    int buf = 0, seg = 0;
    while (pos < end) {
        const int mt = int(pos / P.row_tiles);
        const int rt0 = int(pos - int64_t(mt) * P.row_tiles);
        const int rt1 = int(min(int64_t(P.row_tiles), rt0 + (end - pos)));
        pos += rt1 - rt0;
        const TileRows g = find_tile_rows(C, P.rows_per_tile, scan, mt);
        if (g.n <= 0) continue;                           // (bad offsets only)

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

        // ---- activations of this wave's inputs, as matrix operands
        u32x4 xf[KB * 4][MT] = {};
        float xs[MT][4] = {};                              // of columns 4q + r
        const char* xrow[MT];
        bool xok[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            // column v = 16 m + i16: a row, or the value (lower half) or rest
            // (upper half) of an fp32 row
            const int v = m * 16 + i16, r = X32 ? v & (8 * MT - 1) : v;
            const int u = r < g.n ? use_of(C, g.row0 + r) : -1;
            const int64_t xr = u < 0 ? 0 : gather ? u / C.top_k : g.row0 + r;
            xok[m] = u >= 0;
            xrow[m] = static_cast<const char*>(C.x) + xr * C.ldx * (X32 ? 4 : 2);
            if (wv == 0 && q == 0 && r < g.n && !(X32 && v >= 8 * MT))
                use_row[seg][r] = u < 0 ? -1 : (C.flags & PM_GROUPED_SCATTER ? u : g.row0 + r);
        }
        auto load_x = [&](int panel) {
            if (C.cols == 0) return;
            // first of operand f's 8 inputs: c0 + (f / 4) * 128 + (f % 4) * step
            // (computed here each time: kept over the row tiles it would
            // take the registers that hold the weights)
            const int step = kWhole ? 8 : 32;
            int c0 = first_block(panel) * 128 + q * (kWhole ? 32 : 8);
            asm volatile("" : "+v"(c0));
            const int last = C.cols - 8;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float down = 1.0f;
                if constexpr (!X32) {
#pragma unroll
                    for (int f = 0; f < KB * 4; ++f) {
                        const int c = c0 + (f >> 2) * 128 + (f & 3) * step;
                        xf[f][m] = load_x16(xrow[m] + size_t(min(c, last)) * 2, xok[m] && c <= last);
                    }
                    if (KIND == kW4 && C.x_type == PM_BF16) {
                        float big = 0.0f;
#pragma unroll
                        for (int f = 0; f < KB * 4; ++f) big = max_finite(widen_bf16(xf[f][m]), big);
                        const RowScale k = row_scale(big);
#pragma unroll
                        for (int f = 0; f < KB * 4; ++f) {
                            __builtin_amdgcn_sched_barrier(0);
                            xf[f][m] = to_f16(widen_bf16(xf[f][m]), k.up, false);
                        }
                        down = k.down;
                    }
                } else {
                    auto load = [&](int f) {
                        const int c = c0 + (f >> 2) * 128 + (f & 3) * step;
                        return load_x32(xrow[m] + size_t(min(c, last)) * 4, xok[m] && c <= last);
                    };
                    float big = 0.0f;
#pragma unroll
                    for (int f = 0; f < KB * 4; ++f) {
                        if (f % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                        big = max_finite(load(f), big);
                    }
                    const RowScale k = row_scale(big);
                    const bool lo = m * 16 + i16 >= 8 * MT;
                    asm volatile("" : "+v"(c0));
#pragma unroll
                    for (int f = 0; f < KB * 4; ++f) {
                        if (f % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                        xf[f][m] = to_f16(load(f), k.up, lo);
                    }
                    down = lo ? k.down * (1.0f / 2048.0f) : k.down;
                }
                if constexpr (KIND == kW4) {
#pragma unroll
                    for (int f = 0; f < KB * 4; ++f) xf[f][m] = code_order(xf[f][m]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) xs[m][r] = __shfl(down, 4 * q + r);
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        f32x4 acc[kChunk][MT];
        auto multiply = [&](auto slot, int panel, f32x4* a) {
            constexpr int S = decltype(slot)::value;
            f32x4 sum[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) sum[m] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (KIND == kW4) {
                const int c0 = first_block(panel) * 128;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    __builtin_amdgcn_sched_barrier(0);
                    const u32x4 c = kWhole ? w[S][b] : exchange(w[S][b]);
                    f32x4 d[MT];
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
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            d[m] = mfma_x_w<false>(
                                xf[b * 4 + j][m], wf,
                                j % kPer == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : d[m]);
                        if (j % kPer == kPer - 1) {
                            // past the last input there is no scale of this row
                            const bool in = c0 + b * 128 + (kWhole ? 0 : j / kPer * kPer * 32) < C.cols;
                            const float sf =
                                in ? half_bits(sc[S][unit / 2] >> (16 * (unit & 1))) : 0.0f;
#pragma unroll
                            for (int m = 0; m < MT; ++m)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    sum[m][r] = fmaf(d[m][r], sf, sum[m][r]);
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
                for (int f = 0; f < kLoads; ++f)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        sum[m] = mfma_x_w<BF16>(xf[f][m], w[S][f], sum[m]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    a[m][r] = KIND == kW4 ? fmaf(sum[m][r], xs[m][r], a[m][r]) : a[m][r] + sum[m][r];
        };

        const int per_chunk = rw * kChunk;
        // step c of (rtb, panel); c >= kChunk is of the panel or chunk after it
        auto issue_step = [&](auto slot, int c, int rtb, int panel) {
            if (c >= kChunk) {
                c -= kChunk;
                if (++panel == P.panels) {
                    panel = 0;
                    rtb += per_chunk;
                }
            }
            issue(slot, rtb + c * rw + rg, panel);
        };
        steps_to<kSlots - 1>([&](auto c) { issue(c, rt0 + c * rw + rg, 0); });
        int nlog = 0;
        while ((1 << nlog) < g.n) ++nlog;
        const int plog = glu ? 3 : 4;

        for (int rtb = rt0; rtb < rt1; rtb += per_chunk) {
#pragma unroll
            for (int c = 0; c < kChunk; ++c)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[c][m] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int panel = 0; panel < P.panels; ++panel) {
                if (P.panels > 1 || rtb == rt0) load_x(panel);
                steps_to<kChunk>([&](auto c) {
                    constexpr int kNext = (c + kSlots - 1) % kSlots;
                    issue_step(std::integral_constant<int, kNext>{}, c + kSlots - 1, rtb, panel);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(std::integral_constant<int, c % kSlots>{}, panel, acc[c]);
                    // registers: a row tile's decoded weights live in its own step
                    __builtin_amdgcn_sched_barrier(0);
                });
            }
#pragma unroll
            for (int c = 0; c < kChunk; ++c)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    *reinterpret_cast<f32x4*>(&part[buf][wv][c][m * 256 + lane * 4]) = acc[c][m];
            // LDS only: the weights under way are not waited for
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int items = per_chunk << (nlog + plog);
            for (int it = threadIdx.x; it < items; it += kStreamThreads) {
                const int col = it & ((1 << plog) - 1);
                const int r = (it >> plog) & ((1 << nlog) - 1), t = it >> (plog + nlog);
                const int rt = rtb + t, o = rt * per_tile + col;
                if (r >= g.n || rt >= rt1 || o >= out) continue;
                const int yr = use_row[seg][r];
                if (yr < 0) continue;
                const int c = t >> (3 - P.kw_log), first = (t & (rw - 1)) << P.kw_log;
                auto total = [&](int v, int column) {
                    const float* p = &part[buf][first][c][(v >> 4) * 256 +
                                                          (((v >> 2) & 3) * 16 + column) * 4 + (v & 3)];
                    float s = 0.0f;
                    for (int k = 0; k < kw; ++k) s += p[k * kChunk * MT * 256];
                    return s;
                };
                float p0 = total(r, col), p1 = glu ? total(r, col + 8) : 0.0f;
                if (X32) {
                    p0 += total(r + 8 * MT, col);
                    if (glu) p1 += total(r + 8 * MT, col + 8);
                }
                const float y = glu ? silu_up(p0, p1) : p0;
                const int64_t at = int64_t(yr) * C.ldy + o;
                if (C.y_type == PM_F32) store_f32<PM_F32>(C.y, at, y);
                else if (C.y_type == PM_F16) store_f32<PM_F16>(C.y, at, y);
                else store_f32<PM_BF16>(C.y, at, y);
            }
            buf ^= 1;
        }
        seg ^= 1;
    }
#endif
}

template <int KIND, bool BF16, bool X32, int KB, int MT, int GM, bool ZEROS>
hipError_t run_stream(const GroupedCall& C, const StreamPlan& P, hipStream_t st) {
    const int64_t tiles = int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / P.rows_per_tile;
    const unsigned grid = unsigned(std::min<int64_t>(tiles * P.row_tiles, compute_units()));
    hipLaunchKernelGGL((stream_kernel<KIND, BF16, X32, KB, MT, GM, ZEROS>), dim3(grid),
                       dim3(kStreamThreads), 0, st, C, P);
    return hipGetLastError();
}

// The split of the inputs: 4 blocks of 128 per wave where there are as many,
// over up to 8 waves, then panels.
inline StreamPlan plan_stream(const GroupedCall& C, bool x32, int mt, int* kb) {
    StreamPlan P{};
    const int blocks = std::max(1, (C.cols + 127) / 128);
    while (P.kw_log < 3 && (4 << P.kw_log) < blocks) ++P.kw_log;
    const int per = (blocks + (1 << P.kw_log) - 1) >> P.kw_log;
    // (32 columns: registers for 2 blocks)
    *kb = per >= 3 && mt == 1 ? 4 : std::min(per, 2);
    P.panels = (blocks + (*kb << P.kw_log) - 1) / (*kb << P.kw_log);
    const int out = C.flags & PM_GROUPED_SWIGLU ? C.rows / 2 : C.rows;
    const int per_tile = C.flags & PM_GROUPED_SWIGLU ? 8 : 16;
    P.row_tiles = (out + per_tile - 1) / per_tile;
    P.rows_per_tile = 16 * mt / (x32 ? 2 : 1);
    return P;
}

}  // namespace
}  // namespace pm

// Products grouped by expert with 4-bit weights for groups of many rows: tiles
// of 128 rows of 16-bit activations, or 64 of fp32, by 256 weight rows.
//
//   D[m][o] = sum_g scale[o][g] sum_{k in g} x[m][k] (q - z)[o][k]
//
// (v_mfma_f32_16x16x32; q - z is exact in fp16, and (q - z) 2^-15 in bf16, sums
// are fp32.)
// Streamed past 16 columns at a time, the weights are decoded once per 16 rows
// of x, which bounds groups of more than some 16 rows; here once per 128.
//
// 8 waves, each with 32 weight rows and all 128 rows of x.  The codes go from
// memory to registers, 16 bytes per lane and 128 inputs (as in the streamed
// kernel), two blocks of 128 inputs ahead, and are decoded to matrix operands
// there: no wave needs another's.  x goes straight to LDS, three blocks of 128
// inputs x 128 rows (32 KiB), two ahead; one barrier per block.  A wave reads
// 16 rows of a block at a time, the next 16 while these are multiplied.
//
// An fp32 row takes two of the 128: its values times a power of two per row and
// block, rounded to fp16, and the rest (times 2^11) rounded again: off by 2^-23
// of the value, or 2^-50 of the largest.  Every lane holds 16 inputs of a row,
// loaded a block ahead, and converts them while the last block is multiplied.
//
// Measured: 64 experts of 4096 x 4096 with 128 bf16 rows each 333 to 338 us (815
// to 825 TFLOP/s; the streamed kernel 997), the matrix cores 39 % and LDS 20 %
// busy: a wave decodes, then multiplies, and few of its instructions meet the
// other wave's.  64 rows 238 us (500), 32 rows 213 (261); 8 experts with 256 rows
// 90 us (223).  fp32: 752 to 784 us (1930), 405 (968), 318 (489).  Decoding the
// next block between the products took 3 to 15 % longer (registers, and loads
// later by most of a block); starting the tiles of an expert at different blocks
// changed nothing.
//
// LDS holds rows of 128 inputs (256 bytes = 16 pieces).  The four pieces that
// one product takes (a lane quarter's each) come to adjacent places 4 s + q, and
// place p of row r lies at p ^ (r % 16): 16-byte reads are served 16 lanes at a
// time, of two quarters and all rows, which so fall in distinct banks.  Rows past the group and inputs past `cols` read as zero.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_grouped_codes.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kOuts = 256, kBlockK = 128;
constexpr int kStageBytes = 128 * kBlockK * 2;
constexpr int kThreads4 = 512;
// Rows of x per tile, blocks held in LDS.
constexpr int tile4_rows(bool x32) { return x32 ? 64 : 128; }
constexpr int tile4_stages(bool x32) { return x32 ? 2 : 3; }

typedef __attribute__((address_space(3))) void lds_void;

// bf16 activations reach fp32's largest values, so that their products with
// codes and zero points up to 255, summed over 128 inputs, would pass it where
// the scaled result does not.  Their weight operands are (q - z) 2^-15 and the
// scales 2^15 larger: 255 * 128 * 2^-15 < 1.  Nothing is lost at the small end:
// a bf16 value is a multiple of 2^-133, a product of 2^-148, and fp32 holds
// multiples of 2^-149.  (The factor costs 3 % at 32 rows per expert, nothing at
// 128.)
constexpr float kCodeUnit = 1.0f / 32768.0f;

// The 8 codes of word w minus the zero point, as 16-bit operands in order
// (bf16: in units of kCodeUnit).
template <bool BF16>
__device__ inline u32x4 codes_in_order(const CodeBits& k, uint32_t w, f16x2 za, f16x2 zb) {
    const u32x4 c = codes_to_f16(k, w, za, zb);          // 0 4 | 1 5 | 2 6 | 3 7
    if constexpr (!BF16) {
        return u32x4{__builtin_amdgcn_perm(c[1], c[0], 0x05040100u),
                     __builtin_amdgcn_perm(c[3], c[2], 0x05040100u),
                     __builtin_amdgcn_perm(c[1], c[0], 0x07060302u),
                     __builtin_amdgcn_perm(c[3], c[2], 0x07060302u)};
    } else {
        // (8 significant bits: the upper half of the fp32 value is exact)
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t pair = c[i];                  // (a bit_cast of c[i] takes c[0])
            const f16x2 h = __builtin_bit_cast(f16x2, pair);
            lo[i] = __float_as_uint(fmaf(float(h[0]), kCodeUnit, 0.0f));
            hi[i] = __float_as_uint(fmaf(float(h[1]), kCodeUnit, 0.0f));
        }
        return u32x4{__builtin_amdgcn_perm(lo[1], lo[0], 0x07060302u),
                     __builtin_amdgcn_perm(lo[3], lo[2], 0x07060302u),
                     __builtin_amdgcn_perm(hi[1], hi[0], 0x07060302u),
                     __builtin_amdgcn_perm(hi[3], hi[2], 0x07060302u)};
    }
}

template <bool BF16, bool X32, int GM, bool ZEROS>
__global__ __launch_bounds__(kThreads4, 2) void tile4_kernel(const GroupedCall C, int nt) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int kRows = tile4_rows(X32), kStages = tile4_stages(X32), XB = X32 ? 4 : 2;
    constexpr bool kWhole = GM == kGroup128;
    // products between two scales, scales of a block
    constexpr int kPer = kWhole ? 4 : GM == kGroup64 ? 2 : 1, kUnits = 4 / kPer;
    constexpr int kScaleLoads = GM == kAnyGroup ? 4 : 1;
    constexpr int LX = 4, XR = X32 ? 1 : 4;       // a lane's loads of x, rows of them
    constexpr int LW = 2 * (1 + kScaleLoads * (ZEROS ? 2 : 1));   // loads per block
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    int* const ymap = reinterpret_cast<int*>(smem + kStages * kStageBytes);   // [2][kRows]
    int* const before = ymap + 2 * kRows;                                     // [E + 1]
    __shared__ __attribute__((aligned(16))) float xscale[2][X32 ? kRows : 4];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const bool glu = C.flags & PM_GROUPED_SWIGLU, gather = C.flags & PM_GROUPED_GATHER;
    const int out = glu ? C.rows / 2 : C.rows;
    const int n_tiles = tile_table(C, kRows, before) * nt;
    __syncthreads();

    // place of this workgroup in a round of tiles: the 32 of one XCD are
    // consecutive, so that they share weight rows and x rows in its L2
    const int per_xcd = gridDim.x >> 3;
    const int place = gridDim.x & 7 ? blockIdx.x : (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    struct Where {
        int e, row0, n, o0;                       // expert, rows, first output; n 0: no tile
    };
    auto locate = [&](int i) {
        Where w{0, 0, 0, 0};
        if (i < n_tiles) {
            const int mt = i / nt;
            const int e = tile_expert(C, before, mt);
            const RowRange g = group_rows_uniform(C, e);
            const int64_t skip = int64_t(mt - before[e]) * kRows;
            const bool ok = skip >= 0 && skip < g.n;      // (not so only for bad offsets)
            w.e = uni(e);
            w.row0 = uni(ok ? g.row0 + int(skip) : 0);
            w.n = uni(ok ? min(g.n - int(skip), kRows) : 0);
            w.o0 = uni((i - mt * nt) * (glu ? kOuts / 2 : kOuts));
        }
        return w;
    };

    // ---- x: this lane's rows of a block, 4 loads of 4 rows per wave (fp32: of
    // one row, 8 lanes each)
    const int xrow = X32 ? int(threadIdx.x >> 3) : wv * 4 + q;
    // product s takes piece 4 q + s of quarter q where a scale covers the block,
    // else 4 s + q; its place (and back)
    auto place_piece = [](int p) { return kWhole ? (p & 3) * 4 + (p >> 2) : p; };
    const int piece = place_piece(i16 ^ (xrow & 15));
    // (loads only: they are waited for in set_rows, many blocks later)
    auto use_rows = [&](const Where& w, int* u) {
#pragma unroll
        for (int i = 0; i < XR; ++i) u[i] = w.row0 + i * 32 + xrow;
        if (C.order) {
#pragma unroll
            for (int i = 0; i < XR; ++i) u[i] = C.order[min(u[i], C.n_rows - 1)];
        }
    };
    uint32_t pa[XR];
    auto set_rows = [&](const Where& w, const int* u, int parity) {
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            const int r = i * 32 + xrow;
            int use = u[i];
            asm volatile("" : "+v"(use));                // (nothing is done to it before)
            const bool ok = r < w.n && use >= 0 && use < C.n_rows;
            const uint32_t xr = gather ? uint32_t(use) / uint32_t(C.top_k) : uint32_t(r);
            pa[i] = ok ? uint32_t(xr * uint64_t(C.ldx) * XB) +
                                    (X32 ? (lane & 7) * 16 : piece * 16)
                              : kOutside;
            if ((lane & (X32 ? 7 : 15)) == 0)
                ymap[parity * kRows + r] =
                    ok ? (C.flags & PM_GROUPED_SCATTER ? use : w.row0 + r) : -1;
        }
    };
    auto x_buffer = [&](const Where& w) {
        const char* p = static_cast<const char*>(C.x) + (gather ? 0 : size_t(w.row0) * C.ldx * XB);
        const size_t n = w.n == 0 ? 0
                                  : (size_t(gather ? (C.n_rows - 1) / C.top_k : w.n - 1) * C.ldx +
                                     C.cols) * XB;
        return __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<char*>(p)), 0, uni(int(uint32_t(min(n, size_t(kOutside))))),
            kRawBuffer);
    };

    // ---- weights: this lane's two rows (gate and up under SWIGLU)
    const uint32_t row_bytes = uint32_t(C.cols) / 2;
    const size_t w_bytes = size_t(C.rows) * row_bytes;
    const int ng = C.cols / C.group;
    int wrow[2];
    auto set_weights = [&](const Where& w) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int o = w.o0 + (glu ? wv * 16 : wv * 32 + b * 16) + i16;
            wrow[b] = w.n > 0 && o < out ? (glu && b ? out + o : o) : -1;
        }
    };
    auto w_buffer = [&](const Where& w) {
        return __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<char*>(static_cast<const char*>(C.w)) + size_t(w.e) * w_bytes), 0,
            uni(int(uint32_t(w_bytes))), kRawBuffer);
    };
    auto s_buffer = [&](const Where& w) {
        return __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<uint16_t*>(C.scales) + size_t(w.e) * C.rows * ng), 0,
            uni(int(uint32_t(C.rows) * uint32_t(ng) * 2)), kRawBuffer);
    };
    // Zero points of one block are bytes of one aligned word, which is loaded
    // whole: narrower values would be widened at the loop's end, which waits
    // for them.  (A word that holds a zero point is on the same page with it.)
    constexpr bool kZeroWords = ZEROS && GM != kAnyGroup;
    uint32_t zmis = 0;                            // bytes from the word's start to the first
    auto z_buffer = [&](const Where& w) {
        const uint8_t* p = C.zeros + size_t(w.e) * C.rows * ng;
        uint32_t n = uint32_t(C.rows) * uint32_t(ng);
        if constexpr (kZeroWords) {
            zmis = uni(int(reinterpret_cast<uintptr_t>(p) & 3));
            p -= zmis;
            n = (n + zmis + 3) & ~3u;
        }
        return __builtin_amdgcn_make_buffer_rsrc(uni_ptr(const_cast<uint8_t*>(p)), 0, uni(int(n)),
                                                 kRawBuffer);
    };

    // (blocks past the last input hold zeros; a tile has an even number)
    const int T = max(2, ((C.cols + kBlockK - 1) / kBlockK + 1) & ~1);
    int u[XR];
    Where cur = locate(place), nxt;
    if (cur.n == 0) return;
    use_rows(cur, u);
    set_rows(cur, u, 0);
    set_weights(cur);
    auto xb = x_buffer(cur);
    auto wb = w_buffer(cur), sb = s_buffer(cur), zb = z_buffer(cur);
    int kx = 0, kw = 0;
    // fp32: to registers, and from there as two halves to LDS
    u32x4 raw[X32 ? LX : 1];
    auto load_x = [&]() {
#pragma unroll
        for (int j = 0; j < (X32 ? LX : 1); ++j) {
            const bool in = pa[0] != kOutside && kx * kBlockK + (j * 8 + (lane & 7)) * 4 < C.cols;
            uint32_t at = in ? pa[0] + uint32_t(j * 128 + kx * kBlockK * 4) : kOutside;
            asm("" : "+v"(at));                          // (no branches with a load in each)
            raw[j] =
                __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, at, 0, 0));
        }
        ++kx;
    };
    // times a power of two per row and block that brings the largest to [2^14,
    // 2^15); row r holds the values rounded to fp16, row 64 + r the rest, times
    // 2^11, rounded again
    auto split_x = [&](int stage) {
        float v[4 * LX];
        float big = 0.0f;
#pragma unroll
        for (int j = 0; j < (X32 ? LX : 1); ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = raw[j][i];
                v[4 * j + i] = __uint_as_float(bits);
                const float a = fabsf(v[4 * j + i]);
                big = a < INFINITY ? fmaxf(big, a) : big;
            }
        big = fmaxf(big, dpp<0xB1, 0xF>(big));
        big = fmaxf(big, dpp<0x4E, 0xF>(big));
        big = fmaxf(big, dpp<0x141, 0xF>(big));
        const int e = min(max(14 - (int(__float_as_uint(big) >> 23) - 127), -113), 126);
        const float up = __uint_as_float(uint32_t(127 + e) << 23);
        char* const base = smem + stage * kStageBytes + xrow * 256;
#pragma unroll
        for (int j = 0; j < (X32 ? LX : 1); ++j) {
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = v[4 * j + i] * up;
                const _Float16 h = _Float16(s);
                const float back = float(h);
                hi[i] = __builtin_bit_cast(uint16_t, h);
                const _Float16 l = fabsf(back) < INFINITY ? _Float16((s - back) * 2048.0f)
                                                          : _Float16(0.0f);
                lo[i] = __builtin_bit_cast(uint16_t, l);
            }
            const int g = j * 8 + (lane & 7);            // these 4 inputs of the block
            char* at = base + ((place_piece(g >> 1) ^ (xrow & 15)) * 16) + (g & 1) * 8;
            *reinterpret_cast<u32x2*>(at) = u32x2{hi[0] | uint32_t(hi[1]) << 16,
                                                  hi[2] | uint32_t(hi[3]) << 16};
            *reinterpret_cast<u32x2*>(at + 64 * 256) = u32x2{lo[0] | uint32_t(lo[1]) << 16,
                                                             lo[2] | uint32_t(lo[3]) << 16};
        }
        if ((lane & 7) == 0) xscale[stage][xrow] = __uint_as_float(uint32_t(127 - e) << 23);
    };
    auto issue_x = [&](int stage) {
        char* base = smem + stage * kStageBytes + wv * 1024;
        const bool in = kx * kBlockK + piece * 8 < C.cols;
#pragma unroll
        for (int i = 0; i < LX; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lds_void*)(base + i * 8192), 16,
                                                     in ? pa[X32 ? 0 : i] : kOutside,
                                                     kx * kBlockK * 2, 0, 0);
        ++kx;
    };
    u32x4 w[2][2];
    uint32_t sc[2][2][2], zp[2][2], zsh[2][2];    // [slot][weight row]
    auto issue_w = [&](auto slot) {
        constexpr int S = decltype(slot)::value;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool some = wrow[b] >= 0 && kw * kBlockK < C.cols;
            const uint32_t at = chosen(some, uint32_t(wrow[b]) * row_bytes + kw * 64 + q * 16);
            w[S][b] = __builtin_bit_cast(u32x4,
                                         __builtin_amdgcn_raw_buffer_load_b128(wb, at, 0, 0));
            if constexpr (GM == kAnyGroup) {
                uint32_t z = 0;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int c = kw * kBlockK + s * 32;
                    const uint32_t g = uint32_t(wrow[b]) * ng + c / C.group;
                    const bool in = wrow[b] >= 0 && c < C.cols;
                    const uint32_t v =
                        uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sb, chosen(in, g * 2), 0, 0));
                    sc[S][b][s / 2] = s & 1 ? sc[S][b][s / 2] | v << 16 : v;
                    if constexpr (ZEROS)
                        z |= uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(
                                 zb, chosen(in, g), 0, 0))) << (8 * s);
                }
                if constexpr (ZEROS) zp[S][b] = z;
            } else {
                const uint32_t g = uint32_t(wrow[b]) * ng + uint32_t(kw) * kUnits;
                const uint32_t so = chosen(some, g * 2);
                if constexpr (kZeroWords) {
                    const uint32_t at = g + zmis;
                    zsh[S][b] = (at & 3) * 8;
                    zp[S][b] = __builtin_amdgcn_raw_buffer_load_b32(zb, chosen(some, at & ~3u), 0, 0);
                }
                if constexpr (kUnits == 1) {
                    sc[S][b][0] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sb, so, 0, 0));
                } else if constexpr (kUnits == 2) {
                    sc[S][b][0] = __builtin_amdgcn_raw_buffer_load_b32(sb, so, 0, 0);
                } else {
                    const u32x2 v = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_raw_buffer_load_b64(sb, so, 0, 0));
                    sc[S][b][0] = v[0];
                    sc[S][b][1] = v[1];
                }
            }
        }
        ++kw;
    };
    const CodeBits bits = code_bits();
    if constexpr (X32) load_x();
    else issue_x(0);
    __builtin_amdgcn_sched_barrier(0);
    issue_w(std::integral_constant<int, 0>{});
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (X32) {
        split_x(0);
        load_x();
    } else {
        issue_x(1);
    }
    __builtin_amdgcn_sched_barrier(0);
    issue_w(std::integral_constant<int, 1>{});

    // place in a row of x of this lane's 8 inputs of each product
    int place_of[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
        place_of[s] = i16 * 256 + (((s * 4 + q) ^ i16) * 16);
    f32x4 acc[kRows / 16][2];
    int xs = 0, parity = 0, arrived = 0;
    auto step = [&](auto slot, int t) {
        constexpr int S = decltype(slot)::value;
        __builtin_amdgcn_sched_barrier(0);
        // this block of x has arrived, and every wave is done with the last.
        // (Loads and stores complete in order: the two blocks that were under
        // way at a tile's end were waited for before its stores.)
        if (X32 || arrived > 0) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            --arrived;
        } else {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * LW + LX)
                         : "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool last = S == 0 && t == T - 2;
        if constexpr (X32) split_x(S ^ 1);
        if (last) {
            set_rows(nxt, u, parity ^ 1);
            xb = x_buffer(nxt);
            kx = 0;
        }
        if constexpr (X32) load_x();
        else issue_x(xs == 0 ? 2 : xs - 1);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 wf[2][4];
        float sf[2][kUnits];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t zeros4 = 0;
            if constexpr (ZEROS) zeros4 = kZeroWords ? zp[S][b] >> zsh[S][b] : zp[S][b];
            const u32x4 c = kWhole ? w[S][b] : exchange(w[S][b]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f16x2 za = {_Float16(1032.0f), _Float16(1032.0f)};
                f16x2 zc = {_Float16(72.0f), _Float16(72.0f)};
                if constexpr (ZEROS) {
                    const uint32_t z = zeros4 >> (8 * (j / kPer)) & 255u;
                    za = __builtin_bit_cast(f16x2, 0x64006400u | z | z << 16);
                    zc = za - f16x2{_Float16(960.0f), _Float16(960.0f)};
                }
                wf[b][j] = codes_in_order<BF16>(bits, c[j], za, zc);
            }
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                sf[b][k] = half_bits(sc[S][b][k / 2] >> (16 * (k & 1)));
                if constexpr (BF16) sf[b][k] *= 1.0f / kCodeUnit;
                // here, so that the next loads can take the scales' registers (else
                // they are copied at the loop's end, which waits for them)
                asm volatile("" : "+v"(sf[b][k]));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (last) {
            set_weights(nxt);
            wb = w_buffer(nxt);
            sb = s_buffer(nxt);
            zb = z_buffer(nxt);
            kw = 0;
        }
        issue_w(slot);
        __builtin_amdgcn_sched_barrier(0);

        // (fp32: H = 1 is the rest of row m)
        constexpr int H = X32 ? 2 : 1;
        const char* xt = smem + (X32 ? S : xs) * kStageBytes;
        u32x4 fa[2][H][4];
        auto read = [&](int m) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    fa[m & 1][h][s] = *reinterpret_cast<const u32x4*>(
                        xt + (h * 64 + m * 16) * 256 + place_of[s]);
        };
        read(0);
#pragma unroll
        for (int m = 0; m < kRows / 16; ++m) {
            if (m * 16 >= cur.n) break;
            if (m + 1 < kRows / 16) read(m + 1);
            f32x4 xf = {1.f, 1.f, 1.f, 1.f};
            if constexpr (X32) xf = *reinterpret_cast<const f32x4*>(&xscale[S][m * 16 + 4 * q]);
            // a unit's sums meet their scale after the next unit's first products
            f32x4 d[2][2][H];
            auto scale = [&](int k) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float v = d[k & 1][b][0][r], by = sf[b][k];
                        if constexpr (X32) {
                            const float both = fmaf(d[k & 1][b][H - 1][r], 1.0f / 2048.0f, v);
                            acc[m][b][r] = fmaf(both * by, xf[r], acc[m][b][r]);
                        } else {
                            acc[m][b][r] = fmaf(v, by, acc[m][b][r]);
                        }
                    }
            };
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = s / kPer;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        d[k & 1][b][h] = mfma_x_w<BF16>(
                            fa[m & 1][h][s], wf[b][s],
                            s % kPer == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : d[k & 1][b][h]);
                if (s > 0 && s % kPer == 0) scale(k - 1);
            }
            scale(kUnits - 1);
            // here, not where the sums are needed: the products' registers are
            // free then
            asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]));
        }
        xs = xs == 2 ? 0 : xs + 1;
    };

    auto store = [&](int64_t at, float v) {
        if (C.y_type == PM_F32) store_f32<PM_F32>(C.y, at, v);
        else store_f32<BF16 ? PM_BF16 : PM_F16>(C.y, at, v);
    };
    for (int tile = place; cur.n > 0; tile += gridDim.x) {
        // the next tile's place and uses, long before its first loads
        nxt = locate(tile + gridDim.x);
        use_rows(nxt, u);
#pragma unroll
        for (int m = 0; m < kRows / 16; ++m)
#pragma unroll
            for (int b = 0; b < 2; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int t = 0; t < T; t += 2) {
            step(std::integral_constant<int, 0>{}, t);
            step(std::integral_constant<int, 1>{}, t + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!X32) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LW) : "memory");
            arrived = 2;
        }
        const int* rows = ymap + parity * kRows + 4 * q;
#pragma unroll
        for (int m = 0; m < kRows / 16; ++m) {
            if (m * 16 >= cur.n) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int yr = rows[m * 16 + r];
                if (yr < 0) continue;
                const int64_t at = int64_t(yr) * C.ldy;
                if (glu) {
                    const int o = cur.o0 + wv * 16 + i16;
                    if (o < out) store(at + o, silu_up(acc[m][0][r], acc[m][1][r]));
                } else {
                    const int o = cur.o0 + wv * 32 + i16;
                    if (o < out) store(at + o, acc[m][0][r]);
                    if (o + 16 < out) store(at + o + 16, acc[m][1][r]);
                }
            }
        }
        cur = nxt;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last blocks' loads
#endif
}

template <bool BF16, bool X32, int GM, bool ZEROS>
hipError_t run_tiles4(const GroupedCall& C, hipStream_t st) {
    const int out = C.flags & PM_GROUPED_SWIGLU ? C.rows / 2 : C.rows;
    const int per = C.flags & PM_GROUPED_SWIGLU ? kOuts / 2 : kOuts;
    const int nt = (out + per - 1) / per;
    constexpr int kRows = tile4_rows(X32);
    const size_t lds =
        size_t(tile4_stages(X32)) * kStageBytes + (2 * kRows + C.n_experts + 1) * sizeof(int);
    auto* f = tile4_kernel<BF16, X32, GM, ZEROS>;
    static std::atomic<uint64_t> allowed{0};
    hipError_t e = allow_lds(reinterpret_cast<const void*>(f), kTileMaxLds, &allowed);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / kRows) * nt;
    const unsigned grid = unsigned(std::min<int64_t>(tiles, compute_units()));
    hipLaunchKernelGGL(f, dim3(grid), dim3(kThreads4), lds, st, C, nt);
    return hipGetLastError();
}

template <bool BF16, bool X32, bool ZEROS>
hipError_t run_tiles4_group(const GroupedCall& C, hipStream_t st) {
    if (reads_scales_by(C, 128, 1)) return run_tiles4<BF16, X32, kGroup128, ZEROS>(C, st);
    if (reads_scales_by(C, 64, 1)) return run_tiles4<BF16, X32, kGroup64, ZEROS>(C, st);
    if (reads_scales_by(C, 32, 1)) return run_tiles4<BF16, X32, kGroup32, ZEROS>(C, st);
    return run_tiles4<BF16, X32, kAnyGroup, ZEROS>(C, st);
}

template <bool BF16, bool X32>
hipError_t run_tiles4_zeros(const GroupedCall& C, hipStream_t st) {
    return C.zeros ? run_tiles4_group<BF16, X32, true>(C, st)
                   : run_tiles4_group<BF16, X32, false>(C, st);
}

}  // namespace

hipError_t launch_grouped_tiles4(const GroupedCall& C, hipStream_t st) {
    if (C.x_type == PM_F32) return run_tiles4_zeros<false, true>(C, st);
    return C.x_type == PM_BF16 ? run_tiles4_zeros<true, false>(C, st)
                               : run_tiles4_zeros<false, false>(C, st);
}

}  // namespace pm

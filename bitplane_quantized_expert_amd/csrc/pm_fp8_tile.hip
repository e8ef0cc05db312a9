// Products grouped by expert of 8-bit weights and activations, for groups of
// many rows: tiles of 256 or 128 rows by 256 outputs on the matrix cores.
//
//   y[m][o] = sum_b sw[o/128][b] sx[m][b] D_b[o][m],
//   D_b[o][m] = sum of W[o][k] x[m][k] over the 128 inputs of block b
//
// The walk over the tiles is that of the 16-bit tiles (pm_grouped_tile.hip): a
// persistent workgroup of 8 waves per compute unit, operands straight from
// memory to LDS, S stages of one block of 128 inputs (128 bytes a row), pieces of
// 16 bytes at place c ^ (r % 8), the next tile's stages right behind this one's.
// The scales of x come along with a stage, 4 bytes a row; those of W are scalars.
//
// bf16 results: v_mfma_f32_16x16x128_f8f6f4 takes a whole block of 16 x 16 in one
// instruction (32 cycles), from codes as they are.  Its sums of 8 adjacent
// products are cut off 13 bits below the largest one's power of two (measured:
// every one of 13 million random groups equals that model; v_mfma_f32_16x16x32_fp8
// and the 32x32x64 form do the same), 1.5e-5 of results on normal data beside
// the 1.7e-3 of bf16's own rounding; include/pm.h has the bound.  Other results,
// and bf16 ones under PM_GROUPED_FP32_SUMS: the codes become halves in registers,
// exactly, and four v_mfma_f32_16x16x32_f16 take a block (65536 rows over 32 experts
// of 2048 x 4096, gate and up: 1038 us with fp32 sums beside 540; 40960 over 512 of
// 4096 x 1024: 600 beside 513).
// Either way a block's sum meets the factor sw * sx in one fp32 fma per element.
//
// What bounds them, and how it is met:
// - Many rows (65536 over 32 experts of 2048 x 4096, gate and up: 540 to 563 us, 1.95
//   to 2.04 PFLOP/s, the matrix cores 56 % busy): 4 fmas and 4 factors an element
//   of a block beside its 32 cycles of product, all in one wave's order, and SiLU,
//   30 us of it, with the matrix cores idle.  So each
//   product is pinned where it is written, its sums are added two products later
//   (no wait for the result), and the loads of a stage lie a few products apart;
//   left to the compiler the sums wait, in 193 spilled registers.  A product
//   after another in one wave with 4 fmas each reaches 3.9 PFLOP/s by itself.
// - Some rows (4096 x 10 over 512 experts of 4096 x 1024: 514 us, 4.9 TB/s): the
//   weights' way from memory.  128 rows and three stages keep two on their way.
//   The place of a tile comes by scalar loads, since a wait for a vector load is one
//   for all stages before it, and with three stages the first step does not wait
//   for the last tile's stores.
// - Loads of weights past the caches gained 2 % there and lost more elsewhere, such
//   stores of y lost everywhere, loads 1 product apart or 4 lost 1 to 3 %, and all
//   stages' weights before any x at the start lost on small calls.  Priorities of
//   waves (of one of a SIMD's two, or of both between barriers) changed nothing.
// - Halves (fp32 and fp16 results): conversions and four times the products, 848
//   TFLOP/s at 64 experts of 4096 x 2048 with 512 rows each.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_fp8.h"
#include "pm_grouped_codes.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kTileN = 256, kTileK = 128;
constexpr int kTileThreads = 512, kTileWaves = 8;
constexpr int kScaleBytes = kTileThreads * 4;        // of a stage: a lane of every wave

typedef __attribute__((address_space(3))) void lds_void;

// N adjacent outputs of row y + at, those below `left`, 16 bytes at a time.
template <int YT, int N>
__device__ inline void store_row(void* y, int64_t at, int left, const float* v) {
    constexpr int B = YT == PM_F32 ? 4 : 2, P = 16 / B;
    if (left >= N) {
#pragma unroll
        for (int k = 0; k < N; k += P) {
            alignas(16) char o[16];
#pragma unroll
            for (int r = 0; r < P; ++r) store_f32<YT>(o, r, v[k + r]);
            __builtin_memcpy(static_cast<char*>(y) + (at + k) * B, o, 16);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < N; k += 4) store4<YT>(y, at + k, left - k, v + k);
}

// How the scales of the weight rows of a wave fall: one for all (kPlain), one
// for gate and one for up rows (kGlu), or up rows on both sides of a border
// (kGluSplit: the up matrix begins inside a block of 128 rows).
enum { kPlain = 0, kGlu = 1, kGluSplit = 2 };

// BM rows by 256 weight rows, S stages of 128 inputs in LDS.  NATIVE: codes
// multiplied as they are.
template <int YT, bool NATIVE, int MODE, int BM, int S>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_tile_kernel(const GroupedCall C, int nt) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr bool GLU = MODE != kPlain;
    constexpr int kStageA = BM * kTileK, kCodes = kStageA + kTileN * kTileK;
    constexpr int kStage = kCodes + kScaleBytes;
    constexpr int LA = BM / 64, LB = kTileN / 64, L = LA + LB + 1;  // a wave's loads per stage
    constexpr int WM = BM / 2;                    // rows of a wave: 2 x 4 waves
    constexpr int MB = WM / 16, NB = 4, NP = MB * NB;
    constexpr int kApart = (NP - NB) / (2 * (L - NB));        // products between two loads
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    int* const ymap = reinterpret_cast<int*>(smem + S * kStage);          // [2][BM]
    int* const before = ymap + 2 * BM;                                    // [E + 1]
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int out = GLU ? C.rows / 2 : C.rows;
    const int blocks = (C.cols + kTileK - 1) / kTileK, row_blocks = (C.rows + 127) / 128;
    const int n_tiles = tile_table(C, BM, before) * nt;
    __syncthreads();

    const int wm = wv >> 2, wn = wv & 3;
    const int i16 = lane & 15, q = lane >> 4;
    const int r8 = lane >> 3, piece = (lane & 7) ^ r8;
    // place of this workgroup in a round of tiles: the 32 of one XCD are
    // consecutive, so that they share weight rows and x rows in its L2
    const int per_xcd = gridDim.x >> 3;
    const int place = gridDim.x & 7 ? blockIdx.x : (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);

    struct Where {
        int e, row0, n, o0;                       // expert, rows, first output; n 0: no tile
    };
    // A last round of at most half the workgroups is shared out by halves of
    // 128 rows, which take half the time.
    const int full = n_tiles / int(gridDim.x) * int(gridDim.x), rest = n_tiles - full;
    const bool halves = BM == 256 && full > 0 && 2 * rest <= int(gridDim.x);
    auto locate = [&](int i) {
        Where w{0, 0, 0, 0};
        int half = -1;
        if (halves && i >= full) {
            half = (i - full) & 1;
            i = full + ((i - full) >> 1);
        }
        if (i < n_tiles) {
            const int mt = i / nt;
            const int e = tile_expert(C, before, mt);
            // (by scalar loads: a wait for vector loads is one for the stages, too)
            const RowRange g = group_rows_uniform(C, e);
            const int64_t skip = int64_t(mt - before[e]) * BM;
            const bool ok = skip >= 0 && skip < g.n;      // (not so only for bad offsets)
            w.e = uni(e);
            w.row0 = uni(ok ? g.row0 + int(skip) : 0);
            w.n = uni(ok ? min(g.n - int(skip), BM) : 0);
            if (half == 0) w.n = min(w.n, BM / 2);
            if (half == 1) {
                w.row0 += BM / 2;
                w.n = max(w.n - BM / 2, 0);
            }
            w.o0 = uni((i - mt * nt) * (GLU ? kTileN / 2 : kTileN));
        }
        return w;
    };
    const bool gather = C.flags & PM_GROUPED_GATHER;
    const size_t wbytes = size_t(C.rows) * C.cols;
    // the row whose scale this lane loads: the scales of a wave's rows i * 16 +
    // i16 are adjacent in i, so that a lane reads all of its own at once
    const int p_row = wv < BM / 64 ? (wv * 64 + lane) / WM * WM + (lane & (MB - 1)) * 16 +
                                         ((wv * 64 + lane) % WM) / MB
                                   : BM;
    // the uses of this lane's rows and of that of its scale, as they are loaded
    auto load_uses = [&](const Where& w, int* raw) {
#pragma unroll
        for (int i = 0; i <= LA; ++i) {
            const int r = i < LA ? (i * kTileWaves + wv) * 8 + r8 : p_row;
            raw[i] = r < w.n ? w.row0 + r : -1;
            if (C.order && raw[i] >= 0) raw[i] = C.order[raw[i]];
        }
    };
    // offsets of this lane's rows of x and of their scales, and of W per stage
    auto set_x = [&](const Where& w, const int* raw, int parity, uint32_t* pa, uint32_t* ps) {
        int u[LA + 1];
#pragma unroll
        for (int i = 0; i <= LA; ++i) u[i] = raw[i] < C.n_rows ? max(raw[i], -1) : -1;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int r = (i * kTileWaves + wv) * 8 + r8;
            const uint32_t xr = gather ? uint32_t(u[i]) / uint32_t(C.top_k) : uint32_t(r);
            pa[i] = u[i] >= 0 ? uint32_t(xr * uint64_t(C.ldx)) + piece * 16 : kOutside;
            if ((lane & 7) == 0)
                ymap[parity * BM + r] =
                    u[i] < 0 ? -1 : (C.flags & PM_GROUPED_SCATTER ? u[i] : w.row0 + r);
        }
        const uint32_t sr = gather ? uint32_t(u[LA]) / uint32_t(C.top_k) : uint32_t(p_row);
        *ps = u[LA] >= 0 ? sr * uint32_t(blocks) * 4 : kOutside;
    };
    auto set_w = [&](const Where& w, uint32_t* pb) {
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            const int r = (i * kTileWaves + wv) * 8 + r8;
            // LDS slot (block j, row m) of the wave's 64 holds the weight row
            // that gives a lane adjacent outputs: 16 (8 with gate and up)
            const int s = r & 63, j = s >> 4, m = s & 15;
            int o, row;
            if constexpr (GLU) {
                o = w.o0 + (r >> 6) * 32 + (m >> 2) * 8 + (j >> 1) * 4 + (m & 3);
                row = j & 1 ? out + o : o;
            } else {
                o = w.o0 + (r & ~63) + (m >> 2) * 16 + j * 4 + (m & 3);
                row = o;
            }
            pb[i] = o < out ? uint32_t(row) * uint32_t(C.cols) + piece * 16 : kOutside;
        }
    };
    auto buffer_of = [&](const void* p, size_t n) {
        return __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<char*>(static_cast<const char*>(p))), 0,
            uni(int(uint32_t(min(n, size_t(kOutside))))), kRawBuffer);
    };
    auto x_last = [&](const Where& w) { return size_t(gather ? (C.n_rows - 1) / C.top_k : w.n - 1); };
    auto x_buffer = [&](const Where& w) {
        return buffer_of(static_cast<const char*>(C.x) + (gather ? 0 : size_t(w.row0) * C.ldx),
                         w.n == 0 ? 0 : x_last(w) * C.ldx + C.cols);
    };
    auto s_buffer = [&](const Where& w) {
        return buffer_of(C.xscales8 + (gather ? 0 : size_t(w.row0) * blocks),
                         w.n == 0 ? 0 : (x_last(w) + 1) * blocks * 4);
    };
    auto w_buffer = [&](const Where& w) {
        return buffer_of(static_cast<const char*>(C.w) + size_t(w.e) * wbytes, w.n == 0 ? 0 : wbytes);
    };
    // the scales of this wave's weight rows: the first block's address for each
    // of up to three blocks of 128 rows
    typedef const __attribute__((address_space(4))) float* Scales;
    struct WScales {
        Scales a, u0, u1;
    };
    auto w_scales = [&](const Where& w) {
        const float* base = C.wscales8 + size_t(w.e) * row_blocks * blocks;
        auto at = [&](int row) {
            return (Scales)(uni64(reinterpret_cast<uintptr_t>(
                base + size_t(min(row / 128, row_blocks - 1)) * blocks)));
        };
        WScales r;
        if constexpr (GLU) {
            r.a = at(w.o0 + wn * 32);
            r.u0 = at(out + w.o0 + wn * 32);
            r.u1 = MODE == kGluSplit ? at(out + w.o0 + wn * 32 + 127) : r.u0;
        } else {
            r.a = r.u0 = r.u1 = at(w.o0 + wn * 64);
        }
        return r;
    };

    // (stages past the last input hold zeros; a tile has at least S)
    const int T = max(S, blocks);
    uint32_t pa[LA], pb[LB], ps;
    int u[LA + 1];
    Where cur = locate(place), nxt;
    if (cur.n == 0) return;
    set_w(cur, pb);
    auto ra = x_buffer(cur), rb = w_buffer(cur), rs = s_buffer(cur);
    int kk = 0;
    // load k of the L of stage kk into `stage`: the scales, the rows of x, of W
    auto issue = [&](int stage, auto which) {
        constexpr int k = decltype(which)::value;
        char* base = smem + stage * kStage;
        const bool in = kk * kTileK + piece * 16 < C.cols;
        const int ko = kk * kTileK;
        if constexpr (k == 0)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(base + kCodes + wv * 256), 4,
                                                     kk < blocks ? ps : kOutside, kk * 4, 0, 0);
        else if constexpr (k <= LA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_void*)(base + wv * 1024 + (k - 1) * 8192), 16, in ? pa[k - 1] : kOutside,
                ko, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb, (lds_void*)(base + kStageA + wv * 1024 + (k - 1 - LA) * 8192), 16,
                in ? pb[k - 1 - LA] : kOutside, ko, 0, 0);
    };
    // the first stages, that of W in the first while the uses are on their way; the
    // last loads of the last go out between the products of the first
    load_uses(cur, u);
    asm volatile("" ::: "memory");
    for_each<LB>([&](auto k) { issue(0, std::integral_constant<int, 1 + LA + k>{}); });
    set_x(cur, u, 0, pa, &ps);
    for_each<1 + LA>([&](auto k) { issue(0, k); });
    for_each<S - 1>([&](auto i) {
        ++kk;
        for_each<(i < S - 2 ? L : NB)>([&](auto k) { issue(i + 1, k); });
    });
    // stage 0 is needed now; three stages: and stage 1 in the first step
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NB) : "memory");

    const int off0 = i16 * 128 + ((q ^ (i16 & 7)) * 16);
    const int off1 = i16 * 128 + (((4 + q) ^ (i16 & 7)) * 16);
    const int ao = wm * WM * 128, bo = kStageA + wn * 64 * 128;
    const int so = kCodes + (wm * WM + i16 * MB) * 4;
    i32x8 fa[2], fb[NB];
    f32x4 sx[MB / 4];
    f32x4 acc[MB][NB];
    int st = 0, parity = 0;
    auto read8 = [&](int at) {
        const char* base = smem + at;
        const u32x4 a = *reinterpret_cast<const u32x4*>(base + off0);
        const u32x4 b = *reinterpret_cast<const u32x4*>(base + off1);
        return join(a, b);
    };
    auto read_a = [&](int stage, int i) { return read8(stage * kStage + ao + i * 2048); };
    auto read_b = [&](int stage, int j) { return read8(stage * kStage + bo + j * 2048); };
    auto read_s = [&](int stage) {
#pragma unroll
        for (int i = 0; i < MB / 4; ++i)
            sx[i] = *reinterpret_cast<const f32x4*>(smem + stage * kStage + so + i * 16);
    };
    fb[0] = read_b(0, 0);
    fa[0] = read_a(0, 0);
#pragma unroll
    for (int j = 1; j < NB; ++j) fb[j] = read_b(0, j);
    fa[1] = read_a(0, 1);
    read_s(0);

    for (int tile = place; cur.n > 0; tile += gridDim.x) {
        // the next tile's place and uses, long before its first loads
        nxt = locate(tile + gridDim.x);
        load_uses(nxt, u);
        const bool act = cur.n > wm * WM;
        const WScales wsc = w_scales(cur);
        // up rows past the border of a block of 128 rows, bit (j / 2) * 4 + r
        uint32_t beyond = 0;
        if constexpr (MODE == kGluSplit) {
            const int first = out + cur.o0 + wn * 32;
            const int border = first / 128 * 128 + 128;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (first + q * 8 + k >= border) beyond |= 1u << k;
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        // products whose sums are still to be added, and their factors
        f32x4 d1 = {0.f, 0.f, 0.f, 0.f}, d2 = d1, f1 = d1, f2 = d1;
        auto add = [&](f32x4& to, const f32x4& d, const f32x4& f) {
#pragma unroll
            for (int r = 0; r < 4; ++r) to[r] = fmaf(d[r], f[r], to[r]);
            // (here and not later: a result waiting for its sum holds registers)
            asm volatile("" : "+v"(to));
        };
        // the scales of W: loaded a stage ahead
        float na = 0.0f, nu0 = 0.0f, nu1 = 0.0f;
        auto next_scales = [&](int b) {
            na = wsc.a[b];
            if (GLU) nu0 = wsc.u0[b];
            if (MODE == kGluSplit) nu1 = wsc.u1[b];
        };
        next_scales(0);
        auto steps = [&](auto active) {
            constexpr bool ACT = decltype(active)::value;
            for (int t = 0; t < T; ++t) {
                const int after = st + 1 == S ? 0 : st + 1;
                // (none for a stage past the last input: its sums are 0, and
                // an infinite factor would make them NaN)
                const int in = t < blocks ? -1 : 0;
                auto kept = [&](float v) {
                    return __builtin_bit_cast(float, uni(__builtin_bit_cast(int, v) & in));
                };
                const float wa = kept(na), wu0 = kept(nu0), wu1 = kept(nu1);
                f32x4 wu[2];
                if constexpr (MODE == kGluSplit) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) wu[k >> 2][k & 3] = beyond >> k & 1 ? wu1 : wu0;
                }
                HalfOperand ha, hb[NATIVE ? 1 : NB];
                if constexpr (!NATIVE && ACT) {
#pragma unroll
                    for (int j = 0; j < NB; ++j) hb[j] = halves_of(fb[j]);
                }
                // product k = i * NB + j, and the sums of the product before the
                // last: its result has arrived by now
                auto step = [&](auto kc, bool last) {
                    constexpr int k = decltype(kc)::value, i = k / NB, j = k % NB;
                    if constexpr (!NATIVE && j == 0) ha = halves_of(fa[i & 1]);
                    f32x4 d;
                    if constexpr (NATIVE)
                        d = mfma_codes(fb[j], fa[i & 1]);
                    else
                        d = mfma_halves(hb[j], ha);
                    // (the product here and not later: its operands' registers
                    // are taken by the next reads)
                    asm volatile("" ::"v"(d));
                    __builtin_amdgcn_sched_barrier(0);
                    if (last) fb[j] = read_b(after, j);
                    const float x = sx[i >> 2][i & 3];
                    f32x4 f;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        f[r] = MODE == kGluSplit && (j & 1) ? wu[j >> 1][r] * x
                                                            : (GLU && (j & 1) ? wu0 : wa) * x;
                    constexpr int o = (k + NP - 2) % NP;
                    add(acc[o / NB][o % NB], d2, f2);
                    d2 = d1;
                    f2 = f1;
                    d1 = d;
                    f1 = f;
                    __builtin_amdgcn_sched_barrier(0);
                };
                __builtin_amdgcn_sched_barrier(0);
                // the rest of the loads of the stage before: a few products apart, as
                // a compute unit takes one in 16 cycles
                const int before_st = st == 0 ? S - 1 : st - 1;
                if constexpr (ACT) {
                    for_each<NP - NB>([&](auto k) {
                        step(k, false);
                        constexpr int i = k / NB;
                        if constexpr (k % kApart == kApart - 1 && k / kApart < L - NB)
                            issue(before_st, std::integral_constant<int, NB + k / kApart>{});
                        // (behind the first products: a wait for operands in LDS
                        // is one for these, too)
                        if (k == NB - 1) next_scales(min(t + 1, blocks - 1));
                        if (k % NB == NB - 1 && i + 2 < MB) fa[i & 1] = read_a(st, i + 2);
                    });
                } else {
                    for_each<L - NB>([&](auto k) {
                        issue(before_st, std::integral_constant<int, NB + k>{});
                    });
                }
                ++kk;
                __builtin_amdgcn_sched_barrier(0);
                // the next stage has arrived, and every wave has read all of this one
                // (with three stages the first step's has been waited for before the
                // last tile's stores went out: loads and stores complete in order)
                if (S > 2 && t == 0)
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                else
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * L)
                                 : "memory");
                __builtin_amdgcn_sched_barrier(0);
                // (the loads from here on are of the next stage, or the next tile)
                if (t == T - S) {
                    set_x(nxt, u, parity ^ 1, pa, &ps);
                    set_w(nxt, pb);
                    ra = x_buffer(nxt);
                    rb = w_buffer(nxt);
                    rs = s_buffer(nxt);
                    kk = 0;
                }
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (ACT) {
                    fa[MB & 1] = read_a(after, 0);
                    for_each<NB>([&](auto k) {
                        step(std::integral_constant<int, NP - NB + k>{}, true);
                        issue(st, k);
                    });
                    fa[(MB - 1) & 1] = read_a(after, 1);
                    read_s(after);
                } else {
                    for_each<NB>([&](auto k) { issue(st, k); });
                }
                if (!ACT && t == T - 1) {
                    // the next tile may need this wave
                    fa[0] = read_a(after, 0);
                    fa[1] = read_a(after, 1);
#pragma unroll
                    for (int j = 0; j < NB; ++j) fb[j] = read_b(after, j);
                    read_s(after);
                }
                __builtin_amdgcn_sched_barrier(0);
                st = after;
            }
            if (S > 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 3) * L + NB) : "memory");
        };
        if (act) {
            steps(std::true_type{});
            add(acc[MB - 1][NB - 2], d2, f2);
            add(acc[MB - 1][NB - 1], d1, f1);
            const int* rows = ymap + parity * BM + wm * WM + i16;
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int yr = rows[i * 16];
                if (yr < 0) continue;
                const int64_t at = int64_t(yr) * C.ldy;
                // this lane's adjacent outputs: 8 of gate and up, else 16
                float v[GLU ? 8 : 16];
#pragma unroll
                for (int j = 0; j < 4; j += GLU ? 2 : 1)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (GLU)
                            v[2 * j + r] = silu_up(acc[i][j][r], acc[i][j + 1][r]);
                        else
                            v[4 * j + r] = acc[i][j][r];
                    }
                const int o = cur.o0 + (GLU ? wn * 32 + q * 8 : wn * 64 + q * 16);
                store_row<YT, GLU ? 8 : 16>(C.y, at + o, out - o, v);
            }
        } else {
            steps(std::false_type{});
        }
        cur = nxt;
        parity ^= 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last stages' loads
#endif
}

// LDS of a workgroup: the stages, the rows of y, the table of experts.
inline size_t tile_lds(const GroupedCall& C, int bm, int stages) {
    return size_t(stages) * ((bm + kTileN) * kTileK + kScaleBytes) +
           (2 * bm + C.n_experts + 1) * sizeof(int);
}

template <int YT, bool NATIVE, int MODE, int BM, int S>
hipError_t run_tiles8(const GroupedCall& C, hipStream_t st) {
    const int out = MODE != kPlain ? C.rows / 2 : C.rows;
    const int per = MODE != kPlain ? kTileN / 2 : kTileN;
    const int nt = (out + per - 1) / per;
    const size_t lds = tile_lds(C, BM, S);
    auto* f = fp8_tile_kernel<YT, NATIVE, MODE, BM, S>;
    static std::atomic<uint64_t> allowed{0};
    hipError_t e = allow_lds(reinterpret_cast<const void*>(f), kTileMaxLds, &allowed);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / BM) * nt;
    const unsigned grid = unsigned(std::min<int64_t>(tiles, compute_units()));
    hipLaunchKernelGGL(f, dim3(grid), dim3(kTileThreads), lds, st, C, nt);
    return hipGetLastError();
}

template <int YT, bool NATIVE, int BM, int S>
hipError_t run_tiles8_mode(const GroupedCall& C, hipStream_t st) {
    if (!(C.flags & PM_GROUPED_SWIGLU)) return run_tiles8<YT, NATIVE, kPlain, BM, S>(C, st);
    if ((C.rows / 2) % 128 == 0) return run_tiles8<YT, NATIVE, kGlu, BM, S>(C, st);
    return run_tiles8<YT, NATIVE, kGluSplit, BM, S>(C, st);
}

template <int YT>
hipError_t run_exact(const GroupedCall& C, hipStream_t st) {
    return tile_lds(C, 128, 3) <= kTileMaxLds ? run_tiles8_mode<YT, false, 128, 3>(C, st)
                                              : run_tiles8_mode<YT, false, 128, 2>(C, st);
}

}  // namespace

bool fp8_tiles128_fit(const GroupedCall& C) { return tile_lds(C, 128, 3) <= kTileMaxLds; }

hipError_t launch_fp8_tiles(const GroupedCall& C, int rows, hipStream_t st) {
    if (fp8_cuts_off(C))
        return rows == 256 ? run_tiles8_mode<PM_BF16, true, 256, 2>(C, st)
                           : run_tiles8_mode<PM_BF16, true, 128, 3>(C, st);
    switch (C.y_type) {
    case PM_F32: return run_exact<PM_F32>(C, st);
    case PM_F16: return run_exact<PM_F16>(C, st);
    default: return run_exact<PM_BF16>(C, st);
    }
}

}  // namespace pm

// Products grouped by expert for groups of many rows: tiles of 256 or 128 rows
// by 256 outputs on the matrix cores.
//
//   D[o][m] = sum_k W[o][k] x[m][k]   (v_mfma_f32_16x16x32, fp32 sums)
//
// A persistent workgroup of 8 waves per compute unit walks over the tiles of
// the call.  A tile is 256 rows of one expert by 256 weight rows (128 gate
// and 128 up rows under PM_GROUPED_SWIGLU).  64 inputs of both (64 KiB) go
// straight from memory to LDS (buffer_load ... lds), two such stages are held,
// and the stages of the next tile follow those of this one without a break,
// so neither the first loads of a tile nor its stores stop the products.
//
// A wave computes 128 rows x 64 weight rows: 8 x 4 products of 16 x 16, 128
// accumulators (of 256-row tiles).  A stage is worked in two halves of 32 inputs; while the
// products of one half run, the operands of the next half are read from LDS
// into the other set of registers, and the loads of the stage after next are
// issued, one between every few products (a compute unit takes one 1 KiB load
// in 16 cycles; issued together they stall the products).  One barrier per
// stage.
//
// LDS holds rows of 64 inputs (128 bytes = 8 pieces); piece c of row r is
// stored at place c ^ (r % 8), so that the 16-byte reads of 8 consecutive rows
// fall in distinct banks.  The load to LDS writes lanes in order, so the
// exchange is made on the side of the global address.
//
// Inputs past `cols`, rows past the group and weight rows past the matrix are
// given an offset beyond the buffer's end: they read as zero without traffic.
// Of a tile with at most 128 rows the waves of the other half only load, and
// since every SIMD holds one wave of each half, the tile takes half the time.
//
// 128-row tiles (a wave computes 64 x 64) hold three stages: there the weights
// bound the call, and the third stage covers more of memory's latency.
//
// Measured: 65536 rows over 32 uneven experts, 2048 x 4096 bf16 with gate and
// up: 896 to 940 us, 1.2 PFLOP/s, the matrix cores 67 % busy (a large library
// product reaches 1.5 at these sizes; with all stages served by L2 this kernel
// reached 1.35).  Two stages without the half-stage pipeline gave 0.99 PFLOP/s,
// stages of 32 inputs 1.05 to 1.18, two workgroups of 128 x 256 per compute
// unit 0.97, four waves of 128 x 128 1.13.  128-row tiles: 40960 rows over 512
// experts, 4096 x 1024: 935 us, 5.0 TB/s; 1998 rows over 40 experts, 1426 x 1000
// with gate and up: 35 us, 3.4 TB/s (28 where the 116 MB stay in the last cache).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_grouped_codes.h"
#include "pm_grouped_rows.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kTileN = 256, kTileK = 64;
constexpr int kTileThreads = 512, kTileWaves = 8;

typedef __attribute__((address_space(3))) void lds_void;

// BM rows by 256 weight rows, S stages of 64 inputs in LDS.
template <int WT, int YT, bool GLU, int BM, int S>
__global__ __launch_bounds__(kTileThreads, 2) void tile_kernel(const GroupedCall C, int nt) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int kStageA = BM * kTileK * 2, kStage = kStageA + kTileN * kTileK * 2;
    constexpr int LA = BM / 64, LB = kTileN / 64, L = LA + LB;   // a wave's loads per stage
    constexpr int WM = BM / 2;                    // rows of a wave: 2 x 4 waves
    constexpr int MB = WM / 16, NB = 4, NP = MB * NB, NR = MB + NB;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    int* const ymap = reinterpret_cast<int*>(smem + S * kStage);          // [2][BM]
    int* const before = ymap + 2 * BM;                                    // [E + 1]
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int out = GLU ? C.rows / 2 : C.rows;
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
    // 128 rows, which take half the time.  (128-row tiles wait for their
    // weights, which halves would read twice.)
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
            const RowRange g = group_rows(C, e);
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
    // offsets of this lane's rows of x and of W per stage, and the buffers
    const bool gather = C.flags & PM_GROUPED_GATHER;
    const size_t wbytes = size_t(C.rows) * C.cols * 2;
    auto use_rows = [&](const Where& w, int* u) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int r = (i * kTileWaves + wv) * 8 + r8;
            u[i] = r < w.n ? use_of(C, w.row0 + r) : -1;
        }
    };
    auto set_rows = [&](const Where& w, const int* u, int parity, uint32_t* pa, uint32_t* pb) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int r = (i * kTileWaves + wv) * 8 + r8;
            const uint32_t xr = gather ? uint32_t(u[i]) / uint32_t(C.top_k) : uint32_t(r);
            pa[i] = u[i] >= 0 ? uint32_t(xr * uint64_t(C.ldx) * 2) + piece * 16 : kOutside;
            if ((lane & 7) == 0)
                ymap[parity * BM + r] =
                    u[i] < 0 ? -1 : (C.flags & PM_GROUPED_SCATTER ? u[i] : w.row0 + r);
        }
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
            pb[i] = o < out ? uint32_t(row) * uint32_t(C.cols) * 2 + piece * 16 : kOutside;
        }
    };
    const char* xbase = static_cast<const char*>(C.x);
    auto x_buffer = [&](const Where& w) {
        const char* p = gather ? xbase : xbase + size_t(w.row0) * C.ldx * 2;
        const size_t n = w.n == 0 ? 0
                                  : (size_t(gather ? (C.n_rows - 1) / C.top_k : w.n - 1) * C.ldx +
                                     C.cols) * 2;
        return __builtin_amdgcn_make_buffer_rsrc(
            uni_ptr(const_cast<char*>(p)), 0, uni(int(uint32_t(min(n, size_t(kOutside))))),
            kRawBuffer);
    };
    auto w_buffer = [&](const Where& w) {
        const char* p = static_cast<const char*>(C.w) + size_t(w.e) * wbytes;
        return __builtin_amdgcn_make_buffer_rsrc(uni_ptr(const_cast<char*>(p)), 0,
                                                 uni(w.n == 0 ? 0 : int(uint32_t(wbytes))),
                                                 kRawBuffer);
    };

    // (stages past the last input hold zeros; a tile has at least S)
    const int T = max(S, (C.cols + kTileK - 1) / kTileK);
    uint32_t pa[LA], pb[LB];
    int u[LA];
    Where cur = locate(place), nxt;
    if (cur.n == 0) return;
    use_rows(cur, u);
    set_rows(cur, u, 0, pa, pb);
    auto ra = x_buffer(cur), rb = w_buffer(cur);
    int kk = 0;
    auto issue = [&](int stage) {
        char* base = smem + stage * kStage + wv * 1024;
        const bool in = kk * kTileK + piece * 8 < C.cols;
        const int ko = kk * kTileK * 2;
#pragma unroll
        for (int i = 0; i < LA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(base + i * 8192), 16,
                                                     in ? pa[i] : kOutside, ko, 0, 0);
#pragma unroll
        for (int i = 0; i < LB; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(base + kStageA + i * 8192), 16,
                                                     in ? pb[i] : kOutside, ko, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) {
        issue(i);
        ++kk;
    }
    // stage 0 is needed now; three stages: and stage 1 in the first step
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S > 2 ? S - 2 : S - 1) * L) : "memory");

    const int off0 = i16 * 128 + ((q ^ (i16 & 7)) * 16);
    const int off1 = i16 * 128 + (((4 + q) ^ (i16 & 7)) * 16);
    const int ao = wm * WM * 128, bo = kStageA + wn * 64 * 128;
    u32x4 fa[2][MB], fb[2][NB];
    f32x4 acc[MB][NB];
    int st = 0, parity = 0;
    auto read_half = [&](int stage, int h) {
        const char* base = smem + stage * kStage + (h ? off1 : off0);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            fb[h][j] = *reinterpret_cast<const u32x4*>(base + bo + j * 2048);
#pragma unroll
        for (int i = 0; i < MB; ++i)
            fa[h][i] = *reinterpret_cast<const u32x4*>(base + ao + i * 2048);
    };
    auto products = [&](int h) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mfma_x_w<WT == PM_BF16>(fb[h][j], fa[h][i], acc[i][j]);
    };
    read_half(0, 0);

    for (int tile = place; cur.n > 0; tile += gridDim.x) {
        // the next tile's place and uses, long before its first loads
        nxt = locate(tile + gridDim.x);
        use_rows(nxt, u);
        const bool act = cur.n > wm * WM;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto steps = [&](auto active) {
            constexpr bool ACT = decltype(active)::value;
            for (int t = 0; t < T; ++t) {
                const int after = st + 1 == S ? 0 : st + 1;
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (ACT) {
                    read_half(st, 1);
                    products(0);
                    constexpr int R = (NP - 4) / NR;
                    __builtin_amdgcn_sched_group_barrier(0x8, 4, 0);
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x8, R, 0);
                    }
                    __builtin_amdgcn_sched_group_barrier(0x8, NP - 4 - NR * R, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                // the next stage has arrived, and every wave is done with this
                // one.  With three stages the first step's has been waited for
                // before the last tile's stores went out: loads and stores
                // complete in order
                if (S > 2 && t == 0)
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                else
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * L)
                                 : "memory");
                __builtin_amdgcn_sched_barrier(0);
                if (t == T - S) {
                    set_rows(nxt, u, parity ^ 1, pa, pb);
                    ra = x_buffer(nxt);
                    rb = w_buffer(nxt);
                    kk = 0;
                }
                __builtin_amdgcn_sched_barrier(0);
                issue(st);
                ++kk;
                if constexpr (ACT) {
                    read_half(after, 0);
                    products(1);
                    __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
#pragma unroll
                    for (int g = 0; g < L; ++g) {
                        __builtin_amdgcn_sched_group_barrier(0x10, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    }
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    }
                    __builtin_amdgcn_sched_group_barrier(0x8, NP - 2 - L - NR, 0);
                } else if (t == T - 1) {
                    read_half(after, 0);          // the next tile may need this wave
                }
                __builtin_amdgcn_sched_barrier(0);
                st = after;
            }
            if (S > 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 2) * L) : "memory");
        };
        if (act) {
            steps(std::true_type{});
            const int* rows = ymap + parity * BM + wm * WM + i16;
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int yr = rows[i * 16];
                if (yr < 0) continue;
                const int64_t at = int64_t(yr) * C.ldy;
                if constexpr (GLU) {
                    const int o = cur.o0 + wn * 32 + q * 8;
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        float v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = silu_up(acc[i][j][r], acc[i][j + 1][r]);
                        store4<YT>(C.y, at + o + 2 * j, out - o - 2 * j, v);
                    }
                } else {
                    const int o = cur.o0 + wn * 64 + q * 16;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                        store4<YT>(C.y, at + o + 4 * j, out - o - 4 * j, v);
                    }
                }
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
    return size_t(stages) * (bm + kTileN) * kTileK * 2 + (2 * bm + C.n_experts + 1) * sizeof(int);
}

template <int WT, int YT, bool GLU, int BM, int S>
hipError_t run_tiles(const GroupedCall& C, hipStream_t st) {
    const int out = GLU ? C.rows / 2 : C.rows;
    const int per = GLU ? kTileN / 2 : kTileN;
    const int nt = (out + per - 1) / per;
    const size_t lds = tile_lds(C, BM, S);
    auto* f = tile_kernel<WT, YT, GLU, BM, S>;
    static std::atomic<uint64_t> allowed{0};
    hipError_t e = allow_lds(reinterpret_cast<const void*>(f), kTileMaxLds, &allowed);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / BM) * nt;
    const unsigned grid = unsigned(std::min<int64_t>(tiles, compute_units()));
    hipLaunchKernelGGL(f, dim3(grid), dim3(kTileThreads), lds, st, C, nt);
    return hipGetLastError();
}

template <int BM, int S>
hipError_t run_tiles_typed(const GroupedCall& C, hipStream_t st) {
    const bool f32 = C.y_type == PM_F32;
    if (C.flags & PM_GROUPED_SWIGLU) {
        if (C.w_type == PM_F16)
            return f32 ? run_tiles<PM_F16, PM_F32, true, BM, S>(C, st)
                       : run_tiles<PM_F16, PM_F16, true, BM, S>(C, st);
        return f32 ? run_tiles<PM_BF16, PM_F32, true, BM, S>(C, st)
                   : run_tiles<PM_BF16, PM_BF16, true, BM, S>(C, st);
    }
    if (C.w_type == PM_F16)
        return f32 ? run_tiles<PM_F16, PM_F32, false, BM, S>(C, st)
                   : run_tiles<PM_F16, PM_F16, false, BM, S>(C, st);
    return f32 ? run_tiles<PM_BF16, PM_F32, false, BM, S>(C, st)
               : run_tiles<PM_BF16, PM_BF16, false, BM, S>(C, st);
}

}  // namespace

bool tiles128_fit(const GroupedCall& C) { return tile_lds(C, 128, 3) <= kTileMaxLds; }

hipError_t launch_grouped_tiles(const GroupedCall& C, int rows, hipStream_t st) {
    return rows == 128 ? run_tiles_typed<128, 3>(C, st) : run_tiles_typed<256, 2>(C, st);
}

}  // namespace pm

// Products grouped by expert of 8-bit weights and activations, for groups of
// few rows: the weights streamed through registers once, as in
// pm_grouped_stream.h, whose walk over the groups and row tiles this is.
//
//   y[v][o] = sum_b sw[o/128][b] sx[v][b] sum of W[o][k] x[v][k] over block b
//
// Bound by reading the weights.  A wave keeps up to 16 rows of x as halves
// (exact) for its share of the inputs, KB blocks of 128; a row tile of 16 weight
// rows (8 gate and 8 up rows under PM_GROUPED_SWIGLU) costs it two 16-byte loads
// per lane and block, 16 conversions of two codes to halves, four
// v_mfma_f32_16x16x32_f16, and one fma per sum with the block's factor sw * sx.
// The weights are the left operand: a lane's four sums are four adjacent
// outputs of one row of x, so sx is one register per block and lane, sw (one for
// four outputs that begin at a multiple of four rows) one value loaded with the
// weights.
//
// 8 tokens of 512 experts, top-10, 2048 x 4096, gate and up: 116 to 120 us, 5.2 to 5.4
// TB/s; 64 tokens, top-10, 4096 x 1024: 286, 5.4.  (A plain product of two large
// vectors reaches 6.2.)  The matrix cores are 7 % busy; waves wait for memory.  Two
// row tiles of 4 blocks in registers, one at work: four, with x converted anew for
// each, spill and are slower.
#include <hip/hip_runtime.h>

#include "pm_fp8.h"
#include "pm_grouped_stream.h"

namespace pm {

namespace {

// N adjacent scales.
template <int N>
struct Scales8 {
    uint32_t v[N];
};
template <int N>
__device__ inline Scales8<N> load_scales(__amdgpu_buffer_rsrc_t buf, uint32_t at) {
    Scales8<N> r;
    if constexpr (N == 4) {
        const u32x4 d = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[i] = d[i];
    } else if constexpr (N == 2) {
        const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(buf, at, 0, 0));
        r.v[0] = d[0];
        r.v[1] = d[1];
    } else {
        r.v[0] = __builtin_amdgcn_raw_buffer_load_b32(buf, at, 0, 0);
    }
    return r;
}

// SPLIT: a lane's four up rows may lie on both sides of a border between blocks
// of 128 rows (gate and up where rows / 2 is not a multiple of 4).
template <int NW, int KB, bool SPLIT>
__global__ __launch_bounds__(NW * kWave, 2) void fp8_stream_kernel(const GroupedCall C,
                                                                   const StreamPlan P) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int kLoads = KB * 2;
    // row tiles held in registers: one at work, the others on their way
    constexpr int kSlots = KB == 4 ? 2 : 4;
    constexpr int kThreads = NW * kWave, kLogNW = NW == 8 ? 3 : 2;
    // sums of a chunk: [buffer][wave][row tile][column of x][16]
    constexpr int kPart = kSteps * 256;
    __shared__ __attribute__((aligned(16))) float part[2][NW][kPart];
    __shared__ int use_row[2][16];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, q = lane >> 4;
    const int kw = 1 << P.kw_log, rw = NW >> P.kw_log;
    const int ks = wv & (kw - 1), rg = wv >> P.kw_log;
    const bool glu = C.flags & PM_GROUPED_SWIGLU, gather = C.flags & PM_GROUPED_GATHER;
    const int out = glu ? C.rows / 2 : C.rows;
    const int per_tile = glu ? 8 : 16;
    const int blocks = (C.cols + 127) / 128, row_blocks = (C.rows + 127) / 128;

    // a short call's uses are loaded along with the offsets
    const bool few = C.n_rows <= kWave;
    const int u_few = few && lane < C.n_rows ? use_of(C, lane) : -1;
    Eight eight;
    const TileScan scan = scan_tiles<16>(C, &eight);
    // few groups: a whole number of workgroups each; else equal parts of the
    // sequence
    const int wps = scan.total > 0 ? int(gridDim.x) / scan.total : 0;
    const bool apart = wps >= 8;
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
    TileRows g = find_tile_rows<16>(C, scan, mt, &eight);

    const size_t w_bytes = size_t(C.rows) * C.cols;
    const size_t scales = size_t(row_blocks) * blocks;
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
            uni_ptr(const_cast<float*>(C.wscales8) + size_t(g.e) * scales), 0,
            int(uint32_t(scales * 4)), kRawBuffer);

        // ---- the stream of row tiles: chunk by chunk, panel by panel
        u32x4 w[kSlots][kLoads];
        Scales8<KB> sc[kSlots], sd[SPLIT ? kSlots : 1];
        auto matrix_row = [&](int rt, int m) {             // row m of row tile rt
            const int o = rt * per_tile + (glu ? m & 7 : m);
            return rt < rt1 && o < out ? (glu && m >= 8 ? out + o : o) : -1;
        };
        auto first_block = [&](int panel) { return (panel * kw + ks) * KB; };
        auto issue = [&](auto slot, int rt, int panel) {
            constexpr int S = decltype(slot)::value;
            const int row = matrix_row(rt, i16);
            const int kb = first_block(panel);
            const bool some = kb < blocks;
            const uint32_t at =
                chosen(row >= 0 && some, uint32_t(row) * uint32_t(C.cols) + kb * 128 + q * 16);
            // Past `cols` these are the next row's: see multiply
#pragma unroll
            for (int s = 0; s < kLoads; ++s)
                w[S][s] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(wbuf, at + s * 64, 0, 2));
            // of the first of this lane's four rows (and of the last)
            auto scale_at = [&](int m) {
                const int r = matrix_row(rt, m);
                return chosen(r >= 0 && some, (uint32_t(r) / 128 * uint32_t(blocks) + kb) * 4);
            };
            sc[S] = load_scales<KB>(sbuf, scale_at(4 * q));
            if constexpr (SPLIT) {
                // (rows behind the last output have no scale: not used)
                const int o = rt * per_tile + (4 * q & 7);
                sd[S] = load_scales<KB>(sbuf, scale_at(4 * q + max(min(3, out - 1 - o), 0)));
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

        // ---- activations of this wave's inputs, as matrix operands
        int vlog = 2;
        while ((1 << vlog) < g.n) ++vlog;
        if (wv == 0 && lane < g.n)
            use_row[seg][lane] =
                u_lane < 0 ? -1 : (C.flags & PM_GROUPED_SCATTER ? u_lane : g.row0 + lane);
        HalfOperand xf[KB];
        float xs[KB];
        auto load_x = [&](int panel) {
            const int u = __shfl(u_lane, i16);
            const int64_t xr = u < 0 ? 0 : gather ? u / C.top_k : g.row0 + i16;
            const char* p = static_cast<const char*>(C.x) + xr * C.ldx;
            const float* sp = C.xscales8 + xr * blocks;
            const int kb = first_block(panel);
            int c = kb * 128 + q * 16;
            asm volatile("" : "+v"(c));                    // (addresses are not kept)
            u32x4 d[kLoads];
#pragma unroll
            for (int f = 0; f < kLoads; ++f)
                d[f] = *reinterpret_cast<const u32x4*>(p + max(min(c + f * 64, C.cols - 16), 0));
#pragma unroll
            for (int b = 0; b < KB; ++b) xs[b] = sp[min(kb + b, blocks - 1)];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool ok = u >= 0 && c + (2 * b + h) * 64 < C.cols;
                    const u32x4 v = ok ? d[2 * b + h] : u32x4{0, 0, 0, 0};
                    xf[b].k[2 * h] = codes_f16(v[0], v[1]);
                    xf[b].k[2 * h + 1] = codes_f16(v[2], v[3]);
                }
                xs[b] = u >= 0 && kb + b < blocks ? xs[b] : 0.0f;
            }
        };
        steps_to<kSlots - 2>([&](auto c) {
            issue(std::integral_constant<int, c + 1>{}, rt0 + (c + 1) * rw + rg, 0);
        });

        auto multiply = [&](auto slot, int rt, int panel, f32x4& a) {
            constexpr int S = decltype(slot)::value;
            const int kb = first_block(panel);
            // weights past the last input are of another row, and may be NaN: 0
            // in their place, and no scale
            if ((kb + KB) * 128 > C.cols) {
#pragma unroll
                for (int f = 0; f < kLoads; ++f)
                    if (kb * 128 + f * 64 + q * 16 >= C.cols) w[S][f] = u32x4{0, 0, 0, 0};
            }
            int border = 0;                                // rows past it take sd
            if constexpr (SPLIT) {
                const int r = max(matrix_row(rt, 4 * q), 0);
                border = r / 128 * 128 + 128 - r;
            }
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                __builtin_amdgcn_sched_barrier(0);
                const f32x4 d = mfma_halves(halves_of(join(w[S][2 * b], w[S][2 * b + 1])), xf[b]);
                const bool in = kb + b < blocks;
                const float f = (in ? __uint_as_float(sc[S].v[b]) : 0.0f) * xs[b];
                float f2 = f;
                if constexpr (SPLIT) f2 = (in ? __uint_as_float(sd[S].v[b]) : 0.0f) * xs[b];
#pragma unroll
                for (int r = 0; r < 4; ++r) a[r] = fmaf(d[r], SPLIT && r >= border ? f2 : f, a[r]);
            }
        };

        f32x4 acc[kSteps];
        int nlog = 0;
        while ((1 << nlog) < g.n) ++nlog;
        const int plog = glu ? 3 : 4;
        // row tiles of a wave per chunk, and floats of one
        const int clog = P.panels > 1 ? 2 : min(4, 6 - vlog);
        const int tile_floats = 16 << vlog;
        if (C.cols > 0) load_x(0);
        bool first = true;
        for (int rtb = rt0, step = 0; rtb < rt1; rtb += rw << clog) {
            int here = 0;                                  // row tiles of the chunk so far
            do {
#pragma unroll
                for (int c = 0; c < kSteps; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
                for (int panel = 0; panel < P.panels; ++panel) {
                    if (P.panels > 1 && !first) load_x(panel);
                    first = false;
                    steps_to<kSteps>([&](auto c) {
                        constexpr int kNext = (c + kSlots - 1) % kSlots;
                        issue_step(std::integral_constant<int, kNext>{}, c + kSlots - 1, step, panel);
                        __builtin_amdgcn_sched_barrier(0);
                        const int rt = rt0 + (step + c) * rw + rg;
                        if (C.cols > 0 && rt < rt1)
                            multiply(std::integral_constant<int, c % kSlots>{}, rt, panel, acc[c]);
                        // registers: a row tile's halves live in its own step
                        __builtin_amdgcn_sched_barrier(0);
                    });
                }
                // column i16, sums 4q .. 4q + 3
                if (i16 < 1 << vlog) {
#pragma unroll
                    for (int c = 0; c < kSteps; ++c)
                        *reinterpret_cast<f32x4*>(
                            &part[buf][wv][(here + c) * tile_floats + i16 * 16 + 4 * q]) = acc[c];
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
                const float* p = &part[buf][(t & (rw - 1)) << P.kw_log]
                                      [(t >> (kLogNW - P.kw_log)) * tile_floats + r * 16 + col];
                f32x4 p0 = {0.f, 0.f, 0.f, 0.f}, p1 = p0;
#pragma unroll 2
                for (int k = 0; k < kw; ++k, p += kPart) {
                    p0 += *reinterpret_cast<const f32x4*>(p);
                    if (glu) p1 += *reinterpret_cast<const f32x4*>(p + 8);
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
        g = find_tile_rows<16>(C, scan, ++mt, nullptr);
    }
#endif
}

template <int NW, int KB>
hipError_t run_stream8(const GroupedCall& C, const StreamPlan& P, hipStream_t st) {
    const int64_t tiles = int64_t(std::min(C.n_rows, C.n_experts)) + C.n_rows / 16;
    const int64_t most = int64_t(compute_units()) * (8 / NW);
    const bool split = (C.flags & PM_GROUPED_SWIGLU) && C.rows / 2 % 4 != 0;
    auto* f = split ? &fp8_stream_kernel<NW, KB, true> : &fp8_stream_kernel<NW, KB, false>;
    hipLaunchKernelGGL(f, dim3(unsigned(std::min<int64_t>(tiles * P.row_tiles, most))),
                       dim3(NW * kWave), 0, st, C, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_stream(const GroupedCall& C, hipStream_t st) {
    int nw, kb;
    const StreamPlan P = plan_stream(C, &nw, &kb);
    if (nw == 8) return run_stream8<8, 4>(C, P, st);
    switch (kb) {
    case 1: return run_stream8<4, 1>(C, P, st);
    case 2: return run_stream8<4, 2>(C, P, st);
    default: return run_stream8<4, 4>(C, P, st);
    }
}

}  // namespace pm

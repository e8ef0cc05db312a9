// Router on the device: top-k of each token's logits, softmax over the
// selected, and the uses sorted by expert (stable: ascending use number).
//
// Two launches.  route_kernel: one wave per token, a block of tokens per
// workgroup; it leaves ids, weights and, per block, how many uses every
// expert got.  scatter_kernel: one wave per block; the place of a use is the
// exclusive sum of the counts over (expert, block) plus its rank among the
// uses of its block with the same expert.  Counts are integers and ranks
// come from ballots, so the order never depends on timing.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;

// Orders like the logits; 0 for -inf and NaN, which are never selected.
__device__ inline uint32_t order_key(float l) {
    if (!(l > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(l + 0.0f);          // -0 counts as 0
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL, int ROW_MASK>
__device__ inline uint32_t dpp_max(uint32_t v) {
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), CTRL, ROW_MASK, 0xF,
                                                            false));
    return v > o ? v : o;
}

// Maximum over the wave, in every lane.
__device__ inline uint32_t wave_max(uint32_t v) {
    v = dpp_max<0xB1, 0xF>(v);
    v = dpp_max<0x4E, 0xF>(v);
    v = dpp_max<0x141, 0xF>(v);
    v = dpp_max<0x140, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    return __builtin_amdgcn_readlane(v, 63);
}

__device__ inline double wave_sum_f64(double v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// The selection of one token by one wave: lane j < top_k gets selected slot
// j's id (-1: none) and weight.
template <int VPT, int TYPE>
__device__ inline void select_topk(const RouteCall& C, int t, int lane, int* id_out,
                                   float* w_out) {
    uint32_t key[VPT];
    const int64_t base = int64_t(t) * C.ld;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = v * kWave + lane;
        key[v] = e < C.n_experts ? order_key(load_f32<TYPE>(C.logits, base + e)) : 0u;
    }
    int id = -1;
    uint32_t sel = 0;
    for (int j = 0; j < C.top_k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < VPT; ++v) m = m > key[v] ? m : key[v];
        m = wave_max(m);
        if (m == 0) break;                                  // nothing left to select
        // the lowest expert of the largest key: experts ascend with v, then lane
        int e = -1;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const uint64_t hit = __ballot(key[v] == m);
            if (e < 0 && hit) {
                const int l = __builtin_ctzll(hit);
                e = v * kWave + l;
                if (lane == l) key[v] = 0;
            }
        }
        if (lane == j) {
            id = e;
            sel = m;
        }
    }
    const uint32_t top = __builtin_amdgcn_readlane(sel, 0);
    double x = 0.0;
    if (id >= 0) x = sel == top ? 1.0 : exp(double(key_value(sel)) - double(key_value(top)));
    const double sum = wave_sum_f64(x);
    *id_out = id;
    *w_out = id >= 0 ? float(x / sum) : 0.0f;
}

template <int VPT, int TYPE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteCall C) {
    extern __shared__ uint32_t hist[];                      // [n_experts]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const bool sort = C.offsets != nullptr;
    if (sort) {
        for (int e = threadIdx.x; e < C.n_experts; e += kRouteThreads) hist[e] = 0;
        __syncthreads();
    }
    const int t0 = blockIdx.x * C.block_tokens;
    const int t1 = min(C.n_tokens - t0, C.block_tokens) + t0;
    for (int t = t0 + wv; t < t1; t += kRouteWaves) {
        int id;
        float w;
        select_topk<VPT, TYPE>(C, t, lane, &id, &w);
        if (lane < C.top_k) {
            const size_t u = size_t(t) * C.top_k + lane;
            C.ids[u] = id;
            C.w[u] = w;
            if (sort && id >= 0) atomicAdd(&hist[id], 1u);
        }
    }
    if (sort) {
        __syncthreads();
        for (int e = threadIdx.x; e < C.n_experts; e += kRouteThreads)
            C.hist[size_t(blockIdx.x) * C.n_experts + e] = uint16_t(hist[e]);
    }
}

// Sum over the lanes below this one.
__device__ inline uint32_t wave_prefix(uint32_t v, int lane) {
    uint32_t s = v;
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    return s - v;
}

// nb blocks of tokens per workgroup, one wave each.  LDS: next[nb][E], the
// place of the next use of (block, expert).
__global__ __launch_bounds__(kRouteThreads) void scatter_kernel(const RouteCall C, int nb) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_tot[kRouteWaves];
    const int E = C.n_experts;
    uint32_t* next = lds;                                   // [nb][E]
    uint32_t* tot = lds + size_t(nb) * E;                   // [E]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int b0 = blockIdx.x * nb, b1 = min(b0 + nb, C.n_blocks);
    // column sums: the blocks before ours, ours, and all
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        uint32_t s = 0;
        for (int b = 0; b < C.n_blocks; ++b) {
            if (b >= b0 && b < b1) next[(b - b0) * E + e] = s;
            s += C.hist[size_t(b) * E + e];
        }
        tot[e] = s;
    }
    __syncthreads();
    // exclusive sum over the experts: 1024 threads, consecutive chunks
    const int per = (E + kRouteThreads - 1) / kRouteThreads;
    const int e0 = min(int(threadIdx.x) * per, E), e1 = min(e0 + per, E);
    uint32_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += tot[e];
    const uint32_t before = wave_prefix(mine, lane);
    if (lane == 63) wave_tot[wv] = before + mine;
    __syncthreads();
    uint32_t at = before;
    for (int w = 0; w < wv; ++w) at += wave_tot[w];
    for (int e = e0; e < e1; ++e) {
        const uint32_t n = tot[e];
        if (blockIdx.x == 0) {
            C.offsets[e] = int32_t(at);
            if (e == E - 1) C.offsets[E] = int32_t(at + n);
        }
        for (int b = b0; b < b1; ++b) next[(b - b0) * E + e] += at;
        at += n;
    }
    __syncthreads();
    if (wv >= b1 - b0) return;
    const int b = b0 + wv;
    uint32_t* mynext = next + size_t(wv) * E;
    const size_t u0 = size_t(b) * C.block_tokens * C.top_k;
    const size_t u1 = min(size_t(C.n_tokens), size_t(b + 1) * C.block_tokens) * C.top_k;
    const int bits = 32 - __builtin_clz(E);
    for (size_t u = u0; u < u1; u += kWave) {
        const int id = u + lane < u1 ? C.ids[u + lane] : -1;
        uint64_t same = __ballot(id >= 0);
        for (int k = 0; k < bits; ++k) {
            const uint64_t on = __ballot((id >> k) & 1);
            same &= (id >> k) & 1 ? on : ~on;
        }
        if (id >= 0) {
            const uint32_t rank = __builtin_amdgcn_mbcnt_hi(uint32_t(same >> 32),
                                      __builtin_amdgcn_mbcnt_lo(uint32_t(same), 0));
            const uint32_t p = mynext[id];
            C.order[p + rank] = int32_t(u + lane);
            // the group's last lane moves the place on
            if (rank + 1 == uint32_t(__popcll(same))) mynext[id] = p + rank + 1;
        }
    }
}

__global__ void route_nothing_kernel(const RouteCall C) {
    for (int e = threadIdx.x; e <= C.n_experts; e += blockDim.x) C.offsets[e] = 0;
}

template <int VPT>
hipError_t launch_select(const RouteCall& C, hipStream_t st) {
    const dim3 grid(C.n_blocks), block(kRouteThreads);
    const size_t lds = C.offsets ? size_t(C.n_experts) * 4 : 0;
    switch (C.type) {
    case PM_F32: hipLaunchKernelGGL((route_kernel<VPT, PM_F32>), grid, block, lds, st, C); break;
    case PM_F16: hipLaunchKernelGGL((route_kernel<VPT, PM_F16>), grid, block, lds, st, C); break;
    default: hipLaunchKernelGGL((route_kernel<VPT, PM_BF16>), grid, block, lds, st, C); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteCall& C, hipStream_t st) {
    if (C.n_tokens == 0) {
        hipLaunchKernelGGL(route_nothing_kernel, dim3(1), dim3(256), 0, st, C);
        return hipGetLastError();
    }
    const int per_lane = (C.n_experts + kWave - 1) / kWave;
    hipError_t e;
    if (per_lane <= 1) e = launch_select<1>(C, st);
    else if (per_lane <= 2) e = launch_select<2>(C, st);
    else if (per_lane <= 4) e = launch_select<4>(C, st);
    else if (per_lane <= 8) e = launch_select<8>(C, st);
    else if (per_lane <= 16) e = launch_select<16>(C, st);
    else e = launch_select<64>(C, st);
    if (e != hipSuccess || !C.offsets) return e;
    // LDS: (nb + 1) x E words, 60 KiB at most (E <= 4096: nb >= 2)
    const int nb = std::max(1, std::min(kRouteWaves, 15360 / C.n_experts - 1));
    const unsigned grid = unsigned((C.n_blocks + nb - 1) / nb);
    hipLaunchKernelGGL(scatter_kernel, dim3(grid), dim3(kRouteThreads),
                       size_t(nb + 1) * C.n_experts * 4, st, C, nb);
    return hipGetLastError();
}

}  // namespace pm

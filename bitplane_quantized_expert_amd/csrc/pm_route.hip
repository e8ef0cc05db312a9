// Router on the device: top-k of each token's logits, softmax over the
// selected, and the uses sorted by expert (stable: ascending use number).
//
// Selection, one wave per token: a lane holds every 64th logit as an integer
// that orders like it.  The top_k-th largest of the 64 lanes' own maxima, found
// bit by bit with ballots, is a bound that the whole top-k meets and few other
// logits do (two or three of 512); those that meet it are inserted one by one
// into a list that lies sorted across the lanes: about half the vector
// instructions of ten rounds of a wave maximum with removal, for top-10 of 512.
// The softmax (fp64) of up to 4 tokens is taken together, 16 lanes each.
//
// Sorting: calls of few tokens do it in the same launch, in LDS.  Larger
// ones leave, per block of tokens, how many uses every expert got, and
// scatter_kernel adds up the columns of that table: the place of a use is the
// sum over lower experts and earlier blocks, plus its rank among the uses of
// its block with the same expert.  Counts are integers and ranks come from
// ballots, so the order never depends on timing.
//
// Measured (kernel time): 1 token, 512 experts, top-10: 5.6 us in one launch,
// bound by the chain of dependent steps of one wave.  1003 tokens, 60 experts,
// top-4: 4.9 + 6.1 us.  16384 tokens, 512 experts, top-10: 16.1 us (33.6 MB of
// logits, 2.1 TB/s) + 11.5 us of sorting, of which adding up the table's columns
// in every workgroup is the most.  The selection takes 259 vector and 212 scalar
// instructions per token (loads and softmax among them): the vector units are
// busy half of the time, and the waves, 4 on a SIMD, wait for 56 % of theirs, for
// the ballots and insertions of a token follow from one another.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pm_convert.h"
#include "pm_device.h"
#include "pm_routed.h"

namespace pm {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;

// Waves of a workgroup that selects: 32 and 64 logits per lane need up to 256
// registers (with 16 waves, spilled: 67 us for 24 tokens of 4096 experts, now 41;
// of 1500, 56 and now 14).
constexpr int select_waves(int vpt) { return vpt > 32 ? 4 : vpt > 16 ? 8 : kRouteWaves; }

// Orders like the logits; 0 for -inf and NaN, which are never selected.
__device__ inline uint32_t order_key(float l) {
    if (!(l > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(l + 0.0f);          // -0 counts as 0
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL>
__device__ inline double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(b >> 32)), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
// Sum over each 16 lanes, in every lane.
__device__ inline double row16_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    return v;
}

// Every 64th logit of token t, from logit `lane` on.
template <int VPT>
struct Logits {
    float v[VPT];
};
template <int VPT, int TYPE>
__device__ inline Logits<VPT> load_logits(const RouteCall& C, int t, int lane) {
    Logits<VPT> l;
    const int64_t base = int64_t(t) * C.ld;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        l.v[v] = load_f32<TYPE>(C.logits, base + min(v * kWave + lane, C.n_experts - 1));
    return l;
}

// The selection of one token by one wave: lane j < top_k gets the expert and
// key of slot j (key 0: none).
template <int VPT>
__device__ inline void select_topk(const RouteCall& C, const Logits<VPT>& logits, int lane,
                                   uint32_t* key_out, int* id_out) {
    uint32_t key[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        key[v] = v * kWave + lane < C.n_experts ? order_key(logits.v[v]) : 0u;
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < VPT; ++v) m = m > key[v] ? m : key[v];
    // a bound that top_k lanes meet: the largest, or any that just top_k meet
    uint32_t bound = 0;
    for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
        const uint32_t c = bound | bit;
        const int n = __popcll(__ballot(m >= c));
        if (n >= C.top_k) bound = c;
        if (n == C.top_k) break;
    }
    bound = bound ? bound : 1u;
    // list across the lanes, descending: (key, ~expert), 0 for none
    uint32_t mine = 0, low = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        uint64_t hit = __ballot(key[v] >= bound);
        while (hit) {
            const int l = __builtin_ctzll(hit);
            hit &= hit - 1;
            const uint32_t k = __builtin_amdgcn_readlane(key[v], l);
            const uint32_t ne = ~uint32_t(v * kWave + l);
            // lanes that come after it move up by one, the first takes it
            const bool after = (uint64_t(mine) << 32 | low) < (uint64_t(k) << 32 | ne);
            const uint64_t mask = __ballot(after);
            if (mask == 0) continue;
            const int first = __builtin_ctzll(mask);
            if (after) {
                mine = __builtin_amdgcn_update_dpp(int(mine), int(mine), 0x138, 0xF, 0xF, false);
                low = __builtin_amdgcn_update_dpp(int(low), int(low), 0x138, 0xF, 0xF, false);
            }
            mine = lane == first ? k : mine;
            low = lane == first ? ne : low;
        }
    }
    *key_out = lane < C.top_k ? mine : 0;
    *id_out = lane < C.top_k && mine ? int(~low) : -1;
}

// ids and weights of tokens t0, t0 + step, .. of one wave; f(u, id) for each
// lane with a use (id >= 0).
template <int VPT, int TYPE, class F>
__device__ inline void route_tokens(const RouteCall& C, int t0, int t1, int step, int lane, F&& f) {
    // up to 4 tokens share one softmax where 16 lanes hold a token's slots
    const int group = C.top_k <= 16 ? 4 : 1;
    if (t0 >= t1) return;
    Logits<VPT> next = load_logits<VPT, TYPE>(C, t0, lane);
    for (int t = t0; t < t1; t += group * step) {
        uint32_t key = 0, top = 0;
        int id = -1, tok = 0, slot = kWave;
        for (int s = 0; s < group && t + s * step < t1; ++s) {
            uint32_t k;
            int i;
            const Logits<VPT> now = next;
            // the next token's logits are on their way meanwhile
            next = load_logits<VPT, TYPE>(C, min(t + (s + 1) * step, t1 - 1), lane);
            select_topk<VPT>(C, now, lane, &k, &i);
            const uint32_t first = __builtin_amdgcn_readlane(k, 0);
            if (group == 1) {
                key = k;
                id = i;
                slot = lane;
            } else {
                const uint32_t ks = __shfl(k, lane & 15);
                const int is = __shfl(i, lane & 15);
                if (lane >> 4 != s) continue;
                key = ks;
                id = is;
                slot = lane & 15;
            }
            top = first;
            tok = t + s * step;
        }
        double x = 0.0;
        if (key) x = key == top ? 1.0 : exp(double(key_value(key)) - double(key_value(top)));
        double sum = row16_sum_f64(x);
        if (group == 1) {
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
        }
        if (slot < C.top_k) {
            const int64_t u = int64_t(tok) * C.top_k + slot;
            C.ids[u] = key ? id : -1;
            C.w[u] = key ? float(x / sum) : 0.0f;
            if (key) f(u, id);
        }
    }
}

template <int VPT, int TYPE>
__global__ __launch_bounds__(kWave * select_waves(VPT)) void route_kernel(const RouteCall C) {
    extern __shared__ uint32_t hist[];                      // [n_experts]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const bool sort = C.offsets != nullptr;
    if (sort) {
        for (int e = threadIdx.x; e < C.n_experts; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    const int t0 = blockIdx.x * C.block_tokens;
    const int t1 = min(C.n_tokens - t0, C.block_tokens) + t0;
    route_tokens<VPT, TYPE>(C, t0 + wv, t1, blockDim.x >> 6, lane, [&](int64_t, int id) {
        if (sort) atomicAdd(&hist[id], 1u);
    });
    if (sort) {
        __syncthreads();
        uint16_t* row = C.hist + size_t(blockIdx.x) * C.hist_stride;
        for (int e = threadIdx.x; e < C.hist_stride; e += blockDim.x)
            row[e] = e < C.n_experts ? uint16_t(hist[e]) : uint16_t(0);
    }
}

// Exclusive sum over the E counts of LDS, by the whole workgroup; returns the
// sum below the thread's first expert, of `per` adjacent ones.
__device__ inline uint32_t scan_experts(const uint32_t* count, int E, int per, uint32_t* wave_tot) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int e0 = min(int(threadIdx.x) * per, E), e1 = min(e0 + per, E);
    uint32_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += count[e];
    uint32_t s = mine;
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    if (lane == 63) wave_tot[wv] = s;
    __syncthreads();
    uint32_t at = s - mine;
    for (int w = 0; w < wv; ++w) at += wave_tot[w];
    return at;
}

// Places 64 uses: `next` is the place of the next use of each expert.
__device__ inline void place_uses(int32_t* order, uint32_t* next, int id, int64_t u, int bits) {
    uint64_t same = __ballot(id >= 0);
    for (int k = 0; k < bits; ++k) {
        const uint64_t on = __ballot((id >> k) & 1);
        same &= (id >> k) & 1 ? on : ~on;
    }
    if (id >= 0) {
        const uint32_t rank = __builtin_amdgcn_mbcnt_hi(
            uint32_t(same >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(same), 0));
        const uint32_t p = next[id];
        order[p + rank] = int32_t(u);
        // the group's last lane moves the place on
        if (rank + 1 == uint32_t(__popcll(same))) next[id] = p + rank + 1;
    }
}

// A call of few tokens by one workgroup, sorted in LDS.
template <int VPT, int TYPE>
__global__ __launch_bounds__(kWave * select_waves(VPT)) void route_small_kernel(const RouteCall C) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_tot[kRouteWaves];
    const int E = C.n_experts, n = C.n_tokens * C.top_k;
    uint32_t* count = lds;                                  // [E]
    int* ids = reinterpret_cast<int*>(lds + E);             // [n_tokens * top_k]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
    for (int u = threadIdx.x; u < n; u += blockDim.x) ids[u] = -1;
    __syncthreads();
    route_tokens<VPT, TYPE>(C, wv, C.n_tokens, blockDim.x >> 6, lane, [&](int64_t u, int id) {
        atomicAdd(&count[id], 1u);
        ids[u] = id;
    });
    __syncthreads();
    const int per = (E + blockDim.x - 1) / blockDim.x;
    uint32_t at = scan_experts(count, E, per, wave_tot);
    const int e0 = min(int(threadIdx.x) * per, E), e1 = min(e0 + per, E);
    for (int e = e0; e < e1; ++e) {
        const uint32_t c = count[e];
        C.offsets[e] = int32_t(at);
        count[e] = at;
        at += c;
        if (e == E - 1) C.offsets[E] = int32_t(at);
    }
    __syncthreads();
    if (wv != 0) return;
    const int bits = 32 - __builtin_clz(E);
    for (int u = lane; u - lane < n; u += kWave)
        place_uses(C.order, count, u < n ? ids[u] : -1, u, bits);
}

// `subs` waves per workgroup, `spb` of them for each block of tokens.  LDS:
// next[subs][E], the place of the next use of (wave, expert); total[E];
// earlier[E].
__global__ __launch_bounds__(kRouteThreads) void scatter_kernel(const RouteCall C, int subs, int spb) {
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_tot[kRouteWaves];
    const int E = C.n_experts;
    uint32_t* next = lds;
    uint32_t* total = lds + size_t(subs) * E;
    uint32_t* earlier = total + E;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < (subs + 2) * E; i += kRouteThreads) lds[i] = 0;
    __syncthreads();
    const int nb = subs / spb;
    const int b0 = blockIdx.x * nb;
    // the columns: 8 experts per lane and load, the blocks over the waves, 8
    // loads on their way
    const int octs = C.hist_stride / 8;
    const u32x4* table = reinterpret_cast<const u32x4*>(C.hist);
    for (int c = lane; c - lane < octs; c += kWave) {
        uint32_t all[8] = {}, old[8] = {};
        for (int b = wv; b < C.n_blocks; b += 8 * kRouteWaves) {
            u32x4 h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                h[k] = table[size_t(min(b + k * kRouteWaves, C.n_blocks - 1)) * octs +
                             min(c, octs - 1)];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = b + k * kRouteWaves;
                if (at >= C.n_blocks) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    all[2 * i] += h[k][i] & 0xFFFFu;
                    all[2 * i + 1] += h[k][i] >> 16;
                }
                if (at < b0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        old[2 * i] += h[k][i] & 0xFFFFu;
                        old[2 * i + 1] += h[k][i] >> 16;
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (8 * c + k < E) {
                atomicAdd(&total[8 * c + k], all[k]);
                atomicAdd(&earlier[8 * c + k], old[k]);
            }
    }
    // this wave's uses: a part of its block
    const int b = b0 + (wv >> (31 - __builtin_clz(spb)));
    // (all uses are below 2^31, sums of two below 2^32)
    const uint32_t block_uses = uint32_t(C.block_tokens) * C.top_k;
    const uint32_t all_uses = uint32_t(C.n_tokens) * C.top_k;
    const uint32_t start = min(uint32_t(min(b, C.n_blocks)) * block_uses, all_uses);
    const uint32_t stop = min(start + block_uses, all_uses);
    const uint32_t part = ((block_uses + kWave * spb - 1) / (kWave * spb)) * kWave;
    const uint32_t u0 = min(start + (wv & (spb - 1)) * part, stop);
    const uint32_t u1 = wv < subs ? min(u0 + part, stop) : u0;
    uint32_t* mine = next + min(wv, subs - 1) * E;
    // the first round's ids stay in a register
    const int id0 = u0 + lane < u1 ? C.ids[u0 + lane] : -1;
    if (id0 >= 0) atomicAdd(&mine[id0], 1u);
    for (uint32_t u = u0 + kWave + lane; u < u1; u += kWave) {
        const int id = C.ids[u];
        if (id >= 0) atomicAdd(&mine[id], 1u);
    }
    __syncthreads();
    const int per = (E + kRouteThreads - 1) / kRouteThreads;
    uint32_t at = scan_experts(total, E, per, wave_tot);
    const int e0 = min(int(threadIdx.x) * per, E), e1 = min(e0 + per, E);
    for (int e = e0; e < e1; ++e) {
        const uint32_t n = total[e];
        if (blockIdx.x == 0) {
            C.offsets[e] = int32_t(at);
            if (e == E - 1) C.offsets[E] = int32_t(at + n);
        }
        uint32_t place = at + earlier[e];
        for (int w0 = 0; w0 < subs; w0 += 4) {
            uint32_t k[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) k[w] = w0 + w < subs ? next[(w0 + w) * E + e] : 0u;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w0 + w < subs) next[(w0 + w) * E + e] = place;
                place += k[w];
            }
        }
        at += n;
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(E);
    for (uint32_t u = u0; u < u1; u += kWave) {
        const int id = u == u0 ? id0 : u + lane < u1 ? C.ids[u + lane] : -1;
        place_uses(C.order, mine, id, u + lane, bits);
    }
}

__global__ void route_nothing_kernel(const RouteCall C) {
    for (int e = threadIdx.x; e <= C.n_experts; e += blockDim.x) C.offsets[e] = 0;
}

template <int VPT, int TYPE>
hipError_t launch_select_typed(const RouteCall& C, hipStream_t st) {
    // one wave per token, 16 tokens (of more than 1024 experts 8, of more than
    // 2048 4) at a time
    constexpr int kWaves = select_waves(VPT);
    const dim3 block(kWave * std::min(C.n_tokens, kWaves));
    // one launch while a wave has few tokens and the last wave few uses to place:
    // us in one against two launches at 24, 32, 48, 64 tokens: 5.9/7.6, 6.7/8.2,
    // 8.4/8.6, 9.9/8.5 (60 experts, top-4), 7.4/8.3, 8.9/8.7, 11.4/9.2, 14.2/9.3
    // (128, top-8), 9.5/11.2, 11.4/11.4, 15.5/11.5, 18.4/11.7 (512, top-10)
    if (C.offsets && (C.n_tokens <= kWaves ||
                      (C.n_tokens <= 3 * kWaves && C.n_tokens * C.top_k <= 256))) {
        const size_t lds = (size_t(C.n_experts) + size_t(C.n_tokens) * C.top_k) * 4;
        hipLaunchKernelGGL((route_small_kernel<VPT, TYPE>), dim3(1), block, lds, st, C);
        return hipGetLastError();
    }
    const size_t lds = C.offsets ? size_t(C.n_experts) * 4 : 0;
    hipLaunchKernelGGL((route_kernel<VPT, TYPE>), dim3(C.n_blocks), block, lds, st, C);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !C.offsets) return e;
    // as many waves as 60 KiB of LDS serve (E <= 4096: at least 1)
    const int fit = 15360 / C.n_experts - 2;
    const int subs = fit >= 16 ? 16 : fit >= 8 ? 8 : fit >= 4 ? 4 : fit >= 2 ? 2 : 1;
    const int spb = subs >= 16 ? 8 : subs >= 8 ? 4 : 1;
    const int nb = subs / spb;
    hipLaunchKernelGGL(scatter_kernel, dim3(unsigned((C.n_blocks + nb - 1) / nb)),
                       dim3(kRouteThreads), size_t(subs + 2) * C.n_experts * 4, st, C, subs, spb);
    return hipGetLastError();
}

template <int VPT>
hipError_t launch_select(const RouteCall& C, hipStream_t st) {
    switch (C.type) {
    case PM_F32: return launch_select_typed<VPT, PM_F32>(C, st);
    case PM_F16: return launch_select_typed<VPT, PM_F16>(C, st);
    default: return launch_select_typed<VPT, PM_BF16>(C, st);
    }
}

}  // namespace

hipError_t launch_route(const RouteCall& C, hipStream_t st) {
    if (C.n_tokens == 0) {
        hipLaunchKernelGGL(route_nothing_kernel, dim3(1), dim3(256), 0, st, C);
        return hipGetLastError();
    }
    const int per_lane = (C.n_experts + kWave - 1) / kWave;
    if (per_lane <= 1) return launch_select<1>(C, st);
    if (per_lane <= 2) return launch_select<2>(C, st);
    if (per_lane <= 4) return launch_select<4>(C, st);
    if (per_lane <= 8) return launch_select<8>(C, st);
    if (per_lane <= 16) return launch_select<16>(C, st);
    if (per_lane <= 32) return launch_select<32>(C, st);
    return launch_select<64>(C, st);
}

}  // namespace pm

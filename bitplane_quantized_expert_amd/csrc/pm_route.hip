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
// Sorting: see pm_route_sort.h.
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

#include "pm_route_sort.h"

namespace pm {

namespace {

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

// One wave per token, 16 tokens (of more than 1024 experts 8, of more than 2048
// 4) at a time.
template <int VPT, int TYPE>
struct TopkRouter {
    static constexpr int kWaves = select_waves(VPT);
    template <class F>
    __device__ static inline void tokens(const RouteCall& C, int t0, int t1, int step, int lane,
                                         F&& f) {
        route_tokens<VPT, TYPE>(C, t0, t1, step, lane, f);
    }
};

template <int VPT>
hipError_t launch_select(const RouteCall& C, hipStream_t st) {
    switch (C.type) {
    case PM_F32: return launch_routed<TopkRouter<VPT, PM_F32>>(C, st);
    case PM_F16: return launch_routed<TopkRouter<VPT, PM_F16>>(C, st);
    default: return launch_routed<TopkRouter<VPT, PM_BF16>>(C, st);
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

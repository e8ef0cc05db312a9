// Router by scores: sigmoid or softmax of every logit, a bias that only
// selects, the best groups of experts, top-k among them (include/pm.h).  All
// scores are fp64.
#include <hip/hip_runtime.h>

#include "pm_route_sort.h"

namespace pm {

namespace {

constexpr int scored_waves(int vpt) { return vpt > 16 ? 4 : vpt > 8 ? 8 : kRouteWaves; }

template <class T>
__device__ inline T wave_best(T v) {
    for (int d = 1; d < kWave; d <<= 1) {
        const T o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}

// The selection of one token by one wave.
template <int VPT, int TYPE>
__device__ inline void scored_token(const RouteCall& C, int t, int lane, int* id_out, float* w_out) {
    const pm_route_rule& r = C.rule;
    const int64_t base = int64_t(t) * C.ld;
    const bool softmax = r.score == PM_SCORE_SOFTMAX;
    const Logits<VPT> l = load_logits<VPT, TYPE>(C, t, lane);
    double c[VPT];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (v * kWave + lane < C.n_experts && l.v[v] > top) top = l.v[v];
    top = wave_best(top);
    double sum = 0.0;
    if (softmax) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (v * kWave + lane < C.n_experts && l.v[v] > -INFINITY)
                sum += l.v[v] == top ? 1.0 : exp(double(l.v[v]) - double(top));
        for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
    }
    auto score = [&](float x) {
        if (softmax) return (x == top ? 1.0 : exp(double(x) - double(top))) / sum;
        return 1.0 / (1.0 + exp(-double(x)));
    };
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = v * kWave + lane;
        c[v] = -INFINITY;
        if (e < C.n_experts && l.v[v] > -INFINITY) {
            const double b = C.bias ? double(C.bias[e]) : 0.0;
            if (b > -INFINITY) c[v] = score(l.v[v]) + b;
        }
    }
    if (r.n_groups > 1) {
        const int size = C.n_experts / r.n_groups;
        double mine = -INFINITY;                            // lane g: what group g counts
        for (int g = 0; g < r.n_groups; ++g) {
            double a = -INFINITY, b = -INFINITY;            // its two largest
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int e = v * kWave + lane;
                if (e >= g * size && e < (g + 1) * size) {
                    b = fmax(b, fmin(a, c[v]));
                    a = fmax(a, c[v]);
                }
            }
            for (int d = 1; d < kWave; d <<= 1) {
                const double oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
                b = fmax(fmax(b, ob), fmin(a, oa));
                a = fmax(a, oa);
            }
            if (lane == g) mine = r.group_best == 2 && b > -INFINITY ? a + b : a;
        }
        int better = 0;
        for (int g = 0; g < r.n_groups; ++g) {
            const double o = __shfl(mine, g);
            better += o > mine || (o == mine && g < lane);
        }
        const uint64_t keep = __ballot(mine > -INFINITY && better < r.top_groups);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (!((keep >> min((v * kWave + lane) / size, 63)) & 1)) c[v] = -INFINITY;
    }
    int id = -1;
    for (int j = 0; j < C.top_k; ++j) {
        double a = -INFINITY;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (c[v] > a) {
                a = c[v];
                at = v * kWave + lane;
            }
        const double best = wave_best(a);
        if (!(best > -INFINITY)) break;
        int first = a == best ? at : 0x7FFFFFFF;
        for (int d = 1; d < kWave; d <<= 1) first = min(first, __shfl_xor(first, d));
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (v * kWave + lane == first) c[v] = -INFINITY;
        if (lane == j) id = first;
    }
    double s = 0.0;
    if (id >= 0) s = score(load_f32<TYPE>(C.logits, base + id));
    double all = s;
    for (int d = 1; d < kWave; d <<= 1) all += __shfl_xor(all, d);
    if (r.flags & PM_ROUTE_RENORM) s = all > 0.0 ? s / all : 0.0;
    *id_out = id;
    *w_out = float(s * double(r.scale));
}

template <int VPT, int TYPE>
struct ScoredRouter {
    static constexpr int kWaves = scored_waves(VPT);
    template <class F>
    __device__ static inline void tokens(const RouteCall& C, int t0, int t1, int step, int lane,
                                         F&& f) {
        for (int t = t0; t < t1; t += step) {
            int id;
            float w;
            scored_token<VPT, TYPE>(C, t, lane, &id, &w);
            if (lane < C.top_k) {
                const int64_t u = int64_t(t) * C.top_k + lane;
                C.ids[u] = id;
                C.w[u] = id >= 0 ? w : 0.0f;
                if (id >= 0) f(u, id);
            }
        }
    }
};

template <int VPT>
hipError_t launch_scored(const RouteCall& C, hipStream_t st) {
    switch (C.type) {
    case PM_F32: return launch_routed<ScoredRouter<VPT, PM_F32>>(C, st);
    case PM_F16: return launch_routed<ScoredRouter<VPT, PM_F16>>(C, st);
    default: return launch_routed<ScoredRouter<VPT, PM_BF16>>(C, st);
    }
}

}  // namespace

hipError_t launch_route_scored(const RouteCall& C, hipStream_t st) {
    if (C.n_tokens == 0) {
        hipLaunchKernelGGL(route_nothing_kernel, dim3(1), dim3(256), 0, st, C);
        return hipGetLastError();
    }
    const int per_lane = (C.n_experts + kWave - 1) / kWave;
    if (per_lane <= 1) return launch_scored<1>(C, st);
    if (per_lane <= 2) return launch_scored<2>(C, st);
    if (per_lane <= 4) return launch_scored<4>(C, st);
    if (per_lane <= 8) return launch_scored<8>(C, st);
    if (per_lane <= 16) return launch_scored<16>(C, st);
    if (per_lane <= 32) return launch_scored<32>(C, st);
    return launch_scored<64>(C, st);
}

}  // namespace pm

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

// Orders like the numbers; 0 for -inf and NaN.
__device__ inline uint32_t rank_key(float c) {
    if (!(c > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(c + 0.0f);
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ inline float rank_value(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ inline float value_at(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Ranks in fp32 and what they may be off by.  The score: e^-l from v_exp_f32 has an
// error of |l| 2^-22 of it at most, 1 / (1 + e) and e / sum by v_rcp_f32 a few 2^-24
// more; so 2^-20 of 1, and 2^-16 of the score itself.  The sum with a bias is
// rounded to 2^-24 of it.  Twice that and more:
__device__ inline float rank_slack(float v, bool bias) {
    return bias ? 0x1p-18f + fabsf(v) * 0x1p-21f : fminf(0x1p-18f, v * 0x1p-14f);
}

template <int VPT>
struct Ranks {
    float c[VPT];                                   // in fp32; -inf: not selected
};

// The list of the experts with the largest ranks in fp32, sorted across the
// lanes, ties by lower id: every expert that the exact ranks may select among
// `held`, or *unsure.
template <int VPT>
__device__ inline void rank_list(const RouteCall& C, const Ranks<VPT>& r, int lane, int held,
                                 uint32_t* key_out, int* id_out, bool* unsure) {
    uint32_t key[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = rank_key(r.c[v]);
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < VPT; ++v) m = max(m, key[v]);
    // a bound that top_k lanes meet: the largest, or any that just top_k meet
    uint32_t bound = 0;
    for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
        const uint32_t c = bound | bit;
        const int n = __popcll(__ballot(m >= c));
        if (n >= C.top_k) bound = c;
        if (n == C.top_k) break;
    }
    const bool bias = C.bias != nullptr;
    if (bound) {
        const float v = rank_value(bound);
        bound = rank_key(v - rank_slack(v, bias));
    }
    bound = bound ? bound : 1u;
    // list across the lanes, descending: (key, ~expert), 0 for none
    uint32_t mine = 0, low = 0;
    int found = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        uint64_t hit = __ballot(key[v] >= bound);
        found += __popcll(hit);
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
    *unsure = false;
    if (found > held) {
        const float last = value_at(rank_value(mine), C.top_k - 1);
        *unsure = !(value_at(rank_value(mine), held - 1) < last - rank_slack(last, bias));
    }
    *key_out = mine;
    *id_out = mine ? int(~low) : -1;
}

// Takes the experts of the groups that do not stay out of the ranks; false where
// fp32 does not tell which do.  `space`: the wave's LDS, padded_at(E) floats.
__device__ inline int padded_at(int e) { return e + (e >> 3); }
template <int VPT>
__device__ inline bool rank_groups(const RouteCall& C, Ranks<VPT>& r, int lane, float* space) {
    const pm_route_rule& rule = C.rule;
    const int n = rule.n_groups, size = C.n_experts / n;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int e = v * kWave + lane;
        if (e < C.n_experts) space[padded_at(e)] = r.c[v];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // 2^log lanes per group
    const int log = 6 - (32 - __builtin_clz(n - 1));
    const int g = lane >> log, j = lane & ((1 << log) - 1);
    float a = -INFINITY, b = -INFINITY;                     // its two largest
    if (g < n)
        for (int i = j; i < size; i += 1 << log) {
            const float c = space[padded_at(g * size + i)];
            b = fmaxf(b, fminf(a, c));
            a = fmaxf(a, c);
        }
    for (int d = 1; d < 1 << log; d <<= 1) {
        const float oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
        b = fmaxf(fmaxf(b, ob), fminf(a, oa));
        a = fmaxf(a, oa);
    }
    const float mine = rule.group_best == 2 && b > -INFINITY ? a + b : a;
    const float slack = 4.0f * (0x1p-18f + fabsf(mine) * 0x1p-21f);
    // groups that count more for certain, and those that may
    int more = 0, maybe = 0;
    for (int k = 0; k < n; ++k) {
        const float o = value_at(mine, k << log);
        more += o > mine + slack;
        maybe += k != g && !(o < mine - slack);
    }
    const bool real = g < n && mine > -INFINITY;
    const bool stays = real && maybe < rule.top_groups;
    if (__ballot(real && !stays && more < rule.top_groups)) return false;
    const uint64_t keep = __ballot(stays);                  // bit of a group: its first lane's
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int of = min(v * kWave + lane, C.n_experts - 1) / size;
        if (!((keep >> (of << log)) & 1)) r.c[v] = -INFINITY;
    }
    return true;
}

template <int VPT, int TYPE>
struct ScoredRouter {
    static constexpr int kWaves = scored_waves(VPT);
    template <class F>
    __device__ static inline void tokens(const RouteCall& C, int t0, int t1, int step, int lane,
                                         F&& f) {
        __shared__ float space[kWaves][VPT * kWave + VPT * 8];
        if (t0 >= t1) return;
        const pm_route_rule& rule = C.rule;
        const bool softmax = rule.score == PM_SCORE_SOFTMAX;
        float bias[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = v * kWave + lane;
            bias[v] = e < C.n_experts ? (C.bias ? C.bias[e] : 0.0f) : -INFINITY;
        }
        // up to 4 tokens share the exact scores where 16 lanes hold a token's
        // slots and a few ranks behind them
        const int held = C.top_k <= 12 ? 16 : kWave, group = kWave / held;
        const int slot = lane & (held - 1);
        Logits<VPT> next = load_logits<VPT, TYPE>(C, t0, lane);
        for (int t = t0; t < t1; t += group * step) {
            int id = -1, tok = -1;
            float top = 0.0f;                               // softmax: the largest logit,
            double sum = 1.0;                               // and the sum
            uint64_t redo = 0;                              // tokens that fp32 leaves open
            for (int s = 0; s < group && t + s * step < t1; ++s) {
                const Logits<VPT> now = next;
                // the next token's logits are on their way meanwhile
                next = load_logits<VPT, TYPE>(C, min(t + (s + 1) * step, t1 - 1), lane);
                Ranks<VPT> r;
                float big = -INFINITY;
                double all = 0.0;
                if (softmax) {
#pragma unroll
                    for (int v = 0; v < VPT; ++v)
                        if (v * kWave + lane < C.n_experts) big = fmaxf(big, now.v[v]);
                    big = wave_best(big);
                    double x[VPT];
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        const bool seen = v * kWave + lane < C.n_experts && now.v[v] > -INFINITY;
                        x[v] = !seen ? 0.0
                                     : now.v[v] == big ? 1.0 : exp(double(now.v[v]) - double(big));
                        all += x[v];
                    }
                    for (int d = 1; d < kWave; d <<= 1) all += __shfl_xor(all, d);
                    const float part = __builtin_amdgcn_rcpf(float(all));
#pragma unroll
                    for (int v = 0; v < VPT; ++v) r.c[v] = float(x[v]) * part;
                } else {
#pragma unroll
                    for (int v = 0; v < VPT; ++v)
                        r.c[v] = __builtin_amdgcn_rcpf(
                            1.0f + __builtin_amdgcn_exp2f(now.v[v] * -1.44269504f));
                }
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    // (a NaN among logit and bias leaves no rank, either)
                    r.c[v] = now.v[v] > -INFINITY ? r.c[v] + bias[v] : -INFINITY;
                }
                bool unsure = false;
                if (rule.n_groups > 1)
                    unsure = !rank_groups<VPT>(C, r, lane, space[threadIdx.x >> 6]);
                uint32_t k = 0;
                int i = -1;
                if (!unsure) rank_list<VPT>(C, r, lane, held, &k, &i, &unsure);
                if (unsure) redo |= uint64_t(1) << s;
                const int is = __shfl(i, slot);
                if (lane / held != s) continue;
                id = is;
                tok = t + s * step;
                top = big;
                sum = all;
            }
            // exact scores, and whether the exact ranks are in this order
            double x = 0.0, c = -INFINITY;
            if (id >= 0) {
                const float l = load_f32<TYPE>(C.logits, int64_t(tok) * C.ld + id);
                if (softmax)
                    x = (l == top ? 1.0 : exp(double(l) - double(top))) / sum;
                else
                    x = 1.0 / (1.0 + exp(-double(l)));
                c = x + (C.bias ? double(C.bias[id]) : 0.0);
            }
            const double after = __shfl_down(c, 1);
            const int id_after = __shfl_down(id, 1);
            const bool order = slot == held - 1 || id_after < 0 || c > after ||
                               (c == after && id < id_after);
            const uint64_t wrong = __ballot(!order);
            for (int s = 0; s < group; ++s)
                if ((wrong >> (s * held)) & (held == kWave ? ~0ull : 0xFFFFull))
                    redo |= uint64_t(1) << s;
            if (slot >= C.top_k) {
                id = -1;
                x = 0.0;
            }
            if (rule.flags & PM_ROUTE_RENORM) {
                double all = row16_sum_f64(x);
                if (held == kWave) {
                    all += __shfl_xor(all, 16);
                    all += __shfl_xor(all, 32);
                }
                x = all > 0.0 ? x / all : 0.0;
            }
            if (tok >= 0 && slot < C.top_k && !((redo >> (lane / held)) & 1)) {
                const int64_t u = int64_t(tok) * C.top_k + slot;
                C.ids[u] = id;
                C.w[u] = id >= 0 ? float(x * double(rule.scale)) : 0.0f;
                if (id >= 0) f(u, id);
            }
            while (redo) {
                const int s = __builtin_ctzll(redo);
                redo &= redo - 1;
                if (t + s * step >= t1) continue;
                int i;
                float w;
                scored_token<VPT, TYPE>(C, t + s * step, lane, &i, &w);
                if (lane < C.top_k) {
                    const int64_t u = int64_t(t + s * step) * C.top_k + lane;
                    C.ids[u] = i;
                    C.w[u] = i >= 0 ? w : 0.0f;
                    if (i >= 0) f(u, i);
                }
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

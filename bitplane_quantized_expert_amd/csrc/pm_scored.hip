// Router by scores: sigmoid or softmax of every logit, a bias that only
// selects, the best groups of experts, top-k among them (include/pm.h).
//
// The rule's scores and ranks are fp64, and which expert is selected may hang on
// their last bits; but an exponential and a division in fp64 for each of a token's
// experts would take several times as long as all the rest.  So a wave ranks its
// token's experts in fp32 first, with a bound on what these ranks are off by:
// groups that stay or fall by more than it, and the few experts that the exact
// ranks may place among the top_k.  These get their exact scores, one lane each
// (16 lanes a token where they suffice), which the weights need in any case, and
// the number of exact ranks above a lane's own is its place.  Where fp32 leaves
// a choice open, the wave ranks the token again, in fp64.
//
// Bound by the chain of dependent steps of a token (the bound by ballots, the
// groups, the candidates), which four waves on a SIMD half hide (59 % of the waves'
// time is waiting): 16384 tokens of 512 experts, sigmoid, 10 of the best 4 of 8
// groups, take 28 us (33.5 MB of logits, 5.4 at the memory's rate).  A token that is
// ranked again takes 6, which the kernel waits for; bounds as close as they are leave
// that to less than one token of these calls on average.  With sorting, a second launch
// (pm_route_sort.h): 38 us, with all ranks in fp64 117, and 102 where each token's
// experts all count the same and each is ranked again.  Experts lie VPT adjacent
// ones to a lane: a row is read by one wide load, and groups of whole lanes need no
// LDS (2 us more where experts were dealt out in turn).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "pm_rank.h"
#include "pm_route_sort.h"

namespace pm {

namespace {

// Waves of a workgroup that selects: each has a token's ranks in LDS, 74 KB
// together, and up to 64 logits per lane in registers.
constexpr int scored_waves(int vpt) { return vpt > 32 ? 2 : vpt > 16 ? 4 : vpt > 8 ? 8 : kRouteWaves; }

// ---------------------------------------------------------------- across the wave
// v and its value in lane i ^ D, in either order, for D = 1, 2, and for D = 4, 8,
// 16, 32 where lanes that differ in lower bits only hold the same.
struct Pair {
    uint32_t a, b;
};
template <int D>
__device__ inline Pair both(uint32_t v) {
    if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return {uint32_t(r[0]), uint32_t(r[1])};
    } else if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return {uint32_t(r[0]), uint32_t(r[1])};
    } else {
        // quad_perm [1,0,3,2], [2,3,0,1], row_half_mirror, row_mirror
        constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
        return {v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), ctrl, 0xF, 0xF, false))};
    }
}
template <int D>
__device__ inline void both(uint32_t v, uint32_t* a, uint32_t* b) {
    const Pair p = both<D>(v);
    *a = p.a;
    *b = p.b;
}
template <int D>
__device__ inline void both(uint64_t v, uint64_t* a, uint64_t* b) {
    const Pair lo = both<D>(uint32_t(v)), hi = both<D>(uint32_t(v >> 32));
    *a = uint64_t(hi.a) << 32 | lo.a;
    *b = uint64_t(hi.b) << 32 | lo.b;
}
// f(1), f(2), .. f(2^(log - 1)) with constant arguments.
template <class F>
__device__ inline void doublings(int log, F&& f) {
    if (log > 0) f(std::integral_constant<int, 1>{});
    if (log > 1) f(std::integral_constant<int, 2>{});
    if (log > 2) f(std::integral_constant<int, 4>{});
    if (log > 3) f(std::integral_constant<int, 8>{});
    if (log > 4) f(std::integral_constant<int, 16>{});
    if (log > 5) f(std::integral_constant<int, 32>{});
}

__device__ inline double wave_sum_f64(double v) {
    v = row16_sum_f64(v);
    uint64_t a, b;
    both<16>(__builtin_bit_cast(uint64_t, v), &a, &b);
    v = __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
    both<32>(__builtin_bit_cast(uint64_t, v), &a, &b);
    return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
}

// ---------------------------------------------------------------- ranks
// A rank as an integer that orders like it, 0 for -inf and NaN (never selected)
// and where it does not count.  (The sum as a value: the compiler may not branch
// round it)
__device__ inline uint32_t rank_key(float c, bool counts = true) {
    const uint32_t b = __float_as_uint(c);                  // (a sum with a score is not -0)
    uint32_t k = b ^ (uint32_t(int(b) >> 31) | 0x80000000u);
    asm("" : "+v"(k));
    return counts && c > -INFINITY ? k : 0u;
}
__device__ inline uint64_t rank_key(double c, bool counts = true) {
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    const uint64_t k = b ^ (uint64_t(int64_t(b) >> 63) | 1ull << 63);
    return counts && c > -INFINITY ? k : 0ull;
}
__device__ inline float rank_value(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ inline double rank_value(uint64_t k) {
    return __builtin_bit_cast(double, k ^ (k >> 63 ? 1ull << 63 : ~0ull));
}

// The lanes below this one among those of a ballot.
__device__ inline int lanes_below(uint64_t lanes) {
    return __builtin_amdgcn_mbcnt_hi(uint32_t(lanes >> 32),
                                     __builtin_amdgcn_mbcnt_lo(uint32_t(lanes), 0));
}

__device__ inline float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ inline double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(
        double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(b >> 32), lane))) << 32 |
                    uint32_t(__builtin_amdgcn_readlane(int(b), lane)));
}

// How far apart in fp32 two ranks (or two groups' sums of two) may be and still
// be the other way round, where the larger of them, or the two of a group, are
// `size`.  A sigmoid is off by less than kSigmoidError (pm_rank.h); a softmax's
// e / sum by 5 roundings of 2^-24 of it (v_rcp_f32: two).  Either side has this error
// twice at most (two ranks, or both of the ranks that are compared).  Sums with a
// bias, a group's sum, and the difference from the bound are each rounded to 2^-24 of
// `size`.
__device__ inline float rank_slack(bool softmax, float size) {
    return (softmax ? 0x1.5p-21f : 2 * kSigmoidError) + size * 0x1.9p-23f;
}
// The same without a bias, of ranks from v down: small scores are told apart as
// well, as they are off by kSigmoidRelative of themselves at most, either side twice
// (2^-14 leaves room), or where they are below kSigmoidSmall by less than that.
__device__ inline float score_slack(bool softmax, float v) {
    return fminf(rank_slack(softmax, v), v * 0x1p-14f + 2 * kSigmoidSmall);
}

template <int VPT>
struct Ranks {                                      // in fp32
    uint32_t key[VPT];
};

// A bound that the top_k largest keys meet: at least top_k of the lanes' own
// largest (m) do, just top_k if any value tells so many apart.
__device__ inline uint32_t rank_bound(uint32_t m, int top_k) {
    uint32_t hi = m, lo = m;
    doublings(6, [&](auto d) {
        const Pair h = both<d>(hi), l = both<d>(lo);
        hi = max(h.a, h.b);
        lo = min(l.a, l.b);
    });
    hi = uni(int(hi));
    lo = uni(int(lo));
    // lo is met by top_k lanes at least, hi + 1 by none
    while (lo < hi) {
        const uint32_t c = lo + ((hi - lo) >> 1) + 1;
        const int n = __popcll(__ballot(m >= c));
        if (n >= top_k) lo = c;
        if (n == top_k) break;
        if (n < top_k) hi = c - 1;
    }
    return lo;
}

// A higher bound, of those that all keys are counted for: top_k keys meet it, and
// few more if any value tells so many apart.
template <int VPT>
__device__ inline uint32_t rank_bound_all(const Ranks<VPT>& r, uint32_t lo, uint32_t hi, int top_k,
                                          int spare) {
    doublings(6, [&](auto d) {
        const Pair p = both<d>(hi);
        hi = max(p.a, p.b);
    });
    hi = uni(int(hi));
    while (lo < hi) {
        const uint32_t c = lo + ((hi - lo) >> 1) + 1;
        int n = 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v) n += __popcll(__ballot(r.key[v] >= c));
        if (n >= top_k) lo = c;
        if (n < top_k)
            hi = c - 1;
        else if (n - top_k <= spare)
            break;
    }
    return lo;
}

// ---------------------------------------------------------------- groups
// How the experts fall into groups.  2^log lanes look at a group; a lane's own
// experts are all of their group where the groups are as many as a power of two
// and the lanes hold as many experts each.
struct Groups {
    int log, size;
    uint32_t part;                                  // ceil(2^32 / size), size > 1
    bool whole;

    __device__ inline int of(int e) const { return size == 1 ? e : __umulhi(uint32_t(e), part); }
};
template <int VPT>
__device__ inline Groups find_groups(const RouteCall& C) {
    Groups g;
    const uint32_t n = C.rule.n_groups;
    g.log = n > 1 ? 6 - (32 - __builtin_clz(n - 1)) : 0;
    g.size = C.n_experts / int(n);
    g.part = 0xFFFFFFFFu / uint32_t(g.size) + 1;
    g.whole = C.n_experts == VPT * kWave && (n & (n - 1)) == 0;
    return g;
}

// The two largest keys of a group.
template <class K>
struct TwoLargest {
    K a = 0, b = 0;

    __device__ inline void take(K c) {
        b = max(b, min(a, c));
        a = max(a, c);
    }
    __device__ inline void join(int log) {          // those of 2^log lanes
        doublings(log, [&](auto d) {
            K a0, a1, b0, b1;
            both<d>(a, &a0, &a1);
            both<d>(b, &b0, &b1);
            a = max(a0, a1);
            b = max(min(a0, a1), max(b0, b1));
        });
    }
};

// Places apart in LDS of experts that the lanes of several groups read at once.
__device__ inline int padded_at(int e) { return e + (e >> 3); }
constexpr int padded_size(int vpt) { return vpt * (kWave + kWave / 8); }

// Takes the experts of the groups that do not stay out of the ranks; false where
// ranks in fp32 do not tell which do.  `space`: the wave's LDS, padded_size(VPT)
// keys.
template <int VPT, bool SOFTMAX>
__device__ inline bool rank_groups(const RouteCall& C, const Groups& groups, Ranks<VPT>& r,
                                   int lane, uint32_t* space) {
    const pm_route_rule& rule = C.rule;
    const int n = rule.n_groups, size = groups.size, log = groups.log;
    const int g = lane >> log, j = lane & ((1 << log) - 1);
    TwoLargest<uint32_t> two;
    if (groups.whole) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) two.take(r.key[v]);
    } else {
        int first = lane * VPT;
        asm volatile("" : "+v"(first));                     // (addresses are not kept)
#pragma unroll
        for (int v = 0; v < VPT; ++v) space[padded_at(first + v)] = r.key[v];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        int base = min(g, n - 1) * size;
        asm volatile("" : "+v"(base));
        for (int i0 = j; i0 - j < size; i0 += 8 << log) {
            uint32_t k[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                k[i] = space[padded_at(base + min(i0 + (i << log), size - 1))];
#pragma unroll
            for (int i = 0; i < 8; ++i) two.take(i0 + (i << log) < size ? k[i] : 0u);
        }
        asm volatile("" ::: "memory");                      // (read before the next token's)
    }
    two.join(log);
    const bool real = g < n && two.a != 0;
    float mine = real ? rank_value(two.a) : -INFINITY, second = 0.0f;
    if (rule.group_best == 2 && two.b != 0) second = rank_value(two.b);
    // groups that count more for certain, and those that may: by the ends of what
    // each may count
    const float off = rank_slack(SOFTMAX, fabsf(mine) + fabsf(second));
    mine += second;
    const float low = real ? mine - off : mine, high = real ? mine + off : mine;
    int more = 0, maybe = -1;
    for (int k = 0; k < n; ++k) {
        const float o = lane_value(low, k << log), p = lane_value(high, k << log);
        more += o > high;
        maybe += !(p < low);
    }
    const bool stays = real && maybe < rule.top_groups;
    if (__ballot(real && !stays && more < rule.top_groups)) return false;
    const uint64_t keep = __ballot(stays);                  // bit of a group: its first lane's
    if (groups.whole) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) r.key[v] = stays ? r.key[v] : 0u;
    } else {
        int first = lane * VPT;
        asm volatile("" : "+v"(first));
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int of = groups.of(min(first + v, C.n_experts - 1));
            r.key[v] = (keep >> (of << log)) & 1 ? r.key[v] : 0u;
        }
    }
    return true;
}

// ---------------------------------------------------------------- scores
// A softmax's largest logit, and its sum.
struct Softmax {
    float top;
    double sum;
};
__device__ inline double softmax_part(float l, float top) {
    return l == top ? 1.0 : exp(double(l) - double(top));
}
__device__ inline double exact_score(bool softmax, const Softmax& s, float l) {
    return softmax ? softmax_part(l, s.top) / s.sum : 1.0 / (1.0 + exp(-double(l)));
}

// The logits of a token: a lane has VPT adjacent ones.  As they are loaded: one a
// word, or (16-bit ones of VPT * 64 experts) two.  0 past the last.
template <int VPT>
struct RawLogits {
    uint32_t d[VPT];
};
template <int VPT>
__device__ inline bool in_pairs(const RouteCall& C) {
    return VPT > 1 && C.type != PM_F32 && C.n_experts == VPT * kWave;
}
template <int VPT>
__device__ inline RawLogits<VPT> load_raw(const RouteCall& C, int t, int lane) {
    RawLogits<VPT> l;
    const int log = C.type == PM_F32 ? 2 : 1;
    char* const row =
        const_cast<char*>(static_cast<const char*>(C.logits)) + (int64_t(t) * C.ld << log);
    if (C.n_experts == VPT * kWave && C.type == PM_F32) {
        __builtin_memcpy(l.d, __builtin_assume_aligned(row + lane * VPT * 4, 4), VPT * 4);
    } else if (in_pairs<VPT>(C)) {
        // (rows need no alignment beyond their element's)
        __builtin_memcpy(l.d, row + lane * VPT * 2, VPT * 2);
    } else {
        const auto buf = __builtin_amdgcn_make_buffer_rsrc(uni_ptr(row), 0, C.n_experts << log,
                                                           0x00020000);
        if (C.type == PM_F32) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                l.d[v] = __builtin_amdgcn_raw_buffer_load_b32(buf, (lane * VPT + v) * 4, 0, 0);
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                l.d[v] = uint16_t(
                    __builtin_amdgcn_raw_buffer_load_b16(buf, (lane * VPT + v) * 2, 0, 0));
        }
    }
    return l;
}
template <int VPT>
struct Widened {
    float v[VPT];
};
template <int VPT>
__device__ inline Widened<VPT> widen(const RouteCall& C, const RawLogits<VPT>& r) {
    Widened<VPT> l;
    if (C.type == PM_F32) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) l.v[v] = __uint_as_float(r.d[v]);
        return l;
    }
    uint32_t h[VPT];
    if (in_pairs<VPT>(C)) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) h[v] = v & 1 ? r.d[v >> 1] >> 16 : r.d[v >> 1] & 0xFFFFu;
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) h[v] = r.d[v];
    }
    if (C.type == PM_BF16) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) l.v[v] = __uint_as_float(h[v] << 16);
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) l.v[v] = __half2float(__ushort_as_half(uint16_t(h[v])));
    }
    return l;
}
__device__ inline float logit(const RouteCall& C, int t, int e) {
    const int64_t at = int64_t(t) * C.ld + e;
    if (C.type == PM_F32) return load_f32<PM_F32>(C.logits, at);
    return C.type == PM_F16 ? load_f32<PM_F16>(C.logits, at) : load_f32<PM_BF16>(C.logits, at);
}

// An expert that the exact ranks may select, with what its rank takes.
struct Candidate {
    int32_t id;
    float logit, bias;
};

// The number of lanes with a larger (key, ~id) among those that share a token: 16
// lanes, or all 64 of which `found` hold one.
__device__ inline int place_of16(uint64_t key, uint32_t low) {
    int n = 0;
    auto turn = [&](auto by) {
        constexpr int ctrl = 0x120 + decltype(by)::value;  // row_ror
        const uint32_t h = __builtin_amdgcn_update_dpp(0, int(key >> 32), ctrl, 0xF, 0xF, false);
        const uint32_t l = __builtin_amdgcn_update_dpp(0, int(key), ctrl, 0xF, 0xF, false);
        const uint32_t o = __builtin_amdgcn_update_dpp(0, int(low), ctrl, 0xF, 0xF, false);
        const uint64_t k = uint64_t(h) << 32 | l;
        n += k > key || (k == key && o > low);
    };
    turn(std::integral_constant<int, 1>{});
    turn(std::integral_constant<int, 2>{});
    turn(std::integral_constant<int, 3>{});
    turn(std::integral_constant<int, 4>{});
    turn(std::integral_constant<int, 5>{});
    turn(std::integral_constant<int, 6>{});
    turn(std::integral_constant<int, 7>{});
    turn(std::integral_constant<int, 8>{});
    turn(std::integral_constant<int, 9>{});
    turn(std::integral_constant<int, 10>{});
    turn(std::integral_constant<int, 11>{});
    turn(std::integral_constant<int, 12>{});
    turn(std::integral_constant<int, 13>{});
    turn(std::integral_constant<int, 14>{});
    turn(std::integral_constant<int, 15>{});
    return n;
}
__device__ inline int place_of64(uint64_t key, uint32_t low, int found) {
    int n = 0;
    for (int i = 0; i < found; ++i) {
        const uint64_t k = uint64_t(uint32_t(__builtin_amdgcn_readlane(int(key >> 32), i))) << 32 |
                           uint32_t(__builtin_amdgcn_readlane(int(key), i));
        const uint32_t o = __builtin_amdgcn_readlane(low, i);
        n += k > key || (k == key && o > low);
    }
    return n;
}

template <int VPT, bool SOFTMAX>
struct ScoredRouter {
    static constexpr int kWaves = scored_waves(VPT);
    struct Space {
        uint64_t key[padded_size(VPT)];
        Candidate listed[kWave];
    };

    template <class F>
    __device__ static inline void tokens(const RouteCall& C, int t0, int t1, int step, int lane,
                                         F&& f) {
        __shared__ Space spaces[kWaves];
        Space* const space = &spaces[threadIdx.x >> 6];
        // 64 tokens in fp32, then those among them that it leaves open (apart, as
        // the registers of the two are not the same)
        for (; t0 < t1; t0 += kWave * step) {
            uint64_t redo = rank_tokens(C, t0, min(t1 - t0, kWave * step) + t0, step, lane, space, f);
            for (; redo; redo &= redo - 1) {
                const int t = t0 + __builtin_ctzll(redo) * step;
                int own = lane;
                asm volatile("" : "+v"(own));               // (nothing of it is kept)
                rank_again(C, t, own, space, f);
            }
        }
    }

private:
    // Up to 64 tokens; returns those that are left, a bit each.
    template <class F>
    __device__ static inline uint64_t rank_tokens(const RouteCall& C, int t0, int t1, int step,
                                                  int lane, Space* space, F&& f) {
        uint64_t left = 0;
        const pm_route_rule& rule = C.rule;
        const bool biased = C.bias != nullptr;
        const Groups groups = find_groups<VPT>(C);
        // -inf: never selected.  (Neither is an expert of a NaN: no rank is one)
        float bias[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = lane * VPT + v;
            bias[v] = e < C.n_experts ? (biased ? C.bias[e] : 0.0f) : -INFINITY;
        }
        // up to 4 tokens share the exact scores where 16 lanes hold a token's
        // candidates
        const int held = C.top_k <= 12 ? 16 : kWave, group = kWave / held;
        const int slot = lane & (held - 1);
        RawLogits<VPT> next = load_raw<VPT>(C, t0, lane);
        for (int t = t0; t < t1; t += group * step) {
            int tok = -1, found = 0;
            Softmax soft{0.0f, 1.0};
            uint32_t redo = 0;                              // of these
            for (int s = 0; s < group && t + s * step < t1; ++s) {
                const Widened<VPT> now = widen(C, next);
                // the next token's logits are on their way meanwhile
                next = load_raw<VPT>(C, min(t + (s + 1) * step, t1 - 1), lane);
                Softmax all{-INFINITY, 0.0};
                Ranks<VPT> r;
                if constexpr (SOFTMAX) {
                    double x[VPT];
                    all = softmax_of(C, now, lane, x);
                    const float part = __builtin_amdgcn_rcpf(float(all.sum));
#pragma unroll
                    for (int v = 0; v < VPT; ++v)
                        r.key[v] = rank_key(float(x[v]) * part + bias[v], now.v[v] > -INFINITY);
                } else {
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        const float x = sigmoid_rank(now.v[v]);
                        r.key[v] = rank_key(x + bias[v], now.v[v] > -INFINITY);
                    }
                }
                bool sure = true;
                if (rule.n_groups > 1)
                    sure = rank_groups<VPT, SOFTMAX>(C, groups, r, lane,
                                            reinterpret_cast<uint32_t*>(space->key));
                // all that may be among the top_k, into this token's lanes
                uint32_t most = r.key[0];
#pragma unroll
                for (int v = 1; v < VPT; ++v) most = max(most, r.key[v]);
                uint32_t least = rank_bound(most, C.top_k);
                int n;
#pragma unroll 1
                for (bool again = false;; again = true) {
                    uint32_t bound = 1;
                    if (least) {
                        const float v = rank_value(least);
                        bound = max(rank_key(v - (biased ? rank_slack(SOFTMAX, fabsf(v))
                                                         : score_slack(SOFTMAX, v))),
                                    1u);
                    }
                    n = 0;
#pragma unroll
                    for (int v = 0; v < VPT; ++v) {
                        const bool hit = r.key[v] >= bound;
                        const uint64_t hits = __ballot(hit);
                        if (hits == 0) continue;
                        const int at = n + lanes_below(hits);
                        if (hit && at < held)
                            space->listed[s * held + at] = {lane * VPT + v, now.v[v], bias[v]};
                        n += __popcll(hits);
                    }
                    // (lanes that hold several of the largest let too many pass)
                    if (n <= held || again || !sure) break;
                    least = rank_bound_all(r, least, most, C.top_k, (held - C.top_k) / 2);
                }
                if (!sure || n > held) redo |= 1u << s;
                if (lane / held == s) {
                    tok = t + s * step;
                    found = n;
                    soft = all;
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            // exact scores and ranks, and the place of each
            int id = -1;
            double x = 0.0;
            uint64_t key = 0;
            if (slot < found) {
                const Candidate c = space->listed[lane];
                id = c.id;
                x = exact_score(SOFTMAX, soft, c.logit);
                key = rank_key(x + double(c.bias));
            }
            asm volatile("" ::: "memory");                  // (read before the next tokens')
            const int place = held == kWave ? place_of64(key, ~uint32_t(id), uni(found))
                                            : place_of16(key, ~uint32_t(id));
            const bool chosen = id >= 0 && place < C.top_k;
            if (!chosen) x = 0.0;
            if (rule.flags & PM_ROUTE_RENORM) {
                const double all = held == kWave ? wave_sum_f64(x) : row16_sum_f64(x);
                x = all > 0.0 ? x / all : 0.0;
            }
            if (tok >= 0 && !((redo >> (lane / held)) & 1)) {
                const int64_t u = int64_t(tok) * C.top_k;
                if (chosen) {
                    C.ids[u + place] = id;
                    C.w[u + place] = float(x * double(rule.scale));
                    f(u + place, id);
                }
                // slots left over
                if (slot >= found && slot < C.top_k) {
                    C.ids[u + slot] = -1;
                    C.w[u + slot] = 0.0f;
                }
            }
            left |= uint64_t(redo) << ((t - t0) / step);
        }
        return left;
    }

    // The largest logit, by the largest of the lanes' keys.
    __device__ static inline float top_of(uint32_t big) {
        doublings(6, [&](auto d) {
            const Pair p = both<d>(big);
            big = max(p.a, p.b);
        });
        return big ? rank_value(big) : -INFINITY;
    }

    __device__ static inline Softmax softmax_of(const RouteCall& C, const Widened<VPT>& l, int lane,
                                                double* x) {
        Softmax all{-INFINITY, 0.0};
        uint32_t big = 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (lane * VPT + v < C.n_experts) big = max(big, rank_key(l.v[v]));
        all.top = top_of(big);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const bool seen = lane * VPT + v < C.n_experts && l.v[v] > -INFINITY;
            x[v] = seen ? softmax_part(l.v[v], all.top) : 0.0;
            all.sum += x[v];
            if (VPT > 4) __builtin_amdgcn_sched_barrier(0);           // (registers)
        }
        all.sum = wave_sum_f64(all.sum);
        return all;
    }

    // A token by its exact ranks.  One wave in some hundred comes here, and the
    // rest may wait for it: its time is that of fetching the code, which loops over
    // ranks in LDS keep short.  Expert v * 64 + lane is a lane's v-th.
    template <class F>
    __device__ static inline void rank_again(const RouteCall& C, int t, int lane, Space* space,
                                             F&& f) {
        constexpr int kAt = VPT < 8 ? VPT : 8;      // loads on their way together
        const pm_route_rule& rule = C.rule;
        uint64_t* const keys = space->key;
        auto at = [&](int v) { return padded_at(v * kWave + lane); };
        // logits and biases, as they are; NaN where there is no expert
        uint32_t big = 0;
#pragma unroll 1
        for (int v0 = 0; v0 < VPT; v0 += kAt) {
            float l[kAt], b[kAt];
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
                const int e = min((v0 + i) * kWave + lane, C.n_experts - 1);
                l[i] = logit(C, t, e);
                b[i] = C.bias ? C.bias[e] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
                if ((v0 + i) * kWave + lane >= C.n_experts) l[i] = NAN;
                big = max(big, rank_key(l[i]));
                keys[at(v0 + i)] = uint64_t(__float_as_uint(b[i])) << 32 | __float_as_uint(l[i]);
            }
        }
        Softmax soft{-INFINITY, 0.0};
        if constexpr (SOFTMAX) {
            soft.top = top_of(big);
#pragma unroll 1
            for (int v = 0; v < VPT; ++v) {
                const float l = __uint_as_float(uint32_t(keys[at(v)]));
                if (l > -INFINITY) soft.sum += softmax_part(l, soft.top);
            }
            soft.sum = wave_sum_f64(soft.sum);
        }
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) {
            const uint64_t k = keys[at(v)];
            const float l = __uint_as_float(uint32_t(k)), b = __uint_as_float(uint32_t(k >> 32));
            keys[at(v)] = rank_key(exact_score(SOFTMAX, soft, l) + double(b),
                                   l > -INFINITY && b > -INFINITY);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (rule.n_groups > 1) {
            const Groups groups = find_groups<VPT>(C);
            const int n = rule.n_groups, log = groups.log, g = lane >> log;
            TwoLargest<uint64_t> two;
#pragma unroll 1
            for (int i = lane & ((1 << log) - 1); i < groups.size; i += 1 << log)
                two.take(keys[padded_at(min(g, n - 1) * groups.size + i)]);
            two.join(log);
            const bool real = g < n && two.a != 0;
            double mine = real ? rank_value(two.a) : -double(INFINITY);
            if (rule.group_best == 2 && two.b != 0) mine += rank_value(two.b);
            int more = 0;
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
                const double o = lane_value(mine, k << log);
                more += o > mine || (o == mine && k < g);
            }
            const uint64_t keep = __ballot(real && more < rule.top_groups);
#pragma unroll 1
            for (int v = 0; v < VPT; ++v) {
                const int of = groups.of(min(v * kWave + lane, C.n_experts - 1));
                if (!((keep >> (of << log)) & 1)) keys[at(v)] = 0;
            }
        }
        uint32_t most = 0;
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) most = max(most, uint32_t(keys[at(v)] >> 32));
        // those above `least`, and `equal` of those that equal it
        uint64_t least = uint64_t(max(rank_bound(most, C.top_k), 1u)) << 32;
        int n = list_above(least, kWave, lane, space);
        if (n > kWave) {
            // more than the list holds: the top_k-th largest itself
            uint64_t lo = ~0ull, hi = 0;
#pragma unroll 1
            for (int v = 0; v < VPT; ++v) {
                const uint64_t k = keys[at(v)];
                hi = max(hi, k);
                if (k >= least) lo = min(lo, k);
            }
            doublings(6, [&](auto d) {
                uint64_t a, b;
                both<d>(hi, &a, &b);
                hi = max(a, b);
                both<d>(lo, &a, &b);
                lo = min(a, b);
            });
            lo = uni64(lo);
            hi = uni64(hi);
            while (lo < hi) {
                const uint64_t c = lo + ((hi - lo) >> 1) + 1;
                if (met_by(c, lane, space) >= C.top_k)
                    lo = c;
                else
                    hi = c - 1;
            }
            n = list_above(lo, C.top_k - (lo == ~0ull ? 0 : met_by(lo + 1, lane, space)), lane,
                           space);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        int id = -1;
        uint64_t key = 0;
        double x = 0.0;
        if (lane < n) {
            id = space->listed[lane].id;
            key = keys[padded_at(id)];
        }
        asm volatile("" ::: "memory");              // (read before the next token's)
        const int place = place_of64(key, ~uint32_t(id), n);
        if (place >= C.top_k) id = -1;
        if (id >= 0) x = exact_score(SOFTMAX, soft, logit(C, t, id));
        if (rule.flags & PM_ROUTE_RENORM) {
            const double all = wave_sum_f64(x);
            x = all > 0.0 ? x / all : 0.0;
        }
        const int64_t u = int64_t(t) * C.top_k;
        if (id >= 0) {
            C.ids[u + place] = id;
            C.w[u + place] = float(x * double(rule.scale));
            f(u + place, id);
        }
        if (lane >= n && lane < C.top_k) {          // (left over)
            C.ids[u + lane] = -1;
            C.w[u + lane] = 0.0f;
        }
    }

    // Lists the experts above `least`, and of those that equal it the first `equal`;
    // returns how many, listed if they are no more than a wave's lanes.
    __device__ static inline int list_above(uint64_t least, int equal, int lane, Space* space) {
        int n = 0, same = 0;
#pragma unroll 1
        for (int v = 0; v < VPT; ++v) {
            const uint64_t k = space->key[padded_at(v * kWave + lane)];
            const uint64_t equals = __ballot(k == least);
            const bool hit = k > least || (k == least && same + lanes_below(equals) < equal);
            const uint64_t hits = __ballot(hit);
            const int at = n + lanes_below(hits);
            if (hit && at < kWave) space->listed[at].id = v * kWave + lane;
            n += __popcll(hits);
            same += __popcll(equals);
        }
        return n;
    }
    __device__ static inline int met_by(uint64_t least, int lane, Space* space) {
        int n = 0;
#pragma unroll 1
        for (int v = 0; v < VPT; ++v)
            n += __popcll(__ballot(space->key[padded_at(v * kWave + lane)] >= least));
        return n;
    }
};

template <int VPT>
hipError_t launch_scored(const RouteCall& C, hipStream_t st) {
    return C.rule.score == PM_SCORE_SOFTMAX ? launch_routed<ScoredRouter<VPT, true>>(C, st)
                                            : launch_routed<ScoredRouter<VPT, false>>(C, st);
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

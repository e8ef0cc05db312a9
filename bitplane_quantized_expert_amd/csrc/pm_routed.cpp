// Entry points of the routed experts on the device (include/pm.h): argument
// checks and launches.  Nothing here allocates (so nothing throws), copies or
// waits, so every call can be captured into a HIP graph.
#include <algorithm>
#include <atomic>

#include "pm_error.h"
#include "pm_routed.h"

using namespace pm;

static pm_status launched(hipError_t e, const char* what) {
    if (e == hipSuccess) return PM_OK;
    return failf(PM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

static bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

static bool type_ok(int t) { return t == PM_F32 || t == PM_F16 || t == PM_BF16; }

// Whether two byte ranges share a byte.
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return na && nb && pa < pb + nb && pb < pa + na;
}

// Bytes from the first element of n rows to the end of the last.
static size_t span(size_t n, int64_t ld, size_t cols, int type) {
    return n == 0 || cols == 0 ? 0 : (size_t(ld) * (n - 1) + cols) * type_bytes(type);
}

// Rows of any buffer and their distance stay below this, so that byte
// addresses of a valid call never wrap.
static constexpr int64_t kMaxLd = int64_t(1) << 31;

// Uses of a call: rounding their number up to a tile, or going on by a few
// waves' tokens, stays within 32 bits.
static bool uses_ok(int64_t n) { return n <= PM_ROUTED_MAX_USES; }

// ---------------------------------------------------------------- device properties
static constexpr int kMaxDevices = 64;

int pm::compute_units() {
    static std::atomic<int> known[kMaxDevices];
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
    n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
        n = 256;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

hipError_t pm::allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & (kMaxDevices - 1));
    if (dev < kMaxDevices && (done->load(std::memory_order_relaxed) & bit)) return hipSuccess;
    // (several threads may set the same value)
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && dev < kMaxDevices) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---------------------------------------------------------------- router
void pm::route_blocks(int n_tokens, int* block_tokens, int* n_blocks) {
    // up to 256 blocks of a multiple of 16 tokens
    const int64_t per = ((int64_t(n_tokens) + 255) / 256 + 15) / 16 * 16;
    // a block holds at most 65520 uses of one expert (16-bit counts)
    *block_tokens = int(std::min<int64_t>(std::max<int64_t>(per, 16), 65520));
    *n_blocks = int((int64_t(n_tokens) + *block_tokens - 1) / *block_tokens);
}

static bool route_sizes_ok(int n_tokens, int n_experts, int top_k) {
    return n_tokens >= 0 && n_experts >= 1 && n_experts <= PM_ROUTE_MAX_EXPERTS && top_k >= 1 &&
           top_k <= PM_ROUTE_MAX_TOPK && top_k <= n_experts &&
           uses_ok(int64_t(n_tokens) * top_k);
}

extern "C" size_t pm_route_workspace_bytes(int n_tokens, int n_experts, int top_k) {
    if (!route_sizes_ok(n_tokens, n_experts, top_k)) return 0;
    int bt, nb;
    route_blocks(n_tokens, &bt, &nb);
    return (size_t(nb) * ((n_experts + 7) & ~7) * sizeof(uint16_t) + 15) & ~size_t(15);
}

extern "C" pm_status pm_route_topk_device(int n_tokens, int n_experts, int top_k,
                                          const void* d_logits, int logits_type, int64_t ld,
                                          int32_t* d_ids, float* d_w, int32_t* d_offsets,
                                          int32_t* d_order, void* d_ws, size_t ws_bytes,
                                          void* stream) {
    if (n_tokens < 0 || n_experts < 1 || top_k < 1 || top_k > n_experts)
        return failf(PM_ERR_ARG, "route: n_tokens=%d n_experts=%d top_k=%d", n_tokens, n_experts,
                     top_k);
    if (n_experts > PM_ROUTE_MAX_EXPERTS || top_k > PM_ROUTE_MAX_TOPK)
        return failf(PM_ERR_SHAPE, "route: n_experts=%d top_k=%d above %d, %d", n_experts, top_k,
                     PM_ROUTE_MAX_EXPERTS, PM_ROUTE_MAX_TOPK);
    if (!route_sizes_ok(n_tokens, n_experts, top_k))
        return failf(PM_ERR_ARG, "route: %d tokens of %d uses", n_tokens, top_k);
    if (!type_ok(logits_type)) return failf(PM_ERR_ARG, "route: logits type %d", logits_type);
    if (ld < n_experts || ld >= kMaxLd)
        return failf(PM_ERR_ARG, "route: row distance %lld for %d experts", (long long)ld,
                     n_experts);
    if ((d_order && !d_offsets) || (d_offsets && !d_order && n_tokens > 0))
        return failf(PM_ERR_ARG, "route: d_offsets and d_order go together");
    if (n_tokens > 0 && (!d_logits || !d_ids || !d_w))
        return failf(PM_ERR_ARG, "route: null device pointer");
    if (!aligned(d_logits, type_bytes(logits_type)) || !aligned(d_ids, 4) || !aligned(d_w, 4) ||
        !aligned(d_offsets, 4) || !aligned(d_order, 4) || !aligned(d_ws, 16))
        return failf(PM_ERR_ARG, "route: misaligned device pointer");
    const size_t need = d_offsets ? pm_route_workspace_bytes(n_tokens, n_experts, top_k) : 0;
    if (need && (!d_ws || ws_bytes < need))
        return failf(PM_ERR_ARG, "route: workspace of %zu bytes, need %zu", d_ws ? ws_bytes : 0,
                     need);
    const size_t uses = size_t(n_tokens) * top_k;
    const size_t in = span(size_t(n_tokens), ld, size_t(n_experts), logits_type);
    const struct { const void* p; size_t n; } out[5] = {
        {d_ids, 4 * uses}, {d_w, 4 * uses}, {d_offsets, d_offsets ? 4 * (size_t(n_experts) + 1) : 0},
        {d_order, d_order ? 4 * uses : 0}, {d_ws, need}};
    for (int a = 0; a < 5; ++a) {
        if (overlap(out[a].p, out[a].n, d_logits, in))
            return failf(PM_ERR_ARG, "route: an output overlaps the logits");
        for (int b = 0; b < a; ++b)
            if (overlap(out[a].p, out[a].n, out[b].p, out[b].n))
                return failf(PM_ERR_ARG, "route: outputs or workspace overlap");
    }
    if (n_tokens == 0 && !d_offsets) return PM_OK;
    RouteCall C{};
    C.logits = d_logits;
    C.ld = ld;
    C.ids = d_ids;
    C.w = d_w;
    C.offsets = d_offsets;
    C.order = d_order;
    C.hist = static_cast<uint16_t*>(d_ws);
    C.hist_stride = (n_experts + 7) & ~7;
    C.n_tokens = n_tokens;
    C.n_experts = n_experts;
    C.top_k = top_k;
    C.type = logits_type;
    route_blocks(n_tokens, &C.block_tokens, &C.n_blocks);
    return launched(launch_route(C, (hipStream_t)stream), "route");
}

// ---------------------------------------------------------------- grouped products
static pm_status check_grouped(pm_grouped_shape s, pm_grouped_rows r, const void* d_x, int x_type,
                               int64_t ldx, const void* d_y, int y_type, int64_t ldy,
                               uint32_t flags) {
    if (s.n_experts < 1 || s.rows < 0 || s.cols < 0)
        return failf(PM_ERR_SHAPE, "grouped: %d experts of %d x %d", s.n_experts, s.rows, s.cols);
    if (s.n_experts > kMaxGroupedExperts)
        return failf(PM_ERR_SHAPE, "grouped: %d experts, above %d", s.n_experts,
                     kMaxGroupedExperts);
    if (int64_t(s.rows) * std::max(s.cols, 1) >= (int64_t(1) << 30))
        return failf(PM_ERR_SHAPE, "grouped: a matrix of %d x %d holds 2^30 weights or more",
                     s.rows, s.cols);
    if (flags & ~uint32_t(PM_GROUPED_GATHER | PM_GROUPED_SCATTER | PM_GROUPED_SWIGLU))
        return failf(PM_ERR_ARG, "grouped: flags 0x%x", flags);
    if ((flags & PM_GROUPED_SWIGLU) && s.rows % 2)
        return failf(PM_ERR_SHAPE, "grouped: gate and up of %d rows together", s.rows);
    if (r.n_rows < 0 || r.top_k < 1 || !uses_ok(r.n_rows))
        return failf(PM_ERR_ARG, "grouped: n_rows=%d top_k=%d", r.n_rows, r.top_k);
    if (y_type != PM_F32 && y_type != x_type)
        return failf(PM_ERR_ARG, "grouped: x of type %d, y of type %d", x_type, y_type);
    const int out = flags & PM_GROUPED_SWIGLU ? s.rows / 2 : s.rows;
    if (ldx < s.cols || ldx >= kMaxLd || ldy < out || ldy >= kMaxLd)
        return failf(PM_ERR_ARG, "grouped: row distances %lld, %lld for %d inputs, %d outputs",
                     (long long)ldx, (long long)ldy, s.cols, out);
    if (r.n_rows == 0 || out == 0) return PM_OK;
    if (!r.d_offsets || !d_y || (s.cols > 0 && !d_x))
        return failf(PM_ERR_ARG, "grouped: null device pointer");
    if (s.cols > 0 && (!aligned(d_x, 16) || (size_t(ldx) * type_bytes(x_type)) % 16))
        return failf(PM_ERR_ARG, "grouped: rows of x are not 16-byte aligned");
    if (!aligned(d_y, type_bytes(y_type)) || !aligned(r.d_offsets, 4) || !aligned(r.d_order, 4))
        return failf(PM_ERR_ARG, "grouped: misaligned device pointer");
    const size_t nx = flags & PM_GROUPED_GATHER ? size_t(r.n_rows - 1) / r.top_k + 1 : r.n_rows;
    const size_t ny = span(r.n_rows, ldy, out, y_type);
    if (overlap(d_x, span(nx, ldx, s.cols, x_type), d_y, ny))
        return failf(PM_ERR_ARG, "grouped: x and y overlap");
    if (overlap(r.d_offsets, 4 * (size_t(s.n_experts) + 1), d_y, ny) ||
        (r.d_order && overlap(r.d_order, 4 * size_t(r.n_rows), d_y, ny)))
        return failf(PM_ERR_ARG, "grouped: y overlaps the offsets or the order");
    return PM_OK;
}

// Whether y of a checked call overlaps `per_expert` bytes of weights at p.
static bool in_weights(pm_grouped_shape s, pm_grouped_rows r, const void* p, size_t per_expert,
                       const void* d_y, int y_type, int64_t ldy, uint32_t flags) {
    const int out = flags & PM_GROUPED_SWIGLU ? s.rows / 2 : s.rows;
    return p && overlap(p, per_expert * s.n_experts, d_y, span(r.n_rows, ldy, out, y_type));
}

static GroupedCall grouped_call(pm_grouped_shape s, pm_grouped_rows r, const void* d_x, int x_type,
                                int64_t ldx, void* d_y, int y_type, int64_t ldy, uint32_t flags) {
    GroupedCall C{};
    C.x = d_x;
    C.y = d_y;
    C.offsets = r.d_offsets;
    C.order = r.d_order;
    C.ldx = ldx;
    C.ldy = ldy;
    C.n_experts = s.n_experts;
    C.rows = s.rows;
    C.cols = s.cols;
    C.n_rows = r.n_rows;
    C.top_k = r.top_k;
    C.x_type = x_type;
    C.y_type = y_type;
    C.flags = flags;
    return C;
}

extern "C" pm_status pm_grouped_gemm(pm_grouped_shape s, int type, const void* d_w,
                                     pm_grouped_rows r, const void* d_x, int64_t ldx, void* d_y,
                                     int y_type, int64_t ldy, uint32_t flags, void* stream) {
    if (type != PM_F16 && type != PM_BF16)
        return failf(PM_ERR_ARG, "grouped: weights of type %d", type);
    if (s.cols % 8)
        return failf(PM_ERR_SHAPE, "grouped: %d inputs, not a multiple of 8", s.cols);
    pm_status st = check_grouped(s, r, d_x, type, ldx, d_y, y_type, ldy, flags);
    if (st) return st;
    if (r.n_rows == 0 || s.rows == 0) return PM_OK;
    if (s.cols > 0 && (!d_w || !aligned(d_w, 16)))
        return failf(PM_ERR_ARG, "grouped: weights null or not 16-byte aligned");
    const size_t weights = size_t(s.rows) * s.cols;
    if (in_weights(s, r, d_w, 2 * weights, d_y, y_type, ldy, flags))
        return failf(PM_ERR_ARG, "grouped: y overlaps the weights");
    GroupedCall C = grouped_call(s, r, d_x, type, ldx, d_y, y_type, ldy, flags);
    C.w = d_w;
    C.w_type = type;
    return launched(launch_grouped(C, kW16, (hipStream_t)stream), "grouped product");
}

extern "C" pm_status pm_grouped_gemm_w4(pm_grouped_shape s, int group, const uint8_t* d_q,
                                        const uint16_t* d_scales, const uint8_t* d_zeros,
                                        pm_grouped_rows r, const void* d_x, int x_type,
                                        int64_t ldx, void* d_y, int y_type, int64_t ldy,
                                        uint32_t flags, void* stream) {
    if (!type_ok(x_type)) return failf(PM_ERR_ARG, "grouped: x of type %d", x_type);
    if (group < 32 || group % 32 || s.cols % group)
        return failf(PM_ERR_SHAPE, "grouped: cols=%d group=%d: need group a positive multiple of "
                     "32, cols a multiple of group", s.cols, group);
    pm_status st = check_grouped(s, r, d_x, x_type, ldx, d_y, y_type, ldy, flags);
    if (st) return st;
    if (r.n_rows == 0 || s.rows == 0) return PM_OK;
    if (s.cols > 0 && (!d_q || !d_scales || !aligned(d_q, 16) || !aligned(d_scales, 2)))
        return failf(PM_ERR_ARG, "grouped: codes or scales null or misaligned");
    const size_t weights = size_t(s.rows) * s.cols, groups = weights / group;
    if (in_weights(s, r, d_q, weights / 2, d_y, y_type, ldy, flags) ||
        in_weights(s, r, d_scales, 2 * groups, d_y, y_type, ldy, flags) ||
        in_weights(s, r, d_zeros, groups, d_y, y_type, ldy, flags))
        return failf(PM_ERR_ARG, "grouped: y overlaps the codes, scales or zero points");
    GroupedCall C = grouped_call(s, r, d_x, x_type, ldx, d_y, y_type, ldy, flags);
    C.w = d_q;
    C.scales = d_scales;
    C.zeros = d_zeros;
    C.group = group;
    return launched(launch_grouped(C, kW4, (hipStream_t)stream), "grouped 4-bit product");
}

// ---------------------------------------------------------------- 4-bit encoder
extern "C" pm_status pm_encode_w4_device(pm_matrix_shape s, const void* d_w, int type,
                                         uint8_t* d_q, uint16_t* d_scales, uint8_t* d_zeros,
                                         void* stream) {
    if (s.rows < 0 || s.cols < 0 || s.group < 32 || s.group % 32 || s.cols % s.group)
        return failf(PM_ERR_SHAPE, "encode: rows=%d cols=%d group=%d: need rows>=0, group a "
                     "positive multiple of 32, cols a multiple of group", s.rows, s.cols, s.group);
    if (!type_ok(type)) return failf(PM_ERR_ARG, "encode: weights of type %d", type);
    const size_t n_groups = size_t(s.rows) * (s.cols / s.group);
    if (n_groups == 0) return PM_OK;
    if (n_groups >= (size_t(1) << 31))
        return failf(PM_ERR_SHAPE, "encode: %zu groups", n_groups);
    if (!d_w || !d_q || !d_scales) return failf(PM_ERR_ARG, "encode: null device pointer");
    if (!aligned(d_w, 16) || !aligned(d_q, 16) || !aligned(d_scales, 2))
        return failf(PM_ERR_ARG, "encode: misaligned device pointer");
    const size_t n = size_t(s.rows) * s.cols;
    const struct { const void* p; size_t n; } buf[4] = {
        {d_w, n * type_bytes(type)}, {d_q, n / 2}, {d_scales, 2 * n_groups},
        {d_zeros, d_zeros ? n_groups : 0}};
    for (int a = 1; a < 4; ++a)
        for (int b = 0; b < a; ++b)
            if (overlap(buf[a].p, buf[a].n, buf[b].p, buf[b].n))
                return failf(PM_ERR_ARG, "encode: buffers overlap");
    return launched(launch_encode_w4(n_groups, s.group, d_w, type, d_q, d_scales, d_zeros,
                                     (hipStream_t)stream), "4-bit encoder");
}

// ---------------------------------------------------------------- combine
extern "C" pm_status pm_combine_uses(int n_tokens, int top_k, int hidden, const void* d_z,
                                     int z_type, int64_t ldz, const float* d_w, void* d_y,
                                     int y_type, int64_t ldy, void* stream) {
    if (n_tokens < 0 || top_k < 1 || hidden < 0 || !uses_ok(int64_t(n_tokens) * top_k))
        return failf(PM_ERR_ARG, "combine: n_tokens=%d top_k=%d hidden=%d", n_tokens, top_k,
                     hidden);
    if (!type_ok(z_type) || (y_type != PM_F32 && y_type != z_type))
        return failf(PM_ERR_ARG, "combine: z of type %d, y of type %d", z_type, y_type);
    if (ldz < hidden || ldz >= kMaxLd || ldy < hidden || ldy >= kMaxLd)
        return failf(PM_ERR_ARG, "combine: row distances %lld, %lld for %d columns",
                     (long long)ldz, (long long)ldy, hidden);
    if (n_tokens == 0 || hidden == 0) return PM_OK;
    if (!d_z || !d_w || !d_y) return failf(PM_ERR_ARG, "combine: null device pointer");
    if (!aligned(d_z, type_bytes(z_type)) || !aligned(d_w, 4) || !aligned(d_y, type_bytes(y_type)))
        return failf(PM_ERR_ARG, "combine: misaligned device pointer");
    const size_t uses = size_t(n_tokens) * top_k;
    const size_t ny = span(n_tokens, ldy, hidden, y_type);
    if (overlap(d_z, span(uses, ldz, hidden, z_type), d_y, ny) || overlap(d_w, 4 * uses, d_y, ny))
        return failf(PM_ERR_ARG, "combine: y overlaps z or w");
    return launched(launch_combine_uses(n_tokens, top_k, hidden, d_z, z_type, ldz, d_w, d_y,
                                        y_type, ldy, (hipStream_t)stream), "combine");
}

// moe_nt.hip -- C entry points of the mixture-of-experts layer.  Kernels:
// moe_product.h, skinny.h, moe_gate.h.
#include "moe_gate.h"
#include "moe_product.h"

namespace {

constexpr int64_t kMaxLd = int64_t(1) << 40;

bool sizes_ok_moe(const moe_nt_weights *w, int64_t T, int topk)
{
    return w && dtype_ok(w->dtype) && w->experts >= 1 && w->experts <= MOE_MAX_EXPERTS &&
           w->hidden >= 1 && w->hidden <= GEMM_MAX_K && T >= 0 && T <= INT32_MAX && topk >= 1 &&
           topk <= MOE_MAX_TOPK;
}

bool inner_ok(const moe_nt_weights *w)
{
    return w->inner >= 1 && w->inner <= MOE_MAX_INNER && (w->group == 0 || group_ok(w->group));
}

// Workspace: tickets (kept at zero between calls), the plan, and a chunk's
// logits, gated rows and their products.  The tickets are as many as the
// longest hidden size needs, one for the router and one for each 32 hidden rows
// (the fewest that a workgroup of the down product takes), 512 KB: a call of
// other sizes then never finds there what this one leaves behind them.
constexpr int64_t kTicketBytes = 4 * (1 + (GEMM_MAX_K + 31) / 32);

struct Layout {
    int64_t plan, logits, h, y, bytes;
};

Layout layout_of(int64_t T, const moe_nt_weights *w, int topk)
{
    auto up = [](int64_t n) { return cdiv(n, 256) * 256; };
    const int64_t chunk = moe_chunk(T, topk), slots = chunk * topk;
    Layout l;
    l.plan = up(kTicketBytes);
    l.logits = l.plan + up(sizeof(Plan));
    l.h = l.logits + up(route_parts(w->hidden, w->experts, chunk) * chunk * w->experts * 4);
    l.y = l.h + up(slots * w->inner * 2);
    l.bytes = l.y + up(slots * w->hidden * 4);
    return l;
}

struct Span {
    const void *p;
    uint64_t n;
};

uint64_t span_bytes(int64_t rows, int64_t cols, int64_t ld)
{
    return rows ? ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * 2u : 0u;
}

// None of `out` overlaps another of them or any of `in`.
template <int A, int B>
bool apart(const Span (&out)[A], const Span (&in)[B])
{
    for (int i = 0; i < A; ++i) {
        for (int j = i + 1; j < A; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return false;
        for (int j = 0; j < B; ++j)
            if (overlap(out[i].p, out[i].n, in[j].p, in[j].n))
                return false;
    }
    return true;
}

WeightRef weight_ref(const void *w, const void *s, const void *z, int group)
{
    WeightRef r{};
    if (group) {
        r.q = (const uint32_t *)w;
        r.s = (const uint16_t *)s;
        r.z = (const uint8_t *)z;
    } else {
        r.w = (const uint16_t *)w;
    }
    return r;
}

// Bytes of a weight of `rows` rows of `cols`, and of its scales (zero points:
// half of that).
uint64_t weight_bytes(int64_t rows, int64_t cols, int group)
{
    return group ? (uint64_t)rows * (uint64_t)cdiv(cols, 128) * 64u
                 : (uint64_t)rows * (uint64_t)cols * 2u;
}
uint64_t scale_bytes(int64_t rows, int64_t cols, int group)
{
    return group ? (uint64_t)rows * (uint64_t)cdiv(cols, group) * 2u : 0u;
}

uint64_t router_bytes(const moe_nt_weights *w)
{
    return (uint64_t)w->experts * (uint64_t)w->hidden * 2u;
}

// The experts' weights, scales and zero points.
struct ExpertSpans {
    Span part[6];

    explicit ExpertSpans(const moe_nt_weights *w)
    {
        const int64_t n13 = w->experts * 2 * w->inner, n2 = w->experts * w->hidden;
        const uint64_t s13 = scale_bytes(n13, w->hidden, w->group);
        const uint64_t s2 = scale_bytes(n2, w->inner, w->group);
        part[0] = {w->w13, weight_bytes(n13, w->hidden, w->group)};
        part[1] = {w->w2, weight_bytes(n2, w->inner, w->group)};
        part[2] = {w->w13_scales, s13};
        part[3] = {w->w2_scales, s2};
        part[4] = {w->w13_zeros, w->w13_zeros ? s13 / 2 : 0};
        part[5] = {w->w2_zeros, w->w2_zeros ? s2 / 2 : 0};
    }
};

// What the two halves share: the activations, the workspace.
int check_common(const void *X, const void *ws, int64_t ws_bytes, int64_t need)
{
    return !X || !aligned_to(X, 2) || !ws || !aligned_to(ws, 256) || ws_bytes < need ? GEMM_EINVAL : GEMM_OK;
}

int check_route(const moe_nt_weights *w, const void *X, const int32_t *ids, const float *weights,
                int64_t T, int64_t ldx, int topk, int flags, const void *ws, int64_t ws_bytes)
{
    if (!sizes_ok_moe(w, T, topk) || !inner_ok(w) || topk > w->experts ||
        (flags & ~MOE_RENORMALIZE) || ldx < w->hidden || ldx > MOE_MAX_LDX)
        return GEMM_EINVAL;
    if (T == 0)
        return GEMM_OK;
    if (!w->router || !aligned_to(w->router, 2) || !ids || !weights || !aligned_to(ids, 4) ||
        !aligned_to(weights, 4))
        return GEMM_EINVAL;
    const int rc = check_common(X, ws, ws_bytes, layout_of(T, w, topk).bytes);
    if (rc != GEMM_OK)
        return rc;
    const uint64_t slots = (uint64_t)T * (uint64_t)topk * 4u;
    return apart<3, 2>({{ids, slots}, {weights, slots}, {ws, (uint64_t)ws_bytes}},
                       {{X, span_bytes(T, w->hidden, ldx)},
                        {w->router, router_bytes(w)}})
               ? GEMM_OK
               : GEMM_EINVAL;
}

int check_experts(const moe_nt_weights *w, const void *X, const int32_t *ids, const float *weights,
                  const void *D, int64_t T, int64_t ldx, int64_t ldd, int topk, const void *ws,
                  int64_t ws_bytes)
{
    if (!sizes_ok_moe(w, T, topk) || !inner_ok(w) || ldx < w->hidden || ldx > MOE_MAX_LDX ||
        ldd < w->hidden || ldd > kMaxLd)
        return GEMM_EINVAL;
    if (T == 0)
        return GEMM_OK;
    if (!w->w13 || !w->w2 || !ids || !weights || !D || !aligned_to(D, 2) || !aligned_to(ids, 4) ||
        !aligned_to(weights, 4))
        return GEMM_EINVAL;
    const uintptr_t wa = w->group ? 16 : 2;
    if (!aligned_to(w->w13, wa) || !aligned_to(w->w2, wa))
        return GEMM_EINVAL;
    if (w->group && (!w->w13_scales || !w->w2_scales || !aligned_to(w->w13_scales, 2) ||
                     !aligned_to(w->w2_scales, 2) || !w->w13_zeros != !w->w2_zeros))
        return GEMM_EINVAL;
    const int rc = check_common(X, ws, ws_bytes, moe_nt_ws_size(T, w, topk));
    if (rc != GEMM_OK)
        return rc;
    const uint64_t slots = (uint64_t)T * (uint64_t)topk * 4u;
    const ExpertSpans e(w);
    return apart<2, 3>({{D, span_bytes(T, w->hidden, ldd)}, {ws, (uint64_t)ws_bytes}},
                       {{X, span_bytes(T, w->hidden, ldx)}, {ids, slots}, {weights, slots}}) &&
                   apart<2, 6>({{D, span_bytes(T, w->hidden, ldd)}, {ws, (uint64_t)ws_bytes}},
                               e.part)
               ? GEMM_OK
               : GEMM_EINVAL;
}

// What the whole layer adds to its halves' checks: the outputs of the one
// against the inputs of the other.
int check_across(const moe_nt_weights *w, const int32_t *ids, const float *weights, const void *D,
                 int64_t T, int64_t ldd, int topk)
{
    const uint64_t slots = (uint64_t)T * (uint64_t)topk * 4u;
    const ExpertSpans e(w);
    return apart<2, 6>({{ids, slots}, {weights, slots}}, e.part) &&
                   apart<1, 1>({{D, span_bytes(T, w->hidden, ldd)}},
                               {{w->router, router_bytes(w)}})
               ? GEMM_OK
               : GEMM_EINVAL;
}

// Likewise of a gate: its values, and its bias against all that is written (D or NULL).
int check_gate(const moe_nt_weights *w, const moe_nt_gate *g, const int32_t *ids,
               const float *weights, const void *D, int64_t T, int64_t ldd, int topk,
               const void *ws, int64_t ws_bytes)
{
    if (!gemm18_moe_gate_ok(g, w->experts, topk))
        return GEMM_EINVAL;
    const uint64_t slots = (uint64_t)T * (uint64_t)topk * 4u;
    const Span bias{g->bias, g->bias ? (uint64_t)w->experts * 4u : 0u};
    const Span out[4] = {{ids, slots},
                         {weights, slots},
                         {D, D ? span_bytes(T, w->hidden, ldd) : 0u},
                         {ws, (uint64_t)ws_bytes}};
    for (const Span &o : out)
        if (overlap(o.p, o.n, bias.p, bias.n))
            return GEMM_EINVAL;
    return GEMM_OK;
}

MoeArgs common_args(const moe_nt_weights *w, const void *X, const int32_t *ids,
                    const float *weights, int64_t T, int64_t ldx, int topk, void *ws)
{
    const Layout l = layout_of(T, w, topk);
    MoeArgs p{};
    p.tickets = (uint32_t *)ws;
    p.plan = (Plan *)((char *)ws + l.plan);
    p.h = (uint16_t *)((char *)ws + l.h);
    p.y = (float *)((char *)ws + l.y);
    p.w13 = weight_ref(w->w13, w->w13_scales, w->w13_zeros, w->group);
    p.w2 = weight_ref(w->w2, w->w2_scales, w->w2_zeros, w->group);
    p.X = (const uint16_t *)X;
    p.router = (const uint16_t *)w->router;
    p.logits = (float *)((char *)ws + l.logits);
    p.ids = (int32_t *)ids;
    p.weights = (float *)weights;
    p.ldx = ldx;
    p.E = (int)w->experts;
    p.H = (int)w->hidden;
    p.I = (int)w->inner;
    p.topk = topk;
    return p;
}

// Moves the arguments on by `T` tokens and sets the next chunk's count.
bool next_chunk(MoeArgs &p, int64_t T, int64_t &done)
{
    if (p.T) {
        p.X += p.T * p.ldx;
        if (p.D)
            p.D += p.T * p.ldd;
        p.ids += (int64_t)p.T * p.topk;
        p.weights += (int64_t)p.T * p.topk;
        done += p.T;
    }
    p.T = moe_chunk(T - done, p.topk);
    return p.T > 0;
}

MoeLaunch launches(const moe_nt_weights *w)
{
    return w->dtype == GEMM_T_BF16 ? gemm18_moe_bf16() : gemm18_moe_f16();
}

// The router, the experts or both, a chunk of tokens at a time.  With a gate the router
// leaves its logits, as for a late choice, and a kernel of its own chooses.
int run(const moe_nt_weights *w, MoeArgs p, int64_t T, bool route, bool experts,
        hipStream_t stream, const GateArgs *gate = nullptr)
{
    if (!experts)
        p.plan = nullptr;
    const MoeLaunch go = launches(w);
    const std::lock_guard<std::mutex> whole(launch_lock(p.tickets));
    for (int64_t done = 0; next_chunk(p, T, done);) {
        p.parts = route_parts(p.H, p.E, p.T);       // no more than the workspace has
        p.late = route && experts && p.T == 1 && p.E <= kLateExperts;
        if (gate) {
            MoeArgs r = p;
            r.late = 1;
            go.route(r, stream);
            GateArgs a = *gate;
            a.logits = p.logits;
            a.ids = p.ids;
            a.weights = p.weights;
            a.T = p.T;
            a.E = p.E;
            a.topk = p.topk;
            a.dtype = GEMM_T_F32;
            a.ldl = p.E;
            a.parts = p.parts;
            a.part_stride = (int64_t)p.T * p.E;
            gemm18_moe_gate(a, stream);
            p.late = 0;
        } else if (route) {
            go.route(p, stream);
        }
        if (experts)
            go.experts(p, w->group, route && !gate, stream);
    }
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

} // namespace

extern "C" {

int64_t moe_nt_ws_size(int64_t T, const moe_nt_weights *w, int topk)
{
    if (!sizes_ok_moe(w, T, topk) || !inner_ok(w) || T == 0)
        return 0;
    return layout_of(T, w, topk).bytes;
}

int moe_nt_route(const moe_nt_weights *w, const void *X, int32_t *ids, float *weights, int64_t T,
                 int64_t ldx, int topk, int flags, void *workspace, int64_t ws_bytes,
                 hipStream_t stream)
{
    const int rc = check_route(w, X, ids, weights, T, ldx, topk, flags, workspace, ws_bytes);
    if (rc != GEMM_OK || T == 0)
        return rc;
    MoeArgs p = common_args(w, X, ids, weights, T, ldx, topk, workspace);
    p.renorm = flags & MOE_RENORMALIZE;
    return run(w, p, T, true, false, stream);
}

int moe_nt_experts(const moe_nt_weights *w, const void *X, const int32_t *ids,
                   const float *weights, void *D, int64_t T, int64_t ldx, int64_t ldd, int topk,
                   void *workspace, int64_t ws_bytes, hipStream_t stream)
{
    const int rc =
        check_experts(w, X, ids, weights, D, T, ldx, ldd, topk, workspace, ws_bytes);
    if (rc != GEMM_OK || T == 0)
        return rc;
    MoeArgs p = common_args(w, X, ids, weights, T, ldx, topk, workspace);
    p.D = (uint16_t *)D;
    p.ldd = ldd;
    return run(w, p, T, false, true, stream);
}

int moe_nt_layer(const moe_nt_weights *w, const void *X, void *D, int32_t *ids, float *weights,
                 int64_t T, int64_t ldx, int64_t ldd, int topk, int flags, void *workspace,
                 int64_t ws_bytes, hipStream_t stream)
{
    int rc = check_route(w, X, ids, weights, T, ldx, topk, flags, workspace, ws_bytes);
    if (rc == GEMM_OK)
        rc = check_experts(w, X, ids, weights, D, T, ldx, ldd, topk, workspace, ws_bytes);
    if (rc == GEMM_OK)
        rc = check_across(w, ids, weights, D, T, ldd, topk);
    if (rc != GEMM_OK || T == 0)
        return rc;
    MoeArgs p = common_args(w, X, ids, weights, T, ldx, topk, workspace);
    p.renorm = flags & MOE_RENORMALIZE;
    p.D = (uint16_t *)D;
    p.ldd = ldd;
    return run(w, p, T, true, true, stream);
}

int moe_nt_route_gated(const moe_nt_weights *w, const moe_nt_gate *g, const void *X,
                       int32_t *ids, float *weights, int64_t T, int64_t ldx, int topk, int flags,
                       void *workspace, int64_t ws_bytes, hipStream_t stream)
{
    int rc = check_route(w, X, ids, weights, T, ldx, topk, flags, workspace, ws_bytes);
    if (rc == GEMM_OK)
        rc = check_gate(w, g, ids, weights, nullptr, T, 0, topk, workspace, ws_bytes);
    if (rc != GEMM_OK || T == 0)
        return rc;
    const GateArgs gate = gemm18_moe_gate_args(g, flags);
    return run(w, common_args(w, X, ids, weights, T, ldx, topk, workspace), T, true, false,
               stream, &gate);
}

int moe_nt_layer_gated(const moe_nt_weights *w, const moe_nt_gate *g, const void *X, void *D,
                       int32_t *ids, float *weights, int64_t T, int64_t ldx, int64_t ldd,
                       int topk, int flags, void *workspace, int64_t ws_bytes,
                       hipStream_t stream)
{
    int rc = check_route(w, X, ids, weights, T, ldx, topk, flags, workspace, ws_bytes);
    if (rc == GEMM_OK)
        rc = check_experts(w, X, ids, weights, D, T, ldx, ldd, topk, workspace, ws_bytes);
    if (rc == GEMM_OK)
        rc = check_across(w, ids, weights, D, T, ldd, topk);
    if (rc == GEMM_OK)
        rc = check_gate(w, g, ids, weights, D, T, ldd, topk, workspace, ws_bytes);
    if (rc != GEMM_OK || T == 0)
        return rc;
    MoeArgs p = common_args(w, X, ids, weights, T, ldx, topk, workspace);
    p.D = (uint16_t *)D;
    p.ldd = ldd;
    const GateArgs gate = gemm18_moe_gate_args(g, flags);
    return run(w, p, T, true, true, stream, &gate);
}

} // extern "C"

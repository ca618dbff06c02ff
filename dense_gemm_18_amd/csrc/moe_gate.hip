// moe_gate.hip -- the choice of experts from logits: softmax or sigmoid scores, a bias
// for the choice alone, groups, the topk largest.  Kernel and C entry point.
#include "moe_gate.h"

namespace {

constexpr int kGateWaves = 4;       // tokens of a workgroup

// The order of logits as unsigned numbers: rising with the value, both zeros alike,
// every NaN below everything, 0 left for what is absent or taken.
__device__ __forceinline__ uint32_t rank_of(float v)
{
    if (!(v == v))
        return 1;
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
    return (u & 0x80000000u ? ~u : u | 0x80000000u) + 1;
}

// A choice as a number that a maximum can take: infinite ones become large and NaN the
// least, above kTaken, which is what is absent or taken.
constexpr double kLeast = -1e300, kNone = -1e301;
__device__ __forceinline__ double rank_of(double v)
{
    v = v > kLeast ? v : v == v ? kLeast : kNone;
    return v < -kLeast ? v : -kLeast;
}

template <class T>
constexpr T kTaken = 0;
template <>
constexpr double kTaken<double> = -__builtin_inf();

__device__ __forceinline__ uint32_t top(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ double top(double a, double b) { return __builtin_fmax(a, b); }

// One step of a reduction by data-parallel moves; lanes without a source get `none`.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v, float none)
{
    return __builtin_bit_cast(float, moved<CTRL, ROWS>(__builtin_bit_cast(uint32_t, v),
                                                       __builtin_bit_cast(uint32_t, none)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v, double none)
{
    const u32x2 a = __builtin_bit_cast(u32x2, v), b = __builtin_bit_cast(u32x2, none);
    return __builtin_bit_cast(double, u32x2{moved<CTRL, ROWS>(a[0], b[0]),
                                            moved<CTRL, ROWS>(a[1], b[1])});
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float from_lane(float v, int lane)
{
    return __builtin_bit_cast(float, from_lane(__builtin_bit_cast(uint32_t, v), lane));
}
__device__ __forceinline__ double from_lane(double v, int lane)
{
    const u32x2 a = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{from_lane(a[0], lane), from_lane(a[1], lane)});
}

// f over the wave, the result in every lane.
template <class T, class F>
__device__ __forceinline__ T over_wave(T v, T none, F &&f)
{
    v = f(v, moved<0x111, 0xf>(v, none));       // 1, 2, 4, 8 lanes up
    v = f(v, moved<0x112, 0xf>(v, none));
    v = f(v, moved<0x114, 0xf>(v, none));
    v = f(v, moved<0x118, 0xf>(v, none));
    v = f(v, moved<0x142, 0xa>(v, none));       // lane 15 of a row into the next
    v = f(v, moved<0x143, 0xc>(v, none));       // lane 31 into the upper half
    return from_lane(v, 63);
}

__device__ __forceinline__ float logit(const GateArgs &p, int64_t t, int e)
{
    const int64_t at = t * p.ldl + e;
    if (p.dtype == GEMM_T_F32) {
        const float *q = (const float *)p.logits + at;
        float v = *q;
        for (int i = 1; i < p.parts; ++i)
            v += q[i * p.part_stride];
        return v;
    }
    const uint16_t bits = ((const uint16_t *)p.logits)[at];
    return p.dtype == GEMM_T_BF16 ? to_float<true>(bits) : to_float<false>(bits);
}

// The groups that stay, as a mask, from the choices (as numbers, absent ones kTaken).
// `lds`: E doubles of this wave.  Each group is scanned by as many lanes as there are for
// each, their two largest are joined, and each group's lane counts the groups before it.
template <int PER>
__device__ __forceinline__ uint64_t groups_of(const GateArgs &p, const double (&c)[PER],
                                              double *lds)
{
    const int lane = threadIdx.x & 63, G = p.groups, n = p.E / G;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lane + 64 * i < p.E)
            lds[lane + 64 * i] = c[i];
    // a wave's LDS operations are done in order
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    int per = 1;                           // lanes of a group
    while (2 * per * G <= 64)
        per *= 2;
    const int g = lane / per;
    double first = kTaken<double>, second = kTaken<double>;
    if (g < G)
        for (int k = lane % per; k < n; k += per) {
            const double v = lds[g * n + k];
            second = top(second, v < first ? v : first);
            first = top(first, v);
        }
    for (int d = 1; d < per; d *= 2) {
        const double a = __shfl_xor(first, d), b = __shfl_xor(second, d);
        second = top(a < first ? a : first, top(second, b));
        first = top(first, a);
    }
    double value = p.group_top == 2 ? first + second : first;
    value = value > kLeast ? value : kLeast;
    int before = 0;
    for (int j = 0; j < G; ++j) {
        const double other = from_lane(value, j * per);
        before += other > value || (other == value && j < g);
    }
    uint64_t keep = __ballot(g < G && lane % per == 0 && before < p.kept);
    if (per > 1) {                         // bit g * per to bit g
        uint64_t packed = 0;
        for (int j = 0; j < G; ++j)
            packed |= (keep >> (j * per) & 1) << j;
        keep = packed;
    }
    return keep;
}

// One token to a wave, expert lane + 64 i in lane's element i.  WIDE: choices in 64 bits,
// else the logits' order.  topk maxima over the wave, each taken at its lowest index; lane
// j keeps the j-th expert and its logit, of which it forms the score at the end.
template <int PER, bool WIDE>
__global__ void __launch_bounds__(kGateWaves * 64) moe_gate_kernel(GateArgs p)
{
    extern __shared__ double choices[];
    using Key = typename std::conditional<WIDE, double, uint32_t>::type;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t t =
        (blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * kGateWaves + wave;
    if (t >= p.T)
        return;
    float v[PER], most = -__builtin_inff();
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = lane + 64 * i < p.E;
        v[i] = in ? logit(p, t, lane + 64 * i) : -__builtin_inff();
        bad |= !(v[i] == v[i]);
        most = __builtin_fmaxf(most, v[i]);
    }
    bad = __any(bad);
    double sum = 1.0;                      // of a softmax
    if (!p.sigmoid) {
        most = over_wave(most, -__builtin_inff(),
                         [](float a, float b) { return __builtin_fmaxf(a, b); });
        bad |= !(__builtin_fabsf(most) < __builtin_inff());
    }
    Key key[PER];
    if constexpr (WIDE) {
        double score[PER];
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                score[i] = 1.0 / (1.0 + exp(-(double)v[i]));
        } else {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                score[i] = exp((double)v[i] - (double)most);
                sum += score[i];
            }
            sum = over_wave(sum, 0.0, [](double a, double b) { return a + b; });
#pragma unroll
            for (int i = 0; i < PER; ++i)
                score[i] /= sum;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            key[i] = e < p.E ? rank_of(score[i] + (p.bias ? (double)p.bias[e] : 0.0))
                             : kTaken<double>;
        }
    } else {
        if (!p.sigmoid && !p.renorm) {
            float each = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                each += expf(v[i] - most);
            sum = over_wave(each, 0.0f, [](float a, float b) { return a + b; });
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = lane + 64 * i < p.E ? rank_of(v[i]) : 0;
    }
    if (p.groups > 1) {
        uint64_t keep;
        if constexpr (WIDE) {
            keep = groups_of<PER>(p, key, choices + wave * p.E);
        } else {
            double c[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                c[i] = (double)key[i];
            keep = groups_of<PER>(p, c, choices + wave * p.E);
        }
        const float per = 1.0f / (float)(p.E / p.groups);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // e + 1/2 is 1 / (2 E) or more of a group away from where the next begins
            const int g = (int)(((float)(lane + 64 * i) + 0.5f) * per);
            if (!(keep >> (g & 63) & 1))
                key[i] = kTaken<Key>;
        }
    }
    int id = 0;
    float chosen = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        Key best = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i)
            best = top(best, key[i]);
        best = over_wave(best, kTaken<Key>, [](Key a, Key b) { return top(a, b); });
        bool found = false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint64_t who = found ? 0 : __ballot(key[i] == best);
            if (who) {
                const int at = __builtin_ctzll(who);
                const float l = from_lane(v[i], at);
                id = lane == j ? at + 64 * i : id;
                chosen = lane == j ? l : chosen;
                key[i] = lane == at ? kTaken<Key> : key[i];
                found = true;
            }
        }
    }
    const bool mine = lane < p.topk;
    double w = 0.0;
    if (mine)
        w = p.sigmoid ? 1.0 / (1.0 + exp(-(double)chosen))
                      : exp((double)chosen - (double)most) / sum;
    if (p.renorm) {
        double all = w;                    // topk <= 16: the first row of lanes
#pragma unroll
        for (int d = 1; d < 16; d *= 2)
            all += __shfl_xor(all, d);
        w = all > 0.0 ? w / all : w;
    }
    if (mine) {
        p.ids[t * p.topk + lane] = id;
        p.weights[t * p.topk + lane] = bad ? __builtin_nanf("") : (float)(w * p.scale);
    }
}

template <int PER>
void launch_gate(const GateArgs &a, hipStream_t stream)
{
    const dim3 grid = tile_grid(cdiv(a.T, kGateWaves));
    const int lds = a.groups > 1 ? kGateWaves * a.E * (int)sizeof(double) : 0;
    if (a.bias || (a.groups > 1 && a.group_top > 1))
        hipLaunchKernelGGL((moe_gate_kernel<PER, true>), grid, dim3(kGateWaves * 64), lds, stream,
                           a);
    else
        hipLaunchKernelGGL((moe_gate_kernel<PER, false>), grid, dim3(kGateWaves * 64), lds,
                           stream, a);
}

constexpr int64_t kMaxLd = int64_t(1) << 40;

} // namespace

void gemm18_moe_gate(const GateArgs &a, hipStream_t stream)
{
    if (a.E <= 64)
        launch_gate<1>(a, stream);
    else if (a.E <= 128)
        launch_gate<2>(a, stream);
    else if (a.E <= 256)
        launch_gate<4>(a, stream);
    else if (a.E <= 512)
        launch_gate<8>(a, stream);
    else
        launch_gate<16>(a, stream);
}

bool gemm18_moe_gate_ok(const moe_nt_gate *g, int64_t E, int topk)
{
    if (!g || (g->scoring != MOE_SOFTMAX && g->scoring != MOE_SIGMOID) || g->groups < 1 ||
        g->groups > MOE_MAX_GROUPS || E % g->groups || !aligned_to(g->bias, 4))
        return false;
    const int64_t n = E / g->groups;
    return g->topk_groups >= 1 && g->topk_groups <= g->groups && topk <= g->topk_groups * n &&
           g->group_top >= 1 && g->group_top <= 2 && g->group_top <= n &&
           __builtin_fabsf(g->scale) < __builtin_inff();
}

GateArgs gemm18_moe_gate_args(const moe_nt_gate *g, int flags)
{
    GateArgs a{};
    a.bias = g->bias;
    a.renorm = flags & MOE_RENORMALIZE;
    a.sigmoid = g->scoring == MOE_SIGMOID;
    // with all groups kept their values do not matter
    a.groups = g->topk_groups == g->groups ? 1 : g->groups;
    a.kept = g->topk_groups;
    a.group_top = g->group_top;
    a.scale = g->scale;
    a.parts = 1;
    return a;
}

extern "C" int moe_nt_choose(const moe_nt_gate *g, const void *logits, int32_t *ids,
                             float *weights, int64_t T, int64_t experts, int64_t ldl, int topk,
                             int flags, int dtype, hipStream_t stream)
{
    if (experts < 1 || experts > MOE_MAX_EXPERTS || T < 0 || T > INT32_MAX || topk < 1 ||
        topk > MOE_MAX_TOPK || topk > experts || (flags & ~MOE_RENORMALIZE) || ldl < experts ||
        ldl > kMaxLd || (!dtype_ok(dtype) && dtype != GEMM_T_F32) ||
        !gemm18_moe_gate_ok(g, experts, topk))
        return GEMM_EINVAL;
    if (T == 0)
        return GEMM_OK;
    const uint64_t size = dtype == GEMM_T_F32 ? 4 : 2;
    if (!logits || !ids || !weights || !aligned_to(logits, size) || !aligned_to(ids, 4) ||
        !aligned_to(weights, 4))
        return GEMM_EINVAL;
    const uint64_t slots = (uint64_t)T * (uint64_t)topk * 4u;
    const uint64_t l = ((uint64_t)(T - 1) * (uint64_t)ldl + (uint64_t)experts) * size;
    const uint64_t b = g->bias ? (uint64_t)experts * 4u : 0u;
    if (overlap(ids, slots, weights, slots) || overlap(ids, slots, logits, l) ||
        overlap(weights, slots, logits, l) || overlap(ids, slots, g->bias, b) ||
        overlap(weights, slots, g->bias, b))
        return GEMM_EINVAL;
    GateArgs a = gemm18_moe_gate_args(g, flags);
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.ldl = ldl;
    a.E = (int)experts;
    a.topk = topk;
    a.dtype = dtype;
    gemm18_moe_gate(a, stream);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

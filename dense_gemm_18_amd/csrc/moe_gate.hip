// moe_gate.hip -- the choice of experts from logits: softmax or sigmoid scores, a bias
// for the choice alone, groups, the topk largest.  Kernel and C entry point.
#include "moe_gate.h"

namespace {

constexpr int kGateWaves = 4;       // of a workgroup

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

constexpr double kTaken = -__builtin_inf();

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

// exp(x - most) with what the difference's rounding, up to 2^-24 of it, leaves out.
__device__ __forceinline__ float exp_below(float x, float most)
{
    const float d = x - most, back = d - x;
    const float rest = (x - (d - back)) + (-most - back);
    const float e = expf(d);
    return __builtin_fmaf(e, rest, e);
}

// PLAIN: one fp32 number for each.
template <bool PLAIN>
__device__ __forceinline__ float logit(const GateArgs &p, int64_t t, int e)
{
    const int64_t at = t * p.ldl + e;
    if constexpr (PLAIN)
        return ((const float *)p.logits)[at];
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
    double first = kTaken, second = kTaken;
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

// A lane's choices as 64-bit numbers, the rank above and below it the complement of the
// expert, so that the larger is the one that comes first, in falling order (Batcher's merge
// exchange).
template <int PER>
__device__ __forceinline__ void sort_lane(uint64_t (&c)[PER])
{
    static_for<0, 4>([&](auto pp) {
        constexpr int p = 1 << decltype(pp)::value;
        if constexpr (p < PER)
            static_for<0, decltype(pp)::value + 1>([&](auto kk) {
                constexpr int k = p >> decltype(kk)::value;
                static_for<0, PER>([&](auto ii) {
                    constexpr int a = decltype(ii)::value, b = a + k;
                    // a runs over the first halves of blocks of 2 k that start at k % p
                    constexpr int at = a - k % p;
                    if constexpr (at >= 0 && at / k % 2 == 0 && b < PER && a / (2 * p) == b / (2 * p)) {
                        const bool swap = c[b] > c[a];
                        const uint64_t x = swap ? c[b] : c[a], y = swap ? c[a] : c[b];
                        c[a] = x;
                        c[b] = y;
                    }
                });
            });
    });
}

__device__ __forceinline__ uint32_t upper(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// rank_of's logit.
__device__ __forceinline__ float of_rank(uint32_t rank)
{
    const uint32_t u = rank - 1;
    return __builtin_bit_cast(float, u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// The topk largest of the lanes' sorted choices, the j-th expert in lane j.  APART: also
// whether each of them is more than `margin` plus 2^-22 of both magnitudes above the one
// after it, the first one left out included.
template <int PER, bool APART>
__device__ __forceinline__ bool take(uint64_t (&c)[PER], int topk, float margin, int &id)
{
    const int lane = threadIdx.x & 63;
    uint32_t rank = 0;                         // of the j-th in lane j, 0: nothing is left
    for (int j = 0; j < topk; ++j) {
        const uint32_t best = over_wave(upper(c[0]), 0u, umax);
        uint64_t who = __ballot(upper(c[0]) == best);
        if (__popcll(who) > 1) {               // equal ones: the lowest expert
            const uint32_t low = upper(c[0]) == best ? (uint32_t)c[0] : 0;
            const uint32_t most = over_wave(low, 0u, umax);
            who = __ballot(upper(c[0]) == best && (uint32_t)c[0] == most);
        }
        const int at = __builtin_ctzll(who);
        const int e = (int)~from_lane((uint32_t)c[0], at);
        id = lane == j ? e : id;
        if constexpr (APART)
            rank = lane == j ? best : rank;
        if (lane == at) {
#pragma unroll
            for (int i = 0; i + 1 < PER; ++i)
                c[i] = c[i + 1];
            c[PER - 1] = 0;
        }
    }
    if constexpr (!APART)
        return true;
    const uint32_t best = over_wave(upper(c[0]), 0u, umax);
    rank = lane == topk ? best : rank;
    const float v = of_rank(rank), next = __shfl_down(v, 1);
    const bool last = __shfl_down(rank, 1) == 0;
    return __all(lane >= topk || last ||
                 v - next > margin + 0x1p-22f * (__builtin_fabsf(v) + __builtin_fabsf(next)));
}

// The groups that stay, from choices in fp32 that are off by `margin` / 2 plus 2^-23 of
// their magnitude at most; false if another order within that would change them.
template <int PER>
__device__ __forceinline__ bool groups_apart(const GateArgs &p, const float (&c)[PER],
                                             float *lds, float margin, uint64_t &keep)
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
    const float none = -__builtin_inff();
    float first = none, second = none;
    if (g < G)
        for (int k = lane % per; k < n; k += per) {
            const float v = lds[g * n + k];
            second = __builtin_fmaxf(second, __builtin_fminf(v, first));
            first = __builtin_fmaxf(first, v);
        }
    for (int d = 1; d < per; d *= 2) {
        const float a = __shfl_xor(first, d), b = __shfl_xor(second, d);
        second = __builtin_fmaxf(__builtin_fminf(a, first), __builtin_fmaxf(second, b));
        first = __builtin_fmaxf(first, a);
    }
    const float value = p.group_top == 2 ? first + second : first;
    // of any group, in magnitude
    const float size = over_wave(
        g < G ? p.group_top == 2 ? __builtin_fabsf(first) + __builtin_fabsf(second)
                                 : __builtin_fabsf(first)
              : 0.0f,
        0.0f, [](float a, float b) { return __builtin_fmaxf(a, b); });
    const float slack = 2.0f * margin + 0x1p-20f * size;
    const float high = value + slack, low = value - slack;
    int surely = 0, perhaps = 0;           // groups before this one
    for (int j = 0; j < G; ++j) {
        const float other = from_lane(value, j * per);
        surely += other > high;
        perhaps += !(other < low);
    }
    perhaps -= 1;                          // itself
    const bool mine = g < G && lane % per == 0;
    const uint64_t stays = __ballot(mine && perhaps < p.kept);
    const uint64_t goes = __ballot(mine && surely >= p.kept);
    keep = 0;
    for (int j = 0; j < G; ++j)
        keep |= (stays >> (j * per) & 1) << j;
    return __popcll(stays) + __popcll(goes) == G;
}

__device__ __forceinline__ int group_at(int e, float per)
{
    // e + 1/2 is 1 / (2 E) or more of a group away from where the next begins
    return (int)(((float)e + 0.5f) * per);
}

// One token to a wave, expert lane + 64 i in lane's element i.  Without WIDE the order of
// the logits is that of the choices.  With it choices are formed in fp32 first, each within
// 2^-19 of the largest score and 2^-23 of itself of what 64 bits would give (an exponential,
// a reciprocal and up to 22 additions); if the chosen ones, and the groups, are further apart
// than that, their order is known, and else this token is done in 64 bits: one in some
// hundreds.  Lane j keeps the j-th expert, of whose logit it forms the score at the end.
// lds: E doubles of this wave, where there are groups.
template <int PER, bool WIDE, bool PLAIN>
__device__ __forceinline__ void gate_token(const GateArgs &p, int64_t t, double *lds)
{
    const int lane = threadIdx.x & 63;
    float v[PER], most = -__builtin_inff();
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = lane + 64 * i < p.E;
        v[i] = in ? logit<PLAIN>(p, t, lane + 64 * i) : -__builtin_inff();
        bad |= !(v[i] == v[i]);
        most = __builtin_fmaxf(most, v[i]);
    }
    bad = __any(bad);
    float sum = 1.0f;                      // of a softmax
    if (!p.sigmoid) {
        most = over_wave(most, -__builtin_inff(),
                         [](float a, float b) { return __builtin_fmaxf(a, b); });
        bad |= !(__builtin_fabsf(most) < __builtin_inff());
    }
    const auto add = [](float a, float b) { return a + b; };
    const float per = 1.0f / (float)(p.E / p.groups);
    int id = 0;
    bool done = true;
    uint64_t c[PER];
    if constexpr (WIDE) {
        float score[PER], scale = 1.0f;
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                // the exponent's rounding, 2^-24 |v|, times score (1 - score) is below 2^-25
                score[i] = __builtin_amdgcn_rcpf(
                    1.0f + __builtin_amdgcn_exp2f(v[i] * -1.44269504f));
        } else {
            float each = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                score[i] = expf(v[i] - most);
                each += score[i];
            }
            scale = 1.0f / over_wave(each, 0.0f, add);
        }
        // `scale` is the largest score, or for a sigmoid above it
        const float margin = 0x1p-18f * scale;
        uint64_t keep = ~0ull;
        float choice[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            choice[i] = score[i] * scale;
            if (p.bias)
                choice[i] += e < p.E ? p.bias[e] : 0.0f;
        }
        if (p.groups > 1)
            done = groups_apart<PER>(p, choice, (float *)lds, margin, keep);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            const bool in = e < p.E && (p.groups == 1 || (keep >> (group_at(e, per) & 63) & 1));
            c[i] = in ? (uint64_t)rank_of(choice[i]) << 32 | (uint32_t)~e : 0;
        }
        sort_lane(c);
        done = done && !bad && take<PER, true>(c, p.topk, margin, id);
        if (!done) {
            // in 64 bits
            double exact[PER];
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    exact[i] = 1.0 / (1.0 + exp(-(double)v[i]));
            } else {
                double every = 0.0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    exact[i] = exp((double)v[i] - (double)most);
                    every += exact[i];
                }
                every = over_wave(every, 0.0, [](double a, double b) { return a + b; });
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    exact[i] /= every;
                sum = (float)every;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 64 * i;
                exact[i] = e < p.E ? rank_of(exact[i] + (p.bias ? (double)p.bias[e] : 0.0))
                                   : kTaken;
            }
            if (p.groups > 1) {
                keep = groups_of<PER>(p, exact, lds);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (!(keep >> (group_at(lane + 64 * i, per) & 63) & 1))
                        exact[i] = kTaken;
            }
            for (int j = 0; j < p.topk; ++j) {
                double best = exact[0];
#pragma unroll
                for (int i = 1; i < PER; ++i)
                    best = top(best, exact[i]);
                best = over_wave(best, kTaken, [](double a, double b) { return top(a, b); });
                bool found = false;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint64_t who = found ? 0 : __ballot(exact[i] == best);
                    if (who) {
                        const int at = __builtin_ctzll(who);
                        id = lane == j ? at + 64 * i : id;
                        exact[i] = lane == at ? kTaken : exact[i];
                        found = true;
                    }
                }
            }
        }
        if (!p.sigmoid && done)
            sum = 1.0f / scale;
    } else {
        if (!p.sigmoid && !p.renorm) {
            float each = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                each += expf(v[i] - most);
            sum = over_wave(each, 0.0f, add);
        }
        uint64_t keep = ~0ull;
        if (p.groups > 1) {
            double ranks[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                ranks[i] = lane + 64 * i < p.E ? (double)rank_of(v[i]) : kTaken;
            keep = groups_of<PER>(p, ranks, lds);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            const bool in = e < p.E && (p.groups == 1 || (keep >> (group_at(e, per) & 63) & 1));
            c[i] = in ? (uint64_t)rank_of(v[i]) << 32 | (uint32_t)~e : 0;
        }
        sort_lane(c);
        take<PER, false>(c, p.topk, 0.0f, id);
    }
    const bool mine = lane < p.topk;
    const float chosen = mine ? logit<PLAIN>(p, t, id) : 0.0f;
    // topk <= 16: sums over the first row of lanes
    float w = 0.0f;
    if (mine)
        w = p.sigmoid ? 1.0f / (1.0f + expf(-chosen)) : exp_below(chosen, most) / sum;
    if (p.renorm) {
        float all = w;
#pragma unroll
        for (int d = 1; d < 16; d *= 2)
            all += __shfl_xor(all, d);
        w /= all;
        if (__any(lane < 16 && !(all > 0x1p-80f))) {     // below fp32's range, or nearly
            double x = 0.0;
            if (mine)
                x = p.sigmoid ? 1.0 / (1.0 + exp(-(double)chosen))
                              : exp((double)chosen - (double)most);
            double every = x;
#pragma unroll
            for (int d = 1; d < 16; d *= 2)
                every += __shfl_xor(every, d);
            w = every > 0.0 ? (float)(x / every) : (float)x;
        }
    }
    if (mine) {
        p.ids[t * p.topk + lane] = id;
        p.weights[t * p.topk + lane] = bad ? __builtin_nanf("") : w * p.scale;
    }
}

template <int PER, bool WIDE, bool PLAIN>
__global__ void __launch_bounds__(kGateWaves * 64) moe_gate_kernel(GateArgs p)
{
    extern __shared__ double choices[];
    const int wave = uniform(threadIdx.x >> 6);
    const int64_t t = (blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * kGateWaves + wave;
    if (t < p.T)
        gate_token<PER, WIDE, PLAIN>(p, t, choices + wave * p.E);
}

// ---- 64, 128 or many tokens of 256 experts --------------------------------

// Reductions over 16 lanes, a token's, the result in each of them.
template <int CTRL>
__device__ __forceinline__ uint32_t turned(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float turned(float v)
{
    return __builtin_bit_cast(float, turned<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <class T, class F>
__device__ __forceinline__ T over_16(T v, F &&f)
{
    v = f(v, turned<0x121>(v));                // rotated by 1, 2, 4 and 8 lanes
    v = f(v, turned<0x122>(v));
    v = f(v, turned<0x124>(v));
    return f(v, turned<0x128>(v));
}
__device__ __forceinline__ float fmost(float a, float b) { return __builtin_fmaxf(a, b); }

// Falling order of a lane's 16 keys or fewer, for keys that are all different.
template <int PER>
__device__ __forceinline__ void sort_keys(uint32_t (&c)[PER])
{
    static_for<0, 4>([&](auto pp) {
        constexpr int p = 1 << decltype(pp)::value;
        if constexpr (p < PER)
            static_for<0, decltype(pp)::value + 1>([&](auto kk) {
                constexpr int k = p >> decltype(kk)::value;
                static_for<0, PER>([&](auto ii) {
                    constexpr int a = decltype(ii)::value, b = a + k, at = a - k % p;
                    if constexpr (at >= 0 && at / k % 2 == 0 && b < PER && a / (2 * p) == b / (2 * p)) {
                        const uint32_t x = c[a], y = c[b];
                        c[a] = x > y ? x : y;
                        c[b] = x > y ? y : x;
                    }
                });
            });
    });
}

// Four tokens to a wave, 16 lanes and PER = E / 16 consecutive experts of a lane to each: a
// reduction is four moves within a row of lanes and serves four tokens.  A key holds a
// choice in 24 bits of fixed point below the token's largest and the expert's complement in
// 8, so that keys differ and a minimum and a maximum order two of them.  Neighbours among the
// chosen closer than what fp32 and the fixed point leave open are ordered again in 64 bits;
// where that does not settle the choice (groups that close, or a third neighbour, or out of
// the fixed point's range; NaN and infinite ones), the whole wave does the token again with
// gate_token: one in ten thousand or so.  16-bit logits without WIDE have their order in the
// upper 16 bits (fp16: 19) of their numbers in fp32: exact.
// 16384 tokens of 256 experts in 8 groups, 8 chosen, a bias: 13 to 18 us (its bytes take 3),
// 277 VALU instructions to a token, 65 % of the issue slots; 26.8 us and 675 instructions with
// a token to a wave, 28.7 in 64 bits throughout.
// span: lanes of a group, a power of two; 0: one group.
template <int PER, bool WIDE, int TYPE>
__global__ void __launch_bounds__(kGateWaves * 64) moe_gate_many_kernel(GateArgs p, int span)
{
    extern __shared__ double choices[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l = lane & 15;
    const int64_t t0 =
        ((blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * kGateWaves + wave) * 4;
    if (t0 >= p.T)
        return;
    const int64_t t = t0 + (lane >> 4);
    const int64_t row = t < p.T ? t : p.T - 1;       // lanes past the end repeat the last
    constexpr bool kExact = !WIDE && TYPE != GEMM_T_F32;
    // the compiler's loads of 16 bytes at whatever alignment the elements have
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    float v[PER], bias[PER];
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        if constexpr (TYPE == GEMM_T_F32) {
            const f32x4 x =
                *(const f32x4_any *)((const float *)p.logits + row * p.ldl + l * PER + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[i + e] = x[e];
        } else {
            const u32x2 x =
                *(const u32x2_any *)((const uint16_t *)p.logits + row * p.ldl + l * PER + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[i + e] = to_float<TYPE == GEMM_T_BF16>(
                    (uint16_t)(x[e >> 1] >> (16 * (e & 1))));
        }
        if (WIDE && p.bias) {
            const f32x4 x = *(const f32x4_any *)(p.bias + l * PER + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                bias[i + e] = x[e];
        }
    }
    bool unclear = false;
    float most = v[0];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        unclear |= !(__builtin_fabsf(v[i]) < __builtin_inff());
        most = fmost(most, v[i]);
    }
    const auto add = [](float a, float b) { return a + b; };
    const bool sums = !p.sigmoid && (WIDE || !p.renorm);
    if (!p.sigmoid)
        most = over_16(most, fmost);
    float sum = 1.0f, scale = 1.0f, choice[PER];
    if (sums) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            choice[i] = expf(v[i] - most);
            sum += choice[i];
        }
        sum = over_16(sum, add);
        scale = 1.0f / sum;
    }
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (p.sigmoid)
                // the exponent's rounding, 2^-24 |v|, times score (1 - score) is below 2^-25
                choice[i] = __builtin_amdgcn_rcpf(
                    1.0f + __builtin_amdgcn_exp2f(v[i] * -1.44269504f));
            else
                choice[i] *= scale;
            if (p.bias)
                choice[i] += bias[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            choice[i] = v[i];
    }
    // What fp32 leaves open between two choices besides 2^-23 of their size.  A sigmoid is off
    // by 2^-22 at most: 2^-23 from the exponential, as much from the reciprocal, less from the
    // rest; a softmax by its sum's 22 additions.
    const float margin = WIDE ? (p.sigmoid ? 0x1p-20f : 0x1p-18f) * scale : 0.0f;
    bool keep = true;
    float largest = choice[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
        largest = fmost(largest, choice[i]);
    if (span) {
        float first = choice[0], second = -__builtin_inff();
#pragma unroll
        for (int i = 1; i < PER; ++i) {
            second = fmost(second, __builtin_fminf(choice[i], first));
            first = fmost(first, choice[i]);
        }
        for (int d = 1; d < span; d *= 2) {
            const float a = __shfl_xor(first, d), b = __shfl_xor(second, d);
            second = fmost(__builtin_fminf(a, first), fmost(second, b));
            first = fmost(first, a);
        }
        const bool two = p.group_top == 2;
        const float value = two ? first + second : first;
        const float size =
            over_16(__builtin_fabsf(first) + (two ? __builtin_fabsf(second) : 0.0f), fmost);
        // without WIDE a value is a logit, and equal ones go by index
        const float slack = WIDE ? 2.0f * margin + 0x1p-20f * size : 0.0f;
        const float high = value + slack, low = value - slack;
        int surely = 0, perhaps = 0;
        for (int j = 0; j < 16; j += span) {
            const float other = __shfl(value, (lane & 48) + j);
            const bool before = j < (l & -span);
            surely += other > high || (!WIDE && before && other == value);
            perhaps += WIDE ? !(other < low) : other > value || (before && other == value);
        }
        perhaps -= WIDE;                              // itself
        keep = perhaps < p.kept;
        unclear |= !keep && surely < p.kept;
    }
    largest = over_16(keep ? largest : -__builtin_inff(), fmost);
    uint32_t key[PER];
    // fixed point: `range` below the largest is 0, what is below that too
    const float range = WIDE ? 2.0f * scale + 0.5f * __builtin_fabsf(largest) : 32.0f;
    const float by = 16777215.0f / range;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t low = 255 - (l * PER + i);
        if constexpr (kExact) {
            key[i] = ((rank_of(v[i]) - 1) & 0xffffff00u) | low;
        } else {
            const float f = (choice[i] - largest) * by + 16777215.0f;
            key[i] = (uint32_t)__builtin_amdgcn_fmed3f(f, 0.0f, 16777215.0f) << 8 | low;
        }
        key[i] = keep ? key[i] : low & 0xfu;
    }
    sort_keys(key);
    uint32_t chosen = 0;                              // the j-th key in lane j
    for (int j = 0; j < p.topk + 2; ++j) {
        const uint32_t best = over_16(key[0], umax);
        chosen = l == j ? best : chosen;
        if (best == key[0]) {
#pragma unroll
            for (int i = 0; i + 1 < PER; ++i)
                key[i] = key[i + 1];
            key[PER - 1] = 0;
        }
    }
    const int id = 255 - (chosen & 255);
    float x;
    if constexpr (TYPE == GEMM_T_F32)
        x = ((const float *)p.logits)[row * p.ldl + id];
    else
        x = to_float<TYPE == GEMM_T_BF16>(((const uint16_t *)p.logits)[row * p.ldl + id]);
    int place = l;
    if constexpr (!kExact) {
        // choices in range are no larger than that; 3 for the fixed point's roundings, which
        // keep the order of what they tell apart
        const float size = WIDE ? __builtin_fabsf(largest) + range : 0.0f;
        const float open = (margin + 0x1p-22f * size) * by + 3.0f;
        const uint32_t c = chosen >> 8;
        const uint32_t one = __shfl_down(chosen, 1) >> 8, two = __shfl_down(chosen, 2) >> 8;
        unclear |= l < p.topk && c < 16;
        unclear |= l == p.topk - 1 && (float)(c - two) < open;
        const bool close = l < p.topk && (float)(c - one) < open;
        if (WIDE && p.bias && !p.sigmoid) {
            unclear |= close;              // a softmax's sum is wanted in 64 bits too
        } else if (__any(close)) {
            // Neighbours too close, but the last of the topk + 2 clearly below: the order of
            // these by their choices in 64 bits settles it.  (Without a bias the logits'.)
            double v64 = x;
            if (WIDE && p.bias)
                v64 = 1.0 / (1.0 + exp(-(double)x)) + (double)p.bias[id];
            const bool in = l < p.topk + 2;
            v64 = in ? v64 : -__builtin_inf();
            place = in ? 0 : 16;
            for (int d = 1; d < 16; ++d) {
                const int from = (lane & 48) + ((l + d) & 15);
                const double other = __shfl(v64, from);
                const int its = __shfl(id, from);      // every lane's, before any branch
                place += (int)(other > v64) | ((int)(other == v64) & (int)(its < id));
            }
        }
    }
    const bool mine = place < p.topk;
    float w = 0.0f;
    if (mine)
        w = p.sigmoid ? 1.0f / (1.0f + expf(-x)) : exp_below(x, most) * scale;
    if (p.renorm) {
        const float all = over_16(w, add);
        unclear |= !(all > 0x1p-80f);
        w /= all;
    }
    const uint64_t again = __ballot(unclear && t < p.T);
    if (mine && t < p.T && !(again >> (lane & 48) & 0xffff)) {
        p.ids[t * p.topk + place] = id;
        p.weights[t * p.topk + place] = w * p.scale;
    }
    for (int r = 0; r < 4; ++r)
        if (again >> (16 * r) & 0xffff)
            gate_token<(PER + 3) / 4, WIDE, TYPE == GEMM_T_F32>(p, t0 + r,
                                                               choices + wave * p.E);
}

template <int PER, int TYPE>
void launch_many(const GateArgs &a, int span, hipStream_t stream)
{
    const dim3 grid = tile_grid(cdiv(a.T, 4 * kGateWaves));
    const int lds = a.groups > 1 ? kGateWaves * a.E * (int)sizeof(double) : 0;
    if (a.bias || (a.groups > 1 && a.group_top > 1))
        hipLaunchKernelGGL((moe_gate_many_kernel<PER, true, TYPE>), grid, dim3(kGateWaves * 64),
                           lds, stream, a, span);
    else
        hipLaunchKernelGGL((moe_gate_many_kernel<PER, false, TYPE>), grid, dim3(kGateWaves * 64),
                           lds, stream, a, span);
}

template <int PER>
void launch_many_typed(const GateArgs &a, int span, hipStream_t stream)
{
    if (a.dtype == GEMM_T_F32)
        launch_many<PER, GEMM_T_F32>(a, span, stream);
    else if (a.dtype == GEMM_T_BF16)
        launch_many<PER, GEMM_T_BF16>(a, span, stream);
    else
        launch_many<PER, GEMM_T_F16>(a, span, stream);
}

// Whether that kernel can take the call, and if so launches it: groups of whole lanes, a
// power of two of them, and few enough chosen for the two after them to have lanes.  In us,
// a token to a wave / four, 8 chosen: 64 experts, 64 tokens 3.3 / 3.0, 16384 8.6 / 4.7; 128,
// bias and 8 groups, 512 tokens 8.0 / 4.5, 16384 18.6 / 11.5; 256, 1024 tokens 4.1 / 4.6 and
// with bias and groups 6.4 / 6.5, 2048 4.3 / 4.7 and 10.6 / 6.6, 16384 11.8 / 7.8 and 23.5 /
// 12.2.
bool launch_many_tokens(const GateArgs &a, hipStream_t stream)
{
    if ((a.E != 64 && a.E != 128 && (a.E != 256 || a.T < 2048)) || a.parts != 1 || a.topk > 14)
        return false;
    int span = 0;
    if (a.groups > 1) {
        span = 16 / a.groups;
        if (span * a.groups != 16)
            return false;
    }
    if (a.E == 64)
        launch_many_typed<4>(a, span, stream);
    else if (a.E == 128)
        launch_many_typed<8>(a, span, stream);
    else
        launch_many_typed<16>(a, span, stream);
    return true;
}

template <int PER>
void launch_gate(const GateArgs &a, hipStream_t stream)
{
    const dim3 grid = tile_grid(cdiv(a.T, kGateWaves));
    const int lds = a.groups > 1 ? kGateWaves * a.E * (int)sizeof(double) : 0;
    const auto go = [&](auto wide, auto plain) {
        hipLaunchKernelGGL(
            (moe_gate_kernel<PER, decltype(wide)::value, decltype(plain)::value>), grid,
            dim3(kGateWaves * 64), lds, stream, a);
    };
    const auto typed = [&](auto wide) {
        if (a.dtype == GEMM_T_F32 && a.parts == 1)
            go(wide, std::true_type{});
        else
            go(wide, std::false_type{});
    };
    if (a.bias || (a.groups > 1 && a.group_top > 1))
        typed(std::true_type{});
    else
        typed(std::false_type{});
}

constexpr int64_t kMaxLd = int64_t(1) << 40;

} // namespace

void gemm18_moe_gate(const GateArgs &a, hipStream_t stream)
{
    if (launch_many_tokens(a, stream))
        return;
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

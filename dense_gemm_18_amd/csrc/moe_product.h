// moe_product.h -- kernels and launches of the mixture-of-experts layer,
// compiled once for each 16-bit type.
#pragma once

#include "skinny.h"

// Tokens of one pass through the kernels: 64, or as many as have 512 slots
// (t * topk + j).
constexpr int kMoeSlots = 512;
inline int moe_chunk(int64_t T, int topk)
{
    const int most = kMoeSlots / topk < 64 ? kMoeSlots / topk : 64;
    return T < most ? (int)T : most;
}

// Which slots (t * topk + j) go to which expert: the experts that have any, in
// rising order, and each one's slots side by side.  In the workspace, for the
// launches that follow.  The order of an expert's slots is that of the LDS
// atomics and changes no result: a slot is a row of its own in every product.
struct Plan {
    struct Item {
        int expert, first, count;    // slots slot[first .. first + count); count 0: none
        int slot;                    // slot[first]
    } item[kMoeSlots];
    int active;                      // items in use
    int slot[kMoeSlots];
    int token[kMoeSlots];        // slot[i] / topk
};

struct MoeArgs {
    const uint16_t *X;             // T rows, ldx apart
    const uint16_t *router;        // E x H
    float *logits;                 // parts x T x E
    int32_t *ids;                  // T x topk
    float *weights;                // T x topk
    WeightRef w13, w2;             // E * 2 * I rows of H, E * H rows of I
    uint16_t *h;                   // T * topk rows of I
    float *y;                      // T * topk rows of H
    Plan *plan;                    // null: the router leaves none
    uint32_t *tickets;             // the router's, then one for each block of the down product
    uint16_t *D;                   // T rows, ldd apart
    int64_t ldx, ldd;
    int T, E, H, I, topk, renorm;
    int parts;                     // pieces of H in the router
    int late;                      // the experts' first kernel chooses, not the router
};
constexpr int kLateExperts = 256;

// One translation unit for each type.  Not exported from the library.
struct MoeLaunch {
    void (*route)(const MoeArgs &, hipStream_t);
    void (*experts)(const MoeArgs &, int group, bool planned, hipStream_t);
};
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_f16();
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_bf16();

namespace {

// Words that several workgroups of one launch share (logits, products of the
// slots, tickets) move with agent-scope relaxed atomics, which on gfx950 are
// loads and stores that every XCD's L2 passes on; no fence, which would write
// back or drop a whole L2.
template <class T>
__device__ __forceinline__ void put(T *p, T v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get(const T *p)
{
    return __hip_atomic_load(const_cast<T *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// True in the last of `count` workgroups to come here: what every one of them
// has put() before is then visible.  The counter goes back to 0 for the next
// launch.  Every thread of the workgroup calls it; `flag` is a word of LDS.
__device__ __forceinline__ bool last_of(uint32_t *counter, uint32_t count, uint32_t *flag)
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);       // this wave's stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before =
            __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = before + 1 == count;
        if (before + 1 == count)
            put(counter, 0u);
    }
    __syncthreads();
    const bool last = *flag;
    asm volatile("" ::: "memory");
    return last;
}

// ---- plan ---------------------------------------------------------------

// By one workgroup.  cnt: MOE_MAX_EXPERTS ints of LDS.  ids(i): slot i's id.
template <class F>
__device__ __forceinline__ void make_plan(Plan *plan, int n, int topk, int E, int *cnt,
                                          F &&ids)
{
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        cnt[e] = 0;
    __syncthreads();
    int id = -1;
    if (threadIdx.x < n) {               // n <= kMoeSlots <= blockDim.x
        id = ids(threadIdx.x);
        id = (uint32_t)id < (uint32_t)E ? id : -1;
        if (id >= 0)
            atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int at = 0, base = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int c = e0 + lane < E ? cnt[e0 + lane] : 0;
            int sum = c;                               // inclusive prefix sum
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int up = __shfl_up(sum, d);
                sum += lane >= d ? up : 0;
            }
            const uint64_t has = __ballot(c > 0);
            if (c > 0) {
                const int k = at + __popcll(has & ((1ull << lane) - 1));
                plan->item[k].expert = e0 + lane;
                plan->item[k].first = base + sum - c;
                plan->item[k].count = c;
                cnt[e0 + lane] = (base + sum - c) << 16 | k;
            }
            at += __popcll(has);
            base += __shfl(sum, 63);
        }
        // what a launch for as many items as there can be also looks at
        for (int k = at + lane; k < min(E, n); k += 64)
            plan->item[k].count = 0;
        if (lane == 0)
            plan->active = at;
    }
    __syncthreads();
    if (id >= 0) {
        const int place = atomicAdd(&cnt[id], 1 << 16);
        plan->slot[place >> 16] = threadIdx.x;
        plan->token[place >> 16] = threadIdx.x / topk;
    }
    __syncthreads();
    // the first slots, now that all are in place
    if (id >= 0) {
        const int k = cnt[id] & 0xffff;
        plan->item[k].slot = plan->slot[plan->item[k].first];
    }
}

template <int = 0>
__global__ void __launch_bounds__(kMoeSlots) moe_plan_kernel(MoeArgs p)
{
    __shared__ int cnt[MOE_MAX_EXPERTS];
    make_plan(p.plan, p.T * p.topk, p.topk, p.E, cnt, [&](int i) { return p.ids[i]; });
}

// ---- router -------------------------------------------------------------

constexpr int kRouteWaves = 8;
constexpr int kRouteK = 1024;        // of the hidden size, to a workgroup
// Pieces of the hidden size.  One, for a workgroup alone, where the product is
// small: no ticket, no logits through memory.  4 tokens, 8 experts, hidden size
// 1024, 2048, 4096: 4.9, 5.2 and 6.7 us; in pieces 6.1, 6.1 and 6.5.
inline int route_parts(int64_t H, int64_t E, int64_t T)
{
    if (E <= 16 && T <= 16 && H <= 2 * kRouteK)
        return 1;
    return H <= 16 * kRouteK ? (int)cdiv(H, kRouteK) : 16;
}

// Order of logits as unsigned numbers: rising with the value, both zeros
// alike, every NaN below everything.
__device__ __forceinline__ uint32_t order_of(float v)
{
    if (!(v == v))
        return 0;
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Reductions over the wave by data-parallel moves (in order, no LDS): the
// result as a scalar.  `none`: what leaves a value as it is.
template <class T, class F>
__device__ __forceinline__ T reduce_wave(T v, T none, F &&f)
{
    auto step = [&](auto ctrl, auto rows) G18_INLINE {
        const int moved = __builtin_amdgcn_update_dpp(
            __builtin_bit_cast(int, none), __builtin_bit_cast(int, v), decltype(ctrl)::value,
            decltype(rows)::value, 0xf, false);
        v = f(v, __builtin_bit_cast(T, moved));
    };
    step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // 1 up
    step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});  // 2 up
    step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});  // 4 up
    step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});  // 8 up
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // lane 15 on
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // lane 31 on
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The topk largest logits of the tokens first, first + step, ... (NT of them,
// those below T) and their softmax weights, by one wave with PER logits of
// each token per lane (E <= 64 * PER): topk maxima over the wave of the
// logits' order, each taken at its lowest index.  Several tokens at once hide
// the moves' latency (64 tokens, 16 experts: 17 us one after the other by
// counting larger ones, 64 comparisons for each).
template <int PER, int NT>
__device__ __forceinline__ void choose(const float (&v)[NT][PER], const MoeArgs &p, int first,
                                       int step, int *lds_ids)
{
    const int lane = threadIdx.x & 63;
    uint32_t key[NT][PER];
    int place[NT][PER];
    float top[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float most = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // 0: absent or taken
            key[t][i] = lane + 64 * i < p.E ? order_of(v[t][i]) + 1 : 0;
            place[t][i] = INT32_MAX;
            most = __builtin_fmaxf(most, v[t][i]);      // a NaN shows in the sum below
        }
        top[t] = reduce_wave(most, -__builtin_inff(),
                             [](float a, float b) { return __builtin_fmaxf(a, b); });
    }
    for (int j = 0; j < p.topk; ++j) {
        auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                most = larger(most, key[t][i]);
            most = reduce_wave(most, 0u, larger);
            bool found = false;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint64_t who = __ballot(key[t][i] == most);
                const bool mine = !found && who && lane == __builtin_ctzll(who);
                found |= who != 0;
                place[t][i] = mine ? j : place[t][i];
                key[t][i] = mine ? 0 : key[t][i];
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float sum = 0.0f, chosen = 0.0f, w[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            w[i] = lane + 64 * i < p.E ? expf(v[t][i] - top[t]) : 0.0f;
            sum += w[i];
            chosen += place[t][i] < p.topk ? w[i] : 0.0f;
        }
        auto add = [](float a, float b) { return a + b; };
        sum = reduce_wave(sum, 0.0f, add);
        chosen = reduce_wave(chosen, 0.0f, add);
        const float over = p.renorm && sum == sum ? chosen : sum;
        const int token = first + t * step;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (token < p.T && place[t][i] < p.topk) {
                const int slot = token * p.topk + place[t][i];
                p.ids[slot] = lane + 64 * i;
                if (lds_ids)
                    lds_ids[slot] = lane + 64 * i;
                p.weights[slot] = w[i] / over;
            }
    }
}

// Logits of 16 experts for 16 tokens over one of `parts` pieces of the hidden
// size (a router is small: with the whole of it to a workgroup, 64 tokens of
// 4096 against 16 experts took 22 us); the last workgroup adds the pieces in
// order, chooses for every token and makes the plan.  Or, for one token of a
// layer with up to kLateExperts, nobody does: every workgroup of the up kernel
// chooses for itself.
template <bool BF>
using RouteCore = Skinny<BF, 0, 1, 1, kRouteWaves, 1, true>;

template <bool BF, int PER>
__global__ void __launch_bounds__(kRouteWaves * 64) moe_route_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    __shared__ float few[16 * 16];       // the logits of a workgroup on its own
    const bool alone = PER == 1 && gridDim.x * gridDim.y * gridDim.z == 1;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, part = blockIdx.z;
    // pieces of whole steps
    const int steps = (p.H + 127) >> 7;
    const int k0 = part * steps / p.parts * 128;
    RouteCore<BF> c;
    c.W.w = p.router;
    c.row[0] = e0;
    c.rows[0] = p.E - e0;
    c.stride = p.H;
    c.K = min((part + 1) * steps / p.parts * 128, p.H) - k0;
    c.W.w += k0;
    c.M = min(16, p.T - t0);
    c.begin((char *)lds, p.X + t0 * p.ldx + k0, (uint32_t)((c.M - 1) * p.ldx + c.K) * 2u);
    c.run([&](int m) { return (uint32_t)(m * p.ldx) * 2u; });
    float *logits = p.logits + (int64_t)part * p.T * p.E;
    c.join([&](int m, int n, const float(&v)[1]) {
        if (alone && !p.late)
            few[m * 16 + n] = v[0];
        else if (e0 + n < p.E)
            put(logits + (t0 + m) * p.E + e0 + n, v[0]);
    });
    if (p.late)
        return;
    __syncthreads();
    int *cnt = (int *)lds, *ids = cnt + MOE_MAX_EXPERTS;
    if (!alone && !last_of(p.tickets, gridDim.x * gridDim.y * gridDim.z, (uint32_t *)ids))
        return;
    __syncthreads();
    // four of a wave's tokens at a time, all their logits under way at once
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    constexpr int kTokens = PER == 1 ? 4 : PER == 4 ? 2 : 1;
    for (int base = wave; base < p.T; base += kTokens * kRouteWaves) {
        float v[kTokens][PER];
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[k][i] = alone ? few[min(base + k * kRouteWaves, 15) * 16 + min(lane, 15)] : 0.0f;
        // these loads go past L2 and take 2 us: as many as fit at once
        for (int q = alone ? p.parts : 0; q < p.parts; q += 4) {
            float g[4][kTokens][PER];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < kTokens; ++k)
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int t = base + k * kRouteWaves, e = lane + 64 * i;
                        const bool in = q + j < p.parts && t < p.T && e < p.E;
                        g[j][k][i] =
                            get(p.logits + (in ? ((int64_t)(q + j) * p.T + t) * p.E + e : 0));
                    }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < kTokens; ++k)
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        v[k][i] += q + j < p.parts ? g[j][k][i] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[k][i] = lane + 64 * i < p.E ? v[k][i] : -__builtin_inff();
        choose<PER, kTokens>(v, p, base, kRouteWaves, ids);
    }
    __syncthreads();
    if (p.plan && p.T > 1)
        make_plan(p.plan, p.T * p.topk, p.topk, p.E, cnt, [&](int i) { return ids[i]; });
}

// The expert of one token's slot s, by every wave for itself from the logits
// that the launch before has left: the rounds of `choose` up to s.  `write`:
// and all ids and weights, for the launches that follow.  A router that
// chooses itself passes its logits through memory to the last workgroup to
// end.  4096 x 64, 8 chosen, 1536 inner rows in 4 bits: router and up product
// 12.2 + 19.2 us that way, 4.5 + 21.0 this way; 1024 x 8, 2 chosen: 8.1 + 5.7,
// 3.5 + 6.2; the whole layer of 4096 x 256, 8 chosen: 41.4 and 38.1.
template <int PER>
__device__ __forceinline__ int choose_slot(const MoeArgs &p, int s, bool write)
{
    const int lane = threadIdx.x & 63;
    float v[1][PER] = {};
    for (int q = 0; q < p.parts; q += 4) {
        float g[4][PER];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 64 * i;
                g[j][i] = p.logits[q + j < p.parts && e < p.E ? (q + j) * p.E + e : 0];
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[0][i] += q + j < p.parts ? g[j][i] : 0.0f;
    }
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = lane + 64 * i < p.E;
        v[0][i] = in ? v[0][i] : -__builtin_inff();
        key[i] = in ? order_of(v[0][i]) + 1 : 0;
    }
    if (write)
        choose<PER, 1>(v, p, 0, 1, nullptr);
    int expert = 0;
    for (int j = 0; j <= s; ++j) {
        auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            most = larger(most, key[i]);
        most = reduce_wave(most, 0u, larger);
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const uint64_t who = __ballot(key[i] == most);
            expert = who ? __builtin_ctzll(who) + 64 * i : expert;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = lane + 64 * i == expert ? 0 : key[i];
    }
    return expert;
}

// ---- experts ------------------------------------------------------------

constexpr int kMoeWaves = 8;
constexpr int64_t kOneLds = 96 * 1024;   // of the one-token down product, at most

// Waves along K and blocks of 16 hidden rows to a wave of the down product,
// whose K, the inner size, is short.
template <int GS>
constexpr int kDownWaves = GS ? 4 : 8;
template <int GS>
constexpr int kDownRows = 16 * 2 * (kMoeWaves / kDownWaves<GS>);
static_assert(kDownRows<0> >= 32 && kDownRows<128> >= 32, "a ticket for each 32 hidden rows");

template <bool BF, int GS, int RB, int MB>
using UpCore = Skinny<BF, GS, RB, MB, kMoeWaves, 1, false>;
template <bool BF, int GS, int MB>
using DownCore = Skinny<BF, GS, 2, MB, kDownWaves<GS>, kMoeWaves / kDownWaves<GS>, true>;

// h = silu(gate) * up for some of an expert's inner rows and all its slots.
// One workgroup takes 8 * RB gate rows and their 8 * RB up rows, its waves split
// the hidden size.  Bound by reading w13: 64 tokens, 2 of 16 experts, 4096 x
// 4096 bf16, 204 us for 1.07 GB (5.3 TB/s); 16 tokens, 6 of 64, 2048 x 1024,
// 74 us for the 50 experts or so that any token chose (5.7 TB/s); one token,
// 8 of 64, 4096 x 1536 in 4 bits, bf16, 22 us for 53 MB: a workgroup's first loads
// wait for its expert, and unpacking takes the VALU for half of the time.
template <bool BF, int GS, int RB, int MB>
__global__ void __launch_bounds__(kMoeWaves * 64, MB == 1 ? 4 : 2) moe_up_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    const int blocks = (p.I + 8 * RB - 1) / (8 * RB);
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int s = wg / blocks, i0 = wg % blocks * (8 * RB);
    if (s >= (p.T == 1 ? p.topk : min(p.E, p.T * p.topk)))
        return;                  // past the end of a grid with a second dimension
    Plan::Item it;
    if (p.T == 1) {              // a slot is an expert: no plan
        const bool write = wg == 0 && threadIdx.x < 64;
        // (with more rows than 8 for each expert nothing is late)
        it.expert = MB > 1 || !p.late ? p.ids[s]
                    : p.E <= 64       ? choose_slot<1>(p, s, write)
                                      : choose_slot<kLateExperts / 64>(p, s, write);
        it.first = it.slot = s;
        it.count = (uint32_t)it.expert < (uint32_t)p.E;
    } else {
        it = p.plan->item[s];
    }
    const int64_t e = it.expert;
    for (int c0 = 0; c0 < it.count; c0 += 16 * MB) {
        const int count = min(16 * MB, it.count - c0);
        // a single row, the common case of few tokens, needs no further load
        auto slot = [&](int m) {
            return it.count == 1 ? it.slot : p.plan->slot[it.first + c0 + m];
        };
        UpCore<BF, GS, RB, MB> c;
        c.W = p.w13;
        c.row[0] = e * 2 * p.I + i0;
        c.row[1] = c.row[0] + p.I;
        c.rows[0] = c.rows[1] = p.I - i0;
        c.K = p.H;
        c.M = count;
        c.begin((char *)lds, p.X, (uint32_t)((p.T - 1) * p.ldx + p.H) * 2u);
        c.run([&](int m) {
            const int t = it.count == 1 ? it.slot / p.topk : p.plan->token[it.first + c0 + m];
            return (uint32_t)(t * p.ldx) * 2u;
        });
        c.join([&](int m, int n, const float(&v)[RB]) {
#pragma unroll
            for (int r = 0; r < RB / 2; ++r) {
                const int i = i0 + 16 * r + n;
                if (i < p.I) {
                    const float act = v[r] / (1.0f + expf(-v[r]));
                    // in the type that the down product's matrix instructions take
                    p.h[(int64_t)slot(m) * p.I + i] = from_float<BF>(act * v[RB / 2 + r]);
                }
            }
        });
        __syncthreads();
    }
}

// y = W2 h for a block of an expert's hidden rows and all its slots, in fp32;
// the last expert's workgroup of a block then forms each token's weighted
// sum, over its slots in order.  As above, 121 us for 0.54 GB (4.5 TB/s) and 51
// us (4.2 TB/s): K is short, so a workgroup's first loads and its end weigh more.
template <bool BF, int GS, int MB>
__global__ void __launch_bounds__(kMoeWaves * 64, MB == 1 ? 4 : 2) moe_down_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    const int n = p.T * p.topk, blocks = (p.H + kDownRows<GS> - 1) / kDownRows<GS>;
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int s = wg / blocks, block = wg % blocks, h0 = block * kDownRows<GS>;
    if (s >= min(p.E, n))
        return;                  // past the end of a grid with a second dimension
    const Plan::Item it = p.plan->item[s];
    if (it.count == 0 && s > 0)
        return;
    if (it.count > 0) {
        const int64_t e = it.expert;
        for (int c0 = 0; c0 < it.count; c0 += 16 * MB) {
            const int count = min(16 * MB, it.count - c0);
            auto slot = [&](int m) {
                return it.count == 1 ? it.slot : p.plan->slot[it.first + c0 + m];
            };
            DownCore<BF, GS, MB> c;
            c.W = p.w2;
            c.row[0] = e * p.H + h0;
            c.rows[0] = p.H - h0;
            c.K = p.I;
            c.M = count;
            c.begin((char *)lds, p.h, (uint32_t)n * (uint32_t)p.I * 2u);
            c.run([&](int m) { return (uint32_t)slot(m) * (uint32_t)p.I * 2u; });
            c.join([&](int m, int i, const float(&v)[2]) {
                const int h = h0 + (i >> 4) * 32 + (i & 15);
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (h + 16 * r < p.H)
                        put(p.y + (int64_t)slot(m) * p.H + h + 16 * r, v[r]);
            });
            __syncthreads();
        }
        if (!last_of(p.tickets + 1 + block, p.plan->active, (uint32_t *)lds))
            return;
    }
    for (int i = threadIdx.x; i < p.T * kDownRows<GS>; i += kMoeWaves * 64) {
        const int t = i / kDownRows<GS>, h = h0 + i % kDownRows<GS>;
        if (h >= p.H)
            continue;
        float sum = 0.0f;
        // four slots' loads under way at once, those of slots that are left out
        // or past the last without use
        for (int j0 = 0; j0 < p.topk; j0 += 4) {
            float y[4], weight[4];
            int id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int slot = t * p.topk + min(j0 + j, p.topk - 1);
                id[j] = j0 + j < p.topk ? p.ids[slot] : -1;
                weight[j] = p.weights[slot];
                y[j] = get(p.y + (int64_t)slot * p.H + h);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((uint32_t)id[j] < (uint32_t)p.E)
                    sum = __builtin_fmaf(weight[j], y[j], sum);
        }
        p.D[t * p.ldd + h] = from_float<BF>(sum);
    }
}

// One token: its slots' products are one long product, of the experts' rows
// side by side with the gated rows end to end.  A workgroup takes 16 hidden
// rows of every chosen expert, its waves share the (expert, piece of inner)
// pairs, and the weighted sum is their join, in the pairs' order: nothing passes
// through memory.
// 8 of 64 experts, 4096 x 1536 in 4 bits: 12 us, what its loads take; 2 of 8,
// 1024 x 1024: 4.9 us, with the kernels for many tokens 7.2.
template <bool BF, int GS>
using OneCore = Skinny<BF, GS, 1, 1, kMoeWaves, 1, true>;

template <bool BF, int GS>
__global__ void __launch_bounds__(kMoeWaves * 64, 4) moe_down_one_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    using Core = OneCore<BF, GS>;
    const int h0 = blockIdx.x * 16, steps = (p.I + 127) >> 7;
    Core c;
    c.W = p.w2;
    c.K = p.I;
    c.rows[0] = p.H - h0;
    auto bind = [&](int j) {
        const int e = p.ids[j];
        c.row[0] = (int64_t)((uint32_t)e < (uint32_t)p.E ? e : 0) * p.H + h0;
        c.M = 1;
        c.begin((char *)lds, p.h, (uint32_t)p.topk * (uint32_t)p.I * 2u);
        return (uint32_t)e < (uint32_t)p.E;
    };
    // the gated rows, then each expert's scales
    bind(0);
    c.M = p.topk;
    c.chunk = steps * 128;
    c.astride = c.chunk * 2 + 16;
    c.sstride = steps * Core::kGroups + 1;
    c.stage_acts(0, steps, [&](int m) { return (uint32_t)m * (uint32_t)p.I * 2u; });
    uint32_t *scales = (uint32_t *)((char *)lds + p.topk * c.astride);
    if constexpr (GS != 0) {
        // 16 threads along the groups of a row, the rest along the rows of all
        // experts; four rows' loads at once, from a valid place where there is
        // nothing to load
        const int G = (p.I + GS - 1) / GS, groups = steps * Core::kGroups;
        for (int g0 = threadIdx.x & 15; g0 < groups; g0 += 16)
            for (int n0 = threadIdx.x >> 4; n0 < p.topk * 16; n0 += 4 * 32) {
                uint32_t s[4], z[4];
                bool in[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = n0 + 32 * i, e = n < p.topk * 16 ? p.ids[n >> 4] : -1;
                    in[i] = (uint32_t)e < (uint32_t)p.E && g0 < G && h0 + (n & 15) < p.H;
                    const int64_t at =
                        in[i] ? ((int64_t)e * p.H + h0 + (n & 15)) * G + g0 : 0;
                    s[i] = p.w2.s[at];
                    z[i] = p.w2.z ? p.w2.z[at] & 15 : 8;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + 32 * i < p.topk * 16)
                        scales[(n0 + 32 * i) * c.sstride + g0] =
                            (in[i] ? s[i] : 0) | (0x6400u + z[i]) << 16;
            }
    }
    __syncthreads();

    const int units = p.topk * p.parts;
    f32x4 sum[1][1] = {{f32x4{0.0f, 0.0f, 0.0f, 0.0f}}};
    for (int u = c.wave; u < units; u += kMoeWaves) {
        const int j = u / p.parts, part = u % p.parts;
        if (!bind(j))
            continue;
        c.astride = steps * 256 + 16;
        c.sstride = steps * Core::kGroups + 1;
        const char *acts = (const char *)lds + j * c.astride;
        const uint32_t *sc = scales + j * 16 * c.sstride;
        const int first = part * steps / p.parts, last = (part + 1) * steps / p.parts;
        typename Core::template Batch<Core::U> b;
#pragma nounroll
        for (int st = first; st < last; st += Core::U) {
            c.load(b, st, last);
#pragma unroll
            for (int k = 0; k < Core::U; ++k)
                if (st + k < last)
                    c.consume(b, k, st + k, 0, acts, sc);
        }
        const float w = p.weights[j];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[0][0][e] = __builtin_fmaf(w, c.acc[0][0][e], sum[0][0][e]);
    }
    c.M = 1;
    c.acc[0][0] = sum[0][0];
    c.join([&](int, int i, const float(&v)[1]) {
        if (h0 + i < p.H)
            p.D[h0 + i] = from_float<BF>(v[0]);
    });
}

// LDS of that kernel, in bytes.
template <bool BF, int GS>
int64_t one_bytes(int topk, int I)
{
    const int64_t steps = cdiv(I, 128);
    const int64_t need =
        topk * (steps * 256 + 16 +
                (GS ? 16 * 4 * (steps * OneCore<BF, GS>::kGroups + 1) : 0));
    return need > kMoeWaves * 1024 ? need : kMoeWaves * 1024;
}

template <bool BF, int PER>
void launch_route_per(const MoeArgs &p, hipStream_t stream)
{
    const int act = RouteCore<BF>::lds_bytes(p.T < 16 ? p.T : 16, (int)cdiv(cdiv(p.H, 128), p.parts) * 128);
    const int last = (MOE_MAX_EXPERTS + kMoeSlots) * 4;
    hipLaunchKernelGGL((moe_route_kernel<BF, PER>),
                       dim3((unsigned)cdiv(p.E, 16), (unsigned)cdiv(p.T, 16), (unsigned)p.parts),
                       dim3(kRouteWaves * 64), act > last ? act : last, stream, p);
}

template <bool BF>
void launch_route(const MoeArgs &p, hipStream_t stream)
{
    if (p.E <= 64)
        launch_route_per<BF, 1>(p, stream);
    else if (p.E <= 256)
        launch_route_per<BF, 4>(p, stream);
    else
        launch_route_per<BF, 16>(p, stream);
}

template <bool BF>
void launch_experts(const MoeArgs &p, int group, bool planned, hipStream_t stream)
{
    const int n = p.T * p.topk, most = p.E < n ? p.E : n;
    // workgroups for every item of the plan; one token has none, its slots may
    // name an expert twice
    const int slots = p.T == 1 ? n : most;
    if (!planned && p.T > 1)
        hipLaunchKernelGGL((moe_plan_kernel<>), dim3(1), dim3(kMoeSlots), 0, stream, p);
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value;
        auto go = [&](auto mbs) {
            constexpr int MB = decltype(mbs)::value;
            const int rows = n < 16 * MB ? n : 16 * MB;
            auto up = [&](auto rbs) {
                constexpr int RB = decltype(rbs)::value;
                hipLaunchKernelGGL((moe_up_kernel<BF, GS, RB, MB>),
                                   tile_grid(slots * cdiv(p.I, 8 * RB)), dim3(kMoeWaves * 64),
                                   (UpCore<BF, GS, RB, MB>::lds_bytes(rows, p.H)), stream, p);
            };
            // Packed weights, 32 inner rows to a workgroup where rows are long
            // and that leaves four for each CU: 8 KB of a wave's loads are then
            // a smaller part of its work.  Layers in us with 16 and with 32, bf16,
            // groups of 128 and of 64: 2 of 8 experts of 4096 x 8192, 2 tokens
            // (1024 workgroups) 78, 73 and 83, 79; 8 tokens (2048) 176, 152 and
            // 180, 157; 64 tokens, 2 of 16, 4096 x 4096, 268, 230 and 276, 238;
            // with 512 workgroups 51, 49 and 45, 45.  Groups of 32 win and lose a
            // little (the same: 98, 103; 212, 212; 307, 284; 55, 60), and lose where
            // rows are short (2048 x 1024, 6 of 64: 106, 126).
            if (GS && p.H >= 4096 && slots * cdiv(p.I, 32) >= 4 * kCUs)
                up(std::integral_constant<int, GS ? 4 : 2>{});
            else
                up(std::integral_constant<int, 2>{});
            const int64_t one = one_bytes<BF, GS>(p.topk, p.I);
            if (p.T == 1 && one <= kOneLds) {
                // as many pairs as make all waves' work alike
                MoeArgs q = p;
                q.parts = p.topk % 8 == 0 ? 1 : p.topk % 4 == 0 ? 2 : p.topk % 2 == 0 ? 4 : 8;
                hipLaunchKernelGGL((moe_down_one_kernel<BF, GS>),
                                   dim3((unsigned)cdiv(p.H, 16)), dim3(kMoeWaves * 64), (int)one,
                                   stream, q);
                return;
            }
            if (p.T == 1)
                hipLaunchKernelGGL((moe_plan_kernel<>), dim3(1), dim3(kMoeSlots), 0, stream, p);
            hipLaunchKernelGGL((moe_down_kernel<BF, GS, MB>),
                               tile_grid(most * cdiv(p.H, kDownRows<GS>)), dim3(kMoeWaves * 64),
                               (DownCore<BF, GS, MB>::lds_bytes(rows, p.I)), stream, p);
        };
        // 16 rows against one reading of an expert's weights, in registers that
        // let two workgroups share a CU, or 32 where the mean is above 8
        if (n <= 8 * p.E)
            go(std::integral_constant<int, 1>{});
        else
            go(std::integral_constant<int, 2>{});
    });
}

} // namespace

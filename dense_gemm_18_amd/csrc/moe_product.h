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

struct MoeArgs {
    const uint16_t *X;             // T rows, ldx apart
    const uint16_t *router;        // E x H
    float *logits;                 // T x E
    int32_t *ids;                  // T x topk
    float *weights;                // T x topk
    WeightRef w13, w2;             // E * 2 * I rows of H, E * H rows of I
    uint16_t *h;                   // T * topk rows of I
    float *y;                      // T * topk rows of H
    uint16_t *D;                   // T rows, ldd apart
    int64_t ldx, ldd;
    int T, E, H, I, topk, renorm;
};

// One translation unit for each type.  Not exported from the library.
struct MoeLaunch {
    void (*route)(const MoeArgs &, hipStream_t);
    void (*experts)(const MoeArgs &, int group, hipStream_t);
};
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_f16();
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_bf16();

namespace {

// ---- router -------------------------------------------------------------

constexpr int kRouteWaves = 16;

// Logits of 16 experts for 16 tokens; sixteen waves split the hidden size.
template <bool BF>
using RouteCore = Skinny<BF, 0, 1, 1, kRouteWaves, 1, true>;

template <bool BF>
__global__ void __launch_bounds__(kRouteWaves * 64) moe_logits_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    RouteCore<BF> c;
    c.W.w = p.router;
    c.row[0] = e0;
    c.rows[0] = p.E - e0;
    c.K = p.H;
    c.M = min(16, p.T - t0);
    c.begin((char *)lds, p.X + t0 * p.ldx, (uint32_t)((c.M - 1) * p.ldx + p.H) * 2u);
    c.run([&](int m) { return (uint32_t)(m * p.ldx) * 2u; });
    c.join([&](int m, int n, const float(&v)[1]) {
        if (e0 + n < p.E)
            p.logits[(t0 + m) * p.E + e0 + n] = v[0];
    });
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

// The topk largest of E logits and their softmax weights, one wave per token.
// PER logits per lane (E <= 64 * PER).  A key is the order of the logit above
// the complement of its index, so keys differ, equal logits fall by rising
// index, and 0 marks what is taken: topk maxima over the wave.
template <int PER>
__device__ __forceinline__ void choose(const float *logits, int E, int topk, bool renorm,
                                       int32_t *ids, float *weights)
{
    const int lane = threadIdx.x & 63;
    float v[PER];
    uint64_t key[PER];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? logits[e] : -__builtin_inff();
        key[i] = e < E ? (uint64_t)order_of(v[i]) << 32 | (0xffffffffu - (uint32_t)e) : 0;
        top = __builtin_fmaxf(top, v[i]);      // a NaN shows in the sum below
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = __builtin_fmaxf(top, __shfl_xor(top, d));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        sum += lane + 64 * i < E ? expf(v[i] - top) : 0.0f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        sum += __shfl_xor(sum, d);

    float mine = 0.0f, chosen = 0.0f;
    int id = 0;
    for (int j = 0; j < topk; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            best = key[i] > best ? key[i] : best;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint64_t other = __shfl_xor((unsigned long long)best, d);
            best = other > best ? other : best;
        }
        const int e = (int)(0xffffffffu - (uint32_t)best);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] == best)
                key[i] = 0;
        const float p = expf(logits[e] - top);
        chosen += p;
        if (lane == j) {
            id = e;
            mine = p;
        }
    }
    const float over = renorm && sum == sum ? chosen : sum;
    if (lane < topk) {
        ids[lane] = id;
        weights[lane] = mine / over;
    }
}

template <int PER>
__global__ void __launch_bounds__(256) moe_choose_kernel(MoeArgs p)
{
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t < p.T)
        choose<PER>(p.logits + (int64_t)t * p.E, p.E, p.topk, p.renorm,
                    p.ids + (int64_t)t * p.topk, p.weights + (int64_t)t * p.topk);
}

// ---- experts ------------------------------------------------------------

constexpr int kMoeWaves = 8;

// Which slots (t * topk + j) go to which expert: the experts that have any,
// in rising order, and each one's slots side by side.  Every workgroup works
// it out for itself: at most 512 ids, read from L2.  The order of an
// expert's slots is that of the LDS atomics and changes no result: a slot is
// a row of its own in every product.
struct Plan {
    int *cnt;            // E: slots of an expert, then its cursor into `slot`
    int *off;            // active + 1
    uint16_t *act;       // active experts
    uint16_t *slot;      // slots, expert by expert
    int active;
};

__host__ __device__ inline int plan_bytes(int E, int n)
{
    const int a = E < n ? E : n;
    return (E * 4 + (a + 1) * 4 + a * 2 + n * 2 + 4 + 15) / 16 * 16;
}

__device__ __forceinline__ Plan make_plan(char *lds, const int32_t *ids, int n, int E)
{
    // (a short list could be compared pair by pair in registers: 0.5 us less)
    Plan pl;
    const int a = E < n ? E : n;
    pl.cnt = (int *)lds;
    pl.off = pl.cnt + E;
    int *active = pl.off + a + 1;
    pl.act = (uint16_t *)(active + 1);
    pl.slot = pl.act + a;
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        pl.cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if ((uint32_t)ids[i] < (uint32_t)E)
            atomicAdd(&pl.cnt[ids[i]], 1);
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int at = 0, base = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int c = e0 + lane < E ? pl.cnt[e0 + lane] : 0;
            int sum = c;                               // inclusive prefix sum
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int up = __shfl_up(sum, d);
                sum += lane >= d ? up : 0;
            }
            const uint64_t has = __ballot(c > 0);
            if (c > 0) {
                const int k = at + __popcll(has & ((1ull << lane) - 1));
                pl.act[k] = (uint16_t)(e0 + lane);
                pl.off[k] = base + sum - c;
                pl.cnt[e0 + lane] = base + sum - c;
            }
            at += __popcll(has);
            base += __shfl(sum, 63);
        }
        if (lane == 0) {
            pl.off[at] = base;
            *active = at;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if ((uint32_t)ids[i] < (uint32_t)E)
            pl.slot[atomicAdd(&pl.cnt[ids[i]], 1)] = (uint16_t)i;
    pl.active = uniform(*active);
    __syncthreads();
    return pl;
}

// Rows that run against one reading of an expert's weights, as the registers
// allow (packed weights need some for a group's sums).
template <int GS>
constexpr int kRowsAtOnce = GS ? 32 : 64;

// f(integral_constant<int, MB>): blocks of 16 rows for `count` of them.
template <int GS, class F>
__device__ __forceinline__ void with_blocks(int count, F &&f)
{
    if (count <= 16)
        f(std::integral_constant<int, 1>{});
    else if (GS != 0 || count <= 32)
        f(std::integral_constant<int, 2>{});
    else if constexpr (GS == 0)
        f(std::integral_constant<int, 4>{});
}

// Blocks of 16 hidden rows to a workgroup of the down product: its K, the inner
// size, is short, and four blocks of packed weights are the bytes of one of
// 16-bit ones.
template <int GS>
constexpr int kDownBlocks = GS ? 4 : 2;

template <bool BF, int GS, int MB>
using UpCore = Skinny<BF, GS, 2, MB, kMoeWaves, 1, false>;
template <bool BF, int GS, int MB>
using DownCore = Skinny<BF, GS, kDownBlocks<GS>, MB, kMoeWaves, 1, true>;

// h = silu(gate) * up for 16 of an expert's inner rows and all its slots.
// One workgroup takes the 16 gate rows and their 16 up rows, eight waves
// split the hidden size.
template <bool BF, int GS>
__global__ void __launch_bounds__(kMoeWaves * 64, 2) moe_up_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    const int n = p.T * p.topk, blocks = (p.I + 15) / 16;
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int s = wg / blocks, i0 = wg % blocks * 16;
    const Plan pl = make_plan((char *)lds, p.ids, n, p.E);
    if (s >= pl.active)
        return;
    char *smem = (char *)lds + plan_bytes(p.E, n);
    const int64_t e = uniform(pl.act[s]);
    const int end = uniform(pl.off[s + 1]);
    for (int c0 = uniform(pl.off[s]); c0 < end; c0 += kRowsAtOnce<GS>) {
        const int count = min(kRowsAtOnce<GS>, end - c0);
        with_blocks<GS>(count, [&](auto mbs) {
            UpCore<BF, GS, decltype(mbs)::value> c;
            c.W = p.w13;
            c.row[0] = e * 2 * p.I + i0;
            c.row[1] = c.row[0] + p.I;
            c.rows[0] = c.rows[1] = p.I - i0;
            c.K = p.H;
            c.M = count;
            c.begin(smem, p.X, (uint32_t)((p.T - 1) * p.ldx + p.H) * 2u);
            c.run([&](int m) {
                return (uint32_t)(pl.slot[c0 + m] / p.topk * p.ldx) * 2u;
            });
            c.join([&](int m, int i, const float(&v)[2]) {
                if (i0 + i < p.I) {
                    const float act = v[0] / (1.0f + expf(-v[0]));
                    p.h[(int64_t)pl.slot[c0 + m] * p.I + i0 + i] = from_float<BF>(act * v[1]);
                }
            });
        });
        __syncthreads();
    }
}

// y = W2 h for a block of an expert's hidden rows and all its slots, in fp32.
template <bool BF, int GS>
__global__ void __launch_bounds__(kMoeWaves * 64, 2) moe_down_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    constexpr int RB = kDownBlocks<GS>;
    const int n = p.T * p.topk, blocks = (p.H + 16 * RB - 1) / (16 * RB);
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int s = wg / blocks, h0 = wg % blocks * (16 * RB);
    const Plan pl = make_plan((char *)lds, p.ids, n, p.E);
    if (s >= pl.active)
        return;
    char *smem = (char *)lds + plan_bytes(p.E, n);
    const int64_t e = uniform(pl.act[s]);
    const int end = uniform(pl.off[s + 1]);
    for (int c0 = uniform(pl.off[s]); c0 < end; c0 += kRowsAtOnce<GS>) {
        const int count = min(kRowsAtOnce<GS>, end - c0);
        with_blocks<GS>(count, [&](auto mbs) {
            DownCore<BF, GS, decltype(mbs)::value> c;
            c.W = p.w2;
            c.row[0] = e * p.H + h0;
            c.rows[0] = p.H - h0;
            c.K = p.I;
            c.M = count;
            c.begin(smem, p.h, (uint32_t)n * (uint32_t)p.I * 2u);
            c.run([&](int m) { return (uint32_t)pl.slot[c0 + m] * (uint32_t)p.I * 2u; });
            c.join([&](int m, int i, const float(&v)[RB]) {
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    if (h0 + 16 * r + i < p.H)
                        p.y[(int64_t)pl.slot[c0 + m] * p.H + h0 + 16 * r + i] = v[r];
            });
        });
        __syncthreads();
    }
}

// The weighted sum over a token's slots, in order.
template <bool BF>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs p)
{
    const int t = blockIdx.y, h = blockIdx.x * 256 + threadIdx.x;
    if (h >= p.H)
        return;
    float sum = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const int slot = t * p.topk + j;
        if ((uint32_t)p.ids[slot] < (uint32_t)p.E)
            sum = __builtin_fmaf(p.weights[slot], p.y[(int64_t)slot * p.H + h], sum);
    }
    p.D[t * p.ldd + h] = from_float<BF>(sum);
}

template <bool BF>
void launch_route(const MoeArgs &p, hipStream_t stream)
{
    hipLaunchKernelGGL((moe_logits_kernel<BF>),
                       dim3((unsigned)cdiv(p.E, 16), (unsigned)cdiv(p.T, 16)),
                       dim3(kRouteWaves * 64), RouteCore<BF>::lds_bytes(p.T < 16 ? p.T : 16, p.H),
                       stream, p);
    const dim3 grid((unsigned)cdiv(p.T, 4));
    if (p.E <= 64)
        hipLaunchKernelGGL((moe_choose_kernel<1>), grid, dim3(256), 0, stream, p);
    else if (p.E <= 256)
        hipLaunchKernelGGL((moe_choose_kernel<4>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((moe_choose_kernel<16>), grid, dim3(256), 0, stream, p);
}

template <bool BF>
void launch_experts(const MoeArgs &p, int group, hipStream_t stream)
{
    const int n = p.T * p.topk, most = p.E < n ? p.E : n;
    const int plan = plan_bytes(p.E, n);
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value;
        const int rows = n < kRowsAtOnce<GS> ? n : kRowsAtOnce<GS>;
        const int up = plan + UpCore<BF, GS, 1>::lds_bytes(rows, p.H);
        const int down = plan + DownCore<BF, GS, 1>::lds_bytes(rows, p.I);
        hipLaunchKernelGGL((moe_up_kernel<BF, GS>), tile_grid(most * cdiv(p.I, 16)),
                           dim3(kMoeWaves * 64), up, stream, p);
        hipLaunchKernelGGL((moe_down_kernel<BF, GS>),
                           tile_grid(most * cdiv(p.H, 16 * kDownBlocks<GS>)),
                           dim3(kMoeWaves * 64), down, stream, p);
    });
    hipLaunchKernelGGL((moe_combine_kernel<BF>), dim3((unsigned)cdiv(p.H, 256), (unsigned)p.T),
                       dim3(256), 0, stream, p);
}

} // namespace

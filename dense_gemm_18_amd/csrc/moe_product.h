// moe_product.h -- kernels and launches of the mixture-of-experts layer,
// compiled once for each 16-bit type.
#pragma once

#include "skinny.h"

// Tokens of one pass through the kernels: 64, or as many as have 512 slots
// (t * topk + j), whose 16 columns of fp32 are what the down product keeps in
// LDS.
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
    uint16_t *D;                   // T rows, ldd apart
    int64_t ldx, ldd;
    int T, E, H, I, topk, renorm;
    int parts;                     // pieces of I in the down product
};

// One translation unit for each type.  Not exported from the library.
struct MoeLaunch {
    void (*route)(const MoeArgs &, hipStream_t);
    void (*experts)(const MoeArgs &, int group, hipStream_t);
};
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_f16();
__attribute__((visibility("hidden"))) MoeLaunch gemm18_moe_bf16();

namespace {

// A value that every lane of the wave has, as a scalar: branches on it are
// the wave's.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- router -------------------------------------------------------------

constexpr int kRouteWaves = 16;

// Logits of 16 experts for 16 tokens; sixteen waves split the hidden size.
template <bool BF>
__global__ void __launch_bounds__(kRouteWaves * 64) moe_logits_kernel(MoeArgs p)
{
    __shared__ f32x4 red[kRouteWaves * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    WeightRef W{};
    W.w = p.router;
    Skinny<BF, 0, 1, 1> c;
    c.init(p.H);
    c.bind(0, W, min(e0 + (lane & 15), p.E - 1));
    c.bind_act(0, p.X + (int64_t)min(t0 + (lane & 15), p.T - 1) * p.ldx);
    c.run(wave, (p.H + 127) >> 7, kRouteWaves);
    const f32x4 part[1] = {c.acc[0][0]};
    reduce_waves<1>(part, red, kRouteWaves, [&](int m, int n, const float(&v)[1]) {
        if (t0 + m < p.T && e0 + n < p.E)
            p.logits[(int64_t)(t0 + m) * p.E + e0 + n] = v[0];
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

// f(integral_constant<int, MB>): blocks of 16 rows for `count` of up to 64.
template <class F>
__device__ __forceinline__ void with_blocks(int count, F &&f)
{
    if (count <= 16)
        f(std::integral_constant<int, 1>{});
    else if (count <= 32)
        f(std::integral_constant<int, 2>{});
    else
        f(std::integral_constant<int, 4>{});
}

// h = silu(gate) * up for 16 of an expert's inner rows and all its slots.
// One workgroup takes the 16 gate rows and their 16 up rows, eight waves
// split the hidden size.
template <bool BF, int GS>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_up_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    f32x4 *red = lds;                                  // kMoeWaves * 2 * 64
    const int n = p.T * p.topk, blocks = (p.I + 15) / 16;
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int s = wg / blocks, i0 = wg % blocks * 16;
    const Plan pl = make_plan((char *)(lds + kMoeWaves * 2 * 64), p.ids, n, p.E);
    if (s >= pl.active)
        return;
    const int64_t e = uniform(pl.act[s]);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = e * 2 * p.I + min(i0 + (lane & 15), p.I - 1);
    const int end = uniform(pl.off[s + 1]);
    for (int c0 = uniform(pl.off[s]); c0 < end; c0 += 64) {
        const int count = min(64, end - c0);
        with_blocks(count, [&](auto mbs) {
            constexpr int MB = decltype(mbs)::value;
            Skinny<BF, GS, 2, MB> c;
            c.init(p.H);
            c.bind(0, p.w13, row);
            c.bind(1, p.w13, row + p.I);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int slot = pl.slot[c0 + min(16 * m + (lane & 15), count - 1)];
                c.bind_act(m, p.X + (int64_t)(slot / p.topk) * p.ldx);
            }
            c.run(wave, (p.H + 127) >> 7, kMoeWaves);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                const f32x4 part[2] = {c.acc[0][mb], c.acc[1][mb]};
                reduce_waves<2>(part, red, kMoeWaves, [&](int m, int i, const float(&v)[2]) {
                    if (16 * mb + m < count && i0 + i < p.I) {
                        const int64_t slot = pl.slot[c0 + 16 * mb + m];
                        const float act = v[0] / (1.0f + expf(-v[0]));
                        p.h[slot * p.I + i0 + i] = from_float<BF>(act * v[1]);
                    }
                });
            }
        });
    }
}

// 16 columns of y for every token: the waves share the (expert, piece of
// inner) pairs, each leaves its slots' sums in LDS at places of their own, and
// the weighted sum over a token's slots follows in order.
template <bool BF, int GS>
__global__ void __launch_bounds__(kMoeWaves * 64) moe_down_kernel(MoeArgs p)
{
    extern __shared__ f32x4 lds[];
    const int n = p.T * p.topk;
    float *y = (float *)lds;                           // parts * n * 16
    const int h0 = blockIdx.x * 16;
    const Plan pl = make_plan((char *)(y + p.parts * n * 16), p.ids, n, p.E);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int steps = (p.I + 127) >> 7;
    for (int u = wave; u < pl.active * p.parts; u += kMoeWaves) {
        const int s = u / p.parts, part = u % p.parts;
        const int64_t e = uniform(pl.act[s]);
        const int end = uniform(pl.off[s + 1]);
        for (int c0 = uniform(pl.off[s]); c0 < end; c0 += 64) {
            const int count = min(64, end - c0);
            with_blocks(count, [&](auto mbs) {
                constexpr int MB = decltype(mbs)::value;
                Skinny<BF, GS, 1, MB> c;
                c.init(p.I);
                c.bind(0, p.w2, e * p.H + min(h0 + (lane & 15), p.H - 1));
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    c.bind_act(m, p.h + (int64_t)pl.slot[c0 + min(16 * m + (lane & 15),
                                                                  count - 1)] * p.I);
                c.run(part * steps / p.parts, (part + 1) * steps / p.parts, 1);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = 16 * mb + 4 * (lane >> 4) + r;
                        if (m < count)
                            y[(part * n + pl.slot[c0 + m]) * 16 + (lane & 15)] = c.acc[0][mb][r];
                    }
            });
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * 16; i += blockDim.x) {
        const int t = i >> 4, col = i & 15;
        float sum = 0.0f;
        for (int j = 0; j < p.topk; ++j) {
            const int slot = t * p.topk + j;
            if ((uint32_t)p.ids[slot] < (uint32_t)p.E) {
                float v = 0.0f;
                for (int part = 0; part < p.parts; ++part)
                    v += y[(part * n + slot) * 16 + col];
                sum = __builtin_fmaf(p.weights[slot], v, sum);
            }
        }
        if (h0 + col < p.H)
            p.D[t * p.ldd + h0 + col] = from_float<BF>(sum);
    }
}

template <bool BF>
void launch_route(const MoeArgs &p, hipStream_t stream)
{
    hipLaunchKernelGGL((moe_logits_kernel<BF>),
                       dim3((unsigned)cdiv(p.E, 16), (unsigned)cdiv(p.T, 16)),
                       dim3(kRouteWaves * 64), 0, stream, p);
    const dim3 grid((unsigned)cdiv(p.T, 4));
    if (p.E <= 64)
        hipLaunchKernelGGL((moe_choose_kernel<1>), grid, dim3(256), 0, stream, p);
    else if (p.E <= 256)
        hipLaunchKernelGGL((moe_choose_kernel<4>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((moe_choose_kernel<16>), grid, dim3(256), 0, stream, p);
}

template <bool BF>
void launch_experts(const MoeArgs &args, int group, hipStream_t stream)
{
    MoeArgs p = args;
    const int n = p.T * p.topk, most = p.E < n ? p.E : n;
    // two pairs or more per wave where the experts alone give fewer
    p.parts = (int)cdiv(2 * kMoeWaves, most);
    if (p.parts > kMoeSlots / n)
        p.parts = kMoeSlots / n;
    const int plan = plan_bytes(p.E, n);
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value;
        hipLaunchKernelGGL((moe_up_kernel<BF, GS>), tile_grid(most * cdiv(p.I, 16)),
                           dim3(kMoeWaves * 64), kMoeWaves * 2 * 64 * 16 + plan, stream, p);
        hipLaunchKernelGGL((moe_down_kernel<BF, GS>), dim3((unsigned)cdiv(p.H, 16)),
                           dim3(kMoeWaves * 64), p.parts * n * 64 + plan, stream, p);
    });
}

} // namespace

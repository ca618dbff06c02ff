// w4_product.h -- kernel and launches of the 4-bit weight product, compiled
// once for each 16-bit type.
#pragma once

#include "skinny.h"

constexpr int kW4Waves = 8;

struct W4Args {
    const uint16_t *A;
    WeightRef W;
    uint16_t *D;
    int64_t lda, ldd;
    int M, N, K;
    int tiles_n;
    int64_t tiles;
};

// Launches of the product, one translation unit for each type.  Not exported
// from the library.
__attribute__((visibility("hidden"))) void gemm18_w4_f16(const W4Args &a, int group,
                                                         hipStream_t stream);
__attribute__((visibility("hidden"))) void gemm18_w4_bf16(const W4Args &a, int group,
                                                          hipStream_t stream);

namespace {

// One workgroup: 16 * RB columns n and 16 * MB rows m of D, its eight waves
// taking the 128-wide steps of K in turn (so that together they read whole
// lines of a weight row) and their sums joined in LDS.
template <bool BF, int GS, int RB, int MB>
__global__ void __launch_bounds__(kW4Waves * 64) gemm_w4_kernel(W4Args p)
{
    __shared__ f32x4 red[kW4Waves * RB * 64];
    const int64_t tile = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    if (tile >= p.tiles)
        return;
    const int64_t n0 = tile % p.tiles_n * (16 * RB), m0 = tile / p.tiles_n * (16 * MB);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

    Skinny<BF, GS, RB, MB> c;
    c.init(p.K);
    // rows past the end repeat the last one; their results are not stored
#pragma unroll
    for (int r = 0; r < RB; ++r)
        c.bind(r, p.W, min(n0 + 16 * r + (lane & 15), (int64_t)p.N - 1));
#pragma unroll
    for (int m = 0; m < MB; ++m)
        c.bind_act(m, p.A + min(m0 + 16 * m + (lane & 15), (int64_t)p.M - 1) * p.lda);
    c.run(wave, (p.K + 127) >> 7, kW4Waves);

#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        f32x4 part[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r)
            part[r] = c.acc[r][mb];
        reduce_waves<RB>(part, red, kW4Waves, [&](int m, int n, const float(&v)[RB]) {
            const int64_t mm = m0 + 16 * mb + m;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int64_t nn = n0 + 16 * r + n;
                if (mm < p.M && nn < p.N)
                    p.D[mm * p.ldd + nn] = from_float<BF>(v[r]);
            }
        });
    }
}

template <bool BF, int GS, int RB, int MB>
void launch_w4_tile(W4Args a, hipStream_t stream)
{
    a.tiles_n = (int)cdiv(a.N, 16 * RB);
    a.tiles = a.tiles_n * cdiv(a.M, 16 * MB);
    hipLaunchKernelGGL((gemm_w4_kernel<BF, GS, RB, MB>), tile_grid(a.tiles), dim3(kW4Waves * 64),
                       0, stream, a);
}

template <bool BF>
void launch_w4(const W4Args &a, int group, hipStream_t stream)
{
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value ? decltype(gs)::value : 128;
        if (a.M <= 16)
            launch_w4_tile<BF, GS, 1, 1>(a, stream);
        else if (a.M <= 32)
            launch_w4_tile<BF, GS, 2, 2>(a, stream);
        else
            launch_w4_tile<BF, GS, 2, 4>(a, stream);
    });
}

} // namespace

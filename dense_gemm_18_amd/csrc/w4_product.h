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
    uint32_t tiles_m, tiles_n;
};

// Launches of the product, one translation unit for each type.  Not exported
// from the library.
__attribute__((visibility("hidden"))) void gemm18_w4_f16(const W4Args &a, int group,
                                                         hipStream_t stream);
__attribute__((visibility("hidden"))) void gemm18_w4_bf16(const W4Args &a, int group,
                                                          hipStream_t stream);

namespace {

// One workgroup: 16 * RB * NW columns n and 16 * MB rows m of D.
template <bool BF, int GS, int RB, int MB, int NW>
__global__ void __launch_bounds__(kW4Waves * 64, 2) gemm_w4_kernel(W4Args p)
{
    extern __shared__ f32x4 lds[];
    using Core = Skinny<BF, GS, RB, MB, kW4Waves / NW, NW, true>;
    // a grid of 2^32 work-items or more has a second dimension
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const uint32_t tn = wg % p.tiles_n, tm = wg / p.tiles_n;
    if (tm >= p.tiles_m)
        return;
    const int n0 = tn * Core::kRows, m0 = tm * (16 * MB);
    Core c;
    c.W = p.W;
    c.row[0] = n0;
    c.rows[0] = p.N - n0;
    c.K = p.K;
    c.M = min(16 * MB, p.M - m0);
    c.begin((char *)lds, p.A + (int64_t)m0 * p.lda,
            (uint32_t)((c.M - 1) * p.lda + p.K) * 2u);
    c.run([&](int m) { return (uint32_t)(m * p.lda) * 2u; });
    uint16_t *D = p.D + (int64_t)m0 * p.ldd + n0;
    c.join([&](int m, int n, const float(&v)[RB]) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int nn = (n >> 4) * (16 * RB) + 16 * r + (n & 15);
            if (n0 + nn < p.N)
                D[m * p.ldd + nn] = from_float<BF>(v[r]);
        }
    });
}

template <bool BF, int GS, int RB, int MB, int NW>
void launch_w4_tile(W4Args a, hipStream_t stream)
{
    using Core = Skinny<BF, GS, RB, MB, kW4Waves / NW, NW, true>;
    a.tiles_n = (uint32_t)cdiv(a.N, Core::kRows);
    a.tiles_m = (uint32_t)cdiv(a.M, 16 * MB);
    const int rows = a.M < 16 * MB ? a.M : 16 * MB;
    hipLaunchKernelGGL((gemm_w4_kernel<BF, GS, RB, MB, NW>),
                       tile_grid((int64_t)a.tiles_n * a.tiles_m), dim3(kW4Waves * 64),
                       Core::lds_bytes(rows, a.K), stream, a);
}

template <bool BF>
void launch_w4(const W4Args &a, int group, hipStream_t stream)
{
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value ? decltype(gs)::value : 128;
        if (a.M <= 16 && a.N >= 64 * kCUs)
            launch_w4_tile<BF, GS, 4, 1, 1>(a, stream);
        else if (a.M <= 16 && a.N >= 32 * kCUs)
            launch_w4_tile<BF, GS, 2, 1, 1>(a, stream);
        else if (a.M <= 16)
            launch_w4_tile<BF, GS, 1, 1, 1>(a, stream);
        else if (a.M <= 32)
            launch_w4_tile<BF, GS, 2, 2, 1>(a, stream);
        else
            launch_w4_tile<BF, GS, 2, 4, 2>(a, stream);
    });
}

} // namespace

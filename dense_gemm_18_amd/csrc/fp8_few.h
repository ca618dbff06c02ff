// fp8_few.h -- the FP8 product of few rows: kernel and launch, on the core of skinny.h.
#pragma once

#include "skinny.h"

struct Fp8FewArgs {
    const uint16_t *A, *B;         // rows of K pairs of FP8 bytes
    uint16_t *D;
    const float *row, *col;        // M and N scales, or null
    float scale;
    int M, N, K, bf;
    uint32_t tiles_m, tiles_n;
};

namespace {

// One workgroup's tile of D, 16 * MB rows and as many columns as Core has weight rows.
template <int MB, class Core>
__global__ void __launch_bounds__(Core::kThreads, 2) gemm_fp8_few_kernel(Fp8FewArgs p)
{
    extern __shared__ f32x4 lds[];
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const uint32_t tn = wg / p.tiles_m, tm = wg % p.tiles_m;
    if (tn >= p.tiles_n)
        return;
    const int n0 = tn * Core::kRows, m0 = tm * (16 * MB);
    Core c;
    c.W.w = p.B;
    c.row[0] = n0;
    c.rows[0] = p.N - n0;
    c.K = p.K;
    c.M = min(16 * MB, p.M - m0);
    c.begin((char *)lds, p.A + (int64_t)m0 * p.K, (uint32_t)c.M * (uint32_t)p.K * 2u);
    c.run([&](int m) { return (uint32_t)m * (uint32_t)p.K * 2u; });
    c.join([&](int m, int n, const auto &v) {
        constexpr int RB = sizeof(v) / sizeof(v[0]);
        m += m0;
        const float row = p.row ? p.row[m] : 1.0f;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int nn = n0 + (n >> 4) * (16 * RB) + 16 * r + (n & 15);
            if (nn < p.N) {
                const float d = v[r] * (p.col ? p.scale * p.col[nn] : p.scale) * row;
                p.D[(int64_t)m * p.N + nn] = p.bf ? from_float<true>(d) : from_float<false>(d);
            }
        }
    });
}

template <int F8, int RB, int MB, int KW, int NW>
void launch_few_tile(Fp8FewArgs a, hipStream_t stream)
{
    using Core = Skinny<false, 0, RB, MB, KW, NW, true, F8>;
    a.tiles_n = (uint32_t)cdiv(a.N, Core::kRows);
    a.tiles_m = (uint32_t)cdiv(a.M, 16 * MB);
    hipLaunchKernelGGL((gemm_fp8_few_kernel<MB, Core>),
                       tile_grid((int64_t)a.tiles_n * a.tiles_m), dim3(Core::kThreads),
                       Core::lds_bytes(a.M < 16 * MB ? a.M : 16 * MB, a.K), stream, a);
}

// Which tile serves a product of M x N x K bytes best, if it is one of these: rows x
// columns of 0 leave it to the tiles of gemm_kernels.h, which give a compute unit 64 x 64.
// Where those are few, smaller ones let every unit read.  Operands at multiples of 4 bytes
// only: at others a load of 16 takes several times as long.  Measured in us, weights out of
// the last-level cache, 64 x 64 (from 65 rows on 128 x 128) / the tile taken:
//   1 x 4096 x 4096     10.1 /  6.2 (16 x 16)     16 x 4096 x 8192    17.1 / 11.6
//   8 x 16384 x 4096    15.8 / 13.6 (16 x 32)     1 x 16384 x 8192    26.9 / 23.7
//   32 x 4096 x 4096    11.4 / 10.8 (32 x 16)     64 x 2048 x 4096    12.2 /  8.8
//   128 x 1024 x 4096   15.4 /  9.0               256 x 1024 x 8192   25.4 / 20.0 (32 x 32)
// and where another is better: 16 x 16384 x 8192, whose activations pass the LDS, 27.1 / 36.3
// (16 x 32); 32 x 8192 x 4096 12.0 / 13.1 (32 x 32); 64 x 4096 x 4096 12.9 / 15.9 (32 x 32).
struct FewTile {
    int rows, columns;
};
inline FewTile few_tile(const void *A, const void *B, int64_t M, int64_t N, int64_t K)
{
    if (K % 4 != 0 || !aligned_to(A, 4) || !aligned_to(B, 4))
        return {0, 0};
    if (M <= 16) {
        const bool whole = M * (cdiv(K, 256) * 256 + 16) <= kActBytes;
        if (N <= 16 * kCUs || (N <= 32 * kCUs && !whole))
            return {16, 16};
        return whole ? FewTile{16, 32} : FewTile{0, 0};
    }
    if (cdiv(M, 32) * cdiv(N, 16) <= kCUs)
        return {32, 16};
    if (M > 64 && cdiv(M, 32) * cdiv(N, 32) <= kCUs)
        return {32, 32};
    return {0, 0};
}

template <int F8>
void launch_few(const Fp8FewArgs &a, FewTile t, hipStream_t stream)
{
    if (t.rows == 16 && t.columns == 16)
        launch_few_tile<F8, 1, 1, 8, 1>(a, stream);
    else if (t.rows == 16)
        launch_few_tile<F8, 1, 1, 4, 2>(a, stream);
    else if (t.columns == 16)
        launch_few_tile<F8, 1, 2, 8, 1>(a, stream);
    else
        launch_few_tile<F8, 2, 2, 8, 1>(a, stream);
}

} // namespace

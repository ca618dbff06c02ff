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

// What a kernel adds to a tile's sums before they are rounded: nothing.  Others have
// `lds_at`, where their part of the LDS begins, bytes(rows) of it, first(), what a thread
// loads before the product, stage(), which every thread calls with that after it, and at(),
// the addend of the tile's row m in column n.
struct NoPlus {
    static constexpr bool kNone = true;
    int bytes(int) const { return 0; }
    __device__ __forceinline__ NoPlus first(int, int) const { return {}; }
};

// One workgroup's tile of D, 16 * MB rows and as many columns as Core has
// weight rows.  Few rows are bound by reading the weights: 1 x 16384 x 8192 with
// zero points, 70 MB, takes 15.4 us in fp16 (4.5 TB/s; 14 us from HBM and 10 from
// the last-level cache for the reading alone) and 17.8 in bfloat16, whose
// unpacking takes the VALU for 63 % of the time; the launch, the first loads and
// the join are 4 of it, all that 1 x 1024 x 1024 has.
template <bool BF, int MB, class Core, class Plus = NoPlus>
__global__ void __launch_bounds__(Core::kThreads, 2) gemm_w4_kernel(W4Args p, Plus plus)
{
    extern __shared__ f32x4 lds[];
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
    const auto held = plus.first(m0, c.M);
    c.begin((char *)lds, p.A + (int64_t)m0 * p.lda,
            (uint32_t)((c.M - 1) * p.lda + p.K) * 2u);
    c.run([&](int m) { return (uint32_t)(m * p.lda) * 2u; });
    if constexpr (!Plus::kNone)
        plus.stage((char *)lds, m0, c.M, held);
    uint16_t *D = p.D + (int64_t)m0 * p.ldd + n0;
    c.join([&](int m, int n, const auto &v) {
        constexpr int RB = sizeof(v) / sizeof(v[0]);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int nn = (n >> 4) * (16 * RB) + 16 * r + (n & 15);
            if (n0 + nn < p.N) {
                float d = v[r];
                if constexpr (!Plus::kNone)
                    d += plus.template at<BF>((const char *)lds, m, n0 + nn);
                D[m * p.ldd + nn] = from_float<BF>(d);
            }
        }
    });
}

template <bool BF, int MB, class Core, class Plus>
void launch_w4_tile(W4Args a, int lds, hipStream_t stream, Plus plus)
{
    if constexpr (!Plus::kNone) {
        plus.lds_at = lds;
        lds += plus.bytes(a.M < 16 * MB ? a.M : 16 * MB);
    }
    a.tiles_n = (uint32_t)cdiv(a.N, Core::kRows);
    a.tiles_m = (uint32_t)cdiv(a.M, 16 * MB);
    hipLaunchKernelGGL((gemm_w4_kernel<BF, MB, Core, Plus>),
                       tile_grid((int64_t)a.tiles_n * a.tiles_m), dim3(Core::kThreads), lds,
                       stream, a, plus);
}

// Activations that LDS holds whole: every wave walks its eighth of K freely.
template <bool BF, int GS, int RB, class Plus>
void launch_w4_resident(const W4Args &a, hipStream_t stream, const Plus &plus)
{
    using Core = Skinny<BF, GS, RB, 1, kW4Waves, 1, true>;
    launch_w4_tile<BF, 1, Core>(a, Core::lds_bytes(a.M, a.K), stream, plus);
}

template <bool BF, int GS, int RB, int MB, int KW, int NW, int CS, class Plus>
void launch_w4_piped(const W4Args &a, hipStream_t stream, const Plus &plus)
{
    using Core = Piped<BF, GS, RB, MB, KW, NW, CS>;
    launch_w4_tile<BF, MB, Core>(a, Core::kLds, stream, plus);
}

// Resident: activations within kActBytes, where no wave waits for another until
// the end.  Otherwise the chunked core.  A tile's time hardly depends on how
// many compute units have one, and larger tiles read the activations less
// often: so each takes the largest tile that gives every compute unit one, and
// the smallest if none does.  Measured at K = 8192, fp16, in us, by columns:
//                         16384    8192    4096    1024
//   16 rows, 16 x 64       17.5    15.4    15.0    13.4
//            16 x 32       20.5    12.5    11.4    10.2
//            16 x 16       26.5    14.9     9.6     8.1
//   32 rows, 32 x 64       21.4    19.4    18.7
//            32 x 32       25.3    17.8    14.9
//   64 rows, 64 x 64       31.8    29.7    28.1    27.4
//            32 x 64       35.1    21.6    19.5    17.9
//            32 x 32       47.2    25.6    15.8    13.9
// Of the 16 x 64 tile the chunked form has 16 waves and a compute unit to itself,
// the resident one 8 waves and, with up to 80 KB of LDS, another beside it.  The
// latter wins where there are more tiles than compute units and its scales, which
// all have to be there before it starts, are few (64 groups).  Time of the chunked
// form over the resident one's, one row, fp16 (bf16 is within 0.05 of it but for
// groups of 64 at K = 8192, 0.91 to 0.96):
//   K                     512   1024   2048   4096   8192  16384
//   16384 columns, 256 tiles, one to a compute unit
//     groups of 128      0.94   0.99   0.89   0.84   0.89   0.88
//                32      1.00   0.96   0.91   0.70   0.65   0.61
//   18000 to 65536 columns
//     groups of 128      1.16+  1.19+  1.09+  1.04+  1.05+  0.89-0.96
//                64      1.18+  1.18+  1.05+  1.02+  0.88-0.95  0.71+
//                32      1.26+  1.20+  1.12+  0.83-0.91  0.62+  0.56+
//   four rows, for which K = 8192 takes 82 KB and more
//     groups of 128      1.16+  1.19+  1.08+  1.01+  0.85-0.90
// most: rows that a tile may have (16, 32 or 64).
template <bool BF, class Plus = NoPlus>
void launch_w4(const W4Args &a, int group, hipStream_t stream, const Plus &plus = Plus{},
               int most = 64)
{
    const auto fills = [&](int rows, int columns) {
        return cdiv(a.M, rows) * cdiv(a.N, columns) >= kCUs;
    };
    with_group(group, [&](auto gs) {
        constexpr int GS = decltype(gs)::value ? decltype(gs)::value : 128;
        const bool whole =
            a.M <= 16 && (int64_t)a.M * (cdiv(a.K, 128) * 256 + 16) <= kActBytes;
        const int beside = Skinny<BF, GS, 4, 1, kW4Waves, 1, true>::lds_bytes(a.M, a.K);
        if (whole && cdiv(a.N, 64) > kCUs && cdiv(a.K, GS) <= 64 && beside <= 80 * 1024) {
            launch_w4_resident<BF, GS, 4>(a, stream, plus);
        } else if (whole && !fills(16, 64)) {
            if (fills(16, 32))
                launch_w4_resident<BF, GS, 2>(a, stream, plus);
            else
                launch_w4_resident<BF, GS, 1>(a, stream, plus);
        } else if (a.M <= 16 && fills(16, 64)) {
            launch_w4_piped<BF, GS, 2, 1, 8, 2, 8>(a, stream, plus);
        } else if (a.M <= 16 && fills(16, 32)) {
            launch_w4_piped<BF, GS, 2, 1, 8, 1, 8>(a, stream, plus);
        } else if (a.M > 32 && most >= 64 && fills(64, 64)) {
            launch_w4_piped<BF, GS, 2, 4, 4, 2, 4>(a, stream, plus);
        } else if (a.M > 16 && most >= 32 && fills(32, 64)) {
            launch_w4_piped<BF, GS, 2, 2, 4, 2, 4>(a, stream, plus);
        } else if (a.M > 16 && most >= 32 && fills(32, 32)) {
            launch_w4_piped<BF, GS, 1, 2, 4, 2, 4>(a, stream, plus);
        } else {
            launch_w4_piped<BF, GS, 1, 1, 8, 1, 8>(a, stream, plus);
        }
    });
}

} // namespace

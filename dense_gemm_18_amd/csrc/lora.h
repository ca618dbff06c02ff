// lora.h -- kernels and launches of the low-rank adapters beside a shared projection,
// compiled once for each 16-bit type.
#pragma once

#include "lora_nt.h"
#include "w4_product.h"

// Rows of a tile of the first product.
constexpr int kLoraRows = 32;
// Values of u that a tile of the projection holds in LDS: its rows times the rank.
constexpr int kLoraHeld = 4096;

struct LoraArgs {
    const uint16_t *X, *A, *B;
    const float *s;                // null: 1
    const int32_t *ids;
    float *u;                      // parts x M x rank, scaled; rows without an adapter unset
    uint16_t *D;
    int64_t ldx;
    int M, N, K, rank, count, parts;
    int items, rblocks;            // of a tile: adapters at most, blocks of their rows
};

// Pieces of K in the first product, and with them of u: as many as give each compute unit
// two workgroups, of 512 elements or more.
inline int lora_parts(int64_t M, int64_t K)
{
    const int64_t tiles = cdiv(M, kLoraRows);
    int64_t p = 2 * kCUs / tiles;
    p = p > 8 ? 8 : p < 1 ? 1 : p;
    return (int)(p < cdiv(K, 512) ? p : cdiv(K, 512));
}

// One translation unit for each type.  Not exported from the library.
struct LoraLaunch {
    // u
    void (*shrink)(LoraArgs, hipStream_t);
    // D from the weight's tiles with the adapters' part added, for a group or 16-bit weights
    void (*fused)(const LoraArgs &, const W4Args &, int group, hipStream_t);
    // the adapters' part alone into dense rows of D
    void (*expand)(const LoraArgs &, hipStream_t);
};
__attribute__((visibility("hidden"))) LoraLaunch gemm18_lora_f16();
__attribute__((visibility("hidden"))) LoraLaunch gemm18_lora_bf16();

namespace {

// 16 bytes at any 2-byte alignment (one global load).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// The first `count` of the 8 elements at p, zero for the others; nothing past them is
// accessed.
__device__ __forceinline__ u32x4 eight_of(const uint16_t *p, int count)
{
    if (count >= 8)
        return *(const u32x4_any *)p;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < count)
            v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
}

__device__ __forceinline__ int adapter_of(const LoraArgs &p, int64_t m)
{
    const int id = m < p.M ? p.ids[m] : -1;
    return (uint32_t)id < (uint32_t)p.count ? id : -1;
}

// The rows of a tile, one to a lane, that have the `item`-th of the tile's adapters (by
// their first rows); 0 if there are fewer.
__device__ __forceinline__ uint64_t rows_of(int id, int item)
{
    uint64_t left = __ballot(id >= 0);
    while (left) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __ballot(id == a);
        if (item-- == 0)
            return same;
        left &= ~same;
    }
    return 0;
}

// u of one adapter's rows in a tile, for 16 * RB of its rank and one piece of K, on the
// core of skinny.h with A's rows as the weight: each workgroup looks for its item among the
// tile's ids and gathers its rows, so an adapter is read once for the rows that have it and
// no row is multiplied with another's.
template <bool BF, int RB, int MB>
__device__ __forceinline__ void lora_item(const LoraArgs &p, char *lds, const int *list, int rows,
                                          int64_t m0, int a, int rb, int part)
{
    const int steps = (p.K + 127) >> 7;
    const int k0 = part * steps / p.parts * 128;
    Skinny<BF, 0, RB, MB, 8, 1, true> c;
    c.W.w = p.A + k0;
    c.row[0] = (int64_t)a * p.rank + rb * (16 * RB);
    c.rows[0] = p.rank - rb * (16 * RB);
    c.stride = p.K;
    c.K = min((part + 1) * steps / p.parts * 128, p.K) - k0;
    c.M = rows;
    c.begin(lds, p.X + m0 * p.ldx + k0,
            (uint32_t)((min((int64_t)kLoraRows, p.M - m0) - 1) * p.ldx + c.K) * 2u);
    c.run([&](int m) { return (uint32_t)(list[m] * p.ldx) * 2u; });
    const float s = p.s ? p.s[a] : 1.0f;
    float *u = p.u + ((int64_t)part * p.M + m0) * p.rank + rb * (16 * RB);
    c.join([&](int m, int n, const float(&v)[RB]) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (rb * (16 * RB) + 16 * r + n < p.rank)
                u[(int64_t)list[m] * p.rank + 16 * r + n] = v[r] * s;
    });
}

template <bool BF, int RB>
__global__ void __launch_bounds__(512, 2) lora_shrink_kernel(LoraArgs p)
{
    extern __shared__ f32x4 lds[];
    __shared__ int list[kLoraRows];
    int64_t wg = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int part = (int)(wg % p.parts);
    wg /= p.parts;
    const int rb = (int)(wg % p.rblocks);
    wg /= p.rblocks;
    const int item = (int)(wg % p.items);
    const int64_t m0 = wg / p.items * kLoraRows;
    if (m0 >= p.M)
        return;
    const int lane = threadIdx.x & 63;
    const int id = lane < kLoraRows ? adapter_of(p, m0 + lane) : -1;
    const uint64_t mask = rows_of(id, item);
    if (!mask)
        return;
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(mask));
    if (threadIdx.x < 64 && (mask >> lane & 1))
        list[__popcll(mask & ((1ull << lane) - 1))] = lane;
    __syncthreads();
    const int rows = __popcll(mask);
    if (rows <= 16)
        lora_item<BF, RB, 1>(p, (char *)lds, list, rows, m0, a, rb, part);
    else
        lora_item<BF, RB, 2>(p, (char *)lds, list, rows, m0, a, rb, part);
}

template <bool BF, int RB>
void launch_shrink(LoraArgs p, hipStream_t stream)
{
    p.rblocks = (int)cdiv(p.rank, 16 * RB);
    const int rows = p.M < kLoraRows ? p.M : kLoraRows;
    const int k = (int)cdiv(cdiv(p.K, 128), p.parts) * 128;
    const int one = Skinny<BF, 0, RB, 1, 8, 1, true>::lds_bytes(rows < 16 ? rows : 16, k);
    const int two = Skinny<BF, 0, RB, 2, 8, 1, true>::lds_bytes(rows, k);
    hipLaunchKernelGGL((lora_shrink_kernel<BF, RB>),
                       tile_grid(cdiv(p.M, kLoraRows) * p.items * p.rblocks * p.parts), dim3(512),
                       one > two ? one : two, stream, p);
}

// As many of an adapter's rows to a workgroup as there are, where the tiles alone fill
// the compute units; else 16, for more workgroups.
template <bool BF>
void lora_shrink(LoraArgs p, hipStream_t stream)
{
    p.items = p.count < kLoraRows ? p.count : kLoraRows;
    p.items = p.items < p.M ? p.items : p.M;
    const bool many = cdiv(p.M, kLoraRows) * p.parts >= kCUs;
    if (p.rank <= 16 || !many)
        launch_shrink<BF, 1>(p, stream);
    else if (p.rank <= 32)
        launch_shrink<BF, 2>(p, stream);
    else
        launch_shrink<BF, 4>(p, stream);
}

// ---- beside the projection's tiles ---------------------------------------

// The addend of a tile: u of its rows and their adapters wait in LDS, an output reads its
// row of B.
struct LoraPlus {
    static constexpr bool kNone = false;
    const float *u;
    const uint16_t *B;
    const int32_t *ids;
    int M, N, rank, count, parts;
    int lds_at;

    __host__ __device__ int stride() const { return (rank + 7) & ~7; }
    int bytes(int rows) const { return rows * (stride() + 4) * 4; }

    // Row m's adapter is the word before its u.
    __device__ __forceinline__ void stage(char *lds, int m0, int rows) const
    {
        const int ld = stride() + 4;
        float *to = (float *)(lds + lds_at);
        for (int i = threadIdx.x; i < rows * ld; i += blockDim.x) {
            const int m = i / ld, j = i - m * ld - 4;
            const int id = ids[m0 + m];
            const bool in = (uint32_t)id < (uint32_t)count;
            float v = 0.0f;
            if (j < 0)
                v = __builtin_bit_cast(float, in ? id : -1);
            else if (in && j < rank)
                for (int q = 0; q < parts; ++q)
                    v += u[((int64_t)q * M + m0 + m) * rank + j];
            to[i] = v;
        }
    }

    template <bool BF>
    __device__ __forceinline__ float at(const char *lds, int m, int n) const
    {
        const float *from = (const float *)(lds + lds_at) + m * (stride() + 4);
        const int a = __builtin_bit_cast(int, from[3]);
        if (a < 0)
            return 0.0f;
        const uint16_t *b = B + ((int64_t)a * N + n) * rank;
        float sum = 0.0f;
        for (int j = 0; j < rank; j += 8) {
            const u32x4 v = eight_of(b + j, rank - j);
            const f32x4 x = *(const f32x4 *)(from + 4 + j), y = *(const f32x4 *)(from + 8 + j);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(e < 4 ? x[e & 3] : y[e & 3],
                                     to_float<BF>((uint16_t)(v[e >> 1] >> (16 * (e & 1)))), sum);
        }
        return sum;
    }
};

template <bool BF, int RB, int MB, int KW, int NW>
void launch_lora_dense(const W4Args &w, const LoraPlus &plus, hipStream_t stream)
{
    using Core = Skinny<BF, 0, RB, MB, KW, NW, true>;
    launch_w4_tile<BF, MB, Core>(w, Core::lds_bytes(w.M < 16 * MB ? w.M : 16 * MB, w.K), stream,
                                 plus);
}

template <bool BF>
void lora_fused(const LoraArgs &p, const W4Args &w, int group, hipStream_t stream)
{
    LoraPlus plus{p.u, p.B, p.ids, p.M, p.N, p.rank, p.count, p.parts, 0};
    const int held = kLoraHeld / plus.stride();
    const int most = held >= 64 ? 64 : held >= 32 ? 32 : 16;
    if (group) {
        launch_w4<BF>(w, group, stream, plus, most);
        return;
    }
    if (p.M <= 16 || most < 32) {
        if (p.N <= 16 * kCUs)
            launch_lora_dense<BF, 1, 1, 8, 1>(w, plus, stream);
        else
            launch_lora_dense<BF, 1, 1, 4, 2>(w, plus, stream);
    } else if (cdiv(p.M, 32) * cdiv(p.N, 16) <= kCUs) {
        launch_lora_dense<BF, 1, 2, 8, 1>(w, plus, stream);
    } else {
        launch_lora_dense<BF, 2, 2, 8, 1>(w, plus, stream);
    }
}

// ---- the adapters' part alone --------------------------------------------

constexpr int kExpandColumns = 512;

// 64 rows of the adapters' part, kExpandColumns columns of it.  u, summed and rounded to the
// 16-bit type (each row times a power of two that leaves its largest near 1, taken off
// afterwards), is in LDS; for each adapter of the tile every row is multiplied with its B
// and only the rows that have it are stored: what is infinite in one adapter stays out of
// the others' rows.
template <bool BF>
__global__ void __launch_bounds__(256) lora_expand_kernel(LoraArgs p)
{
    using x8 = typename Elem<BF>::x8;
    extern __shared__ f32x4 lds[];
    __shared__ float unscale[64];
    const int columns = (p.N + kExpandColumns - 1) / kExpandColumns;
    const uint32_t wg = blockIdx.x + blockIdx.y * gridDim.x;
    const int64_t m0 = (int64_t)(wg / columns) * 64;
    if (m0 >= p.M)
        return;
    const int n0 = (int)(wg % columns) * kExpandColumns;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int id = adapter_of(p, m0 + lane);
    const int ks = (p.rank + 31) / 32, ld = ks * 32 + 8;       // 16-bit elements of a row
    uint16_t *held = (uint16_t *)lds;
    for (int m = wave; m < 64; m += 4) {
        const bool in = __builtin_amdgcn_readlane(id, m) >= 0;
        float v[LORA_MAX_RANK / 64], most = 0.0f;
#pragma unroll
        for (int i = 0; i < LORA_MAX_RANK / 64; ++i) {
            const int j = lane + 64 * i;
            v[i] = 0.0f;
            if (in && j < p.rank)
                for (int q = 0; q < p.parts; ++q)
                    v[i] += p.u[((int64_t)q * p.M + m0 + m) * p.rank + j];
            most = __builtin_fmaxf(most, __builtin_fabsf(v[i]));
        }
#pragma unroll
        for (int d = 32; d; d /= 2)
            most = __builtin_fmaxf(most, __shfl_xor(most, d));
        // 2^e <= most < 2^(e + 1); what is 0 or not finite stays as it is
        int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
        e = e == 128 || most == 0.0f ? 0 : e < -126 ? -126 : e;
        if (lane == 0)
            unscale[m] = __builtin_ldexpf(1.0f, e);
#pragma unroll
        for (int i = 0; i < LORA_MAX_RANK / 64; ++i)
            if (lane + 64 * i < ks * 32)
                held[m * ld + lane + 64 * i] = from_float<BF>(__builtin_ldexpf(v[i], -e));
    }
    __syncthreads();
    const int c = lane >> 4, col = lane & 15;
    const bool whole = p.N % 4 == 0 && ((uintptr_t)p.D & 7) == 0;
    auto store = [&](int m, int n, const f32x4 &v) G18_INLINE {
        uint16_t *to = p.D + (m0 + m) * (int64_t)p.N + n;
        if (whole) {
            if (n < p.N)
                *(u32x2 *)to = u32x2{from_float<BF>(v[0]) | (uint32_t)from_float<BF>(v[1]) << 16,
                                     from_float<BF>(v[2]) | (uint32_t)from_float<BF>(v[3]) << 16};
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.N)
                    to[r] = from_float<BF>(v[r]);
        }
    };
    int row[4];                    // the adapters of this lane's rows; -2: past the end
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        row[b] = __shfl(id, 16 * b + col);
        row[b] = m0 + 16 * b + col < p.M ? row[b] : -2;
    }
    uint64_t left = __ballot(id >= 0);
    const bool bare = __ballot(id < 0 && m0 + lane < p.M) != 0;
    for (int nb = wave * 16; nb < kExpandColumns && n0 + nb < p.N; nb += 64) {
        const int n = n0 + nb;
        if (bare) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (row[b] == -1)
                    store(16 * b + col, n + 4 * c, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        }
        for (uint64_t rest = left; rest;) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(rest));
            rest &= ~__ballot(id == a);
            const uint16_t *B = p.B + ((int64_t)a * p.N + min(n + col, p.N - 1)) * p.rank;
            f32x4 acc[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < ks; ++k) {
                const x8 w = __builtin_bit_cast(x8, eight_of(B + k * 32 + 8 * c,
                                                            p.rank - k * 32 - 8 * c));
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    acc[b] = mfma16<BF>(
                        w, *(const x8 *)(held + (16 * b + col) * ld + k * 32 + 8 * c), acc[b]);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (row[b] == a)
                    store(16 * b + col, n + 4 * c, acc[b] * unscale[16 * b + col]);
        }
    }
}

template <bool BF>
void lora_expand(const LoraArgs &p, hipStream_t stream)
{
    const int lds = 64 * ((int)cdiv(p.rank, 32) * 32 + 8) * 2;
    hipLaunchKernelGGL((lora_expand_kernel<BF>),
                       tile_grid(cdiv(p.M, 64) * cdiv(p.N, kExpandColumns)), dim3(256), lds,
                       stream, p);
}

} // namespace

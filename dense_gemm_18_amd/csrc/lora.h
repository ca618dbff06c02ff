// lora.h -- kernels and launches of the low-rank adapters beside a shared projection,
// compiled once for each 16-bit type.
#pragma once

#include "lora_nt.h"
#include "w4_product.h"

// Rows of a tile of the first product, and of one where there are many.
constexpr int kLoraRows = 32;
constexpr int kLoraMany = 64;
// Pieces of u at most.
constexpr int kLoraParts = 8;
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
    int items, rblocks;            // workgroups for a tile's adapters, blocks of their rows
    int columns, split;            // of a workgroup of the second product; who share adapters
};

// Whether the first product runs on the tiles of more rows, 64 of the rank to a workgroup.
inline bool lora_many(int64_t M, int64_t rank) { return M > 512 && rank > 32; }

// Tiles of the first product, with the blocks of the rank that take a workgroup each there.
inline int64_t lora_tiles(int64_t M, int64_t rank)
{
    return lora_many(M, rank) ? cdiv(M, kLoraMany) * cdiv(rank, 64) : cdiv(M, kLoraRows);
}

// Pieces of K in the first product, and with them of u, at most: what the workspace has room
// for.  Of 512 elements or more; the fewer the tiles, the more of them.
inline int lora_parts(int64_t M, int64_t K, int64_t rank)
{
    const int64_t tiles = lora_tiles(M, rank);
    const int64_t most = lora_many(M, rank) || tiles < 8 ? kLoraParts : 4;
    int64_t p = tiles < 8 ? kLoraParts : kCUs / tiles;
    p = p > most ? most : p < 1 ? 1 : p;
    return (int)(p < cdiv(K, 512) ? p : cdiv(K, 512));
}

// One translation unit for each type.  Not exported from the library.
struct LoraLaunch {
    // u
    void (*shrink)(const LoraArgs &, hipStream_t);
    // D from the weight's tiles with the adapters' part added, for a group or 16-bit weights
    void (*fused)(const LoraArgs &, const W4Args &, int group, hipStream_t);
    // the adapters' part alone into dense rows of D
    void (*expand)(LoraArgs, hipStream_t);
};
__attribute__((visibility("hidden"))) LoraLaunch gemm18_lora_f16();
__attribute__((visibility("hidden"))) LoraLaunch gemm18_lora_bf16();

namespace {

// 16 bytes at any 2-byte alignment (one global load).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

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
// core of skinny.h with A's rows as the weight: each workgroup looks for its items among the
// tile's ids and gathers their rows, so an adapter is read once for the rows that have it
// and no row is multiplied with another's.
template <bool BF, int RB, int MB, int NW>
__device__ __forceinline__ void lora_item(const LoraArgs &p, char *lds, const int *list, int rows,
                                          int64_t m0, int tile, int a, int rb, int part)
{
    constexpr int kEach = 16 * RB * NW;
    const int steps = (p.K + 127) >> 7;
    const int k0 = part * steps / p.parts * 128;
    Skinny<BF, 0, RB, MB, 8 / NW, NW, true> c;
    c.W.w = p.A + k0;
    c.row[0] = (int64_t)a * p.rank + rb * kEach;
    c.rows[0] = p.rank - rb * kEach;
    c.stride = p.K;
    c.K = min((part + 1) * steps / p.parts * 128, p.K) - k0;
    c.M = rows;
    const float s = p.s ? p.s[a] : 1.0f;       // on its way before the rest
    c.begin(lds, p.X + m0 * p.ldx + k0,
            (uint32_t)((min((int64_t)tile, p.M - m0) - 1) * p.ldx + c.K) * 2u);
    c.run([&](int m) { return (uint32_t)(list[m] * p.ldx) * 2u; });
    float *u = p.u + ((int64_t)part * p.M + m0) * p.rank;
    c.join([&](int m, int n, const float(&v)[RB]) {
        const int j = rb * kEach + (n >> 4) * (16 * RB) + (n & 15);
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (j + 16 * r < p.rank)
                u[(int64_t)list[m] * p.rank + j + 16 * r] = v[r] * s;
    });
}

// RB * NW: blocks of 16 of the rank; TM: rows of a tile.
template <bool BF, int RB, int NW, int TM>
__global__ void __launch_bounds__(512, 2) lora_shrink_kernel(LoraArgs p)
{
    extern __shared__ f32x4 lds[];
    __shared__ int list[TM];
    // Items vary slowest: those that find no adapter are then the last workgroups.  (Between
    // the others, and dealt to the XCDs by turns, they left half of these idle: 34 us instead
    // of 19 for 2048 rows of 8192, rank 64, with a second item to each tile.)
    int64_t wg = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t tiles = (p.M + (int64_t)TM - 1) / TM;
    const int part = (int)(wg % p.parts);
    wg /= p.parts;
    const int rb = (int)(wg % p.rblocks);
    wg /= p.rblocks;
    const int64_t m0 = wg % tiles * TM;
    wg /= tiles;
    if (wg >= p.items)
        return;
    const int lane = threadIdx.x & 63;
    const int id = lane < TM ? adapter_of(p, m0 + lane) : -1;
    for (int item = (int)wg;; item += p.items) {
        const uint64_t mask = rows_of(id, item);
        if (!mask)
            return;
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(mask));
        __syncthreads();                  // the item before is done with the list
        if (threadIdx.x < 64 && (mask >> lane & 1))
            list[__popcll(mask & ((1ull << lane) - 1))] = lane;
        __syncthreads();
        const int rows = __popcll(mask);
        if (rows <= 16)
            lora_item<BF, RB, 1, NW>(p, (char *)lds, list, rows, m0, TM, a, rb, part);
        else if (TM <= 32 || rows <= 32)
            lora_item<BF, RB, 2, NW>(p, (char *)lds, list, rows, m0, TM, a, rb, part);
        else if constexpr (TM > 32)
            lora_item<BF, RB, 4, NW>(p, (char *)lds, list, rows, m0, TM, a, rb, part);
    }
}

template <bool BF, int RB, int NW, int TM>
void launch_shrink(LoraArgs p, hipStream_t stream)
{
    p.rblocks = (int)cdiv(p.rank, 16 * RB * NW);
    const int rows = p.M < TM ? p.M : TM;
    const int k = (int)cdiv(cdiv(p.K, 128), p.parts) * 128;
    constexpr int KW = 8 / NW;
    int lds = Skinny<BF, 0, RB, 1, KW, NW, true>::lds_bytes(rows < 16 ? rows : 16, k);
    const int two = Skinny<BF, 0, RB, 2, KW, NW, true>::lds_bytes(rows < 32 ? rows : 32, k);
    lds = lds > two ? lds : two;
    if constexpr (TM > 32) {
        const int four = Skinny<BF, 0, RB, 4, KW, NW, true>::lds_bytes(rows, k);
        lds = lds > four ? lds : four;
    }
    hipLaunchKernelGGL((lora_shrink_kernel<BF, RB, NW, TM>),
                       tile_grid(cdiv(p.M, TM) * p.items * p.rblocks * p.parts), dim3(512), lds,
                       stream, p);
}

// How a tile of rows is shared.  Few tiles are a decode step, whose rows may all have
// adapters of their own: a workgroup for each, K in as many pieces as fill the compute units.
// Many are prompts, with one or two adapters to a tile.  A compute unit loads 25 bytes or so
// in a ns, which bounds them: tiles of 64 rows and 64 of the rank read X and the adapters
// least often.  Measured, K = 8192, in us: 64 rows of 32 adapters of rank 16 in 4 pieces 8.8,
// in 2 10.4, in 8 14.0; 2048 rows in runs of 220, rank 64, tiles of 32 rows, in 4 pieces 28.8,
// in 8 32.7, of 64 rows 32.6 and 20.4 (with a second workgroup for a tile's adapters 26.0);
// 1024 rows 16.6 and 13.1.
inline LoraArgs lora_shared(LoraArgs p)
{
    const bool many = lora_many(p.M, p.rank);
    const int rows = many ? kLoraMany : kLoraRows;
    const int64_t tiles = lora_tiles(p.M, p.rank);
    const int most = lora_parts(p.M, p.K, p.rank);
    int items = p.count < rows ? p.count : rows;
    items = items < p.M ? items : p.M;
    if (!many && tiles < 8) {
        const int64_t fill = kCUs / (tiles * items);
        p.parts = (int)(fill < 1 ? 1 : fill < most ? fill : most);
    } else {
        p.parts = most;
        const int64_t fill = many ? cdiv(kCUs, tiles * most)
                             : tiles < 32 ? 8 : cdiv(2 * kCUs, tiles * most);
        items = (int)(items < fill ? items : fill);
    }
    p.items = items;
    return p;
}

template <bool BF>
void lora_shrink(const LoraArgs &p, hipStream_t stream)
{
    const int64_t tiles = cdiv(p.M, kLoraRows);
    if (lora_many(p.M, p.rank))
        launch_shrink<BF, 2, 2, kLoraMany>(p, stream);
    else if (p.rank <= 16 || p.M <= 16 || (p.rank <= 32 && tiles < 8))
        launch_shrink<BF, 1, 1, kLoraRows>(p, stream);
    else
        launch_shrink<BF, 2, 1, kLoraRows>(p, stream);
}

// ---- beside the projection's tiles ---------------------------------------

// The addend of a tile: u of its rows and their adapters wait in LDS, an output reads its
// row of B.  A thread's first value of u is on its way before the weights are: its pieces by
// unconditional loads, together, with nothing that waits for the row's adapter: one row of 4096 x
// 4096 with 8 pieces 10.1 us, 10.4 with rank 64, the product alone 9.4; with a loop over the
// pieces after the product 10.5 and 11.8.  Rank 12 takes what 16 does; 0.35 us more with its last
// four loaded one by one.
struct LoraPlus {
    static constexpr bool kNone = false;
    const float *u;
    const uint16_t *B;
    const int32_t *ids;
    int M, N, rank, count, parts;
    int lds_at;

    struct Value {
        int id;
        float x[kLoraParts];
    };

    __host__ __device__ int stride() const { return (rank + 7) & ~7; }
    int bytes(int rows) const { return rows * (stride() + 4) * 4; }

    // What value i of the tile is made of.
    __device__ __forceinline__ Value load(int i, int m0, int rows) const
    {
        const int ld = stride() + 4, m = i / ld, j = i - m * ld - 4;
        const auto at = range(u + (int64_t)m0 * rank,
                              (uint32_t)(((int64_t)(parts - 1) * M + rows) * rank * 4));
        const uint32_t off = m < rows && (uint32_t)j < (uint32_t)rank
                                 ? (uint32_t)(m * rank + j) * 4u : kOob;
        Value v;
        v.id = __builtin_amdgcn_raw_buffer_load_b32(range(ids + m0, (uint32_t)rows * 4u),
                                                    (uint32_t)m * 4u, 0, 0);
#pragma unroll
        for (int q = 0; q < kLoraParts; ++q)
            v.x[q] = __builtin_bit_cast(
                float, __builtin_amdgcn_raw_buffer_load_b32(
                           at, q < parts ? off + (uint32_t)q * (uint32_t)M * (uint32_t)rank * 4u : kOob,
                           0, 0));
        return v;
    }

    __device__ __forceinline__ Value first(int m0, int rows) const
    {
        return load(threadIdx.x, m0, rows);
    }

    // Row m's adapter is the word before its u.
    __device__ __forceinline__ void stage(char *lds, int m0, int rows, Value v) const
    {
        const int ld = stride() + 4, all = rows * ld;
        float *to = (float *)(lds + lds_at);
        for (int i = threadIdx.x; i < all;) {
            const bool in = (uint32_t)v.id < (uint32_t)count;
            float sum = v.x[0];
#pragma unroll
            for (int q = 1; q < kLoraParts; ++q)
                sum += v.x[q];
            to[i] = i % ld < 4 ? __builtin_bit_cast(float, in ? v.id : -1) : in ? sum : 0.0f;
            i += blockDim.x;
            if (i < all)
                v = load(i, m0, rows);
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
        // the last `count` of eight of B and of u, from j on
        auto piece = [&](u32x4 v, int j, int count) G18_INLINE {
            const float *x = from + 4 + j;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(
                    e >= 8 - count ? x[e] : 0.0f,
                    e >= 8 - count ? to_float<BF>((uint16_t)(v[e >> 1] >> (16 * (e & 1)))) : 0.0f,
                    sum);
        };
        auto eight = [&](int j) G18_INLINE { return *(const u32x4_any *)(b + j); };
        int j = 0;
        for (; j + 16 <= rank; j += 16) {        // two loads on their way together
            const u32x4 v = eight(j), w = eight(j + 8);
            piece(v, j, 8);
            piece(w, j + 8, 8);
        }
        // What is left, fewer than 16, ends with the row's last eight: no branch around a load.
        const int left = rank - j;
        if (left > 8) {
            const u32x4 v = eight(j), w = eight(rank - 8);
            piece(v, j, 8);
            piece(w, rank - 8, left - 8);
        } else if (left && rank >= 8) {
            piece(eight(rank - 8), rank - 8, left);
        } else if (left) {
            uint16_t v[8];
#pragma unroll
            for (int e = 0; e < 7; ++e)
                v[e] = b[e < rank ? e : rank - 1];
#pragma unroll
            for (int e = 0; e < 7; ++e)
                sum = __builtin_fmaf(e < rank ? from[4 + e] : 0.0f,
                                     e < rank ? to_float<BF>(v[e]) : 0.0f, sum);
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

// Tiles of 16-bit weights, rank 16, 32 adapters, in us: one row of 16384 x 4096 in tiles of
// 16 x 32 24.4, of 16 x 16 26.0, 5120 x 2048 8.3 and 9.2, but 12288 x 8192 45.5 and 35.7, 8192 x
// 6144 21.7 and 20.6, 4096 x 4096 11.7 and 9.9; 64 rows of 2048 x 4096 in tiles of 32 x 16 17.5,
// of 32 x 32 19.5, 128 rows 23.2 and 19.9.  A weight of 268 MB, 16384 x 8192, goes by at 5.8
// TB/s.
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
        if (p.N <= 16 * kCUs || p.K > 4096)
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

// 64 rows of the adapters' part, p.columns columns of it.  u, summed and rounded to the
// 16-bit type (each row times a power of two that leaves its largest near 1, taken off
// afterwards), is in LDS.  Each wave takes pairs of an adapter and 64 columns: the adapter's
// rows of B, which come straight to registers, meet every 16 rows that hold one of its own,
// and only its own are stored, so what is infinite in one adapter stays out of the others'
// rows.  The rows of B of several pairs travel at once, the first ones' while u is summed.
// Results go through the wave's own LDS 16 rows at a time, whole
// 128-byte lines of a row leave together.  Where there are few tiles, p.split workgroups share
// one's adapters.  KS: pieces of 32 of the
// rank.
constexpr int kExpandLine = 64 * 2 + 16;         // bytes of a staged row

// TAIL: the rank is no multiple of 8.  (Past 128 that form spills 33 registers of a lane.)
template <bool BF, int KS, bool TAIL>
__global__ void __launch_bounds__(512, 2) lora_expand_kernel(LoraArgs p)
{
    using x8 = typename Elem<BF>::x8;
    constexpr int kLd = KS * 32 + 8;             // 16-bit elements of a row of u
    constexpr int kAhead = TAIL ? 1 : KS == 1 ? 4 : KS == 2 ? 2 : 1;   // pairs of a wave at once
    extern __shared__ f32x4 lds[];
    __shared__ float unscale[64];
    __shared__ int adapter[64];
    __shared__ uint64_t has[64], with[64];
    const int blocks = (p.N + p.columns - 1) / p.columns;
    // Workgroups are dealt to the eight XCDs by turns: each gets tiles that follow one
    // another, so that what it reads of u and B passes its L2 once.
    const uint32_t all = ((uint32_t)p.M + 63u) / 64u * p.split * blocks;
    const uint32_t dealt = blockIdx.x + blockIdx.y * gridDim.x;
    if (dealt >= all)
        return;
    uint32_t wg = dealt % 8 * (all / 8) + min(dealt % 8, all % 8) + dealt / 8;
    const int n0 = (int)(wg % blocks) * p.columns;
    wg /= blocks;
    const int share = (int)(wg % p.split);
    const int64_t m0 = (int64_t)(wg / p.split) * 64;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int id = adapter_of(p, m0 + lane);
    uint16_t *held = (uint16_t *)lds;
    char *stage = (char *)lds + 64 * kLd * 2 + wave * (16 * kExpandLine);
    // The tile's adapters by their first rows, eight rows to a wave, and of these the ones
    // that are this workgroup's.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = 8 * wave + i;
        const uint64_t same = __ballot(id == __builtin_amdgcn_readlane(id, m));
        if (lane == 0)
            with[m] = same;
    }
    __syncthreads();
    const uint64_t mine = with[lane];
    const uint64_t firsts = __ballot(id >= 0 && __builtin_ctzll(mine) == lane);
    const int total = __popcll(firsts), index = __popcll(firsts & ((1ull << lane) - 1));
    const int count = (total - share + p.split - 1) / p.split;
    if (wave == 0 && (firsts >> lane & 1) && index % p.split == share) {
        adapter[index / p.split] = id;
        has[index / p.split] = mine;
    }
    __syncthreads();
    const int c = lane >> 4, col = lane & 15;
    const int cols = (min(p.columns, p.N - n0) + 63) >> 6, pairs = count * cols;
    using Rows = x8[4][KS];
    // Unconditional buffer loads, rows past N and what is past the rank out of range: a
    // branch around loads would wait for each.  A rank that is no multiple of 8 leaves
    // elements of the next row behind the last, which are cleared; where it is odd the last
    // element may be half of the range's last word, which reads as 0, and is loaded alone.
    auto fetch = [&](Rows &w, int pair) G18_INLINE {
        const int k = uniform(pair / cols), n = n0 + (pair - k * cols) * 64;
        const int rows = min(64, p.N - n), a = uniform(adapter[k]);
        const auto rs = range(p.B + ((int64_t)a * p.N + n) * p.rank,
                              (uint32_t)(rows * p.rank) * 2u);
        u32x4 v[4][KS];
        [[maybe_unused]] uint32_t end[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t row = (uint32_t)((col + 16 * i) * p.rank) * 2u;
#pragma unroll
            for (int q = 0; q < KS; ++q)
                v[i][q] = load_b128(rs, 32 * q + 8 * c < p.rank ? row + (32 * q + 8 * c) * 2u
                                                                : kOob);
            if (TAIL && (p.rank & 1))
                end[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                    rs, row + (p.rank - 1) * 2u, 0, 0);
        }
        if constexpr (TAIL) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < KS; ++q) {
                    const int left = p.rank - 32 * q - 8 * c;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t keep = left > 2 * j + 1 ? 0xffffffffu
                                              : left > 2 * j   ? 0xffffu
                                                               : 0u;
                        v[i][q][j] =
                            left == 2 * j + 1 && (p.rank & 1) ? end[i] : v[i][q][j] & keep;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < KS; ++q)
                w[i][q] = __builtin_bit_cast(x8, v[i][q]);
    };
    Rows w[kAhead];
    auto fetch_from = [&](int first) G18_INLINE {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (first + 8 * i < pairs)
                fetch(w[i], first + 8 * i);
    };
    fetch_from(wave);
    {
        // eight lanes to a row
        const int m = threadIdx.x >> 3, j0 = threadIdx.x & 7;
        const bool in = __shfl(id, m) >= 0;
        // pieces of u as many at a time as registers take, unconditionally
        constexpr int kAtOnce = KS <= 2 ? 4 : KS == 4 ? 2 : 1;
        const auto at = range(p.u + m0 * p.rank,
                              (uint32_t)(((int64_t)(p.parts - 1) * p.M +
                                          min((int64_t)64, p.M - m0)) * p.rank * 4));
        float v[KS * 4], most = 0.0f;
#pragma unroll
        for (int i = 0; i < KS * 4; ++i)
            v[i] = 0.0f;
        for (int q = 0; q < p.parts; q += kAtOnce) {
            float x[kAtOnce][KS * 4];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const bool piece = in && q + k < p.parts;
                const uint32_t row =
                    ((uint32_t)(q + k) * (uint32_t)p.M + (uint32_t)m) * (uint32_t)p.rank;
#pragma unroll
                for (int i = 0; i < KS * 4; ++i)
                    x[k][i] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(
                                   at, piece && j0 + 8 * i < p.rank ? (row + j0 + 8 * i) * 4u
                                                                    : kOob, 0, 0));
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                for (int i = 0; i < KS * 4; ++i)
                    v[i] += x[k][i];
        }
#pragma unroll
        for (int i = 0; i < KS * 4; ++i)
            most = __builtin_fmaxf(most, __builtin_fabsf(v[i]));
#pragma unroll
        for (int d = 1; d < 8; d *= 2)
            most = __builtin_fmaxf(most, __shfl_xor(most, d));
        // 2^e <= most < 2^(e + 1); what is 0 or not finite stays as it is
        int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
        e = e == 128 || most == 0.0f ? 0 : e < -126 ? -126 : e;
        if (j0 == 0)
            unscale[m] = __builtin_ldexpf(1.0f, e);
#pragma unroll
        for (int i = 0; i < KS * 4; ++i)
            held[m * kLd + j0 + 8 * i] = from_float<BF>(__builtin_ldexpf(v[i], -e));
    }
    __syncthreads();
    const int vec = p.N % 4 != 0 || ((uintptr_t)p.D & 7) ? 0 : p.N % 8 || ((uintptr_t)p.D & 15)
                                                                   ? 1 : 2;
    auto packed = [&](const f32x4 &v) G18_INLINE {
        return u32x2{from_float<BF>(v[0]) | (uint32_t)from_float<BF>(v[1]) << 16,
                     from_float<BF>(v[2]) | (uint32_t)from_float<BF>(v[3]) << 16};
    };
    auto store = [&](int m, int n, u32x2 v) G18_INLINE {
        uint16_t *to = p.D + (m0 + m) * (int64_t)p.N + n;
        if (vec) {
            if (n < p.N)
                *(u32x2 *)to = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.N)
                    to[r] = (uint16_t)(v[r >> 1] >> (16 * (r & 1)));
        }
    };
    auto consume = [&](const Rows &w, int pair) G18_INLINE {
        const int k = pair / cols, n = n0 + (pair - k * cols) * 64;
        const uint64_t rows = has[k];
        const bool lines = vec == 2 && n + 64 <= p.N;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t mine = uniform((int)(rows >> (16 * b)) & 0xffff);
            if (!mine)
                continue;
            x8 a[KS];
#pragma unroll
            for (int q = 0; q < KS; ++q)
                a[q] = *(const x8 *)(held + (16 * b + col) * kLd + q * 32 + 8 * c);
            const float by = unscale[16 * b + col];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < KS; ++q)
                    acc = mfma16<BF>(w[i][q], a[q], acc);
                const u32x2 v = packed(acc * by);
                if (lines)
                    *(u32x2 *)(stage + col * kExpandLine + i * 32 + c * 8) = v;
                else if (mine >> col & 1)
                    store(16 * b + col, n + 16 * i + 4 * c, v);
            }
            if (!lines)
                continue;
            // the wave's own writes come before its reads, and those before its next writes
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = 8 * i + (lane >> 3);
                const u32x4 v = *(const u32x4 *)(stage + m * kExpandLine + (lane & 7) * 16);
                if (mine >> m & 1)
                    *(u32x4 *)(p.D + (m0 + 16 * b + m) * (int64_t)p.N + n + (lane & 7) * 8) = v;
            }
            asm volatile("" ::: "memory");
        }
    };
    for (int first = wave; first < pairs; first += 8 * kAhead) {
        if (first != wave)
            fetch_from(first);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (first + 8 * i < pairs)
                consume(w[i], first + 8 * i);
    }
    // rows without an adapter
    const uint64_t bare = __ballot(id < 0 && m0 + lane < p.M);
    if (bare && share == 0)
        for (int i = wave; i < 4 * cols; i += 8)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (bare >> (16 * b + col) & 1)
                    store(16 * b + col, n0 + 16 * i + 4 * c, u32x2{0, 0});
}

template <bool BF, int KS>
void launch_expand(const LoraArgs &p, hipStream_t stream)
{
    const auto go = [&](auto tail) {
        hipLaunchKernelGGL((lora_expand_kernel<BF, KS, decltype(tail)::value>),
                           tile_grid(cdiv(p.M, 64) * cdiv(p.N, p.columns) * p.split), dim3(512),
                           64 * (KS * 32 + 8) * 2 + 8 * 16 * kExpandLine, stream, p);
    };
    if (p.rank % 8)
        go(std::true_type{});
    else
        go(std::false_type{});
}

// As many columns to a workgroup, 64 to 1024, as leave each compute unit one; and where even
// 64 are not few enough, several that share a tile's adapters, down to eight for each.
// Measured, in us: 64 x 16384, 32 adapters of rank 16, 64 columns 13.3, 128 18, two sharing
// 14.7; 64 x 8192 12.8 and, two sharing, 10.5; 2048 x 8192, rank 16, 512 columns 10.6, 256 14.3;
// rank 64 in 8 parts of u 512 columns 27.8, 1024 23.1.  (Since then u's parts travel together
// and an XCD's tiles follow one another: 64 x 16384 12.5 to 11.2, 2048 x 8192, rank 64, 28.1 to
// 26.1 in a trace: 34 MB written at 1.3 TB/s, after u's parts and the adapters' rows.)
template <bool BF>
void lora_expand(LoraArgs p, hipStream_t stream)
{
    const auto wgs = [&] { return cdiv(p.M, 64) * cdiv(p.N, p.columns); };
    p.columns = 1024;
    while (p.columns > 64 && wgs() < kCUs)
        p.columns /= 2;
    const int64_t most = cdiv(p.count < 64 ? p.count : 64, 8), fill = kCUs / wgs();
    p.split = (int)(fill < most ? fill : most);
    p.split = p.split > 1 ? p.split : 1;
    if (p.rank <= 32)
        launch_expand<BF, 1>(p, stream);
    else if (p.rank <= 64)
        launch_expand<BF, 2>(p, stream);
    else if (p.rank <= 128)
        launch_expand<BF, 4>(p, stream);
    else
        launch_expand<BF, 8>(p, stream);
}

} // namespace

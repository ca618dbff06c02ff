// skinny.h -- the product core of few rows against many weight rows that the
// 4-bit product, the router and the expert kernels share.  Everything here has
// internal linkage.
//
// A workgroup owns 16 * RB * NW weight rows and 16 * MB activation rows; its
// KW * NW waves are NW bands of rows times KW pieces of K, joined in LDS at
// the end.  K is walked in steps of 128.  Each of a step's four
// v_mfma_f32_16x16x32 takes the activations as its first operand and the
// weights as its second, so a lane loads weights of one row n = lane % 16
// (elements 8c .. 8c+7 of the 32, with c = lane / 16) and its accumulators
// hold column n, rows m = 4c .. 4c+3: a group's scale is one value per lane,
// that of the row the lane loads.
//
// Weights go straight to registers, each used by one wave only, and are the
// only vector loads of the inner loop: activations, scales and zero points are
// staged in LDS a chunk of K at a time.  Measured on 1 x 16384 x 8192 with
// 4-bit weights that the last-level cache holds (10.4 us for reading them and
// nothing else, 6.5 TB/s): 13.0 us with activations in LDS, 17.4 with
// activations as vector loads, and 5.4 more with a scale load per step, which
// asks L2 for as many lines as the weights do.  A ring of prefetched steps
// (2, 3 or 4 deep) was slower than eight waves that each wait for their batch.
#pragma once

#include <mutex>

#include "gemm_types.h"
#include "moe_nt.h"

// A weight matrix as a kernel sees it: 16-bit rows, or packed rows with
// scales and zero points.
struct WeightRef {
    const uint16_t *w;     // 16-bit weights
    const uint32_t *q;     // packed ones
    const uint16_t *s;
    const uint8_t *z;      // may be null: 8
};

namespace {

// A value that every lane of the wave has, as a scalar: branches on it are
// the wave's.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <bool BF>
__device__ __forceinline__ float to_float(uint16_t bits)
{
    if constexpr (BF)
        return __builtin_bit_cast(float, (uint32_t)bits << 16);
    else
        return (float)__builtin_bit_cast(_Float16, bits);
}

// Round to nearest even.
template <bool BF>
__device__ __forceinline__ uint16_t from_float(float v)
{
    return __builtin_bit_cast(uint16_t, (typename Elem<BF>::T)v);
}

// What a product with packed bfloat16 weights has to be multiplied by: they go to
// the matrix units times 2^-11 (still exact), so that a group's sum of at most 128
// terms of 15 |A| stays in fp32's range wherever A does.  fp16's does anyway.
template <bool BF, int GS>
constexpr float kUnscale = BF && GS != 0 ? 0x1p11f : 1.0f;

// Eight 4-bit values of one packed word less their zero point (bfloat16: times
// 2^-11), exact in either type.  A value in the low bits of the mantissa of 1024
// (fp16) is that number plus q, one four bits up 1024 + 16 q: one mask-and-or makes
// two of them, and one shift serves all.
//
// fp16 takes 1024 + z off both halves in one packed instruction, or has a packed
// fma with 1/16 and 64 + z: 9 instructions for 8 weights.  bfloat16 has no packed
// arithmetic on gfx950: a mixed fma reads each half as fp16 and leaves the number
// in fp32, and the upper halves of two go together: 17 instructions.  (The matrix
// units could see 128 + q, for 7, with (128 + z) times the activations' sum taken
// off afterwards.  Those sums are of terms up to 143 |A| where the result has 15
// |A| or less, so an activation that stands out left its rounding where its weight
// is 0.  Exact numbers take 3 to 12 % longer up to 32 rows, 7 x 16384 x 8192 in
// groups of 128 18.0 us for 16.7, up to 28 % in the resident tile, and 3 to 8 %
// less from 64 rows on: matrix instructions for the activations' sums are saved.)
// sz: 1024 + z in fp16, in its upper half.
template <bool BF>
__device__ __forceinline__ typename Elem<BF>::x8 unpack8(uint32_t w, uint32_t sz)
{
    // the constants in registers: v_and_or_b32 takes no literals
    uint32_t mask = 0x000f000fu, mask4 = 0x00f000f0u, magic = 0x64006400u;
    asm("" : "+s"(mask));
    asm("" : "+s"(mask4));
    asm("" : "+v"(magic));
    const auto pair = [&](int t) G18_INLINE {
        return __builtin_bit_cast(f16x2,
                                  ((t < 2 ? w : w >> 8) & (t & 1 ? mask4 : mask)) | magic);
    };
    u32x4 v;
    if constexpr (!BF) {
        uint32_t off = (sz >> 16) | (sz & 0xffff0000u);
        asm("" : "+v"(off));      // seen as two equal halves it would be split up again
        const f16x2 z = __builtin_bit_cast(f16x2, off);
        const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
        // 64 + z, from 1024 + z
        const f16x2 z4 = z - f16x2{(_Float16)960.0f, (_Float16)960.0f};
#pragma unroll
        for (int t = 0; t < 4; ++t)
            v[t] = __builtin_bit_cast(
                uint32_t, t & 1 ? __builtin_elementwise_fma(pair(t), sixteenth, -z4) : pair(t) - z);
        return __builtin_bit_cast(f16x8, v);
    } else {
        const float z = (float)__builtin_bit_cast(f16x2, sz)[1];
        const float off = z * 0x1p-11f, off4 = (z - 960.0f) * 0x1p-11f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f16x2 q = pair(t);
            const float by = t & 1 ? 0x1p-15f : 0x1p-11f, less = t & 1 ? off4 : off;
            const float lo = __builtin_fmaf((float)q[0], by, -less);
            const float hi = __builtin_fmaf((float)q[1], by, -less);
            // exact: the upper halves are the numbers
            v[t] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi),
                                         __builtin_bit_cast(uint32_t, lo), 0x07060302u);
        }
        return __builtin_bit_cast(bf16x8, v);
    }
}

// A range of memory for buffer loads; loads outside it return 0 and cost
// nothing.  `base` and `bytes` are the wave's.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)bytes, kRsrcFlags);
}

__device__ __forceinline__ u32x4 load_b128(__amdgpu_buffer_rsrc_t rs, uint32_t off)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

// LDS of a product: activations, then scales, up to these sizes.
constexpr int kActBytes = 66 * 1024;
constexpr int kScaleBytes = 32 * 1024;

// The matrix instruction of pairs of 16-byte pieces of FP8 rows; F8 = 1 + fa + 2 * fb with
// the formats of the activations and of the weights (0: E4M3, 1: E5M2).
template <int F8>
__device__ __forceinline__ f32x4 mfma_pair(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c)
{
    constexpr int fa = (F8 - 1) & 1, fb = (F8 - 1) >> 1;
    const auto both = [](u32x4 x, u32x4 y) G18_INLINE {
        return __builtin_bit_cast(i32x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(both(a0, a1), both(b0, b1), c, fa, fb,
                                                            0, 0, 0, 0);
}

// One workgroup's product.  GS: 0 for 16-bit weights, else the group.
// JOINED: the workgroup's weight rows follow each other; else (RB even, NW == 1)
// each half of the blocks starts at a row of its own.  F8 (GS 0): activations and weights
// are rows of pairs of FP8 bytes, K counts the pairs.
template <bool BF, int GS, int RB, int MB, int KW, int NW, bool JOINED, int F8 = 0>
struct Skinny {
    using x8 = typename Elem<BF>::x8;
    static constexpr int kThreads = KW * NW * 64;
    static constexpr int kGroups = GS ? 128 / (GS ? GS : 1) : 1;   // groups in a step
    static constexpr int NR = JOINED ? 1 : 2;
    static constexpr int kRows = 16 * RB * NW;                    // weight rows
    // Steps a wave asks for at once: 8 KB, 64 KB for eight waves, which at 25
    // bytes per ns and CU is 2.5 us of latency.
    static constexpr int U = GS == 0 ? (RB == 1 ? 2 : 1) : RB == 4 ? 2 : 4;

    // What the caller sets: the weights, the rows that exist from each
    // start, K, the number of activation rows.
    WeightRef W;
    int64_t row[NR];
    int rows[NR];
    int K, M;
    int stride = 0;              // 16-bit weights: elements between rows, 0 for K
    f32x4 acc[RB][MB];

    char *lds;
    int wave, G, chunk, astride, sstride;
    __amdgpu_buffer_rsrc_t wr[NR], sr[NR], zr[NR], ar;
    uint32_t woff[RB], zdef;       // zdef: 8 where there are no zero points

    // LDS for any number of activation rows up to `most` (with fewer rows the
    // chunk may be longer, so this bounds the two together).
    static int lds_bytes(int most, int K)
    {
        const int64_t all = cdiv(K, 128) * 128;
        const int64_t need = most * (all * 2 + 16) +
                             (GS ? (int64_t)kRows * (all / 128 * kGroups + 1) * 4 : 0);
        const int cap = kActBytes + (GS ? kScaleBytes : 0), red = KW * NW * RB * 1024;
        return need > cap ? cap : need > red ? (int)need : red;
    }
    // Rows of a chunk in LDS are 16 bytes longer than the chunk, so that the 16
    // rows that a fragment read touches lie in different banks.
    static constexpr int act_bytes(int M, int chunk) { return M * (chunk * 2 + 16); }
    static constexpr int scale_bytes(int chunk)
    {
        return GS ? kRows * (chunk / 128 * kGroups + 1) * 4 : 0;
    }
    // K of a chunk: all of it, or what the LDS holds, in whole steps and, where
    // it can be, the same number for each of the KW waves.
    static __host__ __device__ constexpr int chunk_of(int M, int K)
    {
        const int all = (K + 127) / 128;
        int steps = (kActBytes / M - 16) / 256;
        if (GS && steps > kScaleBytes / (kRows * 4 * kGroups) - 1)
            steps = kScaleBytes / (kRows * 4 * kGroups) - 1;
        if (steps >= all)
            return all * 128;
        if (steps > KW)
            steps -= steps % KW;
        return steps * 128;
    }

    __device__ __forceinline__ int lane() const { return threadIdx.x & 63; }
    __device__ __forceinline__ int kw() const { return NW == 1 ? wave : wave % KW; }
    __device__ __forceinline__ int nw() const { return NW == 1 ? 0 : wave / KW; }

    // The activations: `bytes` from `base`.
    __device__ __forceinline__ void begin(char *smem, const uint16_t *base, uint32_t bytes)
    {
        ar = range(base, bytes);
        lds = smem;
        wave = uniform(threadIdx.x >> 6);
        G = GS ? (K + GS - 1) / (GS ? GS : 1) : 0;
        chunk = chunk_of(M, K);
        astride = chunk * 2 + 16;
        sstride = chunk / 128 * kGroups + 1;
        const uint32_t row_bytes =
            GS ? (uint32_t)((K + 127) >> 7) * 64u : (uint32_t)(stride ? stride : K) * 2u;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int n = min(rows[i], kRows / NR);
            wr[i] = range(GS ? (const char *)W.q + row[i] * row_bytes
                             : (const char *)W.w + row[i] * row_bytes,
                          GS ? n * row_bytes : n ? (n - 1) * row_bytes + K * 2u : 0);
            if constexpr (GS != 0) {
                sr[i] = range(W.s + row[i] * G, n * G * 2);
                zr[i] = range(W.z ? W.z + row[i] * G : nullptr, W.z ? n * G : 0);
            }
        }
        zdef = W.z ? 0 : 8;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int at = JOINED ? (nw() * RB + r) * 16 : r % (RB / NR) * 16;
            woff[r] = (at + (lane() & 15)) * row_bytes + (lane() >> 4) * 16;
#pragma unroll
            for (int m = 0; m < MB; ++m)
                acc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    template <int N>
    struct Batch {
        u32x4 v[N][RB][GS ? 1 : 4];
    };

    // N steps from st on; nothing where a step is `end` or later.  Unconditional
    // loads with an offset past the range there: a branch around loads would
    // leave the compiler waiting for all of them.
    template <int N>
    __device__ __forceinline__ void load(Batch<N> &b, int st, int end) const
    {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const uint32_t o =
                    woff[r] + (st + u < end ? (uint32_t)(st + u) * (GS ? 64u : 256u) : kOob);
#pragma unroll
                for (int j = 0; j < (GS ? 1 : 4); ++j)
                    b.v[u][r][j] = load_b128(wr[r / (RB / NR)], o + 64u * j);
            }
    }

    // Activations k0 .. k0 + 128 * steps - 1 of every row, zero from K on.
    // `at(m)`: the byte of `ar` where row m starts.  Pieces of all the rows a
    // thread has to do with are under way at once: each wait is for memory.
    template <class F>
    __device__ __forceinline__ void stage_acts(int k0, int steps, F &&at) const
    {
        // a power of two of threads along a row, the rest along the rows
        const int per_row = steps * 16;
        constexpr int kLog = 31 - __builtin_clz(kThreads);
        int shift = kLog;
        while (shift > 4 && (1 << (shift - 1)) >= per_row)
            --shift;
        const int c0 = threadIdx.x & ((1 << shift) - 1), dc = 1 << shift;
        const int m0 = threadIdx.x >> shift, dm = kThreads >> shift;
        const int total = ((per_row + dc - 1) >> shift) * ((M + dm - 1) >> (kLog - shift));
        int c = 0, m = 0;
        auto batch = [&](auto count) G18_INLINE {
            constexpr int kBatch = decltype(count)::value;
            u32x4 v[kBatch];
            int dst[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = (c0 + c) * 8, row = m0 + m;
                const bool in = c0 + c < per_row && row < M, whole = k0 + k + 8 <= K;
                const uint32_t src = at(min(row, M - 1)) + (uint32_t)(k0 + k) * 2u;
                v[i] = load_b128(ar, in && whole ? src : kOob);
                // the 8 elements that K ends among come below
                dst[i] = in && (whole || k0 + k >= K) ? row * astride + k * 2 : -1;
                c += dc;
                if (c >= per_row) {
                    c = 0;
                    m += dm;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (dst[i] >= 0)
                    *(u32x4 *)(lds + dst[i]) = v[i];
        };
        for (int left = total; left > 0; left -= 4) {
            if (left > 2)
                batch(std::integral_constant<int, 4>{});
            else if (left == 2)
                batch(std::integral_constant<int, 2>{});
            else
                batch(std::integral_constant<int, 1>{});
        }
        if ((K & 7) && k0 + steps * 128 > K) {
            const int k = (K & ~7) + (threadIdx.x & 7);
            for (int m = threadIdx.x >> 3; m < M; m += kThreads / 8)
                *(uint16_t *)(lds + m * astride + (k - k0) * 2) =
                    (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                        ar, k < K ? at(m) + 2u * k : kOob, 0, 0);
        }
    }

    // Scale and zero point of each row's groups in one word: the scale's bits
    // below, above them the fp16 number that unpack8 takes off, 1024 + z.  Groups from G on, and rows past the end, have the scale 0.
    __device__ __forceinline__ void stage_scales(int k0, int steps) const
    {
        uint32_t *dst = (uint32_t *)(lds + act_bytes(M, chunk));
        const int g0 = k0 / (GS ? GS : 1), groups = steps * kGroups;
        // the waves' halves take the two blocks of rows, where there are two;
        // 16 threads or more along the groups of a row
        constexpr int kBatch = 4, kPart = kThreads / NR, kEach = kRows / NR;
        constexpr int kAlong = kPart / kEach > 16 ? kPart / kEach : 16;
        const int i = NR == 1 ? 0 : wave / (kPart / 64), t = threadIdx.x % kPart;
        const auto scales = NR > 1 && i ? sr[NR - 1] : sr[0];
        const auto zeros = NR > 1 && i ? zr[NR - 1] : zr[0];
        for (int n = t / kAlong; n < kEach; n += kPart / kAlong) {
            uint32_t *to = dst + (i * kEach + n) * sstride;
            for (int g = t % kAlong; g < groups; g += kAlong * kBatch) {
                uint32_t s[kBatch], z[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int gg = g0 + g + kAlong * k;
                    const uint32_t o = gg < G ? (uint32_t)(n * G + gg) : kOob;
                    s[k] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scales,
                                                                          2 * o + (o & kOob), 0, 0);
                    z[k] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(zeros, o, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (g + kAlong * k < groups)
                        to[g + kAlong * k] =
                            s[k] | (0x6400u + ((z[k] | zdef) & 15u)) << 16;
            }
        }
    }

    // The 8 elements of a row of 16-bit weights of which `left` (any number)
    // come before K; the others become zero.  Where K is odd, a buffer load,
    // which checks its range by the dword, loses the last element if nothing
    // follows it: it comes from `end`.
    __device__ __forceinline__ u32x4 mend(u32x4 v, int left, uint32_t end) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t keep = left > 2 * i + 1 ? 0xffffffffu : left > 2 * i ? 0xffffu : 0u;
            v[i] = left == 2 * i + 1 && (K & 1) ? end : v[i] & keep;
        }
        return v;
    }

    // Step u of a batch, step `st` of the chunk that starts at k0 and whose
    // activations and scales are at `acts` and `scales`.
    template <int N>
    __device__ __forceinline__ void consume(Batch<N> &b, int u, int st, int k0,
                                            const char *acts, const uint32_t *scales)
    {
        const int c = lane() >> 4;
        x8 a[MB][4];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            // rows past the last repeat it; their results are not used
            const char *p = acts + min(16 * m + (lane() & 15), M - 1) * astride + st * 256 + c * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a[m][j] = *(const x8 *)(p + 64 * j);
        }
        if constexpr (GS == 0) {
            if (k0 + st * 128 + 128 > K) {
                const int left = K - k0 - st * 128 - 8 * c;
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const uint32_t end = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                        wr[r / (RB / NR)], woff[r] - 16u * c + (uint32_t)(K - 1) * 2u, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        b.v[u][r][j] = mend(b.v[u][r][j], left - 32 * j, end);
                }
            }
            if constexpr (F8 != 0) {
#pragma unroll
                for (int j = 0; j < 4; j += 2)
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            acc[r][m] = mfma_pair<F8>(__builtin_bit_cast(u32x4, a[m][j]),
                                                      __builtin_bit_cast(u32x4, a[m][j + 1]),
                                                      b.v[u][r][j], b.v[u][r][j + 1], acc[r][m]);
                return;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[r][m] = mfma16<BF>(a[m][j], __builtin_bit_cast(x8, b.v[u][r][j]),
                                               acc[r][m]);
        } else {
            constexpr int per = 4 / kGroups;       // matrix instructions per group
            const uint32_t *sp =
                scales + ((JOINED ? nw() * RB * 16 : 0) + (lane() & 15)) * sstride + st * kGroups;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const uint32_t sz = sp[r * 16 * sstride + k];
                    const float sc = to_float<BF>((uint16_t)sz);
                    f32x4 sum[MB];
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        sum[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < per; ++i) {
                        const x8 f = unpack8<BF>(b.v[u][r][0][k * per + i], sz);
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            sum[m] = mfma16<BF>(a[m][k * per + i], f, sum[m]);
                    }
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][m][e] = __builtin_fmaf(sc, sum[m][e], acc[r][m][e]);
                }
            }
        }
    }

    // The product, each wave's part of it in `acc`.  `at(m)`: the byte of the
    // activations where row m starts.
    template <class F>
    __device__ __forceinline__ void run(F &&at)
    {
        const int total = (K + 127) >> 7, per = chunk >> 7;
        for (int s0 = 0; s0 < total; s0 += per) {
            const int steps = min(per, total - s0);
            int st = kw() * steps / KW;
            const int end = (kw() + 1) * steps / KW;
            Batch<U> b;
            load(b, s0 + st, s0 + end);
            if (s0 > 0)
                __syncthreads();          // the chunk before has been read
            stage_acts(s0 * 128, steps, at);
            if constexpr (GS != 0)
                stage_scales(s0 * 128, steps);
            __syncthreads();
#pragma nounroll
            while (st < end) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (st + u < end)
                        consume(b, u, st + u, s0 * 128, lds,
                                (const uint32_t *)(lds + act_bytes(M, chunk)));
                st += U;
                if (st < end)
                    load(b, s0 + st, s0 + end);
            }
        }
    }

    // Joins the KW waves of each band in LDS, in order, and hands
    // f(m, n, v) the sums v[r] of activation row m and row n of each block r
    // of band n / 16 (n in [0, 16 * NW)).  Every thread of the workgroup calls.
    template <class F>
    __device__ __forceinline__ void join(F &&f)
    {
        f32x4 *red = (f32x4 *)lds;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RB; ++r)
                red[((nw() * KW + kw()) * RB + r) * 64 + lane()] = acc[r][mb];
            __syncthreads();
            for (int i = threadIdx.x; i < 256 * NW; i += kThreads) {
                const int n = i & 15, m = (i >> 4) & 15, band = i >> 8;
                float v[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const float *p = (const float *)(red + (band * KW * RB + r) * 64 +
                                                     (m >> 2) * 16 + n) + (m & 3);
                    v[r] = 0.0f;
#pragma unroll
                    for (int w = 0; w < KW; ++w)
                        v[r] += p[w * RB * 256];
                    v[r] *= kUnscale<BF, GS>;
                }
                if (16 * mb + m < M)
                    f(16 * mb + m, band * 16 + n, v);
            }
        }
    }
};

// The same product where the activations do not fit the LDS: chunks of CS steps
// of K in two LDS buffers.  While one is consumed, the activations and scales of
// the chunk after travel to registers, and the weights of the next two are
// there already; one barrier ends the chunk.  Rows of packed weights that follow
// each other.
// 64 x 16384 x 8192, fp16, groups of 128, one workgroup to a CU: 31 us, of
// which reading the weights alone takes 14.  By counters the matrix units are
// busy for 25 % of it, the VALU (unpacking, 195 instructions for a step's 32
// matrix instructions) for 37 %, the LDS for 41 %, and with two waves to a SIMD
// these follow each other more than they overlap: without consuming it takes
// 18 us, without fetching activations 30 of then 37.  Wider rows in LDS (fewer
// bank conflicts), scheduling groups and unconditional steps changed nothing;
// the waves' halves one phase apart, one reading LDS while the other multiplies,
// took 32 to 36 us by where the fetches stood (smaller tiles more); four waves
// to a SIMD need 128 registers, which this tile does not have.
template <bool BF, int GS, int RB, int MB, int KW, int NW, int CS>
struct Piped : Skinny<BF, GS, RB, MB, KW, NW, true> {
    using Base = Skinny<BF, GS, RB, MB, KW, NW, true>;
    using Base::kGroups;
    using Base::kRows;
    using Base::kThreads;
    static constexpr int kSteps = CS / KW;                   // of a wave, in a chunk
    static constexpr int kStride = CS * 256 + 16;            // of activation rows in LDS
    static constexpr int kScales = CS * kGroups + 1;         // of scale rows, words
    static constexpr int kActs = 16 * MB * kStride;
    static constexpr int kBuffer = kActs + kRows * kScales * 4;
    static constexpr int NA = 16 * MB * CS * 16 / kThreads;  // 16-byte pieces of a thread
    static constexpr int NS = (kRows * CS * kGroups + kThreads - 1) / kThreads;
    static_assert(CS % KW == 0 && 16 * MB * CS * 16 % kThreads == 0, "whole pieces");
    static constexpr int kLds = 2 * kBuffer > KW * NW * RB * 1024 ? 2 * kBuffer
                                                                  : KW * NW * RB * 1024;

    struct Next {
        u32x4 a[NA];
        uint32_t s[NS], z[NS];
    };

    // The thread's pieces lie in one column, kRowStep rows apart: offsets into
    // memory and LDS differ by constants.
    static constexpr int kRowStep = kThreads / (CS * 16);
    static_assert(kThreads % (CS * 16) == 0, "one column");
    uint32_t row_bytes;             // between activation rows

    __device__ __forceinline__ int column() const { return threadIdx.x % (CS * 16); }
    __device__ __forceinline__ int first_row() const { return threadIdx.x / (CS * 16); }

    // What the thread stages of the chunk from k0 on (nothing from K on; rows
    // from M on are past the activations' range).
    __device__ __forceinline__ void fetch(Next &x, int k0) const
    {
        const int K = this->K, G = this->G;
        // all of the column's 8 elements; `store` fetches those that K ends among
        const bool in = k0 + column() * 8 + 8 <= K;
        const uint32_t o =
            in ? first_row() * row_bytes + (uint32_t)(k0 + column() * 8) * 2u : kOob;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            x.a[i] = load_b128(this->ar, o + (uint32_t)(i * kRowStep) * row_bytes);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int idx = i * kThreads + threadIdx.x, n = idx / (CS * kGroups);
            const int g = k0 / GS + idx % (CS * kGroups);
            const uint32_t o = g < G && n < kRows ? (uint32_t)(n * G + g) : kOob;
            x.s[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(this->sr[0],
                                                                    2 * o + (o & kOob), 0, 0);
            x.z[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(this->zr[0], o, 0, 0);
        }
    }

    __device__ __forceinline__ void store(const Next &x, int k0, char *buf) const
    {
        char *p = buf + first_row() * kStride + column() * 16;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            *(u32x4 *)(p + i * kRowStep * kStride) = x.a[i];
        uint32_t *scales = (uint32_t *)(buf + kActs);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int idx = i * kThreads + threadIdx.x;
            const int n = idx / (CS * kGroups), g = idx % (CS * kGroups);
            if (n < kRows)
                scales[n * kScales + g] =
                    x.s[i] | (0x6400u + ((x.z[i] | this->zdef) & 15u)) << 16;
        }
        // the 8 elements that K ends among, of which `fetch` left zeros
        const int K = this->K;
        if ((K & 7) && k0 <= K && k0 + CS * 128 > K) {
            __syncthreads();
            const int k = (K & ~7) + (threadIdx.x & 7);
            for (int m = threadIdx.x >> 3; m < 16 * MB; m += kThreads / 8)
                *(uint16_t *)(buf + m * kStride + (k - k0) * 2) =
                    (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                        this->ar, k < K ? m * row_bytes + 2u * k : kOob, 0, 0);
        }
    }

    // `at(m)` is m times at(1) here.
    template <class F>
    __device__ __forceinline__ void run(F &&at)
    {
        row_bytes = at(1);
        this->astride = kStride;
        this->sstride = kScales;
        const int total = (this->K + 127) >> 7, mine = this->kw() * kSteps;
        typename Base::template Batch<kSteps> even, odd;
        Next x;
        fetch(x, 0);
        this->load(even, mine, total);
        this->load(odd, CS + mine, total);
        store(x, 0, this->lds);
        fetch(x, CS * 128);
        __syncthreads();
        // The chunk from step s0 on, whose weights are in b and whose activations
        // are in `buf`.  Two copies of this make the loop: a copy of registers
        // that a load is still to fill would wait for it.
        auto chunk = [&](auto &b, int s0, char *buf, char *other) G18_INLINE {
            store(x, (s0 + CS) * 128, other);
            fetch(x, (s0 + 2 * CS) * 128);
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
                if (s0 + mine + u < total)
                    this->consume(b, u, mine + u, s0 * 128, buf, (const uint32_t *)(buf + kActs));
            this->load(b, s0 + 2 * CS + mine, total);
            __syncthreads();
        };
#pragma nounroll
        for (int s0 = 0; s0 < total; s0 += 2 * CS) {
            chunk(even, s0, this->lds, this->lds + kBuffer);
            chunk(odd, s0 + CS, this->lds + kBuffer, this->lds);
        }
    }
};

// Held while a call enqueues launches that hand each other results in
// `workspace`: those of another host thread's call on the same stream come before
// or after all of them.  Calls with other workspaces seldom meet.
inline std::mutex &launch_lock(const void *workspace)
{
    static std::mutex locks[64];
    return locks[(((uintptr_t)workspace >> 8) * 0x9e3779b97f4a7c15ull) >> 58];
}

inline bool overlap(const void *p, uint64_t pn, const void *q, uint64_t qn)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return pn && qn && a < b + qn && b < a + pn;
}

inline bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }
inline bool dtype_ok(int dtype) { return dtype == GEMM_T_F16 || dtype == GEMM_T_BF16; }
inline bool aligned_to(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// f(integral_constant<int, g>) for g the group (0, 32, 64 or 128).
template <class F>
inline void with_group(int group, F &&f)
{
    switch (group) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case 32: f(std::integral_constant<int, 32>{}); break;
    case 64: f(std::integral_constant<int, 64>{}); break;
    default: f(std::integral_constant<int, 128>{}); break;
    }
}

} // namespace

// skinny.h -- the product core of few rows against many weight rows that the
// 4-bit product and the expert kernels share.  Everything here has internal
// linkage.
//
// One wave owns 16 * RB weight rows and 16 * MB activation rows and walks K
// in steps of 128.  Each of a step's four v_mfma_f32_16x16x32 takes the
// activations as its first operand and the weights as its second, so a lane
// loads weights of one row n = lane % 16 (elements 8c .. 8c+7 of the 32, with
// c = lane / 16) and its accumulators hold column n, rows m = 4c .. 4c+3:
// a group's scale is one value per lane, that of the row the lane loads.
// Nothing goes through LDS on the way in: a weight is used by one wave only,
// and the activations, which every workgroup re-reads, come from L1 and L2.
#pragma once

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

// 16 bytes at any 2-byte alignment (one global load on gfx950).
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4 load16(const uint16_t *p) { return *(const u32x4_a2 *)p; }

// The first `count` of the 8 elements at p, zero for the others; nothing
// past them is accessed.
__device__ __forceinline__ u32x4 load16_part(const uint16_t *p, int count)
{
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count)
            v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
}

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

// Eight 4-bit values of one packed word as 16-bit integers, exact.  A value
// in the low bits of the mantissa of 1024 (fp16) or 128 (bfloat16) is that
// number plus q: one mask-and-or for two of them.  fp16 then subtracts
// 1024 + z from both halves in one packed instruction, exactly, leaving q - z.
// bfloat16 has no packed subtraction on gfx950: its 128 + q go to the matrix
// unit as they are, and the caller takes (128 + z) * sum(A) off in fp32 (7
// instructions for 8 weights; EXACT, which subtracts in fp32 and packs again,
// takes 35 and leaves (q - z) * 2^-12).
template <bool BF, bool EXACT>
__device__ __forceinline__ typename Elem<BF>::x8 unpack8(uint32_t w, uint32_t z)
{
    constexpr uint32_t magic = BF ? 0x43004300u : 0x64006400u;
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t)
        v[t] = ((w >> (4 * t)) & 0x000f000fu) | magic;
    if constexpr (!BF) {
        const uint32_t mz = 0x64006400u + z + (z << 16);
        const u32x4 m = {mz, mz, mz, mz};
        return __builtin_bit_cast(f16x8, v) - __builtin_bit_cast(f16x8, m);
    } else {
        if constexpr (EXACT) {
            const float off = (float)(128u + z);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float lo = (__builtin_bit_cast(float, v[t] << 16) - off) * 0x1p-12f;
                const float hi =
                    (__builtin_bit_cast(float, v[t] & 0xffff0000u) - off) * 0x1p-12f;
                v[t] = (__builtin_bit_cast(uint32_t, lo) >> 16) |
                       (__builtin_bit_cast(uint32_t, hi) & 0xffff0000u);
            }
        }
        return __builtin_bit_cast(bf16x8, v);
    }
}

// One wave's share of a product.  GS: 0 for 16-bit weights, else the group.
template <bool BF, int GS, int RB, int MB>
struct Skinny {
    using x8 = typename Elem<BF>::x8;
    static constexpr int kStep = 128;
    static constexpr int kGroups = GS ? kStep / (GS ? GS : 1) : 1;   // groups a step spans

    struct WBuf {
        u32x4 v[RB][GS ? 1 : 4];
        uint16_t s[RB][kGroups];
        uint8_t z[RB][kGroups];
    };
    struct ABuf {
        u32x4 v[MB][4];
    };

    // Per lane: the start of its weight rows and activation rows.
    const uint16_t *w16[RB];
    const uint32_t *q[RB];
    const uint16_t *s[RB];
    const uint8_t *z[RB];
    const uint16_t *a[MB];
    int K, G;
    f32x4 acc[RB][MB];

    __device__ __forceinline__ void init(int k)
    {
        K = k;
        G = GS ? (k + GS - 1) / (GS ? GS : 1) : 0;
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                acc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // The lane's row of block r is `row` of the matrix.
    __device__ __forceinline__ void bind(int r, const WeightRef &W, int64_t row)
    {
        const int c = (threadIdx.x & 63) >> 4;
        if constexpr (GS == 0) {
            w16[r] = W.w + row * K + 8 * c;
        } else {
            q[r] = W.q + row * ((int64_t)((K + 127) >> 7) * 16) + 4 * c;
            s[r] = W.s + row * G;
            z[r] = W.z ? W.z + row * G : nullptr;
        }
    }

    __device__ __forceinline__ void bind_act(int m, const uint16_t *row)
    {
        a[m] = row + 8 * ((threadIdx.x & 63) >> 4);
    }

    __device__ __forceinline__ void load_w(WBuf &b, int st) const
    {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            if constexpr (GS == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b.v[r][j] = load16(w16[r] + (int64_t)st * 128 + 32 * j);
            } else {
                b.v[r][0] = *(const u32x4 *)(q[r] + (int64_t)st * 16);
                load_scales(b, r, st);
            }
        }
    }

    __device__ __forceinline__ void load_scales(WBuf &b, int r, int st) const
    {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            // the last step may hold fewer groups than kGroups: scale 0
            const int at = st * kGroups + g;
            b.s[r][g] = at < G ? s[r][at] : (uint16_t)0;
            b.z[r][g] = z[r] && at < G ? z[r][at] & 15 : 8;
        }
    }

    __device__ __forceinline__ void load_a(ABuf &b, int st) const
    {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b.v[m][j] = load16(a[m] + (int64_t)st * 128 + 32 * j);
    }

    // The step that K ends in: elements from K on are zero in both operands
    // (of packed weights, in the activations alone: those weights are finite).
    __device__ __forceinline__ void load_tail(WBuf &wb, ABuf &ab, int st) const
    {
        const int left = K - st * 128 - 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = left - 32 * j;
#pragma unroll
            for (int m = 0; m < MB; ++m)
                ab.v[m][j] = load16_part(a[m] + (int64_t)st * 128 + 32 * j, n);
            if constexpr (GS == 0)
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    wb.v[r][j] = load16_part(w16[r] + (int64_t)st * 128 + 32 * j, n);
        }
        if constexpr (GS != 0)
            load_w(wb, st);
    }

    template <bool EXACT>
    __device__ __forceinline__ void consume(const WBuf &wb, const ABuf &ab)
    {
        consume<EXACT>(wb, ab, acc);
    }

    template <bool EXACT>
    __device__ __forceinline__ void consume(const WBuf &wb, const ABuf &ab,
                                            f32x4 (&acc)[RB][MB]) const
    {
        if constexpr (GS == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[r][m] = mfma16<BF>(__builtin_bit_cast(x8, ab.v[m][j]),
                                               __builtin_bit_cast(x8, wb.v[r][j]), acc[r][m]);
        } else {
            constexpr int per = 4 / kGroups;       // matrix instructions per group
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                f32x4 sum[RB][MB], asum[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    asum[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        sum[r][m] = asum[m];
                }
#pragma unroll
                for (int i = 0; i < per; ++i) {
                    const int j = g * per + i;
                    if constexpr (BF && !EXACT) {
                        // the activations' own sum, in every column
                        const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            asum[m] = mfma16<BF>(__builtin_bit_cast(x8, ab.v[m][j]),
                                                 __builtin_bit_cast(x8, one), asum[m]);
                    }
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const x8 f = unpack8<BF, EXACT>(wb.v[r][0][j], wb.z[r][g]);
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            sum[r][m] =
                                mfma16<BF>(__builtin_bit_cast(x8, ab.v[m][j]), f, sum[r][m]);
                    }
                }
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const float sc = to_float<BF>(wb.s[r][g]);
                    const float off = (float)(128u + wb.z[r][g]);
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = sum[r][m][e];
                            if constexpr (BF && !EXACT)
                                v = __builtin_fmaf(-off, asum[m][e], v);
                            acc[r][m][e] = __builtin_fmaf(sc, v, acc[r][m][e]);
                        }
                }
            }
        }
    }

    // The steps first, first + stride, ... below `last`, the next one's loads
    // in flight while one is consumed; `last` is at most ceil(K / 128).  The
    // activations are fetched ahead too where that takes few registers.
    __device__ __forceinline__ void run(int first, int last, int stride)
    {
        constexpr bool kAheadA = MB == 1;
        const int full = min(last, K >> 7);
        WBuf w0, w1;
        ABuf a0, a1;
        int st = first;
        if (st < full) {
            load_a(a0, st);
            load_w(w0, st);
            while (st + 2 * stride < full) {
                if (kAheadA)
                    load_a(a1, st + stride);
                load_w(w1, st + stride);
                consume<false>(w0, a0);
                load_a(a0, st + (kAheadA ? 2 : 1) * stride);
                load_w(w0, st + 2 * stride);
                consume<false>(w1, kAheadA ? a1 : a0);
                if (!kAheadA)
                    load_a(a0, st + 2 * stride);
                st += 2 * stride;
            }
            if (st + stride < full) {
                if (kAheadA)
                    load_a(a1, st + stride);
                load_w(w1, st + stride);
                consume<false>(w0, a0);
                if (!kAheadA)
                    load_a(a0, st + stride);
                consume<false>(w1, kAheadA ? a1 : a0);
                st += 2 * stride;
            } else {
                consume<false>(w0, a0);
                st += stride;
            }
        }
        if (st < last) {          // K % 128 != 0, and its step is this wave's
            load_tail(w0, a0, st);
            consume<false>(w0, a0);
        }
        if constexpr (BF && GS != 0) {
            // An activation that is infinite, or so large that 128 times it
            // overflows, leaves infinity minus infinity where q - z itself
            // would not: such sums, and no others, are formed again with the
            // exact weights.
            bool odd = false;
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        odd |= !finite(acc[r][m][e]);
            if (__any(odd))
                run_exact(first, last, stride);
        }
    }

    static __device__ __forceinline__ bool finite(float v)
    {
        return __builtin_fabsf(v) < __builtin_inff();
    }

    // The weights go in times 2^-12, so that a group's sum of at most 128
    // terms of 15 |A| cannot pass fp32 where A does not.
    __device__ __forceinline__ void run_exact(int first, int last, int stride)
    {
        f32x4 sum[RB][MB];
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                sum[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        WBuf wb;
        ABuf ab;
        for (int st = first; st < last; st += stride) {
            if (st < K >> 7) {
                load_a(ab, st);
                load_w(wb, st);
            } else {
                load_tail(wb, ab, st);
            }
            consume<true>(wb, ab, sum);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!finite(acc[r][m][e]))
                        acc[r][m][e] = sum[r][m][e] * 0x1p12f;
    }
};

// Adds the waves' accumulators of one block of 16 rows m in LDS, in wave order,
// and hands f(m, n, v) the sums v[r] of row m and row n of each weight block r.
// red: waves * RB * 64 vectors.  Every wave of the workgroup calls it.
template <int RB, class F>
__device__ __forceinline__ void reduce_waves(const f32x4 (&acc)[RB], f32x4 *red, int waves, F &&f)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RB; ++r)
        red[(wave * RB + r) * 64 + lane] = acc[r];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
        float v[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const float *p = (const float *)(red + r * 64 + (m >> 2) * 16 + n) + (m & 3);
            v[r] = 0.0f;
            for (int w = 0; w < waves; ++w)
                v[r] += p[w * RB * 256];
        }
        f(m, n, v);
    }
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

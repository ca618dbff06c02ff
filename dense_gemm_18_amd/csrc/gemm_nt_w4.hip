// gemm_nt_w4.hip -- C entry points of the 4-bit weight operators, and the
// kernels that quantise a weight and reverse it.  The product's kernels:
// w4_product.h, skinny.h.
#include "w4_product.h"

namespace {

typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

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

// A lane's place among the words (or units) of an N-row weight, `words` to a
// row, and the step from one to the next of its own: a division at the start
// only.
struct Walk {
    int64_t n;
    int at;

    __device__ __forceinline__ Walk(int words)
    {
        const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
        n = i / words;
        at = (int)(i - n * words);
    }
    __device__ __forceinline__ void next(int words, int64_t rows, int rest)
    {
        n += rows;
        at += rest;
        if (at >= words) {
            at -= words;
            ++n;
        }
    }
};

// rint(x / s) for 16-bit x and s, and `rs` = 1 / s within 1 ulp: x / s is a
// half-integer or at least 2^-12 from one (both have at most 11 bits), and
// fma(x, rs, 768) - 768 puts it on a grid of 2^-14, where the half-integers
// are, less than 2^-18 from where it was.  Three instructions for a
// correctly rounded division's ten and a rint.
__device__ __forceinline__ float nearest(float x, float rs)
{
    return __builtin_rintf(__builtin_fmaf(x, rs, 768.0f) - 768.0f);
}

// Quantisation, 32 consecutive elements of a row per lane: four 16-byte loads,
// four packed words.  Lanes follow K, so a group is one lane or 2 or 4
// neighbours, whose extremes take an exchange or two; a 64-byte block's words
// leave by four lanes together.  2.5 bytes and more per element bound it: 80 us
// for 16384 x 8192 bf16 in groups of 32 with zero points, 4.4 TB/s.  With 8
// elements per lane the group's arithmetic and the addresses, done by every
// lane, were the bound (30 VALU instructions to an element, 115 us), though
// 1024 x 1024 took 3.5 us instead of 4.2.  Elements past the last whole unit
// are loaded when they are worked on: a second branch of `fetch` would wait
// for the first one's loads.
template <bool BF, int GS>
__global__ void __launch_bounds__(256) quantize_kernel(const uint16_t *__restrict__ W,
                                                       uint32_t *__restrict__ Q,
                                                       uint16_t *__restrict__ S,
                                                       uint8_t *__restrict__ Z, int64_t N, int K,
                                                       int64_t ldw, int64_t step_rows,
                                                       int step_rest)
{
    constexpr int kLanes = GS / 32;
    struct Unit {
        u32x4 v[4];
    };
    const int units = ((K + 127) >> 7) * 4, G = (K + GS - 1) / GS;
    // every lane of a group of 4 runs the same number of times: units and the
    // grid's lanes are multiples of 4
    auto fetch = [&](const Walk &w) {
        Unit x = {};
        if (w.n < N && w.at * 32 + 32 <= K) {    // or when it is worked on
            const uint16_t *src = W + w.n * ldw + w.at * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x.v[i] = load16(src + 8 * i);
        }
        return x;
    };
    Walk w(units);
    Unit ahead = fetch(w);
    while (w.n < N) {
        // the next unit's elements are under way while this one's are worked on
        const int64_t n = w.n;
        const int at = w.at, k = at * 32;
        Unit raw = ahead;
        w.next(units, step_rows, step_rest);
        ahead = fetch(w);
        if (k + 32 > K) {
            const uint16_t *src = W + n * ldw + k;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw.v[i] = load16_part(src + 8 * i, K - k - 8 * i);
        }
        // The largest value, at least 0, and the negative one of the largest
        // magnitude, as bits, two at a time: signed 16-bit integers have the one
        // as their maximum, unsigned ones the other (or a number below 2^15
        // where none is negative).  An infinity or a NaN is the largest of either.
        s16x2 up = {0, 0};
        u16x2 down = {0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t pair = raw.v[i >> 2][i & 3];
            up = __builtin_elementwise_max(up, __builtin_bit_cast(s16x2, pair));
            down = __builtin_elementwise_max(down, __builtin_bit_cast(u16x2, pair));
        }
        // over the group's lanes
        auto widest = [](auto v) {
            auto step = [&](auto ctrl) {
                const int moved = __builtin_amdgcn_update_dpp(
                    0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false);
                v = __builtin_elementwise_max(v, __builtin_bit_cast(decltype(v), moved));
            };
            if constexpr (kLanes > 1)
                step(std::integral_constant<int, 0xb1>{});       // lane ^ 1
            if constexpr (kLanes > 2)
                step(std::integral_constant<int, 0x4e>{});       // lane ^ 2
            return (uint16_t)(v[0] > v[1] ? v[0] : v[1]);
        };
        const uint16_t up_bits = widest(up), lowest = widest(down);
        const uint16_t down_bits = lowest & 0x8000 ? lowest & 0x7fff : 0;
        constexpr uint16_t kInf = BF ? 0x7f80 : 0x7c00;
        const bool any = up_bits >= kInf || down_bits >= kInf;
        const float hi = to_float<BF>(up_bits), lo = -to_float<BF>(down_bits);
        const uint16_t bits =
            from_float<BF>(Z ? (hi - lo) / 15.0f : __builtin_fmaxf(hi, -lo) / 7.0f);
        const float s = to_float<BF>(bits);
        const bool live = s > 0.0f && !any;
        const float rs = live ? __builtin_amdgcn_rcpf(s) : 0.0f;
        const bool slow = __any(rs > 0x1p100f);          // 1 / s may have overflowed
        // q is the nearest number between `least` and `most`, plus z: where the
        // group is not live, all of them become z
        float z = 8.0f, least = -8.0f, most = 7.0f;
        if (Z) {
            const float r = slow ? __builtin_rintf(-lo / s) : nearest(-lo, rs);
            z = live ? __builtin_fminf(r, 15.0f) : 8.0f;
            least = -z;
            most = 15.0f - z;
        }
        least = live ? least : 0.0f;
        most = live ? most : 0.0f;
        uint32_t *dst = Q + n * (units * 4) + (at & ~3) * 4 + (at & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            auto x = [&](int e) {
                return to_float<BF>((uint16_t)(raw.v[i][e >> 1] >> (16 * (e & 1))));
            };
            float r[8];
            if (slow) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    r[e] = __builtin_rintf(x(e) / s);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    r[e] = nearest(x(e), rs);
            }
            // the digits of two numbers to the base 16, exact in fp32
            float half[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                half[h] = z * 4369.0f;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    half[h] = __builtin_fmaf(
                        __builtin_amdgcn_fmed3f(r[2 * d + h], least, most),
                        (float)(1 << (4 * d)), half[h]);
            }
            uint32_t word = (uint32_t)half[0] | (uint32_t)half[1] << 16;
            if (k + 8 * i + 8 > K) {             // bits past the row's end are 0
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + 8 * i + e >= K)
                        word &= ~(15u << (4 * (e >> 1) + 16 * (e & 1)));
            }
            dst[4 * i] = word;
        }
        if (at % kLanes == 0 && k < K) {
            const int64_t g = n * G + k / GS;
            S[g] = any ? (BF ? 0x7fc0 : 0x7e00) : bits;
            if (Z)
                Z[g] = (uint8_t)z;
        }
    }
}

// The reverse: one packed word, eight elements per lane.  Bound by writing:
// 66 us for 16384 x 8192 bf16 in groups of 32, 5.4 TB/s in all.
template <bool BF, int GS>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint32_t *__restrict__ Q,
                                                         const uint16_t *__restrict__ S,
                                                         const uint8_t *__restrict__ Z,
                                                         uint16_t *__restrict__ W, int64_t N,
                                                         int K, int64_t ldw, int64_t step_rows,
                                                         int step_rest)
{
    const int words = ((K + 127) >> 7) * 16, G = (K + GS - 1) / GS;
    for (Walk w(words); w.n < N; w.next(words, step_rows, step_rest)) {
        const int64_t n = w.n;
        const int at = w.at, k = at * 8;
        if (k >= K)
            continue;
        const int j = (at >> 2) & 3, c = at & 3;
        const uint32_t word = Q[n * words + (at & ~15) + 4 * c + j];
        const int64_t g = n * G + k / GS;
        const float s = to_float<BF>(S[g]);
        const float z = Z ? (float)(Z[g] & 15) : 8.0f;
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = (float)((word >> (4 * (e >> 1) + 16 * (e & 1))) & 15u);
            v[e >> 1] |= (uint32_t)from_float<BF>((q - z) * s) << (16 * (e & 1));
        }
        uint16_t *dst = W + n * ldw + k;
        if (k + 8 <= K) {
            *(u32x4_a2 *)dst = v;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (k + e < K)
                    dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
    }
}

constexpr int64_t kMaxLd = int64_t(1) << 40;

uint64_t packed_bytes(int64_t N, int64_t K) { return (uint64_t)N * (uint64_t)cdiv(K, 128) * 64u; }

// Bytes that rows of `cols` elements `ld` apart span.
uint64_t span_bytes(int64_t rows, int64_t cols, int64_t ld)
{
    return rows && cols ? ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * 2u : 0u;
}

// The checks every entry point shares: sizes, group, type, and the packed
// weight's pointers.
bool weight_ok(const void *Q, const void *S, int64_t N, int64_t K, int group, int dtype)
{
    if (!sizes_ok(0, N, K) || !group_ok(group) || !dtype_ok(dtype))
        return false;
    if (N && K && (!Q || !S))
        return false;
    return aligned_to(Q, 16) && aligned_to(S, 2);
}

template <class F>
void for_type(int dtype, F &&f)
{
    if (dtype == GEMM_T_BF16)
        f(std::true_type{});
    else
        f(std::false_type{});
}

// Workgroups of 256 lanes for `lanes` of them, up to 32 per CU.
unsigned lane_grid(int64_t lanes)
{
    const int64_t wgs = cdiv(lanes, 256);
    return (unsigned)(wgs < 8192 ? wgs : 8192);
}

// Shared by the two directions; W is written where dequantize is set.
int convert(const void *W, const void *Q, const void *S, const void *Z, int64_t N, int64_t K,
            int64_t ldw, int group, int dtype, bool dequantize, hipStream_t stream)
{
    if (!weight_ok(Q, S, N, K, group, dtype) || ldw < K || ldw > kMaxLd)
        return GEMM_EINVAL;
    if ((N && K && !W) || !aligned_to(W, 2))
        return GEMM_EINVAL;
    const uint64_t groups = (uint64_t)N * (uint64_t)cdiv(K, group);
    const struct { const void *p; uint64_t n; bool out; } part[4] = {
        {W, span_bytes(N, K, ldw), dequantize},
        {Q, packed_bytes(N, K), !dequantize},
        {S, groups * 2u, !dequantize},
        {Z, Z ? groups : 0u, !dequantize}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if ((part[i].out || part[j].out) &&
                overlap(part[i].p, part[i].n, part[j].p, part[j].n))
                return GEMM_EINVAL;
    if (N == 0 || K == 0)
        return GEMM_OK;
    // a lane has one word, or the four that it quantises
    const int64_t words = cdiv(K, 128) * (dequantize ? 16 : 4);
    const dim3 grid(lane_grid(N * words));
    const int64_t stride = (int64_t)grid.x * 256;
    const int64_t step_rows = stride / words;
    const int step_rest = (int)(stride % words);
    for_type(dtype, [&](auto bf) {
        with_group(group, [&](auto gs) {
            constexpr bool BF = decltype(bf)::value;
            constexpr int GS = decltype(gs)::value ? decltype(gs)::value : 128;
            if (dequantize)
                hipLaunchKernelGGL((dequantize_kernel<BF, GS>), grid, dim3(256), 0, stream,
                                   (const uint32_t *)Q, (const uint16_t *)S, (const uint8_t *)Z,
                                   (uint16_t *)W, N, (int)K, ldw, step_rows, step_rest);
            else
                hipLaunchKernelGGL((quantize_kernel<BF, GS>), grid, dim3(256), 0, stream,
                                   (const uint16_t *)W, (uint32_t *)Q, (uint16_t *)S,
                                   (uint8_t *)Z, N, (int)K, ldw, step_rows, step_rest);
        });
    });
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

// Zeroes the N columns of M rows `ldd` apart (the empty sum).
__global__ void zero_rows_kernel(uint16_t *__restrict__ D, int64_t M, int64_t N, int64_t ldd)
{
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < M * N;
         i += (int64_t)gridDim.x * 256)
        D[i / N * ldd + i % N] = 0;
}

} // namespace

extern "C" {

int64_t gemm_w4_packed_bytes(int64_t N, int64_t K)
{
    return sizes_ok(0, N, K) ? (int64_t)packed_bytes(N, K) : 0;
}

int gemm_w4_quantize(const void *W, void *Q, void *S, void *Z, int64_t N, int64_t K, int64_t ldw,
                     int group, int dtype, hipStream_t stream)
{
    return convert(W, Q, S, Z, N, K, ldw, group, dtype, false, stream);
}

int gemm_w4_dequantize(const void *Q, const void *S, const void *Z, void *W, int64_t N, int64_t K,
                       int64_t ldw, int group, int dtype, hipStream_t stream)
{
    return convert(W, Q, S, Z, N, K, ldw, group, dtype, true, stream);
}

int64_t gemm_nt_w4_ws_size(int64_t M, int64_t N, int64_t K)
{
    if (!sizes_ok(M, N, K) || M <= GEMM_W4_DIRECT_M || N == 0)
        return 0;
    return cdiv(N * K * 2, 256) * 256;
}

int gemm_nt_w4(const void *A, const void *Q, const void *S, const void *Z, void *D, int64_t M,
               int64_t N, int64_t K, int64_t lda, int64_t ldd, int group, int dtype,
               void *workspace, int64_t ws_bytes, hipStream_t stream)
{
    if (!sizes_ok(M, N, K) || !weight_ok(Q, S, N, K, group, dtype))
        return GEMM_EINVAL;
    if (lda < K || lda > GEMM_W4_MAX_LDA || ldd < N || ldd > kMaxLd || ws_bytes < 0)
        return GEMM_EINVAL;
    if ((M && K && !A) || (M && N && !D) || !aligned_to(A, 2) || !aligned_to(D, 2))
        return GEMM_EINVAL;
    if (ws_bytes && (!workspace || !aligned_to(workspace, 256)))
        return GEMM_EINVAL;
    const uint64_t d_bytes = span_bytes(M, N, ldd);
    const uint64_t groups = (uint64_t)N * (uint64_t)cdiv(K, group);
    const struct { const void *p; uint64_t n; } in[4] = {{A, span_bytes(M, K, lda)},
                                                         {Q, packed_bytes(N, K)},
                                                         {S, groups * 2u},
                                                         {Z, Z ? groups : 0u}};
    for (const auto &x : in)
        if (overlap(D, d_bytes, x.p, x.n) || overlap(workspace, (uint64_t)ws_bytes, x.p, x.n))
            return GEMM_EINVAL;
    if (overlap(D, d_bytes, workspace, (uint64_t)ws_bytes))
        return GEMM_EINVAL;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if (K == 0) {
        const int64_t wgs = cdiv(M * N, 256);
        hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256),
                           0, stream, (uint16_t *)D, M, N, ldd);
        return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
    }
    const int64_t need = gemm_nt_w4_ws_size(M, N, K);
    if (need && ws_bytes >= need && lda == K && ldd == N) {
        // one more rounding of the weights, to the type that the 16-bit product's
        // matrix instructions take, and the weight unpacked once instead of for
        // every 64 rows
        const std::lock_guard<std::mutex> both(launch_lock(workspace));
        const int rc = gemm_w4_dequantize(Q, S, Z, workspace, N, K, K, group, dtype, stream);
        if (rc != GEMM_OK)
            return rc;
        return dtype == GEMM_T_BF16 ? gemm_nt_bf16(A, workspace, D, M, N, K, stream)
                                    : gemm_nt_f16(A, workspace, D, M, N, K, stream);
    }
    W4Args a{};
    a.A = (const uint16_t *)A;
    a.W.q = (const uint32_t *)Q;
    a.W.s = (const uint16_t *)S;
    a.W.z = (const uint8_t *)Z;
    a.D = (uint16_t *)D;
    a.lda = lda;
    a.ldd = ldd;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    if (dtype == GEMM_T_BF16)
        gemm18_w4_bf16(a, group, stream);
    else
        gemm18_w4_f16(a, group, stream);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

} // extern "C"

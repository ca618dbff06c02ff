// rms_norm.hip -- the root-mean-square norm with the residual's addition, into 16
// bits or into FP8 operands: kernels and C entry points.
#include "rms_norm.h"
#include "skinny.h"

namespace {

// 16 and 8 bytes at any alignment that their elements have (one global access each).
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

struct NormArgs {
    const uint16_t *X, *R, *W;
    void *Y;                   // 16-bit elements or FP8 bytes
    uint16_t *S;
    float *scales;
    int64_t T, ldx, ldr, ldy, lds;
    int H;
    float eps, scale;          // scale: where there are no scales
};

// The first `count` of the 8 elements at p, zero for the others; nothing past them is
// accessed.
__device__ __forceinline__ u32x4 load_eight(const uint16_t *p, int count)
{
    if (count >= 8)
        return *(const u32x4_a2 *)p;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < count)
            v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
}

template <bool BF>
__device__ __forceinline__ float element(const u32x4 &v, int e)
{
    return to_float<BF>((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
}

template <bool BF>
__device__ __forceinline__ void store_eight(uint16_t *p, const float (&v)[8], int count)
{
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = from_float<BF>(v[2 * i]) | (uint32_t)from_float<BF>(v[2 * i + 1]) << 16;
    if (count >= 8) {
        *(u32x4_a2 *)p = u;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < count)
            p[i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
}

// Largest numbers of the two formats.
template <int FP8>
constexpr float kMost = FP8 == GEMM_FP8_E5M2 ? 57344.0f : 448.0f;

// Eight FP8 bytes of v, each held within the format's range first (a NaN stays one).
template <int FP8>
__device__ __forceinline__ u32x2 eight_bits(const float (&v)[8])
{
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = v[i] > kMost<FP8> ? kMost<FP8> : v[i];
        c[i] = c[i] < -kMost<FP8> ? -kMost<FP8> : c[i];
    }
    u32x2 u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = 0;
        if constexpr (FP8 == GEMM_FP8_E5M2) {
            w = __builtin_amdgcn_cvt_pk_bf8_f32(c[4 * i], c[4 * i + 1], w, false);
            w = __builtin_amdgcn_cvt_pk_bf8_f32(c[4 * i + 2], c[4 * i + 3], w, true);
        } else {
            w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], w, true);
        }
        u[i] = (uint32_t)w;
    }
    return u;
}

__device__ __forceinline__ void store_bytes(uint8_t *p, u32x2 u, int count)
{
    if (count >= 8) {
        *(u32x2_a1 *)p = u;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < count)
            p[i] = (uint8_t)(u[i >> 2] >> (8 * (i & 3)));
}

// f over the W waves of a row, in the same order in each of them.  `red`: W floats of LDS,
// others than the last reduction's.
template <int W, class F>
__device__ __forceinline__ float over_row(float v, float *red, F &&f)
{
#pragma unroll
    for (int d = 32; d; d /= 2)
        v = f(v, __shfl_xor(v, d));
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v = f(v, red[w]);
    }
    return v;
}

// The larger magnitude; anything that is not finite counts as infinite.
__device__ __forceinline__ float wider(float most, float v)
{
    const float a = __builtin_fabsf(v);
    return __builtin_fmaxf(most, a < __builtin_inff() ? a : __builtin_inff());
}

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }

// What a row is multiplied by first, and eps by its square, where the sum of squares leaves
// fp32's range: 2^22 squares of 2^128 times 2^-80 are in it, and so are, times 2^80, those of
// the smallest numbers there are.  Where the mean and eps are above 2^-120, squares that vanish,
// 2^-150 each, do not count.
__device__ __forceinline__ float range_of(float sum, int H, float eps)
{
    return sum == __builtin_inff() ? 0x1p-80f : sum / (float)H + eps < 0x1p-120f ? 0x1p80f : 1.0f;
}
// What s is multiplied by.
__device__ __forceinline__ float inverse(float sum, int H, float eps)
{
    return 1.0f / __builtin_sqrtf(sum / (float)H + eps);
}

// A row's scale by its largest |y|, and what y is multiplied by to get q.  1 / scale
// passes fp32's range where scale is below 2^-127: `slow`, divide.
struct Scale {
    float scale, by;
    bool slow;
};
template <int FP8>
__device__ __forceinline__ Scale scale_of(float most)
{
    Scale s;
    s.scale = most / kMost<FP8>;
    const bool live = s.scale > 0.0f && s.scale < __builtin_inff();
    s.slow = live && s.scale < 0x1p-100f;
    s.by = live && !s.slow ? 1.0f / s.scale : 0.0f;
    s.scale = most < __builtin_inff() ? s.scale : __builtin_nanf("");
    return s;
}

__device__ __forceinline__ Scale given_scale(float scale)
{
    const bool slow = scale < 0x1p-100f;
    return {scale, slow ? 0.0f : 1.0f / scale, slow};
}

template <int FP8>
__device__ __forceinline__ u32x2 scaled_bits(const float (&y)[8], const Scale &s)
{
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        q[e] = s.slow ? y[e] / s.scale : s.by == 0.0f ? 0.0f : y[e] * s.by;
    return eight_bits<FP8>(q);
}

// A row in the registers of W waves, V times 8 elements to a lane: one pass over memory, which
// bounds it.  FP8: the format, or -1 for 16-bit rows.
template <bool BF, int FP8, int W, int V>
__global__ void __launch_bounds__(W == 1 ? 256 : W * 64) rms_norm_kernel(NormArgs p)
{
    __shared__ float red[3][W];
    const int64_t wg = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t t = W == 1 ? wg * 4 + (threadIdx.x >> 6) : wg;
    if (t >= p.T)
        return;
    const int at = (W == 1 ? threadIdx.x & 63 : threadIdx.x) * 8;
    u32x4 x[V], r[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int k = at + i * W * 512;
        x[i] = load_eight(p.X + t * p.ldx + k, p.H - k);
        r[i] = p.R ? load_eight(p.R + t * p.ldr + k, p.H - k) : u32x4{0, 0, 0, 0};
        w[i] = p.W ? load_eight(p.W + k, p.H - k) : u32x4{0, 0, 0, 0};
    }
    float s[V][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[i][e] = element<BF>(x[i], e);
            if (p.R)
                s[i][e] += element<BF>(r[i], e);
            sum = __builtin_fmaf(s[i][e], s[i][e], sum);
        }
        const int k = at + i * W * 512;
        if (p.S)
            store_eight<BF>(p.S + t * p.lds + k, s[i], p.H - k);
    }
    sum = over_row<W>(sum, red[0], plus);
    float eps = p.eps;
    const float range = range_of(sum, p.H, eps);
    if (range != 1.0f) {
        sum = 0.0f;
        eps = eps * range * range;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[i][e] *= range;
                sum = __builtin_fmaf(s[i][e], s[i][e], sum);
            }
        sum = over_row<W>(sum, red[1], plus);
    }
    const float by = inverse(sum, p.H, eps);
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[i][e] *= by;
            if (p.W)
                s[i][e] *= element<BF>(w[i], e);
            if constexpr (FP8 >= 0)
                most = wider(most, s[i][e]);
        }
    }
    if constexpr (FP8 < 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = at + i * W * 512;
            store_eight<BF>((uint16_t *)p.Y + t * p.ldy + k, s[i], p.H - k);
        }
    } else {
        Scale q;
        if (p.scales) {
            q = scale_of<FP8>(over_row<W>(most, red[2], larger));
            if (at == 0)
                p.scales[t] = q.scale;
        } else {
            q = given_scale(p.scale);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = at + i * W * 512;
            store_bytes((uint8_t *)p.Y + t * p.ldy + k, scaled_bits<FP8>(s[i], q), p.H - k);
        }
    }
}

// Rows of any length, by 16 waves: over the squares, over |y| where scales are wanted,
// and to write, each pass reading the row again (out of the caches: 4096 rows of 40960 take
// 343 us, 3.4 TB/s).
template <bool BF, int FP8>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(NormArgs p)
{
    __shared__ float red[3][16];
    const int64_t t = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    if (t >= p.T)
        return;
    const int at = threadIdx.x * 8;
    auto row = [&](int k, float(&s)[8]) G18_INLINE {
        const u32x4 x = load_eight(p.X + t * p.ldx + k, p.H - k);
        const u32x4 r = p.R ? load_eight(p.R + t * p.ldr + k, p.H - k) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = element<BF>(x, e);
            if (p.R)
                s[e] += element<BF>(r, e);
        }
    };
    auto squares = [&](float range) G18_INLINE {
        float sum = 0.0f, s[8];
        for (int k = at; k < p.H; k += 8192) {
            row(k, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(s[e] * range, s[e] * range, sum);
        }
        return sum;
    };
    float eps = p.eps;
    float sum = over_row<16>(squares(1.0f), red[0], plus);
    const float range = range_of(sum, p.H, eps);
    if (range != 1.0f) {
        eps = eps * range * range;
        sum = over_row<16>(squares(range), red[1], plus);
    }
    const float by = inverse(sum, p.H, eps);
    auto normed = [&](int k, const float(&s)[8], float(&y)[8]) G18_INLINE {
        const u32x4 w = p.W ? load_eight(p.W + k, p.H - k) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = s[e] * range * by;
            if (p.W)
                y[e] *= element<BF>(w, e);
        }
    };
    float s[8], y[8];
    [[maybe_unused]] Scale q{p.scale, 0.0f, false};
    if constexpr (FP8 >= 0) {
        if (p.scales) {
            float most = 0.0f;
            for (int k = at; k < p.H; k += 8192) {
                row(k, s);
                normed(k, s, y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    most = wider(most, y[e]);
            }
            q = scale_of<FP8>(over_row<16>(most, red[2], larger));
            if (at == 0)
                p.scales[t] = q.scale;
        } else {
            q = given_scale(p.scale);
        }
    }
    for (int k = at; k < p.H; k += 8192) {
        row(k, s);
        normed(k, s, y);
        if (p.S)
            store_eight<BF>(p.S + t * p.lds + k, s, p.H - k);
        if constexpr (FP8 < 0)
            store_eight<BF>((uint16_t *)p.Y + t * p.ldy + k, y, p.H - k);
        else
            store_bytes((uint8_t *)p.Y + t * p.ldy + k, scaled_bits<FP8>(y, q), p.H - k);
    }
}

// ---- host ----

// A grid dimension holds at most 2^32 - 1 work-items.
inline dim3 row_grid(int64_t wgs)
{
    constexpr int64_t kMaxX = int64_t(1) << 21;
    return wgs <= kMaxX ? dim3((unsigned)wgs) : dim3((unsigned)kMaxX, (unsigned)cdiv(wgs, kMaxX));
}

template <bool BF, int FP8, int W, int V>
void launch_rows(const NormArgs &p, hipStream_t stream)
{
    hipLaunchKernelGGL((rms_norm_kernel<BF, FP8, W, V>), row_grid(W == 1 ? cdiv(p.T, 4) : p.T),
                       dim3(W == 1 ? 256 : W * 64), 0, stream, p);
}

// Waves to a row: with few rows a lane has few elements, with many a row few waves, as little
// waits for the others then.  In us (residual, weights, E4M3 rows with scales; waves x eights of
// a lane):
//   row                 1024              2048              4096              8192
//   256 rows    4x1 3.8 1x2 4.2   4x1 4.0 1x4 6.0   4x2 5.1 16x1 5.9   16x1 7.4 4x4 7.8
//   512         4x1 4.3 1x2 4.4   4x1 4.8 1x4 6.2   4x2 6.8 16x1 9.1  16x1 11.3 4x4 10.9
//   2048        4x1 8.8 1x2 6.6  4x1 10.8 1x4 10.9  4x2 15.1 4x4 19.6 16x1 30.8 4x4 27.5
//   16384      4x1 40.3 1x2 24.8 4x1 46.3 1x4 45.4  4x2 81.5 4x4 91.4  16x1 196 4x4 163
// one row of 16384 16x2 5.6, three passes 7.3; 2048 rows of 32768 16x4 112, three passes 144.
// 16384 rows of 8192 move 939 MB, 5.8 TB/s: more than a copy of 1 GiB (5.1).
template <bool BF, int FP8>
void launch_norm(const NormArgs &p, hipStream_t stream)
{
    const bool few = p.T <= kCUs;
    if (p.H <= 512)
        launch_rows<BF, FP8, 1, 1>(p, stream);
    else if (p.H <= 1024 && !few)
        launch_rows<BF, FP8, 1, 2>(p, stream);
    else if (p.H <= 2048)
        launch_rows<BF, FP8, 4, 1>(p, stream);
    else if (p.H <= 4096)
        launch_rows<BF, FP8, 4, 2>(p, stream);
    else if (p.H <= 8192 && !few)
        launch_rows<BF, FP8, 4, 4>(p, stream);
    else if (p.H <= 8192)
        launch_rows<BF, FP8, 16, 1>(p, stream);
    else if (p.H <= 16384)
        launch_rows<BF, FP8, 16, 2>(p, stream);
    else if (p.H <= 32768)
        launch_rows<BF, FP8, 16, 4>(p, stream);
    else
        hipLaunchKernelGGL((rms_norm_long_kernel<BF, FP8>), row_grid(p.T), dim3(1024), 0, stream,
                           p);
}

constexpr int64_t kMaxLd = int64_t(1) << 40;

// Bytes that T rows of H elements `ld` apart span.
uint64_t span_bytes(int64_t T, int64_t H, int64_t ld, int size)
{
    return ((uint64_t)(T - 1) * (uint64_t)ld + (uint64_t)H) * (uint64_t)size;
}

// Shared by both entry points; `format` -1: 16-bit rows.
int norm_call(const void *X, const void *R, const void *W, void *Y, float *scales, void *S,
              int64_t T, int64_t H, int64_t ldx, int64_t ldr, int64_t ldy, int64_t lds, float eps,
              float scale, int format, int dtype, hipStream_t stream)
{
    if (T < 0 || T > INT32_MAX || H < 1 || H > GEMM_MAX_K || !dtype_ok(dtype) ||
        !(eps >= 0.0f && eps < __builtin_inff()))
        return GEMM_EINVAL;
    if (ldx < H || ldy < H || (R && ldr < H) || (S && lds < H) || ldx > kMaxLd || ldy > kMaxLd ||
        (R && ldr > kMaxLd) || (S && lds > kMaxLd))
        return GEMM_EINVAL;
    if (T == 0)
        return GEMM_OK;
    if (S && !R)
        return GEMM_EINVAL;
    if (format >= 0 && !scales && !(scale > 0.0f && scale < __builtin_inff()))
        return GEMM_EINVAL;
    const bool wide = format < 0;
    if (!X || !Y || !aligned_to(X, 2) || !aligned_to(R, 2) || !aligned_to(W, 2) ||
        !aligned_to(S, 2) || !aligned_to(Y, wide ? 2 : 1) || !aligned_to(scales, 4))
        return GEMM_EINVAL;
    struct Part {
        const void *p;
        int64_t ld;
        uint64_t n;
        bool out, row;             // row: of the 16-bit rows that may be one and the same
    } part[6] = {{X, ldx, span_bytes(T, H, ldx, 2), false, true},
                 {R, ldr, R ? span_bytes(T, H, ldr, 2) : 0, false, true},
                 {W, 0, W ? (uint64_t)H * 2u : 0, false, false},
                 {Y, ldy, span_bytes(T, H, ldy, wide ? 2 : 1), true, wide},
                 {S, lds, S ? span_bytes(T, H, lds, 2) : 0, true, true},
                 {scales, 0, scales ? (uint64_t)T * 4u : 0, true, false}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j) {
            const bool same = part[i].p == part[j].p && part[i].ld == part[j].ld &&
                              part[i].row && part[j].row && !(part[i].out && part[j].out);
            if ((part[i].out || part[j].out) && !same &&
                overlap(part[i].p, part[i].n, part[j].p, part[j].n))
                return GEMM_EINVAL;
        }
    NormArgs p{};
    p.X = (const uint16_t *)X;
    p.R = (const uint16_t *)R;
    p.W = (const uint16_t *)W;
    p.Y = Y;
    p.S = (uint16_t *)S;
    p.scales = scales;
    p.T = T;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldy = ldy;
    p.lds = lds;
    p.H = (int)H;
    p.eps = eps;
    p.scale = scale;
    auto go = [&](auto bf) {
        constexpr bool BF = decltype(bf)::value;
        if (format < 0)
            launch_norm<BF, -1>(p, stream);
        else if (format == GEMM_FP8_E4M3)
            launch_norm<BF, GEMM_FP8_E4M3>(p, stream);
        else
            launch_norm<BF, GEMM_FP8_E5M2>(p, stream);
    };
    if (dtype == GEMM_T_BF16)
        go(std::true_type{});
    else
        go(std::false_type{});
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

} // namespace

extern "C" {

int rms_norm(const void *X, const void *R, const void *W, void *Y, void *S, int64_t T, int64_t H,
             int64_t ldx, int64_t ldr, int64_t ldy, int64_t lds, float eps, int dtype,
             hipStream_t stream)
{
    return norm_call(X, R, W, Y, nullptr, S, T, H, ldx, ldr, ldy, lds, eps, 1.0f, -1, dtype,
                     stream);
}

int rms_norm_fp8(const void *X, const void *R, const void *W, void *Q, float *scales, void *S,
                 int64_t T, int64_t H, int64_t ldx, int64_t ldr, int64_t ldq, int64_t lds,
                 float eps, float scale, int format, int dtype, hipStream_t stream)
{
    if (format != GEMM_FP8_E4M3 && format != GEMM_FP8_E5M2)
        return GEMM_EINVAL;
    return norm_call(X, R, W, Q, scales, S, T, H, ldx, ldr, ldq, lds, eps, scale, format, dtype,
                     stream);
}

} // extern "C"

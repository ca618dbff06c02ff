// lora_nt.hip -- C entry points of the low-rank adapters beside a shared projection.
// Kernels: lora.h, w4_product.h, skinny.h, and the dense products'.
#include "gemm_add.h"
#include "lora.h"

namespace {

constexpr int64_t kMaxLd = int64_t(1) << 40;

bool sizes_ok_lora(int64_t M, int64_t N, int64_t K, int64_t rank, int group)
{
    return sizes_ok(M, N, K) && rank >= 1 && rank <= LORA_MAX_RANK &&
           (group == 0 || group_ok(group));
}

uint64_t span_bytes(int64_t rows, int64_t cols, int64_t ld)
{
    return rows && cols ? ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * 2u : 0u;
}

int64_t up256(int64_t n) { return cdiv(n, 256) * 256; }

// Whether a call with dense rows goes through the large tiles of the dense products: u, then
// the adapters' part into D, then the product added to it.  Packed weights: where they are
// unpacked anyway.  16-bit weights: where the tiles for few rows are not the better ones,
// which take one pass and one launch, but read the activations once for every 16 or 32
// columns.  Measured with 32 adapters of rank 16, tiles for few rows / large, in us:
//   columns                     2048          4096          8192         16384
//   K 4096   1 row         8.0 / 16.5    9.9 / 17.3   15.0 / 19.0   24.5 / 31.4
//            8             9.2 / 16.7   11.1 / 17.5   16.1 / 19.2   26.6 / 32.0
//           16            11.1 / 16.9   13.6 / 17.6   20.0 / 19.6   36.5 / 33.2
//           32            17.4 / 18.2   20.4 / 19.3   27.1 / 21.7   45.5 / 36.1
//           64            17.5 / 20.3   23.0 / 22.5   42.5 / 25.9   82.1 / 39.4
//          128            19.9 / 25.9   30.8 / 29.3   81.6 / 35.7  145.8 / 63.9
//   K 2048  32 rows                                   17.0 / 16.3   24.8 / 24.1
//   K 1024  32 rows                                    9.8 / 13.2   15.0 / 17.2
//   K 8192   1 row        11.8 / 25.3   15.3 / 25.9   24.8 / 30.3   46.0 / 53.9
//            8            15.2 / 25.5   20.4 / 26.2   33.2 / 30.7   58.7 / 55.4
//           16            19.5 / 25.7   27.2 / 26.5   39.7 / 31.2   65.6 / 57.3
//           32            30.2 / 27.8   36.1 / 28.5   48.9 / 33.3   76.5 / 61.2
//           64            30.8 / 33.2   38.6 / 34.2   72.1 / 40.6  135.8 / 64.2
// Up to 16 rows it is whether LDS holds the activations whole that tells them apart.
bool large(int64_t M, int64_t N, int64_t K, int group)
{
    if (group)
        return M > GEMM_W4_DIRECT_M;
    if (M <= 16)
        return N > 16 * kCUs && M * (cdiv(K, 128) * 256 + 16) > kActBytes;
    if (M <= 32 && K <= 2048)
        return false;
    return N > 8 * kCUs || cdiv(M, 32) * cdiv(N, 32) > kCUs;
}

// D = +0 (K == 0).
__global__ void zero_d_kernel(uint16_t *__restrict__ D, int64_t M, int64_t N, int64_t ldd)
{
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < M * N;
         i += (int64_t)gridDim.x * 256)
        D[i / N * ldd + i % N] = 0;
}

} // namespace

extern "C" {

int64_t gemm_nt_lora_ws_size(int64_t M, int64_t N, int64_t K, int64_t rank, int group)
{
    if (!sizes_ok_lora(M, N, K, rank, group) || M == 0 || N == 0 || K == 0)
        return 0;
    int64_t bytes = up256(lora_parts(M, K, rank) * M * rank * 4);
    if (group && large(M, N, K, group))
        bytes += up256(N * K * 2);
    return bytes;
}

int gemm_nt_lora(const void *X, const void *W, const void *S, const void *Z,
                 const lora_nt_adapters *a, const int32_t *ids, void *D, int64_t M, int64_t N,
                 int64_t K, int64_t ldx, int64_t ldd, int group, int dtype, void *workspace,
                 int64_t ws_bytes, hipStream_t stream)
{
    if (!a || !sizes_ok_lora(M, N, K, a->rank, group) || a->count < 0 || a->count > INT32_MAX ||
        !dtype_ok(dtype) || ldx < K || ldx > LORA_MAX_LDX || ldd < N || ldd > kMaxLd ||
        ws_bytes < 0)
        return GEMM_EINVAL;
    if (M == 0 || N == 0)
        return GEMM_OK;
    const uint64_t count = (uint64_t)a->count, rank = (uint64_t)a->rank;
    const uint64_t w_bytes = group ? (uint64_t)N * (uint64_t)cdiv(K, 128) * 64u
                                   : (uint64_t)N * (uint64_t)K * 2u;
    const uint64_t groups = group ? (uint64_t)N * (uint64_t)cdiv(K, group) : 0u;
    const uint64_t d_bytes = span_bytes(M, N, ldd);
    const struct { const void *p; uint64_t n; bool need; uintptr_t align; } in[] = {
        {X, span_bytes(M, K, ldx), true, 2}, {W, w_bytes, true, group ? 16u : 2u},
        {S, groups * 2u, true, 2},           {Z, Z ? groups : 0u, false, 1},
        {a->A, count * rank * (uint64_t)K * 2u, true, 2},
        {a->B, count * rank * (uint64_t)N * 2u, true, 2},
        {a->s, a->s ? count * 4u : 0u, false, 4},
        {ids, (uint64_t)M * 4u, true, 4}};
    for (const auto &x : in)
        if ((x.need && x.n && !x.p) || !aligned_to(x.p, x.align))
            return GEMM_EINVAL;
    const int64_t need = gemm_nt_lora_ws_size(M, N, K, a->rank, group);
    if (!D || !aligned_to(D, 2) || ws_bytes < need ||
        (ws_bytes && (!workspace || !aligned_to(workspace, 256))))
        return GEMM_EINVAL;
    for (const auto &x : in)
        if (overlap(D, d_bytes, x.p, x.n) || overlap(workspace, (uint64_t)ws_bytes, x.p, x.n))
            return GEMM_EINVAL;
    if (overlap(D, d_bytes, workspace, (uint64_t)ws_bytes))
        return GEMM_EINVAL;
    if (K == 0) {
        const int64_t wgs = cdiv(M * N, 256);
        hipLaunchKernelGGL(zero_d_kernel, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0,
                           stream, (uint16_t *)D, M, N, ldd);
        return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
    }
    LoraArgs p{};
    p.X = (const uint16_t *)X;
    p.A = (const uint16_t *)a->A;
    p.B = (const uint16_t *)a->B;
    p.s = a->s;
    p.ids = ids;
    p.u = (float *)workspace;
    p.D = (uint16_t *)D;
    p.ldx = ldx;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.rank = (int)a->rank;
    p.count = (int)a->count;
    p.parts = 1;
    if (p.count)
        p = lora_shared(p);
    const bool bf = dtype == GEMM_T_BF16;
    const LoraLaunch go = bf ? gemm18_lora_bf16() : gemm18_lora_f16();
    const std::lock_guard<std::mutex> whole(launch_lock(workspace));
    if (p.count)
        go.shrink(p, stream);
    if (ldx == K && ldd == N && large(M, N, K, group)) {
        const void *weight = W;
        if (group) {
            void *unpacked = (char *)workspace + up256(lora_parts(M, K, a->rank) * M * a->rank * 4);
            const int rc =
                gemm_w4_dequantize(W, S, Z, unpacked, N, K, K, group, dtype, stream);
            if (rc != GEMM_OK)
                return rc;
            weight = unpacked;
        }
        go.expand(p, stream);
        (bf ? gemm18_add_bf16 : gemm18_add_f16)(X, weight, D, p.M, p.N, p.K, stream);
    } else {
        W4Args w{};
        w.A = (const uint16_t *)X;
        if (group) {
            w.W.q = (const uint32_t *)W;
            w.W.s = (const uint16_t *)S;
            w.W.z = (const uint8_t *)Z;
        } else {
            w.W.w = (const uint16_t *)W;
        }
        w.D = (uint16_t *)D;
        w.lda = ldx;
        w.ldd = ldd;
        w.M = p.M;
        w.N = p.N;
        w.K = p.K;
        go.fused(p, w, group, stream);
    }
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ELAUNCH;
}

} // extern "C"

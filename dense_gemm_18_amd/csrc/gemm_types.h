// gemm_types.h -- element and vector types, the 16 x 16 x 32 matrix
// instruction and the small host helpers that every translation unit of the
// library shares.  Everything here has internal linkage.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_nt_f16.h"

// Kernel-local lambdas must always inline: an out-of-line call would keep
// every array they capture by reference in scratch memory.
#define G18_INLINE __attribute__((always_inline))

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Element type of A, B and D: fp16, or bfloat16 (BF).  Both are 2 bytes,
// so loads, LDS layout and swizzle are shared; the MFMA, the fragment vector
// type and the fp32 -> storage conversion (round to nearest even) differ.
template <bool BF>
struct Elem {
    using T = _Float16;
    using x8 = f16x8;
    using x4 = f16x4;
};
template <>
struct Elem<true> {
    using T = __bf16;
    using x8 = bf16x8;
    using x4 = bf16x4;
};
template <class T>
struct Vec4 {
    using type = f16x4;
};
template <>
struct Vec4<__bf16> {
    using type = bf16x4;
};

template <bool BF>
__device__ __forceinline__ f32x4 mfma16(typename Elem<BF>::x8 b, typename Elem<BF>::x8 a, f32x4 c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, c, 0, 0, 0);
}

// Compile-time loop: f(integral_constant<int, I>) for I = B .. E-1, so that
// register arrays are only ever indexed by constants.
template <int B, int E, class F>
__device__ __forceinline__ void static_for(F &&f)
{
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

constexpr uint32_t kOob = 0x80000000u;   // a buffer offset past every range
constexpr int kRsrcFlags = 0x00020000;   // gfx9 buffer descriptor word 3

// ---- host ----

constexpr int kCUs = 256;          // of an MI355X

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Sizes every entry point accepts: M, N in [0, 2^31 - 1], K in [0, GEMM_MAX_K].
inline bool sizes_ok(int64_t M, int64_t N, int64_t K)
{
    return M >= 0 && N >= 0 && K >= 0 && M <= INT32_MAX && N <= INT32_MAX && K <= GEMM_MAX_K;
}

// Grid of a one-tile-per-workgroup launch: at least `tiles` workgroups.  A
// grid dimension holds at most 2^32 - 1 work-items, so tile counts above
// 2^22 (workgroups of up to 512 lanes) spread over y; the kernel numbers its
// tile blockIdx.x + blockIdx.y * gridDim.x and skips those past the last.
inline dim3 tile_grid(int64_t tiles)
{
    constexpr int64_t kMaxX = int64_t(1) << 22;
    if (tiles <= kMaxX)
        return dim3((unsigned)tiles);
    return dim3((unsigned)kMaxX, (unsigned)cdiv(tiles, kMaxX));
}

} // namespace

// epilogue.cuh -- the epilogue shared by the fused products:
//
//   C[m, n] = act(s acc + bias[n]) + R[m, n]
//
// The fused kernels put the weight's rows (n) on the accumulator's TMEM lanes and the
// tokens (m) on its columns.  A thread then owns one n for a whole tile: bias[n] and
// the weight's scale are one register each, a warp's 32 lanes write 32 consecutive
// elements of a token's row (whole 32-byte sectors when the row is aligned), and no
// shared-memory transpose or TMA store is needed -- so N, the pitches and the
// alignment of C and R are free.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace nvg {

struct EpiArgs {
    const float* bias;   // [N] or null
    const void* res;     // or null
    void* out;
    int64_t ld_res, ldc;
    int act, res_dtype, out_dtype;
    int M, N;
};

// One column of C: token m0 + j of row pitch ld, this thread's n.  A whole chunk runs
// without a test per token (each test is a branch, and a branch per element keeps the
// accesses from being in flight together); only the last tokens' chunk tests.
template <int C, typename F>
__device__ __forceinline__ void for_tokens(int m0, int M, F f) {
    if (m0 + C <= M) {
#pragma unroll
        for (int j = 0; j < C; ++j) f(j);
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (m0 + j < M) f(j);
    }
}

// R[m0 + j, n] for j < C (0 where there is none).  R may be C itself: a thread reads
// each element before it, and nobody else, writes it, so these are plain loads.
template <int C>
__device__ __forceinline__ void epilogue_residual(const EpiArgs& e, int m0, int n, float (&r)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j) r[j] = 0.0f;
    if (!e.res || n >= e.N) return;
    const int64_t at = m0 * e.ld_res + n;
    if (e.res_dtype == NVFP4_DTYPE_BF16) {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(e.res) + at;
        for_tokens<C>(m0, e.M, [&](int j) { r[j] = __bfloat162float(p[j * e.ld_res]); });
    } else {
        const float* p = static_cast<const float*>(e.res) + at;
        for_tokens<C>(m0, e.M, [&](int j) { r[j] = p[j * e.ld_res]; });
    }
}

// v: the scaled products of tokens m0 .. m0 + C - 1 for this thread's n, bias added.
// expf and erff are CUDA's full-range functions; x / (1 + e^-x) runs to -0 for very
// negative x (its denominator overflows to infinity).
template <int C>
__device__ __forceinline__ void epilogue_store(const EpiArgs& e, int m0, int n, float (&v)[C], const float (&r)[C]) {
    if (e.act == GEMM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = __fdiv_rn(v[j], 1.0f + expf(-v[j]));
    } else if (e.act == GEMM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = 0.5f * v[j] * (1.0f + erff(v[j] * 0.70710678118654752f));
    } else if (e.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];   // NaN stays NaN
    }
    if (n >= e.N) return;
    const int64_t at = m0 * e.ldc + n;
    if (e.out_dtype == NVFP4_DTYPE_BF16) {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(e.out) + at;
        for_tokens<C>(m0, e.M, [&](int j) { p[j * e.ldc] = __float2bfloat16_rn(v[j] + r[j]); });
    } else {
        float* p = static_cast<float*>(e.out) + at;
        for_tokens<C>(m0, e.M, [&](int j) { p[j * e.ldc] = v[j] + r[j]; });
    }
}

}  // namespace nvg

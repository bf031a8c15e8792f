// epilogue.cuh -- the epilogue shared by the fused products:
//
//   C[m, n] = act(acc[m, n] s[m] t[n] + bias[n]) + R[m, n]
//
// The fused kernels put the weight's rows (n) on the accumulator's TMEM lanes and the
// tokens (m) on its columns.  A thread then owns one n for a whole tile: bias[n] and
// the weight's scale are one register each, a warp's 32 lanes write 32 consecutive
// elements of a token's row (whole 32-byte sectors when the row is aligned), and no
// shared-memory transpose or TMA store is needed -- so N, the pitches and the
// alignment of C and R are free.
//
// What bounds it is the number of instructions per element: without its stores an
// earlier form (24 instructions) took 71 of 80 us on 8192 x 12352 outputs, where the
// products of K = 128 alone took 15.  Hence the arithmetic in pairs (one f32x2
// instruction for two tokens), running row pointers (base + j * pitch for each took up to
// 7 % longer), and no test per token in whole chunks.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace nvg {

struct EpiArgs {
    const float* bias;   // [N] or null
    const void* res;     // or null
    void* out;
    uint32_t ld_res, ldc;   // row pitches in bytes
    int act, res_dtype, out_dtype;
    int M, N;
};

// ------------------------------------------------------ pairs of float32 ---
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 ex2(F2 a) {
    float x, y;
    split(a, x, y);
    return f2(ex2(x), ex2(y));
}
__device__ __forceinline__ F2 rcp(F2 a) {
    float x, y;
    split(a, x, y);
    return f2(rcp(x), rcp(y));
}

// x / (1 + e^-x).  The exponent's rounding costs 2^-24 |x log2 e| relative in e^-x, and
// e^-x weighs less than 1 / |x| in the result: within 4 x 2^-24 |x| throughout.  e^-x
// overflowing to infinity gives -0 for very negative x.
__device__ __forceinline__ F2 silu(F2 x) {
    return x * rcp(f2(1.0f, 1.0f) + ex2(x * f2(-1.44269504f, -1.44269504f)));
}

__device__ __forceinline__ F2 relu(F2 x) {
    float a, b;
    split(x, a, b);
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(a));   // NaN stays NaN
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(b));
    return f2(a, b);
}

// x Phi(x) = max(x, 0) - |x| h with h = Phi(-|x|) = erfc(|x| / sqrt 2) / 2 by the rational
// approximation 7.1.26 of Abramowitz and Stegun's Handbook (absolute error of erfc at most
// 1.5e-7, so 0.75e-7 |x| here).  |x| is held at 20, where h has underflowed: infinities
// come out as infinity and 0.
__device__ __forceinline__ F2 gelu(F2 x) {
    float a, b;
    split(x, a, b);
    const F2 r = relu(x);
    const F2 c = f2(fminf(fabsf(a), 20.0f), fminf(fabsf(b), 20.0f));
    const F2 z = c * f2(0.70710678f, 0.70710678f);
    const F2 t = rcp(fma(z, f2(0.3275911f, 0.3275911f), f2(1.0f, 1.0f)));
    // minus one half of the polynomial
    F2 p = fma(t, f2(-0.5f * 1.061405429f, -0.5f * 1.061405429f), f2(0.5f * 1.453152027f, 0.5f * 1.453152027f));
    p = fma(p, t, f2(-0.5f * 1.421413741f, -0.5f * 1.421413741f));
    p = fma(p, t, f2(0.5f * 0.284496736f, 0.5f * 0.284496736f));
    p = fma(p, t, f2(-0.5f * 0.254829592f, -0.5f * 0.254829592f));
    return fma(c, t * p * ex2(z * z * f2(-1.44269504f, -1.44269504f)), r);
}

// R[m0 + j, n] for j < C, as stored (bf16 in the low half), loaded ahead of its use.  R
// may be the output itself: a thread reads each element before it, and nobody else,
// writes it, so these are plain loads.  Past the last token the last one is read.
template <int C>
struct EpiResidual {
    uint32_t raw[C];
    __device__ __forceinline__ void load(const EpiArgs& e, int m0, int n) {
        const int last = e.M - 1 - m0;
        if (!e.res || n >= e.N || last < 0) return;   // nothing of it is used
        const char* row = static_cast<const char*>(e.res) + static_cast<int64_t>(m0) * e.ld_res;
        if (e.res_dtype == NVFP4_DTYPE_BF16) {
            row += 2 * static_cast<int64_t>(n);
            load_rows<uint16_t>(row, e.ld_res, last);
        } else {
            row += 4 * static_cast<int64_t>(n);
            load_rows<uint32_t>(row, e.ld_res, last);
        }
    }
    template <typename T>
    __device__ __forceinline__ void load_rows(const char* row, uint32_t pitch, int last) {
        if (last >= C - 1) {
#pragma unroll
            for (uint32_t j = 0; j < C; ++j) {
                raw[j] = *reinterpret_cast<const T*>(row);
                row += pitch;
            }
        } else {
#pragma unroll
            for (uint32_t j = 0; j < C; ++j)
                raw[j] = *reinterpret_cast<const T*>(row + static_cast<uint64_t>(min(j, static_cast<uint32_t>(last))) * pitch);
        }
    }
};

// Scales of `count` tokens from m0 on into a warp's own shared memory (16-byte aligned).
__device__ __forceinline__ void stage_token_scales(const float* sA, int M, int m0, int count, float* s, int lane) {
    __syncwarp();   // the previous tile's reads are done
    for (int i = lane; i < count; i += 32) s[i] = m0 + i < M ? sA[m0 + i] : 0.0f;
    __syncwarp();
}

template <int C, typename F>
__device__ __forceinline__ void store_rows(int count, F put) {
    if (count >= C) {
#pragma unroll
        for (uint32_t j = 0; j < C; ++j) put(j);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < C; ++j)
            if (static_cast<int>(j) < count) put(j);
    }
}

// acc: the products of tokens m0 .. m0 + C - 1 for this thread's n; s: their scales in
// shared memory, or null; t: the factor they share.
template <int C, bool kTokenScales>
__device__ __forceinline__ void epilogue_store(const EpiArgs& e, int m0, int n, const uint32_t (&acc)[C],
                                               const EpiResidual<C>& res, const float* s, float t, float bias) {
    constexpr int P = C / 2;
    F2 v[P];
    const F2 t2 = f2(t, t), b2 = f2(bias, bias);
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = f2(__uint_as_float(acc[2 * j]), __uint_as_float(acc[2 * j + 1]));
    if constexpr (kTokenScales) {
        static_assert(C % 4 == 0, "token scales are read four at a time");
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            const float4 sj = *reinterpret_cast<const float4*>(s + 2 * j);
            v[j] = v[j] * f2(sj.x, sj.y);
            v[j + 1] = v[j + 1] * f2(sj.z, sj.w);
        }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = fma(v[j], t2, b2);
    if (e.act == GEMM_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = silu(v[j]);
    } else if (e.act == GEMM_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = gelu(v[j]);
    } else if (e.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = relu(v[j]);
    }
    if (n >= e.N) return;
    if (e.res) {
        const int shift = e.res_dtype == NVFP4_DTYPE_BF16 ? 16 : 0;
#pragma unroll
        for (int j = 0; j < P; ++j)
            v[j] = v[j] + f2(__uint_as_float(res.raw[2 * j] << shift), __uint_as_float(res.raw[2 * j + 1] << shift));
    }
    const int count = e.M - m0;   // tokens left from this chunk on
    char* row = static_cast<char*>(e.out) + static_cast<int64_t>(m0) * e.ldc;
    if (e.out_dtype == NVFP4_DTYPE_BF16) {
        row += 2 * static_cast<int64_t>(n);
        uint32_t w[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float x, y;
            split(v[j], x, y);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(y), "f"(x));
        }
        auto put = [&](uint32_t j) {
            *reinterpret_cast<uint16_t*>(row) =
                static_cast<uint16_t>(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu);
            row += e.ldc;
        };
        store_rows<C>(count, put);
    } else {
        row += 4 * static_cast<int64_t>(n);
        float x[C];
#pragma unroll
        for (int j = 0; j < P; ++j) split(v[j], x[2 * j], x[2 * j + 1]);
        auto put = [&](uint32_t j) {
            *reinterpret_cast<float*>(row) = x[j];
            row += e.ldc;
        };
        store_rows<C>(count, put);
    }
}

}  // namespace nvg

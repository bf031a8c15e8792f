// norm.cu -- the block's pre-norm in front of a projection, with an 8-bit output:
// the residual stream's addition, RMS normalisation and row-wise E4M3 quantisation
// in one pass, and the row quantiser alone (weights, the scan's output).
//
//   h = x + r                      (rounded once, to r's type)
//   n = h w / sqrt(mean(h^2) + eps)
//   S = max|n| / 448,  code = E4M3(n (1 / S))          one S per row
//
// The pages keep the norms unquantised ("Minima" section of the review page) and
// compare W4A4 with recipes that hold these projections at 8 bits; they give no
// formula for either, so both are the usual ones.
//
// One pass over the data: a row stays in registers between its load and its codes.
// With p = RN(h w) and n = RN(p rstd), the row's largest |n| is RN(rstd max|p|)
// exactly, because rounding after a product with one positive factor keeps order;
// the sum of squares and max|p| therefore travel through one reduction, and a row
// costs one barrier instead of two.  Magnitudes are compared as integers (sign
// cleared), where NaN sorts above infinity and infinity above every number, so a
// value that is not finite reaches the row's scale instead of being skipped.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace nvg {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100: below it a row's scale is 1
constexpr int kMaxRowCols = 32768;                     // 1024 threads x 32 values
constexpr int kWarpRowCols = 1024;                     // at most this: one warp per row

// V consecutive values as float, loaded or stored as one or two vector accesses.
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(p + i);
        f[i] = u.x; f[i + 1] = u.y; f[i + 2] = u.z; f[i + 3] = u.w;
    }
}
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&f)[V]) {
    uint32_t w[V / 2];
    if constexpr (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    uint32_t u;
    memcpy(&u, &b, 4);
    return u;
}
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
}
// Four E4M3 codes, nearest even, saturating at 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}

struct RowArgs {
    const void* x;
    const void* r;        // residual, or null
    const float* w;
    void* h;              // x + r, in r's type
    uint8_t* codes;       // or null
    float* scale;
    __nv_bfloat16* n;     // or null
    unsigned int* amax;   // or null: folds max|n| of the bf16 n
    int64_t rows, ld_x, ld_r, ld_h, ld_c, ld_n;
    int cols;
    float eps;
};

struct NoResidual {};   // TR when nothing is added

// TX: type of x; TR: type of r and h (NoResidual: h = x, not written); kNorm: false
// for the plain row quantiser; V values per vector, NV vectors per thread and row.
// R = 0: a CTA per row.  R > 0: a warp takes R rows at a time, all their loads in
// flight together.  T: most threads of a CTA; 384 and 512 keep registers for two CTAs an
// SM, so that one works while the other waits for its row; four rows a warp for five (65536 x
// 128 fp32: 11.4 us, with four 12.3).
template <typename TX, typename TR, bool kNorm, int V, int NV, int R, int T>
__global__ void __launch_bounds__(T, T == 384 || T == 512 ? 2 : R == 4 && std::is_same<TR, NoResidual>::value ? 5 : 0)
    row_kernel(const RowArgs a) {
    constexpr bool kAdd = !std::is_same<TR, NoResidual>::value;
    constexpr int N = R ? R : 1;
    using RT = typename std::conditional<kAdd, TR, float>::type;
    pdl_wait_and_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = R ? lane : threadIdx.x;
    const int stride = R ? 32 : blockDim.x;
    const int64_t row0 = R ? (static_cast<int64_t>(blockIdx.x) * 8 + warp) * N : blockIdx.x;
    const int64_t left = a.rows - row0;   // rows of this group: left, at most N
    if (R && left <= 0) return;
    const int nvec = a.cols / V;

    float v[N][NV][V];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const TX* x = static_cast<const TX*>(a.x) + (row0 + k) * a.ld_x;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * stride;
            if (c < nvec && k < left) {
                load_vec<V>(x + c * V, v[k][i]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][i][e] = 0.0f;
            }
        }
    }
    if constexpr (kAdd) {
        // 32 values a thread in 64 registers: the residual in two halves
        constexpr int HALF = NV * V > 16 && T >= 512 ? NV / 2 : NV;
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += HALF) {
            float rv[N][HALF][V];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const RT* r = static_cast<const RT*>(a.r) + (row0 + k) * a.ld_r;
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    const int c = t + (i0 + i) * stride;
                    if (c < nvec && k < left) load_vec<V>(r + c * V, rv[k][i]);
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                RT* h = static_cast<RT*>(a.h) + (row0 + k) * a.ld_h;
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    const int c = t + (i0 + i) * stride;
                    if (c < nvec && k < left) {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[k][i0 + i][e] = round_to(v[k][i0 + i][e] + rv[k][i][e], static_cast<const RT*>(nullptr));
                        store_vec<V>(h + c * V, v[k][i0 + i]);
                    }
                }
            }
        }
    }

    float ss[N];
    uint32_t top[N];   // bits of the largest magnitude
#pragma unroll
    for (int k = 0; k < N; ++k) {
        ss[k] = 0.0f;
        top[k] = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * stride;
        if constexpr (kNorm) {
            float wv[V];
#pragma unroll
            for (int e = 0; e < V; ++e) wv[e] = 0.0f;
            if (c < nvec) {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 u = __ldg(reinterpret_cast<const float4*>(a.w + c * V + e));
                    wv[e] = u.x; wv[e + 1] = u.y; wv[e + 2] = u.z; wv[e + 3] = u.w;
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    ss[k] = fmaf(v[k][i][e], v[k][i][e], ss[k]);
                    v[k][i][e] *= wv[e];
                }
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) top[k] = max(top[k], __float_as_uint(v[k][i][e]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) top[k] = __reduce_max_sync(0xffffffffu, top[k]);
    if constexpr (kNorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], o);
    }
    if constexpr (R == 0) {
        __shared__ float s_ss[32];
        __shared__ uint32_t s_top[32];
        if (lane == 0) {
            s_ss[warp] = ss[0];
            s_top[warp] = top[0];
        }
        __syncthreads();
        const int nwarps = blockDim.x >> 5;
        top[0] = __reduce_max_sync(0xffffffffu, lane < nwarps ? s_top[lane] : 0u);
        if constexpr (kNorm) {
            ss[0] = lane < nwarps ? s_ss[lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], o);
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (k >= left) break;
        const int64_t row = row0 + k;
        float rstd = 1.0f;
        if constexpr (kNorm) {
            rstd = rsqrtf(ss[k] / static_cast<float>(a.cols) + a.eps);
        }
        // A row whose sum of squares, largest |h w| or largest |n| is not a finite fp32 number has no
        // norm: NaN throughout.  (Summing scaled squares, so that the mean alone counts, takes 2 %
        // longer, and 14 % with 4096 x 16384 bf16, for |h| over 1e17.)  0 ss is NaN for such a sum.
        const float amax = kNorm ? fmaf(0.0f, ss[k], __fmul_rn(__uint_as_float(top[k]), rstd)) : __uint_as_float(top[k]);
        const bool finite = amax <= 3.402823466e38f;
        if (kNorm && !finite) rstd = __uint_as_float(0x7FC00000u);
        // NaN and infinity both give a NaN scale: the row decodes to NaN, not to numbers
        const float S = amax < kAmaxFloor ? 1.0f : finite ? __fdiv_rn(amax, kE4m3Max) : __uint_as_float(0x7FC00000u);
        const float inv = __frcp_rn(S);
        if constexpr (kNorm) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][i][e] *= rstd;
            if (a.n) {
                __nv_bfloat16* n = a.n + row * a.ld_n;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = t + i * stride;
                    if (c < nvec) store_vec<V>(n + c * V, v[k][i]);
                }
                if (a.amax && t == 0) {
                    // rounding keeps order: the largest bf16 |n| is the rounded largest |n|
                    const uint32_t b =
                        finite ? __float_as_uint(round_to(amax, static_cast<const __nv_bfloat16*>(nullptr))) : 0x7FC00000u;
                    if (b > *static_cast<volatile unsigned int*>(a.amax)) atomicMax(a.amax, b);
                }
            }
        }
        if (a.codes) {
            uint8_t* q = a.codes + row * a.ld_c;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = t + i * stride;
                if (c < nvec) {
                    uint32_t w[V / 4];
#pragma unroll
                    for (int e = 0; e < V; e += 4)
                        w[e / 4] = e4m3x4(v[k][i][e] * inv, v[k][i][e + 1] * inv, v[k][i][e + 2] * inv,
                                          v[k][i][e + 3] * inv);
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2*>(q + c * 8) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t*>(q + c * 4) = w[0];
                }
            }
            if (t == 0) a.scale[row] = S;
        }
    }
}

template <typename TX, typename TR, bool kNorm, int NV, int R>
cudaError_t warp_rows_launch(const RowArgs& a, cudaStream_t st) {
    return launch_pdl(row_kernel<TX, TR, kNorm, 4, NV, R, 256>, dim3(static_cast<unsigned>((a.rows + 8 * R - 1) / (8 * R))),
                      dim3(256), 0, st, a);
}

// Up to 1024 columns a warp per row, about 16 values a lane and, for short rows, several
// rows at once (65536 x 128 fp32: 13.8 us with one row, 11.4 with four).  Longer rows a
// CTA per row, 16 values a thread: with 32768 x 5120 that reads and writes at the copy
// rate (fp32 x, bf16 residual: 233 us; 8 values 279, 32 values 295).  Few rows want more
// threads a row instead (norm of 1237 x 4112: 14.0 us with 8 values, 15.2 with 16; of 4096
// x 5120: 30.2 and 29.4).  Rows over 6144 are kept to two CTAs an SM (4096 x 8192, fp32 x:
// 60 and 54 us; rows of 5120 lose by it, 30.0 and 33.4).  Rows over 8192 take 32 values, in
// CTAs of at most 384 or 512 threads (4096 x 12288, fp32 x, bf16 residual: 102 us in one
// CTA of 768 threads, 91 in two of 384; 4096 x 16384 bf16 with a bf16 n: 118 and 100).
template <typename TX, typename TR, bool kNorm>
cudaError_t row_launch(const RowArgs& a, cudaStream_t st) {
    if (a.cols <= 128) return warp_rows_launch<TX, TR, kNorm, 1, 4>(a, st);
    if (a.cols <= 256) return warp_rows_launch<TX, TR, kNorm, 2, 2>(a, st);
    if (a.cols <= 512) return warp_rows_launch<TX, TR, kNorm, 4, 1>(a, st);
    if (a.cols <= kWarpRowCols) return warp_rows_launch<TX, TR, kNorm, 8, 1>(a, st);
    // 16-byte vectors of the wider type
    constexpr bool kWide = std::is_same<TX, float>::value || std::is_same<TR, float>::value;
    constexpr int V = kWide ? 4 : 8;
    constexpr int U = 8 / V;                    // vectors per 8 values
    const int nvec = a.cols / V;
    auto threads = [&](int nv) { return dim3(static_cast<unsigned>(((nvec + nv - 1) / nv + 31) / 32 * 32)); };
    const dim3 grid(static_cast<unsigned>(a.rows));
    const bool few = a.rows <= static_cast<int64_t>(num_sms()) * (kNorm ? 10 : 1);
    if (few && nvec <= 1024 * U) return launch_pdl(row_kernel<TX, TR, kNorm, V, U, 0, 1024>, grid, threads(U), 0, st, a);
    if (nvec <= 384 * 2 * U)
        return launch_pdl(row_kernel<TX, TR, kNorm, V, 2 * U, 0, 1024>, grid, threads(2 * U), 0, st, a);
    if (nvec <= 512 * 2 * U)
        return launch_pdl(row_kernel<TX, TR, kNorm, V, 2 * U, 0, 512>, grid, threads(2 * U), 0, st, a);
    if (nvec <= 384 * 4 * U)
        return launch_pdl(row_kernel<TX, TR, kNorm, V, 4 * U, 0, 384>, grid, threads(4 * U), 0, st, a);
    if (nvec <= 512 * 4 * U)
        return launch_pdl(row_kernel<TX, TR, kNorm, V, 4 * U, 0, 512>, grid, threads(4 * U), 0, st, a);
    return launch_pdl(row_kernel<TX, TR, kNorm, V, 4 * U, 0, 1024>, grid, threads(4 * U), 0, st, a);
}

template <typename TX>
cudaError_t norm_launch(const RowArgs& a, int r_dtype, cudaStream_t st) {
    if (!a.r) return row_launch<TX, NoResidual, true>(a, st);
    return r_dtype == NVFP4_DTYPE_BF16 ? row_launch<TX, __nv_bfloat16, true>(a, st) : row_launch<TX, float, true>(a, st);
}

bool known_dtype(int32_t t) { return t == NVFP4_DTYPE_BF16 || t == NVFP4_DTYPE_FP32; }
int64_t dtype_bytes(int32_t t) { return t == NVFP4_DTYPE_BF16 ? 2 : 4; }

// One row-major matrix argument: pitch and 16-byte alignment.
nvfp4_status check_rows(const void* p, int32_t dtype, int64_t ld, int64_t cols, const char* name) {
    if (ld < cols) return fail(NVFP4_ERR_INVALID_ARG, std::string("row pitch of ") + name + " smaller than cols");
    if (!aligned16(p) || (ld * dtype_bytes(dtype)) % 16)
        return fail(NVFP4_ERR_MISALIGNED, std::string(name) + " or its row pitch not 16-byte aligned");
    return NVFP4_OK;
}

nvfp4_status check_size(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1) return fail(NVFP4_ERR_INVALID_ARG, "rows and cols must be >= 1");
    if (cols % 16 || cols > kMaxRowCols)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "cols must be a multiple of 16, at most 32768");
    if (rows > (int64_t(1) << 31) - 256) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "rows too large");
    return NVFP4_OK;
}

}  // namespace

nvfp4_status validate_fp8(const fp8_tensor* t, const char* name) {
    if (!t) return fail(NVFP4_ERR_INVALID_ARG, std::string(name) + " is null");
    if (!t->codes || !t->scale) return fail(NVFP4_ERR_INVALID_ARG, std::string(name) + " has a null buffer");
    if (t->rows < 1 || t->cols < 1) return fail(NVFP4_ERR_INVALID_ARG, std::string(name) + " is empty");
    if (t->cols % 16 || t->cols > (int64_t(1) << 24))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, std::string(name) + " cols must be a multiple of 16, at most 2^24");
    if (t->rows > (int64_t(1) << 31) - 256) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, std::string(name) + " too large");
    if (t->ld < t->cols) return fail(NVFP4_ERR_INVALID_ARG, std::string(name) + " ld < cols");
    if (!aligned16(t->codes) || t->ld % 16)
        return fail(NVFP4_ERR_MISALIGNED, std::string(name) + " codes or ld not 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(t->scale) % 4)
        return fail(NVFP4_ERR_MISALIGNED, std::string(name) + " scale not 4-byte aligned");
    return NVFP4_OK;
}

}  // namespace nvg

extern "C" nvfp4_status fp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld,
                                     const fp8_tensor* out, nvfp4_stream_t stream) {
    using namespace nvg;
    if (!x) return fail(NVFP4_ERR_INVALID_ARG, "x is null");
    if (!known_dtype(x_dtype)) return fail(NVFP4_ERR_INVALID_ARG, "bad x_dtype");
    nvfp4_status s = check_size(rows, cols);
    if (s != NVFP4_OK) return s;
    if ((s = validate_fp8(out, "out")) != NVFP4_OK) return s;
    if (out->rows != rows || out->cols != cols) return fail(NVFP4_ERR_INVALID_ARG, "out shape differs from x");
    if ((s = check_rows(x, x_dtype, ld, cols, "x")) != NVFP4_OK) return s;
    RowArgs a = {};
    a.x = x;
    a.codes = out->codes;
    a.scale = out->scale;
    a.rows = rows;
    a.ld_x = ld;
    a.ld_c = out->ld;
    a.cols = static_cast<int>(cols);
    const cudaError_t e = x_dtype == NVFP4_DTYPE_BF16
                              ? row_launch<__nv_bfloat16, NoResidual, false>(a, as_stream(stream))
                              : row_launch<float, NoResidual, false>(a, as_stream(stream));
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "fp8_quantize launch");
}

extern "C" nvfp4_status add_rmsnorm_quantize(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual,
                                             int32_t residual_dtype, int64_t ld_residual, const float* w, float eps,
                                             int64_t rows, int64_t cols, void* h, int64_t ld_h, const fp8_tensor* out,
                                             void* norm_bf16, int64_t ld_norm, unsigned int* amax_word,
                                             nvfp4_stream_t stream) {
    using namespace nvg;
    if (!x || !w) return fail(NVFP4_ERR_INVALID_ARG, "x or w is null");
    if (!known_dtype(x_dtype)) return fail(NVFP4_ERR_INVALID_ARG, "bad x_dtype");
    if (!(eps > 0.0f) || !(eps <= 3.402823466e38f)) return fail(NVFP4_ERR_INVALID_ARG, "eps must be positive and finite");
    if (!out && !norm_bf16) return fail(NVFP4_ERR_INVALID_ARG, "neither out nor norm_bf16 is given");
    if (amax_word && !norm_bf16) return fail(NVFP4_ERR_INVALID_ARG, "amax_word needs norm_bf16");
    if (reinterpret_cast<uintptr_t>(amax_word) % 4) return fail(NVFP4_ERR_MISALIGNED, "amax_word not 4-byte aligned");
    if ((residual == nullptr) != (h == nullptr))
        return fail(NVFP4_ERR_INVALID_ARG, "residual and h are given together or not at all");
    nvfp4_status s = check_size(rows, cols);
    if (s != NVFP4_OK) return s;
    if ((s = check_rows(x, x_dtype, ld_x, cols, "x")) != NVFP4_OK) return s;
    if (!aligned16(w)) return fail(NVFP4_ERR_MISALIGNED, "w not 16-byte aligned");
    if (residual) {
        if (!known_dtype(residual_dtype)) return fail(NVFP4_ERR_INVALID_ARG, "bad residual_dtype");
        if ((s = check_rows(residual, residual_dtype, ld_residual, cols, "residual")) != NVFP4_OK) return s;
        if ((s = check_rows(h, residual_dtype, ld_h, cols, "h")) != NVFP4_OK) return s;
    }
    if (h && ((h == residual && ld_h != ld_residual) || (h == x && (x_dtype != residual_dtype || ld_h != ld_x))))
        return fail(NVFP4_ERR_INVALID_ARG, "h may be residual or x only with the same type and pitch");
    if (norm_bf16 && (norm_bf16 == x || norm_bf16 == residual || norm_bf16 == h))
        return fail(NVFP4_ERR_INVALID_ARG, "norm_bf16 overlaps x, residual or h");
    if (norm_bf16 && (s = check_rows(norm_bf16, NVFP4_DTYPE_BF16, ld_norm, cols, "norm_bf16")) != NVFP4_OK) return s;
    if (out) {
        if ((s = validate_fp8(out, "out")) != NVFP4_OK) return s;
        if (out->rows != rows || out->cols != cols) return fail(NVFP4_ERR_INVALID_ARG, "out shape differs from x");
    }
    RowArgs a = {};
    a.x = x;
    a.r = residual;
    a.w = w;
    a.h = h;
    a.codes = out ? out->codes : nullptr;
    a.scale = out ? out->scale : nullptr;
    a.n = static_cast<__nv_bfloat16*>(norm_bf16);
    a.amax = amax_word;
    a.rows = rows;
    a.ld_x = ld_x;
    a.ld_r = ld_residual;
    a.ld_h = ld_h;
    a.ld_c = out ? out->ld : 0;
    a.ld_n = ld_norm;
    a.cols = static_cast<int>(cols);
    a.eps = eps;
    const cudaError_t e = x_dtype == NVFP4_DTYPE_BF16 ? norm_launch<__nv_bfloat16>(a, residual_dtype, as_stream(stream))
                                                      : norm_launch<float>(a, residual_dtype, as_stream(stream));
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "add_rmsnorm_quantize launch");
}

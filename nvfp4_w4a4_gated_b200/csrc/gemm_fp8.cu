// gemm_fp8.cu -- 8-bit product with a fused epilogue:
//
//   C[m, n] = act(sA[m] sB[n] sum_k A[m, k] B[n, k] + bias[n]) + R[m, n]
//
// A [M x K] and B [N x K] hold E4M3 codes with one fp32 scale a row (fp8_quantize,
// add_rmsnorm_quantize).  The row scales factor out of the sum, so the tensor cores
// see plain E4M3 operands (tcgen05.mma kind::f8f6f4, f32 accumulators in TMEM) and the
// scales are applied once per output element.
//
// Both kernels put B's rows (n) on the accumulator's lanes and A's rows (the tokens)
// on its columns; see epilogue.cuh for why.  Operand tiles are 128 bytes of K wide,
// staged by TMA with the 128-byte swizzle; K's tail is zero-filled by the copies.
// Every wait is bounded: on expiry the kernel records a code in the device error word
// and returns.
#include "epilogue.cuh"

namespace nvg {

nvfp4_status validate_fp8(const fp8_tensor* t, const char* name);

namespace {

constexpr int kTileK = 128;   // E4M3 values (bytes) of K per stage

// Instruction descriptor of tcgen05.mma kind::f8f6f4: E4M3 x E4M3, both K-major,
// f32 accumulate.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_fp8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tiled TMA load into this CTA's shared memory that signals an mbarrier of either CTA
// of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

struct Fp8Args {
    const float* sA;   // [M] token scales
    const float* sB;   // [N] weight-row scales
    int K;
    unsigned int* err;
    EpiArgs epi;
};

// ------------------------------------------------------------ CTA-pair kernel --
// Long prefills.  A cluster of two CTAs computes 256 weight rows x 256 tokens: CTA r
// holds weight rows [128 r, 128 r + 128) of the tile and tokens [128 r, ...) of the
// tile's tokens, 32 KB a stage for 128 x 256 x 128 products each.  The odd CTA's
// copies signal the even CTA's barriers directly, so the issuing thread waits on one
// barrier a stage.  Two accumulators of 256 columns fill TMEM: the epilogue warps
// drain one while the next tile's products fill the other.  Sixteen of them, because
// short K is bound by the epilogue's instructions (epilogue.cuh): 8192 x 4096 x 256 with
// SiLU took 43 us with eight and 38 with sixteen.  For long K the power limit binds: in
// a loop, 8192 x 12352 x 5120 runs at 1.1 to 1.3 GHz and 2.4 PFLOP/s, 0.87 of the
// sustained rate (twice the measured sustained bf16 rate).
struct Pair {
        static constexpr int STAGES = 6;                     // 4 to 7 measured the same
    static constexpr int EPI_WARPS = 16;
    static constexpr int EPI_COLS = 1024 / EPI_WARPS;   // token columns per epilogue warp
    static constexpr int A_BYTES = 128 * kTileK;   // own weight rows
    static constexpr int B_BYTES = 128 * kTileK;   // own half of the tokens
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * EPI_COLS * 4 + 256 + 1024;
    static constexpr uint32_t IDESC = idesc_e4m3(256, 256);
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::THREADS, 1)
    w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ Fp8Args args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    float* scales = reinterpret_cast<float*>(smem + Pair::STAGES * Pair::STAGE_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + Pair::EPI_WARPS * Pair::EPI_COLS);   // even CTA's are used
    uint64_t* empty = full + Pair::STAGES;
    uint64_t* acc_full = empty + Pair::STAGES;   // [2]
    uint64_t* acc_free = acc_full + 2;           // [2] even CTA's are used: both CTAs' epilogue warps
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_free + 2);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_m = (args.epi.M + 255) / 256, num_n = (args.epi.N + 255) / 256;
    const int num_tiles = num_m * num_n;
    const int num_kt = (args.K + kTileK - 1) / kTileK;
    unsigned int* err = args.err;
    // Tiles run in bands of 8 token tiles, weight tiles slowest inside a band: the
    // tiles in flight then share about as many token rows as weight rows.
    auto tile_mn = [&](int tile, int& m_idx, int& n_idx) {
        const int band = tile / (8 * num_n), first = band * 8;
        const int width = min(8, num_m - first), in = tile - band * 8 * num_n;
        m_idx = first + in % width;
        n_idx = in / width;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < Pair::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 2 * Pair::EPI_WARPS);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, 512);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_and_trigger();

    // A role of one thread is entered through elect.sync: the compiler then knows that one
    // lane runs it and issues each tcgen05.mma straight from uniform registers.  Behind
    // `lane == 0` the issue itself was the limit: without copies and epilogue this loop ran
    // at 2.69 PFLOP/s (8192 x 8192 x 4096), elected at 4.06; the whole kernel 2.28 -> 2.89.
    if (warp == 0) {
        if (elect_one()) {
            // ---------------------------------------------------- producer --
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int tile = pair; tile < num_tiles && ok; tile += npairs) {
                int m_idx, n_idx;
                tile_mn(tile, m_idx, n_idx);
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, err, kErrTimeoutTma)) {
                        ok = false;
                        break;
                    }
                    // the even CTA's barrier counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * Pair::STAGE_BYTES);
                    const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
                    uint8_t* st = smem + stage * Pair::STAGE_BYTES;
                    tma_load_2d_pair(st, &tmW, bar, kt * kTileK, n_idx * 256 + rank * 128);
                    tma_load_2d_pair(st + Pair::A_BYTES, &tmX, bar, kt * kTileK, m_idx * 256 + rank * 128);
                    if (++stage == Pair::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // -------------------------------------------------- MMA (even CTA) --
            const uint32_t peer_acc_full = mapa_shared(smem_u32(acc_full), 1);
            const uint32_t peer_empty = mapa_shared(smem_u32(empty), 1);
            uint32_t stage = 0, phase = 0;
            int local = 0;
            bool ok = true;
            for (int tile = pair; tile < num_tiles && ok; tile += npairs, ++local) {
                const int buf = local & 1;
                const uint32_t acc = tmem + buf * 256;
                if (local >= 2 &&
                    !mbar_wait_cluster(&acc_free[buf], ((local >> 1) - 1) & 1, err, kErrTimeoutMma))
                    break;
                tc_fence_after();
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait_cluster(&full[stage], phase, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + stage * Pair::STAGE_BYTES), b = a + Pair::A_BYTES;
                    const int nk = min(4, (args.K - kt * kTileK + 31) / 32);
                    for (int j = 0; j < nk; ++j)
                        mma_fp8_pair(acc, sdesc_kmajor_sw128(a + j * 32), sdesc_kmajor_sw128(b + j * 32), Pair::IDESC,
                                     (kt > 0 || j > 0) ? 1u : 0u);
                    mma_commit_pair(smem_u32(&empty[stage]));
                    mma_commit_pair(peer_empty + stage * 8);
                    if (++stage == Pair::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair(smem_u32(&acc_full[buf]));
                mma_commit_pair(peer_acc_full + buf * 8);
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue --
        const int q = warp & 3, part = (warp - 2) >> 2;   // lane quarter, share of the columns
        const EpiArgs& e = args.epi;
        float* s = scales + (warp - 2) * Pair::EPI_COLS;
        int local = 0;
        for (int tile = pair; tile < num_tiles; tile += npairs, ++local) {
            int m_idx, n_idx;
            tile_mn(tile, m_idx, n_idx);
            const int buf = local & 1;
            const int n = n_idx * 256 + rank * 128 + q * 32 + lane;
            const int m_base = m_idx * 256 + part * Pair::EPI_COLS;
            // everything that does not depend on the accumulator, before the wait for it
            const float sb = n < e.N ? args.sB[n] : 0.0f;
            const float bias = e.bias && n < e.N ? e.bias[n] : 0.0f;
            EpiResidual<16> cur, next;
            cur.load(e, m_base, n);
            stage_token_scales(args.sA, e.M, m_base, Pair::EPI_COLS, s, lane);
            // the warp stays together whichever of its lanes saw the budget run out
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[buf], (local >> 1) & 1, err, kErrTimeoutEpi))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + part * Pair::EPI_COLS;
#pragma unroll 1
            for (int c = 0; c < Pair::EPI_COLS; c += 16) {
                uint32_t acc[16];
                tmem_ld_32x32b_x16(taddr + c, acc);
                if (c + 16 < Pair::EPI_COLS) next.load(e, m_base + c + 16, n);
                tmem_wait_ld();
                if (c + 16 == Pair::EPI_COLS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_free[buf]), 0));
                }
                epilogue_store<16, true>(e, m_base + c, n, acc, cur, s + c, sb, bias);
                cur = next;
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------ split-K kernel --
// Short token counts (decode, small batches), where the weight's bytes are the cost.
// One tile of 128 weight rows x BN tokens per cluster; the SPLIT CTAs of the cluster
// take SPLIT consecutive ranges of K (none empty: the launch keeps four k-tiles each), so that weights with few row tiles still
// occupy every SM.  The partial accumulators meet in shared memory: each CTA leaves
// its own there and then adds, in rank order, the BN / SPLIT token columns that are
// its share, read from every CTA of the cluster.  The order is fixed: no atomics, the
// same bits every time.
template <int BN, int SPLIT>
struct Small {
    static constexpr int A_BYTES = 128 * kTileK;
    static constexpr int B_BYTES = BN * kTileK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 98304 / STAGE_BYTES;             // two CTAs an SM
    static constexpr int RING = STAGES * STAGE_BYTES;
    static constexpr int COLS = BN / SPLIT;                        // token columns per CTA at the end
    static constexpr int SMEM = RING + 4 * COLS * 4 + 256 + 1024;
    static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
    static constexpr int CHUNK = COLS < 16 ? COLS : 16;
    static constexpr int THREADS = 192;
    static constexpr uint32_t IDESC = idesc_e4m3(128, BN);
    static_assert(RING >= 128 * BN * 4, "the partial accumulators reuse the ring");
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int BN, int SPLIT>
__global__ void __launch_bounds__(192)
    w8a8_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ Fp8Args args) {
    using G = Small<BN, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    float* scales = reinterpret_cast<float*>(smem + G::RING);
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + (4 * G::COLS + 3) / 4 * 4);
    uint64_t* empty = full + G::STAGES;
    uint64_t* acc_full = empty + G::STAGES;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = SPLIT > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int num_m = (args.epi.M + BN - 1) / BN;
    const int tile = blockIdx.x / SPLIT;
    const int n_idx = tile / num_m, m_idx = tile - n_idx * num_m;
    const int num_kt = (args.K + kTileK - 1) / kTileK;
    const int kt0 = num_kt * rank / SPLIT, kt1 = num_kt * (rank + 1) / SPLIT;
    unsigned int* err = args.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, G::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_and_trigger();

    const int q = warp & 3;
    const int n = n_idx * 128 + q * 32 + lane;
    const EpiArgs& e = args.epi;
    float sb = 0.0f, bias = 0.0f;
    EpiResidual<G::CHUNK> cur;
    float* s = scales + (warp - 2) * G::COLS;
    if (warp == 0) {
        if (elect_one()) {
            for (int kt = kt0, i = 0; kt < kt1; ++kt, ++i) {
                const int stage = i % G::STAGES;
                if (!mbar_wait(&empty[stage], ((i / G::STAGES) & 1) ^ 1, err, kErrTimeoutTma)) break;
                mbar_arrive_expect_tx(&full[stage], G::STAGE_BYTES);
                uint8_t* st = smem + stage * G::STAGE_BYTES;
                tma_load_2d(st, &tmW, &full[stage], kt * kTileK, n_idx * 128);
                tma_load_2d(st + G::A_BYTES, &tmX, &full[stage], kt * kTileK, m_idx * BN);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            bool ok = true;
            for (int kt = kt0, i = 0; kt < kt1; ++kt, ++i) {
                const int stage = i % G::STAGES;
                if (!mbar_wait(&full[stage], (i / G::STAGES) & 1, err, kErrTimeoutMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(smem + stage * G::STAGE_BYTES), b = a + G::A_BYTES;
                const int nk = min(4, (args.K - kt * kTileK + 31) / 32);
                for (int j = 0; j < nk; ++j)
                    mma_fp8(tmem, sdesc_kmajor_sw128(a + j * 32), sdesc_kmajor_sw128(b + j * 32), G::IDESC,
                            (i > 0 || j > 0) ? 1u : 0u);
                mma_commit(&empty[stage]);
            }
            if (ok) mma_commit(acc_full);
        }
    } else {
        // what does not depend on the accumulator, before the wait for it
        if (n < e.N) {
            sb = args.sB[n];
            if (e.bias) bias = e.bias[n];
        }
        cur.load(e, m_idx * BN + rank * G::COLS, n);
        stage_token_scales(args.sA, e.M, m_idx * BN + rank * G::COLS, G::COLS, s, lane);
        mbar_wait(acc_full, 0, err, kErrTimeoutEpi);   // expired: the error word says that C is not valid
        tc_fence_after();
    }
    __syncwarp();

    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if constexpr (SPLIT > 1) {
        // partial accumulators, [column][lane row]: the ring is free, its last product done
        float* part = reinterpret_cast<float*>(smem);
        if (warp >= 2) {
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                uint32_t acc[16];
                tmem_ld_32x32b_x16(taddr + c, acc);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = __uint_as_float(acc[j]);
            }
        }
        cluster_sync();
    }
    if (warp >= 2) {
#pragma unroll 1
        for (int c = 0; c < G::COLS; c += G::CHUNK) {
            const int col = rank * G::COLS + c, m0 = m_idx * BN + col;
            uint32_t acc[G::CHUNK];
            EpiResidual<G::CHUNK> next;
            if (c + G::CHUNK < G::COLS) next.load(e, m0 + G::CHUNK, n);
            if constexpr (SPLIT > 1) {
                const uint32_t at = smem_u32(smem) + (col * 128 + q * 32 + lane) * 4;
                float sum[G::CHUNK];
#pragma unroll
                for (int from_rank = 0; from_rank < SPLIT; ++from_rank) {
                    const uint32_t from = mapa_shared(at, from_rank);
#pragma unroll
                    for (int j = 0; j < G::CHUNK; ++j) {
                        const float p = ld_shared_cluster(from + j * 512);
                        sum[j] = from_rank ? sum[j] + p : p;
                    }
                }
#pragma unroll
                for (int j = 0; j < G::CHUNK; ++j) acc[j] = __float_as_uint(sum[j]);
            } else {
                tmem_ld_cols<G::CHUNK>(taddr + c, acc);
                tmem_wait_ld();
            }
            epilogue_store<G::CHUNK, true>(e, m0, n, acc, cur, s + c, sb, bias);
            cur = next;
        }
    }
    tc_fence_before();
    if constexpr (SPLIT > 1)
        cluster_sync();   // nobody leaves while its shared memory is being read
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

// ----------------------------------------------------------------- host side --
template <typename Kern>
cudaError_t launch_cluster_pdl(Kern kernel, unsigned grid, int threads, int smem, int cluster, cudaStream_t st,
                               const CUtensorMap& tw, const CUtensorMap& tx, const Fp8Args& args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tw, tx, args);
}

nvfp4_status launch_pair(const fp8_tensor& A, const fp8_tensor& B, const Fp8Args& args, cudaStream_t st) {
    CUtensorMap tw, tx;
    nvfp4_status s = make_tmap_u8_sw128_ld(&tw, B.codes, B.rows, B.cols, B.ld, 128, kTileK);
    if (s == NVFP4_OK) s = make_tmap_u8_sw128_ld(&tx, A.codes, A.rows, A.cols, A.ld, 128, kTileK);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce once;
    static std::atomic<int> resident[64];   // pairs that fit at once, per device
    int dev = 0;
    cudaGetDevice(&dev);
    s = once_per_device(once, [&]() -> nvfp4_status {
        cudaError_t e = cudaFuncSetAttribute(w8a8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pair::SMEM);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(w8a8 pair smem)");
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms() / 2 * 2);
        cfg.blockDim = dim3(Pair::THREADS);
        cfg.dynamicSmemBytes = Pair::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, w8a8_pair_kernel, &cfg);
        if (e != cudaSuccess || n < 1) return cuda_fail(e, "w8a8 pair occupancy");
        resident[dev].store(n < num_sms() / 2 ? n : num_sms() / 2, std::memory_order_relaxed);
        return NVFP4_OK;
    });
    if (s != NVFP4_OK) return s;
    const int64_t tiles = ((A.rows + 255) / 256) * ((B.rows + 255) / 256);
    const int most = resident[dev].load(std::memory_order_relaxed);
    const unsigned pairs = static_cast<unsigned>(tiles < most ? tiles : most);
    const cudaError_t e =
        launch_pdl(w8a8_pair_kernel, dim3(pairs * 2), dim3(Pair::THREADS), Pair::SMEM, st, tw, tx, args);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "w8a8_gemm pair launch");
}

template <int BN, int SPLIT>
nvfp4_status launch_small(const fp8_tensor& A, const fp8_tensor& B, const Fp8Args& args, cudaStream_t st) {
    using G = Small<BN, SPLIT>;
    CUtensorMap tw, tx;
    nvfp4_status s = make_tmap_u8_sw128_ld(&tw, B.codes, B.rows, B.cols, B.ld, 128, kTileK);
    if (s == NVFP4_OK) s = make_tmap_u8_sw128_ld(&tx, A.codes, A.rows, A.cols, A.ld, BN, kTileK);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce once;
    if ((s = smem_limit_once(once, w8a8_small_kernel<BN, SPLIT>, G::SMEM, "cudaFuncSetAttribute(w8a8 small smem)")) !=
        NVFP4_OK)
        return s;
    const int64_t tiles = ((A.rows + BN - 1) / BN) * ((B.rows + 127) / 128);
    const cudaError_t e = launch_cluster_pdl(w8a8_small_kernel<BN, SPLIT>, static_cast<unsigned>(tiles * SPLIT),
                                             G::THREADS, G::SMEM, SPLIT, st, tw, tx, args);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "w8a8_gemm launch");
}

template <int BN>
nvfp4_status launch_split(int split, const fp8_tensor& A, const fp8_tensor& B, const Fp8Args& args, cudaStream_t st) {
    switch (split) {
        case 8: return launch_small<BN, 8>(A, B, args, st);
        case 4: return launch_small<BN, 4>(A, B, args, st);
        case 2: return launch_small<BN, 2>(A, B, args, st);
        default: return launch_small<BN, 1>(A, B, args, st);
    }
}

}  // namespace

nvfp4_status validate_epilogue(const gemm_epilogue* e, int64_t M, int64_t N, EpiArgs* out) {
    if (!e) return fail(NVFP4_ERR_INVALID_ARG, "epilogue is null");
    if (!e->out) return fail(NVFP4_ERR_INVALID_ARG, "out is null");
    auto known = [](int32_t t) { return t == NVFP4_DTYPE_BF16 || t == NVFP4_DTYPE_FP32; };
    if (!known(e->out_dtype)) return fail(NVFP4_ERR_INVALID_ARG, "bad out_dtype");
    if (e->act < GEMM_ACT_NONE || e->act > GEMM_ACT_RELU) return fail(NVFP4_ERR_INVALID_ARG, "bad act");
    if (e->ldc < N) return fail(NVFP4_ERR_INVALID_ARG, "ldc < N");
    constexpr int64_t kMostPitch = (int64_t(1) << 30) - 1;   // 32-bit byte pitches in the kernels
    if (e->ldc > kMostPitch || (e->residual && e->ld_residual > kMostPitch))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "row pitch of out or residual too large");
    auto aligned = [](const void* p, int32_t t) {
        return reinterpret_cast<uintptr_t>(p) % (t == NVFP4_DTYPE_BF16 ? 2 : 4) == 0;
    };
    if (!aligned(e->out, e->out_dtype) || (e->bias && !aligned(e->bias, NVFP4_DTYPE_FP32)))
        return fail(NVFP4_ERR_MISALIGNED, "out or bias not aligned to its type");
    if (e->residual) {
        if (!known(e->residual_dtype)) return fail(NVFP4_ERR_INVALID_ARG, "bad residual_dtype");
        if (e->ld_residual < N) return fail(NVFP4_ERR_INVALID_ARG, "ld_residual < N");
        if (!aligned(e->residual, e->residual_dtype))
            return fail(NVFP4_ERR_MISALIGNED, "residual not aligned to its type");
        if (e->residual == e->out && (e->residual_dtype != e->out_dtype || e->ld_residual != e->ldc))
            return fail(NVFP4_ERR_INVALID_ARG, "out may be residual only with the same type and pitch");
    }
    out->bias = e->bias;
    out->res = e->residual;
    out->out = e->out;
    auto bytes = [](int64_t ld, int32_t t) { return static_cast<uint32_t>(ld * (t == NVFP4_DTYPE_BF16 ? 2 : 4)); };
    out->ld_res = e->residual ? bytes(e->ld_residual, e->residual_dtype) : 0;
    out->ldc = bytes(e->ldc, e->out_dtype);
    out->act = e->act;
    out->res_dtype = e->residual_dtype;
    out->out_dtype = e->out_dtype;
    out->M = static_cast<int>(M);
    out->N = static_cast<int>(N);
    return NVFP4_OK;
}

static nvfp4_status w8a8_launch(const fp8_tensor& A, const fp8_tensor& B, const Fp8Args& args, cudaStream_t st) {
    const int64_t M = A.rows, N = B.rows;
    const int sms = num_sms();
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (M > 128 && pair_tiles * 2 >= sms) return launch_pair(A, B, args, st);
    const int64_t n_tiles = (N + 127) / 128;
    const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t tiles = n_tiles * ((M + bn - 1) / bn);
    // K ranges: double them while the CTAs still fit on the SMs two at a time and each
    // keeps at least four k-tiles
    const int64_t num_kt = (args.K + kTileK - 1) / kTileK;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * sms && num_kt / (split * 2) >= 4) split *= 2;
    if (bn == 16) return launch_split<16>(split, A, B, args, st);
    if (bn == 32) return launch_split<32>(split, A, B, args, st);
    if (bn == 64) return launch_split<64>(split, A, B, args, st);
    return launch_split<128>(split, A, B, args, st);
}

}  // namespace nvg

extern "C" nvfp4_status w8a8_gemm(const fp8_tensor* A, const fp8_tensor* B, const gemm_epilogue* epilogue,
                                  nvfp4_stream_t stream) {
    using namespace nvg;
    nvfp4_status s = validate_fp8(A, "A");
    if (s == NVFP4_OK) s = validate_fp8(B, "B");
    if (s != NVFP4_OK) return s;
    if (A->cols != B->cols) return fail(NVFP4_ERR_INVALID_ARG, "A and B have different K");
    if (A->rows > (int64_t(1) << 30) || B->rows > (int64_t(1) << 30))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "M or N too large");
    Fp8Args args = {};
    if ((s = validate_epilogue(epilogue, A->rows, B->rows, &args.epi)) != NVFP4_OK) return s;
    args.sA = A->scale;
    args.sB = B->scale;
    args.K = static_cast<int>(A->cols);
    args.err = device_error_word();
    if (!args.err) return fail(NVFP4_ERR_CUDA, "device error word unavailable");
    return w8a8_launch(*A, *B, args, as_stream(stream));
}

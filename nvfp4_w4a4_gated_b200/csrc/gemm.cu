// gemm.cu -- block-scaled FP4 x FP4 GEMM on the sm_100a tensor cores.
//
//   C[M x N] = S_A * S_B * sum_k (e2m1(A) * e4m3(sfA))[m,k] * (e2m1(B) * e4m3(sfB))[n,k]
//
// The fused in_proj of the layer (q|k|v|z|a|b under one harmonised weight
// scale, review page of "Why Gated DeltaNet Survives 4-Bit Quantization",
// paper sec.6) and the out_proj both run through this kernel.
//
// Design (one persistent CTA per SM, 10 warps):
//   warp 0      TMA producer: A tile [128 x 256] and B tile [BN x 256] codes
//               (128-byte swizzle, one 128-byte row per operand row) plus the
//               matching 512-byte scale atoms (bulk copies) into a STAGES-deep
//               shared-memory ring guarded by full/empty mbarriers;
//   warp 1      TMEM owner and MMA issuer: per k-tile 4 x tcgen05.mma
//               kind::mxf4nvf4 (M=128, N=BN, K=64 each) accumulate in TMEM;
//               tcgen05.commit frees the stage and the scale slot and, after
//               the last k-tile, signals the tile;
//   warps 6..9  scale writers: the MMA reads A row m's four E4M3 scales of a
//               k-block as one 32-bit word at TMEM lane m, column base + m/32,
//               and, for accumulator rows of lane quarter q, B row n's word at
//               lane 32q + n%32, column base + n/32.  Each warp takes one lane
//               quarter and tcgen05.st's those words from the staged atoms into
//               one of two TMEM scale slots.
//               tcgen05.cp does the same through the tensor pipe.  Issued
//               behind `lane == 0` it took ~40 % of this kernel's time; the
//               fused products (gemm_fused.cu) issue it behind elect.sync,
//               where it is cheap.  Not measured here in that form;
//   warps 2..5  epilogue: tcgen05.ld of the f32 accumulator (warp w reads
//               TMEM lanes 32*(w%4)...), scale by S_A*S_B, write 32 x 32
//               sub-tiles to shared memory (128-byte swizzle) and TMA-store
//               them, so every global write is a full 128-byte row segment.
// Two accumulator buffers of BN columns; for BN = 256 they overlap in 96
// columns (TMEM also holds two scale-factor slots) and the epilogue drains the
// shared columns first, so the next tile's MMAs start after three 32-column
// chunks and the rest of the drain overlaps them.  Every wait is bounded: on expiry the kernel records a code in the
// device error word and returns.
#include <cstdlib>
#include <cstring>

#include "common.cuh"

namespace nvg {

namespace {

constexpr int BM = 128;
constexpr int K_TILE_BYTES = 128;  // 256 FP4 values per operand row per stage
constexpr int TMEM_COLS = 512;
// TMEM plan (512 columns): two f32 accumulator buffers of BN columns (buffer 1
// starts at ACC_OFF; for BN = 256 the two overlap) and, at the top, two slots
// of scale factors used by alternate k-tiles so the scale copies of k-tile
// kt+1 never overwrite what the MMAs of k-tile kt still read.  A slot holds 4
// k-blocks x 4 columns for A and 4 k-blocks x (BN/128 x 4) columns for B.
template <int BN>
struct TmemPlan {
    static constexpr int SFA_COLS = 16;
    static constexpr int SFB_COLS = 4 * (BN / 128) * 4;
    static constexpr int SLOT = SFA_COLS + SFB_COLS;
    static constexpr int SF_BASE = 512 - 2 * SLOT;
    static constexpr int ACC_OFF = (2 * BN <= SF_BASE) ? BN : SF_BASE - BN;
    static constexpr int NCH = BN / 32;                                  // 32-column epilogue chunks
    static constexpr int OVL = (BN - ACC_OFF + 31) / 32;                 // chunks shared by both buffers
    static constexpr int FIRST = (ACC_OFF < BN) ? ACC_OFF / 32 : 0;      // buffer 0 drains from here
    static constexpr int RELEASE_AFTER = OVL > 0 ? OVL : 1;              // chunks drained before release
    __device__ static uint32_t sfa(uint32_t tmem, int slot, int j) { return tmem + SF_BASE + slot * SLOT + 4 * j; }
    __device__ static uint32_t sfb(uint32_t tmem, int slot, int j) {
        return tmem + SF_BASE + slot * SLOT + SFA_COLS + j * (BN / 128) * 4;
    }
};

template <int BN>
struct Cfg {
    static constexpr int STAGES = BN == 256 ? 3 : 5;
    static constexpr int A_BYTES = BM * K_TILE_BYTES;
    static constexpr int B_BYTES = BN * K_TILE_BYTES;
    static constexpr int SFA_BYTES = 4 * 512;
    static constexpr int SFB_BYTES = (BN / 128) * 4 * 512;
    using TP = TmemPlan<BN>;
    static constexpr int ACC_OFF = TP::ACC_OFF;
    static constexpr int STG_BYTES = 4 * 2 * 32 * 32 * 4;  // per epilogue warp: two 32 x 32 f32 sub-tiles
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM = STAGES * (A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES) + STG_BYTES + BAR_BYTES + 1024;
    static constexpr uint32_t IDESC = idesc_nvf4(BM, BN);
};

// Write 32 consecutive f32 values of row `lane` into a 32 x 32 sub-tile laid out
// with the 128-byte swizzle the C tensor map expects (16-byte chunk c of row r
// at chunk position c ^ (r % 8)); scaled by alpha.
__device__ __forceinline__ void stage_row(float* tile, int lane, const uint32_t (&v)[32], float alpha) {
    char* row = reinterpret_cast<char*>(tile) + lane * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float4 f = make_float4(alpha * __uint_as_float(v[4 * c]), alpha * __uint_as_float(v[4 * c + 1]),
                               alpha * __uint_as_float(v[4 * c + 2]), alpha * __uint_as_float(v[4 * c + 3]));
        *reinterpret_cast<float4*>(row + ((c ^ (lane & 7)) << 4)) = f;
    }
}

template <int BN>
__global__ void __launch_bounds__(320, 1)
    w4a4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const uint8_t* __restrict__ sfA,
                     const uint8_t* __restrict__ sfB, const float* __restrict__ scaleA,
                     const float* __restrict__ scaleB, int M, int N, int K, unsigned int* __restrict__ err) {
    using G = Cfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    uint8_t* sA = smem;
    uint8_t* sB = sA + G::STAGES * G::A_BYTES;
    uint8_t* sSFA = sB + G::STAGES * G::B_BYTES;
    uint8_t* sSFB = sSFA + G::STAGES * G::SFA_BYTES;
    float* sStage = reinterpret_cast<float*>(sSFB + G::STAGES * G::SFB_BYTES);  // 1024-byte aligned
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sStage) + G::STG_BYTES);
    uint64_t* empty = full + G::STAGES;
    uint64_t* acc_full = empty + G::STAGES;
    uint64_t* tmem_free = acc_full + 1;
    uint64_t* sf_full = tmem_free + 1;   // [2] scale slot written (4 writer warps, after the stage landed)
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sf_full + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_m = (M + BM - 1) / BM, num_n = (N + BN - 1) / BN;
    const int num_tiles = num_m * num_n;
    const int kb_total = K / 64;                 // 64-wide k-blocks = scale atoms along K
    const int num_kt = (kb_total + 3) / 4;       // 256-wide k-tiles
    const int sfb_row_blocks = (N + 127) / 128;
    // Tile order: the smaller operand stays in L2 while the larger one streams once.
    // With M > N (the layer's long prefills: A of 32768 x 5120 against a weight of
    // 12352 x 5120) the n tiles of one m run back to back, so each A tile is read
    // while it is hot and the weight is the operand that is reused; otherwise the m
    // tiles of one n do.
    const bool n_fast = M > N;
    auto tile_mn = [&](int tile, int& m_idx, int& n_idx) {
        if (n_fast) {
            m_idx = tile / num_n;
            n_idx = tile - m_idx * num_n;
        } else {
            n_idx = tile / num_m;
            m_idx = tile - n_idx * num_m;
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(tmem_free, 4);
        for (int i = 0; i < 2; ++i) mbar_init(&sf_full[i], 4);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmC);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_and_trigger();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- producer --
            uint32_t stage = 0, phase = 0;
            for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
                int m_idx, n_idx;
                tile_mn(tile, m_idx, n_idx);
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, err, kErrTimeoutTma)) goto producer_done;
                    const int nkb = min(4, kb_total - kt * 4);
                    int nb_valid = 0;
#pragma unroll
                    for (int nb = 0; nb < BN / 128; ++nb) nb_valid += (n_idx * (BN / 128) + nb < sfb_row_blocks);
                    const uint32_t bytes = G::A_BYTES + G::B_BYTES + nkb * 512 * (1 + nb_valid);
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    tma_load_2d(sA + stage * G::A_BYTES, &tmA, &full[stage], kt * K_TILE_BYTES, m_idx * BM);
                    tma_load_2d(sB + stage * G::B_BYTES, &tmB, &full[stage], kt * K_TILE_BYTES, n_idx * BN);
                    bulk_load(sSFA + stage * G::SFA_BYTES, sfA + ((int64_t)m_idx * kb_total + kt * 4) * 512,
                              nkb * 512, &full[stage]);
#pragma unroll
                    for (int nb = 0; nb < BN / 128; ++nb) {
                        const int rb = n_idx * (BN / 128) + nb;
                        if (rb < sfb_row_blocks)
                            bulk_load(sSFB + stage * G::SFB_BYTES + nb * 2048,
                                      sfB + ((int64_t)rb * kb_total + kt * 4) * 512, nkb * 512, &full[stage]);
                    }
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        producer_done:;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // --------------------------------------------------------- MMA --
            uint32_t stage = 0, phase = 0, kt_all = 0;
            int local = 0;
            for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++local) {
                const uint32_t acc = tmem + (local & 1) * G::ACC_OFF;
                if (local > 0) {
                    if (!mbar_wait(tmem_free, (local - 1) & 1, err, kErrTimeoutMma)) break;
                    tc_fence_after();
                }
                bool ok = true;
                for (int kt = 0; kt < num_kt; ++kt) {
                    // the scale writers fill a slot only after this stage's copies landed,
                    // so their signal covers the stage too
                    const int slot = static_cast<int>(kt_all & 1u);
                    if (!mbar_wait(&sf_full[slot], (kt_all >> 1) & 1u, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    ++kt_all;
                    tc_fence_after();
                    const int nkb = min(4, kb_total - kt * 4);
                    const uint32_t a_base = smem_u32(sA + stage * G::A_BYTES);
                    const uint32_t b_base = smem_u32(sB + stage * G::B_BYTES);
                    for (int j = 0; j < nkb; ++j) {
                        mma_nvf4(acc, sdesc_kmajor_sw128(a_base + j * 32), sdesc_kmajor_sw128(b_base + j * 32),
                                 G::IDESC, G::TP::sfa(tmem, slot, j), G::TP::sfb(tmem, slot, j),
                                 (kt > 0 || j > 0) ? 1u : 0u);
                    }
                    mma_commit(&empty[stage]);
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit(acc_full);
            }
        }
    } else if (warp >= 6) {
        // ----------------------------------------------------- scale writers --
        const int q = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        uint32_t stage = 0, phase = 0, kt_all = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
            for (int kt = 0; kt < num_kt; ++kt) {
                const int slot = static_cast<int>(kt_all & 1u);
                if (!mbar_wait(&full[stage], phase, err, kErrTimeoutEpi)) {
                    ok = false;
                    break;
                }
                const int nkb = min(4, kb_total - kt * 4);
                // A: the MMA reads row m's word at lane m, column base + m/32 -> this
                // quarter writes its own rows' words into column base + q.
                // B: output rows of lane quarter q read B row n's word at lane
                // 32q + n%32, column base + n/32 -> every quarter holds all four
                // words of each 128-row atom (16 bytes per lane).
                // The words are read into registers before the slot is free, so only
                // the TMEM stores remain once it is.
                const uint8_t* a = sSFA + stage * G::SFA_BYTES + lane * 16 + q * 4;
                const uint8_t* b = sSFB + stage * G::SFB_BYTES + lane * 16;
                uint32_t wa[4];
                uint4 wb[4][BN / 128];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < nkb) {
                        wa[j] = *reinterpret_cast<const uint32_t*>(a + j * 512);
#pragma unroll
                        for (int nb = 0; nb < BN / 128; ++nb)
                            wb[j][nb] = *reinterpret_cast<const uint4*>(b + nb * 2048 + j * 512);
                    }
                }
                // the slot was last used by k-tile kt_all - 2, whose MMAs completing also
                // released its stage: wait on that stage's empty barrier for that use
                if (kt_all >= 2) {
                    const uint32_t prev = kt_all - 2;
                    if (!mbar_wait(&empty[prev % G::STAGES], (prev / G::STAGES) & 1u, err, kErrTimeoutEpi)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < nkb) {
                        tmem_st_32x32b_x1(G::TP::sfa(tmem, slot, j) + lane_base + q, wa[j]);
#pragma unroll
                        for (int nb = 0; nb < BN / 128; ++nb)
                            tmem_st_32x32b_x4(G::TP::sfb(tmem, slot, j) + nb * 4 + lane_base, wb[j][nb]);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sf_full[slot]);
                ++kt_all;
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue --
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const float alpha = __fmul_rn(*scaleA, *scaleB);
        float* stg = sStage + (warp - 2) * 2 * 32 * 32;
        // C is a stream that no later tile reads: its lines leave L2 first, so the
        // operand that is reused keeps its place
        const uint64_t c_policy = l2_policy_evict_first();
        int local = 0;
        for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++local) {
            int m_idx, n_idx;
            tile_mn(tile, m_idx, n_idx);
            const int buf = local & 1;
            if (!mbar_wait(acc_full, local & 1, err, kErrTimeoutEpi)) break;
            tc_fence_after();
            const int row0 = m_idx * BM + q * 32;
            // buffer 0 drains the columns it shares with buffer 1 first
            auto chunk_col = [&](int ci) { return buf == 0 ? (ci + G::TP::FIRST) % G::TP::NCH : ci; };
            auto chunk_addr = [&](int ci) {
                return tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::ACC_OFF + chunk_col(ci) * 32;
            };
            auto store_chunk = [&](int ci, const uint32_t (&v)[32]) {
                // staging tile (ci & 1) is free once the store issued two chunks ago has read it
                float* tile = stg + (ci & 1) * 32 * 32;
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
                stage_row(tile, lane, v, alpha);
                fence_proxy_async_smem();
                __syncwarp();
                const int col0 = n_idx * BN + chunk_col(ci) * 32;
                if (lane == 0 && row0 < M && col0 < N) tma_store_2d_hint(&tmC, tile, col0, row0, c_policy);
                if (lane == 0) bulk_commit();
            };
            // the chunks the next tile's accumulator reuses go to registers first, so the
            // MMA warp can start that tile before they are staged and stored
            constexpr int RA = G::TP::RELEASE_AFTER;
            uint32_t vr[RA][32];
#pragma unroll
            for (int ci = 0; ci < RA; ++ci) tmem_ld_32x32b_x32(chunk_addr(ci), vr[ci]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tmem_free);
#pragma unroll
            for (int ci = 0; ci < RA; ++ci) store_chunk(ci, vr[ci]);
#pragma unroll 1
            for (int ci = RA; ci < G::TP::NCH; ++ci) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(chunk_addr(ci), v);
                tmem_wait_ld();
                store_chunk(ci, v);
            }
        }
        if (lane == 0) bulk_wait<0>();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------ CTA-pair kernel --
// Cluster of 2 CTAs computes a 256 x 256 tile: CTA r holds A rows [128r, 128r+128)
// of the tile and B rows [128r, 128r+128) of its N range, plus the scale atoms for
// its A rows and for all 256 B rows.  Each CTA's warps 6..9 write those scales into
// its own TMEM (tcgen05.st) and report to the even CTA, which issues
// tcgen05.mma.cta_group::2 (M=256, N=256, K=64); each CTA's TMEM receives its
// 128 rows of the accumulator.  Per stage a CTA loads 16 + 16 KB of codes instead of
// 16 + 32 KB, so operand bytes per FLOP drop by a third.
//   - The odd CTA's warp 1 relays "my stage is full" to the even CTA with a
//     remote mbarrier arrive.
//   - The even CTA's MMA thread commits stage-empty and tile-done separately to
//     each CTA's barriers.
//   - Both CTAs' epilogue warps report a drained overlap chunk to the even CTA.
struct CfgPair {
    static constexpr int STAGES = 5;
    static constexpr int A_BYTES = BM * K_TILE_BYTES;         // own 128 A rows
    static constexpr int B_BYTES = 128 * K_TILE_BYTES;        // own half of the 256 B rows
    static constexpr int SFA_BYTES = 4 * 512;                 // own A rows, 4 k-blocks
    static constexpr int SFB_BYTES = 2 * 4 * 512;             // all 256 B rows, 4 k-blocks
    static constexpr int BN = 256;
    using TP = TmemPlan<256>;
    static constexpr int ACC_OFF = TP::ACC_OFF;
    static constexpr int STG_BYTES = 4 * 2 * 32 * 32 * 4;
    static constexpr int BAR_BYTES = 512;
    static constexpr int SMEM = STAGES * (A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES) + STG_BYTES + BAR_BYTES + 1024;
    static constexpr uint32_t IDESC = idesc_nvf4(256, 256);
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
    w4a4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmC, const uint8_t* __restrict__ sfA,
                          const uint8_t* __restrict__ sfB, const float* __restrict__ scaleA,
                          const float* __restrict__ scaleB, int M, int N, int K, unsigned int* __restrict__ err) {
    using G = CfgPair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    uint8_t* sA = smem;
    uint8_t* sB = sA + G::STAGES * G::A_BYTES;
    uint8_t* sSFA = sB + G::STAGES * G::B_BYTES;
    uint8_t* sSFB = sSFA + G::STAGES * G::SFA_BYTES;
    float* sStage = reinterpret_cast<float*>(sSFB + G::STAGES * G::SFB_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sStage) + G::STG_BYTES);
    uint64_t* empty = full + G::STAGES;
    uint64_t* peer_full = empty + G::STAGES;   // even CTA only: the odd CTA's stage landed
    uint64_t* acc_full = peer_full + G::STAGES;
    uint64_t* tmem_free = acc_full + 1;        // even CTA only: 4 + 4 epilogue warps
    uint64_t* sf_full = tmem_free + 1;         // [2] even CTA only: 4 + 4 scale-writer warps
    uint64_t* sf_free = sf_full + 2;           // [2] both CTAs: the MMAs of that slot completed
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sf_free + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_mp = (M + 255) / 256, num_n = (N + 255) / 256;
    const int num_tiles = num_mp * num_n;
    const int kb_total = K / 64;
    const int num_kt = (kb_total + 3) / 4;
    const int sfa_row_blocks = (M + 127) / 128;
    const int sfb_row_blocks = (N + 127) / 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&peer_full[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(tmem_free, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sf_full[i], 8);
            mbar_init(&sf_free[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmC);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- producer --
            uint32_t stage = 0, phase = 0;
            for (int tile = pair; tile < num_tiles; tile += npairs) {
                const int mp = tile % num_mp, n_idx = tile / num_mp;
                const int rbA = mp * 2 + static_cast<int>(rank);
                const bool sfa_ok = rbA < sfa_row_blocks;
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, err, kErrTimeoutTma)) goto producer_done;
                    const int nkb = min(4, kb_total - kt * 4);
                    int nb_valid = 0;
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) nb_valid += (n_idx * 2 + nb < sfb_row_blocks);
                    const uint32_t bytes = G::A_BYTES + G::B_BYTES + nkb * 512 * ((sfa_ok ? 1 : 0) + nb_valid);
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    tma_load_2d(sA + stage * G::A_BYTES, &tmA, &full[stage], kt * K_TILE_BYTES, rbA * BM);
                    tma_load_2d(sB + stage * G::B_BYTES, &tmB, &full[stage], kt * K_TILE_BYTES,
                                n_idx * 256 + static_cast<int>(rank) * 128);
                    if (sfa_ok)
                        bulk_load(sSFA + stage * G::SFA_BYTES, sfA + ((int64_t)rbA * kb_total + kt * 4) * 512,
                                  nkb * 512, &full[stage]);
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        const int rb = n_idx * 2 + nb;
                        if (rb < sfb_row_blocks)
                            bulk_load(sSFB + stage * G::SFB_BYTES + nb * 2048,
                                      sfB + ((int64_t)rb * kb_total + kt * 4) * 512, nkb * 512, &full[stage]);
                    }
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        producer_done:;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // -------------------------------------------------- MMA (even CTA) --
            const uint32_t peer_acc_full = mapa_shared(smem_u32(acc_full), 1);
            uint32_t stage = 0, phase = 0, kt_all = 0;
            int local = 0;
            bool ok = true;
            for (int tile = pair; tile < num_tiles && ok; tile += npairs, ++local) {
                const uint32_t acc = tmem + (local & 1) * G::ACC_OFF;
                if (local > 0) {
                    if (!mbar_wait(tmem_free, (local - 1) & 1, err, kErrTimeoutMma)) break;
                    tc_fence_after();
                }
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait(&full[stage], phase, err, kErrTimeoutMma) ||
                        !mbar_wait(&peer_full[stage], phase, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    const int slot = static_cast<int>(kt_all & 1u);
                    // both CTAs' scale writers have filled this slot of their TMEM
                    if (!mbar_wait_cluster(&sf_full[slot], (kt_all >> 1) & 1u, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    ++kt_all;
                    tc_fence_after();
                    const int nkb = min(4, kb_total - kt * 4);
                    const uint32_t a_base = smem_u32(sA + stage * G::A_BYTES);
                    const uint32_t b_base = smem_u32(sB + stage * G::B_BYTES);
                    for (int j = 0; j < nkb; ++j) {
                        mma_nvf4_pair(acc, sdesc_kmajor_sw128(a_base + j * 32), sdesc_kmajor_sw128(b_base + j * 32),
                                      G::IDESC, G::TP::sfa(tmem, slot, j), G::TP::sfb(tmem, slot, j),
                                      (kt > 0 || j > 0) ? 1u : 0u);
                    }
                    mma_commit_pair(smem_u32(&empty[stage]));
                    mma_commit_pair(mapa_shared(smem_u32(&empty[stage]), 1));
                    mma_commit_pair(smem_u32(&sf_free[slot]));
                    mma_commit_pair(mapa_shared(smem_u32(&sf_free[slot]), 1));
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair(smem_u32(acc_full));
                mma_commit_pair(peer_acc_full);
            }
        } else if (lane == 0) {
            // ------------------------------------------- relay (odd CTA) --
            uint32_t stage = 0, phase = 0;
            for (int tile = pair; tile < num_tiles; tile += npairs) {
                bool ok = true;
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait(&full[stage], phase, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_cluster(mapa_shared(smem_u32(&peer_full[stage]), 0));
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
        }
    } else if (warp >= 6) {
        // ----------------------------------------------------- scale writers --
        // Same TMEM layout as the single-CTA kernel, in each CTA's own TMEM: its A
        // rows' words (x1, column base + q) and all 256 B rows' words (x4 per atom).
        const int q = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        uint32_t stage = 0, phase = 0, kt_all = 0;
        bool ok = true;
        for (int tile = pair; tile < num_tiles && ok; tile += npairs) {
            for (int kt = 0; kt < num_kt; ++kt) {
                const int slot = static_cast<int>(kt_all & 1u);
                if (!mbar_wait(&full[stage], phase, err, kErrTimeoutEpi) ||
                    (kt_all >= 2 && !mbar_wait(&sf_free[slot], ((kt_all >> 1) - 1) & 1u, err, kErrTimeoutEpi))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int nkb = min(4, kb_total - kt * 4);
                const uint8_t* a = sSFA + stage * G::SFA_BYTES + lane * 16 + q * 4;
                const uint8_t* b = sSFB + stage * G::SFB_BYTES + lane * 16;
                for (int j = 0; j < nkb; ++j) {
                    tmem_st_32x32b_x1(G::TP::sfa(tmem, slot, j) + lane_base + q,
                                      *reinterpret_cast<const uint32_t*>(a + j * 512));
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb)
                        tmem_st_32x32b_x4(G::TP::sfb(tmem, slot, j) + nb * 4 + lane_base,
                                          *reinterpret_cast<const uint4*>(b + nb * 2048 + j * 512));
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sf_full[slot]), 0));
                ++kt_all;
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue --
        const int q = warp & 3;
        const float alpha = __fmul_rn(*scaleA, *scaleB);
        float* stg = sStage + (warp - 2) * 2 * 32 * 32;
        const uint32_t leader_tmem_free = mapa_shared(smem_u32(tmem_free), 0);
        int local = 0;
        for (int tile = pair; tile < num_tiles; tile += npairs, ++local) {
            const int mp = tile % num_mp, n_idx = tile / num_mp;
            const int buf = local & 1;
            if (!mbar_wait(acc_full, local & 1, err, kErrTimeoutEpi)) break;
            tc_fence_after();
            const int row0 = (mp * 2 + static_cast<int>(rank)) * BM + q * 32;
#pragma unroll 1
            for (int ci = 0; ci < G::TP::NCH; ++ci) {
                const int c = buf == 0 ? (ci + G::TP::FIRST) % G::TP::NCH : ci;
                const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::ACC_OFF + c * 32;
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr, v);
                tmem_wait_ld();
                if (ci == G::TP::RELEASE_AFTER - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(leader_tmem_free);
                }
                float* tile = stg + (ci & 1) * 32 * 32;
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
                stage_row(tile, lane, v, alpha);
                fence_proxy_async_smem();
                __syncwarp();
                const int col0 = n_idx * 256 + c * 32;
                if (lane == 0 && row0 < M && col0 < N) tma_store_2d(&tmC, tile, col0, row0);
                if (lane == 0) bulk_commit();
            }
        }
        if (lane == 0) bulk_wait<0>();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

nvfp4_status launch_gemm_pair(const nvfp4_tensor& A, const nvfp4_tensor& B, float* C, int64_t ldc, cudaStream_t st) {
    using G = CfgPair;
    const int M = static_cast<int>(A.rows), N = static_cast<int>(B.rows), K = static_cast<int>(A.cols);
    CUtensorMap ta, tb, tc;
    nvfp4_status s = make_tmap_u8_sw128(&ta, A.codes, A.rows, A.cols / 2, BM, K_TILE_BYTES);
    if (s != NVFP4_OK) return s;
    s = make_tmap_u8_sw128(&tb, B.codes, B.rows, B.cols / 2, 128, K_TILE_BYTES);
    if (s != NVFP4_OK) return s;
    s = make_tmap_f32_sw128(&tc, C, A.rows, B.rows, ldc, 32, 32);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce attr_once;
    if ((s = smem_limit_once(attr_once, w4a4_gemm_pair_kernel, G::SMEM, "cudaFuncSetAttribute(gemm pair smem)")) !=
        NVFP4_OK)
        return s;
    unsigned int* err = device_error_word();
    if (!err) return fail(NVFP4_ERR_CUDA, "device error word unavailable");
    const int tiles = ((M + 255) / 256) * ((N + 255) / 256);
    const int pairs = tiles < num_sms() / 2 ? tiles : num_sms() / 2;
    w4a4_gemm_pair_kernel<<<pairs * 2, 320, G::SMEM, st>>>(ta, tb, tc, A.sf, B.sf, A.global_scale, B.global_scale, M,
                                                          N, K, err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "w4a4_gemm pair launch");
    return NVFP4_OK;
}

template <int BN>
nvfp4_status launch_gemm(const nvfp4_tensor& A, const nvfp4_tensor& B, float* C, int64_t ldc, cudaStream_t st) {
    using G = Cfg<BN>;
    const int M = static_cast<int>(A.rows), N = static_cast<int>(B.rows), K = static_cast<int>(A.cols);
    CUtensorMap ta, tb, tc;
    nvfp4_status s = make_tmap_u8_sw128(&ta, A.codes, A.rows, A.cols / 2, BM, K_TILE_BYTES);
    if (s != NVFP4_OK) return s;
    s = make_tmap_u8_sw128(&tb, B.codes, B.rows, B.cols / 2, BN, K_TILE_BYTES);
    if (s != NVFP4_OK) return s;
    s = make_tmap_f32_sw128(&tc, C, A.rows, B.rows, ldc, 32, 32);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce attr_once;
    if ((s = smem_limit_once(attr_once, w4a4_gemm_kernel<BN>, G::SMEM, "cudaFuncSetAttribute(gemm smem)")) != NVFP4_OK)
        return s;
    unsigned int* err = device_error_word();
    if (!err) return fail(NVFP4_ERR_CUDA, "device error word unavailable");
    const int tiles = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
    const int grid = tiles < num_sms() ? tiles : num_sms();
    const cudaError_t e = launch_pdl(w4a4_gemm_kernel<BN>, dim3(grid), dim3(320), G::SMEM, st, ta, tb, tc, A.sf, B.sf,
                                     A.global_scale, B.global_scale, M, N, K, err);
    if (e != cudaSuccess) return cuda_fail(e, "w4a4_gemm launch");
    return NVFP4_OK;
}

}  // namespace

nvfp4_status validate_tensor(const nvfp4_tensor* t, const char* name);

// Kernel choice.  NVFP4_GEMM_VARIANT=pair|single|narrow forces one (tests
// cover each); by default the single-CTA 128 x 256 kernel takes problems with
// at least one tile per SM and the 128 x 128 kernel smaller / decode shapes.
// The CTA-pair kernel measured slower (a cross-SM round trip per k-tile on its
// two-slot scale ring) and is only used on request.
static int gemm_variant_override() {
    const char* e = getenv("NVFP4_GEMM_VARIANT");
    if (e && !strcmp(e, "pair")) return 1;
    if (e && !strcmp(e, "single")) return 2;
    if (e && !strcmp(e, "narrow")) return 3;
    return 0;
}

nvfp4_status gemm_launch(const nvfp4_tensor& A, const nvfp4_tensor& B, float* C, int64_t ldc, cudaStream_t st) {
    const int64_t M = A.rows, N = B.rows;
    switch (gemm_variant_override()) {
        case 1: return launch_gemm_pair(A, B, C, ldc, st);
        case 2: return launch_gemm<256>(A, B, C, ldc, st);
        case 3: return launch_gemm<128>(A, B, C, ldc, st);
        default: break;
    }
    const int64_t tiles256 = ((M + BM - 1) / BM) * ((N + 255) / 256);
    if (N <= 128 || tiles256 < num_sms()) return launch_gemm<128>(A, B, C, ldc, st);
    return launch_gemm<256>(A, B, C, ldc, st);
}

}  // namespace nvg

extern "C" nvfp4_status w4a4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, float* C, int64_t ldc,
                                  nvfp4_stream_t stream) {
    using namespace nvg;
    nvfp4_status s = validate_tensor(A, "A");
    if (s != NVFP4_OK) return s;
    s = validate_tensor(B, "B");
    if (s != NVFP4_OK) return s;
    if (A->cols != B->cols) return fail(NVFP4_ERR_INVALID_ARG, "A and B have different K");
    if (!C) return fail(NVFP4_ERR_INVALID_ARG, "C is null");
    if (B->rows % 4) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "N must be a multiple of 4");
    if (ldc < B->rows) return fail(NVFP4_ERR_INVALID_ARG, "ldc < N");
    if (!aligned16(C) || ldc % 4) return fail(NVFP4_ERR_MISALIGNED, "C / ldc not 16-byte aligned");
    if (A->rows > (int64_t(1) << 30) || B->rows > (int64_t(1) << 30))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "M or N too large");
    return gemm_launch(*A, *B, C, ldc, as_stream(stream));
}

// gemm_fused.cu -- products with a fused epilogue, for 8-bit and for NVFP4 operands:
//
//   C[m, n] = act(p[m, n] + bias[n]) + R[m, n]
//   8-bit:  p = sA[m] sB[n] sum_k e4m3(A)[m, k] e4m3(B)[n, k]        (one scale a row)
//   NVFP4:  p = S_A S_B sum_k (e2m1(A) e4m3(sfA))[m, k] (e2m1(B) e4m3(sfB))[n, k]
//
// The 8-bit operands' row scales factor out of the sum, so the tensor cores see plain
// E4M3 (tcgen05.mma kind::f8f6f4) and the scales are applied once per output element;
// the NVFP4 block scales go to the tensor cores (kind::mxf4nvf4).  Accumulators are
// float32 in TMEM.
//
// All kernels put B's rows (n, the weight) on the accumulator's lanes and A's rows (the
// tokens) on its columns; see epilogue.cuh for why.  Operand tiles are 128 bytes of a
// row wide (128 E4M3 or 256 E2M1 values) and a tensor-core step 32 bytes, so both kinds
// share one geometry: TMA with the 128-byte swizzle fills a ring of stages, K's tail is
// zero-filled by the copies.  NVFP4 stages also hold the tile's 512-byte scale atoms
// (128 rows x 64 values); tcgen05.cp takes each to TMEM just before the step that
// reads it.
//
// Single-thread roles are entered through elect.sync: the compiler then knows that one
// lane runs them and issues each tcgen05 instruction straight from uniform registers.
// Behind `lane == 0` the issue itself was the limit: without copies and epilogue the
// 8-bit pair kernel's loop ran at 2.69 PFLOP/s (8192 x 8192 x 4096), elected at 4.06.
//
// Every wait is bounded: on expiry the kernel records a code in the device error word,
// waits (again bounded) for the copies and products it has in flight, frees its TMEM and
// returns; what it has not stored by then it does not store.
#include "epilogue.cuh"

namespace nvg {

nvfp4_status validate_fp8(const fp8_tensor* t, const char* name);
nvfp4_status validate_tensor(const nvfp4_tensor* t, const char* name);

namespace {

constexpr int kTileK = 128;         // bytes of K per stage
constexpr int kStepK = 32;          // bytes of K per tensor-core step
constexpr int kAtoms = 4;           // NVFP4: scale atoms of a 128-row block per stage
constexpr int kAtomBytes = 512;

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

// One 512-byte scale atom (32 rows x 16 bytes, no swizzle, 8-row groups 128 bytes
// apart) from shared memory to four TMEM columns, replicated to the four 32-lane
// quarters; in a pair, each CTA's shared memory at this offset to its own TMEM.
__device__ __forceinline__ uint64_t sdesc_scale_atom(uint32_t saddr) { return sdesc_noswz(saddr, 16, 128); }
__device__ __forceinline__ void cp_scale_atom(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void cp_scale_atom_pair(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
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

struct Maps {
    CUtensorMap w, x;       // codes of the weight and of the tokens
    CUtensorMap sw, sx;     // NVFP4: their scale atoms
    CUtensorMap tail;       // pair kernel: codes of the tokens in boxes of a narrow tile
};

struct FusedArgs {
    const float* sA;   // 8-bit: [M] token scales; NVFP4: the tensor's scale
    const float* sB;   // 8-bit: [N] weight-row scales; NVFP4: the tensor's scale
    int row_bytes;     // bytes of a row's K codes
    int tail_from;     // pair kernel: the tiles from this one on are cut into
    int tail_shift;    //   2^tail_shift narrow ones
    int chain_tiles;   // 8-bit, kernels with chains: k-tiles summed in one chain at most
    int stalled_rank;  // split-K kernel: the CTA of each cluster that copies nothing (-1; self-test)
    unsigned int* err;
    EpiArgs epi;
};

// ------------------------------------------------------------ CTA-pair kernel --
// Long prefills.  A cluster of two CTAs computes 256 weight rows x 256 tokens: CTA r
// holds weight rows [128 r, 128 r + 128) of the tile and tokens [128 r, ...) of the
// tile's tokens, so a stage brings 32 KB of codes for 128 x 256 outputs.  The odd CTA's
// copies signal the even CTA's barriers directly, so the issuing thread waits on one
// barrier a stage.
//
// Two accumulators of 256 columns, one drained while the other is filled.  With E4M3
// they are all of TMEM.  With NVFP4 the scale columns of one stage take the top 48 (the
// tensor pipe runs one thread's copies and products in order, so the next stage's copies
// come after the products that read this one's), and the accumulators share columns 208 ..
// 255: each epilogue warp reads its part of those first, into registers, and then lets the
// next tile begin.  (Two alternating stages of scale columns and 96 shared ones made the
// next tile wait for a second round of reads: 4096 x 5120 x 4096 54 us, now 50.)
//
// Sixteen epilogue warps, because short K is bound by the epilogue's instructions:
// 8-bit 8192 x 4096 x 256 with SiLU took 43 us with eight and 38 with sixteen.  For long
// K the power limit binds: in a loop, 8-bit 8192 x 12352 x 5120 runs at 1.1 to 1.3 GHz
// and 2.4 PFLOP/s, 0.87 of twice the measured sustained bf16 rate.
//
// Tiles left over for a last round that they do not fill are cut into narrow ones of 128
// or 64 tokens (NVFP4 128, a scale block), if all of these fit that round: it then ends
// after half or a quarter of a tile's epilogue and a shorter loop.
template <bool kFp4>
struct Pair {
    static constexpr int A_BYTES = 128 * kTileK;                            // own weight rows
    static constexpr int B_BYTES = 128 * kTileK;                            // own half of the tokens
    static constexpr int SFA_BYTES = kFp4 ? kAtoms * kAtomBytes : 0;        // own weight rows
    static constexpr int SFB_BYTES = kFp4 ? 2 * kAtoms * kAtomBytes : 0;    // all 256 tokens
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGES = kFp4 ? 5 : 6;                             // 4 to 7 measured the same (8-bit)
    static constexpr int EPI_WARPS = 16;
    static constexpr int EPI_COLS = 1024 / EPI_WARPS;                       // token columns per epilogue warp
    static constexpr int SCALES = kFp4 ? 0 : EPI_WARPS * EPI_COLS * 4;      // token scales of each warp
    static constexpr int SMEM = STAGES * STAGE_BYTES + SCALES + 256 + 1024;
    __host__ __device__ static constexpr uint32_t idesc(int N) { return kFp4 ? idesc_nvf4(256, N) : idesc_e4m3(256, N); }
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    // TMEM columns: per step of a stage 4 scale columns for A and 8 for B
    static constexpr int SF_STEP = 12, SF_BASE = 512 - kAtoms * SF_STEP;
    static constexpr int ACC_OFF = kFp4 ? SF_BASE - 256 : 256;
    static constexpr int SHARED = (256 - ACC_OFF) / 16;                     // 16-column chunks in both accumulators
};
static_assert(Pair<true>::SMEM <= 232448 && Pair<false>::SMEM <= 232448, "shared memory of one CTA");

// Sums of 8-bit products in several chains of k-tiles, see fused_launch.  The first chain goes
// to one accumulator and each later one to another; the epilogue warps add the second to the
// first, rounding to nearest, before the next chain begins, and the last chain as they read it.
struct Chains {
    int count, tiles;
    // first tile after chain i
    __device__ __forceinline__ int end(int i) const { return (tiles * (i + 1) + count - 1) / count; }
};

// C columns of both accumulators, added (rounded to nearest), in acc.
template <int C>
__device__ __forceinline__ void add_chain(uint32_t first, uint32_t second, uint32_t (&acc)[C]) {
    uint32_t last[C];
    tmem_ld_cols<C>(first, acc);
    tmem_ld_cols<C>(second, last);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < C; ++j) acc[j] = __float_as_uint(__uint_as_float(acc[j]) + __uint_as_float(last[j]));
}

// kChains (8-bit): two or more chains, the first in the first accumulator.
template <bool kFp4, bool kChains>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair<kFp4>::THREADS, 1)
    fused_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ FusedArgs args) {
    using G = Pair<kFp4>;
    static_assert(!(kFp4 && kChains), "chains are for 8-bit operands");
    // one accumulator signal per tile instead of one per buffer
    constexpr bool kOneSignal = kFp4 || kChains;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    float* scales = reinterpret_cast<float*>(smem + G::STAGES * G::STAGE_BYTES);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::STAGES * G::STAGE_BYTES + G::SCALES);   // even CTA's are used
    uint64_t* empty = full + G::STAGES;
    // kChains: [0] for the tile, [1] for each join of chains
    uint64_t* acc_full = empty + G::STAGES;   // [2] by buffer
    uint64_t* acc_free = acc_full + 2;        // even CTA's are used; [2] by buffer, or one with a phase a tile (kOneSignal)
    uint64_t* drained = acc_free + 2;         // products in flight, after an expired wait
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_m = (args.epi.M + 255) / 256, num_n = (args.epi.N + 255) / 256;
    const int tail_from = args.tail_from, tail_shift = args.tail_shift;
    const int num_units = tail_from + ((num_m * num_n - tail_from) << tail_shift);
    const int num_kt = (args.row_bytes + kTileK - 1) / kTileK;
    const Chains chains = {kChains ? max(2, (num_kt + args.chain_tiles - 1) / args.chain_tiles) : 1, num_kt};
    unsigned int* err = args.err;
    // Tiles run in bands of 16 token tiles, weight tiles slowest inside a band, so that the
    // tiles in flight share rows of both operands (8192 x 12352 x 5120 fp32 under a steady load:
    // bands of 4, 8, 16, 32 take 484, 471, 464, 472 us; on another card 8 and 16 take 486, 479).
    struct Unit {
        int m0, n_idx, shift;   // first token, weight tile, 256 >> shift tokens
    };
    auto unit_of = [&](int u) {
        Unit r;
        r.shift = u < tail_from ? 0 : tail_shift;
        const int cut = u - tail_from, tile = u < tail_from ? u : tail_from + (cut >> tail_shift);
        const int band = tile / (16 * num_n), first = band * 16;
        const int width = min(16, num_m - first), in = tile - band * 16 * num_n;
        r.n_idx = in / width;
        r.m0 = (first + in % width) * 256 + (u < tail_from ? 0 : (cut & ((1 << tail_shift) - 1)) << (8 - tail_shift));
        return r;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 2 * G::EPI_WARPS);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, 512);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&maps.w);
        prefetch_tmap(&maps.x);
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_and_trigger();

    if (warp == 0) {
        if (elect_one()) {
            // ---------------------------------------------------- producer --
            const int kb_total = args.row_bytes / kStepK;   // NVFP4: scale atoms along K
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int u = pair; u < num_units && ok; u += npairs) {
                const Unit w = unit_of(u);
                const CUtensorMap* x = w.shift ? &maps.tail : &maps.x;
                const uint32_t bytes = G::A_BYTES + (G::B_BYTES >> w.shift) + G::SFA_BYTES + (G::SFB_BYTES >> w.shift);
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, err, kErrTimeoutTma)) {
                        ok = false;
                        break;
                    }
                    // the even CTA's barrier counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
                    const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
                    uint8_t* st = smem + stage * G::STAGE_BYTES;
                    tma_load_2d_pair(st, &maps.w, bar, kt * kTileK, w.n_idx * 256 + rank * 128);
                    tma_load_2d_pair(st + G::A_BYTES, x, bar, kt * kTileK, w.m0 + (rank * 128 >> w.shift));
                    if constexpr (kFp4) {
                        // four atoms of each 128-row block; past K's end or the last block they
                        // belong to rows or steps that are not used, or are zero-filled
                        uint8_t* sf = st + G::A_BYTES + G::B_BYTES;
                        tma_load_2d_pair(sf, &maps.sw, bar, 0, (w.n_idx * 2 + rank) * kb_total + kt * kAtoms);
                        for (int b = 0; b < 2 >> w.shift; ++b)
                            tma_load_2d_pair(sf + G::SFA_BYTES + b * kAtoms * kAtomBytes, &maps.sx, bar, 0,
                                             (w.m0 / 128 + b) * kb_total + kt * kAtoms);
                    }
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // after an expired wait no CTA ends before its copies (both CTAs' count here; a stage
            // that was never filled does not wait)
            if (!ok && rank == 0) {
                for (uint32_t s = 0; s < G::STAGES; ++s)
                    mbar_wait_cluster(&full[s], s < stage ? phase : phase ^ 1u, err, kErrTimeoutTma);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            // -------------------------------------------------- MMA (even CTA) --
            const uint32_t peer_acc_full = mapa_shared(smem_u32(acc_full), 1);
            const uint32_t peer_empty = mapa_shared(smem_u32(empty), 1);
            uint32_t stage = 0, phase = 0, joins = 0;
            int local = 0;
            bool ok = true;
            for (int u = pair; u < num_units && ok; u += npairs, ++local) {
                const int buf = kChains ? 0 : local & 1, shift = u < tail_from ? 0 : tail_shift;
                int chain = 0, chain_from = 0, chain_end = chains.end(0);
                const uint32_t idesc = shift == 0 ? G::idesc(256) : shift == 1 ? G::idesc(128) : G::idesc(64);
                // 8-bit: this buffer's last tile has been read.  NVFP4: the shared columns of the
                // tile before have been; its readers had by then finished the tile before it.
                // Chains: all of the tile before has been read.
                if (kOneSignal ? local >= 1 && !mbar_wait_cluster(acc_free, (local - 1) & 1, err, kErrTimeoutMma)
                         : local >= 2 && !mbar_wait_cluster(&acc_free[buf], ((local >> 1) - 1) & 1, err, kErrTimeoutMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int kt = 0; kt < num_kt; ++kt) {
                    if (kChains && kt == chain_end) {
                        if (chain) {
                            // the second accumulator is added to the first, then free
                            mma_commit_pair(smem_u32(&acc_full[1]));
                            mma_commit_pair(peer_acc_full + 8);
                            if (!mbar_wait_cluster(&acc_free[1], joins++ & 1, err, kErrTimeoutMma)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        chain_from = kt;
                        chain_end = chains.end(++chain);
                    }
                    if (!mbar_wait_cluster(&full[stage], phase, err, kErrTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + stage * G::STAGE_BYTES), b = a + G::A_BYTES;
                    const int nk = min(4, (args.row_bytes - kt * kTileK + kStepK - 1) / kStepK);
                    const uint32_t acc = tmem + (kChains ? (chain > 0) * 256 : buf * G::ACC_OFF);
                    for (int j = 0; j < nk; ++j) {
                        const uint64_t da = sdesc_kmajor_sw128(a + j * kStepK), db = sdesc_kmajor_sw128(b + j * kStepK);
                        const uint32_t accumulate = (j > 0 || kt > chain_from) ? 1u : 0u;
                        if constexpr (kFp4) {
                            const uint32_t sfa = tmem + G::SF_BASE + j * G::SF_STEP, sfb = sfa + 4;
                            const uint32_t src = b + G::B_BYTES + j * kAtomBytes;
                            cp_scale_atom_pair(sfa, sdesc_scale_atom(src));
                            cp_scale_atom_pair(sfb, sdesc_scale_atom(src + G::SFA_BYTES));
                            if (shift == 0)
                                cp_scale_atom_pair(sfb + 4, sdesc_scale_atom(src + G::SFA_BYTES + kAtoms * kAtomBytes));
                            mma_nvf4_pair(acc, da, db, idesc, sfa, sfb, accumulate);
                        } else {
                            mma_fp8_pair(acc, da, db, idesc, accumulate);
                        }
                    }
                    mma_commit_pair(smem_u32(&empty[stage]));
                    mma_commit_pair(peer_empty + stage * 8);
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair(smem_u32(&acc_full[buf]));
                mma_commit_pair(peer_acc_full + buf * 8);
            }
            if (!ok) {
                mma_commit_pair(smem_u32(drained));
                mbar_wait_cluster(drained, 0, err, kErrTimeoutMma);
            }
        }
    } else {
        // ---------------------------------------------------------- epilogue --
        const int q = warp & 3, part = (warp - 2) >> 2;   // lane quarter, share of the columns
        const EpiArgs& e = args.epi;
        float* s = scales + (warp - 2) * G::EPI_COLS;
        const float whole = kFp4 ? __fmul_rn(*args.sA, *args.sB) : 0.0f;
        int local = 0;
        uint32_t joins = 0;
        for (int u = pair; u < num_units; u += npairs, ++local) {
            const Unit w = unit_of(u);
            const int buf = kChains ? 0 : local & 1, m_tile = w.m0;
            const int n = w.n_idx * 256 + rank * 128 + q * 32 + lane;
            // the i-th 16 columns of this warp; NVFP4: interleaved, whole tiles from the shared
            // columns on
            const int first = kFp4 && buf == 0 && w.shift == 0 ? G::ACC_OFF : 0;
            auto column = [&](int i) {
                return kFp4 ? ((part + 4 * i) * 16 + first) & 255 : part * (G::EPI_COLS >> w.shift) + i * 16;
            };
            const int rounds = 4 >> w.shift;
            // everything that does not depend on the accumulator, before the wait for it
            const float t = kFp4 ? whole : n < e.N ? args.sB[n] : 0.0f;
            const float bias = e.bias && n < e.N ? e.bias[n] : 0.0f;
            EpiResidual<16> cur, next;
            cur.load(e, m_tile + column(0), n);
            if constexpr (!kFp4) stage_token_scales(args.sA, e.M, m_tile + column(0), G::EPI_COLS, s, lane);
            if constexpr (kChains) {
                const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
                bool ok = true;
                for (int c = 2; c < chains.count && ok; ++c) {
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[1], joins++ & 1, err, kErrTimeoutEpi));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < rounds; ++i) {
                        uint32_t acc[16];
                        add_chain(taddr + column(i), taddr + 256 + column(i), acc);
                        tmem_st_32x32b_x16(taddr + column(i), acc);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_free[1]), 0));
                    __syncwarp();
                }
                if (!ok) break;
            }
            // the warp stays together whichever of its lanes saw the budget run out
            if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_full[buf], (kChains ? local : local >> 1) & 1, err, kErrTimeoutEpi))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::ACC_OFF;
            // the round after which this warp has read all that the next tile may overwrite
            const int last_shared = kFp4 && w.shift == 0 ? (G::SHARED - 1 - part) / 4 : rounds - 1;
#pragma unroll 1
            for (int i = 0; i < rounds; ++i) {
                uint32_t acc[16];
                const int c = column(i);
                // lanes past N take another path through the loads and stores of C and R, and
                // TMEM instructions want the warp together
                __syncwarp();
                if constexpr (kChains)
                    add_chain(taddr + c, taddr + 256 + c, acc);
                else
                    tmem_ld_32x32b_x16(taddr + c, acc);
                if (i + 1 < rounds) next.load(e, m_tile + column(i + 1), n);
                __syncwarp();
                tmem_wait_ld();
                if (i == last_shared) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_free[kOneSignal ? 0 : buf]), 0));
                }
                epilogue_store<16, !kFp4>(e, m_tile + c, n, acc, cur, s + i * 16, t, bias);
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
// take SPLIT consecutive ranges of K (none empty: the launch keeps four k-tiles each),
// so that weights with few row tiles still occupy every SM.  The partial accumulators
// meet in shared memory: each CTA leaves its own there and then adds, in rank order,
// the token columns that are its share, read from every CTA of the cluster.
// The order is fixed: no atomics, the same bits every time.
// kChains (8-bit): a CTA's range of K in two or more chains.
template <bool kFp4, int BN, int SPLIT, bool kChains>
struct Small {
    static_assert(!(kFp4 && kChains), "chains are for 8-bit operands");
    static constexpr int A_BYTES = 128 * kTileK;
    static constexpr int B_BYTES = BN * kTileK;
    static constexpr int SF_BYTES = kFp4 ? kAtoms * kAtomBytes : 0;   // of the weight rows, and of the tokens
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * SF_BYTES;
    // three CTAs an SM up to 32 tokens, two above (one token x 5120 x 4096, 8-bit: 5.4 us with
    // three, 6.0 with two, 6.8 with one)
    static constexpr int CTAS = BN <= 32 ? 3 : 2;
    static constexpr int STAGES = (BN <= 32 ? 73728 : 110592) / STAGE_BYTES;
    static constexpr int RING = STAGES * STAGE_BYTES;
    // token columns are finished in chunks, a run of them by each CTA of the cluster (a run of
    // two chunks of 16 would be unrolled, and spill)
    static constexpr int COLS = BN / SPLIT;
    static constexpr int CHUNK = SPLIT == 3 ? BN / 8 : COLS == 32 ? 8 : COLS < 16 ? COLS : 16;
    static constexpr int CHUNKS = BN / CHUNK;
    static constexpr int SCALES = kFp4 ? 0 : 4 * BN * 4;
    static constexpr int SMEM = RING + SCALES + 256 + 1024;
    static constexpr int ACC_COLS = BN < 32 ? 32 : BN;
    static constexpr int SF_STEP = 8;                                 // scale columns of a step: 4 for A, 4 for B
    static constexpr int USED_COLS = ACC_COLS + (kFp4 ? kAtoms * SF_STEP : kChains ? ACC_COLS : 0);
    static constexpr int TMEM_COLS = USED_COLS <= 32 ? 32 : USED_COLS <= 64 ? 64 : USED_COLS <= 128 ? 128 : 256;
    static constexpr int THREADS = 192;
    static constexpr uint32_t IDESC = kFp4 ? idesc_nvf4(128, BN) : idesc_e4m3(128, BN);
    static_assert(RING >= 128 * BN * 4, "the partial accumulators reuse the ring");
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <bool kFp4, int BN, int SPLIT, bool kChains>
__global__ void __launch_bounds__(192, Small<kFp4, BN, SPLIT, kChains>::CTAS)
    fused_small_kernel(const __grid_constant__ Maps maps, const __grid_constant__ FusedArgs args) {
    using G = Small<kFp4, BN, SPLIT, kChains>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align1024_shared(smem_raw);
    float* scales = reinterpret_cast<float*>(smem + G::RING);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::RING + (G::SCALES + 15) / 16 * 16);
    uint64_t* empty = full + G::STAGES;
    uint64_t* acc_full = empty + G::STAGES;
    uint64_t* drained = acc_full + 1;   // products in flight, after an expired wait
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
    volatile uint32_t* expired = tmem_holder + 1;   // [4] by lane quarter: a CTA of the cluster has no sum to join
    uint64_t* chain_full = reinterpret_cast<uint64_t*>(tmem_holder + 6);   // kChains: a chain to join,
    uint64_t* chain_free = chain_full + 1;                                 //   its accumulator free again

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = SPLIT > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int num_m = (args.epi.M + BN - 1) / BN;
    const int tile = blockIdx.x / SPLIT;
    const int n_idx = tile / num_m, m_idx = tile - n_idx * num_m;
    const int num_kt = (args.row_bytes + kTileK - 1) / kTileK;
    const int kt0 = num_kt * rank / SPLIT, kt1 = num_kt * (rank + 1) / SPLIT;
    const Chains chains = {kChains ? (kt1 - kt0 + args.chain_tiles - 1) / args.chain_tiles : 1, kt1 - kt0};
    unsigned int* err = args.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drained, 1);
        fence_mbar_init();
        for (int i = 0; i < 4; ++i) expired[i] = 0;
        if (kChains) {
            mbar_init(chain_full, 1);
            mbar_init(chain_free, 4);
            fence_mbar_init();
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, G::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&maps.w);
        prefetch_tmap(&maps.x);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (SPLIT > 1) cluster_arrive();   // the others may write `expired`
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait_and_trigger();

    const int q = warp & 3;
    const int n = n_idx * 128 + q * 32 + lane;
    bool ok = true;   // this warp's sum is there, and those it joins
    const EpiArgs& e = args.epi;
    const int m_tile = m_idx * BN;
    const int chunk0 = G::CHUNKS * rank / SPLIT, chunk1 = G::CHUNKS * (rank + 1) / SPLIT;
    float t = 0.0f, bias = 0.0f;
    EpiResidual<G::CHUNK> cur;
    float* s = scales + (warp - 2) * BN;
    if (warp == 0) {
        if (elect_one()) {
            const int kb_total = args.row_bytes / kStepK;   // NVFP4: scale atoms along K
            int i = 0;
            for (int kt = kt0; kt < kt1 && rank != args.stalled_rank; ++kt, ++i) {
                const int stage = i % G::STAGES;
                if (!mbar_wait(&empty[stage], ((i / G::STAGES) & 1) ^ 1, err, kErrTimeoutTma)) break;
                mbar_arrive_expect_tx(&full[stage], G::STAGE_BYTES);
                uint8_t* st = smem + stage * G::STAGE_BYTES;
                tma_load_2d(st, &maps.w, &full[stage], kt * kTileK, n_idx * 128);
                tma_load_2d(st + G::A_BYTES, &maps.x, &full[stage], kt * kTileK, m_idx * BN);
                if constexpr (kFp4) {
                    // the tokens' atoms are those of the 128-row block that the tile begins
                    // (the launch takes BN < 128 for a single tile only)
                    uint8_t* sf = st + G::A_BYTES + G::B_BYTES;
                    tma_load_2d(sf, &maps.sw, &full[stage], 0, n_idx * kb_total + kt * kAtoms);
                    tma_load_2d(sf + G::SF_BYTES, &maps.sx, &full[stage], 0, m_idx * kb_total + kt * kAtoms);
                }
            }
            // after an expired wait the CTA does not end before its copies
            if (i < kt1 - kt0)
                for (int k = max(0, i - G::STAGES); k < i; ++k)
                    mbar_wait(&full[k % G::STAGES], (k / G::STAGES) & 1, err, kErrTimeoutTma);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            bool ok = true;
            uint32_t joins = 0;
            int chain = 0, chain_from = 0, chain_end = chains.end(0);
            for (int kt = kt0, i = 0; kt < kt1; ++kt, ++i) {
                const int stage = i % G::STAGES;
                if (kChains && i == chain_end) {
                    if (chain) {
                        mma_commit(chain_full);
                        if (!mbar_wait(chain_free, joins++ & 1, err, kErrTimeoutMma)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    chain_from = i;
                    chain_end = chains.end(++chain);
                }
                if (!mbar_wait(&full[stage], (i / G::STAGES) & 1, err, kErrTimeoutMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(smem + stage * G::STAGE_BYTES), b = a + G::A_BYTES;
                const int nk = min(4, (args.row_bytes - kt * kTileK + kStepK - 1) / kStepK);
                for (int j = 0; j < nk; ++j) {
                    const uint64_t da = sdesc_kmajor_sw128(a + j * kStepK), db = sdesc_kmajor_sw128(b + j * kStepK);
                    const uint32_t accumulate = (i > chain_from || j > 0) ? 1u : 0u;
                    const uint32_t acc = kChains && chain ? tmem + G::ACC_COLS : tmem;
                    if constexpr (kFp4) {
                        const uint32_t sfa = tmem + G::ACC_COLS + j * G::SF_STEP, sfb = sfa + 4;
                        const uint32_t src = b + G::B_BYTES + j * kAtomBytes;
                        cp_scale_atom(sfa, sdesc_scale_atom(src));
                        cp_scale_atom(sfb, sdesc_scale_atom(src + G::SF_BYTES));
                        mma_nvf4(acc, da, db, G::IDESC, sfa, sfb, accumulate);
                    } else {
                        mma_fp8(acc, da, db, G::IDESC, accumulate);
                    }
                }
                mma_commit(&empty[stage]);
            }
            if (ok) {
                mma_commit(acc_full);
            } else {
                mma_commit(drained);
                mbar_wait(drained, 0, err, kErrTimeoutMma);
            }
        }
    } else {
        // what does not depend on the accumulator, before the wait for it
        if (n < e.N) {
            t = kFp4 ? __fmul_rn(*args.sA, *args.sB) : args.sB[n];
            if (e.bias) bias = e.bias[n];
        }
        cur.load(e, m_tile + chunk0 * G::CHUNK, n);
        if constexpr (!kFp4) stage_token_scales(args.sA, e.M, m_tile, BN, s, lane);
        if constexpr (kChains) {
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
            for (int c = 2; c < chains.count && ok; ++c) {
                ok = __all_sync(0xffffffffu, mbar_wait(chain_full, c & 1, err, kErrTimeoutEpi));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < BN; j += 16) {
                    uint32_t acc[16];
                    add_chain(taddr + j, taddr + G::ACC_COLS + j, acc);
                    tmem_st_32x32b_x16(taddr + j, acc);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(chain_free);
                __syncwarp();
            }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(acc_full, 0, err, kErrTimeoutEpi));
        tc_fence_after();
    }
    __syncwarp();

    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if constexpr (SPLIT > 1) {
        // partial accumulators, [column][lane row]: the ring is free, its last product done
        // (after an expired wait it may not be, and there is no sum: every CTA of the cluster is
        // told, and none stores this quarter.  Asking all of them instead costs remote reads:
        // one token x 5120 x 4096 5.3 and 5.6 us, without either 5.1)
        float* part = reinterpret_cast<float*>(smem);
        cluster_wait();
        if (warp >= 2) {
            if (!ok && lane < SPLIT) st_shared_cluster(mapa_shared(smem_u32(const_cast<uint32_t*>(expired + q)), lane), 1);
            __syncwarp();
#pragma unroll 1
            for (int c = 0; ok && c < BN; c += 16) {
                uint32_t acc[16];
                if (kChains && chains.count > 1) {
                    add_chain(taddr + c, taddr + G::ACC_COLS + c, acc);
                } else {
                    tmem_ld_32x32b_x16(taddr + c, acc);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = __uint_as_float(acc[j]);
            }
        }
        cluster_sync();
        if (warp >= 2) ok = expired[q] == 0;
    }
    if (warp >= 2) {
#pragma unroll 1
        for (int k = chunk0; k < chunk1; ++k) {
            const int c = k * G::CHUNK;
            uint32_t acc[G::CHUNK];
            EpiResidual<G::CHUNK> next;
            if (k + 1 < chunk1) next.load(e, m_tile + c + G::CHUNK, n);
            if constexpr (SPLIT > 1) {
                const uint32_t at = smem_u32(smem) + (c * 128 + q * 32 + lane) * 4;
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
                __syncwarp();   // as in the pair kernel
                if constexpr (kChains) {
                    add_chain(taddr + c, taddr + G::ACC_COLS + c, acc);
                } else {
                    tmem_ld_cols<G::CHUNK>(taddr + c, acc);
                    tmem_wait_ld();
                }
            }
            epilogue_store<G::CHUNK, !kFp4>(e, m_tile + c, ok ? n : e.N, acc, cur, s + c, t, bias);
            cur = next;
        }
    }
    __syncwarp();
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
// One operand as the launches see it.
struct Operand {
    const uint8_t* codes;
    const uint8_t* sf;     // NVFP4: scale atoms
    int64_t rows, row_bytes, ld;
};

nvfp4_status operand_maps(const Operand& o, int box_rows, CUtensorMap* codes, CUtensorMap* atoms) {
    nvfp4_status s = make_tmap_u8_sw128_ld(codes, o.codes, o.rows, o.row_bytes, o.ld, box_rows, kTileK);
    if (s == NVFP4_OK && o.sf)
        s = make_tmap_atoms(atoms, o.sf, (o.rows + 127) / 128 * (o.row_bytes / kStepK), kAtoms);
    return s;
}

template <bool kFp4, bool kChains>
nvfp4_status launch_pair(const Operand& X, const Operand& W, const FusedArgs& args, cudaStream_t st) {
    using G = Pair<kFp4>;
    Maps maps = {};
    nvfp4_status s = operand_maps(W, 128, &maps.w, &maps.sw);
    if (s == NVFP4_OK) s = operand_maps(X, 128, &maps.x, &maps.sx);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce once;
    static std::atomic<int> resident[64];   // pairs that fit at once, per device
    int dev = 0;
    cudaGetDevice(&dev);
    s = once_per_device(once, [&]() -> nvfp4_status {
        cudaError_t e = cudaFuncSetAttribute(fused_pair_kernel<kFp4, kChains>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(fused pair smem)");
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms() / 2 * 2);
        cfg.blockDim = dim3(G::THREADS);
        cfg.dynamicSmemBytes = G::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, fused_pair_kernel<kFp4, kChains>, &cfg);
        if (e != cudaSuccess || n < 1) return cuda_fail(e, "fused pair occupancy");
        resident[dev].store(n < num_sms() / 2 ? n : num_sms() / 2, std::memory_order_relaxed);
        return NVFP4_OK;
    });
    if (s != NVFP4_OK) return s;
    const int64_t tiles = ((X.rows + 255) / 256) * ((W.rows + 255) / 256);
    const int64_t most = resident[dev].load(std::memory_order_relaxed);
    const int64_t left = tiles % most;
    FusedArgs a = args;
    a.tail_shift = !kFp4 && left * 4 <= most ? 2 : left * 2 <= most ? 1 : 0;
    a.tail_from = static_cast<int>(tiles - left);
    if (a.tail_shift && left) {
        s = make_tmap_u8_sw128_ld(&maps.tail, X.codes, X.rows, X.row_bytes, X.ld, 128 >> a.tail_shift, kTileK);
        if (s != NVFP4_OK) return s;
    }
    const int64_t units = a.tail_from + (left << a.tail_shift);
    const unsigned pairs = static_cast<unsigned>(units < most ? units : most);
    const cudaError_t e = launch_pdl(fused_pair_kernel<kFp4, kChains>, dim3(pairs * 2), dim3(G::THREADS), G::SMEM, st, maps, a);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "fused pair launch");
}

template <bool kFp4, int BN, int SPLIT, bool kChains = false>
nvfp4_status launch_small(const Operand& X, const Operand& W, const FusedArgs& args, cudaStream_t st) {
    using G = Small<kFp4, BN, SPLIT, kChains>;
    if constexpr (!kFp4 && !kChains) {
        const int64_t num_kt = (args.row_bytes + kTileK - 1) / kTileK;
        if ((num_kt + SPLIT - 1) / SPLIT > args.chain_tiles) return launch_small<kFp4, BN, SPLIT, true>(X, W, args, st);
    }
    if (args.stalled_rank >= SPLIT) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "K is not split for these sizes");
    Maps maps = {};
    nvfp4_status s = operand_maps(W, 128, &maps.w, &maps.sw);
    if (s == NVFP4_OK) s = operand_maps(X, BN, &maps.x, &maps.sx);
    if (s != NVFP4_OK) return s;
    static PerDeviceOnce once;
    if ((s = smem_limit_once(once, fused_small_kernel<kFp4, BN, SPLIT, kChains>, G::SMEM, "cudaFuncSetAttribute(fused small smem)")) !=
        NVFP4_OK)
        return s;
    const int64_t tiles = ((X.rows + BN - 1) / BN) * ((W.rows + 127) / 128);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * SPLIT));
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = SPLIT;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fused_small_kernel<kFp4, BN, SPLIT, kChains>, maps, args);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "fused small launch");
}

template <bool kFp4, int BN>
nvfp4_status launch_split(int split, const Operand& X, const Operand& W, const FusedArgs& args, cudaStream_t st) {
    if constexpr (BN < 128)
        if (split == 4) return launch_small<kFp4, BN, 4>(X, W, args, st);
    if constexpr (BN > 32)
        if (split == 3) return launch_small<kFp4, BN, 3>(X, W, args, st);
    return split == 2 ? launch_small<kFp4, BN, 2>(X, W, args, st) : launch_small<kFp4, BN, 1>(X, W, args, st);
}

// k-tiles that an 8-bit product sums in one chain at most.  The tensor cores' float32
// accumulation does not round to nearest: against float64 its error grows with the number of
// steps (activations with hot channels, of the result's norm: K = 3712, one chain, 7.1e-7; 5120
// 9.6e-7 in one, 4.4e-7 in two; 28672 3.7e-6 in two, 5.7e-7 in eight; operands of one sign about
// 2.3 times that).  So a float32 result takes at least two chains from 30 tiles (K = 3840) on, of
// at most 30 each, and stays within 7.5e-7 (one sign: 1.7e-6) at any K.  A bf16 result's own
// rounding is 1.7e-3; 512 tiles, by the same growth (K^1.3), are near 3e-5.
// In the pair kernel chains cost the overlap of a tile's epilogue with the next tile's products,
// and from the third on a wait for the join (8192 x 12352 x 5120 fp32 under a steady load: 479 us
// in two, 447 in one; 2048 x 5120 x 17408: 177 in five, 166 in two).  Leaving the first chain's
// sum in the result instead keeps the overlap, but under the power limit the extra traffic
// costs more (5 %); three stages and that sum in shared memory: three stages alone take 20 %
// more.  In the split-K kernel chains cost little (64 x 5120 x 17408: 21.8 us in two a CTA, 21.7
// in one).
// NVFP4 products take one chain: a step adds 64 products, and the error is 4.5e-8 at K = 5120,
// 6.9e-7 at 28672 (one sign: 1.9e-7, 5.7e-6); 256 accumulator columns, their second copy and the
// scales are more than TMEM has.
constexpr int kChainTiles = 30;
constexpr int kChainTilesBf16 = 512;

// The pair kernel from 32 tiles of 256 x 256 on, when there are more than 128 tokens
// (8-bit, 512 x 5120 x 4096, 40 tiles: 15.9 us against 17.2 for the best split; 256 x 5120
// x 4096, 20 tiles: 13.0 against 12.3).  Below that the split-K kernel: the narrowest
// token tile that holds the tokens (an NVFP4 tile has to begin a 128-row scale block, so
// more than 128 tokens take tiles of 128).  K is split, four k-tiles at least each:
//   up to 32 tokens, in 2 or 4 while the CTAs stay within 1.5 per SM (one token x 5120 x
//     4096, 8-bit: 5.3 us in 4, 6.5 in 2, 10.8 whole);
//   above, in as many of at most 4 (3 for 128 tokens) as leave one CTA per SM, because the
//     joining moves 32 or 64 KB a CTA (64 x 5120 x 4096: 7.0 us in 3, 8.0 in 4, 8.2 in 2;
//     128 x 5120 x 4096: 8.8 in 3, 10.2 in 2), else in 2 within 1.5 per SM (64 x 12352 x
//     5120: 15.4 in 2, 17.9 whole; in 3 the clusters no longer fit at once, 22).
template <bool kFp4>
nvfp4_status fused_launch(const Operand& X, const Operand& W, const FusedArgs& args, cudaStream_t st) {
    const int64_t M = X.rows, N = W.rows;
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256);
    const int64_t num_kt = (args.row_bytes + kTileK - 1) / kTileK;
    const bool wide = args.epi.out_dtype == NVFP4_DTYPE_FP32;
    if (M > 128 && pair_tiles >= 32) {
        if (args.stalled_rank >= 0) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "K is not split for these sizes");
        if constexpr (!kFp4)
            if (num_kt > args.chain_tiles || (wide && num_kt == kChainTiles)) return launch_pair<false, true>(X, W, args, st);
        return launch_pair<kFp4, false>(X, W, args, st);
    }
    const int64_t n_tiles = (N + 127) / 128, most = num_sms() * 3 / 2;
    const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const int64_t tiles = n_tiles * ((M + bn - 1) / bn);
    auto fits = [&](int split, int64_t ctas) { return tiles * split <= ctas && num_kt / split >= 4; };
    int split = fits(2, most) ? 2 : 1;
    if (bn <= 32) {
        if (fits(4, most)) split = 4;
    } else if (fits(3, num_sms())) {
        split = bn < 128 && fits(4, num_sms()) ? 4 : 3;
    }
    if (!kFp4 && wide && num_kt >= kChainTiles && split == 1) split = 2;
    if (bn == 16) return launch_split<kFp4, 16>(split, X, W, args, st);
    if (bn == 32) return launch_split<kFp4, 32>(split, X, W, args, st);
    if (bn == 64) return launch_split<kFp4, 64>(split, X, W, args, st);
    return launch_split<kFp4, 128>(split, X, W, args, st);
}

nvfp4_status fused_args(const gemm_epilogue* e, int64_t M, int64_t N, FusedArgs* args) {
    if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30)) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "M or N too large");
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
    auto bytes = [](int64_t ld, int32_t t) { return static_cast<uint32_t>(ld * (t == NVFP4_DTYPE_BF16 ? 2 : 4)); };
    EpiArgs& epi = args->epi;
    epi.bias = e->bias;
    epi.res = e->residual;
    epi.out = e->out;
    epi.ld_res = e->residual ? bytes(e->ld_residual, e->residual_dtype) : 0;
    epi.ldc = bytes(e->ldc, e->out_dtype);
    epi.act = e->act;
    epi.res_dtype = e->residual_dtype;
    epi.out_dtype = e->out_dtype;
    epi.M = static_cast<int>(M);
    epi.N = static_cast<int>(N);
    args->stalled_rank = -1;
    args->chain_tiles = e->out_dtype == NVFP4_DTYPE_FP32 ? kChainTiles : kChainTilesBf16;
    args->err = device_error_word();
    if (!args->err) return fail(NVFP4_ERR_CUDA, "device error word unavailable");
    return NVFP4_OK;
}

}  // namespace

}  // namespace nvg

namespace nvg {
static nvfp4_status w8a8_launch(const fp8_tensor* A, const fp8_tensor* B, const gemm_epilogue* epilogue, int stalled_rank,
                                nvfp4_stream_t stream) {
    nvfp4_status s = validate_fp8(A, "A");
    if (s == NVFP4_OK) s = validate_fp8(B, "B");
    if (s != NVFP4_OK) return s;
    if (A->cols != B->cols) return fail(NVFP4_ERR_INVALID_ARG, "A and B have different K");
    FusedArgs args = {};
    if ((s = fused_args(epilogue, A->rows, B->rows, &args)) != NVFP4_OK) return s;
    args.stalled_rank = stalled_rank;
    args.sA = A->scale;
    args.sB = B->scale;
    args.row_bytes = static_cast<int>(A->cols);
    const Operand x = {A->codes, nullptr, A->rows, A->cols, A->ld}, w = {B->codes, nullptr, B->rows, B->cols, B->ld};
    return fused_launch<false>(x, w, args, as_stream(stream));
}
}  // namespace nvg

extern "C" nvfp4_status w8a8_gemm(const fp8_tensor* A, const fp8_tensor* B, const gemm_epilogue* epilogue,
                                  nvfp4_stream_t stream) {
    return nvg::w8a8_launch(A, B, epilogue, -1, stream);
}

extern "C" nvfp4_status nvfp4_selftest_split_expiry(const fp8_tensor* A, const fp8_tensor* B,
                                                    const gemm_epilogue* epilogue, nvfp4_stream_t stream) {
    return nvg::w8a8_launch(A, B, epilogue, 1, stream);
}

extern "C" nvfp4_status w4a4_gemm_fused(const nvfp4_tensor* A, const nvfp4_tensor* B, const gemm_epilogue* epilogue,
                                        nvfp4_stream_t stream) {
    using namespace nvg;
    nvfp4_status s = validate_tensor(A, "A");
    if (s == NVFP4_OK) s = validate_tensor(B, "B");
    if (s != NVFP4_OK) return s;
    if (A->cols != B->cols) return fail(NVFP4_ERR_INVALID_ARG, "A and B have different K");
    FusedArgs args = {};
    if ((s = fused_args(epilogue, A->rows, B->rows, &args)) != NVFP4_OK) return s;
    args.sA = A->global_scale;
    args.sB = B->global_scale;
    args.row_bytes = static_cast<int>(A->cols / 2);
    const Operand x = {A->codes, A->sf, A->rows, A->cols / 2, A->cols / 2};
    const Operand w = {B->codes, B->sf, B->rows, B->cols / 2, B->cols / 2};
    return fused_launch<true>(x, w, args, as_stream(stream));
}

// grouped_sm100.cu - block-scaled FP4 products over groups of rows: the three
// GEMMs of a linear layer whose weight is a stack of E experts and whose
// tokens are sorted by expert, group e having any number m_e of rows (none,
// too) that only the device knows (offsets, int32 [E + 1]).
//
// The activations are quantized in a padded layout: group e starts at row
// p_e = sum_{i<e} 128 ceil(m_i / 128), the rows up to the next group are zero.
// So a group starts at a whole 512-byte scale atom along the rows (Fprop,
// Dgrad), and along the tokens (Wgrad) its blocks, rotations and 64-element
// MMA steps hold no other group's tokens.
//   rows:  D[off_e + i][n] = gA gB sum_k A[p_e + i][k] B_e[n][k], i < m_e.
//          B_e is a part of B along its rows (Fprop: W as [E N x K]) or along
//          the reduction axis (Dgrad: W^T as [K x E N]).
//   wgrad: D[e] = gA gB sum over group e's tokens t of A[.][t] B[.][t]^T.
//
// The main kernel is the dense CTA-pair kernel (256 x 256 tiles, tcgen05
// cta_group::2, the same warp roles and rings) with another walk: every role
// steps through prefix sums of the groups' tile counts in shared memory, which
// the CTA builds once from the offsets. A tile never
// spans two groups. Rows of D past a group belong to the next one: 32-row
// boxes that are full leave by TMA, the one a group's end cuts is written row
// by row from the registers.
#include "groups.cuh"
#include "qfp4_device.cuh"
#include "qfp4_internal.h"

namespace qfp4 {
namespace {

// One tile of the walk.
struct GroupTile {
    int e;       // group
    int m0, n0;  // first row (within the group, or of its D in wgrad) and column
    int k0, k;   // first element of the reduction in A, its length
};

// Every role steps through the tiles by itself. In rows mode the groups are
// walked along with the tiles (a CTA's next tile is rarely more than a group or
// two ahead), so that no role searches for its group.
template <bool WGRAD, int TILE_M>
struct GroupWalk {
    const GroupTable& g;
    int e = 0;  // group of the last tile
    __device__ __forceinline__ explicit GroupWalk(const GroupTable& t) : g(t) {}
    static __device__ __forceinline__ int num_n(const GroupedParams& p) { return (p.N + kGemmBN - 1) / kGemmBN; }
    static __device__ __forceinline__ int num_m(const GroupedParams& p) { return (p.M + TILE_M - 1) / TILE_M; }
    __device__ __forceinline__ int total(const GroupedParams& p) const {
        return (WGRAD ? p.E * num_m(p) : g.tiles[p.E]) * num_n(p);
    }
    // Tile t < total(), t rising; within a group in the dense kernel's order.
    __device__ __forceinline__ GroupTile at(const GroupedParams& p, int t) {
        GroupTile r;
        const int nn = num_n(p);
        int mb, nb;
        if constexpr (WGRAD) {
            const int nm = num_m(p), i = t % (nm * nn);
            r.e = t / (nm * nn);
            tile_coords<P_GROUP_M>(i, nm, nn, mb, nb);
            r.k0 = g.padded[r.e];
            r.k = g.padded[r.e + 1] - r.k0;
        } else {
            while (t >= g.tiles[e + 1] * nn) ++e;
            const int first = g.tiles[e], tm = g.tiles[e + 1] - first, i = t - first * nn;
            r.e = e;
            tile_coords<P_GROUP_M>(i, tm, nn, mb, nb);
            r.k0 = 0;
            r.k = p.K;
        }
        r.m0 = mb * TILE_M;
        r.n0 = nb * kGemmBN;
        return r;
    }
};

// Rows cut by a group's end: this lane's 32 words (128 bytes) of its row to D
// from column x, by 16-byte stores (N is a multiple of 8).
__device__ __forceinline__ void store_row_words(const GroupedParams& p, const uint32_t* v, int row, int x) {
    const int esz = p.out_f32 ? 4 : 2, per = 16 / esz;
    uint8_t* d = static_cast<uint8_t*>(p.D) + (row * p.ldd + x) * esz;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (x + j * per < p.N)
            __stcs(chk(reinterpret_cast<uint4*>(d + 16 * j), p.D, ((int64_t)(p.T - 1) * p.ldd + p.N) * esz),
                   make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
}

// Epilogue of one tile for one warp: 32 rows x 128 columns from D row `row`, nv
// of the rows stored; zero: the sum of an empty group. The accumulator goes back
// to the MMA warp as soon as the values are in registers: all 128 columns
// packed to bf16, or the last 96 in fp32 after the first 32 are stored.
template <typename Release>
__device__ __forceinline__ void group_epilogue(const GroupedParams& p, const CUtensorMap* tmD, uint32_t taddr, int row,
                                               int nv, int n0, float scale, bool zero, uint32_t obox, int lane,
                                               Release release) {
    // 32 words (128 bytes) of each lane's row, from column x: a whole box of 32
    // rows through shared memory (128-byte swizzle) by TMA, which clips the
    // columns past N
    const uint32_t rbase = obox + (uint32_t)lane * 128u;
    auto box = [&](const uint32_t* v, int x) {
        if (nv < 32) {
            if (lane < nv) store_row_words(p, v, row + lane, x);
            return;
        }
        if (lane == 0) bulk_wait_group_read0();  // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sts128(rbase + ((uint32_t)(j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0 && x < p.N) {
            if (p.accumulate)
                tma_reduce_add_2d(tmD, obox, x, row);
            else
                tma_store_2d(tmD, obox, x, row);
            bulk_commit_group();
        }
    };
    __syncwarp();  // loads from tensor memory are the whole warp's
    if (!p.out_f32) {
        uint32_t w[64];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t acc[64];
            tmem_ld_32x32b_x32(taddr + 64 * h, acc);
            tmem_ld_32x32b_x32(taddr + 64 * h + 32, acc + 32);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) w[32 * h + c] = zero ? 0u : pack_bf16(acc[2 * c], acc[2 * c + 1], scale);
        }
        tc_fence_before();
        __syncwarp();
        release();
#pragma unroll
        for (int h = 0; h < 2; ++h) box(w + 32 * h, n0 + 64 * h);
    } else {
        auto scaled = [&](uint32_t* v) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                const float2 t = __fmul2_rn(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                            make_float2(scale, scale));
                v[c] = zero ? 0u : __float_as_uint(t.x);
                v[c + 1] = zero ? 0u : __float_as_uint(t.y);
            }
        };
        uint32_t acc[96];
        tmem_ld_32x32b_x32(taddr, acc);
        tc_wait_ld();
        scaled(acc);
        box(acc, n0);
        __syncwarp();
        tmem_ld_32x32b_x32(taddr + 32, acc);
        tmem_ld_32x32b_x32(taddr + 64, acc + 32);
        tmem_ld_32x32b_x32(taddr + 96, acc + 64);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        release();
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            scaled(acc + 32 * b);
            box(acc + 32 * b, n0 + 32 * (b + 1));
        }
    }
}

// Five ring stages and one box per epilogue warp, as the dense kernel. The
// weight gradient's sums are short (a group's tokens) and its stores heavy, yet
// the operand loads want the stages more than the stores boxes: 16 groups of
// 1024 tokens, 2816 x 2048 in fp32, 81.7 us; 4 stages and 2 boxes 85.5; 3 and 3
// 103.6 (4.5 TB/s of output; a plain fill of memory reaches 3.7 here).
constexpr int GP_SMEM = P_SMEM + (int)sizeof(GroupTable);
static_assert(GP_SMEM <= 227 * 1024, "shared memory of one CTA");

template <int FMT, bool WGRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSFA, const __grid_constant__ CUtensorMap tmSFB,
                        const __grid_constant__ CUtensorMap tmD, const GroupedParams p) {
    constexpr int SF_K = (FMT == kNvfp4) ? 64 : 128;
    constexpr int ATOMS_PER_KT = BK / SF_K;  // 4 or 2
    constexpr uint32_t AB_TX = 2u * (P_A + P_B);          // both CTAs, on the leader
    constexpr uint32_t SF_TX = 3u * ATOMS_PER_KT * 512u;  // this CTA's scale boxes
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = base;
    uint8_t* sB = sA + P_STAGES * P_A;
    uint8_t* sSFA = sB + P_STAGES * P_B;
    uint8_t* sSFB = sSFA + P_STAGES * P_SFA;
    uint8_t* sOut = sSFB + P_STAGES * P_SFB;  // kEpiWarps boxes, 1024-byte aligned
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + kEpiWarps * P_OUT_BOX);
    uint64_t* empty = full + P_STAGES;
    uint64_t* sf_load = empty + P_STAGES;    // this CTA's scale atoms of stage s landed
    uint64_t* sf_full = sf_load + P_STAGES;  // scale slot s written in both CTAs (leader's)
    uint64_t* acc_full = sf_full + P_STAGES;
    uint64_t* acc_empty = acc_full + 1;
    uint64_t* drain = acc_empty + 1;  // every MMA the leader issued has completed (both CTAs)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    GroupTable& groups = *reinterpret_cast<GroupTable*>(sOut + kEpiWarps * P_OUT_BOX + 512);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cid = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmSFA);
        prefetch_tmap(&tmSFB);
        prefetch_tmap(&tmD);
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sf_load[s], 1);
            mbar_init(&sf_full[s], 2 * kScaleWarps);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * kEpiWarps);
        mbar_init(drain, 1);
        fence_mbarrier_init();
    }
    if (warp == 0) tmem_alloc_pair(tmem_slot, TMEM_COLS);
    pdl_wait();  // the offsets and the operands are written (and the previous readers of D done)
    pdl_launch_dependents();
    if (warp == 1) build_groups(groups, p.offsets, p.E, p.T, 2 * BM, lane);
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated, groups known
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    GroupWalk<WGRAD, 2 * BM> walk(groups);
    const int total = walk.total(p);

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += nclusters) {
                const GroupTile w = walk.at(p, t);
                const int arow = (WGRAD ? 0 : groups.padded[w.e]) + w.m0 + (int)rank * BM;
                const int brow = (WGRAD ? 0 : w.e * p.b_rows) + w.n0;
                const int bk0 = WGRAD ? w.k0 : w.e * p.b_k;
                const int kt_n = (w.k + BK - 1) / BK;
                const bool b_half = w.n0 + 128 >= p.N;  // columns of the second CTA's B rows are not stored
                for (int kt = 0; kt < kt_n; ++kt, ++it) {
                    const int s = it % P_STAGES;
                    if (it >= P_STAGES && !mbar_wait_cluster(&empty[s], ((it / P_STAGES) + 1) & 1)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sf_load[s], SF_TX);
                    tma_load_3d(sSFA + s * P_SFA, &tmSFA, &sf_load[s], 0, w.k0 / SF_K + kt * ATOMS_PER_KT, arow / 128);
                    tma_load_3d(sSFB + s * P_SFB, &tmSFB, &sf_load[s], 0, bk0 / SF_K + kt * ATOMS_PER_KT, brow / 128);
                    const uint32_t bar_leader = mapa_shared(smem_u32(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], b_half ? AB_TX - P_B : AB_TX);
                    tma_load_2d_pair(sA + s * P_A, &tmA, bar_leader, w.k0 / 2 + kt * (BK / 2), arow);
                    if (rank == 0 || !b_half)
                        tma_load_2d_pair(sB + s * P_B, &tmB, bar_leader, bk0 / 2 + kt * (BK / 2), brow + (int)rank * 128);
                }
            }
            drain_loads(rank == 0 ? full : nullptr, sf_load, P_STAGES, it);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader CTA only) ----------------
        if (lane == 0 && rank == 0) {
            const uint64_t a_desc0 = sw128_desc(smem_u32(sA)), b_desc0 = sw128_desc(smem_u32(sB));
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = cid; t < total && ok; t += nclusters, ++lt) {
                const GroupTile w = walk.at(p, t);
                if (lt > 0 && !mbar_wait_cluster(acc_empty, (lt - 1) & 1)) break;
                tc_fence_after();
                for (int k = 0; k < w.k; k += BK) {
                    if (!mbar_wait_cluster(&sf_full[s], ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_ktile<FMT, true, 2 * BM>(tmem + TMEM_D, a_desc0 + (uint64_t)(s * (P_A >> 4)),
                                                 b_desc0 + (uint64_t)(s * (P_B >> 4)), tmem + sfa_col(s),
                                                 tmem + sfb_col(s), min(BK, w.k - k) / 64, k == 0);
                    tc_commit_pair(&empty[s]);  // frees stage s and scale slot s in both CTAs
                    if (++s == P_STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                tc_commit_pair(acc_full);  // both CTAs' accumulators are complete
            }
            tc_commit_pair(drain);
            (void)mbar_wait(drain, 0);
        }
    } else if (warp < kFirstEpiWarp) {
        // ---------------- scale writers (both CTAs) ----------------
        const uint32_t tmem_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = cid; t < total && ok; t += nclusters) {
            const int k_len = walk.at(p, t).k;
            for (int k = 0; k < k_len; k += BK) {
                if (!mbar_wait_cluster(&sf_load[s], ph)) {
                    ok = false;
                    break;
                }
                write_scales<ATOMS_PER_KT>(tmem_lane, s, smem_u32(sSFA + s * P_SFA), smem_u32(sSFB + s * P_SFB), lane,
                                           warp & 3);
                if (rank == 0 && !mbar_wait_cluster(&full[s], ph)) {
                    ok = false;
                    break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sf_full[s]), 0));
                if (++s == P_STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const int lq = warp & 3;
        const int chalf = (warp - kFirstEpiWarp) >> 2;
        const float scale = __fmul_rn(__ldg(p.ga), __ldg(p.gb));
        const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);
        const uint32_t obox = smem_u32(sOut) + (uint32_t)(warp - kFirstEpiWarp) * P_OUT_BOX;
        int lt = 0;
        for (int t = cid; t < total; t += nclusters, ++lt) {
            const GroupTile w = walk.at(p, t);
            if (!mbar_wait_cluster(acc_full, lt & 1)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(lq * 32) << 16) + TMEM_D + chalf * 128;
            const int m = w.m0 + (int)rank * BM + lq * 32;  // within the group
            const int nv = min(32, (WGRAD ? p.M : groups.size(w.e)) - m);
            const int row = (WGRAD ? w.e * p.M : groups.row[w.e]) + m;
            // an empty group's weight gradient is zero; added to D it changes nothing
            const bool zero = WGRAD && w.k == 0;
            group_epilogue(p, &tmD, taddr, row, zero && p.accumulate ? 0 : nv, w.n0 + chalf * 128, scale, zero, obox,
                           lane, [&] {
                               if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
                           });
        }
        if (lane == 0) bulk_wait_group0();  // this warp's stores are complete
    }

    tc_fence_before();
    cluster_sync();  // no CTA leaves while its peer may still signal it
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
        tmem_relinquish_pair();
    }
}

// Few rows per group (the rows product alone): single CTAs on 128 x 256 tiles,
// as the dense single-CTA kernel. A pair's second CTA would multiply rows that
// are no group's, and there would be half as many tiles in flight. Bound by the
// weights' arrival (488 rows of 64 groups, 1408 x 2048: 107 MB in 23.9 us, of
// which about 5 are the start and the end; pairs 30.0, tiles of 128 x 128 25.3).
constexpr int GS_SMEM = SMEM_BYTES + (int)sizeof(GroupTable);
static_assert(GS_SMEM <= 227 * 1024, "shared memory of one CTA");

template <int FMT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_grouped_single_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                               const GroupedParams p) {
    constexpr int SF_K = (FMT == kNvfp4) ? 64 : 128;
    constexpr int ATOMS_PER_KT = BK / SF_K;  // 4 or 2
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = base;
    uint8_t* sB = sA + STAGES * A_STAGE;
    uint8_t* sSFA = sB + STAGES * B_STAGE;
    uint8_t* sSFB = sSFA + STAGES * SFA_STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(sSFB + STAGES * SFB_STAGE);
    uint64_t* empty = full + STAGES;
    uint64_t* sf_load = empty + STAGES;
    uint64_t* sf_full = sf_load + STAGES;
    uint64_t* acc_full = sf_full + STAGES;
    uint64_t* acc_empty = acc_full + 1;
    uint64_t* drain = acc_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    GroupTable& groups = *reinterpret_cast<GroupTable*>(sSFB + STAGES * SFB_STAGE + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KT = (p.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&sf_load[s], 1);
            mbar_init(&sf_full[s], kScaleWarps);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, kEpiWarps);
        mbar_init(drain, 1);
        fence_mbarrier_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, TMEM_COLS);
    pdl_wait();  // the offsets and the operands are written (and the previous readers of D done)
    pdl_launch_dependents();
    if (warp == 1) build_groups(groups, p.offsets, p.E, p.T, BM, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    GroupWalk<false, BM> walk(groups);
    const int total = walk.total(p);

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const GroupTile w = walk.at(p, t);
                const int arow = groups.padded[w.e] + w.m0, brow = w.e * p.b_rows + w.n0, bk0 = w.e * p.b_k;
                const int nrb = w.n0 + 128 < p.N ? 2 : 1;  // B row blocks of this group
                for (int kt = 0; kt < KT; ++kt, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES && !mbar_wait(&empty[s], ((it / STAGES) + 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const int atoms = (min(BK, p.K - kt * BK) + SF_K - 1) / SF_K;
                    mbar_arrive_expect_tx(&sf_load[s], atoms * 512 * (1 + nrb));
                    const int64_t katom = (int64_t)kt * ATOMS_PER_KT;
                    bulk_load(sSFA + s * SFA_STAGE, p.sfa + ((int64_t)(arow / 128) * p.atoms_a + katom) * 512, atoms * 512,
                              &sf_load[s]);
                    for (int rb = 0; rb < nrb; ++rb)
                        bulk_load(sSFB + s * SFB_STAGE + rb * (ATOMS_PER_KT * 512),
                                  p.sfb + ((int64_t)(brow / 128 + rb) * p.atoms_b + bk0 / SF_K + katom) * 512, atoms * 512,
                                  &sf_load[s]);
                    mbar_arrive_expect_tx(&full[s], A_STAGE + nrb * P_B);
                    tma_load_2d(sA + s * A_STAGE, &tmA, &full[s], kt * (BK / 2), arow);
                    for (int rb = 0; rb < nrb; ++rb)
                        tma_load_2d(sB + s * B_STAGE + rb * P_B, &tmB, &full[s], bk0 / 2 + kt * (BK / 2), brow + 128 * rb);
                }
            }
            drain_loads(full, sf_load, STAGES, it);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            const uint64_t a_desc0 = sw128_desc(smem_u32(sA)), b_desc0 = sw128_desc(smem_u32(sB));
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++lt) {
                if (lt > 0 && !mbar_wait(acc_empty, (lt - 1) & 1)) break;
                tc_fence_after();
                for (int kt = 0; kt < KT; ++kt) {
                    if (!mbar_wait(&sf_full[s], ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_ktile<FMT, false, BM>(tmem + TMEM_D, a_desc0 + (uint64_t)(s * (A_STAGE >> 4)),
                                              b_desc0 + (uint64_t)(s * (B_STAGE >> 4)), tmem + sfa_col(s),
                                              tmem + sfb_col(s), min(BK, p.K - kt * BK) / 64, kt == 0);
                    tc_commit(&empty[s]);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                tc_commit(acc_full);
            }
            tc_commit(drain);
            (void)mbar_wait(drain, 0);
        }
    } else if (warp < kFirstEpiWarp) {
        // ---------------- scale writers ----------------
        const uint32_t tmem_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            for (int kt = 0; kt < KT; ++kt) {
                if (!mbar_wait(&sf_load[s], ph)) {
                    ok = false;
                    break;
                }
                write_scales<ATOMS_PER_KT>(tmem_lane, s, smem_u32(sSFA + s * SFA_STAGE), smem_u32(sSFB + s * SFB_STAGE),
                                           lane, warp & 3);
                if (!mbar_wait(&full[s], ph)) {
                    ok = false;
                    break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sf_full[s]);
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else {
        // ---------------- epilogue: each lane stores its row ----------------
        const int lq = warp & 3;
        const int chalf = (warp - kFirstEpiWarp) >> 2;
        const float scale = __fmul_rn(__ldg(p.ga), __ldg(p.gb));
        int lt = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++lt) {
            const GroupTile w = walk.at(p, t);
            if (!mbar_wait(acc_full, lt & 1)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(lq * 32) << 16) + TMEM_D + chalf * 128;
            const int m = w.m0 + lq * 32 + lane, n0 = w.n0 + chalf * 128;
            const bool mine = m < groups.size(w.e);
            const int row = groups.row[w.e] + m;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t acc[64];
                __syncwarp();  // loads from tensor memory are the whole warp's
                tmem_ld_32x32b_x32(taddr + 64 * h, acc);
                tmem_ld_32x32b_x32(taddr + 64 * h + 32, acc + 32);
                tc_wait_ld();
                if (h == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty);
                }
                if (mine) {
                    if (!p.out_f32) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) acc[c] = pack_bf16(acc[2 * c], acc[2 * c + 1], scale);
                        store_row_words(p, acc, row, n0 + 64 * h);
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; ++c) acc[c] = __float_as_uint(__fmul_rn(__uint_as_float(acc[c]), scale));
                        store_row_words(p, acc, row, n0 + 64 * h);
                        store_row_words(p, acc + 32, row, n0 + 64 * h + 32);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
        tmem_relinquish();
    }
}

}  // namespace

cudaError_t launch_gemm_grouped(const GroupedParams& p, int fmt, bool wgrad, bool pair, const CUtensorMap* tmapA,
                                const CUtensorMap* tmapB, const CUtensorMap* tmapSFA, const CUtensorMap* tmapSFB,
                                const CUtensorMap* tmapD, cudaStream_t s, int sms) {
    // the tile count is known on the device only: an upper bound sizes the grid
    const int64_t num_n = (p.N + kGemmBN - 1) / kGemmBN;
    if (!pair) {
        const int64_t tiles = std::min<int64_t>(p.T, p.T / 128 + p.E) * num_n;
        auto run = [&](auto* kern) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GS_SMEM);
            if (e != cudaSuccess) return e;
            const dim3 grid((unsigned)std::min<int64_t>(sms, tiles));
            return launch_pdl(kern, grid, dim3(kGemmThreads), GS_SMEM, s, *tmapA, *tmapB, p);
        };
        const cudaError_t e =
            fmt == kNvfp4 ? run(gemm_grouped_single_kernel<kNvfp4>) : run(gemm_grouped_single_kernel<kMxfp4>);
        count_launch();
        return e;
    }
    const int64_t num_m = wgrad ? (int64_t)p.E * ((p.M + 255) / 256) : std::min<int64_t>(p.T, p.T / 256 + p.E);
    const int clusters = (int)std::max<int64_t>(1, std::min<int64_t>(sms / 2, num_m * num_n));
    auto run = [&](auto* kern) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GP_SMEM);
        if (e != cudaSuccess) return e;
        return launch_pdl(kern, dim3(2 * clusters), dim3(kGemmThreads), GP_SMEM, s, *tmapA, *tmapB, *tmapSFA, *tmapSFB,
                          *tmapD, p);
    };
    cudaError_t e;
    if (fmt == kNvfp4)
        e = wgrad ? run(gemm_grouped_kernel<kNvfp4, true>) : run(gemm_grouped_kernel<kNvfp4, false>);
    else
        e = wgrad ? run(gemm_grouped_kernel<kMxfp4, true>) : run(gemm_grouped_kernel<kMxfp4, false>);
    count_launch();
    return e;
}

}  // namespace qfp4

// nm_ffn.cu -- a feed-forward block's sparse projections beyond the plain
// product: the gated first half (both projections, activation and product in
// one kernel) and a projection with the low-rank adapters of many requests.
//
// One persistent CTA-pair kernel serves both (k_ffn<MODE, OP>).  As in
// k_gemm_wide, a pair holds two accumulators of 256 rows x bn <= 240 tokens in
// tensor memory that share every B tile, which keeps the shared-memory feed of
// the sparse tensor core at 78% of its rate instead of 66%.
//   OP_GLU   accumulator 0 = 256 rows of the gate projection, accumulator 1 =
//            the same 256 rows of the up projection, so a thread of the
//            epilogue finds g and u of the same feature and token in tensor
//            memory: H = act(g) u needs no second pass and G, U reach memory
//            only when the caller keeps them for a backward pass.
//   OP_LORA  accumulators 0 and 1 = rows 0..255 and 256..511 of the tile, as in
//            k_gemm_wide.  After the K' blocks of the projection come the
//            blocks of the adapters: for each adapter that occurs among the
//            tile's tokens, D += B[a] V_a^T with dense tcgen05.mma on the same
//            accumulators, where V_a holds scale[a] X A[a]^T of that adapter's
//            tokens and zero in the other rows (k_lora_shrink).  The adapters'
//            share so joins the projection's in fp32 and Y is written once.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "nm_common.cuh"
#include "nm_gemm.cuh"
#include "nm_host.cuh"

namespace nm {

enum { OP_GLU = 0, OP_LORA = 1 };
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_RELU2 = 2 };

struct FfnCfg {
    static constexpr int BN_MAX = 240;          // tokens per tile (both CTAs)
    static constexpr int A_BYTES = BM * 128;    // 128 rows x 64 values
    static constexpr int OFF_A0 = 0, OFF_A1 = A_BYTES, OFF_E0 = 2 * A_BYTES, OFF_E1 = OFF_E0 + EBLK_BYTES;
    static constexpr int OFF_B = OFF_E1 + EBLK_BYTES;  // two atoms of bn/2 tokens x 64 columns
    static constexpr int MAX_STAGES = 6;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 384;
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM_BYTES = 232448;
    static constexpr int SMEM_STAGES = SMEM_BYTES - BAR_BYTES - 1024;
    static constexpr int TMEM_COLS = 512;
    static constexpr int TMEM_D0 = 0, TMEM_E0 = 240, TMEM_E1 = 248, TMEM_D1 = 256;
    static_assert(OFF_B % 1024 == 0, "operand alignment");
    static int stage_bytes(int bn) { return OFF_B + bn * 128; }
    static int stages(int bn) {
        const int s = SMEM_STAGES / stage_bytes(bn);
        return s < MAX_STAGES ? s : MAX_STAGES;
    }
};

// stream-K slot of one epilogue warp: 32 rows x up to 256 columns (OP_GLU: 128
// of each accumulator), [column][row]
constexpr int FFN_SLOT_FLOATS = 32 * 256;
inline size_t ffn_sk_bytes(int64_t pairs) {
    return static_cast<size_t>(pairs) * 2 * 8 * (FFN_SLOT_FLOATS * 4 + 8);
}

struct FfnMaps {
    CUtensorMap a0, a1, e0, e1;  // values and metadata of the two accumulators' weights
    CUtensorMap b, b2;           // activations; 6:8: the gathered middle windows
    CUtensorMap lb, lv;          // OP_LORA: the adapters' B, the shrunk activations V
};

struct FfnArgs {
    int64_t T, R, nkb;
    int bn, stages, stage_bytes;
    int early;  // loads of X and the weights need not wait for the preceding kernel
    uint16_t *Y, *G, *U;
    int64_t ldy, ldgu;
    int act;
    // OP_LORA: adapters per token tile, the tile's first slot, a slot's adapter;
    // at most ext_cap slots per tile, rb blocks of 64 ranks per slot
    const int32_t *tile_cnt, *tile_base, *slot_adapter;
    int ext_cap, rb;
    uint8_t *sk_ws;
    uint64_t seq;
    int sk;
};

__device__ __forceinline__ float act_of(float g, int act) {
    // silu g / (1 + e^-g); gelu (tanh form) g / (1 + e^-2z), since
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z); e^x overflowing to inf gives 0
    if (act == ACT_RELU2) return g < 0.0f ? 0.0f : g * g;
    const float z = act == ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return __fdividef(g, 1.0f + __expf(-z));
}

template <int MODE, int OP>
__global__ void __launch_bounds__(FfnCfg::THREADS, 1)
    k_ffn(const __grid_constant__ FfnMaps tm, const __grid_constant__ FfnArgs p) {
    using C = FfnCfg;
    const int S = p.stages;
    const bool sk = p.sk != 0;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::SMEM_STAGES / 1024 * 1024);
    uint64_t *full = bars, *empty = bars + C::MAX_STAGES;
    uint64_t *acc_full = bars + 2 * C::MAX_STAGES, *acc_empty = acc_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int bn = p.bn, bh = bn >> 1;
    const int b_atom = bh * 128;
    const int64_t nkb = p.nkb, T = p.T;
    const int64_t Rpad = (p.R + 255) / 256 * 256;
    constexpr int TILE_ROWS = OP == OP_GLU ? 256 : 512;
    const int64_t n_t = (T + bn - 1) / bn;
    const int64_t n_m = (Rpad + TILE_ROWS - 1) / TILE_ROWS;
    const int64_t ntiles = n_t * n_m;
    const int64_t nkt = OP == OP_LORA ? nkb + static_cast<int64_t>(p.ext_cap) * p.rb : nkb;
    auto stage = [&](int s) { return smem + s * p.stage_bytes; };
    // K' blocks of a tile: the projection's, then rb per adapter among its tokens
    auto tile_blocks = [&](int64_t nt) -> int64_t {
        return OP == OP_LORA && p.ext_cap > 0 ? nkb + static_cast<int64_t>(__ldcg(p.tile_cnt + nt)) * p.rb : nkb;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * C::EPI_WARPS);
        fence_barrier_init();
        prefetch_tmap(&tm.a0);
        prefetch_tmap(&tm.e0);
        prefetch_tmap(&tm.b);
        if (OP == OP_GLU) {
            prefetch_tmap(&tm.a1);
            prefetch_tmap(&tm.e1);
        }
        if (MODE == PMODE_SP68T) prefetch_tmap(&tm.b2);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // everything above overlaps the preceding kernel's tail (programmatic
    // dependent launch).  With `early` the producer loads what is older than
    // that kernel (X, the packed weights) and waits before its first block that
    // is not; the MMA warp reads global memory only for the adapter counts.
    if (warp >= 2 || !p.early) grid_dep_wait();

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t it = 0;
            bool ok = true, dep_done = p.early == 0;
            SegIter seg(sk, cluster, nclusters, ntiles, nkt);
            int64_t tile, kb0, kb1;
            const uint32_t b_bytes = 2u * static_cast<uint32_t>(b_atom);
            while (ok && seg.next(tile, kb0, kb1)) {
                int64_t nt, mt;
                tile_coords(tile, n_t, n_m, BAND_ROWS / TILE_ROWS, nt, mt);
                const bool has1 = OP == OP_GLU || mt * 512 + 256 < Rpad;
                const int32_t arow = static_cast<int32_t>(mt * TILE_ROWS + rank * 128);
                const int32_t arow1 = OP == OP_GLU ? arow : arow + 256;
                const int32_t brow = static_cast<int32_t>(nt * bn + rank * bh);
                const int64_t e0 = (arow >> 7) * nkb, e1 = (arow1 >> 7) * nkb;
                const uint32_t tx = 2u * ((has1 ? 2u : 1u) * (C::A_BYTES + EBLK_BYTES) + b_bytes);
                const CUtensorMap *ta1 = OP == OP_GLU ? &tm.a1 : &tm.a0, *te1 = OP == OP_GLU ? &tm.e1 : &tm.e0;
                int64_t vend = kb1;                // the tile's blocks that this segment runs
                int32_t slot0 = 0, a_next = 0;     // its first slot; the next block's adapter
                bool adapters_known = false;
                for (int64_t v = kb0; v < vend; ++v) {
                    const bool ext = OP == OP_LORA && v >= nkb;
                    const int64_t kb = ext ? v : (MODE == PMODE_SP68T ? visit68(v, nkb) : v);
                    const bool mid = MODE == PMODE_SP68T && !ext && (kb % 3) == 2;
                    if ((mid || ext) && !dep_done) {  // written by the kernels just before
                        grid_dep_wait();
                        dep_done = true;
                    }
                    if (ext && !adapters_known) {
                        adapters_known = true;
                        const int64_t nb = tile_blocks(nt);
                        if (nb < vend) vend = nb;
                        if (v >= vend) break;
                        slot0 = __ldcg(p.tile_base + nt);
                        a_next = __ldcg(p.slot_adapter + slot0 + static_cast<int>(v - nkb) / p.rb);
                    }
                    if (it >= S && !mbar_wait(&empty[s], ph ^ 1u)) { ok = false; break; }
                    const uint32_t bar = mapa_shared(&full[s], 0);
                    uint8_t *st = stage(s);
                    if (ext) {
                        const int slot = static_cast<int>(v - nkb) / p.rb;
                        const int32_t rk = static_cast<int32_t>((v - nkb) - static_cast<int64_t>(slot) * p.rb) * 64;
                        const int32_t gs = slot0 + slot, a = a_next;
                        if (v + 1 < vend) a_next = __ldcg(p.slot_adapter + slot0 + static_cast<int>(v + 1 - nkb) / p.rb);
                        if (rank == 0)
                            mbar_arrive_expect_tx(&full[s], 2u * ((has1 ? 2u : 1u) * C::A_BYTES + b_bytes / 2));
                        tma_load_3d_pair(st + C::OFF_A0, &tm.lb, bar, rk, arow, a);
                        if (has1) tma_load_3d_pair(st + C::OFF_A1, &tm.lb, bar, rk, arow + 256, a);
                        tma_load_2d_pair(st + C::OFF_B, &tm.lv, bar, rk, gs * bn + static_cast<int32_t>(rank) * bh);
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], tx);
                        const int32_t ka = static_cast<int32_t>(kb * 64);
                        tma_load_2d_pair(st + C::OFF_A0, &tm.a0, bar, ka, arow);
                        tma_load_2d_pair(st + C::OFF_E0, &tm.e0, bar, 0, static_cast<int32_t>((e0 + kb) * 8));
                        if (has1) {
                            tma_load_2d_pair(st + C::OFF_A1, ta1, bar, ka, arow1);
                            tma_load_2d_pair(st + C::OFF_E1, te1, bar, 0, static_cast<int32_t>((e1 + kb) * 8));
                        }
                        const int64_t x0 = MODE == PMODE_SP24 ? kb * 128
                                           : (mid ? (kb / 3) * 128 : (kb / 3) * 256 + (kb % 3) * 128);
                        const CUtensorMap *tb = mid ? &tm.b2 : &tm.b;
                        tma_load_2d_pair(st + C::OFF_B, tb, bar, static_cast<int32_t>(x0), brow);
                        tma_load_2d_pair(st + C::OFF_B + b_atom, tb, bar, static_cast<int32_t>(x0 + 64), brow);
                    }
                    ++it;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok && rank == 0) {  // let copies already issued land before exiting
                for (int64_t j = (it > S ? it - S : 0); j < it; ++j)
                    mbar_wait(&full[j % S], static_cast<uint32_t>((j / S) & 1));
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = make_idesc_bf16(256, bn, true, 0);
            const uint32_t idesc_dense = make_idesc_bf16(256, bn, false, 0);
            int s = 0;
            uint32_t ph = 0;
            int64_t ti = 0;
            bool ok = true, dep_done = p.early == 0;
            SegIter seg(sk, cluster, nclusters, ntiles, nkt);
            int64_t tile, kb0, kb1;
            for (; ok && seg.next(tile, kb0, kb1); ++ti) {
                int64_t nt, mt;
                tile_coords(tile, n_t, n_m, BAND_ROWS / TILE_ROWS, nt, mt);
                const bool has1 = OP == OP_GLU || mt * 512 + 256 < Rpad;
                if (ti >= 1 && !mbar_wait_cluster(acc_empty, static_cast<uint32_t>((ti - 1) & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d0 = tmem_base + C::TMEM_D0, d1 = tmem_base + C::TMEM_D1;
                const uint32_t te0 = tmem_base + C::TMEM_E0, te1 = tmem_base + C::TMEM_E1;
                const int64_t base_end = OP == OP_LORA && kb1 > nkb ? nkb : kb1;
                for (int64_t kb = kb0; kb < base_end; ++kb) {
                    if (!mbar_wait(&full[s], ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t st = smem_u32(stage(s));
                    tmem_cp_128x128b_pair(te0, make_sdesc(st + C::OFF_E0, 2048, 128, 0));
                    if (has1) tmem_cp_128x128b_pair(te1, make_sdesc(st + C::OFF_E1, 2048, 128, 0));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t bd = make_sdesc(st + C::OFF_B + (j >> 1) * b_atom + (j & 1) * 64, 16, 1024, 2);
                        const uint32_t acc = (kb > kb0 || j > 0) ? 1u : 0u;
                        const uint32_t id = idesc | static_cast<uint32_t>(j & 1);
                        mma_sp_bf16_pair(d0, make_sdesc(st + C::OFF_A0 + j * 32, 16, 1024, 2), bd,
                                         te0 + (j & ~1), id, acc);
                        if (has1)
                            mma_sp_bf16_pair(d1, make_sdesc(st + C::OFF_A1 + j * 32, 16, 1024, 2), bd,
                                             te1 + (j & ~1), id, acc);
                    }
                    mma_commit_pair(&empty[s]);
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (OP == OP_LORA && ok && kb1 > nkb) {
                    if (!dep_done) {
                        grid_dep_wait();
                        dep_done = true;
                    }
                    const int64_t nb = tile_blocks(nt), end = nb < kb1 ? nb : kb1;
                    for (int64_t v = kb0 > nkb ? kb0 : nkb; v < end; ++v) {
                        if (!mbar_wait(&full[s], ph)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t st = smem_u32(stage(s));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t bd = make_sdesc(st + C::OFF_B + j * 32, 16, 1024, 2);
                            const uint32_t acc = (v > kb0 || j > 0) ? 1u : 0u;
                            mma_bf16_pair(d0, make_sdesc(st + C::OFF_A0 + j * 32, 16, 1024, 2), bd, idesc_dense, acc);
                            if (has1)
                                mma_bf16_pair(d1, make_sdesc(st + C::OFF_A1 + j * 32, 16, 1024, 2), bd, idesc_dense,
                                              acc);
                        }
                        mma_commit_pair(&empty[s]);
                        if (++s == S) { s = 0; ph ^= 1u; }
                    }
                }
                if (ok) mma_commit_pair(acc_full);
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // ---------------------------------------------------------- epilogue
        // OP_GLU : warp = lane quarter q x token half h, both accumulators
        // OP_LORA: warp = lane quarter q x accumulator h, all tokens
        const int q = warp & 3, h = (warp - 4) >> 2, we = warp - 4;
        constexpr int NACC = OP == OP_GLU ? 2 : 1;
        const uint32_t acc_empty_cl = mapa_shared(acc_empty, 0);
        float *slots = reinterpret_cast<float *>(p.sk_ws);
        uint64_t *flags = reinterpret_cast<uint64_t *>(p.sk_ws + static_cast<size_t>(nclusters) * 2 * 8 *
                                                                     FFN_SLOT_FLOATS * 4);
        const int64_t total = ntiles * nkt;
        auto has_work = [&](int64_t cc) { return (cc + 1) * total / nclusters > cc * total / nclusters; };
        auto slot_of = [&](int64_t cc) {
            return slots + static_cast<size_t>((cc * 2 + rank) * 8 + we) * FFN_SLOT_FLOATS + lane;
        };
        SegIter seg(sk, cluster, nclusters, ntiles, nkt);
        int64_t tile, kb0, kb1, ti = 0;
        for (; seg.next(tile, kb0, kb1); ++ti) {
            int64_t nt, mt;
            tile_coords(tile, n_t, n_m, BAND_ROWS / TILE_ROWS, nt, mt);
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full, static_cast<uint32_t>(ti & 1)))) break;
            tc_fence_after();
            const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
            const uint32_t tacc[2] = {tq + (OP == OP_LORA && h ? C::TMEM_D1 : C::TMEM_D0), tq + C::TMEM_D1};
            const int64_t tok0 = nt * bn;
            const int nv = static_cast<int>(T - tok0 < bn ? T - tok0 : bn);  // real tokens of the tile
            const int nch = (nv + 15) / 16;                                  // their chunks of 16
            int c_lo = 0, c_hi = nch;
            if (OP == OP_GLU) {
                const int half = (bn / 16 + 1) / 2;
                c_lo = h ? half : 0;
                c_hi = h ? nch : (nch < half ? nch : half);
            } else if (h && mt * 512 + 256 >= Rpad) {
                c_hi = 0;
            }
            if (sk && kb0 > 0) {
                // later part of a split tile: the fp32 partial (real tokens) goes to
                // the owner.  A range that holds only blocks of absent adapters ran
                // no MMA: its part is zero, not what tensor memory holds.
                const bool none = OP == OP_LORA && kb0 >= tile_blocks(nt);
                float *slot = slot_of(cluster);
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    uint32_t v[NACC][16];
#pragma unroll
                    for (int a = 0; a < NACC; ++a) tmem_ld_32x32b_x16(tacc[a] + c * 16, v[a]);
                    tmem_ld_wait();
#pragma unroll
                    for (int a = 0; a < NACC; ++a)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c * 16 + j < nv)
                                __stcg(slot + (((c - c_lo) * NACC + a) * 16 + j) * 32,
                                       none ? 0.0f : __uint_as_float(v[a][j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty_cl);
                __threadfence();
                __syncwarp();
                if (lane == 0 && cluster != g_test_withhold_flag_cluster)
                    st_release_u64(flags + (cluster * 2 + rank) * 8 + we, p.seq);
                continue;
            }
            int64_t last_contrib = cluster;
            if (sk && kb1 < nkt) {
                // owner of a split tile (always this cluster's last segment): wait for
                // the clusters after this one that hold the rest, each lane polling one
                // flag, and clear it once seen, so that a replay of the same launch
                // (the same sequence number) waits for its own partial sums
                while (last_contrib + 1 < nclusters &&
                       (last_contrib + 1) * total / nclusters < (tile + 1) * nkt)
                    ++last_contrib;
                bool got = true;
                for (int64_t base = cluster + 1; base <= last_contrib && got; base += 32) {
                    const int64_t cc = base + lane;
                    bool mine = true;
                    if (cc <= last_contrib && has_work(cc)) {
                        uint64_t *fl = flags + (cc * 2 + rank) * 8 + we;
                        mine = sk_wait_flag(fl, p.seq);
                        if (mine) *reinterpret_cast<volatile uint64_t *>(fl) = 0;
                    }
                    got = __all_sync(0xffffffffu, mine);
                }
            }
            const int64_t row = mt * TILE_ROWS + (OP == OP_LORA ? h * 256 : 0) + rank * 128 + q * 32 + lane;
            const bool rok = row < p.R;
            uint32_t pk[8][8];
            // two passes of eight chunks (OP_GLU: one); the accumulator is released
            // once the last chunk is in registers, before its stores
#pragma unroll 1
            for (int c8 = c_lo; c8 < c_hi || c8 == c_lo; c8 += 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int c = c8 + k;
                    if (c < c_hi) {
                        uint32_t v[NACC][16];
                        float f[NACC][16];
#pragma unroll
                        for (int a = 0; a < NACC; ++a) tmem_ld_32x32b_x16(tacc[a] + c * 16, v[a]);
                        tmem_ld_wait();
#pragma unroll
                        for (int a = 0; a < NACC; ++a)
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[a][j] = __uint_as_float(v[a][j]);
                        if (last_contrib > cluster) {
                            for (int64_t cc = cluster + 1; cc <= last_contrib; ++cc) {
                                if (!has_work(cc)) continue;
                                const float *ps = slot_of(cc) + (c - c_lo) * NACC * 16 * 32;
#pragma unroll
                                for (int a = 0; a < NACC; ++a)
#pragma unroll
                                    for (int j = 0; j < 16; ++j)
                                        if (c * 16 + j < nv) f[a][j] += __ldcg(ps + (a * 16 + j) * 32);
                            }
                        }
                        if (OP == OP_GLU) {
                            const int64_t t = tok0 + c * 16;
                            if (p.G != nullptr && rok) {
                                uint16_t *gp = p.G + t * p.ldgu + row, *up = p.U + t * p.ldgu + row;
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    const uint32_t g2 = pack_bf16x2(f[0][j], f[0][j + 1]);
                                    const uint32_t u2 = pack_bf16x2(f[1][j], f[1][j + 1]);
                                    if (c * 16 + j < nv) {
                                        gp[j * p.ldgu] = static_cast<uint16_t>(g2 & 0xFFFFu);
                                        up[j * p.ldgu] = static_cast<uint16_t>(u2 & 0xFFFFu);
                                    }
                                    if (c * 16 + j + 1 < nv) {
                                        gp[(j + 1) * p.ldgu] = static_cast<uint16_t>(g2 >> 16);
                                        up[(j + 1) * p.ldgu] = static_cast<uint16_t>(u2 >> 16);
                                    }
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[0][j] = act_of(f[0][j], p.act) * f[NACC - 1][j];
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) pk[k][i] = pack_bf16x2(f[0][2 * i], f[0][2 * i + 1]);
                    }
                }
                if (c8 + 8 >= c_hi) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(acc_empty_cl);
                }
                if (rok) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int c = c8 + k;
                        if (c < c_hi) {
                            uint16_t *yp = p.Y + (tok0 + c * 16) * p.ldy + row;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (c * 16 + 2 * i < nv) yp[0] = static_cast<uint16_t>(pk[k][i] & 0xFFFFu);
                                if (c * 16 + 2 * i + 1 < nv) yp[p.ldy] = static_cast<uint16_t>(pk[k][i] >> 16);
                                yp += 2 * p.ldy;
                            }
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// adapters: which of them a token tile holds, and V = scale X A^T
//
// The requests' tokens are consecutive: request i has tokens [indptr[i],
// indptr[i+1]) and adapter ids[i] (-1: none); tokens behind the last request
// have none.  A slot is one (token tile, adapter that occurs in it); its V is
// [bn x r], zero in the rows of other tokens.  Tile i's slots start at i * cap
// (few adapters) or at i + (the request of its first token): along the batch
// each tile or request border starts at most one new pair, so that numbering
// leaves every tile room and needs requests + tiles slots in all.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    k_lora_plan(const int32_t *__restrict__ indptr, const int32_t *__restrict__ ids, int32_t requests,
                int32_t adapters, int64_t T, int bn, int cap, int by_cap, int64_t nslots,
                int32_t *__restrict__ token_slot, int32_t *__restrict__ tile_cnt,
                int32_t *__restrict__ tile_base, int32_t *__restrict__ slot_adapter) {
    __shared__ int32_t adp[256];
    __shared__ int32_t slot_at[256];
    __shared__ int32_t warp_cnt[8];
    __shared__ int32_t first_q;
    grid_dep_launch();
    const int tile = blockIdx.x, i = threadIdx.x, warp = i >> 5, lane = i & 31;
    const int64_t t = static_cast<int64_t>(tile) * bn + i;
    bool bad = false;
    if (tile == 0) {  // the whole list once: ascending, within [0, T], known adapters
        for (int q = i; q < requests; q += 256) {
            const int32_t lo = __ldg(indptr + q), hi = __ldg(indptr + q + 1), a = __ldg(ids + q);
            bad |= lo < 0 || lo > hi || hi > T || a < -1 || a >= adapters;
        }
    }
    int32_t a = -1;
    if (i < bn && t < T) {
        int lo = 0, hi = requests;  // the first request that ends behind t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(indptr + mid + 1) > t) hi = mid; else lo = mid + 1;
        }
        if (lo < requests && __ldg(indptr + lo) <= t) {
            a = __ldg(ids + lo);
            if (a < 0 || a >= adapters) a = -1;
        }
        if (i == 0) first_q = lo;
    }
    adp[i] = a;
    __syncthreads();
    int first = i;
    if (a >= 0) {
        for (int k = 0; k < i; ++k)
            if (adp[k] == a) {
                first = k;
                break;
            }
    }
    const bool opens = a >= 0 && first == i;
    const uint32_t b = __ballot_sync(0xffffffffu, opens);
    if (lane == 0) warp_cnt[warp] = __popc(b);
    __syncthreads();
    int before = __popc(b & ((1u << lane) - 1u)), cnt = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) before += warp_cnt[w];
        cnt += warp_cnt[w];
    }
    const int64_t base = by_cap ? static_cast<int64_t>(tile) * cap : tile + static_cast<int64_t>(first_q);
    // a list out of order could ask for more: what does not fit is left out
    int64_t room = nslots - base;
    if (room < 0) room = 0;
    if (room > cap) room = cap;
    if (opens) slot_at[i] = before < room ? before : -1;
    if (opens && before < room) slot_adapter[base + before] = a;
    bad |= cnt > room;
    __syncthreads();
    if (i < bn) token_slot[t] = a >= 0 ? slot_at[first] : -1;
    if (i == 0) {
        tile_cnt[tile] = static_cast<int32_t>(cnt < room ? cnt : room);
        tile_base[tile] = static_cast<int32_t>(base < nslots ? base : 0);
    }
    if (bad) raise_error(ERRBIT_DEVICE);
    grid_dep_wait();  // completes after the staging kernel before it, for the GEMM's sake
}

// eight bf16 of a row from column k on, zero past K
__device__ __forceinline__ uint4 row8(const uint16_t *__restrict__ row, int64_t k, int64_t K) {
    if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < K) w[j >> 1] |= static_cast<uint32_t>(__ldg(row + k + j)) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// V of one (slot, 32 tokens, 64 ranks): K in blocks of 32, block w, w + 8, ...
// to warp w; a thread's 16-byte loads of X and A cover the same eight columns,
// which the two mma k-steps of a block take in a permuted order (the same one
// for both, so the sum is the product's).  The eight warps' fp32 sums meet in
// shared memory in a fixed order.  grid: x = 32-token chunks of a tile, y =
// token tiles, z = rank block + rb x slot lane.
constexpr int SHRINK_TOKENS = 32, SHRINK_RANKS = 64;
constexpr int SHRINK_SMEM = 8 * SHRINK_TOKENS * SHRINK_RANKS * 4;

__global__ void __launch_bounds__(256)
    k_lora_shrink(const uint16_t *__restrict__ X, int64_t T, int64_t K, int64_t ldx,
                  const uint16_t *__restrict__ A, int64_t lda, int64_t sda, int r, const float *__restrict__ scale,
                  const int32_t *__restrict__ token_slot, const int32_t *__restrict__ tile_cnt,
                  const int32_t *__restrict__ tile_base, const int32_t *__restrict__ slot_adapter, int bn, int rb,
                  uint16_t *__restrict__ V) {
    extern __shared__ float red[];  // [warp][token][rank]
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
    const int64_t tile = blockIdx.y, t0 = tile * bn + blockIdx.x * SHRINK_TOKENS;
    const int in_tile = blockIdx.x * SHRINK_TOKENS;
    const int rk = static_cast<int>(blockIdx.z % rb) * SHRINK_RANKS;
    const int lanes_z = gridDim.z / rb;
    const int nr = r - rk < SHRINK_RANKS ? r - rk : SHRINK_RANKS, nn = nr / 8;
    grid_dep_wait();
    const int my = in_tile + lane < bn ? __ldcg(token_slot + t0 + lane) : -1;
    const int cnt = __ldcg(tile_cnt + tile);
    const int64_t base = __ldcg(tile_base + tile);
    for (int j = blockIdx.z / rb; j < cnt; j += lanes_z) {
        const uint32_t mem = __ballot_sync(0xffffffffu, my == j);  // the same in every warp
        uint16_t *vrow = V + ((base + j) * bn + in_tile) * static_cast<int64_t>(r) + rk;
        const int rows = bn - in_tile < SHRINK_TOKENS ? bn - in_tile : SHRINK_TOKENS;
        if (mem == 0) {
            for (int e = threadIdx.x; e < rows * nn; e += 256)
                *reinterpret_cast<uint4 *>(vrow + static_cast<int64_t>(e / nn) * r + (e % nn) * 8) =
                    make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        const int32_t ad = __ldcg(slot_adapter + base + j);
        const uint16_t *arow = A + ad * sda + static_cast<int64_t>(rk) * lda;
        float acc[2][8][4];
#pragma unroll
        for (int mtile = 0; mtile < 2; ++mtile)
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mtile][n][e] = 0.0f;
        const bool hi = (mem >> 16) != 0u;
#pragma unroll 2
        for (int64_t k0 = warp * 32; k0 < K; k0 += 256) {
            const int64_t k = k0 + tg * 8;
            uint4 x[2][2], b[8];
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int mtile = 0; mtile < 2; ++mtile)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int tok = mtile * 16 + u * 8 + g;
                    x[mtile][u] = (mem >> tok) & 1u ? row8(X + (t0 + tok) * ldx, k, K) : zero;
                }
#pragma unroll
            for (int n = 0; n < 8; ++n)
                b[n] = n < nn ? row8(arow + static_cast<int64_t>(n * 8 + g) * lda, k, K) : zero;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n >= nn) break;
                mma_16816(acc[0][n], x[0][0].x, x[0][1].x, x[0][0].y, x[0][1].y, b[n].x, b[n].y);
                mma_16816(acc[0][n], x[0][0].z, x[0][1].z, x[0][0].w, x[0][1].w, b[n].z, b[n].w);
                if (hi) {
                    mma_16816(acc[1][n], x[1][0].x, x[1][1].x, x[1][0].y, x[1][1].y, b[n].x, b[n].y);
                    mma_16816(acc[1][n], x[1][0].z, x[1][1].z, x[1][0].w, x[1][1].w, b[n].z, b[n].w);
                }
            }
        }
        float *mine = red + warp * SHRINK_TOKENS * SHRINK_RANKS;
#pragma unroll
        for (int mtile = 0; mtile < 2; ++mtile)
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n >= nn) break;
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    *reinterpret_cast<float2 *>(mine + (mtile * 16 + u * 8 + g) * SHRINK_RANKS + n * 8 + 2 * tg) =
                        make_float2(acc[mtile][n][2 * u], acc[mtile][n][2 * u + 1]);
            }
        __syncthreads();
        const float sc = __ldg(scale + ad);
        const int half = nr / 2;
        for (int e = threadIdx.x; e < rows * half; e += 256) {
            const int tok = e / half, c = 2 * (e % half);
            float s0 = 0.0f, s1 = 0.0f;
            if ((mem >> tok) & 1u) {
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float2 f = *reinterpret_cast<const float2 *>(red + (w * SHRINK_TOKENS + tok) * SHRINK_RANKS + c);
                    s0 += f.x;
                    s1 += f.y;
                }
                s0 *= sc;
                s1 *= sc;
            }
            *reinterpret_cast<uint32_t *>(vrow + static_cast<int64_t>(tok) * r + c) = pack_bf16x2(s0, s1);
        }
        __syncthreads();
    }
}

}  // namespace nm

// ===========================================================================
// host side
// ===========================================================================
using namespace nm;

namespace {

// CTA pairs of k_ffn<MODE, OP> that can be resident at once on the current
// device (0 on a CUDA error), cached per device
template <int MODE, int OP>
int64_t ffn_pairs() {
    using Cfg = FfnCfg;
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cache[dev] == 0) {
        if (!set_smem_attr<k_ffn<MODE, OP>>(Cfg::SMEM_BYTES)) return 0;
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(2 * static_cast<unsigned>(sm_count() / 2), 1, 1);
        q.blockDim = dim3(Cfg::THREADS, 1, 1);
        q.dynamicSmemBytes = Cfg::SMEM_BYTES;
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 2;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k_ffn<MODE, OP>, &q) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 0;
        }
        cache[dev] = n < sm_count() / 2 ? n : sm_count() / 2;
    }
    int64_t res = cache[dev];
    const int forced = g_sched_clusters.load();
    if (forced > 0 && forced < res) res = forced;
    if (res > NM_GEMM_STREAMK_MAX_CLUSTERS) res = NM_GEMM_STREAMK_MAX_CLUSTERS;
    return res < 1 ? 1 : res;
}

// tokens per tile: the fewest tiles of at most 240 tokens or, when that is
// several, one or two more, whichever needs the least (waves over the resident
// pairs) x (N/2 + 32 clocks an MMA of N tokens costs per K' step)
int ffn_bn(int64_t T, int64_t n_m, int64_t pairs) {
    const int64_t nt0 = (T + FfnCfg::BN_MAX - 1) / FfnCfg::BN_MAX;
    const int64_t nt_last = nt0 >= 2 ? nt0 + 2 : nt0;
    int64_t best = 0, best_cost = 0;
    for (int64_t nt = nt0; nt <= nt_last; ++nt) {
        const int64_t bn = ((T + nt - 1) / nt + 15) / 16 * 16;
        const int64_t tiles = ((T + bn - 1) / bn) * n_m;
        const int64_t cost = ((tiles + pairs - 1) / pairs) * (bn + 32);
        if (best == 0 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    return static_cast<int>(best);
}

template <int MODE, int OP>
nm_status launch_ffn(const FfnMaps &maps, FfnArgs p, int64_t pairs, void *sk_ws, size_t sk_ws_bytes,
                     cudaStream_t s) {
    using Cfg = FfnCfg;
    const int64_t Rpad = (p.R + 255) / 256 * 256;
    const int64_t rows = OP == OP_GLU ? 256 : 512;
    const int64_t ntiles = ((p.T + p.bn - 1) / p.bn) * ((Rpad + rows - 1) / rows);
    const int policy = g_sched_policy.load();
    const bool sk_ok = sk_ws != nullptr && sk_ws_bytes >= ffn_sk_bytes(pairs);
    const bool sk = sk_ok && (policy == 2 || (policy == 0 && 2 * ntiles <= pairs));
    const int64_t clusters = sk ? pairs : (ntiles < pairs ? ntiles : pairs);
    p.stage_bytes = Cfg::stage_bytes(p.bn);
    p.stages = Cfg::stages(p.bn);
    p.sk = sk ? 1 : 0;
    p.sk_ws = sk ? static_cast<uint8_t *>(sk_ws) : nullptr;
    p.seq = sk ? next_seq() : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, k_ffn<MODE, OP>, maps, p) != cudaSuccess) return NM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

bool pattern_ok(int m) { return m == 4 || m == 6 || m == 8 || m == 10; }

// values and metadata of one packed operand
bool packed_maps(CUtensorMap *a, CUtensorMap *e, const void *packed, const PackedGeom &g) {
    const uint8_t *meta = static_cast<const uint8_t *>(packed) + g.vals_bytes;
    return make_tmap_bf16(a, packed, g.Rpad, g.KLpad / 2, g.KLpad / 2, 64, BM, true) &&
           make_tmap_2d(e, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, meta, (g.Rpad / BM) * g.nkb * 8, 256, 256, 256, 8,
                        false);
}

nm_status check_ffn_sizes(int64_t T, int64_t K, int64_t R, int m) {
    if (T < 1 || K < 1 || R < 1 || T > 0x7FFFFFFF - 256 || K > 0x7FFFFFFF / 4 || R > 0x7FFFFFFF - 512)
        return NM_ERR_SHAPE;
    if (!pattern_ok(m)) return NM_ERR_UNSUPPORTED;
    const PackedGeom g = packed_geom(R, K, m);
    if (g.nkb > 0x7FFFFFFF / 8 || (g.Rpad / BM) * g.nkb * 8 > 0x7FFFFFFF) return NM_ERR_SHAPE;
    return NM_OK;
}

// stages the activations where the pattern needs it and encodes the B maps
nm_status stage_b(const uint16_t *X, int64_t T, int64_t K, int64_t ldx, int m, const PackedGeom &g, const GemmWs &w,
                  void *ws, int bn, FfnMaps *maps, cudaStream_t s) {
    uint16_t *stage = static_cast<uint16_t *>(ws);
    const uint32_t bh = static_cast<uint32_t>(bn / 2);
    const uint16_t *src = X;
    int64_t cols = K, ld = ldx;
    nm_status st = NM_OK;
    if (m == 8) {
        st = launch_gather_mid(X, T, K, ldx, g.G, stage, w.ld, s);
    } else if (m != 4) {
        st = lift_activations(X, T, K, ldx, m, stage, w.ld, s);
        src = stage;
        cols = w.cols;
        ld = w.ld;
    }
    if (st != NM_OK) return st;
    if (!make_tmap_bf16(&maps->b, src, T, cols, ld, 64, bh, true)) return NM_ERR_CUDA;
    maps->b2 = maps->b;
    if (m == 8 && !make_tmap_bf16(&maps->b2, stage, T, w.cols, w.ld, 64, bh, true)) return NM_ERR_CUDA;
    return NM_OK;
}

// sizes of the adapters' part of the workspace, for any tile width: slots of
// bn rows number at most min(requests + tiles, tiles x cap) with cap =
// min(requests, adapters, bn), bn <= 240 and tiles x bn < T + 240
struct LoraWs {
    int64_t token_slot, tiles, slots, v_rows;  // elements of each region
    size_t o_token, o_cnt, o_base, o_adapter, o_v, bytes;
};

LoraWs lora_ws(int64_t T, int64_t r, int64_t requests, int64_t adapters) {
    LoraWs l{};
    const int64_t bnm = FfnCfg::BN_MAX;
    int64_t cap = requests < adapters ? requests : adapters;
    if (cap > bnm) cap = bnm;
    l.token_slot = T + bnm;
    l.tiles = T / 16 + 2;
    const int64_t by_req = requests + l.tiles, by_cap = l.tiles * cap;
    l.slots = by_req < by_cap ? by_req : by_cap;
    const int64_t rows_req = (requests + 1) * bnm + T, rows_cap = (T + bnm) * cap;
    l.v_rows = rows_req < rows_cap ? rows_req : rows_cap;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    size_t o = 0;
    l.o_token = o, o += up(static_cast<size_t>(l.token_slot) * 4);
    l.o_cnt = o, o += up(static_cast<size_t>(l.tiles) * 4);
    l.o_base = o, o += up(static_cast<size_t>(l.tiles) * 4);
    l.o_adapter = o, o += up(static_cast<size_t>(l.slots) * 4);
    l.o_v = o, o += up(static_cast<size_t>(l.v_rows) * static_cast<size_t>(r) * 2);
    l.bytes = o;
    return l;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

extern "C" size_t nm_sparse_glu_workspace_bytes(int64_t T, int64_t K, int m) {
    if (T < 1 || K < 1 || !pattern_ok(m)) return 0;
    return sk_offset(gemm_ws(T, K, m)) + ffn_sk_bytes(NM_GEMM_STREAMK_MAX_CLUSTERS);
}

extern "C" nm_status nm_sparse_glu(const uint16_t *X, int64_t T, int64_t K, int64_t ldx, const void *packed_gate,
                                   const void *packed_up, int64_t R, int m, int act, uint16_t *H, int64_t ldh,
                                   uint16_t *G, uint16_t *U, int64_t ldgu, void *ws, size_t ws_bytes,
                                   void *stream) {
    if (!X || !packed_gate || !packed_up || !H || (G == nullptr) != (U == nullptr)) return NM_ERR_NULL;
    nm_status st = check_ffn_sizes(T, K, R, m);
    if (st != NM_OK) return st;
    if (act < ACT_SILU || act > ACT_RELU2) return NM_ERR_UNSUPPORTED;
    if (ldx < K || ldh < R || (G && ldgu < R)) return NM_ERR_SHAPE;
    if (!aligned16(X) || !aligned16(packed_gate) || !aligned16(packed_up) || !aligned16(H) || (ldx % 8) != 0 ||
        (ldh % 8) != 0 || (G && (!aligned16(G) || !aligned16(U) || (ldgu % 8) != 0)) || (ws && !aligned16(ws)))
        return NM_ERR_ALIGN;
    const GemmWs w = gemm_ws(T, K, m);
    if (w.bytes > 0 && (!ws || ws_bytes < w.bytes)) return NM_ERR_WORKSPACE;
    const PackedGeom g = packed_geom(R, K, m);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t pairs = m == 8 ? ffn_pairs<PMODE_SP68T, OP_GLU>() : ffn_pairs<PMODE_SP24, OP_GLU>();
    if (pairs == 0) return NM_ERR_CUDA;
    FfnMaps maps{};
    FfnArgs p{};
    p.T = T;
    p.R = R;
    p.nkb = g.nkb;
    p.bn = ffn_bn(T, g.Rpad / 256, pairs);
    p.early = m == 8 ? 1 : 0;  // the gather runs just before; X and the weights are older
    p.Y = H;
    p.ldy = ldh;
    p.G = G;
    p.U = U;
    p.ldgu = ldgu;
    p.act = act;
    if (!packed_maps(&maps.a0, &maps.e0, packed_gate, g) || !packed_maps(&maps.a1, &maps.e1, packed_up, g))
        return NM_ERR_CUDA;
    st = stage_b(X, T, K, ldx, m, g, w, ws, p.bn, &maps, s);
    if (st != NM_OK) return st;
    const size_t sko = sk_offset(w);
    void *skw = ws && ws_bytes > sko ? static_cast<uint8_t *>(ws) + sko : nullptr;
    const size_t skb = skw ? ws_bytes - sko : 0;
    return m == 8 ? launch_ffn<PMODE_SP68T, OP_GLU>(maps, p, pairs, skw, skb, s)
                  : launch_ffn<PMODE_SP24, OP_GLU>(maps, p, pairs, skw, skb, s);
}

extern "C" size_t nm_sparse_gemm_lora_workspace_bytes(int64_t T, int64_t K, int m, int64_t r, int64_t adapters,
                                                      int64_t requests) {
    if (T < 1 || K < 1 || !pattern_ok(m) || r < 8 || r > NM_LORA_MAX_RANK || (r % 8) != 0 || adapters < 1 ||
        requests < 0)
        return 0;
    return sk_offset(gemm_ws(T, K, m)) + up256(ffn_sk_bytes(NM_GEMM_STREAMK_MAX_CLUSTERS)) +
           lora_ws(T, r, requests, adapters).bytes;
}

extern "C" nm_status nm_sparse_gemm_lora(const uint16_t *X, int64_t T, int64_t K, int64_t ldx, const void *packed,
                                         int64_t R, int m, const uint16_t *A, int64_t lda, int64_t sda,
                                         const uint16_t *B, int64_t ldb, int64_t sdb, const float *scale,
                                         int64_t adapters, int64_t r, const int32_t *indptr, const int32_t *ids,
                                         int64_t requests, uint16_t *Y, int64_t ldy, void *ws, size_t ws_bytes,
                                         void *stream) {
    if (!X || !packed || !A || !B || !scale || !indptr || (requests > 0 && !ids) || !Y || !ws) return NM_ERR_NULL;
    nm_status st = check_ffn_sizes(T, K, R, m);
    if (st != NM_OK) return st;
    if (r < 8 || r > NM_LORA_MAX_RANK || (r % 8) != 0) return NM_ERR_UNSUPPORTED;
    if (adapters < 1 || adapters > 0x7FFFFFFF || requests < 0 || requests > 0x7FFFFFFF / 256 || ldx < K || ldy < R ||
        lda < K || ldb < r || sda < (r - 1) * lda + K || sdb < (R - 1) * ldb + r)
        return NM_ERR_SHAPE;
    if (!aligned16(X) || !aligned16(packed) || !aligned16(A) || !aligned16(B) || !aligned16(Y) || !aligned16(ws) ||
        (ldx % 8) != 0 || (ldy % 8) != 0 || (lda % 8) != 0 || (ldb % 8) != 0 || (sda % 8) != 0 || (sdb % 8) != 0 ||
        ((reinterpret_cast<uintptr_t>(scale) | reinterpret_cast<uintptr_t>(indptr) |
          reinterpret_cast<uintptr_t>(ids)) & 3u) != 0)
        return NM_ERR_ALIGN;
    if (ws_bytes < nm_sparse_gemm_lora_workspace_bytes(T, K, m, r, adapters, requests)) return NM_ERR_WORKSPACE;
    const GemmWs w = gemm_ws(T, K, m);
    const LoraWs l = lora_ws(T, r, requests, adapters);
    if (l.v_rows > 0x7FFFFFFF || l.slots > 0x7FFFFFFF) return NM_ERR_SHAPE;
    const PackedGeom g = packed_geom(R, K, m);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t pairs = m == 8 ? ffn_pairs<PMODE_SP68T, OP_LORA>() : ffn_pairs<PMODE_SP24, OP_LORA>();
    if (pairs == 0 || !set_smem_attr<k_lora_shrink>(SHRINK_SMEM)) return NM_ERR_CUDA;
    uint8_t *skw = static_cast<uint8_t *>(ws) + sk_offset(w);
    const size_t skb = ffn_sk_bytes(NM_GEMM_STREAMK_MAX_CLUSTERS);
    uint8_t *lw = skw + up256(skb);
    int32_t *token_slot = reinterpret_cast<int32_t *>(lw + l.o_token);
    int32_t *tile_cnt = reinterpret_cast<int32_t *>(lw + l.o_cnt);
    int32_t *tile_base = reinterpret_cast<int32_t *>(lw + l.o_base);
    int32_t *slot_adapter = reinterpret_cast<int32_t *>(lw + l.o_adapter);
    uint16_t *V = reinterpret_cast<uint16_t *>(lw + l.o_v);

    FfnMaps maps{};
    FfnArgs p{};
    p.T = T;
    p.R = R;
    p.nkb = g.nkb;
    p.bn = ffn_bn(T, (g.Rpad + 511) / 512, pairs);
    p.early = m == 4 || m == 8 ? 1 : 0;  // 4:6 and 8:10 read the lifted activations from the first block on
    p.Y = Y;
    p.ldy = ldy;
    p.rb = static_cast<int>((r + 63) / 64);
    const int64_t tiles = (T + p.bn - 1) / p.bn;
    int64_t cap = requests < adapters ? requests : adapters;
    if (cap > p.bn) cap = p.bn;
    p.ext_cap = static_cast<int>(cap);
    const int by_cap = tiles * cap <= requests + tiles ? 1 : 0;
    const int64_t nslots = by_cap ? tiles * cap : requests + tiles;
    p.tile_cnt = tile_cnt;
    p.tile_base = tile_base;
    p.slot_adapter = slot_adapter;
    if (tiles > 65535) return NM_ERR_SHAPE;
    if (!packed_maps(&maps.a0, &maps.e0, packed, g)) return NM_ERR_CUDA;
    maps.a1 = maps.a0;
    maps.e1 = maps.e0;
    if (cap > 0) {
        if (!make_tmap_bf16_3d(&maps.lb, B, adapters, R, r, ldb, sdb, 64, BM) ||
            !make_tmap_bf16(&maps.lv, V, nslots * p.bn, r, r, 64, static_cast<uint32_t>(p.bn / 2), true))
            return NM_ERR_CUDA;
    } else {
        maps.lb = maps.a0;
        maps.lv = maps.a0;
        if (m == 4) p.early = 0;  // no kernel of this call runs before the GEMM
    }
    st = stage_b(X, T, K, ldx, m, g, w, ws, p.bn, &maps, s);
    if (st != NM_OK) return st;
    if (cap > 0) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = s;
        cfg.attrs = attr;
        // behind the staging kernel the plan may start early; else it is this
        // call's first kernel and follows the stream's earlier work
        cfg.numAttrs = m == 4 ? 0 : 1;
        if (cudaLaunchKernelEx(&cfg, k_lora_plan, indptr, ids, static_cast<int32_t>(requests),
                               static_cast<int32_t>(adapters), T, p.bn, p.ext_cap, by_cap, nslots, token_slot,
                               tile_cnt, tile_base, slot_adapter) != cudaSuccess)
            return NM_ERR_CUDA;
        const int64_t chunks = (p.bn + SHRINK_TOKENS - 1) / SHRINK_TOKENS;
        int64_t lanes = 2 * sm_count() / (tiles * chunks) + 1;
        if (lanes > cap) lanes = cap;
        cfg.gridDim = dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(tiles),
                           static_cast<unsigned>(lanes * p.rb));
        cfg.dynamicSmemBytes = SHRINK_SMEM;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, k_lora_shrink, X, T, K, ldx, A, lda, sda, static_cast<int>(r), scale,
                               const_cast<const int32_t *>(token_slot), const_cast<const int32_t *>(tile_cnt),
                               const_cast<const int32_t *>(tile_base), const_cast<const int32_t *>(slot_adapter),
                               p.bn, p.rb, V) != cudaSuccess)
            return NM_ERR_CUDA;
    }
    return m == 8 ? launch_ffn<PMODE_SP68T, OP_LORA>(maps, p, pairs, skw, skb, s)
                  : launch_ffn<PMODE_SP24, OP_LORA>(maps, p, pairs, skw, skb, s);
}

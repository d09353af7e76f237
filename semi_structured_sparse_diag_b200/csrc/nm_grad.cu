// nm_grad.cu -- the backward pass of the gated feed-forward's first half
// H = act(G) U, G = X Wg^T, U = X Wu^T with (m-2):m sparse Wg, Wu:
//   dG = dH U act'(G),  dU = dH act(G)                      (k_glu_grad)
//   dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X        (k_gemm_grad)
// and the masked dense form of a pruned weight (k_densify).
//
// The transpose of an (m-2):m matrix is not (m-2):m along its rows, so dX
// takes the masked weights in dense form; all three products run on the dense
// tensor cores.  No operand is transposed in memory: a matrix whose
// contraction runs down its rows (Wg, Wu in dX; dG, dU and X in dW) is read by
// TMA as it lies and handed to tcgen05.mma as an MN-major operand.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "nm_common.cuh"
#include "nm_gemm.cuh"
#include "nm_host.cuh"

namespace nm {

// act(g) and act'(g) in fp32.  silu: s = 1/(1+e^-g), s(1 + g(1-s)).  gelu (tanh
// form), with z = c(g + a g^3): s = 1/(1+e^-2z) = (1 + tanh z)/2, slope
// s + 2 g s (1-s) c (1 + 3 a g^2).  relu^2: 2 max(g, 0).
__device__ __forceinline__ void act_and_slope(float g, int act, float &f, float &d) {
    if (act == NM_ACT_RELU2) {
        const float r = g < 0.0f ? 0.0f : g;
        f = r * r;
        d = 2.0f * r;
        return;
    }
    if (act == NM_ACT_SILU) {
        const float e = __expf(-g), s = __fdividef(1.0f, 1.0f + e);
        f = g * s;
        d = s * (1.0f + g * (1.0f - s));
        return;
    }
    const float z2 = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float s = __fdividef(1.0f, 1.0f + __expf(-z2));
    f = g * s;
    // where s (1 - s) has vanished the slope is s, though g^2 may overflow
    const float t = s * (1.0f - s);
    d = t == 0.0f ? s : s + g * t * 1.5957691216057308f * (1.0f + 0.134145f * g * g);
}

// dG and dU, one rounding to bf16 each (they are tensor-core operands next).
// A thread takes eight columns of a row: three 16-byte loads, two stores.
// grid: x over 8-column chunks, y (+65535 z) over rows.
__global__ void __launch_bounds__(256)
    k_glu_grad(const uint16_t *__restrict__ dH, int64_t lddh, const uint16_t *__restrict__ G,
               const uint16_t *__restrict__ U, int64_t ldgu, int64_t T, int64_t R, int act,
               uint16_t *__restrict__ dG, uint16_t *__restrict__ dU, int64_t ldd) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8;
    if (t >= T || c >= R) return;
    const uint16_t *hp = dH + t * lddh + c, *gp = G + t * ldgu + c, *up = U + t * ldgu + c;
    uint32_t h[4], g[4], u[4], og[4], ou[4];
    if (c + 8 <= R) {
        *reinterpret_cast<uint4 *>(h) = __ldg(reinterpret_cast<const uint4 *>(hp));
        *reinterpret_cast<uint4 *>(g) = __ldg(reinterpret_cast<const uint4 *>(gp));
        *reinterpret_cast<uint4 *>(u) = __ldg(reinterpret_cast<const uint4 *>(up));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = g[i] = u[i] = 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (c + 2 * i + e < R) {
                    h[i] |= static_cast<uint32_t>(hp[2 * i + e]) << (16 * e);
                    g[i] |= static_cast<uint32_t>(gp[2 * i + e]) << (16 * e);
                    u[i] |= static_cast<uint32_t>(up[2 * i + e]) << (16 * e);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float rg[2], ru[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            auto val = [&](uint32_t w) { return __uint_as_float(e ? (w & 0xFFFF0000u) : (w << 16)); };
            float f, d;
            act_and_slope(val(g[i]), act, f, d);
            rg[e] = val(h[i]) * val(u[i]) * d;
            ru[e] = val(h[i]) * f;
        }
        og[i] = pack_bf16x2(rg[0], rg[1]);
        ou[i] = pack_bf16x2(ru[0], ru[1]);
    }
    // the rows of dG and dU are padded to 8 columns: whole chunks
    *reinterpret_cast<uint4 *>(dG + t * ldd + c) = *reinterpret_cast<uint4 *>(og);
    *reinterpret_cast<uint4 *>(dU + t * ldd + c) = *reinterpret_cast<uint4 *>(ou);
}

// ---------------------------------------------------------------------------
// The three products, in one launch unless they are large: dense bf16 operands,
// fp32 accumulation, bf16 results.  Persistent CTA pairs, 256 x 256 tiles, two
// accumulators in tensor memory (the epilogue of a tile overlaps the next tile's
// MMAs), six 32 KB stages; warps as in k_gemm_pair, with the loading and the issuing
// warp in step and one lane of each at work.  8192 tokens, 11008 x 4096, in a loop
// of seconds at the power cap: 93% of cuBLAS' rate for the same products (dX some
// 1.14 ms to 1.05, dWg and dWu 1.17 to 1.09; 1.2 GHz against 1.4 to 1.5).
//   dX  [T x K]: A = dG, then dU [T x R] (K-major), B = Wg, then Wu [R x K]
//       (MN-major); the contraction is R twice.
//   dWg, dWu [R x K]: A = dG or dU [T x R], B = X [T x K], both MN-major,
//       contraction T.
// MN-major operand tiles: TMA boxes of 64 columns x 64 contraction rows
// (128-byte swizzle): rows of 128 bytes are consecutive contraction steps, so
// eight of them make a swizzle atom (1024 bytes, the descriptor's stride
// offset) and the next 64 columns lie one box (8192 bytes, the leading
// offset) further; a k-step of 16 advances by two atoms.
//
// The tiles of dX come first, then those of dWg and dWu.  With few tokens dX
// has too few tiles for the device and a long contraction (and reads all of Wg
// and Wu): a cluster of `split` pairs then shares one tile of it, each with its
// part of the contraction, and the fp32 sums are added through distributed
// shared memory, in the pairs' order, as in the gated product (SPLIT).
// ---------------------------------------------------------------------------
struct GradCfg {
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int MAX_SPLIT = MAX_PAIRS;
    static constexpr int SUM_BYTES = 256 * 128 * 4;        // a CTA's sums, over the idle stages
    static constexpr int EPI_WARPS = 8;
    static constexpr int EPI_BYTES = EPI_WARPS * 32 * 128;  // 32 rows x 64 columns bf16 each
    static constexpr int THREADS = 384;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 256 + 1024;
    static_assert(SMEM_BYTES <= 232448 && SUM_BYTES <= STAGES * STAGE_BYTES, "shared memory");
};

struct GradMaps {
    CUtensorMap g[2];              // dG, dU as dX's A (boxes 64 x 128)
    CUtensorMap w[2];              // Wg, Wu (boxes 64 x 64)
    CUtensorMap gt[2], x;          // dG, dU and X as operands of dW (boxes 64 x 64)
    CUtensorMap dx, dw[2];         // the results
};

struct GradArgs {
    int64_t T, R, K;
    int64_t tiles_x, tiles_w;      // tiles of dX; of dWg (and of dWu)
    int split;
    uint16_t *dX;
    int64_t lddx;
    const uint32_t *mask[2];       // keep bits of dWg, dWu (or NULL: all kept)
    int64_t mask_words;            // per row
};

// The tiles of one pair, in order.  dX: the cluster's tile (SPLIT, at most one
// each) or pair, pair + pairs, ..  dW: likewise, but where the last round of dX
// leaves pairs out (out0 and up), those come first, and first take `extra` tiles
// each, about as much work.
struct GradIter {
    int64_t n_x, n_w, pairs, pair, out0, extra, jx, jw;
    __device__ GradIter(const GradArgs &p, int64_t cluster, int64_t part, int64_t clusters)
        : n_x(p.tiles_x), n_w(2 * p.tiles_w), pairs(clusters * p.split), pair(cluster * p.split + part), jx(0), jw(0) {
        if (p.split > 1) {
            out0 = n_x * p.split;  // pairs of clusters without a tile of dX
            jx = cluster < n_x ? cluster : n_x;
        } else {
            out0 = n_x % pairs == 0 ? pairs : n_x % pairs;
            jx = pair;
        }
        // in blocks of the contraction; with few tokens a tile of dW takes as long as
        // its epilogue, some six blocks
        const int64_t bx = 2 * ((p.R + 63) / 64) / p.split, bw = (p.T + 63) / 64;
        const int64_t c = bw > 6 ? bw : 6;
        extra = n_x == 0 ? 0 : (bx + c / 2) / c;
        if (extra * (pairs - out0) > n_w) extra = 0;
        split = p.split;
    }
    int split;
    // false: no more.  is_x: a tile of dX; else src and the tile of dW
    __device__ bool next(bool &is_x, int &src, int64_t &tile) {
        src = 0;
        if (jx < n_x) {
            is_x = true;
            tile = jx;
            jx = split > 1 ? n_x : jx + pairs;
            return true;
        }
        is_x = false;
        const int64_t given = extra * (pairs - out0);  // handed out in advance
        int64_t idx;
        if (pair >= out0 && jw < extra)
            idx = (pair - out0) * extra + jw;
        else
            idx = given + (pair >= out0 ? pair - out0 : pair + pairs - out0) + (jw - (pair >= out0 ? extra : 0)) * pairs;
        ++jw;
        if (idx >= n_w) return false;
        src = idx >= n_w / 2 ? 1 : 0;
        tile = idx - src * (n_w / 2);
        return true;
    }
};

template <bool SPLIT>
__global__ void __launch_bounds__(GradCfg::THREADS, 1)
    k_gemm_grad(const __grid_constant__ GradMaps tm, const __grid_constant__ GradArgs p) {
    using C = GradCfg;
    constexpr int S = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *epi_smem = smem + S * C::STAGE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + C::EPI_BYTES);
    uint64_t *full = bars, *empty = bars + S, *acc_full = bars + 2 * S, *acc_empty = acc_full + 2;
    uint64_t *sum_ready = acc_full + 4, *sum_free = acc_full + 5;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 6);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank(), rank = crank & 1u, leader = crank & ~1u;
    const int split = SPLIT ? p.split : 1, part = SPLIT ? static_cast<int>(crank >> 1) : 0;
    const int64_t cluster = blockIdx.x / (2 * split), nclusters = gridDim.x / (2 * split);
    const int64_t n_n = (p.K + 255) / 256;                        // column tiles of every result
    const int64_t m_x = (p.T + 255) / 256, m_w = (p.R + 255) / 256;
    const int nkr = static_cast<int>((p.R + 63) / 64), nkt = static_cast<int>((p.T + 63) / 64);
    const int x0 = static_cast<int>(2ll * nkr * part / split), x1 = static_cast<int>(2ll * nkr * (part + 1) / split);
    constexpr int64_t BAND = 16;  // row tiles per band of the tile order

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);
        }
        mbar_init(sum_ready, split * C::EPI_WARPS);
        mbar_init(sum_free, split * C::EPI_WARPS);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_wait();
    grid_dep_launch();  // the stream's next kernel may set itself up

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        const bool lead = elect_one() != 0u;
        const uint32_t st0 = smem_u32(smem), full0 = mapa_shared(full, leader);
        int s = 0;
        uint32_t ph = 0;
        int64_t it = 0, tile;
        bool ok = true, is_x, shared_sums = false;
        int src;
        GradIter tiles(p, cluster, part, nclusters);
        while (ok && tiles.next(is_x, src, tile)) {
            int64_t nt, mt;
            tile_coords(tile, n_n, is_x ? m_x : m_w, BAND, nt, mt);
            const int32_t m0 = static_cast<int32_t>(mt * 256 + rank * 128);
            const int32_t n0 = static_cast<int32_t>(nt * 256 + rank * 128);
            // SPLIT: the sums of the tile of dX lie over the stages until all have read them
            if (SPLIT && shared_sums) {
                if (!mbar_wait_cluster_warp(sum_free, 0)) { ok = false; break; }
                fence_proxy_async_smem();
            }
            shared_sums = SPLIT && is_x;
            const int v1 = is_x ? x1 : nkt;
            for (int v = is_x ? x0 : 0; v < v1; ++v, ++it) {
                if (it >= S && !mbar_wait_warp(&empty[s], ph ^ 1u)) { ok = false; break; }
                if (lead) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * C::STAGE_BYTES);
                    const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                    const uint32_t sa = st0 + static_cast<uint32_t>(s) * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    if (is_x) {
                        const int which = v >= nkr ? 1 : 0;
                        const int32_t k0 = (v - which * nkr) * 64;
                        tma_load_2d_pair_at(sa, &tm.g[which], bar, k0, m0);
                        tma_load_2d_pair_at(sb, &tm.w[which], bar, n0, k0);
                        tma_load_2d_pair_at(sb + 8192, &tm.w[which], bar, n0 + 64, k0);
                    } else {
                        tma_load_2d_pair_at(sa, &tm.gt[src], bar, m0, v * 64);
                        tma_load_2d_pair_at(sa + 8192, &tm.gt[src], bar, m0 + 64, v * 64);
                        tma_load_2d_pair_at(sb, &tm.x, bar, n0, v * 64);
                        tma_load_2d_pair_at(sb + 8192, &tm.x, bar, n0 + 64, v * 64);
                    }
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok && rank == 0) {  // let copies already issued land before exiting
            for (int64_t j = (it > S ? it - S : 0); j < it; ++j)
                mbar_wait_warp(&full[j % S], static_cast<uint32_t>((j / S) & 1));
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const bool lead = elect_one() != 0u;
            // bits 15 and 16: A and B are MN-major
            const uint32_t idesc = make_idesc_bf16(256, 256, false, 0) | (1u << 16);
            const uint16_t both = static_cast<uint16_t>(3u << leader);
            const uint32_t st0 = smem_u32(smem);
            const uint64_t ak = make_sdesc(st0, 16, 1024, 2), am = make_sdesc(st0, 8192, 1024, 2);
            const uint64_t bm = make_sdesc(st0 + C::A_BYTES, 8192, 1024, 2);
            int s = 0;
            uint32_t ph = 0;
            int64_t ti = 0, tile;
            bool ok = true, is_x;
            int src;
            GradIter tiles(p, cluster, part, nclusters);
            for (; ok && tiles.next(is_x, src, tile); ++ti) {
                const int buf = static_cast<int>(ti & 1);
                const uint32_t aph = static_cast<uint32_t>((ti >> 1) & 1);
                if (ti >= 2 && !mbar_wait_cluster_warp(&acc_empty[buf], aph ^ 1u)) break;
                tc_fence_after();
                const uint32_t dcol = tmem_base + static_cast<uint32_t>(buf * 256);
                const int n = is_x ? x1 - x0 : nkt;
                const uint64_t ad = is_x ? ak : am, astep = is_x ? 32 >> 4 : 2048 >> 4;
                const uint32_t id = idesc | (is_x ? 0u : 1u << 15);
                for (int v = 0; v < n; ++v) {
                    if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = static_cast<uint64_t>(static_cast<uint32_t>(s) * (C::STAGE_BYTES >> 4));
                    if (lead) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_bf16_pair(dcol, ad + so + j * astep, bm + so + j * (2048 >> 4), id,
                                          (v > 0 || j > 0) ? 1u : 0u);
                        mma_commit_pair_mask(&empty[s], both);
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (ok && lead) mma_commit_pair_mask(&acc_full[buf], both);
                __syncwarp();
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // ---------------------------------------------------------- epilogue
        // lane = row of the tile's lane quarter q, 128 columns of half h; 64
        // columns at a time through shared memory (128-byte rows, swizzled as
        // the store's tensor map expects) and out by TMA
        const int q = warp & 3, h = (warp - 4) >> 2;
        uint8_t *out = epi_smem + (warp - 4) * 4096;
        const uint32_t acc_empty0 = mapa_shared(&acc_empty[0], leader), acc_empty1 = mapa_shared(&acc_empty[1], leader);
        int64_t ti = 0, tile;
        bool is_x;
        int src;
        GradIter tiles(p, cluster, part, nclusters);
        for (; tiles.next(is_x, src, tile); ++ti) {
            int64_t nt, mt;
            tile_coords(tile, n_n, is_x ? m_x : m_w, BAND, nt, mt);
            const int buf = static_cast<int>(ti & 1);
            if (!mbar_wait_warp(&acc_full[buf], static_cast<uint32_t>((ti >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(buf * 256 + h * 128);
            const int64_t row = mt * 256 + rank * 128 + q * 32 + lane;
            const int64_t col0 = nt * 256 + h * 128;
            if constexpr (SPLIT) {
                if (is_x) {
                    // [4 columns][row][column] fp32 over the stages, which are idle: every
                    // load of the tile has been used
                    float4 *mine = reinterpret_cast<float4 *>(smem) + (h * 32) * 128 + q * 32 + lane;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tb + c * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mine[(c * 8 + i) * 128] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                                  __uint_as_float(v[4 * i + 2]),
                                                                  __uint_as_float(v[4 * i + 3]));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(buf ? acc_empty1 : acc_empty0);
                    if (lane < split) mbar_arrive_cluster(mapa_shared(sum_ready, 2 * lane + rank));
                    if (!mbar_wait_cluster_warp(sum_ready, 0)) break;
                    const uint32_t off = smem_u32(mine);
                    uint32_t from[C::MAX_SPLIT];
#pragma unroll
                    for (int i = 0; i < C::MAX_SPLIT; ++i)
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                     : "=r"(from[i]) : "r"(off), "r"(2 * (i < split ? i : part) + rank));
#pragma unroll 1
                    for (int g = 32 * part / split; g < 32 * (part + 1) / split; ++g) {  // this pair's columns
                        float4 pv[C::MAX_SPLIT];
#pragma unroll
                        for (int i = 0; i < C::MAX_SPLIT; ++i)
                            if (i < split) pv[i] = ld_dsmem_f32x4(from[i] + static_cast<uint32_t>(g * 2048));
                        float4 f = pv[0];
#pragma unroll
                        for (int i = 1; i < C::MAX_SPLIT; ++i)
                            if (i < split) {
                                f.x += pv[i].x;
                                f.y += pv[i].y;
                                f.z += pv[i].z;
                                f.w += pv[i].w;
                            }
                        const int64_t col = col0 + g * 4;
                        if (row < p.T && col < p.K) {
                            const uint32_t lo = pack_bf16x2(f.x, f.y), hi = pack_bf16x2(f.z, f.w);
                            uint16_t *dst = p.dX + row * p.lddx + col;
                            if (col + 4 <= p.K) {
                                *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
                            } else {
                                dst[0] = static_cast<uint16_t>(lo & 0xFFFFu);
                                if (col + 1 < p.K) dst[1] = static_cast<uint16_t>(lo >> 16);
                                if (col + 2 < p.K) dst[2] = static_cast<uint16_t>(hi & 0xFFFFu);
                            }
                        }
                    }
                    __syncwarp();
                    fence_proxy_async_smem();  // the stages go back to TMA
                    if (lane < split) mbar_arrive_cluster(mapa_shared(sum_free, 2 * lane + rank));
                    continue;
                }
            }
            const uint32_t *mrow = !is_x && p.mask[src] != nullptr && row < p.R ? p.mask[src] + row * p.mask_words
                                                                                 : nullptr;
            const int64_t rows = is_x ? p.T : p.R;
            const CUtensorMap *tc = is_x ? &tm.dx : (src ? &tm.dw[1] : &tm.dw[0]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t v[64], w[32];
                tmem_ld_32x32b_x64(tb + c * 64, v);
                uint32_t keep[2] = {~0u, ~0u};
                if (mrow != nullptr) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int64_t word = (col0 + c * 64) / 32 + k;
                        keep[k] = word < p.mask_words ? __ldg(mrow + word) : 0u;
                    }
                }
                tmem_ld_wait();
                if (c == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(buf ? acc_empty1 : acc_empty0);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    uint32_t x = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    const uint32_t kb = keep[i >> 4] >> (2 * (i & 15));
                    x &= ((kb & 1u) ? 0xFFFFu : 0u) | ((kb & 2u) ? 0xFFFF0000u : 0u);
                    w[i] = x;
                }
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(out + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && mt * 256 + rank * 128 + q * 32 < rows && col0 + c * 64 < p.K) {
                    tma_store_2d(tc, out, static_cast<int32_t>(col0 + c * 64),
                                 static_cast<int32_t>(mt * 256 + rank * 128 + q * 32));
                    bulk_commit_group();
                }
            }
        }
        if (lane == 0) bulk_wait_group0();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // also: no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// W = mask (.) V in dense form from the kept values and the mask.  One thread
// per mask word (32 columns).  Every group holds n kept values, so a word's
// first value sits at (groups before it) n + the kept positions of the group
// that the word's start cuts.  grid: x over words, y (+65535 z) over rows.
// 11008 x 4096: 2:4 52 us, 6:8 51, floors 22 and 25 (141 and 163 MB); bound by a
// two-byte load per kept value.  It runs once a training step beside products of
// milliseconds.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128)
    k_densify(const uint16_t *__restrict__ vals, const uint32_t *__restrict__ mask, int64_t R, int64_t K, int n,
              int m, int64_t G, int64_t words, uint16_t *__restrict__ W, int64_t ldw) {
    const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r >= R || w >= words) return;
    const uint32_t *mrow = mask + r * words;
    const uint32_t prev = w > 0 ? __ldg(mrow + w - 1) : 0u, cur = __ldg(mrow + w);
    const uint32_t next = w + 1 < words ? __ldg(mrow + w + 1) : 0u;
    const int64_t g0 = 32 * w / m;
    const int cut = static_cast<int>(32 * w - g0 * m);  // bits of group g0 in the previous word
    int64_t at = g0 * n + (cut > 0 ? __popc(prev >> (32 - cut)) : 0);
    const int64_t len = G * n;
    const uint16_t *vrow = vals + r * len;
    bool bad = false;
    for (int64_t g = cut > 0 ? g0 + 1 : g0; g * m < 32 * w + 32 && g < G; ++g) {  // groups that start here
        const int b = static_cast<int>(g * m - 32 * w);
        const uint32_t bits = __funnelshift_r(cur, next, b) & ((1u << m) - 1u);
        bad |= __popc(bits) != n;
    }
    uint32_t o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        o[i] = 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if ((cur >> (2 * i + e)) & 1u) {
                if (at < len) o[i] |= static_cast<uint32_t>(__ldg(vrow + at)) << (16 * e);
                ++at;
            }
    }
    uint16_t *dst = W + r * ldw + 32 * w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (32 * w + 8 * i + 8 <= K) {
            reinterpret_cast<uint4 *>(dst)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (32 * w + 8 * i + e < K)
                    dst[8 * i + e] = static_cast<uint16_t>(o[4 * i + e / 2] >> (16 * (e & 1)));
        }
    }
    if (bad) raise_error(ERRBIT_DEVICE);
}

}  // namespace nm

// ===========================================================================
// host side
// ===========================================================================
using namespace nm;

namespace {

int64_t padded8(int64_t n) { return (n + 7) / 8 * 8; }

size_t grad_bytes(int64_t T, int64_t R) {  // one of dG, dU
    return (static_cast<size_t>(T) * static_cast<size_t>(padded8(R)) * 2 + 255) / 256 * 256;
}

template <bool SPLIT>
int64_t grad_clusters(int split) {
    return resident_clusters_of<k_gemm_grad<SPLIT>>(split, GradCfg::THREADS, GradCfg::SMEM_BYTES);
}

nm_status launch_grad(const GradMaps &maps, GradArgs p, cudaStream_t s) {
    using Cfg = GradCfg;
    // pairs per tile of dX: the least of (contraction blocks of a pair) x ~600
    // clocks + the exchange of 128 KB of sums at some 18 bytes a clock; a split
    // needs a cluster for every tile.  nm_gemm_set_schedule: 1 never splits, 2
    // always where that holds, and its cluster count bounds the clusters.
    const int policy = g_sched_policy.load(), bound = g_sched_clusters.load();
    auto bounded = [&](int64_t n) { return bound > 0 && bound < n ? static_cast<int64_t>(bound) : n; };
    int split = 1;
    int64_t clusters = bounded(grad_clusters<false>(1));
    const int64_t blocks = 2 * ((p.R + 63) / 64);
    int64_t best = policy == 2 ? INT64_MAX : blocks * 600;
    for (int i = 2; i <= Cfg::MAX_SPLIT && p.tiles_x > 0 && i <= blocks && policy != 1; ++i) {
        const int64_t cost = (blocks + i - 1) / i * 600 + 10000;
        if (cost >= best) continue;
        const int64_t n = bounded(grad_clusters<true>(i));
        if (n < p.tiles_x) continue;
        best = cost;
        split = i;
        clusters = n;
    }
    if (clusters < 1) return NM_ERR_CUDA;
    const int64_t want = split > 1 ? p.tiles_x + (2 * p.tiles_w + split - 1) / split : p.tiles_x + 2 * p.tiles_w;
    if (clusters > want) clusters = want;
    p.split = split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * split * clusters), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = split > 1 ? cudaLaunchKernelEx(&cfg, k_gemm_grad<true>, maps, p)
                                    : cudaLaunchKernelEx(&cfg, k_gemm_grad<false>, maps, p);
    if (e != cudaSuccess) return NM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

}  // namespace

extern "C" size_t nm_sparse_glu_backward_workspace_bytes(int64_t T, int64_t R) {
    if (T < 1 || R < 1) return 0;
    return 2 * grad_bytes(T, R);
}

extern "C" nm_status nm_sparse_glu_backward(const uint16_t *dH, int64_t lddh, const uint16_t *X, int64_t T, int64_t K,
                                            int64_t ldx, const uint16_t *G, const uint16_t *U, int64_t ldgu,
                                            const uint16_t *Wg, const uint16_t *Wu, int64_t R, int64_t ldw, int act,
                                            const uint32_t *mask_gate, const uint32_t *mask_up, int m, uint16_t *dX,
                                            int64_t lddx, uint16_t *dWg, uint16_t *dWu, int64_t lddw, void *ws,
                                            size_t ws_bytes, void *stream) {
    const bool need_w = dWg != nullptr || dWu != nullptr;
    if (!dH || !G || !U || !ws || (!dX && !need_w) || (dX && (!Wg || !Wu)) || (need_w && (!X || !dWg || !dWu)) ||
        (mask_gate == nullptr) != (mask_up == nullptr))
        return NM_ERR_NULL;
    if (T < 1 || K < 1 || R < 1 || T > 0x7FFFFFFF - 512 || K > 0x7FFFFFFF - 512 || R > 0x7FFFFFFF - 512 ||
        lddh < R || ldgu < R || (need_w && (ldx < K || lddw < K)) || (dX && (ldw < K || lddx < K)))
        return NM_ERR_SHAPE;
    if (act < NM_ACT_SILU || act > NM_ACT_RELU2 || (mask_gate && (m < 2 || m > 16))) return NM_ERR_UNSUPPORTED;
    if (!aligned16(dH) || !aligned16(G) || !aligned16(U) || !aligned16(ws) || (lddh % 8) != 0 || (ldgu % 8) != 0 ||
        (dX && (!aligned16(Wg) || !aligned16(Wu) || !aligned16(dX) || (ldw % 8) != 0 || (lddx % 8) != 0)) ||
        (need_w && (!aligned16(X) || !aligned16(dWg) || !aligned16(dWu) || (ldx % 8) != 0 || (lddw % 8) != 0)) ||
        ((reinterpret_cast<uintptr_t>(mask_gate) | reinterpret_cast<uintptr_t>(mask_up)) & 3u) != 0)
        return NM_ERR_ALIGN;
    if (ws_bytes < nm_sparse_glu_backward_workspace_bytes(T, R)) return NM_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint16_t *dG = static_cast<uint16_t *>(ws);
    uint16_t *dU = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + grad_bytes(T, R));
    const int64_t ldd = padded8(R);

    GradMaps maps{};
    GradArgs p{};
    p.T = T;
    p.R = R;
    p.K = K;
    if (dX) {
        if (!make_tmap_bf16(&maps.g[0], dG, T, R, ldd, 64, 128, true) ||
            !make_tmap_bf16(&maps.g[1], dU, T, R, ldd, 64, 128, true) ||
            !make_tmap_bf16(&maps.w[0], Wg, R, K, ldw, 64, 64, true) ||
            !make_tmap_bf16(&maps.w[1], Wu, R, K, ldw, 64, 64, true) ||
            !make_tmap_bf16(&maps.dx, dX, T, K, lddx, 64, 32, true))
            return NM_ERR_CUDA;
        p.tiles_x = ((T + 255) / 256) * ((K + 255) / 256);
        p.dX = dX;
        p.lddx = lddx;
    }
    if (need_w) {
        if (!make_tmap_bf16(&maps.gt[0], dG, T, R, ldd, 64, 64, true) ||
            !make_tmap_bf16(&maps.gt[1], dU, T, R, ldd, 64, 64, true) ||
            !make_tmap_bf16(&maps.x, X, T, K, ldx, 64, 64, true) ||
            !make_tmap_bf16(&maps.dw[0], dWg, R, K, lddw, 64, 32, true) ||
            !make_tmap_bf16(&maps.dw[1], dWu, R, K, lddw, 64, 32, true))
            return NM_ERR_CUDA;
        p.tiles_w = ((R + 255) / 256) * ((K + 255) / 256);
        p.mask[0] = mask_gate;
        p.mask[1] = mask_up;
        p.mask_words = mask_gate ? ((K + m - 1) / m * m + 31) / 32 : 0;
    }
    const int64_t chunks = (R + 7) / 8;
    dim3 grid(static_cast<unsigned>((chunks + 255) / 256), static_cast<unsigned>(T < 65535 ? T : 65535),
              static_cast<unsigned>((T + 65534) / 65535));
    if (!launch_dependent(k_glu_grad, grid, 256, s, dH, lddh, G, U, ldgu, T, R, act, dG, dU, ldd)) return NM_ERR_CUDA;
    // With rounds of dX enough that the last one costs little, dX has a launch of
    // its own: pairs at work on dW beside it push its operands out of L2 (8192
    // tokens, 11008 x 4096: 2.00 ms and 4.7 GB read, against 2.05 ms and 5.8 GB)
    if (dX && need_w && p.tiles_x >= 4 * (sm_count() / 2)) {
        GradArgs x = p;
        x.tiles_w = 0;
        const nm_status st = launch_grad(maps, x, s);
        if (st != NM_OK) return st;
        p.tiles_x = 0;
    }
    return launch_grad(maps, p, s);
}

extern "C" nm_status nm_sparse_densify(const uint16_t *vals, const uint32_t *mask, int64_t R, int64_t K, int n, int m,
                                       uint16_t *W, int64_t ldw, void *stream) {
    if (!vals || !mask || !W) return NM_ERR_NULL;
    if (R < 1 || K < 1 || ldw < K || K > 0x7FFFFFFF - 64 || R > 65535LL * 65535LL) return NM_ERR_SHAPE;
    if (m < 2 || m > 16 || n < 1 || n >= m) return NM_ERR_UNSUPPORTED;
    if (!aligned16(W) || (ldw % 8) != 0 || (reinterpret_cast<uintptr_t>(vals) & 1u) ||
        (reinterpret_cast<uintptr_t>(mask) & 3u))
        return NM_ERR_ALIGN;
    const int64_t G = (K + m - 1) / m, words = (G * m + 31) / 32;
    dim3 grid(static_cast<unsigned>((words + 127) / 128), static_cast<unsigned>(R < 65535 ? R : 65535),
              static_cast<unsigned>((R + 65534) / 65535));
    k_densify<<<grid, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(vals, mask, R, K, n, m, G, words, W, ldw);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

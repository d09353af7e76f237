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

enum { GACT_SILU = 0, GACT_GELU = 1, GACT_RELU2 = 2 };

// act(g) and act'(g) in fp32.  silu: s = 1/(1+e^-g), s(1 + g(1-s)).  gelu (tanh
// form), with z = c(g + a g^3): s = 1/(1+e^-2z) = (1 + tanh z)/2, slope
// s + 2 g s (1-s) c (1 + 3 a g^2).  relu^2: 2 max(g, 0).
__device__ __forceinline__ void act_and_slope(float g, int act, float &f, float &d) {
    if (act == GACT_RELU2) {
        const float r = g < 0.0f ? 0.0f : g;
        f = r * r;
        d = 2.0f * r;
        return;
    }
    if (act == GACT_SILU) {
        const float e = __expf(-g), s = __fdividef(1.0f, 1.0f + e);
        f = g * s;
        d = s * (1.0f + g * (1.0f - s));
        return;
    }
    const float z2 = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float s = __fdividef(1.0f, 1.0f + __expf(-z2));
    f = g * s;
    d = s + g * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * g * g);
}

// dG and dU, one rounding to bf16 each (they are tensor-core operands next).
// A thread takes eight columns of a row: three 16-byte loads, two stores.
// grid: x over 8-column chunks, y (+65535 z) over rows.
__global__ void __launch_bounds__(256)
    k_glu_grad(const uint16_t *__restrict__ dH, int64_t lddh, const uint16_t *__restrict__ G,
               const uint16_t *__restrict__ U, int64_t ldgu, int64_t T, int64_t R, int act,
               uint16_t *__restrict__ dG, uint16_t *__restrict__ dU, int64_t ldd) {
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
// C[M x N] = sum over the contraction of A and B, dense bf16 operands, fp32
// accumulation, bf16 C.  Persistent CTA pairs, 256 x 256 tiles, two
// accumulators in tensor memory (the epilogue of a tile overlaps the next
// tile's MMAs), six 32 KB stages; warps as in k_gemm_pair.
//   GRAD_X : A = dG, then dU [T x R] (K-major), B = Wg, then Wu [R x K]
//            (MN-major); the contraction is R twice.  C = dX [T x K].
//   GRAD_W : A = dG or dU [T x R], B = X [T x K], both MN-major, contraction T.
//            Two problems side by side: tiles of dWg, then of dWu.
// MN-major operand tiles: TMA boxes of 64 columns x 64 contraction rows
// (128-byte swizzle): rows of 128 bytes are consecutive contraction steps, so
// eight of them make a swizzle atom (1024 bytes, the descriptor's stride
// offset) and the next 64 columns lie one box (8192 bytes, the leading
// offset) further; a k-step of 16 advances by two atoms.
// ---------------------------------------------------------------------------
enum { GRAD_X = 0, GRAD_W = 1 };

struct GradCfg {
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int EPI_WARPS = 8;
    static constexpr int EPI_BYTES = EPI_WARPS * 32 * 128;  // 32 rows x 64 columns bf16 each
    static constexpr int THREADS = 384;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + 256 + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct GradMaps {
    CUtensorMap a[2], b[2], c[2];
};

struct GradArgs {
    int64_t M, N, nkb;             // rows, columns; contraction blocks of 64 of one source
    const uint32_t *mask[2];       // GRAD_W: keep bits of C's columns (or NULL: all kept)
    int64_t mask_words;            // words per row
};

template <int KIND>
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int64_t n_n = (p.N + 255) / 256, n_m = (p.M + 255) / 256;
    const int64_t per = n_n * n_m;                                // tiles of one problem
    const int64_t ntiles = KIND == GRAD_W ? 2 * per : per;
    const int64_t nkb = KIND == GRAD_X ? 2 * p.nkb : p.nkb;
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
        fence_barrier_init();
        prefetch_tmap(&tm.a[0]);
        prefetch_tmap(&tm.b[0]);
        prefetch_tmap(&tm.c[0]);
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

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t it = 0;
            bool ok = true;
            for (int64_t tile = cluster; tile < ntiles && ok; tile += nclusters) {
                const int src = KIND == GRAD_W && tile >= per ? 1 : 0;
                int64_t nt, mt;
                tile_coords(tile - src * per, n_n, n_m, BAND, nt, mt);
                const int32_t m0 = static_cast<int32_t>(mt * 256 + rank * 128);
                const int32_t n0 = static_cast<int32_t>(nt * 256 + rank * 128);
                for (int64_t v = 0; v < nkb; ++v) {
                    if (it >= S && !mbar_wait(&empty[s], ph ^ 1u)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * C::STAGE_BYTES);
                    const uint32_t bar = mapa_shared(&full[s], 0);
                    uint8_t *sa = smem + s * C::STAGE_BYTES, *sb = sa + C::A_BYTES;
                    const int which = KIND == GRAD_W ? src : (v >= p.nkb ? 1 : 0);
                    const int32_t k0 = static_cast<int32_t>((KIND == GRAD_X && which ? v - p.nkb : v) * 64);
                    if (KIND == GRAD_X) {
                        tma_load_2d_pair(sa, &tm.a[which], bar, k0, m0);
                    } else {
                        tma_load_2d_pair(sa, &tm.a[which], bar, m0, k0);
                        tma_load_2d_pair(sa + 8192, &tm.a[which], bar, m0 + 64, k0);
                    }
                    const CUtensorMap *tb = &tm.b[KIND == GRAD_X ? which : 0];
                    tma_load_2d_pair(sb, tb, bar, n0, k0);
                    tma_load_2d_pair(sb + 8192, tb, bar, n0 + 64, k0);
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
            // bits 15 and 16: A and B are MN-major
            const uint32_t idesc = make_idesc_bf16(256, 256, false, 0) | (1u << 16) | (KIND == GRAD_W ? 1u << 15 : 0u);
            int s = 0;
            uint32_t ph = 0;
            int64_t ti = 0;
            bool ok = true;
            for (int64_t tile = cluster; tile < ntiles && ok; tile += nclusters, ++ti) {
                const int buf = static_cast<int>(ti & 1);
                const uint32_t aph = static_cast<uint32_t>((ti >> 1) & 1);
                if (ti >= 2 && !mbar_wait_cluster(&acc_empty[buf], aph ^ 1u)) break;
                tc_fence_after();
                const uint32_t dcol = tmem_base + static_cast<uint32_t>(buf * 256);
                for (int64_t v = 0; v < nkb; ++v) {
                    if (!mbar_wait(&full[s], ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(smem + s * C::STAGE_BYTES), b0 = a0 + C::A_BYTES;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16_pair(dcol,
                                      KIND == GRAD_X ? make_sdesc(a0 + j * 32, 16, 1024, 2)
                                                     : make_sdesc(a0 + j * 2048, 8192, 1024, 2),
                                      make_sdesc(b0 + j * 2048, 8192, 1024, 2), idesc, (v > 0 || j > 0) ? 1u : 0u);
                    mma_commit_pair(&empty[s]);
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (ok) mma_commit_pair(&acc_full[buf]);
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // ---------------------------------------------------------- epilogue
        // lane = row of the tile's lane quarter q, 128 columns of half h; 64
        // columns at a time through shared memory (128-byte rows, swizzled as
        // the store's tensor map expects) and out by TMA
        const int q = warp & 3, h = (warp - 4) >> 2;
        uint8_t *out = epi_smem + (warp - 4) * 4096;
        const uint32_t acc_empty_cl[2] = {mapa_shared(&acc_empty[0], 0), mapa_shared(&acc_empty[1], 0)};
        int64_t ti = 0;
        for (int64_t tile = cluster; tile < ntiles; tile += nclusters, ++ti) {
            const int src = KIND == GRAD_W && tile >= per ? 1 : 0;
            int64_t nt, mt;
            tile_coords(tile - src * per, n_n, n_m, BAND, nt, mt);
            const int buf = static_cast<int>(ti & 1);
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], static_cast<uint32_t>((ti >> 1) & 1)))) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(buf * 256 + h * 128);
            const int64_t row = mt * 256 + rank * 128 + q * 32 + lane;
            const int64_t col0 = nt * 256 + h * 128;
            const uint32_t *mrow = KIND == GRAD_W && p.mask[src] != nullptr && row < p.M
                                       ? p.mask[src] + row * p.mask_words : nullptr;
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
                    if (lane == 0) mbar_arrive_cluster(acc_empty_cl[buf]);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    uint32_t x = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    if (KIND == GRAD_W) {
                        const uint32_t kb = keep[i >> 4] >> (2 * (i & 15));
                        x &= ((kb & 1u) ? 0xFFFFu : 0u) | ((kb & 2u) ? 0xFFFF0000u : 0u);
                    }
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
                if (lane == 0 && mt * 256 + rank * 128 + q * 32 < p.M && col0 + c * 64 < p.N) {
                    tma_store_2d(&tm.c[src], out, static_cast<int32_t>(col0 + c * 64),
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
    cluster_sync_all();
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

template <int KIND>
nm_status launch_grad(const GradMaps &maps, const GradArgs &p, int64_t ntiles, cudaStream_t s) {
    using Cfg = GradCfg;
    if (!set_smem_attr<k_gemm_grad<KIND>>(Cfg::SMEM_BYTES)) return NM_ERR_CUDA;
    const int64_t pairs = sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (ntiles < pairs ? ntiles : pairs)), 1, 1);
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
    if (cudaLaunchKernelEx(&cfg, k_gemm_grad<KIND>, maps, p) != cudaSuccess) return NM_ERR_CUDA;
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
    if (act < GACT_SILU || act > GACT_RELU2 || (mask_gate && (m < 2 || m > 16))) return NM_ERR_UNSUPPORTED;
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

    GradMaps mx{}, mw{};
    if (dX && (!make_tmap_bf16(&mx.a[0], dG, T, R, ldd, 64, 128, true) ||
               !make_tmap_bf16(&mx.a[1], dU, T, R, ldd, 64, 128, true) ||
               !make_tmap_bf16(&mx.b[0], Wg, R, K, ldw, 64, 64, true) ||
               !make_tmap_bf16(&mx.b[1], Wu, R, K, ldw, 64, 64, true) ||
               !make_tmap_bf16(&mx.c[0], dX, T, K, lddx, 64, 32, true)))
        return NM_ERR_CUDA;
    if (need_w && (!make_tmap_bf16(&mw.a[0], dG, T, R, ldd, 64, 64, true) ||
                   !make_tmap_bf16(&mw.a[1], dU, T, R, ldd, 64, 64, true) ||
                   !make_tmap_bf16(&mw.b[0], X, T, K, ldx, 64, 64, true) ||
                   !make_tmap_bf16(&mw.c[0], dWg, R, K, lddw, 64, 32, true) ||
                   !make_tmap_bf16(&mw.c[1], dWu, R, K, lddw, 64, 32, true)))
        return NM_ERR_CUDA;
    const int64_t chunks = (R + 7) / 8;
    dim3 grid(static_cast<unsigned>((chunks + 255) / 256), static_cast<unsigned>(T < 65535 ? T : 65535),
              static_cast<unsigned>((T + 65534) / 65535));
    k_glu_grad<<<grid, 256, 0, s>>>(dH, lddh, G, U, ldgu, T, R, act, dG, dU, ldd);
    if (cudaGetLastError() != cudaSuccess) return NM_ERR_CUDA;
    if (dX) {
        GradArgs p{};
        p.M = T;
        p.N = K;
        p.nkb = (R + 63) / 64;
        mx.c[1] = mx.c[0];
        const nm_status st = launch_grad<GRAD_X>(mx, p, ((T + 255) / 256) * ((K + 255) / 256), s);
        if (st != NM_OK) return st;
    }
    if (need_w) {
        GradArgs p{};
        p.M = R;
        p.N = K;
        p.nkb = (T + 63) / 64;
        p.mask[0] = mask_gate;
        p.mask[1] = mask_up;
        p.mask_words = mask_gate ? ((K + m - 1) / m * m + 31) / 32 : 0;
        mw.b[1] = mw.b[0];
        return launch_grad<GRAD_W>(mw, p, 2 * ((R + 255) / 256) * ((K + 255) / 256), s);
    }
    return NM_OK;
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

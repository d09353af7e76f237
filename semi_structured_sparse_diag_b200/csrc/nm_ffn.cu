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
// Where the time goes (device time, 11008 x 4096 2:4 projections): one token
// through gate and up 20.0 us, 101 MB of operands at 5.1 TB/s (78% of a measured
// copy): HBM, and some 5 us of start and tail.  8192 tokens with G and U kept
// 713 us in a long run, which the power cap bounds (1.4 GHz); 494 us at
// 1965 MHz, the tensor pipe 68% active: 15 us of products and 5 us of epilogue a
// tile, the latter bound by all SMs' stores at once.  8192 tokens with rank 64
// adapters 330 to 380 us, of which the product 284 and V 41.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "nm_common.cuh"
#include "nm_gemm.cuh"
#include "nm_host.cuh"

namespace nm {

enum { OP_GLU = 0, OP_LORA = 1 };

// epilogue warps: what a tile waits for is their latency, so the plain kernel has
// sixteen; the exchange of a split needs more registers than that leaves
constexpr int ffn_epi_warps(bool split) { return split ? 8 : 16; }
constexpr int ffn_threads(bool split) { return 128 + 32 * ffn_epi_warps(split); }

struct FfnCfg {
    static constexpr int BN_MAX = 240;          // tokens per tile (both CTAs)
    static constexpr int A_BYTES = BM * 128;    // 128 rows x 64 values
    static constexpr int OFF_A0 = 0, OFF_A1 = A_BYTES, OFF_E0 = 2 * A_BYTES, OFF_E1 = OFF_E0 + EBLK_BYTES;
    static constexpr int OFF_B = OFF_E1 + EBLK_BYTES;  // two atoms of bn/2 tokens x 64 columns
    static constexpr int MAX_STAGES = 6;
    static constexpr int MAX_SPLIT = MAX_PAIRS; // CTA pairs that share a tile's K' blocks
    static constexpr int BAR_BYTES = 256;
    static constexpr int SMEM_BYTES = 232448;
    static constexpr int SMEM_DATA = (SMEM_BYTES - BAR_BYTES - 1024) / 1024 * 1024;
    // without a split: the epilogue's output staging, 1 KB a warp
    static constexpr int OUT_BYTES = ffn_epi_warps(false) * 1024, OFF_OUT = SMEM_DATA - OUT_BYTES;
    static constexpr int TMEM_COLS = 512;
    static constexpr int TMEM_D0 = 0, TMEM_E0 = 240, TMEM_E1 = 248, TMEM_D1 = 256;
    static_assert(OFF_B % 1024 == 0, "operand alignment");
    static int stage_bytes(int bn) { return OFF_B + bn * 128; }
    static int sum_bytes(int bn) { return bn * 1024; }  // both accumulators of a CTA in fp32
};

struct FfnMaps {
    CUtensorMap a0, a1, e0, e1;  // values and metadata of the two accumulators' weights
    CUtensorMap b, b2;           // activations; 6:8: the gathered middle windows
    CUtensorMap lb, lv;          // OP_LORA: the adapters' B, the shrunk activations V
};

struct FfnArgs {
    int64_t T, R, nkb;
    int bn, stages, stage_bytes;
    int split;    // CTA pairs of a cluster that share a tile
    int sum_off;  // split > 1: where a CTA leaves its fp32 sums in shared memory
    int early;    // loads of X and the weights need not wait for the preceding kernel
    int stream_out;  // outputs larger than L2 can keep: written to be evicted first
    uint16_t *Y, *G, *U;
    int64_t ldy, ldgu;
    int act;
    // OP_LORA: rows per tile (512, or 256: one accumulator)
    int tile_rows;
    // adapters per token tile, the tile's first slot, a slot's adapter; a slot is
    // rb pieces of `width` ranks, a stage takes 64 / width pieces; tile_cnt NULL:
    // no adapters at all
    const int32_t *tile_cnt, *tile_base, *slot_adapter;
    int rb, width;
    // OP_LORA, for repair_tile: what the tensor maps read, and the requests.  src: the
    // activations of the K' blocks in order (6:8: of the first two thirds, X; mid:
    // the rest), src_cols columns
    const uint16_t *src, *mid, *vals, *B, *V;
    const uint8_t *meta;
    int64_t src_ld, src_cols, mid_ld, mid_cols, ldb, sdb;
    const int32_t *indptr, *ids;
    int32_t requests;
    int r;
};

// __expf and __fdividef: good to 2^-21 (1 + |x|) and 2 units, far below the rounding
// to bf16 that follows (the quotient of a divisor above 2^126, |g| > 87, is 0 for
// 1e-36).  silu g / (1 + e^-g); gelu (tanh form) g / (1 + e^-2z), since (1 + tanh z) / 2 =
// 1 / (1 + e^-2z); e^x overflowing to inf gives 0; max(g, 0)^2 keeps a NaN
template <int ACT>
__device__ __forceinline__ float act_fn(float g) {
    if (ACT == NM_ACT_RELU2) return g < 0.0f ? 0.0f : g * g;
    const float z = ACT == NM_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return __fdividef(g, 1.0f + __expf(-z));
}

// g[i] = act(g[i]) u[i]
template <int N>
__device__ __forceinline__ void gate(float (&g)[N], const float (&u)[N], int act) {
    if (act == NM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = act_fn<NM_ACT_SILU>(g[i]) * u[i];
    } else if (act == NM_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = act_fn<NM_ACT_GELU>(g[i]) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = act_fn<NM_ACT_RELU2>(g[i]) * u[i];
    }
}

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ bool bf16_nan(uint16_t v) { return (v & 0x7FFFu) > 0x7F80u; }

// columns c .. c + 3 of a row of n columns, zero past its end; c a multiple of 4
__device__ __forceinline__ uint2 row4(const uint16_t *__restrict__ row, int64_t c, int64_t n) {
    if (c + 4 <= n) return __ldg(reinterpret_cast<const uint2 *>(row + c));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c + j < n) w[j >> 1] |= static_cast<uint32_t>(__ldg(row + c + j)) << (16 * (j & 1));
    return make_uint2(w[0], w[1]);
}

// A tile multiplies the B of each of its adapters by all of its tokens, with V = 0
// for the tokens of other adapters, and 0 times an infinity or a NaN in B is a NaN
// in the output of a token that has nothing to do with that adapter.  Then no
// output of that feature is finite for any token of the tile, so a thread of the
// epilogue that has seen that of all of its tokens (one bitwise AND an output; a
// few NaN tokens, as behind the last request, do not look like it) sends its CTA
// back to its outputs when all else is done: those that are NaN, and whose feature
// holds such a value in the B of an adapter that is not the token's, are computed
// again by the formula, with the token's own adapter alone.  A NaN of the token's
// own stays as it is.  A warp takes a feature, REDO of its tokens at a time (what the registers of the
// kernel allow); lane s has slot s of a K' block.
// Tokens t_lo .. t_hi - 1 of the tile, `rows` rows of this CTA; own: 256 entries of
// shared memory.  By all threads of the block.
template <int REDO>
__device__ __forceinline__ void repair_tile(const FfnArgs &p, bool mid68, int64_t nt, int64_t mt, int rows, int rank,
                                            int t_lo, int t_hi, int16_t *own) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int cnt = __ldcg(p.tile_cnt + nt), per = p.r / 8;
    const int64_t base = __ldcg(p.tile_base + nt), tok0 = nt * p.bn;
    const int nraw = static_cast<int>(mid68 ? 2 * (p.nkb / 3) : p.nkb), nkb = static_cast<int>(p.nkb);
    if (cnt == 0) return;
    __syncthreads();  // the tile before has been read
    for (int t = t_lo + threadIdx.x; t < t_hi; t += blockDim.x) {
        // the token's adapter is that of the last request that starts at or before it
        int32_t lo = 0, hi = p.requests + 1;
        while (lo < hi) {
            const int32_t q = lo + (hi - lo) / 2;
            if (__ldg(p.indptr + q) <= tok0 + t)
                lo = q + 1;
            else
                hi = q;
        }
        const int32_t q = lo - 1;
        const int32_t a = q >= 0 && q < p.requests && tok0 + t < __ldg(p.indptr + q + 1) ? __ldg(p.ids + q) : -1;
        int slot = -1;
        for (int s = 0; s < cnt; ++s)
            if (__ldcg(p.slot_adapter + base + s) == a) slot = s;
        own[t] = static_cast<int16_t>(slot);
    }
    __syncthreads();
#pragma unroll 1
    for (int rr = warp; rr < rows; rr += nwarps) {
        const int64_t row = mt * p.tile_rows + (rr >> 7) * 256 + rank * 128 + (rr & 127);
        if (row >= p.R) continue;
        int first = cnt, last = -2;  // slots with such a value at this feature; -2: not looked at yet
#pragma unroll 1
        for (int t32 = t_lo; t32 < t_hi && last != -1; t32 += 32) {
            const int t = t32 + lane < t_hi ? t32 + lane : t_lo;
            const uint32_t y = t32 + lane < t_hi ? p.Y[(tok0 + t) * p.ldy + row] & 0x7FFFu : 0x7F80u;
            const bool nan = y > 0x7F80u;
            if (__any_sync(0xffffffffu, y < 0x7F80u)) break;  // a finite output: no such B at this feature
            if (!__any_sync(0xffffffffu, nan)) continue;
            if (last == -2) {
                for (int e = lane; e < cnt * per; e += 32) {
                    const int s = e / per;
                    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(
                        p.B + __ldcg(p.slot_adapter + base + s) * p.sdb + row * p.ldb + (e - s * per) * 8));
                    bool odd = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = i == 0 ? b.x : i == 1 ? b.y : i == 2 ? b.z : b.w;
                        odd |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
                    }
                    if (odd) {
                        if (s < first) first = s;
                        if (s > last) last = s;
                    }
                }
                first = __reduce_min_sync(0xffffffffu, first);
                last = __reduce_max_sync(0xffffffffu, last < 0 ? -1 : last);
                if (last == -1) break;
            }
            uint32_t todo = __ballot_sync(0xffffffffu, nan && (first != own[t] || last != own[t]));
#pragma unroll 1
            while (todo != 0) {
                int tk[REDO], n = 0;  // up to REDO of the tokens; the last one repeated
#pragma unroll
                for (int u = 0; u < REDO; ++u) {
                    tk[u] = todo != 0 ? t32 + __ffs(todo) - 1 : tk[u > 0 ? u - 1 : 0];
                    n += todo != 0;
                    todo &= todo - 1;
                }
                float sum[REDO] = {};
                // this lane's slot: its pair of values and the nibble of their two
                // positions, in the order of packed_geom's blocks (a byte of the metadata
                // holds two slots of one of 128 rows, in tensor-memory order)
                const int r7 = rr & 127, pr = lane >> 1;
                const int byte = ((r7 & 7) + 8 * ((pr >> 1) & 1) + 16 * (r7 >> 4)) * 16 + 4 * (pr >> 2) +
                                 2 * ((r7 >> 3) & 1) + (pr & 1);
                const uint32_t *v = reinterpret_cast<const uint32_t *>(p.vals + row * nkb * 64) + lane;
                const uint8_t *e = p.meta + (row >> 7) * nkb * EBLK_BYTES + byte;
#pragma unroll 1
                for (int half = 0; half < (mid68 ? 2 : 1); ++half) {
                    const uint16_t *src = half ? p.mid : p.src;
                    const int64_t ld = half ? p.mid_ld : p.src_ld, cols = half ? p.mid_cols : p.src_cols;
#pragma unroll 2
                    for (int k = 0; k < (half ? nkb - nraw : nraw); ++k) {
                        const int64_t kb = !mid68 ? k : (half ? 3 * k + 2 : 3 * (k >> 1) + (k & 1));
                        const uint32_t pair = __ldg(v + kb * 32);
                        const uint32_t nib = static_cast<uint32_t>(__ldg(e + kb * EBLK_BYTES)) >> (4 * (lane & 1));
#pragma unroll
                        for (int u = 0; u < REDO; ++u) {
                            const uint2 x = row4(src + (tok0 + tk[u]) * ld, k * 128 + 4 * lane, cols);
                            const uint32_t x0 = nib & 2u ? x.y : x.x, x1 = nib & 8u ? x.y : x.x;
                            sum[u] = fmaf(__uint_as_float(pair << 16), __uint_as_float(nib & 1u ? x0 & 0xFFFF0000u : x0 << 16), sum[u]);
                            sum[u] = fmaf(__uint_as_float(pair & 0xFFFF0000u),
                                          __uint_as_float(nib & 4u ? x1 & 0xFFFF0000u : x1 << 16), sum[u]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < REDO; ++u) {
                    const int s = own[tk[u]];
                    if (s >= 0) {
                        const uint16_t *b = p.B + __ldcg(p.slot_adapter + base + s) * p.sdb + row * p.ldb;
                        const uint16_t *vs = p.V + ((base + s) * p.bn + tk[u]) * p.r;
#pragma unroll 1
                        for (int j = lane; j < p.r; j += 32)
                            sum[u] = fmaf(__uint_as_float(static_cast<uint32_t>(__ldcg(vs + j)) << 16),
                                          __uint_as_float(static_cast<uint32_t>(__ldg(b + j)) << 16), sum[u]);
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
                    if (lane == 0 && u < n) p.Y[(tok0 + tk[u]) * p.ldy + row] = static_cast<uint16_t>(pack_bf16x2(sum[u], 0.0f));
                }
            }
        }
    }
}

// A cluster of `split` pairs computes a tile: pair j takes the j-th part of its
// K' blocks (and of its adapters' blocks).  With split > 1 every CTA leaves the
// fp32 sums of its 128 + 128 rows in shared memory, and pair j adds the parts
// of all pairs for its share of the tokens, reading them through distributed
// shared memory in the pairs' order (so results do not depend on timing), and
// finishes those tokens.  Nothing goes through global memory and nothing
// outlives the launch.
// (SPLIT is a template parameter because the exchange's registers would spill
// in the plain epilogue, which held up the next tile: 850 -> 1390 us for the
// gate and up projections of 8192 tokens.)
template <int MODE, int OP, bool SPLIT>
__global__ void __launch_bounds__(ffn_threads(SPLIT), 1)
    k_ffn(const __grid_constant__ FfnMaps tm, const __grid_constant__ FfnArgs p) {
    using C = FfnCfg;
    constexpr int EPI_WARPS = ffn_epi_warps(SPLIT);
    const int S = p.stages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::SMEM_DATA);
    uint64_t *full = bars, *empty = bars + C::MAX_STAGES;
    uint64_t *acc_full = bars + 2 * C::MAX_STAGES, *acc_empty = acc_full + 1;
    uint64_t *sum_ready = acc_full + 2, *sum_free = acc_full + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank(), rank = crank & 1u, leader = crank & ~1u;
    const int split = SPLIT ? p.split : 1, part = SPLIT ? static_cast<int>(crank >> 1) : 0;
    const int64_t cluster = blockIdx.x / (2 * split), nclusters = gridDim.x / (2 * split);
    const int bn = p.bn, bh = bn >> 1;
    const int b_atom = bh * 128;
    const int64_t nkb = p.nkb, T = p.T;
    const int64_t Rpad = (p.R + 255) / 256 * 256;
    const int tile_rows = OP == OP_GLU ? 256 : p.tile_rows;
    // rows per band of the tile order: OP_GLU's rows have two weights each (8192
    // tokens, 11008 x 4096: 492 MB read with 2816 rows and streamed outputs, 631
    // with 4096 and plain stores, 681 us against 692 at the power cap)
    constexpr int band_rows = OP == OP_GLU ? 2816 : static_cast<int>(BAND_ROWS);
    const int64_t n_t = (T + bn - 1) / bn;
    const int64_t n_m = (Rpad + tile_rows - 1) / tile_rows;
    const int64_t ntiles = n_t * n_m;
    const int64_t kb0 = nkb * part / split, kb1 = nkb * (part + 1) / split;  // this pair's K' blocks
    auto stage = [&](int s) { return smem + s * p.stage_bytes; };
    // accumulator 1 in use: rows 256.. of the tile exist
    auto second = [&](int64_t mt) { return OP == OP_GLU || (tile_rows == 512 && mt * 512 + 256 < Rpad); };
    // this pair's pieces of the adapters of token tile nt
    auto adapter_pieces = [&](int64_t nt, int &x0, int &x1) {
        const int per = 64 / p.width, n = __ldcg(p.tile_cnt + nt) * p.rb, stages = (n + per - 1) / per;
        x0 = stages * part / split * per;
        x1 = stages * (part + 1) / split * per;
        if (x1 > n) x1 = n;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * EPI_WARPS);
        mbar_init(sum_ready, split * EPI_WARPS);
        mbar_init(sum_free, split * EPI_WARPS);
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
    // the stream's next kernel may set itself up on SMs that this one leaves
    grid_dep_launch();
    // OP_LORA: a feature of this thread had no finite sum for any of its tokens
    constexpr uint32_t EXPONENT = 0x7F800000u;
    bool odd = false;

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        // (the warp in step, one lane issues: as below)
        const bool lead = elect_one() != 0u;
        const uint32_t st0 = smem_u32(smem), full0 = mapa_shared(full, leader);
        const uint32_t b_bytes = 2u * static_cast<uint32_t>(b_atom);
        const CUtensorMap *ta1 = OP == OP_GLU ? &tm.a1 : &tm.a0, *te1 = OP == OP_GLU ? &tm.e1 : &tm.e0;
        const int nraw = 2 * static_cast<int>(nkb / 3);
        int s = 0;
        uint32_t ph = 0;
        int64_t it = 0;
        bool ok = true, dep_done = p.early == 0;
        for (int64_t tile = cluster; tile < ntiles && ok; tile += nclusters) {
            int64_t nt, mt;
            tile_coords(tile, n_t, n_m, band_rows / tile_rows, nt, mt);
            const bool has1 = second(mt);
            const int32_t arow = static_cast<int32_t>(mt * tile_rows + rank * 128);
            const int32_t arow1 = OP == OP_GLU ? arow : arow + 256;
            const int32_t brow = static_cast<int32_t>(nt * bn + rank * bh);
            const int32_t e0 = static_cast<int32_t>((arow >> 7) * nkb * 8), e1 = static_cast<int32_t>((arow1 >> 7) * nkb * 8);
            const uint32_t tx = 2u * ((has1 ? 2u : 1u) * (C::A_BYTES + EBLK_BYTES) + b_bytes);
            for (int v = static_cast<int>(kb0); v < static_cast<int>(kb1); ++v, ++it) {
                // 6:8: tiles of X first, the gathered middle windows last (visit68)
                const bool mid = MODE == PMODE_SP68T && v >= nraw;
                const int kb = MODE != PMODE_SP68T ? v : (mid ? 3 * (v - nraw) + 2 : 3 * (v >> 1) + (v & 1));
                const int xc = MODE != PMODE_SP68T ? v * 128 : (mid ? v - nraw : v) * 128;
                if (mid && !dep_done) {  // written by the kernel just before
                    grid_dep_wait();
                    dep_done = true;
                }
                if (it >= S && !mbar_wait_warp(&empty[s], ph ^ 1u)) { ok = false; break; }
                if (lead) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], tx);
                    const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                    const uint32_t st = st0 + static_cast<uint32_t>(s) * p.stage_bytes;
                    tma_load_2d_pair_at(st + C::OFF_A0, &tm.a0, bar, kb * 64, arow);
                    if (has1) tma_load_2d_pair_at(st + C::OFF_A1, ta1, bar, kb * 64, arow1);
                    const CUtensorMap *tb = mid ? &tm.b2 : &tm.b;
                    tma_load_2d_pair_at(st + C::OFF_B, tb, bar, xc, brow);
                    tma_load_2d_pair_at(st + C::OFF_B + b_atom, tb, bar, xc + 64, brow);
                    tma_load_2d_pair_at(st + C::OFF_E0, &tm.e0, bar, 0, e0 + kb * 8);
                    if (has1) tma_load_2d_pair_at(st + C::OFF_E1, te1, bar, 0, e1 + kb * 8);
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            if (OP == OP_LORA && ok && p.tile_cnt != nullptr) {
                if (!dep_done) {
                    grid_dep_wait();
                    dep_done = true;
                }
                int x0, x1;
                adapter_pieces(nt, x0, x1);
                const int32_t slot0 = __ldcg(p.tile_base + nt);
                const int per = 64 / p.width, piece = p.width * 2;  // bytes per row of a piece
                int32_t a_next = x0 < x1 ? __ldcg(p.slot_adapter + slot0 + x0 / p.rb) : 0;
                for (int x = x0; x < x1; x += per, ++it) {
                    if (it >= S && !mbar_wait_warp(&empty[s], ph ^ 1u)) { ok = false; break; }
                    const int n = x1 - x < per ? x1 - x : per;
                    const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                    const uint32_t st = st0 + static_cast<uint32_t>(s) * p.stage_bytes;
                    if (lead && rank == 0)
                        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * n * piece * ((has1 ? 2 : 1) * BM + bh)));
                    for (int k = 0; k < n; ++k) {
                        const int32_t a = a_next, slot = slot0 + (x + k) / p.rb, rk = ((x + k) % p.rb) * 64;
                        if (x + k + 1 < x1) a_next = __ldcg(p.slot_adapter + slot0 + (x + k + 1) / p.rb);
                        if (lead) {
                            tma_load_3d_pair_at(st + C::OFF_A0 + k * piece * BM, &tm.lb, bar, rk, arow, a);
                            if (has1)
                                tma_load_3d_pair_at(st + C::OFF_A1 + k * piece * BM, &tm.lb, bar, rk, arow + 256, a);
                            tma_load_3d_pair_at(st + C::OFF_B + k * piece * bh, &tm.lv, bar, rk,
                                                static_cast<int32_t>(rank) * bh, slot);
                        }
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
        }
        if (!ok && rank == 0) {  // let copies already issued land before exiting
            for (int64_t j = (it > S ? it - S : 0); j < it; ++j)
                mbar_wait_warp(&full[j % S], static_cast<uint32_t>((j / S) & 1));
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        // The whole warp runs the loop and one elected lane issues, on operand
        // descriptors that differ from those of stage 0 by one addition: with
        // N = 16 the tensor core waits for the issuing thread, not for data.
        if (rank == 0) {
            const bool lead = elect_one() != 0u;
            const uint32_t idesc = make_idesc_bf16(256, bn, true, 0);
            const uint16_t both = static_cast<uint16_t>(3u << leader);
            const uint32_t st0 = smem_u32(smem);
            const uint64_t a0d = make_sdesc(st0 + C::OFF_A0, 16, 1024, 2), a1d = make_sdesc(st0 + C::OFF_A1, 16, 1024, 2);
            const uint64_t b0d = make_sdesc(st0 + C::OFF_B, 16, 1024, 2);
            const uint64_t b1d = make_sdesc(st0 + C::OFF_B + b_atom, 16, 1024, 2);
            const uint64_t e0d = make_sdesc(st0 + C::OFF_E0, 2048, 128, 0), e1d = make_sdesc(st0 + C::OFF_E1, 2048, 128, 0);
            const uint32_t step = static_cast<uint32_t>(p.stage_bytes) >> 4;
            const uint32_t d0 = tmem_base + C::TMEM_D0, d1 = tmem_base + C::TMEM_D1;
            const uint32_t te0 = tmem_base + C::TMEM_E0, te1 = tmem_base + C::TMEM_E1;
            const int nblocks = static_cast<int>(kb1 - kb0);
            int s = 0;
            uint32_t ph = 0;
            int64_t ti = 0;
            bool ok = true, dep_done = p.early == 0;
            for (int64_t tile = cluster; tile < ntiles && ok; tile += nclusters, ++ti) {
                int64_t nt, mt;
                tile_coords(tile, n_t, n_m, band_rows / tile_rows, nt, mt);
                const bool has1 = second(mt);
                if (ti >= 1 && !mbar_wait_cluster_warp(acc_empty, static_cast<uint32_t>((ti - 1) & 1))) break;
                tc_fence_after();
                for (int kb = 0; kb < nblocks; ++kb) {
                    if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = static_cast<uint64_t>(static_cast<uint32_t>(s) * step);
                    if (lead) {
                        tmem_cp_128x128b_pair(te0, e0d + so);
                        if (has1) tmem_cp_128x128b_pair(te1, e1d + so);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t bd = (j >> 1 ? b1d : b0d) + so + (j & 1) * 4;
                            const uint32_t acc = j > 0 || kb > 0 ? 1u : 0u;
                            const uint32_t id = idesc | static_cast<uint32_t>(j & 1);
                            mma_sp_bf16_pair(d0, a0d + so + j * 2, bd, te0 + (j & ~1), id, acc);
                            if (has1) mma_sp_bf16_pair(d1, a1d + so + j * 2, bd, te1 + (j & ~1), id, acc);
                        }
                        mma_commit_pair_mask(&empty[s], both);
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (OP == OP_LORA && ok && p.tile_cnt != nullptr) {
                    if (!dep_done) {
                        grid_dep_wait();
                        dep_done = true;
                    }
                    int x0, x1;
                    adapter_pieces(nt, x0, x1);
                    const uint32_t idesc_dense = make_idesc_bf16(256, bn, false, 0);
                    const int per = 64 / p.width, piece = p.width * 2, steps = p.width / 16;
                    const uint32_t layout = p.width == 16 ? 6 : (p.width == 32 ? 4 : 2);
                    for (int x = x0; x < x1; x += per) {  // on top of this pair's K' blocks
                        if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
                        tc_fence_after();
                        if (lead) {
                            const uint32_t st = st0 + static_cast<uint32_t>(s) * p.stage_bytes;
                            const int n = (x1 - x < per ? x1 - x : per) * steps;
                            for (int k = 0; k < n; ++k) {  // k-steps of 16 ranks
                                const int pc = k / steps, in = (k % steps) * 32;
                                const uint64_t bd = make_sdesc(st + C::OFF_B + pc * piece * bh + in, 16, 8 * piece, layout);
                                const uint32_t at = st + pc * piece * BM + in;
                                mma_bf16_pair(d0, make_sdesc(at + C::OFF_A0, 16, 8 * piece, layout), bd, idesc_dense, 1u);
                                if (has1)
                                    mma_bf16_pair(d1, make_sdesc(at + C::OFF_A1, 16, 8 * piece, layout), bd, idesc_dense,
                                                  1u);
                            }
                            mma_commit_pair_mask(&empty[s], both);
                        }
                        __syncwarp();
                        if (++s == S) { s = 0; ph ^= 1u; }
                    }
                }
                if (ok && lead) mma_commit_pair_mask(acc_full, both);
                __syncwarp();
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------- epilogue
        // a warp = lane quarter q x a part of the tokens, and of both accumulators
        // where one warp needs both (OP_GLU), or of one of them: then half of the
        // parts are of each accumulator, if there are two
        const int q = warp & 3, grp = (warp - 4) >> 2;
        constexpr int NACC = OP == OP_GLU ? 2 : 1, GRPS = EPI_WARPS / 4;
        const bool by_tokens = OP == OP_GLU || tile_rows == 256;
        const uint32_t acc_empty_cl = mapa_shared(acc_empty, leader);
        int64_t ti = 0;
        for (int64_t tile = cluster; tile < ntiles; tile += nclusters, ++ti) {
            int64_t nt, mt;
            tile_coords(tile, n_t, n_m, band_rows / tile_rows, nt, mt);
            if (!mbar_wait_warp(acc_full, static_cast<uint32_t>(ti & 1))) break;
            tc_fence_after();
            const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
            const int acc0 = by_tokens ? 0 : grp & 1;  // the (first) accumulator of this warp
            const int tp = by_tokens ? grp : grp >> 1, ntp = by_tokens ? GRPS : GRPS / 2;  // its part of the tokens
            const uint32_t tacc[2] = {tq + (acc0 ? C::TMEM_D1 : C::TMEM_D0), tq + C::TMEM_D1};
            const int64_t tok0 = nt * bn;
            const int nv = static_cast<int>(T - tok0 < bn ? T - tok0 : bn);  // real tokens of the tile
            const int nch = (nv + 15) / 16;                                  // their chunks of 16
            const bool active = acc0 == 0 || second(mt);
            const int per = (bn / 16 + ntp - 1) / ntp, c_lo = tp * per;
            const int c_hi = !active ? c_lo : (c_lo + per < nch ? c_lo + per : nch);
            // 16 tokens of the accumulators
            auto load_chunk = [&](int c, float (&f)[NACC][16]) {
                uint32_t v[NACC][16];
#pragma unroll
                for (int a = 0; a < NACC; ++a) tmem_ld_32x32b_x16(tacc[a] + c * 16, v[a]);
                tmem_ld_wait();
#pragma unroll
                for (int a = 0; a < NACC; ++a)
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[a][j] = __uint_as_float(v[a][j]);
            };
            const int64_t row = mt * tile_rows + acc0 * 256 + rank * 128 + q * 32 + lane;
            const bool rok = row < p.R;
            if constexpr (SPLIT) {
                // this CTA's sums in its shared memory: [accumulator][4 tokens][row][token], fp32
                float4 *mine = reinterpret_cast<float4 *>(smem + p.sum_off) + acc0 * (bn / 4) * 128 + q * 32 + lane;
                if (ti >= 1 && !mbar_wait_cluster_warp(sum_free, static_cast<uint32_t>((ti - 1) & 1)))
                    break;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    float f[NACC][16];
                    load_chunk(c, f);
#pragma unroll
                    for (int a = 0; a < NACC; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mine[(a * (bn / 4) + c * 4 + j) * 128] =
                                make_float4(f[a][4 * j], f[a][4 * j + 1], f[a][4 * j + 2], f[a][4 * j + 3]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty_cl);
                if (lane < split) mbar_arrive_cluster(mapa_shared(sum_ready, 2 * lane + rank));
                if (!mbar_wait_cluster_warp(sum_ready, static_cast<uint32_t>(ti & 1))) break;
                // this pair's share of the tokens, four at a time; all the parts of
                // GROUPS x 4 tokens are in flight before the first is used
                constexpr int GROUPS = OP == OP_GLU ? 1 : 2;
                uint32_t all = ~0u;  // AND of the sums' bits
                const int ng = (nv + 3) / 4, g1 = active ? ng * (part + 1) / split : 0;
                const int gstep = ntp;
                const uint32_t off = smem_u32(mine);
                uint32_t from[C::MAX_SPLIT];
#pragma unroll
                for (int i = 0; i < C::MAX_SPLIT; ++i)
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(from[i]) : "r"(off), "r"(2 * (i < split ? i : part) + rank));
#pragma unroll 1
                for (int g = ng * part / split + tp; g < g1; g += gstep * GROUPS) {
                    float4 pv[C::MAX_SPLIT][GROUPS][NACC];
#pragma unroll
                    for (int i = 0; i < C::MAX_SPLIT; ++i)
                        if (i < split) {
#pragma unroll
                            for (int u = 0; u < GROUPS; ++u)
#pragma unroll
                                for (int a = 0; a < NACC; ++a) {
                                    const int gg = g + u * gstep < g1 ? g + u * gstep : g;
                                    pv[i][u][a] = ld_dsmem_f32x4(from[i] + static_cast<uint32_t>((a * (bn / 4) + gg) * 2048));
                                }
                        }
#pragma unroll
                    for (int u = 0; u < GROUPS; ++u) {
                        if (g + u * gstep >= g1) break;
                        float f[NACC][4];
#pragma unroll
                        for (int a = 0; a < NACC; ++a) {
                            f[a][0] = pv[0][u][a].x;
                            f[a][1] = pv[0][u][a].y;
                            f[a][2] = pv[0][u][a].z;
                            f[a][3] = pv[0][u][a].w;
#pragma unroll
                            for (int i = 1; i < C::MAX_SPLIT; ++i)
                                if (i < split) {
                                    f[a][0] += pv[i][u][a].x;
                                    f[a][1] += pv[i][u][a].y;
                                    f[a][2] += pv[i][u][a].z;
                                    f[a][3] += pv[i][u][a].w;
                                }
                        }
                        const int t = (g + u * gstep) * 4;
                        if (OP == OP_GLU && p.G != nullptr && rok) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (t + j < nv) {
                                    const int64_t at = (tok0 + t + j) * p.ldgu + row;
                                    p.G[at] = static_cast<uint16_t>(pack_bf16x2(f[0][j], 0.0f));
                                    p.U[at] = static_cast<uint16_t>(pack_bf16x2(f[NACC - 1][j], 0.0f));
                                }
                        }
                        if (OP == OP_GLU) gate(f[0], f[NACC - 1], p.act);
                        if (OP == OP_LORA)
#pragma unroll
                            for (int j = 0; j < 4; ++j) all &= __float_as_uint(f[0][j]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (t + j < nv && rok)
                                p.Y[(tok0 + t + j) * p.ldy + row] = static_cast<uint16_t>(pack_bf16x2(f[0][j], 0.0f));
                    }
                }
                __syncwarp();
                if (lane < split) mbar_arrive_cluster(mapa_shared(sum_free, 2 * lane + rank));
                odd |= ng * part / split + tp < g1 && (all & EXPONENT) == EXPONENT;
            }
            if constexpr (!SPLIT) {
                // 32 rows x 16 tokens at a time, as 8 x 8 blocks: out of tensor memory in
                // the layout of a matrix fragment, transposed by stmatrix on the way to
                // the warp's 1 KB of shared memory ([token][32 rows], 16-byte pieces
                // swizzled against bank conflicts), and out as 64 bytes a token.  (Two-byte
                // stores straight from registers, a row to each lane, took 14 us a tile
                // where the products take 15 and this takes 5, for 8192 tokens through
                // 11008 x 4096 projections with G and U kept; with eight warps instead of
                // sixteen the kernel took 524 us instead of 494 at 1965 MHz.)  The
                // accumulators are released once the last chunk is in registers.
                const int64_t row0 = mt * tile_rows + acc0 * 256 + rank * 128 + q * 32;
                const uint32_t buf = smem_u32(smem) + C::OFF_OUT + static_cast<uint32_t>(warp - 4) * 1024u;
                const int bi = lane >> 3, st_tok = (lane & 7) + 8 * (bi >> 1);
                uint32_t st_at[2];  // where this lane's row of the blocks of lanes 0..15, 16..31 goes
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    st_at[u] = static_cast<uint32_t>(st_tok * 64 + ((((bi & 1) + 2 * u) ^ ((st_tok >> 1) & 3)) << 4));
                auto emit = [&](uint16_t *dst, int64_t ld, int c, const float (&f)[16]) {
                    __syncwarp();  // the piece before has been read
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        stmatrix_x4_trans(buf + st_at[u], pack_bf16x2(f[8 * u], f[8 * u + 1]),
                                          pack_bf16x2(f[8 * u + 2], f[8 * u + 3]), pack_bf16x2(f[8 * u + 4], f[8 * u + 5]),
                                          pack_bf16x2(f[8 * u + 6], f[8 * u + 7]));
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int tok = (lane >> 2) + 8 * u, piece = lane & 3;
                        uint4 v;
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(buf + static_cast<uint32_t>(tok * 64 + ((piece ^ ((tok >> 1) & 3)) << 4))));
                        const int64_t r = row0 + piece * 8;
                        if (c * 16 + tok < nv && r < p.R) {
                            uint16_t *o = dst + (tok0 + c * 16 + tok) * ld + r;
                            if (r + 8 <= p.R) {
                                if (p.stream_out)
                                    __stcs(reinterpret_cast<uint4 *>(o), v);
                                else
                                    *reinterpret_cast<uint4 *>(o) = v;
                            } else {
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (r + e < p.R) o[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                            }
                        }
                    }
                };
                uint32_t all[4] = {~0u, ~0u, ~0u, ~0u};  // ANDs of the bits of this thread's four rows
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    uint32_t v[NACC][2][8];
#pragma unroll
                    for (int a = 0; a < NACC; ++a)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            tmem_ld_16x256b_x2(tacc[a] + (static_cast<uint32_t>(u * 16) << 16) + c * 16, v[a][u]);
                    tmem_ld_wait();
                    if (c + 1 == c_hi) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(acc_empty_cl);
                    }
                    float f[NACC][16];
#pragma unroll
                    for (int a = 0; a < NACC; ++a)
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[a][j] = __uint_as_float(v[a][j >> 3][j & 7]);
                    if (OP == OP_GLU) {
                        if (p.G != nullptr) {
                            emit(p.G, p.ldgu, c, f[0]);
                            emit(p.U, p.ldgu, c, f[NACC - 1]);
                        }
                        gate(f[0], f[NACC - 1], p.act);
                    }
                    if (OP == OP_LORA)
#pragma unroll
                        for (int j = 0; j < 16; ++j) all[2 * (j >> 3) + ((j >> 1) & 1)] &= __float_as_uint(f[0][j]);
                    emit(p.Y, p.ldy, c, f[0]);
                }
                if (OP == OP_LORA)
#pragma unroll
                    for (int i = 0; i < 4; ++i) odd |= c_lo < c_hi && (all[i] & EXPONENT) == EXPONENT;
                if (c_lo >= c_hi) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(acc_empty_cl);
                }
            }
        }
    }
    tc_fence_before();
    const bool redo = OP == OP_LORA ? __syncthreads_or(odd) && p.tile_cnt != nullptr : (__syncthreads(), false);
    cluster_sync_all();  // also: no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
    if (OP == OP_LORA && redo) {
        grid_dep_wait();
        for (int64_t tile = cluster; tile < ntiles; tile += nclusters) {
            int64_t nt, mt;
            tile_coords(tile, n_t, n_m, band_rows / tile_rows, nt, mt);
            const int nv = static_cast<int>(T - nt * bn < bn ? T - nt * bn : bn), ng = (nv + 3) / 4;
            const int t_lo = 4 * (ng * part / split), t_hi = 4 * (ng * (part + 1) / split);  // what this pair stored
            repair_tile<SPLIT ? 8 : 4>(p, MODE == PMODE_SP68T, nt, mt, second(mt) ? 256 : 128, static_cast<int>(rank), t_lo,
                        t_hi < nv ? t_hi : nv, reinterpret_cast<int16_t *>(smem));
        }
    }
}

// ---------------------------------------------------------------------------
// adapters: which of them a token tile holds, and V = scale X A^T
//
// The requests' tokens are consecutive: request i has tokens [indptr[i],
// indptr[i+1]) and adapter ids[i] (-1: none); tokens behind the last request
// have none.  A slot is one (token tile, adapter that occurs in it); its V is
// [bn x r], zero in the rows of other tokens.  Tile i's slots start at i * cap
// (few adapters) or at i + (the requests that end before it): along the batch
// each tile or request border starts at most one new pair, so that numbering
// leaves every tile room and needs requests + tiles slots in all.
//
// k_lora_shrink, one (tile, slot, rank block of <= 64) per cluster of up to
// SHRINK_PARTS blocks that split K (grid: x over parts and tiles, of which there
// may be more than 65535, y over slots and rank blocks).  Every block first works
// out its tile's slots (one pass over the list, a hash of the adapters; about a
// microsecond, less than a kernel of its own would take to start), then, for its
// slots, lists the slot's tokens and multiplies 32 of them at a time with mma.sync:
// a slot of up to 32 tokens has its K split over the warps too, a larger one has
// groups of 32 tokens side by side in the warps.  A thread's 16-byte loads of X
// and A cover the same eight columns, which the two k-steps of a block of 32
// columns take in a permuted order (the same one for both operands), so neither
// passes through shared memory.  The warps' and then the blocks' fp32 sums are
// added in a fixed order, through shared and distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int SHRINK_GROUP = 32, SHRINK_RANKS = 64, SHRINK_WARPS = 4, SHRINK_THREADS = 32 * SHRINK_WARPS;
constexpr int SHRINK_PARTS = 8;      // blocks of a cluster, at most
constexpr int SHRINK_HASH = 512;     // more than twice the tokens of a tile

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

struct ShrinkArgs {
    const uint16_t *X, *A;
    const float *scale;
    const int32_t *indptr, *ids;
    int64_t T, K, ldx, lda, sda, nslots;
    int32_t requests, adapters;
    int r, rb, bn, cap, by_cap;
    int first;  // the call's first kernel (else it follows the staging kernel)
    int parts;  // blocks of a cluster
    int32_t *tile_cnt, *tile_base, *slot_adapter;
    uint16_t *V;
};

struct TilePlan {
    int32_t start[256];            // per token of the tile: the request that starts there, -1: none
    int32_t slot[256];             // the token's slot, -1: none
    int32_t adapter[256];          // of a slot
    int32_t keys[SHRINK_HASH], first[SHRINK_HASH];
    int32_t warp_max[8], warp_cnt[8];
    int32_t list[256];             // the tokens of the slot at hand
    int32_t before, cnt, base;
};

// Fills in plan.slot, .adapter, .cnt and .base of token tile `tile`; true if the
// list is out of order or names an unknown adapter (then what it asks for
// beyond the slots there are is left out).  The blocks of a cluster each make the
// plan of their tile and meet at as many barriers as it has slots and tokens, so it
// depends on the list alone: of requests that a wrong list starts on one token the
// last in the list counts, not the last to be written.
__device__ bool plan_tile(const ShrinkArgs &p, int64_t tile, TilePlan &plan) {
    constexpr int NT = SHRINK_THREADS;
    const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
    const int64_t t0 = tile * p.bn, t1 = t0 + p.bn;
    bool bad = false;
    for (int k = i; k < 256; k += NT) plan.start[k] = -1;
    for (int k = i; k < SHRINK_HASH; k += NT) {
        plan.keys[k] = -1;
        plan.first[k] = 256;
    }
    if (i == 0) plan.before = 0;
    __syncthreads();
    int before = 0;
    for (int32_t q = i; q < p.requests; q += NT) {
        const int32_t lo = __ldg(p.indptr + q), hi = __ldg(p.indptr + q + 1), a = __ldg(p.ids + q);
        const bool odd = lo < 0 || lo > hi || hi > p.T || a < -1 || a >= p.adapters;
        bad |= odd;
        before += hi <= t0;
        if (!odd && lo < hi && hi > t0 && lo < t1) {
            const int at = lo > t0 ? static_cast<int>(lo - t0) : 0;
            atomicMax(&plan.start[at], q);
        }
    }
    if (before) atomicAdd(&plan.before, before);
    __syncthreads();
    // the last start at or before each token (two tokens a thread: i and i + 128)
    int mine[2], a[2], h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        int m = plan.start[i + u * NT] >= 0 ? i + u * NT : -1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, m, d);
            if (lane >= d && o > m) m = o;
        }
        mine[u] = m;
        if (lane == 31) plan.warp_max[u * SHRINK_WARPS + warp] = m;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int tok = i + u * NT;
        for (int w = 0; w < u * SHRINK_WARPS + warp; ++w)
            if (plan.warp_max[w] > mine[u]) mine[u] = plan.warp_max[w];
        a[u] = -1;
        h[u] = 0;
        if (tok < p.bn && mine[u] >= 0) {
            const int32_t q = plan.start[mine[u]];
            if (t0 + tok < __ldg(p.indptr + q + 1)) a[u] = __ldg(p.ids + q);
        }
        if (a[u] >= 0) {
            h[u] = static_cast<int>((static_cast<uint32_t>(a[u]) * 2654435761u) >> 23);
            while (true) {  // at most 240 keys in 512 places
                const int32_t old = atomicCAS(&plan.keys[h[u]], -1, a[u]);
                if (old == -1 || old == a[u]) break;
                h[u] = (h[u] + 1) & (SHRINK_HASH - 1);
            }
            atomicMin(&plan.first[h[u]], tok);
        }
    }
    __syncthreads();
    uint32_t b[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        b[u] = __ballot_sync(0xffffffffu, a[u] >= 0 && plan.first[h[u]] == i + u * NT);
        if (lane == 0) plan.warp_cnt[u * SHRINK_WARPS + warp] = __popc(b[u]);
    }
    __syncthreads();
    const int64_t base = p.by_cap ? tile * p.cap : tile + plan.before;
    int64_t room = p.nslots - base;
    if (room > p.cap) room = p.cap;
    if (room < 0) room = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if ((b[u] >> lane) & 1u) {  // the first token of its adapter: slots in the order of first tokens
            int at = __popc(b[u] & ((1u << lane) - 1u));
            for (int w = 0; w < u * SHRINK_WARPS + warp; ++w) at += plan.warp_cnt[w];
            const bool fits = at < room;
            bad |= !fits;
            plan.keys[h[u]] = fits ? at : -1;  // every probe is over: the key's place now holds the slot
            if (fits) plan.adapter[at] = a[u];
        }
    }
    if (i == 0) {
        int cnt = 0;
        for (int w = 0; w < 2 * SHRINK_WARPS; ++w) cnt += plan.warp_cnt[w];
        plan.cnt = cnt < room ? cnt : static_cast<int>(room);
        plan.base = base < p.nslots ? static_cast<int32_t>(base) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) plan.slot[i + u * NT] = a[u] >= 0 ? plan.keys[h[u]] : -1;
    __syncthreads();
    return bad;
}

// NN: 8-rank columns of a block (a rank block has nr / 8 <= NN of them)
template <int NN>
__global__ void __launch_bounds__(SHRINK_THREADS)
    k_lora_shrink(const __grid_constant__ ShrinkArgs p) {
    constexpr int NR = NN * 8;
    __shared__ TilePlan plan;
    __shared__ __align__(16) float red[SHRINK_WARPS][SHRINK_GROUP][NR];
    // as the call's first kernel it waits for the stream's earlier work before it
    // lets the product start, whose early loads rely on that
    if (p.first) grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
    const int part = static_cast<int>(cluster_ctarank()), parts = p.parts;
    const int64_t tile = blockIdx.x / static_cast<unsigned>(parts), t0 = tile * p.bn;
    const int rk = static_cast<int>(blockIdx.y % p.rb) * SHRINK_RANKS;
    const int lanes_z = gridDim.y / p.rb;
    const int nr = p.r - rk < NR ? p.r - rk : NR, nn = nr / 8;
    const bool bad = plan_tile(p, tile, plan);
    if (bad) raise_error(ERRBIT_DEVICE);
    const int cnt = plan.cnt;
    const int64_t base = plan.base;
    if (part == 0 && blockIdx.y == 0) {  // what the product reads
        for (int k = threadIdx.x; k < cnt; k += SHRINK_THREADS) p.slot_adapter[base + k] = plan.adapter[k];
        if (threadIdx.x == 0) {
            p.tile_cnt[tile] = cnt;
            p.tile_base[tile] = static_cast<int32_t>(base);
        }
    }
    for (int j = blockIdx.y / p.rb; j < cnt; j += lanes_z) {  // the same in every block of the cluster
        uint16_t *vslot = p.V + (base + j) * p.bn * static_cast<int64_t>(p.r) + rk;
        // the slot's tokens in ascending order; the other rows are zero
        uint32_t b[2];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            b[u] = __ballot_sync(0xffffffffu, plan.slot[threadIdx.x + u * SHRINK_THREADS] == j);
            if (lane == 0) plan.warp_cnt[u * SHRINK_WARPS + warp] = __popc(b[u]);
        }
        __syncthreads();
        int n = 0;
        for (int w = 0; w < 2 * SHRINK_WARPS; ++w) n += plan.warp_cnt[w];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if ((b[u] >> lane) & 1u) {
                int at = __popc(b[u] & ((1u << lane) - 1u));
                for (int w = 0; w < u * SHRINK_WARPS + warp; ++w) at += plan.warp_cnt[w];
                plan.list[at] = threadIdx.x + u * SHRINK_THREADS;
            }
        for (int e = part * SHRINK_THREADS + threadIdx.x; e < p.bn * nn; e += parts * SHRINK_THREADS) {
            const int tok = e / nn;
            if (plan.slot[tok] != j)
                *reinterpret_cast<uint4 *>(vslot + static_cast<int64_t>(tok) * p.r + (e - tok * nn) * 8) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        const int32_t ad = plan.adapter[j];
        const uint16_t *arow = p.A + ad * p.sda + static_cast<int64_t>(rk + g) * p.lda;
        const float sc = __ldg(p.scale + ad);
        const bool one = n <= SHRINK_GROUP;  // one group: the warps split K as well
        for (int first = 0; first < n; first += SHRINK_WARPS * SHRINK_GROUP) {
            const int g0 = one ? 0 : first + warp * SHRINK_GROUP;   // this warp's group of the list
            float acc[2][NN][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int c = 0; c < NN; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][c][e] = 0.0f;
            // rows past the list's end repeat its first token, columns past nr the
            // first rank: their sums are not read
            const uint16_t *xr[2][2], *ar[NN];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int at = g0 + mt * 16 + u * 8 + g;
                    xr[mt][u] = p.X + (t0 + plan.list[at < n ? at : 0]) * p.ldx + tg * 8;
                }
#pragma unroll
            for (int c = 0; c < NN; ++c) ar[c] = arow + static_cast<int64_t>(c < nn ? c * 8 : 0) * p.lda + tg * 8;
            const bool hi = g0 + 16 < n;  // more than 16 tokens: the second m-tile
            const int stride = 32 * parts * (one ? SHRINK_WARPS : 1);
            const int K = static_cast<int>(p.K), whole = K & ~31;
            int k = 32 * (one ? part * SHRINK_WARPS + warp : part);
            if (g0 >= n) k = K;
            auto mma = [&](const uint4 (&x)[2][2], const uint4 (&a)[NN]) {
#pragma unroll
                for (int c = 0; c < NN; ++c) {
                    mma_16816(acc[0][c], x[0][0].x, x[0][1].x, x[0][0].y, x[0][1].y, a[c].x, a[c].y);
                    mma_16816(acc[0][c], x[0][0].z, x[0][1].z, x[0][0].w, x[0][1].w, a[c].z, a[c].w);
                    if (hi) {
                        mma_16816(acc[1][c], x[1][0].x, x[1][1].x, x[1][0].y, x[1][1].y, a[c].x, a[c].y);
                        mma_16816(acc[1][c], x[1][0].z, x[1][1].z, x[1][0].w, x[1][1].w, a[c].z, a[c].w);
                    }
                }
            };
#pragma unroll NN <= 2 ? 4 : 2
            for (; k < whole; k += stride) {
                uint4 x[2][2], a[NN];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    x[0][u] = __ldg(reinterpret_cast<const uint4 *>(xr[0][u] + k));
                    x[1][u] = hi ? __ldg(reinterpret_cast<const uint4 *>(xr[1][u] + k)) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int c = 0; c < NN; ++c) a[c] = __ldg(reinterpret_cast<const uint4 *>(ar[c] + k));
                mma(x, a);
            }
            if (k == whole && k < K) {  // the last, ragged block of columns: one warp's
                uint4 x[2][2], a[NN];
                const int64_t left = K - k - tg * 8;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) x[mt][u] = row8(xr[mt][u] + k, 0, left);
#pragma unroll
                for (int c = 0; c < NN; ++c) a[c] = row8(ar[c] + k, 0, left);
                mma(x, a);
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int c = 0; c < NN; ++c) {
                    if (c >= nn) break;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        *reinterpret_cast<float2 *>(&red[warp][mt * 16 + u * 8 + g][c * 8 + 2 * tg]) =
                            make_float2(acc[mt][c][2 * u], acc[mt][c][2 * u + 1]);
                }
            const int groups = one ? 1 : SHRINK_WARPS;
            if (one) {
                __syncthreads();
                for (int e = threadIdx.x; e < n * nr; e += SHRINK_THREADS) {
                    const int tok = e / nr, c = e - tok * nr;
                    float s = red[0][tok][c];
#pragma unroll
                    for (int w = 1; w < SHRINK_WARPS; ++w) s += red[w][tok][c];
                    red[0][tok][c] = s;
                }
            }
            cluster_sync_all();
            // the round's tokens, one in `parts` to each block, added over the blocks
            const int left = n - first < groups * SHRINK_GROUP ? n - first : groups * SHRINK_GROUP;
            const int half = nr / 2;
            for (int e = threadIdx.x; e < (left + parts - 1 - part) / parts * half; e += SHRINK_THREADS) {
                const int i = e / half, c = 2 * (e - i * half), tok = i * parts + part;
                const uint32_t at = smem_u32(&red[0][0][0]) + static_cast<uint32_t>((tok * NR + c) * 4);
                float v0[SHRINK_PARTS], v1[SHRINK_PARTS], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int w = 0; w < SHRINK_PARTS; ++w) {
                    uint32_t from;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(w < parts ? w : part));
                    v0[w] = w < parts ? ld_dsmem_f32(from) : 0.0f;
                    v1[w] = w < parts ? ld_dsmem_f32(from + 4) : 0.0f;
                }
#pragma unroll
                for (int w = 0; w < SHRINK_PARTS; ++w)
                    if (w < parts) {
                        s0 += v0[w];
                        s1 += v1[w];
                    }
                *reinterpret_cast<uint32_t *>(vslot + static_cast<int64_t>(plan.list[first + tok]) * p.r + c) =
                    pack_bf16x2(s0 * sc, s1 * sc);
            }
            cluster_sync_all();  // the sums have been read and may be overwritten
        }
    }
    if (!p.first) grid_dep_wait();  // completes after the staging kernel, for the product's sake
}

// The same for tiles whose slots hold many tokens (prompts): V of a whole token
// tile by tcgen05.mma, M = 128 tokens (twice for tiles wider than that), N = the
// rank block, X and A through TMA.  Rows of other adapters' tokens are computed
// and dropped.  A cluster of SHRINK_PARTS blocks splits K; warp 0 loads, warp 1
// issues, then all four move the fp32 sums to shared memory, and block i adds
// the parts for its share of the tokens.  (mma.sync from registers, as above,
// runs into the L1 cache's rate, eight lines to a load: 92 us for 8192 tokens of
// 4096 columns, rank 64; this 41 us, of which 11 are the reading of X.  Bound by
// the start and the exchange of short blocks; two blocks an SM hide part of it,
// one took 57 us.)
struct WideShrink {
    static constexpr int STAGES = 2, X_BYTES = 2 * 128 * 128, A_BYTES = SHRINK_RANKS * 128;
    static constexpr int STAGE_BYTES = X_BYTES + A_BYTES;
    static constexpr int SUM_LD = SHRINK_RANKS + 4;  // floats per token: 16-byte pieces without bank conflicts
    // the sums lie over the stages, so that two blocks fit on an SM
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + static_cast<int>(sizeof(TilePlan)) + 256 + 1024;
    static_assert(256 * SUM_LD * 4 <= STAGES * STAGE_BYTES && 2 * (SMEM_BYTES + 1024) <= 233472, "shared memory");
};

__global__ void __launch_bounds__(SHRINK_THREADS, 2)
    k_lora_shrink_wide(const __grid_constant__ ShrinkArgs p, const __grid_constant__ CUtensorMap tmx,
                       const __grid_constant__ CUtensorMap tma) {
    using C = WideShrink;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    float *sums = reinterpret_cast<float *>(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::STAGES * C::STAGE_BYTES);
    uint64_t *full = bars, *empty = bars + C::STAGES, *done = bars + 2 * C::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    TilePlan &plan = *reinterpret_cast<TilePlan *>(bars + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = static_cast<int>(cluster_ctarank());
    const int64_t tile = blockIdx.x / SHRINK_PARTS, t0 = tile * p.bn;
    const int rk = static_cast<int>(blockIdx.y % p.rb) * SHRINK_RANKS;
    const int lanes_z = gridDim.y / p.rb;
    const int nr = p.r - rk < SHRINK_RANKS ? p.r - rk : SHRINK_RANKS;
    const int nkb = static_cast<int>((p.K + 63) / 64);
    const int kb0 = nkb * part / SHRINK_PARTS, kb1 = nkb * (part + 1) / SHRINK_PARTS;
    const bool two = p.bn > 128;
    if (p.first) grid_dep_wait();
    grid_dep_launch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        fence_barrier_init();
        prefetch_tmap(&tmx);
        prefetch_tmap(&tma);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    const bool bad = plan_tile(p, tile, plan);  // synchronises the block
    tc_fence_after();
    if (bad) raise_error(ERRBIT_DEVICE);
    const uint32_t tmem_base = *tmem_slot;
    const int cnt = plan.cnt;
    const int64_t base = plan.base;
    if (part == 0 && blockIdx.y == 0) {  // what the product reads
        for (int k = threadIdx.x; k < cnt; k += SHRINK_THREADS) p.slot_adapter[base + k] = plan.adapter[k];
        if (threadIdx.x == 0) {
            p.tile_cnt[tile] = cnt;
            p.tile_base[tile] = static_cast<int32_t>(base);
        }
    }
    int s = 0, it = 0;
    uint32_t ph = 0, dph = 0;
    bool ok = true;
    for (int j = blockIdx.y / p.rb; j < cnt; j += lanes_z) {  // the same in every block of the cluster
        const int32_t ad = plan.adapter[j];
        if (warp == 0) {
            const bool lead = elect_one() != 0u;
            int ls = s, li = it;
            uint32_t lp = ph;
            for (int kb = kb0; kb < kb1 && ok; ++kb, ++li) {
                if (li >= C::STAGES && !mbar_wait_warp(&empty[ls], lp ^ 1u)) ok = false;
                if (ok && lead) {
                    uint8_t *st = smem + ls * C::STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[ls], static_cast<uint32_t>((two ? C::X_BYTES : C::X_BYTES / 2) + C::A_BYTES));
                    tma_load_2d(st, &tmx, &full[ls], kb * 64, static_cast<int32_t>(t0));
                    if (two) tma_load_2d(st + C::X_BYTES / 2, &tmx, &full[ls], kb * 64, static_cast<int32_t>(t0 + 128));
                    tma_load_3d(st + C::X_BYTES, &tma, &full[ls], kb * 64, rk, ad);
                }
                __syncwarp();
                if (++ls == C::STAGES) { ls = 0; lp ^= 1u; }
            }
        } else if (warp == 1) {
            const bool lead = elect_one() != 0u;
            const uint32_t idesc = make_idesc_bf16(128, static_cast<uint32_t>((nr + 15) / 16 * 16), false, 0);
            const uint64_t xd = make_sdesc(smem_u32(smem), 16, 1024, 2), yd = make_sdesc(smem_u32(smem) + C::X_BYTES / 2, 16, 1024, 2);
            const uint64_t ad0 = make_sdesc(smem_u32(smem) + C::X_BYTES, 16, 1024, 2);
            int ls = s;
            uint32_t lp = ph;
            for (int kb = kb0; kb < kb1 && ok; ++kb) {
                if (!mbar_wait_warp(&full[ls], lp)) ok = false;
                tc_fence_after();
                if (ok && lead) {
                    const uint64_t so = static_cast<uint64_t>(static_cast<uint32_t>(ls) * (C::STAGE_BYTES >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t acc = kb > kb0 || k > 0 ? 1u : 0u;
                        mma_bf16(tmem_base, xd + so + 2 * k, ad0 + so + 2 * k, idesc, acc);
                        if (two) mma_bf16(tmem_base + SHRINK_RANKS, yd + so + 2 * k, ad0 + so + 2 * k, idesc, acc);
                    }
                    mma_commit(&empty[ls]);
                    if (kb + 1 == kb1) mma_commit(done);
                }
                __syncwarp();
                if (++ls == C::STAGES) { ls = 0; lp ^= 1u; }
            }
        }
        const int n = kb1 - kb0;  // every warp keeps count of the stages
        it += n;
        s += n % C::STAGES;
        if (s >= C::STAGES) s -= C::STAGES;
        ph = static_cast<uint32_t>((it / C::STAGES) & 1);
        if (n > 0) {
            if (!mbar_wait_warp(done, dph)) ok = false;
            dph ^= 1u;
        }
        tc_fence_after();
        // sums [token][rank]: warp = 32 tokens of each half
        for (int half = 0; half < (two ? 2 : 1); ++half) {
            float *row = sums + (half * 128 + warp * 32 + lane) * C::SUM_LD;
            for (int c = 0; c < nr; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(warp * 32) << 16) + half * SHRINK_RANKS + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4 *>(row + c + 4 * i) =
                        n > 0 ? make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]))
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
        tc_fence_before();
        cluster_sync_all();
        tc_fence_after();
        const float sc = __ldg(p.scale + ad);
        uint16_t *vslot = p.V + (base + j) * p.bn * static_cast<int64_t>(p.r) + rk;
        const int quads = nr / 4;
        for (int e = threadIdx.x; e < (p.bn + SHRINK_PARTS - 1 - part) / SHRINK_PARTS * quads; e += SHRINK_THREADS) {
            const int i = e / quads, c = 4 * (e - i * quads), tok = i * SHRINK_PARTS + part;
            uint2 out = make_uint2(0u, 0u);
            if (plan.slot[tok] == j) {
                const uint32_t at = smem_u32(sums + tok * C::SUM_LD + c);
                float4 v[SHRINK_PARTS];
#pragma unroll
                for (int w = 0; w < SHRINK_PARTS; ++w) {
                    uint32_t from;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(w));
                    v[w] = ld_dsmem_f32x4(from);
                }
                float4 f = v[0];
#pragma unroll
                for (int w = 1; w < SHRINK_PARTS; ++w) {
                    f.x += v[w].x;
                    f.y += v[w].y;
                    f.z += v[w].z;
                    f.w += v[w].w;
                }
                out = make_uint2(pack_bf16x2(f.x * sc, f.y * sc), pack_bf16x2(f.z * sc, f.w * sc));
            }
            *reinterpret_cast<uint2 *>(vslot + static_cast<int64_t>(tok) * p.r + c) = out;
        }
        fence_proxy_async_smem();
        cluster_sync_all();  // the sums have been read; TMA may write there again
    }
    // a wait that ran out: let copies already issued land before exiting
    if (!ok && warp == 0)
        for (int q = it > C::STAGES ? it - C::STAGES : 0; q < it; ++q)
            mbar_wait_warp(&full[q % C::STAGES], static_cast<uint32_t>((q / C::STAGES) & 1));
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 128);
    }
    if (!p.first) grid_dep_wait();  // completes after the staging kernel, for the product's sake
}

}  // namespace nm

// ===========================================================================
// host side
// ===========================================================================
using namespace nm;

namespace {

template <int MODE, int OP>
int64_t ffn_clusters(int split) {
    return split > 1 ? resident_clusters_of<k_ffn<MODE, OP, true>>(split, ffn_threads(true), FfnCfg::SMEM_BYTES)
                     : resident_clusters_of<k_ffn<MODE, OP, false>>(1, ffn_threads(false), FfnCfg::SMEM_BYTES);
}

// How a call is cut: tokens per tile and pairs per tile.
struct FfnPlan {
    int bn, split, stages, sum_off, tile_rows;
    int64_t clusters;
};

// The cheapest in SM clocks by this model: rounds of tiles over the resident
// clusters, each round the K' blocks of a pair (an MMA of N tokens takes N/2 +
// 32 clocks and there are four per accumulator and block; the loads come at some
// 64 bytes a clock) and a fixed part: the epilogue, or with a split the exchange
// of the sums, 512 bytes per token and accumulator at some 18 bytes a clock.
// *sure: false if the device could not be asked about some of them.
template <int MODE, int OP>
bool ffn_search(int64_t T, int64_t Rpad, int64_t nkb, FfnPlan *best, bool *sure) {
    using Cfg = FfnCfg;
    const int forced_split = g_sched_policy.load() == 1 ? 1 : 0;
    const int forced_clusters = g_sched_clusters.load();
    const bool must_split = g_sched_policy.load() == 2 && nkb > 1;
    double best_cost = 0;
    bool found = false;
    const int bn_top = static_cast<int>(T < Cfg::BN_MAX ? (T + 15) / 16 * 16 : Cfg::BN_MAX);
    for (int split = 1; split <= Cfg::MAX_SPLIT && split <= nkb; ++split) {
        if ((forced_split && split > 1) || (must_split && split == 1)) continue;
        int64_t clusters = ffn_clusters<MODE, OP>(split);
        if (clusters < 0) *sure = false;
        if (forced_clusters > 0 && forced_clusters < clusters) clusters = forced_clusters;
        if (clusters < 1) continue;
        for (int v = 0; v < (OP == OP_LORA ? 2 : 1) * (bn_top / 16); ++v) {
            const int bn = bn_top - 16 * (v % (bn_top / 16));
            const int accs = v >= bn_top / 16 ? 1 : 2;  // OP_LORA: 512 rows a tile, or 256
            const int rows = OP == OP_GLU || accs == 1 ? 256 : 512;
            const int64_t tiles = (T + bn - 1) / bn * ((Rpad + rows - 1) / rows), rounds = (tiles + clusters - 1) / clusters;
            const int sb = Cfg::stage_bytes(bn);
            int room = split > 1 ? Cfg::SMEM_DATA : Cfg::OFF_OUT, off = 0;
            if (split > 1) {  // one round: the sums lie over the idle stages
                if (Cfg::sum_bytes(bn) > Cfg::SMEM_DATA) continue;
                if (rounds > 1) room -= Cfg::sum_bytes(bn);
            }
            int stages = room / sb;
            if (stages > Cfg::MAX_STAGES) stages = Cfg::MAX_STAGES;
            if (stages < 2) continue;
            if (split > 1 && rounds > 1) off = stages * sb;
            const double mma = accs * (2.0 * bn + 128);
            const double load = (sb - (accs == 1 ? Cfg::A_BYTES + EBLK_BYTES : 0)) / 64.0;
            const double block = mma > load ? mma : load;
            const double fixed = split > 1 ? 3000 + accs * 28.0 * bn : 1500 + 12.0 * bn;
            const double cost = rounds * (static_cast<double>((nkb + split - 1) / split) * block + fixed);
            if (!found || cost < best_cost) {
                found = true;
                best_cost = cost;
                *best = FfnPlan{bn, split, stages, off, rows, tiles < clusters ? tiles : clusters};
            }
        }
    }
    return found;
}

// the same, looked up: the search takes some 10 us of host time.  It depends on
// the sizes, the device and the schedule settings only.
template <int MODE, int OP>
bool ffn_plan(int64_t T, int64_t Rpad, int64_t nkb, FfnPlan *plan) {
    struct Entry {
        int64_t T, Rpad, nkb;
        int dev, policy, clusters;
        bool ok;
        FfnPlan plan;
    };
    static thread_local Entry cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const int policy = g_sched_policy.load(), clusters = g_sched_clusters.load();
    Entry &e = cache[static_cast<size_t>((T * 31 + Rpad / 256) * 31 + nkb) % 64];
    if (!e.ok || e.T != T || e.Rpad != Rpad || e.nkb != nkb || e.dev != dev || e.policy != policy ||
        e.clusters != clusters) {
        e = Entry{T, Rpad, nkb, dev, policy, clusters, false, {}};
        bool sure = true;
        const bool found = ffn_search<MODE, OP>(T, Rpad, nkb, &e.plan, &sure);
        e.ok = found && sure;
        *plan = e.plan;
        return found;
    }
    *plan = e.plan;
    return true;
}

template <int MODE, int OP>
nm_status launch_ffn(const FfnMaps &maps, FfnArgs p, const FfnPlan &plan, cudaStream_t s) {
    using Cfg = FfnCfg;
    p.bn = plan.bn;
    p.split = plan.split;
    p.stages = plan.stages;
    p.stage_bytes = Cfg::stage_bytes(plan.bn);
    p.sum_off = plan.sum_off;
    p.tile_rows = plan.tile_rows;
    p.stream_out = (p.G ? 3 : 1) * p.T * p.R * 2 > (64ll << 20) ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * plan.split * plan.clusters), 1, 1);
    cfg.blockDim = dim3(ffn_threads(plan.split > 1), 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * plan.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = plan.split > 1 ? cudaLaunchKernelEx(&cfg, k_ffn<MODE, OP, true>, maps, p)
                                         : cudaLaunchKernelEx(&cfg, k_ffn<MODE, OP, false>, maps, p);
    if (e != cudaSuccess) return NM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

template <class Kernel, class... Args>
nm_status launch_shrink(Kernel kernel, int parts, dim3 grid, int smem, cudaStream_t s, const Args &...args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(SHRINK_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return NM_ERR_CUDA;
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
    int64_t tiles, slots, v_rows;
    size_t o_cnt, o_base, o_adapter, o_v, bytes;
};

LoraWs lora_ws(int64_t T, int64_t r, int64_t requests, int64_t adapters) {
    LoraWs l{};
    const int64_t bnm = FfnCfg::BN_MAX;
    int64_t cap = requests < adapters ? requests : adapters;
    if (cap > bnm) cap = bnm;
    l.tiles = T / 16 + 2;
    const int64_t by_req = requests + l.tiles, by_cap = l.tiles * cap;
    l.slots = by_req < by_cap ? by_req : by_cap;
    const int64_t rows_req = (requests + 1) * bnm + T, rows_cap = (T + bnm) * cap;
    l.v_rows = rows_req < rows_cap ? rows_req : rows_cap;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    size_t o = 0;
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
    return gemm_ws(T, K, m).bytes;
}

extern "C" nm_status nm_sparse_glu(const uint16_t *X, int64_t T, int64_t K, int64_t ldx, const void *packed_gate,
                                   const void *packed_up, int64_t R, int m, int act, uint16_t *H, int64_t ldh,
                                   uint16_t *G, uint16_t *U, int64_t ldgu, void *ws, size_t ws_bytes,
                                   void *stream) {
    if (!X || !packed_gate || !packed_up || !H || (G == nullptr) != (U == nullptr)) return NM_ERR_NULL;
    nm_status st = check_ffn_sizes(T, K, R, m);
    if (st != NM_OK) return st;
    if (act < NM_ACT_SILU || act > NM_ACT_RELU2) return NM_ERR_UNSUPPORTED;
    if (ldx < K || ldh < R || (G && ldgu < R)) return NM_ERR_SHAPE;
    if (!aligned16(X) || !aligned16(packed_gate) || !aligned16(packed_up) || !aligned16(H) || (ldx % 8) != 0 ||
        (ldh % 8) != 0 || (G && (!aligned16(G) || !aligned16(U) || (ldgu % 8) != 0)) || (ws && !aligned16(ws)))
        return NM_ERR_ALIGN;
    const GemmWs w = gemm_ws(T, K, m);
    if (w.bytes > 0 && (!ws || ws_bytes < w.bytes)) return NM_ERR_WORKSPACE;
    const PackedGeom g = packed_geom(R, K, m);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FfnPlan plan;
    if (!(m == 8 ? ffn_plan<PMODE_SP68T, OP_GLU>(T, g.Rpad, g.nkb, &plan)
                 : ffn_plan<PMODE_SP24, OP_GLU>(T, g.Rpad, g.nkb, &plan)))
        return NM_ERR_CUDA;
    FfnMaps maps{};
    FfnArgs p{};
    p.T = T;
    p.R = R;
    p.nkb = g.nkb;
    p.early = m == 8 ? 1 : 0;  // the gather runs just before; X and the weights are older
    p.Y = H;
    p.ldy = ldh;
    p.G = G;
    p.U = U;
    p.ldgu = ldgu;
    p.act = act;
    if (!packed_maps(&maps.a0, &maps.e0, packed_gate, g) || !packed_maps(&maps.a1, &maps.e1, packed_up, g))
        return NM_ERR_CUDA;
    st = stage_b(X, T, K, ldx, m, g, w, ws, plan.bn, &maps, s);
    if (st != NM_OK) return st;
    return m == 8 ? launch_ffn<PMODE_SP68T, OP_GLU>(maps, p, plan, s) : launch_ffn<PMODE_SP24, OP_GLU>(maps, p, plan, s);
}

extern "C" size_t nm_sparse_gemm_lora_workspace_bytes(int64_t T, int64_t K, int m, int64_t r, int64_t adapters,
                                                      int64_t requests) {
    if (T < 1 || K < 1 || !pattern_ok(m) || r < 8 || r > NM_LORA_MAX_RANK || (r % 8) != 0 || adapters < 1 ||
        requests < 0)
        return 0;
    return up256(gemm_ws(T, K, m).bytes) + lora_ws(T, r, requests, adapters).bytes;
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
    FfnPlan plan;
    if (!(m == 8 ? ffn_plan<PMODE_SP68T, OP_LORA>(T, g.Rpad, g.nkb, &plan)
                 : ffn_plan<PMODE_SP24, OP_LORA>(T, g.Rpad, g.nkb, &plan)))
        return NM_ERR_CUDA;
    uint8_t *lw = static_cast<uint8_t *>(ws) + up256(w.bytes);
    int32_t *tile_cnt = reinterpret_cast<int32_t *>(lw + l.o_cnt);
    int32_t *tile_base = reinterpret_cast<int32_t *>(lw + l.o_base);
    int32_t *slot_adapter = reinterpret_cast<int32_t *>(lw + l.o_adapter);
    uint16_t *V = reinterpret_cast<uint16_t *>(lw + l.o_v);

    FfnMaps maps{};
    FfnArgs p{};
    p.T = T;
    p.R = R;
    p.nkb = g.nkb;
    p.early = m == 4 || m == 8 ? 1 : 0;  // 4:6 and 8:10 read the lifted activations from the first block on
    p.Y = Y;
    p.ldy = ldy;
    p.width = r <= 16 ? 16 : (r <= 32 ? 32 : 64);
    p.rb = static_cast<int>((r + 63) / 64);
    const int64_t tiles = (T + plan.bn - 1) / plan.bn;
    int64_t cap = requests < adapters ? requests : adapters;
    if (cap > plan.bn) cap = plan.bn;
    const int by_cap = tiles * cap <= requests + tiles ? 1 : 0;
    const int64_t nslots = by_cap ? tiles * cap : requests + tiles;
    p.tile_cnt = cap > 0 ? tile_cnt : nullptr;
    p.tile_base = tile_base;
    p.slot_adapter = slot_adapter;
    if (!packed_maps(&maps.a0, &maps.e0, packed, g)) return NM_ERR_CUDA;
    maps.a1 = maps.a0;
    maps.e1 = maps.e0;
    if (cap > 0) {
        if (!make_tmap_bf16_3d(&maps.lb, B, adapters, R, r, ldb, sdb, static_cast<uint32_t>(p.width), BM) ||
            !make_tmap_bf16_3d(&maps.lv, V, nslots, plan.bn, r, r, plan.bn * r, static_cast<uint32_t>(p.width),
                               static_cast<uint32_t>(plan.bn / 2)))
            return NM_ERR_CUDA;
    } else {
        maps.lb = maps.a0;
        maps.lv = maps.a0;
        if (m == 4) p.early = 0;  // no kernel of this call runs before the product
    }
    st = stage_b(X, T, K, ldx, m, g, w, ws, plan.bn, &maps, s);
    if (st != NM_OK) return st;
    const uint16_t *staged = static_cast<const uint16_t *>(ws);
    p.src = m == 4 || m == 8 ? X : staged;
    p.src_ld = m == 4 || m == 8 ? ldx : w.ld;
    p.src_cols = m == 4 || m == 8 ? K : w.cols;
    p.mid = staged;
    p.mid_ld = w.ld;
    p.mid_cols = w.cols;
    p.vals = static_cast<const uint16_t *>(packed);
    p.meta = static_cast<const uint8_t *>(packed) + g.vals_bytes;
    p.B = B;
    p.ldb = ldb;
    p.sdb = sdb;
    p.V = V;
    p.r = static_cast<int>(r);
    p.indptr = indptr;
    p.ids = ids;
    p.requests = static_cast<int32_t>(requests);
    if (cap > 0) {
        ShrinkArgs a{};
        a.X = X;
        a.A = A;
        a.scale = scale;
        a.indptr = indptr;
        a.ids = ids;
        a.T = T;
        a.K = K;
        a.ldx = ldx;
        a.lda = lda;
        a.sda = sda;
        a.nslots = nslots;
        a.requests = static_cast<int32_t>(requests);
        a.adapters = static_cast<int32_t>(adapters);
        a.r = static_cast<int>(r);
        a.rb = p.rb;
        a.bn = plan.bn;
        a.cap = static_cast<int>(cap);
        a.by_cap = by_cap;
        a.first = m == 4 ? 1 : 0;
        a.parts = SHRINK_PARTS;
        a.tile_cnt = tile_cnt;
        a.tile_base = tile_base;
        a.slot_adapter = slot_adapter;
        a.V = V;
        // Prompts take the wide kernel.  Its cost goes with the slots of a tile, the
        // other's with the tokens times the columns, so it needs enough tokens in all
        // (its start is some 8 us: 777 tokens, rank 8: 15.8 us against 12.5), columns
        // (8192 tokens of 16 requests, rank 16, whole call: 712 columns 35.8 us
        // against 25.2, 1000 columns 36.4 against 52.2) and tokens a request; the more
        // of these, the smaller the rank (1500 columns, rank 64, 64 tokens a request:
        // 65.8 against 87.6, 17: 119.8 against 99.9; rank 16: 57.7 against 57.4 at 64,
        // 96.3 against 63.2 at 17; 4096 columns, rank 16: 154 against 185 at 64, 217
        // against 174 at 17; all of 8192 tokens).
        if (T >= 1024 && K >= 896 && T >= 16 * requests &&
            (r > 16 || (T >= 32 * requests && T * K >= 131072 * requests))) {
            CUtensorMap tx, ta;
            if (!set_smem_attr<k_lora_shrink_wide>(WideShrink::SMEM_BYTES) ||
                !make_tmap_bf16(&tx, X, T, K, ldx, 64, 128, true) ||
                !make_tmap_bf16_3d(&ta, A, adapters, r, K, lda, sda, 64, SHRINK_RANKS))
                return NM_ERR_CUDA;
            const dim3 grid(static_cast<unsigned>(SHRINK_PARTS * tiles), static_cast<unsigned>((cap < 2 ? cap : 2) * p.rb));
            st = launch_shrink(k_lora_shrink_wide, SHRINK_PARTS, grid, WideShrink::SMEM_BYTES, s, a, tx, ta);
            if (st != NM_OK) return st;
            return m == 8 ? launch_ffn<PMODE_SP68T, OP_LORA>(maps, p, plan, s)
                          : launch_ffn<PMODE_SP24, OP_LORA>(maps, p, plan, s);
        }
        // all slots side by side, and K in as many parts as fit on the device then
        // (three blocks an SM); more slots than that take turns
        int64_t lanes = cap, at_once = 3 * sm_count() / (tiles * p.rb);
        a.parts = SHRINK_PARTS;
        while (a.parts > 2 && lanes * a.parts > at_once) a.parts /= 2;
        if (lanes * a.parts > 2 * at_once) lanes = 2 * at_once / a.parts + 1;
        if (lanes > cap) lanes = cap;
        const dim3 grid(static_cast<unsigned>(a.parts * tiles), static_cast<unsigned>(lanes * p.rb));
        st = r <= 8    ? launch_shrink(k_lora_shrink<1>, a.parts, grid, 0, s, a)
             : r <= 16 ? launch_shrink(k_lora_shrink<2>, a.parts, grid, 0, s, a)
             : r <= 32 ? launch_shrink(k_lora_shrink<4>, a.parts, grid, 0, s, a)
                       : launch_shrink(k_lora_shrink<8>, a.parts, grid, 0, s, a);
        if (st != NM_OK) return st;
    }
    return m == 8 ? launch_ffn<PMODE_SP68T, OP_LORA>(maps, p, plan, s)
                  : launch_ffn<PMODE_SP24, OP_LORA>(maps, p, plan, s);
}

// nm_gemm.cuh -- what the tcgen05 GEMM kernels of the library share: the packed
// operand's geometry, the order and the split of the work over CTA pairs, the
// stream-K flags, and the host side's schedule settings and activation staging.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <chrono>

#include "nm_common.cuh"
#include "nm_host.cuh"

namespace nm {

constexpr int BM = 128;          // weight rows per tile (MMA M)

constexpr int EBLK_BYTES = 2048; // metadata of 128 rows x 128 lifted columns

// ---------------------------------------------------------------------------
// packed operand layout (opaque to callers):
//   [0, Rpad*KLpad)                  values, row-major [Rpad x KLpad/2] bf16
//   [Rpad*KLpad, + Rpad*KLpad/8)     metadata blocks, (row tile of 128, K'
//                                    block of 128) order, 2048 bytes each
// Rpad = R rounded up to 256 (one CTA pair tile), KLpad = nkb * 128.
//
// K' order.  A K' block holds 32 windows ("slots") of 4 lifted columns.
//   m = 4, 6, 10: natural order: slot s of block kb is window wi = 32*kb + s,
//                 i.e. group wi / nwin, window wi % nwin (nwin = m/2 - 1).
//   m = 8       : blocks come in threes per 32 groups (256 columns of X):
//                 block 3j   : groups 32j .. 32j+15, windows 0 and 2 of each
//                              group = columns 8g .. 8g+7 of X, in X's order;
//                 block 3j+1 : groups 32j+16 .. 32j+31, likewise;
//                 block 3j+2 : window 1 (columns 8g+2 .. 8g+5) of groups
//                              32j .. 32j+31.
//                 Blocks 3j and 3j+1 are plain tiles of X (TMA loads them into
//                 the operand buffer); only block 3j+2 is built by the lift.
// Any consistent K' order gives the same product, because A (values and
// index pairs) and B (lifted activations) are permuted together.
// ---------------------------------------------------------------------------
struct PackedGeom {
    int64_t G, nwin, KL, KLpad, Rpad, nkb, vals_bytes, meta_bytes;
};

__host__ __device__ inline PackedGeom packed_geom(int64_t R, int64_t K, int m) {
    PackedGeom p;
    p.G = (K + m - 1) / m;
    p.nwin = p.G * (m / 2 - 1);
    p.KL = p.nwin * 4;
    p.nkb = m == 8 ? 3 * ((p.G + 31) / 32) : (p.KL + 127) / 128;
    p.KLpad = p.nkb * 128;
    p.Rpad = (R + 255) / 256 * 256;
    p.vals_bytes = p.Rpad * p.KLpad;       // Rpad x KLpad/2 bf16
    p.meta_bytes = p.Rpad * p.KLpad / 8;   // 4 bits per window of 4
    return p;
}

// PMODE_SP68T: 6:8 with every B block a TMA tile -- raw blocks from X, middle
// windows from X_mid (gathered by k_gather_mid before the GEMM).
enum { PMODE_DENSE = 0, PMODE_SP24 = 1, PMODE_SPLIFT = 2, PMODE_SP68 = 3, PMODE_SP68T = 4 };

// 6:8: the K' blocks in the order the library kernel's producer visits them --
// the blocks that are tiles of X itself first, the middle-window blocks (from
// the gathered X_mid) last -- so that the gather launched just before the GEMM
// overlaps the first two thirds of every tile's mainloop.  The packed layout
// is unchanged; only the order of the fp32 accumulation differs.
__device__ __forceinline__ int64_t visit68(int64_t v, int64_t nkb) {
    const int64_t nraw = 2 * (nkb / 3);
    return v < nraw ? 3 * (v >> 1) + (v & 1) : 3 * (v - nraw) + 2;
}

// Output tile order: bands of `gm` row tiles, each band walked token tile
// by token tile (the band's row tiles side by side).  Concurrent CTA pairs
// then share a few row tiles of weights and a few token tiles of X, which stay
// in L2 across the pairs and the waves of a band, instead of every wave
// streaming all of X again.  A bijection on [0, n_t * n_m); every role of a
// kernel uses it, so stream-K ranges over the same linear order.
__device__ __forceinline__ void tile_coords(int64_t tile, int64_t n_t, int64_t n_m, int64_t gm, int64_t &nt,
                                            int64_t &mt) {
    const int64_t band = tile / (gm * n_t);
    const int64_t rem = tile - band * gm * n_t;
    const int64_t rows = n_m - band * gm < gm ? n_m - band * gm : gm;  // row tiles of this band
    nt = rem / rows;
    mt = band * gm + (rem - nt * rows);
}
constexpr int64_t BAND_ROWS = 4096;   // weight rows per band of the tile order

struct SegIter {
    bool sk;
    int64_t nkb, pos, end, step;
    __device__ SegIter(bool sk_, int64_t cluster, int64_t nclusters, int64_t ntiles, int64_t nkb_)
        : sk(sk_), nkb(nkb_) {
        if (sk) {
            const int64_t total = ntiles * nkb;
            pos = cluster * total / nclusters;
            end = (cluster + 1) * total / nclusters;
            step = 0;
        } else {
            pos = cluster;
            end = ntiles;
            step = nclusters;
        }
    }
    __device__ bool more() const { return pos < end; }
    __device__ bool next(int64_t &tile, int64_t &kb0, int64_t &kb1) {
        if (pos >= end) return false;
        if (!sk) {
            tile = pos;
            kb0 = 0;
            kb1 = nkb;
            pos += step;
            return true;
        }
        tile = pos / nkb;
        kb0 = pos - tile * nkb;
        kb1 = kb0 + (end - pos) < nkb ? kb0 + (end - pos) : nkb;
        pos += kb1 - kb0;
        return true;
    }
};

__device__ __forceinline__ void st_release_u64(uint64_t *p, uint64_t v) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

__device__ __forceinline__ uint64_t ld_acquire_u64(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

// bounded wait for a stream-K flag (one lane's answer; one second limit)
__device__ __forceinline__ bool sk_wait_flag(const uint64_t *p, uint64_t seq) {
    if (ld_acquire_u64(p) == seq) return true;
    const uint64_t t0 = global_timer_ns(), limit = wait_limit_ns();
    while (true) {
        __nanosleep(64);
        if (ld_acquire_u64(p) == seq) return true;
        if (global_timer_ns() - t0 > limit) {
            raise_error(ERRBIT_TIMEOUT);
            return false;
        }
    }
}

// The whole warp's wait for one flag: every lane polls and all get the same
// answer.  A flag has one reader, which clears it once seen: the replay of a
// captured launch carries the same sequence number, and must not take the partial
// sums of the replay before it for its own.
__device__ __forceinline__ bool sk_take_flag(uint64_t *p, uint64_t seq, int lane) {
    const bool seen = __all_sync(0xffffffffu, sk_wait_flag(p, seq));
    if (lane == 0 && seen) *static_cast<volatile uint64_t *>(p) = 0;
    return seen;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count() {
    static int n[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return 148;
    if (n[dev] == 0) {
        int v = 0;
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        n[dev] = v > 0 ? v : 148;
    }
    return n[dev];
}

// schedule override (0 = automatic, 1 = whole tiles, 2 = stream-K) and
// cluster count override (0 = as many as fit on the device at once)
inline std::atomic<int> g_sched_policy{0};
inline std::atomic<int> g_sched_clusters{0};

// launch sequence numbers: unique per launch in this process and, being
// seeded from the clock, unlikely to equal a stale flag left by another one
inline uint64_t next_seq() {
    static std::atomic<uint64_t> ctr{
        static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count()) | 1u};
    return ctr.fetch_add(1);
}

// clusters of 2 * pairs blocks of a kernel that can be resident at once on the
// current device, looked up once per device and number of pairs.  -1: a CUDA call
// failed; that is not remembered, so that later calls do not depend on it.
constexpr int MAX_PAIRS = 8;
template <auto kernel>
inline int64_t resident_clusters_of(int pairs, int threads, int smem) {
    static int cache[64][MAX_PAIRS + 1] = {};  // count + 1
    int dev = 0;
    if (pairs > MAX_PAIRS || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    if (cache[dev][pairs] == 0) {
        if (!set_smem_attr<kernel>(smem)) return -1;
        if (pairs > 4 &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return -1;
        }
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(static_cast<unsigned>(2 * pairs * (sm_count() / (2 * pairs))), 1, 1);
        q.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
        q.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = static_cast<unsigned>(2 * pairs);
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &q) != cudaSuccess) {
            cudaGetLastError();
            return -1;
        }
        cache[dev][pairs] = n + 1;
    }
    return cache[dev][pairs] - 1;
}

// extra device memory the online phase needs for (2N-2):2N patterns: the
// gathered middle windows (6:8) or the lifted activations (4:6, 8:10)
struct GemmWs {
    int64_t ld;      // leading dimension (elements) of the staged activations
    int64_t cols;    // their logical width
    size_t bytes;
};

inline GemmWs gemm_ws(int64_t T, int64_t K, int m) {
    GemmWs w{0, 0, 0};
    if (T < 1 || K < 1 || m == 4) return w;
    const int64_t G = (K + m - 1) / m;
    w.cols = m == 8 ? G * 4 : G * (m / 2 - 1) * 4;
    w.ld = (w.cols + 7) / 8 * 8;
    w.bytes = static_cast<size_t>(T) * static_cast<size_t>(w.ld) * 2;
    return w;
}

// the 6:8 middle windows X_mid [T x 4G] (leading dimension ldm) of X
nm_status launch_gather_mid(const uint16_t *X, int64_t T, int64_t K, int64_t ldx, int64_t G,
                            uint16_t *Xmid, int64_t ldm, cudaStream_t s);

// the stream-K region follows the staged activations, 256-byte aligned
inline size_t sk_offset(const GemmWs &w) { return (w.bytes + 255) / 256 * 256; }

}  // namespace nm

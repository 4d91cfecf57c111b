// Q/K/V projection in 8-bit integers with a scale for each token (feature row) and each output channel:
//
//   out[o(r), j] = (sum_c Xq[r, c] Wq[j, c]) * xs[r] * ws[j],   o(r) = inv[r] (slot order) or r
//
// The sum is exact in 32-bit integers (C <= 65536 values of at most 128 * 128).  Its conversion to float rounds beyond
// 2^24, each of the two scales rounds, and a 16-bit result rounds once more.
//
//  - k_project_i8_few   few rows: a warp per output channel, which reads the channel's weights once for up to
//                       eight rows.  Bound by the weights' bytes and by latency.
//  - k_project_i8_tc    many rows: tcgen05 tensor cores.
//  - k_project_i8_tile  many rows whose results are no multiple of 16 bytes, or not aligned to them: 64 x 64 tiles on
//                       the CUDA cores (dp4a).
#include <cuda_bf16.h>

#include <cstring>

#include "bts_internal.cuh"
#include "bts_tc.cuh"
#include "bts_maps.cuh"

namespace bts {
namespace {

template <typename T> __device__ __forceinline__ T out_value(float v);
template <> __device__ __forceinline__ float out_value<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 out_value<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The output of one projection: Q, K and V rows of hd = H d values.
template <typename T>
struct QkvOut {
    T *q, *k, *v;
    int hd;
    __device__ __forceinline__ T *at(int64_t row, int j) const
    {
        const int t = j / hd;
        return (t == 0 ? q : t == 1 ? k : v) + size_t(row) * hd + (j - t * hd);
    }
};

// The output row of feature row r, or -1 where it has no slot; an inv entry that is neither a slot nor says so is
// recorded.
__device__ __forceinline__ int32_t out_row(const int32_t *inv, int64_t r, int64_t npad, uint32_t *status)
{
    if (!inv) return int32_t(r);
    const int32_t o = __ldg(inv + r);
    if (o >= 0 && o < npad) return o;
    if (o != BT_NO_SLOT) record_error(status, BT_ERR_INTERNAL);
    return -1;
}

// Zero rows of Q, K and V in the dummy slots (perm < 0, or recorded: no row of the tensors), which no feature row fills:
// warp w of nw takes runs of 32 slots, and all lanes write each dummy's row.
template <typename T>
__device__ __forceinline__ void zero_dummies(const int32_t *__restrict__ perm, int64_t npad, int64_t rows,
                                             const QkvOut<T> &out, int64_t w, int64_t nw, uint32_t *status)
{
    const int lane = threadIdx.x & 31;
    const int bytes = out.hd * int(sizeof(T));
    const uintptr_t al = reinterpret_cast<uintptr_t>(out.q) | reinterpret_cast<uintptr_t>(out.k) |
                         reinterpret_cast<uintptr_t>(out.v) | uintptr_t(bytes);
    for (int64_t s0 = w * 32; s0 < npad; s0 += nw * 32) {
        const int64_t s = s0 + lane;
        const int32_t r = s < npad ? __ldg(perm + s) : 0;
        uint32_t dead = __ballot_sync(0xffffffffu, s < npad && uint32_t(r) >= uint32_t(rows));  // rows < 2^31
        if (dead && r >= 0 && s < npad && r >= rows) record_error(status, BT_ERR_INTERNAL);
        while (dead) {
            const int64_t slot = s0 + __ffs(int(dead)) - 1;
            dead &= dead - 1;
            const size_t o = size_t(slot) * out.hd;
            if (al % 16 == 0) {
                for (int i = lane; i < bytes / 16; i += 32) {
                    reinterpret_cast<uint4 *>(out.q + o)[i] = make_uint4(0, 0, 0, 0);
                    reinterpret_cast<uint4 *>(out.k + o)[i] = make_uint4(0, 0, 0, 0);
                    reinterpret_cast<uint4 *>(out.v + o)[i] = make_uint4(0, 0, 0, 0);
                }
            } else {
                for (int i = lane; i < out.hd; i += 32)
                    out.q[o + i] = out.k[o + i] = out.v[o + i] = out_value<T>(0.0f);
            }
        }
    }
}

// LB bytes at p as 32-bit words, bytes past `left` as zeros (LB 16 or 4: whole words are there)
template <int LB>
__device__ __forceinline__ void load_words(const int8_t *p, int left, uint32_t (&w)[(LB + 3) / 4])
{
    if constexpr (LB == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (LB == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else {
        w[0] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (b < left) w[0] |= uint32_t(uint8_t(__ldg(p + b))) << (8 * b);
    }
}

constexpr int kFewRows = 8;   // rows that share one read of the weights
constexpr int kFewWarps = 8;

// LB: bytes per load (16, 4; 1 = four single bytes)
template <typename T, int LB>
__global__ void __launch_bounds__(kFewWarps * 32)
    k_project_i8_few(const int8_t *__restrict__ X, const float *__restrict__ xs, int64_t rows, int C,
                     const int8_t *__restrict__ W, const float *__restrict__ ws, int nout, QkvOut<T> out,
                     const int32_t *__restrict__ perm, const int32_t *__restrict__ inv, int64_t npad, uint32_t *status)
{
    constexpr int STEP = LB == 1 ? 4 : LB, NW = (LB + 3) / 4;
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
    if (j < nout) {
        const int8_t *wr = W + size_t(j) * C;
        const float wsj = __ldg(ws + j);
        for (int64_t r0 = 0; r0 < rows; r0 += kFewRows) {
            const int nr = int(min64(kFewRows, rows - r0));
            int32_t acc[kFewRows];
#pragma unroll
            for (int i = 0; i < kFewRows; ++i) acc[i] = 0;
            for (int c = lane * STEP; c < C; c += 32 * STEP) {
                uint32_t wv[NW];
                load_words<LB>(wr + c, C - c, wv);
#pragma unroll
                for (int i = 0; i < kFewRows; ++i)
                    if (i < nr) {
                        uint32_t xv[NW];
                        load_words<LB>(X + size_t(r0 + i) * C + c, C - c, xv);
#pragma unroll
                        for (int e = 0; e < NW; ++e) acc[i] = __dp4a(int(xv[e]), int(wv[e]), acc[i]);
                    }
            }
            int32_t mine = 0;
#pragma unroll
            for (int i = 0; i < kFewRows; ++i) {
                const int32_t s = __reduce_add_sync(0xffffffffu, acc[i]);
                if (lane == i) mine = s;
            }
            if (lane < nr) {
                const int64_t r = r0 + lane;
                const int32_t o = out_row(inv, r, npad, status);
                if (o >= 0) *out.at(o, j) = out_value<T>(float(mine) * __ldg(xs + r) * wsj);
            }
        }
    }
    if (perm)
        zero_dummies(perm, npad, rows, out, int64_t(blockIdx.x) * kFewWarps + (threadIdx.x >> 5),
                     int64_t(gridDim.x) * kFewWarps, status);
}

constexpr int kTile = 64, kTileK = 64;  // rows and channels of a tile; bytes of the row length per step

template <typename T, int LB>
__global__ void __launch_bounds__(256)
    k_project_i8_tile(const int8_t *__restrict__ X, const float *__restrict__ xs, int64_t rows, int C,
                      const int8_t *__restrict__ W, const float *__restrict__ ws, int nout, QkvOut<T> out,
                      const int32_t *__restrict__ perm, const int32_t *__restrict__ inv, int64_t npad,
                      uint32_t *status)
{
    constexpr int KW = kTileK / 4, LD = KW + 1;  // 32-bit words per row of a step; odd stride: no bank conflicts
    __shared__ uint32_t sx[kTile * LD], sw[kTile * LD];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t r0 = int64_t(blockIdx.x) * kTile;
    const int j0 = blockIdx.y * kTile;
    int32_t acc[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = 0;
    for (int c0 = 0; c0 < C; c0 += kTileK) {
#pragma unroll
        for (int u = tid; u < kTile * KW; u += 256) {
            const int r = u / KW, k = u - r * KW, c = c0 + 4 * k;
            uint32_t xv[1] = {0}, wv[1] = {0};
            if (c < C) {
                if (r0 + r < rows) load_words<LB>(X + size_t(r0 + r) * C + c, C - c, xv);
                if (j0 + r < nout) load_words<LB>(W + size_t(j0 + r) * C + c, C - c, wv);
            }
            sx[r * LD + k] = xv[0];
            sw[r * LD + k] = wv[0];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            int xv[4], wv[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                xv[a] = int(sx[(ty + 16 * a) * LD + k]);
                wv[a] = int(sw[(tx + 16 * a) * LD + k]);
            }
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = __dp4a(xv[a], wv[b], acc[a][b]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int64_t r = r0 + ty + 16 * a;
        if (r >= rows) continue;
        const int32_t o = out_row(inv, r, npad, status);
        if (o < 0) continue;
        const float xr = __ldg(xs + r);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int j = j0 + tx + 16 * b;
            if (j < nout) *out.at(o, j) = out_value<T>(float(acc[a][b]) * xr * __ldg(ws + j));
        }
    }
    if (perm && blockIdx.y == 0)
        zero_dummies(perm, npad, rows, out, int64_t(blockIdx.x) * 8 + (tid >> 5), int64_t(gridDim.x) * 8, status);
}

// ---------------------------------------------------------------------------
// Tensor cores (tcgen05.mma kind::i8, 32-bit integer sums in TMEM).  A CTA keeps to one chunk of BN output channels and
// walks the 128-row tiles of X:
//   warps 17-20  loaders.  TMA: one thread fetches 128 x 128-byte boxes (128-byte swizzle; rows and columns outside read
//               zeros).  Otherwise (row lengths or addresses that no tensor map takes) the four warps copy rows, put
//               together from aligned words.
//   warp 16      issues the products, two accumulators of BN columns;
//   warps 0-15   four warps per 32 rows, a quarter of the columns (but at least 32) each: scale, round, pass through
//                4 KB of shared memory of the warp's own, and store 128-byte pieces of rows to the row's slot of Q, K
//                or V.
// W stays in shared memory where the chunk's rows fit (`keep`), else it is fetched with each block of X.
// Bound by the integer products: 65,536 x 256 -> 768 keeps the tensor pipe active for 23 us (4,096 operations a cycle and
// SM, half of what bf16 has); its 118 MB take 18 us.  Measured: 39 us; the rest is the launch, W's arrival, and eleven
// tiles a CTA where 10.4 are due.  Eight storing warps instead of sixteen: 43.  Without TMA the copying warps bound it
// (65,536 x 255: 118 us, six times its bytes' 19; x 99: 77 us).
// ---------------------------------------------------------------------------
struct I8Tile {
    static constexpr int BM = 128, BK = 128, EPI = 16, THREADS = (EPI + 5) * 32;
    static constexpr uint32_t XBLK = BM * BK;
    static constexpr uint32_t OUT = EPI * 4096;      // the epilogue's pieces
    static constexpr uint32_t ROOM = 160 * 1024;     // for W and the ring
    static constexpr int RING = 6;                   // stages, at most
};

__device__ __forceinline__ void mma_i8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// The aligned word at p of a matrix that begins and ends at the given addresses; a word that reaches out of it comes byte by
// byte, with zeros outside.
__device__ __forceinline__ uint32_t word_at(uintptr_t p, uintptr_t begin, uintptr_t end)
{
    if (p >= begin && p + 4 <= end) return __ldg(reinterpret_cast<const uint32_t *>(p));
    uint32_t x = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (p + b >= begin && p + b < end) x |= uint32_t(uint8_t(__ldg(reinterpret_cast<const int8_t *>(p + b)))) << (8 * b);
    return x;
}

// Columns c0 .. c0 + 127 of row r of the [n][C] bytes at M by a warp: lane l gets bytes 4l .. 4l + 3, zeros outside.  No
// alignment needed: neighbouring lanes read neighbouring words, and each shifts its own and the next lane's together.
struct RowWords {
    uint32_t x, last;
    int left, sh;
    // INSIDE: no word of the row reaches out of the matrix, and the loads wait for nothing
    template <bool INSIDE>
    __device__ __forceinline__ void load(const int8_t *__restrict__ M, int64_t n, int C, int64_t r, int c0, int lane)
    {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(M), end = begin + size_t(n) * C;
        const uintptr_t a = begin + size_t(r) * C + c0, w = a & ~uintptr_t(3);
        left = r < n ? min(128, C - c0) : 0;
        sh = int(a & 3) * 8;
        const int words = left ? (int(a & 3) + left + 3) >> 2 : 0;  // up to 33
        x = last = 0u;
        if constexpr (INSIDE) {
            if (lane < words) x = __ldg(reinterpret_cast<const uint32_t *>(w) + lane);
            if (lane == 31 && words > 32) last = __ldg(reinterpret_cast<const uint32_t *>(w) + 32);
        } else {
            if (lane < words) x = word_at(w + 4 * lane, begin, end);
            if (lane == 31 && words > 32) last = word_at(w + 128, begin, end);
        }
    }
    __device__ __forceinline__ uint32_t get(int lane) const
    {
        uint32_t next = __shfl_down_sync(0xffffffffu, x, 1);
        next = lane == 31 ? last : next;
        const uint32_t y = __funnelshift_r(x, next, sh);
        const int rest = left - 4 * lane;  // bytes of this word inside the row
        return rest >= 4 ? y : rest <= 0 ? 0u : y & ((1u << (8 * rest)) - 1u);
    }
};

template <typename T, int BN, bool TMA>
__global__ void __launch_bounds__(I8Tile::THREADS, 1)
    k_project_i8_tc(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const int8_t *__restrict__ X, const float *__restrict__ xs, int64_t rows, int C,
                    const int8_t *__restrict__ W, const float *__restrict__ ws, int nout, QkvOut<T> out,
                    const int32_t *__restrict__ perm, const int32_t *__restrict__ inv, int64_t npad, int64_t tiles,
                    int nch, int stages, bool keep, uint32_t *status)
{
    using L = I8Tile;
    constexpr uint32_t WBLK = BN * L::BK, SBO = 1024, SW128 = 2;
    // S32 sums of S8 and S8, both K-major, M = 128
    constexpr uint32_t IDESC = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(BN >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    constexpr uint32_t COLS = BN == 256 ? 512 : BN == 128 ? 256 : 128;  // two accumulators
    extern __shared__ __align__(1024) uint8_t psm[];
    __shared__ __align__(8) uint64_t sWFull, sFull[L::RING], sEmpty[L::RING], sAccFull[2], sAccEmpty[2];
    __shared__ __align__(16) float sScale[BN];
    __shared__ uint32_t sTmem;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int KB = (C + L::BK - 1) / L::BK;
    const int chunk = int(blockIdx.x) % nch;
    const int64_t groups = int64_t(gridDim.x) / nch, first = int64_t(blockIdx.x) / nch;
    const uint32_t base = (smem_u32(psm) + 1023u) & ~1023u;
    uint8_t *gbase = psm + (base - smem_u32(psm));
    const uint32_t ring = L::OUT + (keep ? uint32_t(KB) * WBLK : 0);  // offsets from base: pieces, W, ring
    const uint32_t stage = L::XBLK + (keep ? 0 : WBLK);
    constexpr uint32_t LOADERS = TMA ? 1 : 4;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sTmem)),
                     "r"(COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        auto init = [](uint64_t *b, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n) : "memory");
        };
        init(&sWFull, LOADERS);
        for (int i = 0; i < L::RING; ++i) {
            init(&sFull[i], LOADERS);
            init(&sEmpty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            init(&sAccFull[i], 1);
            init(&sAccEmpty[i], L::EPI);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int j = tid; j < BN; j += L::THREADS) sScale[j] = chunk * BN + j < nout ? __ldg(ws + chunk * BN + j) : 0.0f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sTmem;

    if (warp > L::EPI) {
        if (TMA) {
            if (perm && warp > L::EPI + 1)  // these three have nothing to load
                zero_dummies(perm, npad, rows, out, int64_t(blockIdx.x) * 3 + warp - L::EPI - 2, int64_t(gridDim.x) * 3,
                             status);
            if (warp == L::EPI + 1 && lane == 0) {
                bool ok = true;
                if (keep) {
                    mbar_expect_tx(smem_u32(&sWFull), uint32_t(KB) * WBLK);
                    for (int k = 0; k < KB; ++k)
                        tma_load_2d(base + L::OUT + k * WBLK, &tmW, k * L::BK, chunk * BN, smem_u32(&sWFull));
                }
                int i = 0;
                for (int64_t tile = first; tile < tiles && ok; tile += groups)
                    for (int k = 0; k < KB && ok; ++k, ++i) {
                        const int s = i % stages;
                        if (i >= stages) ok = mbar_wait(smem_u32(&sEmpty[s]), ((i / stages) - 1) & 1, status);
                        if (ok) {
                            const uint32_t full = smem_u32(&sFull[s]), at = base + ring + s * stage;
                            mbar_expect_tx(full, stage);
                            tma_load_2d(at, &tmX, k * L::BK, int32_t(tile * L::BM), full);
                            if (!keep) tma_load_2d(at + L::XBLK, &tmW, k * L::BK, chunk * BN, full);
                        }
                    }
                // the copies in flight
                if (keep) mbar_wait(smem_u32(&sWFull), 0, status);
                for (int k = i - 1; k >= 0 && k >= i - stages; --k)
                    mbar_wait(smem_u32(&sFull[k % stages]), (k / stages) & 1, status);
            }
        } else {
            const int lw = warp - L::EPI - 1;  // 0 .. 3: every fourth row
            auto block = [&](const int8_t *M, int64_t n, int64_t r0, int nr, int k, uint32_t off) {
                const bool inside = r0 > 0 && r0 + nr < n && C >= 4;  // a word at least before and after the rows
#pragma unroll 1
                for (int r1 = lw; r1 < nr; r1 += 32) {  // eight rows under way at a time: sixteen spill
                    RowWords v[8];
                    if (inside) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i].load<true>(M, n, C, r0 + r1 + 4 * i, k * L::BK, lane);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i].load<false>(M, n, C, r0 + r1 + 4 * i, k * L::BK, lane);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r1 + 4 * i;
                        *reinterpret_cast<uint32_t *>(gbase + off + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                                      (lane & 3) * 4) = v[i].get(lane);
                    }
                }
            };
            auto arrive = [&](uint64_t *bar) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
            };
            bool ok = true;
            if (keep) {
                for (int k = 0; k < KB; ++k) block(W, nout, chunk * BN, BN, k, L::OUT + k * WBLK);
                arrive(&sWFull);
            }
            int i = 0;
            for (int64_t tile = first; tile < tiles && ok; tile += groups)
                for (int k = 0; k < KB && ok; ++k, ++i) {
                    const int s = i % stages;
                    if (i >= stages) ok = mbar_wait(smem_u32(&sEmpty[s]), ((i / stages) - 1) & 1, status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    block(X, rows, tile * L::BM, L::BM, k, ring + s * stage);
                    if (!keep) block(W, nout, chunk * BN, BN, k, ring + s * stage + L::XBLK);
                    arrive(&sFull[s]);
                }
        }
        __syncwarp();
    } else if (warp == L::EPI) {
        // ---------------- products (one thread) ----------------
        if (lane == 0) {
            bool ok = !keep || mbar_wait(smem_u32(&sWFull), 0, status);
            tc_fence_after();
            int i = 0, ai = 0;
            for (int64_t tile = first; tile < tiles && ok; tile += groups, ++ai) {
                const int ab = ai & 1;
                if (ai >= 2) ok = mbar_wait(smem_u32(&sAccEmpty[ab]), ((ai >> 1) - 1) & 1, status);
                tc_fence_after();
                const uint32_t acc = tmem + uint32_t(ab) * BN;
                for (int k = 0; k < KB && ok; ++k, ++i) {
                    const int s = i % stages;
                    ok = mbar_wait(smem_u32(&sFull[s]), (i / stages) & 1, status);
                    tc_fence_after();
                    if (ok) {
                        const uint32_t xa = base + ring + s * stage;
                        const uint32_t wa = keep ? base + L::OUT + k * WBLK : xa + L::XBLK;
                        const int nk = min(4, (C - k * L::BK + 31) / 32);  // zeros beyond the row length
                        for (int kk = 0; kk < nk; ++kk)
                            mma_i8(acc, smem_desc_sw(xa + 32 * kk, 16, SBO, SW128),
                                   smem_desc_sw(wa + 32 * kk, 16, SBO, SW128), IDESC, (k | kk) != 0);
                    }
                    mma_commit(smem_u32(&sEmpty[s]));  // the stage is free once these products are done
                }
                mma_commit(smem_u32(&sAccFull[ab]));
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue ----------------
        constexpr int PC = 128 / int(sizeof(T));      // columns of a piece (128 bytes)
        constexpr int CE = 16 / int(sizeof(T));       // columns of a chunk (16 bytes)
        constexpr int CW = BN >= 128 ? BN / 4 : 32;   // columns of a warp
        const int quarter = warp >> 2;
        const uint32_t lb = uint32_t((warp & 3) * 32) << 16;
        uint8_t *piece = gbase + warp * 4096;
        bool ok = true;
        int ai = 0;
        for (int64_t tile = first; tile < tiles && ok; tile += groups, ++ai) {
            const int64_t row = tile * L::BM + (warp & 3) * 32 + lane;
            int32_t orow = -1;
            float xr = 0.0f;
            if (row < rows) {
                xr = __ldg(xs + row);
                orow = inv ? __ldg(inv + row) : int32_t(row);
                if (uint32_t(orow) >= uint32_t(npad)) {  // not a slot: never write it (without inv, npad is rows)
                    if (orow != BT_NO_SLOT && quarter == 0 && chunk == 0) record_error(status, BT_ERR_INTERNAL);
                    orow = -1;
                }
            }
            const int ab = ai & 1;
            ok = mbar_wait(smem_u32(&sAccFull[ab]), (ai >> 1) & 1, status);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const uint32_t acc = tmem + uint32_t(ab) * BN + uint32_t(quarter * CW) + lb;
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += PC) {
                const int jl = quarter * CW + c0, j0 = chunk * BN + jl;
                if (jl >= BN || j0 >= nout || !ok) break;  // the same for every thread of the warp
#pragma unroll
                for (int q = 0; q < PC; q += 32) {
                    if (c0 + q >= CW) break;
                    uint32_t v[32];
                    tmem_ld32_nowait(acc + c0 + q, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 32; g += CE) {
                        uint4 o;
                        float f[CE];
#pragma unroll
                        for (int e = 0; e < CE; e += 4) {
                            const float4 w = *reinterpret_cast<const float4 *>(sScale + jl + q + g + e);
                            f[e] = float(int(v[g + e])) * xr * w.x;
                            f[e + 1] = float(int(v[g + e + 1])) * xr * w.y;
                            f[e + 2] = float(int(v[g + e + 2])) * xr * w.z;
                            f[e + 3] = float(int(v[g + e + 3])) * xr * w.w;
                        }
                        if constexpr (sizeof(T) == 4) {
                            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                           __float_as_uint(f[3]));
                        } else {
                            uint32_t b[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                                b[e] = *reinterpret_cast<const uint32_t *>(&t);
                            }
                            o = make_uint4(b[0], b[1], b[2], b[3]);
                        }
                        const int c = (q + g) / CE;  // chunk 0 .. 7 of the piece
                        *reinterpret_cast<uint4 *>(piece + lane * 128 + ((c ^ (lane & 7)) << 4)) = o;
                    }
                }
                __syncwarp();
                // 4 rows of 128 bytes at a time
                const int c = lane & 7, j = j0 + c * CE;
                const bool in = c * CE < CW - c0 && j < nout;  // 3 H d is a multiple of a chunk
                const int t = j / out.hd;
                T *dst = (t == 0 ? out.q : t == 1 ? out.k : out.v) + (j - t * out.hd);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = i * 4 + (lane >> 3);
                    const int32_t to = __shfl_sync(0xffffffffu, orow, r);
                    const uint4 o = *reinterpret_cast<const uint4 *>(piece + r * 128 + ((c ^ (r & 7)) << 4));
                    if (to >= 0 && in) *reinterpret_cast<uint4 *>(dst + size_t(to) * out.hd) = o;
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sAccEmpty[ab])) : "memory");
        }
        if (!TMA && perm)
            zero_dummies(perm, npad, rows, out, int64_t(blockIdx.x) * L::EPI + warp, int64_t(gridDim.x) * L::EPI, status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS) : "memory");
    }
}

template <typename T>
struct I8Args {
    const int8_t *X;
    const float *xs;
    int64_t rows;
    int C;
    const int8_t *W;
    const float *ws;
    int nout;
    QkvOut<T> out;
    const int32_t *perm, *inv;
    int64_t npad;
    bool tma;
    int sms;
    uint32_t *status;
    cudaStream_t st;
};

template <typename T, int BN, bool TMA>
bt_status run_project_tc(const I8Args<T> &a)
{
    using L = I8Tile;
    static std::atomic<bool> set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BT_ERR_CUDA;
    if (dev < 0 || dev >= 64) return BT_ERR_UNSUPPORTED;
    const bt_status s = setup_once(set[dev], [&]() -> bt_status {
        return cudaFuncSetAttribute(k_project_i8_tc<T, BN, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(L::ROOM + L::OUT + 1024)) == cudaSuccess
                   ? BT_OK
                   : BT_ERR_CUDA;
    });
    if (s != BT_OK) return s;
    CUtensorMap mx, mw;
    memset(&mx, 0, sizeof mx);
    memset(&mw, 0, sizeof mw);
    if (TMA && (!matrix_map(&mx, a.X, a.rows, a.C, 1, L::BK, L::BM) || !matrix_map(&mw, a.W, a.nout, a.C, 1, L::BK, BN)))
        return BT_ERR_CUDA;
    const int KB = (a.C + L::BK - 1) / L::BK;
    const int64_t wbytes = int64_t(KB) * BN * L::BK;
    const bool keep = wbytes + 2 * int64_t(L::XBLK) <= int64_t(L::ROOM);  // and two stages beside it
    const uint32_t stage = L::XBLK + (keep ? 0 : BN * L::BK);
    int stages = int((L::ROOM - (keep ? uint32_t(wbytes) : 0)) / stage);
    if (stages > L::RING) stages = L::RING;
    const size_t smem = L::OUT + 1024 + (keep ? size_t(wbytes) : 0) + size_t(stages) * stage;
    const int nch = (a.nout + BN - 1) / BN;
    const int64_t tiles = (a.rows + L::BM - 1) / L::BM;
    int64_t groups = a.sms / nch;
    if (groups < 1) groups = 1;
    if (groups > tiles) groups = tiles;
    k_project_i8_tc<T, BN, TMA><<<unsigned(groups * nch), L::THREADS, smem, a.st>>>(
        mx, mw, a.X, a.xs, a.rows, a.C, a.W, a.ws, a.nout, a.out, a.perm, a.inv, a.npad, tiles, nch, stages, keep,
        a.status);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <typename T, bool TMA>
bt_status launch_project_tc(const I8Args<T> &a)
{
    // wide chunks read X less often; narrow ones spread few rows over more SMs
    const int64_t tiles = (a.rows + 127) / 128;
    if (a.C <= 512 && tiles * ((a.nout + 255) / 256) >= a.sms) return run_project_tc<T, 256, TMA>(a);
    if (tiles * ((a.nout + 127) / 128) >= a.sms) return run_project_tc<T, 128, TMA>(a);
    return run_project_tc<T, 64, TMA>(a);
}

template <typename T>
bt_status launch_project_i8(const int8_t *X, const float *xs, int64_t rows, int C, const int8_t *W, const float *ws,
                            int H, int d, const int32_t *perm, const int32_t *inv, int64_t npad, void *Q, void *K,
                            void *V, cudaStream_t st)
{
    uint32_t *status = stream_status(st);
    if (!status) return BT_ERR_CUDA;
    const int hd = H * d, nout = 3 * hd;
    const QkvOut<T> out{static_cast<T *>(Q), static_cast<T *>(K), static_cast<T *>(V), hd};
    const uintptr_t ali = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(W);
    const int lb = C % 16 == 0 && ali % 16 == 0 ? 16 : C % 4 == 0 && ali % 4 == 0 ? 4 : 1;
    const uintptr_t alo = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) |
                          reinterpret_cast<uintptr_t>(V) | uintptr_t(hd * int(sizeof(T)));
    if (rows > 4 * kFewRows && alo % 16 == 0) {
        int dev = 0;
        const int sms = device_sms(&dev);
        if (sms == 0) return BT_ERR_CUDA;
        const I8Args<T> a{X, xs, rows, C, W, ws, nout, out, perm, inv, npad, lb == 16, sms, status, st};
        return lb == 16 ? launch_project_tc<T, true>(a) : launch_project_tc<T, false>(a);
    }
    if (rows <= 4 * kFewRows) {
        const unsigned grid = unsigned((nout + kFewWarps - 1) / kFewWarps);
        auto kern = lb == 16 ? k_project_i8_few<T, 16> : lb == 4 ? k_project_i8_few<T, 4> : k_project_i8_few<T, 1>;
        kern<<<grid, kFewWarps * 32, 0, st>>>(X, xs, rows, C, W, ws, nout, out, perm, inv, npad, status);
    } else {
        const dim3 grid(unsigned((rows + kTile - 1) / kTile), unsigned((nout + kTile - 1) / kTile));
        auto kern = lb == 1 ? k_project_i8_tile<T, 1> : k_project_i8_tile<T, 4>;
        kern<<<grid, 256, 0, st>>>(X, xs, rows, C, W, ws, nout, out, perm, inv, npad, status);
    }
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

}  // namespace
}  // namespace bts

using namespace bts;

extern "C" bt_status bt_qkv_project_i8(const int8_t *Xq, const float *xs, int64_t rows, int32_t C, const int8_t *Wq,
                                       const float *ws, int32_t H, int32_t d, bt_dtype dt, const int32_t *perm,
                                       const int32_t *inv, int64_t npad, void *Q, void *K, void *V, void *stream)
{
    if (rows < 0 || C < 1 || H < 1 || d < 1) return BT_ERR_ARG;
    if (dt != BT_F32 && dt != BT_BF16) return BT_ERR_ARG;
    if (perm && npad < 0) return BT_ERR_ARG;
    if (!perm) npad = rows;
    if (rows == 0 && npad == 0) return BT_OK;
    if (!Wq || !ws || !Q || !K || !V) return BT_ERR_ARG;
    if (rows > 0 && (!Xq || !xs || (perm && !inv))) return BT_ERR_ARG;
    if (rows > 0x7FFFFFFF || npad > 0x7FFFFFFF || int64_t(H) * d > 65535 / 3 || C > 65536) return BT_ERR_UNSUPPORTED;
    const uintptr_t es = dt == BT_F32 ? 4 : 2;
    const uintptr_t al = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) |
                         reinterpret_cast<uintptr_t>(V);
    const uintptr_t al4 = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws) |
                          reinterpret_cast<uintptr_t>(perm) | reinterpret_cast<uintptr_t>(inv);
    if (al % es || al4 % 4) return BT_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!perm) inv = nullptr;
    return dt == BT_F32
               ? launch_project_i8<float>(Xq, xs, rows, C, Wq, ws, H, d, perm, inv, npad, Q, K, V, st)
               : launch_project_i8<__nv_bfloat16>(Xq, xs, rows, C, Wq, ws, H, d, perm, inv, npad, Q, K, V, st);
}

namespace bts {
namespace {

constexpr size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Layout of the layer's workspace.
struct LayerWs {
    size_t xq, xs, one, inv, total;  // bytes of the 8-bit rows, their scales, one of Q, K, V, the inverse of perm
    LayerWs(int64_t npad, int64_t rows, int64_t C, int64_t hd, bt_dtype dt)
    {
        const int64_t n = npad > rows ? npad : rows;
        xq = up256(size_t(rows) * C);
        xs = up256(size_t(rows) * 4);
        one = up256(size_t(n) * hd * (dt == BT_F32 ? 4 : 2));
        inv = up256(size_t(rows) * 4);
        total = xq + xs + 3 * one + inv;
    }
};

}  // namespace
}  // namespace bts

extern "C" size_t bt_projected_i8_workspace_size(int64_t npad, int64_t rows, int32_t C, int32_t H, int32_t d,
                                                 bt_dtype dt)
{
    if (npad < 0 || rows < 0 || npad > 0x7FFFFFFF || rows > 0x7FFFFFFF || C < 1 || H < 1 || d < 1 ||
        (dt != BT_F32 && dt != BT_BF16))
        return 0;
    const size_t n = LayerWs(npad, rows, C, int64_t(H) * d, dt).total;
    return n ? n : 256;  // 0 says that the sizes are refused; an empty batch is none of those
}

extern "C" bt_status bt_projected_ball_attention_i8(const void *X, const void *R, const float *gamma, float eps,
                                                    const int32_t *perm, int64_t npad, int64_t rows, int32_t C,
                                                    const int8_t *Wq, const float *ws, int32_t m, int32_t H, int32_t d,
                                                    bt_dtype dt, void *Hout, void *O, void *work, size_t work_bytes,
                                                    void *stream)
{
    if (npad < 0 || rows < 0 || C < 1 || H < 1) return BT_ERR_ARG;
    if (dt != BT_F32 && dt != BT_BF16) return BT_ERR_ARG;
    if (m < 1 || m > 256 || (d != 32 && d != 64)) return BT_ERR_SHAPE;
    if (npad % m) return BT_ERR_SHAPE;
    if (!perm && rows < npad) return BT_ERR_ARG;
    if (rows == 0) return BT_OK;  // dummy slots write nothing
    if (!X || !Wq || !ws || !O || reinterpret_cast<uintptr_t>(O) % 16) return BT_ERR_ARG;
    const size_t need = bt_projected_i8_workspace_size(npad, rows, C, H, d, dt);
    if (need == 0) return BT_ERR_UNSUPPORTED;
    if (!work || work_bytes < need) return BT_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(work) & 255u) return BT_ERR_ARG;
    // what the steps would refuse, before the first of them is enqueued
    if (int64_t(H) * d > 65535 / 3 || C > 65536) return BT_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(perm)) % 4) return BT_ERR_ARG;
    const LayerWs l(npad, rows, C, int64_t(H) * d, dt);
    uint8_t *p = static_cast<uint8_t *>(work);
    int8_t *xq = reinterpret_cast<int8_t *>(p);
    float *xs = reinterpret_cast<float *>(p + l.xq);
    uint8_t *q = p + l.xq + l.xs, *k = q + l.one, *v = k + l.one;
    int32_t *inv = reinterpret_cast<int32_t *>(v + l.one);
    bt_status s = bt_rms_norm_i8(X, R, gamma, rows, C, eps, dt, Hout, xq, xs, stream);
    if (s != BT_OK || npad == 0) return s;
    // the shapes of bt_ball_attention_tree: whole tiles in slot order; else, and where slots are too few for the rows (an
    // inverse has no more rows than slots), the attention gathers rows
    const bool tree = perm && dt == BT_BF16 && d == 32 && H % 2 == 0 && npad >= 128 && rows <= npad && rows < 0x7FFFFFFF &&
                      (m == 16 || m == 32 || m == 64 || m == 128);
    if (tree) {
        // the workspace may hold another call's inverse: a row that no slot names must not be taken for one of its slots
        if (cudaMemsetAsync(inv, 0x80, size_t(rows) * 4, static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return BT_ERR_CUDA;
        s = bt_invert_perm(perm, npad, rows, inv, stream);
        if (s != BT_OK) return s;
        s = bt_qkv_project_i8(xq, xs, rows, C, Wq, ws, H, d, dt, perm, inv, npad, q, k, v, stream);
        if (s != BT_OK) return s;
        return bt_ball_attention_tree(q, k, v, perm, npad, rows, m, H, d, dt, O, stream);
    }
    s = bt_qkv_project_i8(xq, xs, rows, C, Wq, ws, H, d, dt, nullptr, nullptr, 0, q, k, v, stream);
    if (s != BT_OK) return s;
    return bt_ball_attention(q, k, v, perm, npad, rows, m, H, d, dt, O, stream);
}

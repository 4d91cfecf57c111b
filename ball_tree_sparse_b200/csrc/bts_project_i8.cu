// Q/K/V projection in 8-bit integers with a scale for each token (feature row) and each output channel:
//
//   out[o(r), j] = (sum_c Xq[r, c] Wq[j, c]) * xs[r] * ws[j],   o(r) = inv[r] (slot order) or r
//
// The sum is exact in 32-bit integers (C <= 65536 values of at most 128 * 128), so only the two scales and the
// output's type round.
//
//  - k_project_i8_few   few rows: a warp per output channel, which reads the channel's weights once for up to
//                       eight rows.  Bound by the weights' bytes and by latency.
//  - k_project_i8_tile  any row length or alignment, many rows: 64 x 64 tiles on the CUDA cores (dp4a).
#include <cuda_bf16.h>

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

// The output row of feature row r, or -1 (recorded) where inv names no slot.
__device__ __forceinline__ int32_t out_row(const int32_t *inv, int64_t r, int64_t npad, uint32_t *status)
{
    if (!inv) return int32_t(r);
    const int32_t o = __ldg(inv + r);
    if (o >= 0 && o < npad) return o;
    record_error(status, BT_ERR_INTERNAL);
    return -1;
}

// Zero rows of Q, K and V in the dummy slots (perm < 0), which no feature row fills: warp w of nw takes runs of
// 32 slots, and all lanes write each dummy's row.
template <typename T>
__device__ __forceinline__ void zero_dummies(const int32_t *__restrict__ perm, int64_t npad, const QkvOut<T> &out,
                                             int64_t w, int64_t nw)
{
    const int lane = threadIdx.x & 31;
    const int bytes = out.hd * int(sizeof(T));
    const uintptr_t al = reinterpret_cast<uintptr_t>(out.q) | reinterpret_cast<uintptr_t>(out.k) |
                         reinterpret_cast<uintptr_t>(out.v) | uintptr_t(bytes);
    for (int64_t s0 = w * 32; s0 < npad; s0 += nw * 32) {
        const int64_t s = s0 + lane;
        uint32_t dead = __ballot_sync(0xffffffffu, s < npad && __ldg(perm + s) < 0);
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
        zero_dummies(perm, npad, out, int64_t(blockIdx.x) * kFewWarps + (threadIdx.x >> 5),
                     int64_t(gridDim.x) * kFewWarps);
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
        zero_dummies(perm, npad, out, int64_t(blockIdx.x) * 8 + (tid >> 5), int64_t(gridDim.x) * 8);
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
    return LayerWs(npad, rows, C, int64_t(H) * d, dt).total;
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
    const LayerWs l(npad, rows, C, int64_t(H) * d, dt);
    uint8_t *p = static_cast<uint8_t *>(work);
    int8_t *xq = reinterpret_cast<int8_t *>(p);
    float *xs = reinterpret_cast<float *>(p + l.xq);
    uint8_t *q = p + l.xq + l.xs, *k = q + l.one, *v = k + l.one;
    int32_t *inv = reinterpret_cast<int32_t *>(v + l.one);
    bt_status s = bt_rms_norm_i8(X, R, gamma, rows, C, eps, dt, Hout, xq, xs, stream);
    if (s != BT_OK || npad == 0) return s;
    // the shapes of bt_ball_attention_tree: whole tiles in slot order; else the attention gathers rows
    const bool tree = perm && dt == BT_BF16 && d == 32 && H % 2 == 0 && npad >= 128 && rows < 0x7FFFFFFF &&
                      (m == 16 || m == 32 || m == 64 || m == 128);
    if (tree) {
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

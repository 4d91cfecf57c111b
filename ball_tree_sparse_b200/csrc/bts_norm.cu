// Root-mean-square norm of the feature rows, with the residual's addition, outputs in the features' type or in
// 8-bit integers with a scale per row, and the backward pass.
//
//   h = round(x + r)                      (h = x without a residual; rounded to the features' type, as stored)
//   y = h * rs * w,  rs = (mean(h^2) + eps)^(-1/2)
//   8 bits: scale = max|y| / 127,  q = rint(y / scale)
//   backward, g = w dy:  dx = rs (g - h rs^2 mean(g h)) + dh,   dw = sum over rows of dy h rs
//
// Every kernel is bound by memory: a row is read once, held in registers between the reduction and the store, and
// written once.  A row belongs to `tpr` threads (a power of two: part of a warp, a warp, or up to 8 warps), each
// holding up to NV vectors of VEC elements, vector i of thread t at element (i * tpr + t) * VEC, so that neighbouring
// threads read neighbouring bytes.  The vector is the widest that the row length and the pointers allow.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "bts_internal.cuh"

namespace bts {
namespace {

constexpr int kMaxEpt = 32;                       // elements of a row that one thread holds
constexpr int kNormThreads = 256;                 // of a block, at most; a block of more has too few registers each
constexpr int kNormMaxC = kMaxEpt * kNormThreads;  // a row's threads fit one block

template <int BYTES>
struct Raw;
template <> struct Raw<1> { using type = uint8_t; };
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

// VEC elements of T as one aligned access
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p)
{
    using R = typename Raw<int(sizeof(T)) * VEC>::type;
    union { R r; Pack<T, VEC> k; } u;
    u.r = *reinterpret_cast<const R *>(p);
    return u.k;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &k)
{
    using R = typename Raw<int(sizeof(T)) * VEC>::type;
    union { R r; Pack<T, VEC> k; } u;
    u.k = k;
    *reinterpret_cast<R *>(p) = u.r;
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC floats of the weight, in 16-byte pieces where VEC allows
template <int VEC>
__device__ __forceinline__ void load_weight(const float *w, float (&f)[VEC])
{
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 t = __ldg(reinterpret_cast<const float4 *>(w + e));
            f[e] = t.x; f[e + 1] = t.y; f[e + 2] = t.z; f[e + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = __ldg(w + e);
    }
}

// Reduction over the tpr threads of a row; every thread gets the result.  The order of the additions depends on
// tpr alone.  tpr > 32: `red` holds one value per warp, and the whole block (one row) calls it together.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int tpr, float *red)
{
    const int o0 = tpr < 32 ? tpr : 32;
    for (int o = o0 >> 1; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (tpr > 32) {
        const int nw = tpr >> 5, lane = threadIdx.x & 31;
        __syncthreads();  // the previous reduction's values are read
        if (lane == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < nw ? red[lane] : 0.0f;  // maxima are of absolute values
        for (int o = nw >> 1; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = MAX ? fmaxf(v, u) : v + u;
        }
        v = __shfl_sync(0xffffffffu, v, 0);
    }
    return v;
}

// One row per group of tpr threads.  I8: q and scale instead of Y.  norm == false: y = h (quantisation alone).
// X, R and Hout may be the same tensor: a thread reads its elements before it writes them, so these loads are
// plain ones.
template <typename T, int VEC, int NV, bool I8>
__global__ void __launch_bounds__(kNormThreads)
    k_rms_norm(const T *X, const T *R, const float *__restrict__ w, int64_t rows, int C, int tpr, float eps,
                           bool norm, T *Hout, T *Y, int8_t *Q, float *scale)
{
    __shared__ float red[32];
    const int rpb = int(blockDim.x) / tpr, t = int(threadIdx.x) % tpr;
    const int64_t row = int64_t(blockIdx.x) * rpb + int(threadIdx.x) / tpr;
    const bool live = row < rows;  // dead groups stay for the shuffles
    const size_t base = live ? size_t(row) * C : 0;

    float h[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        Pack<T, VEC> k;
        if (live && c < C) {
            k = load_pack<T, VEC>(X + base + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i * VEC + e] = widen(k.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i * VEC + e] = 0.0f;
        }
    }
    if (R) {
        Pack<T, VEC> rr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) rr[i] = load_pack<T, VEC>(R + base + c);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) {
                Pack<T, VEC> k;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    k.v[e] = narrow<T>(h[i * VEC + e] + widen(rr[i].v[e]));
                    h[i * VEC + e] = widen(k.v[e]);
                }
                if (Hout) store_pack<T, VEC>(Hout + base + c, k);
            }
        }
    }
    if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) ss = fmaf(h[i], h[i], ss);
        ss = row_reduce<false>(ss, tpr, red);
        const float rs = rsqrtf(ss / float(C) + eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
            if (w && c < C) load_weight<VEC>(w + c, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i * VEC + e] = h[i * VEC + e] * rs * f[e];
        }
    }
    if constexpr (!I8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) {
                Pack<T, VEC> k;
#pragma unroll
                for (int e = 0; e < VEC; ++e) k.v[e] = narrow<T>(h[i * VEC + e]);
                store_pack<T, VEC>(Y + base + c, k);
            }
        }
    } else {
        // a value that is not finite makes the maximum infinite: the row's scale becomes NaN and its values 0
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            const float a = fabsf(h[i]);
            mx = fmaxf(mx, a <= FLT_MAX ? a : INFINITY);
        }
        mx = row_reduce<true>(mx, tpr, red);
        const bool bad = mx > FLT_MAX;
        const float s = bad ? nanf("") : mx / 127.0f;
        if (live && t == 0) scale[row] = s;
        const bool zero = bad || s == 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) {
                Pack<int8_t, VEC> k;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float v = zero ? 0.0f : h[i * VEC + e] / s;
                    k.v[e] = int8_t(max(-127, min(127, __float2int_rn(v))));
                }
                store_pack<int8_t, VEC>(Q + base + c, k);
            }
        }
    }
}

// Backward: every group of threads walks rows blockIdx.x * rpb + group, + gridDim.x * rpb, ...; a thread adds up
// its columns' part of dw in registers, the block's groups add theirs in shared memory in the order of the groups,
// and the block writes one row of `part` ([gridDim.x][C]).  k_norm_dw adds those rows in order, so that equal
// calls give equal bits.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kNormThreads)
    k_rms_norm_bwd(const T *dY, const T *dH, const T *H, const float *__restrict__ w, int64_t rows, int C,
                               int tpr, float eps, T *dX, float *__restrict__ part)
{
    extern __shared__ float acc_sm[];  // [groups][C] while the block's groups are joined
    __shared__ float red[32];
    const int rpb = int(blockDim.x) / tpr, t = int(threadIdx.x) % tpr, grp = int(threadIdx.x) / tpr;
    float dw[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) dw[i] = 0.0f;
    const int64_t step = int64_t(gridDim.x) * rpb;
    // the block's groups take the same number of turns, so that the reductions find every thread
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < rows; r0 += step) {
        const int64_t row = r0 + grp;
        const bool live = row < rows;
        const size_t base = live ? size_t(row) * C : 0;
        Pack<T, VEC> hk[NV], yk[NV], uk[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) {
                hk[i] = load_pack<T, VEC>(H + base + c);
                yk[i] = load_pack<T, VEC>(dY + base + c);
                if (dH) uk[i] = load_pack<T, VEC>(dH + base + c);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) hk[i].v[e] = yk[i].v[e] = narrow<T>(0.0f);
            }
        }
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
            if (w && c < C) load_weight<VEC>(w + c, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float h = widen(hk[i].v[e]);
                ss = fmaf(h, h, ss);
                gh = fmaf(widen(yk[i].v[e]) * f[e], h, gh);
            }
        }
        ss = row_reduce<false>(ss, tpr, red);
        gh = row_reduce<false>(gh, tpr, red);
        const float rs = rsqrtf(ss / float(C) + eps);
        const float k2 = rs * rs * (gh / float(C));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < C) {
                float f[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
                if (w) load_weight<VEC>(w + c, f);
                Pack<T, VEC> k;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = widen(hk[i].v[e]), y = widen(yk[i].v[e]);
                    float x = rs * (y * f[e] - h * k2);
                    if (dH) x += widen(uk[i].v[e]);
                    k.v[e] = narrow<T>(x);
                    dw[i * VEC + e] = fmaf(y, h * rs, dw[i * VEC + e]);
                }
                store_pack<T, VEC>(dX + base + c, k);
            }
        }
    }
    if (!part) return;
    float *out = part + size_t(blockIdx.x) * C;
    if (rpb == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (c < C)
#pragma unroll
                for (int e = 0; e < VEC; ++e) out[c + e] = dw[i * VEC + e];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        if (c < C)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc_sm[grp * C + c + e] = dw[i * VEC + e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        float a = 0.0f;
        for (int g = 0; g < rpb; ++g) a += acc_sm[g * C + c];
        out[c] = a;
    }
}

// dw[c] = sum over the n rows of part: a warp's lanes hold 32 columns, the block's 32 warps every 32nd row.
__global__ void __launch_bounds__(1024) k_norm_dw(const float *__restrict__ part, int n, int C, float *__restrict__ dw)
{
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (c < C)
#pragma unroll 4
        for (int r = wy; r < n; r += 32) a += part[size_t(r) * C + c];
    sm[wy][lane] = a;
    __syncthreads();
    // warp wy adds column wy of the block: one value per lane
    float v = sm[lane][wy];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 32 + wy < C) dw[blockIdx.x * 32 + wy] = v;
}

struct NormShape {
    int vec, nv, tpr, threads;
};

// The widest vector that C and the addresses allow; then as few threads per row as hold it in NV <= 32 / VEC
// vectors each when there are rows enough to fill the SMs, else as many as the row has vectors.
template <typename T>
NormShape norm_shape(int64_t rows, int C, uintptr_t al, uintptr_t al_q, uintptr_t al_w)
{
    const int es = int(sizeof(T));
    NormShape s;
    s.vec = 1;
    for (int v = 16 / es; v > 1; v >>= 1) {
        if (es == 2 && v == 4) continue;  // not instantiated
        if (es == 4 && v == 2) continue;
        if (C % v == 0 && al % uintptr_t(v * es) == 0 && al_q % uintptr_t(v) == 0 &&
            al_w % uintptr_t(v >= 4 ? 16 : 4) == 0) {
            s.vec = v;
            break;
        }
    }
    const int cv = C / s.vec;                      // vectors per row
    const int most = kMaxEpt / s.vec;              // vectors per thread
    int tpr = 1;
    while (tpr * most < cv) tpr <<= 1;
    // few rows: spread each over more threads, down to one vector each
    while (tpr < cv && tpr < kNormThreads && rows * tpr < 148 * 512) tpr <<= 1;
    s.tpr = tpr;
    s.threads = tpr > 32 ? tpr : kNormThreads;  // a row of more than a warp has the block to itself
    const int need = (cv + tpr - 1) / tpr;
    s.nv = need <= 1 ? 1 : need <= most / 4 ? most / 4 : most;
    if (s.nv < 1) s.nv = 1;
    return s;
}

template <typename T, int VEC, int NV, bool I8>
bt_status run_norm(const NormShape &s, const void *X, const void *R, const float *w, int64_t rows, int C, float eps,
                   bool norm, void *Hout, void *Y, int8_t *Q, float *scale, cudaStream_t st)
{
    const int rpb = s.threads / s.tpr;
    const int64_t grid = (rows + rpb - 1) / rpb;
    if (grid > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    k_rms_norm<T, VEC, NV, I8><<<unsigned(grid), s.threads, 0, st>>>(
        static_cast<const T *>(X), static_cast<const T *>(R), w, rows, C, s.tpr, eps, norm, static_cast<T *>(Hout),
        static_cast<T *>(Y), Q, scale);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <typename T, bool I8>
bt_status launch_norm(const void *X, const void *R, const float *w, int64_t rows, int C, float eps, bool norm,
                      void *Hout, void *Y, int8_t *Q, float *scale, cudaStream_t st)
{
    const uintptr_t al = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(R) |
                         reinterpret_cast<uintptr_t>(Hout) | reinterpret_cast<uintptr_t>(Y);
    const NormShape s = norm_shape<T>(rows, C, al, reinterpret_cast<uintptr_t>(Q), reinterpret_cast<uintptr_t>(w));
#define BTS_NORM(V, N)                                                                                     \
    if (s.vec == V && s.nv == N)                                                                           \
        return run_norm<T, V, N, I8>(s, X, R, w, rows, C, eps, norm, Hout, Y, Q, scale, st);
    if constexpr (sizeof(T) == 2) {
        BTS_NORM(8, 1) BTS_NORM(8, 4) BTS_NORM(2, 1) BTS_NORM(2, 4) BTS_NORM(2, 16)
    } else {
        BTS_NORM(4, 1) BTS_NORM(4, 2) BTS_NORM(4, 8)
    }
    BTS_NORM(1, 1) BTS_NORM(1, 8) BTS_NORM(1, 32)
#undef BTS_NORM
    return BT_ERR_INTERNAL;
}

constexpr int kBwdBlocks = 148 * 4;  // rows of partial sums of dw

template <typename T, int VEC, int NV>
bt_status run_bwd(const NormShape &s, const void *dY, const void *dH, const void *H, const float *w, int64_t rows,
                  int C, float eps, void *dX, float *part, int64_t blocks, cudaStream_t st)
{
    const int rpb = s.threads / s.tpr;
    const size_t smem = part && rpb > 1 ? size_t(rpb) * C * 4 : 0;
    // rpb * C <= threads / tpr * tpr * 32 values: at most 32 KB
    k_rms_norm_bwd<T, VEC, NV><<<unsigned(blocks), s.threads, smem, st>>>(
        static_cast<const T *>(dY), static_cast<const T *>(dH), static_cast<const T *>(H), w, rows, C, s.tpr, eps,
        static_cast<T *>(dX), part);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <typename T>
bt_status launch_bwd(const void *dY, const void *dH, const void *H, const float *w, int64_t rows, int C, float eps,
                     void *dX, float *dw, float *part, cudaStream_t st)
{
    const uintptr_t al = reinterpret_cast<uintptr_t>(dY) | reinterpret_cast<uintptr_t>(dH) |
                         reinterpret_cast<uintptr_t>(H) | reinterpret_cast<uintptr_t>(dX);
    int64_t blocks = 0;
    if (rows > 0) {
        const NormShape s = norm_shape<T>(rows, C, al, 0, reinterpret_cast<uintptr_t>(w));
        const int rpb = s.threads / s.tpr;
        blocks = (rows + rpb - 1) / rpb;
        if (blocks > kBwdBlocks) blocks = kBwdBlocks;
        bt_status r = BT_ERR_INTERNAL;
#define BTS_BWD(V, N) \
    if (s.vec == V && s.nv == N) r = run_bwd<T, V, N>(s, dY, dH, H, w, rows, C, eps, dX, dw ? part : nullptr, blocks, st);
        if constexpr (sizeof(T) == 2) {
            BTS_BWD(8, 1) BTS_BWD(8, 4) BTS_BWD(2, 1) BTS_BWD(2, 4) BTS_BWD(2, 16)
        } else {
            BTS_BWD(4, 1) BTS_BWD(4, 2) BTS_BWD(4, 8)
        }
        BTS_BWD(1, 1) BTS_BWD(1, 8) BTS_BWD(1, 32)
#undef BTS_BWD
        if (r != BT_OK) return r;
    }
    if (dw) k_norm_dw<<<unsigned((C + 31) / 32), 1024, 0, st>>>(part, int(blocks), C, dw);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

// element alignment of a tensor's address
bool aligned(const void *p, int es) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(es) == 0; }

bt_status norm_args(const void *X, const void *R, const float *w, int64_t rows, int32_t C, float eps, bt_dtype dt,
                    const void *Hout)
{
    if (rows < 0 || C < 1 || !(eps >= 0.0f) || eps > FLT_MAX) return BT_ERR_ARG;
    if (dt != BT_F32 && dt != BT_BF16) return BT_ERR_ARG;
    if (rows > 0 && !X) return BT_ERR_ARG;
    if (Hout && !R) return BT_ERR_ARG;  // without a residual the stream is X
    const int es = dt == BT_F32 ? 4 : 2;
    if (!aligned(X, es) || !aligned(R, es) || !aligned(Hout, es) || !aligned(w, 4)) return BT_ERR_ARG;
    if (C > kNormMaxC) return BT_ERR_UNSUPPORTED;
    return BT_OK;
}

}  // namespace
}  // namespace bts

using namespace bts;

extern "C" bt_status bt_rms_norm(const void *X, const void *R, const float *w, int64_t rows, int32_t C, float eps,
                                 bt_dtype dt, void *Hout, void *Y, void *stream)
{
    const bt_status a = norm_args(X, R, w, rows, C, eps, dt, Hout);
    if (a != BT_OK) return a;
    if (rows == 0) return BT_OK;
    if (!Y || !aligned(Y, dt == BT_F32 ? 4 : 2)) return BT_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == BT_F32 ? launch_norm<float, false>(X, R, w, rows, C, eps, true, Hout, Y, nullptr, nullptr, st)
                        : launch_norm<__nv_bfloat16, false>(X, R, w, rows, C, eps, true, Hout, Y, nullptr, nullptr, st);
}

extern "C" bt_status bt_rms_norm_i8(const void *X, const void *R, const float *w, int64_t rows, int32_t C, float eps,
                                    bt_dtype dt, void *Hout, int8_t *Yq, float *scale, void *stream)
{
    const bt_status a = norm_args(X, R, w, rows, C, eps, dt, Hout);
    if (a != BT_OK) return a;
    if (rows == 0) return BT_OK;
    if (!Yq || !scale || !aligned(scale, 4)) return BT_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == BT_F32 ? launch_norm<float, true>(X, R, w, rows, C, eps, true, Hout, nullptr, Yq, scale, st)
                        : launch_norm<__nv_bfloat16, true>(X, R, w, rows, C, eps, true, Hout, nullptr, Yq, scale, st);
}

extern "C" bt_status bt_quantize_i8(const void *X, int64_t rows, int32_t C, bt_dtype dt, int8_t *Xq, float *scale,
                                    void *stream)
{
    const bt_status a = norm_args(X, nullptr, nullptr, rows, C, 0.0f, dt, nullptr);
    if (a != BT_OK) return a;
    if (rows == 0) return BT_OK;
    if (!Xq || !scale || !aligned(scale, 4)) return BT_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == BT_F32
               ? launch_norm<float, true>(X, nullptr, nullptr, rows, C, 0.0f, false, nullptr, nullptr, Xq, scale, st)
               : launch_norm<__nv_bfloat16, true>(X, nullptr, nullptr, rows, C, 0.0f, false, nullptr, nullptr, Xq,
                                                  scale, st);
}

extern "C" size_t bt_rms_norm_backward_workspace_size(int64_t rows, int32_t C)
{
    if (rows < 0 || C < 1 || C > kNormMaxC) return 0;
    const int64_t n = rows < 1 ? 1 : rows < kBwdBlocks ? rows : kBwdBlocks;
    return (size_t(n) * C * 4 + 255) & ~size_t(255);
}

extern "C" bt_status bt_rms_norm_backward(const void *dY, const void *dH, const void *H, const float *w, int64_t rows,
                                          int32_t C, float eps, bt_dtype dt, void *dX, float *dw, void *ws,
                                          size_t ws_bytes, void *stream)
{
    const bt_status a = norm_args(H, nullptr, w, rows, C, eps, dt, nullptr);
    if (a != BT_OK) return a;
    const int es = dt == BT_F32 ? 4 : 2;
    if (rows > 0 && (!dY || !dX)) return BT_ERR_ARG;
    if (!aligned(dY, es) || !aligned(dH, es) || !aligned(dX, es) || !aligned(dw, 4)) return BT_ERR_ARG;
    if (dw) {  // the partial sums of dw
        if (!ws || ws_bytes < bt_rms_norm_backward_workspace_size(rows, C)) return BT_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(ws) & 255u) return BT_ERR_ARG;
    }
    if (rows == 0 && !dw) return BT_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == BT_F32 ? launch_bwd<float>(dY, dH, H, w, rows, C, eps, dX, dw, static_cast<float *>(ws), st)
                        : launch_bwd<__nv_bfloat16>(dY, dH, H, w, rows, C, eps, dX, dw, static_cast<float *>(ws), st);
}

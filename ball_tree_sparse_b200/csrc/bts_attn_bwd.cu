// Backward pass of ball attention, with the probabilities recomputed.
//
// For every ball and head, over the ball's real rows i (query) and j (key), with the gradient dO of the output:
//
//   s_ij = q_i . k_j / sqrt(d),  p_ij = exp(s_ij - max_j s_ij) / sum_j exp(s_ij - max_j s_ij)
//   dV_j = sum_i p_ij dO_i
//   dP_ij = dO_i . v_j,  delta_i = sum_j p_ij dP_ij,  dS_ij = p_ij (dP_ij - delta_i)
//   dQ_i = sum_j dS_ij k_j / sqrt(d),  dK_j = sum_i dS_ij q_i / sqrt(d)
//
// A ball's keys all fit one tile, so a row's maximum, sum and delta come from the tile itself: the pass needs
// neither the forward output nor statistics kept by it, and reads Q, K, V and dO and writes dQ, dK and dV once.
//
// k_ball_bwd_simt  float (any m), and bf16 balls of more than 128 slots: CUDA cores, everything in float.
#include <cuda_bf16.h>

#include <cmath>

#include "bts_internal.cuh"
#include "bts_tc.cuh"
#include "bts_maps.cuh"

namespace bts {
namespace {

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}
__device__ __forceinline__ bool finite4(const float4 &v)
{
    return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
}

// ---------------------------------------------------------------------------
// CUDA cores.  One CTA per (tile, head).  A tile is MP slots' room for as many whole balls as fit (one where
// m > MP / 2); its K and V stay in shared memory in float, and its queries come 32 at a time:
//   A  S and dP of 32 queries x MP keys: warp w has rows w, w + NW, ...; lane l the keys l, l + 32, ..., so a row's
//      statistics are warp reductions.  P and dS go to shared memory.
//   B  dV += P^T dO and dK += dS^T Q: a thread keeps KPT keys x 4 columns of each over all queries.
//   C  dQ = dS K of the 32 queries.
// Rows are padded by 16 bytes, which keeps the 16-byte accesses of A, B and C free of bank conflicts.
// Bound by the float pipe and shared-memory loads together (A: 40 cycles of loads to 32 of products).
// ---------------------------------------------------------------------------
template <int D, int MP>
struct BwdSimt {
    static constexpr int QT = 32;
    static constexpr int NT = MP <= 64 ? 128 : 256;
    static constexpr int LD = D + 4, LP = MP + 4;
    static constexpr int NW = NT / 32, RPW = QT / NW, CPL = MP / 32;
    static constexpr int DG = D / 4, NKG = NT / DG, KPT = MP / NKG;
    static constexpr size_t BYTES = sizeof(float) * (2 * MP * LD + 2 * QT * LD + 2 * QT * LP) + 4 * MP;
};

template <typename T, int D, int MP>
__global__ void __launch_bounds__(BwdSimt<D, MP>::NT)
    k_ball_bwd_simt(const T *__restrict__ Q, const T *__restrict__ K, const T *__restrict__ V,
                    const T *__restrict__ dO, const int32_t *__restrict__ perm, int64_t npad, int64_t rows, int m,
                    int spt, int H, float scale, T *__restrict__ dQ, T *__restrict__ dK, T *__restrict__ dV,
                    uint32_t *status)
{
    using L = BwdSimt<D, MP>;
    constexpr int LD = L::LD, LP = L::LP;
    extern __shared__ __align__(16) float bsm[];
    float *sK = bsm, *sV = sK + MP * LD, *sQ = sV + MP * LD, *sG = sQ + L::QT * LD;  // sG: rows of dO
    float *sP = sG + L::QT * LD, *sS = sP + L::QT * LP;                              // P and dS
    int32_t *sRow = reinterpret_cast<int32_t *>(sS + L::QT * LP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = int(blockIdx.x) % H;
    const int64_t tile = int64_t(blockIdx.x) / H;
    const size_t hs = size_t(H) * D;

    bool any = false;
    for (int j = tid; j < MP; j += L::NT) {
        const int64_t slot = tile * spt + j;
        int32_t r = -1;
        if (j < spt && slot < npad) r = perm ? perm[slot] : int32_t(slot);
        if (r >= rows) {  // not a row of the tensors: never read or write it
            if (h == 0) record_error(status, BT_ERR_INTERNAL);
            r = -1;
        }
        sRow[j] = r < 0 ? -1 : r;
        any |= r >= 0;
    }
    if (!__syncthreads_or(any)) return;  // a tile of dummies
    bool odd = false;  // some value is not finite: 0 * value must not reach another ball
    for (int e = tid; e < MP * L::DG; e += L::NT) {
        const int j = e / L::DG, c = (e - j * L::DG) * 4;
        const int32_t r = sRow[j];
        float4 kv = make_float4(0, 0, 0, 0), vv = kv;
        if (r >= 0) {
            kv = load4(K + size_t(r) * hs + h * D + c);
            vv = load4(V + size_t(r) * hs + h * D + c);
        }
        odd |= !finite4(kv);
        *reinterpret_cast<float4 *>(sK + j * LD + c) = kv;
        *reinterpret_cast<float4 *>(sV + j * LD + c) = vv;
    }
    const int kg = tid / L::DG, c0 = (tid - kg * L::DG) * 4;  // phase B: keys kg * KPT .., columns c0 ..
    float av[L::KPT][4], ak[L::KPT][4];
#pragma unroll
    for (int i = 0; i < L::KPT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) av[i][e] = ak[i][e] = 0.0f;

    for (int q0 = 0; q0 < spt; q0 += L::QT) {
        for (int e = tid; e < L::QT * L::DG; e += L::NT) {
            const int j = e / L::DG, c = (e - j * L::DG) * 4;
            const int32_t r = q0 + j < MP ? sRow[q0 + j] : -1;
            float4 qv = make_float4(0, 0, 0, 0), gv = qv;
            if (r >= 0) {
                qv = load4(Q + size_t(r) * hs + h * D + c);
                gv = load4(dO + size_t(r) * hs + h * D + c);
            }
            odd |= !finite4(qv) || !finite4(gv);
            *reinterpret_cast<float4 *>(sQ + j * LD + c) = qv;
            *reinterpret_cast<float4 *>(sG + j * LD + c) = gv;
        }
        const bool guard = __syncthreads_or(odd) && spt > m;
        {
            float s[L::RPW][L::CPL], g[L::RPW][L::CPL];
#pragma unroll
            for (int i = 0; i < L::RPW; ++i)
#pragma unroll
                for (int j = 0; j < L::CPL; ++j) s[i][j] = g[i][j] = 0.0f;
#pragma unroll 2
            for (int k = 0; k < D; k += 4) {
                float4 qv[L::RPW], gv[L::RPW];
#pragma unroll
                for (int i = 0; i < L::RPW; ++i) {
                    qv[i] = *reinterpret_cast<const float4 *>(sQ + (warp + i * L::NW) * LD + k);
                    gv[i] = *reinterpret_cast<const float4 *>(sG + (warp + i * L::NW) * LD + k);
                }
#pragma unroll
                for (int j = 0; j < L::CPL; ++j) {
                    const float4 kv = *reinterpret_cast<const float4 *>(sK + (lane + 32 * j) * LD + k);
                    const float4 vv = *reinterpret_cast<const float4 *>(sV + (lane + 32 * j) * LD + k);
#pragma unroll
                    for (int i = 0; i < L::RPW; ++i) {
                        s[i][j] = fmaf(qv[i].x, kv.x, s[i][j]);
                        s[i][j] = fmaf(qv[i].y, kv.y, s[i][j]);
                        s[i][j] = fmaf(qv[i].z, kv.z, s[i][j]);
                        s[i][j] = fmaf(qv[i].w, kv.w, s[i][j]);
                        g[i][j] = fmaf(gv[i].x, vv.x, g[i][j]);
                        g[i][j] = fmaf(gv[i].y, vv.y, g[i][j]);
                        g[i][j] = fmaf(gv[i].z, vv.z, g[i][j]);
                        g[i][j] = fmaf(gv[i].w, vv.w, g[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < L::RPW; ++i) {
                const int ri = warp + i * L::NW, r = q0 + ri;
                const bool qok = r < MP && sRow[r < MP ? r : 0] >= 0;
                const int b0 = (r / m) * m;
                uint32_t ok = 0;
#pragma unroll
                for (int j = 0; j < L::CPL; ++j) {
                    const int key = lane + 32 * j;
                    if (qok && key >= b0 && key < b0 + m && sRow[key] >= 0) ok |= 1u << j;
                }
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < L::CPL; ++j)
                    if ((ok >> j) & 1u) mx = fmaxf(mx, s[i][j] * scale);
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                float den = 0.0f, dl = 0.0f;
#pragma unroll
                for (int j = 0; j < L::CPL; ++j) {
                    const bool on = (ok >> j) & 1u;
                    s[i][j] = on ? expf(s[i][j] * scale - mx) : 0.0f;
                    den += s[i][j];
                    if (on) dl = fmaf(s[i][j], g[i][j], dl);
                }
                for (int o = 16; o > 0; o >>= 1) {
                    den += __shfl_xor_sync(0xffffffffu, den, o);
                    dl += __shfl_xor_sync(0xffffffffu, dl, o);
                }
                const float inv = qok ? 1.0f / den : 0.0f;  // a real query is a key of its own ball: den >= 1
                const float delta = dl * inv;
#pragma unroll
                for (int j = 0; j < L::CPL; ++j) {
                    const float p = s[i][j] * inv;
                    sP[ri * LP + lane + 32 * j] = p;
                    sS[ri * LP + lane + 32 * j] = (ok >> j) & 1u ? p * (g[i][j] - delta) : 0.0f;
                }
            }
        }
        __syncthreads();
        // B
        if (!guard) {
#pragma unroll 2
            for (int q = 0; q < L::QT; ++q) {
                const float4 gv = *reinterpret_cast<const float4 *>(sG + q * LD + c0);
                const float4 qv = *reinterpret_cast<const float4 *>(sQ + q * LD + c0);
                float p[L::KPT], s[L::KPT];
                if constexpr (L::KPT >= 4) {
#pragma unroll
                    for (int i = 0; i < L::KPT; i += 4) {
                        *reinterpret_cast<float4 *>(p + i) =
                            *reinterpret_cast<const float4 *>(sP + q * LP + kg * L::KPT + i);
                        *reinterpret_cast<float4 *>(s + i) =
                            *reinterpret_cast<const float4 *>(sS + q * LP + kg * L::KPT + i);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < L::KPT; ++i) {
                        p[i] = sP[q * LP + kg * L::KPT + i];
                        s[i] = sS[q * LP + kg * L::KPT + i];
                    }
                }
#pragma unroll
                for (int i = 0; i < L::KPT; ++i) {
                    av[i][0] = fmaf(p[i], gv.x, av[i][0]);
                    av[i][1] = fmaf(p[i], gv.y, av[i][1]);
                    av[i][2] = fmaf(p[i], gv.z, av[i][2]);
                    av[i][3] = fmaf(p[i], gv.w, av[i][3]);
                    ak[i][0] = fmaf(s[i], qv.x, ak[i][0]);
                    ak[i][1] = fmaf(s[i], qv.y, ak[i][1]);
                    ak[i][2] = fmaf(s[i], qv.z, ak[i][2]);
                    ak[i][3] = fmaf(s[i], qv.w, ak[i][3]);
                }
            }
        } else {
            for (int q = 0; q < L::QT; ++q)
#pragma unroll
                for (int i = 0; i < L::KPT; ++i)
                    if ((q0 + q) / m == (kg * L::KPT + i) / m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            av[i][e] = fmaf(sP[q * LP + kg * L::KPT + i], sG[q * LD + c0 + e], av[i][e]);
                            ak[i][e] = fmaf(sS[q * LP + kg * L::KPT + i], sQ[q * LD + c0 + e], ak[i][e]);
                        }
        }
        // C
        for (int u = tid; u < L::QT * L::DG; u += L::NT) {
            const int ri = u / L::DG, c = (u - ri * L::DG) * 4;
            const int32_t r = q0 + ri < MP ? sRow[q0 + ri] : -1;
            if (r < 0) continue;
            const int b0 = guard ? ((q0 + ri) / m) * m : 0, b1 = guard ? b0 + m : MP;
            float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (!guard) {
#pragma unroll 2
                for (int j = 0; j < MP; j += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(sS + ri * LP + j);
                    const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 kv = *reinterpret_cast<const float4 *>(sK + (j + e) * LD + c);
                        a[0] = fmaf(ws[e], kv.x, a[0]);
                        a[1] = fmaf(ws[e], kv.y, a[1]);
                        a[2] = fmaf(ws[e], kv.z, a[2]);
                        a[3] = fmaf(ws[e], kv.w, a[3]);
                    }
                }
            } else {
                for (int j = b0; j < b1; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = fmaf(sS[ri * LP + j], sK[j * LD + c + e], a[e]);
            }
            store4(dQ + size_t(r) * hs + h * D + c, a[0] * scale, a[1] * scale, a[2] * scale, a[3] * scale);
        }
        __syncthreads();  // Q, dO, P and dS are read
    }
#pragma unroll
    for (int i = 0; i < L::KPT; ++i) {
        const int32_t r = sRow[kg * L::KPT + i];
        if (r < 0) continue;
        store4(dV + size_t(r) * hs + h * D + c0, av[i][0], av[i][1], av[i][2], av[i][3]);
        store4(dK + size_t(r) * hs + h * D + c0, ak[i][0] * scale, ak[i][1] * scale, ak[i][2] * scale,
               ak[i][3] * scale);
    }
}

struct BwdArgs {
    const void *Q, *K, *V, *dO;
    const int32_t *perm;
    int64_t npad, rows;
    int m, H;
    void *dQ, *dK, *dV;
    cudaStream_t st;
};

template <typename T, int D, int MP>
bt_status run_simt(const BwdArgs &a)
{
    constexpr size_t smem = BwdSimt<D, MP>::BYTES;
    static std::atomic<bool> set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BT_ERR_CUDA;
    if (dev < 0 || dev >= 64) return BT_ERR_UNSUPPORTED;
    const bt_status s = setup_once(set[dev], [&]() -> bt_status {
        return cudaFuncSetAttribute(k_ball_bwd_simt<T, D, MP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(smem)) == cudaSuccess
                   ? BT_OK
                   : BT_ERR_CUDA;
    });
    if (s != BT_OK) return s;
    uint32_t *status = stream_status(a.st);
    if (!status) return BT_ERR_CUDA;
    const int spt = MP / a.m * a.m;  // slots of a tile: whole balls
    const int64_t grid = (a.npad + spt - 1) / spt * a.H;
    if (grid > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    k_ball_bwd_simt<T, D, MP><<<unsigned(grid), BwdSimt<D, MP>::NT, smem, a.st>>>(
        static_cast<const T *>(a.Q), static_cast<const T *>(a.K), static_cast<const T *>(a.V),
        static_cast<const T *>(a.dO), a.perm, a.npad, a.rows, a.m, spt, a.H, 1.0f / sqrtf(float(D)),
        static_cast<T *>(a.dQ), static_cast<T *>(a.dK), static_cast<T *>(a.dV), status);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <typename T, int D>
bt_status launch_simt(const BwdArgs &a)
{
    if (a.m <= 32) return run_simt<T, D, 32>(a);
    if (a.m <= 64) return run_simt<T, D, 64>(a);
    if (a.m <= 128) return run_simt<T, D, 128>(a);
    return run_simt<T, D, 256>(a);
}

}  // namespace
}  // namespace bts

using namespace bts;

extern "C" bt_status bt_ball_attention_backward(const void *Q, const void *K, const void *V, const void *dO,
                                                const int32_t *perm, int64_t npad, int64_t rows, int32_t m, int32_t H,
                                                int32_t d, bt_dtype dt, void *dQ, void *dK, void *dV, void *stream)
{
    if (npad < 0 || rows < 0 || H < 1) return BT_ERR_ARG;
    if (m < 1 || m > 256 || (d != 32 && d != 64)) return BT_ERR_SHAPE;
    if (npad % m) return BT_ERR_SHAPE;
    if (dt != BT_F32 && dt != BT_BF16) return BT_ERR_ARG;
    if (!perm && rows < npad) return BT_ERR_ARG;
    if (npad == 0 || rows == 0) return BT_OK;  // no slot, or no row that a slot could name
    if (!Q || !K || !V || !dO || !dQ || !dK || !dV) return BT_ERR_ARG;
    if (npad > 0x7FFFFFFF || rows >= 0x7FFFFFFF || H > 65535) return BT_ERR_UNSUPPORTED;
    const uintptr_t al = reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K) |
                         reinterpret_cast<uintptr_t>(V) | reinterpret_cast<uintptr_t>(dO) |
                         reinterpret_cast<uintptr_t>(dQ) | reinterpret_cast<uintptr_t>(dK) |
                         reinterpret_cast<uintptr_t>(dV);
    if (al % 16 || reinterpret_cast<uintptr_t>(perm) % 4) return BT_ERR_ARG;
    const BwdArgs a{Q, K, V, dO, perm, npad, rows, m, H, dQ, dK, dV, static_cast<cudaStream_t>(stream)};
    if (dt == BT_F32) return d == 32 ? launch_simt<float, 32>(a) : launch_simt<float, 64>(a);
    return d == 32 ? launch_simt<__nv_bfloat16, 32>(a) : launch_simt<__nv_bfloat16, 64>(a);
}

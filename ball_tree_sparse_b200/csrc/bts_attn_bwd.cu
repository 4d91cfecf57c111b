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
// k_ball_bwd_tc    bf16, m <= 128: tcgen05 tensor cores, persistent CTAs, rows gathered by TMA.
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

// ---------------------------------------------------------------------------
// Tensor cores.  A tile is up to 128 slots (as many whole balls as fit); the CTAs are persistent, one per SM.
//   warps 0-7   group 0, warps 8-15 group 1: a group works on one head of a tile at a time, two threads per query row
//               (TMEM lane), 64 keys each;
//   warps 16, 17  producers: load perm and gather the rows of Q, K, V and dO by TMA (tile::gather4, 128-byte pieces,
//               128-byte swizzle) into a stage.
// d = 32: the two groups take the two heads of a pair, whose 64 bytes of a row are one piece (an item: tile, pair);
// two stages, one producer.  d = 64: every group has its own items (tile, head), one stage and a producer, so that one
// group computes while the other one's rows arrive.
// Per head:
//   S = Q K^T and dP = dO V^T           TMEM columns [0, 128) and [128, 256) of the group
//   e = exp2(s - own max), sums of e and e dP over the thread's 64 keys, joined with the other half's through
//   shared memory; P = e / sum as bf16 into the group's 32 KB of shared memory ([query][key], two blocks of 64 keys,
//   128-byte swizzle); dS = P (dP - delta) as bf16 into TMEM over S
//   dV = P^T dO                         A read transposed (MN-major); beside dS
//   dQ = dS K                           A from TMEM; over dP
//   dS to shared memory over P once dV is done
//   dK = dS^T Q                         beside dQ
// P and dS take turns in one buffer, because two would leave no room for the second stage.  While one group waits for
// the tensor cores, the other one computes; dV is stored while dK is computed, and dQ and dK while the next item's S
// and dP are.
// A key of another ball or a dummy has P = dS = 0.  Where a tile holds several balls, a value of one ball that is not
// finite would still reach the others as 0 * value: a result that is not finite is therefore summed again over the
// ball's own slots (`mend`).
// ---------------------------------------------------------------------------
template <int D>
struct BwdTc {
    static constexpr bool OWN = D == 64;                  // a group has its own items, stage and producer
    static constexpr uint32_t TENSOR = 128 * 128;         // one of Q, K, V, dO of a stage: 128 rows of 128 bytes
    static constexpr uint32_t STAGE = 4 * TENSOR;
    static constexpr uint32_t BLK = 128 * 128;            // 128 queries, 64 keys of P or dS
    static constexpr uint32_t PBUF = 2 * BLK;
    static constexpr uint32_t P_OFF = 2 * STAGE;
    static constexpr uint32_t BYTES = P_OFF + 2 * PBUF + 1024;
    static constexpr int THREADS = 640;
    // Registers of a thread: at launch, then of a group's threads and of a producer's (setmaxnreg).
    static constexpr int REGS = 96, REGS_G = 112, REGS_P = 32;
    static_assert(512 * REGS_G + 128 * REGS_P <= THREADS * REGS, "the split is of what the block was launched with");
};

__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_ld_nowait(uint32_t taddr, uint32_t (&r)[N])
{
    if constexpr (N == 16) tmem_ld16_nowait(taddr, r);
    else tmem_ld32_nowait(taddr, r);
}

// Barrier of one group's 256 threads.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 256;" ::"r"(g + 1) : "memory"); }

// The same, and whether `p` holds for any of them.
__device__ __forceinline__ bool group_any(int g, bool p)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tbar.red.or.pred b, %1, 256, a;\n\t"
                 "selp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(r)
                 : "r"(g + 1), "r"(uint32_t(p))
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&t);
}

// Byte offset of element (row, col) of a [128][64] bf16 block with 128-byte swizzle
__device__ __forceinline__ uint32_t swz(int row, int col)
{
    return uint32_t(row * 128 + ((((col >> 3) ^ (row & 7)) << 4) | ((col & 7) << 1)));
}

template <int D>
__global__ void __launch_bounds__(BwdTc<D>::THREADS, 1)
    k_ball_bwd_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                  const int32_t *__restrict__ perm, int64_t npad, int64_t rows, int m, int spt, int H, float scale,
                  float sl2, int items, __nv_bfloat16 *__restrict__ dQ, __nv_bfloat16 *__restrict__ dK,
                  __nv_bfloat16 *__restrict__ dV, uint32_t *status)
{
    using L = BwdTc<D>;
    constexpr bool OWN = L::OWN;
    constexpr int HALF_D = D / 2;
    constexpr uint32_t SBO = 1024, SW128 = 2, MN_A = 1u << 15;
    constexpr uint32_t IDESC_S = idesc_bf16(128, false);        // S, dP
    constexpr uint32_t IDESC_Q = idesc_bf16(D, true);           // dQ: A as it lies in TMEM
    constexpr uint32_t IDESC_T = idesc_bf16(D, true) | MN_A;    // dV, dK: A transposed
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ __align__(8) uint64_t sFull[2], sEmpty[2], sBarS[2], sBarG[2], sBarV[2], sBarO[2];
    __shared__ int32_t sRows[2][128];
    __shared__ uint32_t sMask[2][4];  // real slots of the tile
    __shared__ int32_t sItem[2];      // -1: no more work
    __shared__ float sX[2][2][3][128];  // per group and half: a row's max, sum and sum of e dP
    __shared__ uint32_t sTmem;
    __shared__ int sAbort[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int HP = OWN ? H : (H + 1) >> 1;  // items of a tile
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    uint8_t *gbase = dsm + (base - smem_u32(dsm));

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sTmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < 2; ++i) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sFull[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&sEmpty[i])), "r"(OWN ? 1 : 2)
                         : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sBarS[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sBarG[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sBarV[i])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&sBarO[i])) : "memory");
            sAbort[i] = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sTmem;

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REGS_P));
        // ---------------- producer: lane l has rows 4l .. 4l+3 of the tile ----------------
        const int g = warp - 16;
        if (g < (OWN ? 2 : 1)) {  // the other warps fill their warpgroup
            constexpr int NS = OWN ? 1 : 2;  // stages of this producer
            const int first = OWN ? 2 * int(blockIdx.x) + g : int(blockIdx.x);
            const int step = (OWN ? 2 : 1) * int(gridDim.x);
            const int32_t oob = int32_t(rows);  // a row outside the tensor reads zeros
            auto load_rows = [&](int item, int32_t(&r)[4]) {
                const int64_t s0 = int64_t(item / HP) * spt + 4 * lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[i] = -1;
                    if (item < items && 4 * lane + i < spt && s0 + i < npad)
                        r[i] = perm ? __ldg(perm + s0 + i) : int32_t(s0 + i);
                }
            };
            int item = first, it = 0;
            int32_t cur[4];
            load_rows(item, cur);
            bool ok = true;
            for (; item < items && ok; item += step) {
                int32_t nxt[4];
                load_rows(item + step, nxt);  // items + step < 2^31, checked by the host
                bool live = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (cur[i] >= rows) {  // not a row of the tensors: never read or write it
                        record_error(status, BT_ERR_INTERNAL);
                        cur[i] = -1;
                    }
                    live |= cur[i] >= 0;
                }
                if (__any_sync(0xffffffffu, live)) {  // a tile of dummies has no results
                    const int st = OWN ? g : it & 1;
                    const uint32_t full = smem_u32(&sFull[st]);
                    if (it >= NS) ok = mbar_wait(smem_u32(&sEmpty[st]), ((it / NS) - 1) & 1, status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint32_t nib = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sRows[st][4 * lane + i] = cur[i];
                        nib |= uint32_t(cur[i] >= 0) << i;
                    }
                    nib <<= 4 * (lane & 7);
                    for (int o = 1; o < 8; o <<= 1) nib |= __shfl_xor_sync(0xffffffffu, nib, o);
                    if ((lane & 7) == 0) sMask[st][lane >> 3] = nib;
                    __syncwarp();
                    if (lane == 0) {
                        sItem[st] = item;
                        // arrive (release): the rows, the mask and the item are there; then the bytes of the gathers
                        mbar_expect_tx(full, L::STAGE);
                    }
                    __syncwarp();
                    const uint32_t dst = base + st * L::STAGE + lane * 4 * 128;
                    const int32_t col = (item % HP) * 64;
                    int32_t r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = cur[i] >= 0 ? cur[i] : oob;
                    tma_gather4(dst + 0 * L::TENSOR, &tmQ, col, r[0], r[1], r[2], r[3], full);
                    tma_gather4(dst + 1 * L::TENSOR, &tmK, col, r[0], r[1], r[2], r[3], full);
                    tma_gather4(dst + 2 * L::TENSOR, &tmV, col, r[0], r[1], r[2], r[3], full);
                    tma_gather4(dst + 3 * L::TENSOR, &tmG, col, r[0], r[1], r[2], r[3], full);
                    ++it;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
            }
            // the end, through the next free stage; then wait for the gathers in flight
            const int st = OWN ? g : it & 1;
            if (ok && it >= NS) ok = mbar_wait(smem_u32(&sEmpty[st]), ((it / NS) - 1) & 1, status);
            if (lane == 0) {
                if (ok) {
                    sItem[st] = -1;
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sFull[st])) : "memory");
                }
                // (an emptied stage's last gathers have landed, and its barrier is a phase further)
                for (int k = it - 1; k >= 0 && k >= it - NS + int(ok); --k)
                    mbar_wait(smem_u32(&sFull[OWN ? g : k & 1]), (k / NS) & 1, status);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::REGS_G));
        // ---------------- one head: query row (and key row) r, keys and columns of half `half` ----------------
        const int g = warp >> 3, half = (warp >> 2) & 1, r = tid & 127;
        const bool issuer = (tid & 255) == 0;
        const bool multi = spt > m;  // several balls in a tile
        const uint32_t tS = tmem + 256 * g, tG = tS + 128;
        const uint32_t tD = tS, tV = tS + 64, tQ = tG, tK = tG + 64;  // dS as bf16 pairs, and the results
        const uint32_t lb = uint32_t((warp & 3) * 32) << 16;
        const uint32_t barS = smem_u32(&sBarS[g]), barG = smem_u32(&sBarG[g]), barV = smem_u32(&sBarV[g]),
                       barO = smem_u32(&sBarO[g]);
        const uint32_t pbuf = base + L::P_OFF + g * L::PBUF;
        const uint32_t goff = OWN ? 0 : 64 * g;  // the head's bytes within a piece
        uint8_t *gp = gbase + L::P_OFF + g * L::PBUF;
        uint8_t *prow = gp + half * L::BLK + r * 128;
        const int b0 = r / m * m, b1 = min(b0 + m, spt);  // slots of the row's ball within the tile
        bool ok = true;

        // Waits for item `it`, then issues its S and dP; the same answer for the group's threads.
        auto begin = [&](int it) -> bool {
            const int st = OWN ? g : it & 1;
            ok = ok && mbar_wait(smem_u32(&sFull[st]), (OWN ? it : it >> 1) & 1, status);
            if (!ok) sAbort[g] = 1;
            tc_fence_before();
            group_sync(g);
            tc_fence_after();
            if (sAbort[g]) return false;
            if (sItem[st] < 0) return false;
            if (issuer) {
                const uint32_t s0 = base + st * L::STAGE + goff;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16(tS, smem_desc_sw(s0 + 32 * kk, 16, SBO, SW128),
                             smem_desc_sw(s0 + L::TENSOR + 32 * kk, 16, SBO, SW128), IDESC_S, kk > 0);
                mma_commit(barS);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_bf16(tG, smem_desc_sw(s0 + 3 * L::TENSOR + 32 * kk, 16, SBO, SW128),
                             smem_desc_sw(s0 + 2 * L::TENSOR + 32 * kk, 16, SBO, SW128), IDESC_S, kk > 0);
                mma_commit(barG);
            }
            return true;
        };
        auto store_row = [&](__nv_bfloat16 *T, const uint32_t(&v)[HALF_D], float f, int32_t to, int h) {
            if (to < 0 || h >= H) return;
            uint4 *p = reinterpret_cast<uint4 *>(T + (size_t(to) * H + h) * D + half * HALF_D);
#pragma unroll
            for (int i = 0; i < HALF_D / 8; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16(__uint_as_float(v[8 * i + 2 * e]) * f, __uint_as_float(v[8 * i + 2 * e + 1]) * f);
                p[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        };
        auto bad = [&](const uint32_t(&v)[HALF_D]) {
            bool b = false;
#pragma unroll
            for (int i = 0; i < HALF_D; ++i) b |= (v[i] & 0x7F800000u) == 0x7F800000u;
            return b;
        };
        // sum over the ball's slots x of w(x) * tensor[x][column]; w: row r of the buffer, or its column r.  Only for
        // rows r < spt, whose balls lie within the tile.
        auto mend = [&](uint32_t(&v)[HALF_D], bool column, const uint8_t *tensor) {
            float a[HALF_D];
#pragma unroll
            for (int c = 0; c < HALF_D; ++c) a[c] = 0.0f;
            for (int x = b0; x < b1; ++x) {
                const int q = column ? x : r, k = column ? r : x;
                const float w = __bfloat162float(
                    *reinterpret_cast<const __nv_bfloat16 *>(gp + (k >> 6) * L::BLK + swz(q, k & 63)));
#pragma unroll
                for (int c = 0; c < HALF_D; ++c) {
                    const int col = half * HALF_D + c + int(goff / 2);
                    a[c] = fmaf(w, __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(tensor + swz(x, col))),
                                a[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < HALF_D; ++c) v[c] = __float_as_uint(a[c]);
        };

        bool go = begin(0);
        for (int it = 0; go; ++it) {
            const int st = OWN ? g : it & 1;
            const uint32_t par = it & 1;
            const uint32_t s0 = base + st * L::STAGE + goff;
            const uint8_t *gs0 = gbase + st * L::STAGE;
            const int32_t row = sRows[st][r];
            const int item = sItem[st];
            const int h = OWN ? item % HP : (item % HP) * 2 + g;
            uint32_t cm[2];  // keys of this thread's two groups of 32 that count
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k0 = half * 64 + c * 32;
                const int lo = max(b0 - k0, 0), hi = min(b1 - k0, 32);
                const uint32_t in = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
                cm[c] = row >= 0 ? in & sMask[st][half * 2 + c] : 0u;
            }
            float e[64];
            float mx = -INFINITY;
            ok = ok && mbar_wait(barS, par, status);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t v[32];
                if (__any_sync(0xffffffffu, cm[c] != 0u)) {
                    tmem_ld32_nowait(tS + lb + half * 64 + c * 32, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) e[c * 32 + j] = __uint_as_float(v[j]);
                if (__all_sync(0xffffffffu, cm[c] == 0xffffffffu)) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) mx = fmax3(mx, e[c * 32 + j], e[c * 32 + j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if ((cm[c] >> j) & 1u) mx = fmaxf(mx, e[c * 32 + j]);
                }
            }
            const float mxs = mx == -INFINITY ? 0.0f : mx * sl2;
            float sa = 0.0f, sb = 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (__all_sync(0xffffffffu, cm[c] == 0xffffffffu)) {
#pragma unroll
                    for (int j = c * 32; j < c * 32 + 32; j += 2) {
                        float p0, p1;
                        ffma2_bcast(e[j], e[j + 1], sl2, -mxs, p0, p1);
                        e[j] = ex2(p0);
                        e[j + 1] = ex2(p1);
                        fadd2_acc(sa, sb, e[j], e[j + 1]);
                    }
                } else if (__any_sync(0xffffffffu, cm[c] != 0u)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float p = ex2(fmaf(e[c * 32 + j], sl2, -mxs));
                        e[c * 32 + j] = (cm[c] >> j) & 1u ? p : 0.0f;
                        sa += e[c * 32 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) e[c * 32 + j] = 0.0f;
                }
            }
            ok = ok && mbar_wait(barG, par, status);
            tc_fence_after();
            float la = 0.0f, lc = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t cmc = cm[c >> 1] >> (16 * (c & 1));
                if (__any_sync(0xffffffffu, cm[c >> 1] != 0u)) {
                    uint32_t v[16];
                    tmem_ld16_nowait(tG + lb + half * 64 + c * 16, v);
                    tmem_wait_ld();
                    if (__all_sync(0xffffffffu, cm[c >> 1] == 0xffffffffu)) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            la = fmaf(e[c * 16 + j], __uint_as_float(v[j]), la);
                            lc = fmaf(e[c * 16 + j + 1], __uint_as_float(v[j + 1]), lc);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if ((cmc >> j) & 1u) la = fmaf(e[c * 16 + j], __uint_as_float(v[j]), la);
                    }
                }
            }
            sX[g][half][0][r] = mx;
            sX[g][half][1][r] = sa + sb;
            sX[g][half][2][r] = la + lc;
            tc_fence_before();  // S is read: dS comes over it
            group_sync(g);
            tc_fence_after();
            float fs, delta;  // P = e fs
            {
                const float mo = sX[g][half ^ 1][0][r], so = sX[g][half ^ 1][1][r], lo = sX[g][half ^ 1][2][r];
                const float M = fmaxf(mx, mo);
                const float f0 = mx == -INFINITY ? 0.0f : ex2((mx - M) * sl2);
                const float f1 = mo == -INFINITY ? 0.0f : ex2((mo - M) * sl2);
                // a half without keys adds nothing, whatever its sums hold
                float den = 0.0f, dl = 0.0f;
                if (cm[0] | cm[1]) { den = (sa + sb) * f0; dl = (la + lc) * f0; }
                if (so != 0.0f) { den = fmaf(so, f1, den); dl = fmaf(lo, f1, dl); }
                const float inv = row >= 0 ? 1.0f / den : 0.0f;
                fs = f0 * inv;
                delta = dl * inv;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[8], ds[8];
                if (__any_sync(0xffffffffu, cm[c >> 1] != 0u)) {
                    const uint32_t cmc = cm[c >> 1] >> (16 * (c & 1));
                    uint32_t v[16];
                    tmem_ld16_nowait(tG + lb + half * 64 + c * 16, v);
                    tmem_wait_ld();
                    const bool all = __all_sync(0xffffffffu, cm[c >> 1] == 0xffffffffu);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float p0 = e[c * 16 + k] * fs, p1 = e[c * 16 + k + 1] * fs;
                        float d0 = p0 * (__uint_as_float(v[k]) - delta), d1 = p1 * (__uint_as_float(v[k + 1]) - delta);
                        if (!all) {
                            const bool on0 = (cmc >> k) & 1u, on1 = (cmc >> (k + 1)) & 1u;
                            p0 = on0 ? p0 : 0.0f;
                            p1 = on1 ? p1 : 0.0f;
                            d0 = on0 ? d0 : 0.0f;
                            d1 = on1 ? d1 : 0.0f;
                        }
                        w[k >> 1] = pack_bf16(p0, p1);
                        ds[k >> 1] = pack_bf16(d0, d1);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = ds[j] = 0u;
                }
                *reinterpret_cast<uint4 *>(prow + (((c * 2) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(prow + (((c * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
                tmem_st8(tD + lb + half * 32 + c * 8, ds);
            }
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();
            group_sync(g);
            tc_fence_after();
            if (issuer) {
                if (ok)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16(tV, smem_desc_sw(pbuf + kk * 2048, L::BLK, SBO, SW128),
                                 smem_desc_sw(s0 + 3 * L::TENSOR + kk * 2048, 16, SBO, SW128), IDESC_T, kk > 0);
                mma_commit(barV);
                if (ok)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_ts(tQ, tD + 8 * kk, smem_desc_sw(s0 + L::TENSOR + kk * 2048, 16, SBO, SW128),
                                    IDESC_Q, kk > 0);
            }
            ok = ok && mbar_wait(barV, par, status);
            tc_fence_after();
            uint32_t ds[32], ov[HALF_D];
            tmem_ld32_nowait(tD + lb + half * 32, ds);
            tmem_ld_nowait<HALF_D>(tV + lb + half * HALF_D, ov);
            tmem_wait_ld();
            if (multi && group_any(g, row >= 0 && bad(ov))) {
                if (row >= 0 && bad(ov)) mend(ov, true, gs0 + 3 * L::TENSOR);
                group_sync(g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4 *>(prow + ((j ^ (r & 7)) << 4)) =
                    make_uint4(ds[4 * j], ds[4 * j + 1], ds[4 * j + 2], ds[4 * j + 3]);
            fence_async_smem();
            tc_fence_before();
            group_sync(g);
            tc_fence_after();
            if (issuer) {
                if (ok)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16(tK, smem_desc_sw(pbuf + kk * 2048, L::BLK, SBO, SW128),
                                 smem_desc_sw(s0 + kk * 2048, 16, SBO, SW128), IDESC_T, kk > 0);
                mma_commit(barO);
                if (!multi) mma_commit(smem_u32(&sEmpty[st]));  // the stage is free once these products are done
            }
            if (ok) store_row(dV, ov, 1.0f, row, h);
            ok = ok && mbar_wait(barO, par, status);
            tc_fence_after();
            uint32_t oq[HALF_D], ok_[HALF_D];
            tmem_ld_nowait<HALF_D>(tQ + lb + half * HALF_D, oq);
            tmem_ld_nowait<HALF_D>(tK + lb + half * HALF_D, ok_);
            tmem_wait_ld();
            if (multi) {
                if (group_any(g, row >= 0 && (bad(oq) || bad(ok_)))) {
                    if (row >= 0 && bad(oq)) mend(oq, false, gs0 + L::TENSOR);
                    if (row >= 0 && bad(ok_)) mend(ok_, true, gs0);
                    group_sync(g);
                }
                if (issuer)
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sEmpty[st])) : "memory");
            }
            const int32_t to = ok ? row : -1;
            go = begin(it + 1);  // S and dP of the next item while these rows are stored
            store_row(dQ, oq, scale, to, h);
            store_row(dK, ok_, scale, to, h);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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

template <int D>
bt_status launch_tc(const BwdArgs &a)
{
    using L = BwdTc<D>;
    constexpr size_t smem = L::BYTES;
    static std::atomic<bool> set[64] = {};
    int dev = 0;
    const int sms = device_sms(&dev);
    if (sms == 0) return BT_ERR_CUDA;
    const bt_status s = setup_once(set[dev], [&]() -> bt_status {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, k_ball_bwd_tc<D>) != cudaSuccess) return BT_ERR_CUDA;
        if (at.numRegs < L::REGS) return BT_ERR_INTERNAL;  // the register split would wait for registers for ever
        return cudaFuncSetAttribute(k_ball_bwd_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) ==
                       cudaSuccess
                   ? BT_OK
                   : BT_ERR_CUDA;
    });
    if (s != BT_OK) return s;
    uint32_t *status = stream_status(a.st);
    if (!status) return BT_ERR_CUDA;
    CUtensorMap mq, mk, mv, mg;
    const int64_t cols = int64_t(a.H) * D;
    if (!matrix_map(&mq, a.Q, a.rows, cols, 2, 64, 1) || !matrix_map(&mk, a.K, a.rows, cols, 2, 64, 1) ||
        !matrix_map(&mv, a.V, a.rows, cols, 2, 64, 1) || !matrix_map(&mg, a.dO, a.rows, cols, 2, 64, 1))
        return BT_ERR_CUDA;
    const int spt = 128 / a.m * a.m;  // slots of a tile: whole balls
    const int64_t items = (a.npad + spt - 1) / spt * (L::OWN ? a.H : (a.H + 1) / 2);
    if (items > 0x7FFFFFFF - 2 * sms) return BT_ERR_UNSUPPORTED;
    const int64_t most = L::OWN ? (items + 1) / 2 : items;  // CTAs that have work
    const unsigned grid = unsigned(most < sms ? most : sms);
    const float scale = 1.0f / sqrtf(float(D));
    k_ball_bwd_tc<D><<<grid, BwdTc<D>::THREADS, smem, a.st>>>(
        mq, mk, mv, mg, a.perm, a.npad, a.rows, a.m, spt, a.H, scale, scale * 1.4426950408889634f, int(items),
        static_cast<__nv_bfloat16 *>(a.dQ), static_cast<__nv_bfloat16 *>(a.dK), static_cast<__nv_bfloat16 *>(a.dV),
        status);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
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
    if (m <= 128) return d == 32 ? launch_tc<32>(a) : launch_tc<64>(a);
    return d == 32 ? run_simt<__nv_bfloat16, 32, 256>(a) : run_simt<__nv_bfloat16, 64, 256>(a);
}

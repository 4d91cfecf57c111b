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
// Bound by shared-memory loads (77% of their rate; A: 40 cycles of loads to 32 of products), and by latency, as one to five
// CTAs fit an SM: 14 to 24 TFLOP/s.  65,536 rows of 8 x 32 floats in balls of 128: 0.90 ms, 73 us at the rate of a copy (1.23
// ms without the bound on registers that lets two CTAs of that shape share an SM); in balls of 32 0.39 ms; bf16 in balls of 256
// 1.92 ms, 36 us at the rate of a copy.
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
__global__ void __launch_bounds__(BwdSimt<D, MP>::NT, D == 32 && MP == 128 ? 2 : 1)
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
                    const bool on = (ok >> j) & 1u;
                    const float p = on ? s[i][j] * inv : 0.0f;  // (inv is NaN where the row's scores left float's range)
                    sP[ri * LP + lane + 32 * j] = p;
                    sS[ri * LP + lane + 32 * j] = on ? p * (g[i][j] - delta) : 0.0f;
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
//               128-byte swizzle) into a stage, whose two parts (Q and K; V and dO) fill and empty apart;
//   warps 18, 19  one per group: issues its products, and for d = 32 stores its results while the group computes.
// d = 32: the two groups take the two heads of a pair, whose 64 bytes of a row are one piece (an item: tile, pair), from
// two stages.  d = 64: every group has its own items (tile, head), one stage and a producer, so that one group computes
// while the other one's rows arrive.
// Per head:
//   S = Q K^T and dP = dO V^T           128 columns of TMEM each
//   e = exp2(s - max) over S, sums of e and e dP, by groups of 32 keys; a row's two threads join them through shared
//   memory; P = e / sum as bf16 into the group's 32 KB of shared memory ([query][key], two blocks of 64 keys, 128-byte
//   swizzle); dS = P (dP - delta) as bf16 over dP
//   dV = P^T dO                         A read transposed (MN-major)
//   dQ = dS K                           A from TMEM
//   dS to shared memory over P once dV is done
//   dK = dS^T Q
// P and dS take turns in one buffer, because two would leave no room for the second stage.  e lies in TMEM and not in
// registers, which 640 threads would spill (64 values each beside dP: the spills cost 10 to 40% of the time).  For d = 32
// the next item's S is computed while this one's dS is written.
// P and dS are rounded to bf16 because a product's two operands share one type and dO, K and Q are bf16; the maximum,
// sums, delta and every accumulator stay float.  Each rounding is off by at most 2^-8 of its value, as the results' own is:
// against 64 bits the gradients' RMS error is 0.0024 to 0.0025 of their RMS, 0.0017 where only the results are rounded.
// P as a sum of two bf16 numbers would take that back for twice the products and twice the buffer, which is not there.
// A key of another ball or a dummy has P = dS = 0.  Where a tile holds several balls (MULTI), a value of one ball that is
// not finite would still reach the others as 0 * value: a result that is not finite is therefore summed again over the
// ball's own slots (`mend`).  One ball to a tile (m > 64) goes without those checks, and its dummies, rows of zeros, need a
// mask in S alone: 85 us against 97 for the layer below.
// Measured: 65,536 rows of 8 x 32 in balls of 128, 85 us (235 MB: 2.75 TB/s; 36 us at the rate of a copy); 1,048,576 rows
// of 4 x 32, 604 to 630 us; 70,001 rows of 5 x 64 in balls of 64, 119 us.  A group's chain of waits and arithmetic bounds it:
// 9,700 cycles for an item of d = 32 (5,900 from a tile's arrival to P and dS, 3,800 for the last products), with no unit
// more than half busy; without any loads the layer still takes 80 us, and without the exponentials 80.  The gathers beside
// it are not far behind (58 cycles per request of four rows with two warps issuing: 7,400 cycles), so that a shorter chain
// would meet them next.  The loops over keys are kept rolled: unrolled,
// the code did not fit the instruction cache, and its registers spilled (97 us).
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
    static constexpr int GROUP = 256, THREADS = 640;
    // TMEM columns of a group: S, then e; dP, then dS (bf16 pairs) in columns 0-31 and 64-95 of it.  The results lie beside
    // dS, and dK over it; what does not fit there (d = 64) over e.
    static constexpr uint32_t TMEM = 256, T_G = 128, T_K = T_G, T_V = D == 32 ? T_G + 32 : 0,
                              T_Q = D == 32 ? T_G + 96 : 64;
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

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = r[i + j];
        tmem_st16(taddr + i, v);
    }
}

// Products with operands given as address / 16 and the rest of the descriptor.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint64_t da, uint32_t b, uint64_t db, uint32_t idesc,
                                       uint32_t acc)
{
    mma_bf16(d, da | (a & 0x3FFFu), db | (b & 0x3FFFu), idesc, acc);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint64_t db, uint32_t idesc, uint32_t acc)
{
    mma_bf16_ts(d, a, db | (b & 0x3FFFu), idesc, acc);
}

// Whether an mbarrier's phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.b32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred a;\n\telect.sync _|a, 0xffffffff;\n\tselp.u32 %0, 1, 0, a;\n\t}" : "=r"(p));
    return p != 0;
}

// Named barriers: 1 + g, group g and the warp that issues its products; 3 + g, group g; 5 + 4 g + w, the two warps of
// 32 rows.
template <int N>
__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory"); }
__device__ __forceinline__ void group_sync(int g) { named_sync<256>(3 + g); }

// One arrival for the warp.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Barrier of group g, and whether `p` holds for any of its threads.
__device__ __forceinline__ bool group_any(int g, bool p)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tbar.red.or.pred b, %1, 256, a;\n\t"
                 "selp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(r)
                 : "r"(3 + g), "r"(uint32_t(p))
                 : "memory");
    return r != 0;
}

// Pairs of floats in one packed instruction (sm_100), each lane an IEEE operation.
__device__ __forceinline__ void ffma2_acc(float &a0, float &a1, float x0, float x1, float y0, float y1)
{
    asm("{\n\t.reg .b64 a, x, y;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "fma.rn.f32x2 a, x, y, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ void fmul2(float x0, float x1, float y0, float y1, float &z0, float &z1)
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(z0), "=f"(z1)
        : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ void fadd2(float x0, float x1, float y0, float y1, float &z0, float &z1)
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(z0), "=f"(z1)
        : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
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

// Chunk c (16 bytes) of row r of result n in a group's buffer of P and dS.  The 32 rows of a pair of warps lie in that
// pair's part of the buffer (both blocks); the chunks are swizzled, so that neither writing a row per lane nor reading
// whole rows meets a bank conflict.
template <int D>
__device__ __forceinline__ uint4 *place(const uint8_t *gp, int n, int r, int c)
{
    const int rr = r & 31;
    const int o = D == 32 ? n * 2048 + rr * 64 + (((c + (rr >> 1)) & 3) << 4)
                          : n * 4096 + rr * 128 + ((c ^ (rr & 7)) << 4);
    return reinterpret_cast<uint4 *>(const_cast<uint8_t *>(gp) + (o >> 12) * BwdTc<D>::BLK + (r >> 5) * 4096 + (o & 4095));
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

template <int D, bool MULTI>
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
    // descriptors but for the address, in units of 16 bytes
    constexpr uint64_t DESC0 = (uint64_t(SBO >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(SW128) << 61);
    constexpr uint64_t DESC = DESC0 | (1u << 16), DESC_P = DESC0 | (uint64_t(L::BLK >> 4) << 16);
    constexpr uint32_t IDESC_S = idesc_bf16(128, false);        // S, dP
    constexpr uint32_t IDESC_Q = idesc_bf16(D, true);           // dQ: A as it lies in TMEM
    constexpr uint32_t IDESC_T = idesc_bf16(D, true) | MN_A;    // dV, dK: A transposed
    extern __shared__ __align__(1024) uint8_t dsm[];
    // of a stage's parts (Q and K; V and dO), and of a group
    __shared__ __align__(8) uint64_t sFull[2][2], sEmpty[2][2], sBarS[2], sBarG[2], sBarV[2], sBarO[2], sBarP[2],
        sBarD[2], sBarF[2];
    __shared__ int32_t sRows[2][128];
    __shared__ uint32_t sMask[2][4];  // real slots of the tile
    __shared__ int32_t sItem[2];      // -1: no more work
    __shared__ int32_t sWhole[2];     // no dummies among the tile's 128 slots
    __shared__ float sX[2][2][3][128];  // per group and half: a row's max, sum and sum of e dP
    __shared__ int32_t sOut[2][128];  // d = 32: rows of the results in the buffer
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
            for (int j = 0; j < 2; ++j) {
                mbar_init(&sFull[i][j], 1);
                mbar_init(&sEmpty[i][j], OWN ? 1 : 2);  // d = 32: two groups empty a stage
            }
            mbar_init(&sBarS[i], 1);
            mbar_init(&sBarG[i], 1);
            mbar_init(&sBarV[i], 1);
            mbar_init(&sBarO[i], 1);
            mbar_init(&sBarP[i], 8);
            mbar_init(&sBarD[i], 8);
            mbar_init(&sBarF[i], 1);
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
        if (warp >= 18) {
            // ---------------- products of group g; d = 32: and the stores of its results ----------------
            const int g = __shfl_sync(0xffffffffu, warp, 0) - 18;
            const uint32_t tS = __shfl_sync(0xffffffffu, tmem, 0) + L::TMEM * g;
            const uint32_t barS = smem_u32(&sBarS[g]), barG = smem_u32(&sBarG[g]), barV = smem_u32(&sBarV[g]),
                           barO = smem_u32(&sBarO[g]);
            // operand addresses / 16.  Descriptors are made where they are used: kept in registers, they would spill.
            auto stage16 = [&](int st) {
                uint32_t a = (base + st * L::STAGE + (OWN ? 0 : 64 * g)) >> 4;
                asm volatile("" : "+r"(a));
                return a;
            };
            auto wait = [&](uint64_t *bar, uint32_t par) {
                if (!mbar_wait(smem_u32(bar), par, status)) sAbort[g] = 1;
                __syncwarp();
                tc_fence_after();
            };
            auto issue_s = [&](int st) {
                const uint32_t s0 = stage16(st);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tS, s0 + 2 * kk, DESC, s0 + (L::TENSOR + 32 * kk) / 16, DESC, IDESC_S, kk > 0);
                    mma_commit(barS);
                }
                __syncwarp();
            };
            int h = 0;  // head of the results that wait in the buffer
            for (int it = 0;; ++it) {
                const int st = OWN ? g : it & 1;
                const uint32_t use = (OWN ? it : it >> 1) & 1;
                if (OWN || it == 0) wait(&sFull[st][0], use);
                named_sync<L::GROUP + 32>(1 + g);  // the last results are out of TMEM, and item `it` is there
                tc_fence_after();
                const int item = sItem[st];
                const bool stop = sAbort[g] || item < 0;
                if (!stop) {
                    if (OWN || it == 0) issue_s(st);
                    wait(&sFull[st][1], use);
                    const uint32_t s0 = stage16(st);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tS + L::T_G, s0 + (3 * L::TENSOR + 32 * kk) / 16, DESC,
                                   s0 + (2 * L::TENSOR + 32 * kk) / 16, DESC, IDESC_S, kk > 0);
                        mma_commit(barG);
                    }
                    __syncwarp();
                }
                if constexpr (!OWN) {
                    if (it > 0) {
                        // 8 rows of 64 bytes at a time
                        const int c = lane & 3;
#pragma unroll 2
                        for (int i = 0; i < 16; ++i) {
                            const int r = i * 8 + (lane >> 2);
                            const int32_t to = sOut[g][r];
                            if (to >= 0 && h < H) {
                                const uint8_t *gp = gbase + L::P_OFF + g * L::PBUF;
                                const size_t o = (size_t(to) * H + h) * D + c * 8;
                                *reinterpret_cast<uint4 *>(dV + o) = *place<D>(gp, 0, r, c);
                                *reinterpret_cast<uint4 *>(dQ + o) = *place<D>(gp, 1, r, c);
                                *reinterpret_cast<uint4 *>(dK + o) = *place<D>(gp, 2, r, c);
                            }
                        }
                        warp_arrive(smem_u32(&sBarF[g]));  // the buffer is free
                    }
                    h = (item % HP) * 2 + g;
                }
                if (stop) break;
                wait(&sBarP[g], it & 1);  // P in shared memory, dS in TMEM
                {
                    const uint32_t s0 = stage16(st);
                    uint32_t p0 = (base + L::P_OFF + g * L::PBUF) >> 4;
                    asm volatile("" : "+r"(p0));
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ss(tS + L::T_V, p0 + 128 * kk, DESC_P, s0 + (3 * L::TENSOR + 2048 * kk) / 16, DESC,
                                   IDESC_T, kk > 0);
                        mma_commit(barV);
                        if (OWN && !MULTI) mma_commit(smem_u32(&sEmpty[st][1]));
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ts(tS + L::T_Q, tS + L::T_G + 64 * (kk >> 2) + 8 * (kk & 3),
                                   s0 + (L::TENSOR + 2048 * kk) / 16, DESC, IDESC_Q, kk > 0);
                    }
                    __syncwarp();
                }
                bool ahead = false;  // the next S is on its way: e is not needed any more
                if (!OWN && __all_sync(0xffffffffu, mbar_test(smem_u32(&sFull[st ^ 1][0]), ((it + 1) >> 1) & 1))) {
                    ahead = true;
                    if (sItem[st ^ 1] >= 0) issue_s(st ^ 1);
                }
                wait(&sBarD[g], it & 1);  // dS in shared memory
                {
                    const uint32_t s0 = stage16(st);
                    uint32_t p0 = (base + L::P_OFF + g * L::PBUF) >> 4;
                    asm volatile("" : "+r"(p0));
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ss(tS + L::T_K, p0 + 128 * kk, DESC_P, s0 + 128 * kk, DESC, IDESC_T, kk > 0);
                        mma_commit(barO);
                        if (!MULTI) {  // the stage is free once these products are done
                            mma_commit(smem_u32(&sEmpty[st][0]));
                            if (!OWN) mma_commit(smem_u32(&sEmpty[st][1]));
                        }
                    }
                    __syncwarp();
                }
                if (!OWN && !ahead) {
                    wait(&sFull[st ^ 1][0], ((it + 1) >> 1) & 1);
                    if (!*static_cast<volatile int *>(&sAbort[g]) && sItem[st ^ 1] >= 0) issue_s(st ^ 1);
                }
            }
        } else {
            // ---------------- producer p: lane l has rows 4l .. 4l+3 of the tile ----------------
            // d = 32: part p of the two stages (0: Q, K, and the tile's rows; 1: V, dO); d = 64: both parts of group p's
            // stage, V and dO first, which are free first
            const int p = warp - 16;
            constexpr int NS = OWN ? 1 : 2;
            const int first = OWN ? 2 * int(blockIdx.x) + p : int(blockIdx.x);
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
            auto emptied = [&](int st, int part, int it) {
                bool ok = it < NS || mbar_wait(smem_u32(&sEmpty[st][part]), ((it / NS) - 1) & 1, status);
                return bool(__all_sync(0xffffffffu, ok));
            };
            int item = first, it = 0;
            int32_t cur[4];
            load_rows(item, cur);
            bool ok = true;
            for (; item < items; item += step) {
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
                    const int st = OWN ? p : it & 1;
                    const uint32_t dst = base + st * L::STAGE + lane * 4 * 128;
                    const int32_t col = (item % HP) * 64;
                    if (OWN || p == 1) {
                        ok = emptied(st, 1, it);
                        if (!ok) break;
                        const uint32_t full = smem_u32(&sFull[st][1]);
                        if (lane == 0) mbar_expect_tx(full, 2 * L::TENSOR);
                        __syncwarp();
                        int32_t r[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[i] = cur[i] >= 0 ? cur[i] : oob;
                        tma_gather4(dst + 3 * L::TENSOR, &tmG, col, r[0], r[1], r[2], r[3], full);
                        tma_gather4(dst + 2 * L::TENSOR, &tmV, col, r[0], r[1], r[2], r[3], full);
                    }
                    if (OWN || p == 0) {
                        ok = emptied(st, 0, it);
                        if (!ok) break;
                        const uint32_t full = smem_u32(&sFull[st][0]);
                        uint32_t nib = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sRows[st][4 * lane + i] = cur[i];
                            nib |= uint32_t(cur[i] >= 0) << i;
                        }
                        const bool whole = __all_sync(0xffffffffu, nib == 15u);
                        nib <<= 4 * (lane & 7);
                        for (int o = 1; o < 8; o <<= 1) nib |= __shfl_xor_sync(0xffffffffu, nib, o);
                        if ((lane & 7) == 0) sMask[st][lane >> 3] = nib;
                        if (lane == 0) {
                            sItem[st] = item;
                            sWhole[st] = whole;
                        }
                        __syncwarp();
                        // arrive (release): the rows, the mask and the item are there; then the bytes of the gathers
                        if (lane == 0) mbar_expect_tx(full, 2 * L::TENSOR);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) cur[i] = cur[i] >= 0 ? cur[i] : oob;
                        tma_gather4(dst + 0 * L::TENSOR, &tmQ, col, cur[0], cur[1], cur[2], cur[3], full);
                        tma_gather4(dst + 1 * L::TENSOR, &tmK, col, cur[0], cur[1], cur[2], cur[3], full);
                    }
                    ++it;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
            }
            // the end, through the next free stage; then wait for the gathers in flight
            const int st = OWN ? p : it & 1;
            if (ok && (OWN || p == 0)) {
                ok = emptied(st, 0, it);
                if (ok && lane == 0) {
                    sItem[st] = -1;
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sFull[st][0])) : "memory");
                }
            }
            // (an emptied part's last gathers have landed, and its barrier is a phase further)
            if (lane == 0) {
                if (OWN || p == 1)
                    for (int k = it - 1; k >= 0 && k >= it - NS; --k)
                        mbar_wait(smem_u32(&sFull[OWN ? p : k & 1][1]), (k / NS) & 1, status);
                if (OWN || p == 0)
                    for (int k = it - 1; k >= 0 && k >= it - NS + int(ok); --k)
                        mbar_wait(smem_u32(&sFull[OWN ? p : k & 1][0]), (k / NS) & 1, status);
            }
            __syncwarp();
        }
    } else {
        // ---------------- one head: query row (and key row) r, keys and columns of half `half` ----------------
        const int g = warp >> 3, half = (warp >> 2) & 1, r = tid & 127;
        const uint32_t tS = tmem + L::TMEM * g + (uint32_t((warp & 3) * 32) << 16), tG = tS + L::T_G;
        const uint32_t tV = tS + L::T_V, tQ = tS + L::T_Q, tK = tS + L::T_K;
        const uint32_t barS = smem_u32(&sBarS[g]), barG = smem_u32(&sBarG[g]), barV = smem_u32(&sBarV[g]),
                       barO = smem_u32(&sBarO[g]);
        const int pair = 5 + g * 4 + (warp & 3);  // barrier of the two warps that share 32 rows
        uint8_t *gp = gbase + L::P_OFF + g * L::PBUF;
        uint8_t *prow = gp + half * L::BLK + r * 128;
        const int b0 = r / m * m, b1 = min(b0 + m, spt);  // slots of the row's ball within the tile
        bool ok = true;

        auto bad = [&](const uint32_t(&v)[HALF_D]) {
            bool b = false;
#pragma unroll
            for (int i = 0; i < HALF_D; ++i) b |= (v[i] & 0x7F800000u) == 0x7F800000u;
            return b;
        };
        // sum over the ball's slots x of w(x) * tensor[x][column]; w: row r of the buffer, or its column r.  Only for
        // rows r < spt, whose balls lie within the tile.
        auto mend = [&](uint32_t(&v)[HALF_D], bool column, const uint8_t *tensor) {
#pragma unroll
            for (int c0 = 0; c0 < HALF_D; c0 += 8) {
                float a[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) a[c] = 0.0f;
#pragma unroll 1
                for (int x = b0; x < b1; ++x) {
                    const int q = column ? x : r, k = column ? r : x;
                    const float w = __bfloat162float(
                        *reinterpret_cast<const __nv_bfloat16 *>(gp + (k >> 6) * L::BLK + swz(q, k & 63)));
                    const int col = half * HALF_D + c0 + (OWN ? 0 : 32 * g);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        a[c] = fmaf(w, __bfloat162float(
                                           *reinterpret_cast<const __nv_bfloat16 *>(tensor + swz(x, col + c))), a[c]);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c0 + c] = __float_as_uint(a[c]);
            }
        };
        auto put = [&](int n, const uint32_t(&v)[HALF_D], float f) {
#pragma unroll
            for (int i = 0; i < HALF_D / 8; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_bf16(__uint_as_float(v[8 * i + 2 * e]) * f, __uint_as_float(v[8 * i + 2 * e + 1]) * f);
                *place<D>(gp, n, r, half * (HALF_D / 8) + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        };
        // d = 64: the warp stores 16 of the pair's rows
        auto store = [&](int n, __nv_bfloat16 *T, int32_t row, int h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = half * 16 + i * 4 + (lane >> 3), c = lane & 7;
                const int32_t to = __shfl_sync(0xffffffffu, row, rr);
                if (to >= 0)
                    *reinterpret_cast<uint4 *>(T + (size_t(to) * H + h) * D + c * 8) =
                        *place<D>(gp, n, (r & 96) + rr, c);
            }
        };

        for (int it = 0;; ++it) {
            const int st = OWN ? g : it & 1;
            const uint32_t par = it & 1;
            const uint8_t *gs0 = gbase + st * L::STAGE;
            if (ok) ok = mbar_wait(smem_u32(&sFull[st][0]), (OWN ? it : it >> 1) & 1, status);
            if (!ok) sAbort[g] = 1;
            tc_fence_before();
            named_sync<L::GROUP + 32>(1 + g);
            const int item = sItem[st];
            if (sAbort[g] || item < 0) break;
            const int32_t row = sRows[st][r];
            // the keys of this thread's two groups of 32 that count; several balls: and for the warp, bit c, some count in
            // group c, bit c of all: all
            uint32_t cm[2] = {0xffffffffu, 0xffffffffu};
            [[maybe_unused]] int some = 3, all = 3;
            const bool whole = !MULTI && sWhole[st];
            if (!whole) {
                some = all = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int k0 = half * 64 + c * 32;
                    const int lo = max(b0 - k0, 0), hi = min(b1 - k0, 32);
                    const uint32_t in = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
                    cm[c] = row >= 0 ? in & sMask[st][half * 2 + c] : 0u;
                    if (MULTI) {
                        some |= int(__any_sync(0xffffffffu, cm[c] != 0u)) << c;
                        all |= int(__all_sync(0xffffffffu, cm[c] == 0xffffffffu)) << c;
                    }
                }
            }
            // e = exp2(s - max) over S, the maximum and the sums of e and e dP by groups of 32 keys.  The loops are not
            // unrolled: the instruction cache and the registers of 640 threads are short.
            float m0 = -INFINITY, m1 = -INFINITY, s0 = 0.0f, s1 = 0.0f, l0 = 0.0f, l1 = 0.0f;
            if (ok) ok = mbar_wait(barS, par, status);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                if (MULTI && !((some >> c) & 1)) continue;
                const uint32_t on = c ? cm[1] : cm[0];
                uint32_t e[32], v[32];
                tmem_ld32_nowait(tS + half * 64 + c * 32, e);
                tmem_wait_ld();
                float mx = -INFINITY, sa = 0.0f, sb = 0.0f, la = 0.0f, lb = 0.0f;
                const bool full = MULTI ? (all >> c) & 1 : whole;
                // one ball: what is no key is a dummy, whose rows are zeros, so that only S needs the mask
                if (!full) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((on >> j) & 1u)) e[j] = __float_as_uint(-INFINITY);
                }
                {
                    float my = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        mx = fmax3(mx, __uint_as_float(e[j]), __uint_as_float(e[j + 1]));
                        my = fmax3(my, __uint_as_float(e[j + 2]), __uint_as_float(e[j + 3]));
                    }
                    mx = fmaxf(mx, my);
                }
                const float mxs = mx == -INFINITY ? 0.0f : mx * sl2;
                if (ok) ok = mbar_wait(barG, par, status);
                tc_fence_after();
                tmem_ld32_nowait(tG + half * 64 + c * 32, v);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    float p0, p1;
                    ffma2_bcast(__uint_as_float(e[j]), __uint_as_float(e[j + 1]), sl2, -mxs, p0, p1);
                    e[j] = __float_as_uint(ex2(p0));
                    e[j + 1] = __float_as_uint(ex2(p1));
                    if (MULTI && !full) {  // (a row whose maximum is infinite has NaN beside it too)
                        e[j] = (on >> j) & 1u ? e[j] : 0u;
                        e[j + 1] = (on >> (j + 1)) & 1u ? e[j + 1] : 0u;
                    }
                    fadd2_acc(sa, sb, __uint_as_float(e[j]), __uint_as_float(e[j + 1]));
                }
                tmem_st<32>(tS + half * 64 + c * 32, e);
                tmem_wait_ld();
                if (MULTI && !full) {  // another ball's dP may be anything
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((on >> j) & 1u)) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    ffma2_acc(la, lb, __uint_as_float(e[j]), __uint_as_float(e[j + 1]), __uint_as_float(v[j]),
                              __uint_as_float(v[j + 1]));
                if (c) { m1 = mx; s1 = sa + sb; l1 = la + lb; }
                else { m0 = mx; s0 = sa + sb; l0 = la + lb; }
            }
            if (MULTI && ok) ok = mbar_wait(barG, par, status);  // a warp without keys: dS comes over dP
            float f0, f1, delta;  // P = e f0 in the first group, e f1 in the second
            {
                // sums over a part without keys count for nothing, whatever they hold
                const float mx = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.0f : ex2((m0 - mx) * sl2);
                f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - mx) * sl2);
                float den = 0.0f, dl = 0.0f;
                if (cm[0]) { den = s0 * f0; dl = l0 * f0; }
                if (cm[1]) { den = fmaf(s1, f1, den); dl = fmaf(l1, f1, dl); }
                sX[g][half][0][r] = mx;
                sX[g][half][1][r] = den;
                sX[g][half][2][r] = dl;
                named_sync<64>(pair);
                const float mo = sX[g][half ^ 1][0][r], so = sX[g][half ^ 1][1][r], lo = sX[g][half ^ 1][2][r];
                const float M = fmaxf(mx, mo);
                const float g0 = mx == -INFINITY ? 0.0f : ex2((mx - M) * sl2);
                const float g1 = mo == -INFINITY ? 0.0f : ex2((mo - M) * sl2);
                den *= g0;
                dl *= g0;
                if (so != 0.0f) { den = fmaf(so, g1, den); dl = fmaf(lo, g1, dl); }
                const float inv = row >= 0 ? 1.0f / den : 0.0f;
                f0 *= g0 * inv;
                f1 *= g0 * inv;
                delta = dl * inv;
            }
            if (!OWN && it > 0 && ok) ok = mbar_wait(smem_u32(&sBarF[g]), (it - 1) & 1, status);  // results are stored
            tmem_wait_st();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t w[8], ds[8];
                if (!MULTI || ((some >> (c >> 1)) & 1)) {
                    uint32_t e[16], v[16];
                    const float f = c < 2 ? f0 : f1;
                    tmem_ld16_nowait(tS + half * 64 + c * 16, e);
                    tmem_ld16_nowait(tG + half * 64 + c * 16, v);
                    tmem_wait_ld();
                    if (!MULTI || ((all >> (c >> 1)) & 1)) {
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            float p0, p1, d0, d1;
                            fmul2(__uint_as_float(e[k]), __uint_as_float(e[k + 1]), f, f, p0, p1);
                            fadd2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]), -delta, -delta, d0, d1);
                            fmul2(p0, p1, d0, d1, d0, d1);
                            w[k >> 1] = pack_bf16(p0, p1);
                            ds[k >> 1] = pack_bf16(d0, d1);
                        }
                    } else {
                        const uint32_t on = (c < 2 ? cm[0] : cm[1]) >> (16 * (c & 1));
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            const bool o0 = (on >> k) & 1u, o1 = (on >> (k + 1)) & 1u;
                            const float p0 = o0 ? __uint_as_float(e[k]) * f : 0.0f;
                            const float p1 = o1 ? __uint_as_float(e[k + 1]) * f : 0.0f;
                            w[k >> 1] = pack_bf16(p0, p1);
                            ds[k >> 1] = pack_bf16(o0 ? p0 * (__uint_as_float(v[k]) - delta) : 0.0f,
                                                   o1 ? p1 * (__uint_as_float(v[k + 1]) - delta) : 0.0f);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = ds[j] = 0u;
                }
                *reinterpret_cast<uint4 *>(prow + (((c * 2) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(prow + (((c * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
                tmem_st8(tG + half * 64 + c * 8, ds);
            }
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();
            warp_arrive(smem_u32(&sBarP[g]));
            if (ok) ok = mbar_wait(barV, par, status);
            tc_fence_after();
            if constexpr (MULTI) {  // while P is still there
                uint32_t ov[HALF_D];
                tmem_ld_nowait<HALF_D>(tV + half * HALF_D, ov);
                tmem_wait_ld();
                if (group_any(g, row >= 0 && bad(ov))) {
                    if (row >= 0 && bad(ov)) mend(ov, true, gs0 + 3 * L::TENSOR);
                    tmem_st<HALF_D>(tV + half * HALF_D, ov);
                    tmem_wait_st();
                    fence_async_smem();  // dO is read: the next rows may come over it
                    group_sync(g);
                }
                if (OWN && (tid & 255) == 0)
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sEmpty[st][1])) : "memory");
            }
            {
                uint32_t ds[2][16];
                tmem_ld16_nowait(tG + half * 64, ds[0]);
                tmem_ld16_nowait(tG + half * 64 + 16, ds[1]);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t *x = ds[j >> 2] + 4 * (j & 3);
                    *reinterpret_cast<uint4 *>(prow + ((j ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(smem_u32(&sBarD[g]));
            if (ok) ok = mbar_wait(barO, par, status);
            tc_fence_after();
            uint32_t oq[HALF_D], ok_[HALF_D];
            tmem_ld_nowait<HALF_D>(tQ + half * HALF_D, oq);
            tmem_ld_nowait<HALF_D>(tK + half * HALF_D, ok_);
            tmem_wait_ld();
            if constexpr (MULTI) {
                if (group_any(g, row >= 0 && (bad(oq) || bad(ok_)))) {
                    if (row >= 0 && bad(oq)) mend(oq, false, gs0 + L::TENSOR);
                    if (row >= 0 && bad(ok_)) mend(ok_, true, gs0);
                    fence_async_smem();
                    group_sync(g);
                }
                if ((tid & 255) == 0) {
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sEmpty[st][0])) : "memory");
                    if (!OWN)
                        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&sEmpty[st][1]))
                                     : "memory");
                }
            }
            // The results take the place of dS, whose products are done, and leave from there in whole rows
            put(1, oq, scale);
            tmem_ld_nowait<HALF_D>(tV + half * HALF_D, oq);
            tmem_wait_ld();
            put(0, oq, 1.0f);
            const int32_t to = ok ? row : -1;
            if constexpr (!OWN) {
                put(2, ok_, scale);
                if (half == 0) sOut[g][r] = to;
            } else {
                const int h = item % HP;
                named_sync<64>(pair);
                store(0, dV, to, h);
                store(1, dQ, to, h);
                named_sync<64>(pair);
                put(0, ok_, scale);
                named_sync<64>(pair);
                store(0, dK, to, h);
            }
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

template <int D, bool MULTI>
bt_status run_tc(const BwdArgs &a)
{
    using L = BwdTc<D>;
    constexpr size_t smem = L::BYTES;
    static std::atomic<bool> set[64] = {};
    int dev = 0;
    const int sms = device_sms(&dev);
    if (sms == 0) return BT_ERR_CUDA;
    const bt_status s = setup_once(set[dev], [&]() -> bt_status {
        return cudaFuncSetAttribute(k_ball_bwd_tc<D, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) ==
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
    k_ball_bwd_tc<D, MULTI><<<grid, BwdTc<D>::THREADS, smem, a.st>>>(
        mq, mk, mv, mg, a.perm, a.npad, a.rows, a.m, spt, a.H, scale, scale * 1.4426950408889634f, int(items),
        static_cast<__nv_bfloat16 *>(a.dQ), static_cast<__nv_bfloat16 *>(a.dK), static_cast<__nv_bfloat16 *>(a.dV),
        status);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <int D>
bt_status launch_tc(const BwdArgs &a)
{
    return a.m <= 64 ? run_tc<D, true>(a) : run_tc<D, false>(a);  // two balls or more in a tile, or one
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

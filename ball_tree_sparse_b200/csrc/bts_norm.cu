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
// holding up to NV vectors of VEC elements (16 bytes), vector i of thread t the (i * tpr + t)-th of the row, so that
// neighbouring threads read neighbouring bytes.
// Vectors are aligned in memory, not in the row: where C is no multiple of VEC, row r begins `sh` = r C mod VEC elements
// into its first vector, and the first and last vectors are read and written by element.  All tensors of a call have the
// same shape, so they share the shift.  Only where an address is not aligned is VEC 1.
// Measured (bf16): 1,048,576 x 128 with residual 170 us, 98% of a copy's rate; 65,536 x 256 with residual 26 us (79%);
// 1,048,576 x 128 with residual to 8 bits 176 us (83%: arithmetic); backward, 1,048,576 x 128 189 us (88%), 65,536 x 256
// 32 us (64%), both with dH; odd lengths are bound by the instructions for their edges (100,000 x 333 with residual: 115 us,
// 36%).
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "bts_internal.cuh"
#include "bts_maps.cuh"

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

// Two floats in one register pair and packed instructions on them (sm_100), each half an IEEE operation.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ float2 get() const
    {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
        return f;
    }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The vectors of a row that a thread holds: vector i at column col(i) of C, `p` the row's first element; zeros where it has
// none (or !live).  EDGE: the first and last may reach into the neighbouring rows, whose elements are read with the rest
// (and perhaps while they are written) and dropped by mask_edge.  `end`: less than a vector follows the row, and single
// elements are read where it ends inside one.  All loads are issued before any is used.
template <bool EDGE, typename T, int VEC, int NV, typename F>
__device__ __forceinline__ void load_row(Pack<T, VEC> (&k)[NV], const T *p, int C, bool live, bool end, F &&col)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        if (live && c < C && (!EDGE || (c + VEC > 0 && !(end && c + VEC > C)))) {
            k[i] = load_pack<T, VEC>(p + c);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) k[i].v[e] = T(0.0f);
        }
    }
    if (EDGE && end && live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (c < C && c + VEC > C)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (c + e < C) k[i].v[e] = p[c + e];
        }
    }
}

template <bool EDGE, typename T, int VEC>
__device__ __forceinline__ void mask_edge(Pack<T, VEC> &k, int c, int C)
{
    if constexpr (EDGE)
#pragma unroll
        for (int e = 0; e < VEC; ++e) k.v[e] = unsigned(c + e) < unsigned(C) ? k.v[e] : T(0.0f);
}

template <typename T, int VEC, bool EDGE>
__device__ __forceinline__ void store_part(T *p, const Pack<T, VEC> &k, int c0, int C)
{
    if (!EDGE || (c0 >= 0 && c0 + VEC <= C)) {
        store_pack<T, VEC>(p, k);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (unsigned(c0 + e) < unsigned(C)) p[e] = k.v[e];
    }
}

// The weight's elements c0 ..: in 16-byte pieces where they are whole and aligned
template <int VEC, bool EDGE>
__device__ __forceinline__ void load_weight(const float *w, int c0, int C, float (&f)[VEC])
{
    if constexpr (VEC >= 4 && !EDGE) {
#pragma unroll
        for (int e = 0; e + 3 < VEC; e += 4) {
            const float4 t = __ldg(reinterpret_cast<const float4 *>(w + c0 + e));
            f[e] = t.x; f[e + 1] = t.y; f[e + 2] = t.z; f[e + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = !EDGE || unsigned(c0 + e) < unsigned(C) ? __ldg(w + c0 + e) : 0.0f;
    }
}

// Reductions over the tpr threads of a row; every thread gets the result.  The order of the additions depends on tpr
// alone.  tpr > 32: `red` holds one value per warp of the block, the row's warps meet at a barrier of their own, and a
// value stays until the row's next reduction but one (two halves, `turn`).
__device__ __forceinline__ void row_barrier(int grp, int tpr)
{
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(tpr) : "memory");
}

template <typename V, typename F>
__device__ __forceinline__ V row_reduce(V v, int tpr, V *red, int &turn, F &&join)
{
    const int o0 = tpr < 32 ? tpr : 32;
    for (int o = o0 >> 1; o > 0; o >>= 1) {
        V u;
        if constexpr (sizeof(V) == 8) {
            u.x = __shfl_xor_sync(0xffffffffu, v.x, o);
            u.y = __shfl_xor_sync(0xffffffffu, v.y, o);
        } else {
            u = __shfl_xor_sync(0xffffffffu, v, o);
        }
        v = join(v, u);
    }
    if (tpr > 32) {
        const int nw = tpr >> 5, w = threadIdx.x >> 5, w0 = w & ~(nw - 1);
        V *half = red + 8 * (turn & 1);
        ++turn;
        if ((threadIdx.x & 31) == 0) half[w] = v;
        row_barrier(w0 >> (31 - __clz(nw)), tpr);
        v = half[w0];
        for (int i = 1; i < nw; ++i) v = join(v, half[w0 + i]);
    }
    return v;
}

// One row per group of tpr threads.  I8: q and scale instead of Y.  norm == false: y = h (quantisation alone).
// X, R and Hout may be the same tensor: a thread reads its elements before it writes them, so these loads are
// plain ones.  SHIFT: C is no multiple of VEC.
// Three blocks of 256 threads to an SM where a thread holds 32 elements: two, which the registers would make, leave
// 1,048,576 x 128 bf16 to 8 bits at 217 us instead of 176, and four spill (197).  With a shift the bound spills (30,000 x
// 1,777 floats: 250 us instead of 180).
template <typename T, int VEC, int NV, bool SHIFT, bool I8>
__global__ void __launch_bounds__(kNormThreads, NV * VEC == 32 && !SHIFT ? 3 : 0)
    k_rms_norm(const T *X, const T *R, const float *__restrict__ w, int64_t rows, int C, float invC, int tpr,
               float eps, bool norm, T *Hout, T *Y, int8_t *Q, float *scale)
{
    __shared__ float red[16];
    int turn = 0;
    const int lg = 31 - __clz(tpr), t = int(threadIdx.x) & (tpr - 1);  // tpr is a power of two
    const int64_t row = int64_t(blockIdx.x) * (int(blockDim.x) >> lg) + (int(threadIdx.x) >> lg);
    const bool live = row < rows;  // dead groups stay for the shuffles
    const size_t base = live ? size_t(row) * C : 0;
    const int sh = SHIFT ? int(base & (VEC - 1)) : 0;
    auto col = [&](int i) { return (i * tpr + t) * VEC - sh; };  // first column of vector i; below 0 in the row before
    auto has = [&](int c) { return live && c < C && (!SHIFT || c + VEC > 0); };

    float h[NV * VEC];
    {
        Pack<T, VEC> k[NV], rr[NV];
        const bool end = SHIFT && (rows - 1 - row) * C < VEC;
        load_row<SHIFT>(k, X + base, C, live, end, col);
        if (R) load_row<SHIFT>(rr, R + base, C, live, end, col);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            mask_edge<SHIFT>(k[i], c, C);
            if (R) {
                mask_edge<SHIFT>(rr[i], c, C);
#pragma unroll
                for (int e = 0; e < VEC; ++e) k[i].v[e] = narrow<T>(widen(k[i].v[e]) + widen(rr[i].v[e]));
                if (Hout && has(c)) store_part<T, VEC, SHIFT>(Hout + base + c, k[i], c, C);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i * VEC + e] = widen(k[i].v[e]);
        }
    }
    if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) ss = fmaf(h[i], h[i], ss);
        ss = row_reduce(ss, tpr, red, turn, [](float a, float b) { return a + b; });
        const float rs = rsqrtf(fmaf(ss, invC, eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
            if (w && has(c)) load_weight<VEC, SHIFT>(w, c, C, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i * VEC + e] = h[i * VEC + e] * rs * f[e];
        }
    }
    if constexpr (!I8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (has(c)) {
                Pack<T, VEC> k;
#pragma unroll
                for (int e = 0; e < VEC; ++e) k.v[e] = narrow<T>(h[i * VEC + e]);
                store_part<T, VEC, SHIFT>(Y + base + c, k, c, C);
            }
        }
    } else {
        // a value that is not finite leaves NaN in its product with 0: such a row has scale NaN and values 0
        float mx = 0.0f, nf = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            const int c = col(i / VEC) + i % VEC;
            const float y = !SHIFT || unsigned(c) < unsigned(C) ? h[i] : 0.0f;  // (0 times an infinite 1 / rms is NaN too)
            mx = fmaxf(mx, fabsf(y));
            nf = fmaf(y, 0.0f, nf);
        }
        mx = nf == 0.0f ? mx : INFINITY;
        mx = row_reduce(mx, tpr, red, turn, [](float a, float b) { return fmaxf(a, b); });
        const bool bad = mx > FLT_MAX;
        const float s = bad ? nanf("") : mx / 127.0f;
        if (live && t == 0) scale[row] = s;
        // y / s correctly rounded, from the correctly rounded reciprocal and the exact remainders of the multiply-add
        // (Markstein: from a quotient within one unit in the last place, one step gives the rounded one; the first step
        // gets there).  Adding 1.5 * 2^23 then rounds to a whole number, whose low byte is the result.  Rows of extreme
        // scale, of zeros or with values that are not finite are divided.
        const bool quick = s >= 1e-25f && s <= 1e25f;
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (has(c)) {
                Pack<int8_t, VEC> k;
                if (quick) {
                    uint32_t b[VEC];
                    if constexpr (VEC == 1) {
                        float q = h[i] * inv;
                        q = fmaf(fmaf(-q, s, h[i]), inv, q);
                        q = fmaf(fmaf(-q, s, h[i]), inv, q);
                        k.v[0] = int8_t(__float_as_int(q + 12582912.0f));
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            const F2 y(h[i * VEC + e], h[i * VEC + e + 1]), ns(-s, -s), in(inv, inv);
                            F2 q = y * in;
                            q = fma2(fma2(q, ns, y), in, q);
                            q = fma2(fma2(q, ns, y), in, q);
                            const float2 z = (q + F2(12582912.0f, 12582912.0f)).get();
                            b[e] = __float_as_uint(z.x);
                            b[e + 1] = __float_as_uint(z.y);
                        }
                        uint32_t w[VEC / 4];
#pragma unroll
                        for (int e = 0; e < VEC; e += 4)
                            w[e / 4] = __byte_perm(__byte_perm(b[e], b[e + 1], 0x0040),
                                                   __byte_perm(b[e + 2], b[e + 3], 0x0040), 0x5410);
                        memcpy(&k, w, VEC);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float v = bad || s == 0.0f ? 0.0f : h[i * VEC + e] / s;
                        k.v[e] = int8_t(max(-127, min(127, __float2int_rn(v))));
                    }
                }
                store_part<int8_t, VEC, SHIFT>(Q + base + c, k, c, C);
            }
        }
    }
}

constexpr int kBwdBlocks = 148 * 4;  // rows of partial sums of dw, at most

// Backward: whether the next row is loaded before a row is reduced, and blocks of 256 threads on an SM (what their registers
// leave room for).  Floats: two vectors a thread, two blocks, the next row ahead (65,536 x 512 with dH: 94 us; one vector, no
// row ahead, four blocks: 107).  16 bits have twice the arithmetic to a byte, and more threads do better than rows ahead
// (65,536 x 1024 with dH: 123 us with one vector and four blocks; 143 with three and a row ahead).
template <typename T, int VEC, int NV>
struct BwdShape {
    static constexpr bool AHEAD = sizeof(T) == 4 && NV <= 2 && VEC > 1;
    static constexpr int PER_SM = NV * VEC <= 8 ? (AHEAD ? 2 : 4) : NV * VEC <= 16 ? 2 : 1;
};

// Backward: group G of tpr threads (of NG in the grid) walks rows G, G + NG, ...; NG is a multiple of VEC where there are
// more rows than groups, so a group's rows have the same shift and a thread the same columns in all of them: it keeps its
// part of the weight and of dw in registers.  The block's groups add theirs in shared memory in the order of the groups,
// and the block writes one row of `part` ([gridDim.x][C]).  k_norm_dw adds those rows in order, so that equal calls give
// equal bits.
template <typename T, int VEC, int NV, bool SHIFT>
__global__ void __launch_bounds__(kNormThreads, (BwdShape<T, VEC, NV>::PER_SM))
    k_rms_norm_bwd(const T *dY, const T *dH, const T *H, const float *__restrict__ w, int64_t rows, int C,
                   float invC, int tpr, float eps, T *dX, float *__restrict__ part)
{
    constexpr bool PF = BwdShape<T, VEC, NV>::AHEAD;
    extern __shared__ float acc_sm[];  // [groups][C] while the block's groups are joined
    __shared__ float2 red[16];
    int turn = 0;
    const int lg = 31 - __clz(tpr), rpb = int(blockDim.x) >> lg;
    const int t = int(threadIdx.x) & (tpr - 1), grp = int(threadIdx.x) >> lg;
    const int64_t step = int64_t(gridDim.x) * rpb, G = int64_t(blockIdx.x) * rpb + grp;
    const int sh = SHIFT ? int((size_t(G) * C) & (VEC - 1)) : 0;
    auto col = [&](int i) { return (i * tpr + t) * VEC - sh; };
    auto has = [&](int c) { return c < C && (!SHIFT || c + VEC > 0); };
    float dw[NV * VEC], f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) dw[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i][e] = 1.0f;
        if (w && has(c)) load_weight<VEC, SHIFT>(w, c, C, f[i]);
    }
    struct Row {
        Pack<T, VEC> h[NV], y[NV], u[NV];
    };
    auto fetch = [&](Row &k, int64_t row) {
        const size_t base = size_t(row) * C;
        const bool end = SHIFT && (rows - 1 - row) * C < VEC;
        load_row<SHIFT>(k.h, H + base, C, row < rows, end, col);
        load_row<SHIFT>(k.y, dY + base, C, row < rows, end, col);
        if (dH) load_row<SHIFT>(k.u, dH + base, C, row < rows, end, col);
    };
    Row k;
    if (PF) fetch(k, G);
    // the block's groups take the same number of turns, so that the reductions find every thread
    for (int64_t r0 = int64_t(blockIdx.x) * rpb; r0 < rows; r0 += step) {
        const int64_t row = r0 + grp;
        Row next;
        if (PF) fetch(next, row + step);  // (dX may be dY or dH: another row's, written by nobody else)
        else fetch(k, row);
        float2 s = make_float2(0.0f, 0.0f);  // sums of h^2 and of g h
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            mask_edge<SHIFT>(k.h[i], col(i), C);
            mask_edge<SHIFT>(k.y[i], col(i), C);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float h = widen(k.h[i].v[e]);
                s.x = fmaf(h, h, s.x);
                s.y = fmaf(widen(k.y[i].v[e]) * f[i][e], h, s.y);
            }
        }
        s = row_reduce(s, tpr, red, turn, [](float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); });
        const float rs = rsqrtf(fmaf(s.x, invC, eps));
        const float k2 = rs * rs * (s.y * invC);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (row < rows && has(c)) {
                Pack<T, VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = widen(k.h[i].v[e]), y = widen(k.y[i].v[e]);
                    float x = rs * (y * f[i][e] - h * k2);
                    if (dH) x += widen(k.u[i].v[e]);
                    o.v[e] = narrow<T>(x);
                    dw[i * VEC + e] = fmaf(y, h * rs, dw[i * VEC + e]);
                }
                store_part<T, VEC, SHIFT>(dX + size_t(row) * C + c, o, c, C);
            }
        }
        if (PF) k = next;
    }
    if (!part) return;
    float *out = rpb == 1 ? part + size_t(blockIdx.x) * C : acc_sm + grp * C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (c + e >= 0 && c + e < C) out[c + e] = dw[i * VEC + e];
    }
    if (rpb == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
        float a = 0.0f;
        for (int g = 0; g < rpb; ++g) a += acc_sm[g * C + c];
        part[size_t(blockIdx.x) * C + c] = a;
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
#pragma unroll 8
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
    bool shift;
};

// 16-byte vectors where the addresses are aligned (and the weight's, where the vectors follow its own), else single
// elements.  Then the threads of a row:
//   forward   as few as hold it in 32 / VEC vectors each, but four that share 64 bytes (a row per thread reads bytes far
//             apart), when there are rows enough to fill the SMs; else as many as the row has vectors.  In 8 bits with
//             a shift 16 / VEC where a warp is enough for that (100,000 x 333 bf16: 127 us, 143 with 32 / VEC).
//   backward  a vector each, or two of floats, up to 256 threads: a thread keeps its part of the weight and of dw.
template <typename T>
NormShape norm_shape(int64_t rows, int C, uintptr_t al, uintptr_t al_q, uintptr_t al_w, bool backward,
                     bool i8 = false)
{
    constexpr int V = 16 / int(sizeof(T));
    NormShape s;
    s.vec = V;
    s.shift = C % V != 0;
    auto vectors = [&] { return s.shift ? (C + 2 * (V - 1)) / V : C / s.vec; };  // of a row, at most
    if (al % 16 != 0 || al_q % V != 0 || (!s.shift && al_w % 16 != 0) || vectors() > kMaxEpt / V * kNormThreads) {
        s.vec = 1;
        s.shift = false;
    }
    const int cv = vectors(), most = kMaxEpt / s.vec;  // vectors of a row, and of a thread at most
    int tpr = 1;
    if (backward) {
        while (tpr * (sizeof(T) == 4 ? 2 : 1) < cv && tpr < kNormThreads) tpr <<= 1;
    } else {
        while ((i8 && s.shift && tpr * most / 2 < cv && tpr < 32) || tpr * most < cv || (tpr < 4 && tpr < cv)) tpr <<= 1;
        // few rows: spread each over more threads, down to one vector each
        while (tpr < cv && tpr < kNormThreads && rows * tpr < 148 * 512) tpr <<= 1;
    }
    s.tpr = tpr;
    s.threads = kNormThreads;
    if (!backward && tpr > 32) s.threads = tpr;  // a row of more than a warp has the block to itself
    const int need = (cv + tpr - 1) / tpr;
    s.nv = 1;
    while (s.nv < need) s.nv <<= 1;
    if (s.vec == 1 && s.nv > 1) s.nv = s.nv > 8 ? 32 : 8;
    return s;
}

template <typename T, int VEC, int NV, bool SHIFT, bool I8>
bt_status run_norm(const NormShape &s, const void *X, const void *R, const float *w, int64_t rows, int C, float eps,
                   bool norm, void *Hout, void *Y, int8_t *Q, float *scale, cudaStream_t st)
{
    const int rpb = s.threads / s.tpr;
    const int64_t grid = (rows + rpb - 1) / rpb;
    if (grid > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    k_rms_norm<T, VEC, NV, SHIFT, I8><<<unsigned(grid), s.threads, 0, st>>>(
        static_cast<const T *>(X), static_cast<const T *>(R), w, rows, C, 1.0f / float(C), s.tpr, eps, norm,
        static_cast<T *>(Hout), static_cast<T *>(Y), Q, scale);
    return cudaPeekAtLastError() == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

template <typename T, bool I8>
bt_status launch_norm(const void *X, const void *R, const float *w, int64_t rows, int C, float eps, bool norm,
                      void *Hout, void *Y, int8_t *Q, float *scale, cudaStream_t st)
{
    const uintptr_t al = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(R) |
                         reinterpret_cast<uintptr_t>(Hout) | reinterpret_cast<uintptr_t>(Y);
    const NormShape s =
        norm_shape<T>(rows, C, al, reinterpret_cast<uintptr_t>(Q), reinterpret_cast<uintptr_t>(w), false, I8);
#define BTS_NORM(V, N, S)                                                                                  \
    if (s.vec == V && s.nv == N && s.shift == S)                                                           \
        return run_norm<T, V, N, S, I8>(s, X, R, w, rows, C, eps, norm, Hout, Y, Q, scale, st);
    if constexpr (sizeof(T) == 2) {
        BTS_NORM(8, 1, false) BTS_NORM(8, 2, false) BTS_NORM(8, 4, false)
        BTS_NORM(8, 1, true) BTS_NORM(8, 2, true) BTS_NORM(8, 4, true)
    } else {
        BTS_NORM(4, 1, false) BTS_NORM(4, 2, false) BTS_NORM(4, 4, false) BTS_NORM(4, 8, false)
        BTS_NORM(4, 1, true) BTS_NORM(4, 2, true) BTS_NORM(4, 4, true) BTS_NORM(4, 8, true)
    }
    BTS_NORM(1, 1, false) BTS_NORM(1, 8, false) BTS_NORM(1, 32, false)
#undef BTS_NORM
    return BT_ERR_INTERNAL;
}


template <typename T, int VEC, int NV, bool SHIFT>
bt_status run_bwd(const NormShape &s, const void *dY, const void *dH, const void *H, const float *w, int64_t rows,
                  int C, float eps, void *dX, float *part, int64_t &blocks, cudaStream_t st)
{
    int dev = 0;
    const int sms = device_sms(&dev);
    if (sms == 0) return BT_ERR_CUDA;
    const int rpb = s.threads / s.tpr;
    // one wave; a multiple of 8 blocks, and so of 8 groups, where a group has several rows
    int64_t most = int64_t(sms) * (BwdShape<T, VEC, NV>::PER_SM) / 8 * 8;
    most = most < 8 ? 8 : most > kBwdBlocks ? kBwdBlocks : most;
    blocks = (rows + rpb - 1) / rpb;
    if (blocks > most) blocks = most;
    const size_t smem = part && rpb > 1 ? size_t(rpb) * C * 4 : 0;
    // rpb * C <= threads / tpr * tpr * 32 values: at most 32 KB
    k_rms_norm_bwd<T, VEC, NV, SHIFT><<<unsigned(blocks), s.threads, smem, st>>>(
        static_cast<const T *>(dY), static_cast<const T *>(dH), static_cast<const T *>(H), w, rows, C, 1.0f / float(C),
        s.tpr, eps, static_cast<T *>(dX), part);
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
        const NormShape s = norm_shape<T>(rows, C, al, 0, reinterpret_cast<uintptr_t>(w), true);
        bt_status r = BT_ERR_INTERNAL;
#define BTS_BWD(V, N, S)                         \
    if (s.vec == V && s.nv == N && s.shift == S) \
        r = run_bwd<T, V, N, S>(s, dY, dH, H, w, rows, C, eps, dX, dw ? part : nullptr, blocks, st);
        if constexpr (sizeof(T) == 2) {
            BTS_BWD(8, 1, false) BTS_BWD(8, 2, false) BTS_BWD(8, 4, false)
            BTS_BWD(8, 1, true) BTS_BWD(8, 2, true) BTS_BWD(8, 4, true)
        } else {
            BTS_BWD(4, 1, false) BTS_BWD(4, 2, false) BTS_BWD(4, 4, false) BTS_BWD(4, 8, false)
            BTS_BWD(4, 1, true) BTS_BWD(4, 2, true) BTS_BWD(4, 4, true) BTS_BWD(4, 8, true)
        }
        BTS_BWD(1, 1, false) BTS_BWD(1, 8, false) BTS_BWD(1, 32, false)
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

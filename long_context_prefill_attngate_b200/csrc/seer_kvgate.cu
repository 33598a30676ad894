// seer_kvgate.cu — the gate's key rows from the quantised cache.
//
//   Kt_j = RoPE_j( pool_{t in block j, t < len}(z_t + s_t n_t) @ Wk )
//
// One kernel: a CTA pools sixteen blocks of a head and projects them.
//  * Pooling reads the K half of each record once.  The mean is an MMA too: the codes
//    are the bf16 numbers n 2^-133 on M (as in the decode kernel), a group's scales
//    are two columns of N times a power of two of the block's largest (exact down to
//    2^-116 of it), and z is summed in fp32.  Half an integer operation an element
//    instead of two and two fp32 ones.
//    Max and min (the other pooling) take z + s n element by element; their
//    warps share a block's rows when the CTA has few blocks.
//  * Projection: sixteen pooled rows are the M of an mma.sync m16n8k16 (the
//    refresh of a decode step has one row; a tcgen05 tile would be 1/128
//    full).  Wk is bf16 as it is; a pooled value enters as three bf16 parts,
//    x = hi + mid + lo to 24 bits, so a product loses nothing and the sums are
//    fp32 as with plain fp32 FMAs.
//  * Rotation as in the bf16 cache's key rows: frequency and angle in double,
//    reduced modulo 2 pi, then fp32.
//
// 512 blocks of 8 heads at 4 bits (D = d_gate = 128): 9.9 us for 23 MB, of which the
// pooling of a warp's two blocks, one after the other, is half, the projection and the
// rotation 8 % each (HBM alone would be 3.6 us; issue 40 %, DRAM 19 %: the phases wait for
// one another, and both CTAs of an SM are in the same one).  The last block of 4
// sequences (max+min, 8 bits): 5.0 us, all latency.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kGateThreads = 256;
constexpr int kGateRows = 16;                            // blocks of a CTA: the M of the MMA
constexpr int kPad = 8;                                  // bf16 padding of shared rows: ldmatrix without bank conflicts

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix2_trans(uint32_t &r0, uint32_t &r1, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
}

// A NaN wins, as it does in a sum.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// v[NV] of each of the eight lanes that differ in bits 2..4, joined: the lane
// whose bits are i ends with the values [i NV/8, (i + 1) NV/8) in v[0 ..].
template <bool MAX, int NV>
__device__ __forceinline__ void reduce_scatter(float (&v)[NV], int lane)
{
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        const int off = 16 >> step, n = NV >> (step + 1);
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            const float got = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = MAX ? max_nan(keep, got) : min_nan(keep, got);
        }
    }
}

// Order-preserving keys, a NaN above everything: a maximum by atomicMax.
__device__ __forceinline__ uint32_t max_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return x != x ? 0xFFFFFFFFu : u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_max_key(uint32_t k)
{
    return k == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k);
}

template <int N>
__device__ __forceinline__ void ldg_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N == 8) {
        const uint4 x = load(reinterpret_cast<const uint4 *>(p)), y = load(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    } else if constexpr (N == 4) {
        const uint4 x = load(reinterpret_cast<const uint4 *>(p));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = load(reinterpret_cast<const uint2 *>(p));
        w[0] = x.x, w[1] = x.y;
    } else {
        static_assert(N == 1);
        w[0] = load(reinterpret_cast<const uint32_t *>(p));
    }
}

// Two pooled values as three bf16 parts each.
__device__ __forceinline__ void put_parts(__nv_bfloat16 *at, int part_stride, float x, float y)
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 part = __floats2bfloat162_rn(x, y);
        *reinterpret_cast<__nv_bfloat162 *>(at + i * part_stride) = part;
        x -= __low2float(part);
        y -= __high2float(part);
    }
}

// The mean of block (page, kvh), `rows` tokens of it, by one warp into row[D].
// A lane has the words of its eighth of a row, gid, of four tokens of every 16.
// An A operand's pair is two elements of one word, so its even and odd places sum
// up for different elements: a group's scales stand in two columns of N, once in
// the even places (zero in the odd ones) and once in the odd.
template <int BITS, int D>
__device__ __forceinline__ void pool_mean(const uint8_t *rec, int rows, float *row, int lane)
{
    using F = KvFmt<BITS, D>;
    constexpr int VW = F::R / 32, U = BITS == 4 ? 2 : 1;  // a lane's words of a row, MMAs of a word
    const int gid = lane >> 2, tig = lane & 3;
    // every load of the block first (rows behind its tokens too: their scales count as 0)
    uint32_t w[4][4][VW], par[4][4];                     // [tile][row of the lane]
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = (16 * mt + 4 * i + tig) % 32;  // four whole rows a load
            const int at = BITS == 8 && D == 128 ? ((gid >> 2) ^ (t & 1)) * 64 + (gid & 3) * 16 : gid * (F::R / 8);
            ldg_words(w[mt][i], rec + mt / 2 * F::HALF + t * F::R + at);
        }
    // scales of group gid / 2 and the sum of its zeros
    const int gr = gid >> 1;
    uint32_t smax = 0;
    float zs = 0.f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * mt + 4 * i + tig;
            par[mt][i] = gr < F::NG && t < rows ? load(reinterpret_cast<const uint32_t *>(
                                                            rec + t / 32 * F::HALF + F::kParK + t % 32 * F::PAR) + gr)
                                                : 0u;
        }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            smax = __vmaxu2(smax, par[mt][i]);
            zs = fmaf(kv_zero(par[mt][i]), 0.015625f, zs);
        }
    zs += __shfl_xor_sync(0xffffffffu, zs, 1);
    zs += __shfl_xor_sync(0xffffffffu, zs, 2);
    smax = __reduce_max_sync(0xffffffffu, smax & 0xFFFFu);
    // scales to at most 2^124, those of 2^-3 and below by 2^127: exact in bf16 down to 2^-116 of the largest
    const int uf = min(254, 377 - (int)(smax >> 7));
    const float up = __uint_as_float((uint32_t)uf << 23);
    const unsigned first = gid & 1 ? 0x1044u : 0x4410u, second = gid & 1 ? 0x3244u : 0x4432u;
    float c[VW][U][4];
#pragma unroll
    for (int k = 0; k < VW; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
            c[k][u][0] = c[k][u][1] = c[k][u][2] = c[k][u][3] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t s2 = __byte_perm(__float_as_uint(kv_scale(par[mt][i]) * up),
                                            __float_as_uint(kv_scale(par[mt][i + 1]) * up), 0x7632);
            const uint32_t b0 = __byte_perm(s2, 0u, first), b1 = __byte_perm(s2, 0u, second);
#pragma unroll
            for (int k = 0; k < VW; ++k) {
                uint32_t x = w[mt][i][k], y = w[mt][i + 1][k];
                if constexpr (BITS == 4) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        mma_bf16(c[k][u], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, b0, b1);
                        x >>= 8;
                        y >>= 8;
                    }
                } else {
                    mma_bf16(c[k][0], __byte_perm(x, 0u, 0x4140), __byte_perm(x, 0u, 0x4342), __byte_perm(y, 0u, 0x4140),
                            __byte_perm(y, 0u, 0x4342), b0, b1);
                }
            }
        }
    // a lane holds the sums of the words whose group is tig: 2^133 / up, a 64th of each
    // (as z's), so that blocks of the largest values stay within fp32
    const float down = __uint_as_float((uint32_t)(127 + 133 - 6 - 64 - (uf - 127)) << 23), inv = 64.f / (float)rows;
    constexpr float kUnit = 18446744073709551616.f, kUnitOdd = BITS == 4 ? kUnit * 0.0625f : kUnit;        // 2^64
    const float z = __shfl_sync(0xffffffffu, zs, 8 * tig);
#pragma unroll
    for (int k = 0; k < VW; ++k) {
        int g, e0;                                       // group and first element of the word
        if (BITS == 4) {
            const int wd = gid * VW + k;
            g = wd % F::NG;
            e0 = 32 * g + wd / F::NG * 8;
        } else if (D == 128) {
            g = gid >> 2;
            e0 = 64 * g + 16 * k + 4 * (gid & 3);
        } else {
            g = 0;
            e0 = 16 * (gid * 2 % 4 + k) + 4 * (gid / 2);
        }
        if (tig != g)
            continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float v0 = c[k][u][0] * kUnit * down, v1 = c[k][u][1] * kUnit * down;
            const float v2 = c[k][u][2] * kUnitOdd * down, v3 = c[k][u][3] * kUnitOdd * down;
            float2 *at = reinterpret_cast<float2 *>(row + e0 + 2 * u);
            if (BITS == 4) {                             // elements 2u, 2u + 1 and four further
                at[0] = make_float2((v0 + z) * inv, (v2 + z) * inv);
                at[2] = make_float2((v1 + z) * inv, (v3 + z) * inv);
            } else {
                at[0] = make_float2((v0 + z) * inv, (v1 + z) * inv);
                at[1] = make_float2((v2 + z) * inv, (v3 + z) * inv);
            }
        }
    }
}

// The maxima and minima of the tokens [8 p0, 8 p1) of a block, by one warp,
// joined into keys kx[D] (of the maximum) and kx[D ..] (of minus the minimum).
template <int BITS, int D>
__device__ __forceinline__ void pool_extrema(const uint8_t *rec, int rows, int p0, int p1, uint32_t *kx, int lane)
{
    using F = KvFmt<BITS, D>;
    constexpr int KW = F::R / 16, NV = D / 4, EPW = 32 / BITS;   // a lane's words of a row, its elements, elements of a word
    const int gid = lane >> 2, tig = lane & 3;
    // value of a code's unit: by the parity of the element at 4 bits (2^-20, 2^-24)
    auto unit = [](int e) { return BITS == 4 && e % 2 ? 9.5367431640625e-7f : 5.9604644775390625e-8f; };
    float v[NV], v2[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        v[e] = -INFINITY;
        v2[e] = INFINITY;
    }
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
        const int t = 8 * p + gid;
        if (8 * p >= rows)
            break;
        const uint8_t *half = rec + t / 32 * F::HALF;
        uint32_t code[KW], par[F::NG];
        if constexpr (BITS == 8 && D == 128) {
            uint32_t (&lo)[4] = *reinterpret_cast<uint32_t (*)[4]>(code);
            uint32_t (&hi)[4] = *reinterpret_cast<uint32_t (*)[4]>(code + 4);
            ldg_words(lo, half + t % 32 * F::R + (t & 1) * 64 + tig * 16);
            ldg_words(hi, half + t % 32 * F::R + (~t & 1) * 64 + tig * 16);
        } else {
            ldg_words(code, half + t % 32 * F::R + tig * (F::R / 4));
        }
        ldg_words(par, half + F::kParK + t % 32 * F::PAR);
        const bool in = t < rows;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const uint32_t pr = par[k / (KW / F::NG)];
            const float s = kv_scale(pr), z = kv_zero(pr);
#pragma unroll
            for (int e = 0; e < EPW / 2; ++e) {          // two codes as fp16 subnormals, widened
                const int e0 = BITS == 4 ? e : 2 * e, e1 = BITS == 4 ? e + 4 : 2 * e + 1;
                const uint32_t h = BITS == 4 ? code[k] >> (e / 2 * 8) & (e % 2 ? 0x00F000F0u : 0x000F000Fu)
                                             : __byte_perm(code[k], 0u, e ? 0x4342 : 0x4140);
                const float2 n = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                const float2 x = fma2(n, both(s), both(z * unit(e0)));
                if (in) {
                    v[k * EPW + e0] = max_nan(v[k * EPW + e0], x.x);
                    v[k * EPW + e1] = max_nan(v[k * EPW + e1], x.y);
                    v2[k * EPW + e0] = min_nan(v2[k * EPW + e0], x.x);
                    v2[k * EPW + e1] = min_nan(v2[k * EPW + e1], x.y);
                }
            }
        }
    }
    reduce_scatter<true>(v, lane);
    reduce_scatter<false>(v2, lane);
    // the lane's values of the joined row: NV/8 neighbouring elements, from an even one on
    constexpr int N = NV / 8;
    const int at = gid * N, k = at / EPW;
    const int e0 = (BITS == 4 ? 32 * k + 8 * tig : 16 * k + 4 * tig) + at % EPW;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        atomicMax(kx + e0 + e, max_key(v[e] * (1.f / unit(e))));
        atomicMax(kx + D + e0 + e, max_key(-v2[e] * (1.f / unit(e))));
    }
}

template <int BITS, int D, bool MAXMIN>
__global__ void __launch_bounds__(kGateThreads, 2)
    kv_gate_kernel(KvView kv, int Hkv, int L, const int32_t *lens, int nb, int first, const __nv_bfloat16 *wk,
                   long long wk_stride, int dg, double log_freq, float *kt, int *status)
{
    using F = KvFmt<BITS, D>;
    constexpr int DK = MAXMIN ? 2 * D : D;
    constexpr int XS = DK + kPad;                        // shared row strides (elements)
    extern __shared__ __align__(16) uint8_t gsm[];
    const int dgp = (dg + 7) & ~7, ws = dgp + kPad, ys = dg + 1;
    __nv_bfloat16 *sw = reinterpret_cast<__nv_bfloat16 *>(gsm);          // [DK][ws]
    __nv_bfloat16 *sx = sw + DK * ws;                                    // [3][kGateRows][XS]
    double *sfreq = reinterpret_cast<double *>(sx + 3 * kGateRows * XS); // [dg / 2]
    float *sp = reinterpret_cast<float *>(sfreq + dg / 2);               // [kGateRows][DK] (even)
    float *sy = sp + kGateRows * DK;                                     // [kGateRows][ys]
    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const int j0 = first + (int)blockIdx.x * kGateRows;
    const int valid = min(kGateRows, nb - j0);
    __shared__ int s_page[kGateRows];
    // length and pages on their way while Wk is fetched
    const int len = lens != nullptr ? max(0, min(load(lens + b), L)) : L;
    int page = b * kv.max_blocks + j0 + (int)threadIdx.x;
    if (threadIdx.x < valid && kv.table != nullptr)
        page = load(kv.table + (long long)b * kv.max_blocks + j0 + threadIdx.x);

    // ---- Wk of the head on its way to shared memory
    const __nv_bfloat16 *w = wk + (long long)kvh * wk_stride;
    if (dg % 8 == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        const int ch = dg / 8, lg = 32 - __clz(ch - 1);  // 16-byte pieces of a row; a row's lanes, rounded up to 2^lg
        const int c = lane & ((1 << lg) - 1);
        if (c < ch)
            for (int r = (warp << (5 - lg)) + (lane >> lg); r < DK; r += (kGateThreads / 32) << (5 - lg))
                cp_async16(smem_u32(sw + r * ws + c * 8), w + r * dg + c * 8);
    } else {
        for (int i = threadIdx.x; i < DK * dgp; i += kGateThreads) {
            const int r = i / dgp, c = i % dgp;
            sw[r * ws + c] = c < dg ? w[(long long)r * dg + c] : __float2bfloat16_rn(0.f);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (threadIdx.x < dg / 2)
        sfreq[threadIdx.x] = exp(log_freq * (double)threadIdx.x);
    auto tokens = [&](int i) { return i < valid ? min(64, len - 64 * (j0 + i)) : 0; };
    if (threadIdx.x < valid) {                           // -1: a block without a token, or an entry that names no page
        const bool used = tokens(threadIdx.x) > 0, bad = page < 0 || page >= kv.n_pages;
        if (used && bad)
            set_status(status, kStatusPage);
        s_page[threadIdx.x] = used && !bad ? page : -1;
    }
    uint32_t *kx = reinterpret_cast<uint32_t *>(sp);     // max+min: the keys, no token yet
    if constexpr (MAXMIN)
        for (int i = threadIdx.x; i < valid * DK; i += kGateThreads)
            kx[i] = 0u;
    __syncthreads();

    // ---- pooling (rows of sx behind the last block stay unwritten: their
    // products are rows of their own, which nothing reads)
    constexpr int kWarps = kGateThreads / 32;
    auto record = [&](int i) -> const uint8_t * {        // null where block j0 + i has none
        return s_page[i] < 0 ? nullptr : kv_half<F>(kv, Hkv, s_page[i], kvh, 0);
    };
    if constexpr (MAXMIN) {
        const int parts = valid <= 4 ? kWarps : 1;       // warps that share a block: an eighth costs a fifth of the whole
        for (int u = warp; u < valid * parts; u += kWarps) {
            const int i = u / parts, p = u % parts;
            const uint8_t *rec = record(i);
            if (rec != nullptr)
                pool_extrema<BITS, D>(rec, tokens(i), p * (8 / parts), (p + 1) * (8 / parts), kx + i * DK, lane);
        }
    } else {
        for (int i = warp; i < valid; i += kWarps) {
            const uint8_t *rec = record(i);
            if (rec != nullptr)
                pool_mean<BITS, D>(rec, tokens(i), sp + i * DK, lane);
            else
                for (int e = lane; e < D; e += 32)
                    sp[i * DK + e] = 0.f;
        }
    }
    __syncthreads();
    for (int i = 2 * threadIdx.x; i < valid * DK; i += 2 * kGateThreads) {
        float2 x = *reinterpret_cast<const float2 *>(sp + i);
        if constexpr (MAXMIN) {
            auto value = [&](float key) {                // no token: 0
                const uint32_t k = __float_as_uint(key);
                return k == 0u ? 0.f : i % DK < D ? from_max_key(k) : -from_max_key(k);
            };
            x = make_float2(value(x.x), value(x.y));
        }
        put_parts(sx + i / DK * XS + i % DK, kGateRows * XS, x.x, x.y);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // ---- projection: a warp has eight columns, and eight 64 further on
    constexpr int kColStep = kGateThreads / 32 * 8;
    for (int n0 = warp * 8; n0 < dgp; n0 += 2 * kColStep) {
        const int n1 = n0 + kColStep < dgp ? n0 + kColStep : n0;
        float c[2][4] = {}, cl[2][4] = {};               // by the hi parts, by the other two
#pragma unroll 8
        for (int k0 = 0; k0 < DK; k0 += 16) {
            uint32_t b0, b1, d0, d1, x[4], y[4], z[4];
            ldmatrix2_trans(b0, b1, smem_u32(sw + (k0 + (lane & 15)) * ws + n0));
            ldmatrix2_trans(d0, d1, smem_u32(sw + (k0 + (lane & 15)) * ws + n1));
            const uint32_t xa = smem_u32(sx + (lane & 15) * XS + k0 + (lane >> 4) * 8);
            ldmatrix4(x, xa);
            ldmatrix4(y, xa + kGateRows * XS * 2);
            ldmatrix4(z, xa + 2 * kGateRows * XS * 2);
            mma_bf16(c[0], x, b0, b1);
            mma_bf16(c[1], x, d0, d1);
            mma_bf16(cl[0], y, b0, b1);
            mma_bf16(cl[1], y, d0, d1);
            mma_bf16(cl[0], z, b0, b1);
            mma_bf16(cl[1], z, d0, d1);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = (u ? n1 : n0) + 2 * tig + (e & 1);
                if (col < dg)
                    sy[(gid + (e >> 1) * 8) * ys + col] = c[u][e] + cl[u][e];
            }
    }
    __syncthreads();

    // ---- rotation, pairs (t, t + dg/2) at the position of the block
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const int half = dg / 2, lgh = half > 1 ? 32 - __clz(half - 1) : 0;   // a row's threads, rounded up to 2^lgh
    const int t = threadIdx.x & ((1 << lgh) - 1);
#pragma unroll 4
    for (int r = threadIdx.x >> lgh; r < (t < half ? valid : 0); r += kGateThreads >> lgh) {
        const int j = j0 + r;
        const double ang = (double)j * sfreq[t];
        const double red = ang - rint(ang * (1.0 / kTwoPi)) * kTwoPi;
        float sn, cs;
        sincosf((float)red, &sn, &cs);
        const float y0 = sy[r * ys + t], y1 = sy[r * ys + t + half];
        float *o = kt + ((long long)blockIdx.y * nb + j) * dg + t;
        o[0] = y0 * cs - y1 * sn;
        o[half] = y1 * cs + y0 * sn;
    }
}

constexpr size_t gate_smem(int DK, int dg)
{
    return sizeof(__nv_bfloat16) * ((size_t)DK * (((dg + 7) & ~7) + kPad) + 3 * kGateRows * (DK + kPad)) +
           sizeof(double) * (dg / 2) + sizeof(float) * kGateRows * (DK + dg + 1);
}

template <int BITS, int D, bool MAXMIN>
cudaError_t launch(int B, int Hkv, int L, const KvView &kv, const int32_t *lens, int first, const void *wk,
                   long long wk_stride, int dg, float theta, float *kt, int *status, cudaStream_t stream)
{
    constexpr int DK = MAXMIN ? 2 * D : D;
    const int nb = num_blocks(L);
    // the limit for every d_gate at once: another thread's call may lie between this one and the launch
    constexpr size_t kMost = gate_smem(DK, 256);
    static_assert(kMost <= 226 * 1024);
    const cudaError_t e = cudaFuncSetAttribute(kv_gate_kernel<BITS, D, MAXMIN>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess)
        return e;
    return launch_programmatic(kv_gate_kernel<BITS, D, MAXMIN>, dim3((nb - first + kGateRows - 1) / kGateRows, B * Hkv),
                               kGateThreads, gate_smem(DK, dg), stream, kv, Hkv, L, lens, nb, first,
                               static_cast<const __nv_bfloat16 *>(wk), wk_stride, dg, -2.0 * log((double)theta) / dg, kt,
                               status);
}

} // namespace

cudaError_t launch_gate_keys_quant(int bits, int B, int Hkv, int L, int d, int dg, float theta, bool k_maxmin,
                                   const KvView &kv, const int32_t *lens, const void *wk, long long wk_stride,
                                   int first_block, float *kt, int *status, cudaStream_t stream)
{
    if (first_block >= num_blocks(L))
        return cudaSuccess;
    const auto f = bits == 4 ? (d == 128 ? (k_maxmin ? launch<4, 128, true> : launch<4, 128, false>)
                                         : (k_maxmin ? launch<4, 64, true> : launch<4, 64, false>))
                             : (d == 128 ? (k_maxmin ? launch<8, 128, true> : launch<8, 128, false>)
                                         : (k_maxmin ? launch<8, 64, true> : launch<8, 64, false>));
    return f(B, Hkv, L, kv, lens, first_block, wk, wk_stride, dg, theta, kt, status, stream);
}

} // namespace seer

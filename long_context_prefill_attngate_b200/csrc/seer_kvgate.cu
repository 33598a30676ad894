// seer_kvgate.cu — the gate's key rows from the quantised cache.
//
//   Kt_j = RoPE_j( pool_{t in block j, t < len}(z_t + s_t n_t) @ Wk )
//
// One kernel: a CTA pools sixteen blocks of a head and projects them.
//  * Pooling reads the K half of each record once (HBM-bound for a whole
//    cache): a warp has a block at a time, a lane every fourth of eight rows'
//    words; sums of s n and of z in fp32, the 64 tokens joined by a
//    reduce-scatter over the eight lanes of a row's word.
//  * Projection: sixteen pooled rows are the M of an mma.sync m16n8k16 (the
//    refresh of a decode step has one row; a tcgen05 tile would be 1/128
//    full).  Wk is bf16 as it is; a pooled value enters as three bf16 parts,
//    x = hi + mid + lo to 24 bits, so a product loses nothing and the sums are
//    fp32 as with plain fp32 FMAs.
//  * Rotation as in the bf16 cache's key rows: frequency and angle in double,
//    reduced modulo 2 pi, then fp32.
#include <cuda_bf16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kGateThreads = 256;
constexpr int kGateRows = 16;                            // blocks of a CTA: the M of the MMA
constexpr int kPad = 8;                                  // bf16 padding of shared rows: ldmatrix without bank conflicts

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
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

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

enum { kSum = 0, kMax = 1, kMin = 2 };

__device__ __forceinline__ float join(int op, float a, float b)
{
    return op == kSum ? a + b : op == kMax ? max_nan(a, b) : min_nan(a, b);
}

// v[NV] of each of the eight lanes that differ in bits 2..4, joined: lane bits
// 2..4 = i end with the values [i NV/8, (i + 1) NV/8) in v[0 ..].
template <int OP, int NV>
__device__ __forceinline__ void reduce_scatter(float (&v)[NV], int lane)
{
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        const int off = 16 >> step, n = NV >> (step + 1);
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = join(OP, keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
}

// x[0 .. N) of one pooled row from element e on, as three bf16 parts.
template <int N>
__device__ __forceinline__ void put_parts(__nv_bfloat16 *row, int part_stride, int e, const float *x)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
        const float r = x[i] - __bfloat162float(hi);
        const __nv_bfloat16 mid = __float2bfloat16_rn(r);
        row[e + i] = hi;
        row[part_stride + e + i] = mid;
        row[2 * part_stride + e + i] = __float2bfloat16_rn(r - __bfloat162float(mid));
    }
}

template <int BITS, int D, bool MAXMIN>
__global__ void __launch_bounds__(kGateThreads)
    kv_gate_kernel(KvView kv, int Hkv, int L, const int32_t *lens, int nb, int first, const __nv_bfloat16 *wk,
                   long long wk_stride, int dg, double theta, float *kt, int *status)
{
    using F = KvFmt<BITS, D>;
    constexpr int DK = MAXMIN ? 2 * D : D;
    constexpr int XS = DK + kPad;                        // shared row strides (elements)
    constexpr int KW = F::R / 16, NV = D / 4, EPW = 32 / BITS;   // a lane's words of a row, its elements, elements of a word
    extern __shared__ __align__(16) uint8_t gsm[];
    const int dgp = (dg + 7) & ~7, ws = dgp + kPad, ys = dg + 1;
    __nv_bfloat16 *sw = reinterpret_cast<__nv_bfloat16 *>(gsm);          // [DK][ws]
    __nv_bfloat16 *sx = sw + DK * ws;                                    // [3][kGateRows][XS]
    double *sfreq = reinterpret_cast<double *>(sx + 3 * kGateRows * XS); // [dg / 2]
    float *sy = reinterpret_cast<float *>(sfreq + dg / 2);               // [kGateRows][ys]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const int j0 = first + (int)blockIdx.x * kGateRows;
    const int len = lens != nullptr ? max(0, min(__ldg(lens + b), L)) : L;

    // ---- Wk of the head on its way to shared memory
    const __nv_bfloat16 *w = wk + (long long)kvh * wk_stride;
    if (dg % 8 == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        const int ch = dg / 8;
        for (int i = threadIdx.x; i < DK * ch; i += kGateThreads)
            cp_async16(smem_u32(sw + i / ch * ws + i % ch * 8), w + (long long)i * 8);
    } else {
        for (int i = threadIdx.x; i < DK * dgp; i += kGateThreads) {
            const int r = i / dgp, c = i % dgp;
            sw[r * ws + c] = c < dg ? w[(long long)r * dg + c] : __float2bfloat16_rn(0.f);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (threadIdx.x < dg / 2)
        sfreq[threadIdx.x] = pow(theta, -2.0 * (double)threadIdx.x / (double)dg);

    // ---- pooling: warp w has blocks w, w + 8
    for (int i = warp; i < kGateRows; i += kGateThreads / 32) {
        const int j = j0 + i;
        const int rows = j < nb ? min(64, len - 64 * j) : 0;
        const int page = rows > 0 ? kv_page(kv, b, j, status) : -1;
        float v[NV], v2[MAXMIN ? NV : 1], zs[F::NG];
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            v[e] = MAXMIN ? -INFINITY : 0.f;
            if (MAXMIN)
                v2[e] = INFINITY;
        }
#pragma unroll
        for (int gr = 0; gr < F::NG; ++gr)
            zs[gr] = 0.f;
        if (page >= 0) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, hf);
                uint32_t code[4][KW], par[4][F::NG];
                if (32 * hf >= rows)
                    break;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = gid + 8 * r;
                    if constexpr (BITS == 8 && D == 128) {
                        const uint4 x0 = __ldg(reinterpret_cast<const uint4 *>(half + t * F::R + (t & 1) * 64 + tig * 16));
                        const uint4 x1 = __ldg(reinterpret_cast<const uint4 *>(half + t * F::R + (~t & 1) * 64 + tig * 16));
                        code[r][0] = x0.x, code[r][1] = x0.y, code[r][2] = x0.z, code[r][3] = x0.w;
                        code[r][4] = x1.x, code[r][5] = x1.y, code[r][6] = x1.z, code[r][7] = x1.w;
                    } else if constexpr (KW == 4) {
                        const uint4 x0 = __ldg(reinterpret_cast<const uint4 *>(half + t * F::R + tig * 16));
                        code[r][0] = x0.x, code[r][1] = x0.y, code[r][2] = x0.z, code[r][3] = x0.w;
                    } else {
                        const uint2 x0 = __ldg(reinterpret_cast<const uint2 *>(half + t * F::R + tig * 8));
                        code[r][0] = x0.x, code[r][1] = x0.y;
                    }
#pragma unroll
                    for (int gr = 0; gr < F::NG; ++gr)
                        par[r][gr] = __ldg(reinterpret_cast<const uint32_t *>(half + F::kParK + t * F::PAR) + gr);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = 32 * hf + gid + 8 * r < rows;
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        const int gr = k / (KW / F::NG);
                        const uint32_t p = in ? par[r][gr] : 0u;
                        const float s = kv_scale(p), z = kv_zero(p);
                        if (!MAXMIN && k % (KW / F::NG) == 0)
                            zs[gr] += z;
#pragma unroll
                        for (int e = 0; e < EPW; e += 2) {
                            const uint32_t q0 = code[r][k] >> (e * BITS), q1 = code[r][k] >> ((e + 1) * BITS);
                            const float2 n = add2(make_float2(__uint_as_float((q0 & (uint32_t)F::TOP) | 0x4B000000u),
                                                              __uint_as_float((q1 & (uint32_t)F::TOP) | 0x4B000000u)),
                                                  both(-8388608.f));
                            float &a0 = v[k * EPW + e], &a1 = v[k * EPW + e + 1];
                            if constexpr (MAXMIN) {
                                const float2 x = fma2(n, both(s), both(z));
                                a0 = in ? max_nan(a0, x.x) : a0;
                                a1 = in ? max_nan(a1, x.y) : a1;
                                v2[k * EPW + e] = in ? min_nan(v2[k * EPW + e], x.x) : v2[k * EPW + e];
                                v2[k * EPW + e + 1] = in ? min_nan(v2[k * EPW + e + 1], x.y) : v2[k * EPW + e + 1];
                            } else {
                                const float2 x = fma2(n, both(s), make_float2(a0, a1));
                                a0 = x.x;
                                a1 = x.y;
                            }
                        }
                    }
                }
            }
        }
        // the lane's values of the joined row: NV/8 neighbouring elements
        constexpr int N = NV / 8;
        const int at = gid * N, k = at / EPW;            // value index, its word
        const int e0 = (BITS == 4 ? 32 * k + 8 * tig : 16 * k + 4 * tig) + at % EPW;
        __nv_bfloat16 *row = sx + i * XS;
        reduce_scatter<MAXMIN ? kMax : kSum>(v, lane);
        if constexpr (MAXMIN) {
            reduce_scatter<kMin>(v2, lane);
            if (page < 0)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    v[e] = v2[e] = 0.f;
            put_parts<N>(row, kGateRows * XS, e0, v);
            put_parts<N>(row, kGateRows * XS, D + e0, v2);
        } else {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                for (int gr = 0; gr < F::NG; ++gr)
                    zs[gr] += __shfl_xor_sync(0xffffffffu, zs[gr], off);
            float z = zs[0];
#pragma unroll
            for (int gr = 1; gr < F::NG; ++gr)
                z = k / (KW / F::NG) == gr ? zs[gr] : z;
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[e] = page < 0 ? 0.f : (v[e] + z) / (float)rows;
            put_parts<N>(row, kGateRows * XS, e0, v);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // ---- projection: eight columns at a time
    for (int n0 = warp * 8; n0 < dgp; n0 += kGateThreads / 32 * 8) {
        float c[4] = {0.f, 0.f, 0.f, 0.f}, cl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int k0 = 0; k0 < DK; k0 += 16) {
            uint32_t b0, b1, x[4];
            ldmatrix2_trans(b0, b1, smem_u32(sw + (k0 + (lane & 15)) * ws + n0));
            const uint32_t xa = smem_u32(sx + (lane & 15) * XS + k0 + (lane >> 4) * 8);
            ldmatrix4(x, xa);
            mma_bf16(c, x, b0, b1);
            ldmatrix4(x, xa + kGateRows * XS * 2);
            mma_bf16(cl, x, b0, b1);
            ldmatrix4(x, xa + 2 * kGateRows * XS * 2);
            mma_bf16(cl, x, b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = n0 + 2 * tig + (e & 1);
            if (col < dg)
                sy[(gid + (e >> 1) * 8) * ys + col] = c[e] + cl[e];
        }
    }
    __syncthreads();

    // ---- rotation, pairs (t, t + dg/2) at the position of the block
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const int half = dg / 2;
    for (int i = threadIdx.x; i < kGateRows * half; i += kGateThreads) {
        const int r = i / half, t = i % half, j = j0 + r;
        if (j >= nb)
            break;
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

template <int BITS, int D, bool MAXMIN>
cudaError_t launch(int B, int Hkv, int L, const KvView &kv, const int32_t *lens, int first, const void *wk,
                   long long wk_stride, int dg, float theta, float *kt, int *status, cudaStream_t stream)
{
    constexpr int DK = MAXMIN ? 2 * D : D;
    const int nb = num_blocks(L), dgp = (dg + 7) & ~7;
    const size_t smem = sizeof(__nv_bfloat16) * ((size_t)DK * (dgp + kPad) + 3 * kGateRows * (DK + kPad)) +
                        sizeof(double) * (dg / 2) + sizeof(float) * kGateRows * (dg + 1);
    const cudaError_t e = cudaFuncSetAttribute(kv_gate_kernel<BITS, D, MAXMIN>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    kv_gate_kernel<BITS, D, MAXMIN><<<dim3((nb - first + kGateRows - 1) / kGateRows, B * Hkv), kGateThreads, smem, stream>>>(
        kv, Hkv, L, lens, nb, first, static_cast<const __nv_bfloat16 *>(wk), wk_stride, dg, (double)theta, kt, status);
    return cudaGetLastError();
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

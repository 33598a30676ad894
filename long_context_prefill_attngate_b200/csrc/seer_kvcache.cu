// seer_kvcache.cu — rows of K and V quantised into the cache, and read back.
//
// A group of G elements (32 at 4 bits, 64 at 8) is stored as
//   z = min(x),  s = bf16((max(x) - min(x)) / (2^bits - 1)),
//   n = nearest integer to (x - z) / s, ties to even, at most 2^bits - 1
// and stands for z + s n.  z is an element, so bf16 holds it exactly; the
// rounding of s only moves the levels, since n is taken against the stored s.
// s below 2^-100 is stored as 0, a group with a NaN or a magnitude of 2^126 or
// more as s = 0, z = NaN.
//
// Both directions are bound by HBM: a row costs 2 D bytes on the bf16 side and
// D bits / 8 + 4 D / G on the other.
#include <cuda_bf16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kRowThreads = 256;

// A lane holds eight elements of a row (one 16-byte access on the bf16 side):
// 16 lanes a row at D = 128, 8 at D = 64.
template <int BITS, int D>
struct RowMap {
    using F = KvFmt<BITS, D>;
    static constexpr int CH = D / 8;                     // lanes of a row
    static constexpr int RPW = 32 / CH;                  // rows of a warp's access
    static constexpr int GL = F::G / 8;                  // lanes of a group
    static constexpr int NW = BITS / 4;                  // code words of a lane
};

// Row t of sequence b: the half record that holds it, and its token there; null
// when the row is not to be touched (behind the count, or outside the cache).
template <class F>
__device__ __forceinline__ uint8_t *locate(const KvView &kv, int Hkv, int b, int kvh, int t, int rows,
                                           const int32_t *start, int start_pos, int *tok, int *status)
{
    if (t >= rows)
        return nullptr;
    const long long pos = (long long)(start != nullptr ? __ldg(start + b) : 0) + start_pos + t;
    if (pos < 0 || pos >= 64LL * kv.max_blocks) {
        set_status(status, kStatusPage);
        return nullptr;
    }
    const int page = kv_page(kv, b, (int)(pos / 64), status);
    if (page < 0)
        return nullptr;
    *tok = (int)(pos % 32);
    return kv_half<F>(kv, Hkv, page, kvh, (int)(pos % 64) / 32);
}

// The code words of a V row change lanes between element order (lane c: the
// words of elements 8c .. 8c+7) and the order they lie in (lane c: four bytes
// at offset v_place at 4 bits, eight at 8).  At 4 bits a lane's word is two
// 16-bit runs of chunks 2q and 2q + 1 (q = c % 4) of group c / 4, and a stored
// word is two groups of one chunk: a 2 x 2 exchange within the row.
template <int BITS, int D>
__device__ __forceinline__ int v_place(int t, int c)
{
    using F = KvFmt<BITS, D>;
    if (BITS == 8)
        return t * F::R + ((c % 8) ^ F::v_swizzle(t)) * (8 * F::NG) + (c / 8) * 8;
    const int i = c / 4, q = c % 4;
    const int chunk = F::NG == 4 ? 2 * q + (i >> 1) : 2 * q + i;
    return t * F::R + (chunk ^ F::v_swizzle(t)) * (2 * F::NG) + (F::NG == 4 ? (i & 1) * 4 : 0);
}

template <int D>
__device__ __forceinline__ uint32_t v4_exchange(uint32_t w, int lane, bool store)
{
    const int base = lane & ~(D / 8 - 1), c = lane & (D / 8 - 1), i = c / 4, q = c % 4;
    int s0, s1, half;
    if (D == 128) {
        s0 = store ? 2 * (i & 1) : i >> 1;
        s1 = store ? s0 + 1 : s0 + 2;
        half = store ? i >> 1 : i & 1;
    } else {
        s0 = 0;
        s1 = 1;
        half = i;
    }
    const uint32_t v0 = __shfl_sync(0xffffffffu, w, base + 4 * s0 + q), v1 = __shfl_sync(0xffffffffu, w, base + 4 * s1 + q);
    return __byte_perm(v0, v1, half ? 0x7632 : 0x5410);
}

// At 8 bits a K row's word c lies at 16 p + 4 (c % 4) + (c / 4) % 4: lane c
// stores or loads eight bytes, the words (j, t) and (j + 1, t) with j = c / 2
// of the sixteen elements' index, against words 2c and 2c + 1 in element order.
template <int D>
__device__ __forceinline__ int k8_place(int tok, int c)
{
    using F = KvFmt<8, D>;
    const int p = D == 128 ? (c / 8) ^ (tok & 1) : 0;
    return tok * F::R + p * 64 + (c % 8) / 2 * 16 + (c % 2) * 8;
}

template <int D>
__device__ __forceinline__ uint2 k8_to_store(uint2 w, int lane)
{
    const int base = lane & ~(D / 8 - 1), c = lane & (D / 8 - 1);
    const int t = (c % 8) / 2, src = base + 2 * (4 * (c / 8) + 2 * (c % 2)) + t / 2;
    const uint32_t x0 = __shfl_sync(0xffffffffu, w.x, src), y0 = __shfl_sync(0xffffffffu, w.y, src);
    const uint32_t x1 = __shfl_sync(0xffffffffu, w.x, src + 2), y1 = __shfl_sync(0xffffffffu, w.y, src + 2);
    return t & 1 ? make_uint2(y0, y1) : make_uint2(x0, x1);
}

template <int D>
__device__ __forceinline__ uint2 k8_from_store(uint2 w, int lane)
{
    const int base = lane & ~(D / 8 - 1), c = lane & (D / 8 - 1);
    // words 2c, 2c + 1: j = c / 2, t = 2 (c % 2) and t + 1, each in the lane of (p, t, j pair)
    const int j = c / 2, t = 2 * (c % 2), src = base + 8 * (j / 4) + 2 * t + (j % 4) / 2;
    const uint32_t x0 = __shfl_sync(0xffffffffu, w.x, src), y0 = __shfl_sync(0xffffffffu, w.y, src);
    const uint32_t x1 = __shfl_sync(0xffffffffu, w.x, src + 2), y1 = __shfl_sync(0xffffffffu, w.y, src + 2);
    return j & 1 ? make_uint2(y0, y1) : make_uint2(x0, x1);
}

// U rows per lane, their loads in flight together.
template <int BITS, int D, int U>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(KvView kv, KvRows x, int Hkv, int n, const int32_t *start,
                                                               const int32_t *count, int start_pos, int *status)
{
    using F = KvFmt<BITS, D>;
    using M = RowMap<BITS, D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % M::CH;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const bool is_v = blockIdx.z != 0;
    const int rows = count != nullptr ? min(__ldg(count + b), n) : n;
    const int t0 = (int)blockIdx.x * (kRowThreads / 32 * M::RPW * U) + warp * (M::RPW * U) + lane / M::CH;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(is_v ? x.v : x.k) +
                               (is_v ? b * x.v_stride_b + kvh * x.v_stride_h : b * x.k_stride_b + kvh * x.k_stride_h) + 8 * c;
    const long long st = is_v ? x.v_stride_t : x.k_stride_t;
    if (t0 - lane / M::CH >= rows)
        return;                                          // the whole warp
    uint4 in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u * M::RPW;
        in[u] = t < rows ? __ldg(reinterpret_cast<const uint4 *>(src + t * st)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
        __nv_bfloat162 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
        __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
        __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
#pragma unroll
        for (int off = 1; off < M::GL; off <<= 1) {
            mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        const __nv_bfloat16 lob = __hmin_nan(mn.x, mn.y), hib = __hmax_nan(mx.x, mx.y);
        const float lo = __bfloat162float(lob), hi = __bfloat162float(hib);
        const bool ok = lo > -8.507059173023462e37f && hi < 8.507059173023462e37f;   // 2^126; false for a NaN
        __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, (float)F::TOP));
        if (!ok || __bfloat162float(sb) < 7.888609052210118e-31f)                   // 2^-100
            sb = __float2bfloat16_rn(0.f);
        const float s = __bfloat162float(sb), inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
        const float zr = ok ? lo : 0.f;
        // n: t / s rounded by an addition, then checked against the exact remainder
        // t - n s (a few bits of bf16 products): where the reciprocal's error put
        // it on the wrong side of a half, or at a half on the odd side, it moves by one
        constexpr float kMagic = 12582912.f;             // 1.5 2^23
        float q[8], worst = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
            const float d = v - zr;
            q[e] = fmaf(d, inv, kMagic) - kMagic;
            worst = fmaxf(worst, fabsf(fmaf(-q[e], s, d)));
        }
        if (2.f * worst >= s) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
                const float r = 2.f * fmaf(-q[e], s, v - zr);
                const bool odd = ((int)q[e] & 1) != 0;
                q[e] += r > s || (r == s && odd) ? 1.f : -r > s || (-r == s && odd) ? -1.f : 0.f;
            }
        }
        uint32_t code[M::NW] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t n_e = s > 0.f ? __float_as_uint(fminf(q[e], (float)F::TOP) + kMagic) & (uint32_t)F::TOP : 0u;
            code[e * BITS / 32] |= n_e << (e * BITS % 32);
        }
        const int t = t0 + u * M::RPW;
        int tok = 0;
        uint8_t *half = locate<F>(kv, Hkv, b, kvh, t, rows, start, start_pos, &tok, status);
        uint8_t *base = half + (is_v ? F::kCodeV : 0);
        if constexpr (BITS == 4) {
            const uint32_t out = is_v ? v4_exchange<D>(code[0], lane, true) : code[0];
            if (half != nullptr)
                *reinterpret_cast<uint32_t *>(base + (is_v ? v_place<4, D>(tok, c) : F::k_off(tok, 4 * c))) = out;
        } else {
            uint2 out = make_uint2(code[0], code[1]);
            if (!is_v)
                out = k8_to_store<D>(out, lane);
            if (half != nullptr)
                *reinterpret_cast<uint2 *>(base + (is_v ? v_place<8, D>(tok, c) : k8_place<D>(tok, c))) = out;
        }
        if (half != nullptr && c % M::GL == 0)
            *reinterpret_cast<uint32_t *>(half + (is_v ? F::kParV : F::kParK) + tok * F::PAR + c / M::GL * 4) =
                (uint32_t)__bfloat16_as_ushort(sb) | (ok ? (uint32_t)__bfloat16_as_ushort(lob) : 0x7FC0u) << 16;
    }
}

template <int BITS, int D, int U>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(KvView kv, int Hkv, int n, const int32_t *start,
                                                              const int32_t *count, int start_pos,
                                                              __nv_bfloat16 *k, __nv_bfloat16 *v, int *status)
{
    using F = KvFmt<BITS, D>;
    using M = RowMap<BITS, D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % M::CH;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const bool is_v = k == nullptr || blockIdx.z != 0;
    const int rows = count != nullptr ? min(__ldg(count + b), n) : n;
    const int t0 = (int)blockIdx.x * (kRowThreads / 32 * M::RPW * U) + warp * (M::RPW * U) + lane / M::CH;
    if (t0 - lane / M::CH >= rows)
        return;                                          // the whole warp
    uint32_t code[U][M::NW], par[U];
    bool have[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int tok = 0;
        const uint8_t *half = locate<F>(kv, Hkv, b, kvh, t0 + u * M::RPW, rows, start, start_pos, &tok, status);
        have[u] = half != nullptr;
        code[u][0] = code[u][M::NW - 1] = par[u] = 0u;
        if (have[u]) {
            const uint8_t *base = half + (is_v ? F::kCodeV : 0);
            if constexpr (BITS == 4) {
                code[u][0] = *reinterpret_cast<const uint32_t *>(base + (is_v ? v_place<4, D>(tok, c) : F::k_off(tok, 4 * c)));
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(base + (is_v ? v_place<8, D>(tok, c) : k8_place<D>(tok, c)));
                code[u][0] = w.x;
                code[u][M::NW - 1] = w.y;
            }
            par[u] = *reinterpret_cast<const uint32_t *>(half + (is_v ? F::kParV : F::kParK) + tok * F::PAR + c / M::GL * 4);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (BITS == 4) {
            if (is_v)
                code[u][0] = v4_exchange<D>(code[u][0], lane, false);
        } else if (!is_v) {
            const uint2 w = k8_from_store<D>(make_uint2(code[u][0], code[u][1]), lane);
            code[u][0] = w.x;
            code[u][M::NW - 1] = w.y;
        }
        const float s = kv_scale(par[u]), z = kv_zero(par[u]);
        uint4 r;
        uint32_t *rw = &r.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t q = code[u][(2 * i + e) * BITS / 32] >> ((2 * i + e) * BITS % 32) & (uint32_t)F::TOP;
                f[e] = fmaf(s, __uint_as_float(q | 0x4B000000u) - 8388608.f, z);    // q as a float: 2^23 + q, less 2^23
            }
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
            rw[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (have[u])
            *reinterpret_cast<uint4 *>((is_v ? v : k) + ((long long)blockIdx.y * n + t0 + u * M::RPW) * D + 8 * c) = r;
    }
}

// Rows per lane: four where that still leaves two CTAs an SM, else one.
bool four_rows(int B, int Hkv, int n, int d)
{
    return (long long)B * Hkv * n * 2 >= 4LL * 296 * (kRowThreads / (d / 8));
}

template <int BITS, int D, int U>
cudaError_t write_rows(int B, int Hkv, int n, const KvView &kv, const KvRows &x, const int32_t *start,
                       const int32_t *count, int start_pos, int *status, cudaStream_t stream)
{
    const int per = kRowThreads / (D / 8) * U;
    kv_write_kernel<BITS, D, U><<<dim3((n + per - 1) / per, B * Hkv, 2), kRowThreads, 0, stream>>>(
        kv, x, Hkv, n, start, count, start_pos, status);
    return cudaGetLastError();
}

template <int BITS, int D, int U>
cudaError_t read_rows(int B, int Hkv, int n, const KvView &kv, const int32_t *start, const int32_t *count, int start_pos,
                      void *k, void *v, int *status, cudaStream_t stream)
{
    const int per = kRowThreads / (D / 8) * U;
    kv_read_kernel<BITS, D, U>
        <<<dim3((n + per - 1) / per, B * Hkv, k != nullptr && v != nullptr ? 2 : 1), kRowThreads, 0, stream>>>(
            kv, Hkv, n, start, count, start_pos, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), status);
    return cudaGetLastError();
}

} // namespace

int kv_record_bytes(int bits, int d)
{
    if (bits == 4)
        return d == 128 ? KvFmt<4, 128>::REC : d == 64 ? KvFmt<4, 64>::REC : 0;
    if (bits == 8)
        return d == 128 ? KvFmt<8, 128>::REC : d == 64 ? KvFmt<8, 64>::REC : 0;
    return 0;
}

cudaError_t launch_kv_write(int bits, int B, int Hkv, int n, int d, const KvView &kv, const KvRows &x,
                            const int32_t *start, const int32_t *count, int start_pos, int *status, cudaStream_t stream)
{
    const bool four = four_rows(B, Hkv, n, d);
    auto f = bits == 4 ? (d == 128 ? (four ? write_rows<4, 128, 4> : write_rows<4, 128, 1>)
                                   : (four ? write_rows<4, 64, 4> : write_rows<4, 64, 1>))
                       : (d == 128 ? (four ? write_rows<8, 128, 4> : write_rows<8, 128, 1>)
                                   : (four ? write_rows<8, 64, 4> : write_rows<8, 64, 1>));
    return f(B, Hkv, n, kv, x, start, count, start_pos, status, stream);
}

cudaError_t launch_kv_read(int bits, int B, int Hkv, int n, int d, const KvView &kv, const int32_t *start,
                           const int32_t *count, int start_pos, void *k, void *v, int *status, cudaStream_t stream)
{
    const bool four = four_rows(B, Hkv, n, d);
    auto f = bits == 4 ? (d == 128 ? (four ? read_rows<4, 128, 4> : read_rows<4, 128, 1>)
                                   : (four ? read_rows<4, 64, 4> : read_rows<4, 64, 1>))
                       : (d == 128 ? (four ? read_rows<8, 128, 4> : read_rows<8, 128, 1>)
                                   : (four ? read_rows<8, 64, 4> : read_rows<8, 64, 1>));
    return f(B, Hkv, n, kv, start, count, start_pos, k, v, status, stream);
}

} // namespace seer

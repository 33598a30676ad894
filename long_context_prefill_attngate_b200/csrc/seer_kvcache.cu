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

// One thread per group of a row.
template <int BITS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(KvView kv, KvRows x, int Hkv, int n, const int32_t *start,
                                                               const int32_t *count, int start_pos, int *status)
{
    using F = KvFmt<BITS, D>;
    const long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x;
    const int t = (int)(i / F::NG), gr = (int)(i % F::NG);
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const bool is_v = blockIdx.z != 0;
    const int rows = count != nullptr ? min(count[b], n) : n;
    if (t >= rows)
        return;
    const long long pos = (long long)(start != nullptr ? start[b] : 0) + start_pos + t;
    if (pos < 0 || pos >= 64LL * kv.max_blocks) {
        set_status(status, kStatusPage);
        return;
    }
    const int page = kv_page(kv, b, (int)(pos / 64), status);
    if (page < 0)
        return;
    const __nv_bfloat16 *src =
        static_cast<const __nv_bfloat16 *>(is_v ? x.v : x.k) +
        (is_v ? b * x.v_stride_b + kvh * x.v_stride_h + t * x.v_stride_t
              : b * x.k_stride_b + kvh * x.k_stride_h + t * x.k_stride_t) +
        gr * F::G;
    float lo = INFINITY, hi = -INFINITY;
    bool bad = false;
    for (int e = 0; e < F::G; ++e) {
        const float v = __bfloat162float(src[e]);
        bad |= !(fabsf(v) < 8.507059173023462e37f);      // 2^126; a NaN compares false
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    __nv_bfloat16 sb = __float2bfloat16_rn((hi - lo) / (float)F::TOP);
    if (bad || __bfloat162float(sb) < 7.888609052210118e-31f)    // 2^-100
        sb = __float2bfloat16_rn(0.f);
    const float s = __bfloat162float(sb);
    const uint32_t zb = bad ? 0x7FC0u : __bfloat16_as_ushort(__float2bfloat16_rn(lo));
    const int tok = (int)(pos % 32);
    uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, (int)(pos % 64) / 32);
    uint8_t *codes = half + (is_v ? F::kCodeV : 0);
    *reinterpret_cast<uint32_t *>(half + (is_v ? F::kParV : F::kParK) + tok * F::PAR + gr * 4) =
        (uint32_t)__bfloat16_as_ushort(sb) | zb << 16;
    constexpr int per = 8 / BITS;                         // elements of a byte
    for (int e = 0; e < F::G; e += per) {
        uint32_t byte = 0;
        for (int u = 0; u < per; ++u) {
            // IEEE division of bf16 differences rounds to the right side of a
            // half: a quotient that is not one is further from it than 2^-24
            const float q = s > 0.f ? rintf((__bfloat162float(src[e + u]) - lo) / s) : 0.f;
            byte |= (uint32_t)fminf(q, (float)F::TOP) << (u * BITS);
        }
        const int m = (gr * F::G + e) / per;
        codes[is_v ? F::v_off(tok, m) : F::k_off(tok, m)] = (uint8_t)byte;
    }
}

// One thread per byte-aligned pair of elements.
template <int BITS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(KvView kv, int Hkv, int n, const int32_t *start,
                                                              const int32_t *count, int start_pos,
                                                              __nv_bfloat16 *k, __nv_bfloat16 *v, int *status)
{
    using F = KvFmt<BITS, D>;
    const long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x;
    const int t = (int)(i / (D / 2)), e = (int)(i % (D / 2)) * 2;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const bool is_v = blockIdx.z != 0;
    __nv_bfloat16 *out = is_v ? v : k;
    const int rows = count != nullptr ? min(count[b], n) : n;
    if (t >= rows || out == nullptr)
        return;
    const long long pos = (long long)(start != nullptr ? start[b] : 0) + start_pos + t;
    if (pos < 0 || pos >= 64LL * kv.max_blocks) {
        set_status(status, kStatusPage);
        return;
    }
    const int page = kv_page(kv, b, (int)(pos / 64), status);
    if (page < 0)
        return;
    const int tok = (int)(pos % 32);
    const uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, (int)(pos % 64) / 32);
    const uint8_t *codes = half + (is_v ? F::kCodeV : 0);
    const uint32_t par = *reinterpret_cast<const uint32_t *>(half + (is_v ? F::kParV : F::kParK) + tok * F::PAR +
                                                             e / F::G * 4);
    float q[2];
    for (int u = 0; u < 2; ++u) {
        const int m = (e + u) * BITS / 8;
        const uint32_t byte = codes[is_v ? F::v_off(tok, m) : F::k_off(tok, m)];
        q[u] = (float)(BITS == 8 ? byte : (byte >> (4 * u)) & 15u);
    }
    const float s = kv_scale(par), z = kv_zero(par);
    __nv_bfloat162 r;
    r.x = __float2bfloat16_rn(fmaf(s, q[0], z));
    r.y = __float2bfloat16_rn(fmaf(s, q[1], z));
    *reinterpret_cast<__nv_bfloat162 *>(out + ((long long)blockIdx.y * n + t) * D + e) = r;
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
    const int groups = d / (bits == 4 ? 32 : 64);
    const dim3 grid((unsigned)(((long long)n * groups + kRowThreads - 1) / kRowThreads), B * Hkv, 2);
    if (bits == 4 && d == 128)
        kv_write_kernel<4, 128><<<grid, kRowThreads, 0, stream>>>(kv, x, Hkv, n, start, count, start_pos, status);
    else if (bits == 4)
        kv_write_kernel<4, 64><<<grid, kRowThreads, 0, stream>>>(kv, x, Hkv, n, start, count, start_pos, status);
    else if (d == 128)
        kv_write_kernel<8, 128><<<grid, kRowThreads, 0, stream>>>(kv, x, Hkv, n, start, count, start_pos, status);
    else
        kv_write_kernel<8, 64><<<grid, kRowThreads, 0, stream>>>(kv, x, Hkv, n, start, count, start_pos, status);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(int bits, int B, int Hkv, int n, int d, const KvView &kv, const int32_t *start,
                           const int32_t *count, int start_pos, void *k, void *v, int *status, cudaStream_t stream)
{
    const dim3 grid((unsigned)(((long long)n * d / 2 + kRowThreads - 1) / kRowThreads), B * Hkv, 2);
    auto *kb = static_cast<__nv_bfloat16 *>(k);
    auto *vb = static_cast<__nv_bfloat16 *>(v);
    if (bits == 4 && d == 128)
        kv_read_kernel<4, 128><<<grid, kRowThreads, 0, stream>>>(kv, Hkv, n, start, count, start_pos, kb, vb, status);
    else if (bits == 4)
        kv_read_kernel<4, 64><<<grid, kRowThreads, 0, stream>>>(kv, Hkv, n, start, count, start_pos, kb, vb, status);
    else if (d == 128)
        kv_read_kernel<8, 128><<<grid, kRowThreads, 0, stream>>>(kv, Hkv, n, start, count, start_pos, kb, vb, status);
    else
        kv_read_kernel<8, 64><<<grid, kRowThreads, 0, stream>>>(kv, Hkv, n, start, count, start_pos, kb, vb, status);
    return cudaGetLastError();
}

} // namespace seer

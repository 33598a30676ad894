// seer_kvdecode.cu — block-sparse attention of one new token per sequence over
// the quantised cache.
//
// o[b,h] = sum over t < len in active blocks of softmax(q . k_t * scale) v_t
// with k_t, v_t = z + s n of the cache.
#include <cuda_bf16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kQDT = 128;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Element e of token t's K or V row in a half record.
template <class F, int BITS, bool V>
__device__ __forceinline__ float kv_element(const uint8_t *half, int t, int e)
{
    const int m = e * BITS / 8;
    const uint32_t byte = half[V ? F::kCodeV + F::v_off(t, m) : F::k_off(t, m)];
    const uint32_t par =
        *reinterpret_cast<const uint32_t *>(half + (V ? F::kParV : F::kParK) + t * F::PAR + e / F::G * 4);
    return fmaf(kv_scale(par), (float)(BITS == 8 ? byte : (byte >> (4 * (e & 1))) & 15u), kv_zero(par));
}

// One CTA per (query head, split); the splits share the head's blocks by
// index.  A thread has a key in the scores and an output element in P V.
template <int BITS, int D>
__global__ void __launch_bounds__(kQDT)
    decode_quant_kernel(const __nv_bfloat16 *q_tok, KvView kv, const int32_t *lens, const uint8_t *mask, int Hq, int Hkv,
                        int L, int nb, float scale_log2, int nsplit, float *part, int *status)
{
    using F = KvFmt<BITS, D>;
    __shared__ float s_q[D], s_p[64], s_red[2];
    const int split = blockIdx.x, t = threadIdx.x;
    const long long bh = blockIdx.y;
    const int b = (int)(bh / Hq), h = (int)(bh % Hq), kvh = h / (Hq / Hkv);
    const int len = lens != nullptr ? max(0, min(lens[b], L)) : L;
    if (t < D)
        s_q[t] = __bfloat162float(q_tok[bh * D + t]);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int j = split; 64 * j < len; j += nsplit) {
        if (mask[bh * nb + j] == 0)
            continue;
        const int page = kv_page(kv, b, j, status);
        if (page < 0)
            continue;
        __syncthreads();
        float s = -INFINITY;
        if (t < 64 && 64 * j + t < len) {
            const uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, t / 32);
            float acc = 0.f;
            for (int e = 0; e < D; ++e)
                acc = fmaf(s_q[e], kv_element<F, BITS, false>(half, t % 32, e), acc);
            s = acc * scale_log2;
        }
        float wm = s;
        for (int off = 16; off >= 1; off >>= 1)
            wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, off));
        if (t < 64 && (t & 31) == 0)
            s_red[t / 32] = wm;
        __syncthreads();
        const float m_new = fmaxf(m, fmaxf(s_red[0], s_red[1]));
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        if (t < 64)
            s_p[t] = exp2_approx(s - m_use);
        __syncthreads();
        const float alpha = exp2_approx(m - m_use);
        m = m_new;
        l *= alpha;
        o *= alpha;
        const int keys = min(64, len - 64 * j);
        for (int c = 0; c < keys; ++c) {
            const uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, c / 32);
            l += s_p[c];
            if (t < D)
                o = fmaf(s_p[c], kv_element<F, BITS, true>(half, c % 32, t), o);
        }
    }
    float *out = part + (bh * nsplit + split) * (D + 2);
    if (t < D)
        out[t] = o;
    if (t == 0) {
        out[D] = m;
        out[D + 1] = l;
    }
}

// The splits of one head: weights 2^(m_s - M), o = sum w o / sum w l.
template <int D>
__global__ void __launch_bounds__(D)
    decode_quant_merge_kernel(const float *part, int nsplit, __nv_bfloat16 *o, float *lse)
{
    const long long bh = blockIdx.x;
    const float *pp = part + bh * nsplit * (D + 2);
    float M = -INFINITY;
    for (int s = 0; s < nsplit; ++s)
        M = fmaxf(M, pp[s * (D + 2) + D]);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f, acc = 0.f;
    for (int s = 0; s < nsplit; ++s) {
        const float w = exp2_approx(pp[s * (D + 2) + D] - mu);
        l = fmaf(w, pp[s * (D + 2) + D + 1], l);
        acc = fmaf(w, pp[s * (D + 2) + threadIdx.x], acc);
    }
    o[bh * D + threadIdx.x] = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
    if (lse != nullptr && threadIdx.x == 0)
        lse[bh] = l == 0.f ? -INFINITY : (mu + __log2f(l)) * 0.69314718055994530942f;
}

template <int BITS, int D>
cudaError_t launch(int B, int Hq, int Hkv, int L, float scale_log2, const void *q_tok, const KvView &kv,
                   const int32_t *lens, const uint8_t *mask, void *o, float *lse, float *part, int *status,
                   cudaStream_t stream)
{
    const int nb = num_blocks(L);
    const int ns = decode_splits(B, Hq, nb);
    decode_quant_kernel<BITS, D><<<dim3(ns, B * Hq), kQDT, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(q_tok), kv, lens, mask, Hq, Hkv, L, nb, scale_log2, ns, part, status);
    decode_quant_merge_kernel<D><<<B * Hq, D, 0, stream>>>(part, ns, static_cast<__nv_bfloat16 *>(o), lse);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_decode_quant(int bits, int B, int Hq, int Hkv, int L, int d, float scale_log2, const void *q_tok,
                                const KvView &kv, const int32_t *lens, const uint8_t *mask, void *o, float *lse,
                                float *part, int *status, uint64_t timeout_ns, cudaStream_t stream)
{
    (void)timeout_ns;
    if (bits == 4 && d == 128)
        return launch<4, 128>(B, Hq, Hkv, L, scale_log2, q_tok, kv, lens, mask, o, lse, part, status, stream);
    if (bits == 4)
        return launch<4, 64>(B, Hq, Hkv, L, scale_log2, q_tok, kv, lens, mask, o, lse, part, status, stream);
    if (d == 128)
        return launch<8, 128>(B, Hq, Hkv, L, scale_log2, q_tok, kv, lens, mask, o, lse, part, status, stream);
    return launch<8, 64>(B, Hq, Hkv, L, scale_log2, q_tok, kv, lens, mask, o, lse, part, status, stream);
}

} // namespace seer

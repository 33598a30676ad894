// seer_kvgate.cu — the gate's key rows from the quantised cache.
//
//   Kt_j = RoPE_j( pool_{t in block j, t < len}(z_t + s_t n_t) @ Wk )
//
// The pooling reads the K half of each record once; the projection and the
// rotation are those of the bf16 cache's key rows.
#include <algorithm>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

// One CTA per (head, block), one thread per element of the pooled row.
template <int BITS, int D, bool MAXMIN>
__global__ void __launch_bounds__(D) kv_pool_kernel(KvView kv, int Hkv, int L, const int32_t *lens, int nb, int first,
                                                    float *out, int *status)
{
    using F = KvFmt<BITS, D>;
    const long long bh = (long long)blockIdx.x / (nb - first);
    const int j = first + (int)(blockIdx.x % (nb - first));
    const int b = (int)(bh / Hkv), kvh = (int)(bh % Hkv);
    const int e = threadIdx.x;
    const int len = lens != nullptr ? max(0, min(lens[b], L)) : L;
    int rows = min(64, len - 64 * j);
    const int page = rows > 0 ? kv_page(kv, b, j, status) : -1;
    if (page < 0)
        rows = 0;
    float sum = 0.f, mx = -INFINITY, mn = INFINITY;
    const int m = e * BITS / 8;
    for (int t = 0; t < rows; ++t) {
        const uint8_t *half = kv_half<F>(kv, Hkv, page, kvh, t / 32);
        const uint32_t byte = half[F::k_off(t % 32, m)];
        const uint32_t par =
            *reinterpret_cast<const uint32_t *>(half + F::kParK + (t % 32) * F::PAR + e / F::G * 4);
        const float x = fmaf(kv_scale(par), (float)(BITS == 8 ? byte : (byte >> (4 * (e & 1))) & 15u), kv_zero(par));
        sum += x;
        mx = x > mx || x != x ? x : mx;
        mn = x < mn || x != x ? x : mn;
    }
    const long long row = bh * nb + j;
    if (MAXMIN) {
        out[row * 2 * D + e] = rows > 0 ? mx : 0.f;
        out[row * 2 * D + D + e] = rows > 0 ? mn : 0.f;
    } else {
        out[row * D + e] = rows > 0 ? sum / (float)rows : 0.f;
    }
}

template <int BITS, int D>
void pool(bool maxmin, unsigned grid, KvView kv, int Hkv, int L, const int32_t *lens, int nb, int first, float *out,
          int *status, cudaStream_t stream)
{
    if (maxmin)
        kv_pool_kernel<BITS, D, true><<<grid, D, 0, stream>>>(kv, Hkv, L, lens, nb, first, out, status);
    else
        kv_pool_kernel<BITS, D, false><<<grid, D, 0, stream>>>(kv, Hkv, L, lens, nb, first, out, status);
}

} // namespace

cudaError_t launch_gate_keys_quant(int bits, int B, int Hkv, int L, int d, int dg, float theta, bool k_maxmin,
                                   const KvView &kv, const int32_t *lens, const void *wk, long long wk_stride,
                                   int first_block, float *kt, void *ws, int *status, cudaStream_t stream)
{
    const int nb = num_blocks(L);
    if (first_block >= nb)
        return cudaSuccess;
    float *kp = static_cast<float *>(ws);
    const unsigned grid = (unsigned)((long long)B * Hkv * (nb - first_block));
    if (bits == 4 && d == 128)
        pool<4, 128>(k_maxmin, grid, kv, Hkv, L, lens, nb, first_block, kp, status, stream);
    else if (bits == 4)
        pool<4, 64>(k_maxmin, grid, kv, Hkv, L, lens, nb, first_block, kp, status, stream);
    else if (d == 128)
        pool<8, 128>(k_maxmin, grid, kv, Hkv, L, lens, nb, first_block, kp, status, stream);
    else
        pool<8, 64>(k_maxmin, grid, kv, Hkv, L, lens, nb, first_block, kp, status, stream);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    return launch_project_keys(B, Hkv, nb, k_maxmin ? 2 * d : d, dg, theta, kp, wk, wk_stride, first_block, kt, stream);
}

} // namespace seer

// seer_kv.cuh — the quantised KV cache's record layout (include/seer.h,
// seer_kv_cache) and the page lookup its kernels share.
//
// A record holds 64 tokens of one head: two halves of 32 tokens, each one
// contiguous run [K codes | K params | V codes | V params], so that one bulk
// copy brings 32 tokens of K and V.  The code rows are laid out for the decode
// kernel's mma fragments: a K row gives each of the four lanes that share a
// key its elements of every 16-element MMA step in one run, a V row gives each
// of eight lanes its output elements in one run, and both are swizzled by the
// token so that a warp's shared-memory reads meet no bank twice.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "seer_ptx.cuh"

namespace seer {

// The cache's kernels start while the kernel before them in their stream ends (a
// programmatic launch: between two of them the launch latency, some 2 us of a call
// outside a graph, passes under the first) and wait for it, and for what it wrote,
// before they touch memory.  All threads, first of all.  Loads are plain ones: a
// read-only load (ld.global.nc) would be free to pass the wait.
__device__ __forceinline__ void wait_for_previous_kernel()
{
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

template <class T>
__device__ __forceinline__ T load(const T *p)
{
    return *p;
}

template <class... P, class... A>
cudaError_t launch_programmatic(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    return e == cudaSuccess ? e : cudaGetLastError();    // (and cleared)
}

// What the kernels need of a seer_kv_cache.
struct KvView {
    uint8_t *pages;              // [n_pages, Hkv, record]
    const int32_t *table;        // [B, max_blocks] or null: page b * max_blocks + j
    int n_pages, max_blocks;
};

template <int BITS, int D>
struct KvFmt {
    static_assert(BITS == 4 || BITS == 8, "4 or 8 bits");
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int G = BITS == 4 ? 32 : 64;    // elements that share a scale and a zero
    static constexpr int NG = D / G;
    static constexpr int R = D * BITS / 8;           // bytes of a code row
    static constexpr int PAR = 4 * NG;               // bytes of a row's params: (bf16 scale, bf16 zero) per group
    static constexpr int kParK = 32 * R;             // offsets within a half record
    static constexpr int kCodeV = 32 * (R + PAR);
    static constexpr int kParV = kCodeV + 32 * R;
    static constexpr int HALF = 2 * kCodeV;
    static constexpr int REC = 2 * HALF;
    static constexpr int TOP = (1 << BITS) - 1;

    // Byte offset, within a half's codes, of byte m of token t's row in element
    // order (elements 2m and 2m + 1, low nibble first, at 4 bits; element m at 8).
    __host__ __device__ static int k_off(int t, int m)
    {
        const int c = m / 4, b = m % 4;
        if (BITS == 4)
            return t * R + ((c % 4) * NG + c / 4) * 4 + b;
        const int p = D == 128 ? (c / 16) ^ (t & 1) : c / 16;
        return t * R + (p * 16 + (c / 4) % 4 + (c % 4) * 4) * 4 + b;
    }
    __host__ __device__ static int v_swizzle(int t)
    {
        if (BITS == 4)
            return D == 128 ? ((t >> 2) & 1) * 4 : 0;
        return D == 128 ? ((t >> 1) & 3) * 2 : ((t >> 2) & 1) * 4;
    }
};

// The page of block j of sequence b, or -1 (recorded in the status word) when
// the table names none of the cache's pages.  j is within max_blocks.
__device__ __forceinline__ int kv_page(const KvView &kv, int b, int j, int *status)
{
    const int p = kv.table != nullptr ? load(kv.table + (long long)b * kv.max_blocks + j) : b * kv.max_blocks + j;
    if (p < 0 || p >= kv.n_pages) {
        set_status(status, kStatusPage);
        return -1;
    }
    return p;
}

// Head kvh's record of a page, half h.
template <class F>
__device__ __forceinline__ uint8_t *kv_half(const KvView &kv, int Hkv, int page, int kvh, int h)
{
    return kv.pages + ((long long)page * Hkv + kvh) * F::REC + h * F::HALF;
}

__device__ __forceinline__ float kv_scale(uint32_t par) { return __uint_as_float(par << 16); }
__device__ __forceinline__ float kv_zero(uint32_t par) { return __uint_as_float(par & 0xFFFF0000u); }

} // namespace seer

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
// A row costs 2 D bytes on the bf16 side and D bits / 8 + 4 D / G on the other, so
// HBM is the floor of both directions.  32k rows of 8 heads at 4 bits (D = 128,
// 176 MB): reading back 30.5 us (5.8 TB/s), writing 37.1 us (4.8 TB/s; 32.2 before codes
// next to a half were looked for); at 8 bits 34.1 and 38.1.  Both are near the copy rate
// and bound by their instructions (69 and 72 % of the issue slots, the integer pipe first).
#include <type_traits>

#include <cuda_bf16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kRowThreads = 256;

// A lane holds E elements of a row.  Reading, eight: one 16-byte store each,
// which leaves the kernel at 88 % of the copy rate.  Writing has more instructions an
// element, so there a lane has sixteen, over which the group's extrema, scale and
// addresses are shared (37 us against 45 with eight for a 32k prompt of 8 heads, before
// codes next to a half were looked for).
template <int BITS, int D, int E>
struct RowMap {
    using F = KvFmt<BITS, D>;
    static constexpr int CH = D / E;                     // lanes of a row
    static constexpr int RPW = 32 / CH;                  // rows of a warp's access
    static constexpr int GL = F::G / E;                  // lanes of a group
    static constexpr int NW = E * BITS / 32;             // code words of a lane
};

// A CTA has one page of one head, 64 positions of which the call's rows cover
// [lo, hi): the page is looked up once and every row's address is an offset.
// Rows at positions below 0 or past the cache are recorded and left out.
struct PageRows {
    uint8_t *record;             // null: nothing to do here
    int lo, hi;                  // tokens of the page
    int row0;                    // row of token 0 (may be negative)
};

template <class F>
__device__ __forceinline__ PageRows page_rows(const KvView &kv, int Hkv, int b, int kvh, int n, const int32_t *start,
                                              const int32_t *count, int start_pos, int *status)
{
    PageRows r{nullptr, 0, 0, 0};
    const int rows = count != nullptr ? min(load(count + b), n) : n;
    const long long first = (long long)(start != nullptr ? load(start + b) : 0) + start_pos;
    if (rows <= 0)
        return r;
    // beyond +- 2^22 no row of at most 2^20 meets a cache of at most 2^20 tokens
    const int base = (int)max(-(1LL << 22), min(1LL << 22, first));
    const int j = max(base, 0) / 64 + (int)blockIdx.x;
    if (base < 0 && blockIdx.x == 0)
        set_status(status, kStatusPage);
    r.row0 = 64 * j - base;
    r.lo = max(0, -r.row0);
    r.hi = min(64, rows - r.row0);
    if (r.lo >= r.hi)
        return r;
    if (j >= kv.max_blocks) {
        set_status(status, kStatusPage);
        return r;
    }
    const int page = kv_page(kv, b, j, status);
    if (page >= 0)
        r.record = kv_half<F>(kv, Hkv, page, kvh, 0);
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
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

// Reading: the code words of a V row change lanes from the order they lie in
// (lane c: four bytes at offset v_place at 4 bits, eight at 8) to element order
// (lane c: the words of elements 8c .. 8c+7).  At 4 bits a lane's word is two
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
__device__ __forceinline__ uint32_t v4_exchange(uint32_t w, int lane)
{
    const int base = lane & ~(D / 8 - 1), c = lane & (D / 8 - 1), i = c / 4, q = c % 4;
    const int s0 = D == 128 ? i >> 1 : 0, s1 = D == 128 ? s0 + 2 : 1, half = D == 128 ? i & 1 : i;
    const uint32_t v0 = __shfl_sync(0xffffffffu, w, base + 4 * s0 + q), v1 = __shfl_sync(0xffffffffu, w, base + 4 * s1 + q);
    return __byte_perm(v0, v1, half ? 0x7632 : 0x5410);
}

// At 8 bits a K row's word c lies at 16 p + 4 (c % 4) + (c / 4) % 4: lane c loads
// eight bytes, the words (j, t) and (j + 1, t) with j = c / 2 of the sixteen
// elements' index, against words 2c and 2c + 1 in element order.
template <int D>
__device__ __forceinline__ int k8_place(int tok, int c)
{
    using F = KvFmt<8, D>;
    const int p = D == 128 ? (c / 8) ^ (tok & 1) : 0;
    return tok * F::R + p * 64 + (c % 8) / 2 * 16 + (c % 2) * 8;
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

// A group as it is stored: the extrema of the lane's sixteen elements w, joined over
// the lanes that share the group.
struct Group {
    float lo, s, inv;                                    // inv: about 1 / s, 0 for s = 0
    uint32_t par;
    bool ok;                                             // no NaN, no magnitude of 2^126 or more
    bool open;                                           // see quantise16
};

template <int BITS, int D>
__device__ __forceinline__ Group group_of(const uint32_t (&w)[8])
{
    using F = KvFmt<BITS, D>;
    constexpr int GL = RowMap<BITS, D, 16>::GL;
    __nv_bfloat162 mn, mx, least;                        // of the elements, of their magnitudes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 p = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
        mn = i == 0 ? p : __hmin2_nan(mn, p);
        mx = i == 0 ? p : __hmax2_nan(mx, p);
        least = i == 0 ? __habs2(p) : __hmin2(least, __habs2(p));
    }
#pragma unroll
    for (int off = 1; off < GL; off <<= 1) {
        mn = __hmin2_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mx = __hmax2_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    const __nv_bfloat16 lob = __hmin_nan(mn.x, mn.y), hib = __hmax_nan(mx.x, mx.y);
    const float lo = __bfloat162float(lob), hi = __bfloat162float(hib);
    Group g;
    g.ok = lo > -8.507059173023462e37f && hi < 8.507059173023462e37f;           // 2^126; false for a NaN
    // range / TOP: the product with the rounded reciprocal, corrected once by its exact
    // remainder (Markstein's division on a fused multiply-add, IBM J. Res. Dev. 34, 1990)
    constexpr float kInvTop = 1.f / F::TOP;
    const float range = hi - lo, s0 = range * kInvTop;
    __nv_bfloat16 sb = __float2bfloat16_rn(fmaf(fmaf(s0, -(float)F::TOP, range), kInvTop, s0));
    if (!g.ok || __bfloat162float(sb) < 7.888609052210118e-31f)                 // 2^-100
        sb = __float2bfloat16_rn(0.f);
    g.s = __bfloat162float(sb);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.s));
    g.inv = g.s > 0.f ? g.inv : 0.f;
    g.lo = g.ok ? lo : 0.f;
    g.par = (uint32_t)__bfloat16_as_ushort(sb) | (g.ok ? (uint32_t)__bfloat16_as_ushort(lob) : 0x7FC0u) << 16;
    const float most = fmaxf(fabsf(lo), fabsf(hi)) * 0.000030517578125f;        // 2^-15
    const float r = fmaf(rintf(lo * g.inv), -g.s, lo);   // what -z / s is off an integer, times s
    g.open = g.s > 0.f && ((fminf(__low2float(least), __high2float(least)) < most && fabsf(r) > 0.484f * g.s) ||
                           (fabsf(lo) < most && lo != 0.f));
    return g;
}

// The code words of a lane's sixteen elements.  The quotient of t = x - z by s is
// taken as the group's scale is: one that is a half is one then.  Where x and z are
// within 2^15 of the group's largest, t is exact (23 bits; 24 where neither is far below),
// and with an 8-bit s every other quotient is further from a half than it is off.  Of
// two codes the wrong one may come out where z is further below, or where x is and
// -z / s lies within 2^-6 of a half (x / s is below 2^-7): Group::open, then nearest_codes.
template <int BITS>
__device__ __forceinline__ void quantise16(const uint32_t (&w)[8], const Group &g, uint32_t (&code)[BITS / 2])
{
    constexpr float kTop = (1 << BITS) - 1;
    constexpr uint32_t kMagic = 0x4B400000u;             // 1.5 2^23: adding it leaves the integer in the low bits
    uint32_t pair[8];                                    // n of two elements in the low bits
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        const float2 t = add2(v, both(-g.lo));
        float2 q = mul2(t, both(g.inv));
        q = fma2(fma2(q, both(-g.s), t), both(g.inv), q);
        if (BITS == 8)                                   // s may be up to 2^-8 below the range / 255, not so at 15
            q = make_float2(fminf(q.x, kTop), fminf(q.y, kTop));
        const float2 m = add2(q, both(__uint_as_float(kMagic)));
        pair[i] = __float_as_uint(m.y) * (1u << BITS) + __float_as_uint(m.x);
    }
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code[i] = __byte_perm(__byte_perm(pair[4 * i], pair[4 * i + 1], 0x0040),
                                  __byte_perm(pair[4 * i + 2], pair[4 * i + 3], 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i] = __byte_perm(pair[2 * i], pair[2 * i + 1], 0x5410);
    }
    if (!g.ok)
#pragma unroll
        for (int i = 0; i < BITS / 2; ++i)
            code[i] = 0u;
}

__device__ __forceinline__ float element(const uint32_t (&w)[8], int i)
{
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// Whether a quotient of the lane's lies next to a half.
__device__ __forceinline__ bool next_to_a_half(const uint32_t (&w)[8], const Group &g)
{
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float t = element(w, i) - g.lo;
        most = fmaxf(most, fabsf(fmaf(-rintf(t * g.inv), g.s, t)));
    }
    return most > 0.4999f * g.s;
}

// The codes by the definition, the integers nearest to (x - z) / s, with nothing
// rounded on the way to the decision.  t + e is x - z exactly (Knuth's two-sum).  n0, t
// times the reciprocal rounded, is off by one at most, and only next to a half;
// r = t - n0 s is a float (t and n0 s are within a factor of two of each other, or
// t's last place is above 2^-24 s).  |e| is below every difference that r and s / 2
// can have but 0 (t < 2^9 s), so it decides where they are equal, and nowhere else.
template <int BITS>
__device__ __forceinline__ void nearest_codes(const uint32_t (&w)[8], const Group &g, uint32_t (&code)[BITS / 2])
{
    constexpr int kTop = (1 << BITS) - 1;
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i)
        code[i] = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = element(w, i), t = x - g.lo, back = t - x, e = (x - (t - back)) + (-g.lo - back);
        const float n0 = rintf(t * g.inv), r = fmaf(-n0, g.s, t), half = 0.5f * g.s;
        int n = (int)n0;
        const bool odd = n & 1;
        if (r > half || (r == half && (e > 0.f || (e == 0.f && odd))))
            ++n;
        else if (r < -half || (r == -half && (e < 0.f || (e == 0.f && odd))))
            --n;
        code[i * BITS / 32] |= (uint32_t)(g.ok && g.s > 0.f ? min(n, kTop) : 0) << (i * BITS % 32);
    }
}

// Token tok's code words of a lane (sixteen elements c of the row) to their places in
// the half record `half`.  All lanes of the warp; `mine`: this lane has a row.
template <int BITS, int D, bool V>
__device__ __forceinline__ void store_codes(uint8_t *half, int tok, int c, bool mine, const uint32_t (&code)[BITS / 2])
{
    using F = KvFmt<BITS, D>;
    uint8_t *row = half + (V ? F::kCodeV : 0) + tok * F::R;
    if constexpr (BITS == 4 && !V) {                     // words 2c and 2c + 1
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (mine)
                *reinterpret_cast<uint32_t *>(row + (((2 * c + k) % 4) * F::NG + c / 2) * 4) = code[k];
    } else if constexpr (BITS == 4) {
        // 16-bit runs of chunks 4h .. 4h + 3 (h = c % 2) of group c / 2; a stored word is
        // two groups of one chunk: the lanes of an even and an odd group trade the two
        // upper and the two lower chunks
        const int gr = c / 2, h = c % 2, odd = gr & 1;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? code[0] : code[1], 2);
        const uint32_t lo = odd ? got : code[0], hi = odd ? code[1] : got;        // even group, odd group
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int chunk = 4 * h + 2 * odd + k;
            if (mine)
                *reinterpret_cast<uint32_t *>(row + (chunk ^ F::v_swizzle(tok)) * (2 * F::NG) + (gr >> 1) * 4) =
                    __byte_perm(lo, hi, k ? 0x7632 : 0x5410);
        }
    } else if constexpr (!V) {                           // words 4c .. 4c + 3, sixteen bytes apart
        const int p = D == 128 ? (c / 4) ^ (tok & 1) : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (mine)
                *reinterpret_cast<uint32_t *>(row + (p * 16 + k * 4 + c % 4) * 4) = code[k];
    } else {                                             // runs of chunks 2c and 2c + 1 (of eight) of group c / 4
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (mine)
                *reinterpret_cast<uint2 *>(row + ((2 * c % 8 + k) ^ F::v_swizzle(tok)) * (8 * F::NG) + c / 4 * 8) =
                    make_uint2(code[2 * k], code[2 * k + 1]);
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(KvView kv, KvRows x, int Hkv, int n, const int32_t *start,
                                                               const int32_t *count, int start_pos, int *status)
{
    using F = KvFmt<BITS, D>;
    using M = RowMap<BITS, D, 16>;
    constexpr int NI = 64 / (kRowThreads / 32 * M::RPW);  // rows of a lane for each of K and V
    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % M::CH;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const PageRows r = page_rows<F>(kv, Hkv, b, kvh, n, start, count, start_pos, status);
    if (r.record == nullptr)
        return;
    const __nv_bfloat16 *src[2] = {
        static_cast<const __nv_bfloat16 *>(x.k) + b * x.k_stride_b + kvh * x.k_stride_h + r.row0 * x.k_stride_t + 16 * c,
        static_cast<const __nv_bfloat16 *>(x.v) + b * x.v_stride_b + kvh * x.v_stride_h + r.row0 * x.v_stride_t + 16 * c};
    uint32_t in[2][NI][8];
    auto token = [&](int i) { return (i * (kRowThreads / 32) + warp) * M::RPW; };         // the warp's first
    auto fetch = [&](int is_v, int t, uint32_t (&w)[8]) {
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (t >= r.lo && t < r.hi) {
            const uint4 *at = reinterpret_cast<const uint4 *>(src[is_v] + t * (is_v ? x.v_stride_t : x.k_stride_t));
            a = load(at);
            b = load(at + 1);
        }
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    };
    auto store = [&](auto is_v, int t, const uint32_t (&code)[M::NW]) {
        store_codes<BITS, D, is_v>(r.record + t / 32 * F::HALF, t % 32, c, t >= r.lo && t < r.hi, code);
    };
    auto none = [&](int tw) { return tw + M::RPW <= r.lo || tw >= r.hi; };                  // of the whole warp's rows
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v)
#pragma unroll
        for (int i = 0; i < NI; ++i)
            fetch(is_v, token(i) + lane / M::CH, in[is_v][i]);
    unsigned open = 0u;                                  // items whose codes are not certain yet
    auto rows = [&](auto is_v) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tw = token(i), t = tw + lane / M::CH;
            if (none(tw))
                continue;
            const Group g = group_of<BITS, D>(in[is_v][i]);
            uint32_t code[M::NW];
            quantise16<BITS>(in[is_v][i], g, code);
            store(is_v, t, code);
            if (t >= r.lo && t < r.hi && c % M::GL == 0)
                *reinterpret_cast<uint32_t *>(r.record + t / 32 * F::HALF + (is_v ? F::kParV : F::kParK) + t % 32 * F::PAR +
                                              c / M::GL * 4) = g.par;
            open |= (unsigned)g.open << (is_v * NI + i);
        }
    };
    // Rows with an open lane (one in a thousand of a warp's accesses of normal ones) are
    // read again: kept in registers, or decided on the spot, they would cost every row.
    auto again = [&](auto is_v) {
#pragma unroll 1
        for (int i = 0; i < NI; ++i) {
            if (!__any_sync(0xffffffffu, open >> (is_v * NI + i) & 1u))
                continue;
            const int t = token(i) + lane / M::CH;
            uint32_t w[8], code[M::NW];
            fetch(is_v, t, w);
            const Group g = group_of<BITS, D>(w);
            if (!__any_sync(0xffffffffu, g.open && next_to_a_half(w, g)))
                continue;
            nearest_codes<BITS>(w, g, code);
            store(is_v, t, code);
        }
    };
    rows(std::false_type{});
    rows(std::true_type{});
    if (__any_sync(0xffffffffu, open != 0u)) {
        again(std::false_type{});
        again(std::true_type{});
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(KvView kv, int Hkv, int n, const int32_t *start,
                                                              const int32_t *count, int start_pos,
                                                              __nv_bfloat16 *k, __nv_bfloat16 *v, int *status)
{
    using F = KvFmt<BITS, D>;
    using M = RowMap<BITS, D, 8>;
    constexpr int NI = 64 / (kRowThreads / 32 * M::RPW);
    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % M::CH;
    const int b = blockIdx.y / Hkv, kvh = blockIdx.y % Hkv;
    const PageRows r = page_rows<F>(kv, Hkv, b, kvh, n, start, count, start_pos, status);
    if (r.record == nullptr)
        return;
    uint32_t code[2][NI][M::NW], par[2][NI];
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int t = (i * (kRowThreads / 32) + warp) * M::RPW + lane / M::CH, tok = t % 32;
            code[is_v][i][0] = code[is_v][i][M::NW - 1] = par[is_v][i] = 0u;
            if (t < r.lo || t >= r.hi || (is_v ? v : k) == nullptr)
                continue;
            const uint8_t *half = r.record + t / 32 * F::HALF, *base = half + (is_v ? F::kCodeV : 0);
            if constexpr (BITS == 4) {
                code[is_v][i][0] =
                    *reinterpret_cast<const uint32_t *>(base + (is_v ? v_place<4, D>(tok, c) : F::k_off(tok, 4 * c)));
            } else {
                const uint2 w =
                    *reinterpret_cast<const uint2 *>(base + (is_v ? v_place<8, D>(tok, c) : k8_place<D>(tok, c)));
                code[is_v][i][0] = w.x;
                code[is_v][i][M::NW - 1] = w.y;
            }
            par[is_v][i] =
                *reinterpret_cast<const uint32_t *>(half + (is_v ? F::kParV : F::kParK) + tok * F::PAR + c / M::GL * 4);
        }
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
        __nv_bfloat16 *out = (is_v ? v : k) + ((long long)blockIdx.y * n + r.row0) * D + 8 * c;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tw = (i * (kRowThreads / 32) + warp) * M::RPW, t = tw + lane / M::CH;
            if (tw + M::RPW <= r.lo || tw >= r.hi || (is_v ? v : k) == nullptr)
                continue;                                // the whole warp
            uint32_t(&w)[M::NW] = code[is_v][i];
            if constexpr (BITS == 4) {
                if (is_v)
                    w[0] = v4_exchange<D>(w[0], lane);
            } else if (!is_v) {
                const uint2 x = k8_from_store<D>(make_uint2(w[0], w[1]), lane);
                w[0] = x.x;
                w[M::NW - 1] = x.y;
            }
            const float s = kv_scale(par[is_v][i]), z = kv_zero(par[is_v][i]);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                constexpr int per = 32 / BITS;
                const uint32_t q0 = w[2 * e / per] >> (2 * e % per * BITS), q1 = w[(2 * e + 1) / per] >> ((2 * e + 1) % per * BITS);
                // the code as a float: 2^23 + n, less 2^23.  (The sum rounded to fp32 and then to
                // bf16 is the sum rounded once: fp32 is inexact only where s n is below half a bf16
                // step of z, and then 255 * 255 / 2^16 keeps it away from the middle.)
                float2 f = make_float2(__uint_as_float((q0 & (uint32_t)F::TOP) | 0x4B000000u),
                                       __uint_as_float((q1 & (uint32_t)F::TOP) | 0x4B000000u));
                f = fma2(add2(f, both(-8388608.f)), both(s), both(z));
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                o[e] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if (t >= r.lo && t < r.hi)
                *reinterpret_cast<uint4 *>(out + (long long)t * D) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Pages that n rows can touch: one more than they fill, since they may start anywhere.
unsigned pages_of(int n) { return (unsigned)(n - 1) / 64 + 2; }

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
    const auto f = bits == 4 ? (d == 128 ? kv_write_kernel<4, 128> : kv_write_kernel<4, 64>)
                             : (d == 128 ? kv_write_kernel<8, 128> : kv_write_kernel<8, 64>);
    return launch_programmatic(f, dim3(pages_of(n), B * Hkv), kRowThreads, 0, stream, kv, x, Hkv, n, start, count, start_pos,
                               status);
}

cudaError_t launch_kv_read(int bits, int B, int Hkv, int n, int d, const KvView &kv, const int32_t *start,
                           const int32_t *count, int start_pos, void *k, void *v, int *status, cudaStream_t stream)
{
    const auto f = bits == 4 ? (d == 128 ? kv_read_kernel<4, 128> : kv_read_kernel<4, 64>)
                             : (d == 128 ? kv_read_kernel<8, 128> : kv_read_kernel<8, 64>);
    return launch_programmatic(f, dim3(pages_of(n), B * Hkv), kRowThreads, 0, stream, kv, Hkv, n, start, count, start_pos,
                               static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), status);
}

} // namespace seer

// seer_kvdecode.cu — block-sparse attention of one new token per sequence over
// the quantised cache.
//
//   o[b,h] = sum over t < len in active blocks of softmax(q . k_t * scale) v_t,
//   k_t = z + s n (per group of the row), v_t likewise.
//
// Each active block crosses HBM once per GQA group: a CTA serves up to eight
// query heads of one KV head over the union of their active blocks (a head
// without a block gets p = 0 there).  At 4 bits a token's K and V are 160 bytes
// for 4 D flops per head, so with CUDA-core products the arithmetic, not HBM,
// would set the time (at D = 128 and four heads 2048 flops per 160 bytes); the
// products are mma.sync m16n8k16 with the keys on M (K Q^T) or the output
// elements on M (V^T P) and the heads on N.  Decode has at most eight columns
// of N, which leaves a tcgen05 tile nothing to gain.
//
//  * The codes enter the MMA as they are: n <= 255 in the low bits of an fp16 is
//    the subnormal n 2^-24, so one mask (4 bits) or byte permute (8 bits) makes
//    a pair of operands, and scale and zero are applied outside:
//      q . k   = sum_g s_g (q_g . n_g) + z_g sum(q_g)        per key; the second by an
//                MMA of the params as they lie with sum(q_g) in three bf16 parts
//      sum p v = sum_t (p_t s_t,g) n_t + sum_t p_t z_t,g      p s rounded to fp16
//    q is exact in fp16 after a power of two per head; p s <= 2^15 after a power
//    of two that follows the largest scale seen (as a running maximum, so it
//    holds for any range of V).  p z, the row sums and all accumulators are fp32.
//  * Work of a warp: half records of 32 tokens, each one contiguous bulk copy
//    into the warp's own ring, so no warp waits for another until the end.
//  * P leaves K Q^T with keys across lanes and enters V^T P with keys across a
//    lane's register pair: movmatrix turns each 8 x 8 piece.
//  * Split over the union's blocks by rank, so splits differ by one block at
//    most; a second kernel joins them.
//
// What bounds it: with 8 bits and long caches HBM (128k tokens at density 0.17: the loop
// itself reads 7 TB/s; 37.7 us a call with start, end and join, 22.8 at the copy
// rate).  With 4 bits the instructions of the loop: some 350 a tile of 16 tokens
// and warp, 160 of them on the integer pipe at two cycles each, against 6 cycles
// a token that HBM allows (32k tokens of a layer, all active: 20.7 us, 6.4 at the
// copy rate).  Short ones: a CTA's start and end, some 8,000 cycles of latencies,
// and the join (32k at density 0.1: 11.8 us; 200 tokens: 4.8).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kHeads = 8;                 // query heads of a CTA: the N of the MMA
constexpr int kListMax = 513;             // blocks of a split (decode_quant_split)
constexpr int kNoPage = kMaxNb;           // flag of a list entry; block indices are below it

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: no accumulator to clear.
__device__ __forceinline__ void mma16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma16816_bf16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma16816_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float pow2_field(int field) { return __uint_as_float((uint32_t)field << 23); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Weight of a part (maximum m, sum l) in the whole (maximum M), all in log2 units.
// A part that saw only NaN has no maximum but a sum; one that saw nothing has neither.
__device__ __forceinline__ float split_weight(float m, float l, float M)
{
    return m == -INFINITY ? (l == 0.f ? 0.f : l) : exp2_approx(m - M);
}

// Natural log of l 2^M; -inf where nothing was active.
__device__ __forceinline__ float log_sum(float M, float l)
{
    return l == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + __log2f(l)) * 0.69314718055994530942f;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x;
        w[1] = u.y;
    } else {
        static_assert(N == 1);
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Row of an MMA tile -> token: within eight rows (0,1,3,2,4,5,7,6), so that the
// rows of a K fragment's quarter warp have both parities and the four rows that
// a V fragment reads at once differ in the bits its swizzle uses.
__device__ __forceinline__ int tile_token(int r) { return r ^ ((r >> 1) & 1); }

// q of one head for the MMAs, by one warp: its elements in fp16 times 2^qe, in
// the order of the codes' operands (at 4 bits a word's elements 0,4,1,5,2,6,3,7
// with the odd ones times 2^-4, as the codes' masks give them), its group sums in
// three bf16 parts (for the products with z), and 2^-qe.
template <int D>
struct HeadQ {
    uint16_t f16[D];
    uint16_t sum[3][4];
    float inv;
    uint32_t pad;
};

template <int BITS, int D>
__device__ __forceinline__ void prepare_q(const __nv_bfloat16 *qp, int lane, HeadQ<D> *out)
{
    constexpr int N = D / 32, GL = KvFmt<BITS, D>::G / N;   // elements of a lane, lanes of a group
    float f[N];
    if constexpr (N == 4) {
        const uint2 u = qp != nullptr ? __ldg(reinterpret_cast<const uint2 *>(qp) + lane) : make_uint2(0u, 0u);
        f[0] = __uint_as_float(u.x << 16);
        f[1] = __uint_as_float(u.x & 0xFFFF0000u);
        f[2] = __uint_as_float(u.y << 16);
        f[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
        const uint32_t u = qp != nullptr ? __ldg(reinterpret_cast<const uint32_t *>(qp) + lane) : 0u;
        f[0] = __uint_as_float(u << 16);
        f[1] = __uint_as_float(u & 0xFFFF0000u);
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        mx = fmaxf(mx, fabsf(f[i]));
    // max |q| 2^qe in [2^14, 2^15) where 2^qe is a float; no scaling for infinity
    const int eb = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)) >> 23);
    const int qe = eb == 255 ? 0 : min(141 - eb, 126);
    const float up = pow2_field(127 + qe);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        f[i] *= up;
        s += f[i];
        const int e = N * lane + i;
        const int at = BITS == 4 ? (e & ~7) + (e & 3) * 2 + (e >> 2 & 1) : e;
        out->f16[at] = __half_as_ushort(__float2half_rn(BITS == 4 && e & 1 ? f[i] * 0.0625f : f[i]));
    }
#pragma unroll
    for (int off = 1; off < GL; off <<= 1)
        s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= 5.9604644775390625e-8f;                    // 2^-24: the unit of the codes' products
    if (lane % GL == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const __nv_bfloat16 part = __float2bfloat16_rn(s);
            out->sum[i][lane / GL] = __bfloat16_as_ushort(part);
            s -= __bfloat162float(part);
        }
    if (lane == 0)
        out->inv = pow2_field(127 - qe);
}

struct DecodeArgs {
    const __nv_bfloat16 *q_tok;
    KvView kv;
    const int32_t *lens;
    const uint8_t *mask;
    int B, Hq, Hkv, L, nb, tiles, per_tile, nsplit;
    int slots;                           // of a head tile, shared out by length; 0: nsplit each
    float scale_log2;
    float *part;
    __nv_bfloat16 *o;
    float *lse;
    int *status;
    uint64_t timeout_ns;
};

// Warps of a CTA and half records in flight per warp.  Two CTAs share an SM, so
// that one's start and end (some 8,000 cycles of latencies) pass under the
// other's products; their rings hold 70 to 200 KB, where the SM's share of HBM
// (24 bytes a cycle) needs some 40 KB in flight.
template <int BITS, int D>
struct DecodeCfg {
    static constexpr int W = BITS == 8 && D == 128 ? 6 : 8;
    static constexpr int ST = BITS == 4 && D == 64 ? 4 : 2;
    static constexpr int ring = W * ST * KvFmt<BITS, D>::HALF;
};

// The CTAs of a head tile: nsplit for every sequence or, with lengths given (and
// few enough sequences for one look at them), a number of slots of which every
// sequence has one and a share of the others in proportion to its blocks, so
// that a batch of unequal lengths ends together.  slot_of: the sequence that a
// slot serves, which of its splits it is and how many there are (one warp; false:
// it serves nothing).
constexpr int kBalanced = 64;             // sequences

__device__ __forceinline__ int blocks_of(const DecodeArgs &a, int b)
{
    return b < a.B ? (max(0, min(__ldg(a.lens + b), a.L)) + 63) / 64 : 0;
}

struct Shares {
    int first[2], count[2];               // slots of sequences lane, lane + 32
};

__device__ __forceinline__ Shares shares(const DecodeArgs &a, int lane)
{
    int n[2], before[2], total = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        n[i] = blocks_of(a, lane + 32 * i);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int inc = n[i];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            inc += lane >= off ? v : 0;
        }
        before[i] = total + inc - n[i];
        total += __shfl_sync(0xffffffffu, inc, 31);
    }
    // a rising function of the blocks before, so the shares neither overlap nor leave gaps
    const float rate = total > 0 ? (float)(a.slots - a.B) / (float)total : 0.f;
    Shares s;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s.first[i] = lane + 32 * i + (int)((float)before[i] * rate);
        s.count[i] = lane + 32 * i + 1 + (int)((float)(before[i] + n[i]) * rate) - s.first[i];
    }
    return s;
}

__device__ __forceinline__ bool slot_of(const DecodeArgs &a, int lane, int &b, int &split, int &ns)
{
    const int c = blockIdx.x;
    if (a.slots == 0) {
        b = blockIdx.z;
        split = c;
        ns = a.nsplit;
        return true;
    }
    const Shares s = shares(a, lane);
    b = -1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned hit =
            __ballot_sync(0xffffffffu, lane + 32 * i < a.B && c >= s.first[i] && c < s.first[i] + s.count[i]);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            b = src + 32 * i;
            split = c - __shfl_sync(0xffffffffu, s.first[i], src);
            ns = min(__shfl_sync(0xffffffffu, s.count[i], src), kMaxDecodeSplits);
        }
    }
    return b >= 0 && split < ns;
}

__device__ __forceinline__ int splits_of(const DecodeArgs &a, int b, int lane)
{
    if (a.slots == 0)
        return a.nsplit;
    const Shares s = shares(a, lane);
    return min(__shfl_sync(0xffffffffu, b < 32 ? s.count[0] : s.count[1], b & 31), kMaxDecodeSplits);
}

template <int BITS, int D>
__global__ void __launch_bounds__(DecodeCfg<BITS, D>::W * 32, 2) decode_quant_kernel(const DecodeArgs a)
{
    using F = KvFmt<BITS, D>;
    using C = DecodeCfg<BITS, D>;
    constexpr int W = C::W, ST = C::ST, NG = F::NG, R = F::R;
    constexpr int KS = D / 16;                      // MMA steps of a score; also MMA rows of an output / 16
    constexpr int KW = R / 16, VW = R / 32;         // 32-bit words of a lane's K row, V row
    constexpr int UPG = KS / NG;                    // MMAs of a group
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t s_bar[W * ST];
    __shared__ float2 s_ml[W][kHeads], s_sum[kHeads];
    __shared__ uint32_t s_words[kMaxNb / 32];
    __shared__ uint32_t s_rec[kListMax];            // a block's record from the start of the pages, in 512 bytes
    __shared__ uint16_t s_block[kListMax];
    __shared__ __align__(16) HeadQ<D> s_q[kHeads];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    int b, split, ns;
    if (!slot_of(a, lane, b, split, ns))
        return;
    const int tile = blockIdx.y % a.tiles, kvh = blockIdx.y / a.tiles;
    const int g = a.Hq / a.Hkv;
    const int h0 = kvh * g + tile * a.per_tile;     // first query head, and how many
    const int gt = min(a.per_tile, g - tile * a.per_tile);
    const int len = a.lens != nullptr ? max(0, min(a.lens[b], a.L)) : a.L;
    const uint8_t *mrow = a.mask + ((long long)b * a.Hq + h0) * a.nb;

    if (lane == 0) {
        for (int s = 0; s < ST; ++s)
            mbar_init(smem_u32(&s_bar[warp * ST + s]), 1);
        fence_mbar_init();
    }

    // ---- q, a warp per head (0 where there is none)
    for (int h = warp; h < kHeads; h += W)
        prepare_q<BITS, D>(h < gt ? a.q_tok + ((long long)b * a.Hq + h0 + h) * D : nullptr, lane, &s_q[h]);

    // ---- union of the heads' active blocks, one bit each.  Rows short enough for
    // one round of kMaskWords words of 32 blocks a warp: a block a lane, and its
    // table entry, all loads in flight together (and before the length is known).
    // Longer rows: four blocks a lane, where the rows' alignment allows it, and
    // the table is looked up for this split's blocks alone.
    constexpr int kMaskWords = BITS == 8 && D == 128 ? 6 : 4;
    const int nblk = (len + 63) / 64, nwords = (nblk + 31) / 32;
    const bool one_round = a.nb <= 32 * kMaskWords * W;
    int page[kMaskWords];
    if (one_round || a.nb % 4 != 0 || (reinterpret_cast<uintptr_t>(a.mask) & 3) != 0) {
        for (int c0 = warp; c0 < (c0 == warp ? (a.nb + 31) / 32 : nwords); c0 += kMaskWords * W) {
            int raw[kMaskWords][kHeads];
            // (blocks past the row read its last one: the branches are the warp's)
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i) {
                if (i > 0 && (c0 + i * W) * 32 >= a.nb)
                    continue;
                const int j = min((c0 + i * W) * 32 + lane, a.nb - 1);
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    raw[i][h] = 0;
                    if (h < gt)
                        raw[i][h] = __ldg(mrow + (long long)h * a.nb + j);
                }
                if (one_round) {
                    page[i] = b * a.kv.max_blocks + j;
                    if (a.kv.table != nullptr)
                        page[i] = __ldg(a.kv.table + page[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i) {
                const int c = c0 + i * W;
                if (c >= nwords)
                    continue;
                int any = 0;
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    any |= raw[i][h];
                const unsigned bits = __ballot_sync(0xffffffffu, any != 0 && c * 32 + lane < nblk);
                if (lane == 0)
                    s_words[c] = bits;
            }
        }
    } else {
        for (int c0 = warp; c0 * 4 < nwords; c0 += 4 * W) {
            uint32_t raw[4][kHeads];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = min((c0 + i * W) * 128 + 4 * lane, a.nb - 4);
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    raw[i][h] = 0;
                    if (h < gt)
                        raw[i][h] = __ldg(reinterpret_cast<const uint32_t *>(mrow + (long long)h * a.nb + j));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = (c0 + i * W) * 128 + 4 * lane;
                uint32_t x = 0;
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    x |= raw[i][h];
                // bytes that are not 0 -> four bits -> words of eight lanes
                x = (((x & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | x) >> 7 & 0x01010101u;
                x = x * 0x10204080u >> 28 & ((1u << max(0, min(4, nblk - j))) - 1u);
                x <<= 4 * (lane & 7);
                x |= __shfl_xor_sync(0xffffffffu, x, 1);
                x |= __shfl_xor_sync(0xffffffffu, x, 2);
                x |= __shfl_xor_sync(0xffffffffu, x, 4);
                if ((lane & 7) == 0 && j / 32 < nwords)
                    s_words[j / 32] = x;
            }
        }
    }
    __syncthreads();
    // a score in units of log2: its raw sum times fac (kept off 0 and infinity, so
    // that a masked score's -infinity stays one)
    float fac[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        fac[e] = fminf(fmaxf(s_q[2 * tig + e].inv * (a.scale_log2 * 16777216.f), 1.2e-38f), 3e38f);

    // ---- this split's blocks: ranks [r0, r1) of the union
    int r0, r1;
    {
        // words of a lane: a power of two (32 lanes cover the words)
        const int lg = nwords > 32 ? 32 - __clz((nwords - 1) >> 5) : 0, per = 1 << lg;
        int cnt = 0;
        for (int k = 0; k < per; ++k)
            if (lane * per + k < nwords)
                cnt += __popc(s_words[lane * per + k]);
        int inc = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            inc += lane >= off ? v : 0;
        }
        const int total = __shfl_sync(0xffffffffu, inc, 31);
        // total * split / ns: at most 2^20, and inv is 2^32 / ns rounded up by less
        // than 2^-26 of it, so the product's high word is the quotient (one split:
        // inv is 0 and so is r0)
        const unsigned inv = 0xFFFFFFFFu / (unsigned)ns + 1u;
        r0 = (int)__umulhi((unsigned)(total * split), inv);
        r1 = split + 1 == ns ? total : (int)__umulhi((unsigned)(total * (split + 1)), inv);
        // an entry: the block, with kNoPage where its table entry names no page
        // (recorded; page 0 is copied in its place and none of its tokens counts)
        auto entry = [&](int i, int j, int pg) {
            const bool bad = pg < 0 || pg >= a.kv.n_pages;
            if (bad)
                set_status(a.status, kStatusPage);
            s_block[i] = (uint16_t)(bad ? j | kNoPage : j);
            s_rec[i] = ((uint32_t)(bad ? 0 : pg) * a.Hkv + kvh) * (F::REC / 512);
        };
        auto list = [&](int c, int pg) {            // this lane's block of word c
            int base = __shfl_sync(0xffffffffu, inc - cnt, c >> lg);
            for (int k = c >> lg << lg; k < c; ++k)
                base += __popc(s_words[k]);
            const unsigned w = s_words[c];
            const int r = base + __popc(w & ((1u << lane) - 1u));
            if ((w >> lane & 1u) && r >= r0 && r < r1) {
                if (one_round)
                    entry(r - r0, c * 32 + lane, pg);
                else
                    s_block[r - r0] = (uint16_t)(c * 32 + lane);
            }
        };
        if (one_round) {
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i)
                if (warp + i * W < nwords)
                    list(warp + i * W, page[i]);
        } else {
            for (int c = warp; c < nwords; c += W)
                list(c, 0);
            __syncthreads();
            for (int i = threadIdx.x; i < r1 - r0; i += W * 32) {
                const int j = s_block[i], at = b * a.kv.max_blocks + j;
                entry(i, j, a.kv.table != nullptr ? __ldg(a.kv.table + at) : at);
            }
        }
    }
    __syncthreads();

    const int n_units = 2 * (r1 - r0);              // half records
    uint8_t *my = ring + warp * ST * F::HALF;
    const uint32_t my_bar = smem_u32(&s_bar[warp * ST]);
    auto first_token = [&](int u) { return 64 * (s_block[u >> 1] & (kNoPage - 1)) + 32 * (u & 1); };
    auto issue = [&](int u, int st) {               // lane 0
        if (u >= n_units || first_token(u) >= len)
            return;
        mbar_arrive_expect_tx(my_bar + 8 * st, F::HALF);
        bulk_copy(smem_u32(my + st * F::HALF), a.kv.pages + (unsigned long long)s_rec[u >> 1] * 512 + (u & 1) * F::HALF,
                  F::HALF, my_bar + 8 * st);
    };
    auto head_byte = [&](int u) {
        return u < n_units && lane < gt ? (int)__ldg(mrow + (long long)lane * a.nb + (s_block[u >> 1] & (kNoPage - 1))) : 0;
    };
    if (lane == 0)
        for (int s = 0; s < ST; ++s)
            issue(warp + s * W, s);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, zacc[NG][2], acc[KS][4];
    int ve = 27;                                    // exponent field of V's largest scale so far
#pragma unroll
    for (int i = 0; i < KS; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
        zacc[gr][0] = zacc[gr][1] = 0.f;

    // this lane's places in a half record: K row and params of tile row gid (row
    // gid + 8 and the second tile a whole number of rows further, with the same
    // swizzle), V words of tile columns 2 tig and 2 tig + 1
    const int tr = tile_token(gid), t0 = tile_token(2 * tig), t1 = tile_token(2 * tig + 1);
    const int at_k = tr * R + (BITS == 8 && D == 128 ? (tr & 1) * 64 + tig * 16 : tig * (R / 4));
    const int at_p = tr * F::PAR, at_z = F::kParK + at_p + (tig < NG ? tig * 4 : 0);
    const int at_v0 = F::kCodeV + t0 * R + (gid ^ F::v_swizzle(t0)) * (R / 8);
    const int at_v1 = F::kCodeV + t1 * R + (gid ^ F::v_swizzle(t1)) * (R / 8);

    int mb = head_byte(warp);
    int it = 0;
    for (int u = warp; u < n_units; u += W, ++it) {
        const unsigned hbits = __ballot_sync(0xffffffffu, mb != 0 || lane >= gt);
        mb = head_byte(u + W);
        int keys = len - first_token(u);
        if (keys <= 0)
            break;                                  // the empty half of the last block: nothing follows
        if (s_block[u >> 1] & kNoPage)
            keys = 0;
        const int st = it % ST;
        {
            const uint32_t bar = my_bar + 8 * st, parity = (it / ST) & 1;
            bool done = mbar_test_wait(bar, parity);
            if (!done) {
                const uint64_t t0 = globaltimer();
                while (!done && globaltimer() - t0 < a.timeout_ns)
                    done = mbar_try_wait_sleep(bar, parity, 20000u);
            }
            if (!__all_sync(0xffffffffu, done)) {
                // give up: wait for this warp's copies in flight, contribute nothing
                set_status(a.status, kStatusTimeout);
                for (int s = 0; s < ST; ++s) {
                    const int w = it + s;
                    const int uu = warp + w * W;
                    if (uu < n_units && first_token(uu) < len)
                        mbar_drain(my_bar + 8 * (w % ST), (w / ST) & 1, 200000000ull);
                }
                m[0] = m[1] = -INFINITY;
                l[0] = l[1] = 0.f;
                break;
            }
        }
        const uint8_t *h = my + st * F::HALF;
        // q's operands of column gid (read for every half record: the registers are
        // P V's afterwards) and the one against the params as they lie, (s, z) of
        // group tig: 0 for s, q's sum for z
        uint32_t qf[KS][2], qz[3];
        {
            const HeadQ<D> &q = s_q[gid];
#pragma unroll
            for (int i = 0; i < KS; i += 2) {
                if (BITS == 4) {                    // a word's eight elements: two MMA steps
                    const uint4 x = *reinterpret_cast<const uint4 *>(q.f16 + 16 * i + 8 * tig);
                    qf[i][0] = x.x;
                    qf[i][1] = x.y;
                    qf[i + 1][0] = x.z;
                    qf[i + 1][1] = x.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(q.f16 + 16 * (i + k) + 4 * tig);
                        qf[i + k][0] = x.x;
                        qf[i + k][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                qz[i] = tig < NG ? (uint32_t)q.sum[i][tig] << 16 : 0u;
        }

        // ---- raw scores of two 16-token tiles
        float s[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            const uint8_t *ha = h + at_k + 16 * mt * R, *hp = h + F::kParK + at_p + 16 * mt * F::PAR;
            uint32_t ka[KW], kb[KW], pa[NG], pb[NG];
            if constexpr (BITS == 8 && D == 128) {  // the other half of the row is 64 bytes up or down
                uint32_t (&a0)[4] = *reinterpret_cast<uint32_t (*)[4]>(ka);
                uint32_t (&a1)[4] = *reinterpret_cast<uint32_t (*)[4]>(ka + 4);
                uint32_t (&b0)[4] = *reinterpret_cast<uint32_t (*)[4]>(kb);
                uint32_t (&b1)[4] = *reinterpret_cast<uint32_t (*)[4]>(kb + 4);
                const uint8_t *hb = ha + (tr & 1 ? -64 : 64);
                load_words(a0, ha);
                load_words(a1, hb);
                load_words(b0, ha + 8 * R);
                load_words(b1, hb + 8 * R);
            } else {
                load_words(ka, ha);
                load_words(kb, ha + 8 * R);
            }
            load_words(pa, hp);
            load_words(pb, hp + 8 * F::PAR);
            {                                       // z sum(q) of the groups: the params themselves are the operand
                                                    // (lanes past the last group: their q sums are 0)
                const uint32_t wa = *reinterpret_cast<const uint32_t *>(h + at_z + 16 * mt * F::PAR);
                const uint32_t wb = *reinterpret_cast<const uint32_t *>(h + at_z + (16 * mt + 8) * F::PAR);
                mma16816_bf16_0(s[mt], wa, wb, wa, wb, qz[0], qz[1]);
                mma16816_bf16(s[mt], wa, wb, 0u, 0u, qz[2], 0u);
            }
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                float c[4];
#pragma unroll
                for (int i = 0; i < UPG; ++i) {
                    const int ks = gr * UPG + i;
                    uint32_t x[4];
                    if (BITS == 4) {
                        const uint32_t wa = ka[ks / 2] >> (8 * (ks % 2)), wb = kb[ks / 2] >> (8 * (ks % 2));
                        x[0] = wa & 0x000F000Fu;
                        x[1] = wb & 0x000F000Fu;
                        x[2] = wa & 0x00F000F0u;
                        x[3] = wb & 0x00F000F0u;
                    } else {
                        x[0] = __byte_perm(ka[ks], 0u, 0x4140);
                        x[1] = __byte_perm(kb[ks], 0u, 0x4140);
                        x[2] = __byte_perm(ka[ks], 0u, 0x4342);
                        x[3] = __byte_perm(kb[ks], 0u, 0x4342);
                    }
                    if (i == 0)
                        mma16816_0(c, x[0], x[1], x[2], x[3], qf[ks][0], qf[ks][1]);
                    else
                        mma16816(c, x[0], x[1], x[2], x[3], qf[ks][0], qf[ks][1]);
                }
                const float sa = kv_scale(pa[gr]), sb = kv_scale(pb[gr]);
                s[mt][0] = fmaf(sa, c[0], s[mt][0]);
                s[mt][1] = fmaf(sa, c[1], s[mt][1]);
                s[mt][2] = fmaf(sb, c[2], s[mt][2]);
                s[mt][3] = fmaf(sb, c[3], s[mt][3]);
            }
        }
        const bool all_heads = hbits == 0xffffffffu;
        const bool act0 = hbits >> (2 * tig) & 1u, act1 = hbits >> (2 * tig + 1) & 1u;
        if (keys < 32) {                            // the sequence's last tokens
            __syncwarp();                           // (keeps this a branch)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (16 * mt + tr + (e & 2) * 4 >= keys)
                        s[mt][e] = -INFINITY;
        }

        // ---- V's params (zero behind the length) and the power of two for p s
        uint32_t vp[2][2][NG];                      // [tile][row, row + 8]
        uint32_t vmax = 0;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                load_words(vp[mt][hf], h + F::kParV + at_p + (16 * mt + 8 * hf) * F::PAR);
        if (keys < 32) {
            __syncwarp();
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
                        if (16 * mt + tr + 8 * hf >= keys)
                            vp[mt][hf][gr] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (NG == 1)
                vmax = __vmaxu2(vmax, vp[i / 2][i % 2][0]);
#pragma unroll
            for (int gr = 0; gr + 1 < NG; gr += 2)
                vmax = __vimax3_u16x2(vmax, vp[i / 2][i % 2][gr], vp[i / 2][i % 2][gr + 1]);
        }
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            mx[e] = fmaxf(fmaxf(s[0][e], s[0][e + 2]), fmaxf(s[1][e], s[1][e + 2]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
            vmax = __vmaxu2(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
        }
        const int ve_new = max(ve, (int)(vmax >> 7 & 0xFFu));
        // a head that left the block out: its maximum stays and its p are 0
        const bool more0 = act0 && mx[0] > m[0], more1 = act1 && mx[1] > m[1];
        if (__any_sync(0xffffffffu, more0 || more1 || ve_new != ve)) {
            float alpha[2];
            const float m_new[2] = {more0 ? mx[0] : m[0], more1 ? mx[1] : m[1]};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                alpha[e] = m_new[e] == m[e] ? 1.f : exp2_approx((m[e] - m_new[e]) * fac[e]);
                m[e] = m_new[e];
            }
            const float down = ve - ve_new > -127 ? pow2_field(127 + ve - ve_new) : 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][e] *= alpha[e & 1] * down;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                zacc[gr][0] *= alpha[0];
                zacc[gr][1] *= alpha[1];
            }
            l[0] *= alpha[0];
            l[1] *= alpha[1];
            ve = ve_new;
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : -m[0] * fac[0], m[1] == -INFINITY ? 0.f : -m[1] * fac[1]};
        const float up = pow2_field(268 - ve);      // 2^14 over the power of two below the largest scale

        // ---- P V
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = exp2_approx(fmaf(s[mt][e], fac[e & 1], mu[e & 1]));
            if (!all_heads) {
                p[0] = act0 ? p[0] : 0.f;
                p[1] = act1 ? p[1] : 0.f;
                p[2] = act0 ? p[2] : 0.f;
                p[3] = act1 ? p[3] : 0.f;
            }
            l[0] += p[0] + p[2];
            l[1] += p[1] + p[3];
            uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
            load_words(v0, h + at_v0 + 16 * mt * R);
            load_words(v1, h + at_v1 + 16 * mt * R);
            load_words(v2, h + at_v0 + (16 * mt + 8) * R);
            load_words(v3, h + at_v1 + (16 * mt + 8) * R);
            float pu[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pu[e] = p[e] * up;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                const float sa = kv_scale(vp[mt][0][gr]), sb = kv_scale(vp[mt][1][gr]);
                const float za = kv_zero(vp[mt][0][gr]), zb = kv_zero(vp[mt][1][gr]);
                const uint32_t b0 = movmatrix(pack_half2(pu[0] * sa, pu[1] * sa));
                const uint32_t b1 = movmatrix(pack_half2(pu[2] * sb, pu[3] * sb));
                if (act0)                           // a NaN of V stays out of heads that left the block out
                    zacc[gr][0] = fmaf(p[0], za, fmaf(p[2], zb, zacc[gr][0]));
                if (act1)
                    zacc[gr][1] = fmaf(p[1], za, fmaf(p[3], zb, zacc[gr][1]));
                if constexpr (BITS == 4) {
                    const unsigned sel = gr & 1 ? 0x7632u : 0x5410u;
                    // lower rows: an element; upper rows: the byte, that element plus 16 times the next
                    const uint32_t x01 = __byte_perm(v0[gr / 2], v1[gr / 2], sel), x23 = __byte_perm(v2[gr / 2], v3[gr / 2], sel);
#pragma unroll
                    for (int i = 0; i < UPG; ++i) {
                        const uint32_t y01 = i ? __byte_perm(x01, 0u, 0x4341) : x01 & 0x00FF00FFu;
                        const uint32_t y23 = i ? __byte_perm(x23, 0u, 0x4341) : x23 & 0x00FF00FFu;
                        mma16816(acc[gr * UPG + i], y01 & 0x000F000Fu, y01, y23 & 0x000F000Fu, y23, b0, b1);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < UPG; ++i) {
                        const int w = 2 * gr + i / 2;
                        const unsigned sel = i & 1 ? 0x7632u : 0x5410u;
                        const uint32_t x01 = __byte_perm(v0[w], v1[w], sel), x23 = __byte_perm(v2[w], v3[w], sel);
                        mma16816(acc[gr * UPG + i], __byte_perm(x01, 0u, 0x4240), __byte_perm(x01, 0u, 0x4341),
                                 __byte_perm(x23, 0u, 0x4240), __byte_perm(x23, 0u, 0x4341), b0, b1);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            issue(u + ST * W, st);
    }

    // ---- sums over the lanes that share a head, then over the warps
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
                zacc[gr][e] += __shfl_xor_sync(0xffffffffu, zacc[gr][e], off);
        }
    __syncwarp();
    if (gid == 0) {
        s_ml[warp][2 * tig] = make_float2(m[0] == -INFINITY ? m[0] : m[0] * fac[0], l[0]);
        s_ml[warp][2 * tig + 1] = make_float2(m[1] == -INFINITY ? m[1] : m[1] * fac[1], l[1]);
    }
    float *so = reinterpret_cast<float *>(my);      // [kHeads][D], over this warp's ring
    {
        const float un = pow2_field(ve - 14);       // with 2^24 the inverse of `up` and the codes' unit
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                for (int i = 0; i < UPG; i += 2) {
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float lo = acc[gr * UPG + i + k][e], hi = acc[gr * UPG + i + k][e + 2];
                        v[2 * k] = lo * un * 16777216.f + zacc[gr][e];
                        v[2 * k + 1] = (BITS == 4 ? (hi - lo) * un * 1048576.f : hi * un * 16777216.f) + zacc[gr][e];
                    }
                    const float4 r = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(so + (2 * tig + e) * D + F::G * gr + gid * (F::G / 8) + 2 * i) = r;
                }
    }
    __syncthreads();
    for (int hh = warp; hh < gt; hh += W) {         // the warps' weights for a head
        const float2 ml = lane < W ? s_ml[lane][hh] : make_float2(-INFINITY, 0.f);
        float M = ml.x;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float wt = split_weight(ml.x, ml.y, M);
        float lt = wt * ml.y;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            lt += __shfl_xor_sync(0xffffffffu, lt, off);
        if (lane < W)
            s_ml[lane][hh].x = wt;
        if (lane == 0)
            s_sum[hh] = make_float2(M, lt);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < gt * D; i += W * 32) {
        const int hh = i / D, c = i % D;
        const float lt = s_sum[hh].y;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float wt = s_ml[w][hh].x;
            if (wt != 0.f)
                sum = fmaf(wt, *reinterpret_cast<const float *>(ring + w * ST * F::HALF + i * 4), sum);
        }
        const long long bh = (long long)b * a.Hq + h0 + hh;
        if (ns == 1) {
            a.o[bh * D + c] = __float2bfloat16_rn(lt == 0.f ? 0.f : sum / lt);
            if (c == 0 && a.lse != nullptr)
                a.lse[bh] = log_sum(s_sum[hh].x, lt);
        } else {
            float *out = a.part + (bh * kMaxDecodeSplits + split) * (D + 2);
            out[c] = sum;
            if (c == 0) {
                out[D] = s_sum[hh].x;
                out[D + 1] = lt;
            }
        }
    }
}

// The splits of one head: weights 2^(m_s - M), o = sum w o / sum w l.  Q threads
// share an output element, every Q-th split each, and their first loads are in
// flight before a weight is known.  Four from nine splits on: one latency, not
// one per eight splits (128k tokens, 37 splits: 2.7 us less of 40.8); one for few
// (1024 heads of two splits: 90 us a call, 96 with four).
template <int D, int Q>
__global__ void __launch_bounds__(Q * D) decode_quant_merge_kernel(const DecodeArgs a)
{
    constexpr int N = Q == 4 ? kMaxDecodeSplits / 4 : 8;
    __shared__ float s_w[kMaxDecodeSplits], s_part[Q][D];
    const long long bh = blockIdx.x;
    const int lane = threadIdx.x & 31, c = threadIdx.x % D, q = threadIdx.x / D;
    const int nsplit = splits_of(a, blockIdx.x / a.Hq, lane);
    if (nsplit == 1)
        return;                                     // written by its one split
    const float *pp = a.part + bh * kMaxDecodeSplits * (D + 2);
    float v[N], ms[2], ls[2], M = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 32 * i;
        ms[i] = s < nsplit ? pp[s * (D + 2) + D] : -INFINITY;
        ls[i] = s < nsplit ? pp[s * (D + 2) + D + 1] : 0.f;
    }
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = s0 + Q * i + q;
            v[i] = s < nsplit ? pp[s * (D + 2) + c] : 0.f;
        }
    };
    load(0);
    M = fmaxf(ms[0], ms[1]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float w = split_weight(ms[i], ls[i], M);
        l = fmaf(w, ls[i], l);
        if (threadIdx.x < 32)
            s_w[lane + 32 * i] = w;                 // 0 past the last split
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, off);
    __syncthreads();
    float acc = 0.f;
    for (int s0 = 0; s0 < nsplit; s0 += N * Q) {
        if (s0 > 0)
            load(s0);
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc = fmaf(s_w[s0 + Q * i + q], v[i], acc);
    }
    if constexpr (Q > 1) {
        s_part[q][c] = acc;
        __syncthreads();
        if (q != 0)
            return;
        acc = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i)
            acc += s_part[i][c];
    }
    a.o[bh * D + c] = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
    if (a.lse != nullptr && c == 0)
        a.lse[bh] = log_sum(M, l);
}

// Estimated time, in us, of `ctas` CTAs with `blocks` blocks each:
//   a CTA's start and end     6 alone on its SM, 7.5 for two at once, per wave
//   a block                   0.4 for a CTA alone, 0.31 of the SM for two
//   the second kernel         2 and 0.04 a split
// Measured (4 bits, D = 128): 8 units (a sequence's head tile) of 512 blocks, all
// active: 18 splits 20.7 us, 24: 23.8, 37: 19.8; a tenth active: 9: 15.2, 18: 11.8,
// 37: 12.4; 128 units of 256: 1 split 97 us, 2: 86, 4: 91.
double decode_quant_us(long long ctas, double blocks, double splits, int sms)
{
    const long long load = (ctas + sms - 1) / sms, waves = (load + 1) / 2;
    return (load == 1 ? 6.0 + 0.4 * blocks : 7.5 * (double)waves + 0.31 * (double)load * blocks) +
           (splits > 1.0 ? 2.0 + 0.04 * splits : 0.0);
}

// How a call is split (nsplit, slots): the least estimated time with half of the
// blocks active (the mask is on the device) and at least a block for every
// second warp.  Lengths given: one or two CTAs per SM in all, where there are
// enough for every sequence's tiles, shared out by length: a batch of 8 from 32k
// tokens down takes 45 us with 4 splits each, 39 so.  Not for two or three
// sequences, whose CTAs pair up on the SMs (64k and 37k tokens at 8 bits: 42 us with
// 18 splits each, 45 shared out), and in whole splits where a sequence has few
// (16 of 16k tokens: 88 us with two each, 90 with 37 slots).
void decode_quant_split(DecodeArgs &a, int sms)
{
    const int tiles = a.Hkv * a.tiles;
    const int lo = (a.nb + kListMax - 2) / (kListMax - 1);            // a split's block list has to fit
    const int cap = a.nb / 4 < kMaxDecodeSplits ? a.nb / 4 : kMaxDecodeSplits;
    double best_us = 1e30;
    a.nsplit = lo;
    a.slots = 0;
    for (int ns = lo; ns <= cap; ++ns) {
        const double us = decode_quant_us((long long)a.B * tiles * ns, 0.5 * a.nb / ns, ns, sms);
        if (us < best_us) {
            best_us = us;
            a.nsplit = ns;
        }
    }
    if (a.lens == nullptr || a.B < 4 || a.B > kBalanced)
        return;
    best_us = 1e30;
    for (int load = 1; load <= 2; ++load) {
        int slots = load * sms / tiles;
        if (slots < 4 * a.B)
            slots -= slots % a.B;
        // a sequence's share of slots - B is at least that of its blocks in B * nb
        if (slots < a.B * (1 + lo) || slots > a.B * (1 + cap))
            continue;
        const double each = (double)slots / a.B;
        const double us = decode_quant_us((long long)slots * tiles, 0.5 * a.nb / each, each, sms);
        if (us < best_us) {
            best_us = us;
            a.slots = slots;
        }
    }
}

template <int BITS, int D>
cudaError_t launch(DecodeArgs a, cudaStream_t stream)
{
    using C = DecodeCfg<BITS, D>;
    const int g = a.Hq / a.Hkv;
    a.tiles = (g + kHeads - 1) / kHeads;
    a.per_tile = (g + a.tiles - 1) / a.tiles;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_quant_kernel<BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ring);
    if (e != cudaSuccess)
        return e;
    decode_quant_split(a, sms);
    const dim3 grid(a.slots > 0 ? a.slots : a.nsplit, a.Hkv * a.tiles, a.slots > 0 ? 1 : a.B);
    decode_quant_kernel<BITS, D><<<grid, C::W * 32, C::ring, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || (a.slots == 0 && a.nsplit == 1))
        return e;
    if ((a.slots > 0 ? a.slots / a.B : a.nsplit) > 8)
        decode_quant_merge_kernel<D, 4><<<a.B * a.Hq, 4 * D, 0, stream>>>(a);
    else
        decode_quant_merge_kernel<D, 1><<<a.B * a.Hq, D, 0, stream>>>(a);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_decode_quant(int bits, int B, int Hq, int Hkv, int L, int d, float scale_log2, const void *q_tok,
                                const KvView &kv, const int32_t *lens, const uint8_t *mask, void *o, float *lse,
                                float *part, int *status, uint64_t timeout_ns, cudaStream_t stream)
{
    DecodeArgs a{};
    a.q_tok = static_cast<const __nv_bfloat16 *>(q_tok);
    a.kv = kv;
    a.lens = lens;
    a.mask = mask;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.L = L;
    a.nb = num_blocks(L);
    a.scale_log2 = scale_log2;
    a.part = part;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.status = status;
    a.timeout_ns = timeout_ns;
    if (bits == 4)
        return d == 128 ? launch<4, 128>(a, stream) : launch<4, 64>(a, stream);
    return d == 128 ? launch<8, 128>(a, stream) : launch<8, 64>(a, stream);
}

} // namespace seer

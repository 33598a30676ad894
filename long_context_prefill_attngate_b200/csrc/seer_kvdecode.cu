// seer_kvdecode.cu — block-sparse attention of one new token per sequence over
// the quantised cache.
//
//   o[b,h] = sum over t < len in active blocks of softmax(q . k_t * scale) v_t,
//   k_t = z + s n (per group of the row), v_t likewise.
//
// Each active block crosses HBM once per GQA group: a CTA serves up to eight, or
// sixteen, query heads of one KV head over the union of their active blocks (a
// head without a block gets p = 0 there).  At 4 bits a token's K and V are 160 bytes
// for 4 D flops per head, so with CUDA-core products the arithmetic, not HBM,
// would set the time (at D = 128 and four heads 2048 flops per 160 bytes); the
// products are mma.sync m16n8k16 with the keys on M (K Q^T) or the output
// elements on M (V^T P) and the heads on N; with more than eight heads the other
// way round (Sums<.., 16>).  Sixteen rows at most leave a tcgen05 tile nothing to
// gain.
//
//  * The codes enter the MMA as they are: n <= 255 in the low bits of a bf16 is
//    n 2^-133 (below 128 a subnormal, from there on the first binade, which has the
//    same step), so one mask (4 bits) or byte permute (8 bits) makes a pair of
//    operands, and scale and zero are applied outside:
//      q . k   = sum_g s_g (q_g . n_g) + z_g sum(q_g)        per key; the second by an
//                MMA of the params as they lie with sum(q_g) in three bf16 parts
//      sum p v = sum_t (p_t s_t,g) (n_t - c) + sum_t p_t (z_t,g + c s_t,g)
//    q is bf16 already, times a power of two per head: exact down to 2^-116 of the
//    head's largest element.  p s is two bf16 parts, which leave at most 2^-16 of it
//    (one fp16 leaves 2^-11 and has no room for scales 2^20 apart), times a power of two
//    that follows the largest scale in the blocks that the head chose: the parts keep
//    their bits down to 2^-100 of it, whatever other heads read.  c is the middle of the
//    codes: without it the sum of p s n, some sqrt(tokens) times what is left after the
//    zeros, loses as much more to the accumulators' rounding (16k tokens: 2^-13 of o).
//    p z, the row sums and all accumulators are fp32.
//  * The running maximum moves when a score is 2^6 above it, so the accumulators
//    are rescaled a few times per warp; p is 2^-26 at the maximum and reaches 2^-20.
//    It is subtracted before the factor of the exponent: of scores beyond 2^24 the
//    product's rounding alone would be more than p's whole range.
//  * Work of a warp: half records of 32 tokens, each one contiguous bulk copy
//    into the warp's own ring, so no warp waits for another until the end.
//  * P leaves K Q^T with keys across lanes and enters V^T P with keys across a
//    lane's register pair: movmatrix turns each 8 x 8 piece.
//  * Split over the union's blocks by rank, so splits differ by one block at
//    most; a second kernel joins them.
//
// What bounds it: with 8 bits and long caches HBM and what is around the loop (128k
// tokens at density 0.17: 35.5 us with start, end and join, 22.8 at the copy rate).
// With 4 bits the loop (32k tokens of a layer, all active: 19.6 us, 6.4 at the copy rate):
// its warps issue in 51 % of the cycles (47 % with sixteen heads, whose registers allow
// eight warps an SM) and no pipe is busier than 41 %, so the latency of a warp's chain,
// scores to maximum to exponential to P V, is not hidden.  Short ones: a CTA's start and
// end, some 8,000 cycles of latencies, and the join (32k at density 0.1: 11.8 us; 200
// tokens: 4.6).
#include <cuda_bf16.h>

#include "seer_internal.h"
#include "seer_kv.cuh"

namespace seer {

namespace {

constexpr int kListMax = 513;             // blocks of a split (decode_quant_split)
constexpr int kSlack = 6;                  // a maximum moves when a score is 2^kSlack above it
// p is 2^-kTop at the running maximum, so at most 2^-20: 2^20 tokens of values below
// 2^126 sum up within fp32.
constexpr float kTop = 26.f;
constexpr int kNoPage = kMaxNb;           // flag of a list entry; block indices are below it
// p s times scale_up(ve) is below 2^124 for scales whose exponent field is at
// most ve; what the accumulators hold times kUnit and scale_un(ve) is in units of
// V again.  ve is at least kLeastScale: p times scale_up stays a float.
constexpr int kLeastScale = 143;
constexpr int kSlackScale = 8;             // ve moves that much past a scale that is above it
constexpr float kUnit = 18446744073709551616.f;   // 2^64 of the codes' 2^133

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: no accumulator to clear.
__device__ __forceinline__ void mma16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two values as kParts bf16 pairs each, every one the rounding of what the ones
// before left: a part holds 8 bits, so two leave at most 2^-16 of a value.
constexpr int kParts = 2;

__device__ __forceinline__ void split(float x, float y, uint32_t (&part)[kParts])
{
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[i]) : "f"(y), "f"(x));
        if (i + 1 < kParts) {
            x -= __uint_as_float(part[i] << 16);
            y -= __uint_as_float(part[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ float pow2_field(int field) { return __uint_as_float((uint32_t)field << 23); }

// Codes of V less the middle of their range (8 of 16, 128 of 256; the byte of two
// 4-bit codes less 136), so that the accumulators hold what is about the size of
// the result and not of sum p s n.  Exact: below 2^8 units.
constexpr uint32_t kMid4 = 0x00080008u, kMidByte = 0x00880088u, kMid8 = 0x00800080u;

__device__ __forceinline__ uint32_t less(uint32_t n, uint32_t mid)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(n), "r"(mid));
    return r;
}

__device__ __forceinline__ float scale_up(int ve) { return pow2_field(397 - ve); }
__device__ __forceinline__ float scale_un(int ve) { return pow2_field(127 + 133 - 64 - (397 - ve - 127)); }

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

// Natural log of l 2^M; -inf where nothing was active.  (l is at least 2^-kTop.)
__device__ __forceinline__ float log_sum(float M, float l)
{
    return l == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M - kTop) + __log2f(l * 67108864.f)) * 0.69314718055994530942f;
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

// q for the MMAs: row gid of w holds head gid, or heads gid and gid + 8.  First
// its elements (bf16) times 2^qe in the order of the codes' operands (at 4 bits
// a word's elements 0,4,1,5,2,6,3,7 with the odd ones times 2^-4, as the codes'
// masks give them), 16 bytes a lane at a time: two steps' B operands of eight
// heads, one step's A operand of sixteen.  Then its group sums in three bf16
// parts for the products with z: an operand step meets the params' words (s, z)
// of a token as they lie, 0 in the place of s and a part in that of z.  Rows are
// 16 banks apart, so eight lanes read 16 bytes each without a conflict.
template <int BITS, int D, int H>
struct QShared {
    static constexpr int NG = KvFmt<BITS, D>::NG, P = H == 16 ? 2 : 1;
    static constexpr int STEPS = NG == 4 ? 2 : 1;   // MMA steps of z sum(q)
    static constexpr int kSum = P * D / 2;
    static constexpr int LEN = kSum + P * 8 * STEPS;
    uint32_t w[H / P][LEN + (48 - LEN % 32) % 32];
    float inv[H];                                   // 2^(109 - qe)

    // Element e's half word.
    __device__ __forceinline__ static int at(int h, int e)
    {
        const int ks = BITS == 4 ? e / 32 * 2 + (e >> 1 & 1) : e / 16, tig = BITS == 4 ? e / 8 % 4 : e / 4 % 4;
        const int reg = BITS == 4 ? e & 1 : e >> 1 & 1, half = BITS == 4 ? e >> 2 & 1 : e & 1;
        const int word = P == 1 ? (ks / 2 * 4 + tig) * 4 + ks % 2 * 2 + reg : (ks * 4 + tig) * 4 + reg * 2 + h / 8;
        return 2 * word + half;
    }
    // The word of register r of a step that meets group gr's params: part i, or 0 for the places left.
    static constexpr int kPlaces = NG == 1 ? 8 : 4;
    __device__ __forceinline__ static int at_sum(int h, int gr, int i)
    {
        const int step = NG == 4 ? i >> 1 : 0;
        const int tig = NG == 4 ? (gr >> 1) + 2 * (i & 1) : NG == 2 ? i : i >> 1;
        const int r = NG == 4 ? gr & 1 : NG == 2 ? gr : i & 1;
        return kSum + (P == 1 ? (tig * STEPS + step) * 2 + r : (tig * STEPS + step) * 4 + r * 2 + h / 8);
    }
    // The byte, within a token's params, of the word that lane tig's register r meets.
    __device__ __forceinline__ static int par_at(int tig, int r) { return NG == 4 ? 8 * (tig & 1) + 4 * r : NG == 2 ? 4 * r : 0; }

    // Head h by one warp: a lane's elements from memory (0 where qp is null) ...
    static constexpr int N = D / 32;
    using Raw = uint32_t[N / 2];
    __device__ __forceinline__ static void fetch(Raw &u, const __nv_bfloat16 *qp, int lane)
    {
        if constexpr (N == 4) {
            const uint2 x = qp != nullptr ? load(reinterpret_cast<const uint2 *>(qp) + lane) : make_uint2(0u, 0u);
            u[0] = x.x;
            u[1] = x.y;
        } else {
            u[0] = qp != nullptr ? load(reinterpret_cast<const uint32_t *>(qp) + lane) : 0u;
        }
    }
    // ... and into its row.
    __device__ __forceinline__ void prepare(const Raw &u, int h, int lane)
    {
        constexpr int GL = KvFmt<BITS, D>::G / N;   // lanes of a group
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            mx = fmaxf(mx, fabsf(f[i]));
        // max |q| 2^qe in [2^123, 2^124) where 2^qe is a float; no scaling for infinity
        const int eb = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)) >> 23);
        const int qe = eb == 255 ? 0 : min(250 - eb, 127);
        const float up = pow2_field(127 + qe), up_sum = pow2_field(127 + qe - 109);
        uint32_t *row = w[h % 8];
        uint16_t *half = reinterpret_cast<uint16_t *>(row);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s += f[i] * up_sum;
            half[at(h, N * lane + i)] = (uint16_t)(__float_as_uint(f[i] * (BITS == 4 && i & 1 ? up * 0.0625f : up)) >> 16);
        }
#pragma unroll
        for (int off = 1; off < GL; off <<= 1)
            s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= 5.9604644775390625e-8f;                // 2^(qe - 109) 2^-24: the unit of the codes' products, 2^qe 2^-133
        if (lane % GL == 0)
#pragma unroll
            for (int i = 0; i < kPlaces; ++i) {
                const __nv_bfloat16 part = __float2bfloat16_rn(s);
                row[at_sum(h, lane / GL, i)] = i < 3 ? (uint32_t)__bfloat16_as_ushort(part) << 16 : 0u;
                s -= __bfloat162float(part);
            }
        if (lane == 0)
            inv[h] = pow2_field(127 + 109 - qe);
    }
};

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

// Warps of a CTA, for P CTAs per SM, and half records in flight per warp.  Of two
// CTAs one's start and end (some 8,000 cycles of latencies) pass under the other's
// products; one has twice the warps for its list and half the splits to join.  The
// rings hold 70 to 200 KB, where the SM's share of HBM (24 bytes a cycle) needs some
// 40 KB in flight.  Sixteen heads: at D = 128 the accumulators leave eight warps of an
// SM their registers (64 units of 256 blocks at 4 bits, p s in one part: 72 us, 74 with
// twelve, which spill; at 8 bits 59 and 65), at D = 64 twelve.
template <int BITS, int D, int H, int P>
struct DecodeCfg {
    static constexpr int W = (H == 16 ? (D == 128 ? 4 : 6) : BITS == 8 && D == 128 ? 6 : 8) * (P == 1 ? 2 : 1);
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
    return b < a.B ? (max(0, min(load(a.lens + b), a.L)) + 63) / 64 : 0;
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

// What a warp sums up for the heads of its CTA, half record by half record.
// Up to eight heads: on N, keys or output elements on M.  Up to four stand in N
// twice (up to two four times), and the places share the groups of a row: each has
// p s and p z of its own, and one B operand serves a group of every place (32k tokens
// of a layer, groups of four, all active, p s in one part: 17.9 us, 19.5 with eight
// columns).
template <int BITS, int D, int H>
struct Sums {
    using F = KvFmt<BITS, D>;
    static constexpr int NG = F::NG, R = F::R;
    static constexpr float kMid = BITS == 4 ? 8.f : 128.f;
    static constexpr int KS = D / 16;               // MMA steps of a score; also MMA rows of an output / 16
    static constexpr int KW = R / 16, VW = R / 32;  // 32-bit words of a lane's K row, V row
    static constexpr int UPG = KS / NG;             // MMAs of a group
    static constexpr int REP = 8 / H, NS = NG / REP;   // places of a head, groups of a place
    static_assert(NS > 0);
    using Q = QShared<BITS, D, H>;

    float m[2], l[2], zacc[NS][2], acc[KS][4], fac[2];
    int ve[2];                                      // exponent field that V's scales stay within
    int gid, tig, tr, at_k, at_p, at_z, at_pv, at_v0, at_v1;

    __device__ __forceinline__ void clear()
    {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void init(const Q &sq, float scale, int lane)
    {
        gid = lane >> 2;
        tig = lane & 3;
        // a score in units of log2: its raw sum times fac (kept off 0 and infinity, so
        // that a masked score's -infinity stays one)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            fac[e] = fminf(fmaxf(sq.inv[(2 * tig + e) & (H - 1)] * scale, 1.2e-38f), 3e38f);
        clear();
        ve[0] = ve[1] = kLeastScale;
#pragma unroll
        for (int i = 0; i < KS; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
        for (int gr = 0; gr < NS; ++gr)
            zacc[gr][0] = zacc[gr][1] = 0.f;
        // this lane's places in a half record: K row and params of tile row gid (row
        // gid + 8 and the second tile a whole number of rows further, with the same
        // swizzle), V words of tile columns 2 tig and 2 tig + 1
        tr = tile_token(gid);
        const int t0 = tile_token(2 * tig), t1 = tile_token(2 * tig + 1);
        at_k = tr * R + (BITS == 8 && D == 128 ? (tr & 1) * 64 + tig * 16 : tig * (R / 4));
        at_p = tr * F::PAR;
        at_z = F::kParK + at_p + Q::par_at(tig, 0);
        at_pv = F::kParV + at_p + 2 * tig / H * 4 * NS;
        at_v0 = F::kCodeV + t0 * R + (gid ^ F::v_swizzle(t0)) * (R / 8);
        at_v1 = F::kCodeV + t1 * R + (gid ^ F::v_swizzle(t1)) * (R / 8);
    }

    // half record h, of which the first `keys` tokens count; hbits: the heads that chose its block
    __device__ __forceinline__ void step(const uint8_t *h, const Q &sq, unsigned hbits, int keys)
    {
        // q's operands of column gid (read for every half record: the registers are
        // P V's afterwards)
        uint32_t qf[KS][2], qz[2 * Q::STEPS];
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
            const uint4 x = *reinterpret_cast<const uint4 *>(&sq.w[gid & (H - 1)][8 * i + 4 * tig]);
            qf[i][0] = x.x;
            qf[i][1] = x.y;
            qf[i + 1][0] = x.z;
            qf[i + 1][1] = x.w;
        }
        load_words(qz, reinterpret_cast<const uint8_t *>(&sq.w[gid & (H - 1)][Q::kSum + 2 * Q::STEPS * tig]));

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
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = *reinterpret_cast<const uint32_t *>(h + at_z + (16 * mt + 8 * (i & 1)) * F::PAR + Q::par_at(0, i >> 1));
                mma16816_0(s[mt], x[0], x[1], x[2], x[3], qz[0], qz[1]);
                if constexpr (Q::STEPS == 2)
                    mma16816(s[mt], x[0], x[1], x[2], x[3], qz[2], qz[3]);
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
        const bool act0 = hbits >> (2 * tig & (H - 1)) & 1u, act1 = hbits >> ((2 * tig & (H - 1)) + 1) & 1u;
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
        uint32_t vp[2][2][NS];                      // [tile][row, row + 8]
        uint32_t vmax = 0;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                load_words(vp[mt][hf], h + at_pv + (16 * mt + 8 * hf) * F::PAR);
        if (keys < 32) {
            __syncwarp();
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int gr = 0; gr < NS; ++gr)
                        if (16 * mt + tr + 8 * hf >= keys)
                            vp[mt][hf][gr] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (NS == 1)
                vmax = __vmaxu2(vmax, vp[i / 2][i % 2][0]);
#pragma unroll
            for (int gr = 0; gr + 1 < NS; gr += 2)
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
        }
        // a head that left the block out: its maximum and power of two stay and its p are 0
        const bool more0 = act0 && (mx[0] - m[0]) * fac[0] > kSlack, more1 = act1 && (mx[1] - m[1]) * fac[1] > kSlack;
        int vm = (int)(vmax >> 7 & 0xFFu);             // of this lane's scales
        if (__any_sync(0xffffffffu, more0 || more1 || (act0 && vm > ve[0]) || (act1 && vm > ve[1]))) {
            vm = __reduce_max_sync(0xffffffffu, vm);
            const bool over0 = act0 && vm > ve[0], over1 = act1 && vm > ve[1];
            float alpha[2], down[2];
            const int ve_new[2] = {over0 ? vm + kSlackScale : ve[0], over1 ? vm + kSlackScale : ve[1]};
            const float m_new[2] = {more0 ? mx[0] : m[0], more1 ? mx[1] : m[1]};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                alpha[e] = m_new[e] == m[e] ? 1.f : exp2_approx((m[e] - m_new[e]) * fac[e]);
                m[e] = m_new[e];
                down[e] = alpha[e] * (ve[e] - ve_new[e] > -127 ? pow2_field(127 + ve[e] - ve_new[e]) : 0.f);
                ve[e] = ve_new[e];
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][e] *= down[e & 1];
#pragma unroll
            for (int gr = 0; gr < NS; ++gr) {
                zacc[gr][0] *= alpha[0];
                zacc[gr][1] *= alpha[1];
            }
            l[0] *= alpha[0];
            l[1] *= alpha[1];
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        const float up[2] = {scale_up(ve[0]), scale_up(ve[1])};

        // ---- P V
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = exp2_approx(fmaf(s[mt][e] - mu[e & 1], fac[e & 1], -kTop));
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
                pu[e] = p[e] * up[e & 1];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float sa = kv_scale(vp[mt][0][j]), sb = kv_scale(vp[mt][1][j]);
                const float za = fmaf(kMid, sa, kv_zero(vp[mt][0][j])), zb = fmaf(kMid, sb, kv_zero(vp[mt][1][j]));
                uint32_t b0[kParts], b1[kParts];
                split(pu[0] * sa, pu[1] * sa, b0);
                split(pu[2] * sb, pu[3] * sb, b1);
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    b0[k] = movmatrix(b0[k]);
                    b1[k] = movmatrix(b1[k]);
                }
                if (act0)                           // a NaN of V stays out of heads that left the block out
                    zacc[j][0] = fmaf(p[0], za, fmaf(p[2], zb, zacc[j][0]));
                if (act1)
                    zacc[j][1] = fmaf(p[1], za, fmaf(p[3], zb, zacc[j][1]));
#pragma unroll
                for (int gr = j; gr < NG; gr += NS) {
                    if constexpr (BITS == 4) {
                        const unsigned sel = gr & 1 ? 0x7632u : 0x5410u;
                        // lower rows: an element; upper rows: the byte, that element plus 16 times the next
                        const uint32_t x01 = __byte_perm(v0[gr / 2], v1[gr / 2], sel);
                        const uint32_t x23 = __byte_perm(v2[gr / 2], v3[gr / 2], sel);
#pragma unroll
                        for (int i = 0; i < UPG; ++i) {
                            const uint32_t y01 = i ? __byte_perm(x01, 0u, 0x4341) : x01 & 0x00FF00FFu;
                            const uint32_t y23 = i ? __byte_perm(x23, 0u, 0x4341) : x23 & 0x00FF00FFu;
                            const uint32_t n0 = less(y01 & 0x000F000Fu, kMid4), n1 = less(y01, kMidByte);
                            const uint32_t n2 = less(y23 & 0x000F000Fu, kMid4), n3 = less(y23, kMidByte);
#pragma unroll
                            for (int k = 0; k < kParts; ++k)
                                mma16816(acc[gr * UPG + i], n0, n1, n2, n3, b0[k], b1[k]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < UPG; ++i) {
                            const int w = 2 * gr + i / 2;
                            const unsigned sel = i & 1 ? 0x7632u : 0x5410u;
                            const uint32_t x01 = __byte_perm(v0[w], v1[w], sel), x23 = __byte_perm(v2[w], v3[w], sel);
                            const uint32_t n0 = less(__byte_perm(x01, 0u, 0x4240), kMid8), n1 = less(__byte_perm(x01, 0u, 0x4341), kMid8);
                            const uint32_t n2 = less(__byte_perm(x23, 0u, 0x4240), kMid8), n3 = less(__byte_perm(x23, 0u, 0x4341), kMid8);
#pragma unroll
                            for (int k = 0; k < kParts; ++k)
                                mma16816(acc[gr * UPG + i], n0, n1, n2, n3, b0[k], b1[k]);
                        }
                    }
                }
            }
        }
    }

    // over the lanes that share a head: maxima and sums to ml[H], outputs to so[H][D]
    __device__ __forceinline__ void finish(float *so, float2 *ml)
    {
        const int h = 2 * tig & (H - 1), place = 2 * tig / H;                 // first head, which of its places
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    zacc[j][e] += __shfl_xor_sync(0xffffffffu, zacc[j][e], off);
            }
        if (gid == 0 && place == 0) {
            ml[h] = make_float2(m[0] == -INFINITY ? m[0] : fmaf(m[0], fac[0], kTop), l[0]);
            ml[h + 1] = make_float2(m[1] == -INFINITY ? m[1] : fmaf(m[1], fac[1], kTop), l[1]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float un = scale_un(ve[e]);
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < UPG; i += 2) {
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float lo = acc[j * UPG + i + k][e], hi = acc[j * UPG + i + k][e + 2];
#pragma unroll
                        for (int r = 1; r < REP; ++r) {
                            lo = place == r ? acc[(r * NS + j) * UPG + i + k][e] : lo;
                            hi = place == r ? acc[(r * NS + j) * UPG + i + k][e + 2] : hi;
                        }
                        v[2 * k] = lo * kUnit * un + zacc[j][e];
                        v[2 * k + 1] = (BITS == 4 ? (hi - lo) * (kUnit * 0.0625f) : hi * kUnit) * un + zacc[j][e];
                    }
                    const float4 r = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(so + (h + e) * D + F::G * (place * NS + j) + gid * (F::G / 8) + 2 * i) = r;
                }
        }
    }
};

// Nine to sixteen heads: on M, keys or output elements on N.  The codes are the
// same operands (an A of sixteen rows is a B of rows 0 to 7 and one of the
// others), unpacked once for twice the heads, and P leaves the scores as V's A
// operand, so nothing is turned.
template <int BITS, int D>
struct Sums<BITS, D, 16> {
    using F = KvFmt<BITS, D>;
    using Q = QShared<BITS, D, 16>;
    static constexpr int NG = F::NG, R = F::R;
    static constexpr float kMid = BITS == 4 ? 8.f : 128.f;
    static constexpr int KS = D / 16, KW = R / 16, VW = R / 32, UPG = KS / NG;

    float m[2], l[2], zacc[NG][2], acc[KS][2][4], fac[2];
    int ve[2], ve_least;                            // exponent field that V's scales stay within; of all heads
    int lane, gid, tig, t0, t1, at_k, at_z, at_v0, at_v1;

    __device__ __forceinline__ void clear()
    {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void init(const Q &sq, float scale, int lane_)
    {
        lane = lane_;
        gid = lane >> 2;
        tig = lane & 3;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
            fac[hh] = fminf(fmaxf(sq.inv[gid + 8 * hh] * scale, 1.2e-38f), 3e38f);
        clear();
        ve[0] = ve[1] = ve_least = kLeastScale;
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][0][e] = acc[i][1][e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
            zacc[gr][0] = zacc[gr][1] = 0.f;
        const int tr = tile_token(gid);
        t0 = tile_token(2 * tig);
        t1 = tile_token(2 * tig + 1);
        at_k = tr * R + (BITS == 8 && D == 128 ? (tr & 1) * 64 + tig * 16 : tig * (R / 4));
        at_z = F::kParK + tr * F::PAR + Q::par_at(tig, 0);
        at_v0 = F::kCodeV + t0 * R + (gid ^ F::v_swizzle(t0)) * (R / 8);
        at_v1 = F::kCodeV + t1 * R + (gid ^ F::v_swizzle(t1)) * (R / 8);
    }

    __device__ __forceinline__ void step(const uint8_t *h, const Q &sq, unsigned hbits, int keys)
    {
        const uint32_t *q = sq.w[gid] + 4 * tig;
        // ---- raw scores of two 16-token tiles, eight keys each time
        float s[2][2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            const uint8_t *ha = h + at_k + 16 * mt * R;
            uint32_t ka[KW], kb[KW];
            if constexpr (BITS == 8 && D == 128) {  // the other half of the row is 64 bytes up or down
                uint32_t (&a0)[4] = *reinterpret_cast<uint32_t (*)[4]>(ka);
                uint32_t (&a1)[4] = *reinterpret_cast<uint32_t (*)[4]>(ka + 4);
                uint32_t (&b0)[4] = *reinterpret_cast<uint32_t (*)[4]>(kb);
                uint32_t (&b1)[4] = *reinterpret_cast<uint32_t (*)[4]>(kb + 4);
                const uint8_t *hb = ha + (gid >> 1 & 1 ^ gid & 1 ? -64 : 64);
                load_words(a0, ha);
                load_words(a1, hb);
                load_words(b0, ha + 8 * R);
                load_words(b1, hb + 8 * R);
            } else {
                load_words(ka, ha);
                load_words(kb, ha + 8 * R);
            }
#pragma unroll
            for (int st = 0; st < Q::STEPS; ++st) { // z sum(q) of the groups, the params as they lie
                const uint4 x = *reinterpret_cast<const uint4 *>(sq.w[gid] + Q::kSum + (tig * Q::STEPS + st) * 4);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    uint32_t w[2];
                    const uint8_t *at = h + at_z + (16 * mt + 8 * nt) * F::PAR;
                    if constexpr (NG == 1)
                        w[0] = w[1] = *reinterpret_cast<const uint32_t *>(at);
                    else
                        load_words(w, at);
                    if (st == 0)
                        mma16816_0(s[mt][nt], x.x, x.y, x.z, x.w, w[0], w[1]);
                    else
                        mma16816(s[mt][nt], x.x, x.y, x.z, x.w, w[0], w[1]);
                }
            }
            uint32_t par[4][NG];                    // of this lane's keys 2 tig, 2 tig + 1 and 8 further
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_words(par[i], h + F::kParK + (16 * mt + (i & 1 ? t1 : t0) + (i >> 1) * 8) * F::PAR);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                float c[2][4];
#pragma unroll
                for (int i = 0; i < UPG; ++i) {
                    const int ks = gr * UPG + i;
                    uint32_t x[4];
                    const uint4 qk = *reinterpret_cast<const uint4 *>(q + 16 * ks);
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
                    if (i == 0) {
                        mma16816_0(c[0], qk.x, qk.y, qk.z, qk.w, x[0], x[2]);
                        mma16816_0(c[1], qk.x, qk.y, qk.z, qk.w, x[1], x[3]);
                    } else {
                        mma16816(c[0], qk.x, qk.y, qk.z, qk.w, x[0], x[2]);
                        mma16816(c[1], qk.x, qk.y, qk.z, qk.w, x[1], x[3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float sa = kv_scale(par[2 * nt][gr]), sb = kv_scale(par[2 * nt + 1][gr]);
                    s[mt][nt][0] = fmaf(sa, c[nt][0], s[mt][nt][0]);
                    s[mt][nt][1] = fmaf(sb, c[nt][1], s[mt][nt][1]);
                    s[mt][nt][2] = fmaf(sa, c[nt][2], s[mt][nt][2]);
                    s[mt][nt][3] = fmaf(sb, c[nt][3], s[mt][nt][3]);
                }
            }
        }
        const bool all_heads = hbits == 0xffffffffu;
        const bool act0 = hbits >> gid & 1u, act1 = hbits >> (gid + 8) & 1u;
        if (keys < 32) {                            // the sequence's last tokens
            __syncwarp();                           // (keeps this a branch)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * i + (e & 1 ? t1 : t0) >= keys)
                        s[i / 2][i % 2][e] = -INFINITY;
        }

        // ---- the power of two for p s (a token a lane), the maxima
        uint32_t vmax = 0;
        {
            uint32_t w[NG];
            load_words(w, h + F::kParV + lane * F::PAR);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
                vmax = __vmaxu2(vmax, w[gr]);
            vmax = lane < keys ? vmax : 0u;
        }
        float mx[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            mx[hh] = fmaxf(s[0][0][2 * hh], s[0][0][2 * hh + 1]);
#pragma unroll
            for (int i = 1; i < 4; ++i)
                mx[hh] = fmaxf(mx[hh], fmaxf(s[i / 2][i % 2][2 * hh], s[i / 2][i % 2][2 * hh + 1]));
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
        }
        // a head that left the block out: its maximum and power of two stay and its p are 0
        const bool more0 = act0 && (mx[0] - m[0]) * fac[0] > kSlack, more1 = act1 && (mx[1] - m[1]) * fac[1] > kSlack;
        int vm = (int)(vmax >> 7 & 0xFFu);             // of this lane's token
        if (__any_sync(0xffffffffu, more0 || more1 || vm > ve_least)) {
            vm = __reduce_max_sync(0xffffffffu, vm);
            const bool over0 = act0 && vm > ve[0], over1 = act1 && vm > ve[1];
            float alpha[2], down[2];
            const int ve_new[2] = {over0 ? vm + kSlackScale : ve[0], over1 ? vm + kSlackScale : ve[1]};
            const float m_new[2] = {more0 ? mx[0] : m[0], more1 ? mx[1] : m[1]};
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                alpha[hh] = m_new[hh] == m[hh] ? 1.f : exp2_approx((m[hh] - m_new[hh]) * fac[hh]);
                m[hh] = m_new[hh];
                down[hh] = alpha[hh] * (ve[hh] - ve_new[hh] > -127 ? pow2_field(127 + ve[hh] - ve_new[hh]) : 0.f);
                ve[hh] = ve_new[hh];
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[i][0][e] *= down[e >> 1];
                    acc[i][1][e] *= down[e >> 1];
                }
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                zacc[gr][0] *= alpha[0];
                zacc[gr][1] *= alpha[1];
            }
            l[0] *= alpha[0];
            l[1] *= alpha[1];
            ve_least = __reduce_min_sync(0xffffffffu, min(ve[0], ve[1]));
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        const float up[2] = {scale_up(ve[0]), scale_up(ve[1])};

        // ---- P V
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float p[2][4], pu[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[nt][e] = exp2_approx(fmaf(s[mt][nt][e] - mu[e >> 1], fac[e >> 1], -kTop));
                if (!all_heads) {
                    p[nt][0] = act0 ? p[nt][0] : 0.f;
                    p[nt][1] = act0 ? p[nt][1] : 0.f;
                    p[nt][2] = act1 ? p[nt][2] : 0.f;
                    p[nt][3] = act1 ? p[nt][3] : 0.f;
                }
                l[0] += p[nt][0] + p[nt][1];
                l[1] += p[nt][2] + p[nt][3];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    pu[nt][e] = p[nt][e] * up[e >> 1];
            }
            uint32_t par[4][NG], v0[VW], v1[VW], v2[VW], v3[VW];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_words(par[i], h + F::kParV + (16 * mt + (i & 1 ? t1 : t0) + (i >> 1) * 8) * F::PAR);
            if (keys < 32) {                        // zero behind the length
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
                        if (16 * mt + (i & 1 ? t1 : t0) + (i >> 1) * 8 >= keys)
                            par[i][gr] = 0u;
            }
            load_words(v0, h + at_v0 + 16 * mt * R);
            load_words(v1, h + at_v1 + 16 * mt * R);
            load_words(v2, h + at_v0 + (16 * mt + 8) * R);
            load_words(v3, h + at_v1 + (16 * mt + 8) * R);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                uint32_t a[4][kParts];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float sa = kv_scale(par[2 * nt][gr]), sb = kv_scale(par[2 * nt + 1][gr]);
                    const float za = fmaf(kMid, sa, kv_zero(par[2 * nt][gr])), zb = fmaf(kMid, sb, kv_zero(par[2 * nt + 1][gr]));
                    split(pu[nt][0] * sa, pu[nt][1] * sb, a[2 * nt]);
                    split(pu[nt][2] * sa, pu[nt][3] * sb, a[2 * nt + 1]);
                    if (act0)                       // a NaN of V stays out of heads that left the block out
                        zacc[gr][0] = fmaf(p[nt][0], za, fmaf(p[nt][1], zb, zacc[gr][0]));
                    if (act1)
                        zacc[gr][1] = fmaf(p[nt][2], za, fmaf(p[nt][3], zb, zacc[gr][1]));
                }
                if constexpr (BITS == 4) {
                    const unsigned sel = gr & 1 ? 0x7632u : 0x5410u;
                    // an element; and the byte, that element plus 16 times the next
                    const uint32_t x01 = __byte_perm(v0[gr / 2], v1[gr / 2], sel), x23 = __byte_perm(v2[gr / 2], v3[gr / 2], sel);
#pragma unroll
                    for (int i = 0; i < UPG; ++i) {
                        const uint32_t y01 = i ? __byte_perm(x01, 0u, 0x4341) : x01 & 0x00FF00FFu;
                        const uint32_t y23 = i ? __byte_perm(x23, 0u, 0x4341) : x23 & 0x00FF00FFu;
                        const uint32_t n0 = less(y01 & 0x000F000Fu, kMid4), n1 = less(y01, kMidByte);
                        const uint32_t n2 = less(y23 & 0x000F000Fu, kMid4), n3 = less(y23, kMidByte);
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            mma16816(acc[gr * UPG + i][0], a[0][k], a[1][k], a[2][k], a[3][k], n0, n2);
                            mma16816(acc[gr * UPG + i][1], a[0][k], a[1][k], a[2][k], a[3][k], n1, n3);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < UPG; ++i) {
                        const int w = 2 * gr + i / 2;
                        const unsigned sel = i & 1 ? 0x7632u : 0x5410u;
                        const uint32_t x01 = __byte_perm(v0[w], v1[w], sel), x23 = __byte_perm(v2[w], v3[w], sel);
                        const uint32_t n0 = less(__byte_perm(x01, 0u, 0x4240), kMid8), n1 = less(__byte_perm(x01, 0u, 0x4341), kMid8);
                        const uint32_t n2 = less(__byte_perm(x23, 0u, 0x4240), kMid8), n3 = less(__byte_perm(x23, 0u, 0x4341), kMid8);
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            mma16816(acc[gr * UPG + i][0], a[0][k], a[1][k], a[2][k], a[3][k], n0, n2);
                            mma16816(acc[gr * UPG + i][1], a[0][k], a[1][k], a[2][k], a[3][k], n1, n3);
                        }
                    }
                }
            }
        }
    }

    // over the lanes that share a head: maxima and sums to ml[16], outputs to so[16][D]
    __device__ __forceinline__ void finish(float *so, float2 *ml)
    {
#pragma unroll
        for (int off = 1; off < 4; off <<= 1)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], off);
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
                    zacc[gr][hh] += __shfl_xor_sync(0xffffffffu, zacc[gr][hh], off);
            }
        if (tig == 0) {
            ml[gid] = make_float2(m[0] == -INFINITY ? m[0] : fmaf(m[0], fac[0], kTop), l[0]);
            ml[gid + 8] = make_float2(m[1] == -INFINITY ? m[1] : fmaf(m[1], fac[1], kTop), l[1]);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const float un = scale_un(ve[hh]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                    for (int i = 0; i < UPG; i += 2) {
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float lo = acc[gr * UPG + i + k][0][2 * hh + e], hi = acc[gr * UPG + i + k][1][2 * hh + e];
                            v[2 * k] = lo * kUnit * un + zacc[gr][hh];
                            v[2 * k + 1] = (BITS == 4 ? (hi - lo) * (kUnit * 0.0625f) : hi * kUnit) * un + zacc[gr][hh];
                        }
                        *reinterpret_cast<float4 *>(so + (gid + 8 * hh) * D + F::G * gr + (2 * tig + e) * (F::G / 8) + 2 * i) =
                            make_float4(v[0], v[1], v[2], v[3]);
                    }
        }
    }
};

template <int BITS, int D, int H, int P>
__global__ void __launch_bounds__(DecodeCfg<BITS, D, H, P>::W * 32, P) decode_quant_kernel(const DecodeArgs a)
{
    using F = KvFmt<BITS, D>;
    using C = DecodeCfg<BITS, D, H, P>;
    constexpr int W = C::W, ST = C::ST;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t s_bar[W * ST];
    __shared__ float2 s_ml[W][H], s_sum[H];
    __shared__ uint32_t s_words[kMaxNb / 32];
    __shared__ uint32_t s_rec[kListMax];            // a block's record from the start of the pages, in 512 bytes
    __shared__ uint16_t s_block[kListMax];
    __shared__ __align__(16) QShared<BITS, D, H> s_q;

    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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

    // ---- q, a warp per head (0 where there is none), its loads in flight together
    {
        typename QShared<BITS, D, H>::Raw raw[(H + W - 1) / W];
#pragma unroll
        for (int i = 0; i < (H + W - 1) / W; ++i) {
            const int h = warp + i * W;
            QShared<BITS, D, H>::fetch(raw[i], h < gt ? a.q_tok + ((long long)b * a.Hq + h0 + h) * D : nullptr, lane);
        }
#pragma unroll
        for (int i = 0; i < (H + W - 1) / W; ++i)
            if (warp + i * W < H)
                s_q.prepare(raw[i], warp + i * W, lane);
    }

    // ---- union of the heads' active blocks, one bit each.  Rows short enough for
    // one round of kMaskWords words of 32 blocks a warp: a block a lane, and its
    // table entry, all loads in flight together (and before the length is known).
    // Longer rows: four blocks a lane, where the rows' alignment allows it, and
    // the table is looked up for this split's blocks alone.
    constexpr int kMaskWords = H == 16 && W < 8 ? 4 : (31 + W) / W;
    const int nblk = (len + 63) / 64, nwords = (nblk + 31) / 32;
    const bool one_round = a.nb <= 32 * kMaskWords * W;
    int page[kMaskWords];
    if (one_round || a.nb % 4 != 0 || (reinterpret_cast<uintptr_t>(a.mask) & 3) != 0) {
        for (int c0 = warp; c0 < (c0 == warp ? (a.nb + 31) / 32 : nwords); c0 += kMaskWords * W) {
            int raw[kMaskWords][H];
            // (blocks past the row read its last one: the branches are the warp's)
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i) {
                if (i > 0 && (c0 + i * W) * 32 >= a.nb)
                    continue;
                const int j = min((c0 + i * W) * 32 + lane, a.nb - 1);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    raw[i][h] = 0;
                    if (h < gt)
                        raw[i][h] = load(mrow + (long long)h * a.nb + j);
                }
                if (one_round) {
                    page[i] = b * a.kv.max_blocks + j;
                    if (a.kv.table != nullptr)
                        page[i] = load(a.kv.table + page[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i) {
                const int c = c0 + i * W;
                if (c >= nwords)
                    continue;
                int any = 0;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    any |= raw[i][h];
                const unsigned bits = __ballot_sync(0xffffffffu, any != 0 && c * 32 + lane < nblk);
                if (lane == 0)
                    s_words[c] = bits;
            }
        }
    } else {
        for (int c0 = warp; c0 * 4 < nwords; c0 += 4 * W) {
            uint32_t raw[4][H];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = min((c0 + i * W) * 128 + 4 * lane, a.nb - 4);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    raw[i][h] = 0;
                    if (h < gt)
                        raw[i][h] = load(reinterpret_cast<const uint32_t *>(mrow + (long long)h * a.nb + j));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = (c0 + i * W) * 128 + 4 * lane;
                uint32_t x = 0;
#pragma unroll
                for (int h = 0; h < H; ++h)
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
                entry(i, j, a.kv.table != nullptr ? load(a.kv.table + at) : at);
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
        return u < n_units && lane < gt ? (int)load(mrow + (long long)lane * a.nb + (s_block[u >> 1] & (kNoPage - 1))) : 0;
    };
    if (lane == 0)
        for (int s = 0; s < ST; ++s)
            issue(warp + s * W, s);

    Sums<BITS, D, H> sums;
    sums.init(s_q, a.scale_log2 * 16777216.f, lane);

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
                sums.clear();
                break;
            }
        }
        sums.step(my + st * F::HALF, s_q, hbits, keys);
        __syncwarp();
        if (lane == 0)
            issue(u + ST * W, st);
    }

    // ---- sums over the lanes that share a head, then over the warps
    __syncwarp();
    sums.finish(reinterpret_cast<float *>(my), s_ml[warp]);              // over this warp's ring
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
// (1024 heads of two splits: 90 us a call, 96 with four; both with an earlier loop).
template <int D, int Q>
__global__ void __launch_bounds__(Q * D) decode_quant_merge_kernel(const DecodeArgs a)
{
    constexpr int N = Q == 4 ? kMaxDecodeSplits / 4 : 8;
    __shared__ float s_w[kMaxDecodeSplits], s_part[Q][D];
    wait_for_previous_kernel();
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

// How a call is cut up: heads and CTAs of an SM, and the estimated time.
struct Plan {
    int H, P;
    double us;
};

// Estimated time, in us, of `ctas` CTAs with `blocks` blocks each:
//                                     to eight heads   sixteen
//   one CTA per SM (P = 1)            7.2              9.2     start and end
//                                     0.3              0.46    a block
//   two (P = 2)                       7.5              9.5     start and end, per wave
//                                     0.31             0.46    a block, of the SM
//   two, but no more CTAs than SMs    6                8
//                                     0.4              0.65
//   the second kernel                 2 and 0.04 a split
// The constants are of the loop with p s in one part, 4 bits, D = 128 and eight columns
// of heads, and order the plans: with two parts a block takes up to a fifth more, of every
// plan.  Measured now, groups of four, D = 128, 8 units (a sequence's head tile) of 512
// blocks, 4 | 8 bits, all active: P = 1, 9 splits 25.9 | 24.7 us, 12: 21.8 | 21.5, 18:
// 19.2 | 20.6; P = 2, 18: 20.6 | 22.2, 37: 18.3 | 21.4; a tenth active: P = 1, 9: 14.4 |
// 14.4, 18: 13.0 | 13.6; P = 2, 18: 12.9 | 14.4, 37: 13.2 | 13.8.  At D = 64, all active: P = 1,
// 18: 14.4 | 15.3; P = 2, 18: 15.1 | 15.6, 37: 13.8 | 14.9.  128 units of 256, P = 2: 1 split
// 111 | 121 us, 2: 93 | 94, 4: 96 | 98.  Sixteen heads, 64 units of 256 blocks, P = 2: 1 split
// 198 | 176 us, 2: 107 | 97, 4: 84 | 75; of 64 blocks: 56 | 50, 35 | 40, 30 | 29.  What is chosen is
// within 5 % of the best of these, but for sixteen heads on sparse masks (below).
double decode_quant_us(const Plan &p, long long ctas, double blocks, double splits, int sms)
{
    const bool two = p.H == 16;
    const long long load = (ctas + sms - 1) / sms, waves = (load + 1) / 2;
    const double merge = splits > 1.0 ? 2.0 + 0.04 * splits : 0.0;
    if (p.P == 1)
        return load > 1 ? 1e30 : (two ? 9.2 : 7.2) + (two ? 0.46 : 0.3) * blocks + merge;
    if (load == 1)
        return (two ? 8.0 : 6.0) + (two ? 0.65 : 0.4) * blocks + merge;
    return (two ? 9.5 : 7.5) * (double)waves + (two ? 0.46 : 0.31) * (double)load * blocks + merge;
}

// The splits (nsplit, slots) of a plan: the least estimated time with half of the
// blocks active (the mask is on the device) and at least a block for every
// second warp.  Lengths given: a CTA for each place on the SMs, where there are
// enough for every sequence's tiles, shared out by length: a batch of 8 from 32k
// tokens down takes 52 us with 4 splits each, 43 so.  Not for two or three
// sequences, whose CTAs pair up on the SMs (64k and 37k tokens at 8 bits: 44 us with
// 18 splits each, 50 in 18 slots, 43 in 37, 45 with one CTA per SM), and in whole splits where
// a sequence has few (16 of 16k tokens, an earlier loop: 88 us with two each, 90 with 37
// slots).
void decode_quant_split(DecodeArgs &a, Plan &p, int sms)
{
    const int g = a.Hq / a.Hkv;
    a.tiles = (g + p.H - 1) / p.H;
    a.per_tile = (g + a.tiles - 1) / a.tiles;
    const int tiles = a.Hkv * a.tiles;
    const int lo = (a.nb + kListMax - 2) / (kListMax - 1);            // a split's block list has to fit
    const int cap = a.nb / 4 < kMaxDecodeSplits ? a.nb / 4 : kMaxDecodeSplits;
    a.nsplit = lo;
    a.slots = 0;
    p.us = decode_quant_us(p, (long long)a.B * tiles * lo, 0.5 * a.nb / lo, lo, sms);
    for (int ns = lo + 1; ns <= cap; ++ns) {
        const double us = decode_quant_us(p, (long long)a.B * tiles * ns, 0.5 * a.nb / ns, ns, sms);
        if (us < p.us) {
            p.us = us;
            a.nsplit = ns;
        }
    }
    if (a.lens == nullptr || a.B == 1 || a.B > kBalanced)
        return;
    if (a.B < 4) {
        if (p.P == 1)
            p.us = 1e30;
        return;
    }
    for (int load = 1; load <= p.P; ++load) {
        int slots = load * sms / tiles;
        if (slots < 4 * a.B)
            slots -= slots % a.B;
        // a sequence's share of slots - B is at least that of its blocks in B * nb
        if (slots < a.B * (1 + lo) || slots > a.B * (1 + cap))
            continue;
        const double each = (double)slots / a.B;
        const double us = decode_quant_us(p, (long long)slots * tiles, 0.5 * a.nb / each, each, sms);
        if (a.slots == 0 || us < p.us) {
            p.us = us;
            a.slots = slots;
        }
    }
}

template <int BITS, int D, int H, int P>
cudaError_t launch(const DecodeArgs &a, cudaStream_t stream)
{
    using C = DecodeCfg<BITS, D, H, P>;
    cudaError_t e = cudaFuncSetAttribute(decode_quant_kernel<BITS, D, H, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::ring);
    if (e != cudaSuccess)
        return e;
    const dim3 grid(a.slots > 0 ? a.slots : a.nsplit, a.Hkv * a.tiles, a.slots > 0 ? 1 : a.B);
    e = launch_programmatic(decode_quant_kernel<BITS, D, H, P>, grid, C::W * 32, C::ring, stream, a);
    if (e != cudaSuccess || (a.slots == 0 && a.nsplit == 1))
        return e;
    if ((a.slots > 0 ? a.slots / a.B : a.nsplit) > 8)
        return launch_programmatic(decode_quant_merge_kernel<D, 4>, dim3(a.B * a.Hq), 4 * D, 0, stream, a);
    return launch_programmatic(decode_quant_merge_kernel<D, 1>, dim3(a.B * a.Hq), D, 0, stream, a);
}

using Launch = cudaError_t (*)(const DecodeArgs &, cudaStream_t);

template <int BITS, int D>
Launch kernel_of(const Plan &p)
{
    if constexpr (KvFmt<BITS, D>::NG == 4)
        if (p.H == 2)
            return p.P == 1 ? launch<BITS, D, 2, 1> : launch<BITS, D, 2, 2>;
    if constexpr (KvFmt<BITS, D>::NG > 1)
        if (p.H == 4)
            return p.P == 1 ? launch<BITS, D, 4, 1> : launch<BITS, D, 4, 2>;
    if (p.H == 16)
        return p.P == 1 ? launch<BITS, D, 16, 1> : launch<BITS, D, 16, 2>;
    return p.P == 1 ? launch<BITS, D, 8, 1> : launch<BITS, D, 8, 2>;
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
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    // Two, four or eight heads a CTA by the heads of a KV head or, for more, sixteen, and one CTA per SM or two of
    // half the warps: what is estimated fastest.  Sixteen for enough blocks (groups of
    // 16, 64 units of 256 blocks, all active: 84 us, 103 by eights; a tenth active, where
    // the union of sixteen heads is larger: 75 and 69), one CTA for one round of long
    // ones (decode_quant_us).
    Plan best{};
    DecodeArgs args = a;
    const int g = Hq / Hkv, groups = d / (bits == 4 ? 32 : 64);
    const int least = g <= 2 && groups == 4 ? 2 : g <= 4 && groups > 1 ? 4 : 8;
    for (int H = least; H <= (g > 8 ? 16 : least); H += H)
        for (int P = 1; P <= 2; ++P) {
            Plan p{H, P, 0.0};
            decode_quant_split(a, p, sms);
            if (best.H == 0 || p.us < best.us) {
                best = p;
                args = a;
            }
        }
    const Launch f = bits == 4 ? (d == 128 ? kernel_of<4, 128>(best) : kernel_of<4, 64>(best))
                               : (d == 128 ? kernel_of<8, 128>(best) : kernel_of<8, 64>(best));
    return f(args, stream);
}

} // namespace seer

// Attention of ragged chunks over a batch's paged TQ3 cache on the tensor cores (tcgen05), for sequences
// with many rows per KV head. Same operation, identities and cutting of the work as tq3_chunk.cu; here a
// segment has NB x 128 rows and a tile of 128 keys is two products per 128 rows:
//     S = Q~ K^T       (128 rows x 128 keys, K = 128 rotated coordinates; both operands in shared memory)
//     O += P V         (128 rows x 128 coordinates, K = 128 keys; P in tensor memory, V in shared memory)
// with K's row j = c[idx_j] f_j coef 2^13 / F and V's row j = c[idx'_j] g_j 2^13 / G in fp16, F the power of
// two at the tile's largest f_j coef, and each row of q~ scaled by a power of two to 2^7 .. 2^8: one factor per
// row and tile leads from S to the logit in log2 units, and it rides on the subtraction of the maximum. G follows
// the largest g_j of the tiles so far and is raised when one is passed by 4 (O is rescaled then). The least
// centroid, 0.1129, leaves fp16's normal range where its factor is 2^-23 of F or G; below that a coordinate is
// off by 2^-25, which moves a logit by 2^-34 softmax_scale |q| |k| at most, k the longest key of the tile, and the
// result by 2^-34 of the longest value (the low halves of split operands reach that from 2^-12 on). Weights are
// off by 2^-31 of the row's largest at most. A value whose factor is not finite becomes zero and poisons its
// key's logits instead: a row that sees it gets NaN, any other is not touched.
//
// One CTA of 20 warps per SM. Warps 0-3 and 4-7 are the softmax of rows 0-127 and 128-255: a thread a row,
// which lies in its tensor-memory lane. Warps 8-11 decode keys and 12-15 values: a thread a record. Warps 16
// and 17 issue the products of a block each; 18 and 19 fill their warpgroup.
//     decode   the eight centroids times the record's factor as a table of two bytes each; indices to the
//              selectors of byte permutes, which fetch the bytes of four operands at a time; 16-byte
//              chunks into the 128-byte-swizzled operand tile (K as K-major B, V as MN-major B)
//     softmax  the maximum of a row of S; M is raised where it is passed by 2^8 (O is rescaled then);
//              w = 2^(s - M), P as fp16 over S's columns that have been read
//     issue    of a block, with a and b the two 64-key halves of a tile:
//              S(0a) S(0b) | P(0a) V(0a) -> O, S(1a) | P(0b) V(0b) -> O, S(1b) | ...
// so that the softmax of one half runs while the tensor core works on the other, and the two blocks of rows
// share it. Products run in the order of their issue: S(i+1 a) may overwrite P(i a), which lies over S(i a).
// For fp32 queries or results the operands are split hi + lo, a product takes three passes (hi hi, hi lo,
// lo hi), and 128 rows and one stage of operands fill the shared memory.
//
// Measured, with the join: 2048 tokens over 16384 keys, 8 KV heads x 4 rows a token, bf16: 594 us at 1965 MHz, 866
// TFLOP/s, about half of what a library product reaches (642 us where the power cap holds 1815 MHz); with fp32 on
// either side 2.04 ms. A tile and 256 rows more take some 4500 cycles (from 6144 to 16384 keys), 5200 with the
// segments' set-ups and ends, of which the products need 2200 and the exponentials (MUFU) 2050; the softmax of a
// half tile takes 2500 to 3000, half of it waits for tensor memory and barriers, with 62% of the issue slots busy.
// 256 rows a CTA because each decoded
// operand then serves two products; with halves of 64 keys a block's softmax and its products overlap (697 us
// without). Loops are rolled where they can be: code that runs once a segment is fetched anew each time, and at
// 170 KB the kernel took 1220 us.
//
// Every wait is bounded; one that runs out sets fault bit 7 and ends its role's part of the segment. The others
// finish theirs or run out after it, and all leave together at the segment's end, before anything is written over
// its operands. Whatever ends a CTA, the warps that issued products wait for them (again with a limit) before the
// tensor memory is freed.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <cuda_fp16.h>

#include "common.cuh"
#include "tcgen05.cuh"
#include "tq3_cache.cuh"
#include "tq3_chunk.cuh"
#include "tq3_common.cuh"

namespace wq {
namespace tq3_chunk_mma {

using namespace tq3_chunk;

constexpr int kBlock = 128;           // rows of a product
constexpr int kThreads = 640;
// registers a thread: 96 at launch; 256 softmax, 256 decode and 128 issue threads share the same 61440
constexpr int kRegsSoftmax = 152, kRegsDecode = 72, kRegsIssue = 32;
static_assert(256 * kRegsSoftmax + 256 * kRegsDecode + 128 * kRegsIssue <= kThreads * 96, "registers");
constexpr int kIssueWarp = 16;
constexpr int kBox = 128 * 128;       // 64 coordinates of a 128-row fp16 operand, in bytes
constexpr int kOp = 2 * kBox;
constexpr uint32_t kMaxPolls = 1u << 24;
constexpr float kLazy = 8.0f, kLift = 6.0f;  // as in tq3_chunk.cu
constexpr int kRecBytes = kTileKeys * tq3_cache::kRec;  // a tile's records of one pool
constexpr int kRecStages = 2;
constexpr int kQBits = 7;             // the largest |q~| of a row is scaled to 2^7 .. 2^8
// A key of factor F has this one, and a value of factor G: factors are below 4 of those, so operands below 2^15.
constexpr float kTop = 8192.0f;

// fp16 operands, fp32 accumulator, M = 128; N = 64 keys, and N = 128 coordinates with an MN-major B.
constexpr uint32_t kIdescS = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

__device__ unsigned int g_fault;

template <bool kWide>
struct Cfg {
    static constexpr int NB = kWide ? 1 : 2;      // blocks of 128 rows
    static constexpr int KS = kWide ? 1 : 2;      // stages of K and of V
    static constexpr int kParts = kWide ? 2 : 1;  // hi (and lo)
    static constexpr int R = NB * kBlock;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + NB * kParts * kOp;
    static constexpr int kOffV = kOffK + KS * kParts * kOp;
    static constexpr int kOffRec = kOffV + KS * kParts * kOp;  // per stage: a tile's key and value records
    static constexpr int kOffFac = kOffRec + kRecStages * 2 * kRecBytes;  // per stage and key: norm, scale of the value
    static constexpr int kOffShared = kOffFac + kRecStages * kTileKeys * 8;
    static constexpr int kSmem = 1024 + kOffShared + 1280;
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    // tensor memory: S, O, and P (over S where two blocks fill the memory)
    static constexpr int kTmemO = NB * 128, kTmemP = kWide ? 256 : 0;
};

struct Tile {          // of a stage
    float ratio, G;    // G before / G, and G
    uint32_t valid[4]; // keys that have a page
};
struct Shared {
    uint64_t full_k[2], full_v[2], free_k[2], free_v[2], q_ready, drain[2];
    uint64_t s_done[2][2], p_ready[2][2], pv_done[2], o_done[2];  // per block (and half of a tile)
    Tile tile[2];
    // what a unit of K stands for, of the last four tiles: keys are decoded up to KS tiles ahead of the one
    // whose S is complete, and a softmax warp may be a tile behind that
    float unit[4];
    uint32_t tmem;
    uint32_t dead;  // a wait has run out
    uint32_t most[2][2][4];  // per tile (alternately), pool and decoding warp: the largest factor
    int64_t scratch[kThreads / 32 + 4];
    Walk<256, kThreads> walk256;
    Walk<128, kThreads> walk128;
};
static_assert(sizeof(Shared) <= 1280, "shared block");
template <bool kWide>
__device__ __forceinline__ Walk<Cfg<kWide>::R, kThreads> &walk_of(Shared &s);
template <>
__device__ __forceinline__ Walk<256, kThreads> &walk_of<false>(Shared &s) { return s.walk256; }
template <>
__device__ __forceinline__ Walk<128, kThreads> &walk_of<true>(Shared &s) { return s.walk128; }

__device__ __forceinline__ uint32_t h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 f2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Operand descriptors as their low words (address, leading offset); the high word is the same for both:
// the next 8 rows 1024 bytes further, version 1, 128-byte swizzle. K-major ignores the leading offset; for
// the same tile as an MN-major operand (its rows are K) it is the step to the next 64 elements, a box.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t k_desc(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t mn_desc(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | (uint32_t)(kBox >> 4) << 16; }
// D[tmem] (+)= A B^T, A and B in shared memory; and with A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}
// Writes 16 consecutive tensor-memory columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Waits for a phase for kWaitLimitNs at most. A poll may suspend the thread for up to kPollNs, so that
// waiting warps leave the issue slots to the others; the clock, which is slow to read, only bounds waits
// whose first polls have failed.
constexpr uint32_t kPollNs = 100000;
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t phase) {
    const uint32_t at = smem_u32(bar);
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 0; it < kMaxPolls; ++it) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok)
                     : "r"(at), "r"(phase), "r"(kPollNs)
                     : "memory");
        if (ok) return true;
        if ((it & 63) == 63) {
            if (t0 == 0)
                t0 = global_ns();
            else if (global_ns() - t0 > kWaitLimitNs)
                return false;
        }
    }
    return false;
}
// The whole warp waits; false sets the fault bit.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase) {
    const bool ok = __all_sync(0xffffffffu, wait_bar(bar, phase));
    if (!ok && (threadIdx.x & 31) == 0) atomicOr(&g_fault, 128u);
    return ok;
}

template <int kBar, int kCount>
__device__ __forceinline__ void named_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(kBar), "n"(kCount) : "memory");
}

// The eight centroids times a factor, rounded to fp16: their low and their high bytes, in two words each.
// Magnitudes 0 .. 3 are indices 4 .. 7 and, negative, 3 .. 0.
struct Table {
    uint32_t lo0, lo1, hi0, hi1;
};
__device__ __forceinline__ Table make_table(uint32_t m01, uint32_t m23) {
    Table t;
    t.lo1 = __byte_perm(m01, m23, 0x6420);
    t.hi1 = __byte_perm(m01, m23, 0x7531);
    t.lo0 = __byte_perm(m01, m23, 0x0246);
    t.hi0 = __byte_perm(m01, m23, 0x1357) ^ 0x80808080u;
    return t;
}
__device__ __forceinline__ void four(const Table &t, uint32_t sel, uint32_t &a, uint32_t &b) {
    const uint32_t lo = __byte_perm(t.lo0, t.lo1, sel), hi = __byte_perm(t.hi0, t.hi1, sel);
    a = __byte_perm(lo, hi, 0x5140);
    b = __byte_perm(lo, hi, 0x7362);
}
// Eight 3-bit indices (the low 24 bits of x) to eight selector nibbles.
__device__ __forceinline__ uint32_t nibbles(uint32_t x) {
    uint32_t y = (x & 0xFFFu) + (x & 0xFFF000u) * 16u;
    y += (y & 0x0FC00FC0u) * 3u;
    return y + (y & 0x38383838u);
}

// The 128 centroids of a record's indices times a factor, into row `row` of an operand, 32 at a time (the
// loop is kept small: the roles' loops share the instruction cache).
template <bool kWide>
__device__ __forceinline__ void expand(unsigned char *op, int row, const uint32_t *rec, float factor) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __fmul_rn(tq3::centroid(4 + i), factor);
    const uint32_t m01 = h2(m[0], m[1]), m23 = h2(m[2], m[3]);
    const Table th = make_table(m01, m23);
    Table tl = {};
    if (kWide)
        tl = make_table(h2(__fsub_rn(m[0], f2(m01).x), __fsub_rn(m[1], f2(m01).y)),
                        h2(__fsub_rn(m[2], f2(m23).x), __fsub_rn(m[3], f2(m23).y)));
#pragma unroll 1
    for (int part = 0; part < 4; ++part) {
        const uint32_t w0 = rec[3 * part], w1 = rec[3 * part + 1], w2 = rec[3 * part + 2];
        // chunk (4 (part & 1) + c) ^ (row & 7), its two low bits apart
        unsigned char *const to = op + (part >> 1) * kBox + row * 128 + (((part & 1) << 6) ^ ((row & 4) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t x = c == 0 ? w0 : c == 1 ? __funnelshift_r(w0, w1, 24) : c == 2 ? __funnelshift_r(w1, w2, 16) : w2 >> 8;
            const uint32_t sel = nibbles(x);
            unsigned char *const chunk = to + ((c ^ (row & 3)) << 4);
            uint4 h;
            four(th, sel, h.x, h.y);
            four(th, sel >> 16, h.z, h.w);
            *reinterpret_cast<uint4 *>(chunk) = h;
            if (kWide) {
                four(tl, sel, h.x, h.y);
                four(tl, sel >> 16, h.z, h.w);
                *reinterpret_cast<uint4 *>(chunk + kOp) = h;
            }
        }
    }
}

// Keys 32 c .. 32 c + 31 of a tile that a row at `pos` sees, as bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t visible(const Args &a, int pos, int j) {
    const int d = pos - j;
    if (d < 0) return 0u;
    uint32_t m = below(d + 1);
    if (a.window) m &= ~below(d - (a.window - 1)) | below(a.sinks - j);
    return m;
}

__device__ __forceinline__ float max32(float m, const float (&x)[32]) {
    float n = x[0];
#pragma unroll
    for (int k = 0; k < 32; k += 4) m = max3(m, x[k], x[k + 1]), n = max3(n, x[k + 2], x[k + 3]);
    return fmaxf(m, n);
}
// w = 2^(S U - M) of 32 columns of S, their sums, and P (hi, and lo behind it) to tensor memory.
template <bool kWide>
__device__ __forceinline__ void weights(const float (&x)[32], f32x2 U2, f32x2 M2, f32x2 (&ps)[2], uint32_t tP) {
    uint32_t p[16], l[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float d0, d1;
        upk2(fma2(pk2(x[2 * k], x[2 * k + 1]), U2, M2), d0, d1);
        d0 = ex2(d0), d1 = ex2(d1);
        ps[k & 1] = add2(ps[k & 1], pk2(d0, d1));
        p[k] = h2(d0, d1);
        if (kWide) l[k] = h2(__fsub_rn(d0, f2(p[k]).x), __fsub_rn(d1, f2(p[k]).y));
    }
    tmem_st16(tP, p);
    if (kWide) tmem_st16(tP + 16, l);
}

// What every role knows of a segment.
template <bool kWide>
struct Segment {
    Seq s;
    Span span;
    int rows, r0, before, take, first, p_hi, nb, b, head;
    bool blind, whole;  // no row sees a key; all of the segment's tiles are this CTA's
    __device__ __forceinline__ Segment(const Args &a, const Walk<Cfg<kWide>::R, kThreads> &w) {
        constexpr int R = Cfg<kWide>::R;
        s = w.seq, span = w.span, b = w.b, head = w.head;
        rows = s.new_tokens * a.group, r0 = w.block * R, before = s.keys - s.new_tokens;
        take = w.take(), first = w.tile;
        p_hi = before + token_of(a, min(r0 + R, rows) - 1);
        nb = Cfg<kWide>::NB == 2 && r0 + kBlock < rows ? 2 : 1;
        blind = p_hi < 0;
        whole = first == 0 && take == w.segment();
    }
};

// Between segments: all roles have left this one, and thread 0 goes to the next. Whether there is one; none
// follows a wait that ran out (`dead`, of any role).
template <bool kWide>
__device__ __forceinline__ bool next_segment(const Args &a, Shared &sh, bool dead) {
    Walk<Cfg<kWide>::R, kThreads> &w = walk_of<kWide>(sh);
    if (dead) sh.dead = 1;
    tc_fence_before();
    __syncthreads();
    const bool over = sh.dead != 0;
    if (threadIdx.x == 0 && !over) {
        if (w.tile == 0 && w.take() != w.segment())
            *reinterpret_cast<Cut *>(a.ws + (int64_t)blockIdx.x * kCutBytes) = w.cut_here();
        w.next(a);
    }
    __syncthreads();
    tc_fence_after();
    return !over && !w.done();
}

// Warps 0 .. 4 NB - 1.
template <bool kWide>
__device__ __forceinline__ void softmax_role(const Args &a, Shared &sh, unsigned char *base, uint32_t tmem) {
    using C = Cfg<kWide>;
    constexpr int KS = C::KS, R = C::R;
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, blk = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + blk * 128 + lanes, tO = tmem + C::kTmemO + blk * 128 + lanes,
                   tP = tmem + C::kTmemP + blk * 128 + lanes;
    uint32_t n_tile = 0, n_s = 0, n_out[2] = {};  // tiles; tiles of this warp's block; results of each block
    float sg[4];
    lane_signs(a, lane, sg);
    for (bool more = !w.done(), dead = false; more; more = next_segment<kWide>(a, sh, dead)) {
        const Segment<kWide> g(a, w);
        const int wr = g.r0 + 32 * warp, n_rows = min(32, g.rows - wr);  // the warp's rows; may be none
        float down = 1.0f;  // of this lane's row: its power of two
        {
            unsigned char *const op = base + C::kOffQ + blk * C::kParts * kOp + (lane >> 4) * kBox + 8 * (lane & 1);
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 8) {  // eight rows at a time, so that their loads and shuffles overlap
                float v[8][4];
                int row[8];  // a row behind the last one repeats it, and counts as zeros
#pragma unroll
                for (int r = 0; r < 8; ++r) row[r] = min(wr + r0 + r, g.rows - 1);
                load_rows<8, !kWide>(a, g.s, g.head, row, lane, v);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[r][i] = r0 + r < n_rows ? __fmul_rn(v[r][i], sg[i]) : 0.0f;
                    row_fwht(v[r], lane);
                    // 2^u and 2^-u that bring the largest |q~| to 2^kQBits, by biased exponents (1 where the
                    // row is not finite)
                    const float m = fmaxf(fmaxf(fabsf(v[r][0]), fabsf(v[r][1])), fmaxf(fabsf(v[r][2]), fabsf(v[r][3])));
                    const int e = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(m)) >> 23);
                    const int up_exp = e == 255 ? 127 : min(253, 254 + kQBits - e);
                    const float up = __uint_as_float((uint32_t)up_exp << 23);
                    if (lane == r0 + r) down = __uint_as_float((uint32_t)(254 - up_exp) << 23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[r][i] = __fmul_rn(v[r][i], up);
                    unsigned char *const to = op + ((warp & 3) * 32 + r0 + r) * 128 + (((lane >> 1 & 7) ^ r) << 4);
                    const uint2 hi = make_uint2(h2(v[r][0], v[r][1]), h2(v[r][2], v[r][3]));
                    *reinterpret_cast<uint2 *>(to) = hi;
                    if (kWide) {
                        const float2 x = f2(hi.x), y = f2(hi.y);
                        *reinterpret_cast<uint2 *>(to + kOp) = make_uint2(h2(__fsub_rn(v[r][0], x.x), __fsub_rn(v[r][1], x.y)),
                                                                          h2(__fsub_rn(v[r][2], y.x), __fsub_rn(v[r][3], y.y)));
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_ready);
        }
        float M = -FLT_MAX, sum = 0.0f, G = 1.0f;
        if (blk < g.nb && !g.blind) {
            const int pos = lane < n_rows ? g.before + token_of(a, wr + lane) : -1;
            // positions of the warp's rows, for tiles that all of them see whole
            const int lo = g.before + token_of(a, min(wr, g.rows - 1)), hi = g.before + token_of(a, min(wr + 31, g.rows - 1));
            float x[32], y[32];
#pragma unroll 1
            for (int i = 0; i < g.take && !dead; ++i) {
                const uint32_t st = (n_tile + i) % KS;
                const int j0 = g.span.tile(g.first + i) * kTileKeys;
                if (!warp_wait(&sh.full_v[st], ((n_tile + i) / KS) & 1u)) {
                    dead = true;
                    break;
                }
                const Tile t = sh.tile[st];
                G = t.G;
                float unit = 1.0f;  // from S to the logit in log2 units
                const bool full = (t.valid[0] & t.valid[1] & t.valid[2] & t.valid[3]) == 0xffffffffu && j0 + kTileKeys <= lo + 1 &&
                                  (a.window == 0 || j0 > hi - a.window || j0 + kTileKeys <= a.sinks);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!warp_wait(&sh.s_done[blk][half], n_s & 1u)) {
                        dead = true;
                        break;
                    }
                    tc_fence_after();
                    // at least 2^-126, so that -inf stays what it is
                    if (half == 0) unit = fmaxf(__fmul_rn(down, sh.unit[(n_tile + i) & 3]), 0x1p-126f);
                    tmem_ld32(tS + 64 * half, x);
                    tmem_ld32(tS + 64 * half + 32, y);
                    float scale = half ? 1.0f : t.ratio;  // of O, before this half's product
                    tmem_wait(x);
                    tmem_wait(y);
                    if (!full) {  // -inf where the row does not see the key
                        const uint32_t on0 = visible(a, pos, j0 + 64 * half) & t.valid[2 * half],
                                       on1 = visible(a, pos, j0 + 64 * half + 32) & t.valid[2 * half + 1];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            x[k] = (on0 >> k & 1u) ? x[k] : -INFINITY;
                            y[k] = (on1 >> k & 1u) ? y[k] : -INFINITY;
                        }
                    }
                    const float mx = __fmul_rn(max32(max32(-INFINITY, x), y), unit);
                    if (__any_sync(0xffffffffu, mx > __fadd_rn(M, kLazy))) {  // every row of the warp takes its own maximum
                        const float m = fmaxf(M, mx), alpha = ex2(__fsub_rn(M, m));
                        M = m;
                        sum = __fmul_rn(sum, alpha);
                        scale = __fmul_rn(scale, alpha);
                    }
                    const float Mo = __fsub_rn(kLift, M);
                    const f32x2 M2 = pk2(Mo, Mo), U2 = pk2(unit, unit);
                    f32x2 ps[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)};
                    // P's columns lie over the half's columns of S
                    weights<kWide>(x, U2, M2, ps, tP + 64 * half);
                    weights<kWide>(y, U2, M2, ps, tP + 64 * half + (kWide ? 32 : 16));
                    float s0, s1;
                    upk2(add2(ps[0], ps[1]), s0, s1);
                    sum = __fadd_rn(sum, __fadd_rn(s0, s1));
                    if ((half || i > 0) && __any_sync(0xffffffffu, scale != 1.0f)) {
                        // the product of the half before has to be in O first
                        if (!warp_wait(&sh.pv_done[blk], (half - 1) & 1u)) {
                            dead = true;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            tmem_ld32(tO + 32 * c, x);
                            tmem_wait(x);
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = __fmul_rn(x[k], scale);
                            tmem_st32(tO + 32 * c, x);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_ready[blk][half]);
                }
                ++n_s;
            }
            // (both blocks': the results pass through the shared memory of both blocks' operands)
            if (!dead && (!warp_wait(&sh.o_done[0], n_out[0] & 1u) || (g.nb == 2 && !warp_wait(&sh.o_done[1], n_out[1] & 1u))))
                dead = true;
            tc_fence_after();
        }
        if (!g.blind) ++n_out[0], n_out[1] += g.nb == 2;
        // the rows: finished, or a part of a cut segment. Their sums pass through shared memory (Q and K:
        // every product is done) from a thread a row to a warp a row
        if (n_rows > 0 && !dead) {
            const float f = g.blind || sum == 0.0f ? 0.0f : __fmul_rn(__frcp_rn(sum), __fmul_rn(G, 1.0f / kTop));
            unsigned char *const stage = base + C::kOffQ + warp * 16384;
            if (!g.blind) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    tmem_ld32(tO + 32 * c, x);
                    tmem_wait(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4 *>(stage + 512 * lane + (((8 * c + k) ^ lane) << 4)) =
                            make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
                __syncwarp();
            }
            float *const slot = slot_at<R>(a, gridDim.x, 2 * blockIdx.x + (g.first == 0));
            const bool whole = g.whole;
#pragma unroll 1
            for (int r0 = 0; r0 < n_rows; r0 += 4) {
                float v[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float fr = __shfl_sync(0xffffffffu, f, r0 + r);
                    const float4 x = *reinterpret_cast<const float4 *>(stage + 512 * (r0 + r) + ((lane ^ (r0 + r)) << 4));
                    v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[r][i] = fr == 0.0f ? 0.0f : __fmul_rn(v[r][i], fr);
                }
                if (whole) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) row_fwht(v[r], lane);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < n_rows) {
                        if (whole)
                            put_row<!kWide>(a, g.s, g.head, wr + r0 + r, lane, sg, v[r]);
                        else
                            *reinterpret_cast<float4 *>(slot + (32 * warp + r0 + r) * 128 + 4 * lane) =
                                make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
                    }
            }
            if (!g.whole && lane < n_rows) {
                slot[R * 128 + 32 * warp + lane] = sum == 0.0f ? -INFINITY : M;
                slot[R * 129 + 32 * warp + lane] = sum;
            }
        }
        n_tile += g.blind ? 0 : g.take;
    }
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Warps 8 .. 11 decode the keys and 12 .. 15 the values: a thread a record.
template <bool kWide>
__device__ __forceinline__ void decode_role(const Args &a, Shared &sh, unsigned char *base) {
    using C = Cfg<kWide>;
    constexpr int KS = C::KS, R = C::R;
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, key = tid & 127;
    const bool values = warp >= 12;  // (one copy of the code for both)
    unsigned char *const recs = base + C::kOffRec + (values ? kRecBytes : 0), *const ops = base + (values ? C::kOffV : C::kOffK);
    uint64_t *const full = values ? sh.full_v : sh.full_k, *const free = values ? sh.free_v : sh.free_k;
    const uint8_t *const pool = values ? a.pools.v : a.pools.k;
    uint32_t n_tile = 0;
    for (bool more = !w.done(), dead = false; more; more = next_segment<kWide>(a, sh, dead)) {
        const Segment<kWide> g(a, w);
        const int take = g.blind ? 0 : g.take;
        // Two steps ahead of a tile its page entry is asked for, one step ahead its record. -1: no row
        // needs this thread's key (of no tile, or behind a window); -2: an entry outside the pool.
        int32_t entry = -1;
        uint32_t have = 0;  // bit i % kRecStages: the key of tile i has a page
        auto ask = [&](int i) {
            entry = -1;
            if (i < take) {
                const int j = g.span.tile(g.first + i) * kTileKeys + key;
                if (j <= g.p_hi && (j >= g.span.from || j < g.span.until)) {
                    entry = __ldg(a.table + g.b * a.pages_per_seq + (j >> a.pools.shift));
                    if (entry < 0) entry = -2;
                }
            }
        };
        auto fetch = [&](int i) {  // the record of tile i, whose entry is in hand
            const uint32_t bit = 1u << (i % kRecStages);
            have &= ~bit;
            if (i < take) {
                const int j = g.span.tile(g.first + i) * kTileKeys + key;
                const bool ok = entry >= 0 && entry < a.pools.n_pages;
                if (entry != -1 && !ok) atomicOr(&g_fault, tq3::kFaultPoolIndex);
                if (ok) have |= bit;
                const int64_t at = ok ? tq3_cache::record_at(a.pools, entry, g.head, j & ((1 << a.pools.shift) - 1)) : 0;
                const uint32_t to = smem_u32(recs + (i % kRecStages) * 2 * kRecBytes) + key * tq3_cache::kRec;
                const uint32_t bytes = ok ? 8 : 0;  // nothing is read for 0 bytes, zeros are written
                const uint8_t *const from = pool + at;
#pragma unroll
                for (int x = 0; x < 7; ++x) cp_async8(to + 8 * x, from + 8 * x, bytes);
                if (!values)
                    cp_async8(smem_u32(base + C::kOffFac + (i % kRecStages) * kTileKeys * 8) + key * 8, a.pools.v + at + 48, bytes);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        float G = 0.0f;
        ask(0);
        fetch(0);
        ask(1);
#pragma unroll 1
        for (int i = 0; i < take; ++i) {
            const uint32_t n = n_tile + i, st = n % KS, use = n / KS;
            fetch(i + 1);
            ask(i + 2);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // a thread reads only what it copied
            const uint32_t *const rec = reinterpret_cast<const uint32_t *>(
                recs + (i % kRecStages) * 2 * kRecBytes + key * tq3_cache::kRec);
            const float2 own = *reinterpret_cast<const float2 *>(rec + 12);
            float factor = __fmul_rn(own.x, own.y);
            if (!values) factor = __fmul_rn(factor, a.coef);
            const bool finite = fabsf(factor) < INFINITY;
            if (values && !finite) factor = 0.0f;
            // the largest finite factor of the tile (the four warps leave together: a warp whose wait ran out
            // says so here)
            const uint32_t top = __reduce_max_sync(0xffffffffu, finite ? __float_as_uint(fabsf(factor)) : 0u);
            if (lane == 0) sh.most[n & 1][values][warp & 3] = dead ? 0xffffffffu : top;
            if (values)
                named_sync<2, 128>();
            else
                named_sync<1, 128>();
            uint32_t all = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) all = max(all, sh.most[n & 1][values][x]);
            if (all == 0xffffffffu) {
                dead = true;
                break;
            }
            // a power of two at or below it, within 2^-100 .. 2^126
            const float up = __uint_as_float(min(253u << 23, max(27u << 23, all & 0x7f800000u)));
            const uint32_t valid = __ballot_sync(0xffffffffu, (have >> (i % kRecStages)) & 1u);
            float ratio = 1.0f;
            if (values) {
                if (G == 0.0f || __uint_as_float(all) > 4.0f * G) {
                    if (up > G) {
                        ratio = __fmul_rn(G, __uint_as_float((254u << 23) - __float_as_uint(up)));  // exact
                        G = up;
                    }
                }
                factor = __fmul_rn(factor, __fmul_rn(kTop, __uint_as_float((254u << 23) - __float_as_uint(G))));
            } else {
                const float2 other = *reinterpret_cast<const float2 *>(base + C::kOffFac + (i % kRecStages) * kTileKeys * 8 + key * 8);
                factor = __fmul_rn(factor, __fmul_rn(kTop, __uint_as_float((254u << 23) - __float_as_uint(up))));
                if (!(fabsf(__fmul_rn(other.x, other.y)) < INFINITY)) factor = __uint_as_float(0x7fffffffu);
            }
            if (n >= KS && !warp_wait(&free[st], (use - 1) & 1u)) {
                dead = true;
                continue;
            }
            if (lane == 0) {
                Tile &t = sh.tile[st];
                if (values) t.valid[warp & 3] = valid;
                if (warp == 12) t.ratio = ratio, t.G = G;
                if (warp == 8) sh.unit[n & 3] = __fmul_rn(up, 1.0f / kTop);
            }
            expand<kWide>(ops + st * C::kParts * kOp, key, rec, factor);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        n_tile += take;
    }
}

// The same value in every lane, so that the compiler keeps it in a uniform register: the tensor-core
// instructions take their operands from those, and moving each there costs more than the product.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// Warps 16 .. 15 + NB, one per block of rows. Returns whether the warp has issued products.
template <bool kWide>
__device__ __forceinline__ bool issue_role(const Args &a, Shared &sh, unsigned char *base, uint32_t tmem_) {
    using C = Cfg<kWide>;
    constexpr int KS = C::KS, R = C::R, kPasses = kWide ? 3 : 1;
    constexpr uint32_t kBlockOp = C::kParts * kOp >> 4, kLo = kOp >> 4, kHalf = 64 * 128 >> 4;  // in units of a descriptor's address
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    uint32_t n_tile = 0, segs = 0, n_s = 0;  // n_s: tiles of the block
    const uint32_t blk = uniform(threadIdx.x / 32 - kIssueWarp);
    const uint32_t tmem = uniform(tmem_), at = uniform(smem_u32(base));
    const uint32_t q = k_desc(at + C::kOffQ) + blk * kBlockOp, k0 = k_desc(at + C::kOffK), v0 = mn_desc(at + C::kOffV);
    const uint32_t tS = tmem + blk * 128, tO = tmem + C::kTmemO + blk * 128, tP = tmem + C::kTmemP + blk * 128;
    for (bool more = !w.done(), dead = false; more; more = next_segment<kWide>(a, sh, dead)) {
        const Segment<kWide> g(a, w);
        const uint32_t take = uniform(g.blind ? 0 : g.take), nb = uniform(g.nb), mine = blk < nb ? take : 0;
        if (mine > 0 && !warp_wait(&sh.q_ready, segs & 1u)) dead = true;
#pragma unroll 1
        for (uint32_t step = 0; step < 2 * mine + 2 && mine > 0 && !dead; ++step) {
            // S of half `half` of tile i, behind the value product of that half of tile i - 1
            const uint32_t i = step >> 1, half = step & 1, n = n_tile + i, st = n % KS, before = (n - 1) % KS;
            if ((i < mine && half == 0 && !warp_wait(&sh.full_k[st], (n / KS) & 1u)) ||
                (i > 0 && ((half == 0 && !warp_wait(&sh.full_v[before], ((n - 1) / KS) & 1u)) ||
                           !warp_wait(&sh.p_ready[blk][half], (n_s + i - 1) & 1u)))) {
                dead = true;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                if (i > 0) {
#pragma unroll
                    for (int ps = 0; ps < kPasses; ++ps) {
                        const uint32_t v = v0 + before * kBlockOp + half * kHalf + (ps == 1 ? kLo : 0);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts(tO, tP + 64 * half + (kWide ? 32 * (ks >> 1) + 8 * (ks & 1) + (ps == 2 ? 16 : 0) : 8 * ks),
                                   v + ks * (2048 >> 4), kIdescO, step > 2 || ps > 0 || ks > 0);
                    }
                    mma_commit(&sh.pv_done[blk]);
                    if (half) mma_commit(&sh.free_v[before]);
                    if (step == 2 * mine + 1) mma_commit(&sh.o_done[blk]);
                }
                if (i < mine) {
#pragma unroll
                    for (int ps = 0; ps < kPasses; ++ps) {
                        const uint32_t qa = q + (ps == 2 ? kLo : 0), k = k0 + st * kBlockOp + half * kHalf + (ps == 1 ? kLo : 0);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t off = (uint32_t)((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                            mma_ss(tS + 64 * half, qa + off, k + off, kIdescS, ps > 0 || ks > 0);
                        }
                    }
                    mma_commit(&sh.s_done[blk][half]);
                    // Hands on what the decoding warps wrote with the keys (`unit`). The softmax must not wait
                    // for the keys' own barrier: the tile two further may already have completed it again.
                    if (half == 0) mbar_arrive(&sh.s_done[blk][0]);
                    if (half) mma_commit(&sh.free_k[st]);
                }
                if (nb < C::NB && half) {  // a block without rows frees its share
                    if (i > 0) mbar_arrive(&sh.free_v[before]);
                    if (i < mine) mbar_arrive(&sh.free_k[st]);
                }
            }
            __syncwarp();
        }
        n_s += mine;
        ++segs;
        n_tile += take;
    }
    return n_s > 0;
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
    using C = Cfg<kWide>;
    constexpr int NB = C::NB, R = C::R;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const base = tq3::tile_base(smem_raw);
    Shared &sh = *reinterpret_cast<Shared *>(base + C::kOffShared);
    const int tid = threadIdx.x, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.full_k[i], 4);
            mbar_init(&sh.full_v[i], 4);
            mbar_init(&sh.free_k[i], NB);
            mbar_init(&sh.free_v[i], NB);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh.s_done[i][h], h == 0 ? 2 : 1);
                mbar_init(&sh.p_ready[i][h], 4);
            }
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.o_done[i], 1);
        }
        mbar_init(&sh.q_ready, 4 * NB);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        sh.dead = 0;
    }
    if (warp == kIssueWarp) tmem_alloc(&sh.tmem, 512);
    // No wait here: the rows kernel, launched before this one in the same call, lets it start only when all
    // that this call reads has been written, and the two share nothing that either writes.
    Cut *const cut = reinterpret_cast<Cut *>(a.ws + (int64_t)blockIdx.x * kCutBytes);
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    {
        Walk<R, kThreads> mine;
        mine.start(a, sh.scratch);
        if (tid == 0) {
            w = mine;
            cut->cut = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    bool issued = false;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        if (warp < 4 * C::NB)
            softmax_role<kWide>(a, sh, base, tmem);
        else
            for (bool more = !w.done(); more;) more = next_segment<kWide>(a, sh, false);
    } else if (warp < 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
        decode_role<kWide>(a, sh, base);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp < kIssueWarp + NB)
            issued = issue_role<kWide>(a, sh, base, tmem);
        else
            for (bool more = !w.done(); more;) more = next_segment<kWide>(a, sh, false);
    }
    pdl_trigger();
    pdl_wait();  // the join behind this kernel also needs the rows kernel's results
    // by the thread that issued them, the products: all done where no wait ran out
    if (issued && elect_one()) {
        mma_commit(&sh.drain[warp - kIssueWarp]);
        if (!mbar_wait_bounded(&sh.drain[warp - kIssueWarp], 0, kMaxPolls)) atomicOr(&g_fault, 128u);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

unsigned int read_and_clear_fault() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof v) != cudaSuccess) return 0x80000000u;
    if (v) cudaMemcpyToSymbol(g_fault, &zero, sizeof zero);
    return v;
}

int64_t workspace() { return tq3_chunk::workspace_bytes<256>(kSms); }

// Follows the rows kernel of the same call, whose results and own ones it leaves to one join.
template <bool kWide>
wq_status run(const Args &a, const Args &few, int few_ctas, cudaStream_t s) {
    using C = Cfg<kWide>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(chunk_kernel<kWide>), C::kSmem)) return WQ_ERR_CUDA;
    launch_pdl(chunk_kernel<kWide>, kSms, kThreads, C::kSmem, s, a);
    launch_join<C::R>(few, few_ctas, a, kSms, s);
    return launch_status();
}
wq_status run(const Args &a, bool wide, const Args &few, int few_ctas, cudaStream_t s) {
    return wide ? run<true>(a, few, few_ctas, s) : run<false>(a, few, few_ctas, s);
}

}  // namespace tq3_chunk_mma
}  // namespace wq

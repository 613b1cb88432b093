// Attention of ragged chunks over a batch's paged TQ3 cache on the tensor cores (tcgen05), for sequences
// with many rows per KV head. Same operation, identities and cutting of the work as tq3_chunk.cu; here a
// segment has NB x 128 rows and a tile of 128 keys is two products per 128 rows:
//     S = Q~ K^T       (128 rows x 128 keys, K = 128 rotated coordinates; both operands in shared memory)
//     O += P V         (128 rows x 128 coordinates, K = 128 keys; P in tensor memory, V in shared memory)
// with K's row j = c[idx_j] f_j coef 2^-u and V's row j = c[idx'_j] g_j 2^13 / G in fp16. 2^u brings the
// largest sum of |q| of the segment's rows, a bound of |q~|, to 2^4 .. 2^5, so that S is the logit in log2 units as it leaves the tensor
// core and the softmax has no per-key factor to apply. What underflows in K then moves a logit by less
// than 2^-13, and only the absolute error of a logit matters. G follows the largest g_j of the tiles so
// far and is raised when one is passed by 4 (O is rescaled then), so a value keeps all its bits down to
// 2^-27 of the largest. A value whose factor is not finite becomes zero and poisons its key's logits
// instead: a row that sees it gets NaN, any other is not touched.
//
// One CTA of 16 warps per SM. Warps 0-3 and 4-7 are the softmax of rows 0-127 and 128-255: a thread a row,
// which lies in its tensor-memory lane. Warps 8-11 decode: a thread a key. Warp 12 issues the products; 13-15
// fill its warpgroup.
//     decode   records of the next tile into registers; indices to selectors of byte permutes, which
//              fetch the bytes of four fp16 centroids at a time; times the factor (hi + lo); 16-byte
//              chunks into the 128-byte-swizzled operand tile (K as K-major B, V as MN-major B)
//     softmax  w = 2^(s - M) in one pass over S with the M that stood, redone with a larger one where a
//              row passes it by 2^8 (O is rescaled then); P as fp16 over S's columns
//     issue    S0(0) S1(0) | P0(i) V(i) -> O0, S0(i+1) | P1(i) V(i) -> O1, S1(i+1) | ...
// so that the tensor core works on one half of the rows while the other half's softmax runs. S(i+1) is
// issued behind O(i), so a row whose S(i+1) has arrived may touch O. For fp32 queries or results the
// operands are split hi + lo, a product takes three passes (hi hi, hi lo, lo hi), and 128 rows and one
// stage of operands fill the shared memory.
//
// Every wait is bounded; one that runs out sets fault bit 7, ends its role, and the others run out after
// it. In-flight products get a bounded chance to finish before the tensor memory is freed.
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
constexpr int kThreads = 512;
// registers a thread: 128 at launch; 256 softmax, 128 decode and 128 issue threads share the same 65536
constexpr int kRegsSoftmax = 184, kRegsDecode = 104, kRegsIssue = 40;
static_assert(256 * kRegsSoftmax + 128 * kRegsDecode + 128 * kRegsIssue <= kThreads * 128, "registers");
constexpr int kBox = 128 * 128;       // 64 coordinates of a 128-row fp16 operand, in bytes
constexpr int kOp = 2 * kBox;
constexpr uint32_t kMaxPolls = 1u << 24;
constexpr float kLazy = 8.0f, kLift = 6.0f;  // as in tq3_chunk.cu
constexpr int kQBits = 4;             // |q~| of a segment is scaled to less than 2^5
constexpr float kVTop = 8192.0f;      // a value of factor G has this one

// fp16 operands, fp32 accumulator, M = N = 128; B of the value product is MN-major.
constexpr uint32_t kIdescS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 16);

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
    static constexpr int kOffShared = kOffV + KS * kParts * kOp;
    static constexpr int kSmem = 1024 + kOffShared + 1024;
    // centroids times kGain: see tq3_chunk.cu
    static constexpr float kGain = kWide ? 1.0f : 1.6196665f;
    // tensor memory: S, O, and P (over S where two blocks fill the memory)
    static constexpr int kTmemO = NB * 128, kTmemP = kWide ? 256 : 0;
};

struct Tile {          // of a stage
    float ratio, G;    // G before / G, and G
    uint32_t valid[4]; // keys that have a page
};
struct Shared {
    uint64_t full_k[2], full_v[2], free_k[2], free_v[2], s_done[2], p_ready[2], o_done[2], q_ready, drain;
    Tile tile[2];
    uint32_t tmem;
    float down;        // 2^-u
    float top[8];      // per softmax warp: the largest sum of |q|
    uint32_t gmax[2][4];
    int64_t scratch[kThreads / 32 + 4];
    Walk<256, kThreads> walk256;
    Walk<128, kThreads> walk128;
};
static_assert(sizeof(Shared) <= 1024, "shared block");
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

// 16-byte chunk `chunk` (elements 8 chunk on) of row `row` of an operand: two boxes of 64 elements, rows
// of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint4 *op_chunk(unsigned char *op, int row, int chunk) {
    return reinterpret_cast<uint4 *>(op + (chunk >> 3) * kBox + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// The same tile as an MN-major operand (rows are K, their elements N): atoms of 64 elements x 8 rows, the
// next 64 elements a box further (leading offset), the next 8 rows 1024 bytes further (stride offset).
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D[tmem] (+)= A[tmem] * B.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t phase) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(phase)
                 : "memory");
    return ok || mbar_wait_bounded(bar, phase, kMaxPolls);
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

// Unnormalised 64-point FWHT of a thread's values. Half `h` of a 128-point one is that of the sums
// (h = 0) or the differences (h = 1) of the two halves of its input, so a thread never holds 128 values.
__device__ __forceinline__ void fwht64(float (&v)[64]) {
#pragma unroll
    for (int i = 0; i < 64; i += 2) {
        const float a = v[i], b = v[i + 1];
        v[i] = __fadd_rn(a, b);
        v[i + 1] = __fsub_rn(a, b);
    }
#pragma unroll
    for (int h = 2; h < 64; h <<= 1)
#pragma unroll
        for (int i = 0; i < 64; i += 2)
            if ((i & h) == 0) {
                const f32x2 a = pk2(v[i], v[i + 1]), b = pk2(v[i + h], v[i + h + 1]);
                upk2(add2(a, b), v[i], v[i + 1]);
                upk2(sub2(a, b), v[i + h], v[i + h + 1]);
            }
}
// Elements e .. e + 7 of a query row.
__device__ __forceinline__ void load8(const Args &a, int64_t at, int e, float (&x)[8]) {
    if (a.q_bf16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at + e));
        x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
        x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
    } else {
        const float4 *const p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at + e);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
}

// Four fp16 centroids a selector: the low and the high bytes of the eight values, in two words each.
struct Table {
    uint32_t lo0, lo1, hi0, hi1;
};
__device__ __forceinline__ Table make_table(const uint16_t (&h)[8]) {
    Table t = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t.lo0 |= (uint32_t)(h[i] & 255) << (8 * i);
        t.lo1 |= (uint32_t)(h[i + 4] & 255) << (8 * i);
        t.hi0 |= (uint32_t)(h[i] >> 8) << (8 * i);
        t.hi1 |= (uint32_t)(h[i + 4] >> 8) << (8 * i);
    }
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

// The 128 centroids of a record's indices times a factor, into row `row` of an operand. hi + lo is the
// factor, as pairs of equal halves.
template <bool kWide>
__device__ __forceinline__ void expand(unsigned char *op, int row, const uint32_t (&w)[12], const Table &th, const Table &tl,
                                       float factor) {
    const uint32_t fh = h2(factor, factor);
    const float rest = __fsub_rn(factor, f2(fh).x);
    const uint32_t fl = h2(rest, rest);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const int o = 24 * c, q = o >> 5, s = o & 31;
        const uint32_t sel = nibbles(s == 0 ? w[q] : s == 8 ? w[q] >> 8 : __funnelshift_r(w[q], w[q + 1 < 12 ? q + 1 : q], s));
        uint32_t ch[4];
        four(th, sel, ch[0], ch[1]);
        four(th, sel >> 16, ch[2], ch[3]);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = mul_h2(ch[i], fh);
        if (kWide) {
            // hi = RN(ch fh); lo = (ch fh - hi) + ch fl + cl fh, the difference exact
            uint32_t cl[4], l[4];
            four(tl, sel, cl[0], cl[1]);
            four(tl, sel >> 16, cl[2], cl[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                l[i] = fma_h2(cl[i], fh, fma_h2(ch[i], fl, fma_h2(ch[i], fh, h[i] ^ 0x80008000u)));
            *op_chunk(op + kOp, row, c) = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = fma_h2(ch[i], fl, h[i]);
        }
        *op_chunk(op, row, c) = make_uint4(h[0], h[1], h[2], h[3]);
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
        p_hi = before + (min(r0 + R, rows) - 1) / a.group;
        nb = Cfg<kWide>::NB == 2 && r0 + kBlock < rows ? 2 : 1;
        blind = p_hi < 0;
        whole = first == 0 && take == w.segment();
    }
};

// Between segments: all roles have left this one, and thread 0 goes to the next.
template <bool kWide>
__device__ __forceinline__ void next_segment(const Args &a, Walk<Cfg<kWide>::R, kThreads> &w, bool advance) {
    tc_fence_before();
    __syncthreads();
    if (advance) {
        if (w.tile == 0 && w.take() != w.segment())
            *reinterpret_cast<Cut *>(a.ws + (int64_t)blockIdx.x * kCutBytes) = w.cut_here();
        w.next(a);
    }
    __syncthreads();
    tc_fence_after();
}

// Warps 0 .. 4 NB - 1. Returns whether a wait ran out (as the other roles do).
template <bool kWide>
__device__ __forceinline__ bool softmax_role(const Args &a, Shared &sh, unsigned char *base, uint32_t tmem) {
    using C = Cfg<kWide>;
    constexpr int NB = C::NB, KS = C::KS, R = C::R;
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool dead = false;
    uint32_t n_tile = 0, n_s = 0, n_out = 0;  // tiles; of this warp's block: S products, results
    while (!w.done()) {
        const Segment<kWide> g(a, w);
        const int blk = warp >> 2;
        const int rr = blk * kBlock + (warp & 3) * 32 + lane, row = g.r0 + rr;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        {
            // |q~| is at most the row's sum of |q|, which decides the scale
            const int64_t at = row < g.rows ? (int64_t)(g.s.start + row / a.group) * a.q_token +
                                                (int64_t)(g.head * a.group + row % a.group) * a.q_head
                                          : -1;
            float m = 0.0f;
            if (at >= 0)
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    float x[8];
                    load8(a, at, 8 * c, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = __fadd_rn(m, fabsf(x[i]));
                }
            if (!(m < INFINITY)) m = 0.0f;  // a row that is not finite spoils only itself
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) sh.top[warp] = m;
            named_sync<1, 128 * NB>();
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) m = fmaxf(m, sh.top[i]);
            // 2^u and 2^-u with u = kQBits - exponent, by biased exponents
            const int e = max(kQBits + 1, min(253, (int)(__float_as_uint(m) >> 23)));
            const int up_exp = min(254, 254 + kQBits - e);
            const float up = __uint_as_float((uint32_t)up_exp << 23);
            if (tid == 0) sh.down = __uint_as_float((uint32_t)(254 - up_exp) << 23);
            unsigned char *const op = base + C::kOffQ + blk * C::kParts * kOp;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                float v[64];
                const float sgn = half ? -1.0f : 1.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float x[8] = {}, y[8] = {};
                    if (at >= 0) load8(a, at, 8 * c, x), load8(a, at, 64 + 8 * c, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[8 * c + i] = __fmaf_rn(__fmul_rn(y[i], sign_of(a.mask, 64 + 8 * c + i)), sgn,
                                                 __fmul_rn(x[i], sign_of(a.mask, 8 * c + i)));
                }
                fwht64(v);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __fmul_rn(v[8 * c + 2 * i], up), y = __fmul_rn(v[8 * c + 2 * i + 1], up);
                        h[i] = h2(x, y);
                        if (kWide) l[i] = h2(__fsub_rn(x, f2(h[i]).x), __fsub_rn(y, f2(h[i]).y));
                    }
                    *op_chunk(op, rr & 127, 8 * half + c) = make_uint4(h[0], h[1], h[2], h[3]);
                    if (kWide) *op_chunk(op + kOp, rr & 127, 8 * half + c) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_ready);
        }
        float M = -FLT_MAX, sum = 0.0f, G = 1.0f;
        const uint32_t tS = tmem + blk * 128 + lanes, tO = tmem + C::kTmemO + blk * 128 + lanes,
                       tP = tmem + C::kTmemP + blk * 128 + lanes;
        if (blk < g.nb && !g.blind && !dead) {
            const int pos = row < g.rows ? g.before + row / a.group : -1;
            // positions of the warp's rows, for tiles that all of them see whole
            const int wr = g.r0 + blk * kBlock + (warp & 3) * 32;
            const int lo = g.before + min(wr, g.rows - 1) / a.group, hi = g.before + min(wr + 31, g.rows - 1) / a.group;
            for (int i = 0; i < g.take; ++i) {
                const uint32_t n = n_tile + i, st = n % KS;
                const int j0 = g.span.tile(g.first + i) * kTileKeys;
                if (!warp_wait(&sh.full_v[st], (n / KS) & 1u) || !warp_wait(&sh.s_done[blk], n_s & 1u)) {
                    dead = true;
                    break;
                }
                ++n_s;
                tc_fence_after();
                const Tile &t = sh.tile[st];
                const bool full = (t.valid[0] & t.valid[1] & t.valid[2] & t.valid[3]) == 0xffffffffu &&
                                  j0 + kTileKeys <= lo + 1 &&
                                  (a.window == 0 || j0 > hi - a.window || j0 + kTileKeys <= a.sinks);
                float scale = t.ratio;  // of O, before this tile's product
                G = t.G;
                uint32_t P[kWide ? 1 : 64];
                float psum;
                for (int pass = 0; pass < 2; ++pass) {
                    const float Mo = __fsub_rn(M, kLift);
                    const f32x2 M2 = pk2(Mo, Mo);
                    float mx = -INFINITY;
                    f32x2 ps = pk2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float x[32];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait(x);
                        if (!full) {
                            const uint32_t on = visible(a, pos, j0 + 32 * c) & t.valid[c];
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(on >> k & 1u)) x[k] = -INFINITY;
                        }
                        uint32_t pk[32];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            mx = max3(mx, x[k], x[k + 1]);
                            float d0, d1;
                            upk2(sub2(pk2(x[k], x[k + 1]), M2), d0, d1);
                            d0 = ex2(d0), d1 = ex2(d1);
                            ps = add2(ps, pk2(d0, d1));
                            const uint32_t h = h2(d0, d1);
                            if (kWide) {
                                pk[k / 2] = h;
                                pk[16 + k / 2] = h2(__fsub_rn(d0, f2(h).x), __fsub_rn(d1, f2(h).y));
                            } else {
                                P[kWide ? 0 : 16 * c + k / 2] = h;
                            }
                        }
                        if (kWide) tmem_st32(tP + 32 * c, *reinterpret_cast<const float(*)[32]>(pk));
                    }
                    float s0, s1;
                    upk2(ps, s0, s1);
                    psum = __fadd_rn(s0, s1);
                    const bool raise = mx > __fadd_rn(M, kLazy);
                    if (!__any_sync(0xffffffffu, raise)) break;
                    // every row of the warp takes its own maximum
                    const float m = fmaxf(M, mx), alpha = ex2(__fsub_rn(M, m));
                    M = m;
                    sum = __fmul_rn(sum, alpha);
                    scale = __fmul_rn(scale, alpha);
                }
                if (i > 0 && __any_sync(0xffffffffu, scale != 1.0f)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __fmul_rn(o[k], scale);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                sum = __fadd_rn(sum, psum);
                if (!kWide) {
                    tmem_st32(tP, *reinterpret_cast<const float(*)[32]>(&P[0]));
                    tmem_st32(tP + 32, *reinterpret_cast<const float(*)[32]>(&P[kWide ? 0 : 32]));
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[blk]);
            }
            if (!dead && !warp_wait(&sh.o_done[blk], n_out & 1u)) dead = true;
            ++n_out;
            tc_fence_after();
        }
        // this thread's row: finished, or a part of a cut segment
        if (blk < g.nb && !dead) {
            const float f = g.blind || sum == 0.0f ? 0.0f : __fmul_rn(__frcp_rn(sum), __fmul_rn(G, 1.0f / (kVTop * C::kGain)));
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const float sgn = half ? -1.0f : 1.0f;
                float v[64];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[32], y[32];
                    if (!g.blind) {
                        tmem_ld32(tO + 32 * c, x);
                        tmem_ld32(tO + 64 + 32 * c, y);
                        tmem_wait(x);
                        tmem_wait(y);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (f == 0.0f) x[i] = y[i] = 0.0f;
                        v[32 * c + i] = g.whole ? __fmul_rn(__fmaf_rn(y[i], sgn, x[i]), f) : __fmul_rn(half ? y[i] : x[i], f);
                    }
                }
                if (row < g.rows && g.whole) {
                    fwht64(v);
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const float flip = half ? sign_of(a.mask, 64 + i) : sign_of(a.mask, i);
                        v[i] = __fmul_rn(__fmul_rn(v[i], tq3::fwht_post()), flip);
                    }
                    const int64_t at = ((int64_t)(g.s.start + row / a.group) * a.pools.heads * a.group + g.head * a.group +
                                        row % a.group) * 128 + 64 * half;
                    if (a.out_bf16) {
                        uint4 *const to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            to[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                               pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
                    } else {
                        float4 *const to = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
#pragma unroll
                        for (int i = 0; i < 16; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                } else if (row < g.rows) {
                    float *const slot = slot_at<R>(a, gridDim.x, 2 * blockIdx.x + (g.first == 0));
                    float4 *const to = reinterpret_cast<float4 *>(slot + rr * 128 + 64 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    slot[R * 128 + rr] = sum == 0.0f ? -INFINITY : M;
                    slot[R * 129 + rr] = sum;
                }
                __syncwarp();
            }
        }
        n_tile += g.blind ? 0 : g.take;
        next_segment<kWide>(a, w, tid == 0);
    }
    return dead;
}

// Warps 8 .. 11.
template <bool kWide>
__device__ __forceinline__ bool decode_role(const Args &a, Shared &sh, unsigned char *base) {
    using C = Cfg<kWide>;
    constexpr int KS = C::KS, R = C::R;
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool dead = false;
    uint32_t n_tile = 0, segs = 0;
    Table th, tl;
    {
        uint16_t hh[8], hl[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = __fmul_rn(tq3::centroid(i), C::kGain);
            const uint32_t p = h2(x, 0.0f);
            hh[i] = (uint16_t)p;
            hl[i] = (uint16_t)h2(__fsub_rn(x, f2(p).x), 0.0f);
        }
        th = make_table(hh);
        tl = make_table(hl);
    }
    while (!w.done()) {
        const Segment<kWide> g(a, w);
        const int key = tid - 256;
        uint2 rk[7], rv[7];
        bool ok = false, ok_next = false;
        // this thread's key of tile i: whether a row needs it, and its records
        auto load = [&](int i) {
            ok_next = false;
            if (i < g.take) {
                const int j = g.span.tile(g.first + i) * kTileKeys + key;
                if (j <= g.p_hi && (j >= g.span.from || j < g.span.until)) {
                    const int32_t page = __ldg(a.table + g.b * a.pages_per_seq + (j >> a.pools.shift));
                    if (page >= 0 && page < a.pools.n_pages) {
                        const int64_t at = tq3_cache::record_at(a.pools, page, g.head, j & ((1 << a.pools.shift) - 1));
#pragma unroll
                        for (int x = 0; x < 7; ++x) {
                            rk[x] = __ldg(reinterpret_cast<const uint2 *>(a.pools.k + at) + x);
                            rv[x] = __ldg(reinterpret_cast<const uint2 *>(a.pools.v + at) + x);
                        }
                        ok_next = true;
                    } else {
                        atomicOr(&g_fault, tq3::kFaultPoolIndex);
                    }
                }
            }
        };
        float G = 0.0f;
        if (!g.blind) {
            load(0);
            if (!dead && !warp_wait(&sh.q_ready, segs & 1u)) dead = true;
        }
        const float coef = __fmul_rn(__fmul_rn(a.coef, 1.0f / C::kGain), sh.down);
        for (int i = 0; i < g.take && !g.blind; ++i) {
            const uint32_t n = n_tile + i, st = n % KS, use = n / KS;
            ok = ok_next;
            uint32_t wk[12], wv[12];
            float fk = 0.0f, gv = 0.0f;
            if (ok) {
#pragma unroll
                for (int x = 0; x < 6; ++x) wk[2 * x] = rk[x].x, wk[2 * x + 1] = rk[x].y, wv[2 * x] = rv[x].x, wv[2 * x + 1] = rv[x].y;
                fk = __fmul_rn(__fmul_rn(__uint_as_float(rk[6].x), __uint_as_float(rk[6].y)), coef);
                gv = __fmul_rn(__uint_as_float(rv[6].x), __uint_as_float(rv[6].y));
                if (!(fabsf(gv) < INFINITY)) fk = __uint_as_float(0x7fffffffu), gv = 0.0f;
            } else {
#pragma unroll
                for (int x = 0; x < 12; ++x) wk[x] = wv[x] = 0u;
            }
            load(i + 1);
            // the largest factor of the tile
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(gv)));
            const uint32_t valid = __ballot_sync(0xffffffffu, ok);
            // (the four warps leave together: a warp whose wait ran out says so here)
            if (lane == 0) sh.gmax[n & 1][warp - 8] = dead ? 0xffffffffu : top;
            named_sync<2, 128>();
            uint32_t all = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) all = max(all, sh.gmax[n & 1][x]);
            if (all == 0xffffffffu) {
                dead = true;
                break;
            }
            const float most = __uint_as_float(all);
            float ratio = 1.0f;
            if (G == 0.0f || most > 4.0f * G) {
                // a power of two at or below it, at least 2^-100; O is rescaled by an exact ratio
                const float up = __uint_as_float(max(27u << 23, __float_as_uint(most) & 0x7f800000u));
                if (up > G) {
                    ratio = __fdiv_rn(G, up);
                    G = up;
                }
            }
            if (n >= KS && !warp_wait(&sh.free_k[st], (use - 1) & 1u)) {
                dead = true;
                continue;
            }
            expand<kWide>(base + C::kOffK + st * C::kParts * kOp, key, wk, th, tl, fk);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full_k[st]);
            if (n >= KS && !warp_wait(&sh.free_v[st], (use - 1) & 1u)) {
                dead = true;
                continue;
            }
            if (lane == 0) {
                sh.tile[st].valid[warp - 8] = valid;
                if (warp == 8) sh.tile[st].ratio = ratio, sh.tile[st].G = G;
            }
            expand<kWide>(base + C::kOffV + st * C::kParts * kOp, key, wv, th, tl, __fmul_rn(gv, __fdiv_rn(kVTop, G)));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full_v[st]);
        }
        ++segs;
        n_tile += g.blind ? 0 : g.take;
        next_segment<kWide>(a, w, false);
    }
    return dead;
}

// Warp 12.
template <bool kWide>
__device__ __forceinline__ bool issue_role(const Args &a, Shared &sh, unsigned char *base, uint32_t tmem) {
    using C = Cfg<kWide>;
    constexpr int NB = C::NB, KS = C::KS, R = C::R;
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    const int lane = threadIdx.x & 31;
    bool dead = false;
    uint32_t n_tile = 0, segs = 0, n_blk[NB] = {};  // n_blk: S products of a block
    while (!w.done()) {
        const Segment<kWide> g(a, w);
        if (!g.blind && !dead && !warp_wait(&sh.q_ready, segs & 1u)) dead = true;
        const uint32_t q0 = smem_u32(base + C::kOffQ);
        auto wait_op = [&](uint64_t *bar, uint32_t phase) {
            if (!dead && !warp_wait(bar, phase)) dead = true;
            tc_fence_after();
        };
        auto issue_s = [&](int blk, uint32_t n) {
            const uint32_t kb = smem_u32(base + C::kOffK + (n % KS) * C::kParts * kOp);
            if (!dead && lane == 0) {
#pragma unroll
                for (int pass = 0; pass < (kWide ? 3 : 1); ++pass) {
                    const uint64_t qa = sw128_desc(q0 + blk * C::kParts * kOp + (pass == 2 ? kOp : 0)),
                                   kd = sw128_desc(kb + (pass == 1 ? kOp : 0));
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (uint32_t)((ks >> 2) * kBox + (ks & 3) * 32) >> 4;
                        mma_bf16(tmem + blk * 128, qa + off, kd + off, kIdescS, pass > 0 || ks > 0);
                    }
                }
                mma_commit(&sh.s_done[blk]);
            }
        };
        auto issue_o = [&](int blk, uint32_t n, bool first) {
            const uint32_t vb = smem_u32(base + C::kOffV + (n % KS) * C::kParts * kOp);
            if (!dead && lane == 0) {
#pragma unroll
                for (int pass = 0; pass < (kWide ? 3 : 1); ++pass) {
                    const uint64_t vd = mn_desc(vb + (pass == 1 ? kOp : 0));
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t p = kWide ? tmem + C::kTmemP + 32 * (ks >> 1) + 8 * (ks & 1) + (pass == 2 ? 16 : 0)
                                                 : tmem + C::kTmemP + blk * 128 + 8 * ks;
                        mma_ts(tmem + C::kTmemO + blk * 128, p, vd + (uint32_t)(ks * 2048 >> 4), kIdescO,
                               !first || pass > 0 || ks > 0);
                    }
                }
            }
        };
        if (!g.blind) {
            for (int i = 0; i <= g.take && !dead; ++i) {
                const uint32_t n = n_tile + i;
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    if (blk >= g.nb) break;
                    if (i > 0) {  // O of tile i - 1
                        if (blk == 0) wait_op(&sh.full_v[(n - 1) % KS], ((n - 1) / KS) & 1u);
                        wait_op(&sh.p_ready[blk], (n_blk[blk] - 1) & 1u);
                        issue_o(blk, n - 1, i == 1);
                        if (!dead && lane == 0) {
                            if (blk == g.nb - 1) mma_commit(&sh.free_v[(n - 1) % KS]);
                            if (i == g.take) mma_commit(&sh.o_done[blk]);
                        }
                    }
                    if (i < g.take) {
                        if (blk == 0) wait_op(&sh.full_k[n % KS], (n / KS) & 1u);
                        issue_s(blk, n);
                        if (!dead && lane == 0 && blk == g.nb - 1) mma_commit(&sh.free_k[n % KS]);
                        ++n_blk[blk];
                    }
                }
            }
        }
        ++segs;
        n_tile += g.blind ? 0 : g.take;
        next_segment<kWide>(a, w, false);
    }
    return dead;
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
    using C = Cfg<kWide>;
    constexpr int NB = C::NB, R = C::R;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const base = tq3::tile_base(smem_raw);
    Shared &sh = *reinterpret_cast<Shared *>(base + C::kOffShared);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.full_k[i], 4);
            mbar_init(&sh.full_v[i], 4);
            mbar_init(&sh.free_k[i], 1);
            mbar_init(&sh.free_v[i], 1);
            mbar_init(&sh.s_done[i], 1);
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.o_done[i], 1);
        }
        mbar_init(&sh.q_ready, 4 * NB);
        mbar_init(&sh.drain, 1);
    }
    if (warp == 12) tmem_alloc(&sh.tmem, 512);
    pdl_wait();
    Cut *const cut = reinterpret_cast<Cut *>(a.ws + (int64_t)blockIdx.x * kCutBytes);
    Walk<R, kThreads> &w = walk_of<kWide>(sh);
    {
        Walk<R, kThreads> mine;
        mine.start(a, sh.scratch);
        if (tid == 0) {
            w = mine;
            cut->cut = 0;
            if (blockIdx.x == 0)
                for (int b = 0; b < a.batch; ++b)
                    if (__ldg(a.kv_len + b) > (a.pages_per_seq << a.pools.shift)) atomicOr(&g_fault, tq3::kFaultPoolIndex);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    bool dead = false;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        if (warp < 4 * C::NB)
            dead = softmax_role<kWide>(a, sh, base, tmem);
        else
            while (!w.done()) next_segment<kWide>(a, w, false);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
        dead = decode_role<kWide>(a, sh, base);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == 12)
            dead = issue_role<kWide>(a, sh, base, tmem);
        else
            while (!w.done()) next_segment<kWide>(a, w, false);
    }
    pdl_trigger();
    // products still in flight after a wait ran out get a bounded chance to finish
    if (warp == 12 && dead && lane == 0) {
        mma_commit(&sh.drain);
        mbar_wait_bounded(&sh.drain, 0, kMaxPolls);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
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

template <bool kWide>
wq_status run(const Args &a, cudaStream_t s) {
    using C = Cfg<kWide>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(chunk_kernel<kWide>), C::kSmem)) return WQ_ERR_CUDA;
    launch_pdl(chunk_kernel<kWide>, kSms, kThreads, C::kSmem, s, a);
    launch_join<C::R>(a, kSms, s);
    return launch_status();
}
wq_status run(const Args &a, bool wide, cudaStream_t s) { return wide ? run<true>(a, s) : run<false>(a, s); }

}  // namespace tq3_chunk_mma
}  // namespace wq

// Writing a paged TQ3 cache as tokens arrive, and reading ragged sequences back: page "tq3_core.py"
// (tq3_quantize, tq3_dequantize) on the pools of tq3_cache.cuh.
//
// Both kernels give a vector to one thread (64 packed fp32 pairs in registers, so the seven FWHT
// stages need no exchange) and a tile of 32 tokens of one head of K or V to one warp. A tile's
// records are then one or a few runs of consecutive places in the pool, moved in 8-byte pieces by
// neighbouring lanes; its rows are moved in 16-byte pieces through shared memory.
//
// append. With z = H (s . x) and m = max|z|: norm = max(|x|, 1e-8), scale = max(m / (sqrt(128) norm),
// 1e-8), idx_i = #{k : B_k scale < z_i / (sqrt(128) norm)}. In exact arithmetic that is B_k T < z_i
// with T = m while neither floor is active. The fast path forms u_i = z_i / T in fp32 and takes
// 3 + ceil(Q(u_i)) with the odd quintic of tq3_common.cuh. fp32 moves z_i by at most
// 7 * 2^-24 * sqrt(128) |x| <= 4.8e-6 T (each stage rounds by 2^-24 of its partial sums, whose
// contributions to z_i are bounded by Cauchy-Schwarz; T >= |x|), T by as much, and the polynomial
// moves a boundary by 3e-7: 1e-5 in u, 4.5e-5 in Q (|Q'| <= 4.4). A vector with a coefficient whose
// Q lies that close to an integer is decided again by the whole warp in fp64, from the input: four
// coefficients a lane. The indices are then those of real arithmetic, unless z_i lies within fp64's error of
// a boundary: 7 * 2^-53 * sqrt(128) |x| of its own, and nearly that of T's, 2^-45 |x| together.
// About one vector in 100 of Gaussian data takes that path; where all do (each has a coefficient of
// exactly 0, as constant vectors have) 32768 tokens x 8 heads of bf16 take 494 us in place of 86. Vectors
// whose fp32 sum of squares leaves [1.1e-16, 1e37] take it too (the floors, overflow of z); an all-zero
// vector does not need it.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tq3_cache.cuh"
#include "tq3_common.cuh"

namespace wq {
namespace tq3_cache {

using tq3::SignMask;

constexpr int kTile = 32;      // tokens per tile, a lane each
// Both bodies are some 2500 instructions long, more than the instruction cache keeps for warps that are each
// somewhere else in it. Append's 12 warps of an SM (what 168 registers a thread allow) are one CTA that meets
// before each item and so shares its fetches: 32768 tokens x 8 heads take 113 us with a CTA a warp, 102 with
// four warps a CTA, 86 with twelve, 92 where they meet twice an item. Read waits for its stores more than for
// instructions and loses by it: 58, 63 and 74 us for 16 sequences of up to 4096 keys.
constexpr int kAppendWarps = 12;
constexpr int kReadCtas = 12;  // per SM, a warp each
constexpr int kSms = 148;
constexpr int kAppendBytes = 16384 + 32 * kRec;  // of a warp: two bf16 tiles or one fp32 tile, and the tile's records
constexpr float kNear = 0.5f - 4.5e-5f;

__device__ unsigned int g_fault;

struct Rows {  // rows of 128 elements: base + token * token_stride + head * head_stride (in bytes)
    const unsigned char *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(take ? 16 : 0)
                 : "memory");
}

template <bool kDefault>
__device__ __forceinline__ uint32_t flip_of(const SignMask &m, int e) {
    return kDefault ? tq3::default_flip(e) : (~(m.w[e >> 5] >> (e & 31)) & 1u) << 31;
}

// The six stages between pairs: h = 1 .. 32 of a vector held as pairs (k, k + 64), h = 2 .. 64 of one
// held as pairs (2k, 2k + 1).
__device__ __forceinline__ void stages_between(f32x2 (&P)[64]) {
#pragma unroll
    for (int h = 1; h <= 32; h <<= 1)
#pragma unroll
        for (int k = 0; k < 64; ++k)
            if ((k & h) == 0) {
                const f32x2 a = P[k], b = P[k + h];
                P[k] = add2(a, b);
                P[k + h] = sub2(a, b);
            }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The record of one row by the whole warp in fp64; lane l holds elements 4 l .. 4 l + 3.
template <bool kBf16>
static __device__ __noinline__ void encode_row_fp64(const unsigned char *row, const SignMask &mask, uint32_t *rec) {
    const int lane = threadIdx.x & 31;
    double z[4];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i;
        const float x = kBf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(row)[e])
                              : reinterpret_cast<const float *>(row)[e];
        ss = fma((double)x, (double)x, ss);
        z[i] = ((mask.w[e >> 5] >> (e & 31)) & 1u) ? (double)x : -(double)x;
    }
    ss = warp_sum(ss);
    {
        const double a = z[0] + z[1], b = z[0] - z[1], c = z[2] + z[3], d = z[2] - z[3];
        z[0] = a + c;
        z[1] = b + d;
        z[2] = a - c;
        z[3] = b - d;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double other = __shfl_xor_sync(0xffffffffu, z[i], o);
            z[i] = (lane & o) ? other - z[i] : z[i] + other;
        }
    double m = fmax(fmax(fabs(z[0]), fabs(z[1])), fmax(fabs(z[2]), fabs(z[3])));
    m = warp_max(m);
    const double root = 11.313708498984760390;  // sqrt(128)
    const double norm = fmax(sqrt(ss), 1e-8);
    double scale = fmax(m / (root * norm), 1e-8);
    const bool over = !((float)norm < INFINITY);  // the page divides by an infinite norm: y = 0
    if (over) scale = 1e-8;
    const double T = scale * (root * norm);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t idx = 3;
        if (!over)
            idx = (z[i] > -(double)0.7992f * T) + (z[i] > -(double)0.4824f * T) + (z[i] > -(double)0.2304f * T) +
                  (z[i] > 0.0) + (z[i] > (double)0.2304f * T) + (z[i] > (double)0.4824f * T) +
                  (z[i] > (double)0.7992f * T);
        bits |= idx << (3 * i);
    }
    bits |= __shfl_down_sync(0xffffffffu, bits, 1) << 12;
    if (!(lane & 1)) {
        unsigned char *b = reinterpret_cast<unsigned char *>(rec) + 3 * (lane >> 1);
        b[0] = (unsigned char)bits;
        b[1] = (unsigned char)(bits >> 8);
        b[2] = (unsigned char)(bits >> 16);
    }
    if (lane == 0) {
        rec[12] = __float_as_uint((float)norm);
        rec[13] = __float_as_uint((float)scale);
    }
}

// ---------------------------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------------------------
template <bool kBf16, bool kDefault>
__global__ void __launch_bounds__(kAppendWarps * 32, 1)
    append_kernel(Rows in, int64_t tokens, const int64_t *__restrict__ slots, Pools pools, SignMask mask) {
    constexpr int kRowBytes = kBf16 ? 256 : 512, kChunks = kRowBytes / 16;
    constexpr int kStages = kBf16 ? 2 : 1;
    extern __shared__ __align__(16) unsigned char smem_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *const smem = smem_all + warp * kAppendBytes;
    uint32_t *const recs = reinterpret_cast<uint32_t *>(smem + kStages * kTile * kRowBytes);  // [32][14]
    const int64_t n_slots = pools.n_pages << pools.shift;
    // items: (tile of tokens, head, K or V), the last fastest; a contiguous share of them for each warp
    const int per_tile = 2 * pools.heads;
    const int64_t items = (tokens + kTile - 1) / kTile * per_tile;
    const int64_t warps = (int64_t)gridDim.x * kAppendWarps, me = (int64_t)blockIdx.x * kAppendWarps + warp;
    const int64_t begin = items * me / warps, end = items * (me + 1) / warps, rounds = (items + warps - 1) / warps;

    auto row_of = [&](int hk, int64_t token) {
        const int64_t head = hk >> 1;
        return (hk & 1) ? in.v + token * in.v_token + head * in.v_head : in.k + token * in.k_token + head * in.k_head;
    };
    auto fetch = [&](int64_t t0, int hk, int stage) {
        unsigned char *const dst = smem + stage * kTile * kRowBytes;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = i * 32 + lane, r = at / kChunks, c = at % kChunks;
            const bool take = t0 + r < tokens;
            cp_async16(dst + r * kRowBytes + ((c ^ (r & 7)) << 4), row_of(hk, take ? t0 + r : t0) + 16 * c, take);
        }
    };

    int64_t tile = begin / per_tile, have = -1, slot = -1;
    int hk = (int)(begin - tile * per_tile);
    if (begin < end) fetch(tile * kTile, hk, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int64_t item = begin; item < begin + rounds; ++item) {
        __syncthreads();
        if (item >= end) continue;
        const int stage = kStages == 2 ? (int)((item - begin) & 1) : 0;
        const int64_t t0 = tile * kTile, token = t0 + lane;
        if (have != tile) {
            slot = token < tokens ? __ldg(slots + token) : -1;
            have = tile;
        }
        const int here = hk;
        if (++hk == per_tile) hk = 0, ++tile;
        if (kStages == 2) {
            if (item + 1 < end) fetch(tile * kTile, hk, stage ^ 1);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();

        // x with the sign flips, as pairs (k, k + 64); the sum of squares; stage h = 64
        f32x2 P[64];
        f32x2 acc[4] = {0ull, 0ull, 0ull, 0ull};
        const unsigned char *const row = smem + stage * kTile * kRowBytes + lane * kRowBytes;
#pragma unroll
        for (int c = 0; c < kChunks / 2; ++c) {
            const uint4 q = *reinterpret_cast<const uint4 *>(row + ((c ^ (lane & 7)) << 4));
            const uint4 p = *reinterpret_cast<const uint4 *>(row + (((c + kChunks / 2) ^ (lane & 7)) << 4));
            const uint32_t w0[4] = {q.x, q.y, q.z, q.w}, w1[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int i = 0; i < (kBf16 ? 8 : 4); ++i) {
                const int k = (kBf16 ? 8 : 4) * c + i;
                const uint32_t ra = !kBf16 ? w0[i & 3] : (i & 1) ? w0[i >> 1] & 0xffff0000u : w0[i >> 1] << 16;
                const uint32_t rb = !kBf16 ? w1[i & 3] : (i & 1) ? w1[i >> 1] & 0xffff0000u : w1[i >> 1] << 16;
                const float a = __uint_as_float(ra ^ flip_of<kDefault>(mask, k));
                const float b = __uint_as_float(rb ^ flip_of<kDefault>(mask, k + 64));
                const f32x2 ab = pk2(a, b);
                acc[k & 3] = fma2(ab, ab, acc[k & 3]);
                P[k] = pk2(__fadd_rn(a, b), __fsub_rn(a, b));
            }
        }
        __syncwarp();
        if (kStages == 1) {
            if (item + 1 < end) fetch(tile * kTile, hk, 0);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        float n2;
        {
            float a, b;
            upk2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a, b);
            n2 = __fadd_rn(a, b);
        }
        stages_between(P);
        float mm[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 64; ++k) {
            float a, b;
            upk2(P[k], a, b);
            mm[k & 3] = max3(mm[k & 3], fabsf(a), fabsf(b));
        }
        const float m = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
        const bool zero = m == 0.0f && n2 == 0.0f;  // (m alone is 0 too where z overflowed to NaN throughout)
        const float norm = zero ? 1e-8f : __fsqrt_rn(n2);
        const float scale = zero ? 1e-8f : __fmul_rn(__fdiv_rn(m, norm), tq3::fwht_post());
        const float r = zero ? 1.0f : __frcp_rn(m);
        const f32x2 R = pk2(r, r);
        const f32x2 Q1 = pk2(tq3::q_coef(1), tq3::q_coef(1)), Q3 = pk2(tq3::q_coef(3), tq3::q_coef(3)),
                    Q5 = pk2(tq3::q_coef(5), tq3::q_coef(5));
        const f32x2 KK = pk2(8388612.0f, 8388612.0f), NC = pk2(-8388609.0f, -8388609.0f), HALF = pk2(3.5f, 3.5f);
        f32x2 W[8];  // 8^j-weighted sums of the indices: group g (low) and group g + 8 (high), exact below 2^24
#pragma unroll
        for (int g = 0; g < 8; ++g) W[g] = 0ull;
        float far[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < 64; ++kk) {
            const int j = kk >> 3, k = 8 * (kk & 7) + j;
            const float w8 = __uint_as_float((127u + 3u * j) << 23);  // 8^j
            const f32x2 u = mul2(P[k], R);
            const f32x2 u2 = mul2(u, u);
            const f32x2 h = fma2(fma2(Q5, u2, Q3), u2, Q1);
            const f32x2 idx = add2(tq3::fma2_rp(h, u, KK), NC);  // 3 + ceil(Q(u))
            W[k >> 3] = fma2(pk2(w8, w8), idx, W[k >> 3]);
            float a, b;  // Q + 1/2 - ceil(Q): beyond kNear, an integer is near
            upk2(fma2(h, u, sub2(HALF, idx)), a, b);
            far[kk & 3] = max3(far[kk & 3], fabsf(a), fabsf(b));
        }
        const float f = fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3]));
        const bool redo = !zero && !(f < kNear && n2 > 1.1e-16f && n2 < 1e37f);

        {
            uint32_t *const rec = recs + 14 * lane;
            uint32_t g24[16];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                float lo, hi;
                upk2(W[g], lo, hi);
                g24[g] = __float2uint_rn(lo);
                g24[g + 8] = __float2uint_rn(hi);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                rec[3 * q] = g24[4 * q] | (g24[4 * q + 1] << 24);
                rec[3 * q + 1] = (g24[4 * q + 1] >> 8) | (g24[4 * q + 2] << 16);
                rec[3 * q + 2] = (g24[4 * q + 2] >> 16) | (g24[4 * q + 3] << 8);
            }
            rec[12] = __float_as_uint(norm);
            rec[13] = __float_as_uint(scale);
        }
        __syncwarp();
        for (uint32_t todo = __ballot_sync(0xffffffffu, redo && slot >= 0 && slot < n_slots); todo; todo &= todo - 1) {
            const int who = __ffs(todo) - 1;
            encode_row_fp64<kBf16>(row_of(here, t0 + who), mask, recs + 14 * who);
        }
        __syncwarp();
        int64_t at = -1;
        if (slot >= n_slots) atomicOr(&g_fault, tq3::kFaultPoolIndex);
        if (slot >= 0 && slot < n_slots)
            at = record_at(pools, slot >> pools.shift, here >> 1, slot & ((int64_t(1) << pools.shift) - 1));
        uint8_t *const pool = (here & 1) ? pools.v : pools.k;
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            const int piece = i * 32 + lane, v = piece / 7, part = piece % 7;
            const int64_t to = __shfl_sync(0xffffffffu, at, v);
            if (to >= 0)
                *reinterpret_cast<uint2 *>(pool + to + 8 * part) =
                    *reinterpret_cast<const uint2 *>(recs + 14 * v + 2 * part);
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------------------------
struct Dense {
    unsigned char *k, *v;  // [tokens][heads][128]
    int64_t tokens;
    const int32_t *table, *start;
    int64_t batch, pages_per_seq;
};

// The record of this lane's token, or -1 (past the last sequence: `skip`; outside the pool or the
// table: zeros and a fault).
__device__ __forceinline__ int64_t place_of(const Dense &d, const Pools &p, int64_t token, bool &skip) {
    skip = true;
    if (token >= d.tokens || token < __ldg(d.start) || token >= __ldg(d.start + d.batch)) return -1;
    int64_t lo = 0, hi = d.batch;  // start[lo] <= token < start[hi]
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        (token < __ldg(d.start + mid) ? hi : lo) = mid;
    }
    skip = false;
    const int64_t j = token - __ldg(d.start + lo), in_page = j & ((int64_t(1) << p.shift) - 1);
    if (j < 0 || (j >> p.shift) >= d.pages_per_seq) return -1;
    const int64_t page = __ldg(d.table + lo * d.pages_per_seq + (j >> p.shift));
    if (page < 0 || page >= p.n_pages) return -1;
    return (page * p.heads << p.shift) + in_page;  // head 0; head h is h pages' worth further
}

template <bool kBf16, bool kDefault>
__global__ void __launch_bounds__(kTile, kReadCtas) read_kernel(Dense d, Pools pools, SignMask mask) {
    constexpr int kRowBytes = kBf16 ? 256 : 512, kChunks = kRowBytes / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x;
    const float cb = tq3::centroid((uint32_t)(lane & 7));  // lane l holds centroid l mod 8
    const int per_tile = 2 * pools.heads;
    const int64_t items = (d.tokens + kTile - 1) / kTile * per_tile;
    // a contiguous share of the items: the tokens' places are found once per tile
    const int64_t begin = items * blockIdx.x / gridDim.x, end = items * (blockIdx.x + 1) / gridDim.x;
    if (begin >= end) return;

    int64_t tile = begin / per_tile, place = -1;
    int hk = (int)(begin - tile * per_tile);
    bool skip = true;
    uint2 rec[7], next[7];
    auto locate = [&]() {
        place = place_of(d, pools, tile * kTile + lane, skip);
        if (!skip && place < 0) atomicOr(&g_fault, tq3::kFaultPoolIndex);
    };
    auto load = [&](uint2 (&r)[7]) {
        const uint8_t *const src = ((hk & 1) ? pools.v : pools.k) + (place + ((int64_t)(hk >> 1) << pools.shift)) * kRec;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            r[i] = place >= 0 ? __ldg(reinterpret_cast<const uint2 *>(src) + i) : make_uint2(0u, 0u);
    };
    locate();
    load(next);
    for (int64_t item = begin; item < end; ++item) {
#pragma unroll
        for (int i = 0; i < 7; ++i) rec[i] = next[i];
        const int64_t t0 = tile * kTile;
        const uint32_t live = __ballot_sync(0xffffffffu, !skip);
        const int here = hk;
        if (item + 1 < end) {
            if (++hk == per_tile) {
                hk = 0;
                ++tile;
                locate();
            }
            load(next);
        }
        // RN(centroid * scale), stage h = 1 (scalar: a packed product must not feed a packed sum), then
        // stages 2 .. 64
        const float norm = __uint_as_float(rec[6].x), scale = __uint_as_float(rec[6].y);
        uint32_t w[13];
#pragma unroll
        for (int i = 0; i < 6; ++i) w[2 * i] = rec[i].x, w[2 * i + 1] = rec[i].y;
        w[12] = 0;
        f32x2 P[64];
#pragma unroll
        for (int k = 0; k < 64; ++k) {
            const int o = 6 * k;
            const uint32_t ia = __funnelshift_r(w[o >> 5], w[(o >> 5) + 1], o & 31);
            const uint32_t ib = __funnelshift_r(w[(o + 3) >> 5], w[((o + 3) >> 5) + 1], (o + 3) & 31);
            const float a = __fmul_rn(__shfl_sync(0xffffffffu, cb, (int)ia), scale);
            const float b = __fmul_rn(__shfl_sync(0xffffffffu, cb, (int)ib), scale);
            P[k] = pk2(__fadd_rn(a, b), __fsub_rn(a, b));
        }
        stages_between(P);
        const f32x2 C = pk2(tq3::fwht_post(), tq3::fwht_post());
        const f32x2 N = pk2(norm, norm);
        unsigned char *const row = smem + lane * kRowBytes;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < (kBf16 ? 4 : 2); ++i) {
                const int k = (kBf16 ? 4 : 2) * c + i;
                float a, b;
                upk2(mul2(mul2(P[k], C), N), a, b);
                a = __uint_as_float(__float_as_uint(a) ^ flip_of<kDefault>(mask, 2 * k));
                b = __uint_as_float(__float_as_uint(b) ^ flip_of<kDefault>(mask, 2 * k + 1));
                if (kBf16) {
                    o[i] = pack_bf16x2(a, b);
                } else {
                    o[2 * i] = __float_as_uint(a);
                    o[2 * i + 1] = __float_as_uint(b);
                }
            }
            *reinterpret_cast<uint4 *>(row + ((c ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        unsigned char *const out = ((here & 1) ? d.v : d.k) + (t0 * pools.heads + (here >> 1)) * kRowBytes;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int at = i * 32 + lane, r = at / kChunks, c = at % kChunks;
            if ((live >> r) & 1u)
                st_stream16(out + (int64_t)r * pools.heads * kRowBytes + 16 * c,
                            *reinterpret_cast<const uint4 *>(smem + r * kRowBytes + ((c ^ (r & 7)) << 4)));
        }
        __syncwarp();
    }
}

unsigned int read_and_clear_fault() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof v) != cudaSuccess) return 0x80000000u;
    if (v) cudaMemcpyToSymbol(g_fault, &zero, sizeof zero);
    return v;
}

template <typename... K, typename... A>
wq_status launch(void (*kernel)(K...), unsigned grid, int threads, size_t smem, cudaStream_t s, A... args) {
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), smem)) return WQ_ERR_CUDA;
    kernel<<<grid, threads, smem, s>>>(args...);
    return launch_status();
}

inline unsigned grid_for(int64_t items, int per_sm) {
    const int64_t most = (int64_t)kSms * per_sm;
    return (unsigned)(items < most ? items : most);
}

}  // namespace tq3_cache
}  // namespace wq

using namespace wq;

extern "C" wq_status tq3_cache_append(const void *k, const void *v, int dtype, int64_t tokens, int64_t kv_heads,
                                      int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                      int64_t v_head_stride, const uint32_t *sign_mask, const int64_t *slots,
                                      uint8_t *k_pool, uint8_t *v_pool, int64_t n_pages, int64_t page_size,
                                      void *stream) {
    if (tokens < 0 || tokens > (int64_t(1) << 40)) return WQ_ERR_SHAPE;
    if (!tq3_cache::pool_shape_ok(n_pages, kv_heads, page_size)) return WQ_ERR_SHAPE;
    if (!valid_dtype(dtype)) return WQ_ERR_DTYPE;
    const int64_t most = int64_t(1) << 40;  // the strides' products with the counts stay within int64
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (s < 0 || s > most || (tokens && s > (int64_t(1) << 59) / tokens)) return WQ_ERR_SHAPE;
    if (tokens == 0) return WQ_OK;
    if (!k || !v || !sign_mask || !slots || !k_pool || !v_pool) return WQ_ERR_NULL;
    const int64_t size = dtype_size(dtype);
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (s * size % 16) return WQ_ERR_ALIGN;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(k_pool, 16) ||
        !aligned(v_pool, 16))
        return WQ_ERR_ALIGN;
    tq3::SignMask m;
    for (int i = 0; i < 4; ++i) m.w[i] = sign_mask[i];
    const tq3_cache::Pools pools{k_pool, v_pool, n_pages, (int)kv_heads, tq3_cache::page_shift(page_size)};
    const tq3_cache::Rows rows{static_cast<const unsigned char *>(k), static_cast<const unsigned char *>(v),
                               k_token_stride * size, k_head_stride * size, v_token_stride * size,
                               v_head_stride * size};
    const unsigned grid = tq3_cache::grid_for((tokens + 31) / 32 * kv_heads * 2, 1);
    using namespace tq3_cache;
    constexpr int threads = 32 * kAppendWarps;
    const size_t smem = kAppendWarps * kAppendBytes;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool def = tq3::is_default(m);
    if (dtype == WQ_BF16 && def)
        return launch(append_kernel<true, true>, grid, threads, smem, s, rows, tokens, slots, pools, m);
    if (dtype == WQ_BF16)
        return launch(append_kernel<true, false>, grid, threads, smem, s, rows, tokens, slots, pools, m);
    if (def)
        return launch(append_kernel<false, true>, grid, threads, smem, s, rows, tokens, slots, pools, m);
    return launch(append_kernel<false, false>, grid, threads, smem, s, rows, tokens, slots, pools, m);
}

extern "C" wq_status tq3_cache_read(const uint8_t *k_pool, const uint8_t *v_pool, int64_t n_pages, int64_t kv_heads,
                                    int64_t page_size, const int32_t *page_table, int64_t batch,
                                    int64_t pages_per_seq, const int32_t *seq_start, int64_t n_tokens,
                                    const uint32_t *sign_mask, void *k_out, void *v_out, int out_dtype,
                                    void *stream) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || batch < 0 || batch > INT32_MAX || pages_per_seq < 0 ||
        pages_per_seq > (int64_t(1) << 31))
        return WQ_ERR_SHAPE;
    if (!tq3_cache::pool_shape_ok(n_pages, kv_heads, page_size)) return WQ_ERR_SHAPE;
    if (!valid_dtype(out_dtype)) return WQ_ERR_DTYPE;
    if (n_tokens == 0 || batch == 0) return WQ_OK;
    if (!k_pool || !v_pool || !page_table || !seq_start || !sign_mask || !k_out || !v_out) return WQ_ERR_NULL;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) || !aligned(seq_start, 4) ||
        !aligned(k_out, 16) || !aligned(v_out, 16))
        return WQ_ERR_ALIGN;
    tq3::SignMask m;
    for (int i = 0; i < 4; ++i) m.w[i] = sign_mask[i];
    const tq3_cache::Pools pools{const_cast<uint8_t *>(k_pool), const_cast<uint8_t *>(v_pool), n_pages, (int)kv_heads,
                                 tq3_cache::page_shift(page_size)};
    const tq3_cache::Dense d{static_cast<unsigned char *>(k_out), static_cast<unsigned char *>(v_out), n_tokens,
                             page_table, seq_start, batch, pages_per_seq};
    const unsigned grid = tq3_cache::grid_for((n_tokens + 31) / 32 * kv_heads * 2, tq3_cache::kReadCtas);
    const size_t smem = 32 * (out_dtype == WQ_BF16 ? 256 : 512);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool def = tq3::is_default(m);
    if (out_dtype == WQ_BF16 && def)
        return tq3_cache::launch(tq3_cache::read_kernel<true, true>, grid, 32, smem, s, d, pools, m);
    if (out_dtype == WQ_BF16)
        return tq3_cache::launch(tq3_cache::read_kernel<true, false>, grid, 32, smem, s, d, pools, m);
    if (def)
        return tq3_cache::launch(tq3_cache::read_kernel<false, true>, grid, 32, smem, s, d, pools, m);
    return tq3_cache::launch(tq3_cache::read_kernel<false, false>, grid, 32, smem, s, d, pools, m);
}

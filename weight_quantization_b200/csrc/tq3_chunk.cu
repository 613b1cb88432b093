// Attention of ragged chunks of new tokens over a batch's paged TQ3 cache (page "tq3_core.py": the
// cache is what tq3_quantize compresses and tq3_dequantize restores), causal, optionally with a
// sliding window and first tokens that stay visible. How the work is cut and joined is in
// tq3_chunk.cuh; this file has the entry point and the kernel for few rows.
//
// With q~ = H (s . q), f_j = norm_j scale_j of key j and g_j that of value j (post = 128^-1/2):
//     logit_ij = softmax_scale post f_j (q~_i . c[idx_j]),
//     out_i    = s . H(sum_j p_ij g_j c[idx'_j]) post / sum_j p_ij,   p_ij = exp(logit_ij - max_i),
// so both products are over centroids alone: 8 values, looked up as pairs (6 bits) in a table that
// every lane has a column of in shared memory (a bank of its own, so no conflict).
//
// The rows kernel: a warp takes 32 keys at a time and 8 rows of one KV head.
// S^T = C_K q~^T and O^T += C_V^T w with m16n8k16: the looked-up pairs are the A operands as they are
// (the 128 coordinates may be summed in any order, so a lane takes the coordinates whose bits it can
// read as whole words), and no decoded key or value ever leaves the registers. In log2 units the
// weights are taken as w_ij = 2^(s_ij + log2 g_j - M_i), which folds the value's factor into the
// exponent, keeps w within fp16's range whatever the norms are, and leaves sum_j w_ij / g_j as the
// softmax's denominator. M_i is raised only when it is passed by 2^8.
//
// Operands are fp16: the centroids times kGain are within 1.4e-5 of fp16 numbers, a row of q~ is scaled by a
// power of two of its own and rounded (2^-11 of each coordinate at most, so a logit moves by
// 2^-11 softmax_scale |q| |k_j| at most), w likewise (2^-11 of a term). A bf16 result is rounded to 2^-8
// afterwards. For fp32 queries or results every operand is split into fp16 hi + lo (2^-22) and a product
// takes three passes, hi hi + hi lo + lo hi. Sums are fp32.
//
// Measured: one token of 8 sequences of 32768 keys, 8 KV heads x 4 rows, bf16: 99 us with the join, 2.4 TB/s
// of records where a copy reaches 6.55. A step of 32 keys is 988 warp instructions, of which the 128 lookups
// are 500; the issue slots are 66% busy, the ALU 61%, the shared-memory pipe 57%, the tensor cores 17%. With fp32
// on either side, 158 us: two CTAs an SM, three passes. Three
// CTAs of more registers in place of four take as long; right shifts as high halves of multiplications, to
// spare the ALU, 108 us; keys ordered so that no record read meets a bank twice, no change.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <cuda_fp16.h>

#include "common.cuh"
#include "tq3_cache.cuh"
#include "tq3_chunk.cuh"
#include "tq3_common.cuh"

namespace wq {
namespace tq3_chunk_mma {  // tq3_chunk_mma.cu
int64_t workspace();
wq_status run(const tq3_chunk::Args &a, bool wide, const tq3_chunk::Args &few, int few_ctas, cudaStream_t s);
unsigned int read_and_clear_fault();
}  // namespace tq3_chunk_mma
namespace tq3_chunk {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kSub = kTileKeys / kWarps;  // keys of a warp's step
constexpr int kPiece = 16;                // keys of an m16n8k16's rows; a copy within a page
static_assert(kSub == 2 * kPiece, "two pieces a step, a lane per key");
constexpr int kStages = 3;
constexpr int kFewRows = 8;  // rows of a block; with more per KV head a sequence may go to the tensor-core kernel
constexpr int kPieceBytes = kPiece * tq3_cache::kRec;
constexpr int kStageBytes = 4 * kPieceBytes;  // a step's key records, then its value records
constexpr float kLazy = 8.0f;   // M_i is raised past this margin (log2 units)
constexpr float kLift = 6.0f;   // weights are at most 2^(kLazy + kLift) < 65504, so 2^-20 of the largest is still normal
constexpr float kTiny = 0x1p-100f;  // least g_j: a zero vector weighs 2^-100 instead

__device__ unsigned int g_fault;

// Shared memory of the rows kernel.
template <bool kWide>
struct Layout {
    static constexpr int kRows = kFewRows;
    static constexpr int kTable = kWide ? 64 * 32 * 8 : 64 * 32 * 4;
    static constexpr int kQ = kRows * 136;  // halves, rows padded by 16 bytes
    // a warp's stages; between segments, its rows' sums (132 floats a row)
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kOffStage = kTable;
    static constexpr int kOffFactor = kOffStage + kWarps * kWarpBytes;  // per warp and key of a step
    static constexpr int kOffQ = kOffFactor + kWarps * kSub * 16;
    static constexpr int kOffStat = kOffQ + (kWide ? 2 : 1) * kQ * 2;  // per warp and row: M, l
    static constexpr int kOffDown = kOffStat + kWarps * kRows * 8;     // per row: from its fp16 q~ to q~, times 2^-12
    static constexpr int kOffInfo = kOffDown + kRows * 4;              // per warp and stage
    static constexpr int kOffScratch = kOffInfo + kWarps * kStages * 8;
    static constexpr int kBytes = kOffScratch + (kWarps + 4) * 8;
    static_assert(kRows * 132 * 4 <= kWarpBytes, "a warp's sums fit its stages");
    static_assert(kOffQ % 16 == 0 && kOffInfo % 8 == 0 && kOffScratch % 8 == 0 && kBytes <= 227 * 1024, "layout");
};

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// x - hi for the two halves of hi = pack_half2(a, b), as a pair again.
__device__ __forceinline__ uint32_t residue_half2(float a, float b, uint32_t hi) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return pack_half2(__fsub_rn(a, h.x), __fsub_rn(b, h.y));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A pair of centroids: hi, and lo where the operands are split.
template <bool kWide>
struct Pair {
    uint32_t hi, lo;
};
// The pair whose 6 bits are bits 7 .. 12 of x; `column` is this lane's column of the table.
template <bool kWide>
__device__ __forceinline__ Pair<kWide> lookup(const unsigned char *table, uint32_t column, uint32_t x) {
    Pair<kWide> p;
    if (kWide) {
        const uint2 v = *reinterpret_cast<const uint2 *>(table + (((x & 0x1f80u) << 1) | column));
        p.hi = v.x, p.lo = v.y;
    } else {
        p.hi = *reinterpret_cast<const uint32_t *>(table + ((x & 0x1f80u) | column));
        p.lo = 0;
    }
    return p;
}
// Bits o .. o + 5 of the words w, moved to bits 7 .. 12.
template <int N>
__device__ __forceinline__ uint32_t field(const uint32_t (&w)[N], int o) {
    const int q = o >> 5, s = o & 31;
    if (s < 7) return w[q] << (7 - s);
    return s > 26 ? __funnelshift_r(w[q], w[q + 1 < N ? q + 1 : q], s - 7) : w[q] >> (s - 7);
}

template <bool kWide>
__device__ __forceinline__ void product(float (&d)[4], const Pair<kWide> &a0, const Pair<kWide> &a1,
                                        const Pair<kWide> &a2, const Pair<kWide> &a3, const uint32_t (&hi)[2],
                                        const uint32_t (&lo)[2]) {
    mma16816(d, a0.hi, a1.hi, a2.hi, a3.hi, hi[0], hi[1]);
    if (kWide) {
        mma16816(d, a0.lo, a1.lo, a2.lo, a3.lo, hi[0], hi[1]);
        mma16816(d, a0.hi, a1.hi, a2.hi, a3.hi, lo[0], lo[1]);
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ int64_t shfl64(int64_t v, int from) {
    const uint32_t lo = __shfl_sync(0xffffffffu, (uint32_t)v, from),
                   hi = __shfl_sync(0xffffffffu, (uint32_t)((uint64_t)v >> 32), from);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// A warp's stream of 32-key steps through its stages: one group of asynchronous copies a step. Pieces
// are looked up 32 at a time (16 steps), a lane each.
struct Steps {
    uint32_t stage;  // shared address of kStages of kStageBytes
    uint2 *info;     // per stage: the keys that have a page, the step's first key
    uint32_t issued, used;
    // of the segment
    int b, head, take, last, from, until;
    // of the 32 pieces in hand: steps that are still to be requested (bit 2 i), and this lane's piece
    int base;
    uint32_t todo;
    int j;
    int64_t at;  // byte offset in its pool, -1 without a page

    __device__ __forceinline__ bool seen(int j0, int n) const { return j0 <= last && (j0 + n > from || j0 < until); }

    template <class W>
    __device__ __forceinline__ void begin(const W &w, int p_hi) {
        b = w.b, head = w.head, take = w.take(), last = p_hi, from = w.span.from, until = w.span.until;
        base = 0, todo = 0;
    }
    // The offset of key j0's page and place in it, or -1 with the fault bit set.
    __device__ __forceinline__ int64_t locate(const Args &a, int j0) const {
        const int32_t page = __ldg(a.table + b * a.pages_per_seq + (j0 >> a.pools.shift));
        if (page >= 0 && page < a.pools.n_pages)
            return tq3_cache::record_at(a.pools, page, head, j0 & ((1 << a.pools.shift) - 1));
        atomicOr(&g_fault, tq3::kFaultPoolIndex);
        return -1;
    }
    template <class W>
    __device__ __forceinline__ void gather(const Args &a, const W &w, int warp, int lane) {
        const int i = base + (lane >> 1);
        bool need = false;
        at = -1;
        j = 0;
        if (i < take) {
            j = w.span.tile(w.tile + i) * kTileKeys + warp * kSub + (lane & 1) * kPiece;
            need = seen(j, kPiece);
            if (need && a.pools.shift >= 4) at = locate(a, j);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, need);
        todo = (m | m >> 1) & 0x55555555u;
        base += 16;
    }
    // Fills the free stages. Every call commits as many groups as make kStages - 1 of them follow the
    // step that is used next, empty ones at the end of a segment.
    template <class W>
    __device__ __forceinline__ void request(const Args &a, const W &w, int warp, int lane, int steps) {
        for (int k = 0; k < steps; ++k) {
            while (todo == 0 && base < take) gather(a, w, warp, lane);
            if (todo) {
                const int p = __ffs(todo) - 1, st = issued % kStages;
                todo &= todo - 1;
                const int j0 = __shfl_sync(0xffffffffu, j, p);
                const uint32_t keys = a.pools.shift >= 4 ? copy_pieces(a, st, p, lane) : copy_small(a, st, j0, lane);
                if (lane == 0) info[st] = make_uint2(keys, (uint32_t)j0);
                ++issued;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    // Two pieces of 16 keys, each within a page, in 16-byte chunks: 56 of each piece in either pool.
    // Shared: key pieces 0 and 1, value pieces 0 and 1.
    __device__ __forceinline__ uint32_t copy_pieces(const Args &a, int st, int p, int lane) const {
        const int64_t a0 = shfl64(at, p), a1 = shfl64(at, p + 1);
        const uint32_t b0 = a0 >= 0 ? 16 : 0, b1 = a1 >= 0 ? 16 : 0;  // nothing is read for 0 bytes
        const int64_t o0 = (a0 >= 0 ? a0 : 0) + 16 * lane, o1 = (a1 >= 0 ? a1 : 0) + 16 * lane;
        const uint8_t *const k0 = a.pools.k + o0, *const k1 = a.pools.k + o1;
        const uint8_t *const v0 = a.pools.v + o0, *const v1 = a.pools.v + o1;
        const uint32_t dst = stage + st * kStageBytes + 16 * lane;
        cp_async16(dst, k0, b0);
        cp_async16(dst + 512, lane < 24 ? k0 + 512 : k1 + 512 - kPieceBytes, lane < 24 ? b0 : b1);
        cp_async16(dst + 1024, k1 + 1024 - kPieceBytes, b1);
        cp_async16(dst + 1536, lane < 16 ? k1 + 1536 - kPieceBytes : v0 + 1536 - 2 * kPieceBytes, lane < 16 ? b1 : b0);
        cp_async16(dst + 2048, v0 + 2048 - 2 * kPieceBytes, b0);
        cp_async16(dst + 2560, lane < 8 ? v0 + 2560 - 2 * kPieceBytes : v1 + 2560 - 3 * kPieceBytes, lane < 8 ? b0 : b1);
        cp_async16(dst + 3072, v1 + 3072 - 3 * kPieceBytes, b1);
        return (a0 >= 0 ? 0xffffu : 0u) | (a1 >= 0 ? 0xffff0000u : 0u);
    }
    // 32 keys in pages of 1 to 8 places, a page a lane, in 8-byte chunks (a lone record is not a multiple
    // of 16 bytes).
    __device__ __forceinline__ uint32_t copy_small(const Args &a, int st, int j0, int lane) const {
        const int shift = a.pools.shift, size = 1 << shift, jp = j0 + (lane << shift);
        const int64_t mine = lane < (kSub >> shift) && seen(jp, size) ? locate(a, jp) : -1;
#pragma unroll 1
        for (int i = 0; i < kStageBytes / 256; ++i) {
            const int c = 32 * i + lane, tensor = c / (7 * kSub), r = c % (7 * kSub) / 7, word = c % 7;
            const int64_t from_at = shfl64(mine, r >> shift);
            const uint8_t *const src = (tensor ? a.pools.v : a.pools.k) +
                                       (from_at >= 0 ? from_at + (r & (size - 1)) * tq3_cache::kRec + 8 * word : 0);
            cp_async8(stage + st * kStageBytes + 8 * c, src, from_at >= 0 ? 8 : 0);
        }
        return __reduce_or_sync(0xffffffffu, mine >= 0 ? ((1u << size) - 1u) << (lane << shift) : 0u);
    }
};
constexpr int kAhead = kStages - 1;  // steps requested beyond the one in use

template <bool kWide>
__global__ void __launch_bounds__(kThreads, kWide ? 2 : 4) rows_kernel(const __grid_constant__ Args a) {
    using L = Layout<kWide>;
    constexpr int R = L::kRows;
    // centroids times kGain: for one fp16 the gain at which all four magnitudes are nearest to fp16 numbers
    constexpr float kGain = kWide ? 16.0f : 1.6196665f;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    unsigned char *const table = smem;
    const uint32_t column = lane * (kWide ? 8 : 4);
    __half *const qs = reinterpret_cast<__half *>(smem + L::kOffQ);
    float4 *const factor = reinterpret_cast<float4 *>(smem + L::kOffFactor) + warp * kSub;
    float *const stat = reinterpret_cast<float *>(smem + L::kOffStat);
    float *const downs = reinterpret_cast<float *>(smem + L::kOffDown);

    for (int i = tid; i < 64 * 32; i += kThreads) {
        const uint32_t f = i >> 5;
        const float x = __fmul_rn(tq3::centroid(f & 7u), kGain), y = __fmul_rn(tq3::centroid(f >> 3), kGain);
        const uint32_t hi = pack_half2(x, y);
        if (kWide)
            reinterpret_cast<uint2 *>(table)[i] = make_uint2(hi, residue_half2(x, y, hi));
        else
            reinterpret_cast<uint32_t *>(table)[i] = hi;
    }
    Steps steps;
    unsigned char *const stages = smem + L::kOffStage + warp * L::kWarpBytes;
    steps.stage = smem_u32(stages);
    steps.info = reinterpret_cast<uint2 *>(smem + L::kOffInfo) + warp * kStages;
    steps.issued = steps.used = 0;
    Walk<R, kThreads> w;
    pdl_wait();  // what follows reads what earlier kernels wrote
    w.start(a, reinterpret_cast<int64_t *>(smem + L::kOffScratch));
    pdl_trigger();
    Cut *const cut = reinterpret_cast<Cut *>(a.ws + (int64_t)blockIdx.x * kCutBytes);
    if (tid == 0) cut->cut = 0;
    if (blockIdx.x == 0)
        for (int b = tid; b < a.batch; b += kThreads)
            if (__ldg(a.kv_len + b) > a.max_keys) atomicOr(&g_fault, tq3::kFaultPoolIndex);

    float sg[4];
    lane_signs(a, lane, sg);
    for (; !w.done(); w.next(a)) {
        const Seq s = w.seq;
        const int rows = s.new_tokens * a.group, r0 = w.block * R, before = s.keys - s.new_tokens;
        const int p_lo = before + token_of(a, r0), p_hi = before + token_of(a, min(r0 + R, rows) - 1);
        const int take = w.take();

        steps.begin(w, p_hi);
        steps.request(a, w, warp, lane, kAhead);

        // q~ of the block's rows, each scaled by the power of two that brings its largest to 2^13 .. 2^14 (1 where
        // it is not finite): a row keeps its bits whatever the size of the others
        {
            constexpr int kEach = R / kWarps;
            float v[kEach][4];
            int row[kEach];  // a row behind the last one repeats it, and counts as zeros
#pragma unroll
            for (int n = 0; n < kEach; ++n) row[n] = min(r0 + kWarps * n + warp, rows - 1);
            load_rows<kEach, !kWide>(a, s, w.head, row, lane, v);
#pragma unroll
            for (int n = 0; n < kEach; ++n) {
                const int r = kWarps * n + warp;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[n][i] = r0 + r < rows ? __fmul_rn(v[n][i], sg[i]) : 0.0f;
                row_fwht(v[n], lane);
                const float m = fmaxf(fmaxf(fabsf(v[n][0]), fabsf(v[n][1])), fmaxf(fabsf(v[n][2]), fabsf(v[n][3])));
                const int e = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(m)) >> 23);
                const int up_exp = e == 255 ? 127 : min(253, 267 - e);
                const float up = __uint_as_float((uint32_t)up_exp << 23);
                if (lane == 0) downs[r] = __fmul_rn(__uint_as_float((uint32_t)(254 - up_exp) << 23), 0x1p-12f);
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __fmul_rn(v[n][i], up);
                uint2 hi = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
                __half *const to = qs + r * 136 + 4 * lane;
                *reinterpret_cast<uint2 *>(to) = hi;
                if (kWide)
                    *reinterpret_cast<uint2 *>(to + L::kQ) =
                        make_uint2(residue_half2(x[0], x[1], hi.x), residue_half2(x[2], x[3], hi.y));
            }
            __syncthreads();
        }
        // (2^12 with the key's factor and 2^-12 with the row's, so that the row's times S stays finite)
        const float coef = __fmul_rn(a.coef, 4096.0f / kGain);
        // lane (g, t): row g, coordinates 32 t .. 32 t + 31, as the B operands of eight products
        uint32_t qh[8][2], ql[kWide ? 8 : 1][2];
        int p[2];  // of rows 2 t and 2 t + 1: positions, scales
        float down[2];
        const __half *const from = qs + g * 136 + 32 * t;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint2 x = *reinterpret_cast<const uint2 *>(from + 4 * j);
            qh[j][0] = x.x, qh[j][1] = x.y;
            if (kWide) {
                const uint2 y = *reinterpret_cast<const uint2 *>(from + L::kQ + 4 * j);
                ql[kWide ? j : 0][0] = y.x, ql[kWide ? j : 0][1] = y.y;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r0 + 2 * t + e;
            p[e] = r < rows ? before + token_of(a, r) : -1;
            down[e] = downs[2 * t + e];
        }
        // the first and the second three bytes of a lane's 48 bits in the two words that hold them
        const uint32_t first = (g & 1) ? 0x5432u : 0x3210u, second = (g & 1) ? 0x7765u : 0x6543u;
        float acc[8][4], M[2], l[2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
        M[0] = M[1] = -FLT_MAX;
        l[0] = l[1] = 0.0f;

        while (steps.used != steps.issued) {
            steps.request(a, w, warp, lane, 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            __syncwarp();
            const int st = steps.used % kStages;
            const uint32_t *const rec = reinterpret_cast<const uint32_t *>(stages + st * kStageBytes);
            const uint32_t *const vrec = rec + 14 * kSub;
            const uint2 mine = steps.info[st];
            const int j0 = (int)mine.y;
            // key `lane`: the logit's factor, log2 of the value's and its reciprocal; one without a page
            // weighs nothing, and neither its records nor an infinite factor reach a sum
            {
                const float2 fk = *reinterpret_cast<const float2 *>(rec + 14 * lane + 12),
                             fv = *reinterpret_cast<const float2 *>(vrec + 14 * lane + 12);
                float gv = __fmul_rn(fv.x, fv.y);
                gv = gv < kTiny ? kTiny : gv;
                float4 x = make_float4(__fmul_rn(__fmul_rn(fk.x, fk.y), coef), lg2(gv), rcp(gv), 0.0f);
                if (!(mine.x >> lane & 1u)) x = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
                factor[lane] = x;
            }
            __syncwarp();

            float S[2][4], live[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // keys g and g + 8 of the piece: words 3 t .. 3 t + 2 of the indices
                uint32_t ka[3], kb[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    ka[i] = rec[14 * (kPiece * x + g) + 3 * t + i], kb[i] = rec[14 * (kPiece * x + g + 8) + 3 * t + i];
#pragma unroll
                for (int e = 0; e < 4; ++e) S[x][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Pair<kWide> a0 = lookup<kWide>(table, column, field(ka, 12 * j)),
                                      a1 = lookup<kWide>(table, column, field(kb, 12 * j)),
                                      a2 = lookup<kWide>(table, column, field(ka, 12 * j + 6)),
                                      a3 = lookup<kWide>(table, column, field(kb, 12 * j + 6));
                    product<kWide>(S[x], a0, a1, a2, a3, qh[j], ql[kWide ? j : 0]);
                }
                const float4 fa = factor[kPiece * x + g], fb = factor[kPiece * x + g + 8];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float4 f = e == 0 ? fa : fb;
                    float s0, s1;
                    upk2(mul2(pk2(S[x][e], S[x][e + 1]), pk2(down[0], down[1])), s0, s1);
                    S[x][e] = __fmaf_rn(s0, f.x, f.y);
                    S[x][e + 1] = __fmaf_rn(s1, f.x, f.y);
                    live[x][e] = live[x][e + 1] = f.z;
                }
            }
            if (!(j0 + kSub <= p_lo + 1 && (a.window == 0 || j0 > p_hi - a.window || j0 + kSub <= a.sinks))) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + kPiece * x + g + 8 * (e >> 1), pos = p[e & 1];
                        const bool on = j <= pos && (a.window == 0 || j > pos - a.window || j < a.sinks);
                        if (!on) S[x][e] = -INFINITY, live[x][e] = 0.0f;
                    }
            }
            bool raise = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m = max3(fmaxf(S[0][e], S[0][e + 2]), S[1][e], S[1][e + 2]);
                raise |= m > __fadd_rn(M[e], kLazy);
            }
            if (__any_sync(0xffffffffu, raise)) {
                float alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = max3(fmaxf(S[0][e], S[0][e + 2]), S[1][e], S[1][e + 2]);
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    m = fmaxf(m, M[e]);
                    alpha[e] = ex2(__fsub_rn(M[e], m));
                    M[e] = m;
                    l[e] = __fmul_rn(l[e], alpha[e]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] = __fmul_rn(acc[i][e], alpha[e & 1]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t ph[2], pl[2];
                float w4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w4[e] = ex2(__fsub_rn(S[x][e], __fsub_rn(M[e & 1], kLift)));
                    l[e & 1] = __fmaf_rn(w4[e], live[x][e], l[e & 1]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = pack_half2(w4[2 * i], w4[2 * i + 1]);
                    ph[i] = transpose8x8(hi);
                    pl[i] = kWide ? transpose8x8(residue_half2(w4[2 * i], w4[2 * i + 1], hi)) : 0u;
                }
                // values of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9: coordinates 16 g .. 16 g + 15, bits 48 g
                // on, as two groups of 24 bits
                uint32_t v[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t *const at = vrec + 14 * (kPiece * x + 2 * t + (i & 1) + 8 * (i >> 1)) + (3 * g >> 1);
                    const uint32_t lo = at[0], hi = at[1];
                    v[i][0] = __byte_perm(lo, hi, first);
                    v[i][1] = __byte_perm(lo, hi, second);
                }
                // per group: pairs (key 2 t, key 2 t + 1) of one coordinate, even ones and odd ones
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    constexpr uint32_t even = 0x1c71c7u, odd = even << 3;
                    const uint32_t e0[1] = {(v[0][h] & even) | ((v[1][h] << 3) & odd)},
                                   o0[1] = {((v[0][h] >> 3) & even) | (v[1][h] & odd)},
                                   e1[1] = {(v[2][h] & even) | ((v[3][h] << 3) & odd)},
                                   o1[1] = {((v[2][h] >> 3) & even) | (v[3][h] & odd)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const Pair<kWide> a0 = lookup<kWide>(table, column, field(e0, 6 * c)),
                                          a1 = lookup<kWide>(table, column, field(o0, 6 * c)),
                                          a2 = lookup<kWide>(table, column, field(e1, 6 * c)),
                                          a3 = lookup<kWide>(table, column, field(o1, 6 * c));
                        product<kWide>(acc[4 * h + c], a0, a1, a2, a3, ph, pl);
                    }
                }
            }
            __syncwarp();  // the stage and the factors are free
            ++steps.used;
        }

        // join the warps: row r by warp r % kWarps. No copy is in flight, so a warp's sums lie where its
        // stages were
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = l[e];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
            const int r = 2 * t + e;
            if (g == 0) *reinterpret_cast<float2 *>(stat + 2 * (warp * R + r)) = make_float2(M[e], x);
            float *const to = reinterpret_cast<float *>(stages) + r * 132 + 16 * g;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2 *>(to + 2 * i) = make_float2(acc[i][e], acc[i][e + 2]);
        }
        __syncthreads();
        const bool whole = w.tile == 0 && take == w.segment();
        float *const slot = slot_at<R>(a, gridDim.x, 2 * blockIdx.x + (w.tile == 0));
        if (!whole && w.tile == 0 && tid == 0) *cut = w.cut_here();
#pragma unroll
        for (int n = 0; n < R / kWarps; ++n) {
            const int r = kWarps * n + warp;
            if (r0 + r >= rows) continue;
            float m = -FLT_MAX, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int x = 0; x < kWarps; ++x) m = fmaxf(m, stat[2 * (x * R + r)]);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float2 ml = *reinterpret_cast<const float2 *>(stat + 2 * (x * R + r));
                const float f = ex2(__fsub_rn(ml.x, m));
                const float4 o = *reinterpret_cast<const float4 *>(smem + L::kOffStage + x * L::kWarpBytes + r * 528 + 16 * lane);
                sum = __fmaf_rn(ml.y, f, sum);
                v[0] = __fmaf_rn(o.x, f, v[0]);
                v[1] = __fmaf_rn(o.y, f, v[1]);
                v[2] = __fmaf_rn(o.z, f, v[2]);
                v[3] = __fmaf_rn(o.w, f, v[3]);
            }
            const float f = sum == 0.0f ? 0.0f : __fmul_rn(__frcp_rn(sum), 1.0f / kGain);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], f);
            if (whole) {
                store_row<!kWide>(a, s, w.head, r0 + r, lane, sg, v);
            } else {
                *reinterpret_cast<float4 *>(slot + r * 128 + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
                if (lane == 0) slot[R * 128 + r] = sum == 0.0f ? -INFINITY : m, slot[R * 129 + r] = sum;
            }
        }
        __syncthreads();
    }
}

unsigned int read_and_clear_fault() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof v) != cudaSuccess) return 0x80000000u;
    if (v) cudaMemcpyToSymbol(g_fault, &zero, sizeof zero);
    return v | tq3_chunk_mma::read_and_clear_fault();
}

constexpr int kParts = 4 * kSms;
inline int64_t rows_workspace() { return (workspace_bytes<kFewRows>(kParts) + 15) & ~int64_t(15); }

template <bool kWide>
wq_status run_rows(const Args &a, cudaStream_t s) {
    using L = Layout<kWide>;
    if (!ensure_dynamic_smem(reinterpret_cast<const void *>(rows_kernel<kWide>), L::kBytes)) return WQ_ERR_CUDA;
    launch_pdl(rows_kernel<kWide>, kParts, kThreads, L::kBytes, s, a);
    return launch_status();
}

}  // namespace tq3_chunk
}  // namespace wq

using namespace wq;

extern "C" int64_t tq3_attention_chunk_workspace(int64_t max_q, int64_t group) {
    if (max_q < 0 || group < 1) return -1;
    return tq3_chunk::rows_workspace() + (max_q > tq3_chunk::kFewRows / group ? tq3_chunk_mma::workspace() : 0);
}

extern "C" wq_status tq3_attention_chunk(const void *q, int q_dtype, int64_t n_tokens, int64_t q_heads,
                                         int64_t q_token_stride, int64_t q_head_stride, const uint8_t *k_pool,
                                         const uint8_t *v_pool, int64_t n_pages, int64_t kv_heads, int64_t page_size,
                                         const int32_t *page_table, int64_t batch, int64_t pages_per_seq,
                                         const int32_t *q_start, const int32_t *kv_len, int64_t max_q, int64_t window,
                                         int64_t sinks, const uint32_t *sign_mask, float softmax_scale, void *out,
                                         int out_dtype, void *workspace, int64_t workspace_bytes, void *stream) {
    if (n_tokens < 0 || n_tokens > INT32_MAX || batch < 0 || batch > INT32_MAX || pages_per_seq < 0 ||
        pages_per_seq > (int64_t(1) << 31) || max_q < 0 || window < 0 || window > INT32_MAX || sinks < 0 ||
        sinks > INT32_MAX || !(fabsf(softmax_scale) < INFINITY))
        return WQ_ERR_SHAPE;
    if (!tq3_cache::pool_shape_ok(n_pages, kv_heads, page_size)) return WQ_ERR_SHAPE;
    if (q_heads < kv_heads || q_heads % kv_heads) return WQ_ERR_SHAPE;
    const int64_t group = q_heads / kv_heads;
    if (group > INT32_MAX || n_tokens > (INT32_MAX - 4096) / group) return WQ_ERR_SHAPE;
    const int64_t most = int64_t(1) << 40;
    for (int64_t s : {q_token_stride, q_head_stride})
        if (s < 0 || s > most || (n_tokens && s > (int64_t(1) << 59) / n_tokens)) return WQ_ERR_SHAPE;
    if (!valid_dtype(q_dtype) || !valid_dtype(out_dtype)) return WQ_ERR_DTYPE;
    if (n_tokens == 0 || batch == 0) return WQ_OK;
    if (!q || !k_pool || !v_pool || !page_table || !q_start || !kv_len || !sign_mask || !out || !workspace)
        return WQ_ERR_NULL;
    if (workspace_bytes < tq3_attention_chunk_workspace(max_q, group)) return WQ_ERR_SHAPE;
    const int64_t size = dtype_size(q_dtype);
    if (q_token_stride * size % 16 || q_head_stride * size % 16) return WQ_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) ||
        !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(out, 16) || !aligned(workspace, 16))
        return WQ_ERR_ALIGN;
    tq3_chunk::Args a;
    a.q = q, a.q_token = q_token_stride, a.q_head = q_head_stride;
    a.pools = tq3_cache::Pools{const_cast<uint8_t *>(k_pool), const_cast<uint8_t *>(v_pool), n_pages, (int)kv_heads,
                               tq3_cache::page_shift(page_size)};
    a.table = page_table, a.q_start = q_start, a.kv_len = kv_len, a.pages_per_seq = pages_per_seq;
    a.batch = (int)batch, a.n_tokens = (int)n_tokens;
    tq3_chunk::set_group(a, (int)group);
    a.max_keys = pages_per_seq > (tq3_chunk::kMaxKeys >> a.pools.shift) ? tq3_chunk::kMaxKeys
                                                                        : (int)(pages_per_seq << a.pools.shift);
    a.window = (int)window, a.sinks = (int)sinks;
    a.rows_from = 0, a.rows_to = INT32_MAX;
    // post * softmax_scale * log2(e), rounded once
    a.coef = (float)(0.08838834764831844055 * (double)softmax_scale * 1.4426950408889634074);
    for (int i = 0; i < 4; ++i) a.mask.w[i] = sign_mask[i];
    a.out = out, a.q_bf16 = q_dtype == WQ_BF16, a.out_bf16 = out_dtype == WQ_BF16;
    a.ws = static_cast<unsigned char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = !a.q_bf16 || !a.out_bf16;
    // Blocks of 8 rows share no decoding, and the tensor-core kernel takes 256 rows with one: a tile of 128 keys
    // costs the former 0.9 us of an SM per 8 rows, the latter 2.6 us whatever the rows are. But the latter also
    // needs some 25 us to set up, transform, join and drain, so it is left out where no sequence has more than
    // 8 rows, and where so little work is left (as far as the host knows: the tables' room stands for the
    // lengths) that the former has three steps a CTA at most, one for split operands. 8 x 4 heads, 32 tokens
    // over 515 keys: 25 us against 34; 64 tokens: 33 against 37; 32 over 1500: 30 against 39; fp32, 3 x up to 37
    // tokens over 1531 keys, 4 heads: 28 against 43 (the second figure is the call's with a table for 131072 keys).
    const int64_t blocks = (n_tokens * group + 7) / 8 + batch;
    const double tiles = (double)blocks * (double)kv_heads * (double)((a.max_keys + 127) / 128);
    const bool few = max_q <= tq3_chunk::kFewRows / group || tiles <= (wide ? 1 : 3) * tq3_chunk::kParts;
    if (!few) a.rows_to = tq3_chunk::kFewRows + 1;
    const wq_status st = wide ? tq3_chunk::run_rows<true>(a, s) : tq3_chunk::run_rows<false>(a, s);
    if (st != WQ_OK) return st;
    if (few) {
        tq3_chunk::launch_join<tq3_chunk::kFewRows>(a, tq3_chunk::kParts, a, 0, s);
        return launch_status();
    }
    tq3_chunk::Args many = a;
    many.rows_from = a.rows_to, many.rows_to = INT32_MAX;
    many.ws += tq3_chunk::rows_workspace();
    return tq3_chunk_mma::run(many, wide, a, tq3_chunk::kParts, s);
}

// Attention of ragged chunks of new tokens over a batch's paged TQ3 cache: what its kernels share.
// Internal to libwq_b200.
//
// The rows of (sequence, KV head) are its new tokens' query heads of that KV head, token by token:
// row r is token r / group, query head h * group + r % group. A segment is a block of R consecutive
// rows of one (sequence, KV head); its work is the list of 128-key tiles that any of its rows sees.
// All tiles of all segments, in the order (sequence, KV head, block, tile), are one line of work that
// is cut into equal parts, one per CTA, whatever the sequences' lengths. Each CTA finds its part from
// q_start and kv_len alone. A segment inside one part is finished there; one that is cut leaves a
// partial result per part (rows normalised by their own sums, with the maxima and sums), which
// the join kernel joins in the order of the parts: the result does not depend on timing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tq3_cache.cuh"
#include "tq3_common.cuh"

namespace wq {
namespace tq3_chunk {

using tq3::SignMask;

constexpr int kTileKeys = 128;
constexpr int kSms = 148;
constexpr int kMaxKeys = 0x7fffffff - 4096;  // keys of a sequence: tile arithmetic stays within int32

struct Args {
    const void *q;
    int64_t q_token, q_head;  // strides in elements
    tq3_cache::Pools pools;
    const int32_t *table, *q_start, *kv_len;
    int64_t pages_per_seq;
    int max_keys;  // of a sequence: what its row of the table holds, kMaxKeys at most
    int batch, n_tokens, group;
    uint32_t group_mul;  // r / group = (umulhi(group_mul, r) + r) >> group_shift for 0 <= r < 2^31
    int group_shift;
    int window, sinks;  // window == 0: none
    int rows_from, rows_to;  // serves the sequences with rows_from <= rows per KV head < rows_to
    float coef;              // post * softmax_scale * log2(e)
    SignMask mask;
    void *out;
    int q_bf16, out_bf16;
    unsigned char *ws;
};

// Multiplier and shift of Args: with 2^(shift - 1) < group <= 2^shift, floor(2^32 (2^shift - group) / group) + 1
// (division by an invariant, rounded up; r + umulhi stays below 2^32).
inline void set_group(Args &a, int group) {
    a.group = group;
    a.group_shift = 0;
    while ((int64_t(1) << a.group_shift) < group) ++a.group_shift;
    a.group_mul = (uint32_t)((((uint64_t(1) << a.group_shift) - (uint64_t)group) << 32) / (uint64_t)group + 1);
}
// The token, from the first of the sequence's new ones, of row r.
__device__ __forceinline__ int token_of(const Args &a, int r) {
    return (int)((__umulhi(a.group_mul, (uint32_t)r) + (uint32_t)r) >> a.group_shift);
}

// A sequence's new tokens and keys, as this launch serves it.
struct Seq {
    int start, new_tokens, keys;
};

__device__ __forceinline__ Seq load_seq(const Args &a, int b) {
    Seq s;
    const int first = __ldg(a.q_start + b), next = __ldg(a.q_start + b + 1), keys = __ldg(a.kv_len + b);
    s.start = min(max(first, 0), a.n_tokens);
    s.new_tokens = min(max(next, s.start), a.n_tokens) - s.start;
    s.keys = min(max(keys, 0), a.max_keys);
    const int rows = s.new_tokens * a.group;
    if (rows < a.rows_from || rows >= a.rows_to) s.new_tokens = 0;
    return s;
}

// The tiles that rows at positions p_lo .. p_hi see: `sinks` tiles from key 0 on, then the tiles from
// `first` on, `n` in all. Keys below `from` are seen only as sinks (below `until`).
struct Span {
    int sinks, first, n;
    int from, until;
    __device__ __forceinline__ int tile(int i) const { return i < sinks ? i : first + i - sinks; }
};

__device__ __forceinline__ Span span_of(const Args &a, int p_lo, int p_hi) {
    Span s;
    s.from = a.window && p_lo >= a.window ? p_lo - a.window + 1 : 0;
    s.until = min(a.sinks, s.from);
    s.first = s.from / kTileKeys;
    s.sinks = min((s.until + kTileKeys - 1) / kTileKeys, s.first);
    s.n = p_hi < 0 ? 0 : s.sinks + p_hi / kTileKeys - s.first + 1;
    return s;
}

template <int R>
__device__ __forceinline__ Span block_span(const Args &a, const Seq &s, int block) {
    const int r0 = block * R, r1 = min(r0 + R, s.new_tokens * a.group) - 1;
    const int before = s.keys - s.new_tokens;
    return span_of(a, before + token_of(a, r0), before + token_of(a, r1));
}

// On the line a segment is setup_units, what loading its queries and storing its results costs in tiles,
// and then its tiles; who has the first tile begins it. A block without a visible key still counts one
// tile: its rows are written as zeros.
template <int R>
__host__ __device__ constexpr int setup_units() {
    return R == 8 ? 2 : 4;
}
template <int R>
__device__ __forceinline__ int blocks_of(const Args &a, const Seq &s) {
    return (s.new_tokens * a.group + R - 1) / R;
}
template <int R>
__device__ __forceinline__ int64_t tiles_of_head(const Args &a, const Seq &s) {
    int64_t n = 0;
#pragma unroll 1
    for (int i = blocks_of<R>(a, s) - 1; i >= 0; --i) n += max(1, block_span<R>(a, s, i).n) + setup_units<R>();
    return n;
}

// Part c of n is [begin(c), begin(c + 1)), the first total % n parts one unit longer. There are as many
// parts as CTAs, or one per unit of the line where it is shorter.
struct Line {
    int64_t each;
    int rest, parts;
    Line() = default;
    // total < 2^47: two steps of a long division by a number below 2^15
    __device__ __forceinline__ Line(int64_t total, int ctas) {
        parts = total < ctas ? (int)total : ctas;
        const uint32_t d = max(parts, 1), high = (uint32_t)(total >> 16), q = high / d;
        const uint32_t low = (high - q * d) << 16 | (uint32_t)(total & 0xffff), r = low / d;
        each = (int64_t)q << 16 | r;
        rest = (int)(low - r * d);
    }
    __device__ __forceinline__ int64_t begin(int c) const { return each * c + min(c, rest); }
};

// Header of a part, for the join: whether its last segment goes on in the next parts, how many parts it
// is in, and which one it is.
struct Cut {
    int cut, n, seq, head, block;
};
constexpr int kCutBytes = 32;

template <int R>
__host__ __device__ constexpr int64_t slot_floats() {
    return R * (128 + 2);
}
// Slot 2c: the segment that part c continues; 2c + 1: the one that it begins and does not finish.
template <int R>
__device__ __forceinline__ float *slot_at(const Args &a, int ctas, int i) {
    return reinterpret_cast<float *>(a.ws + (int64_t)ctas * kCutBytes) + i * slot_floats<R>();
}
template <int R>
constexpr int64_t workspace_bytes(int64_t ctas) {
    return ctas * (kCutBytes + 2 * slot_floats<R>() * 4);
}

// Walks this CTA's part of the line. All threads of the CTA hold the same state.
template <int R, int kThreads>
struct Walk {
    Line line;
    int64_t seg, end;  // on the line: the segment here, the end of the part
    int b, head, block, blocks;
    int tile, count;  // the segment's tiles that are this CTA's: the first one, how many
    Seq seq;
    Span span;

    // `scratch`: kThreads / 32 + 4 int64 in shared memory.
    __device__ __forceinline__ void start(const Args &a, int64_t *scratch) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        constexpr int kWarps = kThreads / 32;
        // the tiles of all sequences, kThreads of them at a time
        int64_t total = 0;
#pragma unroll 1
        for (int base = 0; base < a.batch; base += kThreads) {
            const int i = base + tid;
            int64_t c = i < a.batch ? tiles_of_head<R>(a, load_seq(a, i)) * a.pools.heads : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (base) __syncthreads();
            if (lane == 0) scratch[warp] = c;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += scratch[w];
        }
        line = Line(min(total, int64_t(1) << 46), gridDim.x);
        int64_t at = 0;
        seg = end = 0;
        if ((int)blockIdx.x >= line.parts) return;
        at = line.begin(blockIdx.x);
        end = line.begin(blockIdx.x + 1);
        // the sequence that holds `at`: prefix sums (all of this ends, with valid places, even if the lengths
        // change under the call)
        if (tid == 0) scratch[kWarps] = -1;
        int64_t before = 0;
#pragma unroll 1
        for (int base = 0; base < a.batch; base += kThreads) {
            const int i = base + tid;
            Seq s;
            s.start = s.new_tokens = s.keys = 0;
            if (i < a.batch) s = load_seq(a, i);
            const int64_t c = i < a.batch ? tiles_of_head<R>(a, s) * a.pools.heads : 0;
            int64_t sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            __syncthreads();
            if (lane == 31) scratch[warp] = sum;
            __syncthreads();
            int64_t lead = before;
            int64_t all = before;
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w) {
                const int64_t x = scratch[w];
                all += x;
                if (w < warp) lead += x;
            }
            if (at >= lead + sum - c && at < lead + sum) {
                scratch[kWarps] = i;
                scratch[kWarps + 1] = at - (lead + sum - c);
                scratch[kWarps + 2] = (int64_t)s.start << 32 | s.new_tokens;
                scratch[kWarps + 3] = s.keys;
            }
            before = all;
            if (at < all) break;
        }
        __syncthreads();
        b = (int)scratch[kWarps];
        if (b < 0) {
            seg = end = 0;
            return;
        }
        int64_t off = scratch[kWarps + 1];
        seq.start = (int)(scratch[kWarps + 2] >> 32);
        seq.new_tokens = (int)scratch[kWarps + 2];
        seq.keys = (int)scratch[kWarps + 3];
        blocks = blocks_of<R>(a, seq);
        const int64_t per_head = tiles_of_head<R>(a, seq);
        head = 0;
#pragma unroll 1
        for (; off >= per_head && head + 1 < a.pools.heads; off -= per_head) ++head;
        block = 0;
#pragma unroll 1
        for (;; ++block) {
            span = block_span<R>(a, seq, block);
            const int n = max(1, span.n) + setup_units<R>();
            if (off < n || block + 1 >= blocks) break;
            off -= n;
        }
        seg = at - off;
        if (!settle(at)) next(a);
    }
    __device__ __forceinline__ bool done() const { return seg >= end; }
    __device__ __forceinline__ int segment() const { return max(1, span.n); }
    __device__ __forceinline__ int take() const { return count; }
    // The tiles of the segment here from `at` on that are before the part's end; whether there are any.
    __device__ __forceinline__ bool settle(int64_t at) {
        const int64_t first = seg + setup_units<R>(), stop = min(first + segment(), end);
        tile = (int)(max(at, first) - first);
        count = (int)(stop - first) - tile;
        return count > 0;
    }
    // Of the segment here, which this part begins and does not finish.
    __device__ __forceinline__ Cut cut_here() const {
        Cut c;
        c.cut = 1, c.n = 2;
        const int64_t last = seg + setup_units<R>() + segment();
#pragma unroll 1
        for (int part = blockIdx.x + 2; part < line.parts && line.begin(part) < last; ++part) ++c.n;
        c.seq = b, c.head = head, c.block = block;
        return c;
    }
    __device__ __forceinline__ void next(const Args &a) {
#pragma unroll 1
        do {
            seg += setup_units<R>() + segment();
            if (seg >= end) return;
            if (++block == blocks) {
                block = 0;
                if (++head == a.pools.heads) {
                    head = 0;
#pragma unroll 1
                    do {
                        if (b + 1 >= a.batch) {
                            seg = end;
                            return;
                        }
                        seq = load_seq(a, ++b);
                    } while (seq.new_tokens == 0);
                    blocks = blocks_of<R>(a, seq);
                }
            }
            span = block_span<R>(a, seq, block);
        } while (!settle(seg));
    }
};

// 128-point Walsh-Hadamard transform (unnormalised) of a row that a warp holds, lane l elements
// 4 l .. 4 l + 3.
__device__ __forceinline__ void row_fwht(float (&v)[4], int lane) {
    {
        const float a = __fadd_rn(v[0], v[1]), b = __fsub_rn(v[0], v[1]), c = __fadd_rn(v[2], v[3]),
                    d = __fsub_rn(v[2], v[3]);
        v[0] = __fadd_rn(a, c);
        v[1] = __fadd_rn(b, d);
        v[2] = __fsub_rn(a, c);
        v[3] = __fsub_rn(b, d);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = __shfl_xor_sync(0xffffffffu, v[i], o);
            v[i] = (lane & o) ? __fsub_rn(w, v[i]) : __fadd_rn(v[i], w);
        }
}

__device__ __forceinline__ float sign_of(const SignMask &m, int e) {
    return __uint_as_float(0x3f800000u | (~(m.w[e >> 5] >> (e & 31)) & 1u) << 31);
}

// A lane's four elements of a row: their sign flips.
__device__ __forceinline__ void lane_signs(const Args &a, int lane, float (&sg)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sg[i] = sign_of(a.mask, 4 * lane + i);
}
// Elements 4 l .. 4 l + 3 of N rows, row[n] of (sequence, head) each; kBf16: q is known to be bf16.
template <int N, bool kBf16>
__device__ __forceinline__ void load_rows(const Args &a, const Seq &s, int head, const int (&row)[N], int lane, float (&v)[N][4]) {
    int64_t at[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int token = token_of(a, row[n]);
        at[n] = (int64_t)(s.start + token) * a.q_token + (int64_t)(head * a.group + row[n] - token * a.group) * a.q_head + 4 * lane;
    }
    if (kBf16 || a.q_bf16) {
        uint2 w[N];
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + at[n]));
#pragma unroll
        for (int n = 0; n < N; ++n)
            v[n][0] = bf16_lo(w[n].x), v[n][1] = bf16_hi(w[n].x), v[n][2] = bf16_lo(w[n].y), v[n][3] = bf16_hi(w[n].y);
    } else {
        float4 w[N];
#pragma unroll
        for (int n = 0; n < N; ++n) w[n] = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at[n]));
#pragma unroll
        for (int n = 0; n < N; ++n) v[n][0] = w[n].x, v[n][1] = w[n].y, v[n][2] = w[n].z, v[n][3] = w[n].w;
    }
}

// Stores s . v post as a row of the result; store_row: of H(v), from the rotated basis.
template <bool kBf16>
__device__ __forceinline__ void put_row(const Args &a, const Seq &s, int head, int row, int lane, const float (&sg)[4],
                                        float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], tq3::fwht_post()), sg[i]);
    const int token = token_of(a, row);
    const int64_t at = (((int64_t)(s.start + token) * a.pools.heads + head) * a.group + row - token * a.group) * 128 + 4 * lane;
    if (kBf16 || a.out_bf16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

template <bool kBf16>
__device__ __forceinline__ void store_row(const Args &a, const Seq &s, int head, int row, int lane, const float (&sg)[4],
                                          float (&v)[4]) {
    row_fwht(v, lane);
    put_row<kBf16>(a, s, head, row, lane, sg, v);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Joins the partial results of the segment that part `part` leaves cut: its row r, by a warp.
template <int R>
__device__ __forceinline__ void merge_cut(const Args &a, int part, int ctas, int r) {
    const int lane = threadIdx.x & 31;
    const Cut c = *reinterpret_cast<const Cut *>(a.ws + (int64_t)part * kCutBytes);
    if (!c.cut) return;
    const Seq s = load_seq(a, c.seq);
    const int row = c.block * R + r;
    if (row >= s.new_tokens * a.group) return;
    const float *const slots = slot_at<R>(a, ctas, 2 * part);  // the part's own one is its second
    auto slot = [&](int i) { return slots + (i == 0 ? 1 : 2 * i) * slot_floats<R>(); };
    float top = -INFINITY;
    for (int i = lane; i < c.n; i += 32) top = fmaxf(top, slot(i)[R * 128 + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
    if (top != -INFINITY)
        for (int i0 = 0; i0 < c.n; i0 += 32) {
            const int n = min(32, c.n - i0);
            const float w_mine = lane < n ? __fmul_rn(slot(i0 + lane)[R * 129 + r], ex2(__fsub_rn(slot(i0 + lane)[R * 128 + r], top)))
                                          : 0.0f;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float w = __shfl_sync(0xffffffffu, w_mine, i);
                const float4 x = *reinterpret_cast<const float4 *>(slot(i0 + i) + r * 128 + 4 * lane);
                sum = __fadd_rn(sum, w);
                v[0] = __fmaf_rn(w, x.x, v[0]);
                v[1] = __fmaf_rn(w, x.y, v[1]);
                v[2] = __fmaf_rn(w, x.z, v[2]);
                v[3] = __fmaf_rn(w, x.w, v[3]);
            }
        }
    if (sum != 0.0f) {
        const float f = __frcp_rn(sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], f);
    }
    float sg[4];
    lane_signs(a, lane, sg);
    store_row<false>(a, s, c.head, row, lane, sg, v);
}

// The join of one launch, or of the two that share a call: `few` of R = 8 over few_ctas CTAs, then `many` of
// RM rows over many_ctas.
constexpr int kJoinThreads = 128, kJoinRows = kJoinThreads / 32;
template <int RM>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args few, int few_ctas,
                                                            const __grid_constant__ Args many, int many_ctas) {
    pdl_wait();
    constexpr int kFew = 8 / kJoinRows, kMany = RM / kJoinRows;
    const int warp = threadIdx.x >> 5, i = blockIdx.x, j = i - few_ctas * kFew;
    if (j < 0)
        merge_cut<8>(few, i / kFew, few_ctas, i % kFew * kJoinRows + warp);
    else
        merge_cut<RM>(many, j / kMany, many_ctas, j % kMany * kJoinRows + warp);
}
template <int RM>
cudaError_t launch_join(const Args &few, int few_ctas, const Args &many, int many_ctas, cudaStream_t s) {
    return launch_pdl(join_kernel<RM>, few_ctas * (8 / kJoinRows) + many_ctas * (RM / kJoinRows), kJoinThreads, 0, s, few,
                      few_ctas, many, many_ctas);
}

}  // namespace tq3_chunk
}  // namespace wq

// The paged TQ3 cache shared by a batch of sequences: pools [n_pages][kv_heads][page_size][56 bytes]
// for K and for V (the record of tq3_encode_aos), one page table per sequence for all heads and both
// pools. Internal to libwq_b200.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tq3_common.cuh"

namespace wq {
namespace tq3_cache {

constexpr int kRec = 56;  // bytes of a record

struct Pools {
    uint8_t *k, *v;
    int64_t n_pages;
    int heads;
    int shift;  // log2 of the page size
};

// Byte offset of (page, head, place in the page).
__device__ __forceinline__ int64_t record_at(const Pools &p, int64_t page, int head, int64_t place) {
    return (((page * p.heads + head) << p.shift) + place) * kRec;
}

// Fault bits of the cache kernels (tq3::kFaultPoolIndex), read and cleared by wq_device_fault.
unsigned int read_and_clear_fault();

// log2 of a page size, or -1 if it is not a power of two in 1 .. 2^30.
inline int page_shift(int64_t page_size) {
    if (page_size < 1 || page_size > (int64_t(1) << 30) || (page_size & (page_size - 1))) return -1;
    int s = 0;
    while ((int64_t(1) << s) < page_size) ++s;
    return s;
}

// Bytes of one pool stay within int64 and heads within int32; the counts the entry points accept.
inline bool pool_shape_ok(int64_t n_pages, int64_t heads, int64_t page_size) {
    if (n_pages < 0 || heads < 1 || heads > 65535 || page_shift(page_size) < 0) return false;
    return n_pages <= (int64_t(1) << 52) / (heads * page_size);
}

}  // namespace tq3_cache
}  // namespace wq

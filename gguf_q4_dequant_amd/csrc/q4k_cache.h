// The paged cache and the packed sequences on the device (include/q4k_layer.h),
// shared by the kernels that write the cache and those that read it.
#pragma once

#include "../../include/q4k_layer.h"
#include "q4k_internal.h"

namespace q4k {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half4v __attribute__((ext_vector_type(4)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

// Passed by value in the kernel-argument segment.
struct Paged {
    uint8_t *k;
    uint8_t *v;
    const int *offsets;
    const int *lengths;
    const int *table;
    int count;      // sequences
    int max_pages;  // of a row of the table
    int pages;      // in the pool
    int shift;      // log2 of the page size
    int kv_heads;
    int head_dim;
    int tokens;     // T
    float k_scale;
    float v_scale;
};

// offsets[b], read as if clamped to [0, T].
__device__ __forceinline__ int offset_of(const Paged &p, int b) { return min(max(p.offsets[b], 0), p.tokens); }

// The last sequence b whose start(b) <= at, start ascending with start(0) <= at;
// every lane of the wave passes the same `at` and gets the same b, in [0, count).
// A 64th of the range is kept by one load a lane: one step for 64 sequences, two for
// 4096, three for 65535 (64 at a time they were 1024: storing one token of each of
// 65535 sequences took 2620 us, with this 256, what its bytes take; of 8192, 66 and 29).
template <class Start>
__device__ __forceinline__ int last_started(int count, int64_t at, Start start) {
    const int lane = threadIdx.x & 63;
    int low = 0, span = count;  // b is in [low, low + span)
    while (span > 64) {
        const int step = (span + 63) / 64, i = lane * step;
        const bool begun = i < span && start(low + i) <= at;
        const int more = max(__builtin_popcountll(__ballot(begun)) - 1, 0) * step;
        low += more;
        span = min(step, span - more);
    }
    const bool begun = lane < span && start(low + lane) <= at;
    return low + max(__builtin_popcountll(__ballot(begun)) - 1, 0);
}

// The first element of (index j of sequence b, kv head h) in units of
// elements, or -1 where the index has no page.
__device__ __forceinline__ int64_t place_of(const Paged &p, int b, int64_t j, int h) {
    if (j < 0 || j >= (static_cast<int64_t>(p.max_pages) << p.shift)) return -1;
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + (j >> p.shift)];
    if (page < 0 || page >= p.pages) return -1;
    const int64_t slot = ((static_cast<int64_t>(page) * p.kv_heads + h) << p.shift) + (j & ((1 << p.shift) - 1));
    return slot * p.head_dim;
}

// Checks of what the calls over a cache share; fills *p.  q_heads 0: no queries.
int check_paged(const q4k_kv_cache *cache, const q4k_sequences *sequences, int T, int q_heads, Paged *p);

}  // namespace q4k

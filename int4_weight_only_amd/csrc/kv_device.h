// kv_device.h -- the paged key-value cache as the kernels see it, and the attention mask shared by
// the single-token and the prompt form.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4 {

// A checked w4_kv_cache: strides in elements. The element offset inside one page fits 31 bits
// (the entry points refuse other caches); the offset of a page does not have to.
struct KvView {
    uint16_t *k, *v;
    const int32_t *table;   // [n_seqs][ld_table], table_cols entries used
    const int32_t *kv_len;  // [n_seqs]
    int64_t page_stride, ld_table;
    int32_t slot_stride, head_stride;
    int32_t n_pages, page_shift, page_mask;
    int32_t table_cols, capacity;  // capacity = table_cols * page_size positions
    int32_t n_kv, head_dim, n_seqs;
};

#if defined(__HIPCC__)

// An element of an array that nothing writes while the kernel runs (page tables, lengths): a scalar
// load where the address is uniform, whatever the kernel stores elsewhere.
__device__ __forceinline__ int32_t read_const(const int32_t *p) {
    typedef const __attribute__((address_space(4))) int32_t *const_ptr;
    return *reinterpret_cast<const_ptr>(reinterpret_cast<uintptr_t>(p));
}

// Keys of sequence b; a length outside what its page table can hold is cut to it.
__device__ __forceinline__ int kv_length(const KvView &c, int b) {
    const int n = read_const(c.kv_len + b);
    return n < 0 ? 0 : (n > c.capacity ? c.capacity : n);
}

// Page that holds position pos (0 <= pos < capacity) of the sequence whose table row is `row`.
// An entry outside the cache is moved into it, so that no entry makes an access leave the cache.
__device__ __forceinline__ int kv_page(const KvView &c, const int32_t *row, int pos) {
    const int p = read_const(row + (pos >> c.page_shift));
    return p < 0 ? 0 : (p >= c.n_pages ? c.n_pages - 1 : p);
}

// Element offset of (position, kv head).
__device__ __forceinline__ int64_t kv_offset(const KvView &c, const int32_t *row, int pos,
                                             int head) {
    return static_cast<int64_t>(kv_page(c, row, pos)) * c.page_stride +
           static_cast<int64_t>((pos & c.page_mask) * c.slot_stride + head * c.head_stride);
}

// Where token row t stands: its sequence, that sequence's keys, and its position (below 0: it sees
// no key). False for a row that q_start gives to no sequence. Without q_start each sequence has
// one row, its last token. q_start is nondecreasing; whatever it holds, the position returned is
// below n_keys.
struct RowPlace {
    int seq, n_keys, pos;
};
__device__ __forceinline__ bool place_of_row(const KvView &c, const int32_t *q_start, int t,
                                             RowPlace *r) {
    if (!q_start) {
        r->seq = t;
        r->n_keys = kv_length(c, t);
        r->pos = r->n_keys - 1;
        return true;
    }
    int lo = 0, hi = c.n_seqs - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (read_const(q_start + mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int end = read_const(q_start + lo + 1);
    if (t < read_const(q_start + lo) || t >= end) return false;
    r->seq = lo;
    r->n_keys = kv_length(c, lo);
    r->pos = r->n_keys - (end - t);
    return true;
}

#endif

}  // namespace w4

// paged.cuh -- the paged Q8_0 cache's addressing and the argument checks that its entry points share.
#pragma once

#include "common.cuh"

namespace kvq8 {

constexpr int kMaxSeqs = 4096;        // requests of one call
constexpr int kMaxWindowRows = 64;    // rows of one request's window: one bit each of a 64-bit mask

// A slot is page * page_size + offset.  Planes: codes [n_pages][n_kv_heads][page_size][head_dim], scales
// [n_pages][n_kv_heads][page_size][head_dim / 32], so a page holds page_size consecutive rows of each head.
// The row index below times head_dim (or head_dim / 32) is the element offset; it is 64-bit throughout.
__device__ __forceinline__ int64_t paged_row(int64_t slot, int head, int n_kv_heads, int page_shift) {
    const int64_t page = slot >> page_shift;
    const int off = (int)(slot & ((1 << page_shift) - 1));
    return ((page * n_kv_heads + head) << page_shift) + off;
}

inline int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

inline size_t dtype_size(int dtype) { return dtype == KVQ8_F32 ? 4u : dtype == KVQ8_F16 || dtype == KVQ8_BF16 ? 2u : 0u; }

inline int check_paged(const kvq8_paged_cache* kv) {
    if (!kv || kv->n_kv_heads < 1 || kv->n_pages < 1 || kv->page_size < 1) return KVQ8_ERR_INVALID_ARG;
    if (!kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales) return KVQ8_ERR_INVALID_ARG;
    if (kv->head_dim != 128 && kv->head_dim != 256) return KVQ8_ERR_UNSUPPORTED;
    if (kv->page_size < 16 || kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1))) return KVQ8_ERR_UNSUPPORTED;
    if (kv->n_kv_heads > 4096) return KVQ8_ERR_UNSUPPORTED;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) || !aligned16(kv->v_scales))
        return KVQ8_ERR_MISALIGNED;
    return KVQ8_OK;
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace kvq8

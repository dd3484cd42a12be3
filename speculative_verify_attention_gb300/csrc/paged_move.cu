// paged_move.cu -- rows of a paged cache moved as they are: the last pages that forked sequences go on in
// (kvq8_paged_copy), and the accepted path of a drafted tree to the places behind its context (kvq8_paged_compact).  Both are bound
// by latency: the list or the lengths, then the page ids, then the rows.  The last pages of 260 beams (1 x 256, 16 rows) 2.5 us; 200
// trees of 64 rows, 25 kept (8 x 128), 6.4 us, four trees of 8 2.6 us.
#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kMoveThreads = 128;

struct PagedMove {
    int8_t* codes[2];
    uint16_t* scales[2];
    int n_kv_heads, head_dim, page_shift, n_pages;
};

// ---------------------------------------------------------------- copy

struct CopyList {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;
    int n;
};

// Block (list entry, plane and head): the first rows of a page's head are one run of codes and one of scales.
__global__ void __launch_bounds__(kMoveThreads) paged_copy_kernel(const __grid_constant__ PagedMove p, const __grid_constant__ CopyList c) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int i = blockIdx.x, z = blockIdx.y & 1, h = blockIdx.y >> 1;
    const int from = c.src[i], to = c.dst[i];
    if (from < 0 || from >= p.n_pages || to < 0 || to >= p.n_pages || from == to) return;
    const int page = 1 << p.page_shift, rows = c.rows ? min(max(c.rows[i], 0), page) : page;
    const uint64_t a = paged_row((uint32_t)from << p.page_shift, h, p.n_kv_heads, p.page_shift);
    const uint64_t b = paged_row((uint32_t)to << p.page_shift, h, p.n_kv_heads, p.page_shift);
    const int8_t* codes = p.codes[z];
    const uint16_t* scales = p.scales[z];
    const uint4* src = reinterpret_cast<const uint4*>(codes + a * (uint32_t)p.head_dim);
    uint4* dst = reinterpret_cast<uint4*>(p.codes[z] + b * (uint32_t)p.head_dim);
    const uint32_t blocks = (uint32_t)p.head_dim / kQBlock;
    const uint2* ssrc = reinterpret_cast<const uint2*>(scales + a * blocks);
    uint2* sdst = reinterpret_cast<uint2*>(p.scales[z] + b * blocks);
    const int n = rows * p.head_dim / 16, ns = rows * (int)blocks / 4;
    for (int k = threadIdx.x; k < ns; k += kMoveThreads) sdst[k] = ssrc[k];
    for (int k0 = threadIdx.x; k0 < n; k0 += 4 * kMoveThreads) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k0 + u * kMoveThreads < n) v[u] = src[k0 + u * kMoveThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k0 + u * kMoveThreads < n) dst[k0 + u * kMoveThreads] = v[u];
    }
}

// ---------------------------------------------------------------- compact

struct Compact {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* row_starts;
    const uint64_t* kept;
    int32_t* lens_out;
    int n_seqs, max_pages;
};

// Block (request, plane and head): every row that moves is read into shared memory before the first is written, as a row's
// place may be another's.
__global__ void __launch_bounds__(kMoveThreads) paged_compact_kernel(const __grid_constant__ PagedMove p, const __grid_constant__ Compact c) {
    extern __shared__ __align__(16) uint4 s_rows[];
    __shared__ int s_from[kMaxWindowRows], s_to[kMaxWindowRows];  // cache rows
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x, z = blockIdx.y & 1, h = blockIdx.y >> 1, tid = threadIdx.x;
    const int len = c.lens[b], t = c.row_starts[b + 1] - c.row_starts[b];
    uint64_t kept = c.kept[b];
    const bool good = t >= 0 && t <= kMaxWindowRows && t <= len && len <= ((int64_t)c.max_pages << p.page_shift);
    if (good && t < 64) kept &= (1ull << t) - 1;
    if (c.lens_out && blockIdx.y == 0 && tid == 0) c.lens_out[b] = good ? len - t + __popcll(kept) : len;
    if (!good) return;
    const int stay = __ffsll((long long)~kept) - 1;  // kept places before the first gap are where they go (-1: all 64)
    if (stay < 0) return;
    const int n = __popcll(kept) - stay;             // rows that move
    if (n <= 0) return;
    if (tid < n) {
        uint64_t rest = kept >> stay >> 1;  // the places behind the gap
        for (int k = 0; k < tid; ++k) rest &= rest - 1;
        const int from = len - t + stay + 1 + __ffsll((long long)rest) - 1, to = len - t + stay + tid;
        const int32_t* pages = c.table + (int64_t)b * c.max_pages;
        const int a = pages[from >> p.page_shift], d = pages[to >> p.page_shift], mask = (1 << p.page_shift) - 1;
        const bool there = a >= 0 && a < p.n_pages && d >= 0 && d < p.n_pages;
        s_from[tid] = there ? (int)paged_row(((uint32_t)a << p.page_shift) + (from & mask), h, p.n_kv_heads, p.page_shift) : -1;
        s_to[tid] = there ? (int)paged_row(((uint32_t)d << p.page_shift) + (to & mask), h, p.n_kv_heads, p.page_shift) : -1;
    }
    __syncthreads();
    const uint32_t blocks = (uint32_t)p.head_dim / kQBlock;
    const int lanes = p.head_dim / 16, shift = p.head_dim == 256 ? 4 : 3;  // 16-byte pieces of a row's codes
    const int pieces = blocks / 4;                                         // 8-byte pieces of its scales
    uint2* s_scales = reinterpret_cast<uint2*>(s_rows + n * lanes);
    for (int k = tid; k < n * lanes; k += kMoveThreads) {
        const int row = s_from[k >> shift];
        if (row >= 0) s_rows[k] = reinterpret_cast<const uint4*>(p.codes[z] + (uint64_t)(uint32_t)row * (uint32_t)p.head_dim)[k & (lanes - 1)];
    }
    for (int k = tid; k < n * pieces; k += kMoveThreads) {
        const int row = s_from[pieces == 2 ? k >> 1 : k];
        if (row >= 0) s_scales[k] = reinterpret_cast<const uint2*>(p.scales[z] + (uint64_t)(uint32_t)row * blocks)[pieces == 2 ? k & 1 : 0];
    }
    __syncthreads();
    for (int k = tid; k < n * lanes; k += kMoveThreads) {
        const int row = s_to[k >> shift];
        if (row >= 0) reinterpret_cast<uint4*>(p.codes[z] + (uint64_t)(uint32_t)row * (uint32_t)p.head_dim)[k & (lanes - 1)] = s_rows[k];
    }
    for (int k = tid; k < n * pieces; k += kMoveThreads) {
        const int row = s_to[pieces == 2 ? k >> 1 : k];
        if (row >= 0) reinterpret_cast<uint2*>(p.scales[z] + (uint64_t)(uint32_t)row * blocks)[pieces == 2 ? k & 1 : 0] = s_scales[k];
    }
}

PagedMove paged_move(const kvq8_paged_cache* kv) {
    return PagedMove{{const_cast<int8_t*>(kv->k_codes), const_cast<int8_t*>(kv->v_codes)},
                     {const_cast<uint16_t*>(kv->k_scales), const_cast<uint16_t*>(kv->v_scales)},
                     kv->n_kv_heads, kv->head_dim, log2_of(kv->page_size), kv->n_pages};
}

}  // namespace
}  // namespace kvq8

extern "C" int kvq8_paged_copy(const kvq8_paged_cache* kv, const int32_t* src_pages, const int32_t* dst_pages,
                               const int32_t* rows, int n, kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    if (n < 0) return KVQ8_ERR_INVALID_ARG;
    if (n == 0) return KVQ8_OK;
    if (!src_pages || !dst_pages) return KVQ8_ERR_INVALID_ARG;
    for (const int32_t* q : {src_pages, dst_pages, rows})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    return launch_dependent(paged_copy_kernel, dim3((unsigned)n, 2u * (unsigned)kv->n_kv_heads), kMoveThreads, 0, (cudaStream_t)stream,
                            paged_move(kv), CopyList{src_pages, dst_pages, rows, n});
}

extern "C" int kvq8_paged_compact(const kvq8_paged_cache* kv, const int32_t* page_table, int max_pages, const int32_t* lens,
                                  const int32_t* row_starts, int n_seqs, const uint64_t* kept, int32_t* lens_out,
                                  kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    if (n_seqs < 0 || max_pages < 1) return KVQ8_ERR_INVALID_ARG;
    if (n_seqs == 0) return KVQ8_OK;
    if (!page_table || !lens || !row_starts || !kept) return KVQ8_ERR_INVALID_ARG;
    if (n_seqs > kMaxSeqs) return KVQ8_ERR_UNSUPPORTED;
    for (const int32_t* q : {page_table, lens, row_starts, (const int32_t*)lens_out})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    if (!aligned_to(kept, 8)) return KVQ8_ERR_MISALIGNED;
    // blocks read these while one writes the new lengths
    const size_t lens_bytes = (size_t)n_seqs * 4;
    if (ranges_meet(lens, lens_bytes, lens_out, lens_bytes) || ranges_meet(row_starts, lens_bytes + 4, lens_out, lens_bytes) ||
        ranges_meet(kept, 2 * lens_bytes, lens_out, lens_bytes) || ranges_meet(page_table, lens_bytes * max_pages, lens_out, lens_bytes))
        return KVQ8_ERR_INVALID_ARG;
    const int smem = kMaxWindowRows * (kv->head_dim + kv->head_dim / 16);
    return launch_dependent(paged_compact_kernel, dim3((unsigned)n_seqs, 2u * (unsigned)kv->n_kv_heads), kMoveThreads, smem,
                            (cudaStream_t)stream, paged_move(kv), Compact{page_table, lens, row_starts, kept, lens_out, n_seqs, max_pages});
}

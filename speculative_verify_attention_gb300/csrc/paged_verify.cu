// paged_verify.cu -- verify attention of a batch of windows over a paged Q8_0 cache (attn_verify_paged_q8).
//
// Row t of request b (window of T rows after ctx = len - T cached tokens) sees every key n < ctx and the window
// key ctx + j where bit j of its mask is set (chains: j <= t):
//   o = sum_n p_n v_n / sum_n p_n,  p_n = exp(scale * q . k_n),  k and v = code * scale of their block.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

struct PagedVerifyParams {
    const void* q;
    void* out;
    int64_t q_stride;
    const int8_t* kc;
    const uint16_t* ks;
    const int8_t* vc;
    const uint16_t* vs;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* row_starts;
    const uint64_t* mask;
    int n_rows, n_q_heads, n_kv_heads, n_pages, page_shift, max_pages, n_seqs, max_rows;
    float scale_log2;
};

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// One block per (row, q head): its four warps take every fourth key and keep an online softmax each, merged at the
// end.  A lane holds HD / 32 dims.
template <typename T, int HD>
__global__ void __launch_bounds__(128) paged_verify_rows_kernel(const PagedVerifyParams p) {
    constexpr int D = HD / 32;
    __shared__ int s_seq;
    __shared__ float s_m[4], s_l[4], s_o[4][HD];
    const int row = blockIdx.x, head = blockIdx.y, kvh = head / (p.n_q_heads / p.n_kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) s_seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < p.n_seqs; b += 128)
        if (p.row_starts[b] <= row && row < p.row_starts[b + 1]) s_seq = b;
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const int r0 = p.row_starts[b], rows = p.row_starts[b + 1] - r0, len = p.lens[b];
    if (r0 < 0 || r0 + rows > p.n_rows || rows > p.max_rows || rows > len || (int64_t)len > ((int64_t)p.max_pages << p.page_shift))
        return;
    const int ctx = len - rows;
    const uint64_t m64 = p.mask ? p.mask[row] : (2ull << (row - r0)) - 1;
    float q[D], o[D];
    const T* src = static_cast<const T*>(p.q) + (int64_t)row * p.q_stride + head * HD + lane * D;
#pragma unroll
    for (int d = 0; d < D; ++d) q[d] = to_f32(src[d]) * p.scale_log2, o[d] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int n = warp; n < len; n += 4) {
        if (n >= ctx && !(m64 >> (n - ctx) & 1)) continue;
        const int page = p.table[(int64_t)b * p.max_pages + (n >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) continue;
        const int64_t at = paged_row(((int64_t)page << p.page_shift) + (n & ((1 << p.page_shift) - 1)), kvh, p.n_kv_heads, p.page_shift);
        const float kd = half_bits_to_float(p.ks[at * (HD / 32) + lane * D / 32]);
        const float vd = half_bits_to_float(p.vs[at * (HD / 32) + lane * D / 32]);
        float s = 0.0f;
#pragma unroll
        for (int d = 0; d < D; ++d) s += q[d] * ((float)p.kc[at * HD + lane * D + d] * kd);
#pragma unroll
        for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        const float m2 = fmaxf(m, s), a = exp2f(m - m2), w = exp2f(s - m2);
        l = l * a + w;
        m = m2;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = o[d] * a + w * ((float)p.vc[at * HD + lane * D + d] * vd);
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int d = 0; d < D; ++d) s_o[warp][lane * D + d] = o[d];
    __syncthreads();
    float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    if (top == -INFINITY) top = 0.0f;
    float w[4], total = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = exp2f(s_m[k] - top), total += w[k] * s_l[k];
    T* dst = static_cast<T*>(p.out) + ((int64_t)row * p.n_q_heads + head) * HD;
    for (int d = threadIdx.x; d < HD; d += 128) {
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) y += w[k] * s_o[k][d];
        from_f32(dst[d], total > 0.0f ? y / total : 0.0f);
    }
}

template <typename T>
int launch_rows(const PagedVerifyParams& p, int hd, cudaStream_t s) {
    const dim3 grid((unsigned)p.n_rows, (unsigned)p.n_q_heads);
    if (hd == 128)
        paged_verify_rows_kernel<T, 128><<<grid, 128, 0, s>>>(p);
    else
        paged_verify_rows_kernel<T, 256><<<grid, 128, 0, s>>>(p);
    return launch_status();
}

}  // namespace
}  // namespace kvq8

extern "C" size_t attn_verify_paged_q8_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim, int max_rows) {
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64) return 0;
    if ((head_dim != 128 && head_dim != 256) || max_rows < 1 || max_rows > kvq8::kMaxWindowRows) return 0;
    return 16;
}

extern "C" int attn_verify_paged_q8(const void* q, int dtype, int64_t q_stride, int n_rows, int n_q_heads,
                                    const kvq8_paged_cache* kv, const int32_t* page_table, int max_pages, const int32_t* lens,
                                    const int32_t* row_starts, int n_seqs, int max_rows, const uint64_t* window_mask,
                                    float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                                    kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    if ((dtype != KVQ8_F16 && dtype != KVQ8_BF16) || n_rows < 0 || n_seqs < 0 || max_pages < 1) return KVQ8_ERR_INVALID_ARG;
    if (n_q_heads < 1 || max_rows < 1 || !(softmax_scale > 0.0f) || softmax_scale == INFINITY) return KVQ8_ERR_INVALID_ARG;
    if (n_q_heads % kv->n_kv_heads || n_q_heads / kv->n_kv_heads > 64 || max_rows > kMaxWindowRows || n_seqs > kMaxSeqs ||
        n_rows > (1 << 24))
        return KVQ8_ERR_UNSUPPORTED;
    if (n_rows == 0 || n_seqs == 0) return KVQ8_OK;
    if (!q || !out || !page_table || !lens || !row_starts || q_stride < (int64_t)n_q_heads * kv->head_dim)
        return KVQ8_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < attn_verify_paged_q8_workspace_bytes(n_q_heads, kv->n_kv_heads, kv->head_dim, max_rows))
        return KVQ8_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (q_stride * 2) % 16 || !aligned_to(page_table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(row_starts, 4) || !aligned_to(window_mask, 8))
        return KVQ8_ERR_MISALIGNED;
    PagedVerifyParams p = {q, out, q_stride, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, page_table, lens,
                           row_starts, window_mask, n_rows, n_q_heads, kv->n_kv_heads, kv->n_pages,
                           log2_of(kv->page_size), max_pages, n_seqs, max_rows, softmax_scale * kLog2e};
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == KVQ8_F16 ? launch_rows<__half>(p, kv->head_dim, s) : launch_rows<__nv_bfloat16>(p, kv->head_dim, s);
}

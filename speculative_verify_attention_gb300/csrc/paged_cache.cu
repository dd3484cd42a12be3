// paged_cache.cu -- K and V tokens into the pages of a Q8_0 cache by slot (kvq8_paged_append), and back out of them
// as values (kvq8_paged_read).
//
// Append is the block quantiser of kvq8_append (q8_0_block: scale max|x| / 127 of 32 values, codes x / scale rounded
// half away from zero) over fp32, fp16 or bf16 tokens, the cache row taken from the token's slot.  Read is its
// inverse, code * scale rounded once to the type asked for.  Both are bandwidth-bound: one read and one write of
// each value.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "q8_0.cuh"

namespace kvq8 {
namespace {

constexpr int kPagedThreads = 256;
constexpr int kPagedTok = 4;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 a = __half22float2(u32_as_h2(r.x)), b = __half22float2(u32_as_h2(r.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));  // a bf16 is the upper half of its fp32
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}

struct PagedIO {
    const void* x[2];         // append: K and V tokens; read: unused
    void* y[2];               // read: K and V values
    int64_t tok_stride[2];    // elements between tokens
    int64_t head_stride[2];   // read: elements between heads
    int8_t* codes[2];
    uint16_t* scales[2];
    const int64_t* slots;
    int64_t n_slots;
    int n_tok, n_kv_heads, head_dim, page_shift;
};

// Block (tx, ty): tx consecutive float4 columns of a token row (a multiple of 32, so a warp stays in one row) for
// ty * kPagedTok tokens; grid z is the plane.  Lanes of tokens past the end or with a slot outside the cache
// quantise zeros (every lane takes part in the block's shuffle maximum) and store nothing.
template <typename T>
__global__ void __launch_bounds__(kPagedThreads) paged_append_kernel(const PagedIO p) {
    const int z = blockIdx.z;
    const T* x = static_cast<const T*>(p.x[z]);
    const int f4_head = p.head_dim / 4;
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    const bool col_ok = j < p.n_kv_heads * f4_head;
    const int h = j / f4_head, i = j - h * f4_head;
    const int tok0 = (blockIdx.x * blockDim.y + threadIdx.y) * kPagedTok;
    float4 v[kPagedTok];
    int64_t slot[kPagedTok];
#pragma unroll
    for (int t = 0; t < kPagedTok; ++t) {
        v[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        slot[t] = -1;
        if (col_ok && tok0 + t < p.n_tok) {
            slot[t] = __ldg(p.slots + tok0 + t);
            v[t] = load4<T>(x + (int64_t)(tok0 + t) * p.tok_stride[z] + (int64_t)j * 4);
        }
    }
    const int nb = p.head_dim / kQBlock;
#pragma unroll
    for (int t = 0; t < kPagedTok; ++t) {
        uint16_t scale_bits;
        const uint32_t packed = q8_0_block(v[t], &scale_bits);
        if (slot[t] >= 0 && slot[t] < p.n_slots) {
            const int64_t row = paged_row(slot[t], h, p.n_kv_heads, p.page_shift);
            *reinterpret_cast<uint32_t*>(p.codes[z] + row * p.head_dim + i * 4) = packed;
            if ((i & 7) == 0) p.scales[z][row * nb + (i >> 3)] = scale_bits;
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* dst, const float (&v)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* dst, const float (&v)[8]) {
    uint4 o;
    o.x = h2_as_u32(__floats2half2_rn(v[0], v[1]));
    o.y = h2_as_u32(__floats2half2_rn(v[2], v[3]));
    o.z = h2_as_u32(__floats2half2_rn(v[4], v[5]));
    o.w = h2_as_u32(__floats2half2_rn(v[6], v[7]));
    *reinterpret_cast<uint4*>(dst) = o;
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

// The same block shape over groups of eight values: 8 code bytes and their scale in, eight values out.  A slot
// outside the cache gives zeros.
template <typename T>
__global__ void __launch_bounds__(kPagedThreads) paged_read_kernel(const PagedIO p) {
    const int z = blockIdx.z;
    T* y = static_cast<T*>(p.y[z]);
    const int g_head = p.head_dim / 8;
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    if (j >= p.n_kv_heads * g_head) return;
    const int h = j / g_head, i = j - h * g_head;
    const int tok0 = (blockIdx.x * blockDim.y + threadIdx.y) * kPagedTok;
    uint2 c[kPagedTok];
    uint16_t sc[kPagedTok];
#pragma unroll
    for (int t = 0; t < kPagedTok; ++t) {
        c[t] = make_uint2(0u, 0u);
        sc[t] = 0;
        if (tok0 + t < p.n_tok) {
            const int64_t slot = __ldg(p.slots + tok0 + t);
            if (slot >= 0 && slot < p.n_slots) {
                const int64_t row = paged_row(slot, h, p.n_kv_heads, p.page_shift);
                c[t] = *reinterpret_cast<const uint2*>(p.codes[z] + row * p.head_dim + i * 8);
                sc[t] = p.scales[z][row * (p.head_dim / kQBlock) + (i >> 2)];
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kPagedTok; ++t) {
        if (tok0 + t >= p.n_tok) break;
        const float d = half_bits_to_float(sc[t]);
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = (float)(int8_t)(c[t].x >> (8 * k)) * d;  // exact in fp32: 8 by 11 bits
            v[4 + k] = (float)(int8_t)(c[t].y >> (8 * k)) * d;
        }
        store8<T>(y + (int64_t)(tok0 + t) * p.tok_stride[z] + (int64_t)h * p.head_stride[z] + i * 8, v);
    }
}

// Columns a block covers (a multiple of 32, at most 256) and its token rows.
dim3 paged_block(int cols) {
    const int tx = cols < kPagedThreads ? cols / 32 * 32 : kPagedThreads;
    return dim3((unsigned)tx, (unsigned)(kPagedThreads / tx));
}

template <typename Kernel>
int launch_paged(Kernel* kernel, const PagedIO& p, int cols, cudaStream_t stream) {
    const dim3 block = paged_block(cols);
    const int64_t per = (int64_t)block.y * kPagedTok;
    const int64_t gx = (p.n_tok + per - 1) / per;
    const dim3 grid((unsigned)gx, (unsigned)((cols + block.x - 1) / block.x), 2u);
    kernel<<<grid, block, 0, stream>>>(p);
    return launch_status();
}

PagedIO paged_io(const kvq8_paged_cache* kv, const int64_t* slots, int n_tok) {
    PagedIO p = {};
    p.codes[0] = const_cast<int8_t*>(kv->k_codes);
    p.codes[1] = const_cast<int8_t*>(kv->v_codes);
    p.scales[0] = const_cast<uint16_t*>(kv->k_scales);
    p.scales[1] = const_cast<uint16_t*>(kv->v_scales);
    p.slots = slots;
    p.n_slots = (int64_t)kv->n_pages * kv->page_size;
    p.n_tok = n_tok;
    p.n_kv_heads = kv->n_kv_heads;
    p.head_dim = kv->head_dim;
    p.page_shift = log2_of(kv->page_size);
    return p;
}

}  // namespace
}  // namespace kvq8

extern "C" int kvq8_paged_append(const void* k, const void* v, int dtype, int n_tok, int64_t k_stride, int64_t v_stride,
                                 const kvq8_paged_cache* kv, const int64_t* slots, kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    const size_t esz = dtype_size(dtype);
    if (!esz || n_tok < 0) return KVQ8_ERR_INVALID_ARG;
    if (n_tok == 0) return KVQ8_OK;
    const int64_t row = (int64_t)kv->n_kv_heads * kv->head_dim;
    if (!k || !v || !slots || k_stride < row || v_stride < row) return KVQ8_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || (k_stride * (int64_t)esz) % 16 || (v_stride * (int64_t)esz) % 16 ||
        !aligned_to(slots, 8))
        return KVQ8_ERR_MISALIGNED;
    PagedIO p = paged_io(kv, slots, n_tok);
    p.x[0] = k;
    p.x[1] = v;
    p.tok_stride[0] = k_stride;
    p.tok_stride[1] = v_stride;
    const int cols = (int)(row / 4);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_paged(paged_append_kernel<float>, p, cols, s);
    if (dtype == KVQ8_F16) return launch_paged(paged_append_kernel<__half>, p, cols, s);
    return launch_paged(paged_append_kernel<__nv_bfloat16>, p, cols, s);
}

extern "C" int kvq8_paged_read(const kvq8_paged_cache* kv, const int64_t* slots, int n_tok, int dtype, void* k, void* v,
                               const int64_t* k_strides, const int64_t* v_strides, kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    const int64_t esz = (int64_t)dtype_size(dtype);
    if (!esz || n_tok < 0) return KVQ8_ERR_INVALID_ARG;
    if (n_tok == 0) return KVQ8_OK;
    if (!k || !v || !slots || !k_strides || !v_strides) return KVQ8_ERR_INVALID_ARG;
    PagedIO p = paged_io(kv, slots, n_tok);
    p.y[0] = k;
    p.y[1] = v;
    for (int z = 0; z < 2; ++z) {
        const int64_t* st = z ? v_strides : k_strides;
        p.tok_stride[z] = st[0];
        p.head_stride[z] = st[1];
        if (st[0] < kv->head_dim || st[1] < kv->head_dim) return KVQ8_ERR_INVALID_ARG;
        if ((st[0] * esz) % 16 || (st[1] * esz) % 16) return KVQ8_ERR_MISALIGNED;
    }
    if (!aligned16(k) || !aligned16(v) || !aligned_to(slots, 8)) return KVQ8_ERR_MISALIGNED;
    const int cols = kv->n_kv_heads * (kv->head_dim / 8);
    cudaStream_t s = (cudaStream_t)stream;
    const int padded = cols < 32 ? 32 : cols;  // hd128 with one head has 16 groups a row
    if (dtype == KVQ8_F32) return launch_paged(paged_read_kernel<float>, p, padded, s);
    if (dtype == KVQ8_F16) return launch_paged(paged_read_kernel<__half>, p, padded, s);
    return launch_paged(paged_read_kernel<__nv_bfloat16>, p, padded, s);
}

// paged_cache.cu -- K and V tokens into the pages of a Q8_0 cache by slot (kvq8_paged_append), and back out of them
// as values (kvq8_paged_read).
//
// Append is the block quantiser of kvq8_append (scale max|x| / 127 of 32 values, codes x / scale rounded half away from
// zero) over fp32, fp16 or bf16 tokens, the cache row taken from the token's slot.  Read is its inverse, code * scale
// rounded once to the type asked for.  Both read and write each value once, and are near enough to the memory's rate
// for instructions a value to count: neither has a conversion instruction a value.  16401 tokens of 8 x 128 fp32 into the
// cache and as many slots back as fp16 (238 MB) 48 us in two launches, 4.9 TB/s; with four values a lane and
// conversion instructions 79 us, with twice the tokens a thread 57 us, with fp16 values rounded from fp32 products 52 us.
#include "paged.cuh"
#include "q8_0.cuh"

namespace kvq8 {
namespace {

constexpr int kPagedThreads = 128;
// Tokens of a thread: their loads are in flight together (64 bytes of input in append, 32 of codes in read).
template <typename T>
constexpr int kAppendTok = sizeof(T) == 4 ? 2 : 4;
constexpr int kReadTok = 4;

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

// Block (tx, ty): tx consecutive groups of eight values of a token's row for ty x kAppendTok tokens; grid z is the
// plane.  The four lanes of a 32-value block are in one row (rows hold whole blocks, so a row's groups are a multiple
// of 16, and tx is one too).  Lanes past the row's or the tokens' end, or with a slot outside the cache, quantise zeros
// (every lane takes part in the shuffles) and store nothing.
template <typename T>
__global__ void __launch_bounds__(kPagedThreads) paged_append_kernel(const __grid_constant__ PagedIO p) {
    constexpr int TOK = kAppendTok<T>;
    const int z = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const T* x = static_cast<const T*>(p.x[z]);
    const int g_head = p.head_dim / 8;
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    const bool col_ok = j < p.n_kv_heads * g_head;
    const int h = j / g_head, i = j - h * g_head;
    const int tok0 = (blockIdx.x * blockDim.y + threadIdx.y) * TOK;
    Eight<T> v[TOK];
    int64_t slot[TOK];
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        v[t].clear();
        slot[t] = -1;
        if (col_ok && tok0 + t < p.n_tok) {
            slot[t] = __ldg(p.slots + tok0 + t);
            v[t].load(x + (int64_t)(tok0 + t) * p.tok_stride[z] + (int64_t)j * 8);
        }
    }
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        float f[8];
        v[t].floats(f);
        uint16_t scale_bits;
        const uint2 packed = q8_0_block8(f, &scale_bits);
        if (slot[t] >= 0 && slot[t] < p.n_slots) {
            const uint64_t row = paged_row((uint32_t)slot[t], h, p.n_kv_heads, p.page_shift);
            *reinterpret_cast<uint2*>(p.codes[z] + row * (uint32_t)p.head_dim + i * 8) = packed;
            if ((i & 3) == 0) p.scales[z][row * (uint32_t)(p.head_dim / kQBlock) + (i >> 2)] = scale_bits;
        }
    }
}

// Eight codes times their scale.  fp32 and bf16: 2^23 + (code + 128) by its bits, and a product that is exact in fp32 (8 by 11
// bits); fp16: its product rounds the exact one once as well, subnormals included.
__device__ __forceinline__ void values8(uint2 c, uint16_t scale, float (&v)[8]) {
    const float d = half_bits_to_float(scale);
    const uint32_t lo = c.x ^ 0x80808080u, hi = c.y ^ 0x80808080u;  // code + 128
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = (__uint_as_float(__byte_perm(lo, 0x4b000000u, 0x7440 + k)) - 8388736.0f) * d;
        v[4 + k] = (__uint_as_float(__byte_perm(hi, 0x4b000000u, 0x7440 + k)) - 8388736.0f) * d;
    }
}
__device__ __forceinline__ void store_values(float* dst, uint2 c, uint16_t scale) {
    float v[8];
    values8(c, scale, v);
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_values(__nv_bfloat16* dst, uint2 c, uint16_t scale) {
    float v[8];
    values8(c, scale, v);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store_values(__half* dst, uint2 c, uint16_t scale) {
    const __half2 d = __half2half2(__ushort_as_half(scale));
    const uint32_t lo = c.x ^ 0x80808080u, hi = c.y ^ 0x80808080u;
    uint4 o;
    o.x = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(lo)), d));
    o.y = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(lo)), d));
    o.z = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(hi)), d));
    o.w = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(hi)), d));
    *reinterpret_cast<uint4*>(dst) = o;
}

// The same block shape: eight code bytes and their scale in, eight values out.  A slot outside the cache gives zeros.
template <typename T>
__global__ void __launch_bounds__(kPagedThreads) paged_read_kernel(const __grid_constant__ PagedIO p) {
    const int z = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    T* y = static_cast<T*>(p.y[z]);
    const int g_head = p.head_dim / 8;
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    if (j >= p.n_kv_heads * g_head) return;
    const int h = j / g_head, i = j - h * g_head;
    const int tok0 = (blockIdx.x * blockDim.y + threadIdx.y) * kReadTok;
    uint2 c[kReadTok];
    uint16_t sc[kReadTok];
#pragma unroll
    for (int t = 0; t < kReadTok; ++t) {
        c[t] = make_uint2(0u, 0u);
        sc[t] = 0;
        if (tok0 + t < p.n_tok) {
            const int64_t slot = __ldg(p.slots + tok0 + t);
            if (slot >= 0 && slot < p.n_slots) {
                const uint64_t row = paged_row((uint32_t)slot, h, p.n_kv_heads, p.page_shift);
                c[t] = *reinterpret_cast<const uint2*>(p.codes[z] + row * (uint32_t)p.head_dim + i * 8);
                sc[t] = p.scales[z][row * (uint32_t)(p.head_dim / kQBlock) + (i >> 2)];
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kReadTok; ++t) {
        if (tok0 + t >= p.n_tok) break;
        store_values(y + (int64_t)(tok0 + t) * p.tok_stride[z] + (int64_t)h * p.head_stride[z] + i * 8, c[t], sc[t]);
    }
}

// Whether two of the rows of `len` values at t * tok + h * head (t < n_tok, h < heads) share a value.  Both steps are at least
// len, so rows of one head or one token do not; those h heads apart do where some number of tokens back brings them together.
bool rows_overlap(int64_t tok, int n_tok, int64_t head, int heads, int len) {
    for (int h = 1; h < heads; ++h) {
        const int64_t ahead = h * head, back = ahead / tok < n_tok - 1 ? ahead / tok : n_tok - 1;
        const int64_t next = back + 1 < n_tok - 1 ? back + 1 : n_tok - 1;
        if (ahead - back * tok < len || (next > back && next * tok - ahead < len)) return true;
    }
    return false;
}

// Groups of a row that a block covers and its token rows, whole warps in all: a row's groups are a multiple of 16 (half
// a warp), so an odd multiple takes an even count of rows, or is rounded up where one row fills the block.
dim3 paged_block(int cols) {
    int tx = cols < kPagedThreads ? cols : kPagedThreads, ty = kPagedThreads / tx;
    if (tx % 32) {
        if (ty == 1) tx = (tx + 31) / 32 * 32;
        if (ty > 1) ty &= ~1;
    }
    return dim3((unsigned)tx, (unsigned)ty);
}

template <typename Kernel>
int launch_paged(Kernel* kernel, const PagedIO& p, int cols, int tok, cudaStream_t stream) {
    const dim3 block = paged_block(cols);
    const int64_t per = (int64_t)block.y * tok;
    const int64_t gx = (p.n_tok + per - 1) / per;
    const dim3 grid((unsigned)gx, (unsigned)((cols + block.x - 1) / block.x), 2u);
    return launch_dependent(kernel, grid, block, 0, stream, p);
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
    const int cols = (int)(row / 8);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_paged(paged_append_kernel<float>, p, cols, kAppendTok<float>, s);
    if (dtype == KVQ8_F16) return launch_paged(paged_append_kernel<__half>, p, cols, kAppendTok<__half>, s);
    return launch_paged(paged_append_kernel<__nv_bfloat16>, p, cols, kAppendTok<__nv_bfloat16>, s);
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
    for (int z = 0; z < 2; ++z)
        if (rows_overlap(p.tok_stride[z], n_tok, p.head_stride[z], kv->n_kv_heads, kv->head_dim)) return KVQ8_ERR_INVALID_ARG;
    const int cols = kv->n_kv_heads * (kv->head_dim / 8);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_paged(paged_read_kernel<float>, p, cols, kReadTok, s);
    if (dtype == KVQ8_F16) return launch_paged(paged_read_kernel<__half>, p, cols, kReadTok, s);
    return launch_paged(paged_read_kernel<__nv_bfloat16>, p, cols, kReadTok, s);
}

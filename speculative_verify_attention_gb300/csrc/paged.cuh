// paged.cuh -- the paged Q8_0 cache's addressing and the argument checks that its entry points share.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace kvq8 {

constexpr int kMaxSeqs = 4096;        // requests of one call
constexpr int kMaxWindowRows = 64;    // rows of one request's window: one bit each of a 64-bit mask

// A slot is page * page_size + offset.  Planes: codes [n_pages][n_kv_heads][page_size][head_dim], scales
// [n_pages][n_kv_heads][page_size][head_dim / 32], so a page holds page_size consecutive rows of each head.
// Rows are counted in 32 bits (2^31 of them are more than the device's memory); the row times head_dim (or head_dim / 32) is
// the element offset, in 64 bits.
__device__ __forceinline__ uint32_t paged_row(uint32_t slot, int head, int n_kv_heads, int page_shift) {
    const uint32_t page = slot >> page_shift, off = slot & ((1u << page_shift) - 1);
    return ((page * (uint32_t)n_kv_heads + (uint32_t)head) << page_shift) + off;
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
    if (kv->n_kv_heads > 4096 || (int64_t)kv->n_pages * kv->n_kv_heads * kv->page_size > 0x7fffffffLL) return KVQ8_ERR_UNSUPPORTED;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) || !aligned16(kv->v_scales))
        return KVQ8_ERR_MISALIGNED;
    return KVQ8_OK;
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// 32 bytes that nothing writes while the kernel runs.
__device__ __forceinline__ void load32(uint32_t (&w)[8], const void* at) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(at));
}

// Eight consecutive values in the form they are loaded in, 16 or 32 bytes.
template <typename T>
struct Eight {
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const T* p) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    }
    __device__ __forceinline__ void load_whole(const T* p) { load(p); }  // from their own size's boundary
    __device__ __forceinline__ void put(int i, T v) {
        const uint32_t bits = *reinterpret_cast<const uint16_t*>(&v);
        w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | bits << 16 : (w[i >> 1] & 0xffff0000u) | bits;
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(u32_as_h2(w[k]));
                x[2 * k] = f.x, x[2 * k + 1] = f.y;
            } else {  // a bf16 is the upper half of its fp32
                x[2 * k] = __uint_as_float(w[k] << 16), x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
};
template <>
struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    __device__ __forceinline__ void load(const float* p) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    // (not by the read-only path, which load32 takes: the kernel may write its output to the same place)
    __device__ __forceinline__ void load_whole(const float* p) {
        uint32_t w[8];
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ void put(int i, float x) { v[i] = x; }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i];
    }
};

// A programmatic dependent launch: the kernel's set-up overlaps the end of the kernel before, and it waits for that
// one's writes itself (griddepcontrol.wait).
template <typename Kernel, typename... Args>
inline int launch_dependent(Kernel* kernel, dim3 grid, dim3 block, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace kvq8

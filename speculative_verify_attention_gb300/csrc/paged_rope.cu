// paged_rope.cu -- a step's queries and keys rotated by their positions, and its keys and values quantised into the pages by
// slot, in one launch (kvq8_paged_append_rope).
//
// Pair i of a rotated row turns by positions[axis_of[i]] * f_i:  (a, b) -> (a cos - b sin, b cos + a sin).  A frequency is given
// in turns a position as a 64-bit fraction, so position times frequency, modulo 2^64, is the angle's fraction of a turn whatever
// the position: no rounding but the frequency's own, 2^-64 of a turn a position.  Its two upper bits are the quarter, and what is
// left, within an eighth of a turn of zero, goes through sincospif.
//
// A block works out the sines and cosines of its tokens once for all of their heads; then a thread has sixteen values of a row,
// eight and their partners eight.  Keys are quantised as they come out of the rotation in fp32 (the block quantiser of
// kvq8_paged_append), without a rounding in between.
#include "paged.cuh"
#include "q8_0.cuh"

namespace kvq8 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxAxes = 4;

struct RopeParams {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t* positions;   // [n_axes][n_tok]
    const uint64_t* turns;      // [rot / 2]
    const int32_t* axis_of;     // [rot / 2]
    const int64_t* slots;
    int8_t* codes[2];
    uint16_t* scales[2];
    int64_t n_slots;
    int n_tok, n_q_heads, n_kv_heads, head_shift, page_shift, rot, n_axes;
};

// cos and sin of phase / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // within 2^61
    float s, c;
    sincospif((float)(int32_t)(rest >> 30) * 0x1p-33f, &s, &c);         // half turns
    if (quarter & 1) {
        const float t = c;
        c = -s, s = t;
    }
    if (quarter & 2) c = -c, s = -s;
    return make_float2(c, s);
}

__device__ __forceinline__ void store8(float* dst, const float (&v)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* dst, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = h2_as_u32(__floats2half2_rn(v[2 * k], v[2 * k + 1]));
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight values, not by the read-only path: queries may be rotated in place.
template <typename T>
__device__ __forceinline__ void load_now(Eight<T>& x, const T* from) {
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]) : "l"(from));
}
__device__ __forceinline__ void load_now(Eight<float>& x, const float* from) {
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x.v[0]), "=f"(x.v[1]), "=f"(x.v[2]), "=f"(x.v[3]) : "l"(from));
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x.v[4]), "=f"(x.v[5]), "=f"(x.v[6]), "=f"(x.v[7]) : "l"(from + 4));
}

// (a, b)[i] turned by t[i].
__device__ __forceinline__ void turn(float& a, float& b, float2 t) {
    const float x = a, y = b;
    a = __fmaf_rn(x, t.x, -__fmul_rn(y, t.y));
    b = __fmaf_rn(y, t.x, __fmul_rn(x, t.y));
}

// Eight values at group g of a row, and eight at its partner group h = g + half the groups of their part of the row: the
// rotated part, whose halves turn together (PAIRS: neighbours do, in both groups), or the part behind it.
template <bool PAIRS>
__device__ __forceinline__ void rotate16(float (&a)[8], float (&b)[8], int g, int h, int rot, const float2* t) {
    if (g * 8 >= rot) return;
    if (PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn(a[2 * i], a[2 * i + 1], t[g * 4 + i]);
            turn(b[2 * i], b[2 * i + 1], t[h * 4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(a[i], b[i], t[g * 8 + i]);
    }
}

// Block: `tok` tokens.  The groups g and h of item j of a row: in the rotated part its first and second half, then the same of
// the part behind it; both parts are multiples of 64, so four neighbouring lanes have a 32-value block in each.
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads) paged_rope_kernel(const __grid_constant__ RopeParams p, int tok) {
    extern __shared__ __align__(16) float2 s_turn[];  // [tok][rot / 2]
    const int tid = threadIdx.x, tok0 = blockIdx.x * tok, half = p.rot / 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int toks = min(tok, p.n_tok - tok0);
    for (int i = tid; i < toks * half; i += kRopeThreads) {
        const int t = i / half, j = i - t * half;
        const int axis = p.axis_of ? __ldg(p.axis_of + j) : 0;
        const int64_t pos = axis >= 0 && axis < p.n_axes ? __ldg(p.positions + (int64_t)axis * p.n_tok + tok0 + t) : 0;
        s_turn[i] = cos_sin((uint64_t)pos * __ldg(p.turns + j));
    }
    __syncthreads();
    const int items = 1 << (p.head_shift - 4), hd = 1 << p.head_shift;  // items of a row
    const int rot_items = p.rot / 16, rest = (hd - p.rot) / 16;
    for (int t = 0; t < toks; ++t) {
        const int64_t slot = __ldg(p.slots + tok0 + t);
        if (slot < 0 || slot >= p.n_slots) continue;
        const float2* turns = s_turn + t * half;
        const T* q = static_cast<const T*>(p.q) + (int64_t)(tok0 + t) * p.q_stride;
        T* o = static_cast<T*>(p.q_out) + (int64_t)(tok0 + t) * p.out_stride;
        for (int i = tid; i < p.n_q_heads * items; i += kRopeThreads) {
            const int j = i & (items - 1), row = (i >> (p.head_shift - 4)) << p.head_shift;
            const int g = j < rot_items ? j : rot_items + j, h = g + (j < rot_items ? rot_items : rest);
            Eight<T> ra, rb;
            load_now(ra, q + row + g * 8);
            load_now(rb, q + row + h * 8);
            float a[8], b[8];
            ra.floats(a);
            rb.floats(b);
            rotate16<PAIRS>(a, b, g, h, p.rot, turns);
            store8(o + row + g * 8, a);
            store8(o + row + h * 8, b);
        }
        const int n = 2 * p.n_kv_heads * items;  // keys, then values; every lane of a warp takes part in the shuffles
        for (int i0 = 0; i0 < n; i0 += kRopeThreads) {
            const int i = i0 + tid, j = i & (items - 1), row = i >> (p.head_shift - 4);
            const int z = row >= p.n_kv_heads, head = row - z * p.n_kv_heads;
            const int g = j < rot_items ? j : rot_items + j, h = g + (j < rot_items ? rot_items : rest);
            Eight<T> ra, rb;
            ra.clear();
            rb.clear();
            if (i < n) {
                const T* x = z ? static_cast<const T*>(p.v) + (int64_t)(tok0 + t) * p.v_stride
                               : static_cast<const T*>(p.k) + (int64_t)(tok0 + t) * p.k_stride;
                ra.load(x + (head << p.head_shift) + g * 8);
                rb.load(x + (head << p.head_shift) + h * 8);
            }
            float a[8], b[8];
            ra.floats(a);
            rb.floats(b);
            if (i < n && !z) rotate16<PAIRS>(a, b, g, h, p.rot, turns);
            uint16_t sa, sb;
            const uint2 ca = q8_0_block8(a, &sa), cb = q8_0_block8(b, &sb);
            if (i < n) {
                const uint64_t r = paged_row((uint32_t)slot, head, p.n_kv_heads, p.page_shift);
                int8_t* codes = p.codes[z] + (r << p.head_shift);
                *reinterpret_cast<uint2*>(codes + g * 8) = ca;
                *reinterpret_cast<uint2*>(codes + h * 8) = cb;
                if ((j & 3) == 0) {
                    uint16_t* scales = p.scales[z] + (r << (p.head_shift - 5));
                    scales[g >> 2] = sa;
                    scales[h >> 2] = sb;
                }
            }
        }
    }
}

template <typename T>
int launch_rope(const RopeParams& p, bool pairs, cudaStream_t s) {
    const int tok = p.n_tok >= 2048 ? 4 : 1;
    const unsigned grid = (unsigned)(((int64_t)p.n_tok + tok - 1) / tok);
    const int smem = tok * p.rot / 2 * (int)sizeof(float2);
    if (pairs) return launch_dependent(paged_rope_kernel<T, true>, grid, kRopeThreads, smem, s, p, tok);
    return launch_dependent(paged_rope_kernel<T, false>, grid, kRopeThreads, smem, s, p, tok);
}

}  // namespace
}  // namespace kvq8

extern "C" int kvq8_paged_append_rope(const void* q, const void* k, const void* v, int dtype, int n_tok, int n_q_heads,
                                      int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* positions,
                                      int n_axes, const uint64_t* turns, const int32_t* axis_of, int rot_dim, int pairs,
                                      const kvq8_paged_cache* kv, const int64_t* slots, void* q_out, int64_t out_stride,
                                      kvq8_stream_t stream) {
    using namespace kvq8;
    const int rc = check_paged(kv);
    if (rc != KVQ8_OK) return rc;
    const int64_t esz = (int64_t)dtype_size(dtype);
    if (!esz || n_tok < 0 || n_q_heads < 1 || n_axes < 1) return KVQ8_ERR_INVALID_ARG;
    if (n_tok == 0) return KVQ8_OK;
    const int64_t row = (int64_t)kv->n_kv_heads * kv->head_dim, q_row = (int64_t)n_q_heads * kv->head_dim;
    if (!q || !k || !v || !positions || !turns || !slots || !q_out) return KVQ8_ERR_INVALID_ARG;
    if (q_stride < q_row || out_stride < q_row || k_stride < row || v_stride < row) return KVQ8_ERR_INVALID_ARG;
    // q_out may be q itself; rows of it that meet other rows would be read after they are written
    const uintptr_t out = reinterpret_cast<uintptr_t>(q_out);
    if (q_out == q ? q_stride != out_stride
                   : rows_meet(reinterpret_cast<uintptr_t>(q), q_row * esz, q_stride * esz, out, q_row * esz, out_stride * esz, n_tok))
        return KVQ8_ERR_INVALID_ARG;
    if (rows_meet(reinterpret_cast<uintptr_t>(k), row * esz, k_stride * esz, out, q_row * esz, out_stride * esz, n_tok) ||
        rows_meet(reinterpret_cast<uintptr_t>(v), row * esz, v_stride * esz, out, q_row * esz, out_stride * esz, n_tok))
        return KVQ8_ERR_INVALID_ARG;
    if (rot_dim < 64 || rot_dim % 64 || rot_dim > kv->head_dim || n_axes > kMaxAxes || n_q_heads > 65536) return KVQ8_ERR_UNSUPPORTED;
    for (const void* x : {q, k, v, (const void*)q_out})
        if (!aligned16(x)) return KVQ8_ERR_MISALIGNED;
    for (int64_t st : {q_stride, k_stride, v_stride, out_stride})
        if (st * esz % 16) return KVQ8_ERR_MISALIGNED;
    if (!aligned_to(positions, 4) || !aligned_to(axis_of, 4) || !aligned_to(turns, 8) || !aligned_to(slots, 8)) return KVQ8_ERR_MISALIGNED;
    RopeParams p = {q, k, v, q_out, q_stride, k_stride, v_stride, out_stride, positions, turns, axis_of, slots,
                    {const_cast<int8_t*>(kv->k_codes), const_cast<int8_t*>(kv->v_codes)},
                    {const_cast<uint16_t*>(kv->k_scales), const_cast<uint16_t*>(kv->v_scales)},
                    (int64_t)kv->n_pages * kv->page_size, n_tok, n_q_heads, kv->n_kv_heads, log2_of(kv->head_dim),
                    log2_of(kv->page_size), rot_dim, n_axes};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_rope<float>(p, pairs != 0, s);
    if (dtype == KVQ8_F16) return launch_rope<__half>(p, pairs != 0, s);
    return launch_rope<__nv_bfloat16>(p, pairs != 0, s);
}

// paged_rope.cu -- a step's queries and keys rotated by their positions, and its keys and values quantised into the pages by
// slot, in one launch (kvq8_paged_append_rope).
//
// Pair i of a rotated row turns by positions[axis_of[i]] * f_i:  (a, b) -> (a cos - b sin, b cos + a sin).  A frequency is given
// in turns a position as a 64-bit fraction, so position times frequency, modulo 2^64, is the angle's fraction of a turn whatever
// the position: no rounding but the frequency's own, 2^-64 of a turn a position.  Its two upper bits are the quarter, and what is
// left, within an eighth of a turn of zero, goes through sincospif: cut to 2^-34 of a turn, and rounded to fp32, half a step of which
// is 2^-28 of a turn at most.
//
// A block works out the sines and cosines of its tokens, two or four, once for all of its heads.  A thread has sixteen values of a
// row, eight and their partners eight, the same ones of several heads: its eight sines and cosines stay in its registers.  What it
// will work on next is fetched by asynchronous copies into its own places in shared memory, some heads ahead and on into its next
// tokens, so that neither the sines nor a barrier holds the loads up.  Keys are quantised as they come out of the rotation in fp32
// (the block quantiser of kvq8_paged_append), without a rounding in between.
// Bound: bytes and issue slots together.  16401 tokens of 32q/8kv/hd128 bf16 (372 MB) 65 us, 5.7 TB/s, 84 % of a copy's rate, 63 % of
// the issue slots; 2051 of 24q/4kv/hd256 fp32 (122 MB) 22 us; 32 tokens 3.6 us.  With the next head alone ahead, in registers, 76 and
// 26.5 us; with more blocks an SM (and spills) 74; two or six heads ahead instead of four 66.  Few heads leave some of eight warps idle
// between two barriers, so a block may take two groups of tokens, four warps each: 18788 tokens of 8q/2kv/hd128 bf16 25 us (33 with one),
// 8000 of 12q/1kv/hd256 24.5 (27.6); 16401 of 32q/8kv 72 with two, 67 with one.
#include "paged.cuh"
#include "q8_0.cuh"

namespace kvq8 {
namespace {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
template <typename T>
constexpr int kRopeDepth = sizeof(T) == 4 ? 3 : 4;   // heads of a thread in flight
template <typename T>
constexpr int kRopeBlocks = sizeof(T) == 4 ? 2 : 3;  // of an SM
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
    int n_tok, n_q_heads, n_kv_heads, page_shift, rot, n_axes;
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

// Eight values, four at `dst` and four `apart` behind them.
__device__ __forceinline__ void store8(float* dst, int apart, const float (&v)[8]) {
    *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(dst + apart) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* dst, int, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = h2_as_u32(__floats2half2_rn(v[2 * k], v[2 * k + 1]));
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, int, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T>
__device__ __forceinline__ void from_shared(Eight<T>& x, const uint4* at) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 r = at[i * kRopeThreads];
        reinterpret_cast<uint32_t*>(&x)[4 * i] = r.x, reinterpret_cast<uint32_t*>(&x)[4 * i + 1] = r.y;
        reinterpret_cast<uint32_t*>(&x)[4 * i + 2] = r.z, reinterpret_cast<uint32_t*>(&x)[4 * i + 3] = r.w;
    }
}

// The cosines and sines of a thread's eight pairs.  Halves turn two pairs an instruction: (c, c'), (s, s') and (-s, -s').
template <bool PAIRS>
struct Turns {
    F2 c[4], s[4], minus[4];
    __device__ __forceinline__ void load(const float2* t, int at0, int at1, int) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(t + (i < 2 ? at0 : at1) + 2 * (i & 1));
            c[i] = F2::of(x.x, x.z);
            s[i] = F2::of(x.y, x.w);
            minus[i] = F2::of(-x.y, -x.w);
        }
    }
    // a cos - b sin, b cos + a sin: a product rounded once, and the sum once
    __device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 x = F2::of(a[2 * i], a[2 * i + 1]), y = F2::of(b[2 * i], b[2 * i + 1]);
            fma2(x, c[i], mul2(y, minus[i])).get(a[2 * i], a[2 * i + 1]);
            fma2(y, c[i], mul2(x, s[i])).get(b[2 * i], b[2 * i + 1]);
        }
    }
};
template <>
struct Turns<true> {
    float2 t[8];
    __device__ __forceinline__ void load(const float2* from, int at0, int at1, int far) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(from + ((i & 1 ? at1 : at0) + (i < 2 ? 0 : far)) / 2);
            t[2 * i] = make_float2(x.x, x.y), t[2 * i + 1] = make_float2(x.z, x.w);
        }
    }
    __device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& u = i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)];
            float& v = i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1];
            const float x = u, y = v;
            u = __fmaf_rn(x, t[i].x, -__fmul_rn(y, t[i].y));
            v = __fmaf_rn(y, t[i].x, __fmul_rn(x, t[i].y));
        }
    }
};

// Block (every gridDim.x-th group of two or four tokens, or of twice as many, half of the warps each; a share of the heads): the lanes of a warp are the items of its tokens' rows, its
// heads every eighth (or fourth) of the block's, queries, then keys, then values.  An item is eight values and the eight that lie `far` behind
// them: in the rotated part of a row the same places of its two halves, then of the two halves of the part behind it; both parts are
// multiples of 64, so four neighbouring lanes have a 32-value block in each.  A lane's eight of a block are consecutive (16 bytes); of
// fp32 they are its fourth of the block's first half and of the second, as four lanes' pieces have to fill whole 32-byte sectors.
template <typename T, int HD, bool PAIRS, int SUBS>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks<T>) paged_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kItems = HD / 16, kTokens = 32 / kItems, kAll = kTokens * SUBS, kWarps = kRopeWarps / SUBS, kPieces = (int)sizeof(T) / 2, kDepth = kRopeDepth<T>;  // 16-byte pieces of eight values
    extern __shared__ __align__(16) uint4 s_ring[];               // [kDepth][2 kPieces][threads]
    __shared__ __align__(16) float2 s_turns[2][kAll * HD / 2];  // [tokens][rot / 2], of this group and the next
    const int tid = threadIdx.x, lane = tid & 31, j = lane % kItems, mine = (tid >> 5) / kWarps * kTokens + lane / kItems;
    const int rot_items = p.rot / 16, half = p.rot / 2, stride = (int)gridDim.x * kAll;
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int kApart = kWide ? 16 : 4;  // between a lane's first four values and its next
    const int g = j < rot_items ? j : rot_items + j, far = j < rot_items ? half : (HD - p.rot) / 2;
    const int at = kWide ? (g >> 2) * 32 + (g & 3) * 4 : g * 8;
    const bool turned = j < rot_items;
    // this warp's heads: of the queries, then of the keys, then of the values
    const int step = kWarps * (int)gridDim.y, warp = (int)blockIdx.y * kWarps + (tid >> 5) % kWarps;
    const int all = p.n_q_heads + 2 * p.n_kv_heads, v_first = p.n_q_heads + p.n_kv_heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t ring = smem_u32(s_ring + tid);
    int ahead_tok = (int)blockIdx.x * kAll + mine, ahead = warp, ahead_place = 0;
    auto fetch = [&] {
        if (ahead_tok < p.n_tok && ahead < all) {
            const T* x = ahead < p.n_q_heads ? static_cast<const T*>(p.q) + (int64_t)ahead_tok * p.q_stride + ahead * HD
                         : ahead < v_first   ? static_cast<const T*>(p.k) + (int64_t)ahead_tok * p.k_stride + (ahead - p.n_q_heads) * HD
                                             : static_cast<const T*>(p.v) + (int64_t)ahead_tok * p.v_stride + (ahead - v_first) * HD;
            x += at;
            const uint32_t to = ring + ahead_place * (2 * kPieces * kRopeThreads * 16);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                cp_async_16(to + i * (kRopeThreads * 16), x + i * kApart, 16);
                cp_async_16(to + (kPieces + i) * (kRopeThreads * 16), x + far + i * kApart, 16);
            }
        }
        cp_async_commit();
        ahead += step;
        if (ahead >= all) ahead = warp, ahead_tok += stride;
        ahead_place = ahead_place + 1 == kDepth ? 0 : ahead_place + 1;
    };
    for (int i = 0; i < kDepth; ++i) fetch();
    // as many threads a token as a row has pairs at most; what a group needs of indexes is loaded a group ahead
    const int pair = tid % (HD / 2), pair_tok = tid / (HD / 2);
    uint64_t frequency = 0;
    const int32_t* positions = nullptr;
    if (pair < half) {
        const int axis = p.axis_of ? __ldg(p.axis_of + pair) : 0;
        frequency = __ldg(p.turns + pair);
        if (axis >= 0 && axis < p.n_axes) positions = p.positions + (int64_t)axis * p.n_tok;
    }
    int32_t next_pos[SUBS];
    int64_t next_slot = -1;
    auto indexes = [&](int tok0) {
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
            const int tok = tok0 + u * kTokens + pair_tok;
            next_pos[u] = positions && tok < p.n_tok ? __ldg(positions + tok) : 0;
        }
        next_slot = tok0 + mine < p.n_tok ? __ldg(p.slots + tok0 + mine) : -1;
    };
    indexes((int)blockIdx.x * kAll);
    int buffer = 0, place = 0;
    for (int tok0 = (int)blockIdx.x * kAll; tok0 < p.n_tok; tok0 += stride, buffer ^= 1) {
        const int64_t slot = next_slot;
        const bool there = slot >= 0 && slot < p.n_slots;
#pragma unroll
        for (int u = 0; u < SUBS; ++u)
            if (pair < half) s_turns[buffer][(u * kTokens + pair_tok) * half + pair] = cos_sin((uint64_t)(int64_t)next_pos[u] * frequency);
        if (tok0 + stride < p.n_tok) indexes(tok0 + stride);
        __syncthreads();  // (the other buffer's readers have passed the barrier before)
        Turns<PAIRS> turns;
        if (turned) turns.load(s_turns[buffer] + mine * half, at, at + kApart, far);
        T* o = static_cast<T*>(p.q_out) + (int64_t)(tok0 + mine) * p.out_stride + (warp * HD + at);
        const uint32_t row0 = there ? paged_row((uint32_t)slot, 0, p.n_kv_heads, p.page_shift) : 0;
        for (int head = warp; head < all; head += step) {
            cp_async_wait<kDepth - 1>();
            const uint4* from = s_ring + place * (2 * kPieces * kRopeThreads) + tid;
            place = place + 1 == kDepth ? 0 : place + 1;
            Eight<T> ra, rb;
            from_shared(ra, from);
            from_shared(rb, from + kPieces * kRopeThreads);
            float a[8], b[8];
            ra.floats(a);
            rb.floats(b);
            if (turned && head < v_first) turns.rotate(a, b);
            if (head < p.n_q_heads) {
                if (there) {
                    store8(o, kApart, a);
                    store8(o + far, kApart, b);
                }
                o += step * HD;
            } else {
                uint16_t sa, sb;  // every lane takes part in the shuffles
                const uint2 ca = q8_0_block8(a, &sa), cb = q8_0_block8(b, &sb);
                if (there) {
                    const bool value = head >= v_first;
                    const uint64_t row = row0 + ((uint32_t)(head - (value ? v_first : p.n_q_heads)) << p.page_shift);
                    int8_t* codes = p.codes[value] + (row * HD + at);
                    if (kWide) {
                        *reinterpret_cast<uint32_t*>(codes) = ca.x;
                        *reinterpret_cast<uint32_t*>(codes + kApart) = ca.y;
                        *reinterpret_cast<uint32_t*>(codes + far) = cb.x;
                        *reinterpret_cast<uint32_t*>(codes + far + kApart) = cb.y;
                    } else {
                        *reinterpret_cast<uint2*>(codes) = ca;
                        *reinterpret_cast<uint2*>(codes + far) = cb;
                    }
                    if ((j & 3) == 0) {
                        uint16_t* scales = p.scales[value] + (row * (HD / kQBlock) + (g >> 2));
                        scales[0] = sa;
                        scales[far >> 5] = sb;
                    }
                }
            }
            fetch();  // into the place just read
        }
    }
    cp_async_wait<0>();
}

template <typename T, int HD, bool PAIRS, int SUBS>
int launch_rope(const RopeParams& p, cudaStream_t s) {
    constexpr int kTokens = 32 / (HD / 16) * SUBS, kWarps = kRopeWarps / SUBS;
    const int64_t groups = ((int64_t)p.n_tok + kTokens - 1) / kTokens, full = 152 * kRopeBlocks<T>;
    // as many blocks as the GPU holds; few tokens: their heads over more blocks, a head a warp at last
    const int64_t most = (p.n_q_heads + 2 * p.n_kv_heads + kWarps - 1) / kWarps, share = full / groups;
    const unsigned gy = (unsigned)(share < 1 ? 1 : share < most ? share : most);
    const unsigned gx = (unsigned)(groups < full ? groups : full);
    constexpr int smem = kRopeDepth<T> * (int)sizeof(T) * kRopeThreads * 16;
    static SmemOptIn opt;
    const int rc = opt.ensure(paged_rope_kernel<T, HD, PAIRS, SUBS>, smem);
    if (rc != KVQ8_OK) return rc;
    return launch_dependent(paged_rope_kernel<T, HD, PAIRS, SUBS>, dim3(gx, gy), kRopeThreads, smem, s, p);
}
template <typename T, int HD, bool PAIRS>
int launch_rope(const RopeParams& p, cudaStream_t s) {
    constexpr int kTokens = 32 / (HD / 16);
    const int64_t full = 152 * kRopeBlocks<T>;
    // A block's heads, a head a warp at a time, and half as much again for the sines and the barrier, as often as the blocks come round.
    auto rounds = [&](int subs) {
        const int64_t groups = (p.n_tok + kTokens * subs - 1) / (kTokens * subs), warps = kRopeWarps / subs;
        return (groups + full - 1) / full * (2 * ((p.n_q_heads + 2 * p.n_kv_heads + warps - 1) / warps) + 3);
    };
    return p.n_tok > full * kTokens && rounds(2) < rounds(1) ? launch_rope<T, HD, PAIRS, 2>(p, s)
                                                             : launch_rope<T, HD, PAIRS, 1>(p, s);
}
template <typename T>
int launch_rope(const RopeParams& p, int head_dim, bool pairs, cudaStream_t s) {
    if (head_dim == 128) return pairs ? launch_rope<T, 128, true>(p, s) : launch_rope<T, 128, false>(p, s);
    return pairs ? launch_rope<T, 256, true>(p, s) : launch_rope<T, 256, false>(p, s);
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
    // what says where a later token goes and how far it turns is read while earlier ones' queries are written
    const size_t tok = (size_t)n_tok, half = (size_t)rot_dim / 2;
    const struct {
        const void* at;
        size_t bytes;
    } reads[] = {{positions, tok * n_axes * 4}, {turns, half * 8}, {axis_of, half * 4}, {slots, tok * 8}};
    for (const auto& r : reads)
        if (range_meets_rows(r.at, r.bytes, q_out, q_row * esz, out_stride * esz, n_tok)) return KVQ8_ERR_INVALID_ARG;
    RopeParams p = {q, k, v, q_out, q_stride, k_stride, v_stride, out_stride, positions, turns, axis_of, slots,
                    {const_cast<int8_t*>(kv->k_codes), const_cast<int8_t*>(kv->v_codes)},
                    {const_cast<uint16_t*>(kv->k_scales), const_cast<uint16_t*>(kv->v_scales)},
                    (int64_t)kv->n_pages * kv->page_size, n_tok, n_q_heads, kv->n_kv_heads, log2_of(kv->page_size), rot_dim, n_axes};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_rope<float>(p, kv->head_dim, pairs != 0, s);
    if (dtype == KVQ8_F16) return launch_rope<__half>(p, kv->head_dim, pairs != 0, s);
    return launch_rope<__nv_bfloat16>(p, kv->head_dim, pairs != 0, s);
}

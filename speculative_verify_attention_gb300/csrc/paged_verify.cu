// paged_verify.cu -- verify attention of a batch of windows over a paged Q8_0 cache (attn_verify_paged_q8).
//
// Row t of request b (window of T rows after ctx = len - T cached tokens) sees every key n < ctx and the window
// key ctx + j where bit j of its mask is set (chains: j <= t):
//   o = sum_n p_n v_n / sum_n p_n,  p_n = exp(scale * q . k_n),  k and v = code * scale of their block.
// Scores, references, sums and O are fp32; keys, values and weights enter the products as fp16 (code * scale and the weight
// each rounded once), bf16 queries as fp16 after a scaling by a power of two (exact but for elements 2^25 below the largest
// that is scaled with them).  Each of the three roundings is off by about 2e-4 of its value, as is that of an fp16 output: 4.1e-4
// to 4.3e-4 in all, and 1.7e-3 with bf16 outputs, which is those outputs' own rounding.  The calls over one contiguous cache keep
// pairs of fp16 for K, V and the weights, and fp32 outputs (1.6e-5).  Pairs here would mean every product twice and, in the tile
// kernels, V^ twice in shared memory, which has no room for it at head_dim 256; the outputs are 16 bits wide.
// A row's sum is of its weights as rounded, so that equal values come out as they are.
//
// Three kernels, by the T x group rows of the longest window and KV head:
//   up to 8 (16 at head_dim 128): here, a warp scans for itself on mma.sync;
//   up to 64, many keys an SM:    paged_verify_stream.cu, tcgen05 with keys as the tile's rows and fetch rings;
//   the others:                   paged_verify_rows.cu, tcgen05 with the window's rows as the tile's rows, and teams of CTAs
//                                 above 192.
#include "paged_verify.cuh"

namespace kvq8 {

unsigned int* device_error_flag();

namespace {

// ---------------------------------------------------------------- few rows

// Up to 8 rows a window and KV head (16 at head_dim 128): the tensor-core tiles above would be mostly empty and their
// hand-offs and per-tile instructions would bound the scan, so here a warp does everything for its own 16 keys at a time,
// on mma.sync and without shared memory: loads straight into registers in fragment order, S^T = K^ Q^T, softmax, and
// O^T += V^T P^T with O^T in registers.  All warps run the same short loop and never wait for one another until the
// segment's end, where their (o, m, l) are joined through shared memory.
//   K : lane (g, c) = (lane / 4, lane % 4) holds the 32-value block c of keys g and g + 8: word s of a block feeds k-step s
//       (the contraction runs over the dims in the order block 0's, 1's, 2's, 3's word s), Q is laid out alike;
//   V : lane (g, c) holds dims 16 g .. 16 g + 15 of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9: two keys' bytes interleaved are the
//       fp16 pairs of the transposed operand;
//   P^T comes from the scores' fragments by an 8 x 8 transpose.
// The next 16 keys' codes are requested as soon as a register is free, and 32 keys' further ahead into L2.
template <int HD, int NT>
struct FL {
    // Warps of a CTA and CTAs of an SM.  At head_dim 128 two CTAs of 6 warps have 168 registers a thread; at 256 that
    // spills, and one CTA of 8 warps has 255.  Measured both ways: 64 requests of 8192 tokens at head_dim 128 151 us
    // against 171 us, 20 requests of 16000 tokens at head_dim 256 42 us against 33 us.  (9 to 16 rows at head_dim 128, NT = 2,
    // spill 52 bytes with bf16 queries and 100 with fp16; all other shapes spill nothing.)
    static constexpr int kWarps = HD == 256 ? 8 : 6, kCtas = HD == 256 ? 1 : 2;
    static constexpr int N = 8 * NT, H = HD / 128;           // rows; 128-dim halves
    static constexpr int kSmO = 0, kSmMl = kWarps * N * HD * 4, kSmBytes = kSmMl + kWarps * N * 8;
};

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint4 load16(const int8_t* at) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at));
    return v;
}

template <typename T, int HD, int NT>
__global__ void __launch_bounds__(FL<HD, NT>::kWarps * 32, FL<HD, NT>::kCtas) paged_verify_few_kernel(const __grid_constant__ PagedVerifyParams p) {
    using L = FL<HD, NT>;
    constexpr int W = L::kWarps, H = L::H, N = L::N, KEYS = 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Place place;
    __shared__ long long s_warp[W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    float* s_o = reinterpret_cast<float*>(smem + L::kSmO);        // [warp][row][dim]
    float2* s_ml = reinterpret_cast<float2*>(smem + L::kSmMl);    // [warp][row]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_place<KEYS, W * 32>(p, &place, s_warp);
    __syncthreads();
    Walk<KEYS> walk = walk_from<KEYS>(p, place);
    Segment next;
#pragma unroll 1
    while (walk.next(p, next)) {
        const Segment seg = next;
        const int len = seg.q.len, ctx = len - seg.q.rows, t1 = seg.t1;
        // queries: row 8 n + g, dims 32 c + 4 s .. + 3 of each half, as k-step s of the B operand
        uint32_t q[NT][H][16];
        float cs = p.scale_log2;
        {
            uint32_t top = 0;
            uint4 raw[NT][H][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = 8 * n + g, t = window_row(p, r);
                const uint16_t* src = static_cast<const uint16_t*>(p.q) + (int64_t)(seg.q.row0 + t) * p.q_stride +
                                      (int64_t)(seg.kvh * p.group + r - t * p.group) * HD + 32 * c;
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        raw[n][h][i] = r < seg.n ? __ldg(reinterpret_cast<const uint4*>(src + 128 * h) + i) : make_uint4(0u, 0u, 0u, 0u);
                        top = max(top, Query<T>::top(raw[n][h][i]));
                    }
            }
            float lifted = 1.0f;
            if (Query<T>::kLifted) lifted = lift_of(__reduce_max_sync(0xffffffffu, top));
            cs = p.scale_log2 / lifted;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = raw[n][h][i];
                        q[n][h][4 * i] = Query<T>::pair(v.x, lifted);
                        q[n][h][4 * i + 1] = Query<T>::pair(v.y, lifted);
                        q[n][h][4 * i + 2] = Query<T>::pair(v.z, lifted);
                        q[n][h][4 * i + 3] = Query<T>::pair(v.w, lifted);
                    }
        }
        float o[H * 8][NT][4], neg[NT][2], l[NT][2];
#pragma unroll
        for (int m = 0; m < H * 8; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) o[m][n][0] = o[m][n][1] = o[m][n][2] = o[m][n][3] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) neg[n][0] = neg[n][1] = kLift - kNoRef, l[n][0] = l[n][1] = 0.0f;

        // the cache row of a 16-key group (one page holds it), -1 where there is none
        const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
        auto page_at = [&](int t) { return t < t1 ? __ldg(pages + (((long long)t * KEYS) >> p.page_shift)) : -1; };
        auto row_at = [&](int t, int page) {
            const int off = (int)(((unsigned)t * KEYS) & ((1u << p.page_shift) - 1));
            return page >= 0 && page < p.n_pages ? (((int64_t)page * p.n_kv_heads + seg.kvh) << p.page_shift) + off : (int64_t)-1;
        };
        uint32_t kw[2][H][8], kd[2][H];
        uint4 vw[4][H];
        uint32_t vd[4][H];
        auto load_k = [&](int64_t row, int keys) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool on = row >= 0 && g + 8 * i < keys;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    if (on) {
                        load32(kw[i][h], p.kc + (row + g + 8 * i) * HD + 128 * h + 32 * c);
                        kd[i][h] = __ldg(p.ks + (row + g + 8 * i) * (HD / 32) + 4 * h + c);
                    } else {
#pragma unroll
                        for (int s = 0; s < 8; ++s) kw[i][h][s] = 0u;
                        kd[i][h] = 0u;
                    }
                }
            }
        };
        auto load_v = [&](int64_t row, int keys) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 2 * c + (i & 1) + 8 * (i >> 1);
                const bool on = row >= 0 && key < keys;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    if (on) {
                        vw[i][h] = load16(p.vc + (row + key) * HD + 128 * h + 16 * g);
                        vd[i][h] = __ldg(p.vs + (row + key) * (HD / 32) + 4 * h + (g >> 1));
                    } else {
                        vw[i][h] = make_uint4(0u, 0u, 0u, 0u);
                        vd[i][h] = 0u;
                    }
                }
            }
        };
        int t = seg.t0 + warp;
        int64_t row = row_at(t, page_at(t)), row1 = row_at(t + W, page_at(t + W));
        int page2 = page_at(t + 2 * W);
        auto keys_of = [&](int t) { return (int)min((long long)len - (long long)t * KEYS, (long long)KEYS); };
        if (t < t1) {
            load_k(row, keys_of(t));
            load_v(row, keys_of(t));
        }
#pragma unroll 1
        for (; t < t1; t += W) {
            // the group after the next into L2: 16 rows of codes are consecutive, and so are their scales
            const int64_t row2 = row_at(t + 2 * W, page2);
            page2 = page_at(t + 3 * W);
            if (row2 >= 0) {
                const int8_t* codes = lane < 16 ? p.kc : p.vc;
#pragma unroll
                for (int h = 0; h < H; ++h) prefetch_l2(codes + row2 * HD + ((lane & 15) + 16 * h) * 128);
                if (lane < 2 * H) prefetch_l2((lane < H ? p.ks : p.vs) + row2 * (HD / 32) + (lane % H) * 64);
            }
            float sc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const __half2 d0 = __half2half2(__ushort_as_half((unsigned short)kd[0][h])), d1 = __half2half2(__ushort_as_half((unsigned short)kd[1][h]));
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t w0 = kw[0][h][s] ^ 0x80808080u, w1 = kw[1][h][s] ^ 0x80808080u;
                    const uint32_t a0 = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(w0)), d0));
                    const uint32_t a1 = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(w1)), d1));
                    const uint32_t a2 = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(w0)), d0));
                    const uint32_t a3 = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(w1)), d1));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16_16816(sc[n], a0, a1, a2, a3, q[n][h][2 * s], q[n][h][2 * s + 1]);
                }
            }
            const int keys = row >= 0 ? keys_of(t) : 0, keys1 = t + W < t1 ? keys_of(t + W) : 0;
            load_k(keys1 ? row1 : (int64_t)-1, keys1);
            // masks: keys that are not there, and in the window those without their bit
            const long long key0 = (long long)t * KEYS;
            if (keys < KEYS || key0 + KEYS > ctx) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * n + 2 * c + e, wt = window_row(p, r);
                        uint64_t m = 0;
                        if (r < seg.n) m = p.mask ? __ldg(p.mask + seg.q.row0 + wt) : (2ull << wt) - 1;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int key = g + 8 * i;
                            const long long at = key0 + key - ctx;  // place in the window
                            if (key >= keys || (at >= 0 && !(m >> (at & 63) & 1))) sc[n][2 * i + e] = -INFINITY;
                        }
                    }
            }
            float x[NT][4];
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                float over = -INFINITY;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[n][i] = fmaf(sc[n][i], cs, neg[n][i & 1]);
                        over = fmaxf(over, x[n][i]);
                    }
                if (pass || !__any_sync(0xffffffffu, over > kLazy + kLift)) break;
                // references to the maxima where a score passed one by more than 2^8; sums and O^T follow
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(sc[n][e], sc[n][2 + e]) * cs;
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                        const float ref = kLift - neg[n][e];
                        a[e] = 1.0f;
                        if (m > ref + kLazy) {
                            a[e] = neg[n][e] == kLift - kNoRef ? 0.0f : ex2_approx(ref - m);
                            neg[n][e] = kLift - m;
                        }
                        l[n][e] *= a[e];
                    }
#pragma unroll
                    for (int m = 0; m < H * 8; ++m) o[m][n][0] *= a[0], o[m][n][1] *= a[1], o[m][n][2] *= a[0], o[m][n][3] *= a[1];
                }
            }
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const __half2 h0 = __floats2half2_rn(ex2_approx(x[n][0]), ex2_approx(x[n][1]));
                const __half2 h1 = __floats2half2_rn(ex2_approx(x[n][2]), ex2_approx(x[n][3]));
                const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                l[n][0] += f0.x + f1.x;
                l[n][1] += f0.y + f1.y;
                b0[n] = transpose8(h2_as_u32(h0));
                b1[n] = transpose8(h2_as_u32(h1));
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const __half2 d01 = __halves2half2(__ushort_as_half((unsigned short)vd[0][h]), __ushort_as_half((unsigned short)vd[1][h]));
                const __half2 d23 = __halves2half2(__ushort_as_half((unsigned short)vd[2][h]), __ushort_as_half((unsigned short)vd[3][h]));
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t w0 = (s == 0 ? vw[0][h].x : s == 1 ? vw[0][h].y : s == 2 ? vw[0][h].z : vw[0][h].w) ^ 0x80808080u;
                    const uint32_t w1 = (s == 0 ? vw[1][h].x : s == 1 ? vw[1][h].y : s == 2 ? vw[1][h].z : vw[1][h].w) ^ 0x80808080u;
                    const uint32_t w2 = (s == 0 ? vw[2][h].x : s == 1 ? vw[2][h].y : s == 2 ? vw[2][h].z : vw[2][h].w) ^ 0x80808080u;
                    const uint32_t w3 = (s == 0 ? vw[3][h].x : s == 1 ? vw[3][h].y : s == 2 ? vw[3][h].z : vw[3][h].w) ^ 0x80808080u;
                    const uint32_t lo01 = prmt2<0x5140>(w0, w1), hi01 = prmt2<0x7362>(w0, w1);
                    const uint32_t lo23 = prmt2<0x5140>(w2, w3), hi23 = prmt2<0x7362>(w2, w3);
                    auto half2_of = [&](uint32_t x, __half2 d, bool upper) {
                        return h2_as_u32(__hmul2(u32_as_h2(upper ? biased_bytes_to_half2<0x4342>(x) : biased_bytes_to_half2<0x4140>(x)), d));
                    };
                    const uint32_t a0 = half2_of(lo01, d01, false), a1 = half2_of(lo01, d01, true);
                    const uint32_t a2 = half2_of(lo23, d23, false), a3 = half2_of(lo23, d23, true);
                    const uint32_t e0 = half2_of(hi01, d01, false), e1 = half2_of(hi01, d01, true);
                    const uint32_t e2 = half2_of(hi23, d23, false), e3 = half2_of(hi23, d23, true);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16_16816(o[8 * h + 2 * s][n], a0, a1, a2, a3, b0[n], b1[n]);
                        mma_f16_16816(o[8 * h + 2 * s + 1][n], e0, e1, e2, e3, b0[n], b1[n]);
                    }
                }
            }
            load_v(keys1 ? row1 : (int64_t)-1, keys1);
            row = row1;
            row1 = row2;
        }

        // the warps' parts: (reference, sum) and O of each row; o[m] holds dims 16 g + 2 (m % 8) and the next of half m / 8
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
                const int r = 8 * n + 2 * c + e;
                if (g == 0) s_ml[warp * N + r] = make_float2(neg[n][e] == kLift - kNoRef ? -INFINITY : kLift - neg[n][e], l[n][e]);
#pragma unroll
                for (int m = 0; m < H * 8; ++m)
                    *reinterpret_cast<float2*>(s_o + (warp * N + r) * HD + 128 * (m >> 3) + 16 * g + 2 * (m & 7)) = make_float2(o[m][n][e], o[m][n][2 + e]);
            }
        __syncthreads();
        const bool whole = seg.begins() && seg.ends();
        const int slot = 2 * blockIdx.x + (seg.begins() ? 1 : 0);
#pragma unroll 1
        for (int i = tid; i < seg.n * (HD / 4); i += W * 32) {
            const int r = i / (HD / 4), d = i - r * (HD / 4);
            float m = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) m = fmaxf(m, s_ml[w * N + r].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 ml = s_ml[w * N + r];
                const float a = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
                const float4 v = reinterpret_cast<const float4*>(s_o + (w * N + r) * HD)[d];
                sum += a * ml.y;
                acc.x += a * v.x, acc.y += a * v.y, acc.z += a * v.z, acc.w += a * v.w;
            }
            if (whole) {
                const int t = window_row(p, r);
                const int64_t out_row = (int64_t)(seg.q.row0 + t) * p.n_q_heads + seg.kvh * p.group + r - t * p.group;
                const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // (NaN stays one)
                reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + out_row * HD)[d] =
                    sum != 0.0f ? make_uint2(Query<T>::out(acc.x * inv, acc.y * inv), Query<T>::out(acc.z * inv, acc.w * inv)) : make_uint2(0u, 0u);
            } else {
                reinterpret_cast<float4*>(p.part_o + ((int64_t)slot * p.chunk + r) * HD)[d] = acc;
                if (d == 0) p.part_ml[(int64_t)slot * p.chunk + r] = make_float2(m, sum);
            }
        }
        __syncthreads();  // before the next segment's parts
    }
    if (tid == 0) leave_join<KEYS>(p, place);
}

// ---------------------------------------------------------------- joining the partials

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// The rows of every item that was cut, one after another: o = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c over its
// parts, slot 1 of the CTA that began it and slot 0 of the same place in the later teams.  A row is a warp's, or where there
// are no more rows than blocks a block's, whose warps share its parts (a long context of few rows has a part per CTA).
// The whole call with a block a row throughout, with a warp a row throughout, and so: 16 trees, 9200 rows of two or three
// parts, 215, 193 and 194 us; one chain of 24 rows over 2048 tokens 15.5, 22.3 and 15.1 us, over 20676 28.2, 35.7 and 27.6 us.
template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedVerifyParams p, int n_ctas) {
    constexpr int V = HD / 128;  // float4 columns of a lane
    __shared__ int4 s_join[1024];
    __shared__ int s_first[1025];
    __shared__ float4 s_o[kJoinWarps][HD / 4];
    __shared__ float2 s_ml[kJoinWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int c = tid; c < n_ctas; c += kJoinThreads) s_join[c] = p.joins[c];
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
        for (int c0 = 0; c0 < n_ctas; c0 += 32) {
            const int n = c0 + lane < n_ctas && s_join[c0 + lane].w >= 0 ? s_join[c0 + lane].z >> 16 : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            if (c0 + lane < n_ctas) s_first[c0 + lane] = sum + inc - n;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) s_first[n_ctas] = sum;
    }
    __syncthreads();
    const int tasks = s_first[n_ctas];
    const bool shared = tasks <= (int)gridDim.x;  // a row is the block's
    const int first = shared ? blockIdx.x : blockIdx.x * kJoinWarps + warp, step = shared ? gridDim.x : gridDim.x * kJoinWarps;
    for (int task = first; task < tasks; task += step) {
        int lo = 0, hi = n_ctas;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_first[mid] <= task)
                lo = mid;
            else
                hi = mid;
        }
        const int c0 = lo, r = task - s_first[c0], parts = s_join[c0].w - c0 / p.team + 1;
        auto slot = [&](int i) { return (int64_t)(2 * (c0 + i * p.team) + (i == 0 ? 1 : 0)) * p.chunk + r; };
        // this warp's parts, four at a time, against a running maximum
        float m = -INFINITY, l = 0.0f;
        float4 acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int i0 = shared ? warp : 0, di = shared ? kJoinWarps : 1;
        for (int i = i0; i < parts; i += 4 * di) {
            float2 ml[4];
            float4 o[4][V];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool on = i + u * di < parts;
                const int64_t at = slot(on ? i + u * di : i);
                ml[u] = p.part_ml[at];
                if (!on) ml[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int v = 0; v < V; ++v) o[u][v] = reinterpret_cast<const float4*>(p.part_o)[at * (HD / 4) + 32 * v + lane];
            }
            const float top = fmaxf(m, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
            const float a = m == -INFINITY ? 0.0f : ex2_approx(m - top);
            m = top;
            l *= a;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v].x *= a, acc[v].y *= a, acc[v].z *= a, acc[v].w *= a;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (ml[u].x == -INFINITY && ml[u].y == 0.0f) continue;  // a part that saw no key, or none (its o may be anything)
                const float w = ex2_approx(ml[u].x - m);
                l += w * ml[u].y;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    acc[v].x += w * o[u][v].x, acc[v].y += w * o[u][v].y, acc[v].z += w * o[u][v].z, acc[v].w += w * o[u][v].w;
            }
        }
        const int rr = (s_join[c0].z & 0xffff) + r, t = rr / p.group;
        const int head = s_join[c0].y * p.group + rr - t * p.group;
        uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((int64_t)(s_join[c0].x + t) * p.n_q_heads + head) * HD);
        auto put = [&](int col, float4 o, float sum) {
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            dst[col] = sum != 0.0f ? make_uint2(Query<T>::out(o.x * inv, o.y * inv), Query<T>::out(o.z * inv, o.w * inv)) : make_uint2(0u, 0u);
        };
        if (!shared) {
#pragma unroll
            for (int v = 0; v < V; ++v) put(32 * v + lane, acc[v], l);
            continue;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[warp][32 * v + lane] = acc[v];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (tid < HD / 4) {
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float a = s_ml[w].x == -INFINITY ? 0.0f : ex2_approx(s_ml[w].x - top);
                const float4 x = s_o[w][tid];
                sum += a * s_ml[w].y;
                o.x += a * x.x, o.y += a * x.y, o.z += a * x.z, o.w += a * x.w;
            }
            put(tid, o, sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        sms = 152;
    return sms < 512 ? sms : 512;  // the joining kernel lists at most 1024 CTAs
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

enum { kFew = 0, kTiles = 1 };

struct VerifyPlan {
    int route, ctas, chunk, team;  // CTAs; most rows of one; CTAs that share an item's rows
    size_t ml_off, join_off, bytes;
};

// With more key tiles (of 64) than this an SM, by the tables' capacity, windows of up to 64 rows go to the streaming kernel: it
// has a deep ring of fetches but takes longer to start, and its time grows with the rows.  Requests far shorter than their
// table's width so get the streaming kernel where the other would be faster: the lengths are on the device, and the choice of a
// captured call stays.  Measured, streaming and by rows, us (tiles an SM by capacity):
//   4 KV heads of 256 dims, 6 query heads each: 1 request of 2048 tokens (1), 8 of 2048 (7), 4 of 20676 (34), 8 of 20676 (68), 16 of 20676 (135)
//     24 rows   24 and 15   37 and 27   53 and 52   72 and 83   104 and 136
//     48 rows   29 and 16   46 and 28   68 and 57   86 and 85   124 and 138
//     60 rows   34 and 17   45 and 28   68 and 59   90 and 86   132 and 139
//   8 KV heads of 128 dims, 4 query heads each: 1 of 2048 (2), 8 of 8192 (53), 4 of 20676 (68), 8 of 20676 (135), 16 of 20676 (270)
//     24 rows   24 and 18   53 and 53   60 and 63    87 and 108   142 and 196
//     48 rows   29 and 19   63 and 55   70 and 66   101 and 111   176 and 201
//     60 rows   34 and 20   72 and 57   78 and 67   115 and 112   200 and 203
inline int stream_tiles(int rows) { return rows <= 32 ? 40 : 80; }

// The lengths are on the device, so all of this is by the longest window and the capacity.
VerifyPlan verify_plan(int sms, int group, int hd, int max_rows) {
    VerifyPlan v;
    const int rows = max_rows * group;
    v.route = rows <= (hd == 128 ? 16 : 8) ? kFew : kTiles;
    v.ctas = v.route == kFew ? (hd == 128 ? FL<128, 1>::kCtas : FL<256, 1>::kCtas) * sms : sms;
    v.team = (rows + 191) / 192;
    v.chunk = (rows + v.team - 1) / v.team;
    v.ml_off = up256((size_t)v.ctas * 2 * v.chunk * hd * sizeof(float));
    v.join_off = v.ml_off + up256((size_t)v.ctas * 2 * v.chunk * sizeof(float2));
    v.bytes = v.join_off + (size_t)v.ctas * sizeof(int4);
    return v;
}
// The code plane as rows of head_dim bytes; a box is 128 bytes of `box` consecutive keys of a page.
bool encode_codes(CUtensorMap* map, const int8_t* codes, const kvq8_paged_cache* kv, int box) {
    const EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)kv->head_dim, (cuuint64_t)kv->n_pages * kv->n_kv_heads * kv->page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)kv->head_dim};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, ones[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(codes), dims, strides, boxes, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int HD, int NT>
int launch_few(const PagedVerifyParams& p, const VerifyPlan& v, cudaStream_t s) {
    using L = FL<HD, NT>;
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_few_kernel<T, HD, NT>, L::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    return launch_dependent(paged_verify_few_kernel<T, HD, NT>, v.ctas, L::kWarps * 32, L::kSmBytes, s, p);
}

template <typename T, int HD>
int launch_verify(PagedVerifyParams& p, const VerifyPlan& v, const kvq8_paged_cache* kv, int dtype, cudaStream_t s) {
    int rc;
    if (v.route == kFew) {
        rc = HD == 128 && v.chunk > 8 ? launch_few<T, 128, 2>(p, v, s) : launch_few<T, HD, 1>(p, v, s);
    } else {
        const int64_t tiles = (int64_t)p.n_seqs * p.n_kv_heads * ((((int64_t)p.max_pages << p.page_shift) + 63) / 64);
        if (v.chunk <= 64 && v.team == 1 && tiles > (int64_t)stream_tiles(v.chunk) * v.ctas) {
            p.box = kv->page_size < 64 ? kv->page_size : 64;
            if (!encode_codes(&p.tmap_k, kv->k_codes, kv, p.box) || !encode_codes(&p.tmap_v, kv->v_codes, kv, p.box)) return KVQ8_ERR_CUDA;
            rc = launch_verify_stream(p, dtype, HD, v.chunk, v.ctas, s);
        } else {
            rc = launch_verify_rows(p, dtype, HD, v.chunk, v.ctas, s);
        }
    }
    if (rc != KVQ8_OK) return rc;
    return launch_dependent(paged_join_kernel<T, HD>, 4 * sm_count(), kJoinThreads, 0, s, p, v.ctas);
}

}  // namespace
}  // namespace kvq8

extern "C" size_t attn_verify_paged_q8_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim, int max_rows) {
    using namespace kvq8;
    if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64) return 0;
    if ((head_dim != 128 && head_dim != 256) || max_rows < 1 || max_rows > kMaxWindowRows) return 0;
    return verify_plan(sm_count(), n_q_heads / n_kv_heads, head_dim, max_rows).bytes;
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
    const int group = n_q_heads / kv->n_kv_heads;
    const VerifyPlan v = verify_plan(sm_count(), group, kv->head_dim, max_rows);
    if (!workspace || workspace_bytes < v.bytes) return KVQ8_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (q_stride * 2) % 16 || !aligned_to(page_table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(row_starts, 4) || !aligned_to(window_mask, 8))
        return KVQ8_ERR_MISALIGNED;
    if (!aligned_to(kv->k_codes, 32) || !aligned_to(kv->v_codes, 32)) return KVQ8_ERR_MISALIGNED;  // whole blocks per load
    unsigned int* error = device_error_flag();
    if (!error) return KVQ8_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    PagedVerifyParams p = {q, out, q_stride, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, page_table, lens,
                                 row_starts, window_mask, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + v.ml_off),
                                 reinterpret_cast<int4*>(ws + v.join_off), error, n_rows, n_q_heads, kv->n_kv_heads, group,
                                 kv->n_pages, log2_of(kv->page_size), max_pages, n_seqs, max_rows, v.chunk, v.team,
                                 softmax_scale * kLog2e, 1.0f / (float)group};
    cudaStream_t s = (cudaStream_t)stream;
    if (kv->head_dim == 128)
        return dtype == KVQ8_F16 ? launch_verify<__half, 128>(p, v, kv, dtype, s) : launch_verify<__nv_bfloat16, 128>(p, v, kv, dtype, s);
    return dtype == KVQ8_F16 ? launch_verify<__half, 256>(p, v, kv, dtype, s) : launch_verify<__nv_bfloat16, 256>(p, v, kv, dtype, s);
}

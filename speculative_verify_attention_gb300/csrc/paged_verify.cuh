// paged_verify.cuh -- what the kernels of attn_verify_paged_q8 share: parameters, how the work is cut, queries and codes
// as fp16, and bounded waits.
//
// Work: the (request, KV head) items, each ceil(len / KEYS) key tiles, laid end to end and cut into one equal share per
// CTA (or team of CTAs, for windows of more rows than one holds: CTA k of a team takes the k-th part of each item's rows, so
// the team reads the same tiles at the same time and all but the first find them in L2).  Every CTA works its share out by
// itself from the lengths on the device (one scan over the requests), so nothing waits for the host and a captured call
// follows new lengths.  A share holds at most one item that it did not begin and one that it does not end: those leave a
// partial (o, m, l) in the CTA's two workspace slots, joined by a second kernel; items wholly inside a share are written at
// once.
#pragma once

#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace kvq8 {

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
    float* part_o;     // [grid][2][chunk][HD]
    float2* part_ml;   // [grid][2][chunk] (m in log2 units, l)
    int4* joins;       // [grid]: the item that CTA c begins and does not end (first q row, KV head, rows, last team)
    unsigned int* error;
    int n_rows, n_q_heads, n_kv_heads, group, n_pages, page_shift, max_pages, n_seqs, max_rows, chunk, team;
    float scale_log2, per_group;  // per_group = 1 / group
    // code planes as (head_dim bytes, rows of n_pages * n_kv_heads * page_size), boxes of 128 bytes x `box` keys
    CUtensorMap tmap_k, tmap_v;
    int box;
};

// The tile kernels of paged_verify_stream.cu and paged_verify_rows.cu, for head_dim hd and windows of up to n rows a CTA.
int launch_verify_stream(const PagedVerifyParams& p, int dtype, int hd, int n, int ctas, cudaStream_t s);
int launch_verify_rows(const PagedVerifyParams& p, int dtype, int hd, int n, int ctas, cudaStream_t s);

namespace {

constexpr long long kPatience = 1ll << 31;  // cycles that a wait may take: about a second
constexpr float kLazy = 8.0f;               // the references follow only jumps of more than 2^8
constexpr float kLift = 6.0f;               // p is 2^6 larger than 2^(s - ref): at most 2^14, and fp16 keeps it to 2^-30
constexpr float kNoRef = -1e30f;            // the reference of a row that has seen no key yet
constexpr uint32_t kTmemCols = 512;

// ---------------------------------------------------------------- the shares

// A request as the kernel sees it; tiles = 0 where there is nothing to do or its numbers make no sense.
struct Request {
    int len, rows, row0, tiles;
};

template <int KEYS>
__device__ __forceinline__ Request request_of(const PagedVerifyParams& p, int b) {
    Request q;
    q.row0 = __ldg(p.row_starts + b);
    const int end = __ldg(p.row_starts + b + 1);
    q.len = __ldg(p.lens + b);
    q.rows = end - q.row0;
    const bool good = q.row0 >= 0 && end <= p.n_rows && end > q.row0 && q.rows <= p.max_rows && q.rows <= q.len &&
                      (int64_t)q.len <= ((int64_t)p.max_pages << p.page_shift);
    q.tiles = good ? (int)(((unsigned)q.len + KEYS - 1) / KEYS) : 0;
    return q;
}

// Part of an item: key tiles [t0, t1) for rows [r0, r0 + n) of KV head kvh of request b.
struct Segment {
    int b, kvh, r0, n, t0, t1;
    Request q;
    __device__ __forceinline__ bool begins() const { return t0 == 0; }
    __device__ __forceinline__ bool ends() const { return t1 == q.tiles; }
};

// A CTA's share, segment by segment, in tiles of KEYS keys.
template <int KEYS>
struct Walk {
    int b, kvh, t;
    long long left;
    Request q;

    // (one copy of the code for all roles: it runs once a segment)
    __device__ __noinline__ bool next(const PagedVerifyParams& p, Segment& s) {
#pragma unroll 1
        while (left > 0) {
#pragma unroll 1
            while (kvh == p.n_kv_heads || q.tiles == 0) {
                kvh = 0;
                if (++b >= p.n_seqs) return false;
                q = request_of<KEYS>(p, b);
            }
            // the team's equal parts of the rows, so that no CTA pays for a tile of a few rows; a window of few rows may leave
            // the last CTAs of the team none
            const int rows = q.rows * p.group;
            int r0 = 0, n = rows;
            if (p.team > 1) {
                const int per = (rows + p.team - 1) / p.team;
                r0 = (int)(blockIdx.x % p.team) * per;
                n = min(per, rows - r0);
            }
            const int t0 = t, kv_head = kvh;
            t = (int)min((long long)q.tiles, t0 + left);
            const int t1 = t;
            left -= t1 - t0;
            if (t == q.tiles) {
                t = 0;
                ++kvh;
            }
            // the caller's segment changes only where it gets a new one: after the last, it is still the last
            if (n > 0) {
                s.b = b;
                s.kvh = kv_head;
                s.r0 = r0;
                s.n = n;
                s.t0 = t0;
                s.t1 = t1;
                s.q = q;
                return true;
            }
        }
        return false;
    }
};

// The window row of row rr of an item, rr / group: rr is below 2^12 and group at most 64, so rr + 1/2 is further from a
// multiple of group than the product's rounding.
__device__ __forceinline__ int window_row(const PagedVerifyParams& p, int rr) { return (int)(((float)rr + 0.5f) * p.per_group); }

__device__ __noinline__ long long divide(long long a, long long b) { return a / b; }

// Shares of u units: every team below `shares` gets base of them, the first `rest` one more.
struct Shares {
    long long base, rest;
    int shares;
    __device__ __forceinline__ long long begin(int c) const { return c < shares ? c * base + min((long long)c, rest) : base * shares + rest; }
};

// Exclusive sum over a block of THREADS of one value per thread, and the total; all threads call it.
template <int THREADS>
__device__ __forceinline__ long long block_exclusive(long long v, long long* s_warp, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    return before + inc - v;
}

// A CTA's place: its share [u0, u1) of all units, how they were cut, and where it starts.
struct Place {
    Shares cut;
    long long units, u0, u1;
    int b, kvh, t;
};

// Every thread of the block calls it; `place` and `s_warp` (THREADS / 32 words) are in shared memory, and `place` is whole
// after the block's next barrier.
template <int KEYS, int THREADS>
__device__ __forceinline__ void find_place(const PagedVerifyParams& p, Place* place, long long* s_warp) {
    const int tid = threadIdx.x;
    const int per = (p.n_seqs + THREADS - 1) / THREADS;
    const int b_lo = min(tid * per, p.n_seqs), b_hi = min(b_lo + per, p.n_seqs);
    long long mine = 0, units;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) mine += (long long)request_of<KEYS>(p, b).tiles * p.n_kv_heads;
    const long long before = block_exclusive<THREADS>(mine, s_warp, units);
    if (tid == 0) {
        // no more shares than units: every share of an item that was cut has tiles of it, and so a partial
        Shares cut;
        cut.shares = (int)min(units, (long long)(gridDim.x / p.team));
        cut.base = cut.shares ? divide(units, cut.shares) : 0;
        cut.rest = units - cut.base * cut.shares;
        place->cut = cut;
        place->units = units;
        place->u0 = cut.begin(blockIdx.x / p.team);
        place->u1 = cut.begin(blockIdx.x / p.team + 1);
    }
    __syncthreads();
    const long long u0 = place->u0;
    if (u0 < place->u1 && before <= u0 && u0 < before + mine) {
        long long at = before;
#pragma unroll 1
        for (int b = b_lo; b < b_hi; ++b) {
            const Request q = request_of<KEYS>(p, b);
            const long long here = (long long)q.tiles * p.n_kv_heads;
            if (u0 < at + here) {
                place->b = b;
                place->kvh = (int)divide(u0 - at, q.tiles);
                place->t = (int)(u0 - at - (long long)place->kvh * q.tiles);
                break;
            }
            at += here;
        }
    }
}

template <int KEYS>
__device__ __forceinline__ Walk<KEYS> walk_from(const PagedVerifyParams& p, const Place& place) {
    Walk<KEYS> w;
    w.left = place.u1 - place.u0;
    w.b = p.n_seqs;
    w.kvh = w.t = 0;
    w.q.tiles = 0;
    if (w.left > 0) {
        w.b = place.b;
        w.kvh = place.kvh;
        w.t = place.t;
        w.q = request_of<KEYS>(p, w.b);
    }
    return w;
}

// What one thread leaves for the joining kernel: the item that this CTA begins and does not end, under its number.  It can only
// be the last one that it has rows of; where the share ends on an item without, the one before ended in the share.
template <int KEYS>
__device__ __forceinline__ void leave_join(const PagedVerifyParams& p, const Place& place) {
    int4 join = make_int4(0, 0, 0, -1);
    Walk<KEYS> walk = walk_from<KEYS>(p, place);
    Segment seg;
    bool any = false;
#pragma unroll 1
    while (walk.next(p, seg)) any = true;
    if (any && seg.begins() && !seg.ends()) {
        const long long last = place.u1 - seg.t1 + seg.q.tiles - 1;  // the item's last unit
        const long long longer = place.cut.rest * (place.cut.base + 1);
        const long long team = last < longer ? divide(last, place.cut.base + 1)
                                             : place.cut.rest + divide(last - longer, place.cut.base);
        join = make_int4(seg.q.row0, seg.kvh, seg.r0 | seg.n << 16, (int)team);
    }
    p.joins[blockIdx.x] = join;
}

// ---------------------------------------------------------------- operands

// Sixteen codes as eight fp16 pairs, code * scale rounded once.
__device__ __forceinline__ void values16(uint4 codes, __half2 scale, uint32_t* h) {
    const uint32_t w[4] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u, codes.z ^ 0x80808080u, codes.w ^ 0x80808080u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[2 * e] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(w[e])), scale));
        h[2 * e + 1] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(w[e])), scale));
    }
}

// Queries as fp16 pairs.  fp16 rows go in as they are; bf16 rows of a chunk times one power of two that brings the
// chunk's largest element into [2^14, 2^15), undone in the scores' scale.  A row 2^k below the largest keeps its
// precision to 2^(39 - k) below its own largest, and its scores are as much smaller.
template <typename T>
struct Query;
template <>
struct Query<__half> {
    static constexpr bool kLifted = false;
    static __device__ __forceinline__ uint32_t top(uint4) { return 0u; }
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float) { return w; }
    static __device__ __forceinline__ uint32_t out(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
    static __device__ __forceinline__ uint16_t one(float a) { return __half_as_ushort(__float2half_rn(a)); }
};
template <>
struct Query<__nv_bfloat16> {
    static constexpr bool kLifted = true;
    // The bits of the largest finite magnitude.  NaN and infinity have no part in it: they stay what they are under any
    // power of two, and one of them must not decide how the other rows are scaled.
    static __device__ __forceinline__ uint32_t top(uint4 v) {
        uint32_t t = 0;
        for (uint32_t w : {v.x, v.y, v.z, v.w}) {
            const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
            t = max(t, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
        }
        return t;
    }
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float lifted) {
        return h2_as_u32(__floats2half2_rn(__uint_as_float(w << 16) * lifted, __uint_as_float(w & 0xffff0000u) * lifted));
    }
    static __device__ __forceinline__ uint32_t out(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint16_t one(float a) { return __bfloat16_as_ushort(__float2bfloat16_rn(a)); }
};

// The power of two that brings a finite bf16 magnitude (its bits) into [2^14, 2^15); 1 for zeros and subnormals.
__device__ __forceinline__ float lift_of(uint32_t top) {
    const int e = (int)(top >> 7);
    if (e == 0) return 1.0f;
    return __uint_as_float((uint32_t)min(127 + 127 + 14 - e, 254) << 23);
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one;
}

__device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

// The waits of one role: each gives up after kPatience, and from then on the role runs without waiting, so that every loop
// ends and every named barrier is met; its results mean nothing, and the role reports the time-out when it is done.
struct Waits {
    uint32_t bar;
    bool ok;
    __device__ __forceinline__ void operator()(int id, int phase) {
        if (!ok) return;
        const uint32_t at = bar + 8u * (uint32_t)id, parity = (uint32_t)phase & 1u;
        if (tc::mbar_try_wait(at, parity)) return;
        const long long from = clock64();
#pragma unroll 1
        do {
            if (tc::mbar_try_wait(at, parity)) return;
        } while (clock64() - from < kPatience);
        ok = false;
    }
};

}  // namespace
}  // namespace kvq8

// paged_verify.cu -- verify attention of a batch of windows over a paged Q8_0 cache (attn_verify_paged_q8).
//
// Row t of request b (window of T rows after ctx = len - T cached tokens) sees every key n < ctx and the window
// key ctx + j where bit j of its mask is set (chains: j <= t):
//   o = sum_n p_n v_n / sum_n p_n,  p_n = exp(scale * q . k_n),  k and v = code * scale of their block.
//
// The T x group rows of a window and KV head (t * group + hh) are few and the keys many, so the products are taken
// transposed: keys, then dims, are the M = 128 rows of the tcgen05 tiles, the window's rows their N columns.
//   S^T [128 keys x N]  = K^ [keys x dims] Q^T  : A = K^ in tensor memory, B = Q in shared memory (K-major)
//   O^T [dims x N]     += V^ [keys x dims]^T P^T : A = V^ (MN-major), B = P [keys x rows] (MN-major), shared memory
// A tile costs the tensor cores 2 HD / 16 instructions of N columns (about 44 cycles each up to N = 64) where rows as
// M = 128 cost the full tile whatever the window.
//
// Work: the (request, KV head) items, each ceil(len / 128) key tiles, laid end to end and cut into one equal share per
// team of C CTAs, C = the row chunks of the batch's longest window; CTA k of a team takes the k-th part of each item's
// rows, so the team's CTAs read the same tiles at the same time and all but the first find them in L2.  Every CTA works
// its share out by itself from the lengths on the device (one scan over the requests), so nothing waits for the host
// and a captured call follows new lengths.  A share holds at most one item that it did not begin and one that it does
// not end: those leave a partial (o, m, l) in the CTA's two workspace slots, joined by the second kernel; items wholly
// inside a share are written at once.
//
// Warps of a CTA (every wait is an mbarrier wait with an iteration limit; a role that ran out of patience flags the
// error and goes on without waiting, so every loop ends and every named barrier is met):
//   0-3   softmax, one key per thread: p = 2^(s - ref) against a reference maximum per row kept in shared memory.
//         The references follow only jumps of more than 2^8, found by one vote per tile.
//   4     issues S^T = K^ Q^T
//   5     issues O^T += V^T P^T and, as one more 128-row tile with ones for V, the row sums of the fp16 weights: fp32 sums
//         of what the product uses.  (Exchanges between the lanes cost the softmax warps as much as the softmax, and
//         mma.sync waits behind the products.)
//   8-11  K: one key per thread, codes to fp16 (code * scale, rounded once) into tensor memory
//   12-19 V: units of 8 keys x 4 blocks into a 128-byte-swizzled tile in shared memory, 64 keys at a time
//   20-23 fetch K (20, 21) and V (22, 23) into rings of 64-key slots, most of shared memory: codes by tensor copies of up
//         to a page (128-byte swizzle), scales by asynchronous copies.  A load takes about 2 us under load: an SM's share
//         of the memory's rate is some 90 KB in flight.  (Loads held in the converters' registers had 40 KB in flight,
//         copies issued by the converters took as many instructions as the conversion, and one warp a plane was bound
//         by its issue: 60-100 ns a copy.)
// Keys on page ids outside the pool are not fetched.  Those and the rows behind len in a page enter V^ as zeros, and
// their scores are masked whatever they are.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace kvq8 {

unsigned int* device_error_flag();

namespace {

constexpr int BN = 128;                     // keys of a tile
constexpr int kQkWarp = 4, kPvWarp = 5, kKWarp0 = 8, kVWarp0 = 12, kFetchWarp0 = 20;
constexpr int kVerifyThreads = 768;
constexpr int kSoftThreads = 128;
constexpr uint32_t kPollLimit = 1u << 24;
constexpr float kLazy = 8.0f;               // the references follow only jumps of more than 2^8
constexpr float kLift = 6.0f;               // p is 2^6 larger than 2^(s - ref): at most 2^14, and fp16 keeps it to 2^-30
constexpr float kNoRef = -1e30f;            // the reference of a row that has seen no key yet
constexpr uint32_t kTmemCols = 512;

// Shapes: NMAX rows of a chunk, 32 or 64; NK tiles of K^ in tensor memory, NV of V^ and two of weights in shared memory;
// the fetch rings take what is left of that.  Up to 32 rows the two weight tiles are the halves of one 64-row atom.
template <int HD, int NMAX>
struct VL {
    static constexpr bool kSmall = NMAX <= 32;
    static constexpr int NK = HD == 256 && !kSmall ? 1 : 2, NV = HD == 256 ? 1 : 2;
    static constexpr int kTile = BN * HD * 2;
    static constexpr int kPNext = kSmall ? 64 : BN * 128;  // from one weight tile to the other
    static constexpr int kSmV = 0, kSmQ = NV * kTile, kSmP = kSmQ + HD / 64 * NMAX * 128;
    static constexpr int kSmTab = kSmP + (kSmall ? 1 : 2) * BN * 128;
    // tables: per row reference, lifted negative reference, factor of the last raise, output row and window mask (two
    // segments each); maxima per softmax warp
    static constexpr int kTabRef = 0, kTabNeg = kTabRef + 4 * NMAX, kTabAlpha = kTabNeg + 4 * NMAX,
                         kTabRow = kTabAlpha + 4 * NMAX, kTabMax = kTabRow + 8 * NMAX, kTabMask = kTabMax + 16 * NMAX,
                         kTabMisc = kTabMask + 16 * NMAX;
    static constexpr int kSmScan = kSmTab + kTabMisc + 32, kSmTmem = kSmScan + 64 + (kVerifyThreads / 32) * 8;
    static constexpr int kSmBar = kSmTmem + 16;
    // fetch slots: 64 keys of codes, [128-byte half of the head][key][128 bytes] with the 16-byte chunks of key n at
    // chunk ^ n % 8; their scales apart
    static constexpr int kCodes = 64 * HD, kScales = 64 * HD / 16, kMaxSlots = 16;
    static constexpr int kSmSlots = (kSmBar + (2 * kMaxSlots + 17) * 8 + 1023) / 1024 * 1024;
    static constexpr int kFit = (227 * 1024 - kSmSlots) / (kCodes + kScales), R = kFit < kMaxSlots ? kFit : kMaxSlots;
    // K and V have rings of their own (slots 0 .. RK - 1 and the rest), and a K slot always serves the same half of a tile:
    // every wait is then for the use just before or the one after it, by roles that saw that one, as parities need
    static constexpr int RK = (R + 1) / 2 / 2 * 2, RV = R - RK;
    static constexpr int kSmScales = kSmSlots + R * kCodes, kSmBytes = kSmScales + R * kScales;
    // barriers: fetch slot full / free; 64-key halves of V^ written / used (two of each tile); then pairs by tile: K^
    // written, scores ready, weights ready, product done; then queries ready
    static constexpr int kFull = 0, kFree = R, kV = 2 * R, kVFree = kV + 4, kK = kVFree + 4, kS = kK + 2, kP = kS + 2, kO = kP + 2,
                         kQ = kO + 2;
    static constexpr int kMt = HD / 128;  // 128-dim tiles of O^T; one more of as many columns holds the row sums
    static constexpr uint32_t kTmO = 0, kTmSum = kMt * NMAX, kTmS = kTmSum + NMAX, kTmK = kTmS + 2 * NMAX,
                              kTmOnes = kTmK + NK * HD / 2;
    static_assert(kTmOnes + 16 <= kTmemCols, "tensor memory");
    static_assert(RK >= 2 && RV >= 2 && kSmBytes <= 227 * 1024, "shared memory: a tile of each at least");
    static_assert(kSmQ % 1024 == 0 && kSmP % 1024 == 0, "swizzled tiles stay 1024-byte aligned");
};

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
            s.b = b;
            s.kvh = kvh;
            // the team's equal parts of the rows, so that no CTA pays for a tile of a few rows
            const int rows = q.rows * p.group;
            s.r0 = 0;
            s.n = rows;
            if (p.team > 1) {
                const int per = (rows + p.team - 1) / p.team;
                s.r0 = (int)(blockIdx.x % p.team) * per;
                s.n = min(per, rows - s.r0);
            }
            s.t0 = t;
            s.t1 = (int)min((long long)q.tiles, t + left);
            s.q = q;
            left -= s.t1 - s.t0;
            t = s.t1;
            if (t == q.tiles) {
                t = 0;
                ++kvh;
            }
            if (s.n > 0) return true;  // fewer rows than CTAs in the team: some have none
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

// What one thread leaves for the joining kernel: the item that this CTA begins and does not end, under its number.
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

// ---------------------------------------------------------------- dequantising

// Sixteen codes as eight fp16 pairs, code * scale rounded once.
__device__ __forceinline__ void values16(uint4 codes, __half2 scale, uint32_t* h) {
    const uint32_t w[4] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u, codes.z ^ 0x80808080u, codes.w ^ 0x80808080u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[2 * e] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(w[e])), scale));
        h[2 * e + 1] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(w[e])), scale));
    }
}

// One box of a plane's tensor map into shared memory, completion counted in bytes.  x is 0 or 128: copies start on
// 16-byte boundaries.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
        : "memory");
}

// ---------------------------------------------------------------- queries

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
    // the largest magnitude's bits (NaN and infinity above all)
    static __device__ __forceinline__ uint32_t top(uint4 v) {
        uint32_t t = 0;
        for (uint32_t w : {v.x, v.y, v.z, v.w}) t = max(t, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
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

// The power of two that brings a bf16 magnitude (its bits) into [2^14, 2^15); 1 for zeros, subnormals and what is
// not finite.
__device__ __forceinline__ float lift_of(uint32_t top) {
    const int e = (int)(top >> 7);
    if (e == 0 || e == 255) return 1.0f;
    return __uint_as_float((uint32_t)min(127 + 127 + 14 - e, 254) << 23);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ unsigned short lds16(uint32_t at) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one;
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, 1, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

// Maximum over a warp of floats, by their order-preserving integers.
__device__ __forceinline__ float warp_max(float x) {
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

template <typename T, int HD, int NMAX>
__global__ void __launch_bounds__(kVerifyThreads, 1) paged_verify_kernel(const __grid_constant__ PagedVerifyParams p) {
    using L = VL<HD, NMAX>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem), bar = sbase + L::kSmBar;
    auto B = [&](int id) { return bar + 8u * (uint32_t)id; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSmTmem);
    Place* place = reinterpret_cast<Place*>(smem + L::kSmScan);
    long long* s_warp = reinterpret_cast<long long*>(smem + L::kSmScan + 64);

    if (tid == 0) {
#pragma unroll 1
        for (int s = 0; s < L::R; ++s) {
            tc::mbar_init(B(L::kFull + s), 66);                  // two fetching warps: their bytes and each lane's copies
            tc::mbar_init(B(L::kFree + s), s < L::RK ? 2 : 8);  // the warps that read it
        }
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
            tc::mbar_init(B(L::kV + s), 8);
            tc::mbar_init(B(L::kVFree + s), 1);
        }
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(B(L::kK + s), 4);
            tc::mbar_init(B(L::kS + s), 1);
            tc::mbar_init(B(L::kP + s), 4);
            tc::mbar_init(B(L::kO + s), 1);
        }
        tc::mbar_init(B(L::kQ), 4);
        tc::mbar_init_fence();
    }
    if (warp == kQkWarp) tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    find_place<BN, kVerifyThreads>(p, place, s_warp);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (warp < 4) {
        uint32_t ones[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) ones[i] = 0x3C003C00u;
        tc::tmem_st16(tmem + ((uint32_t)(warp * 32) << 16) + L::kTmOnes, ones);
        tc::tmem_wait_st();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    Walk<BN> walk = walk_from<BN>(p, *place);
    Segment seg;
    bool ok = true;
    // After a time-out the role runs on without waiting.  (Loops in this kernel are kept rolled: the roles' code together
    // should stay in the instruction caches, and stalls for instructions were a quarter of all before.)
    auto wait = [&](int id, int phase) {
        if (!ok) return;
        const uint32_t at = B(id), parity = (uint32_t)phase & 1u;
#pragma unroll 1
        for (uint32_t i = 0; i < kPollLimit; ++i)
            if (tc::mbar_try_wait(at, parity)) return;
        ok = false;
    };

    if (warp == kQkWarp) {
        const uint32_t one = elect_one();
        const uint64_t qd = tc::smem_desc_sw128(sbase + L::kSmQ, 16, 1024);
        int j = 0, segs = 0;
#pragma unroll 1
        while (walk.next(p, seg)) {
            wait(L::kQ, segs++);
            const uint32_t idesc = tc::idesc_f16_f32_ab(BN, (seg.n + 15) & ~15, false, false);
#pragma unroll 1
            for (int t = seg.t0; t < seg.t1; ++t, ++j) {
                wait(L::kK + j % L::NK, j / L::NK);
                if (j >= 2) wait(L::kP + (j & 1), (j - 2) >> 1);  // the scores of tile j - 2 have been read
                tc::fence_after_sync();
                if (one) {
                    const uint32_t d = tmem + L::kTmS + (j & 1) * NMAX, k0 = tmem + L::kTmK + (j % L::NK) * (HD / 2);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        tc::mma_ts(d, k0 + 8 * k, qd + (uint64_t)(((k >> 2) * (NMAX * 128) + (k & 3) * 32) >> 4), idesc,
                                   k > 0 ? 1u : 0u);
                    tc::mma_commit(B(L::kS + (j & 1)));
                }
                __syncwarp();
            }
        }
        if (!ok) atomicOr(p.error, 1u);
    } else if (warp == kPvWarp) {
        const uint32_t one = elect_one();
        const uint64_t vd0 = tc::smem_desc_sw128(sbase + L::kSmV, BN * 128, 1024);
        const uint64_t pd0 = tc::smem_desc_sw128(sbase + L::kSmP, BN * 128, 1024);
        int j = 0;
#pragma unroll 1
        while (walk.next(p, seg)) {
            const uint32_t idesc = tc::idesc_f16_f32_ab(128, (seg.n + 15) & ~15, true, true);
            const uint32_t idesc_sum = tc::idesc_f16_f32_ab(128, (seg.n + 15) & ~15, false, true);
#pragma unroll 1
            for (int t = seg.t0; t < seg.t1; ++t, ++j) {
                wait(L::kP + (j & 1), j >> 1);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int v = 2 * (j % L::NV) + half;
                    wait(L::kV + v, j / L::NV);
                    tc::fence_after_sync();
                    if (one) {
                        const uint64_t vd = vd0 + (uint64_t)(((j % L::NV) * L::kTile + half * 8192) >> 4);
                        const uint64_t pd = pd0 + (uint64_t)(((j & 1) * L::kPNext + half * 8192) >> 4);
                        const uint32_t more = t > seg.t0 || half ? 1u : 0u;
#pragma unroll
                        for (int m = 0; m < L::kMt; ++m)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_ss(tmem + L::kTmO + m * NMAX, vd + (uint64_t)((m * 2 * BN * 128 + k * 2048) >> 4),
                                           pd + (uint64_t)((k * 2048) >> 4), idesc, k > 0 ? 1u : more);
                        tc::mma_commit(B(L::kVFree + v));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_ts(tmem + L::kTmSum, tmem + L::kTmOnes, pd + (uint64_t)((k * 2048) >> 4), idesc_sum, k > 0 ? 1u : more);
                        if (half) tc::mma_commit(B(L::kO + (j & 1)));
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) atomicOr(p.error, 1u);
    } else if (warp < 4) {
        float* ref = reinterpret_cast<float*>(smem + L::kSmTab + L::kTabRef);
        float* neg = reinterpret_cast<float*>(smem + L::kSmTab + L::kTabNeg);
        float* alpha = reinterpret_cast<float*>(smem + L::kSmTab + L::kTabAlpha);
        int* out_row = reinterpret_cast<int*>(smem + L::kSmTab + L::kTabRow);
        float* warp_top = reinterpret_cast<float*>(smem + L::kSmTab + L::kTabMax);
        uint64_t* masks = reinterpret_cast<uint64_t*>(smem + L::kSmTab + L::kTabMask);
        int* misc = reinterpret_cast<int*>(smem + L::kSmTab + L::kTabMisc);  // largest query of each warp
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        float cs = 0.0f, cs_next = 0.0f;

        // Queries of a segment into shared memory ([64-dim atom][row][128 bytes], 16-byte chunks at chunk ^ row % 8)
        // and its rows' tables; rows up to the next 16 are zeros.  Called once every product with the queries before
        // has been read.
        auto stage = [&](const Segment& s, int parity) {
            const int n16 = (s.n + 15) & ~15, pieces = n16 * (HD / 8);
            const int rr = s.r0 + tid, my_t = window_row(p, rr), my_row = s.q.row0 + my_t;
            uint64_t my_mask = 0;
            if (tid < s.n) my_mask = p.mask ? __ldg(p.mask + my_row) : (2ull << my_t) - 1;
            auto at = [&](int i) {  // where piece i (16 bytes of row i / (HD / 8)) lies
                const int r = i / (HD / 8), c = i - r * (HD / 8);
                return L::kSmQ + (c >> 3) * (NMAX * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            };
            // all pieces at once: one round trip to memory
#pragma unroll 4
            for (int i = tid; i < pieces; i += kSoftThreads) {
                const int r = i / (HD / 8), c = i - r * (HD / 8), q_rr = s.r0 + r, t = window_row(p, q_rr);
                const int64_t off = r < s.n ? (int64_t)(s.q.row0 + t) * p.q_stride + (int64_t)(s.kvh * p.group + q_rr - t * p.group) * HD + c * 8 : 0;
                cp_async_16(sbase + at(i), static_cast<const uint16_t*>(p.q) + off, r < s.n ? 16 : 0);
            }
            cp_async_commit();
            cp_async_wait<0>();
            float lifted = 1.0f;
            if (Query<T>::kLifted) {  // a thread reads and rewrites the pieces that it fetched
                uint32_t top = 0;
#pragma unroll 2
                for (int i = tid; i < pieces; i += kSoftThreads) top = max(top, Query<T>::top(*reinterpret_cast<const uint4*>(smem + at(i))));
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) misc[warp] = (int)top;
                soft_sync();
                lifted = lift_of((uint32_t)max(max(misc[0], misc[1]), max(misc[2], misc[3])));
#pragma unroll 2
                for (int i = tid; i < pieces; i += kSoftThreads) {
                    uint4* q16 = reinterpret_cast<uint4*>(smem + at(i));
                    const uint4 v = *q16;
                    *q16 = make_uint4(Query<T>::pair(v.x, lifted), Query<T>::pair(v.y, lifted), Query<T>::pair(v.z, lifted),
                                      Query<T>::pair(v.w, lifted));
                }
            }
            cs_next = p.scale_log2 / lifted;
            if (tid < n16) {
                if (s.q.rows < 64) my_mask &= (1ull << s.q.rows) - 1;
                masks[parity * NMAX + tid] = my_mask;
                out_row[parity * NMAX + tid] = tid < s.n ? my_row * p.n_q_heads + s.kvh * p.group + rr - my_t * p.group : -1;
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B(L::kQ));
        };

        Segment next_seg;
        bool more = walk.next(p, next_seg);
        int j = 0, segs = 0, n16 = 0;
#pragma unroll 1
        while (true) {
            // a segment's queries go in before the one before's output is read: its first scores overlap that
            const int parity = segs & 1;
            if (more) stage(next_seg, parity);
            if (segs > 0) {
                wait(L::kO + ((j - 1) & 1), (j - 1) >> 1);
                tc::fence_after_sync();
                const bool whole = seg.begins() && seg.ends();
                const int slot = 2 * blockIdx.x + (seg.begins() ? 1 : 0);
                const int* rows = out_row + (parity ^ 1) * NMAX;
#pragma unroll 1
                for (int c0 = 0; c0 < n16; c0 += 16) {
                    float inv[16];  // every lane of the sums' tile holds them
                    {
                        uint32_t l[16];
                        tc::tmem_ld16(tmem + lanes + L::kTmSum + c0, l);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float sum = __uint_as_float(l[c]);
                            inv[c] = sum > 0.0f ? 1.0f / sum : 0.0f;
                            if (!whole && tid == c0 + c && tid < seg.n)
                                p.part_ml[(int64_t)slot * p.chunk + tid] = make_float2(ref[tid] == kNoRef ? -INFINITY : ref[tid], sum);
                        }
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int m = 0; m < L::kMt; ++m) {
                        const int dim = m * 128 + tid;
                        uint32_t o[16];
                        tc::tmem_ld16(tmem + lanes + L::kTmO + m * NMAX + c0, o);
                        tc::tmem_wait_ld();
                        if (whole) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const int row = rows[c0 + c];
                                if (row >= 0)
                                    static_cast<uint16_t*>(p.out)[(int64_t)row * HD + dim] =
                                        inv[c] != 0.0f ? Query<T>::one(__uint_as_float(o[c]) * inv[c]) : (uint16_t)0;
                            }
                        } else {
                            float* dst = p.part_o + ((int64_t)slot * p.chunk + c0) * HD + dim;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (c0 + c < seg.n) dst[c * HD] = __uint_as_float(o[c]);
                        }
                    }
                }
                tc::fence_before_sync();
                soft_sync();  // references and output rows have been read
            }
            if (!more) break;
            seg = next_seg;
            cs = cs_next;
            n16 = (seg.n + 15) & ~15;
            const int ctx = seg.q.len - seg.q.rows;
            if (tid < n16) {
                ref[tid] = kNoRef;
                neg[tid] = kLift - kNoRef;
            }
            soft_sync();
            const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
            auto page_of = [&](int t) {  // this thread's key's page, loaded a tile ahead
                const long long key = (long long)t * BN + tid;
                return t < seg.t1 && key < seg.q.len ? __ldg(pages + (key >> p.page_shift)) : 0;
            };
            int page = page_of(seg.t0);
#pragma unroll 1
            for (int t = seg.t0; t < seg.t1; ++t, ++j) {
                const bool bad = page < 0 || page >= p.n_pages;
                page = page_of(t + 1);
                const long long key = (long long)t * BN + tid;
                // what rows see of this key: all of them, none, or those with its bit in their masks
                const int bit = (int)min(key - ctx, (long long)64);
                const bool none = bad || key >= seg.q.len;
                wait(L::kS + (j & 1), j >> 1);
                tc::fence_after_sync();
                const uint32_t scol = tmem + lanes + L::kTmS + (j & 1) * NMAX;
                const bool masked = __any_sync(0xffffffffu, none || bit >= 0);
                auto mask = [&](int c0, float (&x)[16], const uint32_t (&w)[16]) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(w[c]);
                    if (masked) {
                        const uint64_t* m = masks + parity * NMAX + c0;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (none || (bit >= 0 && !(m[c] >> (bit & 63) & 1))) x[c] = -INFINITY;
                    }
                };
                if (j >= 2) wait(L::kO + (j & 1), (j - 2) >> 1);  // the weights of tile j - 2 have been used
                uint8_t* prow = smem + L::kSmP + (L::kSmall ? 0 : (j & 1) * L::kPNext) + tid * 128;
                const int swz = ((L::kSmall ? (j & 1) * 4 : 0) ^ (tid & 7)) << 4;
#pragma unroll 1
                for (int pass = t == seg.t0 ? 0 : 1; pass < 3; ++pass) {
                    if (pass != 1) {
                        // References to the tile's maxima where those are more than 2^8 above; sums and O^T follow.
                        soft_sync();  // every thread has read the old references
#pragma unroll 1
                        for (int c0 = 0; c0 < n16; c0 += 16) {
                            float x[16];
                            uint32_t w[16];
                            tc::tmem_ld16(scol + c0, w);
                            tc::tmem_wait_ld();
                            mask(c0, x, w);
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float m = warp_max(x[c]);
                                if (lane == c) warp_top[warp * NMAX + c0 + c] = m;
                            }
                            __syncwarp();
                        }
                        soft_sync();
                        if (tid < n16) {
                            const float m = cs * fmaxf(fmaxf(warp_top[tid], warp_top[NMAX + tid]),
                                                       fmaxf(warp_top[2 * NMAX + tid], warp_top[3 * NMAX + tid]));
                            const float old = ref[tid];
                            float a = 1.0f;
                            if (m > old + kLazy) {
                                a = old == kNoRef ? 0.0f : ex2_approx(old - m);
                                ref[tid] = m;
                                neg[tid] = kLift - m;
                            }
                            alpha[tid] = a;
                        }
                        if (t > seg.t0) wait(L::kO + ((j - 1) & 1), (j - 1) >> 1);  // every earlier product has landed
                        soft_sync();
                        if (t > seg.t0) {
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int m = 0; m <= L::kMt; ++m)  // the last holds the row sums
#pragma unroll 1
                                for (int c0 = 0; c0 < n16; c0 += 16) {
                                    uint32_t o[16];
                                    tc::tmem_ld16(tmem + lanes + L::kTmO + m * NMAX + c0, o);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c0 + c]);
                                    tc::tmem_st16(tmem + lanes + L::kTmO + m * NMAX + c0, o);
                                }
                            tc::tmem_wait_st();
                        }
                    }
                    // Weights of this key, 16 rows at a time, the next scores on their way meanwhile; does a score pass
                    // its reference by more than 2^8?
                    float over = -INFINITY;
                    uint32_t w[16];
                    tc::tmem_ld16(scol, w);
#pragma unroll 1
                    for (int c0 = 0; c0 < n16; c0 += 16) {
                        float x[16];
                        tc::tmem_wait_ld16(w);
                        mask(c0, x, w);
                        if (c0 + 16 < n16) tc::tmem_ld16(scol + c0 + 16, w);
                        uint32_t h[8];
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 r = *reinterpret_cast<const float4*>(neg + c0 + c);
                            const float e0 = fmaf(x[c], cs, r.x), e1 = fmaf(x[c + 1], cs, r.y), e2 = fmaf(x[c + 2], cs, r.z),
                                        e3 = fmaf(x[c + 3], cs, r.w);
                            over = fmaxf(over, fmaxf(fmaxf(e0, e1), fmaxf(e2, e3)));
                            h[c / 2] = h2_as_u32(__floats2half2_rn(ex2_approx(e0), ex2_approx(e1)));
                            h[c / 2 + 1] = h2_as_u32(__floats2half2_rn(ex2_approx(e2), ex2_approx(e3)));
                        }
                        *reinterpret_cast<uint4*>(prow + (swz ^ (c0 << 1))) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(prow + (swz ^ (c0 << 1) ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    if (!soft_any(over > kLazy + kLift)) break;
                }
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(B(L::kP + (j & 1)));
            }
            ++segs;
            more = walk.next(p, next_seg);
        }
        if (!ok) atomicOr(p.error, 1u);
    } else if (warp >= kFetchWarp0) {
        // Two warps a plane; each fetches 32 of a slot's 64 keys: scales a key per lane, codes in boxes of `box` keys, which
        // lie in one page (a box of 64 keys: the first warp its lower 128 bytes, the second the upper).  The pages are
        // looked up a tile ahead.
        const int f = warp - kFetchWarp0, part = f & 1;
        const bool is_v = f >= 2;
        const CUtensorMap* map = is_v ? &p.tmap_v : &p.tmap_k;
        const uint16_t* scales = is_v ? p.vs : p.ks;
        const int first = is_v ? L::RK : 0, ring = is_v ? L::RV : L::RK;
        int slot = first, turn = 0, issued = 0, t = 0, page = -1;
        bool have = false;
        // lane l < 4 stands for 16 keys of half l / 2, the part's first or second (the slot's first, in a box of 64)
        const bool whole_slot = p.box == 64;
        auto key_of = [&](int tile) { return (long long)tile * BN + 64 * (lane >> 1) + (whole_slot ? 0 : 32 * part + 16 * (lane & 1)); };
        auto ahead = [&]() {
            if (!have || ++t >= seg.t1) {
                have = walk.next(p, seg);
                t = seg.t0;
                if (!have) return;
            }
            page = lane < 4 && key_of(t) < seg.q.len ? __ldg(p.table + (int64_t)seg.b * p.max_pages + (key_of(t) >> p.page_shift)) : -1;
        };
        ahead();
#pragma unroll 1
        while (have) {
            const bool on = page >= 0 && page < p.n_pages;
            const int off = (int)(key_of(t) & ((1 << p.page_shift) - 1));
            const int row = on ? (((page * p.n_kv_heads) + seg.kvh) << p.page_shift) + off : -1;
            ahead();
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (turn > 0) wait(L::kFree + slot, turn - 1);
                const uint32_t full = B(L::kFull + slot), dst = sbase + L::kSmSlots + slot * L::kCodes + part * 4096;
                const int r0 = __shfl_sync(0xffffffffu, row, 2 * half), r1 = __shfl_sync(0xffffffffu, row, 2 * half + 1);
                // scales of key 32 part + lane
                const int r = whole_slot || lane < 16 ? r0 : r1;
                if (r >= 0) {
                    const uint16_t* sc = scales + ((int64_t)r + (whole_slot ? 32 * part + lane : lane & 15)) * (HD / 32);
                    const uint32_t to = sbase + L::kSmScales + slot * L::kScales + (32 * part + lane) * (HD / 16);
                    if (HD == 256)
                        cp_async_16(to, sc, 16);
                    else
                        cp_async_8(to, sc, 8);
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
                if (elect_one()) {
                    if (p.box == 16) {
                        tc::mbar_arrive_expect_tx(full, (uint32_t)((r0 >= 0) + (r1 >= 0)) * 16 * HD);
#pragma unroll
                        for (int x = 0; x < HD / 128; ++x) {
                            if (r0 >= 0) tma_load_2d(dst + x * 8192, map, 128 * x, r0, full);
                            if (r1 >= 0) tma_load_2d(dst + x * 8192 + 2048, map, 128 * x, r1, full);
                        }
                    } else if (p.box == 32) {
                        tc::mbar_arrive_expect_tx(full, r0 >= 0 ? 32 * HD : 0);
#pragma unroll
                        for (int x = 0; x < HD / 128; ++x)
                            if (r0 >= 0) tma_load_2d(dst + x * 8192, map, 128 * x, r0, full);
                    } else {
                        const int x = HD == 256 ? part : 0;
                        const bool mine = r0 >= 0 && (HD == 256 || part == 0);
                        tc::mbar_arrive_expect_tx(full, mine ? 64 * 128 : 0);
                        if (mine) tma_load_2d(dst - part * 4096 + x * 8192, map, 128 * x, r0, full);
                    }
                }
                __syncwarp();
                ++issued;
                if (++slot == first + ring) slot = first, ++turn;
            }
        }
        // the block is not left while a copy into its memory is in flight
#pragma unroll 1
        for (int i = max(0, issued - ring); i < issued; ++i) {
            if (!ok) atomicOr(p.error, 1u);
            ok = true;
            wait(L::kFull + first + i % ring, i / ring);
        }
        if (!ok) atomicOr(p.error, 1u);
    } else if (warp >= kVWarp0) {
        // V^: lanes 0-7 hold the eight keys of one block, so that their 16-byte loads and swizzled stores fall into
        // different banks.  Scales of keys that are not there become zero, and so do their values.
        constexpr int U = HD / 128;
        const int w = warp - kVWarp0, nn = lane & 7, jj = lane >> 3;
        const uint32_t src0 = sbase + L::kSmSlots + (8 * w + nn) * 128 + ((nn ^ (2 * jj)) << 4);
        const uint32_t scale0 = sbase + L::kSmScales + (8 * w + nn) * (HD / 16) + jj * 2;
        // [64-dim atom][key][128 bytes], 16-byte chunks at chunk ^ key % 8; block jj of a unit: chunks 4 (jj % 2) ..
        const uint32_t dst0 = sbase + L::kSmV + (jj >> 1) * (BN * 128) + w * 1024 + nn * 128 + (((4 * (jj & 1)) ^ nn) << 4);
        int slot = L::RK, turn = 0, j = 0;
#pragma unroll 1
        while (walk.next(p, seg)) {
            const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
            const int len = seg.q.len, t1 = seg.t1;
            auto page_of = [&](int t) {  // lane g < 2: of this warp's keys of half g, loaded a tile ahead
                const long long key = (long long)t * BN + 64 * lane + 8 * w;
                return lane < 2 && t < t1 && key < len ? __ldg(pages + (key >> p.page_shift)) : 0;
            };
            int page = page_of(seg.t0);
#pragma unroll 1
            for (int t = seg.t0; t < t1; ++t, ++j) {
                const uint32_t bad = __ballot_sync(0xffffffffu, page < 0 || page >= p.n_pages);
                page = page_of(t + 1);
                const long long key = (long long)t * BN + 8 * w + nn;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int v = 2 * (j % L::NV) + half;
                    wait(L::kFull + slot, turn);
                    if (j >= L::NV) wait(L::kVFree + v, j / L::NV - 1);  // the half of tile j - NV has been used
                    __syncwarp();
                    const bool there = !(bad >> half & 1) && key + 64 * half < len;
                    const uint32_t dst = dst0 + (j % L::NV) * L::kTile + half * 8192, src = src0 + slot * L::kCodes;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint16_t sc = lds16(scale0 + slot * L::kScales + 8 * u);
                        const __half2 scale = __half2half2(__ushort_as_half(there ? sc : (uint16_t)0));
                        uint32_t h[16];
                        values16(lds128(src + u * 8192), scale, h);
                        values16(lds128((src + u * 8192) ^ 16), scale, h + 8);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            sts128((dst + u * (2 * BN * 128)) ^ (c << 4), make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]));
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive(B(L::kFree + slot));
                        tc::mbar_arrive(B(L::kV + v));
                    }
                    if (++slot == L::R) slot = L::RK, ++turn;
                }
            }
        }
        if (!ok) atomicOr(p.error, 1u);
    } else if (warp >= kKWarp0) {
        // K^: thread = key = tensor-memory lane
        const int w = warp - kKWarp0, half = w >> 1, n = (w & 1) * 32 + lane;
        const uint32_t lanes = (uint32_t)(w * 32) << 16;
        const uint32_t src0 = sbase + L::kSmSlots + n * 128 + ((n & 7) << 4), scale0 = sbase + L::kSmScales + n * (HD / 16);
        int slot = half, turn = 0, j = 0;
#pragma unroll 1
        while (walk.next(p, seg)) {
            const int t1 = seg.t1;
#pragma unroll 1
            for (int t = seg.t0; t < t1; ++t, ++j) {
                wait(L::kFull + slot, turn);
                if (j >= L::NK) wait(L::kS + ((j - L::NK) & 1), (j - L::NK) >> 1);  // K^ of tile j - NK has been used
                tc::fence_after_sync();
                __syncwarp();
                const uint32_t to = tmem + lanes + L::kTmK + (j % L::NK) * (HD / 2);
#pragma unroll 1
                for (int u = 0; u < HD / 128; ++u) {  // four blocks
                    const uint32_t src = src0 + slot * L::kCodes + u * 8192;
                    const uint2 sc = lds64(scale0 + slot * L::kScales + 8 * u);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const __half2 s2 = u32_as_h2(k ? sc.y : sc.x);
                        uint32_t h[32];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            values16(lds128(src ^ ((4 * k + c) << 4)), c < 2 ? __low2half2(s2) : __high2half2(s2), h + 8 * c);
                        tc::tmem_st32(to + 64 * u + 32 * k, h);
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(B(L::kFree + slot));
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(B(L::kK + j % L::NK));
                slot += 2;
                if (slot >= L::RK) slot -= L::RK, ++turn;
            }
        }
        if (!ok) atomicOr(p.error, 1u);
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kQkWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0) leave_join<BN>(p, *place);
}

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
    // against 171 us, 20 requests of 16000 tokens at head_dim 256 42 us against 33 us.
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
__device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

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
                const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
                reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + out_row * HD)[d] =
                    sum > 0.0f ? make_uint2(Query<T>::out(acc.x * inv, acc.y * inv), Query<T>::out(acc.z * inv, acc.w * inv)) : make_uint2(0u, 0u);
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

constexpr int kJoinThreads = 256;

// The rows of every item that was cut, one after another over the blocks: o = sum_c 2^(m_c - m) o_c / sum_c
// 2^(m_c - m) l_c over its parts, slot 1 of the CTA that began it and slot 0 of the same place in the later teams.
template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedVerifyParams p, int n_ctas) {
    constexpr int kCols = HD / 4, kGroups = kJoinThreads / kCols;
    __shared__ int4 s_join[1024];
    __shared__ int s_first[1025];
    __shared__ float4 s_o[kGroups][kCols];
    __shared__ float s_l[kGroups], s_m[kJoinThreads / 32];
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
    const int col = tid % kCols, grp = tid / kCols;
    for (int task = blockIdx.x; task < s_first[n_ctas]; task += gridDim.x) {
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
        float m = -INFINITY;
        for (int i = tid; i < parts; i += kJoinThreads) m = fmaxf(m, p.part_ml[slot(i)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) s_m[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, s_m[w]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.0f;
#pragma unroll 4
        for (int i = grp; i < parts; i += kGroups) {
            const float2 ml = p.part_ml[slot(i)];
            const float4 o = reinterpret_cast<const float4*>(p.part_o)[slot(i) * kCols + col];
            const float w = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
            l += w * ml.y;
            acc.x += w * o.x, acc.y += w * o.y, acc.z += w * o.z, acc.w += w * o.w;
        }
        s_o[grp][col] = acc;
        if (col == 0) s_l[grp] = l;
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int g = 1; g < kGroups; ++g) {
                const float4 o = s_o[g][col];
                acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
                l += s_l[g];
            }
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const int rr = (s_join[c0].z & 0xffff) + r, t = rr / p.group;
            const int head = s_join[c0].y * p.group + rr - t * p.group;
            uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((int64_t)(s_join[c0].x + t) * p.n_q_heads + head) * HD);
            dst[col] = l > 0.0f ? make_uint2(Query<T>::out(acc.x * inv, acc.y * inv), Query<T>::out(acc.z * inv, acc.w * inv))
                                : make_uint2(0u, 0u);
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

enum { kFew = 0, kSome = 1, kMany = 2 };

struct VerifyPlan {
    int route, ctas, chunk, team;  // CTAs; most rows of one; CTAs that share an item's rows
    size_t ml_off, join_off, bytes;
};

// By the rows of the batch's longest window and KV head: up to 8 (16 at head_dim 128) the kernel in which each warp scans
// for itself; up to 32 the tensor-core tiles with the deeper fetch ring; above that teams of CTAs with up to 64 rows each.
VerifyPlan verify_plan(int sms, int group, int hd, int max_rows) {
    VerifyPlan v;
    const int rows = max_rows * group;
    v.route = rows <= (hd == 128 ? 16 : 8) ? kFew : rows <= 32 ? kSome : kMany;
    v.ctas = v.route == kFew ? (hd == 128 ? FL<128, 1>::kCtas : FL<256, 1>::kCtas) * sms : sms;
    v.team = v.route == kMany ? (rows + 63) / 64 : 1;
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

template <typename T, int HD, int N>
int launch_tiles(const PagedVerifyParams& p, const VerifyPlan& v, cudaStream_t s) {
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_kernel<T, HD, N>, VL<HD, N>::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    return launch_dependent(paged_verify_kernel<T, HD, N>, v.ctas, kVerifyThreads, VL<HD, N>::kSmBytes, s, p);
}

template <typename T, int HD, int NT>
int launch_few(const PagedVerifyParams& p, const VerifyPlan& v, cudaStream_t s) {
    using L = FL<HD, NT>;
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_few_kernel<T, HD, NT>, L::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    return launch_dependent(paged_verify_few_kernel<T, HD, NT>, v.ctas, L::kWarps * 32, L::kSmBytes, s, p);
}

template <typename T, int HD>
int launch_verify(const PagedVerifyParams& p, const VerifyPlan& v, cudaStream_t s) {
    int rc;
    if (v.route == kFew)
        rc = HD == 128 && v.chunk > 8 ? launch_few<T, 128, 2>(p, v, s) : launch_few<T, HD, 1>(p, v, s);
    else
        rc = v.route == kSome ? launch_tiles<T, HD, 32>(p, v, s) : launch_tiles<T, HD, 64>(p, v, s);
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
        n_rows > (1 << 24) || (int64_t)kv->n_pages * kv->n_kv_heads * kv->page_size > 0x7fffffffLL)
        return KVQ8_ERR_UNSUPPORTED;  // the last: rows of a plane are tensor-map coordinates
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
    p.box = kv->page_size < 64 ? kv->page_size : 64;
    if (!encode_codes(&p.tmap_k, kv->k_codes, kv, p.box) || !encode_codes(&p.tmap_v, kv->v_codes, kv, p.box)) return KVQ8_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    if (kv->head_dim == 128)
        return dtype == KVQ8_F16 ? launch_verify<__half, 128>(p, v, s) : launch_verify<__nv_bfloat16, 128>(p, v, s);
    return dtype == KVQ8_F16 ? launch_verify<__half, 256>(p, v, s) : launch_verify<__nv_bfloat16, 256>(p, v, s);
}

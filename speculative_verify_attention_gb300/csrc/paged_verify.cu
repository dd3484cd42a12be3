// paged_verify.cu -- verify attention of a batch of windows over a paged Q8_0 cache (attn_verify_paged_q8).
//
// Row t of request b (window of T rows after ctx = len - T cached tokens) sees every key n < ctx and the window
// key ctx + j where bit j of its mask is set (chains: j <= t):
//   o = sum_n p_n v_n / sum_n p_n,  p_n = exp(scale * q . k_n),  k and v = code * scale of their block.
//
// The T x group rows (row t, head hh of one KV head: t * group + hh) are the M = 128 rows of a tcgen05 tile, so a
// key tile is read and dequantised once for all of them:
//   S = Q K^T : A = Q from tensor memory (fp16 pairs), B = K^ [keys][dims] in shared memory (K-major)
//   O += P V^ : A = P from tensor memory, B = V^ [keys][dims] (MN-major), fp32 accumulation in tensor memory
// Work: the (request, KV head, 128-row chunk) items, each ceil(len / BN) key tiles, laid end to end and cut into one
// equal share per SM.  Every CTA works its share out by itself from the lengths on the device (one scan over the
// requests), so nothing waits for the host and a captured call follows new lengths.  A share holds at most one item
// that it did not begin and one that it does not end: those leave a partial (o, m, l) in the CTA's two workspace
// slots, joined by the second kernel; items wholly inside a share are written at once.
//
// Warps of a CTA (each wait between them is an mbarrier wait with an iteration limit):
//   0-3   softmax: one row per thread, running maximum and sum in registers (fp32), P back to tensor memory
//   4     issues the MMAs (one thread), owns tensor memory
//   5-12  dequantise: codes and scales from global memory straight into registers, two tiles ahead, then fp16
//         (code * scale, rounded once) into three-deep K^ and V^ rings in shared memory.  A thread takes whole
//         32-value blocks (one 32-byte load and one scale); lanes 0-7 hold eight consecutive keys of the same block,
//         whose swizzled 16-byte stores fall into different banks.
// Rows behind len and keys on page ids outside the pool are not read: they enter as zeros and are masked.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc.cuh"

namespace kvq8 {

unsigned int* device_error_flag();

namespace {

constexpr int kRows = 128;                  // rows of a tile
constexpr int kIssueWarp = 4, kDeqWarp0 = 5, kDeqWarps = 8;
constexpr int kVerifyThreads = (kDeqWarp0 + kDeqWarps) * 32;
constexpr int kStages = 3;                  // K^ and V^ tiles in shared memory
constexpr uint32_t kPollLimit = 1u << 24;
constexpr float kLazy = 8.0f;               // the running maximum follows only jumps of more than 2^8
constexpr float kLift = 6.0f;               // p is 2^6 larger than 2^(s - m): at most 2^14, and fp16 keeps it to 2^-30
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr int keys_per_tile(int hd) { return hd == 128 ? 128 : 64; }

// Barriers, a ring of kStages each: K^ written, V^ written, S complete (and K^ free), P written, PV complete (and V^
// free).  Tile j uses entry j % kStages; its next use needs tile j + kStages, which needs every wait on this one.
enum { kBarK = 0, kBarV = kStages, kBarS = 2 * kStages, kBarP = 3 * kStages, kBarO = 4 * kStages, kBarQ = 5 * kStages,
       kBarCount = 5 * kStages + 1 };

template <int HD>
struct VL {
    static constexpr int BN = keys_per_tile(HD);
    static constexpr int kTile = BN * HD * 2;              // bytes of one fp16 tile
    static constexpr int kSmK = 0, kSmV = kStages * kTile, kSmBar = 2 * kStages * kTile;
    static constexpr int kSmTmem = kSmBar + kBarCount * 8, kSmScan = (kSmTmem + 4 + 15) / 16 * 16;
    static constexpr int kSmBytes = kSmScan + 64 + (kVerifyThreads / 32) * 8;
    static constexpr uint32_t kTmQ = 0, kTmO = HD / 2, kTmS = kTmO + HD;
    static constexpr uint32_t kIdescS = tc::idesc_f16_f32(kRows, BN, false), kIdescO = tc::idesc_f16_f32(kRows, HD, true);
    // a dequantising warp covers 8 keys x 4 blocks at a time; passes per plane and tile
    static constexpr int kUnits = BN * HD / 32 / 32 / kDeqWarps;
    static_assert(kUnits == 2, "two passes");
    static constexpr int kPages = HD == 256 ? 1 : 2;       // distinct keys of a thread per tile
    static_assert(kTmS + 2 * BN <= kTmemCols, "tensor memory");
    static_assert(kSmBytes <= 227 * 1024, "shared memory");
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
    float* part_o;     // [grid][2][part_rows][HD]
    float2* part_ml;   // [grid][2][part_rows] (m in log2 units, l)
    int4* joins;       // [grid]: the item that CTA c begins and does not end (first q row, KV head, rows, last CTA)
    unsigned int* error;
    int n_rows, n_q_heads, n_kv_heads, group, n_pages, page_shift, max_pages, n_seqs, max_rows, part_rows;
    float scale_log2;
};

// ---------------------------------------------------------------- the shares

// A request as the kernel sees it; items = 0 where there is nothing to do or its numbers make no sense.
struct Request {
    int len, rows, row0, tiles, items;
};

template <int BN>
__device__ __forceinline__ Request request_of(const PagedVerifyParams& p, int b) {
    Request q;
    q.row0 = __ldg(p.row_starts + b);
    const int end = __ldg(p.row_starts + b + 1);
    q.len = __ldg(p.lens + b);
    q.tiles = q.items = q.rows = 0;
    if (q.row0 < 0 || end > p.n_rows || end <= q.row0) return q;
    q.rows = end - q.row0;
    if (q.rows > p.max_rows || q.rows > q.len || (int64_t)q.len > ((int64_t)p.max_pages << p.page_shift)) return q;
    q.tiles = (int)(((int64_t)q.len + BN - 1) / BN);
    q.items = p.n_kv_heads * ((q.rows * p.group + kRows - 1) / kRows);
    return q;
}

// Part of an item: key tiles [t0, t1) for rows [r0, r0 + n) of KV head kvh of request b.
struct Segment {
    int b, kvh, r0, n, t0, t1;
    Request q;
    __device__ __forceinline__ bool begins() const { return t0 == 0; }
    __device__ __forceinline__ bool ends() const { return t1 == q.tiles; }
};

// A CTA's share, segment by segment.  Each role walks it on its own.
struct Walk {
    int b, item, t;
    long long left;
    Request q;

    template <int BN>
    __device__ __forceinline__ bool next(const PagedVerifyParams& p, Segment& s) {
        if (left <= 0) return false;
        while (item >= q.items) {
            item = 0;
            if (++b >= p.n_seqs) return false;
            q = request_of<BN>(p, b);
        }
        const int chunks = q.items / p.n_kv_heads;
        s.b = b;
        s.kvh = item / chunks;
        s.r0 = (item - s.kvh * chunks) * kRows;
        s.n = min(kRows, q.rows * p.group - s.r0);
        s.t0 = t;
        s.t1 = (int)min((long long)q.tiles, t + left);
        s.q = q;
        left -= s.t1 - s.t0;
        t = s.t1;
        if (t == q.tiles) {
            t = 0;
            ++item;
        }
        return true;
    }
};

// Exclusive sum over the block of one value per thread, and the total; all threads call it.
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
    for (int w = 0; w < kVerifyThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    return before + inc - v;
}

// ---------------------------------------------------------------- dequantising

struct Block {           // one 32-value block: its codes and its scale
    uint32_t w[8];
    uint32_t scale;
};

__device__ __forceinline__ void load_block(Block& x, const int8_t* codes, const uint16_t* scales, int64_t block, bool on) {
    if (on) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]), "=r"(x.w[7])
                     : "l"(codes + block * 32));
        x.scale = __ldg(scales + block);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.w[i] = 0u;
        x.scale = 0u;
    }
}

// The block as fp16, code * scale rounded once, at [key n][block] of a 128-byte-swizzled tile: 64-dim atoms of BN
// rows of 128 bytes, the 16-byte chunks of row n stored at chunk ^ (n % 8).
template <int BN>
__device__ __forceinline__ void store_block(const Block& x, uint8_t* tile, int n, int block) {
    const __half2 sc = __half2half2(__ushort_as_half((unsigned short)x.scale));
    uint8_t* row = tile + (block >> 1) * (BN * 128) + (n >> 3) * 1024 + (n & 7) * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t w = x.w[2 * k + e] ^ 0x80808080u;
            h[2 * e] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4140>(w)), sc));
            h[2 * e + 1] = h2_as_u32(__hmul2(u32_as_h2(biased_bytes_to_half2<0x4342>(w)), sc));
        }
        *reinterpret_cast<uint4*>(row + (((4 * (block & 1) + k) ^ (n & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// ---------------------------------------------------------------- queries and output

// Sixteen-byte pieces of a query row as fp16 pairs.  fp16 rows go in as they are; bf16 rows times a power of two that
// brings their largest element into [2^7, 2^8), undone in the score's scale.
template <typename T>
struct Query;
template <>
struct Query<__half> {
    static __device__ __forceinline__ float lift(const uint4*, int) { return 1.0f; }
    static __device__ __forceinline__ float drop(float) { return 1.0f; }
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float) { return w; }
    static __device__ __forceinline__ uint32_t out(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
};
template <>
struct Query<__nv_bfloat16> {
    static __device__ __forceinline__ float lift(const uint4* row, int pieces) {
        uint32_t top = 0;
        for (int c = 0; c < pieces; ++c) {
            const uint4 v = __ldg(row + c);
            for (uint32_t w : {v.x, v.y, v.z, v.w}) top = max(top, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
        }
        const int e = (int)(top >> 7);                      // biased exponent
        if (e == 0 || e == 255) return 1.0f;                // zeros and subnormals; not finite
        return __uint_as_float((uint32_t)min(127 + 127 + 7 - e, 254) << 23);
    }
    static __device__ __forceinline__ float drop(float lifted) { return 1.0f / lifted; }  // a power of two: exact
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float lifted) {
        return h2_as_u32(__floats2half2_rn(__uint_as_float(w << 16) * lifted, __uint_as_float(w & 0xffff0000u) * lifted));
    }
    static __device__ __forceinline__ uint32_t out(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// Bit c = a row with window mask m sees key key0 + c: keys before ctx, then its mask's bits.
__device__ __forceinline__ uint64_t seen64(long long key0, int ctx, uint64_t m) {
    const long long before = ctx - key0;  // keys of this group before the window
    if (before >= 64) return ~0ull;
    if (before > 0) return ((1ull << before) - 1) | (m << before);
    return before > -64 ? m >> -before : 0ull;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kVerifyThreads, 1) paged_verify_kernel(const __grid_constant__ PagedVerifyParams p) {
    using L = VL<HD>;
    constexpr int BN = L::BN;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem), bar = sbase + L::kSmBar;
    auto B = [&](int id) { return bar + 8u * (uint32_t)id; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSmTmem);
    long long* s_start = reinterpret_cast<long long*>(smem + L::kSmScan);  // the request of the first unit, units into it
    long long* s_warp = s_start + 8;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(B(kBarK + s), kDeqWarps);
            tc::mbar_init(B(kBarV + s), kDeqWarps);
            tc::mbar_init(B(kBarS + s), 1);
            tc::mbar_init(B(kBarP + s), 4);
            tc::mbar_init(B(kBarO + s), 1);
        }
        tc::mbar_init(B(kBarQ), 4);
        tc::mbar_init_fence();
    }
    if (warp == kIssueWarp) tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // this CTA's share of the units
    const int per = (p.n_seqs + kVerifyThreads - 1) / kVerifyThreads;
    const int b_lo = min(tid * per, p.n_seqs), b_hi = min(b_lo + per, p.n_seqs);
    long long mine = 0, units;
    for (int b = b_lo; b < b_hi; ++b) {
        const Request q = request_of<BN>(p, b);
        mine += (long long)q.tiles * q.items;
    }
    const long long before = block_exclusive(mine, s_warp, units);
    // no more shares than units: every share of an item that was cut has tiles of it, and so a partial
    const long long shares = units < gridDim.x ? units : (long long)gridDim.x, me = blockIdx.x;
    const long long u0 = me < shares ? me * units / shares : units, u1 = me < shares ? (me + 1) * units / shares : units;
    if (u0 < u1 && before <= u0 && u0 < before + mine) {
        long long at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            const Request q = request_of<BN>(p, b);
            const long long here = (long long)q.tiles * q.items;
            if (u0 < at + here) {
                s_start[0] = b;
                s_start[1] = u0 - at;
                break;
            }
            at += here;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Walk walk;
    walk.left = u1 - u0;
    walk.b = p.n_seqs;
    walk.item = walk.t = 0;
    walk.q.items = 0;
    if (u0 < u1) {
        walk.b = (int)s_start[0];
        walk.q = request_of<BN>(p, walk.b);
        walk.item = (int)(s_start[1] / walk.q.tiles);
        walk.t = (int)(s_start[1] - (long long)walk.item * walk.q.tiles);
    }
    Segment seg;
    bool ok = true;

    if (warp == kIssueWarp) {
        if (lane == 0) {
            const uint64_t kdesc0 = tc::smem_desc_sw128(sbase + L::kSmK, 16, 1024);
            const uint64_t vdesc0 = tc::smem_desc_sw128(sbase + L::kSmV, BN * 128, 1024);
            int st = 0, s_ph = 0, q_ph = 0, sb = 0;  // ring entry and phase of tile j; S buffer j % 2
            auto pv = [&](int st1, int ph1, int sb1, bool first) {
                if (!tc::mbar_wait(B(kBarP + st1), ph1, kPollLimit) || !tc::mbar_wait(B(kBarV + st1), ph1, kPollLimit)) return false;
                tc::fence_after_sync();
                const uint64_t vd = vdesc0 + (uint64_t)((st1 * L::kTile) >> 4);
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    tc::mma_ts(tmem + L::kTmO, tmem + L::kTmS + sb1 * BN + k * 8, vd + (uint64_t)((k * 2048) >> 4), L::kIdescO,
                               (!first || k > 0) ? 1u : 0u);
                tc::mma_commit(B(kBarO + st1));
                return true;
            };
            while (ok && walk.next<BN>(p, seg)) {
                if (!tc::mbar_wait(B(kBarQ), q_ph, kPollLimit)) { ok = false; break; }
                q_ph ^= 1;
                tc::fence_after_sync();
                int st1 = 0, ph1 = 0, sb1 = 0;
                for (int t = seg.t0; t < seg.t1; ++t) {
                    if (!tc::mbar_wait(B(kBarK + st), s_ph, kPollLimit)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint64_t kd = kdesc0 + (uint64_t)((st * L::kTile) >> 4);
                    // S overwrites the columns that held P of tile j - 2, whose PV was issued before (issue order holds)
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        tc::mma_ts(tmem + L::kTmS + sb * BN, tmem + L::kTmQ + k * 8,
                                   kd + (uint64_t)((((k >> 2) * (BN * 128)) + (k & 3) * 32) >> 4), L::kIdescS, k > 0 ? 1u : 0u);
                    tc::mma_commit(B(kBarS + st));
                    if (t > seg.t0 && !pv(st1, ph1, sb1, t - 1 == seg.t0)) { ok = false; break; }
                    st1 = st, ph1 = s_ph, sb1 = sb;
                    sb ^= 1;
                    if (++st == kStages) st = 0, s_ph ^= 1;
                }
                if (ok && !pv(st1, ph1, sb1, seg.t1 - 1 == seg.t0)) ok = false;
            }
            if (!ok) atomicOr(p.error, 1u);
        }
        __syncwarp();
    } else if (warp < 4) {
        const int r = warp * 32 + lane;
        const uint32_t rows_tm = tmem + ((uint32_t)(warp * 32) << 16);
        int st = 0, ph = 0, sb = 0;
        while (ok && walk.next<BN>(p, seg)) {
            const bool busy = warp * 32 < seg.n, valid = r < seg.n;  // a warp without rows only keeps the barriers going
            const int rr = seg.r0 + (valid ? r : 0), t_row = rr / p.group;
            const int head = seg.kvh * p.group + rr - t_row * p.group, row = seg.q.row0 + t_row;
            const int ctx = seg.q.len - seg.q.rows;
            uint64_t m64 = 0;
            float cs = p.scale_log2;
            if (busy) {
                if (valid) {
                    m64 = p.mask ? __ldg(p.mask + row) : (2ull << t_row) - 1;
                    if (seg.q.rows < 64) m64 &= (1ull << seg.q.rows) - 1;
                }
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (int64_t)row * p.q_stride +
                                                                  (int64_t)head * HD);
                const float lifted = Query<T>::lift(src, HD / 8);
                cs *= Query<T>::drop(lifted);
#pragma unroll 1
                for (int c = 0; c < HD / 64; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 v = __ldg(src + c * 8 + k);
                        w[4 * k] = Query<T>::pair(v.x, lifted);
                        w[4 * k + 1] = Query<T>::pair(v.y, lifted);
                        w[4 * k + 2] = Query<T>::pair(v.z, lifted);
                        w[4 * k + 3] = Query<T>::pair(v.w, lifted);
                    }
                    tc::tmem_st32(rows_tm + L::kTmQ + 32 * c, w);
                }
                tc::tmem_wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B(kBarQ));

            float m = -INFINITY, l = 0.0f;
            const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
            // page ids of the tile's 16-key groups, one per lane, loaded a tile ahead
            auto page_of = [&](int t) {
                const long long key = (long long)t * BN + 16 * lane;
                return lane < BN / 16 && t < seg.t1 && key < seg.q.len ? __ldg(pages + (key >> p.page_shift)) : 0;
            };
            int page = busy ? page_of(seg.t0) : 0;
            int o_st = 0, o_ph = 0;
            for (int t = seg.t0; t < seg.t1; ++t) {
                if (!__all_sync(0xffffffffu, tc::mbar_wait(B(kBarS + st), ph, kPollLimit))) { ok = false; break; }
                tc::fence_after_sync();
                if (busy) {
                    const uint32_t bad = __ballot_sync(0xffffffffu, page < 0 || page >= p.n_pages);
                    page = page_of(t + 1);
                    const uint32_t scol = rows_tm + L::kTmS + sb * BN;
                    const long long key0 = (long long)t * BN;
                    const bool whole = key0 + BN <= ctx && !bad;
                    auto load = [&](int h, float (&x)[64]) {  // scores of keys 64 h .. 64 h + 63 of the tile
                        uint32_t a[32], b[32];
                        tc::tmem_ld32(scol + 64 * h, a);
                        tc::tmem_ld32(scol + 64 * h + 32, b);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(a[c]), x[32 + c] = __uint_as_float(b[c]);
                        if (!whole) {
                            uint64_t see = seen64(key0 + 64 * h, ctx, m64);
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                if (bad >> (4 * h + g) & 1) see &= ~(0xffffull << (16 * g));
                            const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                if (!(lo >> c & 1)) x[c] = -INFINITY;
                                if (!(hi >> c & 1)) x[32 + c] = -INFINITY;
                            }
                        }
                    };
                    float x[64], top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int h = 0; h < BN / 64; ++h) {
                        load(h, x);
#pragma unroll
                        for (int c = 0; c < 64; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
                    }
                    const float m_new = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cs);
                    const bool raise = m_new > m + kLazy || (m == -INFINITY && m_new != -INFINITY);
                    if (__any_sync(0xffffffffu, raise)) {
                        float a = 1.0f;
                        if (raise) {
                            a = m == -INFINITY ? 0.0f : ex2_approx(m - m_new);
                            m = m_new;
                            l *= a;
                        }
                        if (t > seg.t0) {  // every earlier PV has landed before its rows are scaled
                            if (!__all_sync(0xffffffffu, tc::mbar_wait(B(kBarO + o_st), o_ph, kPollLimit))) { ok = false; break; }
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < HD / 32; ++c) {
                                uint32_t o[32];
                                tc::tmem_ld32(rows_tm + L::kTmO + 32 * c, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                                tc::tmem_st32(rows_tm + L::kTmO + 32 * c, o);
                            }
                        }
                    }
                    const bool live = m != -INFINITY;
                    const float off = live ? kLift - m : 0.0f;
#pragma unroll 1
                    for (int h = 0; h < BN / 64; ++h) {
                        if (BN > 64) load(h, x);
                        uint32_t pk[32];
                        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float a = live ? ex2_approx(fmaf(x[2 * c], cs, off)) : 0.0f;
                            const float b = live ? ex2_approx(fmaf(x[2 * c + 1], cs, off)) : 0.0f;
                            sum[2 * (c & 1)] += a;
                            sum[2 * (c & 1) + 1] += b;
                            pk[c] = h2_as_u32(__floats2half2_rn(a, b));
                        }
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        // P of half h goes over columns 32 h .. 32 h + 31, whose scores have been read
                        tc::tmem_st32(scol + 32 * h, pk);
                    }
                    tc::tmem_wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(B(kBarP + st));
                o_st = st, o_ph = ph;
                sb ^= 1;
                if (++st == kStages) st = 0, ph ^= 1;
            }
            if (!ok) break;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(B(kBarO + o_st), o_ph, kPollLimit))) { ok = false; break; }
            tc::fence_after_sync();
            if (busy) {
                const bool whole = seg.begins() && seg.ends();
                const int slot = 2 * blockIdx.x + (seg.begins() ? 1 : 0);
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + ((int64_t)row * p.n_q_heads + head) * HD);
                float4* part = reinterpret_cast<float4*>(p.part_o + ((int64_t)slot * p.part_rows + (valid ? r : 0)) * HD);
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32(rows_tm + L::kTmO + 32 * c, o);
                    tc::tmem_wait_ld();
                    if (!valid) continue;
                    auto f = [&](int k) { return __uint_as_float(o[k]); };
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = l > 0.0f ? Query<T>::out(f(8 * k + 2 * e) * inv, f(8 * k + 2 * e + 1) * inv) : 0u;
                            dst[4 * c + k] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) part[8 * c + k] = make_float4(f(4 * k), f(4 * k + 1), f(4 * k + 2), f(4 * k + 3));
                    }
                }
                if (valid && !whole) p.part_ml[(int64_t)slot * p.part_rows + r] = make_float2(m, l);
            }
            tc::fence_before_sync();
        }
        if (!ok) atomicOr(p.error, 1u);
    } else {
        // blocks of this thread in a tile: hd256, blocks jj and 4 + jj of key 8 w + nn; hd128, block jj of keys
        // 8 w + nn and 64 + 8 w + nn
        const int w = warp - kDeqWarp0, nn = lane & 7, jj = lane >> 3;
        int st = 0, ph = 0;
        Block kx[2][2], vx[2][2];
        // the tile whose page ids are being fetched: a tile ahead of the loads
        int page[L::kPages], off[L::kPages];
        int t = 0;
        bool have = false;
        auto ahead = [&]() {
            if (!have || ++t >= seg.t1) {
                have = walk.next<BN>(p, seg);
                t = seg.t0;
                if (!have) return;
            }
            const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
#pragma unroll
            for (int i = 0; i < L::kPages; ++i) {
                const long long key = (long long)t * BN + 64 * i + 8 * w + nn;
                off[i] = (int)key & ((1 << p.page_shift) - 1);
                page[i] = key < seg.q.len ? __ldg(pages + (key >> p.page_shift)) : -1;
            }
        };
        auto block_at = [&](int u, int kvh, bool& on) {  // block index of pass u in the planes
            const int i = L::kPages == 1 ? 0 : u;
            on = page[i] >= 0 && page[i] < p.n_pages;
            const int64_t row = (((int64_t)page[i] * p.n_kv_heads + kvh) << p.page_shift) + off[i];
            return row * (HD / 32) + (HD == 256 ? 4 * u + jj : jj);
        };
        auto key_of = [&](int u) { return HD == 256 ? 8 * w + nn : 64 * u + 8 * w + nn; };
        auto blk_of = [&](int u) { return HD == 256 ? 4 * u + jj : jj; };
        bool full[2];
        auto load_tile = [&](Block (&k)[2], Block (&v)[2], bool& f) {
            f = have;
            if (!have) return;
            bool on[2];
            int64_t at[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) at[u] = block_at(u, seg.kvh, on[u]);
#pragma unroll
            for (int u = 0; u < 2; ++u) load_block(k[u], p.kc, p.ks, at[u], on[u]);
#pragma unroll
            for (int u = 0; u < 2; ++u) load_block(v[u], p.vc, p.vs, at[u], on[u]);
            ahead();
        };
        bool reused = false;  // the ring has gone round once
        auto put_tile = [&](const Block (&k)[2], const Block (&v)[2]) {
            if (reused && !__all_sync(0xffffffffu, tc::mbar_wait(B(kBarS + st), ph ^ 1, kPollLimit))) return false;
#pragma unroll
            for (int u = 0; u < 2; ++u) store_block<BN>(k[u], smem + L::kSmK + st * L::kTile, key_of(u), blk_of(u));
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B(kBarK + st));
            if (reused && !__all_sync(0xffffffffu, tc::mbar_wait(B(kBarO + st), ph ^ 1, kPollLimit))) return false;
#pragma unroll
            for (int u = 0; u < 2; ++u) store_block<BN>(v[u], smem + L::kSmV + st * L::kTile, key_of(u), blk_of(u));
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B(kBarV + st));
            if (++st == kStages) st = 0, ph ^= 1, reused = true;
            return true;
        };
        ahead();
        load_tile(kx[0], vx[0], full[0]);
        load_tile(kx[1], vx[1], full[1]);
        while (true) {
            if (!full[0]) break;
            if (!put_tile(kx[0], vx[0])) { ok = false; break; }
            load_tile(kx[0], vx[0], full[0]);
            if (!full[1]) break;
            if (!put_tile(kx[1], vx[1])) { ok = false; break; }
            load_tile(kx[1], vx[1], full[1]);
        }
        if (!ok && lane == 0) atomicOr(p.error, 1u);
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kIssueWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0) {
        // the last segment, if its item goes on in later CTAs: they are joined under this CTA's number
        int4 join = make_int4(0, 0, 0, -1);
        if (u0 < u1) {
            walk.left = u1 - u0;
            walk.b = (int)s_start[0];
            walk.q = request_of<BN>(p, walk.b);
            walk.item = (int)(s_start[1] / walk.q.tiles);
            walk.t = (int)(s_start[1] - (long long)walk.item * walk.q.tiles);
            while (walk.next<BN>(p, seg)) {}
            if (seg.begins() && !seg.ends()) {
                const long long last = u1 - seg.t1 + seg.q.tiles - 1;  // the item's last unit
                join = make_int4(seg.q.row0, seg.kvh, seg.r0 | seg.n << 16, (int)(((last + 1) * shares - 1) / units));
            }
        }
        p.joins[blockIdx.x] = join;
    }
}

// ---------------------------------------------------------------- joining the partials

constexpr int kJoinThreads = 256;

// The rows of every item that was cut, one after another over the blocks: o = sum_c 2^(m_c - m) o_c / sum_c
// 2^(m_c - m) l_c over its parts, slot 1 of the CTA that began it and slot 0 of the later ones.
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
        const int c0 = lo, r = task - s_first[c0], parts = s_join[c0].w - c0 + 1;
        auto slot = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * p.part_rows + r; };
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
    return sms < 1024 ? sms : 1024;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct VerifyPlan {
    int part_rows;
    size_t ml_off, join_off, bytes;
};

VerifyPlan verify_plan(int ctas, int group, int hd, int max_rows) {
    VerifyPlan v;
    v.part_rows = max_rows * group < kRows ? max_rows * group : kRows;
    v.ml_off = up256((size_t)ctas * 2 * v.part_rows * hd * sizeof(float));
    v.join_off = v.ml_off + up256((size_t)ctas * 2 * v.part_rows * sizeof(float2));
    v.bytes = v.join_off + (size_t)ctas * sizeof(int4);
    return v;
}

// Launched as programmatic dependents: their set-up overlaps the end of the kernel before, and they wait for all of
// its writes before they read or write anything (griddepcontrol.wait).
template <typename Kernel, typename... Args>
int launch_dependent(Kernel* kernel, int grid, int threads, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? KVQ8_OK : KVQ8_ERR_CUDA;
}

template <typename T, int HD>
int launch_verify(const PagedVerifyParams& p, int ctas, cudaStream_t s) {
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_kernel<T, HD>, VL<HD>::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    const int rc = launch_dependent(paged_verify_kernel<T, HD>, ctas, kVerifyThreads, VL<HD>::kSmBytes, s, p);
    if (rc != KVQ8_OK) return rc;
    return launch_dependent(paged_join_kernel<T, HD>, 4 * ctas, kJoinThreads, 0, s, p, ctas);
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
    const int ctas = sm_count(), group = n_q_heads / kv->n_kv_heads;
    const VerifyPlan v = verify_plan(ctas, group, kv->head_dim, max_rows);
    if (!workspace || workspace_bytes < v.bytes) return KVQ8_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (q_stride * 2) % 16 || !aligned_to(page_table, 4) ||
        !aligned_to(lens, 4) || !aligned_to(row_starts, 4) || !aligned_to(window_mask, 8))
        return KVQ8_ERR_MISALIGNED;
    if (!aligned_to(kv->k_codes, 32) || !aligned_to(kv->v_codes, 32)) return KVQ8_ERR_MISALIGNED;  // whole blocks per load
    unsigned int* error = device_error_flag();
    if (!error) return KVQ8_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    const PagedVerifyParams p = {q, out, q_stride, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, page_table, lens,
                                 row_starts, window_mask, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + v.ml_off),
                                 reinterpret_cast<int4*>(ws + v.join_off), error, n_rows, n_q_heads, kv->n_kv_heads, group,
                                 kv->n_pages, log2_of(kv->page_size), max_pages, n_seqs, max_rows, v.part_rows,
                                 softmax_scale * kLog2e};
    cudaStream_t s = (cudaStream_t)stream;
    const bool hd128 = kv->head_dim == 128;
    if (dtype == KVQ8_F16)
        return hd128 ? launch_verify<__half, 128>(p, ctas, s) : launch_verify<__half, 256>(p, ctas, s);
    return hd128 ? launch_verify<__nv_bfloat16, 128>(p, ctas, s) : launch_verify<__nv_bfloat16, 256>(p, ctas, s);
}

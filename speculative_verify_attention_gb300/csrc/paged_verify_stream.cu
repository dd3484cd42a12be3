// paged_verify_stream.cu -- verify attention over pages for windows of up to 64 rows and long contexts: keys stream through
// a deep ring of fetches.
//
// The T x group rows of a window and KV head (t * group + hh) are few and the keys many, so the products are taken
// transposed: keys, then dims, are the M = 128 rows of the tcgen05 tiles, the window's rows their N columns.
//   S^T [128 keys x N]  = K^ [keys x dims] Q^T  : A = K^ in tensor memory, B = Q in shared memory (K-major)
//   O^T [dims x N]     += V^ [keys x dims]^T P^T : A = V^ (MN-major), B = P [keys x rows] (MN-major), shared memory
// A tile costs the tensor cores 2 HD / 16 instructions of N columns (about 44 cycles each up to N = 64) where rows as
// M = 128 cost the full tile whatever the window.
//
// Warps of a CTA:
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
// Measured (24 / 4 heads of 256 dims): 8 requests of 32768 tokens, 30 rows 91 us, 4.1 TB/s; every 28672 tokens more cost
// 53 us, which is the memory's rate, and 36 us do not depend on the length.
#include "paged_verify.cuh"

namespace kvq8 {
namespace {

constexpr int BN = 128;                     // keys of a tile
constexpr int kQkWarp = 4, kPvWarp = 5, kKWarp0 = 8, kVWarp0 = 12, kFetchWarp0 = 20;
constexpr int kVerifyThreads = 768;
constexpr int kSoftThreads = 128;
// Shapes: NMAX rows of a chunk, 32 or 64; NK tiles of K^ in tensor memory, NV of V^ and two of weights in shared memory;
// the fetch rings take what is left of that.  Up to 32 rows the two weight tiles are the halves of one 64-row atom.
template <int HD, int NMAX>
struct SL {
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

// One box of a plane's tensor map into shared memory, completion counted in bytes.  x is 0 or 128: copies start on
// 16-byte boundaries.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
        : "memory");
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
__global__ void __launch_bounds__(kVerifyThreads, 1) paged_verify_stream_kernel(const __grid_constant__ PagedVerifyParams p) {
    using L = SL<HD, NMAX>;
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
    // (Loops in this kernel are kept rolled: the roles' code together should stay in the instruction caches, and stalls for
    // instructions were a quarter of all before.)
    Waits wait = {bar, true};

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
        if (!wait.ok) atomicOr(p.error, 1u);
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
        if (!wait.ok) atomicOr(p.error, 1u);
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
                            inv[c] = sum != 0.0f ? 1.0f / sum : 0.0f;  // (NaN stays one)
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
        if (!wait.ok) atomicOr(p.error, 1u);
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
            if (!wait.ok) atomicOr(p.error, 1u);
            wait.ok = true;
            wait(L::kFull + first + i % ring, i / ring);
        }
        if (!wait.ok) atomicOr(p.error, 1u);
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
        if (!wait.ok) atomicOr(p.error, 1u);
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
        if (!wait.ok) atomicOr(p.error, 1u);
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kQkWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0) leave_join<BN>(p, *place);
}

template <typename T, int HD, int N>
int launch(const PagedVerifyParams& p, int ctas, cudaStream_t s) {
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_stream_kernel<T, HD, N>, SL<HD, N>::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    return launch_dependent(paged_verify_stream_kernel<T, HD, N>, ctas, kVerifyThreads, SL<HD, N>::kSmBytes, s, p);
}

template <typename T, int HD>
int launch(const PagedVerifyParams& p, int n, int ctas, cudaStream_t s) {
    return n <= 32 ? launch<T, HD, 32>(p, ctas, s) : launch<T, HD, 64>(p, ctas, s);
}

}  // namespace

int launch_verify_stream(const PagedVerifyParams& p, int dtype, int hd, int n, int ctas, cudaStream_t s) {
    if (hd == 128) return dtype == KVQ8_F16 ? launch<__half, 128>(p, n, ctas, s) : launch<__nv_bfloat16, 128>(p, n, ctas, s);
    return dtype == KVQ8_F16 ? launch<__half, 256>(p, n, ctas, s) : launch<__nv_bfloat16, 256>(p, n, ctas, s);
}

}  // namespace kvq8

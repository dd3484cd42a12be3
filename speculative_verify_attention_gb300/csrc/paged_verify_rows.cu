// paged_verify_rows.cu -- verify attention over pages for windows of many rows: one CTA holds up to 192 rows.
//
// A tile is 64 keys.  S [rows x keys] = Q K^ with Q's rows as the M = 128 rows of the tcgen05 tile (Q and K^ K-major in
// shared memory), so a softmax thread owns a row: its maximum, reference and sum are registers and need no exchange.
// O^T [dims x rows] += V^ [keys x dims]^T P^T with dims as the M rows (A = V^ MN-major, B = P K-major as a softmax thread wrote
// it): up to 192 rows are its N columns and O^T takes 384 of tensor memory's 512 columns at head_dim 256, the scores the
// rest.  Rows 128 .. 191 are a second M = 128 tile, of rows 64 .. 191.  So a tile is dequantised once for 192 rows, where 64
// rows a CTA dequantise it three times.
//
// Warps (512 threads, 128 registers each):
//   0-3   softmax of rows 0 .. 127; 6, 7: of rows 128 .. 191.  References follow only jumps of more than 2^8, by one vote a
//         group and tile; the group then rescales its columns of O^T.
//   4     issues all products; 5: sleeps, and rescales the second group's columns in its lanes when that raises (4 too)
//   8-15  convert K (8-11) and V: a 32-value block at a time, loaded into registers a tile ahead and asked into L2 a tile
//         earlier, times its scale and rounded once to fp16, into rings of tiles (128-byte swizzle)
// Measured: 16 requests of 20676 tokens (24 / 4 heads of 256 dims, 32-row trees, 144 rows a KV head on average) 194 us, of
// which 45 us do not depend on the length; without loads 188, without conversion as well 181, with a quarter of O^T's products
// 185, without the exponentials 191, without any of these 133: what is left is the hand-offs from one role to the next, which
// one tile of scores a group puts in a row.  24 rows 136 us.
// Steps: one ring for K and V, and scores in tensor memory until the weights are made 254 us; rings of their own 236; the issuing
// warp's descriptors as constants instead of worked out from the tile's number 204; a barrier a tile instead of one for each
// half 195.  Slower: issuing from a single thread's loop 260 (its operands are no longer uniform), from two warps 257, whatever
// is ready first 277, O^T before the scores 265; two tiles of weights and a shorter ring 381; loads two tiles ahead 233.
#include "paged_verify.cuh"

namespace kvq8 {
namespace {

constexpr int BN = 64;                      // keys of a tile
constexpr int kMmaWarp = 4, kHelpWarp = 5, kConvWarp0 = 8;
constexpr int kAhead = 1;                   // tiles between the one being loaded and the one asked into L2
constexpr int kVerifyThreads = 512;
constexpr int kSoftThreads = 192;           // warps 0-3, 6 and 7
// Shapes: NMAX rows of a CTA, 64 or 192, in groups of 128 and 64 (the softmax warps of the lanes); H halves of a tile, of K^
// by dims (64 keys x 128) and of V^ by keys (256 dims x 32; at head_dim 128 all 64), 16 KB each.
template <int HD, int NMAX>
struct RL {
    static constexpr int H = HD / 128, kMt = HD / 128, kGroups = NMAX > 128 ? 2 : 1, kBuf = NMAX > 128 ? 1 : 2;
    static constexpr int kSlot = 64 * 128 * 2, kVKeys = 64 / H;
    static constexpr int kSmQ = 0, kSmP = kSmQ + HD / 64 * NMAX * 128;  // Q: [64-dim atom][row][128 bytes]; P: [row][64 keys]
    static constexpr int kSmRing = kSmP + kBuf * NMAX * 128;
    // tables: 1 / sum and the factor of the last raise (by tile parity) per row, output rows of two segments, largest query per warp
    static constexpr int kTabInv = 0, kTabAlpha = 4 * NMAX, kTabRow = 12 * NMAX, kTabMisc = 20 * NMAX, kTabScan = kTabMisc + 48,
                         kTabTmem = kTabScan + 64 + (kVerifyThreads / 32 + 1) / 2 * 16, kTabBar = kTabTmem + 16;
    static constexpr int kTabBytes = kTabBar + 20 * 8;
    // K^ has a ring of two tiles, V^ of kBuf: K^ of tile j + 1 is wanted while the softmax of tile j runs, V^ of tile j only after
    // it.  In tensor memory two tiles of scores: one of each group, or two of the one, which then has two of weights and of V^ too.
    static constexpr int kTile = H * kSlot, kSmV = kSmRing + 2 * kTile, kSmTab = kSmV + kBuf * kTile, kSmBytes = kSmTab + kTabBytes;
    // barriers: K^ ready / used; V^ ready; a tile of scores ready / read; weights ready; product done (so weights and V^ used);
    // queries ready
    static constexpr int kK = 0, kKFree = 2, kV = 4, kS = 6, kSFree = 8, kP = 10, kO = 12, kQ = 14, kRaise = 15, kR = 16;
    static constexpr uint32_t kTmO = 0, kTmS = kMt * NMAX;
    static_assert(kGroups * kBuf == 2 && kTmS + 128 <= kTmemCols, "tensor memory");
    static_assert(kSmBytes <= 227 * 1024 && kSmP % 1024 == 0 && kSmRing % 1024 == 0, "swizzled tiles are 1024-byte aligned");
};

// Into the whole of a register: two 16-bit values that share one would have to wait for each other.
__device__ __forceinline__ void load_u16(uint32_t& v, const uint16_t* at) {
    asm volatile("{\n .reg .u16 h;\n ld.global.nc.u16 h, [%1];\n cvt.u32.u16 %0, h;\n}\n" : "=r"(v) : "l"(at));
}
// The two halves of h to two fp32 sums, one addition each as for fp32 values (with conversions 16 trees take 195 us, not 194).
__device__ __forceinline__ void add_halves(float (&sum)[2], uint32_t h) {
    asm("{\n .reg .f16 lo, hi;\n mov.b32 {lo, hi}, %2;\n add.f32.f16 %0, lo, %0;\n add.f32.f16 %1, hi, %1;\n}\n"
        : "+f"(sum[0]), "+f"(sum[1])
        : "r"(h));
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 3, 192;" ::: "memory"); }
// The softmax warps of a group: four (0), or two (1).
__device__ __forceinline__ void group_sync(int g) {
    if (g == 0)
        asm volatile("bar.sync 1, 128;" ::: "memory");
    else
        asm volatile("bar.sync 2, 64;" ::: "memory");
}
__device__ __forceinline__ bool group_any(int g, bool v) {
    uint32_t r;
    if (g == 0)
        asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, 1, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n" : "=r"(r) : "r"((uint32_t)v) : "memory");
    else
        asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n bar.red.or.pred b, 2, 64, a;\n selp.u32 %0, 1, 0, b;\n}\n" : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}

template <typename T, int HD, int NMAX>
__global__ void __launch_bounds__(kVerifyThreads, 1) paged_verify_rows_kernel(const __grid_constant__ PagedVerifyParams p) {
    using L = RL<HD, NMAX>;
    constexpr int H = L::H, kGroups = L::kGroups;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* tab = smem + L::kSmTab;
    const uint32_t sbase = smem_u32(smem), bar = sbase + L::kSmTab + L::kTabBar;
    auto B = [&](int id) { return bar + 8u * (uint32_t)id; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tab + L::kTabTmem);
    Place* place = reinterpret_cast<Place*>(tab + L::kTabScan);
    long long* s_warp = reinterpret_cast<long long*>(tab + L::kTabScan + 64);
    static_assert(sizeof(Place) <= 64, "a place's room");

    if (tid == 0) {
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(B(L::kK + g), 4);
            tc::mbar_init(B(L::kKFree + g), 1);
            tc::mbar_init(B(L::kV + g), 4);
            tc::mbar_init(B(L::kS + g), 1);
            tc::mbar_init(B(L::kSFree + g), kGroups > 1 && g ? 2 : 4);
            tc::mbar_init(B(L::kP + g), kGroups > 1 ? 6 : 4);
            tc::mbar_init(B(L::kO + g), 1);
        }
        tc::mbar_init(B(L::kQ), 6);
        tc::mbar_init(B(L::kRaise), 2);
        tc::mbar_init(B(L::kR), 1);
        tc::mbar_init_fence();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    find_place<BN, kVerifyThreads>(p, place, s_warp);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Walk<BN> walk = walk_from<BN>(p, *place);
    Segment seg;
    Waits wait = {bar, true};

    float* alpha = reinterpret_cast<float*>(tab + L::kTabAlpha);
    // By tile parity: the second group raised references; the last such tile's columns (0 at the end) and number.
    int* raised_b = reinterpret_cast<int*>(tab + L::kTabMisc + 24);
    const int quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;  // the tensor-memory lanes that this warp reaches
    // Columns [c0, c1) of O^T times the factors of their rows, in this warp's lanes.
    auto rescale = [&](int j, int c0, int c1) {
        const float* a = alpha + (j & 1) * NMAX;
#pragma unroll 1
        for (int m = 0; m < L::kMt; ++m)
#pragma unroll 1
            for (int c = c0; c < c1; c += 16) {
                uint32_t o[16];
                tc::tmem_ld16(tmem + lanes + L::kTmO + m * NMAX + c, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a[c + i]);
                tc::tmem_st16(tmem + lanes + L::kTmO + m * NMAX + c, o);
            }
        tc::tmem_wait_st();
    };
    // weights and products of tile j: their buffer and phase
    auto pb = [](int j) { return L::kBuf > 1 ? j & 1 : 0; };
    auto pp = [](int j) { return L::kBuf > 1 ? j >> 1 : j; };

    if (warp == kMmaWarp) {
        // All products, issued by one lane.  It is the chain that every tile goes through, so the descriptors are constants: a
        // tile's place in the rings is its number's parity (or fixed), and the code is there once for each.
        const uint32_t one = elect_one();
        const uint64_t qd = tc::smem_desc_sw128(sbase + L::kSmQ, 16, 1024);
        const uint64_t pd = tc::smem_desc_sw128(sbase + L::kSmP, 16, 1024);
        const uint64_t kd0 = tc::smem_desc_sw128(sbase + L::kSmRing, 16, 1024);
        const uint64_t vd0 = tc::smem_desc_sw128(sbase + L::kSmV, L::kVKeys * 128, 1024);
        const uint32_t idesc_s = tc::idesc_f16_f32_ab(128, BN, false, false);
        int raises = 0;
        // S of a group and tile j, whose parity is ODD
        auto scores = [&](auto odd, int g, int j, bool both) {
            constexpr int ODD = decltype(odd)::value;
            const int b = kGroups > 1 ? g : ODD;  // the group's tile of scores
            if (j >= L::kBuf) wait(L::kSFree + b, j / L::kBuf - 1);
            if (g == 0) wait(L::kK + ODD, j >> 1);
            tc::fence_after_sync();
            if (one) {
                if (g == 0 || both) {
#pragma unroll
                    for (int k = 0; k < 8 * H; ++k)
                        tc::mma_ss(tmem + L::kTmS + b * 64, qd + (uint64_t)(((k >> 2) * NMAX * 128 + g * 64 * 128 + (k & 3) * 32) >> 4),
                                   kd0 + (uint64_t)((ODD * L::kTile + (k >> 2) * 64 * 128 + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
                }
                tc::mma_commit(B(L::kS + b));
                if (g == kGroups - 1) tc::mma_commit(B(L::kKFree + ODD));
            }
            __syncwarp();
        };
        // O^T (+)= V^T P^T of tile j
        auto product = [&](auto odd, int j, uint32_t idesc, int n16, uint32_t more) {
            constexpr int ODD = decltype(odd)::value, kBufP = L::kBuf > 1 ? ODD : 0;
            wait(L::kP + kBufP, pp(j));
            if (kGroups > 1 && more && raised_b[ODD]) {  // its rows' columns in the lanes of the warps that it lacks
                wait(L::kO + pb(j - 1), pp(j - 1));
                tc::fence_after_sync();
                rescale(j, 128, n16);
                wait(L::kR, raises++);
                tc::fence_before_sync();
                __syncwarp();
            }
            wait(L::kV + kBufP, pp(j));
            tc::fence_after_sync();
            if (one) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int m = 0; m < L::kMt; ++m)
#pragma unroll
                        for (int k = 0; k < L::kVKeys / 16; ++k)
                            tc::mma_ss(tmem + L::kTmO + m * NMAX, vd0 + (uint64_t)((kBufP * L::kTile + h * L::kSlot + m * 2 * L::kVKeys * 128 + k * 2048) >> 4),
                                       pd + (uint64_t)((kBufP * NMAX * 128 + h * L::kVKeys * 2 + k * 32) >> 4), idesc, h > 0 || k > 0 ? 1u : more);
                tc::mma_commit(B(L::kO + kBufP));
            }
            __syncwarp();
        };
        constexpr std::integral_constant<int, 0> even{};
        constexpr std::integral_constant<int, 1> odd{};
        int j = 0, segs = 0;
#pragma unroll 1
        while (walk.next(p, seg)) {
            wait(L::kQ, segs++);
            const int n16 = (seg.n + 15) & ~15;
            const uint32_t idesc_o = tc::idesc_f16_f32_ab(128, n16, true, false);
            const bool both = kGroups > 1 && seg.n > 128;
            const int t0 = seg.t0, t1 = seg.t1;
#pragma unroll 1
            for (int t = t0; t <= t1; ++t) {
                // the scores of tile t, number j, then the product of the tile before
                const uint32_t more = t - 1 > t0 ? 1u : 0u;
                if (j & 1) {
                    if (t < t1) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) scores(odd, g, j, both);
                    }
                    if (t > t0) product(even, j - 1, idesc_o, n16, more);
                } else {
                    if (t < t1) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) scores(even, g, j, both);
                    }
                    if (t > t0) product(odd, j - 1, idesc_o, n16, more);
                }
                if (t < t1) ++j;
            }
        }
        if (kGroups > 1 && lane < 2) {
            raised_b[2] = 0;
            tc::mbar_arrive(B(L::kRaise));
        }
        if (!wait.ok) atomicOr(p.error, 1u);
    } else if (warp == kHelpWarp) {
        // When the second group raises references: their columns in lanes 32-63 (the product's warp has lanes 0-31).  It
        // sleeps between raises, so its patience is for the whole scan; the last signal says that there is nothing to do.
        if (kGroups > 1) {
#pragma unroll 1
            for (int raises = 0;; ++raises) {
#pragma unroll 1
                for (int i = 0; i < 64; ++i) {
                    wait.ok = true;
                    wait(L::kRaise, raises);
                    if (wait.ok) break;
                }
                const int n16 = raised_b[2];
                if (!wait.ok || n16 == 0) break;
                tc::fence_after_sync();
                rescale(raised_b[3], 128, n16);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(B(L::kR));
            }
            if (!wait.ok) atomicOr(p.error, 1u);
        }
    } else if (warp < kConvWarp0) {
        float* inv = reinterpret_cast<float*>(tab + L::kTabInv);
        int* out_row = reinterpret_cast<int*>(tab + L::kTabRow);
        int* misc = reinterpret_cast<int*>(tab + L::kTabMisc);  // largest query of each warp
        const int g = warp >> 2, sid = g ? tid - 64 : tid;
        // this thread's row of the CTA's: lane of the group's scores; the second group's are rows 64 .. 191, its first 64 lanes
        // repeating rows of the first (a 64-row tile would cost the tensor cores as much)
        const int row = g * 64 + quad * 32 + lane;
        const bool owner = g == 0 ? row < NMAX : kGroups > 1;
        float cs = 0.0f, cs_next = 0.0f;
        uint64_t next_mask = 0;

        // Queries of a segment into shared memory (16-byte chunks of row r at chunk ^ r % 8) and its rows' table.  Called
        // once every product with the queries before has been read.  Rows that are not there keep what was there: what
        // comes of them stays in lanes and columns that nobody reads.
        auto stage = [&](const Segment& s, int parity) {
            const int pieces = s.n * (HD / 8);
            auto at = [&](int i) {  // where piece i (16 bytes of row i / (HD / 8)) lies
                const int r = i / (HD / 8), c = i - r * (HD / 8);
                return L::kSmQ + (c >> 3) * (NMAX * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            };
            // all pieces at once: one round trip to memory
#pragma unroll 4
            for (int i = sid; i < pieces; i += kSoftThreads) {
                const int r = i / (HD / 8), c = i - r * (HD / 8), q_rr = s.r0 + r, t = window_row(p, q_rr);
                const int64_t off = (int64_t)(s.q.row0 + t) * p.q_stride + (int64_t)(s.kvh * p.group + q_rr - t * p.group) * HD + c * 8;
                cp_async_16(sbase + at(i), static_cast<const uint16_t*>(p.q) + off, 16);
            }
            cp_async_commit();
            next_mask = 0;
            if (owner && row < s.n) {
                const int rr = s.r0 + row, t = window_row(p, rr), my_row = s.q.row0 + t;
                next_mask = p.mask ? __ldg(p.mask + my_row) : (2ull << t) - 1;
                if (s.q.rows < 64) next_mask &= (1ull << s.q.rows) - 1;
                out_row[parity * NMAX + row] = my_row * p.n_q_heads + s.kvh * p.group + rr - t * p.group;
            }
            cp_async_wait<0>();
            float lifted = 1.0f;
            if (Query<T>::kLifted) {  // a thread reads and rewrites the pieces that it fetched
                uint32_t top = 0;
#pragma unroll 2
                for (int i = sid; i < pieces; i += kSoftThreads) top = max(top, Query<T>::top(*reinterpret_cast<const uint4*>(smem + at(i))));
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) misc[sid >> 5] = (int)top;
                soft_sync();
                uint32_t most = 0;
#pragma unroll
                for (int w = 0; w < kSoftThreads / 32; ++w) most = max(most, (uint32_t)misc[w]);
                lifted = lift_of(most);
#pragma unroll 2
                for (int i = sid; i < pieces; i += kSoftThreads) {
                    uint4* q16 = reinterpret_cast<uint4*>(smem + at(i));
                    const uint4 v = *q16;
                    *q16 = make_uint4(Query<T>::pair(v.x, lifted), Query<T>::pair(v.y, lifted), Query<T>::pair(v.z, lifted),
                                      Query<T>::pair(v.w, lifted));
                }
            }
            cs_next = p.scale_log2 / lifted;
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B(L::kQ));
        };

        Segment next_seg;
        bool more = walk.next(p, next_seg);
        int j = 0, segs = 0;
#pragma unroll 1
        while (true) {
            // a segment's queries go in before the one before's output is read: its first scores overlap that
            const int parity = segs & 1;
            if (more) stage(next_seg, parity);
            if (segs > 0) {
                wait(L::kO + pb(j - 1), pp(j - 1));
                tc::fence_after_sync();
                const bool whole = seg.begins() && seg.ends();
                const int slot = 2 * blockIdx.x + (seg.begins() ? 1 : 0), n = seg.n;
                const int* rows = out_row + (parity ^ 1) * NMAX;
                // a warp's 32 lanes of the first 128-dim tile, and of the second: warps 6 and 7 those of 2 and 3, warps 0 and 1
                // their own as well
                for (int m = g ? 1 : 0; m < (g == 0 && quad < 2 ? L::kMt : L::kMt == 1 ? 1 - g : 1 + g); ++m) {
                    const int dim = m * 128 + quad * 32 + lane;
#pragma unroll 1
                    for (int c0 = 0; c0 < n; c0 += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tmem + lanes + L::kTmO + m * NMAX + c0, o);
                        tc::tmem_wait_ld();
                        if (whole) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (c0 + c < n) {
                                    const float f = inv[c0 + c];
                                    static_cast<uint16_t*>(p.out)[(int64_t)rows[c0 + c] * HD + dim] =
                                        f != 0.0f ? Query<T>::one(__uint_as_float(o[c]) * f) : (uint16_t)0;
                                }
                        } else {
                            float* dst = p.part_o + ((int64_t)slot * p.chunk + c0) * HD + dim;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (c0 + c < n) dst[c * HD] = __uint_as_float(o[c]);
                        }
                    }
                }
                tc::fence_before_sync();
                soft_sync();  // the tables have been read
            }
            if (!more) break;
            seg = next_seg;
            cs = cs_next;
            const uint64_t window = next_mask;
            // (walk and segments live in local memory, which this much shared memory leaves little cache for: the loop below
            // reads none of them)
            const bool mine = owner && row < seg.n, live = __any_sync(0xffffffffu, mine);
            const int t0 = seg.t0, t1 = seg.t1, len = seg.q.len, ctx = len - seg.q.rows, n16 = (seg.n + 15) & ~15;
            float ref = kNoRef, neg = kLift - kNoRef, l = 0.0f;
            const int32_t* pages = p.table + (int64_t)seg.b * p.max_pages;
            auto page_of = [&](int t) {  // lane x < 4: of keys 16 x .. of the tile, loaded a tile ahead
                const long long key = (long long)t * BN + 16 * lane;
                return lane < 4 && t < t1 && key < len ? __ldg(pages + (key >> p.page_shift)) : 0;
            };
            int page = page_of(t0);
            if (g < kGroups) {
#pragma unroll 1
                for (int t = t0; t < t1; ++t, ++j) {
                    const uint32_t bad = __ballot_sync(0xffffffffu, page < 0 || page >= p.n_pages);
                    page = page_of(t + 1);
                    // the tile's keys that this row sees
                    uint64_t sees = ~0ull;
                    const long long past = (long long)ctx - (long long)t * BN;  // cached keys from the tile's first on
                    if (past < BN) sees = past > 0 ? ((1ull << past) - 1) | window << past : window >> -past;
                    if (bad) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (bad >> x & 1) sees &= ~(0xffffull << (16 * x));
                    }
                    const int b = kGroups > 1 ? g : j & 1;
                    wait(L::kS + b, j / L::kBuf);
                    tc::fence_after_sync();
                    // The scores in registers, so that their place is free for the next tile's at once; those of unseen keys -inf.
                    uint32_t x[64];
                    if (live) tc::tmem_ld64(tmem + lanes + L::kTmS + b * 64, x);
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(B(L::kSFree + b));
                    bool raise = false;
                    float top = 0.0f;
                    if (live) {
                        if (!__all_sync(0xffffffffu, sees == ~0ull)) {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                if (!((c < 32 ? (uint32_t)sees : (uint32_t)(sees >> 32)) >> (c & 31) & 1)) x[c] = 0xff800000u;
                        }
                        float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 64; ++c) most[c & 3] = fmaxf(most[c & 3], __uint_as_float(x[c]));
                        top = cs * fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                        raise = mine && top > ref + kLazy;
                    }
                    // references of the group to the tile's maxima where those are more than 2^8 above; sums and O^T follow
                    const bool raised = group_any(g, raise);
                    if (raised) {
                        float a = 1.0f;
                        if (raise) {
                            a = ref == kNoRef ? 0.0f : ex2_approx(ref - top);
                            ref = top;
                            neg = kLift - top;
                            l *= a;
                        }
                        if (owner) alpha[(j & 1) * NMAX + row] = a;
                    }
                    if (kGroups > 1 && warp == 6 && lane == 0) raised_b[j & 1] = raised;
                    if (live) {
                        float part[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float e0 = ex2_approx(fmaf(__uint_as_float(x[c]), cs, neg));
                            const float e1 = ex2_approx(fmaf(__uint_as_float(x[c + 1]), cs, neg));
                            x[c / 2] = h2_as_u32(__floats2half2_rn(e0, e1));
                            add_halves(part, x[c / 2]);
                        }
                        l += part[0] + part[1];
                    }
                    if (j >= L::kBuf) wait(L::kO + pb(j), pp(j) - 1);  // the weights before in this place have been used
                    if (raised && t > t0) {
                        wait(L::kO + pb(j - 1), pp(j - 1));  // every product so far has landed
                        tc::fence_after_sync();
                        group_sync(g);
                        if (g && lane == 0) {
                            raised_b[2] = n16;
                            raised_b[3] = j;
                            tc::mbar_arrive(B(L::kRaise));
                        }
                        rescale(j, 128 * g, g == 0 ? min(n16, 128) : n16);
                    }
                    if (live && owner) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            sts128(sbase + L::kSmP + pb(j) * NMAX * 128 + row * 128 + ((c ^ (row & 7)) << 4),
                                   make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]));
                    }
                    tc::fence_proxy_async_smem();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(B(L::kP + pb(j)));
                }
            } else {
                j += seg.t1 - seg.t0;
            }
            if (mine) {
                inv[row] = l != 0.0f ? 1.0f / l : 0.0f;  // (NaN stays one)
                if (!(seg.begins() && seg.ends()))
                    p.part_ml[(int64_t)(2 * blockIdx.x + (seg.begins() ? 1 : 0)) * p.chunk + row] =
                        make_float2(ref == kNoRef ? -INFINITY : ref, l);
            }
            soft_sync();  // every score has been read, so the queries are free
            ++segs;
            more = walk.next(p, next_seg);
        }
        if (!wait.ok) atomicOr(p.error, 1u);
    } else {
        // Four warps a plane, each at its own pace.  A thread converts two 32-value blocks of each half tile: lanes 0-7 the same
        // block of eight keys, so that their swizzled 16-byte stores fall into different banks.  A tile's codes are loaded while
        // the one before is converted, and the one after it is asked into L2.
        const int w = (warp - kConvWarp0) & 3, nn = lane & 7, jj = lane >> 3;
        const bool is_v = warp >= kConvWarp0 + 4;
        const int8_t* plane = is_v ? p.vc : p.kc;
        const uint16_t* scales = is_v ? p.vs : p.ks;
        // half s of a tile is its keys 32 s .. (V at head_dim 256), or its dims 128 s ..; block i of the thread in it the other
        // way round: its keys are 32 x + 8 w + nn, its blocks 4 y + jj
        const bool by_keys = is_v && H == 2;
        const uint32_t next = by_keys ? 8192 : 4096;  // from block 0 to block 1
        const uint32_t dst = sbase + (is_v ? L::kSmV : L::kSmRing) + (jj >> 1) * (by_keys ? 4096 : 8192) + (8 * w + nn) * 128 + (((4 * (jj & 1)) ^ nn) << 4);
        uint32_t codes[H][2][8], scale[H][2];
        uint32_t row[2];
        bool there[2] = {false, false};
        int t = 0, t1 = 0, len = 0, kvh = 0;
        const int32_t* pages = p.table;
        int page[kAhead + 2];  // lane x < 4: page of keys 16 x .. of the tile and of the next ones
        bool have = false;
        auto page_of = [&](int u) {
            const long long key = (long long)u * BN + 16 * lane;
            return lane < 4 && u < t1 && key < len ? __ldg(pages + (key >> p.page_shift)) : -1;
        };
        // The cache row of key `key` of tile u, whose page is among `ids`.
        auto row_of = [&](int ids, int u, int key, uint32_t& row) {
            const int id = __shfl_sync(0xffffffffu, ids, key >> 4);
            const uint32_t off = ((uint32_t)u * BN + key) & ((1u << p.page_shift) - 1);
            row = (((uint32_t)id * p.n_kv_heads + kvh) << p.page_shift) + off;
            return id >= 0 && id < p.n_pages && (long long)u * BN + key < len;
        };
        auto ahead = [&]() {
            if (have && ++t < t1) {
#pragma unroll
                for (int x = 0; x <= kAhead; ++x) page[x] = page[x + 1];
            } else {
                have = walk.next(p, seg);
                if (!have) return;
                t = seg.t0, t1 = seg.t1, len = seg.q.len, kvh = seg.kvh;
                pages = p.table + (int64_t)seg.b * p.max_pages;
#pragma unroll
                for (int x = 0; x <= kAhead; ++x) page[x] = page_of(t + x);
            }
            page[kAhead + 1] = page_of(t + kAhead + 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) there[x] = row_of(page[0], t, 32 * x + 8 * w + nn, row[x]);
            // a 128-byte line of codes of the tile after next per thread, and the scales
            uint32_t line;
            if (row_of(page[kAhead], t + kAhead, 16 * w + (lane >> 1), line) && (H == 2 || !(lane & 1))) {
                prefetch_l2(plane + (uint64_t)line * HD + 128 * (lane & 1));
                if ((lane & 15) == 0) prefetch_l2(scales + (uint64_t)line * (HD / 32));
            }
        };
        // What is not there gets scale 0, and any codes.
        auto load = [&](int s) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = by_keys ? s : i, block = 4 * (by_keys ? i : s) + jj;
                const uint64_t r = x ? row[1] : row[0];
                scale[s][i] = 0;
                if (x ? there[1] : there[0]) {
                    load32(codes[s][i], plane + r * HD + 32 * block);
                    load_u16(scale[s][i], scales + r * (HD / 32) + block);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < 2 * H; ++i)
#pragma unroll
            for (int x = 0; x < 8; ++x) codes[i >> 1][i & 1][x] = 0u;
        ahead();
        if (have) {
#pragma unroll
            for (int s = 0; s < H; ++s) load(s);
        }
#pragma unroll 1
        for (int j = 0; have; ++j) {
            ahead();
            // the place's last use: of K^ by the scores of tile j - 2, of V^ by the product of tile j - kBuf
            const int place = is_v ? pb(j) : j & 1, free = is_v ? L::kO + place : L::kKFree + place, last = (is_v ? pp(j) : j >> 1) - 1;
            const bool is_free = last < 0 || tc::mbar_try_wait(B(free), (uint32_t)last & 1u);
            const uint32_t to = dst + place * L::kTile;
#pragma unroll
            for (int s = 0; s < H; ++s) {
                uint32_t v[2][16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 d = __half2half2(__ushort_as_half((unsigned short)scale[s][i]));
                    uint32_t(&c)[8] = codes[s][i];
                    values16(make_uint4(c[0], c[1], c[2], c[3]), d, v[i]);
                    values16(make_uint4(c[4], c[5], c[6], c[7]), d, v[i] + 8);
                }
                if (have) load(s);
                if (s == 0 && !is_free) wait(free, last);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        sts128((to + s * L::kSlot + i * next) ^ (c << 4), make_uint4(v[i][4 * c], v[i][4 * c + 1], v[i][4 * c + 2], v[i][4 * c + 3]));
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(B((is_v ? L::kV : L::kK) + place));
        }
        if (!wait.ok) atomicOr(p.error, 1u);
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0) leave_join<BN>(p, *place);
}

template <typename T, int HD, int N>
int launch(const PagedVerifyParams& p, int ctas, cudaStream_t s) {
    static SmemOptIn opt;
    if (opt.ensure(paged_verify_rows_kernel<T, HD, N>, RL<HD, N>::kSmBytes) != KVQ8_OK) return KVQ8_ERR_CUDA;
    return launch_dependent(paged_verify_rows_kernel<T, HD, N>, ctas, kVerifyThreads, RL<HD, N>::kSmBytes, s, p);
}

template <typename T, int HD>
int launch(const PagedVerifyParams& p, int n, int ctas, cudaStream_t s) {
    return n <= 64 ? launch<T, HD, 64>(p, ctas, s) : launch<T, HD, 192>(p, ctas, s);
}

}  // namespace

int launch_verify_rows(const PagedVerifyParams& p, int dtype, int hd, int n, int ctas, cudaStream_t s) {
    if (hd == 128) return dtype == KVQ8_F16 ? launch<__half, 128>(p, n, ctas, s) : launch<__nv_bfloat16, 128>(p, n, ctas, s);
    return dtype == KVQ8_F16 ? launch<__half, 256>(p, n, ctas, s) : launch<__nv_bfloat16, 256>(p, n, ctas, s);
}

}  // namespace kvq8

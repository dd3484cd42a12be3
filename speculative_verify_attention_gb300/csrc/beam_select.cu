// beam_select.cu -- beam search's choice: of every request's beams and the whole vocabulary the n_out best continuations.
//
// Row r (a beam) with score c continues with value v at  total = c + x[v] - log sum_v exp x[v],  ordered by weight * total.
// The n_out best of a request lie among the n_out best of each of its rows, which are the n_out best logits x.
//
// One pass over the logits.  A warp holds groups of a kilobyte of consecutive values in registers and leaves behind each group's
// maximum, and one partial sum of exponentials of all that it has held: 1/200 of what it read.  Ordered by (maximum descending, place
// ascending), the n_out best groups hold the row's n_out best values: a value outside them has n_out values before it, one in each.
// So the second kernel, a block per row, picks those groups, reads them again and picks the values; a request's blocks form a
// cluster, which joins their lists through shared memory.  Where there are many rows it has a warp per row and a block per request
// instead, and where the vocabulary is small that kernel does it all.
// Bound: the logits' bytes in the first kernel, latency in the others.  48 requests of 8 beams over 248320 bf16 logits (159 MB), 16 of
// each: 34.2 us, of which the scan 27.5 (5.8 TB/s, 85 % of a copy's rate; issue slots 69 % busy) and the second kernel 6.7; one request of
// 4 fp32 beams 6.7 us; 21 of up to 5 over 106299 fp16 logits (21 MB) 11.7 us.  As first built, with groups picked by rounds of five
// barriers and the join by the last block to finish: 74, 26 and 31 us.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kScanThreads = 256;
// Values of a group: a kilobyte.  A warp holds 1024 values at once, kLoads times eight a lane.
template <typename T>
constexpr int kGroup = 1024 / (int)sizeof(T);
constexpr int kChunk = 1024, kLoads = kChunk / 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kManyChunks = 152 * 40;  // chunks that the GPU's warps hold at once
constexpr int kSearchThreads = 256;
constexpr int kPickThreads = kSearchThreads + 32;
constexpr int kMaxOut = 64;
constexpr int kKeep = 4;           // groups of a row that a searching thread keeps: all of 262144 fp32 values
constexpr int kPartKeep = 8;       // parts of a row that a lane of the summing warp keeps
// Tiles of 256 values that a searching lane loads at once: 24 registers.
template <typename T, bool VEC>
constexpr int kFetch = sizeof(T) == 2 && VEC ? 6 : 3;
constexpr int kGroupCap = 256;     // groups, and values, that the second kernel keeps of a row
constexpr int kListCap = 512;

// The sum of exp over a warp's values, whose maximum is m: s * 2^e, or s * exp(m) where |m| >= kLarge (e would not be near
// m log2 e there).  s is NaN if a value is NaN or +infinite.
struct Part {
    float m, e, s;
};
constexpr float kLarge = 0x1p20f;
// log2 of what s is to be multiplied by.
__device__ __forceinline__ double scale_of_part(float m, float e) { return fabsf(m) < kLarge ? (double)e : (double)m * (double)kLog2e; }

struct SelectParams {
    const void* logits;
    int64_t stride;
    const int32_t* row_starts;
    const float* scores;
    const float* weights;
    const int32_t* ended;
    int32_t* parents;
    int32_t* tokens;
    float* totals;
    // workspace
    float* group_max;       // [n_rows][n_groups]
    Part* parts;            // [n_rows][n_parts]
    int n_rows, vocab, n_seqs, n_out, n_groups, n_parts, n_chunks, turns;
};

// fp32 as whole numbers of the same order (-0 as 0).
__device__ __forceinline__ int32_t ordered(float x) {
    const int32_t b = __float_as_int(x + 0.0f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int32_t o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }
__device__ __forceinline__ int64_t ordered(double x) {
    const int64_t b = __double_as_longlong(x + 0.0);
    return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// Unique and ascending in quality: larger values first, of equal ones the lower place.
__device__ __forceinline__ uint64_t key_of(int32_t ord, uint32_t place) {
    return (uint64_t)((uint32_t)ord ^ 0x80000000u) << 32 | (0xffffffffu - place);
}
__device__ __forceinline__ float key_value(uint64_t k) { return from_ordered((int32_t)((uint32_t)(k >> 32) ^ 0x80000000u)); }
__device__ __forceinline__ uint32_t key_place(uint64_t k) { return 0xffffffffu - (uint32_t)k; }

// Whether request b has rows, and which.
__device__ __forceinline__ bool rows_of(const SelectParams& p, int b, int& first, int& rows) {
    first = __ldg(p.row_starts + b);
    const int last = __ldg(p.row_starts + b + 1);
    rows = last - first;
    return first >= 0 && first < last && last <= p.n_rows && rows <= kMaxWindowRows;
}

template <typename T>
constexpr uint32_t kLowestWord = 0xff800000u;  // -inf, or two of them
template <>
constexpr uint32_t kLowestWord<__half> = 0xfc00fc00u;
template <>
constexpr uint32_t kLowestWord<__nv_bfloat16> = 0xff80ff80u;

// How a warp reads 256 consecutive values of a row, eight a lane, -inf outside the row.
//   VEC: eight consecutive ones a load; the row starts on their size and holds whole groups of them.
//   Rows of odd length in 16 bits: the two 16-byte pieces around a lane's eight, and where among those they start (`shift`, of the row
//     alone) comes to a funnel shift a word; 320 rows of 106299 bf16 values 22.5 us (by selections 26; 106304 values 19.4).
//   SPREAD, of fp32 and where rows are read as wholes: a value a load, neighbours to neighbouring lanes (100 fp32 rows of 106299: 13.6 us;
//     by three pieces and selections 17.6.  4000 bf16 rows of 1001 as wholes 11.8 us, by pieces 16.9).
template <typename T, bool VEC, bool SPREAD = sizeof(T) == 4 && !VEC>
struct Tile {
    static constexpr bool kSpread = SPREAD;
    // the place of value e of a lane, in the 256 from `at` on
    static __device__ __forceinline__ int place(int at, int lane, int e) { return kSpread ? at + e * 32 + lane : at + lane * 8 + e; }

    // 16 bits, odd: pieces of eight values, each from its own size's boundary on
    static __device__ __forceinline__ bool whole(int from, int vocab) { return from >= 0 && from + 8 <= vocab; }
    static __device__ __forceinline__ void pieces(uint32_t (&w)[8], const T* row, int from, int vocab) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint4 r = make_uint4(kLowestWord<T>, kLowestWord<T>, kLowestWord<T>, kLowestWord<T>);
            if (whole(from + 8 * k, vocab)) r = __ldg(reinterpret_cast<const uint4*>(row + from + 8 * k));
            w[4 * k] = r.x, w[4 * k + 1] = r.y, w[4 * k + 2] = r.z, w[4 * k + 3] = r.w;
        }
    }
    // the row's first and last piece
    static __device__ __forceinline__ void ends(uint32_t (&w)[8], const T* row, int from, int vocab) {
#pragma unroll
        for (int k = 0; k < 2; ++k, from += 8) {
            if (from <= -8 || from >= vocab || whole(from, vocab)) continue;
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = kLowestWord<T> & 0xffffu;
                if (from + i >= 0 && from + i < vocab) v[i] = *reinterpret_cast<const uint16_t*>(row + from + i);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * k + i] = v[2 * i] | v[2 * i + 1] << 16;
        }
    }
    // N times 256 values, from at[u] on
    template <int N>
    static __device__ __forceinline__ void load(Eight<T> (&x)[N], const T* row, const int (&at)[N], int vocab, int lane) {
        if constexpr (kSpread) {
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = place(at[u], lane, e);
                    x[u].put(e, i < vocab ? __ldg(row + i) : static_cast<T>(-INFINITY));
                }
        } else if constexpr (VEC) {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int i = at[u] + lane * 8;
                if (i < vocab) {
                    x[u].load_whole(row + i);
                } else {
#pragma unroll
                    for (int k = 0; k < (int)sizeof(T) * 2; ++k) reinterpret_cast<uint32_t*>(&x[u])[k] = kLowestWord<T>;
                }
            }
        } else {
            const int shift = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)), bits = (shift & 1) * 16;
            uint32_t w[N][8];
#pragma unroll
            for (int u = 0; u < N; ++u) pieces(w[u], row, at[u] + lane * 8 - shift, vocab);
#pragma unroll
            for (int u = 0; u < N; ++u) ends(w[u], row, at[u] + lane * 8 - shift, vocab);
            auto take = [&](auto words) {  // one branch for all, as the shift is the warp's
#pragma unroll
                for (int u = 0; u < N; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u].w[i] = __funnelshift_r(w[u][i + words.value], w[u][i + words.value + 1], bits);
            };
            if (shift < 2)
                take(std::integral_constant<int, 0>{});
            else if (shift < 4)
                take(std::integral_constant<int, 1>{});
            else if (shift < 6)
                take(std::integral_constant<int, 2>{});
            else
                take(std::integral_constant<int, 3>{});
        }
    }
};

// The largest of eight values; NaN loses.
__device__ __forceinline__ float largest(const Eight<float>& x) {
    float m = fmaxf(x.v[0], x.v[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) m = fmaxf(m, x.v[i]);
    return m;
}
__device__ __forceinline__ float largest(const Eight<__half>& x) {
    const __half2 m = __hmax2(__hmax2(u32_as_h2(x.w[0]), u32_as_h2(x.w[1])), __hmax2(u32_as_h2(x.w[2]), u32_as_h2(x.w[3])));
    return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float largest(const Eight<__nv_bfloat16>& x) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(x.w);
    const __nv_bfloat162 m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float warp_max(float x) {  // NaN loses here too
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

// The exponentials of a chunk join a lane's sum, m the largest value of both.
// A sum's error, relative to it: 2^-22 of the exponential (which is exact of whole numbers, so scaling by it costs nothing), 2^-24 for
// each addition a value goes through (9 here, one a chunk of its lane, 5 between lanes), 2^-24 (H + 1/2) of the exponents' rounding and
// 1.4e-8 H of log2 e's, H <= ln V the entropy of the row's distribution.  Less than 3e-6 for all sizes but for the parts' own rounding
// (add_parts: V / 1024 of them, 2^-33 each); rows of 1000 to 248320 values, of 80 types, spreads and
// routes, were 2.7e-7 off at most.
template <typename T>
__device__ __forceinline__ void add_to(Part& sum, const Eight<T> (&v8)[kLoads], float m) {
    if (fabsf(m) < kLarge) {
        const float e = rintf(m * kLog2e);
        float s = sum.s;
        if (fabsf(sum.m) < kLarge)
            s *= ex2_approx(sum.e - e);
        else if (sum.m > -INFINITY)
            s *= exp2f((float)(scale_of_part(sum.m, sum.e) - (double)e));
        float add[kLoads];  // (short chains: a value goes through 10 additions and one for each chunk after its own)
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            float v[8];
            v8[u].floats(v);
            add[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) add[u] += ex2_approx(__fmaf_rn(v[i], kLog2e, -e));
        }
        sum = {m, e, s + ((add[0] + add[1]) + (add[2] + add[3]))};
    } else {
        const bool any = fabsf(m) < INFINITY;
        float s = sum.m > -INFINITY ? sum.s * exp2f((float)(scale_of_part(sum.m, sum.e) - scale_of_part(m, 0.0f))) : sum.s;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            float v[8];
            v8[u].floats(v);  // of -inf alone nothing; a NaN or +inf makes the sum NaN
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                s += any ? ex2_approx((v[0] - m) * kLog2e) : v[0] == -INFINITY ? 0.0f : NAN;
#pragma unroll
                for (int w = 0; w < 7; ++w) v[w] = v[w + 1];
            }
        }
        sum = {m, 0.0f, s};
    }
}

// log2 near 1 + (i + 1/2) / 32, i < 32, made when this file is compiled: 64-bit arithmetic is slow here (2 a clock on a multiprocessor).
struct LogValues {
    float inverse[32];
    double log_of[32];
    constexpr LogValues() : inverse{}, log_of{} {
        for (int i = 0; i < 32; ++i) {
            inverse[i] = (float)(64.0 / (64 + 2 * i + 1));
            const double z = (1.0 - inverse[i]) / (1.0 + inverse[i]);  // -log(inverse) = 2 (z + z^3/3 + z^5/5 + ...), z <= 1/3
            double s = 0.0;
            for (int k = 41; k >= 1; k -= 2) s = s * z * z + 1.0 / k;
            log_of[i] = 2.0 * z * s * 1.4426950408889634074;
        }
    }
};
__device__ const LogValues kLogs{};
// One entry a lane, loaded ahead of its use.
struct LogTable {
    float inverse;
    double log_of;
    __device__ __forceinline__ explicit LogTable(int lane) : inverse(kLogs.inverse[lane]), log_of(kLogs.log_of[lane]) {}
    // log2 of a sum in units of 2^-32, by the lane nearest to its mantissa m and the series of log2(1 + f), 1 + f = m * inverse,
    // |f| <= 1/64.  f is exact to half a step of fp32 (2^-31) for m's upper 24 bits, and so is what is added for the others; with the
    // series' terms the result is off by 2^-28 at most.  All lanes of the warp; a sum of 0 gives no more than some number.
    __device__ __forceinline__ double log2_of(unsigned long long sum) const {
        const int top = 63 - __clzll((long long)(sum | 1));
        const uint64_t mantissa = sum << 1 << (63 - top);  // behind the leading one
        const int near = (int)(mantissa >> 59);
        const float i = __shfl_sync(0xffffffffu, inverse, near);
        const float f = __fmaf_rn(__uint_as_float(0x3f800000u | (uint32_t)(mantissa >> 41)), i, -1.0f) +
                        (float)((uint32_t)(mantissa >> 17) & 0xffffffu) * 0x1p-47f * i;
        const float tail = f * f * (-0.5f + f * (1.0f / 3.0f + f * (-0.25f + f * (0.2f + f * (-1.0f / 6.0f)))));
        return (double)(top - 32) + (__shfl_sync(0xffffffffu, log_of, near) + (double)((f + tail) * 1.44269504f));
    }
};
// log sum exp, of a sum whose log2 is that and whose values' largest is top
__device__ __forceinline__ double norm_of(float top, float e, double log2_sum) {
    return fabsf(top) < kLarge ? ((double)e + log2_sum) * (1.0 / (double)kLog2e) : (double)top + log2_sum * 0.69314718055994530942;
}

// A row's parts, scaled by powers of two to the largest one's and added as whole numbers of 2^-32, so that their order does not matter.
// True where a value was NaN or +infinite.  All lanes of a warp.
__device__ __forceinline__ bool add_parts(const Part* parts, int n, int lane, float& top, float& e, unsigned long long& sum) {
    int32_t m = ordered(-INFINITY);
    bool bad = false;
    Part kept[kPartKeep];
#pragma unroll
    for (int u = 0; u < kPartKeep; ++u) kept[u] = u * 32 + lane < n ? parts[u * 32 + lane] : Part{-INFINITY, -INFINITY, 0.0f};
    auto look = [&](const Part& q) {
        m = max(m, ordered(q.m));
        bad |= q.s != q.s;
    };
#pragma unroll
    for (int u = 0; u < kPartKeep; ++u) look(kept[u]);
    for (int i = kPartKeep * 32 + lane; i < n; i += 32) look(parts[i]);
    top = from_ordered(__reduce_max_sync(0xffffffffu, m));
    bad = __any_sync(0xffffffffu, bad);
    e = rintf(top * kLog2e);
    const bool plain = fabsf(top) < kLarge;
    sum = 0;
    auto add = [&](const Part& q) {
        float v = 0.0f;
        if (plain && fabsf(q.m) < kLarge)
            v = q.e - e > -126.0f ? q.s * __int_as_float((127 + (int)(q.e - e)) << 23) : 0.0f;
        else if (q.m > -INFINITY)
            v = q.s * exp2f((float)(scale_of_part(q.m, q.e) - scale_of_part(top, e)));
        sum += __float2ull_rn(v * 0x1p32f);
    };
#pragma unroll
    for (int u = 0; u < kPartKeep; ++u) add(kept[u]);
    for (int i = kPartKeep * 32 + lane; i < n; i += 32) add(parts[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return bad;
}

// A warp takes p.turns chunks of a row, and is one of its n_parts.  The sum so far is of 2^(x log2 e - e), e a whole number near the
// largest value so far (one rounding a value); a larger one scales it by a power of two.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ SelectParams p) {
    constexpr int kPerGroup = kGroup<T> / 256;  // loads of a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.ended && __ldg(p.ended + row) >= 0) return;
    const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
    Part sum = {-INFINITY, -INFINITY, 0.0f};
    int chunk = (int)blockIdx.x * p.turns * kScanWarps + warp;
    for (int turn = 0; turn < p.turns && chunk < p.n_chunks; ++turn, chunk += kScanWarps) {
        Eight<T> v8[kLoads];
        int at[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) at[u] = chunk * kChunk + u * 256;
        Tile<T, VEC>::load(v8, x, at, p.vocab, lane);
        float top[kLoads / kPerGroup], m = -INFINITY;
#pragma unroll
        for (int g = 0; g < kLoads / kPerGroup; ++g) {
            top[g] = warp_max(kPerGroup == 1 ? largest(v8[g]) : fmaxf(largest(v8[g * kPerGroup]), largest(v8[g * kPerGroup + kPerGroup - 1])));
            m = fmaxf(m, top[g]);
        }
        if (lane == 0) {
            float* to = p.group_max + (int64_t)row * p.n_groups + chunk * (kLoads / kPerGroup);
            if (kPerGroup == 1)
                *reinterpret_cast<float4*>(to) = make_float4(top[0], top[1], top[kLoads / kPerGroup - 2], top[kLoads / kPerGroup - 1]);
            else
                *reinterpret_cast<float2*>(to) = make_float2(top[0], top[1]);
        }
        add_to(sum, v8, fmaxf(m, sum.m));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
    if (lane == 0) p.parts[(int64_t)row * p.n_parts + (int)blockIdx.x * kScanWarps + warp] = sum;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The threads that search (the others of the block sum).
__device__ __forceinline__ void search_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct alignas(16) Search {
    uint64_t key[kListCap];      // candidates, as key_of
    uint64_t best[kMaxOut];      // the row's best, in order
    uint32_t group[kGroupCap];
    int32_t top[kSearchThreads];
    uint64_t above;              // keys below this are none of the best (slow path)
    int32_t bound;               // values below this are none of the best
    int n_groups, n;
};

// The best n_out of the n keys, in order.  All searching threads; the keys are different.
__device__ __forceinline__ void rank_keys(Search& s, int n, int n_out) {
    for (int i = threadIdx.x; i < n; i += kSearchThreads) {
        const uint64_t mine = s.key[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s.key[j] > mine;
        if (rank < n_out) s.best[rank] = mine;
    }
    search_sync();
}

// A bound of the row's n_out best, from a share's maximum in every `lanes` threads: the n_out-th best of them.
__device__ __forceinline__ void find_bound(Search& s, int32_t m, int lanes, int n_out) {
    const int tid = threadIdx.x, tops = kSearchThreads / lanes;
    for (int o = 1; o < lanes; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (tid % lanes == 0) s.top[tid / lanes] = m;
    search_sync();
    if (tid < tops) {
        m = s.top[tid];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < tops / 4; ++j) {
            const int4 o = reinterpret_cast<const int4*>(s.top)[j];
            rank += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
        }
        if (rank < n_out) atomicMin(&s.bound, m);
    }
    search_sync();
}

// The values of n tiles that reach least become candidates.
template <typename T, bool VEC, typename At>
__device__ __forceinline__ void gather(Search& s, const T* x, float least, int n, int vocab, At at_of) {
    constexpr int kTiles = kFetch<T, VEC>;
    const int lane = threadIdx.x & 31;
    for (int i0 = threadIdx.x >> 5; i0 < n; i0 += kTiles * (kSearchThreads / 32)) {
        Eight<T> v8[kTiles];
        {
            int at[kTiles];
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
                const int i = i0 + u * (kSearchThreads / 32);
                at[u] = i < n ? at_of(i) : vocab;
            }
            Tile<T, VEC>::load(v8, x, at, vocab, lane);
        }
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
            if (!(largest(v8[u]) >= least)) continue;
            const int at = at_of(i0 + u * (kSearchThreads / 32));
            float v[8];
            v8[u].floats(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!(v[e] >= least)) continue;
                const int place = atomicAdd(&s.n, 1);  // (one for all that a lane has is no faster)
                if (place < kListCap) s.key[place] = key_of(ordered(v[e]), (uint32_t)Tile<T, VEC>::place(at, lane, e));
            }
        }
    }
    search_sync();
}

// The candidates of a row of too few groups for a bound: by shares of the row itself, which is read twice.
template <typename T, bool VEC>
__device__ __noinline__ void gather_all(Search& s, const SelectParams& p, const T* x) {
    const int lane = threadIdx.x & 31, tiles = (p.vocab + 255) / 256;
    const int32_t lowest = ordered(-INFINITY);
    constexpr int kTiles = kFetch<T, VEC>;
    int32_t m = lowest;
    for (int i0 = threadIdx.x >> 5; i0 < tiles; i0 += kTiles * (kSearchThreads / 32)) {
        Eight<T> v8[kTiles];
        int at[kTiles];
#pragma unroll
        for (int u = 0; u < kTiles; ++u) at[u] = min((i0 + u * (kSearchThreads / 32)) * 256, p.vocab);
        Tile<T, VEC>::load(v8, x, at, p.vocab, lane);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) m = max(m, ordered(largest(v8[u])));
    }
    find_bound(s, m, p.n_out <= 16 ? 4 : 2, p.n_out);
    gather<T, VEC>(s, x, from_ordered(max(s.bound, lowest + 1)), tiles, p.vocab, [](int i) { return i * 256; });
}

// Where more groups or values reach the bound than the lists hold (many equal values): the row's groups, and then the best ones'
// values, a key a thread at a time; a full list is cut back to its best n_out, below which nothing is taken any more.
template <typename T, bool VEC>
__device__ __noinline__ int pick_slowly(Search& s, const SelectParams& p, const T* x, const float* gm) {
    const int tid = threadIdx.x, n_out = p.n_out;
    auto cut = [&] {
        const int n = s.n;
        rank_keys(s, n, n_out);
        const int m = min(n, n_out);
        if (tid < m) s.key[tid] = s.best[tid];
        if (tid == 0) {
            s.n = m;
            if (m == n_out) s.above = s.best[n_out - 1];
        }
        search_sync();
    };
    auto add = [&](uint64_t k) {
        const bool full = s.n + kSearchThreads > kListCap;
        search_sync();  // every thread has seen the same count before the first one adds to it
        if (full) cut();
        if (k > s.above) s.key[atomicAdd(&s.n, 1)] = k;
        search_sync();
    };
    search_sync();
    if (tid == 0) s.n = 0, s.above = 0;
    search_sync();
#pragma unroll 1
    for (int g0 = 0; g0 < p.n_groups; g0 += kSearchThreads) add(g0 + tid < p.n_groups ? key_of(ordered(gm[g0 + tid]), (uint32_t)(g0 + tid)) : 0);
    cut();
    const int groups = s.n;
    if (tid < groups) s.group[tid] = key_place(s.key[tid]);
    search_sync();
    if (tid == 0) s.n = 0, s.above = 0;
    search_sync();
#pragma unroll 1
    for (int i = 0; i < groups * (kGroup<T> / kSearchThreads); ++i) {
        const int at = (int)s.group[i / (kGroup<T> / kSearchThreads)] * kGroup<T> + i % (kGroup<T> / kSearchThreads) * kSearchThreads + tid;
        const float v = at < p.vocab ? to_float(x[at]) : -INFINITY;
        add(v > -INFINITY ? key_of(ordered(v), (uint32_t)at) : 0);
    }
    cut();
    return s.n;
}

// What the blocks of a request's cluster have found: each has its rows' totals and tokens, n_out places a row (block c has the
// rows c, c + cluster, ...), and all rows' orders.
struct Lists {
    int64_t* order;     // weight * total, descending, ordered as whole numbers
    float* total;
    int32_t* token;
    __device__ Lists(unsigned char* at, int rows, int n_out)
        : order(reinterpret_cast<int64_t*>(at)), total(reinterpret_cast<float*>(order + kMaxWindowRows * n_out)),
          token(reinterpret_cast<int32_t*>(total + rows * n_out)) {}
};
__host__ __device__ __forceinline__ int lists_bytes(int cluster, int n_out) {
    const int rows = (kMaxWindowRows + cluster - 1) / cluster;
    return rows * n_out * 8 + kMaxWindowRows * n_out * 8;
}

// The places of the continuations of a request's rows me, me + size, ... among all of its rows', each row's in order.
// Continuations of all rows are ordered by (order descending, row, place in the row).  For 2^l <= n_out the ceil(n_out / 2^l)-th best of
// the rows' 2^l-th continuations has n_out continuations before it or is the n_out-th.  The best of these bounds leaves at most
// n_out / 2^l rounded up that have a 2^l-th one, so at most (levels) n_out + 2^levels in all, which are counted off against each other.
// Where there is little to place, eight lanes a continuation search the other rows for it instead: 48 requests of 8 beams 34.8 us (this
// way 36.0); searched for always, 125 requests of 32 beams over 1000 values, 64 of each, took 123 us (this way 32).
struct alignas(16) Placed {
    int64_t order;
    int32_t id, pad;  // row * kMaxOut + place
};
constexpr int kLevels = 7;  // 2^6 = kMaxOut
struct PlaceBounds {
    int64_t order[kLevels];
    int32_t id[kLevels];
    int n;
    __device__ __forceinline__ void clear(int i) {
        if (i < kLevels) order[i] = INT64_MIN, id[i] = -1;
        if (i == kLevels) n = 0;
    }
};
__host__ __device__ __forceinline__ int placed_bytes(int n_out) { return (kLevels * n_out + 128) * (int)sizeof(Placed); }

__device__ __forceinline__ bool before(int64_t a, int32_t a_id, int64_t b, int32_t b_id) { return a > b || (a == b && a_id < b_id); }

// The block's threads, all of them; `at` has been cleared and all orders and counts have been written before a barrier.
__device__ __forceinline__ void place_all(const SelectParams& p, const Lists& lists, const int* counts, PlaceBounds& at, Placed* list, int first,
                                          int rows, int me, int size, int64_t to) {
    const int tid = threadIdx.x, lane = tid & 31, n_out = p.n_out, warps = (int)blockDim.x >> 5;
    auto put = [&](int r, int j, int rank) {
        const int mine = (r - me) / size * n_out + j;
        p.parents[to + rank] = first + r;
        p.tokens[to + rank] = lists.token[mine];
        p.totals[to + rank] = lists.total[mine];
    };
    if (rows == 1) {
        for (int j = tid; j < counts[0]; j += (int)blockDim.x) put(0, j, j);
        return;
    }
    const int mine_rows = (rows - me + size - 1) / size;
    if (rows <= 8 && mine_rows * n_out <= (int)blockDim.x / 4) {
        for (int c0 = 0; c0 < mine_rows * n_out; c0 += (int)blockDim.x / 8) {
            const int c = c0 + tid / 8, at = c / n_out, j = c - at * n_out, r = me + at * size, q = tid % 8;
            const bool there = c < mine_rows * n_out && j < counts[r];
            const int64_t mine = there ? lists.order[r * n_out + j] : 0;
            int lo = 0, hi = there && q < rows && q != r ? counts[q] : 0;  // how many of row q come before
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (before(lists.order[q * n_out + mid], q, mine, r))
                    lo = mid + 1;
                else
                    hi = mid;
            }
#pragma unroll
            for (int o = 1; o < 8; o *= 2) lo += __shfl_xor_sync(0xffffffffu, lo, o);
            if (q == 0 && there && j + lo < n_out) put(r, j, j + lo);
        }
        return;
    }
    for (int l = tid >> 5; l < kLevels && n_out >> l; l += warps) {
        const int j = (1 << l) - 1, place = (n_out + j) >> l;
        for (int r = lane; r < rows; r += 32) {
            if (j >= counts[r]) continue;
            const int64_t mine = lists.order[r * n_out + j];
            int rank = 0;
            for (int q = 0; q < rows; ++q) rank += j < counts[q] && before(lists.order[q * n_out + j], q, mine, r);
            if (rank == place - 1) at.order[l] = mine, at.id[l] = r * kMaxOut + j;
        }
    }
    __syncthreads();
    int64_t bound = INT64_MIN;
    int32_t bound_id = INT32_MAX;
#pragma unroll
    for (int l = 0; l < kLevels; ++l)
        if (at.id[l] >= 0 && before(at.order[l], at.id[l], bound, bound_id)) bound = at.order[l], bound_id = at.id[l];
    for (int r = tid >> 5; r < rows; r += warps)
        for (int j = lane; j < counts[r]; j += 32) {
            const int64_t o = lists.order[r * n_out + j];
            if (!before(bound, bound_id, o, r * kMaxOut + j)) list[atomicAdd(&at.n, 1)] = {o, r * kMaxOut + j, 0};
        }
    __syncthreads();
    const int n = at.n;
    for (int i = tid; i < n; i += (int)blockDim.x) {
        const Placed mine = list[i];
        const int r = mine.id / kMaxOut;
        if (r % size != me) continue;
        int rank = 0;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const Placed o = list[k];
            rank += before(o.order, o.id, mine.order, mine.id);
        }
        if (rank < n_out) put(r, mine.id % kMaxOut, rank);
    }
}
// The places that no continuation has.
__device__ __forceinline__ void fill_rest(const SelectParams& p, const int* counts, int rows, int64_t to) {
    const int tid = threadIdx.x, n_out = p.n_out;
    int n_all = 0;
    for (int r = 0; r < rows; ++r) n_all += counts[r];
    for (int k = n_all + tid; k < n_out; k += (int)blockDim.x) {
        p.parents[to + k] = p.tokens[to + k] = -1;
        p.totals[to + k] = -INFINITY;
    }
}

// A cluster of blocks: one request.  A block's first eight warps look for a row's best values, the ninth sums its exponentials.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPickThreads, 3) beam_pick_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ __align__(16) unsigned char s_lists[];
    __shared__ Search s;
    __shared__ PlaceBounds s_places;
    __shared__ double s_base;  // the row's score less its log sum exp
    __shared__ int s_found, s_counts[kMaxWindowRows];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int size = (int)cluster.num_blocks(), me = (int)cluster.block_rank(), b = (int)blockIdx.x / size;
    const int tid = threadIdx.x, n_out = p.n_out;
    const int lane = tid & 31;
    const bool sums = tid >= kSearchThreads;
    const LogTable logs(lane);  // for the summing warp
    s_places.clear(tid);
    cluster_arrive();  // (a block's shared memory is written by others once it has started)
    const Lists lists(s_lists, (kMaxWindowRows + size - 1) / size, n_out);
    const int64_t to = (int64_t)b * n_out;
    // (the scan lets this kernel start when it has waited for what came before it, so the call's own inputs may be read already)
    int first, rows;
    const bool any = rows_of(p, b, first, rows);
    float score = 0.0f, weight = 1.0f;
    int ended = -1;
    auto about = [&](int row) {
        if (p.scores) score = __ldg(p.scores + row);
        if (p.weights) weight = __ldg(p.weights + row);
        if (p.ended) ended = __ldg(p.ended + row);
    };
    if (any && me < rows) about(first + me);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!any) {
        for (int k = tid; k < n_out && me == 0; k += kPickThreads) {
            p.parents[to + k] = p.tokens[to + k] = -1;
            p.totals[to + k] = -INFINITY;
        }
        cluster_wait();
        return;
    }
    const int32_t lowest = ordered(-INFINITY);
    for (int mine = me; mine < rows; mine += size) {
        const int row = first + mine;
        const float* gm = p.group_max + (int64_t)row * p.n_groups;
        if (mine != me) about(row);
        int32_t k[kKeep];
        if (!sums) {
#pragma unroll
            for (int u = 0; u < kKeep; ++u) {
                const int g = u * kSearchThreads + tid;
                k[u] = g < p.n_groups ? ordered(__ldg(gm + g)) : lowest;
            }
        }
        if (tid == 0) s.n_groups = s.n = 0, s.bound = 0x7fffffff;
        const bool usable = fabsf(score) < INFINITY && weight > 0.0f && weight < INFINITY, live = usable && ended < 0;
        if (live && !sums) {
            const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
            int found = kListCap + 1;
            if (4 * p.n_groups < 5 * n_out) {
                gather_all<T, VEC>(s, p, x);
                found = s.n;
            } else {
                // a bound: the n_out-th best of 64, 128 or 256 shares of the groups, 5/4 n_out at least; about 1.1 n_out groups reach it
                const int lanes = n_out <= 16 && p.n_groups >= 5 * n_out ? 4 : 2 * p.n_groups >= 5 * n_out ? 2 : 1;
                int32_t m = k[0];
#pragma unroll
                for (int u = 1; u < kKeep; ++u) m = max(m, k[u]);
                for (int g = kKeep * kSearchThreads + tid; g < p.n_groups; g += kSearchThreads) m = max(m, ordered(__ldg(gm + g)));
                find_bound(s, m, lanes, n_out);
                // the groups that reach it, and their values that do; -inf is none
                const int32_t bound = max(s.bound, lowest + 1);
                auto group = [&](int32_t key, int g) {
                    if (key < bound) return;
                    const int at = atomicAdd(&s.n_groups, 1);
                    if (at < kGroupCap) s.group[at] = (uint32_t)g;
                };
#pragma unroll
                for (int u = 0; u < kKeep; ++u) group(k[u], u * kSearchThreads + tid);
                for (int g = kKeep * kSearchThreads + tid; g < p.n_groups; g += kSearchThreads) group(ordered(__ldg(gm + g)), g);
                search_sync();
                const int groups = s.n_groups;
                if (groups <= kGroupCap) {
                    constexpr int kPerGroup = kGroup<T> / 256;
                    gather<T, VEC>(s, x, from_ordered(bound), groups * kPerGroup, p.vocab,
                                   [&](int i) { return (int)s.group[i / kPerGroup] * kGroup<T> + i % kPerGroup * 256; });
                    found = s.n;
                }
            }
            if (found <= kListCap)
                rank_keys(s, found, n_out);
            else
                found = pick_slowly<T, VEC>(s, p, x, gm);
            if (tid == 0) s_found = min(found, n_out);
        } else if (live) {
            float top, e;
            unsigned long long sum;
            const bool bad = add_parts(p.parts + (int64_t)row * p.n_parts, p.n_parts, lane, top, e, sum);
            const double log2_sum = logs.log2_of(sum);
            if (lane == 0) {
                const double norm = norm_of(top, e, log2_sum);
                s_base = bad || sum == 0 ? (double)INFINITY : (double)score - norm;
            }
        }
        __syncthreads();
        int count = usable ? 1 : 0;
        double total = (double)score;
        int32_t token = ended;
        if (live) {
            count = fabs(s_base) < (double)INFINITY ? s_found : 0;
            if (tid < count) {
                total = (double)key_value(s.best[tid]) + s_base;
                token = (int32_t)key_place(s.best[tid]);
            }
        }
        if (mine == me) cluster_wait();
        if (tid < count) {
            const int at = mine / size * n_out + tid;
            lists.total[at] = (float)total;
            lists.token[at] = token;
            const int64_t order = ordered(p.weights ? total * (double)weight : total);
            for (int c = 0; c < size; ++c) cluster.map_shared_rank(lists.order, c)[mine * n_out + tid] = order;
        }
        if (tid < size) cluster.map_shared_rank(s_counts, tid)[mine] = count;
        __syncthreads();
    }
    if (me >= rows) cluster_wait();
    cluster.sync();
    if (me < rows) {  // each block places its own rows' continuations among all
        Placed* list = reinterpret_cast<Placed*>(s_lists + lists_bytes(size, n_out));
        place_all(p, lists, s_counts, s_places, list, first, rows, me, size, to);
        if (me == 0) fill_rest(p, s_counts, rows, to);
    }
}

// A block per request and a warp per row.  64-bit arithmetic is slow: behind the scan, where the rows of a block come to it at once, it is
// done for all of them together, a thread each (912 rows of 32000 24.4 us, a warp each 28.7); rows that are read as wholes do it by
// themselves (2048 rows of 8000 15.9 us, together 18.6).
//   SCANNED: after beam_scan_kernel, where there are so many rows that blocks for each would queue.
//   Else in one launch, for small vocabularies: the row is read (and a second time from L1, if it is more than the lanes hold at once).
// The bound is the n_out-th best of 32, 64 or 128 shares, which the lanes have of the groups or of the row.
// 4000 rows of 1000 bf16 values, 16 of each 250 requests: 12.1 us in one launch (68 by beam_pick_kernel); one row 3.5 (6.0).  2048 rows
// of 32000, 8 of each 256: 36 (62).  (Logits that no call has read before; of those in L2 4000 rows of 1000 take 11.5 us.)
constexpr int kRowWarps = 16;
constexpr int kRowList = 384;   // candidates of a row
template <bool SCANNED>
struct alignas(16) RowSearch {  // (read 16 bytes at a time)
    uint64_t key[kRowList];     // first the candidates' places, in its second half
    uint64_t best[kMaxOut];
    int32_t share[128];
    int n, pad[3];              // candidates
    uint32_t group[SCANNED ? kRowList : 4];
};
static_assert(sizeof(RowSearch<true>) % 16 == 0 && offsetof(RowSearch<true>, share) % 16 == 0 && offsetof(Search, top) % 16 == 0);
static_assert(kRowList >= kMaxOut + 256);
template <bool SCANNED>
struct RowBlock {
    int counts[kMaxWindowRows];
};
template <>
struct RowBlock<true> {
    unsigned long long sum[kMaxWindowRows];  // of exponentials, in units of 2^-32
    double base[kMaxWindowRows];
    float top[kMaxWindowRows], e[kMaxWindowRows], score[kMaxWindowRows], weight[kMaxWindowRows];
    int32_t ended[kMaxWindowRows];  // -2: the row is not usable
    int counts[kMaxWindowRows];
};

// The best n_out of a warp's n keys, in order.
template <typename S>
__device__ __forceinline__ void rank_row(S& s, int n, int n_out, int lane) {
    for (int i = lane; i < n; i += 32) {
        const uint64_t key = s.key[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s.key[j] > key;
        if (rank < n_out) s.best[rank] = key;
    }
    __syncwarp();
}

// A row of which more values reach `least` than the list holds (many equal ones): those above the list's worst, a full list cut back to
// its best n_out.
template <typename S, typename T>
__device__ __noinline__ int search_slowly(S& s, const T* x, int vocab, float least, int n_out, int lane) {
    int n = 0;
    uint64_t above = 0;
    auto cut = [&] {
        __syncwarp();
        rank_row(s, n, n_out, lane);
        n = min(n, n_out);
        for (int i = lane; i < n; i += 32) s.key[i] = s.best[i];
        __syncwarp();
        if (n == n_out) above = s.key[n - 1];
    };
    for (int at = 0; at < vocab; at += 256) {
        uint64_t key[8];
        int hits = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = at + e * 32 + lane;
            const float v = i < vocab ? to_float(x[i]) : -INFINITY;
            key[e] = i < vocab && v >= least ? key_of(ordered(v), (uint32_t)i) : 0;
            hits += __popc(__ballot_sync(0xffffffffu, key[e] > above));
        }
        if (!hits) continue;
        if (n + hits > kRowList) cut();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t who = __ballot_sync(0xffffffffu, key[e] > above);
            if (key[e] > above) s.key[n + __popc(who & ((1u << lane) - 1))] = key[e];
            n += __popc(who);
        }
    }
    cut();
    return n;
}

template <typename T, bool VEC, bool SCANNED>
__global__ void __launch_bounds__(32 * kRowWarps) beam_rows_kernel(const __grid_constant__ SelectParams p) {
    constexpr int kPerGroup = kGroup<T> / 256;
    using Rows = Tile<T, VEC, !VEC && (sizeof(T) == 4 || !SCANNED)>;
    extern __shared__ __align__(16) unsigned char s_lists[];
    __shared__ RowBlock<SCANNED> s_all;
    __shared__ PlaceBounds s_places;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5, b = blockIdx.x, n_out = p.n_out;
    const LogTable logs(lane);
    for (int i = tid; i <= kLevels; i += (int)blockDim.x) s_places.clear(i);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Lists lists(s_lists, kMaxWindowRows, n_out);
    unsigned char* behind = s_lists + lists_bytes(1, n_out);
    RowSearch<SCANNED>& s = reinterpret_cast<RowSearch<SCANNED>*>(behind + placed_bytes(n_out))[warp];
    int first, rows;
    if (!rows_of(p, b, first, rows)) rows = 0;
    const int32_t lowest = ordered(-INFINITY);
    // one continuation: of a row at its end itself, else by its key
    auto list = [&](int at, uint64_t key, int ended, double base, float weight) {
        const double total = ended >= 0 ? base : (double)key_value(key) + base;
        lists.order[at] = ordered(p.weights ? total * (double)weight : total);
        lists.total[at] = (float)total;
        lists.token[at] = ended >= 0 ? ended : (int32_t)key_place(key);
    };
    for (int mine = warp; mine < rows; mine += warps) {
        const int row = first + mine;
        const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
        Eight<T> v8[kLoads];
        auto load = [&](int chunk, int vocab) {
            int at[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) at[u] = chunk * kChunk + u * 256;
            Rows::load(v8, x, at, vocab, lane);
        };
        const float score = p.scores ? __ldg(p.scores + row) : 0.0f, weight = p.weights ? __ldg(p.weights + row) : 1.0f;
        int ended = p.ended ? max(__ldg(p.ended + row), -1) : -1;  // any value below zero: the row goes on
        if (!SCANNED) load(0, ended < 0 ? p.vocab : 0);  // of a row at its end no value (a branch instead: 97 registers, 12.0 -> 16.8 us)
        if (!(fabsf(score) < INFINITY && weight > 0.0f && weight < INFINITY)) ended = -2;
        float top = 0.0f, e = 0.0f;
        unsigned long long sum = 0;
        int count = ended >= 0;
        double base = (double)score;
        if (ended == -1) {
            const float* gm = p.group_max + (int64_t)row * p.n_groups;
            int32_t most[4] = {lowest, lowest, lowest, lowest};
            bool bad;
            if (SCANNED) {
                for (int g0 = lane; g0 < p.n_groups; g0 += 128)
#pragma unroll
                    for (int u = 0; u < 4; ++u) most[u] = max(most[u], g0 + u * 32 < p.n_groups ? ordered(__ldg(gm + g0 + u * 32)) : lowest);
                bad = add_parts(p.parts + (int64_t)row * p.n_parts, p.n_parts, lane, top, e, sum);
            } else {
                Part part = {-INFINITY, -INFINITY, 0.0f};
                for (int chunk = 0;;) {
                    float m = -INFINITY;
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        const float l = largest(v8[u]);
                        most[u] = max(most[u], ordered(l));
                        m = fmaxf(m, l);
                    }
                    add_to(part, v8, fmaxf(warp_max(m), part.m));
                    if (++chunk == p.n_chunks) break;
                    load(chunk, p.vocab);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) part.s += __shfl_xor_sync(0xffffffffu, part.s, o);
                top = part.m, e = part.e;
                bad = !(part.s < INFINITY);
                sum = bad ? 0 : __float2ull_rn(part.s * 0x1p32f);  // exact: part.s is 0, or about 0.7 at least
            }
            if (!SCANNED) base -= norm_of(top, e, logs.log2_of(sum));
            int32_t reach = 0x7fffffff;
            auto rank = [&](auto n) {  // n shares a lane
                __syncwarp();
                if (lane == 0) s.n = 0;
#pragma unroll
                for (int u = 0; u < n.value; ++u) s.share[u * 32 + lane] = most[u];
                __syncwarp();
                int better[n.value] = {};
#pragma unroll
                for (int j = 0; j < 8 * n.value; ++j) {
                    const int4 o = reinterpret_cast<const int4*>(s.share)[j];
#pragma unroll
                    for (int u = 0; u < n.value; ++u) better[u] += (o.x > most[u]) + (o.y > most[u]) + (o.z > most[u]) + (o.w > most[u]);
                }
#pragma unroll
                for (int u = 0; u < n.value; ++u)
                    if (better[u] < n_out) reach = min(reach, most[u]);
            };
            if (n_out > 32) {
                rank(std::integral_constant<int, 4>{});
            } else {
                most[0] = max(most[0], most[2]), most[1] = max(most[1], most[3]);
                if (n_out > 16) {
                    rank(std::integral_constant<int, 2>{});
                } else {
                    most[0] = max(most[0], most[1]);
                    rank(std::integral_constant<int, 1>{});
                }
            }
            const int32_t bound = max(__reduce_min_sync(0xffffffffu, reach), lowest + 1);
            const float least = from_ordered(bound);
            uint32_t* groups = s.group;
            uint32_t* places = reinterpret_cast<uint32_t*>(s.key) + kRowList;
            int tiles = p.n_chunks * kLoads;
            if (SCANNED) {
                int n = 0;
                for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
                    const bool hit = g0 + lane < p.n_groups && ordered(__ldg(gm + g0 + lane)) >= bound;
                    const uint32_t who = __ballot_sync(0xffffffffu, hit);
                    const int at = n + __popc(who & ((1u << lane) - 1));
                    if (hit && at < kRowList) groups[at] = (uint32_t)(g0 + lane);
                    n += __popc(who);
                }
                __syncwarp();
                tiles = n <= kRowList ? n * kPerGroup : 0;
                if (n > kRowList && lane == 0) s.n = n;
            }
            for (int t = 0; t < tiles; t += kLoads) {
                int at[kLoads];
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = t + u;
                    if (SCANNED)
                        at[u] = i < tiles ? (int)groups[i / kPerGroup] * kGroup<T> + i % kPerGroup * 256 : p.vocab;
                    else
                        at[u] = i * 256;
                }
                if (SCANNED || p.n_chunks > 1) Rows::load(v8, x, at, p.vocab, lane);
                uint32_t hit = 0;
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    if (!(largest(v8[u]) >= least)) continue;
                    float v[8];
                    v8[u].floats(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) hit |= (v[i] >= least ? 1u : 0u) << (u * 8 + i);
                }
                if (hit == 0) continue;
                for (int place = atomicAdd(&s.n, __popc(hit)); hit; hit &= hit - 1, ++place) {
                    const int i = __ffs(hit) - 1;
                    int from = at[0];
#pragma unroll
                    for (int u = 1; u < kLoads; ++u) from = i >= u * 8 ? at[u] : from;
                    if (place < kRowList) places[place] = (uint32_t)Rows::place(from, lane, i & 7);
                }
            }
            __syncwarp();
            const int n = s.n;
            if (n <= kRowList) {
                // (the keys of 32 reach no further into the places than those that have been read)
                for (int i0 = 0; i0 < n; i0 += 32) {
                    const int i = i0 + lane;
                    const uint32_t place = i < n ? places[i] : 0u;
                    __syncwarp();
                    if (i < n) s.key[i] = key_of(ordered(to_float(x[place])), place);
                    __syncwarp();
                }
                rank_row(s, n, n_out, lane);
                count = min(n, n_out);
            } else {
                count = search_slowly(s, x, p.vocab, least, n_out, lane);
            }
            if (bad || sum == 0) count = 0;
        }
        for (int k = lane; k < count; k += 32) {
            if (SCANNED)
                lists.order[mine * n_out + k] = (int64_t)s.best[k];
            else
                list(mine * n_out + k, s.best[k], ended, base, weight);
        }
        if (lane == 0) {
            s_all.counts[mine] = count;
            if constexpr (SCANNED) {
                s_all.sum[mine] = sum;
                s_all.top[mine] = top;
                s_all.e[mine] = e;
                s_all.score[mine] = score;
                s_all.weight[mine] = weight;
                s_all.ended[mine] = ended;
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if constexpr (SCANNED) {
        for (int r0 = warp * 32; r0 < rows; r0 += warps * 32) {
            const int r = min(r0 + lane, rows - 1);
            const double log2_sum = logs.log2_of(s_all.sum[r]);
            const double base = (double)s_all.score[r] - (s_all.ended[r] == -1 ? norm_of(s_all.top[r], s_all.e[r], log2_sum) : 0.0);
            if (r0 + lane < rows) s_all.base[r] = base;
        }
        __syncthreads();
        for (int c = tid; c < rows * n_out; c += (int)blockDim.x) {
            const int r = c / n_out;
            if (c - r * n_out < s_all.counts[r]) list(c, (uint64_t)lists.order[c], s_all.ended[r], s_all.base[r], s_all.weight[r]);
        }
        __syncthreads();
    }
    const int64_t to = (int64_t)b * n_out;
    if (rows) place_all(p, lists, s_all.counts, s_places, reinterpret_cast<Placed*>(behind), first, rows, 0, 1, to);
    fill_rest(p, s_all.counts, rows, to);
}

// What the sizes give: chunks, groups and parts of a row.  A warp takes two chunks of 16-bit values where there are many (320 rows of
// 248320: the call 33.4 us, 34.8 with one, 33.2 with four; 96 rows 16.5 and 16.8), else one (160 rows of fp32: 29.9 us, 30.2 with two).
void plan(SelectParams& p, size_t value_bytes) {
    p.n_chunks = (p.vocab + kChunk - 1) / kChunk;
    p.n_groups = p.n_chunks * (int)value_bytes;
    const int64_t all = (int64_t)p.n_chunks * p.n_rows;
    p.turns = value_bytes == 2 && all >= 3 * kManyChunks ? 2 : 1;
    p.n_parts = (p.n_chunks + kScanWarps * p.turns - 1) / (kScanWarps * p.turns) * kScanWarps;
}

// The workspace's arrays, in order of their alignment; the size where base is null.
size_t carve(SelectParams& p, unsigned char* base) {
    size_t at = 0;
    auto take = [&](auto*& ptr, size_t n) {
        ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(base + at);
        at += (n * sizeof(*ptr) + 15) / 16 * 16;
    };
    const size_t rows = (size_t)p.n_rows;
    take(p.group_max, rows * p.n_groups);
    take(p.parts, rows * p.n_parts);
    return at;
}

bool select_shape(int n_rows, int vocab, int n_seqs, int n_out) {
    return n_rows <= 65535 && vocab <= (1 << 30) && n_seqs <= kMaxSeqs && n_out <= kMaxOut;
}

// A warp per row (beam_rows_kernel) or a block per row (beam_pick_kernel)?  bf16, beams of 8 (of 4 where there is one request), n_out 8
// (4), us, twenty calls in a graph, each on logits that have left L2; a row read as a whole / a warp per row after the scan / a block per
// row after it:
//   rows    vocab 1000         vocab 4096         vocab 8000         vocab 32000        vocab 106304
//   4       4.1 / 25 / 6.4     6.3 / 7.4 / 7.7    9.7 / 7.3 / 6.9    28 / 8.0 / 6.9     - / 8.8 / 7.0
//   304     5.7 / 37 / 8.0     8.8 / 15 / 8.8     14.5 / 15 / 13.2   42 / 17 / 12.2     - / 26 / 18.9
//   608     5.8 / 33 / 14.0    9.5 / 16 / 16.0    14.9 / 16 / 22.4   42 / 21.1 / 21.8   - / 36.7 / 34.6
//   912     5.8 / 36 / 19.9    10.0 / 17 / 22.7   15.1 / 17 / 28.7   42 / 24.4 / 31.0   - / 46.4 / 50.3
//   2048    7.2 / 46 / 39.6    12.0 / 20 / 43.5   17.3 / 21 / 54.1   62 / 36.0 / 61.7   - / 80.7 / 103.7
// Of 32 continuations 1024 rows, 16 of each request, 16.3 / - / 35 at 4096, 53 / 38.5 / 57.7 at 32000, - / 69.8 / 74.7 at 106304.
// The rule goes by the rows alone, and there are sizes where it takes the slower side.  With a warp per row a request has one block, so
// few requests of many beams leave multiprocessors idle; of 32 continuations: 24 requests of 32 beams 39 / - / 34.7 at 8000, 100 / 53.8 /
// 55.9 at 32000, - / 90.7 / 63.2 at 106304; 12 of 64 77 / - / 42.2, 200 / 94 / 61.7, - / 151 / 69.8; 5 of 64 72.6 / - / 40.3 at 8000.  And
// of 64 continuations, which always go to a block per row above kSmallVocab, 64 requests of 32 beams took 41.4 / - / 72.9 at 4096 and
// - / 179 / 185 at 106304; 4 rows of 4096 values 6.3 as wholes and 7.7 as the rule has it.
constexpr int kSmallVocab = 2048;    // rows of no more are read as a whole,
constexpr int kMediumVocab = 10240;  // and of no more where there are more than kSomeRows of them
constexpr int kSomeRows = 152 * 2, kManyRows = 152 * 5;
constexpr int kFewOut = 32;
template <typename T, bool VEC>
int launch_select(const SelectParams& p, cudaStream_t s) {
    auto rows_kernel = [&](auto kernel, SmemOptIn& opt, int row_bytes) {
        int warps = 1;  // a row each, by the mean of the requests' rows
        while (warps < kRowWarps && (int64_t)warps * p.n_seqs < p.n_rows) warps *= 2;
        const int opted = opt.ensure(kernel, lists_bytes(1, kMaxOut) + placed_bytes(kMaxOut) + kRowWarps * row_bytes);
        if (opted != KVQ8_OK) return opted;
        return launch_dependent(kernel, (unsigned)p.n_seqs, 32u * (unsigned)warps,
                                lists_bytes(1, p.n_out) + placed_bytes(p.n_out) + warps * row_bytes, s, p);
    };
    const bool few_out = p.n_out <= kFewOut, few_groups = 4 * p.n_groups < 5 * p.n_out;
    if (p.vocab <= kSmallVocab || (few_out && (p.vocab <= kMediumVocab ? p.n_rows > kSomeRows : p.n_rows > kManyRows && few_groups))) {
        static SmemOptIn opt;
        return rows_kernel(beam_rows_kernel<T, VEC, false>, opt, (int)sizeof(RowSearch<false>));
    }
    const dim3 grid((unsigned)(p.n_parts / kScanWarps), (unsigned)p.n_rows);
    const int rc = launch_dependent(beam_scan_kernel<T, VEC>, grid, kScanThreads, 0, s, p);
    if (rc != KVQ8_OK) return rc;
    if (p.n_rows > kManyRows && few_out) {
        static SmemOptIn opt;
        return rows_kernel(beam_rows_kernel<T, VEC, true>, opt, (int)sizeof(RowSearch<true>));
    }
    // A block a row, by the mean of the requests' rows.  Clusters of 16 where the GPU holds all of them at once: 12 requests of 32 beams, 64
    // of each, over 106304 bf16 logits 48.6 us (of 8: 72.6), 19 of 16 beams, 16 of each, 22.4 (26.7); 24 of 16 beams, 16 of each, 32.9 us (of
    // 8: 28.9).
    int cluster = 1;
    while (cluster < 8 && (int64_t)cluster * p.n_seqs < p.n_rows) cluster *= 2;
    if ((int64_t)p.n_seqs * 8 < p.n_rows && p.n_seqs * 16 <= kSomeRows) cluster = 16;
    static SmemOptIn opt;
    const int opted = opt.ensure(beam_pick_kernel<T, VEC>, lists_bytes(1, kMaxOut) + placed_bytes(kMaxOut), true);
    if (opted != KVQ8_OK) return opted;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_seqs * cluster));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = (size_t)(lists_bytes(cluster, p.n_out) + placed_bytes(p.n_out));
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, beam_pick_kernel<T, VEC>, p));
}

}  // namespace
}  // namespace kvq8

extern "C" size_t beam_select_workspace_bytes(int n_rows, int vocab, int n_seqs, int n_out) {
    using namespace kvq8;
    if (n_rows < 1 || vocab < 1 || n_seqs < 1 || n_out < 1 || !select_shape(n_rows, vocab, n_seqs, n_out)) return 0;
    SelectParams p = {};
    p.n_rows = n_rows, p.vocab = vocab, p.n_seqs = n_seqs, p.n_out = n_out;
    plan(p, 4);  // the groups of fp32 are the most
    return carve(p, nullptr);
}

extern "C" int beam_select(const void* logits, int dtype, int64_t logits_stride, int n_rows, int vocab, const int32_t* row_starts,
                           int n_seqs, const float* scores, const float* weights, const int32_t* ended, int n_out,
                           int32_t* parents, int32_t* tokens, float* totals, void* workspace, size_t workspace_bytes,
                           kvq8_stream_t stream) {
    using namespace kvq8;
    const size_t esz = dtype_size(dtype);
    if (!esz || n_rows < 0 || n_seqs < 0 || vocab < 1 || n_out < 1) return KVQ8_ERR_INVALID_ARG;
    if (n_seqs == 0) return KVQ8_OK;
    if (n_rows == 0) return KVQ8_ERR_INVALID_ARG;
    if (!logits || !row_starts || !parents || !tokens || !totals || logits_stride < vocab) return KVQ8_ERR_INVALID_ARG;
    if (!select_shape(n_rows, vocab, n_seqs, n_out)) return KVQ8_ERR_UNSUPPORTED;
    const size_t need = beam_select_workspace_bytes(n_rows, vocab, n_seqs, n_out);
    if (!workspace || workspace_bytes < need) return KVQ8_ERR_WORKSPACE;
    if (!aligned_to(logits, esz) || !aligned16(workspace)) return KVQ8_ERR_MISALIGNED;
    for (const void* q : {(const void*)row_starts, (const void*)scores, (const void*)weights, (const void*)ended,
                          (const void*)parents, (const void*)tokens, (const void*)totals})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    // (a request's outputs are written while others' inputs are still read)
    const size_t bytes = (size_t)n_seqs * n_out * 4, rows = (size_t)n_rows * 4;
    const void* const outs[] = {parents, tokens, totals};
    for (int i = 0; i < 3; ++i) {
        if (ranges_meet(outs[i], bytes, row_starts, ((size_t)n_seqs + 1) * 4) || ranges_meet(outs[i], bytes, scores, rows) ||
            ranges_meet(outs[i], bytes, weights, rows) || ranges_meet(outs[i], bytes, ended, rows) || ranges_meet(outs[i], bytes, workspace, need) ||
            range_meets_rows(outs[i], bytes, logits, (int64_t)(vocab * esz), logits_stride * (int64_t)esz, n_rows))
            return KVQ8_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (ranges_meet(outs[i], bytes, outs[j], bytes)) return KVQ8_ERR_INVALID_ARG;
    }
    SelectParams p = {};
    p.logits = logits, p.stride = logits_stride, p.row_starts = row_starts, p.scores = scores, p.weights = weights;
    p.ended = ended, p.parents = parents, p.tokens = tokens, p.totals = totals;
    p.n_rows = n_rows, p.vocab = vocab, p.n_seqs = n_seqs, p.n_out = n_out;
    plan(p, esz);
    carve(p, static_cast<unsigned char*>(workspace));
    // eight values a load where every row starts on their size and holds whole groups of eight
    const bool vec = vocab % 8 == 0 && logits_stride % 8 == 0 && aligned_to(logits, 8 * esz);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return vec ? launch_select<float, true>(p, s) : launch_select<float, false>(p, s);
    if (dtype == KVQ8_F16) return vec ? launch_select<__half, true>(p, s) : launch_select<__half, false>(p, s);
    return vec ? launch_select<__nv_bfloat16, true>(p, s) : launch_select<__nv_bfloat16, false>(p, s);
}

// beam_select.cu -- beam search's choice: of every request's beams and the whole vocabulary the n_out best continuations.
//
// Row r (a beam) with score c continues with value v at  total = c + x[v] - log sum_v exp x[v],  ordered by weight * total.
// The n_out best of a request lie among the n_out best of each of its rows, which are the n_out best logits x.
//
// One pass over the logits.  A warp holds four groups of 256 consecutive values in registers and leaves behind each group's
// maximum and one partial sum of exponentials: 1/100 of what it read.  Ordered by (maximum descending, place ascending), the
// n_out best groups hold the row's n_out best values: a value outside them has n_out values before it, one in each.  So the
// second kernel, a block per row, picks those groups, reads them again, picks the values, and the last block of a request to
// finish joins its rows' lists.
// Bound: the logits' bytes in the first kernel; latency in the second.
#include <float.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kScanThreads = 256;
constexpr int kGroup = 256;        // values of a group: eight a lane
// Groups that a warp holds at once: 128 bytes of fp32, as many values twice of the others.
template <typename T>
constexpr int kWarpGroups = sizeof(T) == 4 ? 4 : 8;
constexpr int kPadGroups = 8;      // a row's groups are counted in these
constexpr int kSearchThreads = 256;
constexpr int kPickThreads = kSearchThreads + 32;
constexpr int kMaxOut = 64;
constexpr int kKeep = 4;           // groups of a row that a searching thread keeps
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
    int32_t* group_max;     // [n_rows][n_groups], ordered as whole numbers
    Part* parts;            // [n_rows][n_parts]
    int64_t* list_order;    // [n_rows][n_out] weight * total, descending, ordered as whole numbers
    float* list_total;
    int32_t* list_token;
    int32_t* list_count;    // [n_rows]
    int32_t* seq_of;        // [n_rows]
    uint32_t* done;         // [n_seqs] rows finished
    int n_rows, vocab, n_seqs, n_out, n_groups, n_parts;
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

// Eight values of a group, -inf behind the row's end.
template <typename T, bool VEC>
__device__ __forceinline__ void load_eight(Eight<T>& x, const T* row, int at, int vocab) {
    if (VEC) {
        if (at < vocab) {
            x.load_whole(row + at);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.put(i, T(-INFINITY));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.put(i, at + i < vocab ? row[at + i] : T(-INFINITY));
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ SelectParams p) {
    const int lane = threadIdx.x & 31, row = blockIdx.y;
    const int part = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && row == 0) {  // the request of every row; what the second kernel counts; requests without rows
        for (int b = threadIdx.x; b < p.n_seqs; b += kScanThreads) {
            int first, rows;
            p.done[b] = 0u;
            if (rows_of(p, b, first, rows)) {
                for (int r = 0; r < rows; ++r) p.seq_of[first + r] = b;
            } else {
                for (int k = 0; k < p.n_out; ++k) {
                    const int64_t o = (int64_t)b * p.n_out + k;
                    p.parents[o] = p.tokens[o] = -1;
                    p.totals[o] = -INFINITY;
                }
            }
        }
    }
    if (part >= p.n_parts || (p.ended && __ldg(p.ended + row) >= 0)) return;
    const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
    constexpr int G = kWarpGroups<T>;
    Eight<T> raw[G];
#pragma unroll
    for (int u = 0; u < G; ++u) load_eight<T, VEC>(raw[u], x, (part * G + u) * kGroup + lane * 8, p.vocab);
    int32_t top[G], most = ordered(-INFINITY);
#pragma unroll
    for (int u = 0; u < G; ++u) {
        float v[8];
        raw[u].floats(v);
        float m = fmaxf(v[0], v[1]);
#pragma unroll
        for (int i = 2; i < 8; ++i) m = fmaxf(m, v[i]);
        if (!(m > -INFINITY)) m = -INFINITY;
        top[u] = __reduce_max_sync(0xffffffffu, ordered(m));
        most = max(most, top[u]);
    }
    const float m = from_ordered(most);
    // 2^(x log2 e - e) with e a rounded multiple near the maximum: one rounding a value, and parts join by powers of two
    const float e = rintf(m * kLog2e);
    const bool plain = fabsf(m) < kLarge, any = fabsf(m) < INFINITY;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < G; ++u) {
        float v[8];
        raw[u].floats(v);
        if (plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s += ex2_approx(__fmaf_rn(v[i], kLog2e, -e));
        } else {  // of -inf alone nothing; a NaN or +inf makes the sum NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) s += any ? ex2_approx((v[i] - m) * kLog2e) : v[i] == -INFINITY ? 0.0f : NAN;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
        p.parts[(int64_t)row * p.n_parts + part] = Part{m, e, s};
        int4* to = reinterpret_cast<int4*>(p.group_max + (int64_t)row * p.n_groups + part * G);
#pragma unroll
        for (int u = 0; u < G; u += 4) to[u / 4] = make_int4(top[u], top[u + 1], top[u + 2], top[u + 3]);
    }
}

// The threads that search (the others of the block sum).
__device__ __forceinline__ void search_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct Search {
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

// Where more groups or values reach the bound than the lists hold (many equal values): the row's groups, and then the best ones'
// values, a key a thread at a time; a full list is cut back to its best n_out, below which nothing is taken any more.
template <typename T, bool VEC>
__device__ __noinline__ int pick_slowly(Search& s, const SelectParams& p, const T* x, const int32_t* gm) {
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
        if (s.n + kSearchThreads > kListCap) cut();
        if (k > s.above) s.key[atomicAdd(&s.n, 1)] = k;
        search_sync();
    };
    search_sync();
    if (tid == 0) s.n = 0, s.above = 0;
    search_sync();
#pragma unroll 1
    for (int g0 = 0; g0 < p.n_groups; g0 += kSearchThreads) add(g0 + tid < p.n_groups ? key_of(gm[g0 + tid], (uint32_t)(g0 + tid)) : 0);
    cut();
    const int groups = s.n;
    if (tid < groups) s.group[tid] = key_place(s.key[tid]);
    search_sync();
    if (tid == 0) s.n = 0, s.above = 0;
    search_sync();
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
        const int at = (int)s.group[g] * kGroup + tid;
        const float v = at < p.vocab ? to_float(x[at]) : -INFINITY;
        add(v > -INFINITY ? key_of(ordered(v), (uint32_t)at) : 0);
    }
    cut();
    return s.n;
}

// Block: one row.  Its first eight warps look for the row's best values, the ninth sums its exponentials.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPickThreads, 4) beam_pick_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ __align__(16) unsigned char s_join[];  // the join: the rows' orders
    __shared__ Search s;
    __shared__ double s_norm;
    __shared__ int s_last, s_found, s_count[kMaxWindowRows];
    const int tid = threadIdx.x, row = blockIdx.x, n_out = p.n_out;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t* gm = p.group_max + (int64_t)row * p.n_groups;
    const int b = __ldg(p.seq_of + row);
    const float score = p.scores ? __ldg(p.scores + row) : 0.0f, weight = p.weights ? __ldg(p.weights + row) : 1.0f;
    const int ended = p.ended ? __ldg(p.ended + row) : -1;
    int32_t k[kKeep];
    const int32_t lowest = ordered(-INFINITY);
    if (tid < kSearchThreads) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
            const int g = u * kSearchThreads + tid;
            k[u] = g < p.n_groups && ended < 0 ? __ldg(gm + g) : lowest;
        }
    }
    if (tid == 0) s.n_groups = s.n = 0, s.bound = 0x7fffffff;
    int first, rows;
    if (b < 0 || b >= p.n_seqs || !rows_of(p, b, first, rows) || row < first || row >= first + rows) return;
    const bool usable = fabsf(score) < INFINITY && weight > 0.0f && weight < INFINITY, live = usable && ended < 0;
    if (live && tid < kSearchThreads) {
        // a bound: the n_out-th best of the threads' best groups
        int32_t m = k[0];
#pragma unroll
        for (int u = 1; u < kKeep; ++u) m = max(m, k[u]);
        for (int g = kKeep * kSearchThreads + tid; g < p.n_groups; g += kSearchThreads) m = max(m, __ldg(gm + g));
        s.top[tid] = m;
        search_sync();
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < kSearchThreads / 4; ++j) {
            const int4 o = reinterpret_cast<const int4*>(s.top)[j];
            rank += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
        }
        if (rank < n_out) atomicMin(&s.bound, m);
        search_sync();
        // the groups that reach it, and their values that do; -inf is none
        const int32_t bound = max(s.bound, lowest + 1);
        auto group = [&](int32_t key, int g) {
            if (key < bound) return;
            const int at = atomicAdd(&s.n_groups, 1);
            if (at < kGroupCap) s.group[at] = (uint32_t)g;
        };
#pragma unroll
        for (int u = 0; u < kKeep; ++u) group(k[u], u * kSearchThreads + tid);
        for (int g = kKeep * kSearchThreads + tid; g < p.n_groups; g += kSearchThreads) group(__ldg(gm + g), g);
        search_sync();
        const int groups = s.n_groups;
        const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
        int found = groups <= kGroupCap ? 0 : kListCap + 1;
        if (!found) {
#pragma unroll 2
            for (int i = tid >> 5; i < groups; i += kSearchThreads / 32) {
                const int at = (int)s.group[i] * kGroup + (tid & 31) * 8;
                Eight<T> raw;
                load_eight<T, VEC>(raw, x, at, p.vocab);
                float v[8];
                raw.floats(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int32_t o = ordered(v[e]);
                    if (o < bound || v[e] != v[e]) continue;
                    const int to = atomicAdd(&s.n, 1);
                    if (to < kListCap) s.key[to] = key_of(o, (uint32_t)(at + e));
                }
            }
            search_sync();
            found = s.n;
        }
        if (found <= kListCap)
            rank_keys(s, found, n_out);
        else
            found = pick_slowly<T, VEC>(s, p, x, gm);
        if (tid == 0) s_found = min(found, n_out);
    } else if (live) {
        // parts scaled by powers of two to the largest one's, added as whole numbers of 2^-32, so that their order does not matter
        const int lane = tid & 31;
        const Part* parts = p.parts + (int64_t)row * p.n_parts;
        int32_t m = lowest;
        bool bad = false;
        for (int i = lane; i < p.n_parts; i += 32) {
            const Part q = parts[i];
            m = max(m, ordered(q.m));
            bad |= q.s != q.s;
        }
        const float top = from_ordered(__reduce_max_sync(0xffffffffu, m));
        bad = __any_sync(0xffffffffu, bad);
        const float e = rintf(top * kLog2e);
        const bool plain = fabsf(top) < kLarge;
        unsigned long long sum = 0;
        for (int i = lane; i < p.n_parts; i += 32) {
            const Part q = parts[i];
            float v = 0.0f;
            if (plain && fabsf(q.m) < kLarge)
                v = q.e - e > -126.0f ? q.s * __int_as_float((127 + (int)(q.e - e)) << 23) : 0.0f;
            else if (q.m > -INFINITY)
                v = q.s * exp2f((float)(scale_of_part(q.m, q.e) - scale_of_part(top, e)));
            sum += __float2ull_rn(v * 0x1p32f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            const double total = (double)sum * 0x1p-32;
            const double norm = plain ? ((double)e + log2(total)) * (1.0 / (double)kLog2e) : (double)top + log(total);
            s_norm = bad ? (double)INFINITY : norm;
        }
    }
    __syncthreads();
    const int64_t out0 = (int64_t)row * n_out;
    int count = usable ? 1 : 0;
    double total = (double)score;
    int32_t token = ended;
    if (live) {
        count = fabs(s_norm) < (double)INFINITY ? s_found : 0;
        if (tid < count) {
            total += (double)key_value(s.best[tid]) - s_norm;
            token = (int32_t)key_place(s.best[tid]);
        }
    }
    if (tid < count) {
        p.list_order[out0 + tid] = ordered(total * (double)weight);
        p.list_total[out0 + tid] = (float)total;
        p.list_token[out0 + tid] = token;
    }
    // the last row of a request to be done joins its rows' lists
    if (tid == 0) p.list_count[row] = count;
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(p.done + b, 1u) == (uint32_t)(rows - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    int64_t* order = reinterpret_cast<int64_t*>(s_join);
    if (tid < rows) s_count[tid] = __ldcg(p.list_count + first + tid);
    for (int i = tid; i < rows * n_out; i += kPickThreads) order[i] = __ldcg(p.list_order + (int64_t)first * n_out + i);
    __syncthreads();
    int n_all = 0;
    for (int r = 0; r < rows; ++r) n_all += s_count[r];
    const int64_t to = (int64_t)b * n_out;
    for (int i = tid; i < rows * n_out; i += kPickThreads) {
        const int r = i / n_out, j = i - r * n_out;
        if (j >= s_count[r]) continue;
        const int64_t mine = order[i];
        int rank = j;
        for (int q = 0; q < rows && rank < n_out; ++q) {
            if (q == r) continue;
            const int64_t* o = order + q * n_out;
            int lo = 0, hi = s_count[q];  // how many of row q come before: more, or as much and of a lower row
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (o[mid] > mine || (o[mid] == mine && q < r))
                    lo = mid + 1;
                else
                    hi = mid;
            }
            rank += lo;
        }
        if (rank < n_out) {
            p.parents[to + rank] = first + r;
            p.tokens[to + rank] = __ldcg(p.list_token + (int64_t)first * n_out + i);
            p.totals[to + rank] = __ldcg(p.list_total + (int64_t)first * n_out + i);
        }
    }
    for (int k = n_all + tid; k < n_out; k += kPickThreads) {
        p.parents[to + k] = p.tokens[to + k] = -1;
        p.totals[to + k] = -INFINITY;
    }
}

int groups_of(int vocab) { return (vocab + kGroup * kPadGroups - 1) / (kGroup * kPadGroups) * kPadGroups; }

// The workspace's arrays, in order of their alignment; the size where base is null.
size_t carve(SelectParams& p, unsigned char* base) {
    size_t at = 0;
    auto take = [&](auto*& ptr, size_t n) {
        ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(base + at);
        at += (n * sizeof(*ptr) + 15) / 16 * 16;
    };
    const size_t rows = (size_t)p.n_rows;
    take(p.group_max, rows * p.n_groups);
    take(p.list_order, rows * p.n_out);
    take(p.parts, rows * p.n_parts);
    take(p.list_total, rows * p.n_out);
    take(p.list_token, rows * p.n_out);
    take(p.list_count, rows);
    take(p.seq_of, rows);
    take(p.done, (size_t)p.n_seqs);
    return at;
}

bool select_shape(int n_rows, int vocab, int n_seqs, int n_out) {
    return n_rows <= 65535 && vocab <= (1 << 30) && n_seqs <= kMaxSeqs && n_out <= kMaxOut;
}

template <typename T, bool VEC>
int launch_select(const SelectParams& p, cudaStream_t s) {
    const int warps = kScanThreads / 32;
    const dim3 grid((unsigned)((p.n_parts + warps - 1) / warps), (unsigned)p.n_rows);
    const int rc = launch_dependent(beam_scan_kernel<T, VEC>, grid, kScanThreads, 0, s, p);
    if (rc != KVQ8_OK) return rc;
    return launch_dependent(beam_pick_kernel<T, VEC>, (unsigned)p.n_rows, kPickThreads, kMaxWindowRows * p.n_out * (int)sizeof(int64_t), s, p);
}

}  // namespace
}  // namespace kvq8

extern "C" size_t beam_select_workspace_bytes(int n_rows, int vocab, int n_seqs, int n_out) {
    using namespace kvq8;
    if (n_rows < 1 || vocab < 1 || n_seqs < 1 || n_out < 1 || !select_shape(n_rows, vocab, n_seqs, n_out)) return 0;
    SelectParams p = {};
    p.n_rows = n_rows, p.vocab = vocab, p.n_seqs = n_seqs, p.n_out = n_out;
    p.n_groups = groups_of(vocab);
    p.n_parts = p.n_groups / kWarpGroups<float>;  // fp32 has the most
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
    if (!workspace || workspace_bytes < beam_select_workspace_bytes(n_rows, vocab, n_seqs, n_out)) return KVQ8_ERR_WORKSPACE;
    if (!aligned_to(logits, esz) || !aligned16(workspace)) return KVQ8_ERR_MISALIGNED;
    for (const void* q : {(const void*)row_starts, (const void*)scores, (const void*)weights, (const void*)ended,
                          (const void*)parents, (const void*)tokens, (const void*)totals})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    SelectParams p = {};
    p.logits = logits, p.stride = logits_stride, p.row_starts = row_starts, p.scores = scores, p.weights = weights;
    p.ended = ended, p.parents = parents, p.tokens = tokens, p.totals = totals;
    p.n_rows = n_rows, p.vocab = vocab, p.n_seqs = n_seqs, p.n_out = n_out;
    p.n_groups = groups_of(vocab);
    p.n_parts = p.n_groups / (dtype == KVQ8_F32 ? kWarpGroups<float> : kWarpGroups<__half>);
    carve(p, static_cast<unsigned char*>(workspace));
    // eight values a load where every row starts on their size and holds whole groups of eight
    const bool vec = vocab % 8 == 0 && logits_stride % 8 == 0 && aligned_to(logits, 8 * esz);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return vec ? launch_select<float, true>(p, s) : launch_select<float, false>(p, s);
    if (dtype == KVQ8_F16) return vec ? launch_select<__half, true>(p, s) : launch_select<__half, false>(p, s);
    return vec ? launch_select<__nv_bfloat16, true>(p, s) : launch_select<__nv_bfloat16, false>(p, s);
}

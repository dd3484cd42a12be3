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
constexpr int kWarpGroups = 4;     // groups that a warp holds at once
constexpr int kPickThreads = 256;
constexpr int kMaxOut = 64;
constexpr int kListCap = 1024;     // candidates that the second kernel keeps

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
    double* list_order;     // [n_rows][n_out] weight * total, descending
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
    Eight<T> raw[kWarpGroups];
#pragma unroll
    for (int u = 0; u < kWarpGroups; ++u) load_eight<T, VEC>(raw[u], x, (part * kWarpGroups + u) * kGroup + lane * 8, p.vocab);
    int32_t top[kWarpGroups];
#pragma unroll
    for (int u = 0; u < kWarpGroups; ++u) {
        float v[8];
        raw[u].floats(v);
        float m = fmaxf(v[0], v[1]);
#pragma unroll
        for (int i = 2; i < 8; ++i) m = fmaxf(m, v[i]);
        if (!(m > -INFINITY)) m = -INFINITY;
        top[u] = __reduce_max_sync(0xffffffffu, ordered(m));
    }
    const float m = from_ordered(max(max(top[0], top[1]), max(top[2], top[3])));
    // 2^(x log2 e - e) with e a rounded multiple near the maximum: one rounding a value, and parts join by powers of two
    const float e = rintf(m * kLog2e);
    const bool plain = fabsf(m) < kLarge, any = fabsf(m) < INFINITY;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < kWarpGroups; ++u) {
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
        reinterpret_cast<int4*>(p.group_max)[((int64_t)row * p.n_groups >> 2) + part] = make_int4(top[0], top[1], top[2], top[3]);
    }
}

// A list of at most kListCap keys in shared memory, cut back to its best n_out where it fills up.
struct List {
    uint64_t key[kListCap];
    uint64_t best[kMaxOut];
    uint64_t above;     // keys below this are none of the best
    int n;
};

// The list's n_out best, in order.  All threads; the keys are different.
__device__ __forceinline__ void prune(List& l, int n_out) {
    __syncthreads();
    const int n = l.n;
    for (int i = threadIdx.x; i < n; i += kPickThreads) {
        const uint64_t mine = l.key[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += l.key[j] > mine;
        if (rank < n_out) l.best[rank] = mine;
    }
    __syncthreads();
    const int m = min(n, n_out);
    if ((int)threadIdx.x < m) l.key[threadIdx.x] = l.best[threadIdx.x];
    if (threadIdx.x == 0) {
        l.n = m;
        if (m == n_out) l.above = max(l.above, l.best[n_out - 1]);
    }
    __syncthreads();
}

// Every thread's keys that are not below the list's bound join the list.  All threads.
template <int N>
__device__ __forceinline__ void push(List& l, const uint64_t (&k)[N], int n_out) {
    const uint64_t above = l.above;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += k[i] >= above && k[i];
    const int have = l.n, all = __syncthreads_or(mine) ? mine : -1;
    if (all < 0) return;
    // where all fit, each thread takes its places at once
    __shared__ int s_want;
    if (threadIdx.x == 0) s_want = 0;
    __syncthreads();
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if ((int)(threadIdx.x & 31) >= o) incl += up;
    }
    int base = 0;
    if ((threadIdx.x & 31) == 31) base = atomicAdd(&s_want, incl);
    base = __shfl_sync(0xffffffffu, base, 31);
    __syncthreads();
    const int want = s_want;
    if (have + want <= kListCap) {
        int at = have + base + incl - mine;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (k[i] >= above && k[i]) l.key[at++] = k[i];
        if (threadIdx.x == 0) l.n = have + want;
        __syncthreads();
        return;
    }
    // many equal values: one key a thread at a time, and the bound rises with each cut
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        if (l.n + kPickThreads > kListCap) prune(l, n_out);
        uint64_t key = 0;
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (u == i) key = k[u];
        __syncthreads();
        if (key && key >= l.above) l.key[atomicAdd(&l.n, 1)] = key;
        __syncthreads();
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ __align__(16) unsigned char s_join[];  // the join: 64 rows' orders
    __shared__ List l;
    __shared__ uint64_t s_top[kPickThreads];
    __shared__ unsigned long long s_sum;
    __shared__ int32_t s_m;
    __shared__ double s_norm;
    __shared__ int s_bad, s_last;
    const int tid = threadIdx.x, row = blockIdx.x, n_out = p.n_out;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = p.seq_of[row];
    int first, rows;
    if (b < 0 || b >= p.n_seqs || !rows_of(p, b, first, rows) || row < first || row >= first + rows) return;
    const float score = p.scores ? __ldg(p.scores + row) : 0.0f, weight = p.weights ? __ldg(p.weights + row) : 1.0f;
    const int ended = p.ended ? __ldg(p.ended + row) : -1;
    const bool usable = fabsf(score) < INFINITY && weight > 0.0f && weight < INFINITY;
    const int64_t out0 = (int64_t)row * n_out;
    int count = 0;
    if (ended >= 0) {
        count = usable ? 1 : 0;
        if (tid == 0 && usable) {
            p.list_order[out0] = (double)score * (double)weight;
            p.list_total[out0] = score;
            p.list_token[out0] = ended;
        }
    } else if (usable) {
        // the sum of exponentials: parts scaled by powers of two to the largest one's, added as whole numbers of 2^-32, so
        // that their order does not matter
        if (tid == 0) s_sum = 0, s_m = ordered(-INFINITY), s_bad = 0, l.n = 0, l.above = 1;
        __syncthreads();
        const Part* parts = p.parts + (int64_t)row * p.n_parts;
        int32_t m = ordered(-INFINITY);
        bool bad = false;
        for (int i = tid; i < p.n_parts; i += kPickThreads) {
            m = max(m, ordered(parts[i].m));
            bad |= parts[i].s != parts[i].s;
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((tid & 31) == 0) atomicMax(&s_m, m);
        if (bad) s_bad = 1;
        __syncthreads();
        const float top = from_ordered(s_m);
        const float e = rintf(top * kLog2e);
        const bool plain = fabsf(top) < kLarge;
        unsigned long long sum = 0;
        for (int i = tid; i < p.n_parts; i += kPickThreads) {
            const Part q = parts[i];
            float s = 0.0f;
            if (plain && fabsf(q.m) < kLarge)
                s = q.e - e > -126.0f ? q.s * __int_as_float((127 + (int)(q.e - e)) << 23) : 0.0f;
            else if (q.m > -INFINITY)
                s = q.s * exp2f((float)(scale_of_part(q.m, q.e) - scale_of_part(top, e)));
            sum += __float2ull_rn(s * 0x1p32f);
        }
        if (sum) atomicAdd(&s_sum, sum);
        // the row's best groups: first a bound from the threads' best ones, then those above it
        uint64_t mine = 0;
        const int32_t* gm = p.group_max + (int64_t)row * p.n_groups;
        for (int g = tid; g < p.n_groups; g += kPickThreads) {
            const uint64_t k = key_of(gm[g], (uint32_t)g);
            mine = k > mine ? k : mine;
        }
        s_top[tid] = mine;
        __syncthreads();
        if (tid == 0) s_norm = plain ? ((double)e + log2((double)s_sum * 0x1p-32)) / (double)kLog2e : (double)top + log((double)s_sum * 0x1p-32);
        {
            int rank = 0;
            for (int j = 0; j < kPickThreads; ++j) rank += s_top[j] > mine;
            if (rank == n_out - 1 && mine) l.above = mine;  // threads without a group have the key 0
        }
        __syncthreads();
        for (int g0 = 0; g0 < p.n_groups; g0 += kPickThreads) {
            uint64_t k[1] = {g0 + tid < p.n_groups ? key_of(gm[g0 + tid], (uint32_t)(g0 + tid)) : 0};
            push(l, k, n_out);
        }
        prune(l, n_out);
        const int groups = l.n;
        __shared__ uint32_t s_group[kMaxOut];
        if (tid < groups) s_group[tid] = key_place(l.key[tid]);
        // a value below the last of n_out groups' maxima is none of the best, nor is -inf
        const uint64_t low = groups == n_out ? (l.key[groups - 1] >> 32) << 32 : 0;
        const uint64_t nothing = (key_of(ordered(-INFINITY), 0) >> 32 << 32) + (1ull << 32);
        __syncthreads();
        if (tid == 0) l.n = 0, l.above = low > nothing ? low : nothing;
        __syncthreads();
        const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
        for (int g0 = 0; g0 < groups; g0 += kPickThreads / 32) {
            uint64_t k[8];
            const int g = g0 + (tid >> 5);
            const int at = g < groups ? (int)s_group[g] * kGroup + (tid & 31) * 8 : p.vocab;
            Eight<T> raw;
            load_eight<T, VEC>(raw, x, at, p.vocab);
            float v[8];
            raw.floats(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = at + i < p.vocab && v[i] > -INFINITY ? key_of(ordered(v[i]), (uint32_t)(at + i)) : 0;
            push(l, k, n_out);
        }
        prune(l, n_out);
        const double norm = s_norm;
        count = s_bad || !(fabs(norm) < (double)INFINITY) ? 0 : l.n;
        if (tid < count) {
            const double total = (double)score + ((double)key_value(l.key[tid]) - norm);
            p.list_order[out0 + tid] = total * (double)weight;
            p.list_total[out0 + tid] = (float)total;
            p.list_token[out0 + tid] = (int32_t)key_place(l.key[tid]);
        }
    }
    // the last row of a request to be done joins its rows' lists
    if (tid == 0) p.list_count[row] = count;
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(p.done + b, 1u) == (uint32_t)(rows - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double* order = reinterpret_cast<double*>(s_join);
    __shared__ int s_count[kMaxWindowRows];
    if (tid < rows) s_count[tid] = __ldcg(p.list_count + first + tid);
    __syncthreads();
    int n_all = 0;
    for (int r = 0; r < rows; ++r) n_all += s_count[r];
    for (int i = tid; i < rows * n_out; i += kPickThreads)
        if (i % n_out < s_count[i / n_out]) order[i] = __ldcg(p.list_order + (int64_t)first * n_out + i);
    __syncthreads();
    const int64_t to = (int64_t)b * n_out;
    for (int i = tid; i < rows * n_out; i += kPickThreads) {
        const int r = i / n_out, j = i - r * n_out;
        if (j >= s_count[r]) continue;
        const double mine = order[i];
        int rank = j;
        for (int q = 0; q < rows && rank < n_out; ++q) {
            if (q == r) continue;
            const double* o = order + q * n_out;
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

int groups_of(int vocab) { return (vocab + kGroup * kWarpGroups - 1) / (kGroup * kWarpGroups) * kWarpGroups; }

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
    return launch_dependent(beam_pick_kernel<T, VEC>, (unsigned)p.n_rows, kPickThreads, kMaxWindowRows * p.n_out * (int)sizeof(double), s, p);
}

}  // namespace
}  // namespace kvq8

extern "C" size_t beam_select_workspace_bytes(int n_rows, int vocab, int n_seqs, int n_out) {
    using namespace kvq8;
    if (n_rows < 1 || vocab < 1 || n_seqs < 1 || n_out < 1 || !select_shape(n_rows, vocab, n_seqs, n_out)) return 0;
    SelectParams p = {};
    p.n_rows = n_rows, p.vocab = vocab, p.n_seqs = n_seqs, p.n_out = n_out;
    p.n_groups = groups_of(vocab);
    p.n_parts = p.n_groups / kWarpGroups;
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
    p.n_parts = p.n_groups / kWarpGroups;
    carve(p, static_cast<unsigned char*>(workspace));
    // eight values a load where every row starts on their size and holds whole groups of eight
    const bool vec = vocab % 8 == 0 && logits_stride % 8 == 0 && aligned_to(logits, 8 * esz);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return vec ? launch_select<float, true>(p, s) : launch_select<float, false>(p, s);
    if (dtype == KVQ8_F16) return vec ? launch_select<__half, true>(p, s) : launch_select<__half, false>(p, s);
    return vec ? launch_select<__nv_bfloat16, true>(p, s) : launch_select<__nv_bfloat16, false>(p, s);
}

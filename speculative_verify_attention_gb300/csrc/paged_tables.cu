// paged_tables.cu -- block tables and slots of a step's new tokens, from request lengths (kvq8_paged_tables).
//
// Free pages wait in a ring.  With need = ceil(len / page_size), request b takes max(need - held, 0) pages from the
// ring's head and gives max(held - need, 0) back behind its tail, both in order of request and page, so the result
// does not depend on which thread runs first.  Rows (new tokens) get the slot of their position.
//
// One launch.  Every block scans all requests by itself (three prefix sums kept in shared memory), which replaces
// any exchange between blocks; the rows and the pages moved are then spread over all threads, each finding its
// request by bisection.  The taken pages are read from the ring, not from the table that this call fills, so the
// rows need not wait for the table.  The blocks form one cluster, whose barrier stands between the last read of
// the state (held, ring_state) and its update in place.  Bound: latency (a launch, one load of the lengths, the
// scan, one dependent load of a page id).
#include <cooperative_groups.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;

struct TablesParams {
    const int32_t* lens;
    const int32_t* n_new;
    const int32_t* held;
    int32_t* held_out;
    int32_t* table;
    int32_t* ring;
    const int32_t* ring_state;
    int32_t* ring_out;
    int32_t* row_starts;
    int64_t* slots;
    int32_t* positions;
    int32_t* status;
    int n_seqs, max_pages, n_pages, n_rows, page_shift;
};

// Largest i in [0, n) with first[i] <= x; first is ascending with first[0] <= x.
__device__ __forceinline__ int last_not_above(const int* first, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) paged_tables_kernel(const TablesParams p) {
    extern __shared__ int sm[];
    const int n = p.n_seqs;
    int* s_row = sm;             // [n + 1] first row of each request
    int* s_take = s_row + n + 1; // [n + 1] pages taken before it
    int* s_give = s_take + n + 1;
    int* s_held = s_give + n + 1;
    int* s_base = s_held + n;    // position of its first new token
    __shared__ long long w_sum[3][kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int page = 1 << p.page_shift;
    const int head = p.ring_state[0], count = p.ring_state[1];

    // per-request needs and their exclusive sums, kThreads requests at a time; 64-bit totals, so that no sum of
    // malformed lengths wraps into one that looks right
    long long before[3] = {0, 0, 0};
    bool bad = head < 0 || head >= p.n_pages || count < 0 || count > p.n_pages;
    for (int base = 0; base < n; base += kThreads) {
        const int b = base + tid;
        long long v[3] = {0, 0, 0}, inc[3];
        if (b < n) {
            const int len = p.lens[b], fresh = p.n_new[b], held = p.held[b];
            const bool wrong = len < 0 || fresh < 0 || fresh > len || held < 0 || held > p.max_pages ||
                               (long long)len > ((long long)p.max_pages << p.page_shift);
            bad |= wrong;
            const int need = (int)(((long long)len + page - 1) >> p.page_shift);
            if (!wrong) {
                v[0] = fresh;
                v[1] = max(need - held, 0);
                v[2] = max(held - need, 0);
            }
            s_held[b] = held;
            s_base[b] = len - fresh;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            inc[k] = v[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, inc[k], o);
                if (lane >= o) inc[k] += up;
            }
            if (lane == 31) w_sum[k][warp] = inc[k];
        }
        __syncthreads();
        if (warp < 3) {
            long long w = w_sum[warp][lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += up;
            }
            w_sum[warp][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const long long first = before[k] + inc[k] - v[k] + (warp ? w_sum[k][warp - 1] : 0);
            if (b < n) sm[k * (n + 1) + b] = (int)min(first, (long long)0x7fffffff);
            before[k] += w_sum[k][kThreads / 32 - 1];
        }
        __syncthreads();
    }
    const long long rows = before[0], takes = before[1], gives = before[2];
    bad |= rows > p.n_rows;
    bad |= (long long)count + gives > p.n_pages;  // the ring has no room for the pages given back
    const bool malformed = __syncthreads_or(bad);
    const int status = malformed ? 2 : takes > count ? 1 : 0;

    const int n_threads = kThreads * gridDim.x, id = blockIdx.x * kThreads + tid;
    const int live = status ? 0 : (int)rows;
    for (int r = id; r < p.n_rows; r += n_threads) {
        long long slot = -1;
        int pos = -1;
        if (r < live) {
            const int b = last_not_above(s_row, n, r);
            pos = s_base[b] + r - s_row[b];
            const int k = pos >> p.page_shift, held = s_held[b];
            int pg;
            if (k < held) {
                pg = p.table[(long long)b * p.max_pages + k];
            } else {
                int at = head + s_take[b] + (k - held);
                if (at >= p.n_pages) at -= p.n_pages;
                pg = p.ring[at];
            }
            slot = ((long long)pg << p.page_shift) + (pos & (page - 1));
        }
        p.slots[r] = slot;
        p.positions[r] = pos;
    }
    if (!status) {
        for (int i = id; i < (int)takes; i += n_threads) {
            const int b = last_not_above(s_take, n, i);
            int at = head + i;
            if (at >= p.n_pages) at -= p.n_pages;
            p.table[(long long)b * p.max_pages + s_held[b] + (i - s_take[b])] = p.ring[at];
        }
        for (int i = id; i < (int)gives; i += n_threads) {
            const int b = last_not_above(s_give, n, i);
            const int need = s_held[b] - ((b + 1 < n ? s_give[b + 1] : (int)gives) - s_give[b]);
            int at = head + count;  // head + count + i < 3 n_pages: both terms are at most n_pages
            if (at >= p.n_pages) at -= p.n_pages;
            at += i;
            if (at >= p.n_pages) at -= p.n_pages;
            p.ring[at] = p.table[(long long)b * p.max_pages + need + (i - s_give[b])];
        }
    }
    for (int b = id; b <= n; b += n_threads) p.row_starts[b] = status ? 0 : b < n ? s_row[b] : (int)rows;
    // every block has read held and ring_state; now they may change in place
    cooperative_groups::this_cluster().sync();
    for (int b = id; b < n; b += n_threads) {
        int now = s_held[b];
        if (!status)
            now += ((b + 1 < n ? s_take[b + 1] : (int)takes) - s_take[b]) - ((b + 1 < n ? s_give[b + 1] : (int)gives) - s_give[b]);
        p.held_out[b] = now;
    }
    if (id == 0) {
        int h = head;
        if (!status) {
            h += (int)takes;
            if (h >= p.n_pages) h -= p.n_pages;
        }
        p.ring_out[0] = h;
        p.ring_out[1] = status ? count : count - (int)takes + (int)gives;
        p.status[0] = status;
    }
}

}  // namespace
}  // namespace kvq8

extern "C" int kvq8_paged_tables(const int32_t* lens, const int32_t* n_new, const int32_t* held, int n_seqs, int page_size,
                                 int32_t* page_table, int max_pages, int32_t* free_ring, int n_pages,
                                 const int32_t* ring_state, int32_t* held_out, int32_t* ring_out, int32_t* row_starts,
                                 int64_t* slots, int32_t* positions, int n_rows, int32_t* status, kvq8_stream_t stream) {
    using namespace kvq8;
    if (n_seqs < 1 || max_pages < 1 || n_pages < 1 || n_rows < 0) return KVQ8_ERR_INVALID_ARG;
    if (!lens || !n_new || !held || !page_table || !free_ring || !ring_state || !held_out || !ring_out || !row_starts ||
        !status || (n_rows > 0 && (!slots || !positions)))
        return KVQ8_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) || n_seqs > kMaxSeqs ||
        n_pages > (1 << 30) || n_rows > (1 << 30))
        return KVQ8_ERR_UNSUPPORTED;
    for (const void* q : {(const void*)lens, (const void*)n_new, (const void*)held, (const void*)page_table,
                          (const void*)free_ring, (const void*)ring_state, (const void*)held_out, (const void*)ring_out,
                          (const void*)row_starts, (const void*)positions, (const void*)status})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    if (!aligned_to(slots, 8)) return KVQ8_ERR_MISALIGNED;
    TablesParams p = {lens, n_new, held, held_out, page_table, free_ring, ring_state, ring_out, row_starts, slots,
                      positions, status, n_seqs, max_pages, n_pages, n_rows, log2_of(page_size)};
    const int smem = (5 * n_seqs + 3) * (int)sizeof(int);
    static SmemOptIn opt;
    const int rc = opt.ensure(paged_tables_kernel, (5 * kMaxSeqs + 3) * (int)sizeof(int));
    if (rc != KVQ8_OK) return rc;
    const int want = (n_rows + kThreads - 1) / kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(want < 1 ? 1 : want > kMaxCluster ? kMaxCluster : want);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cfg.gridDim.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, paged_tables_kernel, p));
}

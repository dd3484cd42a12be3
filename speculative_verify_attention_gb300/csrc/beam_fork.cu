// beam_fork.cu -- what a sequence holds follows the beams that were chosen: its row of token counts (token_counts_fork) and
// its pages (kvq8_paged_fork).
//
// parents[i] is the sequence that child i goes on from (< 0: there is no child i).  A sequence's first child, the one of the
// lowest number, takes over what cannot be shared; the others get copies.  Both calls plan in one block (counts of children,
// first children by an atomic minimum, exclusive sums over the children: results do not depend on the order of execution) and
// then spread the work.  Bound: counts by the memory (384 beams over 248320 values, 232 MB: 38 us, 6.1 TB/s, 90 % of a copy's rate),
// pages by the latency of dependent launches and loads (512 beams of up to 8192 tokens, 61 thousand pages: 12 us in three launches; 4
// beams of 2048 tokens 5 us in one).
#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxStates = 65536;

// Exclusive sum of one value a thread, and the total.
__device__ __forceinline__ int block_sums(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (int)(blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += up;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    total = s_warp[31];
    return inc - v + (warp ? s_warp[warp - 1] : 0);
}

// The parents of a planning thread's children, -1: none.  They are asked for first of all.
constexpr int kPlanPer = kMaxSeqs / kPlanThreads;
struct Children {
    int of[kPlanPer];
    __device__ __forceinline__ Children(const int32_t* parents, int n_children) {
#pragma unroll
        for (int u = 0; u < kPlanPer; ++u) {
            const int i = threadIdx.x + u * kPlanThreads;
            of[u] = i < n_children ? parents[i] : -1;
        }
    }
};

// s_first[q]: q's first child (n_children where it has none), s_kids[q]: how many.  True if a parent is out of range.
__device__ __forceinline__ bool families(const Children& c, int n_children, int n_seqs, int* s_first, int* s_kids) {
    for (int q = threadIdx.x; q < n_seqs; q += kPlanThreads) s_first[q] = n_children, s_kids[q] = 0;
    __syncthreads();
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        const int i = threadIdx.x + u * kPlanThreads, q = c.of[u];
        if (q >= n_seqs) bad = true;
        if (q < 0 || q >= n_seqs) continue;
        atomicMin(s_first + q, i);
        atomicAdd(s_kids + q, 1);
    }
    return __syncthreads_or(bad);
}

// ---------------------------------------------------------------- counts

struct CountsFork {
    const int32_t* parents;
    const int32_t* state_of;
    int32_t* state_of_out;
    uint32_t* counts;
    int32_t* status;
    int2* copies;   // workspace [n_children]: rows from and to, -1 where the child copies nothing
    int n_children, n_seqs, n_states, vocab;
};

__global__ void __launch_bounds__(kPlanThreads) counts_fork_plan_kernel(const __grid_constant__ CountsFork p) {
    extern __shared__ int sm[];
    int* s_first = sm;
    int* s_kids = s_first + p.n_seqs;
    int* s_state = s_kids + p.n_seqs;                                    // the sequences' rows: state_of_out may be state_of
    const int n_words = (p.n_states + 31) / 32;
    uint32_t* s_kept = reinterpret_cast<uint32_t*>(s_state + p.n_seqs);  // [n_words] rows that a first child keeps
    int* s_free = reinterpret_cast<int*>(s_kept + n_words);              // [n_words] unkept rows before the word
    __shared__ int s_warp[32];
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Children children(p.parents, p.n_children);
    int states[kPlanPer];
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        const int q = tid + u * kPlanThreads;
        states[u] = q >= p.n_seqs ? -1 : p.state_of ? p.state_of[q] : q;
    }
    for (int w = tid; w < n_words; w += kPlanThreads) s_kept[w] = 0u;
    bool bad = families(children, p.n_children, p.n_seqs, s_first, s_kids);
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        const int q = tid + u * kPlanThreads;
        if (q >= p.n_seqs) continue;
        const int st = states[u] < 0 || states[u] >= p.n_states ? -1 : states[u];
        s_state[q] = st;
        // two sequences that are both gone on from cannot have the same row
        if (st >= 0 && s_kids[q]) bad |= (atomicOr(s_kept + (st >> 5), 1u << (st & 31)) >> (st & 31)) & 1u;
    }
    bad = __syncthreads_or(bad);
    int free_rows = 0;
    for (int w0 = 0; w0 < n_words; w0 += kPlanThreads) {
        const int w = w0 + tid;
        const int rows = w < n_words ? min(32, p.n_states - 32 * w) : 0;
        const int here = rows > 0 ? rows - __popc(s_kept[w]) : 0;
        int total;
        const int before = block_sums(here, s_warp, total);
        if (w < n_words) s_free[w] = free_rows + before;
        free_rows += total;
    }
    __syncthreads();
    int copies = 0;
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        if (u * kPlanThreads >= p.n_children) break;
        const int i = tid + u * kPlanThreads, q = children.of[u];
        int from = -1, state = -1;
        bool copy = false;
        if (q >= 0 && q < p.n_seqs) {
            state = from = s_state[q];
            copy = from >= 0 && s_first[q] != i;
        }
        int total;
        const int k = copies + block_sums(copy, s_warp, total);
        copies += total;
        if (copy) {
            state = -1;
            if (k < free_rows) {  // the k-th row that nobody keeps
                int lo = 0, hi = n_words;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_free[mid] <= k)
                        lo = mid;
                    else
                        hi = mid;
                }
                state = 32 * lo + (int)__fns(~s_kept[lo], 0, k - s_free[lo] + 1);
            }
        }
        if (i < p.n_children) {
            p.copies[i] = copy ? make_int2(from, state) : make_int2(-1, -1);
            p.state_of_out[i] = state;
        }
    }
    const int status = bad ? 2 : copies > free_rows ? 1 : 0;
    if (status) {  // nothing moves
        __syncthreads();
        for (int i = tid; i < p.n_children; i += kPlanThreads) {
            p.copies[i] = make_int2(-1, -1);
            p.state_of_out[i] = -1;
        }
    }
    if (tid == 0) p.status[0] = status;
}

constexpr int kRowThreads = 256;
constexpr int kRowPer = 4;  // 16-byte stores of a thread

// Block (16 KB of a row, child), four or eight 16-byte loads a thread in flight; siblings read a row from L2.  A row that is copied from is
// kept by its first child, and one copied to is kept by nobody, so no block reads what another writes.
//   EVEN: every row starts on 16 bytes and holds whole sixteens of them.
//   Else rows start anywhere among four values: a thread stores on 16 bytes of its row what it shifts together from the 16-byte pieces
//   around it; the ends go by values.  580 beams over 106299 values (154 MB): 31 us (by values 65).
template <bool EVEN>
__global__ void __launch_bounds__(kRowThreads) counts_copy_kernel(const __grid_constant__ CountsFork p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int2 c = p.copies[blockIdx.y];
    if (c.x < 0) return;
    const uint32_t* src = p.counts + (int64_t)c.x * p.vocab;
    uint32_t* dst = p.counts + (int64_t)c.y * p.vocab;
    const int i0 = (int)(blockIdx.x * kRowThreads * kRowPer + threadIdx.x);
    if (EVEN) {
        const int n = p.vocab / 4;
        uint4 v[kRowPer];
#pragma unroll
        for (int k = 0; k < kRowPer; ++k)
            if (i0 + k * kRowThreads < n) v[k] = reinterpret_cast<const uint4*>(src)[i0 + k * kRowThreads];
#pragma unroll
        for (int k = 0; k < kRowPer; ++k)
            if (i0 + k * kRowThreads < n) reinterpret_cast<uint4*>(dst)[i0 + k * kRowThreads] = v[k];
        return;
    }
    const int before = (int)((reinterpret_cast<uintptr_t>(dst) & 15u) / 4), shift = (int)((reinterpret_cast<uintptr_t>(src) / 4 - before) & 3u);
    uint4 a[kRowPer], b[kRowPer];
    auto from = [&](int k) { return (i0 + k * kRowThreads) * 4 - before; };
    auto whole = [&](int k) { return from(k) - shift >= 0 && from(k) - shift + 8 <= p.vocab; };
#pragma unroll
    for (int k = 0; k < kRowPer; ++k)
        if (whole(k)) {
            a[k] = *reinterpret_cast<const uint4*>(src + from(k) - shift);
            b[k] = *reinterpret_cast<const uint4*>(src + from(k) - shift + 4);
        }
#pragma unroll
    for (int k = 0; k < kRowPer; ++k) {
        if (whole(k)) {
            uint4 v = a[k];
            if (shift == 1) v = make_uint4(a[k].y, a[k].z, a[k].w, b[k].x);
            if (shift == 2) v = make_uint4(a[k].z, a[k].w, b[k].x, b[k].y);
            if (shift == 3) v = make_uint4(a[k].w, b[k].x, b[k].y, b[k].z);
            *reinterpret_cast<uint4*>(dst + from(k)) = v;
        } else {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (from(k) + i >= 0 && from(k) + i < p.vocab) v[i] = src[from(k) + i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (from(k) + i >= 0 && from(k) + i < p.vocab) dst[from(k) + i] = v[i];
        }
    }
}

// ---------------------------------------------------------------- pages

struct PagedFork {
    const int32_t* parents;
    const int32_t* lens;
    const int32_t* held;
    const int32_t* table;
    const int32_t* shares;
    const int32_t* ring_state;
    int32_t* ring;
    int32_t* table_out;
    int32_t* lens_out;
    int32_t* held_out;
    int32_t* shares_out;
    int32_t* ring_out;
    int32_t* copy_src;
    int32_t* copy_dst;
    int32_t* copy_rows;
    int32_t* status;
    // workspace
    int32_t* take;      // [n_children] the fresh page of a child, -1: none
    int32_t* holders;   // [n_seqs] children, and kGoesOn: the first one goes on in the last page; kStays: nothing moves
    uint32_t* freed;    // [ceil(n_pages / 32)] pages that nobody holds any more
    int32_t* head;      // the ring's head and count as they were, pages taken, and whether anything moves
    int n_children, n_seqs, max_pages, n_pages, page_shift;
};

constexpr int32_t kGoesOn = 1 << 30, kStays = 1 << 29;
constexpr int kSmallTasks = 128, kSmallPages = 16384;  // what one block does alone
constexpr int kForkThreads = 256;
constexpr int kForkBlocks = 152 * 8;
constexpr int kCopyPer = 4096;  // pages of the pool that a block of the first kernel clears or copies

// Thread id of n: the shares, if they are not updated in place, and no marks.
__device__ __forceinline__ void fork_clear(const PagedFork& p, int id, int n) {
    if (p.shares != p.shares_out)
        for (int i = id; i < p.n_pages; i += n) p.shares_out[i] = p.shares[i];
    for (int i = id; i < (p.n_pages + 31) / 32; i += n) p.freed[i] = 0u;
}

// One block: who goes on from whom, which pages are taken, and the children's lengths and copies.  Returns whether anything moves.
__device__ __forceinline__ bool fork_plan(const PagedFork& p, int* sm, int* s_warp) {
    const int tid = threadIdx.x;
    int* s_first = sm;
    int* s_kids = s_first + p.n_seqs;
    int* s_len = s_kids + p.n_seqs;
    int* s_tail = s_len + p.n_seqs;  // its last page, if that is not full
    const int page = 1 << p.page_shift;
    const int head = p.ring_state[0], count = p.ring_state[1];
    // what the sequences alone say, asked for before the children are counted
    const Children children(p.parents, p.n_children);
    int holds[kPlanPer];  // 0, or kGoesOn; -1: held is wrong, -2: its children's length is
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        const int q = tid + u * kPlanThreads;
        holds[u] = 0;
        if (q >= p.n_seqs) continue;
        const int held = p.held[q], len = p.lens[q];
        s_len[q] = len;
        if (held < 0 || held > p.max_pages) {
            holds[u] = -1;
        } else if (len < 0 || len > ((int64_t)held << p.page_shift)) {
            holds[u] = -2;
        } else if (len & (page - 1)) {
            // a last page that is not full goes to the first child, if no other sequence holds it
            const int tail = p.table[(int64_t)q * p.max_pages + (len >> p.page_shift)];
            if (tail < 0 || tail >= p.n_pages || p.shares[tail] == 0) holds[u] = kGoesOn;
            s_tail[q] = tail;
        }
    }
    bool bad = families(children, p.n_children, p.n_seqs, s_first, s_kids);
    bad |= head < 0 || head >= p.n_pages || count < 0 || count > p.n_pages;
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        const int q = tid + u * kPlanThreads;
        if (q >= p.n_seqs) continue;
        const int kids = s_kids[q];
        bad |= holds[u] == -1 || (holds[u] == -2 && kids);
        s_kids[q] = kids | (kids && holds[u] == kGoesOn ? kGoesOn : 0);
    }
    bad = __syncthreads_or(bad);
    int takes = 0;
#pragma unroll
    for (int u = 0; u < kPlanPer; ++u) {
        if (u * kPlanThreads >= p.n_children) break;
        const int i = tid + u * kPlanThreads, q = children.of[u];
        const bool live = !bad && q >= 0;
        int len = 0;
        bool take = false;
        if (live) {
            len = s_len[q];
            take = (len & (page - 1)) && !(s_first[q] == i && (s_kids[q] & kGoesOn));
        }
        int total;
        const int k = takes + block_sums(take, s_warp, total);
        takes += total;
        if (i < p.n_children) {
            int fresh = -1, src = -1;
            if (take && k < count) {
                fresh = p.ring[head + k >= p.n_pages ? head + k - p.n_pages : head + k];
                src = s_tail[q];
            }
            p.take[i] = fresh;
            p.copy_src[i] = src;
            p.copy_dst[i] = fresh;
            p.copy_rows[i] = take ? len & (page - 1) : 0;
            p.lens_out[i] = len;
            p.held_out[i] = ((len - 1) >> p.page_shift) + 1;  // (rounded up first, a length may pass 31 bits)
        }
    }
    const int status = bad ? 2 : takes > count ? 1 : 0;
    for (int q = tid; q < p.n_seqs; q += kPlanThreads) p.holders[q] = status ? kStays : s_kids[q];
    if (status) {
        __syncthreads();
        for (int i = tid; i < p.n_children; i += kPlanThreads) {
            p.copy_src[i] = p.copy_dst[i] = -1;
            p.copy_rows[i] = p.lens_out[i] = p.held_out[i] = 0;
        }
    }
    if (tid == 0) {
        p.status[0] = status;
        p.head[0] = head, p.head[1] = count, p.head[2] = status ? 0 : takes, p.head[3] = status == 0;
    }
    return status == 0;
}

constexpr int kPiece = 128;  // entries of a table's row that a warp takes

// A lane's four entries of child i's row of the table, from k0 on, from its parent's.
__device__ __forceinline__ void fork_child(const PagedFork& p, int i, int k0) {
    const int need = p.held_out[i], q = p.parents[i], fresh = p.take[i];
    if (need <= 0) return;
    const int tail = fresh >= 0 ? need - 1 : -1;
    const int32_t* from = p.table + (int64_t)q * p.max_pages;
    int32_t* to = p.table_out + (int64_t)i * p.max_pages;
    int v[kPiece / 32];
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u) v[u] = k0 + u * 32 < need ? from[k0 + u * 32] : 0;
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u)
        if (k0 + u * 32 < need) to[k0 + u * 32] = k0 + u * 32 == tail ? fresh : v[u];
}

// What the pages at place k of kTogether sequences gain or lose: each is held by their children from now on, not by themselves.  shares
// counts holders beyond the first, so the last one to let a page go takes it below zero.  A request's beams stand together and share
// most of their pages, which as many children hold again: the changes of neighbours of one page are added up first, and most come
// to nothing.  The atomics that are left go out together: one after another they took longer than all the rest.
constexpr int kTogether = 8;
__device__ __forceinline__ void fork_pages(const PagedFork& p, int group, int k) {
    const int q0 = group * kTogether;
    int page[kTogether], change[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
        const int q = q0 + u;
        const bool there = q < p.n_seqs;
        const int held = there ? p.held[q] : 0, holders = there ? p.holders[q] : kStays, len = there ? p.lens[q] : 0;
        const int kids = holders & ~(kGoesOn | kStays), full = len >> p.page_shift;  // (without children a length means nothing)
        const bool on = k < held && !(holders & kStays);
        page[u] = on ? p.table[(int64_t)q * p.max_pages + k] : -1;
        change[u] = on ? (kids == 0 ? 0 : k < full ? kids : k == full && (holders & kGoesOn) ? 1 : 0) - 1 : 0;
    }
#pragma unroll
    for (int u = 0; u + 1 < kTogether; ++u)
        if (page[u] == page[u + 1]) change[u + 1] += change[u], change[u] = 0;
    int left[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
        if (page[u] < 0 || page[u] >= p.n_pages) change[u] = 0;
        left[u] = change[u] ? atomicAdd(p.shares_out + page[u], change[u]) : 0;
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
        if (change[u] && left[u] + change[u] < 0) atomicOr(p.freed + (page[u] >> 5), 1u << (page[u] & 31));
}

// Warp `warp` of n: a piece of a child's row of the table at a time, or a place a lane of a group of sequences.
__host__ __device__ __forceinline__ int64_t fork_tasks(const PagedFork& p, int64_t& children) {
    children = (int64_t)p.n_children * ((p.max_pages + kPiece - 1) / kPiece);
    return children + (int64_t)((p.n_seqs + kTogether - 1) / kTogether) * ((p.max_pages + 31) / 32);
}
__device__ __forceinline__ void fork_all(const PagedFork& p, int warp, int n) {
    const int pieces = (p.max_pages + kPiece - 1) / kPiece, parts = (p.max_pages + 31) / 32, lane = threadIdx.x & 31;
    int64_t children;
    const int64_t all = fork_tasks(p, children);
    for (int64_t w = warp; w < all; w += n) {
        if (w < children) {
            const int i = (int)(w / pieces);
            fork_child(p, i, (int)(w - (int64_t)i * pieces) * kPiece + lane);
        } else {
            const int group = (int)((w - children) / parts);
            fork_pages(p, group, (int)(w - children - (int64_t)group * parts) * 32 + lane);
        }
    }
}

// After all tasks: the pages that nobody holds any more go behind the ring's tail, in order of their number.  Block `block` of n
// has a part of the marks, and counts those before it itself; a warp writes a word's pages at once.
constexpr int kGiveThreads = 1024;  // or fewer
constexpr int kGiveWords = 64;      // words of marks that a block of the wide form takes, in up to 64 blocks
__device__ __forceinline__ void fork_give(const PagedFork& p, int block, int n, int* s_warp) {
    __shared__ uint32_t s_bits[kGiveThreads];
    __shared__ int s_at[kGiveThreads];
    const int tid = threadIdx.x, threads = (int)blockDim.x, lane = tid & 31;
    const int head = p.head[0], count = p.head[1], takes = p.head[2];
    const bool moved = p.head[3] != 0;
    int given = 0, tail = head + count;
    if (moved) {
        if (tail >= p.n_pages) tail -= p.n_pages;
        const int n_words = (p.n_pages + 31) / 32, per = (n_words + n - 1) / n, first = min(block * per, n_words), last = min(first + per, n_words);
        int before = 0;
#pragma unroll 8
        for (int w = tid; w < first; w += threads) before += __popc(__ldcg(p.freed + w));
        block_sums(before, s_warp, given);
        for (int w0 = first; w0 < last; w0 += threads) {
            const uint32_t bits = w0 + tid < last ? __ldcg(p.freed + w0 + tid) : 0u;
            int total;
            s_at[tid] = given + block_sums(__popc(bits), s_warp, total);
            s_bits[tid] = bits;
            given += total;
            __syncthreads();
            for (int w = tid >> 5; w < min(threads, last - w0); w += threads / 32) {
                const uint32_t word = s_bits[w];
                if (!(word >> lane & 1u)) continue;
                const int id = 32 * (w0 + w) + lane, k = s_at[w] + __popc(word & ((1u << lane) - 1));
                p.shares_out[id] = 0;
                if (k < p.n_pages - count) p.ring[tail + k >= p.n_pages ? tail + k - p.n_pages : tail + k] = id;
            }
            __syncthreads();
        }
    }
    if (block == n - 1 && tid == 0) {  // its sum is the whole one
        const int h = head + takes;
        p.ring_out[0] = moved && h >= p.n_pages ? h - p.n_pages : h;  // (a malformed one is repeated)
        p.ring_out[1] = moved ? count - takes + min(given, p.n_pages - count) : count;
    }
}

// Few entries: everything in one block.
__global__ void __launch_bounds__(kPlanThreads) paged_fork_small_kernel(const __grid_constant__ PagedFork p) {
    extern __shared__ int sm[];
    __shared__ int s_warp[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fork_clear(p, threadIdx.x, kPlanThreads);
    const bool moved = fork_plan(p, sm, s_warp);
    __syncthreads();
    if (moved) fork_all(p, threadIdx.x >> 5, kPlanThreads / 32);
    __syncthreads();
    fork_give(p, 0, 1, s_warp);
}

// Block 0 plans, the others clear.
__global__ void __launch_bounds__(kPlanThreads) paged_fork_plan_kernel(const __grid_constant__ PagedFork p) {
    extern __shared__ int sm[];
    __shared__ int s_warp[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0)
        fork_plan(p, sm, s_warp);
    else
        fork_clear(p, ((int)blockIdx.x - 1) * kPlanThreads + threadIdx.x, kPlanThreads * ((int)gridDim.x - 1));
}


__global__ void __launch_bounds__(kForkThreads) paged_fork_kernel(const __grid_constant__ PagedFork p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fork_all(p, (int)blockIdx.x * (kForkThreads / 32) + (int)(threadIdx.x >> 5), (int)gridDim.x * (kForkThreads / 32));
}

__global__ void __launch_bounds__(kForkThreads) paged_fork_give_kernel(const __grid_constant__ PagedFork p) {
    __shared__ int s_warp[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fork_give(p, (int)blockIdx.x, (int)gridDim.x, s_warp);
}

size_t fork_carve(PagedFork& p, unsigned char* base) {
    size_t at = 0;
    auto take = [&](auto*& ptr, size_t n) {
        ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(base + at);
        at += (n * sizeof(*ptr) + 15) / 16 * 16;
    };
    take(p.take, (size_t)p.n_children);
    take(p.holders, (size_t)p.n_seqs);
    take(p.freed, ((size_t)p.n_pages + 31) / 32);
    take(p.head, 4);
    return at;
}

}  // namespace
}  // namespace kvq8

extern "C" size_t token_counts_fork_workspace_bytes(int n_children) {
    return n_children < 1 || n_children > kvq8::kMaxSeqs ? 0 : ((size_t)n_children * sizeof(int2) + 15) / 16 * 16;
}

extern "C" int token_counts_fork(const int32_t* parents, int n_children, const int32_t* state_of, int n_seqs, uint32_t* counts,
                                 int n_states, int vocab, int32_t* state_of_out, int32_t* status, void* workspace,
                                 size_t workspace_bytes, kvq8_stream_t stream) {
    using namespace kvq8;
    if (n_children < 1 || n_seqs < 1 || n_states < 1 || vocab < 1) return KVQ8_ERR_INVALID_ARG;
    if (!parents || !counts || !state_of_out || !status) return KVQ8_ERR_INVALID_ARG;
    // state_of_out may be state_of itself
    const size_t kids = (size_t)n_children * 4, old = (size_t)n_seqs * 4;
    if (ranges_meet(parents, kids, state_of_out, kids) || (state_of != state_of_out && ranges_meet(state_of, old, state_of_out, kids)))
        return KVQ8_ERR_INVALID_ARG;
    if (n_children > kMaxSeqs || n_seqs > kMaxSeqs || n_states > kMaxStates || vocab > (1 << 30)) return KVQ8_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < token_counts_fork_workspace_bytes(n_children)) return KVQ8_ERR_WORKSPACE;
    for (const void* q : {(const void*)parents, (const void*)state_of, (const void*)counts, (const void*)state_of_out, (const void*)status})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    if (!aligned16(workspace)) return KVQ8_ERR_MISALIGNED;
    // rows are copied by what the plan has written; one of them or the status over it would be followed
    const size_t need = token_counts_fork_workspace_bytes(n_children), all = (size_t)n_states * vocab * 4;
    const struct {
        const void* at;
        size_t bytes;
    } reads[] = {{parents, kids}, {state_of == state_of_out ? nullptr : state_of, old}},
      writes[] = {{counts, all}, {state_of_out, kids}, {status, 4}, {workspace, need}};
    for (const auto& w : writes) {
        for (const auto& r : reads)
            if (ranges_meet(r.at, r.bytes, w.at, w.bytes)) return KVQ8_ERR_INVALID_ARG;
        for (const auto* o = writes; o != &w; ++o)
            if (ranges_meet(o->at, o->bytes, w.at, w.bytes)) return KVQ8_ERR_INVALID_ARG;
    }
    const CountsFork p = {parents, state_of, state_of_out, counts, status, static_cast<int2*>(workspace), n_children, n_seqs, n_states, vocab};
    const int smem = (3 * n_seqs + 2 * ((n_states + 31) / 32)) * 4;
    static SmemOptIn opt;
    int rc = opt.ensure(counts_fork_plan_kernel, (3 * kMaxSeqs + 2 * kMaxStates / 32) * 4);
    if (rc != KVQ8_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    rc = launch_dependent(counts_fork_plan_kernel, 1, kPlanThreads, smem, s, p);
    if (rc != KVQ8_OK) return rc;
    const bool even = vocab % 4 == 0 && aligned16(counts);
    const int per = kRowThreads * kRowPer * 4;
    const dim3 grid((unsigned)((vocab + (even ? 0 : 3) + per - 1) / per), (unsigned)n_children);
    if (even) return launch_dependent(counts_copy_kernel<true>, grid, kRowThreads, 0, s, p);
    return launch_dependent(counts_copy_kernel<false>, grid, kRowThreads, 0, s, p);
}

extern "C" size_t kvq8_paged_fork_workspace_bytes(int n_seqs, int n_children, int n_pages) {
    using namespace kvq8;
    if (n_seqs < 1 || n_children < 1 || n_pages < 1 || n_seqs > kMaxSeqs || n_children > kMaxSeqs || n_pages > (1 << 30)) return 0;
    PagedFork p = {};
    p.n_seqs = n_seqs, p.n_children = n_children, p.n_pages = n_pages;
    return fork_carve(p, nullptr);
}

extern "C" int kvq8_paged_fork(const int32_t* parents, int n_children, const int32_t* lens, const int32_t* held, int n_seqs,
                               int page_size, const int32_t* page_table, int max_pages, const int32_t* shares,
                               int32_t* free_ring, int n_pages, const int32_t* ring_state, int32_t* page_table_out,
                               int32_t* lens_out, int32_t* held_out, int32_t* shares_out, int32_t* ring_out,
                               int32_t* copy_src, int32_t* copy_dst, int32_t* copy_rows, int32_t* status, void* workspace,
                               size_t workspace_bytes, kvq8_stream_t stream) {
    using namespace kvq8;
    if (n_children < 1 || n_seqs < 1 || max_pages < 1 || n_pages < 1) return KVQ8_ERR_INVALID_ARG;
    const void* in[] = {parents, lens, held, page_table, shares, ring_state};
    const void* out[] = {free_ring, page_table_out, lens_out, held_out, shares_out, ring_out, copy_src, copy_dst, copy_rows, status};
    for (const void* q : in)
        if (!q) return KVQ8_ERR_INVALID_ARG;
    for (const void* q : out)
        if (!q) return KVQ8_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) || n_seqs > kMaxSeqs || n_children > kMaxSeqs ||
        n_pages > (1 << 30) || max_pages > (1 << 24))
        return KVQ8_ERR_UNSUPPORTED;
    for (const void* q : in)
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    for (const void* q : out)
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    // the sequences' state is read while the children's is written, and what one kernel writes the next one indexes by
    struct Array {
        const void* at;
        size_t bytes;
    };
    const size_t old = (size_t)n_seqs * 4, kids = (size_t)n_children * 4, pool = (size_t)n_pages * 4;
    const Array reads[] = {{parents, kids}, {lens, old}, {held, old}, {page_table, old * max_pages}, {shares, pool}, {ring_state, 8}};
    const Array writes[] = {{free_ring, pool}, {page_table_out, kids * max_pages}, {lens_out, kids}, {held_out, kids}, {shares_out, pool},
                            {ring_out, 8}, {copy_src, kids}, {copy_dst, kids}, {copy_rows, kids}, {status, 4}};
    for (const Array& w : writes) {
        for (const Array& r : reads) {
            const bool itself = w.at == r.at && ((r.at == shares && w.at == shares_out) || (r.at == ring_state && w.at == ring_out));
            if (!itself && ranges_meet(r.at, r.bytes, w.at, w.bytes)) return KVQ8_ERR_INVALID_ARG;
        }
        for (const Array* o = writes; o != &w; ++o)
            if (ranges_meet(o->at, o->bytes, w.at, w.bytes)) return KVQ8_ERR_INVALID_ARG;
    }
    if (!workspace || workspace_bytes < kvq8_paged_fork_workspace_bytes(n_seqs, n_children, n_pages)) return KVQ8_ERR_WORKSPACE;
    if (!aligned16(workspace)) return KVQ8_ERR_MISALIGNED;
    PagedFork p = {parents, lens, held, page_table, shares, ring_state, free_ring, page_table_out, lens_out, held_out, shares_out,
                   ring_out, copy_src, copy_dst, copy_rows, status, nullptr, nullptr, nullptr, nullptr, n_children, n_seqs,
                   max_pages, n_pages, log2_of(page_size)};
    fork_carve(p, static_cast<unsigned char*>(workspace));
    cudaStream_t s = (cudaStream_t)stream;
    int64_t children;
    const int64_t tasks = fork_tasks(p, children);
    const int smem = 4 * n_seqs * 4;
    static SmemOptIn opt_small, opt_plan;
    if (tasks <= kSmallTasks && n_pages <= kSmallPages) {
        const int rc = opt_small.ensure(paged_fork_small_kernel, 4 * kMaxSeqs * 4);
        return rc != KVQ8_OK ? rc : launch_dependent(paged_fork_small_kernel, 1, kPlanThreads, smem, s, p);
    }
    int rc = opt_plan.ensure(paged_fork_plan_kernel, 4 * kMaxSeqs * 4);
    if (rc != KVQ8_OK) return rc;
    const int clear = (n_pages + kCopyPer - 1) / kCopyPer;
    rc = launch_dependent(paged_fork_plan_kernel, (unsigned)(1 + (clear < 75 ? clear : 75)), kPlanThreads, smem, s, p);
    if (rc != KVQ8_OK) return rc;
    const int64_t blocks = (tasks + kForkThreads / 32 - 1) / (kForkThreads / 32);
    rc = launch_dependent(paged_fork_kernel, (unsigned)(blocks < kForkBlocks ? blocks : kForkBlocks), kForkThreads, 0, s, p);
    if (rc != KVQ8_OK) return rc;
    const int words = (n_pages + 31) / 32, give = (words + kGiveWords - 1) / kGiveWords;
    return launch_dependent(paged_fork_give_kernel, (unsigned)(give < 64 ? give : 64), kForkThreads, 0, s, p);
}

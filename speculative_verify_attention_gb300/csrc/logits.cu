// logits.cu -- logits of a verify step bent by penalties, biases and grammar masks (logits_adjust), and the token
// counts that the penalties read (token_counts).
//
// Row r of request b, value v, with c the times v was generated (counts, plus the window tokens that row r sees)
// and "seen" whether v was generated or stands in the prompt (bit 31 of its count):
//   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   x = x + (bias(v) - (frequency * c + presence * [c > 0]));  x = allowed(v) ? x : -inf
// all in fp32, whatever the type of the logits.
#include <float.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kAdjThreads = 128;
constexpr int kAdjPer = 8;                          // values of one row per thread
constexpr int kAdjChunk = kAdjThreads * kAdjPer;    // vocabulary values per block
constexpr int kAdjDepth = 2;                        // rows whose logits are in flight
constexpr int kAdjRows = 12;                        // rows of a request that a block takes, about
constexpr uint32_t kInPrompt = 0x80000000u;

struct AdjustParams {
    const void* logits;
    float* out;
    int64_t in_stride, out_stride;
    const int32_t* row_starts;
    const float* penalties;        // [n_seqs][3] repetition, frequency, presence
    const uint32_t* counts;        // [n_states][vocab]
    const int32_t* state_of;       // [n_seqs]
    const int32_t* tokens;         // [n_rows] window tokens
    const uint64_t* mask;          // [n_rows]
    const int32_t* bias_starts;    // [n_seqs + 1]
    const int32_t* bias_tokens;
    const float* bias_values;
    const uint32_t* grammar;       // [n_grammar][ceil(vocab / 32)]
    const int32_t* grammar_of;     // [n_rows]
    int n_rows, vocab, n_seqs, n_states, n_bias, n_grammar;
};

// A seen value under the repetition penalty.  x / b by b's rounded reciprocal r and one corrected step, as in scale_of of
// the quantiser: within one unit of the last place (mostly the IEEE quotient) in four operations instead of a called
// division, which bound the kernel where a few percent of the vocabulary was seen (every warp then has such a value).
// An infinite x has no remainder (NaN, which the maximum drops).
__device__ __forceinline__ float repeated(float x, float b, float r) {
    const float q0 = x * r;
    const float q = fmaf(fmaxf(fmaf(-q0, b, x), -FLT_MAX), r, q0);
    return x > 0.0f ? q : __fmul_rn(x, b);
}

// (The functions that round here and below keep products and sums apart, which the compiler could join in one place and not in
// another: then the rows of a request would differ by their route.)
__device__ __forceinline__ float penalty_of(int c, float frequency, float presence) {
    return c > 0 ? __fadd_rn(__fmul_rn(frequency, (float)c), presence) : 0.0f;
}

// The rare value: one that the row's window tokens raise the count of, or any where b or r is not a normal number.
__device__ __noinline__ float bend(float x, uint32_t word, int extra, float b, float frequency, float presence, float bias) {
    const int c = (int)(word & ~kInPrompt) + extra;
    if (c > 0 || word) x = x > 0.0f ? __fdiv_rn(x, b) : __fmul_rn(x, b);
    return __fadd_rn(x, __fsub_rn(bias, penalty_of(c, frequency, presence)));
}

// Block (chunk of the vocabulary, request, share of its rows): a thread owns the same eight values of every row, so the
// penalties and biases of those are worked out once and stay in its registers, and it knows which of the window's
// tokens are among them (`mine`, one bit a token).  Then the rows stream past, kAdjDepth rows' logits in flight.  No
// thread reads what another writes, so the output may be the input.
// Bound by issue: about 180 instructions for a warp's 256 values where every warp has a seen one.  12 requests of 16 to
// 32 rows over 248320 bf16 logits (451 MB) 97 us, 4.7 TB/s; the same with a division called per seen value 182 us, with
// four rows in flight and 6 blocks of an SM (80 registers) 108 us, with 32 rows a block (fewer prologues, a longer tail)
// 121 us, with 8 rows 100 us.  Rows of an odd length go by single values: 106299 of them 74 us, and 100 us with 4 blocks of
// an SM instead of 8.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kAdjThreads, VEC && sizeof(T) == 4 ? 6 : 8) logits_adjust_kernel(const __grid_constant__ AdjustParams p) {
    // (place + 1) << 32 | value of the last entry of the request's list for each value of the chunk, or 0
    __shared__ __align__(16) unsigned long long s_bias[kAdjChunk];
    __shared__ uint32_t s_mine[2][kAdjThreads];             // window tokens among a thread's values
    __shared__ int s_token[kMaxWindowRows];
    const int tid = threadIdx.x, b = blockIdx.y;
    const int v0 = blockIdx.x * kAdjChunk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // what depends on the request alone, asked for together
    const int first = __ldg(p.row_starts + b), last = __ldg(p.row_starts + b + 1);
    const bool on = p.penalties != nullptr;
    float repetition = 1.0f, frequency = 0.0f, presence = 0.0f;
    if (on) repetition = __ldg(p.penalties + 3 * b), frequency = __ldg(p.penalties + 3 * b + 1), presence = __ldg(p.penalties + 3 * b + 2);
    int state = -1, b0 = 0, b1 = 0;
    if (p.counts) state = p.state_of ? __ldg(p.state_of + b) : b;
    if (p.bias_starts) b0 = __ldg(p.bias_starts + b), b1 = __ldg(p.bias_starts + b + 1);
    if (first < 0 || last < first || last > p.n_rows) return;
    const int rows = last - first;
    if (rows <= (int)blockIdx.z || (p.tokens && rows > kMaxWindowRows)) return;
    if (b0 < 0 || b1 < b0 || b1 > p.n_bias) b0 = b1 = 0;
    const bool counted = state >= 0 && state < p.n_states, windows = on && p.tokens;
    const bool odd = !(fabsf(repetition) > 0x1p-100f && fabsf(repetition) < 0x1p100f);

    auto at = [&](int i) { return VEC ? v0 + tid * kAdjPer + i : v0 + i * kAdjThreads + tid; };
    const bool mine_ok = at(0) < p.vocab;  // of VEC all eight values, of the others the first at least
    const int lane = tid & 31, step = gridDim.z, n_rows = (rows - (int)blockIdx.z + step - 1) / step;
    // The block's n-th row is z + n step.  Its grammar: lane n % 32 holds the index of it, 32 rows at a time.
    auto grammar_at = [&](int n) {
        if (!p.grammar || n >= n_rows) return -1;
        const int r = first + (int)blockIdx.z + n * step, g = p.grammar_of ? __ldg(p.grammar_of + r) : r;
        return g < p.n_grammar ? g : -1;
    };
    int grammars = grammar_at(lane);
    const int64_t in_step = (int64_t)step * p.in_stride, out_step = (int64_t)step * p.out_stride;
    const T* src = static_cast<const T*>(p.logits) + (int64_t)(first + (int)blockIdx.z) * p.in_stride;
    float* dst = p.out + (int64_t)(first + (int)blockIdx.z) * p.out_stride;
    const int64_t n_words = (p.vocab + 31) / 32;
    Eight<T> x[kAdjDepth];
    uint32_t allowed[kAdjDepth];  // bit i (VEC: from bit at(0) % 32 on): value i of the row is allowed
    auto load = [&](int k, int n) {  // row n into place k; called for n = 0, 1, 2, ...
        if (n >= n_rows) return;
        if (VEC) {
            if (mine_ok) x[k].load_whole(src + at(0));
        } else {
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i) x[k].put(i, at(i) < p.vocab ? src[at(i)] : T(0.0f));
        }
        src += in_step;
        if ((n & 31) == 0 && n) grammars = grammar_at(n + lane);
        const int g = __shfl_sync(0xffffffffu, grammars, n & 31);
        allowed[k] = ~0u;
        if (g >= 0) {
            const uint32_t* words = p.grammar + g * n_words;
            if (VEC) {
                if (mine_ok) allowed[k] = __ldg(words + (at(0) >> 5));
            } else {
                allowed[k] = 0u;
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i)
                    if (at(i) < p.vocab) allowed[k] |= (__ldg(words + (at(i) >> 5)) >> (at(i) & 31) & 1u) << i;
            }
        }
    };
#pragma unroll
    for (int k = 0; k < kAdjDepth; ++k) load(k, k);
    const uint32_t* counts = p.counts + (int64_t)max(state, 0) * p.vocab;
    uint32_t word[kAdjPer];
#pragma unroll
    for (int i = 0; i < kAdjPer; ++i) word[i] = 0u;
    if (counted) {
        if (VEC) {
            if (at(0) < p.vocab) load32(word, counts + at(0));
        } else {
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i)
                if (at(i) < p.vocab) word[i] = __ldg(counts + at(i));
        }
    }

    uint64_t mine = 0;
    float bias[kAdjPer];
#pragma unroll
    for (int i = 0; i < kAdjPer; ++i) bias[i] = 0.0f;
    if (windows || b1 > b0 || odd) {
        s_mine[0][tid] = s_mine[1][tid] = 0u;
#pragma unroll
        for (int i = 0; i < kAdjPer / 2; ++i) reinterpret_cast<uint4*>(s_bias)[i * kAdjThreads + tid] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (int j = tid; windows && j < rows; j += kAdjThreads) {
            const int v = __ldg(p.tokens + first + j);
            s_token[j] = v;
            if (v >= v0 && v < min(v0 + kAdjChunk, p.vocab))
                atomicOr(&s_mine[j >> 5][VEC ? (v - v0) / kAdjPer : (v - v0) % kAdjThreads], 1u << (j & 31));
        }
        for (int i = tid; i < b1 - b0; i += kAdjThreads) {
            const int v = __ldg(p.bias_tokens + b0 + i);
            const uint32_t value = __float_as_uint(__ldg(p.bias_values + b0 + i));
            if (v >= v0 && v < v0 + kAdjChunk) atomicMax(&s_bias[v - v0], (unsigned long long)(i + 1) << 32 | value);
        }
        __syncthreads();
        mine = (uint64_t)s_mine[1][tid] << 32 | s_mine[0][tid];
#pragma unroll
        for (int i = 0; i < kAdjPer; ++i) bias[i] = __uint_as_float((uint32_t)s_bias[at(i) - v0]);
    }
    // c and the mark of a value, as its penalty and a bit
    const float inverse = 1.0f / repetition;
    uint32_t seen = 0;
    bool touched = false;
    float shift[kAdjPer];  // - (frequency c + presence) + bias
#pragma unroll
    for (int i = 0; i < kAdjPer; ++i) {
        const int c = (int)(word[i] & ~kInPrompt);
        shift[i] = __fsub_rn(bias[i], penalty_of(c, frequency, presence));
        if (word[i]) seen |= 1u << i;
        touched |= word[i] || bias[i] != 0.0f;
    }

    for (int n0 = 0; n0 < n_rows; n0 += kAdjDepth) {
#pragma unroll
        for (int k = 0; k < kAdjDepth; ++k) {
            if (n0 + k >= n_rows) break;
            float y[8];
            x[k].floats(y);
            const uint32_t bits = VEC ? allowed[k] >> (at(0) & 31) : allowed[k];
            load(k, n0 + k + kAdjDepth);
            uint64_t sees = 0;
            if (mine) {
                const int r = (int)blockIdx.z + (n0 + k) * step;
                sees = mine & (p.mask ? __ldg(p.mask + first + r) : (2ull << r) - 1);
            }
            if (sees || (odd && touched)) {
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i) {
                    int extra = 0;
#pragma unroll 1
                    for (uint64_t rest = sees; rest; rest &= rest - 1) extra += s_token[__ffsll((long long)rest) - 1] == at(i);
                    const uint32_t w = counted && at(i) < p.vocab ? __ldg(counts + at(i)) : 0u;
                    const float bias = __uint_as_float((uint32_t)s_bias[at(i) - v0]);
                    y[i] = bend(y[i], w, extra, repetition, frequency, presence, bias);
                }
            } else if (touched) {
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i) {
                    if (seen >> i & 1) y[i] = repeated(y[i], repetition, inverse);
                    y[i] = __fadd_rn(y[i], shift[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i)
                if (!(bits >> i & 1)) y[i] = -INFINITY;
            if (VEC) {
                if (mine_ok)
                    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + at(0)), "f"(y[0]), "f"(y[1]),
                                 "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                                 : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i)
                    if (at(i) < p.vocab) dst[at(i)] = y[i];
            }
            dst += out_step;
        }
    }
}

template <typename T>
int launch_adjust(const AdjustParams& p, bool vec, cudaStream_t s) {
    // about kAdjRows rows a block, by the mean of the requests' rows
    const int shares = (p.n_rows + p.n_seqs * kAdjRows - 1) / (p.n_seqs * kAdjRows);
    const dim3 grid((unsigned)((p.vocab + kAdjChunk - 1) / kAdjChunk), (unsigned)p.n_seqs, (unsigned)(shares < 65535 ? shares : 65535));
    if (vec) return launch_dependent(logits_adjust_kernel<T, true>, grid, kAdjThreads, 0, s, p);
    return launch_dependent(logits_adjust_kernel<T, false>, grid, kAdjThreads, 0, s, p);
}

// ---------------------------------------------------------------- counts

constexpr int kCountThreads = 256;
constexpr int kCountPer = 4;  // tokens of a thread in flight

struct CountParams {
    const int32_t* tokens;
    const int32_t* starts;
    const int32_t* prompt_lens;
    const int32_t* state_of;
    uint32_t* counts;
    int n_tokens, n_states, vocab, n_lists;
};

__device__ __forceinline__ int list_state(const CountParams& p, int list) {
    const int st = p.state_of ? p.state_of[list] : list;
    return st >= 0 && st < p.n_states ? st : -1;
}

// Rows are cleared 16 bytes a thread; a row need not start or end on 16 bytes.
__global__ void __launch_bounds__(kCountThreads) counts_clear_kernel(const CountParams p) {
    // the adds read the lists as soon as this kernel runs: not before what came before it is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int st = list_state(p, blockIdx.y);
    if (st < 0) return;
    uint32_t* row = p.counts + (int64_t)st * p.vocab;
    const int head = min((int)(-(reinterpret_cast<intptr_t>(row) >> 2) & 3), p.vocab), body = (p.vocab - head) / 4;
    const int i0 = blockIdx.x * kCountThreads + threadIdx.x;
    if (i0 < head) row[i0] = 0u;
    if (i0 < p.vocab - head - 4 * body) row[head + 4 * body + i0] = 0u;
    for (int i = i0; i < body; i += gridDim.x * kCountThreads) reinterpret_cast<uint4*>(row + head)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// A thread's first tokens are on their way before the wait for the cleared rows.  The adds commute, so their order does
// not change the counts.
__global__ void __launch_bounds__(kCountThreads) counts_add_kernel(const CountParams p) {
    const int list = blockIdx.y;
    const int st = list_state(p, list);
    const int a = p.starts[list], e = p.starts[list + 1];
    const bool on = st >= 0 && a >= 0 && a <= e && e <= p.n_tokens;
    const int prompt = p.prompt_lens ? max(p.prompt_lens[list], 0) : 0;
    const int step = gridDim.x * kCountThreads, i0 = a + blockIdx.x * kCountThreads + threadIdx.x;
    int tok[kCountPer];
#pragma unroll
    for (int k = 0; k < kCountPer; ++k) tok[k] = on && i0 + k * step < e ? __ldg(p.tokens + i0 + k * step) : -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!on) return;
    uint32_t* row = p.counts + (int64_t)st * p.vocab;
    auto add = [&](int i, int v) {
        if (v < 0 || v >= p.vocab) return;
        if (i - a < prompt)
            atomicOr(row + v, kInPrompt);
        else
            atomicAdd(row + v, 1u);
    };
#pragma unroll
    for (int k = 0; k < kCountPer; ++k) add(i0 + k * step, tok[k]);
    for (int64_t i = i0 + (int64_t)kCountPer * step; i < e; i += step) add((int)i, p.tokens[i]);
}

}  // namespace
}  // namespace kvq8

extern "C" int logits_adjust(const void* logits, int dtype, int64_t logits_stride, int n_rows, int vocab,
                             const int32_t* row_starts, int n_seqs, const float* penalties, const uint32_t* counts,
                             int n_states, const int32_t* state_of, const int32_t* window_tokens,
                             const uint64_t* window_mask, const int32_t* bias_starts, const int32_t* bias_tokens,
                             const float* bias_values, int n_bias, const uint32_t* grammar, int n_grammar,
                             const int32_t* grammar_of, float* out, int64_t out_stride, kvq8_stream_t stream) {
    using namespace kvq8;
    const int64_t esz = (int64_t)dtype_size(dtype);
    if (!esz || n_rows < 0 || n_seqs < 0 || vocab < 1 || n_bias < 0) return KVQ8_ERR_INVALID_ARG;
    if (n_rows == 0 || n_seqs == 0) return KVQ8_OK;
    if (!logits || !out || !row_starts || logits_stride < vocab || out_stride < vocab) return KVQ8_ERR_INVALID_ARG;
    if ((counts || window_tokens) && !penalties) return KVQ8_ERR_INVALID_ARG;
    if (counts && n_states < 1) return KVQ8_ERR_INVALID_ARG;
    if (window_mask && !window_tokens) return KVQ8_ERR_INVALID_ARG;
    if (bias_starts && n_bias > 0 && (!bias_tokens || !bias_values)) return KVQ8_ERR_INVALID_ARG;
    if (grammar && n_grammar < 1) return KVQ8_ERR_INVALID_ARG;
    // in place: only where an element's input and output are the same bytes
    if (static_cast<const void*>(out) == logits && (dtype != KVQ8_F32 || logits_stride != out_stride)) return KVQ8_ERR_INVALID_ARG;
    if (n_seqs > kMaxSeqs || vocab > (1 << 30) || n_rows > 262140) return KVQ8_ERR_UNSUPPORTED;
    if (!aligned_to(logits, (size_t)esz) || !aligned_to(window_mask, 8)) return KVQ8_ERR_MISALIGNED;
    for (const void* q : {(const void*)row_starts, (const void*)penalties, (const void*)counts, (const void*)state_of,
                          (const void*)window_tokens, (const void*)bias_starts, (const void*)bias_tokens,
                          (const void*)bias_values, (const void*)grammar, (const void*)grammar_of, (const void*)out})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    if (static_cast<const void*>(out) != logits &&
        rows_meet(reinterpret_cast<uintptr_t>(logits), vocab * esz, logits_stride * esz, reinterpret_cast<uintptr_t>(out), vocab * 4ll,
                  out_stride * 4, n_rows))
        return KVQ8_ERR_INVALID_ARG;
    AdjustParams p = {logits, out, logits_stride, out_stride, row_starts, penalties, counts, state_of, window_tokens,
                      window_mask, n_bias > 0 ? bias_starts : nullptr, bias_tokens, bias_values, grammar, grammar_of,
                      n_rows, vocab, n_seqs, n_states, n_bias, n_grammar};
    // eight values an access (16 bytes of logits of 16 bits, else 32) where every row starts on that and holds whole groups
    const bool vec = vocab % 8 == 0 && aligned_to(logits, (size_t)(8 * esz)) && logits_stride % 8 == 0 && aligned_to(out, 32) &&
                     out_stride % 8 == 0 && aligned_to(counts, 32);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == KVQ8_F32) return launch_adjust<float>(p, vec, s);
    if (dtype == KVQ8_F16) return launch_adjust<__half>(p, vec, s);
    return launch_adjust<__nv_bfloat16>(p, vec, s);
}

extern "C" int token_counts(const int32_t* tokens, const int32_t* token_starts, int n_lists, int n_tokens,
                            const int32_t* prompt_lens, const int32_t* state_of, int clear, uint32_t* counts, int n_states,
                            int vocab, kvq8_stream_t stream) {
    using namespace kvq8;
    if (n_lists < 0 || n_tokens < 0 || n_states < 1 || vocab < 1) return KVQ8_ERR_INVALID_ARG;
    if (n_lists == 0) return KVQ8_OK;
    if (!token_starts || !counts || (n_tokens > 0 && !tokens)) return KVQ8_ERR_INVALID_ARG;
    if (n_lists > kMaxSeqs || vocab > (1 << 30) || n_tokens > (1 << 30)) return KVQ8_ERR_UNSUPPORTED;
    for (const void* q : {(const void*)tokens, (const void*)token_starts, (const void*)prompt_lens, (const void*)state_of,
                          (const void*)counts})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    const CountParams p = {tokens, token_starts, prompt_lens, state_of, counts, n_tokens, n_states, vocab, n_lists};
    cudaStream_t s = (cudaStream_t)stream;
    if (clear) {
        const int gx = (vocab / 4 + 4 * kCountThreads - 1) / (4 * kCountThreads) + 1;
        const int rc = launch_dependent(counts_clear_kernel, dim3((unsigned)(gx < 128 ? gx : 128), (unsigned)n_lists), kCountThreads, 0, s, p);
        if (rc != KVQ8_OK) return rc;
    }
    if (n_tokens == 0) return KVQ8_OK;
    const int per = kCountThreads * kCountPer, gx = (n_tokens / n_lists + per - 1) / per + 1;
    const dim3 grid((unsigned)(gx < 64 ? gx : 64), (unsigned)n_lists);
    if (clear) return launch_dependent(counts_add_kernel, grid, kCountThreads, 0, s, p);
    counts_add_kernel<<<grid, kCountThreads, 0, s>>>(p);
    return launch_status();
}

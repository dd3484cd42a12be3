// logits.cu -- logits of a verify step bent by penalties, biases and grammar masks (logits_adjust), and the token
// counts that the penalties read (token_counts).
//
// Row r of request b, value v, with c the times v was generated (counts, plus the window tokens that row r sees)
// and "seen" whether v was generated or stands in the prompt (bit 31 of its count):
//   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   x = x - (frequency * c + presence * [c > 0]);  x = x + bias(v);  x = allowed(v) ? x : -inf
// all in fp32, whatever the type of the logits.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace kvq8 {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjPer = 8;                          // values of one row per thread
constexpr int kAdjChunk = kAdjThreads * kAdjPer;    // vocabulary values per block
constexpr int kAdjRows = kAdjThreads / kMaxWindowRows;  // rows per block: a thread for every (row, window token)
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

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight consecutive values, 16-byte aligned (two loads for fp32).
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(u32_as_h2(w[k]));
        x[2 * k] = f.x, x[2 * k + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = __uint_as_float(w[k] << 16), x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
}

struct Penalty {
    float repetition, frequency, presence;
    bool on;
};

__device__ __forceinline__ float bend(float x, uint32_t word, int extra, const Penalty& q, float bias, bool allowed) {
    const int c = (int)(word & ~kInPrompt) + extra;
    if (q.on) {
        if (c > 0 || (word & kInPrompt)) x = x > 0.0f ? x / q.repetition : x * q.repetition;
        x -= q.frequency * (float)c + (c > 0 ? q.presence : 0.0f);
    }
    x += bias;
    return allowed ? x : -INFINITY;
}

// Block (chunk of the vocabulary, group of kAdjRows rows).  The rows' logits are requested before anything else.
// Counts and the bias table of a request are loaded once for its rows of the group.  A row's window tokens change
// few of its values: the thread of (row, window token j) computes that value from the raw logit before any is
// written (the output may be the input) and writes it after the row's plain values.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kAdjThreads) logits_adjust_kernel(const AdjustParams p) {
    __shared__ int s_bias[kAdjChunk];  // last entry of the request's list for each value of the chunk, or -1
    __shared__ int s_seq[kAdjRows];
    const int tid = threadIdx.x;
    const int r0 = blockIdx.y * kAdjRows, v0 = blockIdx.x * kAdjChunk;
    const T* in = static_cast<const T*>(p.logits);
    auto at = [&](int i) { return VEC ? v0 + tid * kAdjPer + i : v0 + i * kAdjThreads + tid; };

    float x[kAdjRows][kAdjPer];
#pragma unroll
    for (int k = 0; k < kAdjRows; ++k) {
        const bool row_ok = r0 + k < p.n_rows;
        const T* src = in + (int64_t)(r0 + k) * p.in_stride;
        if (VEC) {
            if (row_ok && at(0) < p.vocab) load8(src + at(0), x[k]);
        } else {
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i) x[k][i] = row_ok && at(i) < p.vocab ? to_f32(src[at(i)]) : 0.0f;
        }
    }
    if (tid < kAdjRows) s_seq[tid] = -1;
    __syncthreads();
    for (int b = tid; b < p.n_seqs; b += kAdjThreads) {
        const int a = p.row_starts[b], e = p.row_starts[b + 1];
        if (a < 0 || e > p.n_rows || (p.tokens && e - a > kMaxWindowRows)) continue;
#pragma unroll
        for (int k = 0; k < kAdjRows; ++k)
            if (a <= r0 + k && r0 + k < e) s_seq[k] = b;
    }
    __syncthreads();

    for (int k0 = 0; k0 < kAdjRows;) {  // rows k0 .. k1 - 1 belong to one request
        const int b = s_seq[k0];
        int k1 = k0 + 1;
        while (k1 < kAdjRows && s_seq[k1] == b) ++k1;
        if (b < 0) {
            k0 = k1;
            continue;
        }
        const int first = p.row_starts[b], rows = p.row_starts[b + 1] - first;
        Penalty q = {1.0f, 0.0f, 0.0f, p.penalties != nullptr};
        if (q.on) q.repetition = p.penalties[3 * b], q.frequency = p.penalties[3 * b + 1], q.presence = p.penalties[3 * b + 2];
        int state = p.counts ? (p.state_of ? p.state_of[b] : b) : -1;
        if (state < 0 || state >= p.n_states) state = -1;
        const uint32_t* counts = p.counts + (int64_t)max(state, 0) * p.vocab;
        uint32_t word[kAdjPer];
#pragma unroll
        for (int i = 0; i < kAdjPer; ++i) word[i] = 0u;
        if (q.on && state >= 0) {
            if (VEC) {
                if (at(0) < p.vocab) {
                    const uint4 a = __ldg(reinterpret_cast<const uint4*>(counts + at(0)));
                    const uint4 c = __ldg(reinterpret_cast<const uint4*>(counts + at(0)) + 1);
                    word[0] = a.x, word[1] = a.y, word[2] = a.z, word[3] = a.w;
                    word[4] = c.x, word[5] = c.y, word[6] = c.z, word[7] = c.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i)
                    if (at(i) < p.vocab) word[i] = __ldg(counts + at(i));
            }
        }
        int n_bias = 0, bias0 = 0;
        if (p.bias_starts) {
            bias0 = p.bias_starts[b];
            const int e = p.bias_starts[b + 1];
            if (bias0 >= 0 && e <= p.n_bias && e > bias0) n_bias = e - bias0;
        }
        float bias[kAdjPer];
#pragma unroll
        for (int i = 0; i < kAdjPer; ++i) bias[i] = 0.0f;
        if (n_bias) {
            __syncthreads();  // an earlier request's table has been read
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i) s_bias[i * kAdjThreads + tid] = -1;
            __syncthreads();
            for (int i = tid; i < n_bias; i += kAdjThreads) {
                const int v = __ldg(p.bias_tokens + bias0 + i);
                if (v >= v0 && v < v0 + kAdjChunk) atomicMax(&s_bias[v - v0], i);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kAdjPer; ++i) {
                const int e = s_bias[at(i) - v0];
                if (e >= 0) bias[i] = __ldg(p.bias_values + bias0 + e);
            }
        }
        // this thread's window token: (row kw, token j)
        const int kw = tid / kMaxWindowRows, j = tid % kMaxWindowRows;
        int special = -1;
        float special_x = 0.0f;
        if (q.on && p.tokens && kw >= k0 && kw < k1 && j < rows) {
            const int r = r0 + kw;
            const uint64_t all = rows >= 64 ? ~0ull : (1ull << rows) - 1;
            uint64_t m = p.mask ? p.mask[r] : (2ull << (r - first)) - 1;
            m &= all;
            const int v = p.tokens[first + j];
            if ((m >> j & 1) && v >= v0 && v < min(v0 + kAdjChunk, p.vocab)) {
                int extra = 0, lowest = -1;
                for (uint64_t rest = m; rest; rest &= rest - 1) {
                    const int i = __ffsll((long long)rest) - 1;
                    if (p.tokens[first + i] == v) {
                        if (lowest < 0) lowest = i;
                        ++extra;
                    }
                }
                if (lowest == j) {
                    float bv = 0.0f;
                    if (n_bias && s_bias[v - v0] >= 0) bv = p.bias_values[bias0 + s_bias[v - v0]];
                    bool allowed = true;
                    const int g = p.grammar ? (p.grammar_of ? p.grammar_of[r] : r) : -1;
                    if (g >= 0 && g < p.n_grammar)
                        allowed = p.grammar[(int64_t)g * ((p.vocab + 31) / 32) + (v >> 5)] >> (v & 31) & 1;
                    special = v;
                    special_x = bend(to_f32(in[(int64_t)r * p.in_stride + v]), state >= 0 ? counts[v] : 0u, extra, q, bv, allowed);
                }
            }
        }
        __syncthreads();  // every special value has read its logit
#pragma unroll
        for (int k = 0; k < kAdjRows; ++k) {
            if (k < k0 || k >= k1) continue;
            const int r = r0 + k;
            const int g = p.grammar ? (p.grammar_of ? p.grammar_of[r] : r) : -1;
            const bool masked = g >= 0 && g < p.n_grammar;
            const uint32_t* words = p.grammar + (int64_t)max(g, 0) * ((p.vocab + 31) / 32);
            float* dst = p.out + (int64_t)r * p.out_stride;
            if (VEC) {
                if (at(0) < p.vocab) {
                    const uint32_t bits = masked ? __ldg(words + (at(0) >> 5)) >> (at(0) & 31) : 0xffu;
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = bend(x[k][i], word[i], 0, q, bias[i], bits >> i & 1);
                    reinterpret_cast<float4*>(dst + at(0))[0] = make_float4(y[0], y[1], y[2], y[3]);
                    reinterpret_cast<float4*>(dst + at(0))[1] = make_float4(y[4], y[5], y[6], y[7]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kAdjPer; ++i) {
                    if (at(i) >= p.vocab) break;
                    const bool allowed = !masked || (__ldg(words + (at(i) >> 5)) >> (at(i) & 31) & 1);
                    dst[at(i)] = bend(x[k][i], word[i], 0, q, bias[i], allowed);
                }
            }
        }
        __syncthreads();  // the plain values are written
        if (special >= 0) p.out[(int64_t)(r0 + kw) * p.out_stride + special] = special_x;
        k0 = k1;
    }
}

template <typename T>
int launch_adjust(const AdjustParams& p, bool vec, cudaStream_t s) {
    const dim3 grid((unsigned)((p.vocab + kAdjChunk - 1) / kAdjChunk), (unsigned)((p.n_rows + kAdjRows - 1) / kAdjRows));
    if (vec)
        logits_adjust_kernel<T, true><<<grid, kAdjThreads, 0, s>>>(p);
    else
        logits_adjust_kernel<T, false><<<grid, kAdjThreads, 0, s>>>(p);
    return launch_status();
}

// ---------------------------------------------------------------- counts

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

__global__ void __launch_bounds__(256) counts_clear_kernel(const CountParams p) {
    const int st = list_state(p, blockIdx.y);
    if (st < 0) return;
    for (int v = blockIdx.x * 256 + threadIdx.x; v < p.vocab; v += gridDim.x * 256) p.counts[(int64_t)st * p.vocab + v] = 0u;
}

__global__ void __launch_bounds__(256) counts_add_kernel(const CountParams p) {
    const int list = blockIdx.y;
    const int st = list_state(p, list);
    const int a = p.starts[list], e = p.starts[list + 1];
    if (st < 0 || a < 0 || e > p.n_tokens) return;
    const int prompt = a + (p.prompt_lens ? max(p.prompt_lens[list], 0) : 0);
    uint32_t* row = p.counts + (int64_t)st * p.vocab;
    for (int i = a + blockIdx.x * 256 + threadIdx.x; i < e; i += gridDim.x * 256) {
        const int v = p.tokens[i];
        if (v < 0 || v >= p.vocab) continue;
        if (i < prompt)
            atomicOr(row + v, kInPrompt);
        else
            atomicAdd(row + v, 1u);
    }
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
    if (n_seqs > kMaxSeqs || vocab > (1 << 30) || n_rows > kAdjRows * 65535) return KVQ8_ERR_UNSUPPORTED;
    if (!aligned_to(logits, (size_t)esz) || !aligned_to(window_mask, 8)) return KVQ8_ERR_MISALIGNED;
    for (const void* q : {(const void*)row_starts, (const void*)penalties, (const void*)counts, (const void*)state_of,
                          (const void*)window_tokens, (const void*)bias_starts, (const void*)bias_tokens,
                          (const void*)bias_values, (const void*)grammar, (const void*)grammar_of, (const void*)out})
        if (!aligned_to(q, 4)) return KVQ8_ERR_MISALIGNED;
    AdjustParams p = {logits, out, logits_stride, out_stride, row_starts, penalties, counts, state_of, window_tokens,
                      window_mask, n_bias > 0 ? bias_starts : nullptr, bias_tokens, bias_values, grammar, grammar_of,
                      n_rows, vocab, n_seqs, n_states, n_bias, n_grammar};
    // eight-value accesses where every row starts on 16 bytes (logits, counts, output) and rows hold whole groups
    const bool vec = vocab % 8 == 0 && aligned16(logits) && aligned16(out) && (logits_stride * esz) % 16 == 0 &&
                     out_stride % 4 == 0 && (!counts || aligned16(counts));
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
        const int gx = (vocab + 2047) / 2048;
        counts_clear_kernel<<<dim3((unsigned)(gx < 128 ? gx : 128), (unsigned)n_lists), 256, 0, s>>>(p);
        const int rc = launch_status();
        if (rc != KVQ8_OK) return rc;
    }
    if (n_tokens == 0) return KVQ8_OK;
    const int gx = (n_tokens / n_lists + 1023) / 1024 + 1;
    counts_add_kernel<<<dim3((unsigned)(gx < 64 ? gx : 64), (unsigned)n_lists), 256, 0, s>>>(p);
    return launch_status();
}

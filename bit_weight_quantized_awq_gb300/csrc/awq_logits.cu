// awq_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits, in one pass over them:
//   x = x > 0 ? x / rep : x * rep   (token known; by 1 / rep),  x -= freq * count,
//   x -= pres (count > 0),  x += bias,  -inf where the grammar's bit is 0.
//
// Bound: every logit is read and written once (HBM); a row's history has a few
// thousand tokens against a hundred thousand logits. A CTA owns a range of kRange
// vocabulary entries (rounded up to fill the GPU) and a run of rows. It counts the tokens of the row's
// history that fall into its range in shared memory (a counter and a touched bit
// an entry), then takes the logits, fetched a row ahead, 16 bytes at a time; only
// pieces with a touched or biased entry look further. Consecutive rows of one request -- the
// nodes of a drafted tree -- share the counts: only the tokens of the row's own
// path are added before and taken back after it. Counts are whole numbers, so the
// atomics' order does not matter.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kRange = 8192;              // vocabulary entries of a CTA
constexpr int kBitmap = kRange / 32 + 4;  // words of a bitmap of the range: one to spare, and 16-byte pieces
constexpr int kSmemWords = 2 * kRange + 2 * kBitmap;
constexpr unsigned kPrompt = 1u << 31;    // counter: in the prompt; below it the generated count

struct LogitsParams {
    awq_logits_t a;
    unsigned int *status;
    int64_t grammar_words;
    int rows_per_cta;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// `count` (at most 8) bits from bit position `at` of a shared bitmap with a spare word at its end
__device__ __forceinline__ unsigned bits_at(const unsigned *map, int at, int count)
{
    const int w = at >> 5;
    return __funnelshift_r(map[w], map[w + 1], at & 31) & ((1u << count) - 1);
}

// CTAs an SM has room for: a row of 16 or 32 KB is on its way to each
template <typename T>
constexpr int kPerSm = sizeof(T) == 4 ? 2 : 3;

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm<T>)
process_logits_kernel(const __grid_constant__ LogitsParams p)
{
    constexpr int kVec = 16 / sizeof(T);
    constexpr int kHeld = kRange / (kThreads * kVec);   // 16-byte pieces of a row that a thread holds
    constexpr unsigned kAll = (1u << kVec) - 1;
    constexpr int kStep = kThreads * kVec;              // entries between a thread's pieces: whole words of bits
    static_assert(kHeld * kVec == 32 && kStep % 32 == 0, "the grammar's bits of a thread's pieces fill a word");
    extern __shared__ unsigned smem[];
    unsigned *counts = smem;                       // [kRange]
    unsigned *touched = counts + kRange;           // [kBitmap]
    unsigned *biased = touched + kBitmap;          // [kBitmap]
    float *bias = reinterpret_cast<float *>(biased + kBitmap);   // [kRange], set where the bit is
    const awq_logits_t &a = p.a;
    const int tid = threadIdx.x;
    const int64_t v0 = (int64_t)blockIdx.x * kRange;
    const int range = (int)min((int64_t)kRange, a.vocab - v0);
    const int64_t r_lo = (int64_t)blockIdx.y * p.rows_per_cta;
    const int64_t r_hi = min(r_lo + p.rows_per_cta, a.rows);
    unsigned bad = 0;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    auto count_token = [&](int token, unsigned add) {
        const int at = token - (int)v0;
        if (at < 0 || at >= range) {
            if (token >= (int)a.vocab) bad |= kStatusBadIndex;
            return;
        }
        if (add == kPrompt) atomicOr(counts + at, kPrompt);
        else atomicAdd(counts + at, add);
        atomicOr(touched + (at >> 5), 1u << (at & 31));
    };
    auto clamp_offset = [&](int at, int64_t size) {
        if (at < 0 || at > size) bad |= kStatusBadIndex;
        return (int)min(max((int64_t)at, (int64_t)0), size);
    };

    // A row as it is fetched, a row ahead of its turn: the thread's pieces of its
    // logits, the grammar's bits of all of them in one word, its word of the path,
    // and what is known of its request.
    struct Row {
        const T *in;
        const int32_t *mask;       // the grammar's words from the range's first entry on
        int head, pieces;          // elements before the first 16-byte boundary, whole pieces behind it
        int request, history_lo, history_hi, prompt, bias_lo, bias_hi, first;
        float rep, freq, pres;
        unsigned path, allowed;
        uint4 raw[kHeld];
    };
    auto fetch = [&](int64_t r, Row &row) {
        int64_t b = a.row_request ? a.row_request[r] : r;
        if (b < 0 || b >= a.B) {
            if (a.B > 0 || a.row_request) bad |= kStatusBadIndex;
            b = -1;
        }
        row.path = a.tree_mask && tid < a.mask_words * 32 ? (unsigned)a.tree_mask[r * a.mask_words + (tid >> 5)] : 0u;
        row.mask = nullptr;
        if (a.grammar_mask) {
            const int64_t m = a.grammar_rows ? a.grammar_rows[r] : r;
            if (m >= 0 && m < a.grammar_count) row.mask = a.grammar_mask + m * p.grammar_words + (v0 >> 5);
            else if (m != -1 || !a.grammar_rows) bad |= kStatusBadIndex;
        }
        row.in = static_cast<const T *>(a.logits) + r * a.logits_row_stride + v0;
        const T *out = static_cast<const T *>(a.out) + r * a.out_row_stride + v0;
        // all one by one where input and output do not share their alignment
        const unsigned mis_in = (unsigned)(reinterpret_cast<uintptr_t>(row.in) / sizeof(T)) % kVec;
        const unsigned mis_out = (unsigned)(reinterpret_cast<uintptr_t>(out) / sizeof(T)) % kVec;
        row.head = mis_in == mis_out ? min(range, (int)((kVec - mis_in) % kVec)) : range;
        row.pieces = (range - row.head) / kVec;
        row.allowed = ~0u;
        const int at = row.head + tid * kVec;      // the thread's first piece; the others kStep further on each
        const uint4 *piece = reinterpret_cast<const uint4 *>(row.in + at);
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            if (tid + u * kThreads < row.pieces) row.raw[u] = __ldcs(piece + u * kThreads);
        if (row.mask) {
            row.allowed = 0;
            const int32_t *w = row.mask + (at >> 5);
            const bool crosses = (at & 31) + kVec > 32;
#pragma unroll
            for (int u = 0; u < kHeld; ++u)
                if (tid + u * kThreads < row.pieces) {
                    const unsigned lo = (unsigned)w[u * (kStep / 32)], hi = crosses ? (unsigned)w[u * (kStep / 32) + 1] : 0u;
                    row.allowed |= (__funnelshift_r(lo, hi, at & 31) & kAll) << (u * kVec);
                }
        }
        row.request = (int)b;
        row.rep = b >= 0 && a.repetition ? a.repetition[b] : 1.f;
        row.freq = b >= 0 && a.frequency ? a.frequency[b] : 0.f;
        row.pres = b >= 0 && a.presence ? a.presence[b] : 0.f;
        row.history_lo = row.history_hi = row.prompt = row.bias_lo = row.bias_hi = row.first = 0;
        if (b >= 0 && a.history) {
            row.history_lo = a.history_offsets[b];
            row.history_hi = a.history_offsets[b + 1];
            if (a.prompt_lens) row.prompt = a.prompt_lens[b];
        }
        if (b >= 0 && a.bias_tokens) {
            row.bias_lo = a.bias_offsets[b];
            row.bias_hi = a.bias_offsets[b + 1];
        }
        if (b >= 0 && a.draft_tokens) row.first = a.cu_new[b];
    };

    Row row;
    fetch(r_lo, row);
    int have = -2;                                 // request whose counts are held (-1: a row without one)
    float rep = 1.f, inv = 1.f, freq = 0.f, pres = 0.f;
    bool penal = false, any_bias = false;          // else counts change nothing; no bias in the range
    int64_t first = 0;                             // the request's first drafted token
    int my_token = -1;                             // its token number tid
    for (int64_t r = r_lo; r < r_hi; ++r) {
        const int b = row.request;
        if (b != have) {
            have = b;
            rep = row.rep;
            freq = row.freq;
            pres = row.pres;
            penal = rep != 1.f || freq != 0.f || pres != 0.f;
            inv = 1.f / rep;
            first = row.first;
            my_token = -1;
            if (penal && a.draft_tokens && first + tid >= 0 && first + tid < a.rows) my_token = a.draft_tokens[first + tid];
            int h_lo = 0, h_hi = 0;
            if (penal) {
                h_lo = clamp_offset(row.history_lo, a.history_size);
                h_hi = clamp_offset(row.history_hi, a.history_size);
            }
            const int bias_lo = clamp_offset(row.bias_lo, a.bias_size), bias_hi = clamp_offset(row.bias_hi, a.bias_size);
            // the first tokens are on their way while the counts are cleared
            constexpr int kBatch = 8;
            int token[kBatch];
            auto load = [&](int i0) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) token[u] = i0 + u * kThreads < h_hi ? a.history[i0 + u * kThreads] : -1;
            };
            load(h_lo + tid);
            __syncthreads();
            for (int i = tid; i < (kSmemWords - kRange) / 4; i += kThreads)
                reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            for (int i0 = h_lo + tid; i0 - tid < h_hi; i0 += kThreads * kBatch) {
                int now[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) now[u] = token[u];
                load(i0 + kThreads * kBatch);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    count_token(now[u], i0 + u * kThreads - h_lo < row.prompt ? kPrompt : 1u);
            }
            // the request's biases: the first of a token's entries adds all of them up
            bool mine = false;
            for (int i = bias_lo + tid; i < bias_hi; i += kThreads) {
                const int t = a.bias_tokens[i];
                float sum = a.bias_values[i];
                if (i > bias_lo) {
                    const int before = a.bias_tokens[i - 1];
                    if (before > t) bad |= kStatusBadIndex;
                    if (before == t) continue;
                }
                if (t < 0 || t >= a.vocab) bad |= kStatusBadIndex;
                const int at = t - (int)v0;
                if (at < 0 || at >= range) continue;
                for (int k = i + 1; k < bias_hi && a.bias_tokens[k] == t; ++k) sum += a.bias_values[k];
                bias[at] = sum;
                atomicOr(biased + (at >> 5), 1u << (at & 31));
                mine = true;
            }
            any_bias = __syncthreads_or(mine);
        }
        // the row's own path, `sign` 1 to add and -1 (mod 2^32) to take back: token
        // tid from its register, those a longer path has from memory
        const unsigned word = row.path;
        auto path = [&](unsigned sign) {
            if (!penal || !a.draft_tokens || b < 0) return;
            const int64_t last = a.tree_mask ? a.mask_words * 32 : r - first + 1;
            for (int64_t j = tid; j < last; j += kThreads) {
                const unsigned bits = !a.tree_mask ? ~0u : j == tid ? word : (unsigned)a.tree_mask[r * a.mask_words + (j >> 5)];
                if (!((bits >> (j & 31)) & 1u)) continue;
                if (first + j < 0 || first + j >= a.rows) {
                    bad |= kStatusBadIndex;
                    continue;
                }
                const int token = j == tid ? my_token : a.draft_tokens[first + j];
                if (token >= 0) count_token(token, sign);
            }
        };
        path(1u);
        __syncthreads();

        T *out = static_cast<T *>(a.out) + r * a.out_row_stride + v0;
        // entry `at` of the range: its counts and its bias applied to its logit
        auto value = [&](T raw, int at, bool seen, bool has_bias) -> T {
            float x = to_f<T>(raw);
            if (seen) {
                const unsigned c = counts[at], n = c & ~kPrompt;
                if (c) x *= x > 0.f ? inv : rep;
                if (n) x = fmaf(-freq, (float)n, x) - pres;
            }
            if (has_bias) x += bias[at];
            return from_f<T>(x);
        };
        auto one = [&](int at) {
            const bool allowed = !row.mask || ((row.mask[at >> 5] >> (at & 31)) & 1);
            out[at] = allowed ? value(row.in[at], at, bits_at(touched, at, 1), bits_at(biased, at, 1)) : from_f<T>(-INFINITY);
        };
        for (int at = tid; at < row.head; at += kThreads) one(at);
        for (int at = row.head + row.pieces * kVec + tid; at < range; at += kThreads) one(at);
        const int at0 = row.head + tid * kVec;
        const unsigned *seen0 = touched + (at0 >> 5), *bias0 = biased + (at0 >> 5);
        uint4 *to = reinterpret_cast<uint4 *>(out + at0);
#pragma unroll
        for (int u = 0; u < kHeld; ++u) {
            if (tid + u * kThreads >= row.pieces) break;
            const int at = at0 + u * kStep, w = u * (kStep / 32);
            const unsigned t = __funnelshift_r(seen0[w], seen0[w + 1], at0 & 31) & kAll;
            const unsigned bi = any_bias ? __funnelshift_r(bias0[w], bias0[w + 1], at0 & 31) & kAll : 0u;
            const unsigned ok = (row.allowed >> (u * kVec)) & kAll;
            T v[kVec];
            *reinterpret_cast<uint4 *>(v) = row.raw[u];
            if ((t | bi) & ok) {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (((t | bi) >> e) & 1u) v[e] = value(v[e], at + e, (t >> e) & 1u, (bi >> e) & 1u);
            }
            if (ok != kAll) {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (!((ok >> e) & 1)) v[e] = from_f<T>(-INFINITY);
            }
            __stcs(to + u * kThreads, *reinterpret_cast<uint4 *>(v));
        }
        if (r + 1 < r_hi) {
            fetch(r + 1, row);      // under way while the threads meet and the path is taken back
            __syncthreads();
            if (row.request == have) path(0xFFFFFFFFu);
        }
    }
    if (bad) raise_status(p.status, bad);
}

template <typename T>
cudaError_t launch(const awq_logits_t &a, cudaStream_t stream)
{
    LogitsParams p{};
    p.a = a;
    p.status = device_status_word();
    p.grammar_words = (a.vocab + 31) / 32;
    const int64_t ranges = (a.vocab + kRange - 1) / kRange;
    // runs of rows, so long that one wave of CTAs does all of them
    const int64_t want = std::max<int64_t>(1, 152 * kPerSm<T> / ranges);
    p.rows_per_cta = (int)std::max<int64_t>((a.rows + want - 1) / want, (a.rows + 65534) / 65535);
    const size_t smem = kSmemWords * sizeof(unsigned);
    cudaError_t e = cudaFuncSetAttribute(process_logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ranges, (unsigned)((a.rows + p.rows_per_cta - 1) / p.rows_per_cta));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, process_logits_kernel<T>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

cudaError_t launch_process_logits(const awq_logits_t &a, cudaStream_t stream)
{
    if (a.dtype == AWQ_F16) return launch<__half>(a, stream);
    if (a.dtype == AWQ_BF16) return launch<__nv_bfloat16>(a, stream);
    return launch<float>(a, stream);
}

} // namespace awq

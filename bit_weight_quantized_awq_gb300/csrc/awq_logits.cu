// awq_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits, in one pass over them:
//   x = x > 0 ? x / rep : x * rep   (token known),  x -= freq * count,
//   x -= pres (count > 0),  x += bias,  -inf where the grammar's bit is 0.
//
// Bound: every logit is read and written once (HBM); a row's history has a few
// thousand tokens against a hundred thousand logits. A CTA owns a range of kRange
// vocabulary entries (rounded up to fill the GPU) and a run of rows. It counts the tokens of the row's
// history that fall into its range in shared memory (a counter and a touched bit
// an entry), then streams the logits: 16 bytes at a time, and only pieces with a
// touched or biased entry look further. Consecutive rows of one request -- the
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
constexpr int kWords = kRange / 32;
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

template <typename T>
__global__ void __launch_bounds__(kThreads)
process_logits_kernel(const __grid_constant__ LogitsParams p)
{
    constexpr int kVec = 16 / sizeof(T);
    extern __shared__ unsigned smem[];
    unsigned *counts = smem;                       // [kRange]
    unsigned *touched = counts + kRange;           // [kWords + 1]
    unsigned *biased = touched + kWords + 1;       // [kWords + 1]
    const awq_logits_t &a = p.a;
    const int tid = threadIdx.x;
    const int64_t v0 = (int64_t)blockIdx.x * kRange;
    const int range = (int)min((int64_t)kRange, a.vocab - v0);
    const int64_t r_lo = (int64_t)blockIdx.y * p.rows_per_cta;
    const int64_t r_hi = min(r_lo + p.rows_per_cta, a.rows);
    unsigned bad = 0;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    auto count_token = [&](int64_t token, unsigned add) {
        const int64_t at = token - v0;
        if (at < 0 || at >= range) {
            if (token >= a.vocab) bad |= kStatusBadIndex;
            return;
        }
        if (add == kPrompt) atomicOr(counts + at, kPrompt);
        else atomicAdd(counts + at, add);
        atomicOr(touched + (at >> 5), 1u << (at & 31));
    };

    auto clamp_offset = [&](int64_t at, int64_t size) {
        if (at < 0 || at > size) bad |= kStatusBadIndex;
        return min(max(at, (int64_t)0), size);
    };

    int64_t have = -2;                             // request whose counts are held (-1: a row without one)
    for (int64_t r = r_lo; r < r_hi; ++r) {
        int64_t b = a.row_request ? a.row_request[r] : r;
        if (b < 0 || b >= a.B) {
            if (a.B > 0 || a.row_request) bad |= kStatusBadIndex;
            b = -1;
        }
        const float rep = b >= 0 && a.repetition ? a.repetition[b] : 1.f;
        const float freq = b >= 0 && a.frequency ? a.frequency[b] : 0.f;
        const float pres = b >= 0 && a.presence ? a.presence[b] : 0.f;
        const bool penal = rep != 1.f || freq != 0.f || pres != 0.f;   // else counts change nothing
        int bias_lo = 0, bias_hi = 0;
        if (b >= 0 && a.bias_tokens) {
            bias_lo = (int)clamp_offset(a.bias_offsets[b], a.bias_size);
            bias_hi = (int)clamp_offset(a.bias_offsets[b + 1], a.bias_size);
        }
        if (b != have) {
            have = b;
            __syncthreads();
            for (int i = tid; i < kRange + 2 * kWords + 2; i += kThreads) smem[i] = 0;
            __syncthreads();
            if (penal && a.history) {
                const int64_t h_lo = clamp_offset(a.history_offsets[b], a.history_size);
                const int64_t h_hi = clamp_offset(a.history_offsets[b + 1], a.history_size);
                const int64_t prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
                for (int64_t i = h_lo + tid; i < h_hi; i += kThreads)
                    count_token(a.history[i], i - h_lo < prompt ? kPrompt : 1u);
            }
            // the request's biases: entries of the range are marked
            for (int i = bias_lo + tid; i < bias_hi; i += kThreads) {
                const int64_t token = a.bias_tokens[i];
                if (i > bias_lo && a.bias_tokens[i - 1] > token) bad |= kStatusBadIndex;
                if (token < 0 || token >= a.vocab) bad |= kStatusBadIndex;
                const int64_t at = token - v0;
                if (at >= 0 && at < range) atomicOr(biased + (at >> 5), 1u << (at & 31));
            }
        }
        // the row's own path, `sign` 1 to add and -1 (mod 2^32) to take back
        const int64_t first = b >= 0 && a.draft_tokens ? a.cu_new[b] : 0;
        auto path = [&](unsigned sign) {
            if (!penal || !a.draft_tokens || b < 0) return;
            const int64_t last = a.tree_mask ? a.mask_words * 32 : r - first + 1;
            for (int64_t j = tid; j < last; j += kThreads) {
                if (a.tree_mask && !((a.tree_mask[r * a.mask_words + (j >> 5)] >> (j & 31)) & 1)) continue;
                if (first + j < 0 || first + j >= a.rows) {
                    bad |= kStatusBadIndex;
                    continue;
                }
                const int64_t token = a.draft_tokens[first + j];
                if (token >= 0) count_token(token, sign);
            }
        };
        path(1u);
        __syncthreads();

        const int32_t *mask = nullptr;
        if (a.grammar_mask) {
            const int64_t m = a.grammar_rows ? a.grammar_rows[r] : r;
            if (m >= 0 && m < a.grammar_count) mask = a.grammar_mask + m * p.grammar_words;
            else if (m != -1 || !a.grammar_rows) bad |= kStatusBadIndex;
        }
        const T *in = static_cast<const T *>(a.logits) + r * a.logits_row_stride + v0;
        T *out = static_cast<T *>(a.out) + r * a.out_row_stride + v0;

        // the value of entry `at` of the range from its logit; `seen`: it has
        // counts, `bias`: it is in the bias list
        auto value = [&](T raw, int at, bool seen, bool bias, bool allowed) -> T {
            float x = to_f<T>(raw);
            if (seen) {
                const unsigned c = counts[at];
                if (c) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
                if (c & ~kPrompt) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)(c & ~kPrompt))), pres);
            }
            if (bias) {
                const int token = (int)(v0 + at);
                int lo = bias_lo, hi = bias_hi;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (a.bias_tokens[mid] < token) lo = mid + 1;
                    else hi = mid;
                }
                float sum = 0.f;
                for (; lo < bias_hi && a.bias_tokens[lo] == token; ++lo) sum += a.bias_values[lo];
                x += sum;
            }
            return allowed ? from_f<T>(x) : from_f<T>(-INFINITY);
        };
        auto one = [&](int at) {
            const int64_t v = v0 + at;
            const bool allowed = !mask || ((mask[v >> 5] >> (v & 31)) & 1);
            out[at] = value(in[at], at, bits_at(touched, at, 1), bits_at(biased, at, 1), allowed);
        };
        // elements before the first 16-byte boundary, whole pieces, the rest; all
        // one by one where input and output do not share their alignment
        const int mis_in = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kVec);
        const int mis_out = (int)((reinterpret_cast<uintptr_t>(out) / sizeof(T)) % kVec);
        const int head = mis_in == mis_out ? min(range, (kVec - mis_in) % kVec) : range;
        const int pieces = (range - head) / kVec;
        for (int at = tid; at < head; at += kThreads) one(at);
        for (int at = head + pieces * kVec + tid; at < range; at += kThreads) one(at);
        constexpr int kAhead = 4;
        for (int i0 = tid; i0 < pieces; i0 += kThreads * kAhead) {
            uint4 raw[kAhead];
            unsigned allowed[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kThreads;
                allowed[u] = (1u << kVec) - 1;
                if (i >= pieces) continue;
                raw[u] = *reinterpret_cast<const uint4 *>(in + head + i * kVec);
                if (mask) {
                    const int64_t v = v0 + head + i * kVec;
                    const unsigned lo = (unsigned)mask[v >> 5];
                    const unsigned hi = (v & 31) + kVec > 32 ? (unsigned)mask[(v >> 5) + 1] : 0u;
                    allowed[u] &= __funnelshift_r(lo, hi, v & 31);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kThreads;
                if (i >= pieces) continue;
                const int at = head + i * kVec;
                const unsigned t = bits_at(touched, at, kVec), bi = bits_at(biased, at, kVec);
                T v[kVec];
                *reinterpret_cast<uint4 *>(v) = raw[u];
                if (t | bi) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        v[e] = value(v[e], at + e, (t >> e) & 1, (bi >> e) & 1, (allowed[u] >> e) & 1);
                } else if (allowed[u] != (1u << kVec) - 1) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (!((allowed[u] >> e) & 1)) v[e] = from_f<T>(-INFINITY);
                }
                *reinterpret_cast<uint4 *>(out + at) = *reinterpret_cast<uint4 *>(v);
            }
        }
        __syncthreads();
        if (r + 1 < r_hi) path(0xFFFFFFFFu);
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
    // runs of rows: enough CTAs to fill the GPU several times over
    const int64_t want = std::max<int64_t>(1, 152 * 16 / ranges);
    p.rows_per_cta = (int)std::max<int64_t>(std::max<int64_t>(1, a.rows / want), (a.rows + 65534) / 65535);
    const size_t smem = (kRange + 2 * kWords + 2) * sizeof(unsigned);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, process_logits_kernel<T>, p);
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

// awq_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits, in one pass over them:
//   x = x > 0 ? x / rep : x * rep   (token known),  x -= freq * count,
//   x -= pres (count > 0),  x += bias,  -inf where the grammar's bit is 0.
//
// Bound: every logit is read and written once (HBM); a row's history has a few
// thousand tokens against a hundred thousand logits, but most of them are the
// frequent tokens, which lie close together. A CTA owns a range of vocabulary
// entries and a run of rows. Eight warps count the tokens of a request's history
// that fall into the range in shared memory, and who meets an entry first lists it;
// then, row by row, the listed entries are changed, an entry a thread, so that their number
// alone counts and not how they crowd, and 16 bytes at a time are masked and
// stored. A ninth warp brings the rows in, two ahead: logits by bulk copies, and
// beside them whatever the others would have to wait for -- grammar words, path
// words, the request's settings. (With the change made as the logits stream by,
// nearly every warp walked through the few entries of its pieces: 92 us for 580
// rows of 100,000 fp16 logits. With every warp fetching for itself a row ahead, a
// third of the time went into waiting for one conditional load after the other:
// 67 us.) Consecutive rows of one request -- the nodes of a drafted tree -- share
// the counts: only the tokens in which the rows' paths differ are added or taken
// back. Counts are whole numbers, so the atomics' order does not matter.
// Measured: 64 rows of 131072 fp32 logits, histories of up to 4000 tokens: 28 us (13
// without a history; a plain copy takes 14); 580 rows of 100000 bf16 logits of 16
// requests' trees: 53 us, 65% of the copy bandwidth; one row of 32000: 5.6 us.
#include <algorithm>
#include <map>
#include <mutex>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;             // of the eight working warps
// vocabulary entries of a CTA: 16 KB of a row
template <typename T>
constexpr int kRange = 16384 / sizeof(T);
// A counter: in the prompt, in the list of the entries met, and the generated count.
constexpr unsigned kPrompt = 1u << 31, kListed = 1u << 30, kCount = kListed - 1;
// Up to this many tokens of a lane are counted one by one, more of them all at once: 64
// rows of 131072 fp32 logits with histories of up to 4,000 tokens took 27 us so (28 since
// they are divided by the penalty); 30 us all one by one, where a third of the tokens
// fell into one range; with the tokens
// spread evenly 20 us, and 23 all at once.
constexpr int kTurns = 4;
constexpr int kPairs = 2;                 // biases a thread keeps

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

// -inf where a bit of `ok` is 0: two 16-bit values or one fp32 a word
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 v, unsigned ok)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
            if (!((ok >> i) & 1u)) w[i] = 0xFF800000u;
        } else {
            constexpr uint32_t inf = std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
            // bits 2 i and 2 i + 1 at bits 0 and 16, each spread over its half
            const uint32_t keep = (((ok | ok << 15) >> (2 * i)) & 0x00010001u) * 0xFFFFu;
            w[i] = (w[i] & keep) | (inf & ~keep);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kStages = 3;
constexpr int kPathWords = 8;             // words of a path that come with the row: a token a thread

// What comes with a row beside its logits.
template <typename T>
struct RowInfo {
    int request;                          // -1: none
    float rep, freq, pres;
    int history_lo, history_hi, prompt, bias_lo, bias_hi, first;
    int masked;                           // has a grammar mask
    unsigned path[kPathWords];
    unsigned bits[kRange<T> / 32 + 1];    // the grammar's bits of the range
};

// shared memory: the rows' logits, each behind one spare piece and with one after
// it; the counts; a bitmap of the entries with a bias; the list of the entries met;
// what comes with the rows
template <typename T>
constexpr size_t kSmem = kStages * (kRange<T> * sizeof(T) + 32) +
                         (kRange<T> + kRange<T> / 32) * sizeof(unsigned) + kRange<T> * sizeof(uint16_t) +
                         kStages * sizeof(RowInfo<T>);

// CTAs an SM has room for: two rows of 16 KB are on their way to each
template <typename T>
constexpr int kPerSm = sizeof(T) == 4 ? 3 : 2;

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, kPerSm<T>)
process_logits_kernel(const __grid_constant__ LogitsParams p)
{
    constexpr int kVec = 16 / sizeof(T);
    constexpr int kRange = awq::kRange<T>, kBitmap = kRange / 32, kStage = kRange + 2 * kVec;
    constexpr int kHeld = kRange / (kThreads * kVec);   // 16-byte pieces of a row a thread
    constexpr unsigned kAll = (1u << kVec) - 1;
    constexpr int kStep = kThreads * kVec;              // entries between a thread's pieces: whole words of bits
    static_assert(kStep % 32 == 0 && kBitmap <= kThreads, "words of bits");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int listed;
    T *stage = reinterpret_cast<T *>(smem);        // [kStages][kStage]
    unsigned *counts = reinterpret_cast<unsigned *>(stage + kStages * kStage);   // [kRange]
    unsigned *biased = counts + kRange;            // [kBitmap]
    uint16_t *list = reinterpret_cast<uint16_t *>(biased + kBitmap);   // [kRange]
    RowInfo<T> *infos = reinterpret_cast<RowInfo<T> *>(list + kRange);  // [kStages]
    const awq_logits_t &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t v0 = (int64_t)blockIdx.x * kRange;
    const int range = (int)min((int64_t)kRange, a.vocab - v0);
    const int64_t r_lo = (int64_t)blockIdx.y * p.rows_per_cta;
    const int64_t r_hi = min(r_lo + p.rows_per_cta, a.rows);
    unsigned bad = 0;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 2);                // the copy's issue, and the rest
            ptx::mbar_init(ptx::smem_addr(empty + i), kThreads / 32);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    // Where a row's logits of the range lie: elements before the first 16-byte
    // boundary, then whole pieces. All one by one (no pieces) where input and output
    // do not share their alignment.
    auto split = [&](int64_t r, const T *&in, T *&out, int &head, int &pieces) {
        in = static_cast<const T *>(a.logits) + r * a.logits_row_stride + v0;
        out = static_cast<T *>(a.out) + r * a.out_row_stride + v0;
        const unsigned mis_in = (unsigned)(reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kVec;
        const unsigned mis_out = (unsigned)(reinterpret_cast<uintptr_t>(out) / sizeof(T)) % kVec;
        head = mis_in == mis_out ? min(range, (int)((kVec - mis_in) % kVec)) : range;
        pieces = (range - head) / kVec;
    };
    // Entry 0 of a row in its stage: the first piece is on a boundary, one piece in.
    auto entry0 = [&](int s, int head, int pieces) { return stage + s * kStage + kVec - (pieces > 0 ? head : 0); };
    // element number i of those outside the pieces
    auto outside = [&](int i, int head, int pieces) { return i < head ? i : i + pieces * kVec; };

    if (tid >= kThreads) {
        // ------------------------------------------------------------ the rows' way in
        // What a row needs of its request is one word a lane, so that it takes one
        // wait; and the two indices it starts from are asked for a row earlier.
        const int32_t *words = nullptr;
        switch (lane) {
        case 0: words = reinterpret_cast<const int32_t *>(a.repetition); break;
        case 1: words = reinterpret_cast<const int32_t *>(a.frequency); break;
        case 2: words = reinterpret_cast<const int32_t *>(a.presence); break;
        case 3: words = a.history ? a.history_offsets : nullptr; break;
        case 4: words = a.history ? a.history_offsets + 1 : nullptr; break;
        case 5: words = a.history ? a.prompt_lens : nullptr; break;
        case 6: words = a.bias_tokens ? a.bias_offsets : nullptr; break;
        case 7: words = a.bias_tokens ? a.bias_offsets + 1 : nullptr; break;
        case 8: words = a.draft_tokens ? a.cu_new : nullptr; break;
        }
        const int none = lane == 0 ? __float_as_int(1.f) : 0;
        int64_t request = a.row_request ? a.row_request[r_lo] : r_lo;
        int64_t mask_row = a.grammar_rows ? a.grammar_rows[r_lo] : r_lo;
        bool ok = true;
        int64_t r = r_lo;
        for (; r < r_hi; ++r) {
            const int n = (int)(r - r_lo), s = n % kStages;
            ok = ptx::mbar_wait_bounded(ptx::smem_addr(empty + s), ((n / kStages) & 1) ^ 1, nullptr, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const T *in;
            T *out;
            int head, pieces;
            split(r, in, out, head, pieces);
            T *at0 = entry0(s, head, pieces);
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(ptx::smem_addr(full + s), (uint32_t)pieces * 16);
                if (pieces > 0)
                    ptx::bulk_load(ptx::smem_addr(at0 + head), in + head, (uint32_t)pieces * 16, ptx::smem_addr(full + s));
            }
            __syncwarp();
            int64_t b = request, m = a.grammar_mask ? mask_row : -1;
            if (r + 1 < r_hi) {
                request = a.row_request ? a.row_request[r + 1] : r + 1;
                mask_row = a.grammar_rows ? a.grammar_rows[r + 1] : r + 1;
            }
            if (b < 0 || b >= a.B) {
                if ((a.B > 0 || a.row_request) && (b != -1 || !a.row_request)) bad |= kStatusBadIndex;
                b = -1;
            }
            if (m < 0 || m >= a.grammar_count) {
                if (a.grammar_mask && (m != -1 || !a.grammar_rows)) bad |= kStatusBadIndex;
                m = -1;
            }
            RowInfo<T> &info = infos[s];
            int word = none;
            unsigned path = 0, bits[kBitmap / 32 + 1];
            T edge{};
            const int edges = range - pieces * kVec;
            if (words && b >= 0) word = words[b];
            if (a.tree_mask && lane < min((int64_t)kPathWords, a.mask_words)) path = (unsigned)a.tree_mask[r * a.mask_words + lane];
            if (lane < edges) edge = in[outside(lane, head, pieces)];
            const int32_t *grammar = a.grammar_mask + m * p.grammar_words + (v0 >> 5);
            const int have_words = m < 0 ? 0 : (range + 31) / 32;
#pragma unroll
            for (int i = 0; i < kBitmap / 32 + 1; ++i)
                if (lane + 32 * i < have_words) bits[i] = (unsigned)grammar[lane + 32 * i];
            // ---- all of it asked for; now put away
            if (lane < 9) (&info.request)[1 + lane] = word;
            if (lane == 9) info.request = (int)b;
            if (lane == 10) info.masked = m >= 0;
            if (lane < kPathWords) info.path[lane] = path;
#pragma unroll
            for (int i = 0; i < kBitmap / 32 + 1; ++i)
                if (lane + 32 * i < have_words) info.bits[lane + 32 * i] = bits[i];
            if (lane < edges) at0[outside(lane, head, pieces)] = edge;
            for (int i = lane + 32; i < edges; i += 32) at0[outside(i, head, pieces)] = in[outside(i, head, pieces)];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(full + s));
        }
        if (!ok) {
            // the copies on their way land before the shared memory goes
            for (int64_t i = max(r_lo, r - kStages); i < r; ++i)
                ptx::mbar_wait_bounded(ptx::smem_addr(full + (i - r_lo) % kStages), ((i - r_lo) / kStages) & 1, nullptr, nullptr);
        }
        if (bad) raise_status(p.status, bad);
        return;
    }

    // ---------------------------------------------------------------- counts, changes, output
    // Counts a token at an entry of the range. Who meets an entry first lists it; its
    // mark stays when the count goes back to zero, so that none is listed twice.
    auto enlist = [&](int at) {
        atomicOr(counts + at, kListed);
        list[atomicAdd(&listed, 1)] = (uint16_t)at;
    };
    auto count_at = [&](int at, unsigned add) {
        const unsigned was = add == kPrompt ? atomicOr(counts + at, kPrompt) : atomicAdd(counts + at, add);
        if (was == 0) enlist(at);
    };
    auto clamp_offset = [&](int at, int64_t size) {
        if (at < 0 || at > size) bad |= kStatusBadIndex;
        return (int)min(max((int64_t)at, (int64_t)0), size);
    };
    // The entry in the range that pair i of the request's list begins, given its token
    // and those beside it (-1: none), and the sum of all its pairs; -1 if it begins none.
    auto bias_entry = [&](int i, int token, int before, int after, int end, float &sum) {
        const int at = token - (int)v0;
        if (at < 0 || at >= range || before == token) return -1;
        if (after == token)
            for (int k = i + 1; k < end && a.bias_tokens[k] == token; ++k) sum += a.bias_values[k];
        return at;
    };

    int have = -2;                                 // request whose counts are held
    float rep = 1.f, inv = 1.f, freq = 0.f, pres = 0.f;
    bool penal = false;                            // else counts change nothing
    int my_bias[kPairs], more_lo = 0, more_hi = 0; // the entries of this thread's biases; pairs past the threads'
    float my_sum[kPairs];
    int64_t first = 0;                             // the request's first drafted token
    int my_token = -1;                             // its token number tid
    int64_t held = -1;                             // the row whose path is counted, if any
    unsigned held_word = 0;                        // and this thread's word of it
    for (int64_t r = r_lo; r < r_hi; ++r) {
        const int n = (int)(r - r_lo), s = n % kStages;
        const RowInfo<T> &info = infos[s];
        const bool landed = ptx::mbar_wait_bounded(ptx::smem_addr(full + s), (n / kStages) & 1, nullptr, p.status);
        if (!ptx::named_barrier_and(1, kThreads, landed)) break;
        const int b = info.request;
        if (b != have) {
            have = b;
            rep = info.rep;
            freq = info.freq;
            pres = info.pres;
            penal = rep != 1.f || freq != 0.f || pres != 0.f;
            inv = 1.f / rep;
            first = info.first;
            const int h_lo = penal ? clamp_offset(info.history_lo, a.history_size) : 0;
            const int h_hi = penal ? clamp_offset(info.history_hi, a.history_size) : 0;
            const int bias_lo = clamp_offset(info.bias_lo, a.bias_size);
            const int bias_hi = clamp_offset(info.bias_hi, a.bias_size);
            // the first tokens, the thread's pair of the biases and its drafted token
            // are on their way while the counts are cleared
            constexpr int kBatch = 16, kHalf = kBatch / 2;
            int token[kBatch];
            auto load = [&](int i0, int at0, int at1) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u >= at0 && u < at1) token[u] = i0 + u * kThreads < h_hi ? a.history[i0 + u * kThreads] : -1;
            };
            load(h_lo + tid, 0, kHalf);
            if (h_hi - h_lo > kHalf * kThreads) load(h_lo + tid, kHalf, kBatch);
            int bias_token[kPairs], bias_before[kPairs], bias_after[kPairs];
#pragma unroll
            for (int u = 0; u < kPairs; ++u) {
                const int i = bias_lo + u * kThreads + tid;
                bias_token[u] = bias_before[u] = bias_after[u] = -1;
                if (i < bias_hi) {
                    bias_token[u] = a.bias_tokens[i];
                    my_sum[u] = a.bias_values[i];
                    if (i > bias_lo) bias_before[u] = a.bias_tokens[i - 1];
                    if (i + 1 < bias_hi) bias_after[u] = a.bias_tokens[i + 1];
                }
            }
            my_token = -1;
            if (penal && a.draft_tokens && first + tid >= 0 && first + tid < a.rows) my_token = a.draft_tokens[first + tid];
            held = -1;
            held_word = 0;
            for (int i = tid; i < (kRange + kBitmap) / 4; i += kThreads)
                reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0, 0, 0, 0);
            if (tid == 0) listed = 0;
            ptx::named_barrier(1, kThreads);
            int most = -1;
            for (int i0 = h_lo; i0 < h_hi; i0 += kThreads * kBatch) {
                const bool more = h_hi - i0 > kHalf * kThreads;
                if (i0 > h_lo) {
                    load(i0 + tid, 0, kHalf);
                    if (more) load(i0 + tid, kHalf, kBatch);
                }
                // the thread's tokens in the range
                unsigned mine = 0;
                auto look = [&](int at0, int at1) {
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        if (u >= at0 && u < at1) {
                            most = max(most, token[u]);
                            mine |= ((unsigned)token[u] - (unsigned)v0 < (unsigned)range ? 1u : 0u) << u;
                        }
                };
                look(0, kHalf);
                if (more) look(kHalf, kBatch);
                const int in_prompt = info.prompt - (i0 - h_lo) - tid;    // the thread's token u: u * kThreads < this
                if (__reduce_max_sync(0xFFFFFFFFu, __popc(mine)) > kTurns) {
                    unsigned met = 0;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        if ((mine >> u) & 1u) {
                            unsigned *count = counts + (token[u] - (int)v0);
                            const unsigned was = u * kThreads < in_prompt ? atomicOr(count, kPrompt) : atomicAdd(count, 1u);
                            met |= (was == 0 ? 1u : 0u) << u;
                        }
                    int place = met ? atomicAdd(&listed, __popc(met)) : 0;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        if ((met >> u) & 1u) {
                            const int at = token[u] - (int)v0;
                            atomicOr(counts + at, kListed);
                            list[place++] = (uint16_t)at;
                        }
                } else {
                    // few: one of them a turn, so that a warp takes as many turns as its
                    // busiest lane has tokens; the token is in the L1 cache
                    while (mine) {
                        const int u = __ffs(mine) - 1;
                        mine &= mine - 1;
                        const int at = a.history[i0 + tid + u * kThreads] - (int)v0;
                        if ((unsigned)at < (unsigned)range) count_at(at, u * kThreads < in_prompt ? kPrompt : 1u);
                    }
                }
            }
            if (most >= (int)a.vocab) bad |= kStatusBadIndex;
            // the request's biases: the thread's own pair, and those past the threads'
            auto check = [&](int t, int before) {
                if (t < 0 || before > t || t >= a.vocab) bad |= kStatusBadIndex;
            };
#pragma unroll
            for (int u = 0; u < kPairs; ++u) {
                const int i = bias_lo + u * kThreads + tid;
                my_bias[u] = -1;
                if (i >= bias_hi) continue;
                check(bias_token[u], bias_before[u]);
                const int at = bias_entry(i, bias_token[u], bias_before[u], bias_after[u], bias_hi, my_sum[u]);
                if (at >= 0) atomicOr(biased + (at >> 5), 1u << (at & 31));
                my_bias[u] = at;
            }
            more_lo = bias_lo + kPairs * kThreads;
            more_hi = bias_hi;
            for (int i = more_lo + tid; i < more_hi; i += kThreads) {
                const int t = a.bias_tokens[i], at = t - (int)v0;
                check(t, a.bias_tokens[i - 1]);
                if (at >= 0 && at < range) atomicOr(biased + (at >> 5), 1u << (at & 31));
            }
            ptx::named_barrier(1, kThreads);
        }
        // The row's path in place of the one that is counted: where the two differ.
        // Token tid and its bits are at hand, those a longer path has in memory.
        const unsigned my_word = info.path[tid >> 5];
        if (penal && a.draft_tokens && b >= 0) {
            const int64_t last = a.tree_mask ? a.mask_words * 32 : r - first + 1;
            for (int64_t j = tid; j < last; j += kThreads) {
                bool now, was;
                if (a.tree_mask) {
                    const unsigned w = j == tid ? my_word : (unsigned)a.tree_mask[r * a.mask_words + (j >> 5)];
                    const unsigned h = held < 0 ? 0u : j == tid ? held_word : (unsigned)a.tree_mask[held * a.mask_words + (j >> 5)];
                    now = (w >> (j & 31)) & 1u;
                    was = (h >> (j & 31)) & 1u;
                } else {
                    now = true;
                    was = held >= 0 && j <= held - first;
                }
                if (now == was) continue;
                if (first + j < 0 || first + j >= a.rows) {
                    bad |= kStatusBadIndex;
                    continue;
                }
                const int token = j == tid ? my_token : a.draft_tokens[first + j];
                if (token >= (int)a.vocab) bad |= kStatusBadIndex;
                const int at = token - (int)v0;
                if (at >= 0 && at < range) count_at(at, now ? 1u : 0xFFFFFFFFu);
            }
            held = r;
            held_word = my_word;
        }
        const T *in;
        T *out;
        int head, pieces;
        split(r, in, out, head, pieces);
        T *at0 = entry0(s, head, pieces);
        ptx::named_barrier(1, kThreads);

        // ---- the entries that change
        auto change = [&](int at, float sum) {
            float x = to_f<T>(at0[at]);
            const unsigned c = counts[at], times = c & kCount;
            // Where the result is rounded to 16 bits, times the reciprocal: its rounding is
            // 2^-13 of that one or less. (580 rows of 100000: 60.5 us with divisions; 55 with
            // the reciprocal's remainder taken into account; 64 rows of 131072 fp32: 28, and
            // 27 by the reciprocal.)
            if (c & ~kListed) {
                if constexpr (sizeof(T) == 4) x = x > 0.f ? x / rep : x * rep;
                else x *= x > 0.f ? inv : rep;
            }
            if (times) x = fmaf(-freq, (float)times, x) - pres;
            at0[at] = from_f<T>(x + sum);
        };
        const int entries = listed;
        for (int i = tid; i < entries; i += kThreads) {
            const int at = list[i];
            if (!((biased[at >> 5] >> (at & 31)) & 1u)) change(at, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kPairs; ++u)
            if (my_bias[u] >= 0) change(my_bias[u], my_sum[u]);
        for (int i = more_lo + tid; i < more_hi; i += kThreads) {
            float sum = a.bias_values[i];
            const int token = a.bias_tokens[i];
            const int at = bias_entry(i, token, a.bias_tokens[i - 1], token, more_hi, sum);
            if (at >= 0) change(at, sum);
        }
        ptx::named_barrier(1, kThreads);

        // ---- masked and stored
        const bool masks = info.masked != 0;
        const int at1 = head + tid * kVec, shift = at1 & 31;      // the thread's first piece
        const unsigned *bits = info.bits + (at1 >> 5);
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            if (tid + u * kThreads < pieces) {
                uint4 v = reinterpret_cast<const uint4 *>(at0 + head)[tid + u * kThreads];
                if (masks)
                    v = masked<T>(v, __funnelshift_r(bits[u * (kStep / 32)], bits[u * (kStep / 32) + 1], shift) & kAll);
                __stcs(reinterpret_cast<uint4 *>(out + head) + tid + u * kThreads, v);
            }
        for (int i = tid; i < range - pieces * kVec; i += kThreads) {
            const int at = outside(i, head, pieces);
            out[at] = !masks || ((info.bits[at >> 5] >> (at & 31)) & 1) ? at0[at] : from_f<T>(-INFINITY);
        }
        // the stage's next copy comes after these accesses
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(empty + s));
    }
    if (bad) raise_status(p.status, bad);
}

// The kernel's shared memory, allowed once a device.
template <typename T>
cudaError_t prepare()
{
    static std::mutex mu;
    static std::map<int, unsigned> done;   // device -> cache generation
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned gen = cache_generation();
    std::lock_guard<std::mutex> lock(mu);
    const auto it = done.find(dev);
    if (it != done.end() && it->second == gen) return cudaSuccess;
    e = cudaFuncSetAttribute(process_logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<T>);
    if (e == cudaSuccess) done[dev] = gen;
    return e;
}

template <typename T>
cudaError_t launch(const awq_logits_t &a, cudaStream_t stream)
{
    LogitsParams p{};
    p.a = a;
    p.status = device_status_word();
    p.grammar_words = (a.vocab + 31) / 32;
    const int64_t ranges = (a.vocab + kRange<T> - 1) / kRange<T>;
    // runs of rows, so long that one wave of CTAs does all of them
    const int64_t want = std::max<int64_t>(1, 152 * kPerSm<T> / ranges);
    p.rows_per_cta = (int)std::max<int64_t>((a.rows + want - 1) / want, (a.rows + 65534) / 65535);
    constexpr size_t smem = kSmem<T>;
    cudaError_t e = prepare<T>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ranges, (unsigned)((a.rows + p.rows_per_cta - 1) / p.rows_per_cta));
    cfg.blockDim = dim3(kThreads + 32);
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

// awq_beam.cu -- one step of beam search over the logits, and rows of other state by parent.
//
// beam_rows_kernel reads every logit once. The rows are cut into equal chunks of up to 1024
// 16-byte pieces, and those shared out over the CTAs (beam_cut); a producer warp keeps a ring of bulk copies
// under way across rows, so that HBM does not wait while a row's end is worked on. Each thread keeps the
// maximum of what it has read. No list is kept while the logits stream by: the best K of a part
// of a row can only lie with the K threads whose maxima are the greatest (each of them has an element
// at least as great as the K-th greatest maximum, any other thread has none). Those
// threads' pieces, where their chunks' maxima allow, are read a second time, from the L2 cache, and what
// reaches the K-th greatest maximum is sorted out, by counting. Where that is more than there is room for, a sample of
// it gives a better bound, and it is done again. Logits that are equal are told apart by
// their place, so all keys differ, and how the data lie hardly matters to the time.
//
// The sum of exp(x - m) is taken for each chunk and warp by itself and added up in one order,
// so that a row's log-sum-exp does not depend on how the rows are shared out: equal rows (at
// the same place within 16 bytes) have equal ones, and their beams tie as they should.
//
// beam_merge_kernel, a CTA a request, adds up a row's sums and takes the best of the lists of all its
// rows' parts. A bound from the lists' candidates of several numbers leaves few that can be among the first;
// their scores, as pairs of fp32 numbers, since fp64 runs at two operations a clock, decide.
//
// Bound: HBM, one read of the logits; one exponential a logit, and about seven instructions
// around it, issued in 56 % of the cycles. Measured, with the reordering of token histories: 64 requests of 8
// beams over 131,072 bf16 logits 38 us (rows 27.7, merge 6.4, histories 3.5; the read alone 20), 15 of 32
// over 100,003 fp32 logits 50 us (36, 11, 3.2; 28), 4 beams over 32,000 11.5 us
// replayed (17 to 20 a call, the host's). Masked parts cost little more (64 x 8 over 65,536 fp16, of which a mask leaves a
// tenth: 20.7 us, 20.1 without). On the way there: plain loads,
// keys sorted by one warp, sums and merges in fp64 94 and 153 us; the ring and sorted maxima 62 and 103; four small CTAs an
// SM instead of two, fp32 pairs in the merge 50 and 62; eight pieces a thread and packed fp32
// instructions 46 and 57; logits that leave L2 before anything else, so that code and lists stay, 43 and 56 (replayed);
// equal chunks, several bounds in the merge 42 and 53; parts that end with rows 39.5 and 52.
#include <algorithm>
#include <cmath>
#include <numeric>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 128;          // of the working warps
constexpr int kLoads = 8;             // 16-byte pieces of a thread in a chunk at most
constexpr int kMostBeams = 32, kMostEnds = 8, kMostBest = kMostBeams + kMostEnds;
constexpr int kMergeKeys = 6144;      // keys of a request's lists in the merge's shared memory
constexpr int kMergeLists = 640;      // and its lists; beam_cut keeps to both
constexpr int kNoRow = 255;
constexpr int kMostEnding = kMostBeams * kMostEnds;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct BeamParams {
    awq_beam_select_t a;
    unsigned int *status;
    // All rows as a line of chunks, in which a row takes `span` and has `chunks`, cut into `each` for a CTA. The part of
    // a row that one CTA has is a stretch, number CTA + row: its best [best] are in the workspace, and the
    // maximum and sum of each chunk and warp.
    float2 *sums;
    uint64_t *lists;
    int64_t rows, chunks, span, each;
    int chunk, own;                   // pieces of a chunk, and of a thread in it
    int best, merge_lists, fault;     // merge_lists: the most stretches of a request
};

template <typename T>
__device__ __forceinline__ void widen(uint4 v, float (&x)[16 / sizeof(T)])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ float one(const T *p)
{
    if constexpr (sizeof(T) == 4) return *p;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(*p);
    else return __bfloat162float(*p);
}

// 2^x to 2^-22 of its value; what is below the least normal number is 0.
__device__ __forceinline__ float power(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Larger keys are better: the logit, then the lower token. No logit gives 0; both zeros are one value.
__device__ __forceinline__ uint64_t key_of(float x, unsigned token)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    return (uint64_t)(b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u)) << 32 | (0xFFFFFFFFu - token);
}

__device__ __forceinline__ float logit_of(uint64_t key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ unsigned token_of(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// The greatest of the lanes' keys, known to all.
__device__ __forceinline__ uint64_t warp_max(uint64_t key)
{
    const uint32_t high = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32));
    const uint32_t low = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
    return (uint64_t)high << 32 | low;
}

// The `best` greatest of n keys in shared memory into out, in order, 0 after the last; by
// one warp. Keys that are not 0 differ.
__device__ void warp_best(uint64_t *keys, int n, int best, uint64_t *out)
{
    const int lane = threadIdx.x & 31;
    uint64_t mine = 0;
    int at = 0;
    for (int i = lane; i < n; i += 32)
        if (keys[i] > mine) mine = keys[at = i];
    for (int r = 0; r < best; ++r) {
        const uint64_t top = warp_max(mine);
        if (lane == 0) out[r] = top;
        if (top && mine == top) {
            keys[at] = 0;
            mine = 0;
            for (int i = lane; i < n; i += 32)
                if (keys[i] > mine) mine = keys[at = i];
        }
    }
    __syncwarp();
}

// A row as 16-byte pieces from an aligned address at or before it. Pieces `whole` to
// `end` - 1 lie in the row; what is outside them is one by one: `head` elements at its beginning,
// `tail` at its end.
template <typename T>
struct Row {
    static constexpr int kEach = 16 / sizeof(T);
    const T *row;
    const uint4 *pieces;
    int lead, whole, end, head, tail;   // lead: elements of the first piece that are not the row's

    __device__ Row(const T *p, int vocab) : row(p)
    {
        lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        pieces = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
        whole = lead > 0;
        head = lead > 0 ? min(kEach - lead, vocab) : 0;
        end = max((lead + vocab) / kEach, whole);
        tail = max(lead + vocab - end * kEach, 0);
    }
    __device__ unsigned token(int piece) const { return (unsigned)(piece * kEach - lead); }
};

// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t both(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 apart(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

// The greatest of a piece's elements as they are (a NaN gives way to a number), joined with `top`'s.
template <typename T>
__device__ __forceinline__ uint32_t top_of(uint4 v, uint32_t top)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            top = __float_as_uint(fmaxf(__uint_as_float(top), __uint_as_float(w[i])));
        } else if constexpr (std::is_same<T, __half>::value) {
            const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&top), *reinterpret_cast<const __half2 *>(&w[i]));
            top = *reinterpret_cast<const uint32_t *>(&m);
        } else {
            const __nv_bfloat162 m =
                __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&top), *reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            top = *reinterpret_cast<const uint32_t *>(&m);
        }
    }
    return top;
}

template <typename T>
__device__ __forceinline__ float top_value(uint32_t top)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(top);
    float x[16 / sizeof(T)];
    widen<T>(make_uint4(top, top, top, top), x);
    return fmaxf(x[0], x[1]);
}

// The 32 lanes' keys in descending order (a bitonic network).
__device__ __forceinline__ uint64_t warp_sort(uint64_t key)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, key, j);
            const bool greater = ((lane & j) == 0) == ((lane & k) == 0);
            key = (other > key) == greater ? other : key;
        }
    }
    return key;
}

constexpr int kWarps = kThreads / 32;
constexpr int kChunk = kThreads * kLoads;     // pieces at most: 16 KB
constexpr int kStage = kChunk / 2;            // pieces of a stage of the ring, for half of the warps
constexpr int kRoom = 512;            // keys of a part that the list of the best is taken from
constexpr int kPerSm = 4;             // CTAs: while one sorts, the others read
constexpr int kStages = 4;
constexpr int kKnown = 48;            // chunks of a part whose threads' maxima are kept
constexpr int kAtOnce = 4;            // pieces of a thread under way

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, kPerSm)
beam_rows_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int kEach = 16 / sizeof(T);
    extern __shared__ __align__(128) uint4 ring[];       // [kStages][kStage]
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t keys[kRoom], sorted[kWarps][32], leaders[kMostBest];
    __shared__ uint16_t highs[kKnown][kThreads];         // upper halves of the threads' maxima, in their order
    __shared__ uint16_t todo[kMostBest * kKnown];        // kThreads * chunk + thread
    __shared__ int who[kMostBest], listed, todos;
    __shared__ uint64_t least;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), kWarps / 2);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t begin = blockIdx.x * p.each, end = min(begin + p.each, p.rows * p.span);
    auto row_of = [&](int64_t r) {
        return Row<T>(static_cast<const T *>(p.a.logits) + r * p.a.logits_row_stride, (int)p.a.vocab);
    };

    const int first_half = kThreads / 2 * p.own;
    if (warp == kWarps) {
        // ---------------------------------------------------------------- the rows' way in
        if (lane > 0) return;
        const uint64_t policy = ptx::evict_first_policy();
        int64_t issued = 0;
        bool ok = true;
        for (int64_t at = begin, r = begin / p.span; at < end && ok; ++r) {
            const int j0 = (int)(at - r * p.span), j1 = (int)min(p.chunks, j0 + end - at);
            at = (r + 1) * p.span;
            // no beam: nobody looks at it
            if (p.a.scores[r] == -INFINITY) continue;
            const Row<T> row = row_of(r);
            for (int j = j0; j < j1 && ok; ++j) {
                const int i0 = row.whole + j * p.chunk, i2 = min(i0 + p.chunk, row.end);
                if (i0 >= i2) continue;
                for (int half = 0; half < 2; ++half) {
                    // the first half of the threads have the first stage
                    const int i = half ? min(i0 + first_half, i2) : i0, i1 = half ? i2 : min(i0 + first_half, i2);
                    const int s = (int)(issued % kStages);
                    ok = ptx::mbar_wait_bounded(ptx::smem_addr(empty + s), ((issued / kStages) & 1) ^ 1, nullptr, p.status);
                    if (!ok) break;
                    const uint32_t bytes = (uint32_t)(i1 - i) * 16;
                    ptx::mbar_arrive_expect_tx(ptx::smem_addr(full + s), bytes);
                    ++issued;
                    if (bytes == 0) continue;
#ifdef AWQ_FAULT_TEST
                    if (p.fault == 1 && blockIdx.x == 0) continue;
#endif
                    ptx::bulk_load(ptx::smem_addr(ring + s * kStage), row.pieces + i, bytes, ptx::smem_addr(full + s), policy);
                }
            }
        }
        // The copies on their way land before the shared memory goes: the working warps may have given up on them (if
        // not, they wait for the same stages). Those behind one that never lands have had as long
        bool landed = true;
        for (int64_t i = max((int64_t)0, issued - kStages); i < issued && landed; ++i)
            landed = ptx::mbar_wait_bounded(ptx::smem_addr(full + i % kStages), (i / kStages) & 1, nullptr, nullptr);
        return;
    }

    // ---------------------------------------------------------------- maxima, sums, lists
    constexpr uint32_t nothing = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    int64_t used = 0;
    for (int64_t at = begin, r = begin / p.span; at < end; ++r) {
        const int j0 = (int)(at - r * p.span), j1 = (int)min(p.chunks, j0 + end - at);
        at = (r + 1) * p.span;
        if (p.a.scores[r] == -INFINITY) continue;
        const Row<T> row = row_of(r);
        // what is not in whole pieces, one element a thread: the first chunk has the head, the last one the tail
        const bool in_head = j0 == 0 && tid < row.head;
        const bool in_tail = j1 == p.chunks && tid >= 32 && tid - 32 < row.tail;
        const unsigned single_token = in_tail ? row.token(row.end) + tid - 32 : tid;
        // not read-only loads: this kernel may be resident while the one before writes the logits
        const float single = in_head || in_tail ? one(row.row + single_token) : -INFINITY;
        const int single_chunk = in_tail ? j1 - 1 : j0;

        // ---- each thread kLoads neighbouring pieces of a chunk: its maximum, and the warp's sum
        float m = -INFINITY;
        int where = 0;
        bool landed = true;
        for (int j = j0; j < j1; ++j) {
            const int i = row.whole + j * p.chunk, count = min(p.chunk, row.end - i);
            uint4 v[kLoads];
            uint32_t all = nothing;
            if (count > 0) {
                const int64_t stage = 2 * used + tid / (kThreads / 2);
                const int s = (int)(stage % kStages);
#ifdef AWQ_FAULT_TEST
                if (p.fault == 2 && blockIdx.x == 0) {
                    raise_status(p.status, kStatusTimeout);
                    landed = false;
                }
#endif
                landed = landed && ptx::mbar_wait_bounded(ptx::smem_addr(full + s), (stage / kStages) & 1, nullptr, p.status);
                if (!__all_sync(0xFFFFFFFFu, landed)) {
                    landed = false;
                    break;
                }
                ++used;
                // in an order that keeps eight lanes off one another's banks
                const uint4 *from = ring + s * kStage + tid % (kThreads / 2) * p.own;
                if (p.own == kLoads && (warp + 1) * 32 * kLoads <= count) {
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) v[u] = from[(u + tid) % kLoads];
                } else {
                    const int mine = min(p.own, count - tid * p.own);
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        v[u] = make_uint4(nothing, nothing, nothing, nothing);
                        if ((u + tid) % kLoads < mine) v[u] = from[(u + tid) % kLoads];
                    }
                }
#pragma unroll
                for (int u = 0; u < kLoads; ++u) all = top_of<T>(v[u], all);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(empty + s));
            } else {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) v[u] = make_uint4(nothing, nothing, nothing, nothing);
            }
            const float top = top_value<T>(all);
            if (top > m) {
                m = top;
                where = j;
            }
            const float alone = j == single_chunk ? single : -INFINITY;
            uint32_t order = (uint32_t)(key_of(top, 0) >> 32);
            if (j - j0 < kKnown) highs[j - j0][tid] = (uint16_t)(order >> 16);
            order = __reduce_max_sync(0xFFFFFFFFu, max(order, (uint32_t)(key_of(alone, 0) >> 32)));
            const float most = logit_of((uint64_t)order << 32), base = most > -INFINITY ? most : 0.f;
            const uint64_t scale = both(kLog2e, kLog2e);
            auto sum_of = [&](auto exponents) {
                uint64_t s0 = 0, s1 = 0;
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    float x[kEach];
                    widen<T>(v[u], x);
#pragma unroll
                    for (int k = 0; k < kEach; k += 2) {
                        const float2 t = apart(exponents(both(x[k], x[k + 1])));
                        const uint64_t e = both(power(t.x), power(t.y));
                        if (k & 2) s1 = add2(s1, e);
                        else s0 = add2(s0, e);
                    }
                }
                const float2 sums = apart(add2(s0, s1));
                return sums.x + sums.y;
            };
            float sum;
            if (fabsf(base) < 0x1p12f) {
                // 2^(x log2 e - shift), one FMA. Shift's own rounding, d <= 2^-12, is put right to first order, which
                // leaves (d ln 2)^2 / 2 < 2^-26
                const float shift = base * kLog2e;
                const uint64_t minus = both(-shift, -shift);
                sum = sum_of([&](uint64_t x) { return fma2(x, scale, minus); });
                sum = fmaf(sum, -kLn2 * fmaf(base, kLog2e, -shift), sum);
            } else {
                // parts of which a mask leaves nothing, rows far from zero: there d would be anything up to infinity
                const uint64_t minus = both(-base, -base);
                sum = sum_of([&](uint64_t x) { return fma2(add2(x, minus), scale, 0); });
            }
            // a NaN stays one
            sum += power((alone - base) * kLog2e);
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            if (lane == 0) p.sums[(r * p.chunks + j) * kWarps + warp] = make_float2(most, sum);
        }

        // ---- the threads with the greatest maxima: each warp sorts its own, then each key counts those
        // before it in the other warps' lists. Equal maxima go by the place of their pieces, so keys differ
        const uint64_t key = warp_sort(m > -INFINITY ? key_of(m, (unsigned)((where - j0) * kThreads + tid)) : 0);
        sorted[warp][lane] = key;
        if (tid == 0) {
            least = 0;
            todos = listed = 0;
        }
        if (!ptx::named_barrier_and(1, kThreads, landed)) {
            // A wait ran out. What the workspace holds for this row and the share's later ones is from earlier calls:
            // empty lists, and sums that leave their rows without candidates
            for (; r * p.span < end; ++r) {
                for (int k = tid; k < p.best; k += kThreads) p.lists[(blockIdx.x + r) * p.best + k] = 0;
                const int64_t first = max(begin - r * p.span, (int64_t)0), last = min(p.chunks, end - r * p.span);
                for (int64_t i = (r * p.chunks + first) * kWarps + tid; i < (r * p.chunks + last) * kWarps; i += kThreads)
                    p.sums[i] = make_float2(-INFINITY, NAN);
            }
            break;
        }
        if (key && lane < p.best) {
            int rank = lane;
            int low[kWarps] = {};             // keys of warp w that are greater: found bit by bit
#pragma unroll
            for (int step = 32; step; step >>= 1)
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (low[w] + step <= 32 && sorted[w][low[w] + step - 1] > key) low[w] += step;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (w != warp) rank += low[w];
            if (rank < p.best) who[rank] = (int)((0xFFFFFFFFu - (uint32_t)key) % kThreads);
            if (rank == p.best - 1) least = key;
        }
        ptx::named_barrier(1, kThreads);

        // ---- their pieces again: what reaches `least`
        int leads = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) leads += __popc(__ballot_sync(0xFFFFFFFFu, sorted[w][lane] >= max(least, (uint64_t)1)));
        const uint64_t lowest = least;
        const uint32_t lowest_value = (uint32_t)(lowest >> 32);
        const float lowest_logit = lowest ? logit_of(lowest) : -INFINITY;
        uint64_t floor = 0;                   // of keys, once there were too many
        // behind: of a unit whose place is behind that of the least maximum, where only what is greater than it counts
        auto enlist = [&](float x, unsigned token, bool behind) {
            if (!(x > -INFINITY)) return;
            const uint64_t k = key_of(x, token);
            const uint32_t value = (uint32_t)(k >> 32);
            if (value < lowest_value || (behind && value == lowest_value) || k < floor) return;
            // past the room each takes the place of another with the chance that all have: a sample of them
            const unsigned at = atomicAdd(&listed, 1);
            const unsigned slot = at < kRoom ? at : __umulhi(at * 2654435761u, at);
            if (slot < kRoom) keys[slot] = k;
        };
        while (true) {
            enlist(single, single_token, false);
            for (int g0 = j0; g0 < j1; g0 += kKnown) {
                // the units -- chunk j of a leading thread -- whose maximum is great enough
                const int units = leads * min(kKnown, j1 - g0);
                if (g0 > j0 || floor) {
                    ptx::named_barrier(1, kThreads);
                    if (tid == 0) todos = 0;
                    ptx::named_barrier(1, kThreads);
                }
                for (int e = tid; e < units; e += kThreads) {
                    const int j = e / leads, l = who[e - j * leads];
                    if (g0 > j0 || highs[j][l] >= lowest_value >> 16) todo[atomicAdd(&todos, 1)] = (uint16_t)(j * kThreads + l);
                }
                ptx::named_barrier(1, kThreads);
                // Their pieces, kAtOnce of a thread under way. Few have an element that will do: those are taken
                // once more, from L1, so that what follows is there once
                const int pieces = todos * p.own;
                auto piece_of = [&](int e, bool &behind) {
                    if (e >= pieces) return -1;
                    const int unit = todo[e / p.own], j = g0 + unit / kThreads, l = unit % kThreads;
                    const int at = l * p.own + e % p.own, i = row.whole + j * p.chunk + at;
                    behind = ((uint64_t)lowest_value << 32 | (0xFFFFFFFFu - (unsigned)((j - j0) * kThreads + l))) < lowest;
                    return at < p.chunk && i < row.end ? i : -1;
                };
                for (int e0 = tid; e0 < pieces; e0 += kThreads * kAtOnce) {
                    uint4 v[kAtOnce];
                    bool behind;
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        const int i = piece_of(e0 + u * kThreads, behind);
                        v[u] = i >= 0 ? row.pieces[i] : make_uint4(nothing, nothing, nothing, nothing);
                    }
                    unsigned good = 0;
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        float x[kEach];
                        widen<T>(v[u], x);
#pragma unroll
                        for (int k = 0; k < kEach; ++k) good |= (x[k] >= lowest_logit ? 1u : 0u) << (u * kEach + k);
                    }
#pragma unroll 1
                    for (; good; good &= good - 1) {
                        const int bit = __ffs(good) - 1, i = piece_of(e0 + bit / kEach * kThreads, behind);
                        const unsigned token = row.token(i) + bit % kEach;
                        if (i >= 0) enlist(one(row.row + token), token, behind);
                    }
                }
            }
            ptx::named_barrier(1, kThreads);
            const int have = listed;
            if (have <= kRoom) break;
            // too many: `best` at least reach the sample's number `best`, and few more; once more with those
            ptx::named_barrier(1, kThreads);
            if (warp == 0) {
                warp_best(keys, kRoom, p.best, leaders);
                if (lane == 0) listed = 0;
            }
            ptx::named_barrier(1, kThreads);
            floor = leaders[p.best - 1];
        }
        // ---- the best of them in order
        const int have = listed;
        uint64_t *list = p.lists + (blockIdx.x + r) * p.best;
        uint64_t mine[kRoom / kThreads];
        int place[kRoom / kThreads] = {};
#pragma unroll
        for (int u = 0; u < kRoom / kThreads; ++u) mine[u] = tid + u * kThreads < have ? keys[tid + u * kThreads] : ~(uint64_t)0;
#pragma unroll 4
        for (int i = 0; i < have; ++i) {
            const uint64_t other = keys[i];
#pragma unroll
            for (int u = 0; u < kRoom / kThreads; ++u)
                if (u == 0 || have > u * kThreads) place[u] += other > mine[u];
        }
#pragma unroll
        for (int u = 0; u < kRoom / kThreads; ++u)
            if (tid + u * kThreads < have && place[u] < p.best) list[place[u]] = mine[u];
        for (int k = have + tid; k < p.best; k += kThreads) list[k] = 0;
        ptx::named_barrier(1, kThreads);
    }
}

// A sum of fp32 numbers with what its roundings lost (Knuth's two-sum): 2^-47 of it for the price of
// fp32, where fp64 runs at two operations a clock.
struct Sum {
    float high = 0.f, low = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float s = high + x, t = s - high;
        low += (high - (s - t)) + (x - t);
        high = s;
    }
    // low below half of high's last place
    __device__ __forceinline__ void settle()
    {
        const float s = high + low;
        low -= s - high;
        high = s;
    }
};

// Adds ln(x.high + x.low), normal and positive, to `to`: x = 2^e m with m in [2/3, 4/3), ln m by the series of
// 2 atanh(t) in t = (m - 1) / (m + 1), |t| <= 1/5. The quotient has its remainder; what
// is behind the first term, 0.0055 at most, is formed and added in fp32: seven roundings, below 2^-28 in all.
__device__ __forceinline__ void add_log(Sum x, Sum &to)
{
    int bits = __float_as_int(x.high);
    const int e = (bits - 0x3F2AAAAB) >> 23;
    const float scale = __int_as_float((127 - e) << 23);       // a normal number: sums are 1 to 2^28
    const float m = x.high * scale, a = m - 1.f, b = m + 1.f;
    const float r = 1.f / b, t = a * r;
    // (a - t (m + 1)) / (m + 1), of b's own rounding too, and of x.low
    const float rest = fmaf(-t, b, a) - t * (m - (b - 1.f));
    const float t_low = (rest + x.low * scale * (1.f - t)) * r;
    const float s = t * t;
    const float more = t * s * (2.f / 3 + s * (2.f / 5 + s * (2.f / 7 + s * (2.f / 9 + s * (2.f / 11 + s * (2.f / 13))))));
    to.add((float)e * 0.693145751953125f);                     // ln 2 in 14 bits, and the rest
    to.add(2.f * t);
    // of t's remainder the whole series' slope, 2 / (1 - t^2)
    to.low += (float)e * 1.42860682e-6f + 2.f * t_low * (1.f + s * (1.f + s)) + more;
    to.settle();
}

// Order of such sums as whole numbers; no candidate is 0.
__device__ __forceinline__ uint64_t order_of(Sum s)
{
    return (key_of(s.high, 0) & 0xFFFFFFFF00000000ull) | key_of(s.low, 0) >> 32;
}

__global__ void __launch_bounds__(32 * kMostBeams)
beam_merge_kernel(const __grid_constant__ BeamParams p)
{
    extern __shared__ __align__(16) uint64_t merge_smem[];
    __shared__ Sum lses[kMostBeams];                     // of the rows that have candidates
    __shared__ float befores[kMostBeams];
    __shared__ bool sound[kMostBeams];
    __shared__ int first_list[kMostBeams], last_list[kMostBeams], end_tokens[kMostEnds];
    __shared__ uint8_t row_of_list[kMergeLists];
    __shared__ int stopping[kMergeLists];                // of a list's candidates: how many end
    __shared__ uint32_t floor_order;
    __shared__ int ending_at[kMostEnding], picked, endings, told;
    const int beams = (int)p.a.beams, best = p.best, keep = (int)p.a.num_beams, threads = blockDim.x;
    const int ends = (int)p.a.num_ends;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t request = blockIdx.x, r0 = request * beams;
    // a row has one list in each CTA that had a part of it
    const int64_t first = r0 * p.span / p.each + r0;
    if (tid < beams) {
        const int64_t begin = (r0 + tid) * p.span;
        first_list[tid] = (int)(begin / p.each + r0 + tid - first);
        last_list[tid] = (int)((begin + p.chunks - 1) / p.each + r0 + tid - first);
    }
    if (tid == 0) {
        picked = endings = told = 0;
        floor_order = 0;
    }
    // a number that no part has, where a row and a CTA's share end together
    for (int l = tid; l < p.merge_lists; l += threads) {
        row_of_list[l] = kNoRow;
        stopping[l] = 0;
    }
    __syncthreads();
    const int lists = last_list[beams - 1] + 1, candidates = lists * best;
    // picks: those that end, and behind them what reaches `floor`: score, and what goes before at equal scores
    uint64_t *keys = merge_smem;
    ulonglong2 *picks = reinterpret_cast<ulonglong2 *>(keys + (p.merge_lists * best + 1) / 2 * 2);
    int *pick_at = reinterpret_cast<int *>(picks + p.merge_lists * best);
    float *highs = reinterpret_cast<float *>(pick_at + p.merge_lists * best);
    if (warp < beams)
        for (int l = first_list[warp] + lane; l <= last_list[warp]; l += 32) row_of_list[l] = warp;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    // ---- the lists of the request's rows, and a warp a row: its sum
    if (tid < ends) end_tokens[tid] = p.a.end_tokens[tid];
    for (int c = tid; c < candidates; c += threads) keys[c] = p.lists[first * best + c];
    if (warp < beams) {
        const int64_t r = r0 + warp;
        const float before = p.a.scores[r];
        const float2 *row_sums = p.sums + r * p.chunks * kWarps;
        const int64_t parts = p.chunks * kWarps;
        constexpr int kHeld = 8;
        float2 held[kHeld];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            held[i] = lane + 32 * i < parts ? row_sums[lane + 32 * i] : make_float2(-INFINITY, 0.f);
            top = fmaxf(top, held[i].x);
        }
        for (int64_t i = lane + 32 * kHeld; i < parts; i += 32) top = fmaxf(top, row_sums[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        // a chunk without a logit has the sum 0, or NaN
        auto part = [&](float2 s) { return s.x > -INFINITY ? s.y * power((s.x - top) * kLog2e) : s.y; };
        Sum all;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (32 * i < parts) all.add(part(held[i]));
        for (int64_t i = lane + 32 * kHeld; i < parts; i += 32) all.add(part(row_sums[i]));
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            // the same on both lanes of a pair
            const float high = __shfl_xor_sync(0xFFFFFFFFu, all.high, d), low = __shfl_xor_sync(0xFFFFFFFFu, all.low, d);
            const float great = fmaxf(all.high, high), small = fminf(all.high, high);
            const bool bad = !(all.high >= 0.f && high >= 0.f);
            all.low += low;
            all.high = great;
            all.add(small);
            if (bad) all.high = NAN;
        }
        if (lane == 0) {
            // without a beam nothing was written; NaN fails all comparisons
            const bool fine = all.high >= 0.f && top < INFINITY && before < INFINITY;
            if (!fine && before != -INFINITY) raise_status(p.status, kStatusBadIndex);
            sound[warp] = fine && all.high > 0.f && before != -INFINITY;
            befores[warp] = before;
            Sum lse;
            lse.high = top;
            if (sound[warp]) add_log(all, lse);
            lses[warp] = lse;
        }
    }
    __syncthreads();

    // ---- every candidate's score in fp32, with a bound of what that is off by (16 times its roundings); NaN for
    // none. Those that end are put aside
    auto near = [&](uint64_t key, int w, float &off) {
        const float x = logit_of(key);
        off = fabsf(befores[w]) * 0x1p-20f + fabsf(x) * 0x1p-20f + fabsf(lses[w].high) * 0x1p-20f;
        return befores[w] + (x - lses[w].high);
    };
    auto exact = [&](int c) {
        const int w = row_of_list[c / best];
        Sum s;
        s.high = logit_of(keys[c]);
        // below the least fp32 number, where two-sums have no remainder, all are one: -inf
        if (befores[w] + (s.high - lses[w].high) == -INFINITY) return order_of({-INFINITY, 0.f});
        s.add(-lses[w].high);
        s.add(befores[w]);
        s.low -= lses[w].low;
        s.settle();
        return order_of(s);
    };
    for (int c = tid; c < candidates; c += threads) {
        const uint64_t key = keys[c];
        const int w = row_of_list[c / best];
        highs[c] = NAN;
        if (w == kNoRow || key == 0 || !sound[w]) continue;
        bool stops = false;
        for (int i = 0; i < ends; ++i) stops |= end_tokens[i] == (int)token_of(key);
        float off;
        const float s = near(key, w, off);
        if (!stops) {
            highs[c] = s + off;
        } else {
            atomicAdd(&stopping[c / best], 1);
            if (const int i = atomicAdd(&endings, 1); i < kMostEnding) ending_at[i] = c;
        }
    }
    __syncthreads();

    // ---- The first `keep` reach `floor`: with a list's candidate number q (from 0, of those that go on) each
    // list has q + 1 that are as good, so that where ceil(keep / (q + 1)) lists' reach it, `keep` do. Which q gives
    // the highest floor hangs on how unlike the lists are: several are tried
    float *heads = reinterpret_cast<float *>(picks);               // [tries][wide]
    const int least_q = (keep - 1) / lists, wide = (lists + 3) / 4 * 4;
    auto q_of = [&](int k) { return k == 0 ? least_q : (2 << k) - 1; };             // least_q, 3, 7, 15
    int tries = 1;
    while (tries < 4 && q_of(tries) < keep && 4 * (tries + 1) * wide <= 16 * candidates) ++tries;
    for (int i = tid; i < tries * wide; i += threads) {
        const int k = i / wide, l = i - k * wide;
        float head = -INFINITY;
        if (l < lists) {
            const int at = q_of(k) + stopping[l], w = row_of_list[l];
            const uint64_t key = at < best && w != kNoRow && sound[w] ? keys[l * best + at] : 0;
            if (key) {
                float off;
                const float s = near(key, w, off);
                head = s - 2.f * off;
            }
        }
        heads[i] = head;
    }
    __syncthreads();
    for (int i = tid; i < tries * wide; i += threads) {
        const int k = i / wide, l = i - k * wide;
        const float head = heads[i];
        int rank = 0;
#pragma unroll 2
        for (int j = 0; j < lists; j += 4) {
            const float4 h = *reinterpret_cast<const float4 *>(heads + k * wide + j);
            rank += (h.x > head || (h.x == head && j < l)) + (h.y > head || (h.y == head && j + 1 < l)) +
                    (h.z > head || (h.z == head && j + 2 < l)) + (h.w > head || (h.w == head && j + 3 < l));
        }
        if (l < lists && rank == (keep + q_of(k)) / (q_of(k) + 1) - 1) atomicMax(&floor_order, (uint32_t)(key_of(head, 0) >> 32));
    }
    __syncthreads();
    const float floor = floor_order ? logit_of((uint64_t)floor_order << 32) : -INFINITY;
    const int e = min(endings, kMostEnding);
    for (int c = tid; c < candidates + e; c += threads) {
        const bool stops = c >= candidates;
        if (!stops && !(highs[c] >= floor)) continue;
        const int i = stops ? c - candidates : e + atomicAdd(&picked, 1), at = stops ? ending_at[i] : c;
        // equal scores: the lower row (of 32), the greater logit, the lower token (of 2^27)
        picks[i] = make_ulonglong2(exact(at), (uint64_t)(31 - row_of_list[at / best]) << 59 | (keys[at] >> 32) << 27 |
                                                  (keys[at] & 0x7FFFFFF));
        pick_at[i] = at;
    }
    __syncthreads();

    // ---- in order: a candidate's place is the number of those before it
    const int n = e + picked;
    for (int i = tid; i < n; i += threads) {
        const bool stops = i < e;
        const ulonglong2 mine = picks[i];
        const uint64_t s = mine.x;
        auto before = [&](int from, int to) {
            int place = 0;
#pragma unroll 4
            for (int j = from; j < to; ++j) {
                const ulonglong2 other = picks[j];
                place += (int)(other.x > mine.x) | ((int)(other.x == mine.x) & (int)(other.y > mine.y));
            }
            return place;
        };
        int place = before(e, n);
        if (place >= keep) continue;
        if (stops) {
            const int gone = before(0, e);
            if (place + gone >= keep) continue;
            place = gone;
            atomicAdd(&told, 1);
        }
        const int c = pick_at[i];
        const int64_t to = request * keep + place;
        (stops ? p.a.ended_scores : p.a.out_scores)[to] = logit_of(s);
        (stops ? p.a.ended_parents : p.a.out_parents)[to] = (int)r0 + row_of_list[c / best];
        (stops ? p.a.ended_tokens : p.a.out_tokens)[to] = (int)token_of(keys[c]);
    }
    // places without a candidate
    const bool tells = p.a.ended_scores != nullptr;
    if (tells) __syncthreads();
    for (int k = tid; k < 2 * keep; k += threads) {
        const bool stops = k >= keep;
        const int place = stops ? k - keep : k;
        if (place < (stops ? told : n - e) || (stops && !tells)) continue;
        (stops ? p.a.ended_scores : p.a.out_scores)[request * keep + place] = -INFINITY;
        (stops ? p.a.ended_parents : p.a.out_parents)[request * keep + place] = -1;
        (stops ? p.a.ended_tokens : p.a.out_tokens)[request * keep + place] = -1;
    }
}

// ---------------------------------------------------------------------------

// Rows by parent (64 x 8 rows of 2000 tokens: 3.7 us), in pieces of the widest kind that the arrays' addresses, strides and
// sizes allow; all of an array's pieces in a line, kPieces a thread under way.
constexpr int kStateThreads = 256;
constexpr int kStatePieces = 4;
constexpr int kStatesPerLaunch = 64;

struct StateParams {
    struct {
        const char *src;
        char *dst;
        int64_t src_stride, dst_stride, row_pieces, ctas;
        int width;        // log2 of a piece's bytes
    } state[kStatesPerLaunch];
    const int32_t *parents;
    unsigned int *status;
    int64_t rows_out, rows_in;
};

template <typename V>
__device__ __forceinline__ void reorder_pieces(const StateParams &p, int n)
{
    const auto &s = p.state[n];
    const int64_t first = (int64_t)blockIdx.x * kStateThreads * kStatePieces;
    const int64_t row0 = first / s.row_pieces, total = p.rows_out * s.row_pieces;
    const int64_t off0 = first - row0 * s.row_pieces;
    V v[kStatePieces];
    V *to[kStatePieces];
#pragma unroll
    for (int u = 0; u < kStatePieces; ++u) {
        const int e = threadIdx.x + u * kStateThreads;
        to[u] = nullptr;
        if (first + e >= total) continue;
        int64_t row = row0, at = off0 + e;
        if (at >= s.row_pieces) {
            const uint32_t over = (uint32_t)at / (uint32_t)s.row_pieces;
            row += over;
            at -= over * s.row_pieces;
        }
        const int parent = p.parents[row];
        to[u] = reinterpret_cast<V *>(s.dst + row * s.dst_stride) + at;
        v[u] = V{};
        if (parent >= 0 && parent < p.rows_in) v[u] = *(reinterpret_cast<const V *>(s.src + parent * s.src_stride) + at);
        else if (parent != -1) raise_status(p.status, kStatusBadIndex);
    }
#pragma unroll
    for (int u = 0; u < kStatePieces; ++u)
        if (to[u]) *to[u] = v[u];
}

__global__ void __launch_bounds__(kStateThreads)
reorder_kernel(const __grid_constant__ StateParams p)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const int n = blockIdx.y;
    if (blockIdx.x >= p.state[n].ctas) return;
    switch (p.state[n].width) {
    case 4: reorder_pieces<uint4>(p, n); break;
    case 3: reorder_pieces<uint2>(p, n); break;
    case 2: reorder_pieces<uint32_t>(p, n); break;
    case 1: reorder_pieces<uint16_t>(p, n); break;
    default: reorder_pieces<uint8_t>(p, n); break;
    }
}

constexpr size_t merge_bytes(int64_t keys) { return (3 * sizeof(uint64_t) + sizeof(int) + sizeof(float)) * keys + 8; }

template <typename T>
const void *rows_kernel() { return (const void *)beam_rows_kernel<T>; }

} // namespace

// A row is cut into equal chunks of 16 KB at most, and all rows, as a line of chunks, into equal parts, one a CTA. What a
// CTA takes is its start, its chunks, and the end of each part of a row, which sorts out its best. So where few CTAs
// are left idle, parts end with their rows: several parts of each row, or several rows of each part, or a row a part
// for more CTAs than run at once, which go on as others end. In chunks of 16 KB (1.3 us, when all CTAs read) an end costs
// about 3 and the more the more are kept, a start 2. 38 x 7 rows of 151,927 bf16: 20.3 us in two parts each, 22.4 in
// equal ones; 300 x 4 of 100,000: 44 in pairs, 61; 44 x 32 of 33,377, 40 kept: 36.7 one by one, 42.7.
// A part has no more chunks of a row than have their maxima kept (it can, but is slow: what is read again is
// not picked); a row has at most 32 parts, since the merge looks at each list, and a request's lists the room that they have there.
BeamCut beam_cut(int64_t requests, int64_t beams, int64_t vocab, int64_t best, int element_bytes)
{
    if (requests == 0) return {};
    BeamCut c;
    const int64_t pieces = std::max<int64_t>(1, vocab / (16 / element_bytes));      // whole ones at most
    c.chunks = (pieces + kChunk - 1) / kChunk;
    c.chunk = (pieces + c.chunks - 1) / c.chunks;
    // eight pieces a thread, while that gives more threads a part than there are best to be found
    c.own = c.chunk >= kLoads * 64 ? kLoads : (c.chunk + kThreads - 1) / kThreads;
    const int64_t rows = requests * beams, total = rows * c.chunks, most = kPerSm * 152;
    const int64_t lists = std::min<int64_t>(kMergeKeys / best, kMergeLists) - beams - 1;
    double cost = INFINITY;
    // `each` chunks a CTA, of a line in which a row takes `span`; in how many parts of rows they end at most
    auto consider = [&](int64_t each, int64_t span, int64_t ends) {
        const int64_t ctas = (rows * span + each - 1) / each;
        const double waves = ctas <= most ? 1 : std::max(2., (double)ctas / most + 0.3);
        const double takes = waves * (std::min(each, total) + ends * (3 + best / 16.) + 2);
        if (takes < cost) cost = takes, c.each = each, c.span = span, c.ctas = ctas;
    };
    const int64_t least = std::max({(c.chunks + 30) / 31, (beams * c.chunks + lists - 1) / lists, int64_t(1)});
    // several parts of a row, as many as leave each a CTA
    if (const int64_t n = std::min({c.chunks, lists / beams, int64_t(31), most / rows}); n > 1) {
        const int64_t each = (c.chunks + n - 1) / n;
        if (each <= kKnown) consider(each, (c.chunks + each - 1) / each * each, 1);
    }
    // one row, or several
    const int64_t several = (rows + most - 1) / most;
    for (int64_t n = 1; c.chunks <= kKnown && n <= several; n += std::max<int64_t>(1, several - 1))
        consider(n * c.chunks, c.chunks, n);
    // equal parts
    const int64_t equal = (total + most - 1) / most;
    const int64_t each = std::max(least, c.chunks <= kKnown ? equal : std::min<int64_t>(equal, kKnown));
    consider(each, c.chunks, (each + 2 * c.chunks - std::gcd(each, c.chunks) - 1) / c.chunks);
    c.merge_lists = beams * c.span / c.each + beams + 1;
    // 8-byte words of the workspace: best keys a stretch, maximum and sum of each chunk and warp
    c.words = (c.ctas + requests * beams) * best + total * kWarps;
    return c;
}

cudaError_t launch_beam_select(const awq_beam_select_t &a, cudaStream_t stream)
{
    BeamParams p{};
    p.a = a;
    p.status = device_status_word();
    p.best = (int)(a.num_beams + a.num_ends);
    p.rows = a.requests * a.beams;
    const BeamCut c = beam_cut(a.requests, a.beams, a.vocab, p.best, a.dtype == AWQ_F32 ? 4 : 2);
    p.chunks = c.chunks;
    p.chunk = (int)c.chunk;
    p.own = (int)c.own;
    p.each = c.each;
    p.span = c.span;
    p.merge_lists = (int)c.merge_lists;
    p.lists = static_cast<uint64_t *>(a.workspace);
    p.sums = reinterpret_cast<float2 *>(p.lists + (c.ctas + p.rows) * p.best);
#ifdef AWQ_FAULT_TEST
    p.fault = fault_injection();
#endif
    void *args[] = {&p};
    const void *kernel = a.dtype == AWQ_F16 ? rows_kernel<__half>()
                         : a.dtype == AWQ_BF16 ? rows_kernel<__nv_bfloat16>() : rows_kernel<float>();
    constexpr size_t ring = kStages * kStage * sizeof(uint4);
    cudaError_t e = allow_shared(kernel, ring);
    if (e == cudaSuccess)
        e = allow_shared((const void *)beam_merge_kernel, merge_bytes(kMergeKeys));
    if (e == cudaSuccess) e = launch_dependent(kernel, c.ctas, kThreads + 32, ring, stream, args);
    if (e != cudaSuccess) return e;
    // a thread a candidate, as far as that goes: 3 requests of 18 lists of 16 10 us, 13 by 256 threads
    const int64_t candidates = c.merge_lists * p.best;
    const int threads = (int)std::max({int64_t(256), 32 * a.beams, std::min<int64_t>(1024, (candidates + 31) / 32 * 32)});
    return launch_dependent((const void *)beam_merge_kernel, a.requests, threads,
                            merge_bytes(c.merge_lists * p.best), stream, args);
}

cudaError_t launch_reorder_states(const awq_state_t *states, int64_t count, const int32_t *parents, int64_t rows_out,
                                  int64_t rows_in, cudaStream_t stream)
{
    for (int64_t n0 = 0; n0 < count; n0 += kStatesPerLaunch) {
        StateParams p{};
        p.parents = parents;
        p.status = device_status_word();
        p.rows_out = rows_out;
        p.rows_in = rows_in;
        int n = 0;
        int64_t grid = 0;
        for (int64_t i = n0; i < std::min(count, n0 + kStatesPerLaunch); ++i) {
            const awq_state_t &s = states[i];
            if (s.row_bytes == 0) continue;
            // a single row's stride is never used
            const int64_t src_stride = rows_in > 1 ? s.src_row_stride : 0, dst_stride = rows_out > 1 ? s.dst_row_stride : 0;
            const uintptr_t all = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
                                  (uintptr_t)src_stride | (uintptr_t)dst_stride | (uintptr_t)s.row_bytes;
            int width = 0;
            while (width < 4 && (all >> width & 1) == 0) ++width;
            auto &to = p.state[n++];
            to.src = static_cast<const char *>(s.src);
            to.dst = static_cast<char *>(s.dst);
            to.src_stride = src_stride;
            to.dst_stride = dst_stride;
            to.width = width;
            to.row_pieces = s.row_bytes >> width;
            to.ctas = (rows_out * to.row_pieces + kStateThreads * kStatePieces - 1) / (kStateThreads * kStatePieces);
            grid = std::max(grid, to.ctas);
        }
        if (n == 0) continue;
        if (grid >= int64_t(1) << 31) return cudaErrorInvalidValue;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)grid, (unsigned)n);
        cfg.blockDim = dim3(kStateThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void *args[] = {&p};
        cudaError_t e = cudaLaunchKernelExC(&cfg, (const void *)reorder_kernel, args);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

} // namespace awq

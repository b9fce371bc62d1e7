// awq_beam.cu -- one step of beam search over the logits, and rows of other state by parent.
//
// beam_rows_kernel reads every logit once. The rows are a line of chunks of 1024 16-byte
// pieces, cut into equal parts, one a CTA; a producer warp keeps a ring of bulk copies under way
// across rows, so that HBM does not wait while a row's end is worked on. Each thread keeps the
// maximum of what it has read. No list is kept while the logits stream by: the best K of a part
// of a row can only lie with the K threads whose maxima are the greatest (each of them has an element
// at least as great as the K-th greatest maximum, any other thread has none). Those
// threads' pieces, K / 256 of the part, are read a second time, from the L2 cache, and what
// reaches the K-th greatest maximum is sorted out. Logits that are equal are told apart by
// their place, so all keys differ and the time does not depend on the data.
//
// The sum of exp(x - m) is taken for each chunk and warp by itself and added up in one order,
// so that a row's log-sum-exp does not depend on where the line was cut: equal rows (at
// the same place within 16 bytes) have equal ones, and their beams tie as they should.
//
// beam_merge_kernel, a CTA a request, adds up a row's sums in 64 bits, merges the lists of its
// parts, a warp a row, and takes the best over the rows. The logarithms, in fp64, are one a lane of one warp:
// by all warps they took longer than all the rest (fp64 runs at two operations a clock).
//
// Bound: HBM, one read of the logits; one exponential a logit.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;             // 16-byte pieces of a thread under way
constexpr int kMostBeams = 32, kMostEnds = 8, kMostBest = kMostBeams + kMostEnds;
constexpr int kMergeKeys = 8192;      // keys of a request's lists in the merge's shared memory
constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
    awq_beam_select_t a;
    unsigned int *status;
    // All rows as a line of chunks, `chunks` each, cut into `each` for a CTA. The part of a row that one CTA
    // has is a stretch, number CTA + row: its best [best] are in the workspace, and the
    // maximum and sum of each chunk and warp.
    float2 *sums;
    uint64_t *lists;
    int64_t rows, chunks, each;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
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
constexpr int kChunk = kThreads * kLoads;     // pieces: 16 KB, a stage of the ring
constexpr int kStages = 5;

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, 2)
beam_rows_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int kEach = 16 / sizeof(T);
    constexpr int kRoom = kMostBest + kThreads * kEach + 32;
    extern __shared__ __align__(128) uint4 ring[];       // [kStages][kChunk]
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t keys[kRoom], sorted[kWarps][32], leaders[kMostBest];
    __shared__ int who[kMostBest], listed[2];
    __shared__ uint64_t least;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), kWarps);
        }
        ptx::fence_mbar_init();
        listed[0] = listed[1] = 0;
    }
    __syncthreads();
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t begin = blockIdx.x * p.each, end = min(begin + p.each, p.rows * p.chunks);
    auto row_of = [&](int64_t r) {
        return Row<T>(static_cast<const T *>(p.a.logits) + r * p.a.logits_row_stride, (int)p.a.vocab);
    };

    if (warp == kWarps) {
        // ---------------------------------------------------------------- the rows' way in
        if (lane > 0) return;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t at = begin, r = begin / p.chunks; at < end && ok; ++r) {
            const int j0 = (int)(at - r * p.chunks), j1 = (int)min(p.chunks, j0 + end - at);
            at += j1 - j0;
            // no beam: nobody looks at it
            if (p.a.scores[r] == -INFINITY) continue;
            const Row<T> row = row_of(r);
            for (int j = j0; j < j1 && ok; ++j) {
                const int i = row.whole + j * kChunk;
                if (i >= row.end) continue;
                const int s = (int)(issued % kStages);
                ok = ptx::mbar_wait_bounded(ptx::smem_addr(empty + s), ((issued / kStages) & 1) ^ 1, nullptr, p.status);
                if (!ok) break;
                const uint32_t bytes = (uint32_t)min(kChunk, row.end - i) * 16;
                ptx::mbar_arrive_expect_tx(ptx::smem_addr(full + s), bytes);
                ++issued;
#ifdef AWQ_FAULT_TEST
                if (p.fault && blockIdx.x == 0) continue;
#endif
                ptx::bulk_load(ptx::smem_addr(ring + s * kChunk), row.pieces + i, bytes, ptx::smem_addr(full + s));
            }
        }
        // after a wait that ran out: the copies on their way land before the shared memory goes
        for (int64_t i = max((int64_t)0, issued - kStages); i < issued && !ok; ++i)
            ptx::mbar_wait_bounded(ptx::smem_addr(full + i % kStages), (i / kStages) & 1, nullptr, nullptr);
        return;
    }

    // ---------------------------------------------------------------- maxima, sums, lists
    int64_t used = 0;
    int turn = 0;
    for (int64_t at = begin, r = begin / p.chunks; at < end; ++r) {
        const int j0 = (int)(at - r * p.chunks), j1 = (int)min(p.chunks, j0 + end - at);
        at += j1 - j0;
        if (p.a.scores[r] == -INFINITY) continue;
        const Row<T> row = row_of(r);
        // what is not in whole pieces, one element a thread: the first chunk has the head, the last one the tail
        const bool in_head = j0 == 0 && tid < row.head;
        const bool in_tail = j1 == p.chunks && tid >= 32 && tid - 32 < row.tail;
        const unsigned single_token = in_tail ? row.token(row.end) + tid - 32 : tid;
        // not read-only loads: this kernel may be resident while the one before writes the logits
        const float single = in_head || in_tail ? one(row.row + single_token) : -INFINITY;
        const int single_chunk = in_tail ? j1 - 1 : j0;

        // ---- each thread four neighbouring pieces of a chunk: its maximum, and the warp's sum
        float m = -INFINITY;
        int where = 0;
        bool landed = true;
        for (int j = j0; j < j1; ++j) {
            constexpr uint32_t nothing = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
            const int i = row.whole + j * kChunk;
            uint4 v[kLoads];
            uint32_t all = nothing;
            if (i < row.end) {
                const int s = (int)(used % kStages);
                landed = landed && ptx::mbar_wait_bounded(ptx::smem_addr(full + s), (used / kStages) & 1, nullptr, p.status);
                if (!__all_sync(0xFFFFFFFFu, landed)) {
                    landed = false;
                    break;
                }
                ++used;
                const int left = row.end - i - tid * kLoads;
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    // in an order that keeps eight lanes off one another's banks
                    const int piece = (u + (tid >> 1)) % kLoads;
                    v[u] = ring[s * kChunk + tid * kLoads + piece];
                    if (piece >= left) v[u] = make_uint4(nothing, nothing, nothing, nothing);
                    all = top_of<T>(v[u], all);
                }
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
            const uint32_t order = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key_of(fmaxf(top, alone), 0) >> 32));
            const float most = logit_of((uint64_t)order << 32), base = most > -INFINITY ? most : 0.f;
            const uint64_t minus = both(-base, -base), scale = both(kLog2e, kLog2e);
            uint64_t s0 = 0, s1 = 0;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                float x[kEach];
                widen<T>(v[u], x);
#pragma unroll
                for (int k = 0; k < kEach; k += 2) {
                    const float2 t = apart(mul2(add2(both(x[k], x[k + 1]), minus), scale));
                    const uint64_t e = both(power(t.x), power(t.y));
                    if (k & 2) s1 = add2(s1, e);
                    else s0 = add2(s0, e);
                }
            }
            const float2 sum2 = apart(add2(s0, s1));
            // a NaN stays one
            float sum = sum2.x + sum2.y + power((alone - base) * kLog2e);
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            if (lane == 0) p.sums[(r * p.chunks + j) * kWarps + warp] = make_float2(most, sum);
        }

        // ---- the threads with the greatest maxima: each warp sorts its own, then each key counts those
        // before it in the other warps' lists. Equal maxima go by the place of their pieces, so keys differ
        const uint64_t key = warp_sort(m > -INFINITY ? key_of(m, (unsigned)((where - j0) * kThreads + tid)) : 0);
        sorted[warp][lane] = key;
        if (tid == 0) least = 0;
        if (!ptx::named_barrier_and(1, kThreads, landed)) break;
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
        const uint32_t floor_value = (uint32_t)(least >> 32);
        uint64_t floor = 0;                   // of whole keys, once a list has been cut
        const int items = leads * (j1 - j0) * kLoads;
        int *count = &listed[turn & 1];
        auto enlist = [&](float x, unsigned token) {
            const uint64_t k = key_of(x, token);
            if (x > -INFINITY && (uint32_t)(k >> 32) >= floor_value && k >= floor) keys[atomicAdd(count, 1)] = k;
        };
        enlist(single, single_token);
        for (int e0 = 0; e0 < items; e0 += kThreads) {
            const int e = e0 + tid;
            if (e < items) {
                const int l = e / kLoads % leads, j = e / kLoads / leads;
                const int piece = row.whole + (j0 + j) * kChunk + who[l] * kLoads + e % kLoads;
                if (piece < row.end) {
                    float x[kEach];
                    widen<T>(row.pieces[piece], x);
                    // equal to the least maximum: only from its place on, so that no list overflows
                    const uint64_t place = (uint64_t)floor_value << 32 | (0xFFFFFFFFu - (unsigned)(j * kThreads + who[l]));
#pragma unroll
                    for (int k = 0; k < kEach; ++k)
                        if ((uint32_t)(key_of(x[k], 0) >> 32) > floor_value || place >= least) enlist(x[k], row.token(piece) + k);
                }
            }
            ptx::named_barrier(1, kThreads);
            const int have = *count;
            ptx::named_barrier(1, kThreads);
            if (have > kMostBest && e0 + kThreads < items) {      // room for the next round
                if (warp == 0) {
                    warp_best(keys, have, p.best, leaders);
                    for (int k = lane; k < p.best; k += 32) keys[k] = leaders[k];
                    if (lane == 0) *count = p.best;
                }
                ptx::named_barrier(1, kThreads);
                floor = keys[p.best - 1];
            }
        }
        if (items == 0) ptx::named_barrier(1, kThreads);
        const int have = *count;
        const int64_t slot = blockIdx.x + r;
        if (tid == 0) listed[turn & 1 ^ 1] = 0;
        // ---- the best of them in order
        uint64_t *list = p.lists + slot * p.best;
        if (have <= kThreads) {
            if (tid < have) {
                const uint64_t k = keys[tid];
                int rank = 0;
                for (int i = 0; i < have; ++i) rank += keys[i] > k;
                if (rank < p.best) list[rank] = k;
            }
            for (int k = have + tid; k < p.best; k += kThreads) list[k] = 0;
        } else if (warp == 0) {
            warp_best(keys, have, p.best, leaders);
            for (int k = lane; k < p.best; k += 32) list[k] = leaders[k];
        }
        ++turn;
    }
}

// Order of 64-bit scores as whole numbers; no candidate is 0.
__device__ __forceinline__ uint64_t order_of(double s)
{
    const uint64_t b = (uint64_t)__double_as_longlong(s + 0.);
    return b ^ ((int64_t)b < 0 ? ~(uint64_t)0 : (uint64_t)1 << 63);
}

__device__ __forceinline__ double score_of(uint64_t o)
{
    return __longlong_as_double((int64_t)(o >> 63 ? o ^ (uint64_t)1 << 63 : ~o));
}

__global__ void __launch_bounds__(32 * kMostBeams)
beam_merge_kernel(const __grid_constant__ BeamParams p)
{
    extern __shared__ uint64_t merge_smem[];
    __shared__ double sums[kMostBeams], lses[kMostBeams];
    __shared__ float tops[kMostBeams];
    const int beams = (int)p.a.beams, best = p.best, keep = (int)p.a.num_beams;
    uint64_t *scores = merge_smem;                                  // [beams][best + 1]: a row's best, 0 behind the last
    uint64_t *lists = scores + beams * (best + 1);                  // [stretches of all rows][best]
    unsigned *tokens = reinterpret_cast<unsigned *>(lists + p.merge_lists * best);   // [beams][best]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    // ---- a warp a row: its best from its stretches' lists, and its sum
    const int64_t request = blockIdx.x, r = request * beams + warp;
    const float before = p.a.scores[r];
    // one stretch in each CTA that has a part of the row
    const int64_t first = r * p.chunks / p.each + r;
    const int stretches = (int)(((r + 1) * p.chunks - 1) / p.each + r - first) + 1;
    uint64_t *list = lists + (first - (request * beams * p.chunks / p.each + request * beams)) * best;
    uint64_t *mine = scores + warp * (best + 1);
    int have = 0;
    if (before != -INFINITY) {
        const float2 *row_sums = p.sums + r * p.chunks * kWarps;
        const int64_t parts = p.chunks * kWarps;
        float top = -INFINITY;
        double all = 0.;
        for (int i = lane; i < stretches * best; i += 32) list[i] = p.lists[first * best + i];
        for (int64_t i = lane; i < parts; i += 32) top = fmaxf(top, row_sums[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        for (int64_t i = lane; i < parts; i += 32) {
            const float2 s = row_sums[i];
            // a chunk without a logit has the sum 0, or NaN
            all += s.x > -INFINITY ? s.y * power((s.x - top) * kLog2e) : s.y;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
        const bool sound = all >= 0. && top < INFINITY && before < INFINITY;         // not for NaN
        if (!sound && lane == 0) raise_status(p.status, kStatusBadIndex);
        if (lane == 0) {
            tops[warp] = top;
            sums[warp] = sound ? all : 0.;
        }
        __syncwarp();
        if (sound && all > 0.) {
            list += lane * best;      // of a stretch: 0 behind the last
            int at = 0;
            uint64_t head = lane < stretches ? list[0] : 0;
            for (; have < best; ++have) {
                const uint64_t key = warp_max(head);
                if (key == 0) break;
                if (head == key) head = ++at < best ? list[at] : 0;
                if (lane == 0) mine[have] = key;
            }
        }
    }
    __syncthreads();
    if (warp == 0 && lane < beams) lses[lane] = (double)tops[lane] + log(sums[lane]);
    __syncthreads();
    for (int i = lane; i <= best; i += 32) {
        if (i < have) {
            tokens[warp * best + i] = token_of(mine[i]);
            mine[i] = order_of((double)before + ((double)logit_of(mine[i]) - lses[warp]));
        } else {
            mine[i] = 0;
        }
    }
    __syncthreads();
    if (warp > 0) return;

    // ---- the best over the rows, a lane a row
    const int ends = (int)p.a.num_ends;
    const int end = lane < ends ? p.a.end_tokens[lane] : -1;
    int at = 0, live = 0, ended = 0;
    uint64_t head = lane < beams ? scores[lane * (best + 1)] : 0;
    for (int rank = 0; live < keep; ++rank) {
        const uint64_t top = warp_max(head);
        if (top == 0) break;
        // equal scores: the lowest row
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, head == top)) - 1;
        const int token = (int)tokens[w * best + __shfl_sync(0xFFFFFFFFu, at, w)];
        if (lane == w) head = scores[lane * (best + 1) + ++at];
        const bool ends_here = __any_sync(0xFFFFFFFFu, lane < ends && end == token);
        if (ends_here && rank >= keep) continue;
        if (lane == 0) {
            const int64_t to = request * keep + (ends_here ? ended : live);
            (ends_here ? p.a.ended_scores : p.a.out_scores)[to] = (float)score_of(top);
            (ends_here ? p.a.ended_parents : p.a.out_parents)[to] = (int)(request * beams + w);
            (ends_here ? p.a.ended_tokens : p.a.out_tokens)[to] = token;
        }
        if (ends_here) ++ended;
        else ++live;
    }
    for (int k = live + lane; k < keep; k += 32) {
        p.a.out_scores[request * keep + k] = -INFINITY;
        p.a.out_parents[request * keep + k] = -1;
        p.a.out_tokens[request * keep + k] = -1;
    }
    for (int k = ended + lane; ends && k < keep; k += 32) {
        p.a.ended_scores[request * keep + k] = -INFINITY;
        p.a.ended_parents[request * keep + k] = -1;
        p.a.ended_tokens[request * keep + k] = -1;
    }
}

// ---------------------------------------------------------------------------

// Rows by parent, in pieces of the widest kind that the arrays' addresses, strides and
// sizes allow; all of an array's pieces in a line, kPieces a thread under way.
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
    const int64_t first = (int64_t)blockIdx.x * kThreads * kStatePieces;
    const int64_t row0 = first / s.row_pieces, total = p.rows_out * s.row_pieces;
    const int64_t off0 = first - row0 * s.row_pieces;
    V v[kStatePieces];
    V *to[kStatePieces];
#pragma unroll
    for (int u = 0; u < kStatePieces; ++u) {
        const int e = threadIdx.x + u * kThreads;
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

__global__ void __launch_bounds__(kThreads)
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

constexpr size_t merge_bytes(int64_t beams, int64_t lists, int64_t best)
{
    return 8 * lists * best + beams * (8 * (best + 1) + 4 * best);
}

template <typename T>
const void *rows_kernel() { return (const void *)beam_rows_kernel<T>; }

} // namespace

// The line of all rows' chunks, cut into equal parts for as many CTAs as the GPU holds; a row has at
// most 32 stretches (a lane each in the merge), and a request's lists the room that they have there.
BeamCut beam_cut(int64_t requests, int64_t beams, int64_t vocab, int64_t best, int element_bytes)
{
    BeamCut c;
    c.chunks = std::max<int64_t>(1, (vocab / (16 / element_bytes) + kChunk - 1) / kChunk);
    const int64_t total = requests * beams * c.chunks;
    const int64_t lists = kMergeKeys / best - beams - 1;
    c.each = std::max({(total + 2 * 152 - 1) / (2 * 152), (c.chunks + 30) / 31, (beams * c.chunks + lists - 1) / lists,
                       int64_t(1)});
    c.ctas = (total + c.each - 1) / c.each;
    c.merge_lists = beams * c.chunks / c.each + beams + 1;
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
    p.each = c.each;
    p.merge_lists = (int)c.merge_lists;
    p.lists = static_cast<uint64_t *>(a.workspace);
    p.sums = reinterpret_cast<float2 *>(p.lists + (c.ctas + p.rows) * p.best);
#ifdef AWQ_FAULT_TEST
    p.fault = fault_injection();
#endif
    void *args[] = {&p};
    const void *kernel = a.dtype == AWQ_F16 ? rows_kernel<__half>()
                         : a.dtype == AWQ_BF16 ? rows_kernel<__nv_bfloat16>() : rows_kernel<float>();
    constexpr size_t ring = kStages * kChunk * sizeof(uint4);
    cudaError_t e = allow_shared(kernel, ring);
    if (e == cudaSuccess)
        e = allow_shared((const void *)beam_merge_kernel, 8 * kMergeKeys + merge_bytes(kMostBeams, 0, kMostBest));
    if (e == cudaSuccess) e = launch_dependent(kernel, c.ctas, kThreads + 32, ring, stream, args);
    if (e != cudaSuccess) return e;
    return launch_dependent((const void *)beam_merge_kernel, a.requests, 32 * (int)a.beams,
                            merge_bytes(a.beams, c.merge_lists, p.best), stream, args);
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
            to.ctas = (rows_out * to.row_pieces + kThreads * kStatePieces - 1) / (kThreads * kStatePieces);
            grid = std::max(grid, to.ctas);
        }
        if (n == 0) continue;
        if (grid >= int64_t(1) << 31) return cudaErrorInvalidValue;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)grid, (unsigned)n);
        cfg.blockDim = dim3(kThreads);
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

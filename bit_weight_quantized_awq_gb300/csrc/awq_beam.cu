// awq_beam.cu -- one step of beam search over the logits, and rows of other state by parent.
//
// beam_rows_kernel reads every logit once. A CTA takes a stretch of one row; each thread
// keeps the maximum m of what it has read, the 16 bytes it came from, and the sum of
// exp(x - m). No list is kept while the logits stream by: the best K of a stretch can
// only lie with the K threads whose maxima are the greatest (each of them has an element
// at least as great as the K-th greatest maximum, any other thread has none). Those
// threads' pieces, K / kThreads of the stretch, are read a second time, and what
// reaches the K-th greatest maximum is sorted out. Logits that are equal are told apart by
// their token, so all keys differ and the time does not depend on the data.
//
// beam_merge_kernel, a CTA a request, adds up the sums of a row's stretches in 64 bits,
// merges their lists, a warp a row, and takes the best over the rows.
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
    // workspace: of each stretch, maximum and sum [rows][stretches], and its best [rows][stretches][best]
    float2 *sums;
    uint64_t *lists;
    int stretches, best, element;     // element: bytes
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

// A row as 16-byte pieces from an aligned address at or before it.
template <typename T>
struct Row {
    static constexpr int kEach = 16 / sizeof(T);
    const T *row;
    const uint4 *pieces;
    int lead;           // elements of the first piece that are not the row's
    int vocab, count;

    __device__ Row(const T *p, int n) : row(p), vocab(n)
    {
        lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        pieces = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
        count = (lead + n + kEach - 1) / kEach;
    }
    // not read-only loads: this kernel may be resident while the one before writes the logits
    __device__ void load(int i, float (&x)[kEach]) const
    {
        const int first = i * kEach - lead;
        if (first >= 0 && first + kEach <= vocab) {
            widen<T>(pieces[i], x);
        } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                x[j] = first + j >= 0 && first + j < vocab ? one(row + first + j) : -INFINITY;
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_rows_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int kEach = 16 / sizeof(T);
    constexpr int kRoom = kMostBest + kThreads * kEach;
    __shared__ uint64_t keys[kRoom];
    __shared__ uint64_t leaders[kMostBest];
    __shared__ int who[kMostBest];
    __shared__ float part[kThreads / 32];
    __shared__ int listed, chosen;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t r = blockIdx.x / p.stretches;
    const int stretch = (int)(blockIdx.x - r * p.stretches);
    // no beam: the merge does not look at it either
    if (p.a.scores[r] == -INFINITY) return;
    const Row<T> row(static_cast<const T *>(p.a.logits) + r * p.a.logits_row_stride, (int)p.a.vocab);
    const int each = (row.count + p.stretches - 1) / p.stretches;
    const int begin = min(stretch * each, row.count), end = min(begin + each, row.count);

    // ---- maximum and sum of what each thread reads
    float m = -INFINITY, base = 0.f, s = 0.f;      // base: m once it is finite
    int where = -1;
    int i = begin + tid;
    for (; i < end; i += kThreads * kLoads) {
        float x[kLoads][kEach];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            if (i + n * kThreads < end) {
                row.load(i + n * kThreads, x[n]);
            } else {
#pragma unroll
                for (int j = 0; j < kEach; ++j) x[n][j] = -INFINITY;
            }
        }
        float top = m;
        int at = where;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            float t = x[n][0];
#pragma unroll
            for (int j = 1; j < kEach; ++j) t = fmaxf(t, x[n][j]);
            if (t > top) {
                top = t;
                at = i + n * kThreads;
            }
        }
        if (top > m) {
            if (m > -INFINITY) s *= power((base - top) * kLog2e);
            m = base = top;
            where = at;
        }
#pragma unroll
        for (int n = 0; n < kLoads; ++n)
#pragma unroll
            for (int j = 0; j < kEach; ++j) s += power((x[n][j] - base) * kLog2e);
    }

    // ---- the threads with the greatest maxima
    uint64_t mine = 0;
    if (where >= 0) {
        float x[kEach];
        row.load(where, x);
#pragma unroll
        for (int j = kEach - 1; j >= 0; --j)
            if (x[j] == m) mine = key_of(m, where * kEach - row.lead + j);
    }
    keys[tid] = mine;
    if (tid == 0) listed = chosen = 0;
    __syncthreads();
    if (warp == 0) warp_best(keys, kThreads, p.best, leaders);
    __syncthreads();
    const float top = logit_of(leaders[0]);       // of the stretch; leaders[0] is 0 without any logit
    float sum = mine ? s * power((m - top) * kLog2e) : s;      // s that is no number stays so
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) part[warp] = sum;
    const uint64_t least = max(leaders[p.best - 1], (uint64_t)1);
    if (mine >= least) who[atomicAdd(&chosen, 1)] = tid;
    __syncthreads();
    const int64_t slot = r * p.stretches + stretch;
    if (tid == 0) {
        float all = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) all += part[w];
        p.sums[slot] = make_float2(leaders[0] ? top : -INFINITY, all);
    }

    // ---- their pieces again: what reaches `least`, the order of `who` does not matter
    uint64_t floor = least;
    const int leads = chosen, turns = (end - begin + kThreads - 1) / kThreads;
    for (int e0 = 0; e0 < leads * turns; e0 += kThreads) {
        const int e = e0 + tid;
        if (e < leads * turns) {
            const int piece = begin + who[e % leads] + e / leads * kThreads;
            if (piece < end) {
                float x[kEach];
                row.load(piece, x);
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    if (!(x[j] > -INFINITY)) continue;
                    const uint64_t key = key_of(x[j], piece * kEach - row.lead + j);
                    if (key >= floor) keys[atomicAdd(&listed, 1)] = key;
                }
            }
        }
        __syncthreads();
        const int n = listed;
        __syncthreads();
        if (n > kMostBest && e0 + kThreads < leads * turns) {     // room for the next round
            if (warp == 0) {
                warp_best(keys, n, p.best, leaders);
                for (int k = lane; k < p.best; k += 32) keys[k] = leaders[k];
                if (lane == 0) listed = p.best;
            }
            __syncthreads();
            floor = max(leaders[p.best - 1], floor);
        }
    }
    if (warp == 0) {
        warp_best(keys, listed, p.best, leaders);
        for (int k = lane; k < p.best; k += 32) p.lists[slot * p.best + k] = leaders[k];
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
    const int beams = (int)p.a.beams, best = p.best, keep = (int)p.a.num_beams;
    uint64_t *lists = merge_smem;                                                    // [beams][stretches][best]
    uint64_t *scores = lists + beams * p.stretches * best;                           // [beams][best + 1]
    unsigned *tokens = reinterpret_cast<unsigned *>(scores + beams * (best + 1));    // [beams][best]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t request = blockIdx.x, r = request * beams + warp;
    // ---- a warp a row: its log-sum-exp and its best, from the stretches' lists
    const float before = p.a.scores[r];
    const int entries = p.stretches * best;
    uint64_t *list = lists + warp * entries;
    int have = 0;
    if (before != -INFINITY) {
        for (int i = lane; i < entries; i += 32) list[i] = p.lists[r * entries + i];
        __syncwarp();
        const float2 sum = lane < p.stretches ? p.sums[r * p.stretches + lane] : make_float2(-INFINITY, 0.f);
        float top = sum.x;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        double all = top == -INFINITY ? (double)sum.y : (double)sum.y * exp((double)sum.x - (double)top);
        if (sum.x == -INFINITY && sum.y == 0.f) all = 0.;
#pragma unroll
        for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
        const bool sound = all >= 0. && top < INFINITY && before < INFINITY;         // not for NaN
        if (!sound) {
            if (lane == 0) raise_status(p.status, kStatusBadIndex);
        } else if (all > 0.) {
            const double lse = (double)top + log(all);
            list += lane * best;      // of a stretch: none behind the last
            int at = 0;
            uint64_t head = lane < p.stretches ? list[0] : 0;
            for (; have < best; ++have) {
                const uint64_t key = warp_max(head);
                if (key == 0) break;
                if (head == key) head = ++at < best ? list[at] : 0;
                if (lane == 0) {
                    scores[warp * (best + 1) + have] = order_of((double)before + ((double)logit_of(key) - lse));
                    tokens[warp * best + have] = token_of(key);
                }
            }
        }
    }
    if (lane == 0) scores[warp * (best + 1) + have] = 0;
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

constexpr size_t merge_bytes(int64_t beams, int64_t keys, int64_t best)
{
    return 8 * keys + beams * (8 * (best + 1) + 4 * best);
}

template <typename T>
const void *rows_kernel() { return (const void *)beam_rows_kernel<T>; }

} // namespace

// As many stretches as give every SM eight CTAs, each of four pieces a thread at least,
// and a request's lists the room that they have in the merge.
int beam_stretches(int64_t requests, int64_t beams, int64_t vocab, int64_t best, int element_bytes)
{
    const int64_t rows = std::max<int64_t>(requests * beams, 1);
    const int64_t pieces = vocab * element_bytes / (16 * kThreads * kLoads);
    return (int)std::max<int64_t>(
        1, std::min({(8 * 152 + rows - 1) / rows, pieces, int64_t(kMergeKeys) / (beams * best), int64_t(32)}));
}

cudaError_t launch_beam_select(const awq_beam_select_t &a, cudaStream_t stream)
{
    BeamParams p{};
    p.a = a;
    p.status = device_status_word();
    p.element = a.dtype == AWQ_F32 ? 4 : 2;
    const int64_t rows = a.requests * a.beams;
    p.best = (int)(a.num_beams + a.num_ends);
    p.stretches = beam_stretches(a.requests, a.beams, a.vocab, p.best, p.element);
    p.lists = static_cast<uint64_t *>(a.workspace);
    p.sums = reinterpret_cast<float2 *>(p.lists + rows * p.stretches * p.best);
    void *args[] = {&p};
    const void *kernel = a.dtype == AWQ_F16 ? rows_kernel<__half>()
                         : a.dtype == AWQ_BF16 ? rows_kernel<__nv_bfloat16>() : rows_kernel<float>();
    cudaError_t e = allow_shared((const void *)beam_merge_kernel, merge_bytes(kMostBeams, kMergeKeys, kMostBest));
    if (e == cudaSuccess) e = launch_dependent(kernel, rows * p.stretches, kThreads, 0, stream, args);
    if (e != cudaSuccess) return e;
    const size_t smem = merge_bytes(a.beams, a.beams * p.stretches * p.best, p.best);
    return launch_dependent((const void *)beam_merge_kernel, a.requests, 32 * (int)a.beams, smem, stream, args);
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

// awq_paged.cu -- the paged cache of one decoding step: paged_plan_kernel
// (block tables, slot map, positions, ancestor masks from request lengths) and
// kv_append_kernel (the new tokens' keys and values into their slots).
//
// Plan: with have = ceil(ctx / bs) and need = ceil((ctx + new) / bs) - have,
// token i of request b lies at cache position c = ctx + i, in page p = c / bs,
// which is block_table[b, p] for p < have and free_blocks[base(b) + p - have]
// after that, base = the exclusive prefix sum of need. Every CTA computes the
// two prefix sums (of new and need) over all requests by itself, so CTAs need
// nothing from one another, no entry is read that another CTA writes, and the
// step is one launch. Bound: latency (a few KB are read and written). Measured: 256
// requests of one token 3.2 us, 64 trees of up to 60 nodes 5.0 us.
#include <algorithm>
#include <map>
#include <mutex>

#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 512;          // tokens per CTA and round
constexpr unsigned kSumLimit = 1u << 30;  // prefix sums saturate here: no overflow, whatever the lengths

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kSumLimit); }

__device__ __forceinline__ unsigned warp_scan(unsigned v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = sat_add(v, o);
    }
    return v;
}

// Lengths are read as max(length, 0) and capped at the sums' limit.
__device__ __forceinline__ unsigned length_of(int v, unsigned &bad)
{
    if (v < 0) bad |= kStatusBadIndex;
    if (v > (int)kSumLimit / 2) bad |= kStatusTooLarge;
    return (unsigned)min(max(v, 0), (int)kSumLimit / 2);
}

__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const PlanProblem p, unsigned int *status)
{
    extern __shared__ unsigned plan_smem[];
    unsigned *cu = plan_smem;                 // [B + 1] new tokens before request b
    unsigned *base = plan_smem + p.B + 1;     // [B + 1] new blocks before request b
    __shared__ unsigned warp_new[kPlanThreads / 32], warp_need[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(p.block_size) - 1;
    unsigned bad = 0;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    unsigned carry_new = 0, carry_need = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        unsigned n = 0, need = 0;
        if (b < p.B) {
            const unsigned ctx = length_of(p.context_lens[b], bad);
            n = length_of(p.new_lens[b], bad);
            need = ((ctx + n + p.block_size - 1) >> shift) - ((ctx + p.block_size - 1) >> shift);
        }
        const unsigned sn = warp_scan(n, lane), sd = warp_scan(need, lane);
        if (lane == 31) {
            warp_new[warp] = sn;
            warp_need[warp] = sd;
        }
        __syncthreads();
        unsigned before_new = carry_new, before_need = carry_need;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) {
                before_new = sat_add(before_new, warp_new[w]);
                before_need = sat_add(before_need, warp_need[w]);
            }
            carry_new = sat_add(carry_new, warp_new[w]);
            carry_need = sat_add(carry_need, warp_need[w]);
        }
        if (b < p.B) {
            cu[b + 1] = sat_add(before_new, sn);
            base[b + 1] = sat_add(before_need, sd);
        }
        __syncthreads();
    }
    if (tid == 0) {
        cu[0] = 0;
        base[0] = 0;
    }
    __syncthreads();
    const unsigned total = cu[p.B];

    // ---- what there is one of per request, shared out over the CTAs
    for (int b = blockIdx.x * kPlanThreads + tid; b <= p.B; b += gridDim.x * kPlanThreads)
        p.cu_new[b] = (int)min(cu[b], (unsigned)p.max_tokens);
    if (blockIdx.x == 0 && tid == 0) {
        p.counts[0] = (int)total;
        p.counts[1] = (int)base[p.B];
        if (total > (unsigned)p.max_tokens || base[p.B] > (unsigned)p.num_free) bad |= kStatusTooLarge;
    }
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += gridDim.x * (kPlanThreads / 32)) {
        const unsigned first = base[b], count = base[b + 1] - first;
        if (count == 0) continue;
        unsigned ignored = 0;
        const unsigned have = (length_of(p.context_lens[b], ignored) + p.block_size - 1) >> shift;
        if (have + count > (unsigned)p.table_width) bad |= kStatusTooLarge;
        for (unsigned j = lane; j < count; j += 32) {
            if (have + j >= (unsigned)p.table_width || first + j >= (unsigned)p.num_free) break;
            p.block_table[(int64_t)b * p.table_stride + have + j] = p.free_blocks[first + j];
        }
    }

    // ---- the tokens
    for (int64_t t0 = (int64_t)blockIdx.x * kPlanTokens; t0 < p.max_tokens; t0 += (int64_t)gridDim.x * kPlanTokens) {
        const int64_t tt = t0 + tid;
        if (tt >= p.max_tokens) continue;
        const unsigned t = (unsigned)tt;
        if (t >= total) {
            p.slot_map[t] = -1;
            p.positions[t] = 0;
            p.token_request[t] = -1;
            for (int w = 0; w < p.mask_words; ++w) p.tree_mask[(int64_t)t * p.mask_words + w] = 0;
            continue;
        }
        // the last request that starts at or before t: cu[b] <= t < cu[b + 1]
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        const int b = lo;
        const unsigned first = cu[b], i = t - first;
        unsigned ignored = 0;
        const unsigned ctx = length_of(p.context_lens[b], ignored);
        const unsigned have = (ctx + p.block_size - 1) >> shift;
        const unsigned page = (ctx + i) >> shift;
        int block = -1;
        if (page >= (unsigned)p.table_width) {
            bad |= kStatusTooLarge;
        } else if (page < have) {
            block = p.block_table[(int64_t)b * p.table_stride + page];
            if (block < 0) bad |= kStatusBadIndex;
        } else if (base[b] + page - have < (unsigned)p.num_free) {
            block = p.free_blocks[base[b] + page - have];
            // -1 (free_pages' lists have it behind the last free block): none left
            if (block < 0) bad |= block == -1 ? kStatusTooLarge : kStatusBadIndex;
        }
        p.slot_map[t] = block < 0 ? -1 : ((int64_t)block << shift) + ((ctx + i) & (p.block_size - 1));
        p.token_request[t] = b;

        // Depth and ancestors. A parent's index is below its child's, so the
        // walk to the root meets them from the highest word of the mask down:
        // one word is held at a time.
        int32_t *row = p.tree_mask + (int64_t)t * p.mask_words;
        int at = p.mask_words - 1;
        unsigned word = 0, depth = i;
        if ((int64_t)i >= (int64_t)p.mask_words * 32 && p.mask_words > 0) bad |= kStatusTooLarge;
        if (p.parents == nullptr) {
            for (; at >= 0; --at) {
                const int64_t bits = (int64_t)i + 1 - (int64_t)at * 32;
                row[at] = bits >= 32 ? -1 : bits <= 0 ? 0 : (int)((1u << bits) - 1);
            }
        } else {
            depth = 0;
            unsigned node = i;
            while (true) {
                const int w = (int)(node >> 5);
                if (w < p.mask_words) {
                    while (at > w) {
                        row[at--] = (int)word;
                        word = 0;
                    }
                    word |= 1u << (node & 31);
                }
                const int up = p.parents[first + node];
                if (up >= (int)node || up < -1) bad |= kStatusBadIndex;
                if (up < 0 || up >= (int)node) break;
                node = (unsigned)up;
                ++depth;
            }
            while (at >= 0) {
                row[at--] = (int)word;
                word = 0;
            }
        }
        p.positions[t] = (int)(ctx + depth);
    }
    if (bad) raise_status(status, bad);
}

// ---------------------------------------------------------------------------

// Copy of 16-byte pieces: a token's row is kv_heads * head_dim / 8 of them for
// the keys and as many for the values; a CTA takes `per_cta` tokens, each
// thread kAppendPieces loads before the first of its stores, so that enough
// bytes are in flight to cover HBM's latency. Bound: HBM, each byte read and written
// once. Measured: 9 prompts of up to 2048 tokens, 32 heads of 128: 75 us, 92% of
// the copy bandwidth. (With the slots' test after all loads, so that rows need not wait
// for slots: 108 us, at 114 registers.)
constexpr int kAppendThreads = 256;
constexpr int kAppendPieces = 8;

struct AppendParams {
    const char *src[2];
    char *dst[2];
    int64_t src_token[2], src_head[2], dst_block[2], dst_token[2], dst_head[2];   // bytes
    const int64_t *slot_map;
    int64_t tokens, slots;
    int shift;              // log2 of the block size
    int head_pieces, row_pieces, per_cta;
};

__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendParams p, unsigned int *status)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const int64_t t0 = (int64_t)blockIdx.x * p.per_cta;
    const int tokens = (int)min((int64_t)p.per_cta, p.tokens - t0);
    const int pieces = tokens * 2 * p.row_pieces;
    for (int e0 = threadIdx.x; e0 < pieces; e0 += kAppendThreads * kAppendPieces) {
        uint4 v[kAppendPieces];
        char *to[kAppendPieces];
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u) {
            const int e = e0 + u * kAppendThreads;
            to[u] = nullptr;
            if (e >= pieces) continue;
            const int row = e / p.row_pieces, piece = e - row * p.row_pieces;
            const int side = row & 1;
            const int head = piece / p.head_pieces, at = piece - head * p.head_pieces;
            const int64_t t = t0 + (row >> 1);
            const int64_t slot = p.slot_map[t];
            if (slot < 0 || slot >= p.slots) {
                if (slot != -1) raise_status(status, kStatusBadIndex);
                continue;
            }
            to[u] = p.dst[side] + (slot >> p.shift) * p.dst_block[side] +
                    (slot & ((1 << p.shift) - 1)) * p.dst_token[side] + head * p.dst_head[side] + at * 16;
            // not a read-only load: this kernel may be resident while the one before writes k and v
            v[u] = *reinterpret_cast<const uint4 *>(p.src[side] + t * p.src_token[side] + head * p.src_head[side] +
                                                    at * 16);
        }
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u)
            if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = v[u];
    }
}

// The plan kernel's shared memory, two sums a request.
constexpr size_t plan_smem_bytes(int64_t B) { return (size_t)2 * (B + 1) * sizeof(unsigned); }

// Allowed once a device, for the most requests: a limit of a call's own size could be
// lowered by another thread's call before this one's launch.
cudaError_t prepare_plan()
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
    e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)plan_smem_bytes(kMaxRequests));
    if (e == cudaSuccess) done[dev] = gen;
    return e;
}

} // namespace

cudaError_t launch_paged_plan(const PlanProblem &p, cudaStream_t stream)
{
    const size_t smem = plan_smem_bytes(p.B);
    const cudaError_t e = prepare_plan();
    if (e != cudaSuccess) return e;
    // every CTA scans all requests: few CTAs, each with several rounds of tokens once there are many
    const int64_t rounds = ((int64_t)p.max_tokens + kPlanTokens - 1) / kPlanTokens;
    const int64_t by_request = (p.B + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(304, std::max(rounds, std::min<int64_t>(by_request, 32))));
    PlanProblem prob = p;
    unsigned int *status = device_status_word();
    void *args[] = {&prob, &status};
    return launch_dependent((const void *)paged_plan_kernel, grid, kPlanThreads, smem, stream, args);
}

cudaError_t launch_kv_append(const AppendProblem &a, cudaStream_t stream)
{
    AppendParams p{};
    p.src[0] = static_cast<const char *>(a.k);
    p.src[1] = static_cast<const char *>(a.v);
    p.dst[0] = static_cast<char *>(a.k_cache.data);
    p.dst[1] = static_cast<char *>(a.v_cache.data);
    p.src_token[0] = a.k_token_stride * 2;
    p.src_token[1] = a.v_token_stride * 2;
    p.src_head[0] = a.k_head_stride * 2;
    p.src_head[1] = a.v_head_stride * 2;
    const awq_cache_t *c[2] = {&a.k_cache, &a.v_cache};
    for (int s = 0; s < 2; ++s) {
        p.dst_block[s] = c[s]->block_stride * 2;
        p.dst_token[s] = c[s]->token_stride * 2;
        p.dst_head[s] = c[s]->head_stride * 2;
    }
    p.slot_map = a.slot_map;
    p.tokens = a.tokens;
    p.slots = a.num_blocks * a.block_size;
    while ((1 << p.shift) < a.block_size) ++p.shift;
    p.head_pieces = a.head_dim / 8;
    p.row_pieces = a.kv_heads * p.head_pieces;
    p.per_cta = std::max(1, kAppendThreads * kAppendPieces / (2 * p.row_pieces));
    // but four CTAs an SM before one has several tokens (16 x 33 tokens, 8 heads of 128: 2.3 us, and 5.1 without)
    p.per_cta = (int)std::min<int64_t>(p.per_cta, (a.tokens + 607) / 608);
    unsigned int *status = device_status_word();
    void *args[] = {&p, &status};
    return launch_dependent((const void *)kv_append_kernel, (a.tokens + p.per_cta - 1) / p.per_cta, kAppendThreads, 0,
                            stream, args);
}

} // namespace awq

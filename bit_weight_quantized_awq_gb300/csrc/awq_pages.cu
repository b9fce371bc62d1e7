// awq_pages.cu -- the pages of a paged cache between steps: fork_kernel (block tables of
// the beams that go on), copy_pages_kernel (pages within caches), and the kernels that
// list the free blocks and compact the used ones (pages_cluster_kernel, or mark_kernel,
// count_kernel, list_kernel and move_kernel for large caches).
#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {

cudaError_t allow_shared(const void *kernel, size_t bytes)
{
    static std::mutex mu;
    static std::map<std::pair<int, const void *>, unsigned> done;   // -> cache generation
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned gen = cache_generation();
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_pair(dev, kernel);
    const auto it = done.find(key);
    if (it != done.end() && it->second == gen) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done[key] = gen;
    return e;
}

namespace {

// A row's pages: lengths are read as max(length, 0), and none is longer than the table's width.
__device__ __forceinline__ int pages_of(int length, int block_size, int shift, int width, unsigned &bad)
{
    if (length < 0) {
        bad |= kStatusBadIndex;
        return 0;
    }
    const unsigned pages = ((unsigned)length + block_size - 1) >> shift;
    if (pages > (unsigned)width) {
        bad |= kStatusTooLarge;
        return width;
    }
    return (int)pages;
}

// ---------------------------------------------------------------------------
// Fork. Which row is its parent's first and how many rows before it need a block follows
// from the parents and lengths alone; every CTA computes both for all rows by itself, as the plan
// does, so the step is one launch. Bound: latency; the tables are a few KB to a few MB. Measured
// (replayed): 8 rows 3.1 us, 384 rows 4.0 us.

constexpr int kForkThreads = 512;
constexpr int kForkEntries = 2048;          // of a row, a CTA and turn
constexpr int kForkRows = 16384;

__global__ void __launch_bounds__(kForkThreads)
fork_kernel(const __grid_constant__ ForkProblem p, unsigned int *status)
{
    extern __shared__ int fork_smem[];
    int *first = fork_smem;                 // [rows_in] the first row of each parent
    int *rank = fork_smem + p.rows_in;      // [rows_out] 2 * blocks taken before the row + whether it takes one
    __shared__ int sums[kForkThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int shift = __ffs(p.block_size) - 1, mask = p.block_size - 1;
    unsigned bad = 0;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    for (int i = tid; i < p.rows_in; i += kForkThreads) first[i] = p.rows_out;
    __syncthreads();
    for (int r = tid; r < p.rows_out; r += kForkThreads) {
        const int parent = p.parents[r];
        if (parent < -1 || parent >= p.rows_in) bad |= kStatusBadIndex;
        if (parent >= 0 && parent < p.rows_in) atomicMin(&first[parent], r);
    }
    __syncthreads();
    int carry = 0;
    for (int r0 = 0; r0 < p.rows_out; r0 += kForkThreads) {
        const int r = r0 + tid;
        bool need = false;
        if (r < p.rows_out) {
            const int parent = p.parents[r];
            if (parent >= 0 && parent < p.rows_in && first[parent] != r) {
                const int length = p.lens[parent];
                // a length beyond the table's width has no page to copy
                need = length > 0 && (length & mask) && (length >> shift) < p.width;
            }
        }
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, need);
        if (lane == 0) sums[warp] = __popc(votes);
        __syncthreads();
        int before = carry;
        for (int w = 0; w < kForkThreads / 32; ++w) {
            if (w < warp) before += sums[w];
            carry += sums[w];
        }
        if (r < p.rows_out) rank[r] = 2 * (before + __popc(votes & ((1u << lane) - 1))) + need;
        __syncthreads();
    }
    int start = p.free_start ? *p.free_start : 0;
    if (start < 0) {
        bad |= kStatusBadIndex;
        start = 0;
    }
    // -1 (free_pages' lists have it behind the last free block): none left
    auto entry = [&](int n) { return (int64_t)start + n < p.num_free ? p.free_blocks[start + n] : -1; };
    auto fresh = [&](int n) { return max(entry(n), -1); };

    // ---- what there is one of a row
    const int grid_threads = gridDim.x * kForkThreads;
    if (blockIdx.x == 0 && tid == 0) *p.count = carry;
    for (int r = blockIdx.x * kForkThreads + tid; r < p.rows_out; r += grid_threads) {
        const int parent = p.parents[r];
        const bool row = parent >= 0 && parent < p.rows_in;
        const int length = row ? p.lens[parent] : 0;
        pages_of(length, p.block_size, shift, p.width, bad);
        p.new_lens[r] = max(length, 0);
        const int n = rank[r] >> 1;
        if (rank[r] & 1) {
            const int free = entry(n), to = max(free, -1), from = p.table[parent * p.stride + (length >> shift)];
            if (free < 0) bad |= free == -1 ? kStatusTooLarge : kStatusBadIndex;
            if (from < 0) bad |= kStatusBadIndex;
            p.src[n] = to < 0 ? -1 : from;
            p.dst[n] = to;
            p.tokens[n] = length & mask;
        }
        if (r >= carry) p.src[r] = p.dst[r] = p.tokens[r] = -1;
    }

    // ---- the tables
    const int chunks = (p.width + kForkEntries - 1) / kForkEntries;
    for (int64_t u = blockIdx.x; u < (int64_t)p.rows_out * chunks; u += gridDim.x) {
        const int r = (int)(u / chunks), j0 = (int)(u - (int64_t)r * chunks) * kForkEntries + tid;
        const int parent = p.parents[r];
        unsigned ignored = 0;
        const bool row = parent >= 0 && parent < p.rows_in;
        const int have = row ? pages_of(p.lens[parent], p.block_size, shift, p.width, ignored) : 0;
        int v[kForkEntries / kForkThreads];
#pragma unroll
        for (int i = 0; i < kForkEntries / kForkThreads; ++i) {
            const int j = j0 + i * kForkThreads;
            v[i] = -1;
            if (j >= have) continue;
            v[i] = j == have - 1 && (rank[r] & 1) ? fresh(rank[r] >> 1) : p.table[parent * p.stride + j];
        }
#pragma unroll
        for (int i = 0; i < kForkEntries / kForkThreads; ++i) {
            const int j = j0 + i * kForkThreads;
            if (j < p.width) p.new_table[r * p.new_stride + j] = v[i];
        }
    }
    if (bad) raise_status(status, bad);
}

// ---------------------------------------------------------------------------
// Copies of pages, 16 bytes at a time, kCopyPieces of a thread under way. A unit is a
// part of one page of one cache; the CTAs take units in turn, since how many there are is known
// on the device only. Bound: HBM, each byte read and written once. For small copies (2 layers, pages of 16 KB: 2.4
// us) and layouts without long runs; 24 layers of 48 x 8 beams took 189 us so, and 129 in bulk.

constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 8;
constexpr int kCachesPerLaunch = 256;

struct CopyParams {
    char *cache[kCachesPerLaunch];
    const int32_t *src, *dst, *tokens, *count;
    unsigned int *status;
    int64_t pairs;
    int64_t block, token, head;       // strides in bytes
    int caches, num_blocks, block_size, parts;
    int row_pieces, head_pieces;      // of a token, of a head
    bool heads_first;                 // a head's tokens lie together
    int runs, run_token;              // of a page: runs `head` apart, bytes of a token in one
    int fault;
};

__global__ void __launch_bounds__(kCopyThreads, 4)
copy_pages_kernel(const __grid_constant__ CopyParams p)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    int64_t pairs = p.pairs;
    if (p.count) pairs = min(pairs, (int64_t)max(*p.count, 0));
    const int64_t each = (int64_t)p.caches * p.parts;
    for (int64_t u = blockIdx.x; u < pairs * each; u += gridDim.x) {
        const int64_t n = u / each;
        const int rest = (int)(u - n * each), cache = rest / p.parts, part = rest - cache * p.parts;
        const int from = p.src[n], to = p.dst[n];
        int tokens = p.tokens ? p.tokens[n] : p.block_size;
        if (from == -1 || to == -1) continue;
        if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks || tokens < 0 || tokens > p.block_size) {
            if (threadIdx.x == 0) raise_status(p.status, kStatusBadIndex);
            if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) continue;
            tokens = min(max(tokens, 0), p.block_size);
        }
        if (from == to) continue;
        const int pieces = tokens * p.row_pieces, e0 = part * kCopyThreads * kCopyPieces + threadIdx.x;
        const char *src = p.cache[cache] + from * p.block;
        char *dst = p.cache[cache] + to * p.block;
        uint4 v[kCopyPieces];
        int64_t at[kCopyPieces];
#pragma unroll
        for (int k = 0; k < kCopyPieces; ++k) {
            const int e = e0 + k * kCopyThreads;
            at[k] = -1;
            if (e >= pieces) continue;
            int token, head, piece;
            if (p.heads_first) {
                const int row = e / p.head_pieces;
                piece = e - row * p.head_pieces;
                head = row / tokens;
                token = row - head * tokens;
            } else {
                token = e / p.row_pieces;
                piece = e - token * p.row_pieces;
                head = piece / p.head_pieces;
                piece -= head * p.head_pieces;
            }
            at[k] = token * p.token + head * p.head + piece * 16;
            v[k] = *reinterpret_cast<const uint4 *>(src + at[k]);
        }
#pragma unroll
        for (int k = 0; k < kCopyPieces; ++k)
            if (at[k] >= 0) *reinterpret_cast<uint4 *>(dst + at[k]) = v[k];
    }
}

// The same by bulk copies (92 % of the copy bandwidth; 1.5 GB of moved pages 258 us, 284 by the
// kernel above), for pages whose tokens lie in long runs: through a ring in shared memory, kAhead
// loads and as many stores under way, all issued by one lane. The 32 lanes of the CTA look up 32 parts at
// a time. (24 layers of 48 x 8 beams, with the tables: 135 us; with 2 CTAs of twice the parts and ring 142. 8 tokens of 320 bytes
// of pages of 32, 32 layers of 20 x 16 beams: 14.5 and 25; in parts of 4 KB 14, but long pages of few tokens 28 for 23.5.)
constexpr int kRunBytes = 8192;             // of a run at once
constexpr int kRing = 4, kAhead = 2;
constexpr int kBulkPerSm = 6;
// Bytes of a page that is one run, of a run of a head, and of all pages, from which on they are used. 16,000 pages of
// 2 KB: 18 us, and 41 by threads; 128,000 runs of up to 2 KB, 8 to a page: 117 and 69 (1 GB in runs of 8 KB: 334 and
// 370); 8.9 of 16 MB: 6.4 and 8.3.
constexpr int64_t kLeastPage = 1024, kLeastRun = 4096, kLeastBulk = 2 << 20;

__global__ void __launch_bounds__(32)
copy_runs_kernel(const __grid_constant__ CopyParams p)
{
    extern __shared__ __align__(128) char copy_ring[];     // [kRing][kRunBytes]
    __shared__ uint64_t full[kRing];
    __shared__ char *to[kRing];
    __shared__ uint32_t size[kRing];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kRing; ++i) ptx::mbar_init(ptx::smem_addr(full + i), 1);
        ptx::fence_mbar_init();
    }
    __syncwarp();
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    int64_t pairs = p.pairs;
    if (p.count) pairs = min(pairs, (int64_t)max(*p.count, 0));
    // the parts of one number of all pages, then those of the next: where few tokens of each are copied, the
    // later ones are empty
    const int64_t each = (int64_t)p.caches * p.runs, units = pairs * each * p.parts;
    int64_t loads = 0, stores = 0;
    bool ok = true;
    auto store = [&] {
        const int s = (int)(stores % kRing);
        ok = ptx::mbar_wait_bounded(ptx::smem_addr(full + s), (stores / kRing) & 1, nullptr, p.status);
        if (!ok) return;
        ptx::bulk_store(to[s], ptx::smem_addr(copy_ring + s * kRunBytes), size[s]);
        ptx::bulk_commit_group();
        ++stores;
    };
    for (int64_t u0 = blockIdx.x; u0 < units; u0 += 32ll * gridDim.x) {
        const int64_t u = u0 + (int64_t)lane * gridDim.x;
        const char *src = nullptr;
        char *dst = nullptr;
        int bytes = 0;
        if (u < units) {
            const int part = (int)(u / (pairs * each));
            const int64_t within = u - part * (pairs * each), n = within / each;
            const int rest = (int)(within - n * each), cache = rest / p.runs, run = rest - cache * p.runs;
            const int from = p.src[n], dest = p.dst[n];
            int tokens = p.tokens ? p.tokens[n] : p.block_size;
            if (tokens < 0 || tokens > p.block_size) {
                if (from != -1 && dest != -1) raise_status(p.status, kStatusBadIndex);
                tokens = min(max(tokens, 0), p.block_size);
            }
            if (from == -1 || dest == -1 || from == dest) {
            } else if (from < 0 || from >= p.num_blocks || dest < 0 || dest >= p.num_blocks) {
                raise_status(p.status, kStatusBadIndex);
            } else {
                const int64_t at = run * p.head + (int64_t)part * kRunBytes;
                bytes = max(0, min(kRunBytes, tokens * p.run_token - part * kRunBytes));
                src = p.cache[cache] + from * p.block + at;
                dst = p.cache[cache] + dest * p.block + at;
            }
        }
        unsigned some = __ballot_sync(0xFFFFFFFFu, bytes > 0);
        while (some) {
            const int l = __ffs(some) - 1;
            some &= some - 1;
            const uint64_t from = __shfl_sync(0xFFFFFFFFu, (uint64_t)src, l), dest = __shfl_sync(0xFFFFFFFFu, (uint64_t)dst, l);
            const uint32_t n = __shfl_sync(0xFFFFFFFFu, (uint32_t)bytes, l);
            if (lane > 0 || !ok) continue;
            const int s = (int)(loads % kRing);
            // the store that read this place last: at most kRing - kAhead - 1 are committed after it
            ptx::bulk_wait_read<kRing - kAhead - 1>();
            to[s] = reinterpret_cast<char *>(dest);
            size[s] = n;
            ptx::mbar_arrive_expect_tx(ptx::smem_addr(full + s), n);
#ifdef AWQ_FAULT_TEST
            if (!p.fault || blockIdx.x > 0)
#endif
                ptx::bulk_load(ptx::smem_addr(copy_ring + s * kRunBytes), reinterpret_cast<const void *>(from), n,
                               ptx::smem_addr(full + s));
            if (++loads > kAhead) store();
        }
    }
    if (lane > 0) return;
    while (ok && stores < loads) store();
    // after a wait that ran out: the copies on their way land before the shared memory goes
    for (int64_t i = stores; i < loads; ++i)
        ptx::mbar_wait_bounded(ptx::smem_addr(full + i % kRing), (i / kRing) & 1, nullptr, nullptr);
    ptx::bulk_wait_all();
}

// ---------------------------------------------------------------------------
// Used blocks as a bitmap, set from the tables (a bit that is set twice stays set: no
// counts, and no order that results could depend on); then free blocks and moves are
// numbered by the bits before them. Bound for large caches: the work of L2, in which every entry sets a random
// bit (2.2 million of 2.5 million blocks: 17 us of 27; bytes instead of bits are not faster, and ranges of blocks in
// shared memory, joined word by word, 8 % at best).

constexpr int kPageThreads = 512;
constexpr int kListWords = 256;           // of the bitmap, for a CTA

// Sum of v over the threads before this one, and over all.
template <int kThreads = kPageThreads>
__device__ __forceinline__ int block_scan(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before + s - v;
}

__global__ void __launch_bounds__(kPageThreads)
clear_kernel(uint4 *words, int64_t n)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    for (int64_t i = (int64_t)blockIdx.x * kPageThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kPageThreads)
        words[i] = make_uint4(0, 0, 0, 0);
}

// Calls f(row, its pages, entry) for the tables' entries in eights: entry is the first, the next ones lie `apart`
// further. Shared out over `threads` threads of which this is number `thread`, whole warps: neighbouring
// lanes have neighbouring entries, 256 entries of a row a warp; but where there are more short rows than warps,
// a row has no more lanes than it needs. (3,941 rows of a page, free blocks, replayed: 8 us, and 18 with a row a warp, as each
// waits for 16 rows in turn; 80,000 rows: 18 and 228.)
template <typename F>
__device__ __forceinline__ void each_eight(const PagesProblem &p, int64_t thread, int64_t threads, unsigned &bad, F f)
{
    const int shift = __ffs(p.block_size) - 1, lane = threadIdx.x & 31;
    const int parts = (p.width + 255) / 256;
    int share = 5;                       // 2^share lanes a row
    while (share > 0 && 4 << share >= p.width && (int64_t)p.rows > threads >> share) --share;
    const int64_t units = (int64_t)p.rows * parts, beside = 32 >> share;
    for (int64_t u = (thread / 32 * beside) + (lane >> share); u < units; u += threads / 32 * beside) {
        const int r = (int)(parts == 1 ? u : u / parts), part = (int)(u - (int64_t)r * parts);
        f(r, pages_of(p.lens[r], p.block_size, shift, p.width, bad), 256 * part + (lane & ((1 << share) - 1)), 1 << share);
    }
}

// Calls f for every entry of the tables' pages and of `held` that is a block; reports those that are none.
template <typename F>
__device__ __forceinline__ void each_used(const PagesProblem &p, int64_t thread, int64_t threads, unsigned &bad, F f)
{
    auto check = [&](int block) {
        if (block < 0 || block >= p.num_blocks) bad |= kStatusBadIndex;
        else f(block);
    };
    each_eight(p, thread, threads, bad, [&](int r, int have, int j0, int apart) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i * apart < have) v[i] = p.table[r * p.stride + j0 + i * apart];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i * apart < have) check(v[i]);
    });
    for (int64_t i = thread; i < p.num_held; i += threads)
        if (p.held[i] != -1) check(p.held[i]);
}

// The tables with the new numbers that `moved` gives for blocks from `first` on.
template <typename F>
__device__ __forceinline__ void renumber(const PagesProblem &p, int64_t thread, int64_t threads, int first, F moved)
{
    unsigned ignored = 0;
    each_eight(p, thread, threads, ignored, [&](int r, int have, int j0, int apart) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * apart;
            v[i] = j < have ? p.table[r * p.stride + j] : -1;
            if (v[i] >= p.num_blocks || v[i] < 0) v[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v[i] >= first) v[i] = moved(v[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i * apart < p.width) p.new_table[r * p.new_stride + j0 + i * apart] = v[i];
    });
}

// What block b's entry in the lists is: `rank` used blocks lie before it, `used` there are, of which the first
// `stays` below `used` stay; of the others each takes the free block of its own rank there.
__device__ __forceinline__ void list_block(const PagesProblem &p, int b, bool in_use, int rank, int used, int stays)
{
    if (p.free_blocks) {
        p.free_blocks[in_use ? p.num_blocks - 1 - rank : b - rank] = in_use ? -1 : b;
        return;
    }
    if (!in_use && b < used) p.dst[b - rank] = b;
    if (in_use && b >= used) p.src[rank - stays] = b;
    if (!in_use || b < used) p.block_map[b] = in_use ? b : -1;
    if (b < p.num_blocks / 2 && b >= used - stays) p.src[b] = p.dst[b] = -1;
}

__global__ void __launch_bounds__(kPageThreads)
mark_kernel(const __grid_constant__ PagesProblem p, unsigned int *status)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    unsigned bad = 0;
    each_used(p, (int64_t)blockIdx.x * kPageThreads + threadIdx.x, (int64_t)gridDim.x * kPageThreads, bad,
              [&](int b) { atomicOr(&p.workspace[b >> 5], 1u << (b & 31)); });
    if (bad) raise_status(status, bad);
}

// How many blocks of each kListWords words are used.
__global__ void __launch_bounds__(kPageThreads)
count_kernel(const __grid_constant__ PagesProblem p)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const int words = (p.num_blocks + 31) / 32, lane = threadIdx.x & 31;
    const int groups = (words + kListWords - 1) / kListWords;
    for (int g = (blockIdx.x * kPageThreads + threadIdx.x) / 32; g < groups; g += gridDim.x * kPageThreads / 32) {
        int n = 0;
#pragma unroll
        for (int i = lane; i < kListWords; i += 32)
            if (g * kListWords + i < words) n += __popc(p.workspace[g * kListWords + i]);
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0) p.groups[g] = n;
    }
}

// A CTA numbers the blocks of kListWords words, a lane a block. It adds up the counts before them, and
// all of them, by itself.
__global__ void __launch_bounds__(kPageThreads)
list_kernel(const __grid_constant__ PagesProblem p)
{
    __shared__ int sums[kPageThreads / 32], before_word[kListWords];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const int words = (p.num_blocks + 31) / 32, w0 = blockIdx.x * kListWords, w = w0 + tid;
    const int counts = (words + kListWords - 1) / kListWords;
    int before = 0, all = 0, ignored;
    for (int i = tid; i < counts; i += kPageThreads) {
        const int n = p.groups[i];
        all += n;
        if (i < blockIdx.x) before += n;
    }
    const uint32_t word = tid < kListWords && w < words ? p.workspace[w] : 0;
    int used, used_before;
    block_scan(all, sums, used);
    block_scan(before, sums, used_before);
    const int at = used_before + block_scan(__popc(word), sums, ignored);
    if (tid < kListWords) before_word[tid] = at;
    int stays = 0;
    if (!p.free_blocks) {
        int stay = 0;
        for (int i = tid; i < counts; i += kPageThreads)
            if ((i + 1) * (32ll * kListWords) <= used) stay += p.groups[i];
        const int rest = used / (32 * kListWords) * kListWords + tid;      // words of the count that `used` falls into
        if (tid < kListWords && rest * 32 < used) {
            const int left = used - rest * 32;
            stay += __popc(left >= 32 ? p.workspace[rest] : p.workspace[rest] & ((1u << left) - 1));
        }
        block_scan(stay, sums, stays);
        if (tid < kListWords && w < words) p.prefix[w] = at;       // for the ranks that move_kernel looks up
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        if (p.free_blocks) {
            p.counts[0] = p.num_blocks - used;
            p.counts[1] = used;
        } else {
            *p.moves = used - stays;
        }
    }
#pragma unroll 4
    for (int i = warp; i < kListWords; i += kPageThreads / 32) {
        const int b = (w0 + i) * 32 + lane;
        if (w0 + i >= words || b >= p.num_blocks) continue;
        const uint32_t bits = p.workspace[w0 + i];
        list_block(p, b, bits >> lane & 1, before_word[i] + __popc(bits & ((1u << lane) - 1)), used, stays);
    }
}

// The map of the blocks that move, and the tables with the new numbers.
__global__ void __launch_bounds__(kPageThreads)
move_kernel(const __grid_constant__ PagesProblem p)
{
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const int moves = *p.moves;
    const int64_t thread = (int64_t)blockIdx.x * kPageThreads + threadIdx.x, threads = (int64_t)gridDim.x * kPageThreads;
    for (int64_t i = thread; i < moves; i += threads) p.block_map[p.src[i]] = p.dst[i];
    auto before = [&](int b) { return p.prefix[b >> 5] + __popc(p.workspace[b >> 5] & ((1u << (b & 31)) - 1)); };
    // the first block that moves tells how many stay
    const int first = moves > 0 ? p.src[0] : p.num_blocks, stays = moves > 0 ? before(first) : 0;
    renumber(p, thread, threads, first, [&](int b) { return p.dst[before(b) - stays]; });
}

// All of it in one launch of one cluster, for caches of up to kClusterWords words and small tables. Each CTA marks
// its share of the entries in a bitmap of its own, then owns an eighth of the words: joins them from all
// CTAs' bitmaps, counts and lists them. (Free blocks of 256 rows of up to 256 pages: 7.4 us replayed, 14.8 in
// launches of their own for marking and listing; compacted 18.)
constexpr int kCluster = 8, kClusterThreads = 1024;
constexpr int kClusterWords = kCluster * kClusterThreads;       // a word a thread
constexpr int64_t kClusterEntries = 1 << 18;

__global__ void __launch_bounds__(kClusterThreads)
pages_cluster_kernel(const __grid_constant__ PagesProblem p, unsigned int *status)
{
    extern __shared__ uint32_t bitmap[];            // [words]
    __shared__ uint32_t own[kClusterThreads];       // the CTA's words, and the used blocks before them
    __shared__ int prefix[kClusterThreads], sums[kClusterThreads / 32], total;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = ptx::cluster_rank();
    const int words = (p.num_blocks + 31) / 32, each = (words + kCluster - 1) / kCluster;
    const int thread = rank * kClusterThreads + tid, threads = kCluster * kClusterThreads;
    for (int i = tid; i < words; i += kClusterThreads) bitmap[i] = 0;
    __syncthreads();
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    unsigned bad = 0;
    each_used(p, thread, threads, bad, [&](int b) { atomicOr(&bitmap[b >> 5], 1u << (b & 31)); });
    if (bad) raise_status(status, bad);
    ptx::cluster_sync();
    const int w = rank * each + tid;
    uint32_t word = 0;
    if (tid < each && w < words) {
#pragma unroll
        for (int c = 0; c < kCluster; ++c) word |= ptx::cluster_load_u32(ptx::cluster_addr(ptx::smem_addr(bitmap + w), c));
    }
    own[tid] = word;
    int mine;
    int before = block_scan<kClusterThreads>(__popc(word), sums, mine);
    if (tid == 0) total = mine;
    ptx::cluster_sync();
    int used = 0;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) {
        const int n = (int)ptx::cluster_load_u32(ptx::cluster_addr(ptx::smem_addr(&total), c));
        used += n;
        if (c < rank) before += n;
    }
    prefix[tid] = before;
    int stays = used;
    // used blocks before block b, from the CTA that owns its word
    auto used_before = [&](int b) {
        const int at = b >> 5, c = at / each, i = at - c * each;
        return (int)ptx::cluster_load_u32(ptx::cluster_addr(ptx::smem_addr(prefix + i), c)) +
               __popc(ptx::cluster_load_u32(ptx::cluster_addr(ptx::smem_addr(own + i), c)) & ((1u << (b & 31)) - 1));
    };
    if (p.free_blocks) {
        __syncthreads();
    } else {
        ptx::cluster_sync();
        if (used < words * 32) stays = used_before(used);
    }
    if (thread == 0) {
        if (p.free_blocks) {
            p.counts[0] = p.num_blocks - used;
            p.counts[1] = used;
        } else {
            *p.moves = used - stays;
        }
    }
    for (int i = warp; i < each; i += kClusterThreads / 32) {
        const int b = (rank * each + i) * 32 + lane;
        if (b >= p.num_blocks) continue;
        list_block(p, b, own[i] >> lane & 1, prefix[i] + __popc(own[i] & ((1u << lane) - 1)), used, stays);
    }
    if (!p.free_blocks) {
        ptx::cluster_sync();           // the lists are there for all
        for (int i = thread; i < used - stays; i += threads) p.block_map[p.src[i]] = p.dst[i];
        renumber(p, thread, threads, used, [&](int b) { return p.dst[used_before(b) - stays]; });
    }
    ptx::cluster_sync();               // none ends while others read its words
}

} // namespace

cudaError_t launch_fork_pages(const ForkProblem &p, cudaStream_t stream)
{
    cudaError_t e = allow_shared((const void *)fork_kernel, 2 * kForkRows * sizeof(int));
    if (e != cudaSuccess) return e;
    const int64_t chunks = (p.width + kForkEntries - 1) / kForkEntries;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(304, p.rows_out * chunks));
    ForkProblem prob = p;
    unsigned int *status = device_status_word();
    void *args[] = {&prob, &status};
    return launch_dependent((const void *)fork_kernel, grid, kForkThreads,
                            (size_t)(p.rows_in + p.rows_out) * sizeof(int), stream, args);
}

cudaError_t launch_copy_pages(const CopyProblem &c, cudaStream_t stream)
{
    for (int64_t n0 = 0; n0 < c.num_caches; n0 += kCachesPerLaunch) {
        CopyParams p{};
        p.caches = (int)std::min<int64_t>(c.num_caches - n0, kCachesPerLaunch);
        for (int i = 0; i < p.caches; ++i) p.cache[i] = static_cast<char *>(c.caches[n0 + i]);
        p.src = c.src;
        p.dst = c.dst;
        p.tokens = c.tokens;
        p.count = c.count;
        p.status = device_status_word();
        p.pairs = c.pairs;
        p.block = c.layout.block_stride * 2;
        p.token = c.layout.token_stride * 2;
        p.head = c.layout.head_stride * 2;
        p.num_blocks = c.num_blocks;
        p.block_size = c.block_size;
        p.head_pieces = c.head_dim / 8;
        p.row_pieces = c.kv_heads * p.head_pieces;
        p.heads_first = c.layout.head_stride > c.layout.token_stride;
        const int64_t row = c.head_dim * 2, page = row * c.kv_heads * c.block_size;
        const bool whole = p.head == row && p.token == row * c.kv_heads;      // a page is one run
        p.runs = whole ? 1 : c.kv_heads;
        p.run_token = (int)(whole ? row * c.kv_heads : row);
        const bool runs = (whole ? page >= kLeastPage : p.token == row && row * c.block_size >= kLeastRun) &&
                          page * c.pairs * p.caches >= kLeastBulk;
#ifdef AWQ_FAULT_TEST
        p.fault = fault_injection();
#endif
        void *args[] = {&p};
        cudaError_t e;
        if (runs) {
            p.parts = (int)(((int64_t)p.run_token * c.block_size + kRunBytes - 1) / kRunBytes);
            e = allow_shared((const void *)copy_runs_kernel, kRing * kRunBytes);
            if (e == cudaSuccess)
                e = launch_dependent((const void *)copy_runs_kernel,
                                     std::min<int64_t>(152 * kBulkPerSm, c.pairs * p.caches * p.runs * p.parts), 32,
                                     kRing * kRunBytes, stream, args);
        } else {
            p.parts = (c.block_size * p.row_pieces + kCopyThreads * kCopyPieces - 1) / (kCopyThreads * kCopyPieces);
            e = launch_dependent((const void *)copy_pages_kernel, std::min<int64_t>(152 * 4, c.pairs * p.caches * p.parts),
                                 kCopyThreads, 0, stream, args);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pages(const PagesProblem &p, cudaStream_t stream)
{
    PagesProblem prob = p;
    unsigned int *status = device_status_word();
    const int64_t words = (p.num_blocks + 31) / 32;
    void *mark_args[] = {&prob, &status};
    if (words <= kClusterWords && (int64_t)p.rows * p.width + p.num_held <= kClusterEntries) {
        const cudaError_t e = allow_shared((const void *)pages_cluster_kernel, kClusterWords * sizeof(uint32_t));
        if (e != cudaSuccess) return e;
        return launch_dependent((const void *)pages_cluster_kernel, kCluster, kClusterThreads, words * sizeof(uint32_t), stream,
                                mark_args, kCluster);
    }
    uint4 *clear = reinterpret_cast<uint4 *>(p.workspace);
    int64_t n = (words + 3) / 4;
    void *clear_args[] = {&clear, &n};
    cudaError_t e = launch_dependent((const void *)clear_kernel,
                                     std::max<int64_t>(1, std::min<int64_t>(152, n / (4 * kPageThreads))), kPageThreads, 0,
                                     stream, clear_args);
    if (e != cudaSuccess) return e;
    const int64_t pieces = (int64_t)p.rows * ((p.width + 255) / 256);
    const int64_t grid = std::max<int64_t>(
        1, std::min<int64_t>(608, std::max((pieces * 32 + kPageThreads - 1) / kPageThreads,
                                           (p.num_held + kPageThreads - 1) / kPageThreads)));
    e = launch_dependent((const void *)mark_kernel, grid, kPageThreads, 0, stream, mark_args);
    if (e != cudaSuccess) return e;
    prob.prefix = reinterpret_cast<int *>(p.workspace + (words + 3) / 4 * 4);
    prob.groups = prob.prefix + words;
    const int64_t groups = (words + kListWords - 1) / kListWords;
    void *args[] = {&prob};
    e = launch_dependent((const void *)count_kernel, std::min<int64_t>(304, (groups * 32 + kPageThreads - 1) / kPageThreads),
                         kPageThreads, 0, stream, args);
    if (e == cudaSuccess) e = launch_dependent((const void *)list_kernel, groups, kPageThreads, 0, stream, args);
    if (e != cudaSuccess || p.free_blocks) return e;
    return launch_dependent((const void *)move_kernel, grid, kPageThreads, 0, stream, args);
}

} // namespace awq

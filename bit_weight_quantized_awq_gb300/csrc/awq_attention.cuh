// awq_attention.cuh -- what the tree-attention kernels share: how the work of
// a ragged batch is split over the CTAs, and how the pieces of a split row
// block are joined.
//
// Rows. The queries that share one head of the cache are, for a request with n
// new tokens and `group` query heads a key-value head, n * group rows; row r is
// token r / group, head r % group of the group. They are cut into blocks of RB
// rows, the keys into tiles of KT. The work is the row blocks of all (request,
// key-value head) pairs, one after another on a line: a block takes kBlockCost
// units for its beginning and end and its weight for each tile. CTA c of G takes
// the tiles that begin in [c U / G, (c + 1) U / G). So every CTA has the same work
// whatever the lengths are, a long cache is split along its length, and nothing
// but the lengths on the device is needed to find a CTA's range. Where the CTAs
// divide well by the key-value heads, each head has a line of its own and its share
// of the CTAs, neighbouring ones for the heads: they then go through the same
// tokens at the same time, whose keys of all heads lie side by side in HBM.
//
// Pieces. A row block whose tiles fall to several CTAs is a sum of pieces
// (m, l, O): O = sum_j exp2(s_j - m) v_j and l = sum_j exp2(s_j - m), joined by
//   M = max m,  L = sum l exp2(m - M),  out = (sum O exp2(m - M)) / L.
// Each piece is written to a slot of its CTA (one that begins its row block in
// slot 1, any other in slot 0), and the CTA that has a row block's last piece
// writes down what there is to join. A second kernel, launched as a programmatic dependent, joins
// the pieces in the order of the CTAs, so the sum's order is the same in every
// call, and no CTA ever waits for another. (Joined by whichever CTA came last the
// pieces took 10 to 20 us at 256 rows: one CTA's loads, behind a fence.)
//
// Where the bounds allow only a few row blocks of few tiles, none is cut: a CTA has
// each, or (few-row kernel) a cluster, whose CTAs join their parts through shared memory.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace attn {

// What is to be joined because a CTA has the last piece of a split row block.
struct Join {
    int valid;
    int cta0, cta1;         // the pieces: slot 1 of cta0, slot 0 of the line's CTAs after it up to cta1
    int h, rb, token0, rows;
};

struct Params {
    const void *q;
    int64_t q_token_stride, q_head_stride;
    void *out;
    float *lse;
    const int32_t *table;
    int64_t table_stride;
    const void *v_data;     // the values, for the few elements read outside the tiles
    int64_t v_block_stride, v_token_stride, v_head_stride;
    const int32_t *ctx, *cu, *mask;
    float *partials;        // slots, two a CTA
    struct Join *joins;     // one a CTA; null, as the slots, where no row block is cut
    unsigned int *status;
    int table_width, mask_words;
    int B, tokens, q_heads, kv_heads, group, head_dim, num_blocks;
    int shift;              // log2 of the block size
    int min_units;          // a CTA takes at least this many units: one tile at least
    int whole;              // row blocks are not split: one unit each, and nothing to join
    int share;              // log2 of the CTAs (a cluster) that share each row block; 0 unless whole
    int lines;              // 1, or kv_heads: lines of work, one a key-value head (see Work)
    float scale_log2;       // scale * log2(e): scores are kept in powers of two
#ifdef AWQ_FAULT_TEST
    int fault;              // CTA 0's producer issues nothing (fault-test build only)
#endif
};

// ---- the work ----

// One CTA's part of one row block: key tiles tile0 .. tile1 - 1 of `tiles`.
struct Segment {
    int b, h, rb;
    int ctx, n, token0;     // the request: context length, new tokens, first row of q
    int tile0, tile1, tiles;
    int64_t u0;             // the row block's first unit
    __device__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

template <int RB, int KT, int kBlockCost>
struct Work {
    int64_t units, pos, end;   // pos: where this CTA's next row block begins on the line
    int ctas;               // CTAs of the line that take part
    int heads, head0, cta;  // heads of the line, the first of them, and this CTA's number in it
    int b, h, rb, tile, tiles;
    int ctx, n, token0, row_blocks;

    // Tiles of one row block: all keys, or without a mask (causal) those up to
    // the block's last token.
    static __device__ int tiles_of(const Params &p, int ctx, int n, int rb)
    {
        int seen = n;
        if (p.mask == nullptr && n > 1) seen = min(n, ((rb + 1) * RB - 1) / p.group + 1);
        return (ctx + seen + KT - 1) / KT;
    }
    static __device__ int row_blocks_of(const Params &p, int n) { return (n * p.group + RB - 1) / RB; }
    // Units a tile: 1, or 2 where it takes the tensor-core kernel twice as long -- a
    // block of more than 128 rows, and any first block, whose tiles come from HBM
    // (those of the later ones are in L2 by then).
    static __device__ int weight_of(const Params &p, int n, int rb)
    {
        return RB > 128 && (rb == 0 || n * p.group - rb * RB > 128) ? 2 : 1;
    }
    static __device__ int64_t block_units(const Params &p, int ctx, int n, int rb)
    {
        return p.whole ? 1 : kBlockCost + (int64_t)tiles_of(p, ctx, n, rb) * weight_of(p, n, rb);
    }
    static __device__ int64_t head_units(const Params &p, int ctx, int n)
    {
        const int blocks = row_blocks_of(p, n);
        if (blocks == 0 || p.whole) return blocks;
        if (p.mask != nullptr)
            return (blocks - 1) * block_units(p, ctx, n, 0) + block_units(p, ctx, n, blocks - 1);
        int64_t sum = 0;
        for (int rb = 0; rb < blocks; ++rb) sum += block_units(p, ctx, n, rb);
        return sum;
    }
    // a / b of non-negative numbers; most fit 32 bits, whose division takes a tenth of the time
    static __device__ int64_t quotient(int64_t a, int64_t b)
    {
        return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
    }
    __device__ int64_t begin_of(int c) const { return quotient(units * c, ctas); }
    __device__ int cta_of(int64_t u) const { return (int)quotient((u + 1) * ctas - 1, units); }
    // A block's first tile begins at its first unit u0, tile i at u0 + kBlockCost + i
    // weight: the first one that begins at `at` or later.
    static __device__ int first_tile(const Params &p, int64_t at, int64_t u0, int weight, int tiles)
    {
        if (at <= u0) return 0;
        if (p.whole) return tiles;
        const int64_t i = weight == 1 ? at - u0 - kBlockCost : (at - u0 - kBlockCost + 1) >> 1;   // weight is 1 or 2
        return (int)min((int64_t)tiles, max((int64_t)1, i));
    }

    // All threads of the CTA (THREADS of them, a multiple of 32) call this. False if there is
    // nothing to do for this CTA; if the lengths are not valid, for any CTA.
    template <int THREADS>
    __device__ bool find(const Params &p)
    {
        __shared__ int64_t warp_units[THREADS / 32];
        __shared__ struct {
            int64_t before, per_head;
            int b, ctx, token0, n;
        } found;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        if (tid == 0 && p.joins != nullptr) p.joins[blockIdx.x].valid = 0;
        heads = p.lines == 1 ? p.kv_heads : 1;
        head0 = p.lines == 1 ? 0 : blockIdx.x % p.lines;
        cta = p.lines == 1 ? blockIdx.x >> p.share : blockIdx.x / p.lines;
        const int per = (p.B + THREADS - 1) / THREADS;
        const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
        int64_t mine = 0, units0 = 0;          // of the thread's requests, and of the first of them
        int bad = 0, ctx0 = 0, at0 = 0, len0 = 0;
        for (int i = b_lo; i < b_hi; ++i) {
            const int c = p.ctx[i], t0 = p.cu[i], t1 = p.cu[i + 1];
            if (t0 < 0 || t1 < t0 || t1 > p.tokens || c < 0 ||
                (int64_t)c + (t1 - t0) > ((int64_t)p.table_width << p.shift)) {
                bad = 1;
                break;
            }
            const int64_t u = head_units(p, c, t1 - t0);
            mine += u * heads;
            if (i == b_lo) {
                units0 = u;
                ctx0 = c;
                at0 = t0;
                len0 = t1 - t0;
            }
        }
        int64_t su = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t ou = __shfl_up_sync(0xFFFFFFFFu, su, d);
            if (lane >= d) su += ou;
        }
        if (lane == 31) warp_units[warp] = su;
        if (__syncthreads_or(bad)) {
            if (tid == 0 && blockIdx.x == 0) raise_status(p.status, kStatusBadIndex);
            return false;
        }
        units = 0;
        int64_t before = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += warp_units[w];
            units += warp_units[w];
        }
        before += su - mine;
        if (units == 0) return false;
        const int there = p.lines == 1 ? gridDim.x >> p.share : gridDim.x / p.lines;
        if (p.whole && units <= there) {     // a row block a CTA: no divisions, half a microsecond
            ctas = (int)units;
            pos = cta;
            end = cta + 1;
        } else {
            ctas = (int)min((int64_t)there, max((int64_t)1, quotient(units, p.min_units)));
            pos = begin_of(cta);
            end = begin_of(cta + 1);
        }
        if (cta >= ctas) return false;
        if (pos >= before && pos < before + mine) {
            // the request, and what has just been read of it
            int i = b_lo;
            int64_t per_head = units0;
            while (pos >= before + per_head * heads) {
                before += per_head * heads;
                ++i;
                ctx0 = p.ctx[i];
                at0 = p.cu[i];
                len0 = p.cu[i + 1] - at0;
                per_head = head_units(p, ctx0, len0);
            }
            found.b = i;
            found.ctx = ctx0;
            found.token0 = at0;
            found.n = len0;
            found.before = before;
            found.per_head = per_head;
        }
        __syncthreads();
        b = found.b;
        ctx = found.ctx;
        token0 = found.token0;
        n = found.n;
        row_blocks = row_blocks_of(p, n);
        int64_t rem = pos - found.before;
        const int64_t per_head = found.per_head;
        h = per_head == 1 ? (int)rem : (int)quotient(rem, per_head);
        rem -= h * per_head;
        rb = 0;
        if (p.whole) {
            rb = (int)rem;
            rem = 0;
        } else if (p.mask != nullptr) {
            const int64_t full = block_units(p, ctx, n, 0);
            rb = (int)min((int64_t)(row_blocks - 1), quotient(rem, full));
            rem -= rb * full;
        } else {
            for (int64_t u = block_units(p, ctx, n, 0); rem >= u; u = block_units(p, ctx, n, rb)) {
                rem -= u;
                ++rb;
            }
        }
        tiles = tiles_of(p, ctx, n, rb);
        tile = first_tile(p, pos, pos - rem, weight_of(p, n, rb), tiles);
        pos -= rem;
        return true;
    }

    __device__ void load(const Params &p)
    {
        ctx = p.ctx[b];
        token0 = p.cu[b];
        n = p.cu[b + 1] - token0;
        row_blocks = row_blocks_of(p, n);
    }

    __device__ void next_block(const Params &p)
    {
        pos += block_units(p, ctx, n, rb);
        tile = 0;
        if (pos >= end) return;
        if (++rb == row_blocks) {
            rb = 0;
            if (++h == heads) {
                h = 0;
                do {
                    ++b;
                    load(p);
                } while (n == 0);
            }
        }
        tiles = tiles_of(p, ctx, n, rb);
    }

    // The next segment of this CTA's range; every thread walks the same list.
    __device__ bool next(const Params &p, Segment &s)
    {
        if (pos < end && tile == tiles) next_block(p);   // the range began behind a block's last tile
        if (pos >= end) return false;
        s.b = b;
        s.h = head0 + h;
        s.rb = rb;
        s.ctx = ctx;
        s.n = n;
        s.token0 = token0;
        s.tile0 = tile;
        s.tile1 = first_tile(p, end, pos, weight_of(p, n, rb), tiles);
        s.tiles = tiles;
        s.u0 = pos;
        if (s.tile1 <= s.tile0) return false;            // no tile begins in what is left
        next_block(p);
        return true;
    }

    // The slot of this CTA's piece.
    static __device__ int slot_of(const Segment &s) { return 2 * blockIdx.x + (s.tile0 == 0 ? 1 : 0); }
    // One thread of a CTA whose segment is a row block's last piece, of several.
    __device__ void note_join(const Params &p, const Segment &s, int rows) const
    {
        p.joins[blockIdx.x] = Join{1, cta_of(s.u0) * p.lines + (int)blockIdx.x % p.lines, (int)blockIdx.x, s.h, s.rb, s.token0, rows};
    }
};

// ---- masks ----

// Bits of the drafted tokens that token t of the segment's request sees, from
// drafted token j0 on (32 of them; those at or past n are 0).
__device__ __forceinline__ uint32_t seen_bits(const Params &p, const Segment &s, int t, int j0)
{
    if (j0 >= s.n) return 0;
    uint32_t bits;
    if (p.mask == nullptr) {
        const int k = t - j0 + 1;
        bits = k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1;
    } else {
        const int32_t *row = p.mask + (int64_t)(s.token0 + t) * p.mask_words;
        const int w = j0 >> 5, o = j0 & 31;   // j0 >= 0
        const uint32_t lo = w < p.mask_words ? (uint32_t)row[w] : 0u;
        const uint32_t hi = o && w + 1 < p.mask_words ? (uint32_t)row[w + 1] : 0u;
        bits = __funnelshift_r(lo, hi, o);
    }
    const int left = s.n - j0;
    return left >= 32 ? bits : bits & ((1u << left) - 1);
}

// Bits of the keys key0 .. key0 + 31 that token t sees.
__device__ __forceinline__ uint32_t seen32(const Params &p, const Segment &s, int t, int key0)
{
    const int before = s.ctx - key0;   // keys of the context among them
    if (before >= 32) return 0xFFFFFFFFu;
    if (before > 0) return ((1u << before) - 1) | (seen_bits(p, s, t, 0) << before);
    return seen_bits(p, s, t, -before);
}

// ---- page numbers ----

// A producer warp's view of a request's block table: a window of 32 entries, one a
// lane, and the next window already asked for, so that no tile waits for its
// pages' numbers (with each tile's looked up just ahead of it, a warp spent a
// microsecond a tile waiting).
struct Pages {
    const int32_t *table;
    int last;               // the last page of the request
    int base, now, next;    // the window's first page; this lane's entries of both windows
    __device__ int entry(int page) const { return page <= last ? table[page] : 0; }
    __device__ void open(const Params &p, const Segment &s, int first, int lane)
    {
        table = p.table + (int64_t)s.b * p.table_stride;
        last = (s.ctx + s.n - 1) >> p.shift;
        base = first;
        now = entry(base + lane);
        next = entry(base + 32 + lane);
    }
    // This lane's page's block, called by all lanes; pages only grow, and those of one
    // call lie in one window. A number outside the cache is reported, and becomes one
    // past the tensor, where TMA reads zeros.
    __device__ int block(const Params &p, int page, int lane)
    {
        if (__any_sync(0xFFFFFFFFu, page >= base + 32)) {
            base += 32;
            now = next;
            next = entry(base + 32 + lane);
        }
        const int id = __shfl_sync(0xFFFFFFFFu, now, (page - base) & 31);
        if (id >= 0 && id < p.num_blocks) return id;
        if (page <= last) raise_status(p.status, kStatusBadIndex);
        return p.num_blocks;
    }
};

// ---- element types ----

// The softmax weights are rounded to q's type for their product with v: a matrix
// instruction takes both operands in one 16-bit type, and a second product with what the
// rounding left would double that work. Their sum takes them unrounded, in fp32. Relative
// error of the output against 64 bits, its own rounding included: fp16 2.6e-4 to 2.9e-4, bf16
// 2.2e-3 to 2.4e-3; with weights in fp32 2.1e-4 and 1.7e-3.
template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    // Weights are scaled by 2^kBias before they are rounded to fp16, whose
    // normal range starts at 2^-14: small weights then keep all their bits.
    // The factor leaves with the division by the sum, which has it too.
    static constexpr float kBias = 14.f;
    static constexpr uint32_t kExpMask = 0x7C00u;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float to_float(uint16_t v) { return __half2float(__ushort_as_half(v)); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr float kBias = 0.f;   // the exponent range of fp32
    static constexpr uint32_t kExpMask = 0x7F80u;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float to_float(uint16_t v) { return __bfloat162float(__ushort_as_bfloat16(v)); }
};

template <typename T>
__device__ __forceinline__ bool has_nonfinite(uint32_t two)
{
    constexpr uint32_t m = Elem<T>::kExpMask;
    return (two & m) == m || ((two >> 16) & m) == m;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- waiting ----

// ptx::mbar_wait_bounded without a suspend hint: for waits in a chain of short
// steps, where a suspended thread's way back would count.
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *status)
{
    long long t0 = 0;
    for (int i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63) != 63) continue;
        if (t0 == 0) t0 = clock64();
        if (*abort) return false;
        if (clock64() - t0 > ptx::kWaitLimitCycles) {
            *abort = 1;
            if (status) atomicOr(status, 1u);
            return false;
        }
    }
}

// ---- joining ----

// A slot: O as [column / 4][row][4], then m and l of every row.
constexpr int slot_floats(int rb, int dp) { return rb * dp + 2 * rb; }
__host__ __device__ constexpr int slot_at(int rb, int r, int c) { return (c >> 2) * rb * 4 + r * 4 + (c & 3); }
// Floats of the partial sums of `ctas` CTAs: their slots and what is to be joined.
constexpr size_t scratch_floats(int ctas, int rb, int dp)
{
    return (size_t)ctas * (2 * slot_floats(rb, dp) + sizeof(Join) / sizeof(float));
}

__device__ __forceinline__ void store_lse(const Params &p, int token0, int h, int r, float m, float l)
{
    if (p.lse == nullptr) return;
    const int64_t t = token0 + r / p.group;
    const int64_t head = (int64_t)h * p.group + r % p.group;
    p.lse[t * p.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Joins the pieces of the row block whose last one CTA blockIdx.x had. A thread has
// eight columns of one row, or of a part of its pieces: `subs` threads share a
// row's pieces and add up their parts in shared memory. All loads of eight pieces
// are under way at a time -- the pieces come from L2, half a microsecond away, and
// there are seldom more -- so that a join is about one such wait.
constexpr int kJoinThreads = 256;
constexpr int kJoinColumns = 8;
// eight-column groups of a CTA
constexpr int join_groups(int rb) { return rb <= 16 ? 4 : 1; }

template <typename T, int RB, int DP>
__global__ void __launch_bounds__(kJoinThreads)
attention_join_kernel(const __grid_constant__ Params p)
{
    constexpr int kGroups = join_groups(RB), kBatch = 8;
    __shared__ float part[kJoinThreads][kJoinColumns + 1];
    __shared__ float part_m[kJoinThreads], part_l[kJoinThreads];
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const Join j = p.joins[blockIdx.x];
    if (!j.valid) return;
    const int lanes = RB <= 16 ? 16 : (j.rows + 31) & ~31;          // rows, rounded up
    const int per_sub = lanes * kGroups, subs = kJoinThreads / per_sub;
    const int sub = threadIdx.x / per_sub, in_sub = threadIdx.x % per_sub;
    const int r = in_sub % lanes;
    const int col = (blockIdx.y * kGroups + in_sub / lanes) * kJoinColumns;
    const bool works = sub < subs && r < j.rows && col < p.head_dim;
    constexpr int SF = slot_floats(RB, DP);
    float m = -INFINITY, l = 0.f;
    float acc[kJoinColumns];
#pragma unroll
    for (int e = 0; e < kJoinColumns; ++e) acc[e] = 0.f;
    if (works) {
        const int step = subs * p.lines;
        for (int c = j.cta0 + sub * p.lines; c <= j.cta1; c += kBatch * step) {
            float4 v[kBatch][2];
            float mc[kBatch], lc[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int cu = c + u * step;
                mc[u] = -INFINITY;
                if (cu > j.cta1) continue;
                const float *from = p.partials + (int64_t)(2 * cu + (cu == j.cta0 ? 1 : 0)) * SF;
                mc[u] = __ldcg(from + RB * DP + r);
                lc[u] = __ldcg(from + RB * DP + RB + r);
                v[u][0] = __ldcg(reinterpret_cast<const float4 *>(from + slot_at(RB, r, col)));
                v[u][1] = __ldcg(reinterpret_cast<const float4 *>(from + slot_at(RB, r, col + 4)));
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) top = fmaxf(top, mc[u]);
            const float mx = top == -INFINITY ? 0.f : top, w0 = exp2_fast(m - mx);
            l *= w0;
#pragma unroll
            for (int e = 0; e < kJoinColumns; ++e) acc[e] *= w0;
            m = top;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (c + u * step > j.cta1) break;
                const float w = exp2_fast(mc[u] - mx);
                l += lc[u] * w;
                const float *f = reinterpret_cast<const float *>(v[u]);
#pragma unroll
                for (int e = 0; e < kJoinColumns; ++e) acc[e] += f[e] * w;
            }
        }
    }
    if (subs > 1) {
        part_m[threadIdx.x] = m;
        part_l[threadIdx.x] = l;
#pragma unroll
        for (int e = 0; e < kJoinColumns; ++e) part[threadIdx.x][e] = acc[e];
        __syncthreads();
        if (sub != 0 || !works) return;
        float top = m;
        for (int i = 1; i < subs; ++i) top = fmaxf(top, part_m[i * per_sub + in_sub]);
        const float mx = top == -INFINITY ? 0.f : top, w0 = exp2_fast(m - mx);
        l *= w0;
#pragma unroll
        for (int e = 0; e < kJoinColumns; ++e) acc[e] *= w0;
        for (int i = 1; i < subs; ++i) {
            const float w = exp2_fast(part_m[i * per_sub + in_sub] - mx);
            l += part_l[i * per_sub + in_sub] * w;
#pragma unroll
            for (int e = 0; e < kJoinColumns; ++e) acc[e] += part[i * per_sub + in_sub][e] * w;
        }
        m = top;
    }
    if (sub != 0 || !works) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = j.rb * RB + r;
    const int64_t token = j.token0 + row / p.group;
    T *out = static_cast<T *>(p.out) + (token * p.q_heads + (int64_t)j.h * p.group + row % p.group) * p.head_dim + col;
    *reinterpret_cast<uint4 *>(out) =
        make_uint4(Elem<T>::pack(acc[0] * inv, acc[1] * inv), Elem<T>::pack(acc[2] * inv, acc[3] * inv),
                   Elem<T>::pack(acc[4] * inv, acc[5] * inv), Elem<T>::pack(acc[6] * inv, acc[7] * inv));
    if (col == 0) store_lse(p, j.token0, j.h, row, m == -INFINITY ? 0.f : m, l);
}

// What a call's bounds allow, as sizes whose products stay far below 2^63 whatever the
// bounds are: rows a key-value head (a request has no more new tokens than q has), row
// blocks of all heads, key tiles of a request.
inline int64_t rows_bound(const awq_tree_attention_t &a) { return std::min(a.max_new, a.tokens) * (a.q_heads / a.kv_heads); }
inline int64_t blocks_bound(const awq_tree_attention_t &a, int rows)
{
    const int64_t a_head = std::max<int64_t>(1, (rows_bound(a) + rows - 1) / rows);
    return std::min(a.B * a.kv_heads * a_head, int64_t(1) << 31);
}
inline int64_t tiles_bound(const awq_tree_attention_t &a, int keys)
{
    return std::max<int64_t>(1, (a.max_context + a.max_new + keys - 1) / keys);
}

// CTAs of a launch, at most `most` of them, and how its work is laid out: `units` as
// the bounds allow, `min_units` a CTA.
inline int lay_out(Params &p, int most, int64_t units)
{
    const int a_head = most / p.kv_heads;
    p.lines = a_head * p.kv_heads * 10 >= most * 9 ? p.kv_heads : 1;
    const int64_t line = units / p.lines;
    return (int)std::min<int64_t>(most / p.lines, std::max<int64_t>(1, line / p.min_units)) * p.lines;
}

// Launches a main kernel of `ctas` CTAs and, unless there is one only or each has
// whole row blocks, its join; only then does the call need scratch.
template <typename T, int RB, int DP, typename K>
cudaError_t launch_pair(K kernel, int ctas, int threads, int smem, cudaStream_t stream, const CUtensorMap &tk,
                        const CUtensorMap &tv, Params &p)
{
    const bool cut = ctas > 1 && !p.whole;
    if (cut) {
        Scratch sc{};
        if (!get_scratch(stream, scratch_floats(ctas, RB, DP), 0, &sc)) return cudaErrorMemoryAllocation;
        p.partials = sc.partials;
        p.joins = reinterpret_cast<Join *>(sc.partials + (size_t)ctas * 2 * slot_floats(RB, DP));
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << p.share;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.share > 0 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, p);
    if (e != cudaSuccess) return e;
    if (cut) {
        constexpr int kColumns = kJoinColumns * join_groups(RB);
        cfg.gridDim = dim3((unsigned)ctas, (unsigned)(p.head_dim + kColumns - 1) / kColumns);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, attention_join_kernel<T, RB, DP>, p);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

} // namespace attn
} // namespace awq

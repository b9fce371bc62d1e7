// awq_attention.cuh -- what the tree-attention kernels share: how the work of
// a ragged batch is split over the CTAs, and how the pieces of a split row
// block are joined.
//
// Rows. The queries that share one head of the cache are, for a request with n
// new tokens and `group` query heads a key-value head, n * group rows; row r is
// token r / group, head r % group of the group. They are cut into blocks of RB
// rows, the keys into tiles of KT. A unit of work is one (request, key-value
// head, row block, key tile); all units, in that order, form one line, and CTA c
// of G takes the range [c U / G, (c + 1) U / G). So every CTA has the same work
// whatever the lengths are, a long cache is split along its length, and nothing
// but the lengths on the device is needed to find a CTA's range.
//
// Pieces. A row block whose tiles fall to several CTAs is a sum of pieces
// (m, l, O): O = sum_j exp2(s_j - m) v_j and l = sum_j exp2(s_j - m), joined by
//   M = max m,  L = sum l exp2(m - M),  out = (sum O exp2(m - M)) / L.
// Each piece is written to a slot of its CTA (its first segment in slot 0, its
// last in slot 1); the CTA that finishes a row block's last piece -- told by a
// counter -- joins all of them in the order of the CTAs, so the sum's order is
// the same in every call, and no CTA ever waits for another.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace attn {

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
    float *partials;
    unsigned int *counters, *status;
    int table_width, mask_words;
    int B, tokens, q_heads, kv_heads, group, head_dim, num_blocks;
    int shift;              // log2 of the block size
    int min_units;          // a CTA takes at least this many units (fewer pieces to join)
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
    int64_t u0;             // unit of the row block's first tile
    int block;              // counter of the row block
    __device__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

template <int RB, int KT>
struct Work {
    int64_t units, pos, end;
    int ctas;               // CTAs that take part
    int b, h, rb, tile, tiles;
    int ctx, n, token0, row_blocks, block0;

    // Tiles of one row block: all keys, or without a mask (causal) those up to
    // the block's last token.
    static __device__ int tiles_of(const Params &p, int ctx, int n, int rb)
    {
        int seen = n;
        if (p.mask == nullptr) seen = min(n, ((rb + 1) * RB - 1) / p.group + 1);
        return (ctx + seen + KT - 1) / KT;
    }
    static __device__ int row_blocks_of(const Params &p, int n) { return (n * p.group + RB - 1) / RB; }
    static __device__ int64_t head_units(const Params &p, int ctx, int n)
    {
        const int blocks = row_blocks_of(p, n);
        if (p.mask != nullptr) return (int64_t)blocks * tiles_of(p, ctx, n, 0);
        int64_t sum = 0;
        for (int rb = 0; rb < blocks; ++rb) sum += tiles_of(p, ctx, n, rb);
        return sum;
    }
    __device__ int64_t begin_of(int c) const { return units * c / ctas; }
    __device__ int cta_of(int64_t u) const { return (int)(((u + 1) * ctas - 1) / units); }

    // All threads of the CTA (THREADS of them, a multiple of 32) call this. False if there is
    // nothing to do for this CTA; if the lengths are not valid, for any CTA.
    template <int THREADS>
    __device__ bool find(const Params &p)
    {
        __shared__ int64_t warp_units[THREADS / 32];
        __shared__ int warp_blocks[THREADS / 32];
        __shared__ int64_t found_units;
        __shared__ int found_b, found_block;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int per = (p.B + THREADS - 1) / THREADS;
        const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
        int64_t mine = 0;
        int blocks = 0, bad = 0;
        for (int i = b_lo; i < b_hi; ++i) {
            const int c = p.ctx[i], t0 = p.cu[i], t1 = p.cu[i + 1];
            if (t0 < 0 || t1 < t0 || t1 > p.tokens || c < 0 ||
                (int64_t)c + (t1 - t0) > ((int64_t)p.table_width << p.shift)) {
                bad = 1;
                break;
            }
            mine += head_units(p, c, t1 - t0) * p.kv_heads;
            blocks += row_blocks_of(p, t1 - t0) * p.kv_heads;
        }
        int64_t su = mine;
        int sb = blocks;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t ou = __shfl_up_sync(0xFFFFFFFFu, su, d);
            const int ob = __shfl_up_sync(0xFFFFFFFFu, sb, d);
            if (lane >= d) {
                su += ou;
                sb += ob;
            }
        }
        if (lane == 31) {
            warp_units[warp] = su;
            warp_blocks[warp] = sb;
        }
        if (__syncthreads_or(bad)) {
            if (tid == 0 && blockIdx.x == 0) raise_status(p.status, kStatusBadIndex);
            return false;
        }
        units = 0;
        int64_t before = 0;
        int before_blocks = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) {
                before += warp_units[w];
                before_blocks += warp_blocks[w];
            }
            units += warp_units[w];
        }
        before += su - mine;
        before_blocks += sb - blocks;
        if (units == 0) return false;
        ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, units / p.min_units));
        if ((int)blockIdx.x >= ctas) return false;
        pos = begin_of(blockIdx.x);
        end = begin_of(blockIdx.x + 1);
        if (pos >= before && pos < before + mine) {
            int i = b_lo;
            for (;; ++i) {
                const int c = p.ctx[i], len = p.cu[i + 1] - p.cu[i];
                const int64_t u = head_units(p, c, len) * p.kv_heads;
                if (pos < before + u) break;
                before += u;
                before_blocks += row_blocks_of(p, len) * p.kv_heads;
            }
            found_b = i;
            found_units = before;
            found_block = before_blocks;
        }
        __syncthreads();
        b = found_b;
        block0 = found_block;
        load(p);
        int64_t rem = pos - found_units;
        const int64_t per_head = head_units(p, ctx, n);
        h = (int)(rem / per_head);
        rem -= h * per_head;
        rb = 0;
        if (p.mask != nullptr) {
            tiles = tiles_of(p, ctx, n, 0);
            rb = (int)(rem / tiles);
            rem -= (int64_t)rb * tiles;
        } else {
            tiles = tiles_of(p, ctx, n, 0);
            while (rem >= tiles) {
                rem -= tiles;
                tiles = tiles_of(p, ctx, n, ++rb);
            }
        }
        tile = (int)rem;
        return true;
    }

    __device__ void load(const Params &p)
    {
        ctx = p.ctx[b];
        token0 = p.cu[b];
        n = p.cu[b + 1] - token0;
        row_blocks = row_blocks_of(p, n);
    }

    // The next segment of this CTA's range; every thread walks the same list.
    __device__ bool next(const Params &p, Segment &s)
    {
        if (pos >= end) return false;
        const int count = (int)min((int64_t)(tiles - tile), end - pos);
        s.b = b;
        s.h = h;
        s.rb = rb;
        s.ctx = ctx;
        s.n = n;
        s.token0 = token0;
        s.tile0 = tile;
        s.tile1 = tile + count;
        s.tiles = tiles;
        s.u0 = pos - tile;
        s.block = block0 + h * row_blocks + rb;
        pos += count;
        if (pos < end) {
            tile = 0;
            if (++rb == row_blocks) {
                rb = 0;
                if (++h == p.kv_heads) {
                    h = 0;
                    block0 += p.kv_heads * row_blocks;
                    do {
                        ++b;
                        load(p);
                    } while (n == 0);
                }
            }
            tiles = tiles_of(p, ctx, n, rb);
        }
        return true;
    }

    // The slot of CTA c's piece of the row block whose first unit is u0.
    __device__ int slot_of(int c, int64_t u0) const { return 2 * c + (begin_of(c) >= u0 ? 0 : 1); }
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

// ---- element types ----

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

constexpr int slot_floats(int rb, int dp) { return rb * dp + 2 * rb; }

// Writes rows of a finished row block: `v` the four values of columns c .. c + 3.
template <typename T>
__device__ __forceinline__ void store4(const Params &p, const Segment &s, int r, int c, float4 v)
{
    if (c >= p.head_dim) return;
    const int64_t t = s.token0 + r / p.group;
    const int64_t head = (int64_t)s.h * p.group + r % p.group;
    uint2 o;
    o.x = Elem<T>::pack(v.x, v.y);
    o.y = Elem<T>::pack(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (t * p.q_heads + head) * p.head_dim + c) = o;
}

__device__ __forceinline__ void store_lse(const Params &p, const Segment &s, int r, float m, float l)
{
    if (p.lse == nullptr) return;
    const int64_t t = s.token0 + r / p.group;
    const int64_t head = (int64_t)s.h * p.group + r % p.group;
    p.lse[t * p.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// The CTA that finishes the last piece of a row block joins all of them.
// Called by the THREADS consecutive threads whose index is tid, after they have
// written this CTA's piece to its slot; `rows` of the block's RB rows exist.
// red: shared, join_floats(RB, THREADS) floats. bar: a named barrier of these threads.
// kByColumn: a slot's O is stored [column / 4][row][4] instead of [row][column], and
// a thread joins neighbouring columns of one row.
// The pieces lie in L2, half a microsecond away: a thread asks for 16
// four-float values (of E places and 16 / E pieces) before it uses the first.
// Not inlined, its arguments by value: the callers' loops keep their registers.
constexpr int kJoinPieces = 16;   // pieces whose weights are held at a time
constexpr int join_floats(int rb, int threads) { return threads + 2 * rb + kJoinPieces * rb; }

template <typename T, int RB, int DP, int THREADS, bool kByColumn, typename W>
__device__ __noinline__ void join(const Params &p, const W work, const Segment s, int tid, int rows, float *red, int bar)
{
    __shared__ unsigned arrived;
    const int c0 = work.cta_of(s.u0), c1 = work.cta_of(s.u0 + s.tiles - 1);
    __threadfence();
    ptx::named_barrier(bar, THREADS);
    if (tid == 0) {
        const unsigned old = atomicAdd(p.counters + s.block, 1u);
        arrived = old;
        if (old == (unsigned)(c1 - c0)) p.counters[s.block] = 0;   // as the next call expects it
    }
    ptx::named_barrier(bar, THREADS);
    if (arrived != (unsigned)(c1 - c0)) return;
    __threadfence();
    constexpr int SF = slot_floats(RB, DP);
    float *row_m = red + THREADS, *row_l = row_m + RB, *weight = row_l + RB;
    auto slot_at = [&](int c) { return p.partials + (int64_t)work.slot_of(c, s.u0) * SF; };
    // maxima and sums of every row: `subs` threads share a row's pieces
    constexpr int subs = THREADS / RB;
    static_assert(subs >= 1, "a thread a row at least");
    {
        const int r = tid % RB, sub = tid / RB;
        float m = -INFINITY, l = 0.f;
#pragma unroll 8
        for (int c = c0 + sub; c <= c1; c += subs) {
            const float *ml = slot_at(c) + RB * DP + r;
            const float mc = __ldcg(ml), lc = __ldcg(ml + RB);
            const float nm = fmaxf(m, mc), mx = nm == -INFINITY ? 0.f : nm;
            l = l * exp2_fast(m - mx) + lc * exp2_fast(mc - mx);
            m = nm;
        }
        if (subs > 1) {
            red[tid] = m;
            ptx::named_barrier(bar, THREADS);
            float all = -INFINITY;
            for (int i = 0; i < subs; ++i) all = fmaxf(all, red[i * RB + r]);
            l *= exp2_fast(m - (all == -INFINITY ? 0.f : all));
            m = all;
            ptx::named_barrier(bar, THREADS);
            red[tid] = l;
            ptx::named_barrier(bar, THREADS);
            l = 0.f;
            for (int i = 0; i < subs; ++i) l += red[i * RB + r];
        }
        if (sub == 0) {
            row_m[r] = m == -INFINITY ? 0.f : m;
            row_l[r] = l;
            if (r < rows) store_lse(p, s, s.rb * RB + r, row_m[r], l);
        }
    }
    ptx::named_barrier(bar, THREADS);
    constexpr int kPlaces = RB * DP / 4 / THREADS;
    constexpr int E = kByColumn ? 4 : kPlaces < 8 ? kPlaces : 8, PU = 16 / E;
    // by column: the threads' rows, and how many of them share a row's columns
    const int share = kByColumn && rows * 2 <= THREADS ? 2 : 1;
    const int places = kByColumn ? DP / 4 / share : rows * (DP / 4), step = kByColumn ? E : E * THREADS;
    for (int first = 0; first < places; first += step) {
        float4 acc[E];
        int at[E], row[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            int r, c4;
            if (kByColumn) {
                r = share == 2 ? tid & (THREADS / 2 - 1) : tid;
                c4 = ((share == 2 && tid >= THREADS / 2 ? places : 0) + first + i) * 4;
                r = min(r, rows - 1);
            } else {
                const int e = min(first + tid + i * THREADS, places - 1);
                r = e / (DP / 4);
                c4 = (e % (DP / 4)) * 4;
            }
            row[i] = r | (c4 << 16);
            at[i] = kByColumn ? c4 * RB + r * 4 : r * DP + c4;
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int cc = c0; cc <= c1; cc += kJoinPieces) {
            const int n = min(kJoinPieces, c1 - cc + 1);
            if (c1 - c0 >= kJoinPieces || first == 0) {      // the weights held are others, or none
                ptx::named_barrier(bar, THREADS);
#pragma unroll 4
                for (int i = tid; i < n * RB; i += THREADS)
                    weight[i] = exp2_fast(__ldcg(slot_at(cc + i / RB) + RB * DP + i % RB) - row_m[i % RB]);
                ptx::named_barrier(bar, THREADS);
            }
            for (int j = 0; j < n; j += PU) {
                float4 v[PU][E];
#pragma unroll
                for (int u = 0; u < PU; ++u) {
                    const float *slot = slot_at(cc + min(j + u, n - 1));
#pragma unroll
                    for (int i = 0; i < E; ++i) v[u][i] = __ldcg(reinterpret_cast<const float4 *>(slot + at[i]));
                }
#pragma unroll
                for (int u = 0; u < PU; ++u) {
                    if (j + u >= n) break;
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float w = weight[(j + u) * RB + (row[i] & 0xFFFF)];
                        acc[i].x += v[u][i].x * w;
                        acc[i].y += v[u][i].y * w;
                        acc[i].z += v[u][i].z * w;
                        acc[i].w += v[u][i].w * w;
                    }
                }
            }
        }
        if (kByColumn && (share == 2 ? tid & (THREADS / 2 - 1) : tid) >= rows) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (!kByColumn && first + tid + i * THREADS >= places) break;
            const int r = row[i] & 0xFFFF;
            const float l = row_l[r], inv = l == 0.f ? 0.f : 1.f / l;
            store4<T>(p, s, s.rb * RB + r, row[i] >> 16,
                      make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
        }
    }
    ptx::named_barrier(bar, THREADS);
}

} // namespace attn
} // namespace awq

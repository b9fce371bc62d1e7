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
// last in slot 1), and the CTA that has a row block's last piece writes down what
// there is to join. A second kernel, launched as a programmatic dependent, joins
// the pieces in the order of the CTAs, so the sum's order is the same in every
// call, and no CTA ever waits for another. (Joined by whichever CTA came last the
// pieces took 10 to 20 us at 256 rows: one CTA's loads, behind a fence.)
#pragma once

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
    int cta0, slot0;        // CTA of the first piece, and its slot; the others are slot 0 of
    int cta1;               // the CTAs after it up to cta1
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
    struct Join *joins;     // one a CTA
    unsigned int *status;
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
    __device__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

template <int RB, int KT>
struct Work {
    int64_t units, pos, end;
    int ctas;               // CTAs that take part
    int b, h, rb, tile, tiles;
    int ctx, n, token0, row_blocks;

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
        __shared__ int64_t found_units;
        __shared__ int found_b;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        if (tid == 0) p.joins[blockIdx.x].valid = 0;
        const int per = (p.B + THREADS - 1) / THREADS;
        const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
        int64_t mine = 0;
        int bad = 0;
        for (int i = b_lo; i < b_hi; ++i) {
            const int c = p.ctx[i], t0 = p.cu[i], t1 = p.cu[i + 1];
            if (t0 < 0 || t1 < t0 || t1 > p.tokens || c < 0 ||
                (int64_t)c + (t1 - t0) > ((int64_t)p.table_width << p.shift)) {
                bad = 1;
                break;
            }
            mine += head_units(p, c, t1 - t0) * p.kv_heads;
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
            }
            found_b = i;
            found_units = before;
        }
        __syncthreads();
        b = found_b;
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
        pos += count;
        if (pos < end) {
            tile = 0;
            if (++rb == row_blocks) {
                rb = 0;
                if (++h == p.kv_heads) {
                    h = 0;
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
    // One thread of a CTA whose segment is a row block's last piece, of several.
    __device__ void note_join(const Params &p, const Segment &s, int rows) const
    {
        const int c0 = cta_of(s.u0);
        p.joins[blockIdx.x] = Join{1, c0, slot_of(c0, s.u0), (int)blockIdx.x, s.h, s.rb, s.token0, rows};
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

// Joins the pieces of the row block whose last one CTA blockIdx.x had, columns
// 32 blockIdx.y .. + 31. A thread has one row; where the rows are fewer than the
// threads, `subs` of them share a row's pieces and add up their parts in shared
// memory. Eight 16-byte loads a piece, of two pieces, are under way at a time: the
// pieces come from L2.
constexpr int kJoinThreads = 256;

template <typename T, int RB, int DP>
__global__ void __launch_bounds__(kJoinThreads)
attention_join_kernel(const __grid_constant__ Params p)
{
    __shared__ float part[kJoinThreads][33];
    __shared__ float part_m[kJoinThreads], part_l[kJoinThreads];
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    const Join j = p.joins[blockIdx.x];
    const int c0 = blockIdx.y * 32;
    if (!j.valid || c0 >= p.head_dim) return;
    const int lanes = j.rows <= 16 ? 16 : (j.rows + 31) & ~31;      // rows, rounded up
    const int subs = kJoinThreads / lanes;
    const int r = threadIdx.x % lanes, sub = threadIdx.x / lanes;
    constexpr int SF = slot_floats(RB, DP);
    auto slot = [&](int c) { return p.partials + (int64_t)(c == j.cta0 ? j.slot0 : 2 * c) * SF; };
    float m = -INFINITY, l = 0.f;
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
    if (sub < subs && r < j.rows) {
#pragma unroll 8
        for (int c = j.cta0 + sub; c <= j.cta1; c += subs) m = fmaxf(m, __ldcg(slot(c) + RB * DP + r));
        const float mx = m == -INFINITY ? 0.f : m;
        for (int c = j.cta0 + sub; c <= j.cta1; c += 2 * subs) {
            float4 v[2][8];
            float mc[2], lc[2];
            const bool both = c + subs <= j.cta1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u && !both) break;
                const float *from = slot(c + u * subs);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[u][i] = __ldcg(reinterpret_cast<const float4 *>(from + slot_at(RB, r, c0 + 4 * i)));
                mc[u] = __ldcg(from + RB * DP + r);
                lc[u] = __ldcg(from + RB * DP + RB + r);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u && !both) break;
                const float w = exp2_fast(mc[u] - mx);
                l += lc[u] * w;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[4 * i] += v[u][i].x * w;
                    acc[4 * i + 1] += v[u][i].y * w;
                    acc[4 * i + 2] += v[u][i].z * w;
                    acc[4 * i + 3] += v[u][i].w * w;
                }
            }
        }
    }
    if (subs > 1) {
        part_m[threadIdx.x] = m;
        part_l[threadIdx.x] = l;
#pragma unroll
        for (int e = 0; e < 32; ++e) part[threadIdx.x][e] = acc[e];
        __syncthreads();
        if (sub != 0 || r >= j.rows) return;
        float top = m;
        for (int i = 1; i < subs; ++i) top = fmaxf(top, part_m[i * lanes + r]);
        const float mx = top == -INFINITY ? 0.f : top, w0 = exp2_fast(m - mx);
        l *= w0;
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] *= w0;
        for (int i = 1; i < subs; ++i) {
            const float w = exp2_fast(part_m[i * lanes + r] - mx);
            l += part_l[i * lanes + r] * w;
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[e] += part[i * lanes + r][e] * w;
        }
        m = top;
    }
    if (sub != 0 || r >= j.rows) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = j.rb * RB + r;
    const int64_t token = j.token0 + row / p.group;
    T *out = static_cast<T *>(p.out) + (token * p.q_heads + (int64_t)j.h * p.group + row % p.group) * p.head_dim + c0;
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        if (c0 + e < p.head_dim)
            *reinterpret_cast<uint4 *>(out + e) =
                make_uint4(Elem<T>::pack(acc[e] * inv, acc[e + 1] * inv), Elem<T>::pack(acc[e + 2] * inv, acc[e + 3] * inv),
                           Elem<T>::pack(acc[e + 4] * inv, acc[e + 5] * inv), Elem<T>::pack(acc[e + 6] * inv, acc[e + 7] * inv));
    if (blockIdx.y == 0) store_lse(p, j.token0, j.h, row, m == -INFINITY ? 0.f : m, l);
}

// Launches a main kernel of `ctas` CTAs and, unless there is one only, its join.
template <typename T, int RB, int DP, typename K>
cudaError_t launch_pair(K kernel, int ctas, int threads, int smem, cudaStream_t stream, const CUtensorMap &tk,
                        const CUtensorMap &tv, Params &p)
{
    Scratch sc{};
    if (!get_scratch(stream, scratch_floats(ctas, RB, DP), 0, &sc)) return cudaErrorMemoryAllocation;
    p.partials = sc.partials;
    p.joins = reinterpret_cast<Join *>(sc.partials + (size_t)ctas * 2 * slot_floats(RB, DP));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, p);
    if (e != cudaSuccess) return e;
    if (ctas > 1) {
        cfg.gridDim = dim3((unsigned)ctas, (unsigned)(p.head_dim + 31) / 32);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, attention_join_kernel<T, RB, DP>, p);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

} // namespace attn
} // namespace awq

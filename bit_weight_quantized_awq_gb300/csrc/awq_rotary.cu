// awq_rotary.cu -- rotary positions of q and k, into new rows, in place or, with the
// values beside the keys, straight into a paged cache.
//
// Angles. cos and sin of position * frequency have to be right for positions in the
// millions, where an fp32 product is off by whole degrees. The frequency is taken in
// turns, F = frac(inv_freq / 2 pi) as a 64-bit fraction; position * F modulo 2^64 is
// then the rest of a turn (the integer product wraps where whole turns fall away), good to
// position * 2^-63 turns, and its upper 32 bits are the argument of sincospif. 1 / 2 pi is
// three fp32 numbers, whose products with inv_freq are exact as pairs: fp64 runs at two operations a
// clock, which was a tenth of the time.
//
// Bound: HBM, every head read and written once. A CTA takes a few tokens and a part of their heads; the
// cosines and sines are computed once for all of the CTA's heads, by all of its threads, and shared
// through shared memory. Each thread asks for its first kItems pieces before that, so that their way in takes
// no time of its own.
// Measured: 16,383 tokens of 64 / 8 heads of 128 bf16 into a cache 108 us, 92 % of the copy bandwidth
// (torch's copy of as many dense bytes takes 106); 30,001 tokens of 16 / 4 heads of 96 with three axes
// 48 us (a dense copy: 41); one token of 32 heads 4.3 us a call. With places of heads worked out item by
// item the first took 152 us; with more tokens a CTA 121 (twice) and 125 (four times); with two items a thread and
// five CTAs an SM 111; with CTAs of only as many warps as have items 117, since the angles then take two turns. A
// shorter way to the angles (fp32 pairs, own series) changed nothing; a thread with another frequency at each
// angle cost 10 %.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 3;           // of an SM

struct Side {                      // of q, k and v; strides in bytes
    const char *src;
    char *dst;
    int64_t src_token, src_head, dst_block, dst_token, dst_head;
};

struct RotaryParams {
    Side side[3];
    const int32_t *positions, *axes;
    const float *inv_freq;
    const int64_t *slot_map;
    unsigned int *status;
    int64_t tokens, slots;
    int num_axes, half, dim;
    int q_heads, turned_heads, heads;   // heads: with v's
    // A head is `items` items, of which `turns` turn something; `lanes` of them beside each other, `blocks` times.
    // A CTA takes per_cta tokens, `abreast` at once, and part_heads blocks of their heads: one of `parts`.
    int items, turns, lanes, blocks, abreast, per_cta, parts, part_heads;
    int shift;
};

// An item: kHalf: kWidth elements (8, 4, 2 or 1) and those that lie rotary_dim / 2 further; kPairs: kWidth
// elements (8, 4 or 2), neighbouring pairs. As many as rotary_dim / 2, or rotary_dim, is a multiple of: with one pair
// a thread and no loads ahead, 17 heads of 72 of which 36 turn took 80 us for 12,911 tokens, and take 18 in twos.
enum Mode { kHalf, kPairs };

template <int kMode, int kWidth>
constexpr int kItems = kMode == kHalf ? std::min(16, 32 / kWidth) : std::min(16, 64 / kWidth);     // of a thread under way

template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t v)
{
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<__half2 *>(&v));
    else return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}

template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b)
{
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Turns two elements a, b by (c, s).
__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a, y = b;
    a = x * c - y * s;
    b = y * c + x * s;
}

// frac(f / 2 pi) in units of 2^-64.
__device__ __forceinline__ uint64_t in_turns(float f)
{
    constexpr float k0 = 0.15915494f, k1 = 6.4206382e-09f, k2 = 7.342739e-17f;      // their sum is 1 / 2 pi to 2^-76
    auto fixed = [](float x) { return (uint64_t)__float2ll_rn((x - rintf(x)) * 0x1p64f); };
    const float a = f * k0, b = f * k1;
    return fixed(a) + fixed(fmaf(f, k0, -a)) + fixed(b) + fixed(fmaf(f, k1, -b)) + fixed(f * k2);
}

// Cosines and sines of a CTA's tokens and their slots, into shared memory.
__device__ __forceinline__ void angles(const RotaryParams &p, int64_t t0, int tokens, float *cosine, float *sine, int64_t *slots)
{
    for (int i = threadIdx.x; i < tokens; i += kThreads) {
        int64_t slot = p.slot_map ? p.slot_map[t0 + i] : 0;
        if (slot < 0 || slot >= p.slots) {
            if (slot != -1) raise_status(p.status, kStatusBadIndex);
            slot = -1;
        }
        slots[i] = slot;
    }
    // a thread has one frequency and goes through the tokens
    const int across = min(p.half, kThreads), rows = kThreads / across, row = threadIdx.x / across;
    for (int i = threadIdx.x - row * across; i < p.half && row < rows; i += across) {
        const uint64_t turns = in_turns(p.inv_freq[i]);
        const int axis = p.axes ? p.axes[i] : 0;
        const bool known = axis >= 0 && axis < p.num_axes;
        if (!known) raise_status(p.status, kStatusBadIndex);
        const int32_t *positions = p.positions + (known ? axis : 0) * p.tokens + t0;
        for (int t = row; t < tokens; t += rows) {
            const uint64_t rest = known ? turns * (uint64_t)(int64_t)positions[t] : 0;
            sincospif((float)(int32_t)(rest >> 32) * 0x1p-31f, &sine[t * p.half + i], &cosine[t * p.half + i]);
        }
    }
}

template <int kWidth>
struct Vector;
template <> struct Vector<8> { using type = uint4; };
template <> struct Vector<4> { using type = uint2; };
template <> struct Vector<2> { using type = uint32_t; };
template <> struct Vector<1> { using type = uint16_t; };

// n angles, at a multiple of n (or of 4) from an aligned start.
template <int n>
__device__ __forceinline__ void take(const float *from, float (&x)[n])
{
#pragma unroll
    for (int i = 0; i < n; i += n % 4 == 0 ? 4 : n % 2 == 0 ? 2 : 1) {
        if constexpr (n % 4 == 0) {
            const float4 v = *reinterpret_cast<const float4 *>(from + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        } else if constexpr (n % 2 == 0) {
            const float2 v = *reinterpret_cast<const float2 *>(from + i);
            x[i] = v.x, x[i + 1] = v.y;
        } else {
            x[i] = from[i];
        }
    }
}

// A thread has one place in one head, of which all is looked up once, and goes through the CTA's tokens,
// kItems of them under way.
template <typename T, int kMode, int kWidth>
__global__ void __launch_bounds__(kThreads, kCtas)
rotary_kernel(const __grid_constant__ RotaryParams p)
{
    using V = typename Vector<kWidth>::type;
    constexpr int kItems = awq::kItems<kMode, kWidth>, kBytes = 2 * kWidth, kEach = kMode == kHalf ? kWidth : kWidth / 2;
    extern __shared__ __align__(16) char rotary_smem[];
    float *cosine = reinterpret_cast<float *>(rotary_smem), *sine = cosine + p.per_cta * p.half;     // [per_cta][half]
    int64_t *slots = reinterpret_cast<int64_t *>(sine + p.per_cta * p.half);
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t group = blockIdx.x / p.parts, t0 = group * p.per_cta;
    const int tokens = (int)min((int64_t)p.per_cta, p.tokens - t0);
    const int own = threadIdx.x / p.lanes;
    const int beside = own / p.part_heads;              // which of the tokens abreast
    const int block = (int)(blockIdx.x - group * p.parts) * p.part_heads + own - beside * p.part_heads;
    const int h = block / p.blocks, lane = (block - h * p.blocks) * p.lanes + threadIdx.x - own * p.lanes;
    const bool works = beside < p.abreast && h < p.heads && lane < p.items;
    const bool v = h >= p.turned_heads, turns = !v && lane < p.turns;
    const int side = v ? 2 : h >= p.q_heads, number = h - (v ? p.turned_heads : h >= p.q_heads ? p.q_heads : 0);
    // the item's first elements in the head, in bytes, and how far the second are; 0: none
    int at = kBytes * lane, more = 0;
    if (kMode == kHalf) {
        if (turns) {
            more = 2 * p.half;
        } else if (v) {
            more = at + kBytes * p.items < 2 * p.dim ? kBytes * p.items : 0;
        } else {
            at = 4 * p.half + 2 * kBytes * (lane - p.turns);
            more = at + kBytes < 2 * p.dim ? kBytes : 0;
        }
    }
    const int64_t src_token = p.side[side].src_token, dst_token = p.side[side].dst_token, dst_block = p.side[side].dst_block;
    const char *src = p.side[side].src + t0 * src_token + number * p.side[side].src_head + at;
    char *dst = p.side[side].dst + (dst_block ? 0 : t0 * dst_token) + number * p.side[side].dst_head + at;

    V a[kItems], b[kItems];
    const int step = p.abreast * kItems, end = works ? tokens : 0;
    auto load = [&](int t1) {
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int t = t1 + u * p.abreast;
            if (t >= end) continue;
            // not a read-only load: this kernel may be resident while the one before writes q, k and v
            const char *from = src + t * src_token;
            a[u] = *reinterpret_cast<const V *>(from);
            if (kMode == kHalf && more) b[u] = *reinterpret_cast<const V *>(from + more);
        }
    };
    load(beside);
    angles(p, t0, tokens, cosine, sine, slots);
    __syncthreads();
    for (int t1 = beside; t1 < end; t1 += step) {
        if (t1 != beside) load(t1);
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int t = t1 + u * p.abreast;
            if (t >= end) continue;
            char *to = dst;
            if (dst_block) {
                const int64_t slot = slots[t];
                if (slot < 0) continue;
                to += (slot >> p.shift) * dst_block + (slot & ((1 << p.shift) - 1)) * dst_token;
            } else {
                to += t * dst_token;
            }
            if (turns) {
                float c[kEach], d[kEach];
                take(cosine + t * p.half + kEach * lane, c);
                take(sine + t * p.half + kEach * lane, d);
                if constexpr (kWidth == 1) {
                    float2 x = unpack<T>(a[u] | (uint32_t)b[u] << 16);
                    turn(x.x, x.y, c[0], d[0]);
                    const uint32_t y = pack<T>(x.x, x.y);
                    a[u] = (uint16_t)y;
                    b[u] = (uint16_t)(y >> 16);
                } else {
                    uint32_t *va = reinterpret_cast<uint32_t *>(&a[u]), *vb = reinterpret_cast<uint32_t *>(&b[u]);
#pragma unroll
                    for (int q = 0; q < kWidth / 2; ++q) {
                        float2 x = unpack<T>(va[q]);
                        if constexpr (kMode == kHalf) {
                            float2 y = unpack<T>(vb[q]);
                            turn(x.x, y.x, c[2 * q], d[2 * q]);
                            turn(x.y, y.y, c[2 * q + 1], d[2 * q + 1]);
                            vb[q] = pack<T>(y.x, y.y);
                        } else {
                            turn(x.x, x.y, c[q], d[q]);
                        }
                        va[q] = pack<T>(x.x, x.y);
                    }
                }
            }
            *reinterpret_cast<V *>(to) = a[u];
            if (kMode == kHalf && more) *reinterpret_cast<V *>(to + more) = b[u];
        }
    }
}

template <typename T>
const void *kernel_of(Mode mode, int width)
{
    if (mode == kPairs)
        return width == 8 ? (const void *)rotary_kernel<T, kPairs, 8>
               : width == 4 ? (const void *)rotary_kernel<T, kPairs, 4> : (const void *)rotary_kernel<T, kPairs, 2>;
    return width == 8 ? (const void *)rotary_kernel<T, kHalf, 8>
           : width == 4 ? (const void *)rotary_kernel<T, kHalf, 4>
           : width == 2 ? (const void *)rotary_kernel<T, kHalf, 2> : (const void *)rotary_kernel<T, kHalf, 1>;
}

} // namespace

cudaError_t launch_rotary(const awq_rotary_t &a, cudaStream_t stream)
{
    RotaryParams p{};
    const bool append = a.slot_map != nullptr;
    p.side[0] = {(const char *)a.q, (char *)a.q_out, 2 * a.q_token_stride, 2 * a.q_head_stride, 0,
                 2 * a.q_out_token_stride, 2 * a.q_out_head_stride};
    p.side[1] = {(const char *)a.k, (char *)a.k_out, 2 * a.k_token_stride, 2 * a.k_head_stride, 0,
                 2 * a.k_out_token_stride, 2 * a.k_out_head_stride};
    if (append) {
        p.side[1].dst = (char *)a.k_cache.data;
        p.side[1].dst_block = 2 * a.k_cache.block_stride;
        p.side[1].dst_token = 2 * a.k_cache.token_stride;
        p.side[1].dst_head = 2 * a.k_cache.head_stride;
        p.side[2] = {(const char *)a.v, (char *)a.v_cache.data, 2 * a.v_token_stride, 2 * a.v_head_stride,
                     2 * a.v_cache.block_stride, 2 * a.v_cache.token_stride, 2 * a.v_cache.head_stride};
    }
    p.positions = a.positions;
    p.axes = a.axes;
    p.inv_freq = a.inv_freq;
    p.slot_map = a.slot_map;
    p.status = device_status_word();
    p.tokens = a.tokens;
    p.slots = append ? a.num_blocks * a.block_size : 1;
    while (append && (1 << p.shift) < a.block_size) ++p.shift;
    p.num_axes = (int)a.num_axes;
    p.half = (int)a.rotary_dim / 2;
    p.dim = (int)a.head_dim;
    p.q_heads = (int)a.q_heads;
    p.turned_heads = (int)(a.q_heads + a.kv_heads);
    p.heads = p.turned_heads + (append ? (int)a.kv_heads : 0);
    const int R = (int)a.rotary_dim, D = (int)a.head_dim;
    const Mode mode = a.pairs ? kPairs : kHalf;
    int width = 8;
    while ((a.pairs ? R : R / 2) % width) width /= 2;
    p.turns = a.pairs ? R / width : R / 2 / width;
    p.items = a.pairs ? D / width : p.turns + ((D - R) / width + 1) / 2;
    p.blocks = (p.items + kThreads - 1) / kThreads;
    p.lanes = (p.items + p.blocks - 1) / p.blocks;
    // The heads are shared out over CTAs, an item a thread, and few heads let several tokens go abreast. More
    // parts than are needed can leave fewer threads idle, but each works out its tokens' angles, and two angles
    // cost about what an item does: 16,383 x 80 heads of 128 take 107.6 us in 5 parts of 16 heads and 111 in 3 of 27;
    // 10,361 x 40 of 64 22.0 in 2 and 24.0 in one.
    const int at_once = kThreads / p.lanes, all = p.heads * p.blocks, items = std::min(16, (mode == kHalf ? 32 : 64) / width);
    const int least = (all + at_once - 1) / at_once;
    double best = 0;
    for (int n = least; n <= std::min({all, 4 * least, least + 8}); ++n) {
        const int heads = (all + n - 1) / n, abreast = at_once / heads;
        const double score = (double)heads * abreast * all / (n * heads) / (1 + (double)n * p.half / (all * p.lanes));
        if (score > best) best = score, p.parts = n, p.part_heads = heads, p.abreast = abreast;
    }
    // as many tokens for a CTA as keep all its threads at their angles and all its loads under way, but
    // not before there are kCtas CTAs an SM
    const int busy = std::max((kThreads + p.half - 1) / p.half, p.abreast * items);
    p.per_cta = (int)std::max<int64_t>(
        1, std::min<int64_t>({busy, (a.tokens * p.parts + kCtas * 152 - 1) / (kCtas * 152), 4096 / p.half}));
    const int64_t grid = (a.tokens + p.per_cta - 1) / p.per_cta * p.parts;
    const size_t smem = 8 * (size_t)p.per_cta * (p.half + 1);
    void *args[] = {&p};
    const void *kernel = a.dtype == AWQ_F16 ? kernel_of<__half>(mode, width) : kernel_of<__nv_bfloat16>(mode, width);
    return launch_dependent(kernel, grid, kThreads, smem, stream, args);
}

} // namespace awq

// awq_rotary.cu -- rotary positions of q and k, into new rows, in place or, with the
// values beside the keys, straight into a paged cache.
//
// Angles. cos and sin of position * frequency have to be right for positions in the
// millions, where an fp32 product is off by whole degrees. The frequency is taken in
// turns, F = frac(inv_freq / 2 pi) as a 64-bit fraction; position * F modulo 2^64 is
// then the exact rest of a turn (the integer product wraps where whole turns fall away),
// good to position * 2^-53 turns (the division by 2 pi, in fp64, once a CTA), and its upper 32
// bits are the argument of sincospif.
//
// Bound: HBM, every head read and written once. A CTA takes a few tokens; a token's
// cosines and sines are computed once and shared by its heads through shared memory.
// Each thread has the loads of kUnits pieces under way before it needs them.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "awq_device.cuh"
#include "awq_internal.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;          // units of a thread under way

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
    int num_axes, half, head_bytes;
    int turned_heads, q_heads, v_heads;
    int turn_units, head_units, copy_units;   // of a turned head: those that are turned, all; of a head of v
    int token_units, per_cta, shift;
};

// kHalf: 8 elements and the 8 that lie rotary_dim / 2 further; kPairs: 4 neighbouring pairs; kSingle:
// one pair of either kind, for rotary_dim / 2 (or rotary_dim) that is no multiple of 8.
enum Mode { kHalf, kPairs, kSingleHalf, kSinglePairs };

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

// What unit `u` of a token is: a head of q, k or v and a place in it.
struct Unit {
    int side, head, at;      // at: bytes from the head's start
    int turn;                // the first pair that it turns, -1 for a copy
};

template <int kMode>
__device__ __forceinline__ Unit unit_of(const RotaryParams &p, int u)
{
    Unit x;
    const int turned = p.turned_heads * p.head_units;
    if (u >= turned) {
        u -= turned;
        x.side = 2;
        x.head = u / p.copy_units;
        x.at = (u - x.head * p.copy_units) * 16;
        x.turn = -1;
        return x;
    }
    x.head = u / p.head_units;
    const int j = u - x.head * p.head_units;
    x.side = x.head >= p.q_heads;
    if (x.side) x.head -= p.q_heads;
    if (j < p.turn_units) {
        x.turn = kMode == kHalf ? 8 * j : kMode == kPairs ? 4 * j : j;
        x.at = kMode == kHalf ? 16 * j : kMode == kPairs ? 16 * j : kMode == kSingleHalf ? 2 * j : 4 * j;
    } else {
        constexpr int kBytes = kMode == kHalf || kMode == kPairs ? 16 : 2;
        x.turn = -1;
        x.at = 4 * p.half + (j - p.turn_units) * kBytes;
    }
    return x;
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const __grid_constant__ RotaryParams p)
{
    extern __shared__ __align__(16) char rotary_smem[];
    const int tid = threadIdx.x;
    // frequencies in turns, cosines and sines [per_cta][half], slots
    uint64_t *turns = reinterpret_cast<uint64_t *>(rotary_smem);
    int64_t *slots = reinterpret_cast<int64_t *>(turns + p.half);
    float *cosine = reinterpret_cast<float *>(slots + p.per_cta + (p.per_cta + p.half) % 2);
    float *sine = cosine + p.per_cta * p.half;
    ptx::launch_dependents();
    ptx::wait_prerequisites();

    const int64_t t0 = (int64_t)blockIdx.x * p.per_cta;
    const int tokens = (int)min((int64_t)p.per_cta, p.tokens - t0);
    for (int i = tid; i < p.half; i += kThreads) {
        const double f = (double)p.inv_freq[i] * 0.15915494309189533577;    // 1 / (2 pi)
        turns[i] = (uint64_t)((f - floor(f)) * 18446744073709551616.);      // of 2^64
    }
    for (int i = tid; i < tokens; i += kThreads) {
        int64_t slot = p.slot_map ? p.slot_map[t0 + i] : 0;
        if (slot < 0 || slot >= p.slots) {
            if (slot != -1) raise_status(p.status, kStatusBadIndex);
            slot = -1;
        }
        slots[i] = slot;
    }
    __syncthreads();
    for (int e = tid; e < tokens * p.half; e += kThreads) {
        const int t = e / p.half, i = e - t * p.half;
        const int axis = p.axes ? p.axes[i] : 0;
        int position = 0;
        if (axis >= 0 && axis < p.num_axes) position = p.positions[axis * p.tokens + t0 + t];
        else raise_status(p.status, kStatusBadIndex);
        const uint64_t rest = turns[i] * (uint64_t)(int64_t)position;
        sincospif((float)(int32_t)(rest >> 32) * 0x1p-31f, &sine[e], &cosine[e]);
    }
    __syncthreads();

    constexpr bool kVector = kMode == kHalf || kMode == kPairs;
    const int units = tokens * p.token_units;
    for (int e0 = tid; e0 < units; e0 += kThreads * kUnits) {
        uint4 a[kUnits], b[kUnits];
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int e = e0 + n * kThreads;
            if (e >= units) continue;
            const int t = e / p.token_units;
            const Unit x = unit_of<kMode>(p, e - t * p.token_units);
            const Side &s = p.side[x.side];
            const char *from = s.src + (t0 + t) * s.src_token + x.head * s.src_head + x.at;
            if (kVector || x.side == 2) {
                // not a read-only load: this kernel may be resident while the one before writes q, k and v
                a[n] = *reinterpret_cast<const uint4 *>(from);
                if (kMode == kHalf && x.turn >= 0) b[n] = *reinterpret_cast<const uint4 *>(from + 2 * p.half);
            } else if (kMode == kSinglePairs && x.turn >= 0) {
                a[n].x = *reinterpret_cast<const uint32_t *>(from);
            } else {
                a[n].x = *reinterpret_cast<const uint16_t *>(from);
                if (x.turn >= 0) a[n].x |= (uint32_t)*reinterpret_cast<const uint16_t *>(from + 2 * p.half) << 16;
            }
        }
#pragma unroll
        for (int n = 0; n < kUnits; ++n) {
            const int e = e0 + n * kThreads;
            if (e >= units) continue;
            const int t = e / p.token_units;
            const Unit x = unit_of<kMode>(p, e - t * p.token_units);
            const Side &s = p.side[x.side];
            char *to = s.dst;
            if (s.dst_block) {
                const int64_t slot = slots[t];
                if (slot < 0) continue;
                to += (slot >> p.shift) * s.dst_block + (slot & ((1 << p.shift) - 1)) * s.dst_token;
            } else {
                to += (t0 + t) * s.dst_token;
            }
            to += x.head * s.dst_head + x.at;
            const float *c = cosine + t * p.half + x.turn, *d = sine + t * p.half + x.turn;
            if (kMode == kHalf && x.turn >= 0) {
                uint32_t *va = &a[n].x, *vb = &b[n].x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 cc = reinterpret_cast<const float2 *>(c)[i], dd = reinterpret_cast<const float2 *>(d)[i];
                    float2 u = unpack<T>(va[i]), w = unpack<T>(vb[i]);
                    turn(u.x, w.x, cc.x, dd.x);
                    turn(u.y, w.y, cc.y, dd.y);
                    va[i] = pack<T>(u.x, u.y);
                    vb[i] = pack<T>(w.x, w.y);
                }
                *reinterpret_cast<uint4 *>(to + 2 * p.half) = b[n];
            } else if (kMode == kPairs && x.turn >= 0) {
                uint32_t *va = &a[n].x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 u = unpack<T>(va[i]);
                    turn(u.x, u.y, c[i], d[i]);
                    va[i] = pack<T>(u.x, u.y);
                }
            } else if (!kVector && x.turn >= 0) {
                float2 u = unpack<T>(a[n].x);
                turn(u.x, u.y, c[0], d[0]);
                a[n].x = pack<T>(u.x, u.y);
            }
            if (kVector || x.side == 2) {
                *reinterpret_cast<uint4 *>(to) = a[n];
            } else if (kMode == kSinglePairs && x.turn >= 0) {
                *reinterpret_cast<uint32_t *>(to) = a[n].x;
            } else {
                *reinterpret_cast<uint16_t *>(to) = (uint16_t)a[n].x;
                if (x.turn >= 0) *reinterpret_cast<uint16_t *>(to + 2 * p.half) = (uint16_t)(a[n].x >> 16);
            }
        }
    }
}

template <typename T>
const void *kernel_of(int mode)
{
    switch (mode) {
    case kHalf: return (const void *)rotary_kernel<T, kHalf>;
    case kPairs: return (const void *)rotary_kernel<T, kPairs>;
    case kSingleHalf: return (const void *)rotary_kernel<T, kSingleHalf>;
    default: return (const void *)rotary_kernel<T, kSinglePairs>;
    }
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
    p.head_bytes = (int)a.head_dim * 2;
    p.q_heads = (int)a.q_heads;
    p.turned_heads = (int)(a.q_heads + a.kv_heads);
    p.v_heads = append ? (int)a.kv_heads : 0;
    const int R = (int)a.rotary_dim, D = (int)a.head_dim;
    int mode;
    if (a.pairs ? R % 8 == 0 : R % 16 == 0) {
        mode = a.pairs ? kPairs : kHalf;
        p.turn_units = a.pairs ? R / 8 : R / 16;
        p.head_units = p.turn_units + (D - R) / 8;
    } else {
        mode = a.pairs ? kSinglePairs : kSingleHalf;
        p.turn_units = R / 2;
        p.head_units = p.turn_units + (D - R);
    }
    p.copy_units = D / 8;
    p.token_units = p.turned_heads * p.head_units + p.v_heads * p.copy_units;
    // as many tokens as the CTA's threads have units for at once, but four CTAs an SM before one has several
    p.per_cta = std::max(1, kThreads * kUnits / p.token_units);
    p.per_cta = (int)std::min<int64_t>(p.per_cta, (a.tokens + 607) / 608);
    // and no more than the cosines' share of shared memory
    p.per_cta = std::max(1, std::min(p.per_cta, 4096 / p.half));
    const size_t smem = 8 * ((size_t)p.half + p.per_cta + 1) + 8 * (size_t)p.per_cta * p.half;
    void *args[] = {&p};
    const void *kernel = a.dtype == AWQ_F16 ? kernel_of<__half>(mode) : kernel_of<__nv_bfloat16>(mode);
    return launch_dependent(kernel, (a.tokens + p.per_cta - 1) / p.per_cta, kThreads, smem, stream, args);
}

} // namespace awq

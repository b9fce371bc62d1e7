// awq_attention.cu -- attention of a step's new tokens over a paged cache, for
// few rows a key-value head (plain decode, small trees) and for every head_dim up
// to 256; awq_attention_tc.cu takes the calls with many rows.
//
//   out[r, :] = sum_j exp(s_rj - m_r) v_j / sum_j exp(s_rj - m_r),  s_rj = scale q_r . k_j
//
// in one pass over keys and values with a running maximum and sum (awq_attention.cuh
// has the split of the work and the join of its pieces).
//
// Bound: the cache is read once, 4 head_dim bytes a key and head, against
// 4 head_dim flops a row, so 16 rows have 16 flops a byte: HBM. A CTA therefore is
// one producer warp, which asks for key and value tiles (32 keys) with TMA, a page
// with all of its columns a box, as far ahead as shared memory allows (with a box a
// 64 columns the issue of a tile of two pages took 900 cycles instead of 660), and
// three consumer warps that take whole tiles in turn: S = Q K^T and O += P V with
// mma.sync m16n8k16 (16 rows of q, held in registers), the warp's own maximum and
// sum, 1,900 cycles a tile, two thirds of them the products'. A stage of the ring
// always goes to the same warp, and the warps never meet before the segment ends.
// (Four warps with 16 keys each of a common tile went through maximum, sum and
// rescaling four times as often: 6 us for 500 keys instead of 4. A fourth consumer
// and a second producer warp, which leave 168 registers a thread, changed nothing
// beyond 3%.) mma.sync, not tcgen05: at 16 rows a 128-row tcgen05 tile would be
// seven eighths padding and its operands and accumulators would take the detour over
// shared and tensor memory.
// Measured: 64 requests of up to 8192 tokens, 64 / 8 heads of 128, fp16: 197 us, 95%
// of the copy bandwidth; one request of 500 tokens, 32 heads of 128: 9.6 us.
#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "awq_attention.h"
#include "awq_attention.cuh"

namespace awq {
namespace attn {
namespace {

constexpr int kRows = 16;        // rows of q a CTA works on (one mma.sync M)
constexpr int kKeys = 32;        // keys a tile
constexpr int kBlockCost = 2;    // a row block's beginning and end, in tiles
// Row blocks of up to this many tiles are not split: a CTA reads them (1,024 keys)
// in the time that a second kernel would take to join the pieces.
constexpr int kWholeTiles = 32;
// Few row blocks are shared by the CTAs of a cluster, as many (up to kMaxShare) as find
// room on the GPU and have kShareTiles tiles each: one token, 32 heads of 128 over 1,000
// keys took 10.5 us so and 16.5 without, 4 tokens of 64 / 8 heads over 400 keys 10.4 and
// 12.9; with two tiles a CTA, 4 tokens over 100 keys 9.5 instead of 8.0. Beyond
// kSharedTiles a CTA the split and join of the whole GPU is faster: 8 heads over 4,000
// keys (16 tiles) 13.2 us shared and 12.9 split, over 8,000 keys 19.7 and 14.7.
constexpr int kShareLog = 3, kMaxShare = 1 << kShareLog;
constexpr int kShareTiles = 3, kSharedTiles = 16;
constexpr int kWarps = 3;        // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;

// DP: head_dim rounded up to 64, 128 or 256 (TMA fills the rest with zeros).
template <int DP>
struct Cfg {
    static constexpr int kHalves = DP / 64;              // 128-byte columns of a tile
    static constexpr int kTile = kKeys * DP * 2;         // keys or values of one stage
    static constexpr int kStages = DP == 64 ? 12 : 6;    // 96 KB in flight (192 KB at DP = 256)
    static_assert(kStages % kWarps == 0, "a stage always goes to the same warp");
    static constexpr int kMergeOff = kStages * 2 * kTile;
    static constexpr int kMerge = kRows * DP * 4;        // one warp's O
    static constexpr int kRedOff = kMergeOff + kMerge;   // m and l of the warps
    static constexpr int kRed = 2 * kWarps * kRows * 4;
    static constexpr int kBarOff = kRedOff + kRed;
    static constexpr int kSmem = kBarOff + 256 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    ptx::mma_16816(d, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&d)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(addr) : "memory");
}

// A tile lies in shared memory page by page (of 16 or 32 keys), a page by halves of 64
// columns, as TMA writes a box of all of them, in its 128-byte swizzle.
struct Layout {
    uint32_t half, skip;    // bytes between halves; between the pages of 16 keys, beyond their rows'
    // 16-byte piece `c` of row `r`
    __device__ __forceinline__ uint32_t piece(uint32_t tile, int r, int c) const
    {
        return tile + (uint32_t)(c >> 3) * half + (uint32_t)r * 128 + (uint32_t)(r >> 4) * skip +
               (uint32_t)(((c & 7) ^ (r & 7)) << 4);
    }
};

// Tiles of a segment that CTA `rank` of a cluster of 2^share has.
__device__ __forceinline__ void share_of(Segment &s, int share, int rank)
{
    const int n = s.tile1 - s.tile0;
    s.tile1 = s.tile0 + ((n * (rank + 1)) >> share);
    s.tile0 += (n * rank) >> share;
}

// Joins the parts that the CTAs of a cluster have left: at `pairs` m and l of the rows,
// at `parts_o` O as the lanes of warp 0 had it. CTA `rank` does its part of the columns,
// eight a warp and turn; a lane has rows g and g + 8. (A function of its own: inlined, its
// registers were missing in the loop over the tiles at head_dim 256.)
template <typename T, int DP>
__device__ __noinline__ void join_shared(const Params &p, const Segment &s, uint32_t pairs, uint32_t parts_o, int rank,
                                         int row0, int rows)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int parts = 1 << p.share, turns = (DP / 8) >> p.share;
    if (g >= rows) return;
    float fa[kMaxShare], fb[kMaxShare], ka[kMaxShare], kb[kMaxShare];
#pragma unroll
    for (int i = 0; i < kMaxShare; ++i) {
        float2 a = make_float2(-INFINITY, 0.f), b = a;
        if (i < parts) {
            a = ptx::cluster_load2(ptx::cluster_addr(pairs + g * 8, i));
            b = ptx::cluster_load2(ptx::cluster_addr(pairs + (g + 8) * 8, i));
        }
        fa[i] = a.x;
        ka[i] = a.y;
        fb[i] = b.x;
        kb[i] = b.y;
    }
    float top_a = -INFINITY, top_b = -INFINITY, sum_a = 0.f, sum_b = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxShare; ++i) {
        top_a = fmaxf(top_a, fa[i]);
        top_b = fmaxf(top_b, fb[i]);
    }
    const float za = top_a == -INFINITY ? 0.f : top_a, zb = top_b == -INFINITY ? 0.f : top_b;
#pragma unroll
    for (int i = 0; i < kMaxShare; ++i) {
        fa[i] = exp2_fast(fa[i] - za);
        fb[i] = exp2_fast(fb[i] - zb);
        sum_a = fmaf(ka[i], fa[i], sum_a);
        sum_b = fmaf(kb[i], fb[i], sum_b);
    }
    const float ia = sum_a == 0.f ? 0.f : 1.f / sum_a, ib = sum_b == 0.f ? 0.f : 1.f / sum_b;
    auto out_of = [&](int r) {
        const int64_t t = s.token0 + (row0 + r) / p.group, head = (int64_t)s.h * p.group + (row0 + r) % p.group;
        return static_cast<T *>(p.out) + (t * p.q_heads + head) * p.head_dim + t4 * 2;
    };
    T *out_a = out_of(g), *out_b = out_of(g + 8);
    for (int k = warp; k < turns; k += kWarps) {
        const int i = rank * turns + k;
        if (i * 8 >= p.head_dim) break;
        float4 v[kMaxShare], x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kMaxShare; ++j)
            if (j < parts) v[j] = ptx::cluster_load4(ptx::cluster_addr(parts_o + (i * 32 + lane) * 16, j));
#pragma unroll
        for (int j = 0; j < kMaxShare; ++j)
            if (j < parts) {
                x.x += v[j].x * fa[j];
                x.y += v[j].y * fa[j];
                x.z += v[j].z * fb[j];
                x.w += v[j].w * fb[j];
            }
        *reinterpret_cast<uint32_t *>(out_a + i * 8) = Elem<T>::pack(x.x * ia, x.y * ia);
        if (g + 8 < rows) *reinterpret_cast<uint32_t *>(out_b + i * 8) = Elem<T>::pack(x.z * ib, x.w * ib);
    }
    if (rank == 0 && warp == 0 && t4 == 0) {
        store_lse(p, s.token0, s.h, row0 + g, za, sum_a);
        if (g + 8 < rows) store_lse(p, s.token0, s.h, row0 + g + 8, zb, sum_b);
    }
}

// kShared: a cluster has each row block, its CTAs a part of the keys each (few short
// row blocks, which would leave most of the GPU idle). They leave m, l and O in shared
// memory, where all of them read their part of the columns.
template <typename T, int DP, bool kShared>
__global__ void __launch_bounds__(kThreads, DP <= 128 && !kShared ? 2 : 1)
attention_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ Params p)
{
    using C = Cfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + C::kStages;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(empty + C::kStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(empty + i), 1);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    Work<kRows, kKeys, kBlockCost> work;
    if (!work.template find<kThreads>(p)) return;   // its barriers also publish the mbarriers
    Segment s;
    const int rank = kShared ? ptx::cluster_rank() : 0;
    // Every thread of a cluster, a segment: all CTAs have left their part; whether each
    // of them has.
    auto parts_left = [&] {
        ptx::cluster_sync();
        int gave_up = 0;
        for (int r = 0; r < 1 << p.share; ++r)
            gave_up |= __float_as_int(ptx::cluster_load(ptx::cluster_addr(ptx::smem_addr(const_cast<int *>(abort_flag)), r)));
        return gave_up == 0;
    };
    const int box = min(1 << p.shift, kKeys);                // keys of one TMA box
    const Layout lay{(uint32_t)box * 128, box < kKeys ? (C::kHalves - 1) * 16u * 128u : 0u};

    if (warp == kWarps) {
        // ---------------------------------------------------------------- producer
        const int pages = kKeys / box;                       // pages of a tile: 1 or 2
        // A box a lane: page, then keys or values, then the half of head_dim if its
        // columns do not fill the halves (else a box has all halves).
        const int cols = p.head_dim % 64 == 0 ? 1 : C::kHalves;
        const int page = lane / (2 * cols), part = lane % (2 * cols), half = part % cols;
        const CUtensorMap *map = part < cols ? &tm_k : &tm_v;
        const uint32_t to = (part < cols ? 0 : C::kTile) + (page * C::kHalves + half) * lay.half;
        const uint32_t bytes = (uint32_t)(C::kHalves / cols) * lay.half;
        int it = 0;
        bool ok = true;
#ifdef AWQ_FAULT_TEST
        if (p.fault && blockIdx.x == 0) ok = false;
#endif
        while ((ok || kShared) && work.next(p, s)) {
            if (kShared) share_of(s, p.share, rank);
            const int keys = s.ctx + s.n;
            Pages ids;
            ids.open(p, s, (s.tile0 * kKeys) >> p.shift, lane);
            for (int tile = s.tile0; tile < s.tile1 && ok; ++tile, ++it) {
                const int key = tile * kKeys + (page < pages ? page * box : 0);
                const int id = ids.block(p, key >> p.shift, lane);
                const bool mine = page < pages && key < keys;
                const int st = it % C::kStages;
                ok = ptx::mbar_wait_bounded(ptx::smem_addr(empty + st), ((it / C::kStages) & 1) ^ 1, abort_flag, p.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t fb = ptx::smem_addr(full + st);
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, mine));
                if (lane == 0) ptx::mbar_arrive_expect_tx(fb, (uint32_t)count * bytes);
                __syncwarp();
                if (mine)
                    ptx::tma_load_5d(ptx::smem_addr(smem + st * 2 * C::kTile) + to, map, fb, half * 64,
                                     (tile * kKeys) & ((1 << p.shift) - 1), 0, s.h, id);
            }
            if (kShared) {
                const bool all = parts_left();
                ptx::cluster_sync();
                if (!all) {
                    ok = false;
                    break;
                }
            }
        }
        if (!ok) {
            // the copies in flight land before the CTA's shared memory goes
            for (int i = std::max(0, it - C::kStages); i < it; ++i)
                ptx::mbar_wait_bounded(ptx::smem_addr(full + i % C::kStages), (i / C::kStages) & 1, nullptr, nullptr);
        }
        return;
    }

    // -------------------------------------------------------------------- consumers
    const int g = lane >> 2, t4 = lane & 3;
    float *merge = reinterpret_cast<float *>(smem + C::kMergeOff);
    float *warp_m = reinterpret_cast<float *>(smem + C::kRedOff), *warp_l = warp_m + kWarps * kRows;
    int base = 0;                    // tiles of the segments before
    bool ok = true;
    while (work.next(p, s)) {
        if (kShared) share_of(s, p.share, rank);
        const int all_rows = s.n * p.group, row0 = s.rb * kRows;
        const int rows = min(kRows, all_rows - row0);
        // this lane's rows g and g + 8 (the last row again where they do not exist)
        const int ra = min(row0 + g, all_rows - 1), rb = min(row0 + g + 8, all_rows - 1);
        const int ta = ra / p.group, tb = rb / p.group;
        uint32_t qf[DP / 16][4];
        {
            const T *qa = static_cast<const T *>(p.q) + (int64_t)(s.token0 + ta) * p.q_token_stride +
                          (int64_t)(s.h * p.group + ra % p.group) * p.q_head_stride;
            const T *qb = static_cast<const T *>(p.q) + (int64_t)(s.token0 + tb) * p.q_token_stride +
                          (int64_t)(s.h * p.group + rb % p.group) * p.q_head_stride;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                const int c = kk * 16 + t4 * 2;
                qf[kk][0] = c < p.head_dim ? *reinterpret_cast<const uint32_t *>(qa + c) : 0u;
                qf[kk][1] = c < p.head_dim ? *reinterpret_cast<const uint32_t *>(qb + c) : 0u;
                qf[kk][2] = c + 8 < p.head_dim ? *reinterpret_cast<const uint32_t *>(qa + c + 8) : 0u;
                qf[kk][3] = c + 8 < p.head_dim ? *reinterpret_cast<const uint32_t *>(qb + c + 8) : 0u;
            }
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

        // this warp's tiles: those whose place in the ring goes to it
        const int skip = (warp - base % kWarps + kWarps) % kWarps;
        for (int tile = s.tile0 + skip; tile < s.tile1 && ok; tile += kWarps) {
            const int it = base + tile - s.tile0, st = it % C::kStages;
            ok = ptx::mbar_wait_bounded(ptx::smem_addr(full + st), (it / C::kStages) & 1, abort_flag, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t kt = ptx::smem_addr(smem + st * 2 * C::kTile);
            const uint32_t vt = kt + C::kTile;
            // scores: columns 2 t4, 2 t4 + 1 of each eight keys
            float sc[kKeys / 8][4];
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
            const int krow = ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i) {
                    uint32_t b[4];
                    ptx::ldmatrix_x4(lay.piece(kt, i * 16 + krow, kk * 2 + ((lane >> 3) & 1)), b);
                    mma<T>(sc[2 * i], qf[kk], b[0], b[1]);
                    mma<T>(sc[2 * i + 1], qf[kk], b[2], b[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][e] *= p.scale_log2;
            const int key0 = tile * kKeys;
            const bool drafted = key0 + kKeys > s.ctx;       // drafted (or no) keys among them
            uint32_t seen_a = 0xFFFFFFFFu, seen_b = 0xFFFFFFFFu;   // bit k: key0 + k is visible
            if (drafted) {
                seen_a = seen32(p, s, ta, key0);
                seen_b = seen32(p, s, tb, key0);
#pragma unroll
                for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = i * 8 + t4 * 2 + e;
                        if (!((seen_a >> k) & 1u)) sc[i][e] = -INFINITY;
                        if (!((seen_b >> k) & 1u)) sc[i][2 + e] = -INFINITY;
                    }
            }
            float na = -INFINITY, nb = -INFINITY;
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i) {
                na = fmaxf(na, fmaxf(sc[i][0], sc[i][1]));
                nb = fmaxf(nb, fmaxf(sc[i][2], sc[i][3]));
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                na = fmaxf(na, __shfl_xor_sync(0xFFFFFFFFu, na, d));
                nb = fmaxf(nb, __shfl_xor_sync(0xFFFFFFFFu, nb, d));
            }
            // the maximum less the weights' scaling; a row without a visible key keeps -inf
            na = fmaxf(ma, na - Elem<T>::kBias);
            nb = fmaxf(mb, nb - Elem<T>::kBias);
            const float ea = na == -INFINITY ? 0.f : na, eb = nb == -INFINITY ? 0.f : nb;
            if (__any_sync(0xFFFFFFFFu, na != ma || nb != mb)) {
                const float fa = exp2_fast(ma - ea), fb = exp2_fast(mb - eb);
                la *= fa;
                lb *= fb;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    o[i][0] *= fa;
                    o[i][1] *= fa;
                    o[i][2] *= fb;
                    o[i][3] *= fb;
                }
                ma = na;
                mb = nb;
            }
            uint32_t pf[kKeys / 16][4];
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i) {
                sc[i][0] = exp2_fast(sc[i][0] - ea);
                sc[i][1] = exp2_fast(sc[i][1] - ea);
                sc[i][2] = exp2_fast(sc[i][2] - eb);
                sc[i][3] = exp2_fast(sc[i][3] - eb);
                la += sc[i][0] + sc[i][1];
                lb += sc[i][2] + sc[i][3];
                pf[i >> 1][2 * (i & 1)] = Elem<T>::pack(sc[i][0], sc[i][1]);
                pf[i >> 1][2 * (i & 1) + 1] = Elem<T>::pack(sc[i][2], sc[i][3]);
            }
            if (drafted) {
                // Values of keys past the last one may be anything: made zero, so
                // that a weight of zero takes nothing from them. A drafted key's
                // infinities and NaN reach the rows that see it only.
                bool odd = false;
                for (int e = lane; e < kKeys * (DP / 8); e += 32) {
                    const int r = e / (DP / 8), key = key0 + r;
                    const uint32_t at = lay.piece(vt, r, e % (DP / 8));
                    if (key >= s.ctx + s.n) {
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    } else if (key >= s.ctx) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
                        for (int i = 0; i < 4; ++i) odd = odd || has_nonfinite<T>(w[i]);
                    }
                }
                __syncwarp();
                if (__any_sync(0xFFFFFFFFu, odd)) {
                    for (int k = max(0, s.ctx - key0); k < kKeys && key0 + k < s.ctx + s.n; ++k) {
                        const bool sa = (seen_a >> k) & 1u, sb = (seen_b >> k) & 1u;
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) {
                            uint32_t w;
                            const uint32_t at = lay.piece(vt, k, i) + t4 * 4;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint16_t half = (uint16_t)(w >> (16 * e));
                                if ((half & Elem<T>::kExpMask) != Elem<T>::kExpMask) continue;
                                const float v = Elem<T>::to_float(half);
                                if (sa) o[i][e] += v;
                                if (sb) o[i][2 + e] += v;
                            }
                        }
                        __syncwarp();
                        // cleared once all lanes have read it
                        for (int c = lane; c < DP / 2; c += 32) {
                            const uint32_t at = lay.piece(vt, k, c >> 2) + (c & 3) * 4;
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                            if ((w & Elem<T>::kExpMask) == Elem<T>::kExpMask) w &= 0xFFFF0000u;
                            if (((w >> 16) & Elem<T>::kExpMask) == Elem<T>::kExpMask) w &= 0x0000FFFFu;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
                        }
                        __syncwarp();
                    }
                }
                // these stores come before the TMA's next write of the stage
                ptx::fence_proxy_async_smem();
            }
#pragma unroll
            for (int j = 0; j < kKeys / 16; ++j) {
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(lay.piece(vt, j * 16 + (lane & 15), i * 2 + (lane >> 4)), b);
                    mma<T>(o[2 * i], pf[j], b[0], b[1]);
                    mma<T>(o[2 * i + 1], pf[j], b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(empty + st));
        }

        base += s.tile1 - s.tile0;

        // ---- the warps' sums become one, in warp 0
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            la += __shfl_xor_sync(0xFFFFFFFFu, la, d);
            lb += __shfl_xor_sync(0xFFFFFFFFu, lb, d);
        }
        if (t4 == 0) {
            warp_m[warp * kRows + g] = ma;
            warp_m[warp * kRows + g + 8] = mb;
            warp_l[warp * kRows + g] = la;
            warp_l[warp * kRows + g + 8] = lb;
        }
        // all leave together if one gave up
        if (!ptx::named_barrier_and(1, kConsumers, ok)) {
            if (kShared) {           // abort_flag is set: the others of the cluster leave too
                parts_left();
                ptx::cluster_sync();
            }
            return;
        }
        float m2a = -INFINITY, m2b = -INFINITY, l2a = 0.f, l2b = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            m2a = fmaxf(m2a, warp_m[w * kRows + g]);
            m2b = fmaxf(m2b, warp_m[w * kRows + g + 8]);
        }
        const float ea = m2a == -INFINITY ? 0.f : m2a, eb = m2b == -INFINITY ? 0.f : m2b;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            l2a += warp_l[w * kRows + g] * exp2_fast(warp_m[w * kRows + g] - ea);
            l2b += warp_l[w * kRows + g + 8] * exp2_fast(warp_m[w * kRows + g + 8] - eb);
        }
        const float fa = exp2_fast(ma - ea), fb = exp2_fast(mb - eb);
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
            o[i][0] *= fa;
            o[i][1] *= fa;
            o[i][2] *= fb;
            o[i][3] *= fb;
        }
        float4 *mine = reinterpret_cast<float4 *>(merge) + lane;
#pragma unroll 1
        for (int w = 1; w < kWarps; ++w) {
            if (warp == w)
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) mine[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
            ptx::named_barrier(1, kConsumers);
            if (warp == 0)
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    const float4 v = mine[i * 32];
                    o[i][0] += v.x;
                    o[i][1] += v.y;
                    o[i][2] += v.z;
                    o[i][3] += v.w;
                }
            ptx::named_barrier(1, kConsumers);
        }
        if (kShared) {
            // this CTA's part, then the columns that it joins
            float2 *pairs = reinterpret_cast<float2 *>(warp_m);     // m and l of the rows
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) mine[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                if (t4 == 0) {
                    pairs[g] = make_float2(m2a, l2a);
                    pairs[g + 8] = make_float2(m2b, l2b);
                }
            }
            const bool all = parts_left();
            if (all) join_shared<T, DP>(p, s, ptx::smem_addr(pairs), ptx::smem_addr(merge), rank, row0, rows);
            ptx::cluster_sync();
            if (!all) return;
        } else if (s.whole()) {
            if (warp == 0) {
                const float ia = l2a == 0.f ? 0.f : 1.f / l2a, ib = l2b == 0.f ? 0.f : 1.f / l2b;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = g + 8 * half;
                    if (r >= rows) continue;
                    const int64_t t = s.token0 + (row0 + r) / p.group;
                    const int64_t head = (int64_t)s.h * p.group + (row0 + r) % p.group;
                    T *out = static_cast<T *>(p.out) + (t * p.q_heads + head) * p.head_dim;
                    const float inv = half ? ib : ia;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
                        if (i * 8 < p.head_dim)
                            *reinterpret_cast<uint32_t *>(out + i * 8 + t4 * 2) =
                                Elem<T>::pack(o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
                    if (t4 == 0) store_lse(p, s.token0, s.h, row0 + r, half ? eb : ea, half ? l2b : l2a);
                }
            }
        } else {
            if (warp == 0) {
                float *slot = p.partials + (int64_t)work.slot_of(s) * slot_floats(kRows, DP);
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    const int c = i * 8 + t4 * 2;
                    __stcg(reinterpret_cast<float2 *>(slot + slot_at(kRows, g, c)), make_float2(o[i][0], o[i][1]));
                    __stcg(reinterpret_cast<float2 *>(slot + slot_at(kRows, g + 8, c)), make_float2(o[i][2], o[i][3]));
                }
                if (t4 == 0) {
                    __stcg(slot + kRows * DP + g, m2a);
                    __stcg(slot + kRows * DP + g + 8, m2b);
                    __stcg(slot + kRows * DP + kRows + g, l2a);
                    __stcg(slot + kRows * DP + kRows + g + 8, l2b);
                }
            }
            if (threadIdx.x == 0 && s.tile1 == s.tiles) work.note_join(p, s, rows);
        }
    }
}

struct LaunchInfo {
    int sms = 0, ctas = 0;   // CTAs that fit the GPU at once
    cudaError_t err = cudaSuccess;
    unsigned gen = 0;
};

template <typename T, int DP, bool kShared>
LaunchInfo launch_info()
{
    static std::mutex mu;
    static std::map<int, LaunchInfo> cache;
    int dev = 0;
    LaunchInfo li;
    li.err = cudaGetDevice(&dev);
    if (li.err != cudaSuccess) return li;
    const unsigned gen = cache_generation();
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it != cache.end() && it->second.gen == gen) return it->second;
    li.gen = gen;
    int sms = 0, per_sm = 0;
    li.err = cudaFuncSetAttribute(attention_rows_kernel<T, DP, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  Cfg<DP>::kSmem);
    if (li.err == cudaSuccess) li.err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (li.err == cudaSuccess)
        li.err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attention_rows_kernel<T, DP, kShared>, kThreads,
                                                               Cfg<DP>::kSmem);
    li.sms = sms;
    li.ctas = sms * std::max(1, per_sm);
    if (li.err == cudaSuccess) cache[dev] = li;
    return li;
}

template <typename T, int DP>
cudaError_t launch_rows(const awq_tree_attention_t &a, cudaStream_t stream)
{
    const LaunchInfo li = launch_info<T, DP, false>();
    if (li.err != cudaSuccess) return li.err;
    Params p = make_params(a);
    CUtensorMap tk, tv;
    if (!make_cache_map_5d(&tk, a, a.k_cache, kKeys, Cfg<DP>::kHalves) ||
        !make_cache_map_5d(&tv, a, a.v_cache, kKeys, Cfg<DP>::kHalves))
        return cudaErrorInvalidValue;
    // a launch no larger than the work the bounds allow
    const int64_t tiles = tiles_bound(a, kKeys), blocks = blocks_bound(a, kRows);
    const LaunchInfo shared = launch_info<T, DP, true>();
    if (shared.err != cudaSuccess) return shared.err;
    int share = 0;
    while (blocks > 0 && share < kShareLog && (blocks << (share + 1)) <= shared.ctas && (tiles >> (share + 1)) >= kShareTiles) ++share;
    p.whole = tiles <= (share > 0 ? (int64_t)kSharedTiles << share : kWholeTiles);
    p.min_units = p.whole ? 1 : kBlockCost + 8;
    const int64_t units = p.whole ? blocks : blocks * (kBlockCost + tiles);
#ifdef AWQ_FAULT_TEST
    p.fault = fault_injection();
#endif
    if (p.whole) p.share = share;
    if (p.share > 0) {
        p.lines = 1;
        return launch_pair<T, kRows, DP>(attention_rows_kernel<T, DP, true>, (int)blocks << p.share, kThreads, Cfg<DP>::kSmem,
                                         stream, tk, tv, p);
    }
    const int ctas = lay_out(p, li.ctas, units);
    return launch_pair<T, kRows, DP>(attention_rows_kernel<T, DP, false>, ctas, kThreads, Cfg<DP>::kSmem, stream, tk, tv, p);
}

} // namespace

Params make_params(const awq_tree_attention_t &a)
{
    Params p{};
    p.q = a.q;
    p.q_token_stride = a.q_token_stride;
    p.q_head_stride = a.q_head_stride;
    p.out = a.out;
    p.lse = a.lse;
    p.table = a.block_table;
    p.table_stride = a.table_stride;
    p.v_data = a.v_cache.data;
    p.v_block_stride = a.v_cache.block_stride;
    p.v_token_stride = a.v_cache.token_stride;
    p.v_head_stride = a.v_cache.head_stride;
    p.ctx = a.context_lens;
    p.cu = a.cu_new;
    p.mask = a.tree_mask;
    p.status = device_status_word();
    p.table_width = (int)a.table_width;
    p.mask_words = (int)a.mask_words;
    p.B = (int)a.B;
    p.tokens = (int)a.tokens;
    p.q_heads = (int)a.q_heads;
    p.kv_heads = (int)a.kv_heads;
    p.group = (int)(a.q_heads / a.kv_heads);
    p.head_dim = (int)a.head_dim;
    p.num_blocks = (int)a.num_blocks;
    while ((int64_t(1) << p.shift) < a.block_size) ++p.shift;
    p.min_units = 1;
    p.scale_log2 = a.scale * 1.44269504088896341f;
    return p;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode()
{
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return enc;
}

bool make_cache_map(CUtensorMap *m, const awq_tree_attention_t &a, const awq_cache_t &c, int tile_keys)
{
    const auto enc = encode();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.kv_heads, (cuuint64_t)a.block_size,
                          (cuuint64_t)a.num_blocks};
    cuuint64_t strides[3] = {(cuuint64_t)c.head_stride * 2, (cuuint64_t)c.token_stride * 2,
                             (cuuint64_t)c.block_stride * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)std::min<int64_t>(a.block_size, tile_keys), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, a.dtype == AWQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c.data,
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// As halves of 64 columns: 64, tokens, halves, heads, blocks, a box `halves` of them
// (zeros past head_dim). Where the last half is not full, head_dim stays one axis, of
// which a box has 64 columns.
bool make_cache_map_5d(CUtensorMap *m, const awq_tree_attention_t &a, const awq_cache_t &c, int tile_keys, int halves)
{
    const auto enc = encode();
    if (!enc) return false;
    const bool full = a.head_dim % 64 == 0;
    cuuint64_t dims[5] = {(cuuint64_t)(full ? 64 : a.head_dim), (cuuint64_t)a.block_size,
                          (cuuint64_t)(full ? a.head_dim / 64 : 1), (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_blocks};
    cuuint64_t strides[4] = {(cuuint64_t)c.token_stride * 2, 128, (cuuint64_t)c.head_stride * 2,
                             (cuuint64_t)c.block_stride * 2};
    cuuint32_t box[5] = {64, (cuuint32_t)std::min<int64_t>(a.block_size, tile_keys), (cuuint32_t)(full ? halves : 1), 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, a.dtype == AWQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, c.data,
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_rows_any(const awq_tree_attention_t &a, cudaStream_t stream)
{
    const bool f16 = a.dtype == AWQ_F16;
    if (a.head_dim <= 64)
        return f16 ? launch_rows<__half, 64>(a, stream) : launch_rows<__nv_bfloat16, 64>(a, stream);
    if (a.head_dim <= 128)
        return f16 ? launch_rows<__half, 128>(a, stream) : launch_rows<__nv_bfloat16, 128>(a, stream);
    return f16 ? launch_rows<__half, 256>(a, stream) : launch_rows<__nv_bfloat16, 256>(a, stream);
}

} // namespace attn

cudaError_t launch_tree_attention(const awq_tree_attention_t &a, cudaStream_t stream)
{
    const int64_t rows = attn::rows_bound(a);
    if (a.head_dim > 128 || rows <= attn::kRows) return attn::launch_rows_any(a, stream);
    // With more rows the few-row kernel reads its keys once a block of 16. Small calls
    // still take it: if all blocks have a CTA at once (or are two a head), and as long as
    // that costs no more than the tensor-core kernel's longer way in and out: up to about
    // 20,000 tiles of 32 keys, read again by each block. Us with this kernel and with the other:
    //   64 / 8 heads of 128     1 request,  64 tokens, 2000 keys (17k tiles): 33 and 36
    //                           1 request,  64 tokens, 3000 keys (25k): 40 and 36
    //                           1 request,  64 tokens, 4000 keys (33k): 48 and 35
    //                          16 requests,  4 tokens,  400 keys  (3k): 12 and 17
    //                          16 requests,  4 tokens, 2000 keys (16k): 40 and 48
    //                          16 requests,  4 tokens, 3000 keys (24k): 55 and 58
    //                          16 requests,  4 tokens, 4000 keys (32k): 76 and 67
    //                           4 requests, 16 tokens, 4000 keys (32k): 53 and 34
    //   32 / 8 heads of 64      1 request,  64 tokens, 4000 keys (16k): 25 and 28
    //                          16 requests,  8 tokens, 2000 keys (16k): 27 and 34
    //                           4 requests,  5 tokens, 16000 keys (32k): 41 and 38
    // and where not all blocks have a CTA at once, 64 / 8 heads of 128, 400 keys:
    //   16 requests, 8 tokens: 18 and 13; 32 tokens: 42 and 23
    const int64_t blocks = attn::blocks_bound(a, attn::kRows), tiles = attn::tiles_bound(a, attn::kKeys);
    if (blocks * tiles > 20000 || (blocks > 304 && rows > 2 * attn::kRows)) return attn::launch_tc_any(a, stream);
    return attn::launch_rows_any(a, stream);
}

size_t tree_attention_partial_floats(int64_t head_dim, int sms)
{
    // At most four CTAs of the few-row kernel fit an SM's shared memory. The smaller classes
    // of head_dim too: the tensor-core kernel, which ends at 128, has the larger pieces.
    size_t most = 0;
    for (const int dp : {64, 128, 256}) {
        if (dp > 64 && head_dim <= dp / 2) break;
        most = std::max({most, attn::scratch_floats(4 * sms, attn::kRows, dp), attn::tc_partial_floats(sms, dp)});
    }
    return most;
}

} // namespace awq

// awq_attention_tc.cu -- attention of a step's new tokens over a paged cache, for
// many rows a key-value head (drafted trees, chunks of a prompt), on the 5th-generation
// tensor cores; head_dim up to 128. awq_attention.cuh has the split of the work.
//
// A row block is 256 rows (128 where no request has more), a tile 128 keys. Two streams of work alternate on the
// tensor cores, so that one multiplies while the other's softmax runs:
//   more than 128 rows in the block: stream i has rows 128 i .. 128 i + 127 and
//     both take every tile (a tile is read once for 256 rows);
//   128 rows or fewer: both have the same rows, stream i takes tiles i, i + 2, ..,
//     and their two sums are joined at the segment's end.
// For a stream and half a tile (64 keys): S = Q K^T (tcgen05, 128 x 64, into tensor
// memory), the stream's four warps read S (a thread has one row: no shuffles),
// write P = exp2(S - m) over it as 16-bit values, and O += P V takes P from tensor
// memory. Tensor memory is full: S 2 streams x 2 halves x 64, O 2 x DP columns.
// S of the next tile's half is written over P, so it is issued only once the O += P V
// that reads this P has completed: products run in the order of their issue where they
// share accumulator and shape, and these two do not. Meanwhile the softmax has the
// other half and the tensor cores the other stream. (Without that wait 0.5 to 1% less for
// 256 rows and for 128 of head_dim 128, 4% for a tree of 26 over 131072 keys, head_dim
// 64. S of 128 keys at once left the softmax waiting for both products of every tile:
// 4,700 cycles a tile of two streams, twice what either side needs.)
//
// The maximum is lazy: O is rescaled only when a row's maximum has grown by more
// than 2^kSlack since the last time (P then is up to 2^kSlack instead of 1, which
// its floating-point format holds as exactly); after a few tiles that is rare, and
// the accumulator stays where it is.
//
// Bounds: 4 DP flops a row and key against 4 DP bytes a key: HBM below about 280 rows a
// head, then the tensor cores and, close to them, the exponentials (128 x 128 of
// them a stream and tile).
//
// Measured: 12 requests with trees of 64 over up to 16384 keys, 64 / 8 heads of 128,
// fp16: 224 to 238 us, half of the bf16 matrix rate (tensor pipe 56% busy: S in halves
// of 64 keys reads q twice a tile); 16 requests with trees of 13 over up to 6000 keys,
// bf16: 66 us, 59% of the copy bandwidth; a tree of 26 over 131072 keys, 32 / 8 heads
// of 64: 59 us, 68%.
//
//   warps 0, 3  producers of K and of V tiles, a TMA box a page, in one ring, in the
//               order the MMAs take them
//   warps 1, 2  the MMAs of streams 0 and 1: while one waits for its softmax the
//               other keeps the tensor cores busy; warp 1 also has tensor memory
//   warps 4-7   softmax and epilogue of stream 0, warps 8-11 of stream 1
#include <algorithm>
#include <map>
#include <mutex>

#include <cuda.h>

#include "awq_attention.h"
#include "awq_attention.cuh"
#include "awq_tcgen05.cuh"

namespace awq {
namespace attn {
namespace {

constexpr int kKeys = 128;       // keys of a tile
// A row block's beginning and end, in units: 6,000 to 9,000 cycles at 128 rows, where a
// tile takes 1,900 and is one unit, and 20,000 at 256, where it takes 3,200 and is two.
template <int kRows>
constexpr int kBlockCost = kRows > 128 ? 16 : 3;
// Row blocks of up to this many tiles are not split: a CTA reads them (1,024 keys)
// in the time that a second kernel would take to join the pieces.
constexpr int kWholeTiles = 8;
constexpr int kThreads = 384;
constexpr int kSoftmax = 256;    // threads of the softmax warps
constexpr float kSlack = 8.f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kO = 256;     // first column of O 0; S of stream i and half h is at 128 i + 64 h

// kRows: rows of a block, 256, or 128 for calls whose requests have no more -- their
// keys and values come from HBM at the pace of the loads under way, and up to four
// tiles have landed and wait for their turn, so the space of q's other half goes
// to the ring.
template <int DP, int kRows>
struct Cfg {
    static constexpr int kHalves = DP / 64;
    static constexpr int kHalf = kKeys * 128;          // 64 columns of a tile, 128-byte rows
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kQ = kRows / 128 * kTile;
    static constexpr int kSlots = (224 * 1024 - kQ) / kTile;   // 5 or 6 tiles of 32 KB, 12 or 13 of 16 KB
    static constexpr int kBarOff = kQ + kSlots * kTile;
    static constexpr int kSmem = kBarOff + 512 + 1024;
    static_assert(kSmem <= 226 * 1024, "shared memory budget");
};

// fp16 weights are 2^(7 + kSlack) at most, and keep all their bits down to 2^-21 of the maximum
template <typename T>
constexpr float kWeightBias = 0.f;
template <>
constexpr float kWeightBias<__half> = 7.f;

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// two at a time
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <typename T, int DP, int kRows>
__global__ void __launch_bounds__(kThreads, 1)
attention_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ Params p)
{
    using C = Cfg<DP, kRows>;
    constexpr bool kBf16 = !std::is_same<T, __half>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);   // [kSlots] tile landed
    uint64_t *freed = full + C::kSlots;      // [kSlots] MMAs that read the tile are done (two arrivals)
    uint64_t *s_full = freed + C::kSlots;    // [2 streams][2 halves] S is complete
    uint64_t *p_full = s_full + 4;           // [2][2] P is written
    uint64_t *pv_done = p_full + 4;          // [2] the stream's last O += P V is complete
    uint64_t *o_full = pv_done + 2;          // [2] O of the stream and segment is complete
    uint64_t *q_full = o_full + 2;
    uint64_t *drain = q_full + 1;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *odd_flag = abort_flag + 1;   // a drafted value of the segment is infinite or NaN
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            ptx::mbar_init(ptx::smem_addr(full + i), 1);
            ptx::mbar_init(ptx::smem_addr(freed + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) {
                ptx::mbar_init(ptx::smem_addr(s_full + 2 * i + h), 1);
                ptx::mbar_init(ptx::smem_addr(p_full + 2 * i + h), 4);
            }
            ptx::mbar_init(ptx::smem_addr(pv_done + i), 1);
            ptx::mbar_init(ptx::smem_addr(o_full + i), 1);
        }
        ptx::mbar_init(ptx::smem_addr(q_full), kSoftmax);
        ptx::mbar_init(ptx::smem_addr(drain), 2);
        *abort_flag = 0;
        *odd_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
        tc::tmem_relinquish();
        tc::fence_before_sync();
    }
    // all that does not depend on the kernel before comes before this wait
    ptx::launch_dependents();
    ptx::wait_prerequisites();
    Work<kRows, kKeys, kBlockCost<kRows>> work;
    const bool works = work.template find<kThreads>(p);
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (!works) {
        if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    Segment s;

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- producers
        // Warp 0 has the keys, warp 3 the values; a tile takes one of them 700
        // cycles and more to ask for (a box a page, a wait, a barrier), so two.
        const bool values = warp == 3;
        const CUtensorMap *map = values ? &tm_v : &tm_k;
        const int box = min(1 << p.shift, kKeys);
        const int pages = kKeys / box;               // boxes of a tile, one a lane
        const int my_page = lane < pages ? lane * box : 0;
        int base = 0;                                // ring position of the segment's first tile
        bool ok = true;
#ifdef AWQ_FAULT_TEST
        if (p.fault && blockIdx.x == 0) ok = false;
#endif
        uint32_t asked = 0, rounds = 0;              // slots this warp has filled, the parity of the last time
        while (ok && work.next(p, s)) {
            const int keys = s.ctx + s.n, nt = s.tile1 - s.tile0;
            const bool two = kRows > 128 && min(kRows, s.n * p.group - s.rb * kRows) > 128;
            const int ahead = min(nt, two ? 1 : 2);  // K tiles before the first V tile
            Pages ids;
            ids.open(p, s, (s.tile0 * kKeys) >> p.shift, lane);
            for (int j = 0; j < nt; ++j) {
                // the order of the MMAs: K 0 (K 1), then V j, K j + ahead
                const int v_at = ahead + (values ? j : j - ahead) + min(values ? j : j - ahead, nt - ahead);
                const int at = base + (values ? v_at : j < ahead ? j : v_at + 1);
                const int slot = at % C::kSlots;
                const int key = (s.tile0 + j) * kKeys + my_page;
                const int id = ids.block(p, key >> p.shift, lane);
                const bool there = lane < pages && key < keys;
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, there));
                const uint32_t round = (uint32_t)(at / C::kSlots) & 1u;
                ok = __all_sync(0xFFFFFFFFu, ptx::mbar_wait_bounded(ptx::smem_addr(freed + slot), round ^ 1u, abort_flag,
                                                                    p.status));
                if (!ok) break;
                asked |= 1u << slot;
                rounds = (rounds & ~(1u << slot)) | round << slot;
                const uint32_t fb = ptx::smem_addr(full + slot);
                if (lane == 0) ptx::mbar_arrive_expect_tx(fb, (uint32_t)count * C::kHalves * box * 128);
                __syncwarp();
                if (there) {
                    const uint32_t dst = ptx::smem_addr(smem + C::kQ + slot * C::kTile) + (uint32_t)my_page * 128;
                    const int in_page = ((s.tile0 + j) * kKeys) & ((1 << p.shift) - 1) & ~(box - 1);
#pragma unroll
                    for (int half = 0; half < C::kHalves; ++half)
                        ptx::tma_load_4d(dst + half * C::kHalf, map, fb, half * 64, s.h, in_page, id);
                }
                __syncwarp();
            }
            base += 2 * nt;
        }
        if (!ok) {
            // the warp's copies land before the shared memory goes
            for (int i = 0; i < C::kSlots; ++i)
                if ((asked >> i) & 1u)
                    ptx::mbar_wait_bounded(ptx::smem_addr(full + i), (rounds >> i) & 1u, nullptr, nullptr);
        }
    } else if (warp == 1 || warp == 2) {
        // ---------------------------------------------------------------- MMAs
        // The whole warp walks the list and waits; one elected lane issues, so
        // that addresses and descriptors stay in uniform registers: the issue of
        // a product has to take less than the product (512 cycles).
        constexpr uint32_t id_qk = tc::idesc_16bit_f32(128, 64, false, kBf16);
        constexpr uint32_t id_pv = tc::idesc_16bit_f32(128, DP, true, kBf16);
        constexpr uint32_t hi = tc::desc_hi(1024);
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint32_t smem0 = ptx::smem_addr(smem);
        const uint32_t q_lo = tc::desc_lo(smem0, 16);
        const uint32_t k_lo = tc::desc_lo(smem0 + C::kQ, 16), v_lo = tc::desc_lo(smem0 + C::kQ, C::kHalf);
        const uint32_t full0 = ptx::smem_addr(full), freed0 = ptx::smem_addr(freed);
        const int k_steps = (p.head_dim + 15) / 16;
        const int stream = __shfl_sync(0xFFFFFFFFu, warp - 1, 0);
        const uint32_t t_s = tm + stream * 128, t_o = tm + kO + stream * 128;
        const uint32_t s_bar = ptx::smem_addr(s_full + 2 * stream), p_bar = ptx::smem_addr(p_full + 2 * stream);
        const uint32_t done_bar = ptx::smem_addr(pv_done + stream), o_bar = ptx::smem_addr(o_full + stream);
        int slot = 0, seg = 0;
        uint32_t ring = 0, taken = 0;                // parities: of the slot's tile, of P
        uint32_t products = 0;                       // O += P V issued
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xFFFFFFFFu, wait_soon(bar, parity, abort_flag, p.status));
            tc::fence_after_sync();
            return ok;
        };
        auto wait_tile = [&] { return wait(full0 + slot * 8, ring); };
        auto advance = [&](int &i, uint32_t &parity) {
            if (++i == C::kSlots) {
                i = 0;
                parity ^= 1;
            }
        };
        // Every tile of the ring is waited for by both warps, in order, and
        // released by both -- by the end of its product or, where only the other
        // stream takes it, at once: so neither can be a round ahead of or behind
        // the slot's parity.
        auto pass = [&] {
            if (!wait_tile()) return;
            if (lane == 0) ptx::mbar_arrive(freed0 + slot * 8);
            advance(slot, ring);
        };
        // half h of the tile in slot i: 64 rows of 128 bytes are 8 KB
        constexpr uint32_t kHalfKeys = 64 * 128;
        auto qk = [&](int i, int h, int q_half) {
            if (tc::elect_one()) {
                const uint32_t a = q_lo + q_half * (C::kTile >> 4);
                const uint32_t b = k_lo + i * (C::kTile >> 4) + h * (kHalfKeys >> 4);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = ((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
                    if (k < k_steps) tc::mma_f16_ss(t_s + h * 64, a + off, b + off, hi, id_qk, k != 0);
                }
                tc::commit(s_bar + h * 8);
                if (h == 1) tc::commit(freed0 + i * 8);
            }
            __syncwarp();
        };
        auto pv = [&](int i, int h, bool first, bool last) {
            if (tc::elect_one()) {
                const uint32_t b = v_lo + i * (C::kTile >> 4) + h * (kHalfKeys >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_f16_ts(t_o, t_s + h * 64 + k * 8, b + k * (2048 >> 4), hi, id_pv, !first || k != 0);
                tc::commit(done_bar);
                if (h == 1) tc::commit(freed0 + i * 8);
                if (last) tc::commit(o_bar);
            }
            __syncwarp();
        };
        // The last O += P V is complete. After each one, so that the barrier is never
        // more than one phase ahead of what is waited for.
        auto pv_complete = [&] { return wait(done_bar, products++ & 1); };
        while (ok && work.next(p, s)) {
            const int nt = s.tile1 - s.tile0;
            const bool two = kRows > 128 && min(kRows, s.n * p.group - s.rb * kRows) > 128;
            if (!wait(ptx::smem_addr(q_full), seg & 1)) break;
            ++seg;
            // the ring: K 0 (K 1), then V j, K j + ahead; with shared rows this
            // stream takes its own tiles of it and passes over the others
            const int ahead = two ? 1 : 2;
            auto mine = [&](int j) { return two || (j & 1) == stream; };
            for (int j = 0; j < min(ahead, nt) && ok; ++j) {
                if (!mine(j)) {
                    pass();
                    continue;
                }
                if (!wait_tile()) break;
                qk(slot, 0, two ? stream : 0);
                qk(slot, 1, two ? stream : 0);
                advance(slot, ring);
            }
            for (int j = 0; j < nt && ok; ++j) {
                const bool more = j + ahead < nt;
                if (!mine(j)) {
                    pass();
                    if (more && ok) pass();
                    continue;
                }
                int next = slot;                     // of the K tile behind this V tile
                uint32_t next_ring = ring;
                advance(next, next_ring);
                if (!wait_tile() || !wait(p_bar, taken & 1)) break;
                pv(slot, 0, j < ahead, false);
                if (more && !wait(full0 + next * 8, next_ring)) break;
                if (!pv_complete()) break;
                if (more) qk(next, 0, two ? stream : 0);
                if (!wait(p_bar + 8, taken & 1)) break;
                pv(slot, 1, false, !more);
                if (!pv_complete()) break;
                if (more) qk(next, 1, two ? stream : 0);
                ++taken;
                advance(slot, ring);
                if (more) advance(slot, ring);
            }
            // a stream without a tile has its O at once
            if (!two && stream >= nt && ok && lane == 0) ptx::mbar_arrive(o_bar);
            __syncwarp();
        }
        // every MMA issued, of both streams, has completed once `drain` flips
        if (tc::elect_one()) {   // the lane that issued them
            tc::commit(ptx::smem_addr(drain));
            ptx::mbar_wait_bounded(ptx::smem_addr(drain), 0, nullptr, p.status);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax, epilogue
        const int tid = threadIdx.x - 128;
        const int stream = tid >> 7;
        const int quarter = warp & 3;                // tensor-memory lanes this warp may touch
        const int row = quarter * 32 + lane;         // row of the stream's 128
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t t_s = t_lane + stream * 128, t_o = t_lane + kO + stream * 128;
        // the two streams' m and l at a segment's end, [2][128], in q's space
        float *pair_m = reinterpret_cast<float *>(smem), *pair_l = pair_m + 256;
        const bool negative = p.scale_log2 < 0.f;
        const float scale = fabsf(p.scale_log2);
        int base = 0;                                // ring position of the segment's first tile
        uint32_t tiles_done = 0, segs_done = 0;
        bool ok = true;
        while (true) {
            // everybody is done with the segment before: q's space and O are free
            if (!ptx::named_barrier_and(1, kSoftmax, ok)) break;
            if (!work.next(p, s)) break;
            const int nt = s.tile1 - s.tile0;
            const int row0 = s.rb * kRows, rows = min(kRows, s.n * p.group - row0);
            const bool two = kRows > 128 && rows > 128;
            if (tid == 0) *odd_flag = 0;
            {
                // a thread has one 16-byte column and every kStep-th row; eight
                // loads are under way before the first is stored
                constexpr int kStep = kSoftmax / (DP / 8);
                const int c = tid % (DP / 8), limit = two ? 256 : 128;
                const T *q = static_cast<const T *>(p.q) + (int64_t)s.token0 * p.q_token_stride +
                             (int64_t)s.h * p.group * p.q_head_stride + c * 8;
                for (int r0 = tid / (DP / 8); r0 < limit; r0 += 8 * kStep) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i * kStep, qr = row0 + r, token = qr / p.group;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (r < rows && c * 8 < p.head_dim)
                            v[i] = *reinterpret_cast<const uint4 *>(q + token * p.q_token_stride +
                                                                    (qr - token * p.group) * p.q_head_stride);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + i * kStep;
                        if (r >= limit) break;
                        const uint32_t flip = negative ? 0x80008000u : 0u;   // scores are scaled by |scale|
                        const uint32_t dst = ptx::smem_addr(smem) + (uint32_t)(r >> 7) * C::kTile +
                                             (uint32_t)(c >> 3) * C::kHalf + (uint32_t)(r & 127) * 128 +
                                             (uint32_t)(((c & 7) ^ (r & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                     ::"r"(dst), "r"(v[i].x ^ flip), "r"(v[i].y ^ flip), "r"(v[i].z ^ flip),
                                       "r"(v[i].w ^ flip) : "memory");
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(ptx::smem_addr(q_full));
            const int my_row = (two ? stream * 128 : 0) + row;            // of the block
            const bool warp_works = (two ? stream * 128 : 0) + quarter * 32 < rows;
            const int t = min(row0 + my_row, s.n * p.group - 1) / p.group;    // its token
            float m = -INFINITY, l = 0.f;
            bool begun = false;                          // O has a product in it
            for (int j = two ? 0 : stream; j < nt && ok; j += two ? 1 : 2, ++tiles_done) {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                ok = wait_soon(ptx::smem_addr(s_full + 2 * stream + h), tiles_done & 1, abort_flag, p.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                const int key0 = (s.tile0 + j) * kKeys + h * 64;
                const bool drafted = key0 + 64 > s.ctx, tile_drafted = h == 0 && key0 + kKeys > s.ctx;
                if (warp_works) {
                    uint32_t x[64];
                    tc::ld_32x32b_x32(t_s + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                    tc::ld_32x32b_x32(t_s + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                    tc::ld_wait();
                    if (drafted) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t seen = seen32(p, s, t, key0 + c * 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((seen >> e) & 1u)) x[c * 32 + e] = 0xFF800000u;   // -inf
                        }
                    }
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale - kWeightBias<T>;
                    const bool grown = mx > m + kSlack || (m == -INFINITY && mx > -INFINITY);
                    if (__any_sync(0xFFFFFFFFu, grown)) {
                        const float nm = grown ? mx : m;
                        const float f = nm == m ? 1.f : exp2_fast(m - nm);
                        m = nm;
                        l *= f;
                        if (begun) {
                            // The half before may still be added to O. (Those before
                            // it are: this S was issued behind them.)
                            const uint32_t half = 2 * tiles_done + h;
                            ok = wait_soon(ptx::smem_addr(pv_done + stream), (half - 1) & 1, abort_flag, p.status);
                            ok = __all_sync(0xFFFFFFFFu, ok);
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < DP / 32; ++c) {
                                uint32_t o[32];
                                tc::ld_32x32b_x32(t_o + c * 32, o);
                                tc::ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st_32x32b_x32(t_o + c * 32, o);
                            }
                        }
                    }
                    const float mm = m == -INFINITY ? 0.f : m;
                    const float2 scale2 = make_float2(scale, scale), mm2 = make_float2(-mm, -mm);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        float2 a = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, mm2);
                        a.x = exp2_fast(a.x);
                        a.y = exp2_fast(a.y);
                        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], a);
                        w[e >> 1] = Elem<T>::pack(a.x, a.y);
                    }
                    tc::st_32x32b_x32(t_s + h * 64, w);
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc::st_wait();
                }
                begun = true;
                if (tile_drafted) {
                    // The tile's values before this stream's P V reads them: rows
                    // past the last key become zero, and so do infinities and NaN of
                    // drafted keys, which the epilogue gives to the rows that see
                    // them. With two row halves both streams do so, each for its
                    // own product: a second write is the same zero.
                    const int v_at = base + (two ? 1 + j + min(j, nt - 1) : min(2, nt) + j + min(j, max(0, nt - 2)));
                    const int slot = v_at % C::kSlots;
                    ok = wait_soon(ptx::smem_addr(full + slot), (v_at / C::kSlots) & 1, abort_flag, p.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t vt = ptx::smem_addr(smem + C::kQ + slot * C::kTile);
                    const int first = max(0, s.ctx - key0);
                    for (int e = first * (DP / 8) + (tid & 127); e < kKeys * (DP / 8); e += 128) {
                        const int r = e / (DP / 8), c = e % (DP / 8);
                        const uint32_t a = vt + (uint32_t)(c >> 3) * C::kHalf + (uint32_t)r * 128 +
                                           (uint32_t)(((c & 7) ^ (r & 7)) << 4);
                        if (key0 + r >= s.ctx + s.n) {
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                            continue;
                        }
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
                        bool odd = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (has_nonfinite<T>(w[i])) {
                                odd = true;
                                if ((w[i] & Elem<T>::kExpMask) == Elem<T>::kExpMask) w[i] &= 0xFFFF0000u;
                                if (((w[i] >> 16) & Elem<T>::kExpMask) == Elem<T>::kExpMask) w[i] &= 0x0000FFFFu;
                            }
                        if (odd) {
                            *odd_flag = 1;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                         ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(p_full + 2 * stream + h));
                }
                if (!ok) break;
            }
            base += 2 * nt;

            // ---- the segment's end: all MMAs of both streams are done
            for (int st = 0; st < 2; ++st)
                ok = ok && wait_soon(ptx::smem_addr(o_full + st), segs_done & 1, abort_flag, p.status);
            ++segs_done;
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc::fence_after_sync();
            if (!ptx::named_barrier_and(1, kSoftmax, ok)) {
                ok = false;
                break;
            }
            pair_m[stream * 128 + row] = m;
            pair_l[stream * 128 + row] = l;
            ptx::named_barrier(1, kSoftmax);
            // factors of the two streams' O (of this one's alone with two row halves)
            float f0 = 1.f, f1 = 0.f;
            if (!two) {
                const float m0 = pair_m[row], m1 = pair_m[128 + row], l0 = pair_l[row], l1 = pair_l[128 + row];
                m = fmaxf(m0, m1);
                const float mm = m == -INFINITY ? 0.f : m;
                f0 = exp2_fast(m0 - mm);
                f1 = exp2_fast(m1 - mm);
                l = l0 * f0 + l1 * f1;
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const bool whole = s.whole(), odd = *odd_flag != 0;
            float *slot = p.partials + (int64_t)work.slot_of(s) * slot_floats(kRows, DP);
            if (warp_works) {
                const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
                // with shared rows each stream's warps write half of the columns
                const int c_lo = two ? 0 : stream * (DP / 2), c_hi = two ? DP : c_lo + DP / 2;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; c += 32) {
                    __syncwarp();            // rows differ in what they store; tensor memory is read by whole warps
                    uint32_t raw[32];
                    float o[32];
                    tc::ld_32x32b_x32((two ? t_o : t_lane + kO) + c, raw);
                    tc::ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(raw[e]) * f0;
                    if (!two && nt > 1) {
                        tc::ld_32x32b_x32(t_lane + kO + 128 + c, raw);
                        tc::ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] += __uint_as_float(raw[e]) * f1;
                    }
                    if (odd) {
                        for (int key = max(s.ctx, s.tile0 * kKeys); key < min(s.ctx + s.n, s.tile1 * kKeys); ++key) {
                            if (!(seen_bits(p, s, t, key - s.ctx) & 1u)) continue;
                            const int id = p.table[(int64_t)s.b * p.table_stride + (key >> p.shift)];
                            if (id < 0 || id >= p.num_blocks) continue;
                            const T *v = static_cast<const T *>(p.v_data) + id * p.v_block_stride +
                                         (int64_t)(key & ((1 << p.shift) - 1)) * p.v_token_stride + s.h * p.v_head_stride;
#pragma unroll 1
                            for (int e = 0; e < 32; ++e) {
                                if (c + e >= p.head_dim) break;
                                const uint16_t bits = reinterpret_cast<const uint16_t *>(v)[c + e];
                                if ((bits & Elem<T>::kExpMask) != Elem<T>::kExpMask) continue;
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (i == e) o[i] += Elem<T>::to_float(bits);
                            }
                        }
                    }
                    if (whole) {
                        if (my_row < rows) {
                            const int64_t head = (int64_t)s.h * p.group + (row0 + my_row) % p.group;
                            T *out = static_cast<T *>(p.out) + ((int64_t)(s.token0 + t) * p.q_heads + head) * p.head_dim + c;
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                if (c + e < p.head_dim)
                                    *reinterpret_cast<uint4 *>(out + e) =
                                        make_uint4(Elem<T>::pack(o[e], o[e + 1]), Elem<T>::pack(o[e + 2], o[e + 3]),
                                                   Elem<T>::pack(o[e + 4], o[e + 5]), Elem<T>::pack(o[e + 6], o[e + 7]));
                        }
                    } else if (my_row < rows) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            __stcg(reinterpret_cast<float4 *>(slot + slot_at(kRows, my_row, c + e)),
                                   make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                    }
                }
                if (my_row < rows && (two || stream == 0)) {
                    if (whole) {
                        store_lse(p, s.token0, s.h, row0 + my_row, mm, l);
                    } else {
                        __stcg(slot + kRows * DP + my_row, m);
                        __stcg(slot + kRows * DP + kRows + my_row, l);
                    }
                }
            }
            tc::fence_before_sync();
            if (!whole && tid == 0 && s.tile1 == s.tiles) work.note_join(p, s, rows);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

struct LaunchInfo {
    int sms = 0;
    cudaError_t err = cudaSuccess;
    unsigned gen = 0;
};

template <typename T, int DP, int kRows>
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
    li.err = cudaFuncSetAttribute(attention_tc_kernel<T, DP, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP, kRows>::kSmem);
    if (li.err == cudaSuccess) li.err = cudaDeviceGetAttribute(&li.sms, cudaDevAttrMultiProcessorCount, dev);
    if (li.err == cudaSuccess) cache[dev] = li;
    return li;
}

template <typename T, int DP, int kRows>
cudaError_t launch_tc(const awq_tree_attention_t &a, cudaStream_t stream)
{
    const LaunchInfo li = launch_info<T, DP, kRows>();
    if (li.err != cudaSuccess) return li.err;
    Params p = make_params(a);
    // no zero: a masked score, -inf times the scale, has to stay -inf
    if (p.scale_log2 == 0.f) p.scale_log2 = 1e-30f;
    CUtensorMap tk, tv;
    if (!make_cache_map(&tk, a, a.k_cache, kKeys) || !make_cache_map(&tv, a, a.v_cache, kKeys))
        return cudaErrorInvalidValue;
    const int64_t tiles = tiles_bound(a, kKeys), blocks = blocks_bound(a, kRows);
    p.whole = tiles <= kWholeTiles;
    p.min_units = p.whole ? 1 : kBlockCost<kRows> + 4;
    const int64_t units = p.whole ? blocks : blocks * (kBlockCost<kRows> + (kRows > 128 ? 2 : 1) * tiles);
    const int ctas = lay_out(p, li.sms, units);
#ifdef AWQ_FAULT_TEST
    p.fault = fault_injection();
#endif
    return launch_pair<T, kRows, DP>(attention_tc_kernel<T, DP, kRows>, ctas, kThreads, Cfg<DP, kRows>::kSmem, stream, tk, tv, p);
}

} // namespace

template <typename T, int DP>
cudaError_t launch_tc_rows(const awq_tree_attention_t &a, cudaStream_t stream)
{
    return rows_bound(a) <= 128 ? launch_tc<T, DP, 128>(a, stream) : launch_tc<T, DP, 256>(a, stream);
}

cudaError_t launch_tc_any(const awq_tree_attention_t &a, cudaStream_t stream)
{
    const bool f16 = a.dtype == AWQ_F16;
    if (a.head_dim <= 64) return f16 ? launch_tc_rows<__half, 64>(a, stream) : launch_tc_rows<__nv_bfloat16, 64>(a, stream);
    return f16 ? launch_tc_rows<__half, 128>(a, stream) : launch_tc_rows<__nv_bfloat16, 128>(a, stream);
}

size_t tc_partial_floats(int sms, int64_t head_dim)
{
    return head_dim > 128 ? 0 : scratch_floats(sms, 256, head_dim <= 64 ? 64 : 128);
}

} // namespace attn
} // namespace awq

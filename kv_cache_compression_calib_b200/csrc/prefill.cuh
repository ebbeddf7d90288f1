// Causal attention of new tokens over the cache that ends with them (the step around
// "TriAttention：基于三角函数 KV 压缩的高效长推理", 流程详解 step 5): for each (layer l,
// token i of sequence s's n, query head g of KV head h), over slots j <= N - n + i of
// row (l, s, h),
//   s_j = scale * (q . k_j),  out = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}.
//
// 4 d flops per visible (query, key) pair: tensor-core bound for prompts, HBM bound
// (K and V read once) for a few tokens over a long row.  The G query heads of a KV
// head share its keys, so the rows of the product are the (token, head) pairs of one
// KV head in token order: a prompt of n tokens is n * G rows, cut into items of up to
// 256.  One block per SM (12 warps) takes item after item: its first by its place in
// the grid, the next ones from the blocks that the hardware has not launched yet
// (cluster launch control), a sequence's heaviest first, so the grid needs no counter in memory.
//
// For an item's two 128-row query tiles it computes
//   S = Q K^T  and  O += P V,  P = 2^(S scale log2(e) - m),
// on tcgen05.mma (kind::f16, bf16 operands - fp16 where the cache is fp8, below - and fp32
// accumulators in tensor memory):
//   - warps 0-3 and 4-7: the softmax of query tile 0 and 1, one thread per row.  S is
//     read from tensor memory, P (bf16) written back over it as the A operand of P V,
//     which starts on the first half of the keys while the second half's weights are
//     formed.  While one tile's softmax runs, the other tile's products do.
//   - warp 8: brings Q (by TMA where G divides 128) and K and V tiles (128 keys; 64
//     at head dim 256) into a ring in shared memory, 128-byte swizzled, one box per 64
//     dims of a contiguous tile or of a page.  It runs ahead into the next item.
//   - warp 9: issues every product.
//     Many small copies take long to issue: for pages and few rows warp 11 brings V beside it.
//   - warps 10 and 11: see to V tiles that some row sees in part (below), and widen fp8
//     tiles to fp16 from a second ring; warp 10 also finds the next item.
//     Pages of fewer than 8 slots (a swizzle atom) are copied by warps 8, 10 and 11.
// Head dim 256 fits one query tile (its O takes half of tensor memory); its S is
// double-buffered instead.
//
// fp8 caches: e4m3 widens to fp16 by one conversion per two values (to bf16 it takes
// five instructions), exactly.  The queries then have to be fp16 as well: a row is
// scaled by the power of two that brings its largest value to [2^14, 2^15), which its
// score scale takes back, so values down to 2^-31 of the largest keep all eight bits of
// their bf16.  P is fp16, too, whose smallest numbers are not far below 1: the maximum's weight is
// put to 2^10 and may grow to 2^14, so that weights down to 2^-27 of the largest are as good as
// in bf16 (half a step, 2^-8), and all within 2^-35 of the largest.  (At 1 and 2^8, keys 17 nats below an
// attention sink were lost.)
//
// The maximum m a row subtracts is only raised when its weights pass 2^8 (bf16) or 2^14 (fp16),
// which neither these types nor fp32 mind, so O is rescaled rarely.
// Statistics and O are fp32.  P is rounded to bf16 because a product's operands have one type:
// half a step per weight, which brings outputs to 2.3e-3 of the 64-bit rule (norm of the difference)
// where rounding them alone gives 1.7e-3.  Two bf16 parts of P, as the single-token call
// has them, would double the product with V on the unit that bounds prompts.
//
// Keys a row must not see get weight exactly 0, but 0 * NaN is NaN in the product:
// rows of V outside the cache row are zero-filled, and in the tiles that some row sees
// only in part, NaN and infinite values of V are taken out and noted per dim; the
// epilogue gives them back to the rows that see them.
//
// An item of at most 128 rows leaves the second query tile empty: both softmax
// warpgroups then take the same rows, one the even key tiles and one the odd ones, and the
// first merges the two (a "twin" item; one token over a 2K row waits on the chain product -
// softmax - product, not on memory).
//
// Measured (one B200, 32/8 heads of 128): a 32K prompt 7.5 ms, 1.18 PFLOP/s; 16 ragged prompts of
// 100 to 4096 tokens 770 us, 0.94 PFLOP/s; 512 tokens over 32K paged slots 279 us; 3 to 5 tokens over
// 20K to 33K paged slots 104 us, 4.3 TB/s.  Per pair of query tiles and 128 keys the loop takes 3140 cycles, 2048 of
// them the tensor pipe's: each warpgroup's scores, maximum, weights and products are one chain,
// and the other warpgroup hides two thirds of it.
//
// When the items are fewer than the SMs, each row is split over its keys, and
// prefill_join merges the parts.
//
// Every wait is bounded.  A warp whose wait runs out sets the flag and the block's mark, on which the
// others give up in their next long wait; when all have, the block waits (bounded again) for copies and
// products on their way and gives its tensor memory back.
#pragma once

#include <algorithm>

#include <cuda_bf16.h>

#include "keys.cuh"
#include "span.h"
#include "tc.cuh"
#include "tensormap.cuh"

// How a wait tries, when it looks whether its time is over (a try lasts up to some 16 us), and whether
// it gives up before that: the self-test of the waits has them end after a given number of short tries.
#ifndef TRI_WAIT_TRY
#define TRI_WAIT_TRY mbar_test
#define TRI_WAIT_LOOK(it, p) (((it) & 4095u) == 0)
#define TRI_WAIT_OVER(it, p) false
#endif

namespace tri {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;     // rows of a query tile: one per thread of a softmax warpgroup
constexpr int kSlots = 3;      // items known to the block: the next, the current, the last

// How a cache's tiles come: TMA of bf16 rows or pages, TMA of fp8 and widened, or copied
// record by record.
enum { kTma16, kPage16, kTma8, kCopy16, kCopy8 };
enum { kBoth, kKeys, kValues };  // what a TMA warp brings
constexpr uint32_t kMends = 0x80000000u, kOdd = 0x40000000u;  // marks of a copy in flight

template <int D, int SRC, bool FEW>
struct Cfg {
    static constexpr int NT = D == 256 ? 1 : 2;     // query tiles per item
    static constexpr int BN = D == 256 ? 64 : 128;  // keys per tile
    static constexpr int kRowsPer = NT * kRows;     // rows per item
    static constexpr int kStageBytes = BN * D * 2;
    static constexpr int kStages = D == 64 ? 8 : SRC == kTma8 ? 3 : 4;
    static constexpr int kRawBytes = BN * D;  // an fp8 tile
    static constexpr int kRaws = SRC == kTma8 ? (D == 64 ? 4 : 2) : 0;
    static constexpr int kQBytes = kRows * D * 2;  // per query tile
    static constexpr int kSubQ = kRows * 128;      // a 64-dim column of a Q tile
    static constexpr int kSubK = BN * 128;         // ... of a K or V tile
    static constexpr bool kTwins = FEW && D != 256;  // items of at most 128 rows are twin items
    static constexpr bool kTma = SRC == kTma16 || SRC == kPage16;  // bf16 by TMA
    static constexpr bool kF16 = SRC == kTma8 || SRC == kCopy8;  // fp16 operands
    // log2 of a weight of the maximum when it is raised, and of how far weights may pass that before it is
    // raised again.
    static constexpr float kLift = kF16 ? 10.f : 0.f, kRaise = kF16 ? 4.f : 8.f;
    static constexpr int kLoaders = 96;  // threads that copy
    // tensor memory columns
    static constexpr int kTmemS(int b) { return b * BN; }  // S (and P) of tile b, or buffer b
    static constexpr int kTmemO(int t) { return 256 + t * D; }
    // shared memory from a 1024-byte aligned base
    static constexpr int kSmRing = NT * kQBytes;
    static constexpr int kSmRaw = kSmRing + kStages * kStageBytes;
    static constexpr int kSmBad = kSmRaw + kRaws * kRawBytes;  // int [3][D]
    static constexpr int kSmTwin = kSmBad + 3 * D * 4;         // float2 [kRows]
    static constexpr int kSmMisc = kSmTwin + kRows * 8;
};

template <int STAGES, int RAWS>
struct Shared {
    alignas(16) uint4 claim;  // cluster launch control's answer
    uint64_t full[STAGES], empty[STAGES], land[STAGES];
    uint64_t raw_full[RAWS + 1], raw_empty[RAWS + 1];
    uint64_t q_full, q_land, q_empty, claimed, drain, twin_done, keys_begun;
    uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_free[2];
    uint64_t item_full[kSlots], item_empty[kSlots], scanned[kSlots], helpers;
    // Per stage of the ring that copies land in, its last fill, and for the queries their item; with kMends
    // where the fill is mended, kOdd beside it where its phase of land is odd; -1 for none.
    uint32_t in_flight[STAGES + 1];
};

struct Misc {
    uint32_t tmem;
    volatile uint32_t abort_flag;
    volatile uint32_t land;  // bit st: parity of the next phase of land[st]
};

// -------------------------------------------------------------------- waits

// Bounded wait of one role's warp (the clock is read once in 4096 tries).  When it runs out
// the block is told to stop.  The warp gives up only where all its lanes still wait: a lane
// that saw the barrier complete just as others gave up would wait for them in the collective
// instructions that follow.  (A vote on every wait instead: 7% on prompts.)
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, Misc *misc, const PrefillParams &p) {
    unsigned long long t0 = 0;
    for (uint32_t it = 1;; it++) {
        if (TRI_WAIT_TRY(bar, parity)) return true;
        if (TRI_WAIT_LOOK(it, p)) {
            const unsigned long long t = global_ns();
            if (t0 == 0) t0 = t;
            if (__activemask() == 0xffffffffu &&
                __any_sync(0xffffffffu, TRI_WAIT_OVER(it, p) || t - t0 > kStageWaitNs || misc->abort_flag))
                break;
            if (it >= kStageWaitIters) break;
        }
    }
    misc->abort_flag = 1u;
    atomicOr(p.flags, TRI_FLAG_STAGE_TIMEOUT);
    return false;
}

// ------------------------------------------------------------------ the work

struct Block {
    int l, h, seq;
    int n;         // new tokens of the sequence; -1: no work is left
    int rows;      // n * G
    int row0;      // first row of this block
    int len;       // N: slots of the cache row
    int64_t tok0;  // tok_off[seq]
    int64_t lo;    // row_off
    int beg;       // first key tile (of the split)
    int cnt[2];    // key tiles of each query tile, from beg; of a twin item, of each half
    int twin;      // both query tiles are the same rows, tile t taking key tiles t, t + 2, ...
    int place;     // of its part, where rows are split
    volatile uint32_t any_bad;      // a NaN or infinite value of V was taken out
    volatile uint32_t any_missing;  // a slot without a block
    volatile uint32_t mend;         // V tiles seen in part hold NaN or infinities
    __device__ __forceinline__ int tiles() const { return twin ? cnt[0] + cnt[1] : max(cnt[0], cnt[1]); }
};

// x / G for 0 <= x < 2^31, by multiplication: mul = ceil(2^(31 + l) / G), l = ceil(log2 G).
__device__ __forceinline__ int token_of(const PrefillParams &p, int x) {
    return (int)(((unsigned long long)(unsigned)x * p.div_mul) >> p.div_shift);
}
// Last slot row x (of the sequence's rows) sees.
__device__ __forceinline__ int last_seen(const PrefillParams &p, const Block &b, int x) { return b.len - b.n + token_of(p, x); }
// Row x's place among the rows of q, out and lse.
__device__ __forceinline__ int64_t row_of(const PrefillParams &p, const Block &b, int x) {
    const int i = token_of(p, x);
    return ((int64_t)b.l * p.T + b.tok0 + i) * p.geo.Hq + b.h * p.geo.G + (x - i * p.geo.G);
}

// The block's share of the work, by one warp: sequence after sequence, each cut into
// ceil(n G / (128 NT)) blocks, the last rows (most keys) first, each for all heads before the
// next: the shortest items then come last.  (Head after head, every head's long items came
// behind the short ones of the head before: 8K prompt 523 -> 448 us.)
template <int D, bool TWINS>
__device__ __forceinline__ bool find_block(const PrefillParams &p, int idx, int split, Block *out) {
    constexpr int R = kRows * Cfg<D, 0, false>::NT, BN = Cfg<D, 0, false>::BN;
    const Geometry &geo = p.geo;
    const int lane = threadIdx.x & 31;
    int b = idx / (geo.L * geo.H);
    const int lh = idx - b * (geo.L * geo.H);
    const int l = lh / geo.H, h = lh - l * geo.H;
    for (int base = 0; base < geo.S; base += 32) {
        const int s = base + lane;
        // A lane's sequence: its tokens and, before it is known whose they are, its cache row.
        int64_t t0 = 0, n = 0, lo = 0, hi = 0;
        if (s < geo.S) {
            const int64_t r = ((int64_t)l * geo.S + s) * geo.H + h;
            t0 = p.tok_off[s];
            n = p.tok_off[s + 1] - t0;
            lo = geo.row_off[r];
            hi = geo.row_off[r + 1];
            if (t0 < 0 || n < 0 || t0 + n > p.T || (s == 0 && t0 != 0)) {
                atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
                n = 0;
            }
        }
        int upto = (int)((n * geo.G + R - 1) / R);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, b < upto);
        if (here) {
            if (lane == __ffs(here) - 1) {
                if (lo < 0 || hi < lo || hi > geo.total || hi - lo > 0x7fffff00LL) {
                    atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
                    hi = lo = 0;
                }
                const int rows = (int)(n * geo.G), row0 = (upto - 1 - b) * R, old = (int)(hi - lo) - (int)n;
                int c[2] = {0, 0};
#pragma unroll
                for (int t = 0; t < Cfg<D, 0, false>::NT; t++) {
                    const int first = row0 + t * kRows;
                    if (first < rows) c[t] = max(0, old + token_of(p, min(first + kRows, rows) - 1) + BN) / BN;
                }
                const int all = max(c[0], c[1]);
                const int beg = p.splits == 1 ? 0 : (int)((int64_t)all * split / p.splits);
                const int end = p.splits == 1 ? all : (int)((int64_t)all * (split + 1) / p.splits);
                int c0 = max(0, min(c[0], end) - beg), c1 = max(0, min(c[1], end) - beg);
                const bool twin = TWINS && row0 + kRows >= rows;
                if (twin) {
                    c1 = c0 / 2;
                    c0 -= c1;
                }
                Block &w = *out;
                w.l = l;
                w.h = h;
                w.seq = s;
                w.n = (int)n;
                w.rows = rows;
                w.row0 = row0;
                w.len = (int)(hi - lo);
                w.tok0 = t0;
                w.lo = lo;
                w.beg = beg;
                w.cnt[0] = c0;
                w.cnt[1] = c1;
                w.twin = twin;
            }
            if (idx == 0)  // the first block looks at the offsets of the sequences behind its own, too
                for (int x = s + 32; x < geo.S; x += 32)
                    if (p.tok_off[x] > p.tok_off[x + 1] || p.tok_off[x + 1] > p.T) atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
            return true;
        }
        b -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// Record of slot j of the block's row; -1 if its table names none.
__device__ __forceinline__ int64_t record(const Geometry &geo, const Block &b, int j) {
    if (geo.layout != TRI_KV_PAGED) return b.lo + j;
    const int bi = j >> geo.block_shift;
    const int32_t blk = bi < geo.max_blocks ? __ldg(geo.block_table + (int64_t)b.seq * geo.max_blocks + bi) : -1;
    if (blk < 0 || blk >= geo.n_blocks) return -1;
    return ((((int64_t)b.l * geo.n_blocks + blk) << geo.block_shift) | (j & ((1 << geo.block_shift) - 1))) * geo.H + b.h;
}

// Byte of (row, 16-byte chunk c of d) in a swizzled tile whose 64-dim columns are `sub` bytes.
__device__ __forceinline__ uint32_t tile_at(int row, int c, int sub) {
    return (uint32_t)((c >> 3) * sub + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// ------------------------------------------------------------------- loading

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Takes NaN and infinities out of 8 bf16 values of V (dims d0.., slot j), noting for
// each dim the first slot that has one: bad[0] NaN, bad[1] +inf, bad[2] -inf.
template <int D>
__device__ __forceinline__ uint4 take_out(uint4 v, int d0, int j, int *bad, Block *b) {
    b->any_bad = 1u;
    const auto word = [&](uint32_t w, int d) {
#pragma unroll 1
        for (int k = 0; k < 2; k++) {
            const uint32_t x = (w >> (16 * k)) & 0xffffu;
            if ((x & 0x7f80u) != 0x7f80u) continue;
            const int kind = (x & 0x7fu) ? 0 : (x & 0x8000u) ? 2 : 1;
            atomicMin(bad + kind * D + d + k, j);
            w &= ~(0xffffu << (16 * k));
        }
        return w;
    };
    return make_uint4(word(v.x, d0), word(v.y, d0 + 2), word(v.z, d0 + 4), word(v.w, d0 + 6));
}
// Whether one of 8 bf16 values has the exponent of NaN and infinity (some bit of
// 0x80008000): adding 1 to the exponent field then carries into the sign's place, and
// nowhere else.
__device__ __forceinline__ uint32_t special_bits(uint4 v) {
    const auto one = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
    return one(v.x) | one(v.y) | one(v.z) | one(v.w);
}
__device__ __forceinline__ bool has_special(uint4 v) { return (special_bits(v) & 0x80008000u) != 0; }

// Four e4m3 values as fp16 (exact; NaN stays NaN).
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
    return r;
}
// 16 e4m3 values of a tile's row as two chunks of fp16.
__device__ __forceinline__ void widen16(uint4 v, unsigned char *tile, int row, int ch, int sub) {
    const uint2 a = widen4(v.x), b = widen4(v.y), c = widen4(v.z), d = widen4(v.w);
    *reinterpret_cast<uint4 *>(tile + tile_at(row, 2 * ch, sub)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4 *>(tile + tile_at(row, 2 * ch + 1, sub)) = make_uint4(c.x, c.y, d.x, d.y);
}
// Whether one of 16 e4m3 values is NaN.
__device__ __forceinline__ bool has_nan8(uint4 v) {
    const auto one = [](uint32_t x) { return (x & 0x7f7f7f7fu) + 0x01010101u; };
    return ((one(v.x) | one(v.y) | one(v.z) | one(v.w)) & 0x80808080u) != 0;
}
// take_out for 16 e4m3 values (which have no infinities).
__device__ __forceinline__ uint4 take_out8(uint4 v, int d0, int j, int *bad, Block *b) {
    b->any_bad = 1u;
    const auto word = [&](uint32_t w, int d) {
#pragma unroll 1
        for (int k = 0; k < 4; k++)
            if ((w >> (8 * k) & 0x7fu) == 0x7fu) {
                atomicMin(bad + d + k, j);
                w &= ~(0xffu << (8 * k));
            }
        return w;
    };
    return make_uint4(word(v.x, d0), word(v.y, d0 + 4), word(v.z, d0 + 8), word(v.w, d0 + 12));
}

// The order in which an item's key tiles are brought: K_0, V_0, K_1, V_1, ...; with FEW
// K_0, then K_{j+1} before V_j, and the last V.  V_j is held until its weights are formed
// and used, and K_{j+1} behind it would come a copy's latency too late where one tile's
// chain of steps is the bound (4 tokens over 27K slots 105 -> 99 us); in short items the
// first values come too late instead (2K-token prompts 339 -> 345 us).
template <bool FEW>
struct Fill {
    int tile;
    bool v;
    __device__ __forceinline__ Fill(int g, int tiles) {
        const bool last = g == 2 * tiles - 1;
        v = FEW ? last || (g > 0 && g % 2 == 0) : g & 1;
        tile = !FEW ? g >> 1 : last ? tiles - 1 : v ? g / 2 - 1 : (g + 1) / 2;
    }
    static __device__ __forceinline__ int of_k(int j) { return !FEW ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
    static __device__ __forceinline__ int of_v(int j, int tiles) {
        return !FEW ? 2 * j + 1 : j + 1 < tiles ? 2 * j + 2 : 2 * tiles - 1;
    }
};

// Query tile t's first row sees this many slots: key tiles past them are seen in part.
struct Partial {
    int beg, cnt[2], first[2];
    __device__ __forceinline__ Partial(const PrefillParams &p, const Block &b) {
        beg = b.beg;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            cnt[t] = b.twin ? (t ? 0 : b.tiles()) : b.cnt[t];
            first[t] = last_seen(p, b, b.row0 + t * kRows) + 1;
        }
    }
    template <int BN>
    __device__ __forceinline__ bool tile(int j) const {
        const int end = (beg + j + 1) * BN;
        return (j < cnt[0] && end > first[0]) || (j < cnt[1] && end > first[1]);
    }
    // First slot of tile j that some row does not see.
    __device__ __forceinline__ int from(int j) const {
        return min(j < cnt[0] ? first[0] : 0x7fffffff, j < cnt[1] ? first[1] : 0x7fffffff);
    }
};

__device__ __forceinline__ void tma2(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// What the roles of a block share.
template <int D, int SRC, bool FEW>
struct Ctx {
    using C = Cfg<D, SRC, FEW>;
    using Sh = Shared<C::kStages, C::kRaws>;
    const PrefillParams &p;
    unsigned char *sm;
    Sh *sh;
    Block *slots;
    Misc *misc;
    uint32_t tmem;

    // Between the loading warps that fill or mend tiles.
    static constexpr int kHelpers = SRC >= kCopy16 ? 96 : 64;
    __device__ __forceinline__ bool paged() const {
        return SRC == kTma16 ? false : SRC == kPage16 ? true : p.geo.layout == TRI_KV_PAGED;
    }
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t n) const { return role_wait(bar, n & 1u, misc, p); }
    // A barrier of the helpers that gives up as every wait does; `syncs` counts a warp's.
    __device__ __forceinline__ bool sync_helpers(int *syncs) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->helpers);
        return wait(&sh->helpers, (*syncs)++);
    }
    // The n-th item, when it is known; nullptr at the end.
    __device__ __forceinline__ Block *item(int n) const {
        if (!wait(sh->item_full + n % kSlots, n / kSlots)) return nullptr;
        Block *b = slots + n % kSlots;
        return b->n < 0 ? nullptr : b;
    }
    // A warp is done with the n-th item.
    __device__ __forceinline__ void leave(int n) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(sh->item_empty + n % kSlots);
    }
    // Per dim, the first slot whose V is NaN, +inf, -inf there (any_bad of the item says whether any is).
    __device__ __forceinline__ int *bad() const { return reinterpret_cast<int *>(sm + C::kSmBad); }
    // One warp, when no more copies are asked for: those on their way have landed.
    __device__ __forceinline__ void drain_copies() const {
        const int st = threadIdx.x & 31;
        constexpr int RING = SRC == kTma8 ? C::kRaws : C::kStages;
        if (st > C::kStages || sh->in_flight[st] == 0xffffffffu) return;
        const uint32_t mark = sh->in_flight[st];
        if (st == C::kStages) mbar_wait(C::kF16 ? &sh->q_land : &sh->q_full, mark & 1);
        else if (mark & kMends) mbar_wait(sh->land + st, mark & kOdd ? 1u : 0u);
        else mbar_wait(SRC == kTma8 ? sh->raw_full + st : sh->full + st, (mark / RING) & 1);
    }
    __device__ __forceinline__ unsigned char *stage(int f) const { return sm + C::kSmRing + (f % C::kStages) * C::kStageBytes; }
};

// --------------------------------------------------------------- finding work

// Warp 10: the place in the grid of a block that the hardware has not launched, which
// then never will be; -1 when none is left (not to be asked again).
template <int D, int SRC, bool FEW>
__device__ __forceinline__ int claim_block(const Ctx<D, SRC, FEW> &c, int *claims) {
    if ((threadIdx.x & 31) == 0) {
        mbar_arrive_expect_tx(&c.sh->claimed, 16);
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                smem_u32(&c.sh->claim)),
            "r"(smem_u32(&c.sh->claimed))
            : "memory");
    }
    __syncwarp();
    if (!c.wait(&c.sh->claimed, *claims)) {
        mbar_wait(&c.sh->claimed, *claims & 1);  // the answer is on its way into this block's memory
        return -1;
    }
    ++*claims;
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\tld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(&c.sh->claim))
        : "memory");
    fence_async_smem();  // the answer is read before the next one is written
    __syncwarp();
    return got ? (int)x : -1;
}

// Warp 10: the n-th item into its slot, or the word that there is none (false then).
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool next_item(const Ctx<D, SRC, FEW> &c, int n, int *claims) {
    const int lane = threadIdx.x & 31;
    Block *b = c.slots + n % kSlots;
    if (n >= kSlots && !c.wait(c.sh->item_empty + n % kSlots, n / kSlots - 1)) return false;
    __syncwarp();
    if (lane == 0) b->any_bad = b->any_missing = b->mend = 0u;
    int idx = n == 0 ? (int)blockIdx.x : claim_block(c, claims);
    bool found = false;
    while (idx >= 0) {  // the blocks of the grid are a bound: some name no item
        const int unit = c.p.splits == 1 ? idx : idx / c.p.splits;
        found = find_block<D, Ctx<D, SRC, FEW>::C::kTwins>(c.p, unit, idx - unit * c.p.splits, b);
        if (found) break;
        idx = claim_block(c, claims);
    }
    __syncwarp();
    if (lane == 0) {
        if (found) b->place = idx;
        else b->n = -1;
        mbar_arrive(c.sh->item_full + n % kSlots);
    }
    return found;
}

// -------------------------------------------------------------------- loading

// An item's copies by TMA: all of them by warp 8, or the queries and K by warp 8 and V by
// warp 11.
// Where the scan found NaN or infinities, V tiles that are seen in part land on land[stage],
// for the mending warps; fp8 tiles land in the raw ring, for the widening ones.  Pages
// behind the row's end, or that the table does not name, are asked for behind the end of
// the pool, where a copy delivers zeros.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool tma_item(const Ctx<D, SRC, FEW> &c, const CUtensorMap *mk, const CUtensorMap *mv, const CUtensorMap *mq,
                                         Block *b, int n, int fill, int which) {
    using C = Cfg<D, SRC, FEW>;
    constexpr int BN = C::BN;
    constexpr bool RAW = SRC == kTma8;
    const PrefillParams &p = c.p;
    const Geometry &geo = p.geo;
    const int lane = threadIdx.x & 31;
    const bool paged = c.paged();
    const int box = paged ? min(1 << geo.block_shift, BN) : BN;  // slots per copy
    constexpr int kNone = -1, kMissing = -2;
    const int pool_end = (int)(paged ? (int64_t)geo.L * geo.n_blocks << geo.block_shift : geo.total);
    const Partial part(p, *b);
    const int tiles = b->tiles(), len = b->len, beg = b->beg, h = b->h;
    const int64_t lo = b->lo, layer = (int64_t)b->l * geo.n_blocks;
    const int32_t *table = geo.block_table + (int64_t)b->seq * geo.max_blocks;
    // Slot of the pool that a copy starts at for slot j of the row.
    const auto slot_of = [&](int j) -> int {
        if (lane * box >= BN || j >= len) return kNone;
        if (!paged) return (int)(lo + j);
        const int bi = j >> geo.block_shift;
        const int32_t blk = bi < geo.max_blocks ? __ldg(table + bi) : -1;
        if (blk < 0 || blk >= geo.n_blocks) return kMissing;  // a block that the table does not name
        return (int)(((layer + blk) << geo.block_shift) + (j & ((1 << geo.block_shift) - 1)));
    };
    int k_slot = kNone, v_slot = kNone, next = slot_of(beg * BN + lane * box);
    const int total = max(1, 2 * tiles);  // an item without keys still has its queries
    for (int g = 0; g < total; g++) {
        if (g < 2 * tiles) {
            const int f = fill + g;
            const Fill<FEW> what(g, tiles);
            const bool v = what.v;
            // K and V of a tile come from the same slots, which are looked up one tile ahead.
            const int slot = v ? v_slot : next;
            if (!v) {
                k_slot = next;
                next = what.tile + 1 < tiles ? slot_of((beg + what.tile + 1) * BN + lane * box) : kNone;
            }
            if (!FEW || v || g == 0) v_slot = k_slot;
            if (which != kBoth && v != (which == kValues)) continue;
            constexpr int RING = RAW ? C::kRaws : C::kStages;
            const int st = f % RING, round = f / RING;
            if (round > 0 && !c.wait(RAW ? c.sh->raw_empty + st : c.sh->empty + st, round - 1)) return false;
            bool mend = false;
            uint32_t mark = (uint32_t)f;
            if (!RAW && v && part.tile<BN>(what.tile)) {
                if (!c.wait(c.sh->scanned + n % kSlots, n / kSlots)) return false;
                mend = b->mend;
                if (mend) mark = kMends | (mbar_test_now(c.sh->land + st, 0) ? kOdd : 0u);
            }
            uint64_t *bar = RAW ? c.sh->raw_full + st : mend ? c.sh->land + st : c.sh->full + st;
            const uint32_t dst = smem_u32(RAW ? c.sm + C::kSmRaw + st * C::kRawBytes : c.stage(f));
            if (slot == kMissing) {
                b->any_missing = 1u;
                atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
            }
            __syncwarp();
            if (lane == 0) {
                c.sh->in_flight[st] = mark;
                mbar_arrive_expect_tx(bar, RAW ? C::kRawBytes : C::kStageBytes);
            }
            __syncwarp();
            const CUtensorMap *map = v ? mv : mk;
            constexpr int MOST = BN / 8;
            int at[MOST];
#pragma unroll
            for (int i = 0; i < MOST; i++) {
                const int from = __shfl_sync(0xffffffffu, slot, i);
                at[i] = from < 0 ? pool_end : from;
            }
            if (elect_one()) {
                if (!paged) {
                    if (RAW) {
                        tma2(dst, map, 0, at[0], bar);
                    } else {
#pragma unroll
                        for (int x = 0; x < D / 64; x++) tma2(dst + x * C::kSubK, map, 64 * x, at[0], bar);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MOST; i++) {
                        if (i * box >= BN) break;
                        if (RAW) {
                            tma3(dst + i * box * D, map, 0, h, at[i], bar);
                        } else {
#pragma unroll
                            for (int x = 0; x < D / 64; x++) tma3(dst + x * C::kSubK + i * box * 128, map, 64 * x, h, at[i], bar);
                        }
                    }
                }
            }
            __syncwarp();
        }
        if (g == 0 && which == kKeys && lane == 0) mbar_arrive(&c.sh->keys_begun);
        if (g == 0 && p.q_tma && which != kValues) {  // the query tiles, behind the first key tile
            if (n > 0 && !c.wait(&c.sh->q_empty, n - 1)) return false;
            // (both halves of a twin item scale the same rows where they become fp16)
            const bool same = C::kF16 && C::kTwins && b->twin;
            const int nt = same || (C::NT == 2 && b->row0 + kRows < b->rows) ? 2 : 1;
            uint64_t *bar = C::kF16 ? &c.sh->q_land : &c.sh->q_full;
            if (lane == 0) {
                c.sh->in_flight[C::kStages] = (uint32_t)n;
                mbar_arrive_expect_tx(bar, (uint32_t)(nt * C::kQBytes));
            }
            __syncwarp();
            if (elect_one())
                for (int t = 0; t < nt; t++) {
                    const int64_t tok = (int64_t)b->l * p.T + b->tok0 + token_of(p, b->row0 + (same ? 0 : t * kRows));
#pragma unroll
                    for (int x = 0; x < D / 64; x++)
                        tma3(smem_u32(c.sm + t * C::kQBytes + x * C::kSubQ), mq, 64 * x, h * geo.G, (int)tok, bar);
                }
            __syncwarp();
        }
    }
    return true;
}

// Whether an item's V is warp 11's: pages, where warp 10 has time to do the scan alone, that
// is an item of few rows or a long one.  (4 tokens over 27K paged slots 124 -> 106 us;
// 2K-token prompts, with every item so, 395 -> 505 us.)
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool two_loaders(const Ctx<D, SRC, FEW> &c, const Block &b) {
    return FEW && SRC == kPage16 && b.tiles() >= (b.twin ? 4 : 64);
}

// Warp 8 with TMA.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ void tma_warp(const Ctx<D, SRC, FEW> &c, const CUtensorMap *mk, const CUtensorMap *mv, const CUtensorMap *mq) {
    int fill = 0;
    for (int n = 0;; n++) {
        Block *b = c.item(n);
        if (!b || !tma_item(c, mk, mv, mq, b, n, fill, two_loaders(c, *b) ? kKeys : kBoth)) return;
        fill += 2 * b->tiles();
        c.leave(n);
    }
}

// Warps 10 and 11 for one item of a bf16 cache, ahead of its copies: whether the slots
// that some row does not see, up to the end of the last tile as the copies bring it, hold
// NaN or infinite values of V.  Read from global memory: the copies then find them in L2, and
// shared memory, whose bandwidth the products take, is left alone.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ void scan(const Ctx<D, SRC, FEW> &c, Block *b, int step) {
    constexpr int BN = Cfg<D, SRC, FEW>::BN, CH = D / 8, BATCH = 8;
    const Geometry &geo = c.p.geo;
    const int tid = threadIdx.x - 10 * 32;
    const Partial part(c.p, *b);
    const int len = b->len;
    const int seen = min(part.cnt[0] > 0 ? part.first[0] : 0x7fffffff, part.cnt[1] > 0 ? part.first[1] : 0x7fffffff);
    const bool paged = c.paged();
    const int box = paged ? min(1 << geo.block_shift, BN) : BN;
    const Span span = unseen_span(b->beg, b->tiles(), BN, seen, paged ? (int64_t)((len + box - 1) & -box) : geo.total - b->lo);
    const int chunks = span.count * CH;  // counted from the span's start: a row may have 2^31 of them
#pragma unroll 1
    for (int e0 = tid; e0 < chunks; e0 += step * BATCH) {
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            const int e = e0 + step * k;
            const int64_t rec = e < chunks ? record(geo, *b, span.start + e / CH) : -1;
            if (rec >= 0) any |= special_bits(*reinterpret_cast<const uint4 *>(c.p.V + (rec * CH + e % CH) * 16));
        }
        if (any & 0x80008000u) b->mend = 1u;
    }
}

// Warps 10 and 11 for one item of a bf16 cache: V tiles seen in part get zeros behind
// the row and their special values taken out, then pass on to full[stage].
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool mend(const Ctx<D, SRC, FEW> &c, Block *b, int *bad, int fill, int step, int *syncs) {
    using C = Cfg<D, SRC, FEW>;
    constexpr int BN = C::BN, CH = D / 8;
    const int tid = threadIdx.x - 10 * 32;
    const int tiles = b->tiles(), len = b->len, beg = b->beg;
    const Partial part(c.p, *b);
    uint32_t phase = c.misc->land;  // the last item's warps have left it (sync_helpers)
    for (int j = 0; j < tiles; j++) {
        if (!part.tile<BN>(j)) continue;
        const int f = fill + Fill<FEW>::of_v(j, tiles), st = f % C::kStages, key0 = (beg + j) * BN;
        if (!c.wait(c.sh->land + st, phase >> st)) return false;
        phase ^= 1u << st;
        unsigned char *at = c.stage(f);
        const auto chunk = [&](int e) { return reinterpret_cast<uint4 *>(at + tile_at(e / CH, e % CH, C::kSubK)); };
        // Only slots that some row does not see, eight chunks of a thread at once; behind the
        // row's end, zeros.
        constexpr int BATCH = 8;
        const int stop = min(BN, len - key0) * CH;
        for (int e0 = max(0, part.from(j) - key0) * CH + tid; e0 < stop; e0 += step * BATCH) {
            uint32_t any = 0;
#pragma unroll
            for (int k = 0; k < BATCH; k++)
                if (e0 + step * k < stop) any |= special_bits(*chunk(e0 + step * k));
            if (any & 0x80008000u) {
#pragma unroll 1
                for (int e = e0; e < min(stop, e0 + step * BATCH); e += step)
                    if (has_special(*chunk(e))) *chunk(e) = take_out<D>(*chunk(e), 8 * (e % CH), key0 + e / CH, bad, b);
            }
        }
        for (int e = stop + tid; e < BN * CH; e += step) *chunk(e) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
        if (step > 32 && !c.sync_helpers(syncs)) return false;
        if (tid == 0) mbar_arrive(c.sh->full + st);
    }
    if (tid == 0) c.misc->land = phase;
    return true;
}

// Warps 10 and 11 for one item of an fp8 cache: every tile from the raw ring to fp16.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool widen(const Ctx<D, SRC, FEW> &c, Block *b, int *bad, int fill) {
    using C = Cfg<D, SRC, FEW>;
    constexpr int BN = C::BN, CH = D / 16, RAWS = C::kRaws > 0 ? C::kRaws : 1;
    const int tid = threadIdx.x - 10 * 32;
    const int tiles = b->tiles(), len = b->len, beg = b->beg;
    const Partial part(c.p, *b);
    for (int g = 0; g < 2 * tiles; g++) {
        const Fill<FEW> what(g, tiles);
        const int f = fill + g, raw = f % RAWS, st = f % C::kStages, key0 = (beg + what.tile) * BN;
        if (!c.wait(c.sh->raw_full + raw, f / RAWS)) return false;
        if (f >= C::kStages && !c.wait(c.sh->empty + st, f / C::kStages - 1)) return false;
        const bool check = what.v && part.tile<BN>(what.tile);
        const unsigned char *from = c.sm + C::kSmRaw + raw * C::kRawBytes;
        unsigned char *to = c.stage(f);
        constexpr int BATCH = 8;
#pragma unroll 1
        for (int e0 = tid; e0 < BN * CH; e0 += 64 * BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; k++) v[k] = *reinterpret_cast<const uint4 *>(from + 16 * (e0 + 64 * k));
            if (check) {
#pragma unroll
                for (int k = 0; k < BATCH; k++) {
                    const int e = e0 + 64 * k, j = key0 + e / CH;
                    if (j >= len) v[k] = make_uint4(0u, 0u, 0u, 0u);
                    else if (has_nan8(v[k])) v[k] = take_out8(v[k], 16 * (e % CH), j, bad, b);
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; k++) {
                const int e = e0 + 64 * k;
                widen16(v[k], to, e / CH, e % CH, C::kSubK);
            }
        }
        fence_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            mbar_arrive(c.sh->full + st);
            mbar_arrive(c.sh->raw_empty + raw);
        }
    }
    return true;
}

// Warps 8, 10 and 11 for one item, record by record: what TMA does not bring.  bf16
// records are copied asynchronously, kLag fills in flight before the oldest is handed over.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool copy(const Ctx<D, SRC, FEW> &c, Block *b, int *bad, int fill) {
    using C = Cfg<D, SRC, FEW>;
    constexpr int ELEM = SRC == kCopy8 ? 1 : 2;
    constexpr int BN = C::BN, CH = D * ELEM / 16, ALL = BN * CH;  // 16-byte chunks per record, per tile
    constexpr int kLag = 2;
    const PrefillParams &p = c.p;
    const Geometry &geo = p.geo;
    const int tid = threadIdx.x < 288 ? threadIdx.x - 256 : threadIdx.x - 288;
    const int tiles = b->tiles(), len = b->len, beg = b->beg;
    const Partial part(p, *b);
    const auto hand_over = [&](int g) {  // fill g of the item; its V may need special values taken out first
        const Fill<FEW> what(g, tiles);
        if (ELEM == 2 && what.v && part.tile<BN>(what.tile))
            for (int e = tid; e < ALL; e += C::kLoaders) {
                uint4 *at = reinterpret_cast<uint4 *>(c.stage(fill + g) + tile_at(e / CH, e % CH, C::kSubK));
                if (has_special(*at)) *at = take_out<D>(*at, 8 * (e % CH), (beg + what.tile) * BN + e / CH, bad, b);
            }
        fence_async_smem();
        mbar_arrive(c.sh->full + (fill + g) % C::kStages);
    };
    bool ok = true;
    for (int g = 0; g < 2 * tiles; g++) {
        const int f = fill + g;
        if (f >= C::kStages && !c.wait(c.sh->empty + f % C::kStages, f / C::kStages - 1)) { ok = false; break; }
        const Fill<FEW> what(g, tiles);
        const char *src = what.v ? p.V : p.K;
        const int key0 = (beg + what.tile) * BN;
        const bool check = what.v && part.tile<BN>(what.tile);
#pragma unroll 2
        for (int e = tid; e < ALL; e += C::kLoaders) {
            const int row = e / CH, ch = e % CH, j = key0 + row;
            const int64_t rec = j < len ? record(geo, *b, j) : -1;
            if (rec < 0 && j < len) {
                b->any_missing = 1u;
                atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
            }
            if (ELEM == 2) {
                cp16(smem_u32(c.stage(f) + tile_at(row, ch, C::kSubK)), src + (rec < 0 ? 0 : rec) * (2 * D) + 16 * ch, rec >= 0);
            } else {
                uint4 v = rec < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4 *>(src + rec * D + 16 * ch);
                if (check && has_nan8(v)) v = take_out8(v, 16 * ch, j, bad, b);
                widen16(v, c.stage(f), row, ch, C::kSubK);
            }
        }
        if (ELEM == 2) {
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (g >= kLag) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                hand_over(g - kLag);
            }
        } else {
            hand_over(g);
        }
    }
    if (ELEM == 2) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (ok)
            for (int g = max(0, 2 * tiles - kLag); g < 2 * tiles; g++) hand_over(g);
    }
    return ok;
}

// Warps 10 and 11 (and 8, where it copies): item after item.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ void fill_warps(const Ctx<D, SRC, FEW> &c, const CUtensorMap *mk, const CUtensorMap *mv) {
    const int warp = threadIdx.x >> 5;
    int fill = 0, claims = 0, alones = 0, syncs = 0;
    bool more = warp == 10 && next_item(c, 0, &claims);
    for (int n = 0;; n++) {
        // An item is claimed while the one before it runs, not earlier: blocks that are
        // still free should have it.
        if (!Cfg<D, SRC, FEW>::kTma && more) more = next_item(c, n + 1, &claims);
        Block *b = c.item(n);
        if (!b) return;
        int *bad = c.bad();
        bool ok;
        if (n > 0 && c.slots[(n - 1) % kSlots].any_bad) {  // the notes are the last item's until its epilogue is done
            if (!c.wait(c.sh->item_empty + (n - 1) % kSlots, (n - 1) / kSlots)) return;
            __syncwarp();
            for (int e = threadIdx.x & 31; e < 3 * D; e += 32) bad[e] = 0x7fffffff;
            if (!c.sync_helpers(&syncs)) return;
        }
        if constexpr (Cfg<D, SRC, FEW>::kTma) {
            const bool alone = two_loaders(c, *b);  // warp 10 scans and mends alone, warp 11 loads
            const int step = alone ? 32 : 64;
            if (!alone || warp == 10) scan(c, b, step);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(c.sh->scanned + n % kSlots);
            if (alone && warp == 11) {
                // Not before warp 8 has brought the item's first keys: this warp may be items ahead of
                // the ring, where the parity of a stage's barrier says nothing.
                ok = c.wait(&c.sh->keys_begun, alones++) && tma_item(c, mk, mv, mv, b, n, fill, kValues);
            } else {
                ok = c.wait(c.sh->scanned + n % kSlots, n / kSlots);
                if (ok && b->mend) ok = mend(c, b, bad, fill, step, &syncs);
            }
            if (ok && more) {
                if (n > 0) ok = c.wait(c.sh->item_empty + (n - 1) % kSlots, (n - 1) / kSlots);
                more = ok && next_item(c, n + 1, &claims);
            }
        } else if constexpr (SRC == kTma8) {
            ok = widen(c, b, bad, fill);
        } else {
            ok = copy(c, b, bad, fill);
        }
        if (!ok) return;
        fill += 2 * b->tiles();
        if (!c.sync_helpers(&syncs)) return;  // any_bad is final
        c.leave(n);
    }
}

// ------------------------------------------------------------------- products

template <class C, int D>
__device__ __forceinline__ void issue_qk(uint32_t q, uint32_t k, uint32_t d) {
    const uint64_t qd = smem_desc(q, 16, 1024), kd = smem_desc(k, 16, 1024);
#pragma unroll
    for (int i = 0; i < D / 16; i++)
        mma_ss(d, qd + (((i >> 2) * C::kSubQ + (i & 3) * 32) >> 4), kd + (((i >> 2) * C::kSubK + (i & 3) * 32) >> 4),
               idesc(kRows, C::BN, 0, !C::kF16), i > 0);
}
// The product with V over one half of a tile's keys.
template <class C, int D, int HALF>
__device__ __forceinline__ void issue_pv(uint32_t p, uint32_t v, uint32_t d, bool acc) {
    const uint64_t vd = smem_desc(v, C::kSubK, 1024);
    constexpr int K = C::BN / 32;
#pragma unroll
    for (int i = HALF * K; i < (HALF + 1) * K; i++)
        mma_ts(d, p + 8 * i, vd + i * (2048 >> 4), idesc(kRows, D, 1, !C::kF16), acc || i > 0);
}

template <int D, int SRC, bool FEW>
__device__ __forceinline__ void issuer(const Ctx<D, SRC, FEW> &c) {
    using C = Cfg<D, SRC, FEW>;
    const uint32_t q = smem_u32(c.sm), tmem = c.tmem;
    const auto have = [&](int f) {
        const bool ok = c.wait(c.sh->full + f % C::kStages, f / C::kStages);
        fence_after();
        return ok;
    };
    const auto at = [&](int f) { return smem_u32(c.stage(f)); };
    const auto release = [&](int f) { mma_commit(c.sh->empty + f % C::kStages); };
    int fill = 0;
    int done[2] = {0, 0};  // key tiles of query tile t in the items before
    int outs[2] = {0, 0};  // items before in which query tile t had any
    for (int n = 0;; n++) {
        const Block *b = c.item(n);
        if (!b) return;
        const int cnt[2] = {b->cnt[0], b->cnt[1]};
        const int tiles = b->tiles();
        const bool twin = C::kTwins && b->twin;
        c.leave(n);
        if (!c.wait(&c.sh->q_full, n)) return;
        if (tiles == 0) {
            if (elect_one()) mbar_arrive(&c.sh->q_empty);
            __syncwarp();
            continue;
        }
        if (!have(fill)) return;
        if (twin) {
            // key tile j for query tile j & 1; the query rows are those of tile 0
            for (int j = 0; j < min(2, tiles); j++) {
                const int fk = fill + Fill<FEW>::of_k(j);
                if (!have(fk)) return;
                if (elect_one()) {
                    issue_qk<C, D>(q, at(fk), tmem + C::kTmemS(j));
                    mma_commit(c.sh->s_full + j);
                    release(fk);
                    if (j + 1 == tiles) mma_commit(&c.sh->q_empty);
                }
                __syncwarp();
            }
            for (int j = 0; j < tiles; j++) {
                const int t = j & 1, fv = fill + Fill<FEW>::of_v(j, tiles), fk = fill + Fill<FEW>::of_k(j + 2);
                const int before = t ? done[1] : done[0], used = t ? outs[1] : outs[0];
                if (!have(fv)) return;
                if (j < 2 && used > 0 && !c.wait(c.sh->o_free + t, used - 1)) return;
                if (!c.wait(c.sh->p_half + t, before + (j >> 1))) return;
                fence_after();
                if (elect_one()) issue_pv<C, D, 0>(tmem + C::kTmemS(t), at(fv), tmem + C::kTmemO(t), j > 1);
                __syncwarp();
                if (!c.wait(c.sh->p_full + t, before + (j >> 1))) return;
                fence_after();
                if (elect_one()) {
                    issue_pv<C, D, 1>(tmem + C::kTmemS(t), at(fv), tmem + C::kTmemO(t), true);
                    if (j + 2 >= tiles) mma_commit(c.sh->o_done + t);
                    release(fv);
                }
                __syncwarp();
                if (j + 2 < tiles) {
                    if (!have(fk)) return;
                    if (elect_one()) {
                        issue_qk<C, D>(q, at(fk), tmem + C::kTmemS(t));
                        mma_commit(c.sh->s_full + t);
                        release(fk);
                        if (j + 3 == tiles) mma_commit(&c.sh->q_empty);
                    }
                    __syncwarp();
                }
            }
        } else if (C::NT == 2) {
            if (elect_one()) {
#pragma unroll 1
                for (int t = 0; t < 2; t++)
                    if ((t ? cnt[1] : cnt[0]) > 0) {
                        issue_qk<C, D>(q + t * C::kQBytes, at(fill), tmem + C::kTmemS(t));
                        mma_commit(c.sh->s_full + t);
                    }
                release(fill);
                if (tiles == 1) mma_commit(&c.sh->q_empty);
            }
            __syncwarp();
            for (int j = 0; j < tiles; j++) {
                const int fv = fill + Fill<FEW>::of_v(j, tiles), fk = fill + Fill<FEW>::of_k(j + 1);
                bool v = false, k = false;  // V of tile j, K of tile j + 1 have landed
#pragma unroll 1
                for (int t = 0; t < 2; t++) {
                    const int mine = t ? cnt[1] : cnt[0], before = t ? done[1] : done[0], used = t ? outs[1] : outs[0];
                    if (j >= mine) continue;
                    const bool more = j + 1 < mine;
                    if (!v && !have(fv)) return;
                    v = true;
                    if (more && !k) {
                        if (!have(fk)) return;
                        k = true;
                    }
                    // the epilogue before has read this tile's O
                    if (j == 0 && used > 0 && !c.wait(c.sh->o_free + t, used - 1)) return;
                    if (!c.wait(c.sh->p_half + t, before + j)) return;
                    fence_after();
                    if (elect_one()) issue_pv<C, D, 0>(tmem + C::kTmemS(t), at(fv), tmem + C::kTmemO(t), j > 0);
                    __syncwarp();
                    if (!c.wait(c.sh->p_full + t, before + j)) return;
                    fence_after();
                    if (elect_one()) {
                        issue_pv<C, D, 1>(tmem + C::kTmemS(t), at(fv), tmem + C::kTmemO(t), true);
                        if (!more) mma_commit(c.sh->o_done + t);
                        if (t == 1 || j >= cnt[1]) release(fv);  // the last query tile that takes V
                        if (more) {
                            issue_qk<C, D>(q + t * C::kQBytes, at(fk), tmem + C::kTmemS(t));
                            mma_commit(c.sh->s_full + t);
                            if (t == 1 || j + 1 >= cnt[1]) {
                                release(fk);
                                if (j + 2 == tiles) mma_commit(&c.sh->q_empty);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        } else {
            int at_tile = done[0];  // S buffer and phase go by the tiles of all items
            if (elect_one()) {
                issue_qk<C, D>(q, at(fill), tmem + C::kTmemS(at_tile & 1));
                mma_commit(c.sh->s_full + (at_tile & 1));
                release(fill);
                if (tiles == 1) mma_commit(&c.sh->q_empty);
            }
            __syncwarp();
            for (int j = 0; j < tiles; j++, at_tile++) {
                const int fv = fill + Fill<FEW>::of_v(j, tiles), fk = fill + Fill<FEW>::of_k(j + 1), sb = at_tile & 1;
                if (j + 1 < tiles) {
                    if (!have(fk)) return;
                    if (elect_one()) {
                        issue_qk<C, D>(q, at(fk), tmem + C::kTmemS(sb ^ 1));
                        mma_commit(c.sh->s_full + (sb ^ 1));
                        release(fk);
                        if (j + 2 == tiles) mma_commit(&c.sh->q_empty);
                    }
                    __syncwarp();
                }
                if (!have(fv)) return;
                if (j == 0 && outs[0] > 0 && !c.wait(c.sh->o_free, outs[0] - 1)) return;
                if (!c.wait(c.sh->p_half + sb, at_tile >> 1)) return;
                fence_after();
                if (elect_one()) issue_pv<C, D, 0>(tmem + C::kTmemS(sb), at(fv), tmem + C::kTmemO(0), j > 0);
                __syncwarp();
                if (!c.wait(c.sh->p_full + sb, at_tile >> 1)) return;
                fence_after();
                if (elect_one()) {
                    issue_pv<C, D, 1>(tmem + C::kTmemS(sb), at(fv), tmem + C::kTmemO(0), true);
                    release(fv);
                    mma_commit(c.sh->o_done + sb);
                }
                __syncwarp();
            }
        }
        fill += 2 * tiles;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            done[t] += cnt[t];
            outs[t] += cnt[t] > 0;
        }
    }
}

// -------------------------------------------------------------------- softmax

// 32 bytes to global memory: one store where the address is a multiple of 32.
__device__ __forceinline__ void st32(char *to, const uint32_t *w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(to + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Rows of a part: O [kRowsPer][D] fp32, then (m, sum) [kRowsPer].
template <class C, int D>
__device__ __forceinline__ float *part_of(const PrefillParams &p, int64_t place) {
    return p.part + place * (C::kRowsPer * (D + 2));
}

// One item's softmax of query tile t.  `before`: key tiles of this query tile in the
// items before, `outs`: items with any.
template <int D, int SRC, bool FEW>
__device__ __forceinline__ bool softmax(const Ctx<D, SRC, FEW> &c, const Block &b, const int *bad, int t, int n, int before, int outs,
                                        int *twins) {
    using C = Cfg<D, SRC, FEW>;
    constexpr int BN = C::BN;
    const PrefillParams &p = c.p;
    const Geometry &geo = p.geo;
    const int tid = threadIdx.x & 127, lane = tid & 31;
    const bool twin = C::kTwins && b.twin;
    const int base = b.row0 + (twin ? 0 : t * kRows);  // first row of the tile
    const int x = base + tid;
    float scale = p.scale_log2;
    if (C::kF16) {
        // The thread's own row as fp16, scaled by a power of two: one pass for the largest
        // magnitude, one to convert.  TMA has brought the tile to where the result goes, or the row
        // is read from global memory.
        constexpr int CH = D / 8, BATCH = 8;
        const uint4 *row = reinterpret_cast<const uint4 *>(p.q + row_of(p, b, min(x, b.rows - 1)) * D);
        const auto here = [&](int k) { return reinterpret_cast<uint4 *>(c.sm + t * C::kQBytes + tile_at(tid, k, C::kSubQ)); };
        if (p.q_tma ? !c.wait(&c.sh->q_land, n) : n > 0 && !c.wait(&c.sh->q_empty, n - 1)) return false;
        uint32_t top = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < CH; k0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; k++) v[k] = p.q_tma ? *here(k0 + k) : row[k0 + k];
#pragma unroll
            for (int k = 0; k < BATCH; k++)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                             __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
        }
        // exponent field of the largest; up is 2^(127 + 14 - field) in two factors that never overflow
        const int field = (int)(max(top & 0xffffu, top >> 16) >> 7);
        const bool plain = field == 0 || field == 255;  // nothing but zeros and subnormals, or NaN and infinity
        const int up = plain ? 0 : 141 - field;
        const float f1 = __uint_as_float((uint32_t)(127 + up / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
        scale = scale / f1 / f2;
#pragma unroll 1
        for (int k0 = 0; k0 < CH; k0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; k++) v[k] = p.q_tma ? *here(k0 + k) : row[k0 + k];
#pragma unroll
            for (int k = 0; k < BATCH; k++) {
                const auto two = [&](uint32_t w) { return f16x2(bf16lo(w) * f1 * f2, bf16hi(w) * f1 * f2); };
                *here(k0 + k) = make_uint4(two(v[k].x), two(v[k].y), two(v[k].z), two(v[k].w));
            }
        }
        fence_async_smem();
        mbar_arrive(&c.sh->q_full);
    } else if (!p.q_tma) {
        // The query tile: 16-byte chunks, rows behind the sequence's last as zeros; a thread's
        // loads are all issued before the first is stored.
        constexpr int CH = D / 8, PER = kRows * CH / 128, BATCH = PER < 16 ? PER : 16;
        if (n > 0 && !c.wait(&c.sh->q_empty, n - 1)) return false;
#pragma unroll 1
        for (int k0 = 0; k0 < PER; k0 += BATCH) {
            uint4 v[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; k++) {
                const int e = tid + 128 * (k0 + k), x = base + e / CH;
                v[k] = x < b.rows ? *reinterpret_cast<const uint4 *>(p.q + row_of(p, b, x) * D + 8 * (e % CH))
                                  : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < BATCH; k++) {
                const int e = tid + 128 * (k0 + k);
                *reinterpret_cast<uint4 *>(c.sm + t * C::kQBytes + tile_at(e / CH, e % CH, C::kSubQ)) = v[k];
            }
        }
        fence_async_smem();
        mbar_arrive(&c.sh->q_full);
    }

    // rows behind the last see what the last does; they are not written
    const int limit = last_seen(p, b, min(x, b.rows - 1));
    const int first = last_seen(p, b, base);  // no row of the tile sees less
    const int cnt = b.cnt[t], beg = b.beg + (twin ? t : 0), step = twin ? 2 : 1;
    const uint32_t my = c.tmem + ((uint32_t)(tid & ~31) << 16);
    // (The wait for s_full covers every product issued before it: with one query tile, P V of
    // tile j - 2, so of the two o_done barriers none is more than a phase behind its wait.)
    float m = -INFINITY, sum = 0.f;  // m in units of log2, kLift below a maximum: subtracted from scaled scores
    for (int j = 0; j < cnt; j++) {
        const int at = before + j;
        const int sb = C::NT == 2 ? t : at & 1;
        if (!c.wait(c.sh->s_full + sb, C::NT == 2 ? at : at >> 1)) return false;
        fence_after();
        const int key0 = (beg + j * step) * BN;
        // (the loading warps, tiles ahead, may be setting it: the lanes' readings are made one)
        const bool missing = SRC != kTma16 && __any_sync(0xffffffffu, b.any_missing);
        if (key0 + BN - 1 > first || missing) {
            // Some row sees the tile only in part, or slots have no block: minus infinity goes to
            // their columns in tensor memory.  (A rolled loop: this code runs once or twice per
            // item, and fetching 128 unrolled selections took longer than running them.)
#pragma unroll 1
            for (int q = 0; q < BN / 32; q++) {
                uint32_t e[32];
                tmem_ld32(my + C::kTmemS(sb) + 32 * q, e);
                const int jj = key0 + 32 * q, seen = limit + 1 - jj;
                uint32_t bits = seen >= 32 ? 0xffffffffu : seen <= 0 ? 0u : (1u << seen) - 1u;
                if (missing) bits &= ~__ballot_sync(0xffffffffu, jj + lane < b.len && record(geo, b, jj + lane) < 0);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k++)
                    if (!(bits >> k & 1)) e[k] = 0xff800000u;
                tmem_st32(my + C::kTmemS(sb) + 32 * q, e);
            }
            wait_st();
        }
        // The upper half of the keys, then the lower one, which stays in registers for the
        // weights; the upper half is read again after them.  (The weights' code is a loop of
        // two turns: unrolled over all keys it outgrew the instruction cache beside the other
        // warps' code, and a tenth of the warps' time went into fetching.)
        constexpr int HALF = BN / 2;
        uint32_t s[HALF];
        float mx[4];
#pragma unroll
        for (int h = 1; h >= 0; h--) {
#pragma unroll
            for (int k = 0; k < HALF; k += 32) tmem_ld32(my + C::kTmemS(sb) + HALF * h + k, s + k);
            wait_ld();
#pragma unroll
            for (int k = 0; k < HALF; k += 8)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const float u = __uint_as_float(s[k + 2 * q]), v = __uint_as_float(s[k + 2 * q + 1]);
                    mx[q] = h == 1 && k == 0 ? max2(u, v) : max3(mx[q], u, v);
                }
        }
        float top = max2(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
        if (top == INFINITY) top = NAN;  // inf - inf, as the definition has it
        // raise the maximum: always from nothing, else once the weights pass 2^(kLift + kRaise)
        if (__any_sync(0xffffffffu, !(top <= m + (C::kLift + C::kRaise)))) {
            const float mn = top <= m + (C::kLift + C::kRaise) ? m : top - C::kLift;
            if (j > 0) {
                if (C::NT == 1 && !c.wait(c.sh->o_done + ((at - 1) & 1), (at - 1) >> 1)) return false;
                fence_after();
                const float f = mn == m ? 1.f : m == -INFINITY ? 0.f : ex2(m - mn);
#pragma unroll 1
                for (int k = 0; k < D / 32; k++) {
                    uint32_t o[32];
                    tmem_ld32(my + C::kTmemO(t) + 32 * k, o);
                    wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st32(my + C::kTmemO(t) + 32 * k, o);
                }
                sum *= f;
            }
            m = mn;
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const f32x2 scale2 = both(scale), off2 = both(off);
        f32x2 part_sum[2] = {0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; h++) {
            uint32_t pk[HALF / 2];
#pragma unroll
            for (int k = 0; k < HALF / 2; k++) {
                const f32x2 e = fma2(pack2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), scale2, off2);
                float a, d;
                unpack2(e, a, d);
                a = ex2(a);
                d = ex2(d);
                part_sum[k & 1] = add2(part_sum[k & 1], pack2(a, d));
                pk[k] = C::kF16 ? f16x2(a, d) : bf16x2(a, d);
            }
            // P of the lower half lies over S of the lower quarter, P of the upper half over the
            // rest of the lower half: S of the upper half stays until it is read
            if (HALF == 64) tmem_st32(my + C::kTmemS(sb) + 32 * h, pk);
            else tmem_st16(my + C::kTmemS(sb) + 16 * h, pk);
            if (h == 0) {
#pragma unroll
                for (int k = 0; k < HALF; k += 32) tmem_ld32(my + C::kTmemS(sb) + HALF + k, s + k);
            }
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive((h == 0 ? c.sh->p_half : c.sh->p_full) + sb);
            if (h == 0) wait_ld();
        }
        float s0, s1;
        unpack2(add2(part_sum[0], part_sum[1]), s0, s1);
        sum += s0 + s1;
    }
    // ---- epilogue
    if (cnt > 0) {
        const int at = before + cnt - 1;
        if (!c.wait(c.sh->o_done + (C::NT == 2 ? t : at & 1), C::NT == 2 ? outs : at >> 1)) return false;
        fence_after();
    }
    // A twin item: the second warpgroup leaves its statistics and its O to the first.
    float f0 = 1.f, f1 = 0.f;  // what O of query tile t, and of the twin, is worth
    const bool join = twin && b.cnt[1] > 0;
    if (join) {
        float2 *notes = reinterpret_cast<float2 *>(c.sm + C::kSmTwin) + tid;
        if (t == 1) {
            *notes = make_float2(m, sum);
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.sh->twin_done);
            return true;
        }
        if (!c.wait(&c.sh->twin_done, (*twins)++)) return false;
        fence_after();
        const float2 o = *notes;
        const float mn = max2(m, o.x);
        f0 = m == -INFINITY ? 0.f : ex2(m - mn);
        f1 = o.x == -INFINITY ? 0.f : ex2(o.x - mn);
        sum = sum * f0 + o.y * f1;
        m = mn;
    } else if (twin && t == 1) {
        return true;
    }
    const bool nothing = sum == 0.f;
    const bool parts = p.splits > 1;
    const float inv = parts ? 1.f : nothing ? 0.f : 1.f / sum;
    f0 *= inv;
    f1 *= inv;
    if (parts) {
        float *ml = part_of<C, D>(p, b.place) + C::kRowsPer * D + 2 * (x - b.row0);
        ml[0] = nothing ? -INFINITY : m;
        ml[1] = sum;
    } else if (p.lse && x < b.rows) {
        p.lse[row_of(p, b, x)] = nothing ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
    }
    // Each thread writes its own row, 32 bytes (a sector) at a time where the row allows:
    // going through shared memory for whole lines was slower beside the other tile's products.
    char *to = parts ? (char *)(part_of<C, D>(p, b.place) + (x - b.row0) * D)
                     : (char *)(p.out + row_of(p, b, min(x, b.rows - 1)) * D);
    const bool wide = ((uintptr_t)(parts ? (const void *)p.part : (const void *)p.out) & 31) == 0;
    const bool fix = b.any_bad && cnt > 0;
#pragma unroll 1
    for (int k0 = 0; k0 < D; k0 += 32) {
        uint32_t o[32];
        if (cnt > 0) {
            tmem_ld32(my + C::kTmemO(t) + k0, o);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
            if (join) {
                uint32_t o1[32];
                tmem_ld32(my + C::kTmemO(1) + k0, o1);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
            }
            if (k0 == D - 32) {  // O is free for the next item
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c.sh->o_free + t);
                    if (join) mbar_arrive(c.sh->o_free + 1);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] = 0u;
        }
        if (fix) {
            const int *at = bad + k0;
#pragma unroll
            for (int k = 0; k < 32; k++) {
                if (at[D + k] <= limit) o[k] = __float_as_uint(__uint_as_float(o[k]) + INFINITY);
                if (at[2 * D + k] <= limit) o[k] = __float_as_uint(__uint_as_float(o[k]) - INFINITY);
                if (at[k] <= limit) o[k] = 0x7fc00000u;
            }
        }
        if (parts) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st32(to + (k0 + e) * 4, o + e, wide);
        } else if (x < b.rows) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e++)
                w[e] = bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            st32(to + k0 * 2, w, wide);
            st32(to + k0 * 2 + 32, w + 8, wide);
        }
        __syncwarp();
    }
    return true;
}

// -------------------------------------------------------------------- kernels

template <int D, int SRC, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mq) {
    using C = Cfg<D, SRC, FEW>;
    using Sh = typename Ctx<D, SRC, FEW>::Sh;
    extern __shared__ unsigned char smraw[];
    __shared__ Sh sh;
    __shared__ Block slots[kSlots];
    __shared__ Misc misc;
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5;
    constexpr bool COPY = SRC >= kCopy16;
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&misc.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 8 * 32 && !COPY) {  // the copies' descriptors, before the first needs them
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mv)) : "memory");
        if (p.q_tma) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mq)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; i++) {
            mbar_init(sh.full + i, COPY ? C::kLoaders : SRC == kTma8 ? 2 : 1);
            mbar_init(sh.empty + i, 1);
            mbar_init(sh.land + i, 1);
        }
        for (int i = 0; i <= C::kStages; i++) sh.in_flight[i] = 0xffffffffu;
        for (int i = 0; i <= C::kRaws; i++) {
            mbar_init(sh.raw_full + i, 1);
            mbar_init(sh.raw_empty + i, 2);
        }
        mbar_init(&sh.q_full, p.q_tma && !C::kF16 ? 1 : 128 * C::NT);
        mbar_init(&sh.q_land, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.claimed, 1);
        mbar_init(&sh.drain, 1);
        mbar_init(&sh.keys_begun, 1);
        mbar_init(&sh.twin_done, 4);
        mbar_init(&sh.helpers, Ctx<D, SRC, FEW>::kHelpers / 32);
        for (int i = 0; i < 2; i++) {
            mbar_init(sh.s_full + i, 1);
            mbar_init(sh.p_half + i, 4);
            mbar_init(sh.p_full + i, 4);
            mbar_init(sh.o_done + i, 1);
            mbar_init(sh.o_free + i, 4);
        }
        for (int i = 0; i < kSlots; i++) {
            mbar_init(sh.item_full + i, 1);
            mbar_init(sh.scanned + i, 2);
            mbar_init(sh.item_empty + i, 4 * C::NT + 4);  // the softmax warps and warps 8 to 11
        }
        mbar_init_fence();
        misc.abort_flag = misc.land = 0u;
    }
    for (int e = threadIdx.x; e < 3 * D; e += kThreads) reinterpret_cast<int *>(sm + C::kSmBad)[e] = 0x7fffffff;
    fence_before();
    __syncthreads();
    fence_after();
    grid_dependency_wait();
    const Ctx<D, SRC, FEW> c{p, sm, &sh, slots, &misc, misc.tmem};
    // Registers: 384 threads are launched with 168 each; 2 x 208 + 88 = 3 x 168.
    if (warp < 8) {
        regs_up<208>();
        const int t = warp >> 2;
        if (t < C::NT) {
            int before = 0, outs = 0, twins = 0;
            for (int n = 0;; n++) {
                Block *b = c.item(n);
                if (!b) break;
                if (!softmax(c, *b, c.bad(), t, n, before, outs, &twins)) break;
                before += b->cnt[t];
                outs += b->cnt[t] > 0;
                c.leave(n);
            }
        }
    } else {
        regs_down<88>();
        if (warp == 9) {
            issuer(c);
        } else if (warp == 8 && !COPY) {
            tma_warp(c, &mk, &mv, &mq);
        } else {
            fill_warps(c, &mk, &mv);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (misc.abort_flag) {  // after a wait ran out: what is still on its way ends before its memory is released
        if (warp == 9 && elect_one()) {
            mma_commit(&sh.drain);
            mbar_wait(&sh.drain, 0);
        }
        if (warp == 8) c.drain_copies();
        __syncwarp();
        __syncthreads();
    }
    fence_after();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(misc.tmem) : "memory");
    grid_dependents_launch();
}

// Merges the parts of a unit's rows: one warp per row,
//   out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k.
template <int D>
__global__ void __launch_bounds__(256) prefill_join(const __grid_constant__ PrefillParams p) {
    using C = Cfg<D, kTma16, false>;
    constexpr int PER = C::kRowsPer / 8;  // blocks of 8 rows per unit
    __shared__ Block blk;
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    const int unit = blockIdx.x / PER;
    const int r = (int)(blockIdx.x % PER) * 8 + warp;
    if (warp == 0) {
        const bool f = find_block<D, false>(p, unit, 0, &blk);
        if (lane == 0) found = f;
    }
    __syncthreads();
    const int x = blk.row0 + r;
    if (!found || x >= blk.rows) return;
    const auto part = [&](int k) { return part_of<C, D>(p, (int64_t)unit * p.splits + k); };
    const auto ml = [&](int k) { return part(k) + C::kRowsPer * D + 2 * r; };
    float m = -INFINITY;
    for (int k = 0; k < p.splits; k++) m = max2(m, ml(k)[0]);
    float sum = 0.f, o[D / 32] = {0.f};
    for (int k = 0; k < p.splits; k++) {
        const float mk = ml(k)[0];
        if (mk == -INFINITY) continue;
        const float w = exp2f(mk - m);
        sum = fmaf(w, ml(k)[1], sum);
#pragma unroll
        for (int e = 0; e < D / 32; e++) o[e] = fmaf(w, part(k)[r * D + lane + 32 * e], o[e]);
    }
    const int64_t row = row_of(p, blk, x);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < D / 32; e++) {
        const __nv_bfloat16 v = __float2bfloat16_rn(o[e] * inv);
        p.out[row * D + lane + 32 * e] = *reinterpret_cast<const uint16_t *>(&v);
    }
    if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Items per (layer, KV head): sum over sequences of ceil(n G / R), bounded from what the host knows.
inline int64_t most_blocks(int64_t S, int64_t G, int D, int64_t T) {
    const int64_t R = D == 256 ? kRows : 2 * kRows;
    return (T * G + std::min(S, T) * (R - 1)) / R;
}

constexpr int kMostParts = 160;  // parts of split rows the workspace holds: one per SM

// Splits of each row over its keys: as many as fill the SMs while a split keeps at least
// four key tiles of the average row.
inline int splits_of(int64_t units, int64_t keys, int D) {
    const int64_t tiles = keys / (D == 256 ? 64 : 128);
    return (int)std::max<int64_t>(
        1, std::min<int64_t>(std::min(sm_count(), kMostParts) / std::max<int64_t>(1, units), tiles / 4));
}

// The cache as boxes of up to BN slots: [total][d], or the pool's slots [L n_blocks bs][H][d] one
// head at a time.  bf16: 64 dims a box, 128-byte swizzled; fp8: all dims, as stored.
template <int D, int SRC, bool FEW>
bool make_map(CUtensorMap *m, const void *base, const Geometry &geo) {
    auto fn = tensormap_encode_fn();
    if (!fn) return false;
    constexpr int E = SRC == kTma8 ? 1 : 2;
    constexpr cuuint32_t dims = SRC == kTma8 ? D : 64;
    const bool paged = geo.layout == TRI_KV_PAGED;
    const int64_t slots = paged ? (int64_t)geo.L * geo.n_blocks << geo.block_shift : geo.total;
    const cuuint32_t box = (cuuint32_t)std::min<int64_t>(paged ? 1 << geo.block_shift : 256, Cfg<D, SRC, FEW>::BN);
    const cuuint64_t dims3[3] = {D, (cuuint64_t)geo.H, (cuuint64_t)slots}, dims2[2] = {D, (cuuint64_t)slots};
    const cuuint64_t str3[2] = {E * D, (cuuint64_t)geo.H * E * D}, str2[1] = {E * D};
    const cuuint32_t box3[3] = {dims, 1, box}, box2[2] = {dims, box}, ones[3] = {1, 1, 1};
    return fn(m, E == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, paged ? 3 : 2,
              const_cast<void *>(base), paged ? dims3 : dims2, paged ? str3 : str2, paged ? box3 : box2, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, E == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries [L T][Hq][d] as boxes of 64 dims x the G heads of a KV head x 128 / G tokens.
template <int D>
bool make_q_map(CUtensorMap *m, const PrefillParams &p) {
    auto fn = tensormap_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {D, (cuuint64_t)p.geo.Hq, (cuuint64_t)(p.geo.L * p.T)};
    const cuuint64_t str[2] = {2 * D, (cuuint64_t)p.geo.Hq * 2 * D};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.geo.G, (cuuint32_t)(kRows / p.geo.G)}, ones[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p.q), dims, str, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA wants slot numbers of 31 bits, and pages that fill a swizzle atom of 8 rows.
inline bool tma_fits(const Geometry &geo) {
    const int64_t most = 0x7fffffffLL;
    if (geo.layout == TRI_KV_PAGED) return geo.block_shift >= 3 && geo.n_blocks <= (most / geo.L >> geo.block_shift);
    return geo.total >= 1 && geo.total <= most;
}

template <int D, int SRC, bool FEW>
cudaError_t launch_t(PrefillParams p, int64_t units, cudaStream_t s) {
    using C = Cfg<D, SRC, FEW>;
    constexpr size_t smem = C::kSmMisc + 1024;
    static bool attr[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    auto kern = prefill_kernel<D, SRC, FEW>;
    if (!attr[dev & 63]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        attr[dev & 63] = true;
    }
    CUtensorMap mk = {}, mv = {}, mq = {};
    if (SRC < kCopy16 && (!make_map<D, SRC, FEW>(&mk, p.K, p.geo) || !make_map<D, SRC, FEW>(&mv, p.V, p.geo))) return cudaErrorInvalidValue;
    p.q_tma = SRC < kCopy16 && kRows % p.geo.G == 0 && p.geo.L * p.T <= 0x7fffffffLL;
    if (p.q_tma && !make_q_map<D>(&mq, p)) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(kern, dim3((unsigned)(units * p.splits)), dim3(kThreads), smem, s, p, mk, mv, mq);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_pdl(prefill_join<D>, dim3((unsigned)(units * C::kRowsPer / 8)), dim3(256), 0, s, p);
}

template <int D>
cudaError_t launch_d(const PrefillParams &p0, cudaStream_t s) {
    PrefillParams p = p0;
    const Geometry &geo = p.geo;
    const int64_t blocks = most_blocks(geo.S, geo.G, D, p.T), units = blocks * geo.L * geo.H;
    int l = 0;
    while ((1 << l) < geo.G) l++;
    p.div_shift = 31 + l;
    p.div_mul = ((1ull << (31 + l)) + geo.G - 1) / geo.G;
    if (units > 0x7fffffffLL / 64 || p.T * geo.G > 0x7fffff00LL) return cudaErrorInvalidConfiguration;
    p.splits = splits_of(units, geo.total / ((int64_t)geo.L * geo.S * geo.H), D);
    const bool paged = geo.layout == TRI_KV_PAGED;
    if (!tma_fits(geo))
        return geo.elem_bytes == 1 ? launch_t<D, kCopy8, false>(p, units, s) : launch_t<D, kCopy16, false>(p, units, s);
    // The code for few rows (twin items, keys ahead of values, two loaders) costs whole prompts 5 to
    // 8 percent, by its mere presence in the kernel: it has kernels of its own, for sequences of at most
    // one query tile on average.
    const bool few = D != 256 && p.T * geo.G <= kRows * std::min<int64_t>(geo.S, p.T);
    if (geo.elem_bytes == 1) return few ? launch_t<D, kTma8, D != 256>(p, units, s) : launch_t<D, kTma8, false>(p, units, s);
    if (paged) return few ? launch_t<D, kPage16, D != 256>(p, units, s) : launch_t<D, kPage16, false>(p, units, s);
    return few ? launch_t<D, kTma16, D != 256>(p, units, s) : launch_t<D, kTma16, false>(p, units, s);
}

}  // namespace
}  // namespace tri

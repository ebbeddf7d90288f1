// Causal attention of new tokens over the cache that ends with them (the step around
// "TriAttention：基于三角函数 KV 压缩的高效长推理", 流程详解 step 5): for each (layer l,
// token i of sequence s's n, query head g of KV head h), over slots j <= N - n + i of
// row (l, s, h),
//   s_j = scale * (q . k_j),  out = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}.
//
// 4 d flops per visible (query, key) pair: tensor-core bound for prompts, HBM bound
// (K and V read once) for a few tokens over a long row.  The G query heads of a KV
// head share its keys, so a block's rows are the (token, head) pairs of one KV head in
// token order: a prompt of n tokens is n * G rows, cut into blocks of up to 256.
//
// A block (one per SM, 12 warps) computes, for its two 128-row query tiles,
//   S = Q K^T  and  O += P V,  P = 2^(S scale log2(e) - m),
// on tcgen05.mma (kind::f16, bf16 operands, fp32 accumulators in tensor memory):
//   - warps 0-3 and 4-7: the softmax of query tile 0 and 1, one thread per row.  S is
//     read from tensor memory, P (bf16) written back over it as the A operand of P V.
//     While one tile's softmax runs, the other tile's products do.
//   - warps 8, 10, 11: bring K and V tiles (128 keys; 64 at head dim 256) into a ring in
//     shared memory, 128-byte swizzled.  bf16 caches: warp 8 issues TMA copies, one
//     box per 64 dims of a contiguous tile or of a block of pages, and warps 10 and 11
//     only touch V tiles that some row sees in part.  fp8 caches, and blocks too
//     small for a swizzle atom (8 slots): all three copy, fp8 widened to bf16 (exact).
//   - warp 9: issues every product.
// Head dim 256 fits one query tile (its O takes half of tensor memory); its S is
// double-buffered instead.
//
// The maximum m a row subtracts is only raised when its scores pass it by more than
// 2^8 (weights up to 256 lose nothing in bf16 or fp32), so O is rescaled rarely.
// Statistics and O are fp32; P's rounding to bf16 is the operands' common type.
//
// Keys a row must not see get weight exactly 0, but 0 * NaN is NaN in the product:
// rows of V outside the cache row are zero-filled, and in the tiles that some row sees
// only in part, NaN and infinite values of V are taken out and noted per dim; the
// epilogue gives them back to the rows that see them.
//
// When the blocks are fewer than the SMs, each row is split over its keys, and
// prefill_join merges the parts.  Every wait is bounded.
#include <algorithm>

#include <cuda_bf16.h>

#include "keys.cuh"
#include "stage.cuh"
#include "tensormap.cuh"

namespace tri {
namespace {

constexpr int kThreads = 384;
constexpr int kLoaders = 96;  // threads of warps 8, 10 and 11
constexpr int kRows = 128;  // rows of a query tile: one per thread of a softmax warpgroup
constexpr float kRaise = 8.f;  // log2 of the most a weight may pass 1 before the maximum is raised

template <int D>
struct Cfg {
    static constexpr int NT = D == 256 ? 1 : 2;     // query tiles per block
    static constexpr int BN = D == 256 ? 64 : 128;  // keys per tile
    static constexpr int kStageBytes = BN * D * 2;
    static constexpr int kStages = D == 64 ? 8 : D == 128 ? 5 : 4;
    static constexpr int kQBytes = kRows * D * 2;  // per query tile
    static constexpr int kSubQ = kRows * 128;      // a 64-dim column of a Q tile
    static constexpr int kSubK = BN * 128;         // ... of a K or V tile
    // tensor memory columns
    static constexpr int kTmemS(int b) { return b * BN; }  // S (and P) of tile b, or buffer b
    static constexpr int kTmemO(int t) { return 256 + t * D; }
    // shared memory from a 1024-byte aligned base
    static constexpr int kSmRing = NT * kQBytes;
    static constexpr int kSmBad = kSmRing + kStages * kStageBytes;  // int [3][D]
    static constexpr int kSmBar = kSmBad + 3 * D * 4;
    static constexpr int kBars = 3 * kStages + 1 + 2 + 2 + 2 + 1 + 2;
    static constexpr int kSmMisc = kSmBar + kBars * 8;
    static constexpr size_t kSmem = kSmMisc + 64 + 1024;
};

struct Misc {
    uint32_t tmem;
    volatile uint32_t abort_flag;
    volatile uint32_t any_bad;      // a NaN or infinite value of V was taken out
    volatile uint32_t any_missing;  // a slot without a block
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    // start, leading and stride byte offsets in 16-byte units, version 1, 128-byte swizzle
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16 instruction descriptor: fp32 accumulator, bf16 A and B, B K-major or MN-major.
constexpr uint32_t idesc(int M, int N, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
        : "memory");
}
// A from tensor memory (bf16 pairs per 32-bit column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// -------------------------------------------------------------------- waits

// Bounded wait of one role (the clock is read once in 4096 tries).  When it runs out
// the block is told to stop.
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, Misc *misc, unsigned *flags) {
    unsigned long long t0 = 0;
    for (uint32_t it = 1; it < kStageWaitIters; it++) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 4095u) == 0) {
            const unsigned long long t = global_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kStageWaitNs || misc->abort_flag) break;
        }
    }
    misc->abort_flag = 1u;
    atomicOr(flags, TRI_FLAG_STAGE_TIMEOUT);
    return false;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// ---------------------------------------------------------------- arithmetic

// Maxima that keep a NaN: a NaN score makes its row NaN, as the definition does.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two floats per register pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }

// 2^x of two values on the FMA pipe, which the softmax leaves idle while the
// special-function unit is its bound.  x = n + f with n the nearest integer (the
// low bits of x + 1.5 * 2^23) and f in [-1/2, 1/2]; 2^f as 1 + c1 f + .. + c4 f^4,
// the polynomial of least maximal relative error on that interval (2.8e-6, found
// by linear programming); n is added to its exponent.  x is held at -127, where the
// result is exactly 0; x <= kRaise always.
__device__ __forceinline__ void ex2_fma(f32x2 x, float &a, float &b) {
    float lo, hi;
    unpack2(x, lo, hi);
    x = pack2(fmaxf(lo, -127.f), fmaxf(hi, -127.f));
    const f32x2 r = add2(x, both(12582912.f));
    const f32x2 f = add2(x, fma2(r, both(-1.f), both(12582912.f)));
    f32x2 y = fma2(f, both(0.009582853876054287f), both(0.055906426161527634f));
    y = fma2(y, f, both(0.24024099111557007f));
    y = fma2(y, f, both(0.6931241750717163f));
    y = fma2(y, f, both(1.f));
    float r0, r1, y0, y1;
    unpack2(r, r0, r1);
    unpack2(y, y0, y1);
    a = __uint_as_float(__float_as_uint(y0) + (__float_as_uint(r0) << 23));
    b = __uint_as_float(__float_as_uint(y1) + (__float_as_uint(r1) << 23));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------ the work

struct Block {
    int l, h, seq;
    int n;         // new tokens of the sequence
    int rows;      // n * G
    int row0;      // first row of this block
    int len;       // N: slots of the cache row
    int64_t tok0;  // tok_off[seq]
    int64_t lo;    // row_off
    int beg;       // first key tile (of the split)
    int cnt[2];    // key tiles of each query tile, from beg
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
// ceil(n G / (128 NT)) blocks, the last rows (most keys) first.
template <int D>
__device__ __forceinline__ bool find_block(const PrefillParams &p, int idx, int split, Block *out) {
    constexpr int R = kRows * Cfg<D>::NT, BN = Cfg<D>::BN;
    const Geometry &geo = p.geo;
    const int lane = threadIdx.x & 31;
    const int lh = idx / p.blocks;
    int b = idx - lh * p.blocks;
    for (int base = 0; base < geo.S; base += 32) {
        const int s = base + lane;
        int64_t t0 = 0, n = 0;
        if (s < geo.S) {
            t0 = p.tok_off[s];
            n = p.tok_off[s + 1] - t0;
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
                Block w;
                w.l = lh / geo.H;
                w.h = lh - w.l * geo.H;
                w.seq = s;
                w.n = (int)n;
                w.rows = (int)(n * geo.G);
                w.row0 = (upto - 1 - b) * R;
                w.tok0 = t0;
                const int64_t r = ((int64_t)w.l * geo.S + s) * geo.H + w.h;
                int64_t lo = geo.row_off[r], hi = geo.row_off[r + 1];
                if (lo < 0 || hi < lo || hi > geo.total || hi - lo > 0x7fffff00LL) {
                    atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
                    hi = lo = 0;
                }
                w.lo = lo;
                w.len = (int)(hi - lo);
                int c[2] = {0, 0};
                for (int t = 0; t < Cfg<D>::NT; t++) {
                    const int first = w.row0 + t * kRows;
                    if (first < w.rows) c[t] = max(0, last_seen(p, w, min(first + kRows, w.rows) - 1) + BN) / BN;
                }
                const int all = max(c[0], c[1]);
                w.beg = p.splits == 1 ? 0 : (int)((int64_t)all * split / p.splits);
                const int end = p.splits == 1 ? all : (int)((int64_t)all * (split + 1) / p.splits);
                for (int t = 0; t < 2; t++) w.cnt[t] = max(0, min(c[t], end) - w.beg);
                *out = w;
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
__device__ __forceinline__ uint4 take_out(uint4 v, int d0, int j, int *bad, Misc *misc) {
    misc->any_bad = 1u;
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

// Eight e4m3 values (two words) as bf16.
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
    const float2 x = e4m3x2_to_float2(a), y = e4m3x2_to_float2(a >> 16), z = e4m3x2_to_float2(b), w = e4m3x2_to_float2(b >> 16);
    return make_uint4(bf16x2(x.x, x.y), bf16x2(y.x, y.y), bf16x2(z.x, z.y), bf16x2(w.x, w.y));
}

// Query tile t's first row sees this many slots: key tiles past them are seen in part.
struct Partial {
    int beg, cnt[2], first[2];
    __device__ __forceinline__ Partial(const PrefillParams &p, const Block &b) {
        beg = b.beg;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            cnt[t] = b.cnt[t];
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

// The TMA warp of a bf16 cache.  Fill 2j is K, fill 2j+1 V of key tile beg + j.  A V
// tile that is seen in part lands on land[stage], for the mending warps; every other
// fill on full[stage].
template <int D>
__device__ __forceinline__ void tma_loader(const PrefillParams &p, const Block &b, unsigned char *sm, const CUtensorMap *mk,
                                           const CUtensorMap *mv, uint64_t *full, uint64_t *empty, uint64_t *land,
                                           Misc *misc) {
    using C = Cfg<D>;
    constexpr int BN = C::BN;
    const Geometry &geo = p.geo;
    const int lane = threadIdx.x & 31;
    const int tiles = max(b.cnt[0], b.cnt[1]);
    const uint32_t ring = smem_u32(sm + C::kSmRing);
    const Partial part(p, b);
    const bool paged = geo.layout == TRI_KV_PAGED;
    const int64_t lo = b.lo;
    const int len = b.len, beg = b.beg, h = b.h;
    const int32_t *table = geo.block_table + (int64_t)b.seq * geo.max_blocks;
    const int box = paged ? min(1 << geo.block_shift, BN) : BN;  // slots per copy
    const int64_t layer = (int64_t)b.l * geo.n_blocks;
    for (int f = 0; f < 2 * tiles; f++) {
        const int st = f % C::kStages;
        const bool v = f & 1;
        const int key0 = (beg + (f >> 1)) * BN;
        // Slot of the pool the lane's copy starts at (looked up before the wait below).
        int64_t slot = -1;
        const int j = key0 + lane * box;
        const bool mine = lane * box < BN && j < len;
        if (paged && mine) {
            const int bi = j >> geo.block_shift;
            const int32_t blk = bi < geo.max_blocks ? __ldg(table + bi) : -1;
            if (blk >= 0 && blk < geo.n_blocks)
                slot = ((layer + blk) << geo.block_shift) + (j & ((1 << geo.block_shift) - 1));
        } else if (mine) {
            slot = lo + j;
        }
        if (f >= C::kStages && !role_wait(empty + st, ((f / C::kStages) - 1) & 1, misc, p.flags)) break;
        uint64_t *bar = v && part.tile<BN>(f >> 1) ? land + st : full + st;
        const uint32_t dst = ring + st * C::kStageBytes;
        const uint32_t here = __ballot_sync(0xffffffffu, slot >= 0);
        if (here != __ballot_sync(0xffffffffu, mine)) {  // blocks that the table does not name
            misc->any_missing = 1u;
            if (mine && slot < 0) {
                atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
                if (v)  // no weight reaches their keys; their values must be finite
                    for (int x = 0; x < D / 64; x++)
                        for (int e = 0; e < box * 8; e++)
                            *reinterpret_cast<uint4 *>(sm + C::kSmRing + st * C::kStageBytes + x * C::kSubK +
                                                       lane * box * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(__popc(here) * box * D * 2));
        __syncwarp();
        if (slot >= 0) {
            const CUtensorMap *map = v ? mv : mk;
#pragma unroll
            for (int x = 0; x < D / 64; x++) {
                const uint32_t at = dst + x * C::kSubK + lane * box * 128;
                if (paged) tma3(at, map, 64 * x, h, (int)slot, bar);
                else tma2(at, map, 64 * x, (int)slot, bar);
            }
        }
    }
}

// Warps 10 and 11 beside the TMA warp: V tiles seen in part get zeros behind the row and
// their special values taken out, then pass on to full[stage].
template <int D>
__device__ __forceinline__ void mender(const PrefillParams &p, const Block &b, unsigned char *sm, uint64_t *full,
                                       uint64_t *land, int *bad, Misc *misc) {
    using C = Cfg<D>;
    constexpr int BN = C::BN, CH = D / 8;
    const int tid = threadIdx.x - 10 * 32;
    const int tiles = max(b.cnt[0], b.cnt[1]);
    const Partial part(p, b);
    uint32_t phase = 0;  // bit st: parity of land[st]
    for (int j = 0; j < tiles; j++) {
        if (!part.tile<BN>(j)) continue;
        const int st = (2 * j + 1) % C::kStages, key0 = (b.beg + j) * BN;
        if (!role_wait(land + st, (phase >> st) & 1u, misc, p.flags)) break;
        phase ^= 1u << st;
        unsigned char *at = sm + C::kSmRing + st * C::kStageBytes;
        const auto chunk = [&](int e) { return reinterpret_cast<uint4 *>(at + tile_at(e / CH, e % CH, C::kSubK)); };
        // Only slots that some row does not see, eight chunks of a thread at once; behind the
        // row's end, zeros.
        constexpr int BATCH = 8;
        const int stop = min(BN, b.len - key0) * CH;
        for (int e0 = max(0, part.from(j) - key0) * CH + tid; e0 < stop; e0 += 64 * BATCH) {
            uint32_t any = 0;
#pragma unroll
            for (int k = 0; k < BATCH; k++)
                if (e0 + 64 * k < stop) any |= special_bits(*chunk(e0 + 64 * k));
            if (any & 0x80008000u) {
#pragma unroll 1
                for (int e = e0; e < min(stop, e0 + 64 * BATCH); e += 64)
                    if (special_bits(*chunk(e)) & 0x80008000u)
                        *chunk(e) = take_out<D>(*chunk(e), 8 * (e % CH), key0 + e / CH, bad, misc);
            }
        }
        for (int e = stop + tid; e < BN * CH; e += 64) *chunk(e) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        asm volatile("bar.sync 1, 64;" ::: "memory");
        if (tid == 0) mbar_arrive(full + st);
    }
}

// All three warps, for what TMA does not bring: fill 2j is K, fill 2j+1 V of key tile beg + j.  bf16 rows are copied
// asynchronously, kLag fills in flight before the oldest is handed over.
template <int D, int ELEM>
__device__ __forceinline__ void loader(const PrefillParams &p, const Block &b, unsigned char *sm, uint64_t *full,
                                       uint64_t *empty, int *bad, Misc *misc) {
    using C = Cfg<D>;
    constexpr int BN = C::BN, CH = D * ELEM / 16, ALL = BN * CH;  // 16-byte chunks per record, per tile
    constexpr int PER = (ALL + kLoaders - 1) / kLoaders;          // per thread
    constexpr int kLag = 2;
    const Geometry &geo = p.geo;
    const int tid = threadIdx.x < 288 ? threadIdx.x - 256 : threadIdx.x - 288;
    const int tiles = max(b.cnt[0], b.cnt[1]);
    const uint32_t ring = smem_u32(sm + C::kSmRing);
    const Partial part(p, b);
    // Hands fill f over: its V may need special values taken out first.
    const auto hand_over = [&](int f) {
        const int j = f >> 1;
        if (ELEM == 2 && (f & 1) && part.tile<BN>(j)) {
            unsigned char *st = sm + C::kSmRing + (f % C::kStages) * C::kStageBytes;
            for (int e = tid; e < ALL; e += kLoaders) {
                const int row = e / CH, c = e % CH;
                uint4 *at = reinterpret_cast<uint4 *>(st + tile_at(row, c, C::kSubK));
                const uint4 v = *at;
                if (has_special(v)) *at = take_out<D>(v, 8 * c, (b.beg + j) * BN + row, bad, misc);
            }
        }
        fence_async_smem();
        mbar_arrive(full + f % C::kStages);
    };
    for (int f = 0; f < 2 * tiles; f++) {
        const int st = f % C::kStages;
        if (f >= C::kStages && !role_wait(empty + st, ((f / C::kStages) - 1) & 1, misc, p.flags)) break;
        const char *src = f & 1 ? p.V : p.K;
        const int key0 = (b.beg + (f >> 1)) * BN;
        if (ELEM == 2) {
#pragma unroll 4
            for (int e = tid; e < ALL; e += kLoaders) {
                const int row = e / CH, c = e % CH, j = key0 + row;
                int64_t rec = j < b.len ? record(geo, b, j) : -1;
                if (rec < 0 && j < b.len) {
                    misc->any_missing = 1u;
                    atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
                }
                cp16(ring + st * C::kStageBytes + tile_at(row, c, C::kSubK), src + (rec < 0 ? 0 : rec) * (2 * D) + 16 * c,
                     rec >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (f >= kLag) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                hand_over(f - kLag);
            }
        } else {
            uint4 v[PER];
#pragma unroll
            for (int k = 0; k < PER; k++) {
                const int e = tid + kLoaders * k, row = e / CH, c = e % CH, j = key0 + row;
                if (e >= ALL) break;
                const int64_t rec = j < b.len ? record(geo, b, j) : -1;
                if (rec < 0 && j < b.len) {
                    misc->any_missing = 1u;
                    atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
                }
                v[k] = rec < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4 *>(src + rec * D + 16 * c);
            }
            const bool chk = (f & 1) && part.tile<BN>(f >> 1);
#pragma unroll
            for (int k = 0; k < PER; k++) {
                const int e = tid + kLoaders * k, row = e / CH, c = e % CH;
                if (e >= ALL) break;
                uint4 lo = widen8(v[k].x, v[k].y), hi = widen8(v[k].z, v[k].w);
                if (chk && has_special(lo)) lo = take_out<D>(lo, 16 * c, key0 + row, bad, misc);
                if (chk && has_special(hi)) hi = take_out<D>(hi, 16 * c + 8, key0 + row, bad, misc);
                unsigned char *at = sm + C::kSmRing + st * C::kStageBytes;
                *reinterpret_cast<uint4 *>(at + tile_at(row, 2 * c, C::kSubK)) = lo;
                *reinterpret_cast<uint4 *>(at + tile_at(row, 2 * c + 1, C::kSubK)) = hi;
            }
            hand_over(f);
        }
    }
    if (ELEM == 2) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (!misc->abort_flag)
            for (int f = max(0, 2 * tiles - kLag); f < 2 * tiles; f++) hand_over(f);
    }
}

// ------------------------------------------------------------------ products

// True in one lane of a converged warp.  The warp that issues products keeps its
// control flow uniform and elects per batch: operands then sit in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t q, uint32_t k, uint32_t d) {
    using C = Cfg<D>;
    const uint64_t qd = smem_desc(q, 16, 1024), kd = smem_desc(k, 16, 1024);
#pragma unroll
    for (int i = 0; i < D / 16; i++)
        mma_ss(d, qd + (((i >> 2) * C::kSubQ + (i & 3) * 32) >> 4), kd + (((i >> 2) * C::kSubK + (i & 3) * 32) >> 4),
               idesc(kRows, C::BN, 0), i > 0);
}
template <int D, int HALF>
__device__ __forceinline__ void issue_pv(uint32_t p, uint32_t v, uint32_t d, bool acc) {
    using C = Cfg<D>;
    const uint64_t vd = smem_desc(v, C::kSubK, 1024);
#pragma unroll
    for (int i = 0; i < C::BN / 16; i++)
        if (i / (C::BN / 32) == HALF) mma_ts(d, p + 8 * i, vd + i * (2048 >> 4), idesc(kRows, D, 1), acc || i > 0);
}

template <int D>
__device__ __forceinline__ void issuer(const PrefillParams &p, const Block &b, unsigned char *sm, uint32_t tmem,
                                       uint64_t *full, uint64_t *empty, uint64_t *q_full, uint64_t *s_full,
                                       uint64_t *p_full, uint64_t *p_half, uint64_t *o_done, Misc *misc) {
    using C = Cfg<D>;
    const int cnt0 = b.cnt[0], cnt1 = b.cnt[1];
    const int tiles = max(cnt0, cnt1);
    const uint32_t q = smem_u32(sm), ring = smem_u32(sm + C::kSmRing);
    const auto have = [&](int f) {
        const bool ok = role_wait(full + f % C::kStages, (f / C::kStages) & 1, misc, p.flags);
        fence_after();
        return ok;
    };
    const auto at = [&](int f) { return ring + (f % C::kStages) * C::kStageBytes; };
    if (tiles == 0 || !role_wait(q_full, 0, misc, p.flags)) return;
    if (!have(0)) return;
    if (C::NT == 2) {
        if (elect_one()) {
#pragma unroll
            for (int t = 0; t < 2; t++)
                if ((t ? cnt1 : cnt0) > 0) {
                    issue_qk<D>(q + t * C::kQBytes, at(0), tmem + C::kTmemS(t));
                    mma_commit(s_full + t);
                }
            mma_commit(empty);
        }
        __syncwarp();
        for (int j = 0; j < tiles; j++) {
            bool v = false, k = false;  // V of tile j, K of tile j + 1 have landed
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const int cnt = t ? cnt1 : cnt0;
                if (j >= cnt) continue;
                if (!v && !have(2 * j + 1)) return;
                v = true;
                if (j + 1 < cnt && !k) {
                    if (!have(2 * j + 2)) return;
                    k = true;
                }
                if (!role_wait(p_half + t, j & 1, misc, p.flags)) return;
                fence_after();
                if (elect_one()) issue_pv<D, 0>(tmem + C::kTmemS(t), at(2 * j + 1), tmem + C::kTmemO(t), j > 0);
                __syncwarp();
                if (!role_wait(p_full + t, j & 1, misc, p.flags)) return;
                fence_after();
                if (elect_one()) {
                    issue_pv<D, 1>(tmem + C::kTmemS(t), at(2 * j + 1), tmem + C::kTmemO(t), true);
                    if (j + 1 == cnt) mma_commit(o_done + t);
                    // the last query tile that takes V
                    if (t == 1 || j >= cnt1) mma_commit(empty + (2 * j + 1) % C::kStages);
                    if (j + 1 < cnt) {
                        issue_qk<D>(q + t * C::kQBytes, at(2 * j + 2), tmem + C::kTmemS(t));
                        mma_commit(s_full + t);
                        if (t == 1 || j + 1 >= cnt1) mma_commit(empty + (2 * j + 2) % C::kStages);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        if (elect_one()) {
            issue_qk<D>(q, at(0), tmem + C::kTmemS(0));
            mma_commit(s_full);
            mma_commit(empty);
        }
        __syncwarp();
        for (int j = 0; j < tiles; j++) {
            if (j + 1 < tiles) {
                if (!have(2 * j + 2)) return;
                if (elect_one()) {
                    issue_qk<D>(q, at(2 * j + 2), tmem + C::kTmemS((j + 1) & 1));
                    mma_commit(s_full + ((j + 1) & 1));
                    mma_commit(empty + (2 * j + 2) % C::kStages);
                }
                __syncwarp();
            }
            if (!have(2 * j + 1) || !role_wait(p_half + (j & 1), (j >> 1) & 1, misc, p.flags)) return;
            fence_after();
            if (elect_one()) issue_pv<D, 0>(tmem + C::kTmemS(j & 1), at(2 * j + 1), tmem + C::kTmemO(0), j > 0);
            __syncwarp();
            if (!role_wait(p_full + (j & 1), (j >> 1) & 1, misc, p.flags)) return;
            fence_after();
            if (elect_one()) {
                issue_pv<D, 1>(tmem + C::kTmemS(j & 1), at(2 * j + 1), tmem + C::kTmemO(0), true);
                mma_commit(empty + (2 * j + 1) % C::kStages);
                mma_commit(o_done + (j & 1));  // phase j / 2
            }
            __syncwarp();
        }
    }
}

// ------------------------------------------------------------------- softmax

template <int D>
__device__ __forceinline__ void softmax(const PrefillParams &p, const Block &b, int t, int64_t part, unsigned char *sm,
                                        uint32_t tmem, uint64_t *q_full, uint64_t *s_full, uint64_t *p_full,
                                        uint64_t *p_half, uint64_t *o_done, const int *bad, Misc *misc) {
    using C = Cfg<D>;
    constexpr int BN = C::BN;
    const Geometry &geo = p.geo;
    const int tid = threadIdx.x & 127, lane = tid & 31;
    const int base = b.row0 + t * kRows;  // first row of the tile
    // The query tile: 16-byte chunks, rows behind the sequence's last as zeros; a thread's
    // loads are all issued before the first is stored.
    {
        constexpr int CH = D / 8, PER = kRows * CH / 128, BATCH = PER < 16 ? PER : 16;
#pragma unroll
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
                *reinterpret_cast<uint4 *>(sm + t * C::kQBytes + tile_at(e / CH, e % CH, C::kSubQ)) = v[k];
            }
        }
    }
    fence_async_smem();
    mbar_arrive(q_full);

    const int x = base + tid;
    const bool real = x < b.rows;
    // rows behind the last see what the last does; they are not written
    const int limit = last_seen(p, b, min(x, b.rows - 1));
    const int first = last_seen(p, b, base);  // no row of the tile sees less
    const uint32_t my = tmem + ((uint32_t)(tid & ~31) << 16);
    const float scale = p.scale_log2;
    // (The wait for s_full covers every product issued before it: with one query tile, P V of
    // tile j - 2, so of the two o_done barriers none is more than a phase behind its wait.)
    float m = -INFINITY, sum = 0.f;  // m in units of log2: subtracted from scaled scores
    bool ok = true;
    for (int j = 0; j < b.cnt[t]; j++) {
        const int sb = C::NT == 2 ? t : j & 1;
        const uint32_t ph = C::NT == 2 ? j & 1 : (j >> 1) & 1;
        if (!role_wait(s_full + sb, ph, misc, p.flags)) { ok = false; break; }
        fence_after();
        uint32_t s[BN];
#pragma unroll
        for (int c = 0; c < BN / 32; c++) tmem_ld32(my + C::kTmemS(sb) + 32 * c, s + 32 * c);
        wait_ld();
        const int key0 = (b.beg + j) * BN;
        if (key0 + BN - 1 > first) {  // some row sees the tile only in part
#pragma unroll
            for (int k = 0; k < BN; k++)
                if (key0 + k > limit) s[k] = 0xff800000u;
        }
        if (misc->any_missing) {  // slots without a block have no weight
            for (int c = 0; c < BN / 32; c++) {
                const int jj = key0 + 32 * c + lane;
                const uint32_t gone = __ballot_sync(0xffffffffu, jj < b.len && record(geo, b, jj) < 0);
#pragma unroll
                for (int k = 0; k < BN; k++)
                    if ((k >> 5) == c && (gone >> (k & 31) & 1)) s[k] = 0xff800000u;
            }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            constexpr int W = BN / 4;
            mx[c] = max2(__uint_as_float(s[c * W]), __uint_as_float(s[c * W + 1]));
#pragma unroll
            for (int k = 2; k < W; k += 2) mx[c] = max3(mx[c], __uint_as_float(s[c * W + k]), __uint_as_float(s[c * W + k + 1]));
        }
        float top = max2(max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
        if (top == INFINITY) top = NAN;  // inf - inf, as the definition has it
        // raise the maximum: always from nothing, else once the scores pass it by 2^8
        if (__any_sync(0xffffffffu, !(top <= m + kRaise))) {
            const float mn = top <= m + kRaise ? m : top;
            const float f = m == -INFINITY ? 0.f : ex2(m - mn);
            if (j > 0) {
                if (C::NT == 1 && !role_wait(o_done + ((j - 1) & 1), ((j - 1) >> 1) & 1, misc, p.flags)) { ok = false; break; }
                fence_after();
                const float f1 = mn == m ? 1.f : f;
#pragma unroll
                for (int c = 0; c < D / 32; c++) {
                    uint32_t o[32];
                    tmem_ld32(my + C::kTmemO(t) + 32 * c, o);
                    wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f1);
                    tmem_st32(my + C::kTmemO(t) + 32 * c, o);
                }
                sum *= f1;
            }
            m = mn;
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const f32x2 scale2 = both(scale), off2 = both(off);
        f32x2 part_sum[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < BN / 32; c++) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; k++) {
                const f32x2 e = fma2(pack2(__uint_as_float(s[32 * c + 2 * k]), __uint_as_float(s[32 * c + 2 * k + 1])),
                                     scale2, off2);
                float a, d;
                if (k % 4 == 3) {
                    ex2_fma(e, a, d);
                } else {
                    unpack2(e, a, d);
                    a = ex2(a);
                    d = ex2(d);
                }
                part_sum[k & 1] = add2(part_sum[k & 1], pack2(a, d));
                pk[k] = bf16x2(a, d);
            }
            tmem_st16(my + C::kTmemS(sb) + 16 * c, pk);
            if (c == BN / 64 - 1) {
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_half + sb);
            }
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + sb);
        float s0, s1;
        unpack2(add2(part_sum[0], part_sum[1]), s0, s1);
        sum += s0 + s1;
    }
    // ---- epilogue
    if (ok && b.cnt[t] > 0) {
        ok = role_wait(o_done + (C::NT == 2 ? t : (b.cnt[t] - 1) & 1), C::NT == 2 ? 0 : ((b.cnt[t] - 1) >> 1) & 1, misc, p.flags);
        fence_after();
    }
    if (!ok) return;
    const bool nothing = sum == 0.f;
    const float inv = nothing ? 0.f : 1.f / sum;
    const int64_t row = row_of(p, b, min(x, b.rows - 1));
    if (part < 0 && real && p.lse) p.lse[row] = nothing ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
    float *slab = p.part + part * (C::NT * kRows) * (D + 2) + (t * kRows + tid) * (D + 2);
    if (part >= 0) {
        slab[D] = nothing ? -INFINITY : m;
        slab[D + 1] = sum;
    }
    const bool fix = misc->any_bad;
#pragma unroll
    for (int c = 0; c < D / 32; c++) {
        uint32_t o[32];
        if (b.cnt[t] > 0) {
            tmem_ld32(my + C::kTmemO(t) + 32 * c, o);
            wait_ld();
        } else {
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] = 0u;
        }
        if (fix && b.cnt[t] > 0) {
#pragma unroll
            for (int k = 0; k < 32; k++) {
                const int *at = bad + 32 * c + k;
                if (at[D] <= limit) o[k] = __float_as_uint(__uint_as_float(o[k]) + INFINITY);
                if (at[2 * D] <= limit) o[k] = __float_as_uint(__uint_as_float(o[k]) - INFINITY);
                if (at[0] <= limit) o[k] = 0x7fc00000u;
            }
        }
        if (part >= 0) {
#pragma unroll
            for (int k = 0; k < 32; k += 2)
                *reinterpret_cast<uint2 *>(slab + 32 * c + k) = make_uint2(o[k], o[k + 1]);
        } else {
            // through the query tile, which no product reads any more: rows of a warp are
            // its own, and go out as whole 16-byte runs of consecutive rows below
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const auto two = [&](int i) {
                    return bf16x2(__uint_as_float(o[8 * k + i]) * inv, __uint_as_float(o[8 * k + i + 1]) * inv);
                };
                *reinterpret_cast<uint4 *>(sm + t * C::kQBytes + tile_at(tid, 4 * c + k, C::kSubQ)) =
                    make_uint4(two(0), two(2), two(4), two(6));
            }
        }
    }
    if (part < 0) {
        constexpr int CH = D / 8;
        __syncwarp();
#pragma unroll 8
        for (int e = lane; e < 32 * CH; e += 32) {
            const int r = (tid & ~31) + e / CH;
            if (base + r < b.rows)
                *reinterpret_cast<uint4 *>(p.out + row_of(p, b, base + r) * D + 8 * (e % CH)) =
                    *reinterpret_cast<const uint4 *>(sm + t * C::kQBytes + tile_at(r, e % CH, C::kSubQ));
        }
    }
    fence_before();
}

// ------------------------------------------------------------------- kernels

// TMA: a bf16 cache brought by tma_loader; else loader.
template <int D, int ELEM, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smraw[];
    __shared__ Block blk;
    __shared__ int found;
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    int *bad = reinterpret_cast<int *>(sm + C::kSmBad);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::kSmBar), *empty = full + C::kStages;
    uint64_t *q_full = empty + C::kStages, *s_full = q_full + 1, *p_full = s_full + 2, *o_done = p_full + 2,
             *drain = o_done + 2, *land = drain + 1, *p_half = land + C::kStages;
    Misc *misc = reinterpret_cast<Misc *>(sm + C::kSmMisc);
    const int warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const int idx = p.splits == 1 ? blockIdx.x : blockIdx.x / p.splits;
    const int split = (int)blockIdx.x - idx * p.splits;
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&misc->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0) {
        const bool f = find_block<D>(p, idx, split, &blk);
        if ((threadIdx.x & 31) == 0) found = f;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < C::kStages; i++) {
            mbar_init(full + i, TMA ? 1 : kLoaders);
            mbar_init(empty + i, 1);
            mbar_init(land + i, 1);
        }
        mbar_init(q_full, 128 * C::NT);
        mbar_init(drain, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(p_half + i, 4);
            mbar_init(o_done + i, 1);
        }
        mbar_init_fence();
        misc->abort_flag = 0u;
        misc->any_bad = 0u;
        misc->any_missing = 0u;
    }
    for (int e = threadIdx.x; e < 3 * D; e += kThreads) bad[e] = 0x7fffffff;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = misc->tmem;
    if (found) {
    // Registers: 384 threads are launched with 168 each; 2 x 208 + 88 = 3 x 168.
    if (warp < 8) {
        regs_up<208>();
        const int t = warp >> 2;
        if (t < C::NT)
            softmax<D>(p, blk, t, p.splits > 1 ? (int64_t)blockIdx.x : -1, sm, tmem, q_full, s_full, p_full, p_half, o_done, bad, misc);
    } else {
        regs_down<88>();
        if (warp == 9) {
            issuer<D>(p, blk, sm, tmem, full, empty, q_full, s_full, p_full, p_half, o_done, misc);
            __syncwarp();
            if (misc->abort_flag && elect_one()) {  // after a wait ran out: products in flight end before their memory is released
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        } else if (!TMA) {
            loader<D, ELEM>(p, blk, sm, full, empty, bad, misc);
        } else if (warp == 8) {
            tma_loader<D>(p, blk, sm, &mk, &mv, full, empty, land, misc);
        } else {
            mender<D>(p, blk, sm, full, land, bad, misc);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    }
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    grid_dependents_launch();
}

// Merges the splits of a block's rows: one warp per row,
//   out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k.
template <int D>
__global__ void __launch_bounds__(256) prefill_join(const __grid_constant__ PrefillParams p) {
    constexpr int R = kRows * Cfg<D>::NT, PER = R / 8;  // blocks of 8 rows per unit
    __shared__ Block blk;
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    const int idx = blockIdx.x / PER;
    const int r = (int)(blockIdx.x % PER) * 8 + warp;
    if (warp == 0) {
        const bool f = find_block<D>(p, idx, 0, &blk);
        if (lane == 0) found = f;
    }
    __syncthreads();
    const int x = blk.row0 + r;
    if (!found || x >= blk.rows) return;
    const float *slab = p.part + (int64_t)idx * p.splits * R * (D + 2) + (int64_t)r * (D + 2);
    float m = -INFINITY;
    for (int k = 0; k < p.splits; k++) m = max2(m, slab[(int64_t)k * R * (D + 2) + D]);
    float sum = 0.f, o[D / 32] = {0.f};
    for (int k = 0; k < p.splits; k++) {
        const float *s = slab + (int64_t)k * R * (D + 2);
        const float mk = s[D];
        if (mk == -INFINITY) continue;
        const float w = exp2f(mk - m);
        sum = fmaf(w, s[D + 1], sum);
#pragma unroll
        for (int e = 0; e < D / 32; e++) o[e] = fmaf(w, s[lane + 32 * e], o[e]);
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

// Blocks per (layer, KV head): sum over sequences of ceil(n G / R), bounded from what the host knows.
int64_t most_blocks(int64_t S, int64_t G, int D, int64_t T) {
    const int64_t R = D == 256 ? kRows : 2 * kRows;
    return T * G / R + std::min(S, T);
}

constexpr int kMostParts = 160;  // parts of split rows the workspace holds: one per SM

// Splits of each row over its keys: as many as fill the SMs while a split keeps at least
// four key tiles of the average row.
int splits_of(int64_t blocks, int64_t keys, int D) {
    const int64_t tiles = keys / (D == 256 ? 64 : 128);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(sm_count(), kMostParts) / std::max<int64_t>(1, blocks), tiles / 4));
}

// The cache as boxes of 64 dims x up to BN slots, 128-byte swizzled: [total][d], or the
// pool's slots [L n_blocks bs][H][d] one head at a time.
template <int D>
bool make_map(CUtensorMap *m, const void *base, const Geometry &geo) {
    auto fn = tensormap_encode_fn();
    if (!fn) return false;
    const bool paged = geo.layout == TRI_KV_PAGED;
    const int64_t slots = paged ? (int64_t)geo.L * geo.n_blocks << geo.block_shift : geo.total;
    const cuuint32_t box = (cuuint32_t)std::min<int64_t>(paged ? 1 << geo.block_shift : Cfg<D>::BN, Cfg<D>::BN);
    const cuuint64_t dims3[3] = {D, (cuuint64_t)geo.H, (cuuint64_t)slots}, dims2[2] = {D, (cuuint64_t)slots};
    const cuuint64_t str3[2] = {2 * D, (cuuint64_t)geo.H * 2 * D}, str2[1] = {2 * D};
    const cuuint32_t box3[3] = {64, 1, box}, box2[2] = {64, box}, ones[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, paged ? 3 : 2, const_cast<void *>(base), paged ? dims3 : dims2,
              paged ? str3 : str2, paged ? box3 : box2, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA wants slot numbers of 31 bits, and pages that fill a swizzle atom of 8 rows.
bool tma_fits(const Geometry &geo) {
    const bool paged = geo.layout == TRI_KV_PAGED;
    const int64_t most = 0x7fffffffLL;
    if (paged) return geo.block_shift >= 3 && geo.n_blocks <= most / geo.L >> geo.block_shift;
    return geo.total >= 1 && geo.total <= most;
}

template <int D, int ELEM, bool TMA>
cudaError_t launch_t(const PrefillParams &p, int64_t units, cudaStream_t s) {
    static bool attr[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    auto kern = prefill_kernel<D, ELEM, TMA>;
    if (!attr[dev & 63]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        attr[dev & 63] = true;
    }
    CUtensorMap mk = {}, mv = {};
    if (TMA && (!make_map<D>(&mk, p.K, p.geo) || !make_map<D>(&mv, p.V, p.geo))) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(kern, dim3((unsigned)(units * p.splits)), dim3(kThreads), Cfg<D>::kSmem, s, p, mk, mv);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_pdl(prefill_join<D>, dim3((unsigned)(units * Cfg<D>::NT * kRows / 8)), dim3(256), 0, s, p);
}

template <int D>
cudaError_t launch_d(const PrefillParams &p0, cudaStream_t s) {
    PrefillParams p = p0;
    const Geometry &geo = p.geo;
    const int64_t blocks = most_blocks(geo.S, geo.G, D, p.T), units = blocks * geo.L * geo.H;
    p.blocks = (int32_t)blocks;
    int l = 0;
    while ((1 << l) < geo.G) l++;
    p.div_shift = 31 + l;
    p.div_mul = ((1ull << (31 + l)) + geo.G - 1) / geo.G;
    if (units > 0x7fffffffLL / 64 || p.T * geo.G > 0x7fffff00LL) return cudaErrorInvalidConfiguration;
    p.splits = splits_of(units, geo.total / ((int64_t)geo.L * geo.S * geo.H), D);
    if (geo.elem_bytes == 1) return launch_t<D, 1, false>(p, units, s);
    return tma_fits(geo) ? launch_t<D, 2, true>(p, units, s) : launch_t<D, 2, false>(p, units, s);
}

}  // namespace

// Scratch of split rows: at most one part per SM.
size_t prefill_scratch_bytes(int64_t L, int64_t S, int64_t H, int64_t G, int D, int64_t T) {
    const int64_t units = most_blocks(S, G, D, T) * L * H, sms = kMostParts;
    if (units == 0 || units > sms / 2) return 0;
    return (size_t)(sms / units * units) * (D == 256 ? kRows : 2 * kRows) * (D + 2) * sizeof(float);
}

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_d<64>(p, s);
        case 128: return launch_d<128>(p, s);
        case 256: return launch_d<256>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tri

// New tokens into the cache (the cache that "TriAttention：基于三角函数 KV 压缩的高效
// 长推理", 流程详解 steps 2-5, scores, compacts and attends to): per token and head,
// pair f of the query and the key turned by w_f * position,
//   (re, im) -> (re cos - im sin, re sin + im cos),
// the query to q_out, key, value and position to the token's cache slot.
//
// Bound by HBM: every element is read and written once.  A 32K prompt of 64 query and 8 KV
// heads of 128 (1.34 GB) takes 219 us, 6.1 TB/s, 0.94 of a plain copy's rate (272 us with one
// unit of a thread in flight and angles read with bank conflicts); 16 single tokens 3.7 us,
// launch latency.  A block takes `tile`
// tokens at a time.  First the angles: one sine and cosine per (token, pair),
// shared by all query and KV heads through shared memory, from a phase reduced
// exactly as (pos * T_f) mod 2^64 turns, so far positions lose nothing; and
// each token's sequence and place in it.  Then one thread per unit of 8 pairs of one
// head (16 values: two 16-byte loads; 8 + 8 dims of a rotate-half record, 16
// adjacent ones of an interleaved record), whose loads for kBatch units are issued before
// the first is used.  The fp32 rotation is rounded once, to
// bf16 or e4m3 (saturating, as the format's cache holds no infinities).
#include <algorithm>

#include <cuda_bf16.h>

#include "keys.cuh"

namespace tri {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppTile = 8;  // most tokens per block step
constexpr int kBatch = 2;    // units of a thread in flight
// u / units as (u * ceil(2^55 / units)) >> 55: exact while u * units < 2^55, and u < 8 units, units <= 2^26.
constexpr int kDivShift = 55;

// Lanes of one warp: the sequence token t belongs to (the number of sequences that
// end at or before t; S when t lies behind the last sequence).
__device__ __forceinline__ int token_seq(const int64_t *tok_off, int S, int64_t t, int lane) {
    int seq = 0;
    for (int base = 0; base < S; base += 32) {
        const int s = base + lane;
        const bool before = s < S && __ldg(tok_off + s + 1) <= t;
        seq += __popc(__ballot_sync(0xffffffffu, before));
    }
    return seq;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Stores 8 values (fp32) as ELEM-byte elements at dst.
template <int ELEM>
__device__ __forceinline__ void store8(char *dst, const float (&x)[8]) {
    if (ELEM == 2)
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                     pack_bf16(x[6], x[7]));
    else
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
}

struct TokenPlace {
    int64_t tail;  // slots from this token to the end of its rows (n_s - i), 0: no slot
    int seq;       // -1: behind the last sequence
    int pos;
};

template <int D, int ELEM, bool IL>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int F = D / 2, UPH = D / 16;  // units per head
    __shared__ float2 turn[kAppTile][F];  // pair f at 8 f's units apart: [f % 8][f / 8], so that lanes read neighbours
    __shared__ TokenPlace place[kAppTile];
    const Geometry &geo = p.geo;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = p.tile;
    const int64_t tiles = (p.T + tile - 1) / tile;
    const int HQ = p.q ? geo.Hq : 0;
    const int heads = HQ + 2 * geo.H;  // queries, keys, values
    const int units = heads * UPH;

    grid_dependency_wait();
    for (int64_t item = blockIdx.x; item < tiles * geo.L; item += gridDim.x) {
        const int l = (int)(item / tiles);
        const int64_t t0 = (item % tiles) * tile;
        const int nt = (int)std::min<int64_t>(tile, p.T - t0);
        for (int i = warp; i < nt; i += kAppThreads / 32) {
            const int s = token_seq(p.tok_off, geo.S, t0 + i, lane);
            if (lane == 0) {
                TokenPlace w;
                w.seq = s < geo.S ? s : -1;
                w.pos = p.positions[t0 + i];
                w.tail = 0;
                if (s < geo.S) {
                    const int64_t b = p.tok_off[s], e = p.tok_off[s + 1];
                    if (b >= 0 && b <= t0 + i && e > t0 + i && e <= p.T) w.tail = e - (t0 + i);
                    else atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
                }
                place[i] = w;
            }
        }
        for (int e = threadIdx.x; e < nt * F; e += kAppThreads) {
            const int i = e / F, f = e % F;
            const unsigned long long ph = (unsigned long long)(long long)p.positions[t0 + i] * p.turns[f];
            float sn, cs;
            sincospif((float)(long long)ph * 1.0842021724855044e-19f, &sn, &cs);  // 2^-63: half turns
            turn[i][(f % 8) * UPH + f / 8] = make_float2(cs, sn);
        }
        __syncthreads();
        for (int u0 = threadIdx.x; u0 < nt * units; u0 += kAppThreads * kBatch) {
            uint4 ra[kBatch], rb[kBatch];
            int tok[kBatch], head[kBatch], chunk[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; e++) {
                const int u = u0 + e * kAppThreads;
                if (u >= nt * units) {
                    tok[e] = -1;
                    continue;
                }
                const int i = (int)(((unsigned long long)(unsigned)u * p.div_mul) >> kDivShift), x = u - i * units;
                const int hd = x / UPH, c = x % UPH;
                tok[e] = place[i].seq < 0 ? -1 : i;
                head[e] = hd;
                chunk[e] = c;
                if (tok[e] < 0) continue;
                const int64_t row = (int64_t)l * p.T + t0 + i;
                const char *src = hd < HQ ? p.q + row * p.q_stride + (int64_t)hd * (2 * D)
                                  : hd < HQ + geo.H ? p.k + row * p.k_stride + (int64_t)(hd - HQ) * (2 * D)
                                                    : p.v + row * p.v_stride + (int64_t)(hd - HQ - geo.H) * (2 * D);
                ra[e] = *reinterpret_cast<const uint4 *>(src + (IL ? 32 * c : 16 * c));
                rb[e] = *reinterpret_cast<const uint4 *>(src + (IL ? 32 * c + 16 : 16 * c + 2 * F));
            }
#pragma unroll
            for (int e = 0; e < kBatch; e++) {
                if (tok[e] < 0) continue;
                const int i = tok[e], c = chunk[e];
                const bool is_q = head[e] < HQ, is_v = head[e] >= HQ + geo.H;
                const int h = is_q ? head[e] : is_v ? head[e] - HQ - geo.H : head[e] - HQ;
                const int64_t row = (int64_t)l * p.T + t0 + i;
                float a[8], b[8];
                unpack_bf16x8(ra[e], a);
                unpack_bf16x8(rb[e], b);
                if (is_q || (!is_v && p.rotate_keys)) {
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const float2 t = turn[i][k * UPH + c];
                        // interleaved: pairs 0..3 lie in a, 4..7 in b, (re, im) adjacent
                        float &re = !IL ? a[k] : k < 4 ? a[2 * k] : b[2 * k - 8];
                        float &im = !IL ? b[k] : k < 4 ? a[2 * k + 1] : b[2 * k - 7];
                        const float r0 = fmaf(re, t.x, -im * t.y);
                        im = fmaf(re, t.y, im * t.x);
                        re = r0;
                    }
                }
                if (is_q) {
                    char *dst = p.q_out + (row * geo.Hq + h) * (2 * D);
                    store8<2>(dst + (IL ? 32 * c : 16 * c), a);
                    store8<2>(dst + (IL ? 32 * c + 16 : 16 * c + 2 * F), b);
                    continue;
                }
                const TokenPlace w = place[i];
                if (w.tail == 0) continue;
                const int64_t r = ((int64_t)l * geo.S + w.seq) * geo.H + h;
                const int64_t lo = geo.row_off[r], hi = geo.row_off[r + 1];
                const int64_t j = hi - lo - w.tail;  // the token's slot
                if (lo < 0 || hi > geo.total || j < 0) {
                    atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
                    continue;
                }
                int64_t rec = lo + j;
                if (geo.layout == TRI_KV_PAGED) {
                    const int64_t bi = j >> geo.block_shift;
                    const int32_t blk = bi < geo.max_blocks ? __ldg(geo.block_table + (int64_t)w.seq * geo.max_blocks + bi) : -1;
                    if (blk < 0 || blk >= geo.n_blocks) {
                        atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
                        continue;
                    }
                    rec = ((((int64_t)l * geo.n_blocks + blk) << geo.block_shift) | (j & ((1 << geo.block_shift) - 1))) * geo.H + h;
                }
                char *dst = (is_v ? p.V : p.K) + rec * (D * ELEM);
                store8<ELEM>(dst + (IL ? 16 * c : 8 * c) * ELEM, a);
                store8<ELEM>(dst + (IL ? 16 * c + 8 : 8 * c + F) * ELEM, b);
                if (!is_v && c == 0 && p.pos) p.pos[rec] = w.pos;
            }
        }
        __syncthreads();
    }
    grid_dependents_launch();
}

template <int D, int ELEM, bool IL>
cudaError_t launch_t(const AppendParams &p0, cudaStream_t s) {
    AppendParams p = p0;
    const int64_t sms = sm_count(), rows = p.T * p.geo.L;
    // Full tiles once they give every SM eight blocks; single tokens below that.
    p.tile = (int)std::max<int64_t>(1, std::min<int64_t>(kAppTile, rows / (8 * sms)));
    const unsigned units = (unsigned)((p.q ? p.geo.Hq : 0) + 2 * p.geo.H) * (D / 16);
    p.div_mul = ((1ull << kDivShift) + units - 1) / units;
    const int64_t items = (p.T + p.tile - 1) / p.tile * p.geo.L;
    return launch_pdl(append_kernel<D, ELEM, IL>, dim3((unsigned)std::min<int64_t>(items, 8 * sms)), dim3(kAppThreads), 0, s,
                      p);
}

template <int D>
cudaError_t launch_d(const AppendParams &p, cudaStream_t s) {
    if (p.geo.elem_bytes == 2) return p.geo.il ? launch_t<D, 2, true>(p, s) : launch_t<D, 2, false>(p, s);
    return p.geo.il ? launch_t<D, 1, true>(p, s) : launch_t<D, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_d<64>(p, s);
        case 128: return launch_d<128>(p, s);
        case 256: return launch_d<256>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tri

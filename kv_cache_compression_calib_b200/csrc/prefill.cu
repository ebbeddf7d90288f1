// Causal attention of new tokens over the cache that ends with them (the step around
// "TriAttention：基于三角函数 KV 压缩的高效长推理", 流程详解 step 5): for each (layer l,
// token i of sequence s's n, query head g of KV head h), over slots j <= N - n + i of
// row (l, s, h),
//   s_j = scale * (q . k_j),  out = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}.
//
// One warp per (token, head): each lane holds d/32 dims of the query, a key's dot
// product is a warp sum, softmax online in base 2 with fp32 statistics.
#include <algorithm>

#include <cuda_bf16.h>

#include "keys.cuh"

namespace tri {
namespace {

template <int D, int ELEM>
__global__ void __launch_bounds__(128) prefill_kernel(const PrefillParams p) {
    constexpr int E = D / 32;
    const Geometry &geo = p.geo;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t rows = p.T * geo.L * geo.Hq;
    if (item >= rows) return;
    const int g = (int)(item % geo.Hq);
    const int64_t lt = item / geo.Hq, t = lt % p.T;
    const int l = (int)(lt / p.T);
    int s = 0;
    for (; s < geo.S && p.tok_off[s + 1] <= t; s++)
        if (p.tok_off[s + 1] < p.tok_off[s] && lane == 0) atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
    if (s == geo.S) return;
    const int64_t tb = p.tok_off[s], te = p.tok_off[s + 1];
    const int64_t r = ((int64_t)l * geo.S + s) * geo.H + g / geo.G;
    const int64_t lo = geo.row_off[r], hi = geo.row_off[r + 1];
    int64_t seen = hi - lo - (te - t) + 1;
    if (lo < 0 || hi < lo || hi > geo.total || tb < 0 || tb > t || te > p.T) {
        if (lane == 0) atomicOr(p.flags, TRI_FLAG_ROW_OFFSETS);
        seen = 0;
    }
    float q[E], o[E] = {0.f}, m = -INFINITY, sum = 0.f;
    for (int e = 0; e < E; e++) q[e] = __uint_as_float((uint32_t)p.q[item * D + lane * E + e] << 16) * p.scale_log2;
    for (int64_t j = 0; j < seen; j++) {
        int64_t rec = lo + j;
        if (geo.layout == TRI_KV_PAGED) {
            const int64_t bi = j >> geo.block_shift;
            const int32_t blk = bi < geo.max_blocks ? __ldg(geo.block_table + (int64_t)s * geo.max_blocks + bi) : -1;
            if (blk < 0 || blk >= geo.n_blocks) {
                if (lane == 0) atomicOr(p.flags, TRI_FLAG_BLOCK_TABLE);
                continue;
            }
            rec = ((((int64_t)l * geo.n_blocks + blk) << geo.block_shift) | (j & ((1 << geo.block_shift) - 1))) * geo.H +
                  g / geo.G;
        }
        float k[E], v[E];
        for (int e = 0; e < E; e++) {
            const int64_t x = rec * D + lane * E + e;
            if (ELEM == 2) {
                k[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p.K)[x] << 16);
                v[e] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p.V)[x] << 16);
            } else {
                k[e] = e4m3x2_to_float2((uint8_t)p.K[x]).x;
                v[e] = e4m3x2_to_float2((uint8_t)p.V[x]).x;
            }
        }
        float dot = 0.f;
        for (int e = 0; e < E; e++) dot = fmaf(q[e], k[e], dot);
        for (int b = 16; b; b >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, b);
        const float mn = fmaxf(m, dot);
        const float a = m == mn ? 1.f : exp2f(m - mn), w = dot == -INFINITY ? 0.f : exp2f(dot - mn);
        sum = fmaf(sum, a, w);
        for (int e = 0; e < E; e++) o[e] = fmaf(o[e], a, w * v[e]);
        m = mn;
    }
    for (int e = 0; e < E; e++) {
        const __nv_bfloat16 b = __float2bfloat16_rn(sum == 0.f ? 0.f : o[e] / sum);
        p.out[item * D + lane * E + e] = *reinterpret_cast<const uint16_t *>(&b);
    }
    if (p.lse && lane == 0) p.lse[item] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_d(const PrefillParams &p, cudaStream_t s) {
    const int64_t blocks = (p.T * p.geo.L * p.geo.Hq + 3) / 4;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.geo.elem_bytes == 2) prefill_kernel<D, 2><<<(unsigned)blocks, 128, 0, s>>>(p);
    else prefill_kernel<D, 1><<<(unsigned)blocks, 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t prefill_scratch_bytes(int64_t, int64_t, int64_t, int64_t, int, int64_t) { return 0; }

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_d<64>(p, s);
        case 128: return launch_d<128>(p, s);
        case 256: return launch_d<256>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tri

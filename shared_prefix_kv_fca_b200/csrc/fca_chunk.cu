// fca_chunk_attention: the rows of new tokens over the paged cache.
//
// Row (token t of request r, query head h) at position p = L - n + i:
//   s_j = scale q.k_j,  o = sum_{j <= p} exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m)
// over the cached tokens j that the row sees (all L of them in full plans).
#include <algorithm>

#include <cuda_bf16.h>

#include "fca_chunk.h"
#include "fca_device.cuh"

namespace fca {
namespace {

struct ChunkArgs {
    const ChunkItem* items;
    const int32_t* begin;
    const int32_t* end;
    const int32_t* bad;
    const int32_t* bt;
    const int32_t* seq;
    const int32_t* qs;
    const __nv_bfloat16* q;
    int64_t q_stride;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* out;
    float* lse;
    int32_t R, max_blocks, num_blocks, Hq, Hkv, G, full;
    float scale_log2;
    int32_t* err;
};

// One row by one warp: a pass over its tokens with the running maximum and
// sum, lane i holding D / 32 of the row's elements.
template <int D>
__device__ void exact_row(const ChunkArgs& a, int32_t req, int32_t head, const __nv_bfloat16* q, int32_t tok0, int32_t tok1,
                          float (&o)[D / 32], float& m, float& l) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float qf[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        qf[i] = __bfloat162float(q[lane * E + i]);
        o[i] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
    for (int32_t j = tok0; j < tok1; ++j) {
        const int32_t b = a.bt[(int64_t)req * a.max_blocks + j / kBlockSize];
        const int64_t at = (((int64_t)b * kBlockSize + j % kBlockSize) * a.Hkv + head) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += qf[i] * __bfloat162float(a.k[at + i]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale_log2;
        const float top = fmaxf(m, s);
        const float f = top == -INFINITY ? 1.f : exp2f(m - top), p = top == -INFINITY ? 0.f : exp2f(s - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * f + p * __bfloat162float(a.v[at + i]);
    }
}

template <int D>
__global__ void __launch_bounds__(256) k_chunk_rows(ChunkArgs a) {
    const int32_t t = blockIdx.x, head = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (head >= a.Hq || t >= a.qs[a.R]) return;
    int32_t lo = 0, hi = a.R - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (a.qs[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int32_t n = a.qs[lo + 1] - a.qs[lo], L = a.bad[lo] ? 0 : a.seq[lo];
    const int32_t seen = (a.full || L == 0) ? L : L - n + (t - a.qs[lo]) + 1;
    float o[D / 32], m, l;
    exact_row<D>(a, lo, head / a.G, a.q + t * a.q_stride + (int64_t)head * D, 0, seen, o, m, l);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        a.out[((int64_t)t * a.Hq + head) * D + lane * (D / 32) + i] = __float2bfloat16(seen ? o[i] / l : 0.f);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + head] = seen ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace
}  // namespace fca

using namespace fca;

extern "C" fca_status fca_chunk_attention(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                                          fca_chunk_plan_t plan, void* out, float* lse, float scale, void* stream) {
    if (!plan || !k_cache || !v_cache || !(scale > 0.f) || !(scale < INFINITY)) return FCA_ERR_INVALID_ARG;
    if (plan->T > 0 && (!q || !out)) return FCA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u) || q_row_stride % 8 != 0 ||
        q_row_stride < (int64_t)plan->Hq * plan->D)
        return FCA_ERR_INVALID_ARG;
    if (plan->T == 0) return FCA_OK;
    DeviceGuard dg(plan->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ChunkArgs a;
    a.items = plan->items;
    a.begin = plan->begin;
    a.end = plan->end;
    a.bad = plan->bad;
    a.bt = plan->bt;
    a.seq = plan->seq;
    a.qs = plan->qs;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_row_stride;
    a.k = static_cast<const __nv_bfloat16*>(k_cache);
    a.v = static_cast<const __nv_bfloat16*>(v_cache);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.R = plan->R;
    a.max_blocks = plan->max_blocks;
    a.num_blocks = plan->num_blocks;
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.G = plan->G;
    a.full = plan->full;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.err = plan->dev_status;
    const dim3 grid(plan->T, (plan->Hq + 7) / 8);
    if (plan->D == 128)
        k_chunk_rows<128><<<grid, 256, 0, s>>>(a);
    else
        k_chunk_rows<64><<<grid, 256, 0, s>>>(a);
    return note_cuda(cudaGetLastError()) == cudaSuccess ? FCA_OK : FCA_ERR_CUDA;
}

// fca_append_kv: new keys and values into the paged caches.
//
// Row i of k and v ([num_kv_heads][head_dim], rows possibly strided in a wider
// projection output) is copied to token slots[i] of its cache.  No arithmetic:
// bound by memory, 4 bytes moved per element of k and v.  Each thread moves
// kPieces 16-byte pieces of consecutive rows, all loads before the first store
// and none waiting for a slot (the slots are only needed to store), so that a
// CTA has kPieces x 4 KB in flight.
#include "fca_internal.h"

namespace fca {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;

struct AppendArgs {
    const uint4 *k, *v;
    uint4 *k_cache, *v_cache;
    int64_t k_stride, v_stride;  // row strides, 16-byte pieces
    const int32_t* slots;
    int32_t* err;
    uint32_t num_tokens, row;    // row: pieces a row
    int32_t num_slots;
};

__global__ void __launch_bounds__(kThreads) k_append_kv(AppendArgs a) {
    const uint4* __restrict__ src = blockIdx.y ? a.v : a.k;
    uint4* __restrict__ dst = blockIdx.y ? a.v_cache : a.k_cache;
    const int64_t stride = blockIdx.y ? a.v_stride : a.k_stride;
    const uint64_t total = (uint64_t)a.num_tokens * a.row;
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPieces) + threadIdx.x;
    uint4 v[kPieces];
    int32_t slot[kPieces];
    uint32_t piece[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint64_t x = base + i * kThreads;
        slot[i] = -1;
        if (x < total) {
            const uint32_t t = (uint32_t)(x / a.row);
            piece[i] = (uint32_t)(x - (uint64_t)t * a.row);
            slot[i] = __ldg(a.slots + t);
            v[i] = __ldg(src + t * stride + piece[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (slot[i] >= a.num_slots) {
            if (a.err) atomicOr(a.err, kErrStaticBlockId);
        } else if (slot[i] >= 0) {
            dst[(uint64_t)slot[i] * a.row + piece[i]] = v[i];
        }
    }
}

}  // namespace
}  // namespace fca

using namespace fca;

extern "C" fca_status fca_append_kv(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                    const int32_t* slots, int32_t num_tokens, int32_t num_blocks,
                                    int32_t num_kv_heads, int32_t head_dim, void* k_cache, void* v_cache,
                                    int32_t* dev_status, void* stream) {
    if (num_tokens < 0 || num_blocks < 1 || num_kv_heads < 1 || !k_cache || !v_cache ||
        (num_tokens > 0 && (!k || !v || !slots)))
        return FCA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(slots) & 3u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return FCA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || (int64_t)num_blocks * kBlockSize > INT32_MAX) return FCA_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (row > INT32_MAX) return FCA_ERR_UNSUPPORTED;
    if (k_row_stride < row || v_row_stride < row || k_row_stride % 8 != 0 || v_row_stride % 8 != 0)
        return FCA_ERR_INVALID_ARG;
    if (num_tokens == 0) return FCA_OK;
    const size_t cache = (size_t)num_blocks * kBlockSize * row * 2, n = (size_t)num_tokens - 1;
    if (overlap(k_cache, cache, v_cache, cache)) return FCA_ERR_INVALID_ARG;
    for (const void* c : {k_cache, v_cache})
        if (overlap(c, cache, k, (n * k_row_stride + row) * 2) || overlap(c, cache, v, (n * v_row_stride + row) * 2) ||
            overlap(c, cache, slots, 4 * (n + 1)))
            return FCA_ERR_INVALID_ARG;
    AppendArgs a;
    a.k = static_cast<const uint4*>(k);
    a.v = static_cast<const uint4*>(v);
    a.k_cache = static_cast<uint4*>(k_cache);
    a.v_cache = static_cast<uint4*>(v_cache);
    a.k_stride = k_row_stride / 8;
    a.v_stride = v_row_stride / 8;
    a.slots = slots;
    a.err = dev_status;
    a.num_tokens = (uint32_t)num_tokens;
    a.row = (uint32_t)(row / 8);
    a.num_slots = num_blocks * kBlockSize;
    const int64_t ctas = ((int64_t)num_tokens * a.row + kThreads * kPieces - 1) / (kThreads * kPieces);
    if (ctas > INT32_MAX) return FCA_ERR_UNSUPPORTED;
    k_append_kv<<<dim3((unsigned)ctas, 2), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    if (note_cuda(cudaGetLastError()) != cudaSuccess) return FCA_ERR_CUDA;
    return FCA_OK;
}

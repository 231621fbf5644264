// fca_extend_tables: the requests' block tables grown by blocks off a free
// list, and the cache slot of every new token, from the requests' lengths.
//
// With c[r] cached and n[r] new tokens, request r holds h = ceil(c / 16) blocks
// and needs m = ceil((c + n) / 16) - h more.  Two exclusive sums over the
// requests place everything: q_starts[r] = sum n gives the request's rows, and
// first[r] = free_next + sum m its blocks on the list.  Block j >= h of the
// table is free_blocks[first[r] + j - h], so a token's slot needs the table
// itself only where it falls into the last block that was there.  A new
// block's first position is a multiple of 16 that is a new token's, so the
// thread with that token also writes the table entry: one pass over tokens.
//
// The work is a few hundred kilobytes at most and bound by latency: one
// launch, no workspace.  One cluster of CTAs (one CTA for small steps); each CTA
// sums all the lengths itself into its shared memory (reading 2 R integers
// again costs less than passing sums around), the tokens are dealt out over the
// cluster.  Every thread first finds and checks its slots, the CTAs exchange
// the verdict through distributed shared memory, and behind that cluster
// barrier either everything is written or nothing: every input has been read by
// then, so lengths and list position may be updated in place.
#include <algorithm>
#include <cooperative_groups.h>

#include "fca_internal.h"

namespace fca {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kCluster = 8;     // CTAs for large steps (the largest portable cluster)
constexpr int kKeep = 4;        // slots a thread keeps in registers between check and write

struct TablesArgs {
    int32_t* bt;
    const int32_t* cached;
    const int32_t* fresh;
    const int32_t* free_blocks;
    const int32_t* free_next;
    int32_t* seq_lens;
    int32_t* q_starts;
    int32_t* slots;
    int32_t* free_after;
    int32_t* err;
    int32_t R, max_blocks, num_free, num_blocks, num_slots;
};

// Exclusive sum over the CTA's threads of two 64-bit values; totals in ta, tb.
__device__ __forceinline__ void block_scan2(int64_t a, int64_t b, int64_t (*part)[2], int64_t& xa, int64_t& xb,
                                            int64_t& ta, int64_t& tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sa = a, sb = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, sa, o), ub = __shfl_up_sync(0xffffffffu, sb, o);
        if (lane >= o) {
            sa += ua;
            sb += ub;
        }
    }
    if (lane == 31) {
        part[warp][0] = sa;
        part[warp][1] = sb;
    }
    __syncthreads();
    int64_t wa = part[lane][0], wb = part[lane][1];      // kThreads / 32 == 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, wa, o), ub = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
            wa += ua;
            wb += ub;
        }
    }
    ta = __shfl_sync(0xffffffffu, wa, 31);
    tb = __shfl_sync(0xffffffffu, wb, 31);
    const int64_t pa = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
    xa = (warp ? pa : 0) + sa - a;
    xb = (warp ? pb : 0) + sb - b;
}

// Last r in [lo, hi] with start[r] <= t.
__device__ __forceinline__ int32_t find_request(const int32_t* start, int32_t t, int32_t lo, int32_t hi) {
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1) k_extend_tables(TablesArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* const start = sm;                    // [R + 1]
    int32_t* const first = sm + a.R + 1;          // [R] place of the request's first new block on the list
    int32_t* const had = first + a.R;             // [R] cached tokens
    __shared__ int64_t part[kThreads / 32][2];
    __shared__ int32_t verdict[kCluster];
    __shared__ int32_t bits;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t R = a.R;
    if (tid == 0) bits = 0;      // (the scan's barrier lies between this and the first use)

    // lengths of this thread's requests [r0, r1), their sums, and the scan
    const int32_t per = (R + kThreads - 1) / kThreads;
    const int32_t r0 = min(R, tid * per), r1 = min(R, r0 + per);
    const int32_t next = *a.free_next;
    int32_t bad = 0;
    int64_t tokens = 0, blocks = 0;
    for (int32_t r = r0; r < r1; ++r) {
        const int32_t c = a.cached[r], n = a.fresh[r];
        had[r] = c;
        if (c < 0 || n < 0 || (int64_t)c + n > (int64_t)a.max_blocks * kBlockSize) {
            bad |= kErrStaticSeqLen;
            continue;
        }
        tokens += n;
        blocks += (c + n + kBlockSize - 1) / kBlockSize - (c + kBlockSize - 1) / kBlockSize;
    }
    int64_t at_tok, at_blk, all_tok, all_blk;
    block_scan2(tokens, blocks, part, at_tok, at_blk, all_tok, all_blk);
    if (next < 0 || next + all_blk > a.num_free) bad |= kErrNoBlocks;
    if (all_tok > a.num_slots) bad |= kErrNoSlots;
    for (int32_t r = r0; r < r1; ++r) {
        const int32_t c = had[r], n = a.fresh[r];
        start[r] = (int32_t)at_tok;
        first[r] = (int32_t)(next + at_blk);
        if (c < 0 || n < 0 || (int64_t)c + n > (int64_t)a.max_blocks * kBlockSize) continue;
        at_tok += n;
        at_blk += (c + n + kBlockSize - 1) / kBlockSize - (c + kBlockSize - 1) / kBlockSize;
    }
    if (tid == 0) start[R] = (int32_t)all_tok;
    // the sums may only be used to index when no length was refused
    if (bad) atomicOr(&bits, bad);
    __syncthreads();
    bad = bits;

    // Request, position and block id of token t (left alone behind the last one).
    // The searches for the warp's first and last token bound each lane's own.
    const int32_t total = (int32_t)all_tok;
    auto slot_of = [&](int32_t t, int32_t& row, int32_t& col, int32_t& id) {
        const int32_t t0 = t - lane;
        const int32_t lo = find_request(start, min(t0, total - 1), 0, R - 1);
        const int32_t hi = find_request(start, min(t0 + 31, total - 1), lo, R - 1);
        if (t >= total) return;
        const int32_t r = find_request(start, t, lo, hi);
        const int32_t c = had[r], p = c + (t - start[r]), j = p / kBlockSize, h = (c + kBlockSize - 1) / kBlockSize;
        id = j < h ? a.bt[(int64_t)r * a.max_blocks + j] : a.free_blocks[first[r] + j - h];
        row = r;
        col = p;
    };
    const int32_t stride = ranks * kThreads, t_first = rank * kThreads + tid;
    int32_t k_row[kKeep], k_col[kKeep], k_id[kKeep];
    if (!bad) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            k_row[i] = -1;
            const int64_t t = t_first + (int64_t)i * stride;
            if (t - lane < total) {
                slot_of((int32_t)t, k_row[i], k_col[i], k_id[i]);
                if (k_row[i] >= 0 && (k_id[i] < 0 || k_id[i] >= a.num_blocks)) bad |= kErrStaticBlockId;
            }
        }
        for (int64_t t = t_first + (int64_t)kKeep * stride; t - lane < total; t += stride) {
            int32_t row = -1, col = 0, id = 0;
            slot_of((int32_t)t, row, col, id);
            if (row >= 0 && (id < 0 || id >= a.num_blocks)) bad |= kErrStaticBlockId;
        }
    }
    __syncthreads();             // (everyone has read `bits`)
    if (bad) atomicOr(&bits, bad);
    __syncthreads();
    if (tid < ranks) *cluster.map_shared_rank(&verdict[rank], tid) = bits;
    cluster.sync();
    bad = 0;
    for (int i = 0; i < ranks; ++i) bad |= verdict[i];

    for (int32_t r = rank * kThreads + tid; r <= R; r += stride) {
        a.q_starts[r] = bad ? 0 : start[r];
        if (r < R) a.seq_lens[r] = bad ? had[r] : had[r] + start[r + 1] - start[r];
    }
    if (rank == 0 && tid == 0) {
        *a.free_after = bad ? next : next + (int32_t)all_blk;
        if (bad && a.err) atomicOr(a.err, bad);
    }
    if (bad) {
        for (int64_t t = t_first; t < a.num_slots; t += stride) a.slots[t] = -1;
        return;
    }
    auto put = [&](int32_t t, int32_t row, int32_t col, int32_t id) {
        a.slots[t] = row < 0 ? -1 : id * kBlockSize + col % kBlockSize;
        if (row >= 0 && col % kBlockSize == 0) a.bt[(int64_t)row * a.max_blocks + col / kBlockSize] = id;
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int64_t t = t_first + (int64_t)i * stride;
        if (t < a.num_slots) put((int32_t)t, k_row[i], k_col[i], k_id[i]);
    }
    for (int64_t t = t_first + (int64_t)kKeep * stride; t - lane < a.num_slots; t += stride) {
        int32_t row = -1, col = 0, id = 0;
        if (t - lane < total) slot_of((int32_t)t, row, col, id);
        if (t < a.num_slots) put((int32_t)t, row, col, id);
    }
}

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace fca

using namespace fca;

extern "C" fca_status fca_extend_tables(int32_t* block_tables, int32_t max_blocks, const int32_t* cached_lens,
                                        const int32_t* new_lens, int32_t num_requests, const int32_t* free_blocks,
                                        int32_t num_free, const int32_t* free_next, int32_t num_blocks,
                                        int32_t* seq_lens, int32_t* q_starts, int32_t* slots, int32_t num_slots,
                                        int32_t* free_after, int32_t* dev_status, void* stream) {
    if (num_requests < 0 || max_blocks < 1 || num_blocks < 1 || num_free < 0 || num_slots < 0 || !free_next ||
        !free_after || !q_starts || (num_slots > 0 && !slots) || (num_free > 0 && !free_blocks) ||
        (num_requests > 0 && (!block_tables || !cached_lens || !new_lens || !seq_lens)))
        return FCA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)cached_lens, (const void*)new_lens,
                          (const void*)free_blocks, (const void*)free_next, (const void*)seq_lens,
                          (const void*)q_starts, (const void*)slots, (const void*)free_after, (const void*)dev_status})
        if (!aligned4(p)) return FCA_ERR_INVALID_ARG;
    if (seq_lens != cached_lens && overlap(seq_lens, 4 * (size_t)num_requests, cached_lens, 4 * (size_t)num_requests))
        return FCA_ERR_INVALID_ARG;
    if (num_requests > kMaxRequests || (int64_t)num_blocks * kBlockSize > INT32_MAX ||
        (int64_t)max_blocks * kBlockSize > INT32_MAX)
        return FCA_ERR_UNSUPPORTED;
    TablesArgs a;
    a.bt = block_tables;
    a.cached = cached_lens;
    a.fresh = new_lens;
    a.free_blocks = free_blocks;
    a.free_next = free_next;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.slots = slots;
    a.free_after = free_after;
    a.err = dev_status;
    a.R = num_requests;
    a.max_blocks = max_blocks;
    a.num_free = num_free;
    a.num_blocks = num_blocks;
    a.num_slots = num_slots;
    const size_t smem = (3 * (size_t)num_requests + 1) * sizeof(int32_t);
    cudaError_t e = cudaFuncSetAttribute(k_extend_tables, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((3 * (size_t)kMaxRequests + 1) * sizeof(int32_t)));
    if (note_cuda(e) != cudaSuccess) {
        (void)cudaGetLastError();
        return FCA_ERR_CUDA;
    }
    // One CTA while its threads hold every slot between check and write.
    const int ctas = num_slots <= kKeep * kThreads ? 1 : kCluster;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (note_cuda(cudaLaunchKernelEx(&cfg, k_extend_tables, a)) != cudaSuccess) {
        (void)cudaGetLastError();
        return FCA_ERR_CUDA;
    }
    return FCA_OK;
}

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
// The work is a megabyte or two at most and bound by latency and, with many
// tokens, by the instructions of the lookups.  Every CTA sums all the lengths and checks
// all the ids that would be used itself (a few tens of kilobytes from L2), so that
// each comes to the same verdict -- everything is written or nothing -- without an exchange.
// The tokens are dealt out over the warps of all CTAs.  Small steps are one CTA and
// one launch; there, lengths and list position are written behind a barrier, all
// CTA's reads done, and may be updated in place.  Large ones leave those two to a second
// launch of one CTA (2048 prompts, 262144 tokens: 129 us with the tokens' slots found
// by a search each on a cluster of 8 CTAs, 47 us with the lookup below, and 10.8 us over
// 148 CTAs; a decode step of 256 requests takes 6.0 us).
#include <algorithm>

#include "fca_internal.h"

namespace fca {
namespace {

constexpr int kThreads = 1024;
constexpr int kWide = 4;        // tokens a lane has under way at once
constexpr int32_t kMaxSlots = 1 << 30;      // (places of slots are added to in 32 bits)

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
    int32_t lengths;             // whether this launch writes seq_lens and free_after
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
    __shared__ int32_t bits;
    const int rank = blockIdx.x, ranks = gridDim.x;
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

    // the ids that would be used: the list's, and the last blocks that get more tokens
    const int32_t total = (int32_t)all_tok;
    const int32_t stride = ranks * kThreads, mine = rank * kThreads + tid;
    if (!bad) {
        for (int64_t x = tid; x < all_blk; x += kThreads) {
            const int32_t id = a.free_blocks[next + x];
            if (id < 0 || id >= a.num_blocks) bad = kErrStaticBlockId;
        }
        for (int32_t r = tid; r < R; r += kThreads) {
            if (had[r] % kBlockSize == 0 || start[r + 1] == start[r]) continue;
            const int32_t id = a.bt[(int64_t)r * a.max_blocks + had[r] / kBlockSize];
            if (id < 0 || id >= a.num_blocks) bad = kErrStaticBlockId;
        }
    }
    __syncthreads();             // (everyone has read `bits`)
    if (bad) atomicOr(&bits, bad);
    __syncthreads();
    bad = bits;

    for (int32_t r = mine; r <= R; r += stride) {
        a.q_starts[r] = bad ? 0 : start[r];
        if (a.lengths && r < R) a.seq_lens[r] = bad ? had[r] : had[r] + start[r + 1] - start[r];
    }
    if (rank == 0 && tid == 0) {
        if (a.lengths) *a.free_after = bad ? next : next + (int32_t)all_blk;
        if (bad && a.err) atomicOr(a.err, bad);
    }
    if (bad) {
        for (int64_t t = mine; t < a.num_slots; t += stride) a.slots[t] = -1;
        return;
    }
    // Each warp takes a stretch of the slots, kWide tokens a lane at a time.  The request
    // of a window of 32 tokens is found by stepping over the next 32 starts at once: a
    // search from scratch per token costs twenty times the instructions.
    const int32_t windows = (a.num_slots + 31) / 32, warps = stride / 32, warp = mine / 32;
    const int32_t w0 = (int32_t)((int64_t)windows * warp / warps), w1 = (int32_t)((int64_t)windows * (warp + 1) / warps);
    int32_t r_cur = w0 < w1 && w0 * 32 < total ? find_request(start, w0 * 32, 0, R - 1) : 0;
    for (int32_t w = w0; w < w1; w += kWide) {
        int32_t row[kWide], pos[kWide], id[kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
            const int32_t t0 = (w + i) * 32, t = t0 + lane;
            row[i] = -1;
            if (w + i >= w1 || t0 >= total) continue;
            const int32_t t_last = min(t0 + 31, total - 1);
            int32_t next_start, n;
            do {                                   // the request that holds t0
                next_start = start[min(R, r_cur + 1 + lane)];
                n = __popc(__ballot_sync(0xffffffffu, r_cur + 1 + lane < R && next_start <= t0));
                r_cur += n;
            } while (n == 32);
            if (n) next_start = start[min(R, r_cur + 1 + lane)];
            int32_t r = r_cur;
            n = __popc(__ballot_sync(0xffffffffu, r_cur + 1 + lane < R && next_start <= t_last));
            if (n == 32)                           // (many requests without tokens)
                r = find_request(start, min(t, t_last), r_cur, R - 1);
            else
                for (int k = 0; k < n; ++k) r += t >= __shfl_sync(0xffffffffu, next_start, k);
            if (t >= total) continue;
            const int32_t c = had[r], p = c + (t - start[r]), j = p / kBlockSize, h = (c + kBlockSize - 1) / kBlockSize;
            row[i] = r;
            pos[i] = p;
            id[i] = j < h ? a.bt[(int64_t)r * a.max_blocks + j] : a.free_blocks[first[r] + j - h];
        }
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
            const int64_t t = (int64_t)(w + i) * 32 + lane;
            if (w + i >= w1 || t >= a.num_slots) continue;
            a.slots[t] = row[i] < 0 ? -1 : id[i] * kBlockSize + pos[i] % kBlockSize;
            // a block's first position is new exactly when the block is
            if (row[i] >= 0 && pos[i] % kBlockSize == 0) a.bt[(int64_t)row[i] * a.max_blocks + pos[i] / kBlockSize] = id[i];
        }
    }
}

// The lengths and the list position of a large step, from the rows that it was given.
__global__ void __launch_bounds__(kThreads, 1) k_extend_lengths(TablesArgs a) {
    __shared__ int64_t part[kThreads / 32][2];
    int64_t blocks = 0;
    for (int32_t r = threadIdx.x; r < a.R; r += kThreads) {
        const int32_t c = a.cached[r], n = a.q_starts[r + 1] - a.q_starts[r];
        if (n > 0) blocks += (c + n + kBlockSize - 1) / kBlockSize - (c + kBlockSize - 1) / kBlockSize;
        a.seq_lens[r] = c + n;
    }
    int64_t x, y, all, none;
    block_scan2(blocks, 0, part, x, y, all, none);
    if (threadIdx.x == 0) *a.free_after = *a.free_next + (int32_t)all;
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
    if (num_requests > kMaxRequests || (int64_t)num_blocks * kBlockSize > INT32_MAX ||
        (int64_t)max_blocks * kBlockSize > INT32_MAX || num_slots > kMaxSlots)
        return FCA_ERR_UNSUPPORTED;
    // What one CTA writes others may still have to read: outputs, the first six, stand alone.
    const size_t r = (size_t)num_requests;
    const struct { const int32_t* at; size_t n; } buf[10] = {
        {block_tables, r * max_blocks}, {seq_lens, r}, {q_starts, r + 1}, {slots, (size_t)num_slots},
        {free_after, 1}, {dev_status, dev_status ? 1u : 0u}, {cached_lens, r}, {new_lens, r},
        {free_blocks, (size_t)num_free}, {free_next, 1}};
    for (int x = 0; x < 6; ++x)
        for (int y = x + 1; y < 10; ++y) {
            const bool in_place = buf[x].at == buf[y].at && ((x == 1 && y == 6) || (x == 4 && y == 9));
            if (!in_place && overlap(buf[x].at, 4 * buf[x].n, buf[y].at, 4 * buf[y].n)) return FCA_ERR_INVALID_ARG;
        }
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
    // (only what the default limit does not cover asks for more)
    cudaError_t e = smem <= 32 * 1024 ? cudaSuccess
                                      : cudaFuncSetAttribute(k_extend_tables, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                             (int)((3 * (size_t)kMaxRequests + 1) * sizeof(int32_t)));
    if (note_cuda(e) != cudaSuccess) {
        (void)cudaGetLastError();
        return FCA_ERR_CUDA;
    }
    // One CTA while a warp has one round of slots at most (a second launch costs as much as two or
    // three rounds: 19000 slots take 33 us on one CTA, 12.9 us on 5, 8.4 us on 19); else a
    // window a warp, up to one CTA per SM.
    const int64_t want = num_slots <= kWide * kThreads ? 1 : ((int64_t)num_slots + kThreads - 1) / kThreads;
    const int ctas = (int)std::min<int64_t>(want, 148);
    a.lengths = ctas == 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    k_extend_tables<<<ctas, kThreads, smem, s>>>(a);
    if (ctas > 1 && cudaPeekAtLastError() == cudaSuccess) k_extend_lengths<<<1, kThreads, 0, s>>>(a);
    if (note_cuda(cudaGetLastError()) != cudaSuccess) return FCA_ERR_CUDA;
    return FCA_OK;
}

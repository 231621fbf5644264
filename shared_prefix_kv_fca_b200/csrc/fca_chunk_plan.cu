// Plans of the chunk attention: checks, copies of tables and lengths, and the
// work lists, built on the device.
//
// The rows of a request that read one KV head -- n tokens x G query heads -- are
// stacked and cut into tiles of 256.  Tile i of a request with L cached tokens
// sees the first l_i = L - n + ceil(256 (i + 1) / G) of them (the last tile L),
// that is ceil(l_i / 128) stages, and costs so much for each stage and for itself.  All tiles
// of the step, in the order (request, KV head, tile), form one line of
// cost W; CTA c gets the stretch [c Q, (c + 1) Q), Q = W / CTAs.  So every CTA has the
// same work to within a stage, whatever the mix of long and short requests, and
// only tiles on a boundary are cut, at most one per CTA: their pieces write
// partial rows to two fixed slots per CTA, which bounds the workspace by the
// number of SMs instead of by the batch.
//
// Where a tile begins on the line needs the sum of its predecessors' stage
// counts.  Within a request that is a sum of floor((a i + b) / m) over i, which
// has a logarithmic-time recurrence (Euclid's algorithm on a and m), so each tile
// finds its own place: no pass over tiles, no sort.
#include <algorithm>
#include <new>

#include "fca_chunk.h"
#include "fca_device.cuh"

namespace fca {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kListThreads = 256;
constexpr int kSegment = 1024;      // table entries a copy unit
constexpr int kListShared = 4096;   // requests whose offsets the list kernel keeps in shared memory

struct ChunkPlanArgs {
    const int32_t* bt_in;
    const int32_t* seq_in;
    const int32_t* qs_in;
    int32_t R, T, max_blocks, num_blocks, Hkv, G, ctas, full;
    int32_t tile_ctas;              // CTAs of the list kernel that place tiles; the others copy tables
    int32_t* bt;
    int32_t* seq;
    int32_t* qs;
    int32_t* bad;
    int32_t* tile_off;
    int64_t* cost_off;
    int32_t* begin;
    int32_t* end;
    ChunkItem* items;
    ChunkCut* cuts;
    ChunkHeader* hdr;
    int32_t* status;
};

// sum over i in [0, n) of floor((a i + b) / m); a, b, n >= 0, m >= 1; T holds a n + b.
template <typename T>
__device__ int64_t floor_sum_in(T n, T m, T a, T b) {
    int64_t s = 0;
    while (n > 0) {
        if (a >= m) {
            s += (int64_t)(n - 1) * n / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            s += (int64_t)n * (b / m);
            b %= m;
        }
        const T y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const T t = m;
        m = a;
        a = t;
    }
    return s;
}

__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    // (a 64-bit division takes five times a 32-bit one, and the sums are on the way of every launch)
    if (a * n + b < INT32_MAX) return floor_sum_in<uint32_t>((uint32_t)n, (uint32_t)m, (uint32_t)a, (uint32_t)b);
    return floor_sum_in<int64_t>(n, m, a, b);
}

__device__ __forceinline__ int32_t tiles_of(int32_t n, int32_t G) {
    return (int32_t)(((int64_t)n * G + kChunkRows - 1) / kChunkRows);
}

__device__ __forceinline__ int32_t stages_for(int64_t tokens) {
    return (int32_t)((tokens + kChunkStage - 1) / kChunkStage);
}

// Cost of a request's tiles [0, i) of one KV head, i below its tile count (so that all are full).
__device__ int64_t cost_before(int32_t i, int32_t n, int32_t L, int32_t G, bool whole) {
    const int64_t m = (int64_t)kChunkStage * G;
    const int64_t stages = whole ? (int64_t)i * stages_for(L)
                                 : floor_sum(i, m, kChunkRows, (int64_t)(L - n) * G + kChunkRows + m - 1);
    return stages * kChunkStageCost + (int64_t)i * kChunkTileCost;
}

// Cost of a tile of `rows` rows and ns stages.
__device__ __forceinline__ int64_t tile_cost(int64_t rows, int32_t ns) {
    return rows > kChunkRows / 2 ? (int64_t)ns * kChunkStageCost + kChunkTileCost
                                 : (int64_t)ns * kChunkHalfStageCost + kChunkHalfTileCost;
}

// Cost of all of a request's tiles of one KV head.
__device__ __forceinline__ int64_t head_cost(int32_t n, int32_t L, int32_t G, bool whole) {
    const int32_t nt = tiles_of(n, G);
    return cost_before(nt - 1, n, L, G, whole) + tile_cost((int64_t)n * G - (int64_t)(nt - 1) * kChunkRows, stages_for(L));
}

// Lengths checked and copied; tiles and cost before each request; the CTA's
// share.  One CTA: the sums need all requests.
__global__ void __launch_bounds__(kScanThreads) k_chunk_scan(ChunkPlanArgs a) {
    __shared__ int64_t part[32][2];
    __shared__ int32_t status;
    dev::pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t R = a.R, per = (R + kScanThreads - 1) / kScanThreads;
    const int32_t r0 = min(R, tid * per), r1 = min(R, r0 + per);
    if (tid == 0) status = 0;
    __syncthreads();
    // the rows' ranges first: if they are wrong there is no step at all
    int32_t bits = 0;
    if (tid == 0 && (a.qs_in[0] != 0 || a.qs_in[R] > a.T)) bits = kErrStaticSeqLen;
    for (int32_t r = r0; r < r1; ++r)
        if (a.qs_in[r + 1] < a.qs_in[r]) bits = kErrStaticSeqLen;
    const bool refused = __syncthreads_or(bits) != 0;

    int64_t tiles = 0, cost = 0;
    int64_t head = 0;           // the last request's cost, the only one of most threads
    for (int32_t r = r0; r < r1; ++r) {
        const int32_t q0 = a.qs_in[r], n = refused ? 0 : a.qs_in[r + 1] - q0;
        int32_t L = a.seq_in[r];
        if (L < 0 || L > a.max_blocks * kBlockSize || (!a.full && L < n)) {
            bits |= kErrStaticSeqLen;
            L = 0;
        }
        if (n == 0) L = 0;
        a.seq[r] = L;
        a.qs[r] = refused ? 0 : q0;
        a.bad[r] = 0;
        if (n > 0) {
            tiles += (int64_t)tiles_of(n, a.G) * a.Hkv;
            head = head_cost(n, L, a.G, a.full || L == 0);
            cost += a.Hkv * head;
        }
    }
    if (bits) atomicOr(&status, bits);
    int64_t st = tiles, sc = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ut = __shfl_up_sync(0xffffffffu, st, o), uc = __shfl_up_sync(0xffffffffu, sc, o);
        if (lane >= o) {
            st += ut;
            sc += uc;
        }
    }
    if (lane == 31) {
        part[warp][0] = st;
        part[warp][1] = sc;
    }
    __syncthreads();
    int64_t before_t = 0, before_c = 0, W = 0, N = 0;
    for (int w = 0; w < 32; ++w) {
        if (w == warp) {
            before_t = N;
            before_c = W;
        }
        N += part[w][0];
        W += part[w][1];
    }
    int64_t at_t = before_t + st - tiles, at_c = before_c + sc - cost;
    for (int32_t r = r0; r < r1; ++r) {
        a.tile_off[r] = (int32_t)at_t;
        a.cost_off[r] = at_c;
        const int32_t n = refused ? 0 : a.qs_in[r + 1] - a.qs_in[r], L = a.seq[r];
        if (n > 0) {
            at_t += (int64_t)tiles_of(n, a.G) * a.Hkv;
            at_c += a.Hkv * (r + 1 == r1 ? head : head_cost(n, L, a.G, a.full || L == 0));
        }
    }
    const int64_t quota = max((W + a.ctas - 1) / a.ctas, (int64_t)(2 * kChunkMinPiece * kChunkHalfStageCost + kChunkHalfTileCost));
    const int32_t used = (int32_t)((W + quota - 1) / quota);
    if (tid < a.ctas) {
        a.cuts[tid].nrows = 0;
        // the inner boundaries are set by the tiles that they fall into
        if (tid == 0 || tid >= used) a.begin[tid] = 0;
        if (tid >= used) a.end[tid] = 0;
        if (tid == used - 1) a.end[tid] = (int32_t)N + used - 1;
    }
    if (tid == 0) {
        a.tile_off[R] = (int32_t)N;
        a.cost_off[R] = W;
        a.qs[R] = refused ? 0 : a.qs_in[R];
        a.hdr->work = W;
        a.hdr->quota = quota;
        a.hdr->status = status;
        a.hdr->n_tiles = (int32_t)N;
        a.hdr->n_ctas = used;
        a.hdr->n_cuts = 0;
        if (status) atomicOr(a.status, status);
    }
}

// One thread places one tile; the last CTAs copy and check the tables.
__global__ void __launch_bounds__(kListThreads) k_chunk_lists(ChunkPlanArgs a) {
    dev::pdl_wait();
    if ((int32_t)blockIdx.x >= a.tile_ctas) {
        const int32_t segs = (a.max_blocks + kSegment - 1) / kSegment;
        const int64_t units = (int64_t)a.R * segs;
        for (int64_t u = blockIdx.x - a.tile_ctas; u < units; u += gridDim.x - a.tile_ctas) {
            const int32_t r = (int32_t)(u / segs), j0 = (int32_t)(u % segs) * kSegment;
            const int32_t nb = min((a.seq[r] + kBlockSize - 1) / kBlockSize, j0 + kSegment);
            bool bad = false;
            for (int32_t j = j0 + threadIdx.x; j < nb; j += kListThreads) {
                const int64_t at = (int64_t)r * a.max_blocks + j;
                int32_t b = a.bt_in[at];
                if (b < 0 || b >= a.num_blocks) {
                    bad = true;
                    b = a.num_blocks;      // reads as zeros
                }
                a.bt[at] = b;
            }
            if (bad) {
                a.bad[r] = 1;
                atomicOr(&a.hdr->status, kErrStaticBlockId);
                atomicOr(a.status, kErrStaticBlockId);
            }
        }
        return;
    }
    __shared__ int32_t offs[kListShared];
    const int32_t N = a.hdr->n_tiles;
    const int64_t Q = a.hdr->quota;
    const int32_t used = a.hdr->n_ctas;
    const int32_t t = blockIdx.x * kListThreads + threadIdx.x;
    if ((int32_t)blockIdx.x * kListThreads >= N) return;
    const int32_t* off = a.tile_off;
    if (a.R <= kListShared) {               // a search in shared memory instead of L2
        for (int32_t r = threadIdx.x; r < a.R; r += kListThreads) offs[r] = a.tile_off[r];
        off = offs;
        __syncthreads();
    }
    if (t >= N) return;
    int32_t lo = 0, hi = a.R - 1;           // the last request whose tiles begin at or before t
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (off[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int32_t r = lo, q0 = a.qs[r], n = a.qs[r + 1] - q0, L = a.seq[r], G = a.G;
    const bool whole = a.full || L == 0;    // every row sees all L
    const int32_t nt = tiles_of(n, G), head = (t - a.tile_off[r]) / nt, i = (t - a.tile_off[r]) % nt;
    const int64_t s = a.cost_off[r] + head * head_cost(n, L, G, whole) + cost_before(i, n, L, G, whole);
    const int64_t row0 = (int64_t)i * kChunkRows, row1 = min(row0 + kChunkRows, (int64_t)n * G);
    const int32_t seen = whole ? L : (int32_t)((L - n) + (row1 + G - 1) / G);
    const int32_t ns = stages_for(seen);
    const int64_t e = s + tile_cost(row1 - row0, ns);
    const bool half = row1 - row0 <= kChunkRows / 2;
    const int64_t own = half ? kChunkHalfTileCost : kChunkTileCost, per_stage = half ? kChunkHalfStageCost : kChunkStageCost;

    ChunkItem it;
    it.req = r;
    it.head = head;
    it.q0 = q0 + (int32_t)(row0 / G);
    it.rem = (int32_t)(row0 % G);
    it.nrows = (int32_t)(row1 - row0);
    it.lim0 = whole ? L : L - n + (int32_t)(row0 / G);
    it.pad0 = it.pad1 = it.pad2 = 0;

    // Walk the boundaries c Q inside [s, e).  One that would leave a piece under
    // kChunkMinPiece stages moves to the tile's end on that side.
    int32_t owner = s == 0 ? 0 : (int32_t)((s + Q - 1) / Q) - 1;
    int32_t k = 0, first_cut = 0, last_cut = 0;
    for (int32_t c = max(1, (int32_t)((s + Q - 1) / Q)); c < used && (int64_t)c * Q < e; ++c) {
        const int64_t x = max((int64_t)0, (int64_t)c * Q - s - own) / per_stage;     // the boundary's stage
        int32_t next = t, prev_end = t;                             // tiles on the two sides
        if (x < kChunkMinPiece) {
            prev_end = t - 1;
        } else if (ns - x < kChunkMinPiece) {
            next = t + 1;
        } else {
            it.tok0 = k * kChunkStage;
            it.tok1 = (int32_t)x * kChunkStage;
            it.slot = 2 * owner + (k == 0 ? 1 : 0);
            a.items[t + owner] = it;
            k = (int32_t)x;
            if (!first_cut) first_cut = c;
            last_cut = c;
        }
        a.begin[c] = next + c;
        a.end[c - 1] = prev_end + c;
        // behind a boundary moved to the tile's end the tile still belongs to `owner`
        if (next == t) owner = c;
    }
    it.tok0 = k * kChunkStage;
    it.tok1 = seen;
    it.slot = first_cut ? 2 * owner : -1;
    a.items[t + owner] = it;
    if (first_cut) {
        ChunkCut cut;
        cut.cta0 = first_cut - 1;
        cut.cta1 = last_cut;
        cut.q0 = it.q0;
        cut.rem = it.rem;
        cut.nrows = it.nrows;
        cut.head = head;
        cut.pad0 = cut.pad1 = 0;
        a.cuts[first_cut] = cut;
        atomicAdd(&a.hdr->n_cuts, 1);
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Places the plan's arrays behind one another; returns the bytes they take.
size_t place(fca_chunk_plan_s* P, uint8_t* base) {
    size_t at = 0;
    auto put = [&](auto** p, size_t count) {
        *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + at);
        at += align256(std::max<size_t>(count, 1) * sizeof(**p));
    };
    const size_t R = P->R, C = P->ctas;
    put(&P->dev_status, 1);
    put(&P->hdr, 1);
    put(&P->bt, R * P->max_blocks);
    put(&P->seq, R);
    put(&P->qs, R + 1);
    put(&P->bad, R);
    put(&P->tile_off, R + 1);
    put(&P->cost_off, R + 1);
    put(&P->begin, C);
    put(&P->end, C);
    put(&P->items, (size_t)P->cap_items);
    put(&P->cuts, C);
    put(&P->part_o, 2 * C * P->part_rows * P->D);
    put(&P->part_w, 2 * C * P->part_rows);
    return at;
}

cudaError_t build_lists(const fca_chunk_plan_s* P, const int32_t* bt, const int32_t* seq, const int32_t* qs,
                        cudaStream_t stream) {
    ChunkPlanArgs a;
    a.bt_in = bt;
    a.seq_in = seq;
    a.qs_in = qs;
    a.R = P->R;
    a.T = P->T;
    a.max_blocks = P->max_blocks;
    a.num_blocks = P->num_blocks;
    a.Hkv = P->Hkv;
    a.G = P->G;
    a.ctas = P->ctas;
    a.full = P->full;
    a.bt = P->bt;
    a.seq = P->seq;
    a.qs = P->qs;
    a.bad = P->bad;
    a.tile_off = P->tile_off;
    a.cost_off = P->cost_off;
    a.begin = P->begin;
    a.end = P->end;
    a.items = P->items;
    a.cuts = P->cuts;
    a.hdr = P->hdr;
    a.status = P->dev_status;
    a.tile_ctas = (int32_t)((P->cap_items + kListThreads - 1) / kListThreads);
    const int64_t units = (int64_t)P->R * ((P->max_blocks + kSegment - 1) / kSegment);
    const int copy_ctas = (int)std::min<int64_t>(units, 148 * 8);
    k_chunk_scan<<<1, kScanThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // set up while the scan runs, which it waits for
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.tile_ctas + copy_ctas);
    cfg.blockDim = dim3(kListThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_chunk_lists, a);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace fca

using namespace fca;

extern "C" {

fca_status fca_chunk_plan_destroy(fca_chunk_plan_t plan) {
    if (!plan) return FCA_OK;
    DeviceGuard dg(plan->device);
    if (plan->base) {
        // the memory goes back to the pool once nothing that may read it still runs
        cudaDeviceSynchronize();
        cudaFreeAsync(plan->base, cudaStreamLegacy);
        cudaStreamSynchronize(cudaStreamLegacy);
        (void)cudaGetLastError();
    }
    delete plan;
    return FCA_OK;
}

fca_status fca_chunk_plan(const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                          const int32_t* q_starts, int32_t num_requests, int32_t num_tokens, int32_t block_size,
                          int32_t num_blocks, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                          uint32_t flags, fca_chunk_plan_t* out_plan, void* stream) {
    if (!out_plan) return FCA_ERR_INVALID_ARG;
    *out_plan = nullptr;
    if (!block_tables || !seq_lens || !q_starts || num_requests < 1 || num_tokens < 0 || max_blocks < 1 ||
        num_blocks < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        (flags & ~FCA_CHUNK_FULL) || !aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(q_starts))
        return FCA_ERR_INVALID_ARG;
    const int32_t G = num_q_heads / num_kv_heads;
    if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128) || G > kMaxGqa ||
        num_requests > kMaxRequests || max_blocks > (1 << 20) || (int64_t)num_blocks * kBlockSize > INT32_MAX)
        return FCA_ERR_UNSUPPORTED;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int32_t ctas = std::min(sms, kChunkMaxCtas);
    const int64_t rows = (int64_t)num_tokens * G;
    const int64_t cap = num_kv_heads * (rows / kChunkRows + num_requests) + ctas + 1;
    if (rows > INT32_MAX || cap > (1 << 24)) return FCA_ERR_UNSUPPORTED;
    fca_chunk_plan_s* P = new (std::nothrow) fca_chunk_plan_s();
    if (!P) return FCA_ERR_OOM;
    P->device = dev;
    P->R = num_requests;
    P->T = num_tokens;
    P->max_blocks = max_blocks;
    P->num_blocks = num_blocks;
    P->Hq = num_q_heads;
    P->Hkv = num_kv_heads;
    P->D = head_dim;
    P->G = G;
    P->full = (flags & FCA_CHUNK_FULL) != 0;
    P->ctas = ctas;
    P->cap_items = cap;
    P->part_rows = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kChunkRows, rows));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t bytes = place(P, nullptr);
    cudaMemPool_t pool = nullptr;
    cudaError_t e = plan_pool(&pool);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&P->base, bytes, pool, s);
    if (e != cudaSuccess) {
        note_cuda(e);
        (void)cudaGetLastError();
        P->base = nullptr;
        delete P;
        return e == cudaErrorMemoryAllocation ? FCA_ERR_OOM : FCA_ERR_CUDA;
    }
    place(P, static_cast<uint8_t*>(P->base));
    ChunkHeader h{};
    e = cudaMemsetAsync(P->dev_status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = build_lists(P, block_tables, seq_lens, q_starts, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&h, P->hdr, sizeof(h), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(P->dev_status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    fca_status st = FCA_OK;
    if (e != cudaSuccess) {
        note_cuda(e);
        (void)cudaGetLastError();
        st = FCA_ERR_CUDA;
    } else if (h.status & kErrStaticSeqLen) {
        st = FCA_ERR_INVALID_ARG;
    } else if (h.status & kErrStaticBlockId) {
        st = FCA_ERR_BAD_BLOCK_ID;
    }
    if (st != FCA_OK) {
        fca_chunk_plan_destroy(P);
        return st;
    }
    P->may_cut = h.n_cuts > 0;
    *out_plan = P;
    return FCA_OK;
}

fca_status fca_chunk_plan_update(fca_chunk_plan_t plan, const int32_t* block_tables, int32_t max_blocks,
                                 const int32_t* seq_lens, const int32_t* q_starts, int32_t num_requests,
                                 void* stream) {
    if (!plan || !block_tables || !seq_lens || !q_starts || max_blocks != plan->max_blocks ||
        num_requests != plan->R || !aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(q_starts))
        return FCA_ERR_INVALID_ARG;
    DeviceGuard dg(plan->device);
    if (note_cuda(build_lists(plan, block_tables, seq_lens, q_starts, static_cast<cudaStream_t>(stream))) != cudaSuccess)
        return FCA_ERR_CUDA;
    plan->may_cut = true;
    return FCA_OK;
}

fca_status fca_chunk_check_status(fca_chunk_plan_t plan, void* stream, int32_t* code) {
    if (!plan) return FCA_ERR_INVALID_ARG;
    DeviceGuard dg(plan->device);
    int32_t v = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpy(&v, plan->dev_status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(plan->dev_status, 0, sizeof(v)) != cudaSuccess) {
        (void)cudaGetLastError();
        return FCA_ERR_CUDA;
    }
    if (code) *code = v;
    return v ? FCA_ERR_DEVICE_FLAG : FCA_OK;
}

}  // extern "C"

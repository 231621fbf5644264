// fca_chunk_attention: the rows of new tokens over the paged cache, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Row (token t of request r, query head h) at position p = L - n + i:
//   s_j = scale q.k_j,  o = sum_{j <= p} exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m)
// over the cached tokens j that the row sees (all L of them in full plans), in one
// pass over the tokens with a running reference m and running sums.
//
// The rows of a request that read one KV head (tokens x query heads of the
// group) are stacked, so that a K or V stage in shared memory serves them
// all.  A CTA walks its items of the plan (fca_chunk_plan.cu); an item is up to
// 256 stacked rows against a range of tokens, 128 tokens a stage:
//   - above 128 rows: two MMA tiles of 128 rows share every stage, each with its
//     own weights and accumulator, so that the softmax of one tile runs while
//     the tensor core works for the other;
//   - up to 128 rows ("dual"): one tile's rows, but its even and odd stages go
//     to the two halves of the machinery, whose accumulators are joined at
//     the end: few rows are bound by the cache's bytes, and the softmax of a
//     stage (a row is one thread) takes longer than the bytes do.
//
// 384 threads:
//   warps 0-3, 4-7  the warpgroups of tile 0 and tile 1, one thread a row: for
//                each stage they read the scores from tensor memory into
//                registers and write the weights back as bf16; the accumulator is
//                rescaled in place in the rare case that a row's maximum
//                outgrows its reference; at the item's end they normalise and store.
//                Two row sums: of the rounded weights, by which out is divided, and
//                of those before rounding, for lse;
//   warps 8, 9   TMA loads of K, and of V and the queries; one block of 16
//                tokens, or 16 stacked query rows, a box;
//   warps 10, 11 MMA issue: S = Q K^T (operands in shared memory), and
//                O += P V (P from tensor memory).
// Tensor memory holds one score buffer, two weight buffers and two
// accumulators.  The tiles take turns with the scores: a softmax warp copies its
// row of 128 scores to registers and gives the buffer up before it computes
// anything, so that the other tile's Q K^T, and this tile's next, never wait for an
// exponential or a P V.  (With a score buffer per tile and the weights
// written over the scores, a tile's next Q K^T had to wait for its P V:
// 5300 cycles a stage of 256 x 128 instead of then 3300.)
//
// What bounds it.  A stage of 256 x 128 at head_dim 128 needs 2048 tensor cycles,
// 2048 cycles of exponentials (16 a cycle and SM) and 2048 of shared-memory reads,
// and takes 3400 (3300 without the sum of rounded weights): the softmax of the two
// tiles, two warps a scheduler, takes 2350 by itself without that sum.  Where the rest goes
// is not known in full; a second score buffer, which head_dim 64 has room for, gained
// nothing.  Measured: 4096 tokens behind 32768 (32/8/128) 1.99 ms, 1175 TFLOP/s (71% of the
// measured burst rate; 2.37 ms in runs of seconds, at the clock that power leaves); 16 prompts
// of 2048 630 us, 872 TFLOP/s: an item's start and end cost 3.5 us.  Dual items are
// bound by the cache's bytes: 192 x 5 drafted tokens behind 1500-8000 (3.8 GB) 6.4 TB/s, 98% of
// the copy rate; 64 x 5, of which 1024 shared (0.85 GB), 5.2 TB/s, with 15 us of start and
// end.  Tried and slower: exponentials partly by a polynomial on the FMA pipe; 16 softmax
// warps of 64 columns; one warp issuing both products in order; P handed over in halves.
//
// Every wait is bounded (fca_device.cuh); a role that gives up sets the CTA's
// abort flag, the others leave at their next wait, copies and MMAs in flight
// are waited for, and tensor memory is freed.  A parity tells a phase from the
// next one only: whoever waits on a barrier either holds its next phase up or
// is the only one to wait, so that none can fall two phases behind.
#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>

#include "fca_chunk.h"
#include "fca_device.cuh"

namespace fca {
namespace {

constexpr int kStage = kChunkStage;
constexpr int kBlkPerStage = kStage / kBlockSize;
constexpr int kThreads = 384;
constexpr int kKWarp = 8, kVWarp = 9, kQKWarp = 10;
// Registers a thread: the three warpgroups' shares add up to the launch's.
constexpr int kRegsLaunch = 168;
constexpr int kRegsTile = 208, kRegsOthers = 88;
static_assert(2 * kRegsTile + kRegsOthers == 3 * kRegsLaunch, "register shares");
// A row's exponentials are taken against a reference that follows its running
// maximum only when that is 2^8 above it: the accumulator is rescaled in few stages, and
// weights up to 2^8 are as exact in bf16 and fp32 as those up to 1.
constexpr float kRescaleLog2 = 8.f;
constexpr float kLn2 = 0.69314718055994531f;

struct ChunkArgs {
    const ChunkItem* items;
    const int32_t* begin;
    const int32_t* end;
    const int32_t* bad;
    const int32_t* bt;
    const __nv_bfloat16* q;
    int64_t q_stride;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;
    float* part_w;
    int32_t part_rows, max_blocks, num_blocks, T, Hq, Hkv, G;
    uint32_t div_g;     // 65536 / G, rounded up: x / G = x div_g >> 16 for x < kChunkRows + 16
    int32_t q_tma;      // queries by TMA, 16 stacked rows a box: G divides 16
    float scale_log2;
    int32_t* err;
};

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;               // 128-byte swizzle atoms a row
    static constexpr int kTileQ = 128 * D * 2;
    static constexpr int kKV = kStage * D * 2;           // one K or V stage
    static constexpr int kKSlots = D == 128 ? 3 : 5;
    static constexpr int kVSlots = D == 128 ? 2 : 5;
    static constexpr int kOffQ = 0;                      // two tiles
    static constexpr int kOffK = kOffQ + 2 * kTileQ;
    static constexpr int kOffV = kOffK + kKSlots * kKV;
    static constexpr int kOffML = kOffV + kVSlots * kKV; // [3][128] f32: tile 1's row references and sums, for tile 0
    static constexpr int kOffBar = kOffML + 3 * 128 * 4;
    static constexpr int kNumBars = 2 * (kKSlots + kVSlots) + 5 * 2 + 4;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kAlloc = kOffMisc + 32;
    static constexpr uint32_t kColS = 0;                 // scores: 128 fp32 columns
    static constexpr uint32_t kColP = 128;               // tile t's weights: 64 columns of bf16 pairs at 128 + 64 t
    static constexpr uint32_t kColO = 256;               // tile t's accumulator: D columns at 256 + D t
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kColO + 2 * D <= kTmemCols, "tensor memory budget");
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

// An item and what every role derives from it.
struct Work {
    ChunkItem it;
    int32_t ns;         // stages
    int32_t ns0, ns1;   // stages of tile 0 and 1
    bool dual;          // one tile of rows, stages dealt out to both
};

__device__ __forceinline__ int32_t over_g(const ChunkArgs& a, int32_t x) { return (int32_t)((uint32_t)x * a.div_g >> 16); }

// Tokens below which stacked row `row` of the item sees.
__device__ __forceinline__ int32_t row_limit(const ChunkArgs& a, const ChunkItem& it, int32_t row) {
    return min(it.tok1, it.lim0 + over_g(a, it.rem + row) + 1);
}

// Row of q (and of out, in heads) that stacked row `row` is.
__device__ __forceinline__ int32_t row_token(const ChunkArgs& a, const ChunkItem& it, int32_t row, int32_t& qhead) {
    const int32_t x = it.rem + row, t = over_g(a, x);
    qhead = it.head * a.G + x - t * a.G;
    return it.q0 + t;
}

__device__ __forceinline__ Work load_work(const ChunkArgs& a, int32_t i) {
    const int4* p = reinterpret_cast<const int4*>(a.items + i);
    const int4 x = __ldg(p), y = __ldg(p + 1), z = __ldg(p + 2);
    Work w;
    w.it.req = x.x;
    w.it.head = x.y;
    w.it.q0 = x.z;
    w.it.rem = x.w;
    w.it.nrows = y.x;
    w.it.tok0 = y.y;
    w.it.tok1 = y.z;
    w.it.lim0 = y.w;
    w.it.slot = z.x;
    if (__ldg(a.bad + x.x)) w.it.tok1 = w.it.tok0;       // a refused request sees nothing
    w.ns = (w.it.tok1 - w.it.tok0 + kStage - 1) / kStage;
    w.dual = w.it.nrows <= 128;
    if (w.dual) {
        w.ns0 = (w.ns + 1) / 2;
        w.ns1 = w.ns / 2;
    } else {
        // tile 1 holds the item's last row and has all its stages
        w.ns0 = (max(0, row_limit(a, w.it, 127) - w.it.tok0) + kStage - 1) / kStage;
        w.ns1 = w.ns;
    }
    return w;
}

// Byte offset of 16-byte chunk c (< 8) of row r in 64-element atom `atom` of
// a K-major, 128-byte swizzled tile of 128 rows.
__device__ __forceinline__ uint32_t sw128_off(int r, int atom, int c) {
    return atom * (128 * 128) + (r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// mbar_wait by a warp whose lanes go on together.  When a wait is given up (its limit, or the
// abort flag) just as the phase completes, lanes may come back with different answers: all of
// them leave then, since one that went on alone would wait for the others in the next vote,
// without a limit.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err_word) {
    return __all_sync(0xffffffffu, dev::mbar_wait(bar, parity, abort, err_word));
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Waits for this thread's tensor-memory loads; the registers are named so that
// no use of them can be moved before the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&x)[32], uint32_t (&y)[32]) {
    dev::tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        asm volatile("" : "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]));
        asm volatile("" : "+r"(y[i]), "+r"(y[i + 1]), "+r"(y[i + 2]), "+r"(y[i + 3]));
    }
}

__device__ __forceinline__ float as_f(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ void max32(const uint32_t (&x)[32], float& a, float& b) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        a = dev::max3(a, as_f(x[i]), as_f(x[i + 1]));
        b = dev::max3(b, as_f(x[i + 2]), as_f(x[i + 3]));
    }
}

// Weights of 32 scores against the reference (nm = -m): 16 bf16 pairs, and their sum
// before rounding (for lse).
__device__ __forceinline__ void weights32(const uint32_t (&x)[32], float2 sc, float2 nm, uint32_t* p, float2& sum) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 z = dev::fma2(make_float2(as_f(x[i]), as_f(x[i + 1])), sc, nm);
        const float2 e = make_float2(dev::ex2(z.x), dev::ex2(z.y));
        p[i / 2] = dev::pack_bf16x2(e.x, e.y);
        sum = dev::add2(sum, e);
    }
}

// The sum of 64 weights as they were rounded, which is what P V applies: out divided by it stays a
// weighted mean of V.  (Divided by the sum before rounding, a row whose weight sits on one token
// would be off by that weight's rounding, up to 2^-8, in all elements at once.)  Taken behind the
// weights' hand-over, while the tile waits for its next scores, by adds that read a bf16 as it
// lies: 16 prompts of 2048 take 632 us, 603 without this sum, 640 with it among the exponentials,
// 652 with pairs unpacked and added two at a time, 723 with warp products.
__device__ __forceinline__ float rounded_sum(const uint32_t (&p)[32]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        dev::add_bf16x2(s[0], s[1], p[i]);
        dev::add_bf16x2(s[2], s[3], p[i + 1]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Whether V has an inf or NaN in tokens [tok0, tok1), by one warp.
template <int D>
__device__ __noinline__ bool v_not_finite(const ChunkArgs& a, int32_t req, int32_t head, int32_t tok0, int32_t tok1) {
    float x = 0.f;
    for (int32_t j = tok0; j < tok1; ++j) {
        const int32_t b = a.bt[(int64_t)req * a.max_blocks + j / kBlockSize];
        const int64_t at = (((int64_t)b * kBlockSize + j % kBlockSize) * a.Hkv + head) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x = fmaf(__bfloat162float(a.v[at + (threadIdx.x & 31) + 32 * i]), 0.f, x);
    }
    return __any_sync(0xffffffffu, isnan(x));
}

// Rows row0 + i of item `item`, for the bits i of `rows`, by one warp with plain arithmetic, from the
// tokens that they see; the results are written over what is there.  Does nothing where V is finite
// in all that some of them do not see: then they are what they should be.  Rows are taken
// kExactRows at a time and tokens 32 at a time, a lane a token for the scores: 256 stacked rows of 30000
// tokens on every SM at once take 48 ms (512 ms a row at a time).
constexpr int kExactRows = 8;

template <int D>
__device__ __noinline__ void exact_rows(const ChunkArgs& a, int32_t item, int row0, uint32_t rows) {
    constexpr int E = D / 32, N = kExactRows;
    const int lane = threadIdx.x & 31;
    const ChunkItem it = load_work(a, item).it;
    if (!v_not_finite<D>(a, it.req, it.head, max(it.tok0, row_limit(a, it, row0 + __ffs(rows) - 1)), it.tok1)) return;
    while (rows) {
        int r[N];                               // (the last one again where there are fewer)
        int32_t lim[N];
        const __nv_bfloat16* q[N];
        float o[N][E], m[N], l[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (rows) r[k] = row0 + __ffs(rows) - 1;
            else if (k > 0) r[k] = r[k - 1];
            rows &= rows - 1;
            lim[k] = row_limit(a, it, r[k]);
            int32_t qhead;
            const int32_t tok = row_token(a, it, r[k], qhead);
            q[k] = a.q + (int64_t)tok * a.q_stride + qhead * D;
            m[k] = -INFINITY;
            l[k] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) o[k][i] = 0.f;
        }
        const int32_t end = lim[N - 1];         // limits grow with the row
        for (int32_t j0 = it.tok0; j0 < end; j0 += 32) {
            const int32_t j = min(j0 + lane, end - 1);
            const int32_t b = a.bt[(int64_t)it.req * a.max_blocks + j / kBlockSize];
            const int64_t at = (((int64_t)b * kBlockSize + j % kBlockSize) * a.Hkv + it.head) * D;
            float s[N];
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 kx = *reinterpret_cast<const uint4*>(a.k + at + c * 8);
                const uint32_t kw[4] = {kx.x, kx.y, kx.z, kx.w};
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const uint4 qx = *reinterpret_cast<const uint4*>(q[k] + c * 8);
                    const uint32_t qw[4] = {qx.x, qx.y, qx.z, qx.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[k] = fmaf(as_f(kw[e] << 16), as_f(qw[e] << 16), s[k]);
                        s[k] = fmaf(as_f(kw[e] & 0xffff0000u), as_f(qw[e] & 0xffff0000u), s[k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                s[k] = j0 + lane < lim[k] ? s[k] * a.scale_log2 : -INFINITY;
                float top = s[k];
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(m[k], top);
                const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m[k] - ref);
                s[k] = exp2f(s[k] - ref);       // the token's weight
                m[k] = top;
                float sum = s[k];
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[k] = l[k] * f + sum;
#pragma unroll
                for (int i = 0; i < E; ++i) o[k][i] *= f;
            }
            const int n = min(32, end - j0);
#pragma unroll 4
            for (int y = 0; y < n; ++y) {
                const __nv_bfloat16* v = a.v + __shfl_sync(0xffffffffu, at, y) + lane * E;
                float vf[E];
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    const uint32_t vx = *reinterpret_cast<const uint32_t*>(v + i);
                    vf[i] = as_f(vx << 16);
                    vf[i + 1] = as_f(vx & 0xffff0000u);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float w = __shfl_sync(0xffffffffu, s[k], y);
#pragma unroll
                    for (int i = 0; i < E; ++i) o[k][i] = j0 + y < lim[k] ? fmaf(w, vf[i], o[k][i]) : o[k][i];
                }
            }
        }
        __syncwarp();                           // behind what the rows' own lanes wrote
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int32_t qhead;
            const int32_t tok = row_token(a, it, r[k], qhead);
            const int64_t orow = (int64_t)tok * a.Hq + qhead, prow = (int64_t)it.slot * a.part_rows + r[k];
            const float inv = l[k] == 0.f ? 0.f : 1.f / l[k], lw = m[k] + log2f(l[k]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (it.slot < 0)
                    a.out[orow * D + lane * E + i] = __float2bfloat16(o[k][i] * inv);
                else
                    a.part_o[prow * D + lane * E + i] = o[k][i] * inv;
            }
            if (lane == 0) {
                if (it.slot >= 0)
                    a.part_w[prow] = lw;
                else if (a.lse)
                    a.lse[orow] = lw * kLn2;
            }
        }
    }
}

// Whether a lane's row, as it was stored, has an inf or NaN.
template <int D>
__device__ __forceinline__ bool not_finite(const ChunkArgs& a, const ChunkItem& it, int32_t row) {
    bool bad = false;
    if (it.slot < 0) {
        int32_t qhead;
        const int32_t tok = row_token(a, it, row, qhead);
        const __nv_bfloat16* const p = a.out + ((int64_t)tok * a.Hq + qhead) * D;
#pragma unroll 8
        for (int e = 0; e < D; ++e) bad |= !(fabsf(__bfloat162float(p[e])) < INFINITY);
    } else {
        const float* const p = a.part_o + ((int64_t)it.slot * a.part_rows + row) * D;
#pragma unroll 8
        for (int e = 0; e < D; ++e) bad |= !(fabsf(p[e]) < INFINITY);
    }
    return bad;
}

// The rows that are not finite among a warp's rows row0 + lane of all the CTA's items.  A warp comes here
// behind its last item, when it has arrived at every barrier that others wait for: however long it
// takes, no wait with a limit runs meanwhile.
template <int D>
__device__ __noinline__ void exact_items(const ChunkArgs& a, int32_t first, int32_t last, int row0) {
    for (int32_t i = first; i < last; ++i) {
        const ChunkItem it = load_work(a, i).it;
        const int r = row0 + (threadIdx.x & 31);
        const uint32_t again = __ballot_sync(0xffffffffu, r < it.nrows && not_finite<D>(a, it, r));
        if (again) exact_rows<D>(a, i, row0, again);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap tmK,
            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
    using L = Layout<D>;
    dev::pdl_launch_dependents();           // the merge may be set up
    const int32_t first = a.begin[blockIdx.x], last = a.end[blockIdx.x];
    if (first >= last) return;

    extern __shared__ __align__(1024) uint8_t smem[];    // the swizzled operands want 1024-byte alignment
    if (dev::smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrBadItem);
        return;
    }
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);   // [slots] a K slot holds its stage
    uint64_t* k_empty = k_full + L::kKSlots;   // [slots] the products of both tiles reading it have completed
    uint64_t* v_full = k_empty + L::kKSlots;   // [slots]
    uint64_t* v_empty = v_full + L::kVSlots;   // [slots]
    uint64_t* q_full = v_empty + L::kVSlots;   // [2] a query tile is written
    uint64_t* q_free = q_full + 2;             // [2] the last products reading it have completed
    uint64_t* s_full = q_free + 2;             // [2] a stage's scores of the tile are there
    uint64_t* s_free = s_full + 2;             // ... and copied
    uint64_t* p_full = s_free + 1;             // [2] the tile's weights are written
    uint64_t* pv_done = p_full + 2;            // [2] the P V reading them has completed
    uint64_t* x_full = pv_done + 2;            // tile 1's row state of a dual item is written
    uint64_t* x_free = x_full + 1;             // ... and it and the accumulator are read
    uint64_t* mma_done = x_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 16);
    float* ml = reinterpret_cast<float*>(smem + L::kOffML);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kKSlots; ++s) {
            dev::mbar_init(&k_full[s], 1);
            dev::mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < L::kVSlots; ++s) {
            dev::mbar_init(&v_full[s], 1);
            dev::mbar_init(&v_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            dev::mbar_init(&q_full[t], a.q_tma ? 1 : 128);
            dev::mbar_init(&q_free[t], 1);
            dev::mbar_init(&s_full[t], 1);
            dev::mbar_init(&p_full[t], 128);
            dev::mbar_init(&pv_done[t], 1);
        }
        dev::mbar_init(s_free, 128);
        dev::mbar_init(x_full, 128);
        dev::mbar_init(x_free, 128);
        dev::mbar_init(mma_done, 2);
        *abort_flag = 0;
        dev::fence_mbarrier_init();
    }
    if (warp == kQKWarp) {
        dev::tmem_alloc(tmem_slot, L::kTmemCols);
        dev::tmem_relinquish();
    }
    dev::tc_fence_before();
    __syncthreads();
    dev::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < kKWarp) {
        // ------------------------------------------------ a tile's warpgroup
        regs_inc<kRegsTile>();
        const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + L::kColS, p_addr = tmem + lane_base + L::kColP + t * 64,
                       o_addr = tmem + lane_base + L::kColO + t * D;
        bool ok = true, redo = false;
        // Where the head group does not divide a tile (else the V warp loads the queries by TMA):
        // queries of tile t for the next item that has some, from item i on (a dual item's go to
        // tile 0), once the products reading the last ones have completed.
        uint32_t n_q = 0;
        auto load_q = [&](int32_t i) {
            if (a.q_tma) return;
            for (; i < last; ++i) {
                const Work w = load_work(a, i);
                if (t ? w.dual || w.ns == 0 : w.ns0 == 0) continue;
                if (n_q) ok = warp_wait(&q_free[t], (n_q - 1) & 1, abort_flag, a.err);
                if (!ok) return;
                ++n_q;
                constexpr int C = D / 8;            // 16-byte chunks a row
                const uint32_t q_tile = dev::smem_u32(smem + L::kOffQ) + t * L::kTileQ;
#pragma unroll 4
                for (int e = row; e < 128 * C; e += 128) {
                    const int r = e / C, c = e % C, ri = t * 128 + r;
                    int32_t qhead;
                    const int32_t tok = row_token(a, w.it, min(ri, w.it.nrows - 1), qhead);
                    cp_async16(q_tile + sw128_off(r, c >> 3, c & 7), a.q + (int64_t)tok * a.q_stride + qhead * D + c * 8,
                               ri < w.it.nrows ? 16u : 0u);
                }
                cp_async_wait();
                dev::fence_proxy_async_smem();
                dev::mbar_arrive(&q_full[t]);
                return;
            }
        };
        load_q(first);
        uint32_t g = 0, g_other = 0;    // stages of this tile, and of the other, before the item
        uint32_t n_dual = 0;            // items joined from both tiles
        for (int32_t i = first; ok && i < last; ++i) {
            int32_t ns, ns_other, ns_item, lim, n_hot;
            bool dual, live;
            {   // (only what the stages need is kept: the scores take up the registers)
                const Work w = load_work(a, i);
                ns = t ? w.ns1 : w.ns0;
                ns_other = t ? w.ns0 : w.ns1;
                ns_item = w.ns;
                dual = w.dual;
                const int r_item = w.dual ? row : t * 128 + row;         // stacked row within the item
                live = (w.dual ? quarter * 32 : t * 128 + quarter * 32) < w.it.nrows;
                lim = row_limit(a, w.it, min(r_item, w.it.nrows - 1)) - w.it.tok0;   // tokens of the item it sees
                // stages of which every row of this warp sees all
                const int32_t all = max(0, __reduce_min_sync(0xffffffffu, lim)) / kStage;
                n_hot = min(ns, w.dual ? (all - t + 1) >> 1 : all);
            }
            float m = -INFINITY, l = 0.f, lr = 0.f;     // reference (log2 domain), sums of the weights and of the rounded ones
            // Before a stage's first weights: the P V of the tile's stage before has read
            // the last ones.
            auto weights_free = [&]() -> bool {
                const bool up = g == 0 || warp_wait(&pv_done[t], (g - 1) & 1, abort_flag, a.err);
                dev::tc_fence_after();
                return up;
            };
            // Stage x.  In an edge stage (x >= n_hot) some row of the warp does not see all
            // 128 columns: those are set to -inf where they lie first, in a short loop, so that
            // the stage itself is one body of code for all (instructions that run once
            // an item come from far: a second body with masks cost 3500 cycles an item).
            auto stage = [&](int32_t x) -> bool {
                const int32_t j = dual ? 2 * x + t : x;
                if (!warp_wait(&s_full[t], g & 1, abort_flag, a.err)) return false;
                dev::tc_fence_after();
                if (x >= n_hot) {
                    const int nv = lim - j * kStage;             // columns that the row sees
                    const int low = __reduce_min_sync(0xffffffffu, nv), high = __reduce_max_sync(0xffffffffu, nv);
#pragma unroll 1
                    for (int c = max(0, low) / 16 * 16; c < kStage; c += 16) {
                        uint32_t y[16];
                        if (c < high) {
                            dev::tmem_ld16(s_addr + c, y);
                            dev::tc_wait_ld();
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            asm volatile("" : "+r"(y[e]));
                            y[e] = c + e < nv ? y[e] : 0xff800000u;
                        }
                        dev::tmem_st16(s_addr + c, y);
                    }
                    dev::tc_wait_st();
                }
                uint32_t s0[32], s1[32], s2[32], s3[32];
                dev::tmem_ld32(s_addr, s0);
                dev::tmem_ld32(s_addr + 32, s1);
                dev::tmem_ld32(s_addr + 64, s2);
                dev::tmem_ld32(s_addr + 96, s3);
                wait_ld(s0, s1);
                wait_ld(s2, s3);
                dev::tc_fence_before();
                dev::mbar_arrive(s_free);
                float mx = -INFINITY, my = -INFINITY, mz = -INFINITY, mw = -INFINITY;
                max32(s0, mx, my);
                max32(s1, mz, mw);
                max32(s2, mx, my);
                max32(s3, mz, mw);
                mx = fmaxf(dev::max3(mx, my, mz), mw) * a.scale_log2;        // the scale is positive
                float f = 1.f;
                if (mx > m + kRescaleLog2) {
                    f = dev::ex2(m - mx);
                    l *= f;
                    lr *= f;
                    m = mx;
                }
                // (an item's first P V overwrites the accumulator)
                if (x > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                    if (!weights_free()) return false;           // that P V has brought the accumulator up to date
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t ov[16];
                        dev::tmem_ld16(o_addr + c * 16, ov);
                        dev::tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            asm volatile("" : "+r"(ov[e]));
                            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                        }
                        dev::tmem_st16(o_addr + c * 16, ov);
                    }
                }
                const float m0 = m == -INFINITY ? 0.f : m;       // nothing seen yet: every weight is 2^-inf
                const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(-m0, -m0);
                float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                uint32_t p[32], p2[32];
                weights32(s0, sc, nm, p, sum);
                weights32(s1, sc, nm, p + 16, sum2);
                if (!weights_free()) return false;
                dev::tmem_st32(p_addr, p);
                weights32(s2, sc, nm, p2, sum);
                weights32(s3, sc, nm, p2 + 16, sum2);
                dev::tmem_st32(p_addr + 32, p2);
                sum = dev::add2(sum, sum2);
                l += sum.x + sum.y;
                dev::tc_wait_st();
                dev::tc_fence_before();
                dev::mbar_arrive(&p_full[t]);
                lr += rounded_sum(p) + rounded_sum(p2);      // while the tile waits for its next scores
                return true;
            };
            int32_t x = 0;
            if (live) {
#pragma unroll 1
                for (; ok && x < ns; ++x, ++g) ok = stage(x);
            } else {
                // rows that do not exist: the barriers only
#pragma unroll 1
                for (; ok && x < ns; ++x, ++g) {
                    ok = warp_wait(&s_full[t], g & 1, abort_flag, a.err);
                    if (!ok) break;
                    dev::mbar_arrive(s_free);
                    ok = weights_free();
                    if (ok && x == 0) {
                        // what an earlier item left there is cleared, for the same reason as unused query rows
                        uint32_t z[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) z[e] = 0u;
                        dev::tmem_st32(p_addr, z);
                        dev::tmem_st32(p_addr + 32, z);
                        dev::tc_wait_st();
                        dev::tc_fence_before();
                    }
                    if (ok) dev::mbar_arrive(&p_full[t]);
                }
            }
            if (!ok) break;
            g_other += ns_other;
            if (ns && (t == 0 || !dual)) load_q(i + 1);
            if (!ok) break;
            const bool join = dual && ns_item > 1;      // both tiles have stages of the same rows
            if (dual && t == 1) {
                // tile 0 joins the two accumulators
                if (join) {
                    ml[row] = m;
                    ml[128 + row] = l;
                    ml[256 + row] = lr;
                    dev::mbar_arrive(x_full);
                    ok = warp_wait(x_free, n_dual & 1, abort_flag, a.err);
                    ++n_dual;
                }
                continue;
            }
            // ------------------------------------------------ the item's rows
            const Work w = load_work(a, i);
            const int r_item = t * 128 + row;
            const bool mine = r_item < w.it.nrows;
            float c0, c1 = 0.f, lw;             // coefficients of the accumulators; the row's log2 sum
            {
                bool up = ns == 0 || warp_wait(&pv_done[t], (g - 1) & 1, abort_flag, a.err);
                float m1 = -INFINITY, l1 = 0.f, lr1 = 0.f;
                if (join) {
                    up = up && warp_wait(x_full, n_dual & 1, abort_flag, a.err) &&
                         warp_wait(&pv_done[1], (g_other - 1) & 1, abort_flag, a.err);
                    m1 = ml[row];
                    l1 = ml[128 + row];
                    lr1 = ml[256 + row];
                    ++n_dual;
                }
                if (!up) { ok = false; break; }
                dev::tc_fence_after();
                const float M = fmaxf(m, m1), Mf = M == -INFINITY ? 0.f : M;
                const float f0 = dev::ex2(m - Mf), f1 = dev::ex2(m1 - Mf);
                const float sum = l * f0 + l1 * f1, sum_r = lr * f0 + lr1 * f1, inv = sum_r == 0.f ? 0.f : 1.f / sum_r;
                c0 = f0 * inv;
                c1 = f1 * inv;
                lw = M + log2f(sum);            // -inf for a row that saw nothing
            }
            int32_t qhead;
            const int32_t tok = row_token(a, w.it, r_item, qhead);
            const int64_t orow = (int64_t)tok * a.Hq + qhead;
            const int64_t prow = (int64_t)w.it.slot * a.part_rows + r_item;
            const bool whole = w.it.slot < 0;
            float finite = 0.f;                 // NaN once an element is not finite
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                float v[16];
                uint32_t y[16];
                if (ns) {
                    dev::tmem_ld16(o_addr + 16 * c, y);
                    dev::tc_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    asm volatile("" : "+r"(y[e]));
                    v[e] = ns ? as_f(y[e]) * c0 : 0.f;
                }
                if (join) {
                    uint32_t z[16];
                    dev::tmem_ld16(o_addr + D + 16 * c, z);
                    dev::tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        asm volatile("" : "+r"(z[e]));
                        v[e] = fmaf(as_f(z[e]), c1, v[e]);
                    }
                    if (c + 1 == D / 16) {
                        dev::tc_fence_before();
                        dev::mbar_arrive(x_free);
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) finite = fmaf(v[e], 0.f, finite);
                if (mine) {
                    if (whole) {
                        __nv_bfloat16* const bo = a.out + orow * D + 16 * c;
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            *reinterpret_cast<uint4*>(bo + e) =
                                make_uint4(dev::pack_bf16x2(v[e], v[e + 1]), dev::pack_bf16x2(v[e + 2], v[e + 3]),
                                           dev::pack_bf16x2(v[e + 4], v[e + 5]), dev::pack_bf16x2(v[e + 6], v[e + 7]));
                    } else {
                        float* const po = a.part_o + prow * D + 16 * c;
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4*>(po + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
            }
            dev::tc_fence_before();             // (the next item's weights, and so its P V, come behind this)
            if (mine) {
                if (!whole)
                    a.part_w[prow] = lw;
                else if (a.lse)
                    a.lse[orow] = lw * kLn2;
            }
            // A product of weight 0 with an inf or NaN that the row does not see
            // (a later token's) is NaN: a row that is not finite is computed again from
            // the tokens that it does see, if V is not finite in one that it does not.
            redo |= mine && isnan(finite);
        }
        if (ok && __any_sync(0xffffffffu, redo)) exact_items<D>(a, first, last, warp * 32);
    } else {
        regs_dec<kRegsOthers>();
        if (warp == kKWarp || warp == kVWarp) {
            // -------------------------------------------- TMA loads
            // Stage g of the CTA goes to slot g % slots of its ring.  Block ids are
            // read 32 at a time (four stages), a batch ahead.
            const bool is_k = warp == kKWarp;
            const CUtensorMap* tm = is_k ? &tmK : &tmV;
            uint64_t* full = is_k ? k_full : v_full;
            uint64_t* empty = is_k ? k_empty : v_empty;
            const uint32_t NS = is_k ? L::kKSlots : L::kVSlots;
            uint8_t* const ring = smem + (is_k ? L::kOffK : L::kOffV);
            if (lane == 0) dev::tma_prefetch_desc(tm);
            constexpr int kStagesPerBatch = 32 / kBlkPerStage;
            auto fetch = [&](const Work& w, int32_t batch) -> int32_t {
                const int32_t blk = w.it.tok0 / kBlockSize + batch * 32 + lane;
                // past the range: rows beyond the cache, which TMA fills with zeros
                return blk * kBlockSize < w.it.tok1 ? __ldg(a.bt + (int64_t)w.it.req * a.max_blocks + blk) * kBlockSize
                                                    : a.num_blocks * kBlockSize;
            };
            uint32_t g = 0, n_q0 = 0, n_q1 = 0;      // stages, and query tiles, loaded so far
            bool ok = true;
            // The queries of an item go ahead of its first V: the products that read the last
            // ones are done before the slot of that V is free.
            auto load_q = [&](const Work& w) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t& n = b ? n_q1 : n_q0;
                    if (!ok || (b ? w.dual : w.ns0 == 0)) continue;
                    if (lane == 0) {
                        if (n && !dev::mbar_wait(&q_free[b], (n - 1) & 1, abort_flag, a.err))
                            ok = false;
                        else
                            dev::mbar_arrive_expect_tx(&q_full[b], L::kTileQ);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) continue;
                    ++n;
                    // Lane e < 8 loads stacked rows 16 e on.  Boxes without a row of the item are
                    // loaded from rows beyond q, as zeros: products with zeros draw less
                    // power, and the step runs at the clock that power leaves.
                    if (lane < 8) {
                        const int32_t r0 = (w.dual ? 0 : b * 128) + 16 * lane;
                        const int32_t tok = r0 < w.it.nrows ? w.it.q0 + over_g(a, r0) : a.T;
                        for (int hf = 0; hf < L::kHalves; ++hf)
                            dev::tma_load_3d(smem + L::kOffQ + b * L::kTileQ + hf * (128 * 128) + lane * (16 * 128), &tmQ,
                                             &q_full[b], hf * 64, w.it.head * a.G, tok);
                    }
                }
            };
            Work nw = load_work(a, first);
            int32_t nxt = fetch(nw, 0);
            for (int32_t i = first; ok && i < last; ++i) {
                const Work w = nw;
                int32_t cur = nxt;
                if (i + 1 < last) {
                    nw = load_work(a, i + 1);
                    nxt = fetch(nw, 0);             // the next item's first batch, while this one streams
                }
                int32_t more = w.ns > kStagesPerBatch ? fetch(w, 1) : 0;
                if (!is_k && a.q_tma && w.ns) load_q(w);
                if (!ok) break;
                for (int32_t j = 0; j < w.ns; ++j, ++g) {
                    if (j && j % kStagesPerBatch == 0) {
                        cur = more;
                        const int32_t batch = j / kStagesPerBatch + 1;
                        if (batch * kStagesPerBatch < w.ns) more = fetch(w, batch);
                    }
                    // lane e < 8 issues the boxes of the stage's block e
                    const int32_t trow = __shfl_sync(0xffffffffu, cur, (j % kStagesPerBatch) * kBlkPerStage + (lane & 7));
                    const uint32_t s = g % NS;
                    if (lane == 0) {
                        if (g >= NS && !dev::mbar_wait(&empty[s], ((g / NS) - 1) & 1, abort_flag, a.err))
                            ok = false;
                        else
                            dev::mbar_arrive_expect_tx(&full[s], L::kKV);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane < kBlkPerStage) {
                        uint8_t* dst = ring + s * L::kKV + lane * (kBlockSize * 128);
#pragma unroll
                        for (int hf = 0; hf < L::kHalves; ++hf)
                            dev::tma_load_3d(dst + hf * (kStage * 128), tm, &full[s], hf * 64, w.it.head, trow);
                    }
                }
            }
            if (lane == 0) {
                // never leave with copies in flight (each slot's latest load only)
                volatile int never = 0;
                for (uint32_t j = g; j > 0 && j + NS > g; --j)
                    dev::mbar_wait(&full[(j - 1) % NS], ((j - 1) / NS) & 1, &never, a.err);
                if (n_q0) dev::mbar_wait(&q_full[0], (n_q0 - 1) & 1, &never, a.err);
                if (n_q1) dev::mbar_wait(&q_full[1], (n_q1 - 1) & 1, &never, a.err);
            }
        } else {
            // -------------------------------------------- MMA issue
            // The whole warp runs the loop, so that descriptors are computed in uniform
            // registers; one elected thread issues.
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (ok) ok = warp_wait(bar, parity, abort_flag, a.err);
                return ok;
            };
            uint32_t g = 0;                     // stages of the CTA before the item
            Work nxt = load_work(a, first);
            if (warp == kQKWarp) {
                constexpr uint32_t idesc = dev::idesc_bf16_f32(128, kStage, false, false);
                const uint64_t q_desc = dev::smem_desc_sw128(dev::smem_u32(smem + L::kOffQ), 16, 1024);
                const uint64_t k_desc = dev::smem_desc_sw128(dev::smem_u32(smem + L::kOffK), 16, 1024);
                uint32_t n = 0;                 // score tiles so far
                uint32_t loads0 = 0, loads1 = 0;   // query loads so far, by buffer
                for (int32_t i = first; ok && i < last; ++i) {
                    const Work w = nxt;
                    if (i + 1 < last) nxt = load_work(a, i + 1);
                    if (w.ns == 0) continue;
                    if (w.dual || w.ns0) ++loads0;
                    if (!w.dual) ++loads1;
                    for (int32_t j = 0; ok && j < w.ns; ++j) {
                        const uint32_t G = g + j, s = G % L::kKSlots;
                        wait(&k_full[s], (G / L::kKSlots) & 1);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (w.dual ? (j & 1) != t : (t == 0 && j >= w.ns0)) continue;
                            const int b = w.dual ? 0 : t;
                            const int32_t ns_t = w.dual ? w.ns : (t ? w.ns1 : w.ns0);
                            if (j == 0) wait(&q_full[b], ((b ? loads1 : loads0) - 1) & 1);
                            if (n) wait(s_free, (n - 1) & 1);
                            if (!ok) break;
                            dev::tc_fence_after();
                            const uint64_t ad0 = q_desc + ((uint32_t)(b * L::kTileQ) >> 4), bd0 = k_desc + ((s * L::kKV) >> 4);
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < D / 16; ++k) {
                                    const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
                                    dev::tc_mma_ss(tmem + L::kColS, ad0 + off, bd0 + off, idesc, k > 0 ? 1u : 0u);
                                }
                                dev::tc_commit(&s_full[t]);
                                if (j + 1 == ns_t) dev::tc_commit(&q_free[b]);
                            }
                            __syncwarp();
                            ++n;
                        }
                        if (!ok) break;
                        if (elect_one()) dev::tc_commit(&k_empty[s]);
                        __syncwarp();
                    }
                    g += w.ns;
                }
            } else {
                constexpr uint32_t idesc = dev::idesc_bf16_f32(128, D, false, true);
                const uint64_t v_desc = dev::smem_desc_sw128(dev::smem_u32(smem + L::kOffV), kStage * 128, 1024);
                uint32_t c[2] = {0, 0};         // P V so far, by tile
                for (int32_t i = first; ok && i < last; ++i) {
                    const Work w = nxt;
                    if (i + 1 < last) nxt = load_work(a, i + 1);
                    if (w.ns == 0) continue;
                    for (int32_t j = 0; ok && j < w.ns; ++j) {
                        const uint32_t G = g + j, s = G % L::kVSlots;
                        wait(&v_full[s], (G / L::kVSlots) & 1);
                        if (ok && j + 1 == w.ns && w.it.tok1 % kBlockSize) {
                            // The last block's slots behind the range were loaded too and may
                            // hold anything, NaN included: their weights are 0, but 0 x NaN is
                            // not, so V's rows there are cleared.
                            const int r0 = w.it.tok1 - w.it.tok0 - j * kStage, r1 = (r0 + kBlockSize - 1) / kBlockSize * kBlockSize;
                            uint8_t* vs = smem + L::kOffV + s * L::kKV;
                            for (int e = lane; e < (r1 - r0) * 8 * L::kHalves; e += 32) {
                                const int rr = r0 + e / (8 * L::kHalves), c = e % (8 * L::kHalves);
                                *reinterpret_cast<uint4*>(vs + sw128_off(rr, c >> 3, c & 7)) = make_uint4(0, 0, 0, 0);
                            }
                            dev::fence_proxy_async_smem();
                            __syncwarp();
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (w.dual ? (j & 1) != t : (t == 0 && j >= w.ns0)) continue;
                            const int32_t x = w.dual ? j >> 1 : j;
                            const uint64_t bd0 = v_desc + ((s * L::kKV) >> 4);
                            const uint32_t d = tmem + L::kColO + t * D, p = tmem + L::kColP + t * 64;
                            wait(&p_full[t], c[t] & 1);
                            if (!ok) break;
                            dev::tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < kStage / 16; ++k)
                                    dev::tc_mma_ts(d, p + k * 8, bd0 + k * (16 * 128 / 16), idesc, (x == 0 && k == 0) ? 0u : 1u);
                                dev::tc_commit(&pv_done[t]);
                            }
                            __syncwarp();
                            ++c[t];
                        }
                        if (!ok) break;
                        if (elect_one()) dev::tc_commit(&v_empty[s]);
                        __syncwarp();
                    }
                    g += w.ns;
                }
            }
            // every MMA of this warp has retired before tensor memory is freed
            if (elect_one()) dev::tc_commit(mma_done);
            __syncwarp();
            volatile int never = 0;
            dev::mbar_wait(mma_done, 0, &never, a.err);
        }
        __syncwarp();
    }

    dev::tc_fence_before();
    __syncthreads();
    if (warp == kQKWarp) {
        dev::tc_fence_after();
        dev::tmem_dealloc(tmem, L::kTmemCols);
    }
}

// The pieces of a cut tile joined by their weights: a warp a row.
constexpr int kMergeThreads = 256, kMergeSplit = 16;     // CTAs a tile: 2 rows a warp at most

template <int D>
__global__ void __launch_bounds__(kMergeThreads) k_chunk_merge(ChunkArgs a, const ChunkCut* cuts) {
    constexpr int E = D / 32;
    dev::pdl_wait();
    const ChunkCut cut = cuts[blockIdx.x];
    const int lane = threadIdx.x & 31, pieces = cut.cta1 - cut.cta0 + 1;
    for (int32_t row = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5); row < cut.nrows;
         row += kMergeSplit * (kMergeThreads / 32)) {
        auto at = [&](int p) { return (int64_t)(2 * (cut.cta0 + p) + (p == 0 ? 1 : 0)) * a.part_rows + row; };
        float M = -INFINITY;
        for (int p = lane; p < pieces; p += 32) M = fmaxf(M, a.part_w[at(p)]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        if (M == -INFINITY) M = 0.f;
        float o[E], sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int base = 0; base < pieces; base += 32) {
            const int p = base + lane;
            const float f = p < pieces ? dev::ex2(a.part_w[at(p)] - M) : 0.f;
            const int n = min(32, pieces - base);
#pragma unroll 4
            for (int y = 0; y < n; ++y) {
                const float fy = __shfl_sync(0xffffffffu, f, y);
                const float* src = a.part_o + at(base + y) * D + lane * E;
                sum += fy;
                if constexpr (E == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(src);
                    o[0] = fmaf(fy, v.x, o[0]);
                    o[1] = fmaf(fy, v.y, o[1]);
                    o[2] = fmaf(fy, v.z, o[2]);
                    o[3] = fmaf(fy, v.w, o[3]);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(src);
                    o[0] = fmaf(fy, v.x, o[0]);
                    o[1] = fmaf(fy, v.y, o[1]);
                }
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int32_t x = cut.rem + row, t = over_g(a, x);
        const int64_t orow = (int64_t)(cut.q0 + t) * a.Hq + cut.head * a.G + x - t * a.G;
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = dev::pack_bf16x2(o[e] * inv, o[e + 1] * inv);
        if (a.lse && lane == 0) a.lse[orow] = (M + log2f(sum)) * kLn2;
    }
}

template <int D>
cudaError_t launch_chunk(const ChunkArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq, int ctas,
                         cudaStream_t stream) {
    using L = Layout<D>;
    // setmaxnreg hands out what the block was launched with: it has to have been kRegsLaunch a thread
    static std::atomic<bool> checked{false};
    cudaError_t e;
    if (!checked) {
        cudaFuncAttributes at{};
        if ((e = cudaFuncGetAttributes(&at, k_chunk<D>)) != cudaSuccess) return e;
        if (at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        checked = true;
    }
    e = cudaFuncSetAttribute(k_chunk<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    k_chunk<D><<<ctas, kThreads, L::kAlloc, stream>>>(a, tk, tv, tq);
    return cudaGetLastError();
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
    // q is read while rows of out and lse are written already
    const size_t rows = (size_t)plan->T, heads = rows * plan->Hq;
    const size_t cache = (size_t)plan->num_blocks * kBlockSize * plan->Hkv * plan->D * 2;
    const size_t n_out = heads * plan->D * 2, n_lse = lse ? heads * 4 : 0;
    const size_t n_q = ((rows - 1) * q_row_stride + (size_t)plan->Hq * plan->D) * 2;
    if (overlap(out, n_out, lse, n_lse)) return FCA_ERR_INVALID_ARG;
    const struct { const void* at; size_t bytes; } in[3] = {{q, n_q}, {k_cache, cache}, {v_cache, cache}};
    for (const auto& x : in)
        if (overlap(x.at, x.bytes, out, n_out) || overlap(x.at, x.bytes, lse, n_lse)) return FCA_ERR_INVALID_ARG;
    DeviceGuard dg(plan->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap tk, tv;
    if (!make_cache_map(&tk, k_cache, plan->num_blocks, plan->Hkv, plan->D) ||
        !make_cache_map(&tv, v_cache, plan->num_blocks, plan->Hkv, plan->D))
        return FCA_ERR_CUDA;
    ChunkArgs a;
    a.items = plan->items;
    a.begin = plan->begin;
    a.end = plan->end;
    a.bad = plan->bad;
    a.bt = plan->bt;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_row_stride;
    a.k = static_cast<const __nv_bfloat16*>(k_cache);
    a.v = static_cast<const __nv_bfloat16*>(v_cache);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.part_o = plan->part_o;
    a.part_w = plan->part_w;
    a.part_rows = plan->part_rows;
    a.max_blocks = plan->max_blocks;
    a.num_blocks = plan->num_blocks;
    a.T = plan->T;
    a.Hq = plan->Hq;
    a.Hkv = plan->Hkv;
    a.G = plan->G;
    a.div_g = (65536u + plan->G - 1) / plan->G;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.err = plan->dev_status;
    CUtensorMap tq = tk;
    a.q_tma = 16 % plan->G == 0;
    if (a.q_tma && !make_rows_map(&tq, q, plan->T, plan->Hq, plan->D, q_row_stride, plan->G, 16 / plan->G)) return FCA_ERR_CUDA;
    const cudaError_t e = plan->D == 128 ? launch_chunk<128>(a, tk, tv, tq, plan->ctas, s)
                                         : launch_chunk<64>(a, tk, tv, tq, plan->ctas, s);
    if (note_cuda(e) != cudaSuccess) return FCA_ERR_CUDA;
    // A captured attention may run after updates that cut tiles where there are none now.
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (!plan->may_cut && cudaStreamIsCapturing(s, &capture) != cudaSuccess) {
        (void)cudaGetLastError();
        return FCA_ERR_CUDA;
    }
    if (plan->may_cut || capture != cudaStreamCaptureStatusNone) {
        // set up while the tiles run, which it waits for
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(plan->ctas, kMergeSplit);
        cfg.blockDim = dim3(kMergeThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (note_cuda(cudaLaunchKernelEx(&cfg, plan->D == 128 ? k_chunk_merge<128> : k_chunk_merge<64>, a,
                                         (const ChunkCut*)plan->cuts)) != cudaSuccess)
            return FCA_ERR_CUDA;
    }
    return FCA_OK;
}

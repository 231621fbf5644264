// Work lists and plan object of the chunk attention (fca_chunk_plan.cu builds
// them, fca_chunk.cu runs them).  Not part of the C ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fca.h"
#include "fca_internal.h"

namespace fca {

constexpr int kChunkRows = 256;      // stacked query rows a tile: two MMA tiles of 128
constexpr int kChunkStage = 128;     // tokens a pipeline stage
// What a stage and a tile itself (query load, pipeline fill, last P V, storing) cost, in
// units of about 0.25 us: tiles above 128 rows are bound by the softmax and the products, the
// others by the cache's bytes.  A chunk of 1999 tokens (64/8/128) beside 95 decodes takes
// 555 us with equal costs for all stages, 526 us at 4 : 3, 515 us at 8 : 5 and 580 us at 2 : 1
// (head_dim 128, before a second row sum that costs 3% of it; not tried at head_dim 64).
constexpr int kChunkStageCost = 8, kChunkTileCost = 14;
constexpr int kChunkHalfStageCost = 5, kChunkHalfTileCost = 10;
constexpr int kChunkMinPiece = 2;    // fewest stages a tile is cut into
constexpr int kChunkMaxCtas = 256;

// One piece of a tile: `nrows` stacked rows of request `req` and KV head `head`
// over cached tokens [tok0, tok1).  Row i of the tile is row q0 + (rem + i) / G of q,
// query head head * G + (rem + i) % G, and sees tokens below
// min(tok1, lim0 + (rem + i) / G + 1).  A whole tile writes out and lse (slot -1); a piece
// of a cut tile writes its partial rows to `slot`.
struct ChunkItem {
    int32_t req, head, q0, rem;
    int32_t nrows, tok0, tok1, lim0;
    int32_t slot, pad0, pad1, pad2;
};

// A tile that was cut: its pieces are in slot 2 * cta0 + 1 and then 2 * c for
// c in (cta0, cta1].  nrows 0: no record.
struct ChunkCut {
    int32_t cta0, cta1, q0, rem;
    int32_t nrows, head, pad0, pad1;
};

struct ChunkHeader {
    int64_t work;       // total cost
    int64_t quota;      // cost a CTA gets
    int32_t status;     // error bits of the last build
    int32_t n_tiles;
    int32_t n_ctas;     // CTAs with work
    int32_t n_cuts;     // tiles cut
};

}  // namespace fca

struct fca_chunk_plan_s {
    int device = 0;
    int32_t R = 0, T = 0, max_blocks = 0, num_blocks = 0;
    int32_t Hq = 0, Hkv = 0, D = 0, G = 0;
    bool full = false;
    bool may_cut = true;            // whether the lists hold cut tiles, as far as the host knows
    int32_t ctas = 0;               // CTAs the lists are made for
    int32_t part_rows = 0;          // partial rows a slot
    int64_t cap_items = 0;

    int32_t* bt = nullptr;          // [R][max_blocks] copy, ids out of range replaced by num_blocks
    int32_t* seq = nullptr;         // [R] tokens (0 for a refused request)
    int32_t* qs = nullptr;          // [R + 1] first row of each request
    int32_t* bad = nullptr;         // [R] the request's table holds a bad id
    int32_t* tile_off = nullptr;    // [R + 1] tiles before the request
    int64_t* cost_off = nullptr;    // [R + 1] cost before the request
    int32_t* begin = nullptr;       // [ctas] the CTA's items
    int32_t* end = nullptr;         // [ctas]
    fca::ChunkItem* items = nullptr;
    fca::ChunkCut* cuts = nullptr;  // [ctas]
    fca::ChunkHeader* hdr = nullptr;
    int32_t* dev_status = nullptr;
    float* part_o = nullptr;        // [2 ctas][part_rows][D] normalised partial rows
    float* part_w = nullptr;        // [2 ctas][part_rows] log2 of their weights

    void* base = nullptr;           // the one allocation
};

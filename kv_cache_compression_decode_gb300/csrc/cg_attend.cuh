// cg_attend.cuh -- what the attention kernels share: their arguments, the list
// of work that the blocks of a row kernel are dealt, and the launches of the
// shared part and of the joins (sm_103a).
#pragma once

#include <cuda.h>
#include <math.h>

#include "cg_async.cuh"
#include "cg_launch.cuh"

namespace cg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kRows = 16;  // query rows of a row tile

struct Args {
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    const uint32_t *slots, *tables, *lens;
    uint32_t n_slots, n_blocks, n_pool, bshift;
    uint32_t R, nq, g, Hkv;  // requests, query tokens, query heads per KV head, KV heads
    uint32_t P, shared_slot; // shared tokens
    uint32_t nh, ng;         // row kernel: heads that one block takes together (a power of two), groups of them
    uint32_t hlog;           // log2 of nh; a block's warp columns have a head each, or part of its tokens
    uint32_t tlog;           // log2 of the tokens of a tile
    uint32_t rlog;           // log2 of an item's rows
    uint32_t over;           // what a piece's beginning and end cost, in tiles: an item is dealt as that many tiles more
    uint32_t rt;             // items' row ranges of a request
    uint32_t npt;            // row ranges of the whole batch over the shared tokens in the row kernel (0: k_shared has them)
    uint32_t pairs;          // k_shared: pairs of 128-row tiles of the whole batch (0: the row kernel has the shared part)
    uint32_t one;            // k_shared: the batch fits one 128-row tile
    uint32_t n_tc;           // blocks of k_shared
    uint32_t after;          // k_shared: its K and V are made by the kernel before it, which lets it start early
    uint32_t merge_rows;     // rows of a warp of the joins
    uint32_t n_cta;          // blocks of the row kernel
    uint64_t qs[3], os[3];
    float scale2;            // |scale| * log2 e
    uint32_t flip;           // sign bits to flip in q (scale < 0)
    uint32_t *status;
    // workspace
    uint64_t *cum;           // [R + 1] first tile of request r; [R]: tiles of all requests
    uint32_t *tokens;        // [R] tokens of request r (tokens_of)
    // rows of partial results: O [D] and (m, l).  First k_shared's, [piece][2][128];
    // from row part0 on the row kernel's, [piece][column][piece_rows]
    float *part_o;
    float2 *part_ml;
    uint32_t part0;
    uint32_t piece_rows;     // rows of a piece that are stored
};

// Tokens of request r's sequence; 0 for an empty slot and for a request that
// is refused (*bad).
__device__ __forceinline__ uint32_t tokens_of(const Args &a, uint32_t r, bool *bad) {
    const uint32_t s = a.slots ? a.slots[r] : r;
    if (s >= a.n_slots) {
        *bad = true;
        return 0;
    }
    const uint32_t n = a.lens[s];
    // the first query token, which sees n - nq + 1 tokens, has to see all the shared ones
    if (n != 0 && (n > ((uint64_t)a.n_blocks << a.bshift) || (a.P && (uint64_t)n + 1 < (uint64_t)a.P + a.nq))) {
        *bad = true;
        return 0;
    }
    return n;
}

__device__ __forceinline__ uint32_t tiles_of(const Args &a, uint32_t tokens) {
    return (tokens + (1u << a.tlog) - 1u) >> a.tlog;
}
// Places on the work list that an item of `tokens` tokens takes.  (kQuant: k_quant_rows, whose items have a.over places
// more and whose blocks have eight warp columns; k_rows has none more and four.)
template <bool kQuant> __device__ __forceinline__ uint32_t places_of(const Args &a, uint32_t tokens) {
    return tokens ? tiles_of(a, tokens) + (kQuant ? a.over : 0u) : 0u;
}
// Blocks that a list of `total` tiles is dealt to: two tiles each at least.
__device__ __forceinline__ uint64_t shares(const Args &a, uint64_t total) {
    return min((uint64_t)a.n_cta, (total + 1) / 2);
}

// Work list: for each request its row ranges x head groups ("items"), each as
// long as the request's own tokens, then the items of the shared part.  An item
// has a.over places before those of its tiles.  Block c of n takes places
// [c T / n, (c + 1) T / n) of the whole list, so every block has the same share
// whatever the lengths are.  A block's run of tiles of one item is a piece; its
// slot c + item is unique, since along the list each new piece has a larger
// block or a larger item.
struct Piece {
    uint32_t r;        // request; R: the shared part
    uint32_t item;     // number of the item
    uint32_t range, group;
    uint32_t tile0, n; // tiles of the item
    uint32_t of;       // tiles the item has
    uint32_t len;      // tokens in the sequence (request) or P
};

struct Walk {
    uint64_t t, end, base;  // position, end of this block's share, first tile of request r
    uint32_t r;
    const uint32_t *lens;   // tokens of the requests in shared memory, or null
};

// floor(x / y): the numbers are small most of the time, and 64-bit division is long.
__device__ __forceinline__ uint64_t quot(uint64_t x, uint64_t y) {
    return (x | y) >> 32 ? x / y : (uint32_t)x / (uint32_t)y;
}

template <bool kQuant> __device__ __forceinline__ bool next_piece(const Args &a, Walk &w, Piece &p) {
    for (;;) {
        if (w.t >= w.end) return false;
        bool bad = false;
        uint32_t nt = 0, len = 0;  // places of an item of request r
        while (w.r < a.R) {
            len = w.lens ? w.lens[w.r] : tokens_of(a, w.r, &bad);
            nt = len > a.P ? places_of<kQuant>(a, len - a.P) : 0;
            const uint64_t all = (uint64_t)nt * a.rt * a.ng;
            if (w.t < w.base + all) break;
            w.base += all;
            w.r++;
        }
        p.r = w.r;
        if (w.r == a.R) {
            len = a.P;
            nt = places_of<kQuant>(a, a.P);
        }
        if (nt == 0) return false;  // this and the next: lengths that changed under the call leave places over
        const uint64_t at = w.t - w.base;
        const uint32_t local = (uint32_t)quot(at, nt);
        if (w.r == a.R && local >= a.npt * a.ng) return false;
        p.item = w.r * a.rt * a.ng + local;
        p.range = local / a.ng;
        p.group = local - p.range * a.ng;
        const uint32_t from = (uint32_t)(at - (uint64_t)local * nt);
        const uint32_t to = from + (uint32_t)min((uint64_t)(nt - from), w.end - w.t);
        w.t += to - from;
        const uint32_t over = kQuant ? a.over : 0u;
        if (to <= over) continue;  // none of the item's tiles
        p.tile0 = max(from, over) - over;
        p.n = to - over - p.tile0;
        p.of = nt - over;
        p.len = len;
        return true;
    }
}

// This block's share of the work list, found by all of its kThreads threads:
// every thread sums its own run of requests.  misc: a word for each warp and
// two more; lens gets the tokens of up to max_lens requests.  Block 0 writes
// a.cum and a.tokens.
template <uint32_t kThreads, bool kQuant>
__device__ __forceinline__ Walk take_share(const Args &a, uint64_t *misc, uint32_t *lens, uint32_t max_lens) {
    constexpr uint32_t kWarps = kThreads / 32;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t per = (a.R + kThreads - 1) / kThreads;
    const uint32_t r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    const bool keep = a.R <= max_lens;
    uint64_t mine = 0;
    bool bad = false;
    for (uint32_t r = r0; r < r1; r++) {
        const uint32_t n = tokens_of(a, r, &bad);
        if (keep) lens[r] = n;
        if (blockIdx.x == 0) a.tokens[r] = n;
        mine += (uint64_t)(n > a.P ? places_of<kQuant>(a, n - a.P) : 0) * a.rt * a.ng;
    }
    if (bad && blockIdx.x == 0) flag(a.status, CG_ERR_RANGE);
    uint64_t inc = mine;
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(kFull, inc, d);
        if (lane >= d) inc += y;
    }
    if (lane == 31) misc[warp] = inc;
    __syncthreads();
    uint64_t before = inc - mine, own = 0;
    for (uint32_t k = 0; k < kWarps; k++) {
        if (k < warp) before += misc[k];
        own += misc[k];
    }
    const uint64_t total = own + (uint64_t)a.npt * a.ng * places_of<kQuant>(a, a.P);
    if (blockIdx.x == 0) {
        uint64_t at = before;
        for (uint32_t r = r0; r < r1; r++) {
            a.cum[r] = at;
            const uint32_t n = a.tokens[r];  // this thread's own write
            at += (uint64_t)(n > a.P ? places_of<kQuant>(a, n - a.P) : 0) * a.rt * a.ng;
        }
        if (tid == 0) a.cum[a.R] = own;
    }
    const uint64_t n_cta = shares(a, total);
    Walk w;
    w.t = blockIdx.x < n_cta ? quot(blockIdx.x * total, n_cta) : total;
    w.end = blockIdx.x < n_cta ? quot((blockIdx.x + 1ull) * total, n_cta) : total;
    if (mine && w.t >= before && w.t < before + mine) {  // one thread at most
        misc[kWarps] = before;
        misc[kWarps + 1] = r0;
    }
    __syncthreads();
    w.base = w.t < own ? misc[kWarps] : own;
    w.r = w.t < own ? (uint32_t)misc[kWarps + 1] : a.R;
    w.lens = keep ? lens : nullptr;
    return w;
}

// Query row x of an item (of the request, or of the batch in the shared
// part): request, query token, query head.
struct Row {
    uint32_t r, i, h;
    bool valid;
};
__device__ __forceinline__ Row row_of(const Args &a, const Piece &p, uint32_t x, uint32_t head) {
    Row o;
    const uint32_t per = a.nq * a.g;
    if (p.r == a.R) {
        o.r = x / per;
        x -= o.r * per;
        o.valid = o.r < a.R;
    } else {
        o.r = p.r;
        o.valid = x < per;
    }
    o.i = x / a.g;
    o.h = head * a.g + (x - o.i * a.g);
    return o;
}

// log2 of the warp columns of a block of the row kernel
template <bool kQuant> __host__ __device__ constexpr uint32_t columns_log() { return kQuant ? 3 : 2; }

constexpr uint32_t kTcTok = 128, kTcSlots = 5;  // k_shared: tokens of a tile, tiles in flight
constexpr uint32_t kMaxCtas = 304, kMaxTcCtas = 152;  // bounds of the grids that workspaces are sized for: 152 SMs

// The launches of k_shared (a.n_tc is set; a.tables null: block i of the shared tokens is block i of the map; split, bf16
// only: K is the sum of the map's matrices 0 and 2) and of the joins (cg_attend.cu).
cudaError_t launch_shared(uint32_t dtype, uint32_t head_dim, bool split, const CUtensorMap &map, Args &a, int sms, cudaStream_t s);
cudaError_t launch_joins(uint32_t dtype, uint32_t head_dim, bool quant, Args &a, int sms, cudaStream_t s);

// A matrix (channel, row, block, K/V) of 16-bit words, in boxes of `box` channels x `rows` rows; `copies` of them, K and V
// the first two, p->kv_stride apart.
bool make_token_map(const cg_pages *p, const uint16_t *base, uint32_t channels, uint32_t copies, uint32_t box, uint32_t rows,
                    CUtensorMapSwizzle swizzle, CUtensorMap *map);
// What is wrong with a call whatever its pool holds.
bool attention_ok(const cg_pages *p, const cg_attention *a);

}  // namespace cg

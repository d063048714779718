// cg_pages.cu -- page operations on the sequences of a paged pool (sm_103a):
// copy, fork, free, compact.  The tables live on the device; a one-block
// planning kernel turns them into a list of block moves, and one mover
// kernel carries the moves out and writes the new tables.
#include "cg_internal.cuh"
#include "cg_launch.cuh"

namespace cg {
namespace {

constexpr uint32_t kPlanThreads = 512;
constexpr uint32_t kMoveThreads = 256;
constexpr uint32_t kVecs = 8;                    // vectors per lane in one unit of a move
constexpr uint32_t kUnitVecs = 32u * kVecs;      // a warp's unit: 4 KiB with 16-byte vectors

constexpr uint32_t kMaxRowBlocks = 255;  // blocks that check the children's rows beside the plan
static_assert(kMaxRowBlocks <= kMoveThreads, "the mover reads their results a thread to a block");

// Workspace: header, then u32 arrays.  Fork fills per-child entries, compact
// per-move ones; both give the mover (src, dst, rows) lists.
struct PlanWs {
    uint32_t *n_moves;   // header[0]
    uint32_t *held;      // [kMaxRowBlocks] fork: what each row-checking block found
    uint32_t *src, *dst; // [max(n_pool, n_slots)] (fork's destinations are fresh[base])
    uint32_t *rows;      // [n_slots] fork: rows of the move (0: none)
    uint32_t *base;      // [n_slots] fork: the child's first entry in `fresh`
    uint32_t *plen;      // [n_slots] fork: the parent's length
    uint32_t *claimed;   // [n_slots] fork: the slot is a child of this call
    uint32_t *fresh;     // [n_pool] fork: free blocks in ascending order
};

__host__ __device__ inline size_t plan_ws(uint32_t n_pool, uint32_t n_slots, void *ws, PlanWs *w) {
    uint32_t *p = static_cast<uint32_t *>(ws);
    const size_t m = n_pool > n_slots ? n_pool : n_slots;
    size_t o = 64 + 256;
    auto take = [&](size_t n) {
        uint32_t *at = p + o;
        o += n;
        return at;
    };
    PlanWs t;
    t.n_moves = p;
    t.held = p + 64;
    t.src = take(m);
    t.dst = take(m);
    t.rows = take(n_slots);
    t.base = take(n_slots);
    t.plen = take(n_slots);
    t.claimed = take(n_slots);
    t.fresh = take(n_pool);
    if (w) *w = t;
    return round_up(o * 4, 256);
}

// Exclusive sum over the block; *total gets the sum.  Every thread calls it.
template <class N>
__device__ N block_scan(N v, N *total, N *sh) {
    const uint32_t lane = threadIdx.x & 31u, w = threadIdx.x >> 5;
    N x = v;
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const N y = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sh[w] = x;
    __syncthreads();
    if (w == 0) {
        N y = lane < blockDim.x / 32u ? sh[lane] : 0u;
        for (uint32_t d = 1; d < 32; d <<= 1) {
            const N z = __shfl_up_sync(kFull, y, d);
            if (lane >= d) y += z;
        }
        sh[lane] = y;
    }
    __syncthreads();
    const N before = w ? sh[w - 1] : 0u;
    *total = sh[31];
    __syncthreads();
    return before + x - v;
}

struct ForkArgs {
    const uint32_t *parent, *child, *reserve;
    uint32_t n;
};

struct Tab {
    uint32_t *tables, *lens, *refs;
    uint32_t n_slots, n_blocks, n_pool, bshift;
};

// The use counts of blocks 4 tid .. 4 tid + 3 of a run of 2048: bit k set
// where block k is in use (kLive) or free; blocks past the pool are neither.
template <bool kLive>
__device__ __forceinline__ uint32_t use_bits(const Tab &t, uint64_t b) {
    uint32_t v[4];
#pragma unroll
    for (uint32_t k = 0; k < 4; k++) v[k] = b + k < t.n_pool ? t.refs[b + k] : (kLive ? 0u : 1u);
    uint32_t bits = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; k++) bits |= (uint32_t)((v[k] != 0) == kLive) << k;
    return bits;
}
constexpr uint32_t kRun = 4u * kPlanThreads;

// Block 0: check every child, hand out the free blocks, list the tail
// copies.  Any fault leaves n_moves = 0 in the header and nothing changed.
// The other blocks look through the children's rows, a row at a time, for a
// block that is still held; the mover drops the call if one found any.
// The time, 4.6 us, is that of its chain of dependent loads and barriers, so the
// first children, the first run of use counts and the tail blocks are fetched
// beside the checks, by 512 threads (1024, with costlier barriers: 4.8 us).
__global__ void __launch_bounds__(kPlanThreads) k_fork_plan(Tab t, ForkArgs f, PlanWs w, uint32_t *status) {
    let_next_start();
    __shared__ uint32_t sh[32];
    __shared__ uint64_t sh8[32];  // the wanted blocks are summed in 64 bits: each child may ask for up to 2^31
    const uint32_t tid = threadIdx.x, bt = 1u << t.bshift;
    if (blockIdx.x) {
        bool held = false;
        for (uint64_t i = blockIdx.x - 1u; i < f.n; i += gridDim.x - 1u) {
            const uint32_t c = f.child[i];
            if (c >= t.n_slots) continue;  // block 0 refuses the call
            const uint32_t *row = t.tables + (uint64_t)c * t.n_blocks;
#pragma unroll 4
            for (uint64_t k = tid; k < t.n_blocks; k += kPlanThreads) held |= row[k] != CG_NO_BLOCK;
        }
        held = __syncthreads_or(held);
        if (tid == 0) {
            w.held[blockIdx.x - 1u] = held;
            if (held) flag(status, CG_ERR_RANGE);
        }
        return;
    }
    uint32_t fr = use_bits<false>(t, 4u * tid);
    uint32_t p_next = CG_NO_SLOT, c_next = 0, len_next = 0, clen_next = 0, rv_next = 0;
    auto load = [&](uint32_t i) {
        p_next = i < f.n ? f.parent[i] : CG_NO_SLOT;
        c_next = i < f.n ? f.child[i] : 0u;
        rv_next = i < f.n && f.reserve ? f.reserve[i] : 0u;
        len_next = p_next < t.n_slots ? t.lens[p_next] : 0u;
        clen_next = i < f.n && c_next < t.n_slots ? t.lens[c_next] : 0u;
    };
    load(tid);
    for (uint32_t s = tid; s < t.n_slots; s += kPlanThreads) w.claimed[s] = 0;
    __syncthreads();
    uint64_t total = 0;
    bool bad = false;
    for (uint32_t i0 = 0; i0 < f.n; i0 += kPlanThreads) {
        const uint32_t i = i0 + tid;
        uint32_t need = 0, pl = 0, p = CG_NO_SLOT;
        if (i < f.n) {
            if (i0) load(i);
            p = p_next;
            pl = len_next;
            const uint32_t c = c_next;
            if (p != CG_NO_SLOT && p >= t.n_slots) bad = true;
            if (c >= t.n_slots) bad = true;
            else if (clen_next != 0) bad = true;
            else if (atomicExch(&w.claimed[c], 1u) != 0) bad = true;
            const uint64_t rows = (uint64_t)t.n_blocks << t.bshift;
            const uint64_t want = (uint64_t)pl + rv_next;
            if (want > rows) {  // covers pl > rows too
                bad = true;
            } else {
                need = (uint32_t)((want + bt - 1u) >> t.bshift) - (pl >> t.bshift);
                if (pl & (bt - 1u)) w.src[i] = t.tables[(uint64_t)p * t.n_blocks + (pl >> t.bshift)];
            }
        }
        uint64_t sum;
        const uint64_t off = block_scan<uint64_t>(need, &sum, sh8);
        if (i < f.n) {
            w.base[i] = (uint32_t)(total + off);
            w.plen[i] = pl;
            w.rows[i] = pl & (bt - 1u);
        }
        total += sum;
        if (total > t.n_pool) bad = true;
        if (__syncthreads_or(bad)) {
            if (tid == 0) {
                *w.n_moves = 0;
                flag(status, CG_ERR_RANGE);
            }
            return;
        }
    }
    uint32_t found = 0;
    for (uint64_t b0 = 0; b0 < t.n_pool && found < total; b0 += kRun) {
        const uint32_t next = b0 + kRun < t.n_pool ? use_bits<false>(t, b0 + kRun + 4u * tid) : 0u;
        uint32_t sum;
        uint32_t at = found + block_scan<uint32_t>(__popc(fr), &sum, sh);
        for (uint32_t k = 0; k < 4; k++)
            if ((fr >> k) & 1u) {
                if (at < total) w.fresh[at] = (uint32_t)(b0 + 4u * tid + k);
                at++;
            }
        found += sum;
        fr = next;
    }
    if (tid == 0) {
        *w.n_moves = found < total ? 0u : f.n;
        if (found < total) flag(status, CG_ERR_RANGE);
    }
}

// One block: count the blocks in use, pair the ones past that count with the
// holes below it (both in ascending order), move their references.  A run of
// 2048 blocks is counted and scanned in about 3.5 us, and larger pools take one
// scan more a run.
__global__ void __launch_bounds__(kPlanThreads) k_compact_plan(Tab t, uint32_t *remap, PlanWs w) {
    let_next_start();
    __shared__ uint32_t sh[32];
    const uint32_t tid = threadIdx.x;
    uint32_t live = use_bits<true>(t, 4u * tid);
    uint32_t mine = __popc(live), n_live;
#pragma unroll 4
    for (uint64_t b0 = kRun; b0 < t.n_pool; b0 += kRun) mine += __popc(use_bits<true>(t, b0 + 4u * tid));
    block_scan<uint32_t>(mine, &n_live, sh);
    uint32_t movers = 0, holes = 0;
    for (uint64_t b0 = 0; b0 < t.n_pool; b0 += kRun) {
        const uint64_t b = b0 + 4u * tid;
        const uint32_t next = b0 + kRun < t.n_pool ? use_bits<true>(t, b + kRun) : 0u;
        uint32_t mv = 0, ho = 0;
        for (uint32_t k = 0; k < 4; k++) {
            if (b + k >= t.n_pool) break;
            const bool used = (live >> k) & 1u;
            remap[b + k] = used ? (uint32_t)(b + k) : CG_NO_BLOCK;
            if (used && b + k >= n_live) mv |= 1u << k;
            if (!used && b + k < n_live) ho |= 1u << k;
        }
        uint32_t sum;  // both counts in one word: at most 2048 each
        const uint32_t off = block_scan<uint32_t>(__popc(mv) | (__popc(ho) << 16), &sum, sh);
        uint32_t im = movers + (off & 0xFFFFu), ih = holes + (off >> 16);
        for (uint32_t k = 0; k < 4; k++) {
            if ((mv >> k) & 1u) w.src[im++] = (uint32_t)(b + k);
            if ((ho >> k) & 1u) w.dst[ih++] = (uint32_t)(b + k);
        }
        movers += sum & 0xFFFFu;
        holes += sum >> 16;
        live = next;
    }
    __syncthreads();
    movers = min(movers, holes);  // as many of either, unless counts changed under the call
    for (uint32_t i = tid; i < movers; i += kPlanThreads) {
        const uint32_t s = w.src[i], d = w.dst[i];
        remap[s] = d;
        t.refs[d] = t.refs[s];
        t.refs[s] = 0;
    }
    if (tid == 0) *w.n_moves = movers;
}

enum Mode { kCopy, kFork, kCompact };

struct Side {
    uint8_t *pool;
    uint64_t layer, kv, block, token;  // strides in bytes
    uint32_t n_pool;
};

struct MoveArgs {
    Side from, to;
    uint32_t L, bt, row_bytes;
    const uint32_t *src, *dst, *rows;  // rows null: whole blocks
    const uint32_t *n_dev;             // moves; null: n
    uint32_t n;
    Tab t;
    ForkArgs f;
    PlanWs w;
    uint32_t row_blocks;               // fork: blocks that checked rows
    const uint32_t *remap;
    uint32_t *status;
};

template <int V> struct Vec;
template <> struct Vec<16> { using T = uint4; };
template <> struct Vec<8> { using T = uint2; };
template <> struct Vec<4> { using T = uint32_t; };
template <> struct Vec<2> { using T = uint16_t; };

// The children's rows, lengths and references.
__device__ void fork_tables(const MoveArgs &a) {
    for (uint32_t i = blockIdx.x; i < a.f.n; i += gridDim.x) {
        const uint32_t c = a.f.child[i], p = a.f.parent[i], pl = a.w.plen[i], base = a.w.base[i];
        const uint32_t full = pl >> a.t.bshift;
        const uint32_t all = (uint32_t)(((uint64_t)pl + (a.f.reserve ? a.f.reserve[i] : 0u) + a.bt - 1u) >> a.t.bshift);
        uint32_t *row = a.t.tables + (uint64_t)c * a.t.n_blocks;
        const bool no_tail = a.w.rows[i] && a.w.src[i] >= a.t.n_pool;  // nothing to copy: the fresh block stays free
        for (uint32_t k = threadIdx.x; k < a.t.n_blocks; k += blockDim.x) {
            uint32_t b = CG_NO_BLOCK;
            if (k == full && no_tail) {
                flag(a.status, CG_ERR_CORRUPT);
            } else if (k < full) {
                b = a.t.tables[(uint64_t)p * a.t.n_blocks + k];
                if (b < a.t.n_pool) {
                    atomicAdd(&a.t.refs[b], 1u);
                } else {
                    b = CG_NO_BLOCK;
                    flag(a.status, CG_ERR_CORRUPT);
                }
            } else if (k < all) {
                b = a.w.fresh[base + k - full];
                atomicAdd(&a.t.refs[b], 1u);  // not a store: a corrupt parent may name this block too
            }
            row[k] = b;
        }
        if (threadIdx.x == 0) a.t.lens[c] = pl;
    }
}

__device__ void compact_tables(const MoveArgs &a) {
    const uint64_t n = (uint64_t)a.t.n_slots * a.t.n_blocks;
    for (uint64_t k = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; k < n; k += (uint64_t)gridDim.x * blockDim.x) {
        const uint32_t b = a.t.tables[k];
        if (b == CG_NO_BLOCK) continue;
        const uint32_t nb = b < a.t.n_pool ? a.remap[b] : CG_NO_BLOCK;
        if (nb == CG_NO_BLOCK) flag(a.status, CG_ERR_CORRUPT);
        if (nb != b) a.t.tables[k] = nb;
    }
}

// The moves.  A warp takes a unit of 256 vectors of one (move, layer, K/V)
// and has 8 loads a lane in flight before the first store: 96 KB an SM with
// the 24 warps that a copy's 80 registers allow, 64 KB with the 16 warps of a
// fork (110 registers) or a compaction (104).  Bound by DRAM: 500 blocks of 80
// layers, 5.24 GB read and written, take 781 us, 6.7 TB/s (99% of a plain
// copy); 32 tails of one parent, read from L2 and written once each, 671 MB,
// 138 us, 4.9 TB/s of writes (a plain fill of 671 MB takes 168 us, 4.0 TB/s).
template <int V, Mode kMode>
__global__ void __launch_bounds__(kMoveThreads) k_move(MoveArgs a) {
    using T = typename Vec<V>::T;
    if (kMode != kCopy) wait_for_previous();  // the plan
    uint32_t n = a.n_dev ? *a.n_dev : a.n;
    if (kMode == kFork) {
        const bool held = threadIdx.x < a.row_blocks && a.w.held[threadIdx.x];
        if (__syncthreads_or(held)) n = 0;
    }
    if (kMode == kFork && n) fork_tables(a);
    if (kMode == kCompact) compact_tables(a);
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t per_row = a.row_bytes / V;
    const bool flat = a.from.token == a.row_bytes && a.to.token == a.row_bytes;
    const uint64_t most = (uint64_t)per_row * a.bt;
    const uint64_t chunks = (most + kUnitVecs - 1u) / kUnitVecs;
    const uint64_t per_move = chunks * a.L * 2u, units = per_move * n;
    const uint64_t warps = (uint64_t)gridDim.x * (kMoveThreads / 32u);
    for (uint64_t u = (uint64_t)blockIdx.x * (kMoveThreads / 32u) + (threadIdx.x >> 5); u < units; u += warps) {
        const uint32_t m = (uint32_t)(u / per_move);
        const uint64_t r = u - m * per_move;
        const uint32_t slice = (uint32_t)(r / chunks);
        const uint64_t v0 = (r - slice * chunks) * kUnitVecs;
        const uint64_t nv = a.rows ? (uint64_t)per_row * a.rows[m] : most;
        if (v0 >= nv) continue;
        const uint32_t s = a.src[m], d = kMode == kFork ? a.w.fresh[a.w.base[m]] : a.dst[m];
        if (s >= a.from.n_pool || d >= a.to.n_pool) {
            if (lane == 0) flag(a.status, kMode == kCopy ? CG_ERR_RANGE : CG_ERR_CORRUPT);
            continue;
        }
        const uint8_t *ps = a.from.pool + (slice >> 1) * a.from.layer + (slice & 1u) * a.from.kv + s * a.from.block;
        uint8_t *pd = a.to.pool + (slice >> 1) * a.to.layer + (slice & 1u) * a.to.kv + d * a.to.block;
        T x[kVecs];
        uint64_t at[kVecs];
#pragma unroll
        for (uint32_t k = 0; k < kVecs; k++) {
            const uint64_t v = v0 + k * 32u + lane;
            if (v >= nv) continue;
            if (flat) {
                at[k] = v * V;
                x[k] = *reinterpret_cast<const T *>(ps + at[k]);
            } else {
                const uint32_t row = (uint32_t)v / per_row, col = (uint32_t)v - row * per_row;
                at[k] = row * a.to.token + (uint64_t)col * V;
                x[k] = *reinterpret_cast<const T *>(ps + row * a.from.token + (uint64_t)col * V);
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < kVecs; k++)
            if (v0 + k * 32u + lane < nv) *reinterpret_cast<T *>(pd + at[k]) = x[k];
    }
}

// A block per listed slot.  Every entry is taken with an exchange, so that a
// row with gaps loses all of its blocks and a slot named twice is ended once.
// A count may pass below zero for as long as a thread that found no reference
// takes its step back; read as signed, it counts as none all that time, so as
// many rows succeed as there were references (fewer than 2^31), in any order.
// Bound by the chain of two atomics an entry and, where many rows share blocks,
// by those on one count: 256 rows of 1024 entries, 180 thousand references, take
// 8.5 us with cold caches, one slot 3 us.
__global__ void __launch_bounds__(256) k_free(Tab t, const uint32_t *slots, uint32_t n, uint32_t *status) {
    for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
        const uint32_t s = slots[i];
        if (s >= t.n_slots) {
            if (threadIdx.x == 0) flag(status, CG_ERR_RANGE);
            continue;
        }
        uint32_t *row = t.tables + (uint64_t)s * t.n_blocks;
        if (threadIdx.x == 0) t.lens[s] = 0;
        for (uint32_t k = threadIdx.x; k < t.n_blocks; k += blockDim.x) {
            const uint32_t b = atomicExch(&row[k], CG_NO_BLOCK);
            if (b == CG_NO_BLOCK) continue;  // none, or taken by another block of the call
            if (b >= t.n_pool) {
                flag(status, CG_ERR_CORRUPT);
            } else if ((int32_t)atomicSub(&t.refs[b], 1u) <= 0) {
                atomicAdd(&t.refs[b], 1u);
                flag(status, CG_ERR_CORRUPT);
            }
        }
    }
}

Tab tab_of(const cg_pages *p) {
    return Tab{p->tables, p->lens, p->refs, p->n_slots, p->n_blocks, p->n_pool_blocks,
               (uint32_t)__builtin_ctz(p->block_tokens)};
}

Side side_of(const cg_pages *p) {
    return Side{reinterpret_cast<uint8_t *>(p->pool), 2 * p->layer_stride, 2 * p->kv_stride, 2 * p->block_stride,
                2 * p->token_stride, p->n_pool_blocks};
}

// Bytes that every address of a side is a multiple of.
uint64_t align_of(const cg_pages *p) {
    return reinterpret_cast<uintptr_t>(p->pool) | 2 * p->layer_stride | 2 * p->kv_stride | 2 * p->block_stride |
           2 * p->token_stride | 2ull * p->C;
}

template <Mode kMode>
cudaError_t launch_move(const MoveArgs &a, uint64_t align, uint64_t max_moves, uint64_t table_blocks, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int V = align % 16 == 0 ? 16 : align % 8 == 0 ? 8 : align % 4 == 0 ? 4 : 2;
    const uint64_t chunks = ((uint64_t)(a.row_bytes / V) * a.bt + kUnitVecs - 1u) / kUnitVecs;
    uint64_t want = (max_moves * a.L * 2u * chunks + kMoveThreads / 32u - 1u) / (kMoveThreads / 32u);
    want = want < table_blocks ? table_blocks : want;
    const uint64_t most = (uint64_t)sms * 8u;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    const auto k = V == 16 ? k_move<16, kMode> : V == 8 ? k_move<8, kMode> : V == 4 ? k_move<4, kMode> : k_move<2, kMode>;
    return launch_next(k, grid, kMoveThreads, 0, s, kMode != kCopy, a);
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) != 0; }

bool pool_ok(const cg_pages *p) {
    return p && p->pool && p->L && p->C && p->n_pool_blocks && p->block_tokens && p->token_stride >= p->C &&
           (p->block_tokens & (p->block_tokens - 1u)) == 0 && p->n_pool_blocks <= (1u << 31) &&
           (uint64_t)p->C * p->block_tokens <= (1ull << 31) && !misaligned(p->pool, 2);
}

bool state_ok(const cg_pages *p) {
    return pool_ok(p) && p->tables && p->lens && p->refs && p->n_slots && p->n_slots <= (1u << 31) && p->n_blocks &&
           (uint64_t)p->n_blocks * p->block_tokens <= (1ull << 31) && !misaligned(p->tables, 4) &&
           !misaligned(p->lens, 4) && !misaligned(p->refs, 4);
}

// A list of n numbers; an empty one may have no address.
bool ids_ok(const uint32_t *ids, uint32_t n) { return (ids || n == 0) && !misaligned(ids, 4); }

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" cg_status cg_pages_ws_bytes(const cg_pages *p, size_t *ws_bytes) {
    if (!state_ok(p) || !ws_bytes) return CG_ERR_INVALID_ARG;
    *ws_bytes = plan_ws(p->n_pool_blocks, p->n_slots, nullptr, nullptr);
    return CG_OK;
}

extern "C" cg_status cg_pages_copy(const cg_pages *to, const cg_pages *from, const uint32_t *src_ids,
                                   const uint32_t *dst_ids, uint32_t n, uint32_t *dev_status, void *stream) {
    if (!pool_ok(to) || !pool_ok(from) || !ids_ok(src_ids, n) || !ids_ok(dst_ids, n)) return CG_ERR_INVALID_ARG;
    if (to->L != from->L || to->C != from->C || to->block_tokens != from->block_tokens) return CG_ERR_INVALID_ARG;
    if (n == 0) return CG_OK;
    MoveArgs a{};
    a.from = side_of(from);
    a.to = side_of(to);
    a.L = to->L;
    a.bt = to->block_tokens;
    a.row_bytes = 2 * to->C;
    a.src = src_ids;
    a.dst = dst_ids;
    a.n = n;
    a.status = dev_status;
    CG_CUDA_TRY(launch_move<kCopy>(a, align_of(to) | align_of(from), n, 0, static_cast<cudaStream_t>(stream)));
    return CG_OK;
}

extern "C" cg_status cg_pages_fork(const cg_pages *p, const uint32_t *parent, const uint32_t *child,
                                   const uint32_t *reserve, uint32_t n, void *ws, size_t ws_bytes,
                                   uint32_t *dev_status, void *stream) {
    if (!state_ok(p) || !ids_ok(parent, n) || !ids_ok(child, n) || !ws || misaligned(ws, 256) ||
        misaligned(reserve, 4) || n > p->n_slots)
        return CG_ERR_INVALID_ARG;
    PlanWs w;
    if (ws_bytes < plan_ws(p->n_pool_blocks, p->n_slots, ws, &w)) return CG_ERR_RANGE;
    if (n == 0) return CG_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MoveArgs a{};
    a.from = a.to = side_of(p);
    a.L = p->L;
    a.bt = p->block_tokens;
    a.row_bytes = 2 * p->C;
    a.src = w.src;
    a.rows = w.rows;
    a.n_dev = w.n_moves;
    a.t = tab_of(p);
    a.f = ForkArgs{parent, child, reserve, n};
    a.w = w;
    a.status = dev_status;
    a.row_blocks = n < kMaxRowBlocks ? n : kMaxRowBlocks;
    k_fork_plan<<<1 + a.row_blocks, kPlanThreads, 0, s>>>(a.t, a.f, w, dev_status);
    CG_CUDA_TRY(cudaGetLastError());
    CG_CUDA_TRY(launch_move<kFork>(a, align_of(p), n, n, s));
    return CG_OK;
}

extern "C" cg_status cg_pages_free(const cg_pages *p, const uint32_t *slots, uint32_t n, uint32_t *dev_status,
                                   void *stream) {
    if (!state_ok(p) || !ids_ok(slots, n) || n > (1u << 31)) return CG_ERR_INVALID_ARG;
    if (n == 0) return CG_OK;
    k_free<<<n < 65535u ? n : 65535u, 256, 0, static_cast<cudaStream_t>(stream)>>>(tab_of(p), slots, n, dev_status);
    CG_CUDA_TRY(cudaGetLastError());
    return CG_OK;
}

extern "C" cg_status cg_pages_compact(const cg_pages *p, uint32_t *remap, void *ws, size_t ws_bytes,
                                      uint32_t *dev_status, void *stream) {
    if (!state_ok(p) || !remap || misaligned(remap, 4) || !ws || misaligned(ws, 256)) return CG_ERR_INVALID_ARG;
    PlanWs w;
    if (ws_bytes < plan_ws(p->n_pool_blocks, p->n_slots, ws, &w)) return CG_ERR_RANGE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MoveArgs a{};
    a.from = a.to = side_of(p);
    a.L = p->L;
    a.bt = p->block_tokens;
    a.row_bytes = 2 * p->C;
    a.src = w.src;
    a.dst = w.dst;
    a.n_dev = w.n_moves;
    a.t = tab_of(p);
    a.w = w;
    a.remap = remap;
    a.status = dev_status;
    k_compact_plan<<<1, kPlanThreads, 0, s>>>(a.t, remap, w);
    CG_CUDA_TRY(cudaGetLastError());
    const uint64_t entries = (uint64_t)p->n_slots * p->n_blocks;
    CG_CUDA_TRY(launch_move<kCompact>(a, align_of(p), p->n_pool_blocks / 2u, entries / kMoveThreads, s));
    return CG_OK;
}

// cg_attend.cu -- attention of a batch of sequences in a paged pool whose
// leading blocks are shared (sm_103a).
//
// The softmax over a sequence splits at the end of the shared blocks: with
// m the largest score of a part, l = sum e^{s - m} and O = sum e^{s - m} V,
// parts join as m = max m_j, l = sum l_j e^{m_j - m}, O likewise, out = O / l.
// The shared part has the same keys for every request, so the query rows of
// all requests that use one KV head form one matrix against it, and its K
// and V are read once for the batch.  Every part may be split along its
// tokens again; the pieces go to the workspace and a last kernel joins them in
// a fixed order.  Scores are kept in log2 units (scale * log2 e folded in).
// Three kernels, each started while the one before it drains: k_shared (many
// query rows on the shared part, tcgen05), k_rows (a few query rows on their
// tokens, bound by memory), k_merge or k_merge_rows.
#include "cg_attend.cuh"

namespace cg {
namespace {

constexpr uint32_t kTileRows = 64;  // K rows of a tile of k_rows: 64 / nh tokens of nh neighbouring heads

// kR row tiles of 16 query rows a block.
template <uint32_t D, uint32_t kR> struct Smem {
    static constexpr uint32_t kStages = 3 * kR;             // tiles in flight: 96 KB, or 192 KB where one block has an SM
    static constexpr uint32_t kThreads = (4 * kR + 1) * 32; // kR x 4 warps compute, one fetches
    static constexpr uint32_t kTile = kTileRows * D * 2;    // K or V of a tile
    static constexpr uint32_t kStage = 2 * kTile;
    static constexpr uint32_t oBar = kStages * kStage;
    static constexpr uint32_t oMisc = oBar + 2 * kStages * 8;
    static constexpr uint32_t oLens = oMisc + 128;          // tokens of up to kLens requests
    static constexpr uint32_t kLens = 1024;
    static constexpr uint32_t oWeights = oLens + kLens * 4;  // 16 x 16 weights a warp, where rows add up one by one
    static constexpr uint32_t kBytes = oWeights + 4 * kR * kRows * 16 * 4 + 1024;  // and slack to align the tiles to 1 KiB
};

// Query rows in tiles of 16 against their tokens.  A block takes nh = 4
// neighbouring KV heads, 16 tokens at a time: a token's rows of four heads are
// one run of memory (1 KiB with 128 channels), and each warp has a head of its
// own, so that its softmax needs no other warp.  With fewer heads (nh = 2, 1)
// tiles are 32 or 64 tokens long and the warps of a head take every second or
// fourth 16 of them; their results go out as separate parts.  With kR = 2, two
// sets of warps take two row tiles against the same K and V.  One more warp
// fetches the tiles by TMA, 96 KB a block and 192 KB an SM ahead.
// Bound by DRAM: 24 requests of 32 heads, 747 MB of K and V, take 128 us, 5.8
// TB/s (with a block to one head, whose rows are runs of 256 bytes, 168 us).
// Where the pieces are short it is their beginnings and ends, about 2 us each:
// 128 requests of 200 tokens and 32 rows, 101 MB, take 39 us.  The products
// are mma.sync: 16 rows of 16 tokens are too few for the 128-row tcgen05
// tiles, and their unit is 19% busy.
template <class T, uint32_t D, uint32_t kR>
__global__ void __launch_bounds__(Smem<D, kR>::kThreads, 3 - kR) k_rows(const __grid_constant__ CUtensorMap map, const Args a) {
    using S = Smem<D, kR>;
    constexpr uint32_t kStages = S::kStages, kWarps = 4 * kR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (s_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = s_addr(smem);
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t full = sm + S::oBar, empty = full + kStages * 8;
    uint64_t *misc = reinterpret_cast<uint64_t *>(smem + S::oMisc);

    if (tid == 0) {
        for (uint32_t k = 0; k < kStages; k++) {
            bar_init(full + 8 * k, 1);
            bar_init(empty + 8 * k, kWarps);
        }
        fence_bar_init();
    }
    uint32_t *lens = reinterpret_cast<uint32_t *>(smem + S::oLens);
    Walk w = take_share<S::kThreads, false>(a, misc, lens, S::kLens);

    const uint32_t tt = 1u << a.tlog;                 // tokens of a tile
    const uint32_t head_bytes = tt * D * 2, half_bytes = tt * 128;
    Piece p;
    uint32_t it = 0;  // tiles so far: stage it % kStages, parity it / kStages
    if (warp == kWarps) {
        // a box (64 channels x up to tt rows of one block) per lane, at most 32 of them
        const uint32_t rlog = min(a.bshift, a.tlog), subs = tt >> rlog;
        const uint32_t sub = lane % subs, x = lane / subs, half = x % (D / 64), y = x / (D / 64);
        const uint32_t head = y % a.nh, kv = y / a.nh;
        const bool mine_box = kv < 2;
        const uint32_t dst0 = sm + kv * S::kTile + head * head_bytes + half * half_bytes + (sub << rlog) * 128;
        bool ok = true;
        while (ok && next_piece<false>(a, w, p)) {
            const bool shared = p.r == a.R;
            const uint32_t slot = shared ? a.shared_slot : a.slots ? a.slots[p.r] : p.r;
            const uint32_t *row = a.tables + (uint64_t)slot * a.n_blocks;
            const int c = (int)((p.group * a.nh + head) * D + half * 64);
            uint32_t pos = (shared ? 0u : a.P) + (p.tile0 << a.tlog) + (sub << rlog);
            // the block of this lane's box; a box past the sequence lies outside the map and reads zeros
            uint32_t next = mine_box && pos < p.len ? row[pos >> a.bshift] : a.n_pool;
            for (uint32_t k = 0; k < p.n; k++, it++, pos += tt) {
                const uint32_t st = it % kStages, in = pos & ((1u << a.bshift) - 1u);
                uint32_t id = next;
                next = mine_box && pos + tt < p.len && k + 1 < p.n ? row[(pos + tt) >> a.bshift] : a.n_pool;
                if (it >= kStages) ok = bar_wait(empty + 8 * st, (it / kStages - 1) & 1u);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                if (lane == 0) bar_expect(full + 8 * st, S::kStage);
                __syncwarp();
                if (mine_box) {
                    if (id > a.n_pool || (id == a.n_pool && pos < p.len)) {
                        id = a.n_pool;
                        flag(a.status, CG_ERR_RANGE);
                    }
                    tma_box(dst0 + st * S::kStage, &map, c, (int)in, (int)id, (int)kv, full + 8 * st);
                }
            }
        }
        if (!ok) {  // wait for the copies in flight before leaving
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; k++)
                bar_wait(full + 8 * (k % kStages), (k / kStages) & 1u);
            if (lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
        }
        if (a.pairs) wait_for_previous();  // this kernel is complete only after k_shared, whose pieces k_merge reads
        return;
    }

    let_next_start();
    const uint32_t qd = lane & 3u, rw = lane >> 2;
    const uint32_t col = warp & 3u, hd = col % a.nh, part = col / a.nh;  // head of the group, 16 tokens of the tile
    const uint32_t kbase = hd * head_bytes + part * 16 * 128, vbase = S::kTile + kbase;
    bool ok = true;
    // The queries of a piece, and how many of the item's tokens each of this
    // lane's two rows sees.  They are fetched before the results of the piece
    // before it go out.
    uint32_t q[D / 16][4], lim[2], least, own_tokens;
    Row ro[2];
    auto begin = [&]() {
        const bool shared = p.r == a.R;
        own_tokens = least = shared ? a.P : p.len - a.P;
        const uint32_t head = p.group * a.nh + hd, x0 = p.range * (kR * kRows) + (warp >> 2) * kRows;
#pragma unroll
        for (uint32_t e = 0; e < 2; e++) {
            const Row o = ro[e] = row_of(a, p, x0 + rw + 8 * e, head);
            const uint16_t *src = a.q + o.r * a.qs[0] + o.i * a.qs[1] + o.h * a.qs[2] + 2 * qd;
#pragma unroll
            for (uint32_t k = 0; k < D / 16; k++) {
                q[k][e] = o.valid ? *reinterpret_cast<const uint32_t *>(src + 16 * k) : 0u;
                q[k][e + 2] = o.valid ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 8) : 0u;
            }
            lim[e] = own_tokens;
            if (!shared) {
                const uint32_t sees = p.len + 1 + o.i;  // + 1 - nq below
                lim[e] = sees > a.nq + a.P ? min(sees - a.nq - a.P, own_tokens) : 0u;
                least = min(least, p.len + 1 > a.nq + a.P ? p.len + 1 - a.nq - a.P : 0u);
            }
        }
    };
    bool more = next_piece<false>(a, w, p);
    if (more) begin();
    while (more) {
        if (a.flip)
#pragma unroll
            for (uint32_t k = 0; k < D / 16; k++)
#pragma unroll
                for (uint32_t e = 0; e < 4; e++) q[k][e] ^= a.flip;
        float o[D / 8][4];
#pragma unroll
        for (uint32_t d = 0; d < D / 8; d++)
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) o[d][k] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (uint32_t k = 0; k < p.n; k++, it++) {
            const uint32_t st = it % kStages;
            if (ok) ok = bar_wait(full + 8 * st, (it / kStages) & 1u);
            if (!__all_sync(kFull, ok)) {
                ok = false;
                continue;
            }
            const uint32_t tok = ((p.tile0 + k) << a.tlog) + 16 * part;  // this warp's 16 tokens of the item
            if (tok < own_tokens) {
                const uint32_t kb = sm + st * S::kStage + kbase, vb = sm + st * S::kStage + vbase;
                const bool tail = tok + 16 > own_tokens;
                if (tail) {  // rows past the sequence hold anything: V's must not meet the weight 0
                    if (tok + (lane >> 1) >= own_tokens)
                        for (uint32_t b = 16 * (lane & 1u); b < D * 2; b += 32)
                            *reinterpret_cast<uint4 *>(smem + st * S::kStage + vbase + (b >> 7) * half_bytes +
                                                       (lane >> 1) * 128 + (b & 127u)) = make_uint4(0, 0, 0, 0);
                    __syncwarp();
                }
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                {
                    const uint32_t r = (lane >> 4) * 8 + (lane & 7u);
                    const uint32_t rb = kb + r * 128, x = r & 7u, hi = (lane >> 3) & 1u;
#pragma unroll
                    for (uint32_t c = 0; c < D / 16; c++) {
                        uint32_t b[4];
                        ldsm4(b, rb + (c >> 2) * half_bytes + ((((c & 3u) * 2 + hi) ^ x) << 4));
                        Half<T>::mma(s[0], q[c], b[0], b[1]);
                        Half<T>::mma(s[1], q[c], b[2], b[3]);
                    }
                }
                const bool mask = tok + 16 > least;
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (uint32_t n = 0; n < 2; n++)
#pragma unroll
                    for (uint32_t j = 0; j < 4; j++) {
                        const uint32_t e = j >> 1, t = tok + n * 8 + 2 * qd + (j & 1u);
                        s[n][j] *= a.scale2;
                        if (mask && t >= lim[e]) s[n][j] = -INFINITY;
                        mx[e] = fmaxf(mx[e], s[n][j]);
                    }
                float c[2];
                bool moved = false;
#pragma unroll
                for (uint32_t e = 0; e < 2; e++) {
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFull, mx[e], 1));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFull, mx[e], 2));
                    const float nm = fmaxf(m[e], mx[e]);
                    c[e] = m[e] == nm ? 1.f : ex2(m[e] - nm);
                    moved |= m[e] != nm;
                    m[e] = nm;
                }
                if (__any_sync(kFull, moved)) {
#pragma unroll
                    for (uint32_t d = 0; d < D / 8; d++) {
                        o[d][0] *= c[0];
                        o[d][1] *= c[0];
                        o[d][2] *= c[1];
                        o[d][3] *= c[1];
                    }
                    l[0] *= c[0];
                    l[1] *= c[1];
                }
                const float z[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
                for (uint32_t n = 0; n < 2; n++)
#pragma unroll
                    for (uint32_t j = 0; j < 4; j++) {
                        s[n][j] = ex2(s[n][j] - z[j >> 1]);
                        l[j >> 1] += s[n][j];
                    }
                // A token that some of the rows do not see may hold an infinity or a NaN, which
                // the weight 0 would not keep out of their sums: then each row adds its own.
                bool odd = false;
                if (mask && a.nq > 1) {
                    if (tok + (lane >> 1) >= least)
                        for (uint32_t b = 16 * (lane & 1u); b < D * 2; b += 32) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(smem + st * S::kStage + vbase + (b >> 7) * half_bytes +
                                                                             (lane >> 1) * 128 + (b & 127u));
                            constexpr uint32_t kX = Half<T>::kExponent;
                            for (uint32_t z : {y.x, y.y, y.z, y.w}) odd |= (z & kX) == kX || (z >> 16 & kX) == kX;
                        }
                    odd = __any_sync(kFull, odd);
                }
                uint32_t pa[4];  // O is held kHigh times as large until the end of the piece
#pragma unroll
                for (uint32_t k4 = 0; k4 < 4; k4++)
                    pa[k4] = Half<T>::pack(s[k4 >> 1][2 * (k4 & 1u)] * Half<T>::kHigh, s[k4 >> 1][2 * (k4 & 1u) + 1] * Half<T>::kHigh);
                if (!odd) {
                    const uint32_t r = ((lane >> 3) & 1u) * 8 + (lane & 7u);
                    const uint32_t rb = vb + r * 128, x = r & 7u, hi = lane >> 4;
#pragma unroll
                    for (uint32_t d = 0; d < D / 16; d++) {
                        uint32_t b[4];
                        ldsm4_t(b, rb + (d >> 2) * half_bytes + ((((d & 3u) * 2 + hi) ^ x) << 4));
                        Half<T>::mma(o[2 * d], pa, b[0], b[1]);
                        Half<T>::mma(o[2 * d + 1], pa, b[2], b[3]);
                    }
                } else {
                    float2 *wts = reinterpret_cast<float2 *>(smem + S::oWeights) + warp * (kRows * 8);  // [row][token]
                    for (uint32_t k4 = 0; k4 < 4; k4++)
                        wts[(rw + 8 * (k4 & 1u)) * 8 + (k4 >> 1) * 4 + qd] = Half<T>::unpack(pa[k4]);
                    __syncwarp();
#pragma unroll 1
                    for (uint32_t t = 0; t < 16; t++) {
                        const uint8_t *row = smem + st * S::kStage + vbase + t * 128 + 4 * qd;
#pragma unroll
                        for (uint32_t e = 0; e < 2; e++) {
                            if (tok + t >= lim[e]) continue;
                            const float wt = reinterpret_cast<const float *>(wts)[(rw + 8 * e) * 16 + t];
#pragma unroll
                            for (uint32_t d = 0; d < D / 8; d++) {
                                const float2 v = Half<T>::unpack(*reinterpret_cast<const uint32_t *>(
                                    row + (d >> 3) * half_bytes + (((d & 7u) ^ (t & 7u)) << 4)));
                                o[d][2 * e] += wt * v.x;
                                o[d][2 * e + 1] += wt * v.y;
                            }
                        }
                    }
                    __syncwarp();
                }
                if (tail) fence_async();  // the zeros are ordered before the copy that reuses the stage
            }
            __syncwarp();
            if (lane == 0) bar_arrive(empty + 8 * st);
        }

        const Row done[2] = {ro[0], ro[1]};
        constexpr float kLow = 1.f / Half<T>::kHigh;
        const bool answer = a.P == 0 && a.nh == 4 && p.n == p.of;  // the whole sequence
        const uint64_t slot = a.part0 + (((uint64_t)blockIdx.x + p.item) * 4 + col) * a.piece_rows + (warp >> 2) * kRows + rw;
#pragma unroll
        for (uint32_t e = 0; e < 2; e++) {
            l[e] += __shfl_xor_sync(kFull, l[e], 1);
            l[e] += __shfl_xor_sync(kFull, l[e], 2);
            if (!done[e].valid) continue;
            if (answer) {
                const float inv = l[e] == 0.f ? 0.f : kLow / l[e];
                uint16_t *dst = a.out + done[e].r * a.os[0] + done[e].i * a.os[1] + done[e].h * a.os[2] + 2 * qd;
#pragma unroll
                for (uint32_t d = 0; d < D / 8; d++)
                    *reinterpret_cast<uint32_t *>(dst + 8 * d) = Half<T>::pack(o[d][2 * e] * inv, o[d][2 * e + 1] * inv);
                if (a.lse && qd == 0)
                    a.lse[((uint64_t)done[e].r * a.nq + done[e].i) * (a.g * a.Hkv) + done[e].h] =
                        l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * kLn2;
            } else {
                const uint64_t at = slot + 8 * e;
                float *dst = a.part_o + at * D + 2 * qd;
#pragma unroll
                for (uint32_t d = 0; d < D / 8; d++)
                    *reinterpret_cast<float2 *>(dst + 8 * d) = make_float2(o[d][2 * e] * kLow, o[d][2 * e + 1] * kLow);
                if (qd == 0) a.part_ml[at] = make_float2(m[e], l[e]);
            }
        }
        more = next_piece<false>(a, w, p);
        if (more) begin();
    }
    if (!ok && lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
}

// ---------------------------------------------------------------------------
// The shared part for many query rows, on tcgen05.
//
// Rows: a KV head's query rows of all requests, 128 to a tile (the M of the
// matrix instructions, a row per TMEM lane).  A block works on two softmax
// streams, each with a score tile S and an output O in TMEM: with more than
// 128 rows the streams are two row tiles that read the same K and V; with up
// to 128 rows they are the even and the odd token tiles of one row tile.
// While one stream's warps turn S into weights, the tensor cores work on the
// other's.  Token tiles are 128 long: S = Q K^T (both from shared memory),
// P = e^{S - m} goes back into TMEM as the A operand of O += P V, whose V is
// read as it lies in the pool (rows = tokens, the contraction dimension).
// The running maximum m is only raised, and O rescaled, when a tile's maximum
// lies more than 8 (a factor of 2^8) above it; P is kept kShift octaves high,
// so that fp16 weights neither overflow (2^(8 + 6)) nor lose their small end.
// Bound by the tensor cores: 4096 rows on each of 8 heads' 32768 tokens (550
// GFLOP) take 309 us, 1770 TFLOP/s; with 512 rows on 16384 tokens (34 GFLOP,
// 134 MB) 34 us, of which K and V from DRAM are 20.
// ---------------------------------------------------------------------------
// Three warpgroups: two of softmax, one whose first warps fetch tiles and
// issue MMAs.  The launch gives 168 registers a thread; the last group keeps
// 72, so that a softmax thread can hold its row of scores: 2 x 216 + 72 = 3 x 168.
constexpr uint32_t kTcThreads = 384;
constexpr float kGrow = 8.f, kShift = 6.f;

template <uint32_t D> struct TcSmem {
    static constexpr uint32_t kHalf = kTcTok * 128;     // 64 channels x 128 rows
    static constexpr uint32_t kTile = kTcTok * D * 2;   // K, V or Q
    static constexpr uint32_t oQ = kTcSlots * kTile;
    static constexpr uint32_t oBar = oQ + 2 * kTile;
    static constexpr uint32_t kBytes = oBar + 256 + 1024;
};
// TMEM columns.  With D = 64 there is room for P beside S; with D = 128 it
// lies on S, which the MMAs of one shape leave in order.
template <uint32_t D> struct Tmem {
    static constexpr __host__ __device__ uint32_t S(uint32_t s) { return s * 128; }
    static constexpr __host__ __device__ uint32_t O(uint32_t s) { return 256 + s * D; }
    static constexpr __host__ __device__ uint32_t P(uint32_t s) { return D == 64 ? 384 + s * 64 : s * 128; }
};

struct TcPiece {
    uint32_t item, pair, head, tile0, n;
};
// A block's share [t, end) of the list of all items' tiles.  Where it crosses
// from one item to the next, the last item's piece comes first: then every
// block begins near the start of an item and the row tiles of a head go over
// its tokens together, so that the others find in L2 what the first has read.
// (In list order their places in the tokens were spread evenly, and 134 MB of
// K and V went through the 129 MB L2 sixteen times: 358 us, 6 TB/s from DRAM.)
struct TcWalk {
    uint64_t t, end, last;  // last: where the piece of the last item begins, until it has been given out
    uint32_t of;
    __device__ __forceinline__ TcWalk(uint64_t t_, uint64_t end_, uint32_t of_) : t(t_), end(end_), last(end_), of(of_) {
        if (t < end) last = quot(end - 1, of) * of;
        if (last <= t) last = end;
    }
    __device__ __forceinline__ bool next(const Args &a, TcPiece &p) {
        uint64_t from = t, to = end;
        if (last < end) {
            from = last;
            end = last;
        } else if (t >= end) {
            return false;
        }
        p.item = (uint32_t)quot(from, of);
        p.head = p.item / a.pairs;
        p.pair = p.item - p.head * a.pairs;
        p.tile0 = (uint32_t)(from - (uint64_t)p.item * of);
        p.n = (uint32_t)min((uint64_t)(of - p.tile0), to - from);
        if (from == t) t += p.n;
        return true;
    }
};

// kSplit: K is the sum of the map's matrices 0 and 2, a tile of each in turn.
template <class T, uint32_t D, bool kSplit>
__global__ void __launch_bounds__(kTcThreads, 1) k_shared(const __grid_constant__ CUtensorMap map, const Args a) {
    using M = TcSmem<D>;
    constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (s_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = s_addr(smem), tid = threadIdx.x, lane = tid & 31u;
    const uint32_t warp = __shfl_sync(kFull, tid >> 5, 0);
    // barriers: slot full / empty, then per stream: scores ready, weights ready (two halves), output ready;
    // queries ready; drain
    const uint32_t full = sm + M::oBar, empty = full + 8 * kTcSlots, s_rdy = empty + 8 * kTcSlots, p_rdy = s_rdy + 16,
                   o_rdy = p_rdy + 32, q_rdy = o_rdy + 16, drain = q_rdy + 8;
    uint32_t *tm_at = reinterpret_cast<uint32_t *>(smem + M::oBar + 8 * (2 * kTcSlots + 10));
    if (tid == 0) {
        for (uint32_t k = 0; k < 2 * kTcSlots; k++) bar_init(full + 8 * k, 1);
        for (uint32_t s = 0; s < 2; s++) {
            bar_init(s_rdy + 8 * s, 1);
            bar_init(p_rdy + 16 * s, 128);
            bar_init(p_rdy + 16 * s + 8, 128);
            bar_init(o_rdy + 8 * s, 1);
        }
        bar_init(q_rdy, 256);
        bar_init(drain, 1);
        fence_bar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s_addr(tm_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(kFull, *tm_at, 0);  // the same in every lane, and known to be
    let_next_start();

    const uint32_t of = (a.P + kTcTok - 1) / kTcTok;  // tiles of an item
    const uint64_t total = (uint64_t)a.pairs * a.Hkv * of;
    const uint64_t n_cta = min((uint64_t)a.n_tc, total);
    TcWalk walk(blockIdx.x < n_cta ? quot(blockIdx.x * total, n_cta) : total,
                blockIdx.x < n_cta ? quot((blockIdx.x + 1ull) * total, n_cta) : total, of);
    TcPiece p;
    bool ok = true;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {  // fetch: tiles in the order in which the MMA warp uses them
            const uint32_t rows_log = min(a.bshift, 6u), rows = 1u << rows_log, boxes = kTcTok >> rows_log;
            const uint32_t *row = a.tables ? a.tables + (uint64_t)a.shared_slot * a.n_blocks : nullptr;
            uint32_t cnt = 0;
            if (a.after) {  // the kernel before this one makes what is fetched
                wait_for_previous();
                asm volatile("fence.proxy.async.global;" ::: "memory");
            }
            auto fetch = [&](uint32_t tile, uint32_t kv, uint32_t head) {
                if (!ok) return;
                const uint32_t st = cnt % kTcSlots;
                const uint32_t pos = tile * kTcTok + lane * rows;
                uint32_t id = a.n_pool;  // outside the map: reads zeros
                if (lane < boxes && pos < a.P) {
                    id = row ? row[pos >> a.bshift] : pos >> a.bshift;
                    if (id >= a.n_pool) {
                        id = a.n_pool;
                        flag(a.status, CG_ERR_RANGE);
                    }
                }
                if (cnt >= kTcSlots) ok = bar_wait(empty + 8 * st, (cnt / kTcSlots - 1) & 1u);
                ok = __all_sync(kFull, ok);
                if (!ok) return;
                if (lane == 0) bar_expect(full + 8 * st, M::kTile);
                __syncwarp();
                if (lane < boxes)
    #pragma unroll
                    for (uint32_t h = 0; h < D / 64; h++)
                        tma_box(sm + st * M::kTile + h * M::kHalf + lane * rows * 128, &map, (int)(head * D + 64 * h),
                                (int)(pos & ((1u << a.bshift) - 1u)), (int)id, (int)kv, full + 8 * st);
                cnt++;
            };
            while (walk.next(a, p)) {
                const uint32_t ahead = a.one ? 2 : 1;  // score tiles fetched before the first V
                auto fetch_k = [&](uint32_t tile) {
                    fetch(tile, 0, p.head);
                    if constexpr (kSplit) fetch(tile, 2, p.head);
                };
                for (uint32_t k = 0; k < ahead && k < p.n; k++) fetch_k(p.tile0 + k);
                for (uint32_t k = 0; k < p.n; k++) {
                    fetch(p.tile0 + k, 1, p.head);
                    if (k + ahead < p.n) fetch_k(p.tile0 + k + ahead);
                }
            }
            if (!ok) {
                for (uint32_t k = cnt > kTcSlots ? cnt - kTcSlots : 0; k < cnt; k++)
                    bar_wait(full + 8 * (k % kTcSlots), (k / kTcSlots) & 1u);
                if (lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
            }
        } else if (warp == 9) {
            constexpr uint32_t kQk = mma_shape(kBf16, kTcTok, true), kPv = mma_shape(kBf16, D, false);
            uint32_t cnt = 0, piece = 0, np[2] = {0, 0};
            auto slot_ready = [&](uint32_t c) {
                if (ok) ok = __all_sync(kFull, bar_wait(full + 8 * (c % kTcSlots), (c / kTcSlots) & 1u));
                tc_fence_after();
            };
            // scores of stream s from the K in slot c (kSplit: and in the next)
            auto qk = [&](uint32_t s, uint32_t c) {
                if (!ok) return;
                const uint32_t q = mma_desc(sm + M::oQ + (a.one ? 0 : s) * M::kTile, true, 0);
#pragma unroll
                for (uint32_t y = 0; y <= (kSplit ? 1u : 0u); y++) {
                    const uint32_t k = mma_desc(sm + ((c + y) % kTcSlots) * M::kTile, true, 0);
#pragma unroll
                    for (uint32_t x = 0; x < D / 16; x++) {
                        const uint32_t o = ((x >> 2) * M::kHalf + (x & 3u) * 32) >> 4;
                        tc_mma_ss(tm + Tmem<D>::S(s), q + o, k + o, kQk, x != 0 || y);
                    }
                }
                tc_commit(s_rdy + 8 * s);
            };
            auto pv = [&](uint32_t s, uint32_t c, bool first) {
                const uint32_t v = mma_desc(sm + (c % kTcSlots) * M::kTile, false, M::kHalf);
#pragma unroll
                for (uint32_t h = 0; h < 2; h++) {
                    if (ok) ok = __all_sync(kFull, bar_wait(p_rdy + 16 * s + 8 * h, np[s] & 1u));
                    tc_fence_after();
                    if (!ok) return;
#pragma unroll
                    for (uint32_t x = h * (kTcTok / 32); x < (h + 1) * (kTcTok / 32); x++)
                        tc_mma_ts(tm + Tmem<D>::O(s), tm + Tmem<D>::P(s) + 8 * x, v + x * 128, kPv, !first || x != 0);
                }
                np[s]++;
            };
            auto free_slot = [&](uint32_t c) {
                if (ok) tc_commit(empty + 8 * (c % kTcSlots));
            };
            auto done = [&](uint32_t s) {
                if (ok) tc_commit(o_rdy + 8 * s);
            };
            while (walk.next(a, p)) {
                if (ok) ok = __all_sync(kFull, bar_wait(q_rdy, piece++ & 1u));
                tc_fence_after();
                // K's slots: cnt, with kSplit cnt + 1 too
                auto k_ready = [&]() {
                    slot_ready(cnt);
                    if constexpr (kSplit) slot_ready(cnt + 1);
                };
                auto free_k = [&]() {
                    free_slot(cnt++);
                    if constexpr (kSplit) free_slot(cnt++);
                };
                if (a.one) {  // even token tiles: stream 0, odd ones: stream 1
                    for (uint32_t k = 0; k < 2 && k < p.n; k++) {
                        k_ready();
                        qk(k, cnt);
                        free_k();
                    }
                    for (uint32_t k = 0; k < p.n; k++) {
                        const uint32_t s = k & 1u;
                        slot_ready(cnt);
                        pv(s, cnt, k < 2);
                        free_slot(cnt++);
                        if (k + 2 < p.n) {
                            k_ready();
                            qk(s, cnt);
                            free_k();
                        } else {
                            done(s);
                        }
                    }
                } else {
                    k_ready();
                    qk(0, cnt);
                    qk(1, cnt);
                    free_k();
                    for (uint32_t k = 0; k < p.n; k++) {
                        const uint32_t v = cnt++;
                        const bool more = k + 1 < p.n;
                        slot_ready(v);
                        if (more) k_ready();
                        for (uint32_t s = 0; s < 2; s++) {
                            pv(s, v, k == 0);
                            if (s) free_slot(v);
                            if (more) qk(s, cnt);
                            else done(s);
                        }
                        if (more) free_k();
                    }
                }
            }
            if (!ok) {
                tc_commit(drain);
                bar_wait(drain, 0);
                if (lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const uint32_t s = warp >> 2, rl = tid & 127u;            // stream, row (TMEM lane)
        const uint32_t tml = tm + ((warp & 3u) << 21);            // this warp's lanes
        uint32_t ns = 0, piece = 0;
        const uint32_t rows_all = a.R * a.nq * a.g, per = a.nq * a.g;
        while (walk.next(a, p)) {
            // the queries: a warp brings its 32 rows, D / 8 lanes to a row (a
            // thread to a row took 4.6 us, each load touching 32 lines); with
            // one row tile the first stream brings it
            if (!(a.one && s)) {
                const uint32_t x = p.pair * 256 + s * 128 + rl;
                const uint32_t r = x / per, y = x - r * per, i = y / a.g, h = p.head * a.g + (y - i * a.g);
                const uint16_t *mine = x < rows_all ? a.q + r * a.qs[0] + i * a.qs[1] + h * a.qs[2] : nullptr;
                constexpr uint32_t kLanes = D / 8, kPass = 32 / kLanes;  // lanes of a row, rows of a pass
                uint4 v[kLanes];
#pragma unroll
                for (uint32_t k = 0; k < kLanes; k++) {
                    const uint32_t row = k * kPass + lane / kLanes;
                    const uint4 *src = reinterpret_cast<const uint4 *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), row));
                    v[k] = src ? src[lane % kLanes] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (uint32_t k = 0; k < kLanes; k++) {
                    const uint32_t row = (rl & 96u) + k * kPass + lane / kLanes, c = lane % kLanes;
                    v[k].x ^= a.flip;
                    v[k].y ^= a.flip;
                    v[k].z ^= a.flip;
                    v[k].w ^= a.flip;
                    *reinterpret_cast<uint4 *>(smem + M::oQ + s * M::kTile + (c >> 3) * M::kHalf + row * 128 +
                                               (((c & 7u) ^ (row & 7u)) << 4)) = v[k];
                }
            }
            fence_async();
            bar_arrive(q_rdy);

            const uint32_t mine = a.one ? (p.n + 1 - s) / 2 : p.n;
            float m = -INFINITY, l = 0.f;
            for (uint32_t k = 0; k < mine; k++) {
                if (ok) ok = bar_wait(s_rdy + 8 * s, ns++ & 1u);
                ok = __all_sync(kFull, ok);
                if (!ok) continue;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (uint32_t c = 0; c < 4; c++) tc_ld32(x[c], tml + Tmem<D>::S(s) + 32 * c);
                tc_wait_ld();
                const uint32_t tile = p.tile0 + (a.one ? 2 * k + s : k), left = a.P - tile * kTcTok;
                if (left < kTcTok) {
#pragma unroll
                    for (uint32_t c = 0; c < 4; c++)
#pragma unroll
                        for (uint32_t j = 0; j < 32; j++)
                            if (32 * c + j >= left) x[c][j] = 0xFF800000u;
                }
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (uint32_t c = 0; c < 4; c++)
#pragma unroll
                    for (uint32_t j = 0; j < 32; j += 2)
                        mq[(j >> 1) & 3u] = fmaxf(fmaxf(mq[(j >> 1) & 3u], __uint_as_float(x[c][j])), __uint_as_float(x[c][j + 1]));
                float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                mx = mx == -INFINITY ? mx : mx * a.scale2;
                const bool grow = k == 0 || mx - m > kGrow;
                if (__any_sync(kFull, grow)) {
                    const float nm = grow ? fmaxf(m, mx) : m, f = nm == m ? 1.f : ex2(m - nm);
                    m = nm;
                    l *= f;
                    if (k) {  // the MMAs before this tile's scores, and so O, are done
#pragma unroll
                        for (uint32_t c = 0; c < D / 32; c++) {
                            uint32_t o[32];
                            tc_ld32(o, tml + Tmem<D>::O(s) + 32 * c);
                            tc_wait_ld();
#pragma unroll
                            for (uint32_t j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tc_st32(tml + Tmem<D>::O(s) + 32 * c, o);
                        }
                    }
                }
                const float z = m == -INFINITY ? 0.f : kShift - m;
                float su[2] = {0.f, 0.f}, sv[2] = {0.f, 0.f};
#pragma unroll
                for (uint32_t c = 0; c < 2; c++) {  // half a tile: the MMAs on it start while the other half is made
                    uint32_t w[32];
#pragma unroll
                    for (uint32_t j = 0; j < 32; j++) {
                        const uint32_t e = 2 * j;
                        float u, v;
                        fma2(u, v, __uint_as_float(x[2 * c + (e >> 5)][e & 31u]),
                             __uint_as_float(x[2 * c + (e >> 5)][(e & 31u) + 1]), a.scale2, z);
                        u = ex2(u);
                        v = ex2(v);
                        add2(su[j & 1u], sv[j & 1u], u, v);
                        w[j] = Half<T>::pack(u, v);
                    }
                    tc_st32(tml + Tmem<D>::P(s) + 32 * c, w);
                    tc_wait_st();
                    tc_fence_before();
                    bar_arrive(p_rdy + 16 * s + 8 * c);
                }
                l += (su[0] + su[1]) + (sv[0] + sv[1]);
            }
            // the piece's result
            const uint64_t at = (((uint64_t)blockIdx.x + p.item) * 2 + s) * 128 + rl;
            a.part_ml[at] = make_float2(m == -INFINITY ? m : m - kShift, l);
            if (mine) {
                if (ok) ok = bar_wait(o_rdy + 8 * s, piece & 1u);
                ok = __all_sync(kFull, ok);
                piece++;
            }
            if (a.one) group_sync(1, 256);  // the other stream's products read the same queries
            if (mine && ok) {
                // through the queries' shared memory, 8 KB a warp, so that a row goes out in one run
                tc_fence_after();
                const uint32_t stage = M::oQ + s * M::kTile + (warp & 3u) * (M::kTile / 4);
                constexpr uint32_t kCols = D / 2, kUnits = kCols / 4, kRowsOut = 32 / kUnits;  // columns of a pass in 16-byte units
#pragma unroll
                for (uint32_t c = 0; c < 2; c++) {
#pragma unroll
                    for (uint32_t b = 0; b < kCols / 32; b++) {
                        uint32_t o[32];
                        tc_ld32(o, tml + Tmem<D>::O(s) + kCols * c + 32 * b);
                        tc_wait_ld();
#pragma unroll
                        for (uint32_t j = 0; j < 8; j++)
                            *reinterpret_cast<uint4 *>(smem + stage + lane * (kCols * 4) + (((8 * b + j) ^ (lane & 7u)) << 4)) =
                                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    __syncwarp();
                    float *dst = a.part_o + (at - lane) * D + kCols * c;
#pragma unroll
                    for (uint32_t k = 0; k < kUnits; k++) {
                        const uint32_t row = k * kRowsOut + lane / kUnits, u = lane % kUnits;
                        *reinterpret_cast<uint4 *>(dst + row * D + 4 * u) =
                            *reinterpret_cast<const uint4 *>(smem + stage + row * (kCols * 4) + ((u ^ (row & 7u)) << 4));
                    }
                    __syncwarp();
                }
                tc_fence_before();
            }
            group_sync(1, 256);  // both streams are done with the queries and with TMEM
        }
        if (!ok && lane == 0) flag_why(a.status, CG_ERR_TIMEOUT, kWhyWait);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
}

// Where the pieces of a run of query rows lie: three runs of pieces, of
// k_shared, of the shared part in k_rows, of the request's own tokens.  The
// pieces of a row and of the next lie side by side.
struct Runs {
    uint32_t n_tc, n_sh, n_own, n;
    uint32_t tc, sh, own;  // the first piece of the first row
    uint32_t rows;         // rows that this holds for
};

// The rows x0.. of request r and KV head `head`, at most up to x_end.
template <bool kQuant>
__device__ __forceinline__ Runs runs_of(const Args &a, uint32_t r, uint32_t head, uint32_t x0, uint32_t x_end, uint32_t len,
                                        uint64_t own, uint64_t first) {
    constexpr uint32_t clog = columns_log<kQuant>();
    const uint32_t plog = clog - a.hlog;  // log2 of the parts of a row
    const uint32_t over = kQuant ? a.over : 0u;
    const uint32_t group = head >> a.hlog, hd = head & (a.nh - 1u);
    const uint32_t rlog = a.rlog, rmask = (1u << rlog) - 1u;
    const uint32_t nt_sh = a.npt ? places_of<kQuant>(a, a.P) : 0, nt_own = len > a.P ? places_of<kQuant>(a, len - a.P) : 0;
    const uint64_t total = own + (uint64_t)a.npt * a.ng * nt_sh, n_cta = shares(a, total);
    // places [t0, t0 + nt) of the list, an item's tiles, are spread over blocks c0..c1
    auto run = [](uint64_t t0, uint32_t nt, uint64_t n, uint64_t all, uint32_t &c0) {
        c0 = (uint32_t)quot((t0 + 1) * n - 1, all);
        return (uint32_t)quot((t0 + nt) * n - 1, all) - c0 + 1;
    };
    const uint32_t xp = r * (a.nq * a.g) + x0;
    uint32_t x1 = min(x_end, (x0 | rmask) + 1), c0;
    Runs o{};
    if (a.pairs) x1 = min(x1, x0 + 256u - (xp & 255u));
    if (a.npt) x1 = min(x1, x0 + (rmask + 1u) - (xp & rmask));
    o.rows = x1 - x0;
    if (len && a.pairs) {
        const uint32_t of = (a.P + kTcTok - 1) / kTcTok, item = head * a.pairs + (xp >> 8);
        const uint64_t all = (uint64_t)a.pairs * a.Hkv * of;
        o.n_tc = run((uint64_t)item * of, of, min((uint64_t)a.n_tc, all), all, c0) << a.one;
        o.tc = (c0 + item) * 256 + (xp & 255u);
    }
    if (len && a.npt) {
        const uint32_t item = (xp >> rlog) * a.ng + group;
        o.n_sh = run(own + (uint64_t)item * nt_sh + over, nt_sh - over, n_cta, total, c0) << plog;
        o.sh = a.part0 + (((c0 + a.R * a.rt * a.ng + item) << clog) + hd) * a.piece_rows + (xp & rmask);
    }
    if (nt_own) {
        const uint32_t item = (x0 >> rlog) * a.ng + group;
        o.n_own = run(first + (uint64_t)item * nt_own + over, nt_own - over, n_cta, total, c0) << plog;
        o.own = a.part0 + (((c0 + r * a.rt * a.ng + item) << clog) + hd) * a.piece_rows + (x0 & rmask);
    }
    o.n = o.n_tc + o.n_sh + o.n_own;
    return o;
}

// Row of piece e of the first row of `o`.
template <bool kQuant> __device__ __forceinline__ uint32_t place(const Args &a, const Runs &o, uint32_t e) {
    if (e < o.n_tc) return o.tc + (e >> a.one) * 256u + (e & a.one) * 128u;
    constexpr uint32_t clog = columns_log<kQuant>();
    const uint32_t plog = clog - a.hlog;
    const bool sh = e - o.n_tc < o.n_sh;
    const uint32_t f = sh ? e - o.n_tc : e - o.n_tc - o.n_sh;
    return (sh ? o.sh : o.own) + (((f >> plog) << clog) + ((f & ((1u << plog) - 1u)) << a.hlog)) * a.piece_rows;
}

__device__ __forceinline__ uint16_t *out_row(const Args &a, uint32_t r, uint32_t head, uint32_t i, uint32_t j) {
    return a.out + r * a.os[0] + i * a.os[1] + (head * a.g + j) * a.os[2];
}
__device__ __forceinline__ void write_lse(const Args &a, uint32_t r, uint32_t head, uint32_t i, uint32_t j, float m, float l) {
    if (a.lse)
        a.lse[((uint64_t)r * a.nq + i) * (a.g * a.Hkv) + head * a.g + j] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Joins the pieces of many query rows.  A warp takes a.merge_rows rows of one
// request and KV head, a lane D / 32 channels, four pieces at a time (seldom
// are there more): one trip to memory a row.  What counts is warps, since each
// waits for its row: 32768 rows of three pieces took 37 us with 16 warps an SM,
// 27 with 24, 23 with 32 and 21 where twice as many take half as many rows.
template <class T, uint32_t D, bool kQuant>
__global__ void __launch_bounds__(256, 4) k_merge_rows(const Args a) {
    wait_for_previous();
    constexpr uint32_t kLane = D / 32;
    const uint32_t lane = threadIdx.x & 31u, per = a.nq * a.g, chunks = (per + a.merge_rows - 1) / a.merge_rows;
    const uint32_t id = blockIdx.x * 8 + (threadIdx.x >> 5);  // at most 2^31 rows
    if (id >= a.R * a.Hkv * chunks) return;
    const uint32_t rh = id / chunks, r = rh / a.Hkv, head = rh - r * a.Hkv, x_begin = (id - rh * chunks) * a.merge_rows;
    const uint32_t x_end = min(x_begin + a.merge_rows, per);
    const uint32_t len = a.tokens[r];
    const uint64_t own = a.cum[a.R], first = a.cum[r];
    uint32_t i = x_begin / a.g, j = x_begin - i * a.g;  // query token, query head of the KV head
    for (uint32_t x0 = x_begin; x0 < x_end;) {
        const Runs o = runs_of<kQuant>(a, r, head, x0, x_end, len, own, first);
        x0 += o.rows;
        uint32_t at[4];
#pragma unroll
        for (uint32_t e = 0; e < 4; e++) at[e] = e < o.n ? place<kQuant>(a, o, e) : 0;
        const bool done = o.n_own == 1 && a.P == 0;  // k_rows has written the answer
#pragma unroll 1
        for (uint32_t x = 0; x < o.rows; x++) {
            if (!done) {
                float m = -INFINITY, l = 0.f, s[kLane] = {};
#pragma unroll 1
                for (uint32_t e0 = 0; e0 < o.n; e0 += 4) {
                    if (o.n > 4)
#pragma unroll
                        for (uint32_t e = 0; e < 4; e++) at[e] = e0 + e < o.n ? place<kQuant>(a, o, e0 + e) : 0;
                    float2 v[4];
                    float y[4][kLane];
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) {
                        v[e] = make_float2(-INFINITY, 0.f);
                        if (e0 + e < o.n) {
                            v[e] = a.part_ml[at[e] + x];
                            const float *src = a.part_o + (uint64_t)(at[e] + x) * D + kLane * lane;
                            if constexpr (kLane == 4) *reinterpret_cast<float4 *>(y[e]) = *reinterpret_cast<const float4 *>(src);
                            else *reinterpret_cast<float2 *>(y[e]) = *reinterpret_cast<const float2 *>(src);
                        }
                    }
                    float nm = m;
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++)
                        if (v[e].y != 0.f) nm = fmaxf(nm, v[e].x);  // 0: a piece the row sees nothing of; its outputs may be unwritten
                    const float f = m == nm ? 1.f : ex2(m - nm);
                    m = nm;
                    l *= f;
#pragma unroll
                    for (uint32_t k = 0; k < kLane; k++) s[k] *= f;
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) {
                        if (e0 + e >= o.n || v[e].y == 0.f) continue;
                        const float w = v[e].x == m ? 1.f : ex2(v[e].x - m);
                        l += v[e].y * w;
#pragma unroll
                        for (uint32_t k = 0; k < kLane; k++) s[k] += y[e][k] * w;
                    }
                }
                const float inv = l == 0.f ? 0.f : __frcp_rn(l);
                uint16_t *dst = out_row(a, r, head, i, j) + kLane * lane;
                if constexpr (kLane == 4)
                    *reinterpret_cast<uint2 *>(dst) =
                        make_uint2(Half<T>::pack(s[0] * inv, s[1] * inv), Half<T>::pack(s[2] * inv, s[3] * inv));
                else
                    *reinterpret_cast<uint32_t *>(dst) = Half<T>::pack(s[0] * inv, s[1] * inv);
                if (lane == 0) write_lse(a, r, head, i, j, m, l);
            }
            if (++j == a.g) {
                j = 0;
                i++;
            }
        }
    }
}

// Joins the pieces of fewer rows, of which each may have hundreds.  Lane j
// looks at piece j (32 at a time): its maximum, and its weight against the
// largest; then four groups of eight lanes add up every fourth piece, D / 8
// channels a lane, and the groups' sums meet in two halving exchanges.
// kWide, for the fewest rows: a block to a row, its eight warps taking every
// eighth 32 pieces; otherwise a warp takes a.merge_rows rows.  With kQuant,
// whose row kernel has no second block an SM and so at most 152 pieces a range
// and part, few pieces are dealt evenly over the eight warps: 152 of them are
// five rounds of loads a warp instead of eight (one request of 100003 tokens
// 55.4 -> 53.3 us), and from nine pieces on the block's warps share a row
// (with 33: 700 tokens 16.4 us; with nine 14.4).  Loading two pieces of a group before either is added
// spilled and was slower (24 ragged requests 66 -> 68 us).
template <class T, uint32_t D, bool kWide, bool kQuant>
__global__ void __launch_bounds__(256, 3) k_merge(const Args a) {
    wait_for_previous();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t per = a.nq * a.g, chunks = (per + a.merge_rows - 1) / a.merge_rows;
    const uint32_t id = kWide ? blockIdx.x : blockIdx.x * 8 + warp;
    if (id >= a.R * a.Hkv * chunks) return;
    const uint32_t rh = id / chunks, r = rh / a.Hkv, head = rh - r * a.Hkv, x_begin = (id - rh * chunks) * a.merge_rows;
    const uint32_t x_end = min(x_begin + a.merge_rows, per);
    const uint32_t len = a.tokens[r];
    const uint64_t own = a.cum[a.R], first = a.cum[r];
    constexpr uint32_t kPer = D / 8, kFew = kQuant ? 8 : 32;  // pieces that one warp of a block takes alone
    const uint32_t grp = lane >> 3, gl = lane & 7u;
    for (uint32_t x0 = x_begin; x0 < x_end;) {
        const Runs z = runs_of<kQuant>(a, r, head, x0, x_end, len, own, first);
        const uint32_t n = z.n, x_first = x0;
        x0 += z.rows;
        if (z.n_own == 1 && a.P == 0) continue;  // k_rows has written the answer
        if (kWide && n <= kFew && warp) return;
        // pieces that a warp looks at together; a block's eight warps share few evenly
        const uint32_t step = kWide && kQuant && n > kFew ? min(32u, ((n + 31) / 32) * 4) : 32u;
#pragma unroll 1
        for (uint32_t x = 0; x < z.rows; x++) {
            float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
            for (uint32_t k = 0; k < kPer; k++) o[k] = 0.f;
#pragma unroll 1
            for (uint32_t e0 = kWide ? step * warp : 0; e0 < n; e0 += kWide ? 8 * step : 32) {
                const float *s = nullptr;
                float2 v = make_float2(-INFINITY, 0.f);
                if (e0 + lane < n && lane < step) {
                    const uint32_t at = place<kQuant>(a, z, e0 + lane) + x;
                    v = a.part_ml[at];
                    s = a.part_o + (uint64_t)at * D;
                }
                if (v.y == 0.f) {  // a piece the row sees nothing of; its outputs may be unwritten
                    v.x = -INFINITY;
                    s = nullptr;
                }
                float nm = fmaxf(m, v.x);
#pragma unroll
                for (uint32_t d = 16; d; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(kFull, nm, d));
                const float f = m == nm ? 1.f : ex2(m - nm);
                const float w = v.x == nm ? 1.f : ex2(v.x - nm);
                float sum = v.y * w;
#pragma unroll
                for (uint32_t d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
                m = nm;
                l = l * f + sum;
                if (e0)
#pragma unroll
                    for (uint32_t k = 0; k < kPer; k++) o[k] *= f;
                const uint32_t cnt = min(n - e0, step);
#pragma unroll 2
                for (uint32_t b = 0; b < cnt; b += 4) {
                    const float wj = __shfl_sync(kFull, w, b + grp);
                    const float *sj = reinterpret_cast<const float *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(s), b + grp));
                    if (!sj) continue;
#pragma unroll
                    for (uint32_t k = 0; k < kPer / 4; k++) {
                        const float4 y = *reinterpret_cast<const float4 *>(sj + 4 * (gl + 8 * k));
                        o[4 * k] += y.x * wj;
                        o[4 * k + 1] += y.y * wj;
                        o[4 * k + 2] += y.z * wj;
                        o[4 * k + 3] += y.w * wj;
                    }
                }
            }
            // the groups' sums: half of the channels to either pair of groups, then to either group
            __syncwarp();
#pragma unroll
            for (uint32_t k = 0; k < kPer / 2; k++) {
                const float give = grp & 2u ? o[k] : o[k + kPer / 2], keep = grp & 2u ? o[k + kPer / 2] : o[k];
                o[k] = keep + __shfl_xor_sync(kFull, give, 16);
            }
#pragma unroll
            for (uint32_t k = 0; k < kPer / 4; k++) {
                const float give = grp & 1u ? o[k] : o[k + kPer / 4], keep = grp & 1u ? o[k + kPer / 4] : o[k];
                o[k] = keep + __shfl_xor_sync(kFull, give, 8);
            }
            if (kWide && n > kFew) {  // a row a block: the warps' sums meet in shared memory
                __shared__ float2 sh_ml[8];
                __shared__ float sh_o[8][D];
                constexpr uint32_t kOwn = kPer / 4;
                if (lane == 0) sh_ml[warp] = make_float2(m, l);
#pragma unroll
                for (uint32_t k = 0; k < kOwn; k++) sh_o[warp][lane * kOwn + k] = o[k];
                __syncthreads();
                if (warp) return;
#pragma unroll
                for (uint32_t k = 0; k < 8; k++) m = fmaxf(m, sh_ml[k].x);
                l = 0.f;
#pragma unroll
                for (uint32_t k = 0; k < kOwn; k++) o[k] = 0.f;
#pragma unroll
                for (uint32_t b = 0; b < 8; b++) {
                    const float2 v = sh_ml[b];
                    const float w = v.x == m ? 1.f : ex2(v.x - m);
                    l += v.y * w;
#pragma unroll
                    for (uint32_t k = 0; k < kOwn; k++) o[k] += sh_o[b][lane * kOwn + k] * w;
                }
            }
            const float inv = l == 0.f ? 0.f : __frcp_rn(l);
            const uint32_t i = (x_first + x) / a.g, j = x_first + x - i * a.g;
            uint16_t *dst = out_row(a, r, head, i, j);
            if constexpr (D == 128)
                *reinterpret_cast<uint2 *>(dst + 4 * (gl + 8 * grp)) =
                    make_uint2(Half<T>::pack(o[0] * inv, o[1] * inv), Half<T>::pack(o[2] * inv, o[3] * inv));
            else
                *reinterpret_cast<uint32_t *>(dst + 4 * (gl + 8 * (grp >> 1)) + 2 * (grp & 1u)) = Half<T>::pack(o[0] * inv, o[1] * inv);
            if (lane == 0) write_lse(a, r, head, i, j, m, l);
        }
    }
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) != 0; }

struct Plan {
    uint32_t g, nh, ng, range_rows, rt, npt, pairs, one, piece_rows;
    uint64_t items, tc_rows, cum_bytes, o_bytes, bytes;
};

// Who takes the shared part, by its query rows per KV head.  Up to 16: k_rows,
// one row tile (16 rows of 8 heads on 512 / 8192 / 32768 tokens: 15 / 23 / 40
// us a call; with k_shared 20 / 25 / 48).  17 to 32 rows of up to four
// requests: k_rows in blocks of two row tiles (24 rows: 16 / 26 / 44; k_shared
// 21 / 25 / 49).  Of more requests: k_shared, since such blocks are half empty
// on the requests' own tokens (24 requests of one row, 32 heads: 131 us;
// k_rows 150).  More than 32 rows: k_shared.
bool by_tensor(uint64_t rows, uint64_t requests) { return rows > 32 || (rows > kRows && requests > 4); }

bool make_plan(const cg_pages *p, const cg_attention *a, Plan *o) {
    if (!attention_ok(p, a) || (uint64_t)a->n_kv_heads * a->head_dim != p->C) return false;
    o->g = a->n_q_heads / a->n_kv_heads;
    constexpr uint64_t kMost = 1ull << 31;  // query rows; compared before each product, so that none wraps
    const uint64_t per = (uint64_t)a->n_queries * o->g;
    if (per > kMost || per * a->n_requests > kMost) return false;
    const uint64_t all = per * a->n_requests;
    if (all * a->n_kv_heads > kMost) return false;
    o->nh = a->n_kv_heads % 4 == 0 ? 4 : a->n_kv_heads % 2 == 0 ? 2 : 1;
    o->ng = a->n_kv_heads / o->nh;
    const bool tc = a->shared_blocks && by_tensor(all, a->n_requests);
    o->pairs = tc ? (uint32_t)((all + 255) / 256) : 0;
    o->one = all <= 128;
    const bool here = a->shared_blocks && !tc;  // the shared part goes through k_rows too
    const uint64_t most = here ? all : per;
    o->range_rows = most > kRows ? 2 * kRows : kRows;
    o->rt = (uint32_t)((per + o->range_rows - 1) / o->range_rows);
    o->npt = here ? (uint32_t)((all + o->range_rows - 1) / o->range_rows) : 0;
    o->piece_rows = (uint32_t)(most < o->range_rows ? most : o->range_rows);
    o->items = ((uint64_t)a->n_requests * o->rt + o->npt) * o->ng;
    if (o->items > (1ull << 31)) return false;
    o->tc_rows = tc ? ((uint64_t)o->pairs * a->n_kv_heads + kMaxTcCtas) * 256 : 0;
    const uint64_t rows = o->tc_rows + (o->items + kMaxCtas) * 4 * o->piece_rows;  // of partial results
    if (rows > 0xFFFFFFFFull) return false;
    o->cum_bytes = round_up((a->n_requests + 1ull) * 8 + a->n_requests * 4ull, 256);
    o->o_bytes = round_up(rows * a->head_dim * 4, 256);
    o->bytes = o->cum_bytes + o->o_bytes + round_up(rows * 8, 256);
    return true;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

template <class T, uint32_t D, uint32_t kR>
cudaError_t launch_rows(const CUtensorMap &map, Args &a, int sms, cudaStream_t s) {
    using S = Smem<D, kR>;
    cudaError_t e = cudaFuncSetAttribute(k_rows<T, D, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    const uint32_t n = (uint32_t)sms * (3 - kR);
    a.n_cta = n < kMaxCtas ? n : kMaxCtas;
    return launch_next(k_rows<T, D, kR>, a.n_cta, S::kThreads, S::kBytes, s, a.pairs != 0, map, a);
}

template <class T, uint32_t D, bool kSplit>
cudaError_t shared(const CUtensorMap &map, Args &a, int sms, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(k_shared<T, D, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    // An even deal of all tiles lets a block cross from one item to the
    // next, which costs about kCross tiles (the streams drain, new
    // queries come in); where whole blocks per item take no longer than that, deal so.
    constexpr uint64_t kCross = 4;
    // A block gets two token tiles a stream at least: a piece less to join saves more than a tile takes.
    const uint64_t items = (uint64_t)a.pairs * a.Hkv, of = (a.P + kTcTok - 1) / kTcTok, least = a.one ? 4 : 2;
    const uint64_t most = items * ((of + least - 1) / least), sm = (uint64_t)sms < kMaxTcCtas ? sms : kMaxTcCtas;
    const uint64_t n = sm < most ? sm : most, k = n / items;
    a.n_tc = (uint32_t)(k && (of + k - 1) / k <= items * of / n + kCross ? k * items : n);
    return launch_next(k_shared<T, D, kSplit>, a.n_tc, kTcThreads, TcSmem<D>::kBytes, s, a.after != 0, map, a);
}

template <class T, uint32_t D, bool kQuant>
cudaError_t joins(Args &a, int sms, cudaStream_t s) {
    // warps for the joins: as many as an SM holds (many rows: twice that), with a few rows each where there are rows enough
    const uint64_t per = (uint64_t)a.nq * a.g, rh = (uint64_t)a.R * a.Hkv;
    const bool wide = rh * per <= (uint64_t)sms * 4, many = rh * per >= (uint64_t)sms * 16;
    const uint64_t fit = (uint64_t)sms * (many ? 64 : 24) / rh, chunks = fit < 1 ? 1 : fit < per ? fit : per;
    a.merge_rows = wide ? 1 : (uint32_t)((per + chunks - 1) / chunks);
    const uint64_t warps = rh * ((per + a.merge_rows - 1) / a.merge_rows);
    if (wide) return launch_next(k_merge<T, D, true, kQuant>, (unsigned)warps, 256, 0, s, true, a);
    return launch_next(many ? k_merge_rows<T, D, kQuant> : k_merge<T, D, false, kQuant>, (unsigned)((warps + 7) / 8), 256, 0, s, true, a);
}

template <class T, uint32_t D>
cudaError_t rows(const CUtensorMap &map, uint32_t range_rows, Args &a, int sms, cudaStream_t s) {
    return range_rows == kRows ? launch_rows<T, D, 1>(map, a, sms, s) : launch_rows<T, D, 2>(map, a, sms, s);
}

}  // namespace

bool attention_ok(const cg_pages *p, const cg_attention *a) {
    if (!p || !a || !p->pool || !p->tables || !p->lens || !a->q || !a->out) return false;
    if (!p->L || !p->C || !p->n_pool_blocks || p->n_pool_blocks > (1u << 31) - 1u || !p->n_slots || !p->n_blocks)
        return false;
    const uint32_t bt = p->block_tokens;
    if (bt < 8 || (bt & (bt - 1u)) || (uint64_t)p->n_blocks * bt > (1ull << 31) - 64u || p->token_stride < p->C)
        return false;
    if (a->dtype > CG_BF16 || !a->n_requests || !a->n_queries || !a->n_q_heads || !a->n_kv_heads) return false;
    if (a->head_dim != 64 && a->head_dim != 128) return false;
    if (a->n_q_heads % a->n_kv_heads) return false;
    if (a->layer >= p->L || a->shared_blocks > p->n_blocks) return false;
    if (a->shared_blocks && a->shared_slot >= p->n_slots) return false;
    if (!isfinite(a->scale)) return false;
    // the stride of a dimension with one element is never used
    const auto used = [](uint64_t n, uint64_t stride) { return n > 1 ? stride : 0; };
    const uint64_t block = used(p->n_pool_blocks, p->block_stride), layer = used(p->L, p->layer_stride);
    const uint64_t counts[3] = {a->n_requests, a->n_queries, a->n_q_heads};
    uint64_t strides = layer | p->kv_stride | block | p->token_stride;
    for (int k = 0; k < 3; k++) strides |= used(counts[k], a->q_stride[k]) | used(counts[k], a->out_stride[k]);
    if (strides % 8 || misaligned(p->pool, 16) || misaligned(a->q, 16) || misaligned(a->out, 16)) return false;
    if (misaligned(p->tables, 4) || misaligned(p->lens, 4) || misaligned(a->lse, 4) || misaligned(a->slots, 4))
        return false;
    // a tensor map's strides have 40 bits, and its rows and blocks may not be empty strides
    if ((p->kv_stride | block | p->token_stride) >> 39 || !p->kv_stride || (p->n_pool_blocks > 1 && !block)) return false;
    return true;
}

bool make_token_map(const cg_pages *p, const uint16_t *base, uint32_t channels, uint32_t copies, uint32_t box, uint32_t rows,
                    CUtensorMapSwizzle swizzle, CUtensorMap *map) {
    const EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {channels, p->block_tokens, p->n_pool_blocks, copies};
    const cuuint64_t block = p->n_pool_blocks > 1 ? p->block_stride : p->token_stride;  // unused with one block, but checked
    const cuuint64_t strides[3] = {2 * p->token_stride, 2 * block, 2 * p->kv_stride};
    const cuuint32_t boxes[4] = {box, rows, 1, 1}, step[4] = {1, 1, 1, 1};
    // words: fp16 and bf16 are moved alike, and what lies outside the matrix is filled with zeros
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<uint16_t *>(base), dims, strides, boxes, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_shared(uint32_t dtype, uint32_t head_dim, bool split, const CUtensorMap &map, Args &a, int sms, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (dtype == CG_FP16) return head_dim == 128 ? shared<__half, 128, false>(map, a, sms, s) : shared<__half, 64, false>(map, a, sms, s);
    if (split) return head_dim == 128 ? shared<B, 128, true>(map, a, sms, s) : shared<B, 64, true>(map, a, sms, s);
    return head_dim == 128 ? shared<B, 128, false>(map, a, sms, s) : shared<B, 64, false>(map, a, sms, s);
}

template <bool kQuant> cudaError_t launch_joins(uint32_t dtype, uint32_t head_dim, Args &a, int sms, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (head_dim == 128) return dtype == CG_FP16 ? joins<__half, 128, kQuant>(a, sms, s) : joins<B, 128, kQuant>(a, sms, s);
    return dtype == CG_FP16 ? joins<__half, 64, kQuant>(a, sms, s) : joins<B, 64, kQuant>(a, sms, s);
}
cudaError_t launch_joins(uint32_t dtype, uint32_t head_dim, bool quant, Args &a, int sms, cudaStream_t s) {
    return quant ? launch_joins<true>(dtype, head_dim, a, sms, s) : launch_joins<false>(dtype, head_dim, a, sms, s);
}

}  // namespace cg

using namespace cg;

extern "C" cg_status cg_attend_ws_bytes(const cg_pages *p, const cg_attention *a, size_t *ws_bytes) {
    Plan pl;
    if (!ws_bytes || !make_plan(p, a, &pl)) return CG_ERR_INVALID_ARG;
    *ws_bytes = pl.bytes;
    return CG_OK;
}

extern "C" cg_status cg_attend(const cg_pages *p, const cg_attention *at, void *ws, size_t ws_bytes,
                               uint32_t *dev_status, void *stream) {
    Plan pl;
    if (!make_plan(p, at, &pl) || !ws || misaligned(ws, 256)) return CG_ERR_INVALID_ARG;
    if (ws_bytes < pl.bytes) return CG_ERR_RANGE;
    int dev = 0, sms = 0;
    CG_CUDA_TRY(cudaGetDevice(&dev));
    CG_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const uint32_t bshift = (uint32_t)__builtin_ctz(p->block_tokens);
    // boxes of k_rows are at most a tile high, those of k_shared 64 rows
    const uint32_t tt = kTileRows / pl.nh, bt = p->block_tokens;
    CUtensorMap map, rows_map;
    const uint16_t *layer = p->pool + at->layer * p->layer_stride;
    if (!make_token_map(p, layer, p->C, 2, 64, bt < tt ? bt : tt, CU_TENSOR_MAP_SWIZZLE_128B, &rows_map) ||
        !make_token_map(p, layer, p->C, 2, 64, bt < 64 ? bt : 64, CU_TENSOR_MAP_SWIZZLE_128B, &map))
        return CG_ERR_CUDA;
    Args a{};
    a.q = at->q;
    a.out = at->out;
    a.lse = at->lse;
    a.slots = at->slots;
    a.tables = p->tables;
    a.lens = p->lens;
    a.n_slots = p->n_slots;
    a.n_blocks = p->n_blocks;
    a.n_pool = p->n_pool_blocks;
    a.bshift = bshift;
    a.R = at->n_requests;
    a.nq = at->n_queries;
    a.g = pl.g;
    a.Hkv = at->n_kv_heads;
    a.P = at->shared_blocks << bshift;
    a.shared_slot = at->shared_slot;
    a.nh = pl.nh;
    a.ng = pl.ng;
    a.hlog = (uint32_t)__builtin_ctz(pl.nh);
    a.tlog = (uint32_t)__builtin_ctz(tt);
    a.rlog = (uint32_t)__builtin_ctz(pl.range_rows);
    a.rt = pl.rt;
    a.npt = pl.npt;
    for (int k = 0; k < 3; k++) {
        a.qs[k] = at->q_stride[k];
        a.os[k] = at->out_stride[k];
    }
    a.scale2 = fminf(fmaxf(fabsf(at->scale) * kLog2e, 0x1p-149f), 0x1p127f);  // not 0: masked scores are -inf before the product; nor infinite
    a.flip = at->scale < 0.f ? 0x80008000u : 0u;
    a.status = dev_status;
    uint8_t *w = static_cast<uint8_t *>(ws);
    a.cum = reinterpret_cast<uint64_t *>(w);
    a.tokens = reinterpret_cast<uint32_t *>(a.cum + a.R + 1);
    a.part_o = reinterpret_cast<float *>(w + pl.cum_bytes);
    a.part_ml = reinterpret_cast<float2 *>(w + pl.cum_bytes + pl.o_bytes);
    a.piece_rows = pl.piece_rows;
    a.pairs = pl.pairs;
    a.one = pl.one;
    a.part0 = (uint32_t)pl.tc_rows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp16 = at->dtype == CG_FP16;
    if (a.pairs) CG_CUDA_TRY(launch_shared(at->dtype, at->head_dim, false, map, a, sms, s));
    if (at->head_dim == 128)
        CG_CUDA_TRY((fp16 ? rows<__half, 128>(rows_map, pl.range_rows, a, sms, s) : rows<__nv_bfloat16, 128>(rows_map, pl.range_rows, a, sms, s)));
    else
        CG_CUDA_TRY((fp16 ? rows<__half, 64>(rows_map, pl.range_rows, a, sms, s) : rows<__nv_bfloat16, 64>(rows_map, pl.range_rows, a, sms, s)));
    CG_CUDA_TRY(launch_joins(at->dtype, at->head_dim, false, a, sms, s));
    return CG_OK;
}

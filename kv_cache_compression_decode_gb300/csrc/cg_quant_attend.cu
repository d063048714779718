// cg_quant_attend.cu -- attention of a batch of sequences in a paged pool of 4
// or 8 bits (sm_103a).
//
// Parts, pieces and joins are those of cg_attend.cu.  A few query rows go
// against the codes as they lie (cg_quant_rows.cuh).  The shared blocks of many
// rows are bound by the tensor cores: their tokens are read into the workspace
// once, as 16-bit values, and k_shared takes them from there.
#include "cg_quant_rows.cuh"

namespace cg {
namespace {

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) != 0; }

// Whether the shared blocks go through the workspace, by the row ranges that k_quant_rows would take over them (of 8 query
// rows of a KV head, or of 16, which cost half as much again) and the tokens.  Microseconds a call, through the workspace /
// in k_quant_rows, fp16, 8 KV heads: 2048 shared tokens, 64 rows 28 / 21, 128 rows 25 / 25; 8192 tokens, 64 rows 33 / 35,
// 96 rows 33 / 44; 32768 tokens, 48 rows 80 / 69, 64 rows 83 / 91, 128 rows 83 / 163.  bf16, whose K goes in two parts:
// 8192 tokens, 64 rows 39 / 37, 96 rows 38 / 46; 32768 tokens, 64 rows 102 / 97, 96 rows 101 / 136.  The workspace costs
// two launches and about the time of eight ranges.  Up to 64 rows go against the codes at any length: up to 9% slower with
// fp16, up to 5% faster with bf16, without the values' rounding and without their memory.  (8 bits, groups of 32 and heads
// of 64 go by the same rule and were not measured for it.)
bool by_workspace(uint64_t ranges, uint32_t kN, uint64_t tokens, uint32_t heads) {
    const uint64_t half = ranges * (kN == 1 ? 2 : 3);
    return half > 16 && (half - 16) * tokens * heads > 160000;
}
constexpr uint32_t kStageBytes = 214u << 10;  // shared memory for an SM's tiles in flight

struct Plan {
    uint32_t g, nh, ng, hlog, tt, kN, rt, npt, pairs, one, piece_rows;
    uint32_t copies;  // matrices of values in the workspace
    uint64_t tc_rows, cum_bytes, o_bytes, ml_bytes, bytes;
};

bool make_plan(const cg_pages *p, const cg_quant *f, const cg_attention *a, Plan *o) {
    if (!quant_ok(f) || !attention_ok(p, a)) return false;
    if (p->C != quant_row(f) || a->dtype != f->dtype || a->n_kv_heads != f->n_kv_heads || a->head_dim != f->head_dim) return false;
    const uint32_t Hkv = a->n_kv_heads;
    o->g = a->n_q_heads / Hkv;
    constexpr uint64_t kMost = 1ull << 31;  // query rows; compared before each product, so that none wraps
    const uint64_t per = (uint64_t)a->n_queries * o->g;
    if (per > kMost || per * a->n_requests > kMost) return false;
    const uint64_t all = per * a->n_requests;
    if (all * Hkv > kMost) return false;
    // Neighbouring heads of a block, a warp or more to each: eight or four where that leaves no warp without a head,
    // otherwise the next power of two.
    o->hlog = Hkv % 8 == 0 ? 3 : Hkv % 4 == 0 ? 2 : Hkv > 4 ? 3 : Hkv > 2 ? 2 : Hkv - 1;
    o->nh = 1u << o->hlog;
    o->ng = (Hkv + o->nh - 1) / o->nh;
    o->tt = quant_tok(f->bits, f->head_dim) * (kQuantWarps >> o->hlog);
    o->kN = per > 8 ? 2 : 1;
    const uint32_t range = 8 * o->kN;
    const bool tc = a->shared_blocks && by_workspace((all + range - 1) / range, o->kN, (uint64_t)a->shared_blocks * p->block_tokens, Hkv);
    o->pairs = tc ? (uint32_t)((all + 255) / 256) : 0;
    o->one = all <= 128;
    const bool here = a->shared_blocks && !tc;  // the shared part goes through k_quant_rows too
    const uint64_t most = here ? all : per;
    o->rt = (uint32_t)((per + range - 1) / range);
    o->npt = here ? (uint32_t)((all + range - 1) / range) : 0;
    o->piece_rows = (uint32_t)(most < range ? most : range);
    const uint64_t items = ((uint64_t)a->n_requests * o->rt + o->npt) * o->ng;
    if (items > (1ull << 31)) return false;
    o->tc_rows = tc ? ((uint64_t)o->pairs * Hkv + kMaxTcCtas) * 256 : 0;
    const uint64_t rows = o->tc_rows + (items + kMaxCtas) * kQuantWarps * o->piece_rows;  // of partial results
    if (rows > 0xFFFFFFFFull) return false;
    o->cum_bytes = round_up((a->n_requests + 1ull) * 8 + a->n_requests * 4ull, 256);
    o->o_bytes = round_up(rows * a->head_dim * 4, 256);
    o->ml_bytes = round_up(rows * 8, 256);
    o->bytes = o->cum_bytes + o->o_bytes + o->ml_bytes;
    // K and V, and with bf16 what rounding K to its 8 bits left, as a second K: a score is a sum of hundreds of products
    // and lse shows their rounding (2e-3 of it with K alone; fp16's 11 bits leave 6e-6 of it, where the codes leave 6e-7)
    o->copies = f->dtype == CG_BF16 ? 3 : 2;
    if (tc) o->bytes += round_up((uint64_t)a->shared_blocks * p->block_tokens * quant_channels(f) * 2 * o->copies, 256);
    return true;
}

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" cg_status cg_quant_attend_ws_bytes(const cg_pages *p, const cg_quant *f, const cg_attention *a, size_t *ws_bytes) {
    Plan pl;
    if (!ws_bytes || !make_plan(p, f, a, &pl)) return CG_ERR_INVALID_ARG;
    *ws_bytes = pl.bytes;
    return CG_OK;
}

extern "C" cg_status cg_quant_attend(const cg_pages *p, const cg_quant *f, const cg_attention *at, void *ws, size_t ws_bytes,
                                     uint32_t *dev_status, void *stream) {
    Plan pl;
    if (!make_plan(p, f, at, &pl) || !ws || misaligned(ws, 256)) return CG_ERR_INVALID_ARG;
    if (ws_bytes < pl.bytes) return CG_ERR_RANGE;
    int dev = 0, sms = 0;
    CG_CUDA_TRY(cudaGetDevice(&dev));
    CG_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const uint32_t bt = p->block_tokens, bshift = (uint32_t)__builtin_ctz(bt), C = quant_channels(f);
    const uint32_t head_bytes = f->head_dim * f->bits / 8, n_groups = f->head_dim / f->group;

    QuantArgs q{};
    q.cols = (pl.nh * head_bytes + 127) / 128;
    q.pw = pl.nh * n_groups * 4 < 16 ? 16 : pl.nh * n_groups * 4;
    q.tile = pl.tt * q.cols * 128;
    q.ptile = pl.tt * q.pw;
    q.stage = (uint32_t)round_up(2 * (q.tile + q.ptile), 1024);
    const uint32_t room = kStageBytes / q.stage;
    q.n_stages = room < kQuantMaxStages ? room : kQuantMaxStages;
    q.scale2 = fminf(fmaxf(fabsf(at->scale) * 1.4426950408889634f, 0x1p-149f), 0x1p127f);  // not 0: masked scores are -inf before the product; nor infinite

    const uint16_t *layer = p->pool + at->layer * p->layer_stride;
    const uint32_t box = bt < pl.tt ? bt : pl.tt, codes = quant_codes(f);
    CUtensorMap code_map, pair_map, map;
    if (!make_token_map(p, layer, codes, 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B, &code_map) ||
        !make_token_map(p, layer + codes, p->C - codes, 2, q.pw / 2, box, CU_TENSOR_MAP_SWIZZLE_NONE, &pair_map))
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
    a.hlog = pl.hlog;
    a.tlog = (uint32_t)__builtin_ctz(pl.tt);
    a.rlog = pl.kN == 1 ? 3 : 4;
    a.over = 3;
    a.rt = pl.rt;
    a.npt = pl.npt;
    a.pairs = pl.pairs;
    a.one = pl.one;
    for (int k = 0; k < 3; k++) {
        a.qs[k] = at->q_stride[k];
        a.os[k] = at->out_stride[k];
    }
    a.scale2 = q.scale2;
    a.flip = at->scale < 0.f ? 0x80008000u : 0u;
    a.status = dev_status;
    uint8_t *w = static_cast<uint8_t *>(ws);
    a.cum = reinterpret_cast<uint64_t *>(w);
    a.tokens = reinterpret_cast<uint32_t *>(a.cum + a.R + 1);
    a.part_o = reinterpret_cast<float *>(w + pl.cum_bytes);
    a.part_ml = reinterpret_cast<float2 *>(w + pl.cum_bytes + pl.o_bytes);
    a.piece_rows = pl.piece_rows;
    a.part0 = (uint32_t)pl.tc_rows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    if (a.pairs) {
        // the shared tokens' values, [K/V][token][C], as a pool of blocks in their order
        uint16_t *values = reinterpret_cast<uint16_t *>(w + pl.cum_bytes + pl.o_bytes + pl.ml_bytes);
        TokenRows t{};
        t.k = values;
        t.v = values + (uint64_t)a.P * C;
        t.k_rest = pl.copies == 3 ? values + 2ull * a.P * C : nullptr;
        t.n_seqs = 1;
        t.n_rows = t.per = t.fixed = a.P;
        t.ks[1] = t.vs[1] = C;
        t.slot0 = a.shared_slot;
        t.zero = 1;
        CG_CUDA_TRY(quant_read(quant_pool(p, f, at->layer), t, 1, f->dtype, f->bits, dev_status, s));
        cg_pages v{};
        v.C = C;
        v.n_pool_blocks = at->shared_blocks;
        v.block_tokens = bt;
        v.kv_stride = (uint64_t)a.P * C;
        v.block_stride = (uint64_t)bt * C;
        v.token_stride = C;
        if (!make_token_map(&v, values, C, pl.copies, 64, bt < 64 ? bt : 64, CU_TENSOR_MAP_SWIZZLE_128B, &map)) return CG_ERR_CUDA;
        Args b = a;
        b.tables = nullptr;
        b.n_pool = at->shared_blocks;
        b.after = 1;
        CG_CUDA_TRY(launch_shared(at->dtype, at->head_dim, pl.copies == 3, map, b, sms, s));
        a.n_tc = b.n_tc;
    }
    const bool half = f->dtype == CG_FP16;
    const auto rows = f->bits == 4 ? f->head_dim == 128 ? half ? launch_quant_rows_4_128_f : launch_quant_rows_4_128_b
                                                        : half ? launch_quant_rows_4_64_f : launch_quant_rows_4_64_b
                                   : f->head_dim == 128 ? half ? launch_quant_rows_8_128_f : launch_quant_rows_8_128_b
                                                        : half ? launch_quant_rows_8_64_f : launch_quant_rows_8_64_b;
    CG_CUDA_TRY(rows(f->group, pl.kN, code_map, pair_map, a, q, sms, s));
    CG_CUDA_TRY(launch_joins(at->dtype, at->head_dim, true, a, sms, s));
    return CG_OK;
}

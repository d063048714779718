// cg_quant.cuh -- a paged pool in 4 or 8 bits: its format on the host, and the
// two 16-bit types (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cg_internal.cuh"

namespace cg {

inline bool quant_ok(const cg_quant *f) {
    return f && f->dtype <= CG_BF16 && (f->bits == 4 || f->bits == 8) &&
           (f->group == 32 || f->group == 64 || f->group == 128) && (f->head_dim == 64 || f->head_dim == 128) &&
           f->group <= f->head_dim && f->n_kv_heads && f->n_kv_heads <= (1u << 20);
}
inline uint32_t quant_channels(const cg_quant *f) { return f->n_kv_heads * f->head_dim; }
// 16-bit words of a row's codes, and of the whole row
inline uint32_t quant_codes(const cg_quant *f) { return quant_channels(f) * f->bits / 16; }
inline uint32_t quant_row(const cg_quant *f) {
    return (uint32_t)round_up(quant_codes(f) + 2ull * (quant_channels(f) / f->group), 8);
}

// A row of 16-bit values read or written beside the pool.
struct TokenRows {
    uint16_t *k, *v;
    const uint32_t *slots, *first, *start;
    uint32_t n_seqs, n_rows, per;  // per: rows of a sequence where first is null
    uint64_t ks[2], vs[2];
    uint32_t slot0, fixed;         // slots null: sequence r is slot slot0 + r; fixed: its length (0: lens)
    uint16_t *k_rest;              // read: what the rounding of k left, or null
    uint32_t zero;                 // read: rows of a block outside the pool become zeros
};
struct QuantPool {
    uint16_t *pool;  // of the first layer
    const uint32_t *tables, *lens;
    uint32_t n_slots, n_blocks, n_pool, bshift;
    uint64_t layer, kv, block, token;  // strides in words
    uint32_t C, codes, group;
};

// Reads n_layers layers of `rows` (cg_quant.cu).
cudaError_t quant_read(const QuantPool &p, const TokenRows &rows, uint32_t n_layers, uint32_t dtype, uint32_t bits,
                       uint32_t *status, cudaStream_t s);
QuantPool quant_pool(const cg_pages *p, const cg_quant *f, uint32_t layer);

}  // namespace cg

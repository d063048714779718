// cg_quant_rows_8_128_b.cu -- k_quant_rows for 8-bit codes, heads of 128 channels and bf16 (sm_103a).
#define CG_QUANT_BITS 8
#include "cg_quant_rows.cuh"

namespace cg {

CG_QUANT_ROWS(launch_quant_rows_8_128_b) { return launch_rows<__nv_bfloat16, 8, 128>(group, n, codes, pairs, a, q, sms, s); }

}  // namespace cg

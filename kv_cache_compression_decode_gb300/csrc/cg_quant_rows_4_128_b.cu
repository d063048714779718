// cg_quant_rows_4_128_b.cu -- k_quant_rows for 4-bit codes, heads of 128 channels and bf16 (sm_103a).
#define CG_QUANT_BITS 4
#include "cg_quant_rows.cuh"

namespace cg {

CG_QUANT_ROWS(launch_quant_rows_4_128_b) { return launch_rows<__nv_bfloat16, 4, 128>(group, n, codes, pairs, a, q, sms, s); }

}  // namespace cg

// cg_quant_rows_8_128_f.cu -- k_quant_rows for 8-bit codes, heads of 128 channels and fp16 (sm_103a).
#define CG_QUANT_BITS 8
#include "cg_quant_rows.cuh"

namespace cg {

CG_QUANT_ROWS(launch_quant_rows_8_128_f) { return launch_rows<__half, 8, 128>(group, n, codes, pairs, a, q, sms, s); }

}  // namespace cg

// cg_quant_rows_4_64_f.cu -- k_quant_rows for 4-bit codes, heads of 64 channels and fp16 (sm_103a).
#define CG_QUANT_BITS 4
#include "cg_quant_rows.cuh"

namespace cg {

CG_QUANT_ROWS(launch_quant_rows_4_64_f) { return launch_rows<__half, 4, 64>(group, n, codes, pairs, a, q, sms, s); }

}  // namespace cg

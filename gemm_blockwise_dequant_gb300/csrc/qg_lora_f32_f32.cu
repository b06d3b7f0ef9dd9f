// qg_lora_f32_f32.cu -- the row kernels of the adapters for fp32 activations and fp32 adapters.
#include "qg_lora_rows.cuh"

namespace qg {

QG_DEFINE_LAUNCH_ROWS(kF32, kF32)

}  // namespace qg

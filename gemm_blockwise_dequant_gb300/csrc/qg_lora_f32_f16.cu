// qg_lora_f32_f16.cu -- the row kernels of the adapters for fp32 activations and fp16 adapters.
#include "qg_lora_rows.cuh"

namespace qg {

QG_DEFINE_LAUNCH_ROWS(kF32, kF16)

}  // namespace qg

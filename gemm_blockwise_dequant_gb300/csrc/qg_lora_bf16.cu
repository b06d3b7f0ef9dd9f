// qg_lora_bf16.cu -- the row kernels of the adapters for bf16 activations and bf16 adapters.
#include "qg_lora_rows.cuh"

namespace qg {

QG_DEFINE_LAUNCH_ROWS(kBF16, kBF16)

}  // namespace qg

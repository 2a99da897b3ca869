// The mixture-of-experts layer for bf16 rows (moe_layer.h).
#include "moe_layer.h"

namespace lora {
hipError_t launch_moe_bf16(const MoeCall& c, hipStream_t stream) { return launch_moe<BF16>(c, stream); }
}  // namespace lora

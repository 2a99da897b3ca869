// The mixture-of-experts layer for float32 rows (moe_layer.h).
#include "moe_layer.h"

namespace lora {
hipError_t launch_moe_f32(const MoeCall& c, hipStream_t stream) { return launch_moe<F32>(c, stream); }
}  // namespace lora

// The few-rows kernels for bf16 rows (w4_rows.h).
#include "w4_rows.h"

namespace lora {
hipError_t launch_w4_rows_bf16(const W4Call& c, hipStream_t stream) { return launch_rows_of<BF16>(c, stream); }
}  // namespace lora

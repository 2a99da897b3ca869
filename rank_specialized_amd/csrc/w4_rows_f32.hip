// The few-rows kernels for float32 rows (w4_rows.h).
#include "w4_rows.h"

namespace lora {
hipError_t launch_w4_rows_f32(const W4Call& c, hipStream_t stream) { return launch_rows_of<F32>(c, stream); }
}  // namespace lora

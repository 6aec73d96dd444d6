// int8_logits to float32 logits: kernel instances and dispatch.
#include "int8_tiles.hpp"

namespace tsr {

hipError_t launch_int8_dt0(const Int8Args& a, hipStream_t s) { return launch_int8_dt<0>(a, s); }

}  // namespace tsr

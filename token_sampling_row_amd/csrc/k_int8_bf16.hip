// int8_logits to bfloat16 logits: kernel instances and dispatch.
#include "int8_tiles.hpp"

namespace tsr {

hipError_t launch_int8_dt1(const Int8Args& a, hipStream_t s) { return launch_int8_dt<1>(a, s); }

}  // namespace tsr

// The bf16 instantiations of the linear attention kernel (ss_lattn.h).
#include "ss_lattn.h"

namespace ssk {

hipError_t launch_lattn_bf16(const LattnArgs& a, bool vec, hipStream_t stream) { return launch_typed<1>(a, vec, stream); }

}  // namespace ssk

// The fp32 instantiations of the linear attention kernel (ss_lattn.h).
#include "ss_lattn.h"

namespace ssk {

hipError_t launch_lattn_f32(const LattnArgs& a, bool vec, hipStream_t stream) { return launch_typed<0>(a, vec, stream); }

}  // namespace ssk

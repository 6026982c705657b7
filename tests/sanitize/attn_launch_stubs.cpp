// Host-only stand-ins for the kernel launchers behind ss_attn_api.cpp, as launch_stubs.cpp has
// them for ss_api.cpp: each only reports hipSuccess, or the code in SS_STUB_LAUNCH_ERROR.
#include <stdlib.h>

#include "ss_attn_internal.h"

namespace {
hipError_t stub_status()
{
    const char* v = getenv("SS_STUB_LAUNCH_ERROR");
    return v ? static_cast<hipError_t>(atoi(v)) : hipSuccess;
}
}  // namespace

namespace ssk {
hipError_t launch_lattn(const LattnArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_lattn_share(const float*, void*, int64_t, int64_t, int64_t, int64_t, int, hipStream_t)
{
    return stub_status();
}
hipError_t launch_lattn_step(const LattnStepArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_qknorm_fwd(const QknormArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_qknorm_bwd(const QknormArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_sample(const SampleArgs&, int, hipStream_t) { return stub_status(); }
}  // namespace ssk

// Host-only stand-ins for the kernel launchers behind ss_lm_api.cpp, as launch_stubs.cpp has
// them for ss_api.cpp: each only reports hipSuccess, or the code in SS_STUB_LAUNCH_ERROR.
#include <stdlib.h>

#include "ss_lm_internal.h"

namespace {
hipError_t stub_status()
{
    const char* v = getenv("SS_STUB_LAUNCH_ERROR");
    return v ? static_cast<hipError_t>(atoi(v)) : hipSuccess;
}
}  // namespace

namespace ssk {
hipError_t launch_pad_rows(const void*, int64_t, void*, int64_t, int64_t, int64_t, int, hipStream_t) { return stub_status(); }
hipError_t launch_few_grad(const FewGradArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_glu_fwd(const GluArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_glu_bwd(const GluArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_xent_fwd(const XentArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_xent_bwd(const XentArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_glr_fwd(const GlrArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_glr_bwd(const GlrArgs&, int, hipStream_t) { return stub_status(); }
hipError_t launch_glr_step(const GlrStepArgs&, int, hipStream_t) { return stub_status(); }
}  // namespace ssk

// Stand-ins for the launchers of the feed-forward calls, beside host_stubs.cpp
// (tests/test_sanitized_feed_forward.py).  TEST INFRASTRUCTURE ONLY: every
// launcher reports success without doing anything.
#include "launch_ffn.h"

namespace swz {

hipError_t launch_gated(const GatedJob&, hipStream_t) { return hipSuccess; }
hipError_t launch_gated_grad(const GatedJob&, const GatedPlan&, hipStream_t) { return hipSuccess; }
hipError_t launch_quant_w4(const QuantW4Job&, hipStream_t) { return hipSuccess; }
hipError_t launch_dequant_w4(const WeightsW4&, bool, int64_t, int64_t, int, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_gemm_w4(const GemmW4Job&, hipStream_t) { return hipSuccess; }
hipError_t launch_norm(const NormJob&, hipStream_t) { return hipSuccess; }

}  // namespace swz

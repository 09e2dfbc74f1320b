#include "delta.hpp"
namespace ssd {
hipError_t launch_delta_bwd_chain(const DeltaProb&, const DeltaArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_delta_bwd_grads(const DeltaProb&, const DeltaArgs&, hipStream_t) { return hipErrorNotSupported; }
}

// gate_logit.cu -- the gate's choice by the logits themselves (gate.cuh).
#define MOE_GATE_SELECT
#include "gate.cuh"

namespace moe {
template cudaError_t launch_gate_select<kKeyLogit>(const GateArgs &a, cudaStream_t s);
}  // namespace moe

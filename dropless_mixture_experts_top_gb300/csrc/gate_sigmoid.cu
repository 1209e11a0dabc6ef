// gate_sigmoid.cu -- the gate's choice by sigmoids (gate.cuh).
#define MOE_GATE_SELECT
#include "gate.cuh"

namespace moe {
template cudaError_t launch_gate_select<kKeySigmoid>(const GateArgs &a, cudaStream_t s);
}  // namespace moe

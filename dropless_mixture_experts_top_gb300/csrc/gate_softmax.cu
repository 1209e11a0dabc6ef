// gate_softmax.cu -- the gate's choice by softmax probabilities (gate.cuh).
#define MOE_GATE_SELECT
#include "gate.cuh"

namespace moe {
template cudaError_t launch_gate_select<kKeySoftmax>(const GateArgs &a, cudaStream_t s);
}  // namespace moe

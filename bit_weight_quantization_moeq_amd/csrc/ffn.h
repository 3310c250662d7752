// Launchers behind the gated feed-forward block over rows sorted by expert.
#pragma once

#include "grouped.h"

namespace moeq {

// g: x [M][kc], w = gate_up [E][2 nout][kc], out = h [M][nout]; gu: [M][2 nout]
// for the fp32 pre-activations, or null.
hipError_t launch_glu(const GroupedArgs& g, float* gu, hipStream_t s);

// g: x = grad_out [M][kc], w = down [E][kc][nout], out = h [M][nout]; gu (fp32) and
// dgu (bf16) [M][2 nout].
hipError_t launch_glu_backward(const GroupedArgs& g, const float* gu, uint16_t* dgu, hipStream_t s);

}  // namespace moeq

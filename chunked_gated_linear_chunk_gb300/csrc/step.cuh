// step.cuh -- the recurrence token by token on a pool of states (step.cu).
#pragma once

#include "internal.cuh"

namespace glacore {
namespace step {
// p has been checked; slots may be null (sequence b uses slot b).
cudaError_t launch(const glacore_problem *p, bool head_gate, float *state, int64_t n_slots, const int32_t *slots,
                   void *o, int *err, cudaStream_t st);
}  // namespace step
}  // namespace glacore

// Rotary positions (li_rope.cu): launcher.
#pragma once

#include "li_internal.cuh"

namespace li {

// grad: the transposed map (dy in args.x, dx in args.y).
cudaError_t launch_rope(const li_rope_args &a, bool grad, cudaStream_t st);

}  // namespace li

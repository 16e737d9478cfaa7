// Quantised key cache (li_cache.cu): launchers.
#pragma once

#include "li_internal.cuh"

namespace li {

cudaError_t launch_cache_write(const li_cache_args &a, cudaStream_t st);
cudaError_t launch_cache_read(const li_cache_args &a, cudaStream_t st);

}  // namespace li

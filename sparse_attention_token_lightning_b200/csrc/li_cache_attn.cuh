// Attention over selected rows of the E4M3 key cache (li_cache_attn.cu): work split, shared-memory
// plan and launcher.
#pragma once

#include "li_internal.cuh"

namespace li {

struct CacheAttnPlan {
    int N;                      // heads per CTA, padded (16 or 32): MMA N is 2 N (hi and lo parts)
    int head_blocks;            // CTAs' head ranges per row
    int tiles;                  // 128-entry tiles of a row's selection
    int64_t units;              // rows x head_blocks
    int cut_log2;               // CTAs that share a unit
    int grid;
    int blocks;                 // 128-dim blocks of a key (Dm / 128)
    int slots;
    uint32_t p_off, slot_off;
    uint32_t tmem_cols;
};

// False when the argument set does not fit the kernel.
bool cache_attn_plan(const li_cache_attn_args &a, CacheAttnPlan *p);

cudaError_t launch_cache_attention(const li_cache_attn_args &a, const CacheAttnPlan &p, void *out,
                                   float *smax, float *ssum, cudaStream_t st);

}  // namespace li

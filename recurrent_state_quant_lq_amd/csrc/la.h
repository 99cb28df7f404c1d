// Launches of linear attention and of drafted token trees (gfx950); arguments validated
// by the C entry points.
#pragma once

#include "lq_internal.h"

namespace lq {

// Linear attention with a decay per head.  alpha_heads: alpha is [H] instead of one per token.
hipError_t launch_la_prefill(const lq_dims& d, const float* h0, float* h, int T, const void* q, const void* k,
                             const void* v, const float* alpha, bool alpha_heads, const int32_t* lens, void* o,
                             void* workspace, hipStream_t s);
size_t la_workspace_bytes(const lq_dims& d, int T);
constexpr int kLaMaxTokens = 1 << 30;   // token counts and their rounding up to chunks stay in 32 bits
hipError_t launch_la_decode(const lq_dims& d, const lq_state& st, int pos, const int32_t* pos_dev, const void* q,
                            const void* k, const void* v, const float* alpha, bool alpha_heads, void* o,
                            hipStream_t s);

// Drafted token trees; beta null: plain linear attention (no delta rule).
hipError_t launch_tree(const lq_dims& d, const lq_state& st, const int32_t* pos, int N, const int32_t* parent,
                       const void* q, const void* k, const void* v, const float* alpha, bool alpha_heads,
                       const float* beta, void* o, float* tree_m, float* tree_g, hipStream_t s);
hipError_t launch_tree_commit(const lq_dims& d, const lq_state& st, const int32_t* pos, int N, const int32_t* path,
                              int P, const int32_t* n_path, const void* k, const float* tree_m,
                              const float* tree_g, hipStream_t s);
constexpr int kTreeMax = 64;   // nodes per row of a tree step

// Log decay of an alpha in [0, 1] of the lq_la_* calls: alpha = 0 (forget) as -110,
// whose exponential is 0 in fp32, so that differences of prefix sums stay finite.
constexpr float kLogForget = -110.0f;
__device__ __forceinline__ float log_decay(float alpha) { return alpha == 0.0f ? kLogForget : logf(alpha); }

}  // namespace lq

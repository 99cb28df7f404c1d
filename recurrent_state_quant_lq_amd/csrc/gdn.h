// Launches of the serving operators around the recurrent state: prompts of the gated delta
// rule, verification of drafted trees, rows of states moved (gfx950); arguments validated by
// the C entry points.
#pragma once

#include "lq_internal.h"

namespace lq {

// The gated delta rule over a padded batch of prompts.
hipError_t launch_gdn_prefill(const lq_dims& d, const float* h0, float* h, int T, const void* q, const void* k,
                              const void* v, const float* alpha, const float* beta, const int32_t* lens, void* o,
                              void* workspace, hipStream_t s);
size_t gdn_workspace_bytes(const lq_dims& d, int T);
constexpr int kGdnMaxTokens = 1 << 30;  // token counts and their rounding up to chunks stay in 32 bits
constexpr int kGdnMaxHeads = 1 << 23;   // a launch counts its threads in 32 bits
constexpr int kGdnStepTokens = 4;       // prompts of up to this many tokens run as the recurrence

// Drafted trees against the target's probabilities.
constexpr int kVerifyRows = 1 << 21;    // a launch counts its threads in 32 bits
constexpr int64_t kVerifyValues = (int64_t)1 << 36;
struct VerifyArgs {
    const int32_t* pos;
    const int32_t* parent;    // [B,N]
    const int32_t* token;     // [B,N]
    const float* target;      // [N,B,V]
    const float* target0;     // [B,V] or null
    const float* draft;       // [N,B,V] or null
    const float* draft0;      // [B,V] or null
    const float* u;           // [N+1,B]
    int32_t* path;            // [B,P]
    int32_t* n_path;
    int32_t* next;
    double* sums;             // workspace: [B][tiles], then the rows' walks
    int B, W, N, V, P, replace;
};
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);
size_t verify_workspace_bytes(int B, int N, int V);

// Rows of states.  Layer l of dst and src either the same arrays (in place) or disjoint ones.
hipError_t launch_gather(const lq_dims& d, int n_layers, const lq_state* dst, const lq_state* src, int src_rows,
                         const int32_t* index, const int32_t* pos, int32_t* pos_out, hipStream_t s);
constexpr int kGatherInPlace = 2048;    // rows of an in-place gather

}  // namespace lq

// tree.hip -- drafted token trees: the choice of the rule's kernels (tree.h), and the
// commit of an accepted path (gfx950).
#include "tree.h"

namespace lq {
namespace {

struct CommitArgs {
    float* bk;
    float* bm;
    float* bg;
    const int32_t* pos;
    const int32_t* path;
    const int32_t* n_path;
    const void* k;
    const float* tm;
    const float* tg;
    int N, P, W, H, heads, gd;
};

// One workgroup per (b, h): the path's slots, copied.
template <int D, typename TI>
__global__ __launch_bounds__((D < 64 ? 64 : D)) void commit_kernel(CommitArgs a) {
    const int t = threadIdx.x;
    const size_t head = blockIdx.x;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int pos = a.pos[b], n = a.n_path[b];
    if (pos < 0 || pos >= a.W || n < 1 || n > a.P || n > a.W - pos) return;
    const int32_t* path = a.path + (size_t)b * a.P;
    bool ok = true;
    for (int i = 0; i < n; ++i) ok &= path[i] >= 0 && path[i] < a.N;
    if (!ok) return;
    for (int i = 0; i < n; ++i) {
        const int node = path[i];
        const size_t slot = head * a.W + pos + i, from = head * a.N + node;
        if (t < D) {
            a.bk[slot * D + t] = tok_ld<TI>(a.k, ((size_t)node * a.heads + head) * D + t);
            a.bm[slot * D + t] = a.tm[from * D + t];
        }
        if (t < a.gd) a.bg[slot * a.gd + t] = a.tg[from * a.gd + t];
    }
}

template <int D>
hipError_t commit_t(const lq_dims& d, const CommitArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H), block(D < 64 ? 64 : D);
    if (d.io_dtype == LQ_IO_BF16) return launch_kernel(LQ_KERNEL_COMMIT, commit_kernel<D, uint16_t>, grid, block, s, args);
    return launch_kernel(LQ_KERNEL_COMMIT, commit_kernel<D, float>, grid, block, s, args);
}

}  // namespace

hipError_t launch_tree(const lq_dims& d, const lq_state& st, const int32_t* pos, int N, const int32_t* parent,
                       const void* q, const void* k, const void* v, const float* alpha, bool alpha_heads,
                       const float* beta, void* o, float* tree_m, float* tree_g, hipStream_t s) {
    TreeArgs args{st.sq, st.row_scale, st.col_scale, st.comp_idx, st.comp_val, st.buf_k, st.buf_m, st.buf_g,
                  pos, parent, q, k, v, alpha, beta, o, tree_m, tree_g, alpha_heads ? 0 : d.B * d.H,
                  N, d.W, d.C, d.H, d.B * d.H};
    if (!beta) return launch_tree_rule<TREE_LA>(d, args, s);
    return d.decay_mode == LQ_DECAY_PER_KEY ? launch_tree_rule<TREE_KDA>(d, args, s) : launch_tree_rule<TREE_GDN>(d, args, s);
}

hipError_t launch_tree_commit(const lq_dims& d, const lq_state& st, const int32_t* pos, int N, const int32_t* path,
                              int P, const int32_t* n_path, const void* k, const float* tree_m,
                              const float* tree_g, hipStream_t s) {
    CommitArgs args{st.buf_k, st.buf_m, st.buf_g, pos, path, n_path, k, tree_m, tree_g, N, P, d.W, d.H, d.B * d.H,
                    d.decay_mode == LQ_DECAY_PER_KEY ? d.dk : 1};
    switch (d.dk) {
        case 16: return commit_t<16>(d, args, s);
        case 64: return commit_t<64>(d, args, s);
        default: return commit_t<128>(d, args, s);
    }
}

}  // namespace lq

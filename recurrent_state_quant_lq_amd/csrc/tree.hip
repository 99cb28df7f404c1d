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

// One workgroup per (b, h): the path's slots, copied; D/4 lanes per slot (four values
// of each row a lane), all slots of up to 1024/D nodes at once.  A copy of a few rows, bound
// by the latency of path, then rows: 3 us for 16 heads, 7.7 us for 2048 heads (12-node paths).
template <int D, typename TI>
__global__ __launch_bounds__(256) void commit_kernel(CommitArgs a) {
    constexpr int LPS = D / 4, SPP = 256 / LPS;            // lanes per slot, slots per pass
    const int t = threadIdx.x, lane = t & 63;
    const size_t head = blockIdx.x;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int pos = a.pos[b], n = a.n_path[b];
    const int node_l = lane < a.P ? a.path[(size_t)b * a.P + lane] : 0;    // P <= 64
    if (pos < 0 || pos >= a.W || n < 1 || n > a.P || n > a.W - pos) return;
    if (__any(lane < n && (node_l < 0 || node_l >= a.N))) return;          // (every wave sees the whole path)
    const int c = 4 * (t % LPS);
    for (int i = t / LPS; i < n; i += SPP) {
        const int node = a.path[(size_t)b * a.P + i];
        const size_t slot = head * a.W + pos + i, from = head * a.N + node;
        const size_t kf = ((size_t)node * a.heads + head) * D + c;
        float k[4], m[4], g[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = tok_ld<TI>(a.k, kf + u);
        load_floats<4>(a.tm + from * D + c, m);
        if (a.gd > 1) load_floats<4>(a.tg + from * D + c, g);
        else if (c == 0) g[0] = a.tg[from];
        store_floats<4>(a.bk + slot * D + c, k);
        store_floats<4>(a.bm + slot * D + c, m);
        if (a.gd > 1) store_floats<4>(a.bg + slot * D + c, g);
        else if (c == 0) a.bg[slot] = g[0];
    }
}

template <int D>
hipError_t commit_t(const lq_dims& d, const CommitArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H), block(256);
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

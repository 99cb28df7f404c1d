// tree.hip -- a tree of drafted tokens over the int8 state and its window, and
// the commit of an accepted path (gfx950).
//
// Node n with parent p, window-base state Hb (fixed for the window) and context
// c = the window's slots and n's ancestors:
//     g_n = g_p + log alpha_n,   E_c = exp(g_n - g_c),
//     m_n = beta_n (v_n - Hb^T (e^{g_n} o k_n) - sum_c <k_n, E_c o k_c> m_c),
//     o_n = Hb^T (e^{g_n} o q_n) + sum_c <q_n, E_c o k_c> m_c + <q_n, k_n> m_n
// (plain linear attention: m_n = v_n), i.e. the decode step's sums with the
// window continued along the node's path.  The state and the window are read
// once for all N nodes.
//
// One workgroup per (b, h), lane j = channel j = value column j, node after node.
#include "lq_internal.h"

namespace lq {
namespace {

struct TreeArgs {
    const int8_t* sq;
    const float* r;
    const float* s;
    const int32_t* idx;
    const float* cv;
    const float* bk;
    const float* bm;
    const float* bg;
    const int32_t* pos;
    const int32_t* parent;
    const void* q;            // q, k, v, o: fp32 or bf16 (the kernel's TI)
    const void* k;
    const void* v;
    const float* alpha;
    const float* beta;
    void* o;
    float* tm;
    float* tg;
    int alpha_tok;            // token stride of alpha in heads: B*H, or 0 (one decay per head)
    int N, W, C, H, heads;
};

constexpr int WMAX = 32;

// Bit i of masks[n]: node i is an ancestor of node n; here: the nodes that are
// present.  A parent outside [-1, n) or an absent parent leaves a node absent, so
// no later index depends on an unchecked value.
__device__ __forceinline__ uint64_t tree_masks(const int32_t* parent, int N, uint64_t* masks, int8_t* par) {
    uint64_t here = 0;
    for (int n = 0; n < N; ++n) {
        const int p = parent[n];
        const bool root = p == -1, child = p >= 0 && p < n && ((here >> p) & 1u);
        masks[n] = child ? masks[p] | (1ull << p) : 0;
        par[n] = (int8_t)(child ? p : -1);
        if (root || child) here |= 1ull << n;
    }
    return here;
}

template <int D, bool KDA, bool DELTA, typename TI>
__global__ __launch_bounds__((D < 64 ? 64 : D)) void tree_kernel(TreeArgs a) {
    constexpr int NT = D < 64 ? 64 : D, NW = NT / 64, GD = KDA ? D : 1;
    __shared__ uint64_t s_mask[kTreeMax];
    __shared__ int8_t s_par[kTreeMax];
    __shared__ uint64_t s_here;
    __shared__ float sg[kTreeMax * GD];
    __shared__ __align__(16) float sx[2][D], st[2][D];     // r o e^g o (q, k); q, k
    __shared__ float sc[2][WMAX + kTreeMax + 1];           // <q, E k_c>, <k, E k_c>; <q, k> last
    __shared__ float sm[kTreeMax * D];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int W = a.W, C = a.C, N = a.N;
    const int pos = a.pos[b];
    if (pos < 0 || pos > W) return;                        // a row outside its window: untouched
    if (t == 0) s_here = tree_masks(a.parent + (size_t)b * N, N, s_mask, s_par);
    __syncthreads();
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W * GD;
    for (int n = 0; n < N; ++n) {
        if (!((s_here >> n) & 1u)) continue;               // absent: untouched
        const size_t th = (size_t)n * heads + head;
        const int par = s_par[n];
        const uint64_t anc = s_mask[n];
        if (t < D) {
            st[0][t] = tok_ld<TI>(a.q, th * D + t);
            st[1][t] = tok_ld<TI>(a.k, th * D + t);
        }
        if (t < GD) {
            const float al = KDA ? a.alpha[th * D + t] : a.alpha_tok ? a.alpha[(size_t)n * a.alpha_tok + head] : a.alpha[head % (unsigned)a.H];
            const float g = (par >= 0 ? sg[par * GD + t] : pos > 0 ? bg[(size_t)(pos - 1) * GD + t] : 0.0f) +
                            (DELTA ? __logf(al) : log_decay(al));
            sg[n * GD + t] = g;
            a.tg[(head * N + n) * GD + t] = g;
        }
        __syncthreads();
        if (t < D) {
            const float e = expf(sg[n * GD + (KDA ? t : 0)]), r = a.r[head * D + t];
            sx[0][t] = r * (e * st[0][t]);
            sx[1][t] = r * (e * st[1][t]);
        }
        for (int c = w; c <= pos + n; c += NW) {           // slots, nodes before n, n itself
            const int i = c - pos;
            if (i >= 0 && i < n && !((anc >> i) & 1u)) continue;
            float xq = 0.0f, xk = 0.0f;
            for (int ch = lane; ch < D; ch += 64) {
                float kc = i < 0 ? bk[(size_t)c * D + ch] : tok_ld<TI>(a.k, ((size_t)i * heads + head) * D + ch);
                if (KDA && i < n) kc *= expf(sg[n * GD + ch] - (i < 0 ? bg[(size_t)c * GD + ch] : sg[i * GD + ch]));
                xq += st[0][ch] * kc;
                xk += st[1][ch] * kc;
            }
            xq = group_sum<64>(xq);
            xk = group_sum<64>(xk);
            const float e = KDA || i == n ? 1.0f : expf(sg[n] - (i < 0 ? bg[c] : sg[i]));
            if (lane == 0) {
                const int at = i < 0 ? c : WMAX + i;
                sc[0][at] = xq * e;
                sc[1][at] = xk * e;
            }
        }
        __syncthreads();
        if (t < D) {
            float hq = 0.0f, hk = 0.0f;
            for (int c = 0; c < D; c += 16) {
                const v4i x = *reinterpret_cast<const v4i*>(a.sq + head * (size_t)(D * D) + sq_off<D>(c, t));
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const float y = sbyte((uint32_t)x[u / 4], u % 4);
                    hq += y * sx[0][c + u];
                    hk += y * sx[1][c + u];
                }
            }
            const float s = a.s[head * D + t];
            hq *= s;
            hk *= s;
            for (int c = 0; c < C; ++c) {
                const int ic = a.idx[head * C + c] & (D - 1);
                const float y = a.cv[(head * C + c) * D + t] * expf(sg[n * GD + (KDA ? ic : 0)]);
                hq += st[0][ic] * y;
                hk += st[1][ic] * y;
            }
            for (int c = 0; c < pos; ++c) {
                const float m = bm[(size_t)c * D + t];
                hq += sc[0][c] * m;
                hk += sc[1][c] * m;
            }
            for (int i = 0; i < n; ++i)
                if ((anc >> i) & 1u) {
                    hq += sc[0][WMAX + i] * sm[i * D + t];
                    hk += sc[1][WMAX + i] * sm[i * D + t];
                }
            const float v = tok_ld<TI>(a.v, th * D + t);
            const float m = DELTA ? a.beta[th] * (v - hk) : v;
            sm[n * D + t] = m;
            a.tm[(head * N + n) * D + t] = m;
            tok_st<TI>(a.o, th * D + t, hq + sc[0][WMAX + n] * m);
        }
        __syncthreads();                                   // st, sx, sc are rewritten by the next node
    }
}

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

template <int D, typename TI>
hipError_t tree_t(const lq_dims& d, const TreeArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H), block(D < 64 ? 64 : D);
    if (!args.beta) return launch_kernel(LQ_KERNEL_TREE, tree_kernel<D, false, false, TI>, grid, block, s, args);
    if (d.decay_mode == LQ_DECAY_PER_KEY)
        return launch_kernel(LQ_KERNEL_TREE, tree_kernel<D, true, true, TI>, grid, block, s, args);
    return launch_kernel(LQ_KERNEL_TREE, tree_kernel<D, false, true, TI>, grid, block, s, args);
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
    const bool bf16 = d.io_dtype == LQ_IO_BF16;
    switch (d.dk) {
        case 16: return bf16 ? tree_t<16, uint16_t>(d, args, s) : tree_t<16, float>(d, args, s);
        case 64: return bf16 ? tree_t<64, uint16_t>(d, args, s) : tree_t<64, float>(d, args, s);
        default: return bf16 ? tree_t<128, uint16_t>(d, args, s) : tree_t<128, float>(d, args, s);
    }
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

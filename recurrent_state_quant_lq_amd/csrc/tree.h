// Kernels of a drafted token tree over the int8 state and its window (gfx950).
//
// Node n with parent p, window-base state Hb (fixed for the window) and context
// c = the window's slots and n's ancestors:
//     g_n = g_p + log alpha_n,   E_c = exp(g_n - g_c),
//     m_n = beta_n (v_n - Hb^T (e^{g_n} o k_n) - sum_c <k_n, E_c o k_c> m_c),
//     o_n = Hb^T (e^{g_n} o q_n) + sum_c <q_n, E_c o k_c> m_c + <q_n, k_n> m_n
// (plain linear attention: m_n = v_n), i.e. the decode step's sums with the
// window continued along the node's path.  The state and the window are read
// once for all N nodes.
#pragma once

#include "lq_internal.h"
#include "lq_split.h"

namespace lq {

enum TreeRule { TREE_LA = 0, TREE_GDN = 1, TREE_KDA = 2 };

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


// The launch of one rule's kernels (each rule's kernels are a source of their own).
template <int RULE>
hipError_t launch_tree_rule(const lq_dims& d, const TreeArgs& args, hipStream_t s);

#ifdef LQ_TREE_KERNELS
namespace {

// Presence and ancestors of a row's nodes, lane n = node n: own = whether the node's
// parent entry is valid (-1 or an earlier node), mask = its ancestors while every
// entry on the way up is valid.  A node is present if its own entry and all its
// ancestors' are; no index depends on an unchecked value.  sum: of x over the path
// (the node included), by pointer doubling.
struct TreeNode {
    uint64_t mask;
    float sum;
    int parent;               // -1: the last committed token
    bool here;
};
__device__ __forceinline__ TreeNode tree_node(const int32_t* parent, int N, int lane, float x) {
    const int p = lane < N ? parent[lane] : -2;
    const bool own = p == -1 || (p >= 0 && p < lane);
    int jump = own ? p : -1;
    TreeNode t;
    t.parent = jump;
    t.mask = jump >= 0 ? 1ull << jump : 0;
    t.sum = x;
#pragma unroll
    for (int i = 0; i < 6; ++i) {                          // paths of doubling length; at most 64 nodes
        const int from = jump >= 0 ? jump : lane;
        const uint64_t m = __shfl(t.mask, from, 64);
        const float y = __shfl(t.sum, from, 64);
        const int j = __shfl(jump, from, 64);
        if (jump >= 0) {
            t.mask |= m;
            t.sum += y;
            jump = j;
        }
    }
    const uint64_t valid = __ballot(own);
    t.here = own && (t.mask & ~valid) == 0;
    return t;
}

// ---------------------------------------------------------------------------
// node after node: d = 16, and rows that hold a value that is not finite
// ---------------------------------------------------------------------------
// Lane j = channel j = value column j.  Sums run over a node's own context only, so
// a value that is not finite reaches its descendants and nothing else.
template <int D>
struct TreeSimple {
    float x[2][D];            // r o e^g o (q, k)
    float t[2][D];            // q, k
    float c[2][32 + kTreeMax + 1];   // <q, E k_c>, <k, E k_c> of the window and the nodes
};

template <int D, int RULE, typename TI, int NT>
__device__ void tree_simple(const TreeArgs& a, int pos, const uint64_t* s_mask, const int8_t* s_par, uint64_t here,
                            TreeSimple<D>& s) {
    constexpr bool KDA = RULE == TREE_KDA, DELTA = RULE != TREE_LA;
    constexpr int NW = NT / 64, GD = KDA ? D : 1;
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int W = a.W, C = a.C, N = a.N;
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W * GD;
    float* tg = a.tg + head * (size_t)N * GD;              // this workgroup's rows: written, then read back
    float* tm = a.tm + head * (size_t)N * D;
    for (int n = 0; n < N; ++n) {
        if (!((here >> n) & 1u)) continue;                 // absent: untouched
        const size_t th = (size_t)n * heads + head;
        const int par = s_par[n];
        const uint64_t anc = s_mask[n];
        if (t < D) {
            s.t[0][t] = tok_ld<TI>(a.q, th * D + t);
            s.t[1][t] = tok_ld<TI>(a.k, th * D + t);
        }
        if (t < GD) {
            const float al = KDA ? a.alpha[th * D + t] : a.alpha_tok ? a.alpha[(size_t)n * a.alpha_tok + head] : a.alpha[head % (unsigned)a.H];
            tg[n * GD + t] = (par >= 0 ? tg[par * GD + t] : pos > 0 ? bg[(size_t)(pos - 1) * GD + t] : 0.0f) +
                             (DELTA ? logf(al) : log_decay(al));
        }
        __syncthreads();
        if (t < D) {
            const float e = expf(tg[n * GD + (KDA ? t : 0)]), r = a.r[head * D + t];
            s.x[0][t] = r * (e * s.t[0][t]);
            s.x[1][t] = r * (e * s.t[1][t]);
        }
        for (int c = w; c <= pos + n; c += NW) {           // slots, nodes before n, n itself
            const int i = c - pos;
            if (i >= 0 && i < n && !((anc >> i) & 1u)) continue;
            float xq = 0.0f, xk = 0.0f;
            for (int ch = lane; ch < D; ch += 64) {
                float kc = i < 0 ? bk[(size_t)c * D + ch] : tok_ld<TI>(a.k, ((size_t)i * heads + head) * D + ch);
                if (KDA && i < n) kc *= expf(tg[n * GD + ch] - (i < 0 ? bg[(size_t)c * GD + ch] : tg[i * GD + ch]));
                xq += s.t[0][ch] * kc;
                xk += s.t[1][ch] * kc;
            }
            xq = group_sum<64>(xq);
            xk = group_sum<64>(xk);
            const float e = KDA || i == n ? 1.0f : expf(tg[n] - (i < 0 ? bg[c] : tg[i]));
            if (lane == 0) {
                const int at = i < 0 ? c : 32 + i;
                s.c[0][at] = xq * e;
                s.c[1][at] = xk * e;
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
                    hq += y * s.x[0][c + u];
                    hk += y * s.x[1][c + u];
                }
            }
            const float sj = a.s[head * D + t];
            hq *= sj;
            hk *= sj;
            for (int c = 0; c < C; ++c) {
                const int ic = a.idx[head * C + c] & (D - 1);
                const float y = a.cv[(head * C + c) * D + t] * expf(tg[n * GD + (KDA ? ic : 0)]);
                hq += s.t[0][ic] * y;
                hk += s.t[1][ic] * y;
            }
            for (int c = 0; c < pos; ++c) {
                const float m = bm[(size_t)c * D + t];
                hq += s.c[0][c] * m;
                hk += s.c[1][c] * m;
            }
            for (int i = 0; i < n; ++i)
                if ((anc >> i) & 1u) {
                    const float m = tm[i * D + t];
                    hq += s.c[0][32 + i] * m;
                    hk += s.c[1][32 + i] * m;
                }
            const float v = tok_ld<TI>(a.v, th * D + t);
            const float m = DELTA ? a.beta[th] * (v - hk) : v;
            tm[n * D + t] = m;
            tok_st<TI>(a.o, th * D + t, hq + s.c[0][32 + n] * m);
        }
        __syncthreads();                                   // s is rewritten by the next node
    }
}

// Node tables of the workgroup's row, by wave 0.
struct TreeTables {
    uint64_t mask[kTreeMax];
    int8_t par[kTreeMax];
    uint64_t here;
};

template <int D, int RULE, typename TI>
__global__ __launch_bounds__((D < 64 ? 64 : D)) void tree_kernel(TreeArgs a) {
    constexpr int NT = D < 64 ? 64 : D;
    __shared__ TreeTables s_t;
    __shared__ TreeSimple<D> s_s;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int pos = a.pos[b];
    if (pos < 0 || pos > a.W) return;                      // a row outside its window: untouched
    if (threadIdx.x < 64) {
        const TreeNode nd = tree_node(a.parent + (size_t)b * a.N, a.N, threadIdx.x, 0.0f);
        s_t.mask[threadIdx.x] = nd.mask;
        s_t.par[threadIdx.x] = (int8_t)nd.parent;
        const uint64_t here = __ballot(nd.here);
        if (threadIdx.x == 0) s_t.here = here;
    }
    __syncthreads();
    tree_simple<D, RULE, TI, NT>(a, pos, s_t.mask, s_t.par, s_t.here, s_s);
}

// ---------------------------------------------------------------------------
// d >= 64: blocks of 16 nodes on matrix products
// ---------------------------------------------------------------------------
// Wave w owns the 32 value columns 32 w + 2 li + ct.  Per block of 16 nodes:
//   1. the block's q and k rows to LDS as bf16 parts (one for bf16 tokens with a
//      decay per head; else three; per-key decay: rows scaled by e^{g_n - g_pos},
//      at most 1);
//   2. scores against the window's keys (three parts in LDS; per-key decay: scaled by
//      e^{g_pos - g_c}) and the nodes' keys, times E and the ancestor mask; those of
//      k times -beta.  Per-key decay takes the nodes' scores pair by pair, with the
//      exponential of each channel's difference: a product of two factors could
//      overflow;
//   3. one wave inverts the block's I + A, A_{n,i} = beta_n <k_n, E k_i> (strictly
//      lower triangular in node order); the others begin
//   4. the products with the state, r o sq in three bf16 parts in registers;
//   5. R = beta (v - Hb^T k) - A_ctx M_ctx, M = (I + A)^{-1} R, O = Hb^T q + S M on the
//      fp32 matrix instruction: accumulators are its B operand as they are, so M
//      never leaves the registers.
// A product of a masked zero with a value that is not finite would spread it: if any
// m is not finite, the row is computed again node after node.
template <int D, int NB, int WT, int RULE, typename TI>
struct TM {
    static constexpr int NW = D / 32, NT = 64 * NW;
    static constexpr bool KDA = RULE == TREE_KDA, DELTA = RULE != TREE_LA;
    static constexpr int NP = sizeof(TI) == 2 && !KDA ? 1 : 3;     // parts of a token row
    static constexpr int KB = KDA ? 1 : NB;                        // blocks whose keys stay in LDS
    static constexpr int QS = D + 8;                               // shorts per row
    static constexpr int WC = 16 * WT;                             // window columns of the scores
    static constexpr int SS = WC + 16 * NB + 4;                    // floats per score row
    struct Shared {
        TreeTables t;
        float g[kTreeMax], e[kTreeMax], beta[kTreeMax];            // scalar decay: g_n, e^{g_n}
        float wg[32];                                              // scalar decay: the window's g
        __align__(16) uint16_t q[NP][16 * QS];
        __align__(16) uint16_t k[NP][16 * KB * QS];
        __align__(16) uint16_t wk[3][WC * QS];
        __align__(16) float s[2][16 * SS];                         // scores of q; -beta times those of k
        __align__(16) float inv[16 * 20];                          // (I + A)^{-1}
        __align__(16) float gk[KDA ? 16 * NB * D : 4];             // per-key decay: g_n
        __align__(16) float gp[KDA ? D : 4];                       // per-key decay: g of slot pos - 1
    };
    union Space {
        Shared m;
        struct {
            TreeTables t;
            TreeSimple<D> s;
        } f;
    };
};

// c += a b with a in NP parts, b in three; small products first.
template <int NP>
__device__ __forceinline__ v4f mfma_parts(const u32x4 (&a)[NP], const u32x4 (&b)[3], v4f c) {
    if constexpr (NP == 3) return mfma_split(a, b, c);
    c = mfma_bf16(a[0], b[2], c);
    c = mfma_bf16(a[0], b[1], c);
    return mfma_bf16(a[0], b[0], c);
}

template <int D, int NB, int WT, int RULE, typename TI>
__global__ __launch_bounds__((TM<D, NB, WT, RULE, TI>::NT), 2) void tree_mfma_kernel(TreeArgs a) {
    using X = TM<D, NB, WT, RULE, TI>;
    constexpr int NW = X::NW, NT = X::NT, NP = X::NP, KB = X::KB, QS = X::QS, WC = X::WC, SS = X::SS;
    constexpr bool KDA = X::KDA, DELTA = X::DELTA;
    constexpr int NX = DELTA ? 2 : 1, GD = KDA ? D : 1, KS = D / 64;
    __shared__ typename X::Space sp;
    auto& s = sp.m;

    const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int W = a.W, C = a.C, N = a.N;
    const int pos = a.pos[b];
    if (pos < 0 || pos > W) return;                        // a row outside its window: untouched
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W * GD;
    const int col = 32 * w + 2 * li;                       // and col + 1

    // ---- the state's bytes: columns col + ct, channels 64 ks + 16 lg .. + 15 ----
    v4i raw[KS][2];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
            raw[ks][ct] = *reinterpret_cast<const v4i*>(a.sq + head * (size_t)(D * D) + sq_off<D>(64 * ks + 16 * lg, col + ct));

    // ---- node tables ----
    if (w == 0) {
        float al = 0.0f;
        const size_t th = (size_t)min(lane, N - 1) * heads + head;
        if constexpr (!KDA) {
            al = a.alpha_tok ? a.alpha[(size_t)min(lane, N - 1) * a.alpha_tok + head] : a.alpha[head % (unsigned)a.H];
            al = DELTA ? logf(al) : log_decay(al);
        }
        const TreeNode nd = tree_node(a.parent + (size_t)b * N, N, lane, al);
        s.t.mask[lane] = nd.here ? nd.mask : 0;
        s.t.par[lane] = (int8_t)nd.parent;
        const uint64_t here = __ballot(nd.here);
        if (lane == 0) s.t.here = here;
        if constexpr (DELTA) s.beta[lane] = nd.here ? a.beta[th] : 0.0f;
        if constexpr (!KDA) {
            const float g = nd.sum + (pos > 0 ? bg[pos - 1] : 0.0f);
            s.g[lane] = g;
            s.e[lane] = expf(g);
            if (nd.here) a.tg[head * N + lane] = g;
            if (lane < 32) s.wg[lane] = lane < pos ? bg[lane] : 0.0f;
        }
    }
    if constexpr (KDA)
        if (t < D) s.gp[t] = pos > 0 ? bg[(size_t)(pos - 1) * D + t] : 0.0f;
    __syncthreads();
    const uint64_t here = s.t.here;
    if constexpr (KDA) {
        // g of every node, channel t
        if (t < D)
            for (int n = 0; n < 16 * NB; ++n) {
                float g = 0.0f;
                if ((here >> n) & 1u) {
                    const int par = s.t.par[n];
                    g = (par >= 0 ? s.gk[par * D + t] : s.gp[t]) + logf(a.alpha[((size_t)n * heads + head) * D + t]);
                    a.tg[(head * N + n) * D + t] = g;
                }
                s.gk[n * D + t] = g;
            }
        __syncthreads();
    }
    // ---- the window: keys in three parts to LDS, m rows to registers ----
    const int wt = (pos + 15) >> 4;                        // window tiles in use
    for (int e = t; e < 16 * wt * (D / 8); e += NT) {
        const int c = e / (D / 8), c8 = 8 * (e % (D / 8));
        float x[8];
        uint32_t p[3][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = 0.0f;
        if (c < pos) {
            load_floats<8>(bk + (size_t)c * D + c8, x);
            if constexpr (KDA) {
                float gc[8];
                load_floats<8>(bg + (size_t)c * D + c8, gc);
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] *= expf(s.gp[c8 + u] - gc[u]);
            }
        }
        split3<8>(x, p);
#pragma unroll
        for (int m = 0; m < 3; ++m)
            *reinterpret_cast<u32x4*>(&s.wk[m][c * QS + c8]) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
    }
    v4f WM[WT][2];
#pragma unroll
    for (int c = 0; c < WT; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = 16 * c + 4 * lg + v;
            f32x2 x = {0.f, 0.f};
            if (n < pos) x = *reinterpret_cast<const f32x2*>(bm + (size_t)n * D + col);
            WM[c][0][v] = x[0];
            WM[c][1][v] = x[1];
        }
    // ---- r o sq (per-key decay: o e^{g_pos}) in three parts: B operands, half hf of 64 channels ks
    //      holds channels 64 ks + 16 lg + 8 hf .. + 7 ----
    u32x4 st[KS][2][2][3];                                 // [ks][hf][ct][part]
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float r[8];
            load_floats<8>(a.r + head * D + 64 * ks + 16 * lg + 8 * hf, r);
            if constexpr (KDA)
#pragma unroll
                for (int u = 0; u < 8; ++u) r[u] *= expf(s.gp[64 * ks + 16 * lg + 8 * hf + u]);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = sbyte((uint32_t)raw[ks][ct][2 * hf + u / 4], u % 4) * r[u];
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) st[ks][hf][ct][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
        }
    const f32x2 sj = *reinterpret_cast<const f32x2*>(a.s + head * D + col);
    // compensator rows: B operand of two k = 4 steps, row 4 u + lg
    float cb[2][2];
    int ci[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int c = 4 * u + lg;
        f32x2 x = {0.f, 0.f};
        ci[u] = 0;
        if (c < C) {
            ci[u] = a.idx[head * C + c] & (D - 1);
            x = *reinterpret_cast<const f32x2*>(a.cv + (head * C + c) * (size_t)D + col);
            if constexpr (KDA) x *= expf(s.gp[ci[u]]);
        }
        cb[u][0] = x[0];
        cb[u][1] = x[1];
    }

    v4f M[NB][2];
    bool odd = false;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (16 * j >= N) break;
        // values, ahead of the rows' work
        f32x2 vr[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = 16 * j + 4 * lg + v;
            vr[v] = f32x2{0.f, 0.f};
            if ((here >> n) & 1u) {
                const size_t at = ((size_t)n * heads + head) * D + col;
                if constexpr (sizeof(TI) == 4) vr[v] = *reinterpret_cast<const f32x2*>(static_cast<const float*>(a.v) + at);
                else {
                    const uint32_t x = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v) + at);
                    vr[v] = f32x2{lo_f32(x), hi_f32(x)};
                }
            }
        }
        // ---- 1. rows ----
        {
            constexpr int CPR = D / 8;
            static_assert(NT == 16 * CPR, "one 8-channel piece of one row per lane");
            const int row = t / CPR, c8 = 8 * (t % CPR), n = 16 * j + row;
            const size_t at = ((size_t)n * heads + head) * D + c8;
            const bool on = (here >> n) & 1u;              // absent nodes: zeros
            float sc[8];
            if constexpr (KDA)
#pragma unroll
                for (int u = 0; u < 8; ++u) sc[u] = on ? expf(s.gk[n * D + c8 + u] - s.gp[c8 + u]) : 0.0f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (KDA && !DELTA && x) break;
                uint16_t* dst = x ? &s.k[0][((KB > 1 ? 16 * j : 0) + row) * QS + c8] : &s.q[0][row * QS + c8];
                const size_t plane = x ? sizeof(s.k[0]) / 2 : sizeof(s.q[0]) / 2;
                if constexpr (NP == 1) {
                    u32x4 y = {0, 0, 0, 0};
                    if (on) y = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x ? a.k : a.q) + at);
                    *reinterpret_cast<u32x4*>(dst) = y;
                } else {
                    float y[8];
                    uint32_t p[3][4];
#pragma unroll
                    for (int u = 0; u < 8; ++u) y[u] = 0.0f;
                    if (on) {
                        if constexpr (sizeof(TI) == 4) load_floats<8>(static_cast<const float*>(x ? a.k : a.q) + at, y);
                        else {
                            const u32x4 z = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x ? a.k : a.q) + at);
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                y[2 * u] = lo_f32(z[u]);
                                y[2 * u + 1] = hi_f32(z[u]);
                            }
                        }
                        if constexpr (KDA)
#pragma unroll
                            for (int u = 0; u < 8; ++u) y[u] *= sc[u];
                    }
                    split3<8>(y, p);
#pragma unroll
                    for (int m = 0; m < 3; ++m) *reinterpret_cast<u32x4*>(dst + m * plane) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
                }
            }
        }
        __syncthreads();
        // ---- 2. scores ----
        {
            const int nt = wt + (KDA ? 0 : j + 1);         // context tiles of matrix products
            for (int it = w; it < NX * nt; it += NW) {
                const int x = it >= nt, c = x ? it - nt : it;
                const uint16_t* arow = x ? &s.k[0][((KB > 1 ? 16 * j : 0) + li) * QS] : &s.q[0][li * QS];
                const size_t plane = x ? sizeof(s.k[0]) / 2 : sizeof(s.q[0]) / 2;
                v4f acc = {0.f, 0.f, 0.f, 0.f};
                const bool win = c < wt;
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks) {
                    const int ch = 32 * ks + 8 * lg;
                    u32x4 ar[NP];
#pragma unroll
                    for (int m = 0; m < NP; ++m) ar[m] = *reinterpret_cast<const u32x4*>(arow + m * plane + ch);
                    if (win) {
                        u32x4 br[3];
#pragma unroll
                        for (int m = 0; m < 3; ++m) br[m] = *reinterpret_cast<const u32x4*>(&s.wk[m][(16 * c + li) * QS + ch]);
                        acc = mfma_parts<NP>(ar, br, acc);
                    } else if constexpr (NP == 1) {
                        acc = mfma_bf16(ar[0], *reinterpret_cast<const u32x4*>(&s.k[0][(16 * (c - wt) + li) * QS + ch]), acc);
                    } else if constexpr (!KDA) {
                        u32x4 br[3];
#pragma unroll
                        for (int m = 0; m < 3; ++m) br[m] = *reinterpret_cast<const u32x4*>(&s.k[m][(16 * (c - wt) + li) * QS + ch]);
                        acc = mfma_split(ar, br, acc);
                    }
                }
                const int i = 16 * (c - wt) + li;          // node of this lane's column (node tiles)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int r = 4 * lg + v, n = 16 * j + r;
                    float y = acc[v];
                    bool on;
                    if (win) {
                        on = 16 * c + li < pos && ((here >> n) & 1u);
                        if constexpr (!KDA) y *= on ? expf(s.g[n] - s.wg[(16 * c + li) & 31]) : 0.0f;
                    } else {
                        on = (s.t.mask[n] >> i) & 1u;
                        if constexpr (!KDA) y *= on ? expf(s.g[n] - s.g[i]) : 1.0f;
                        if (!x && i == n) on = true;       // <q_n, k_n>
                    }
                    if (DELTA && x) y *= -s.beta[n];
                    s.s[x][r * SS + (win ? 16 * c : WC + 16 * (c - wt)) + li] = on ? y : 0.0f;
                }
            }
            if constexpr (KDA) {
                // node pairs, a row per wave at a time, four ancestors at once (16 lanes each)
                constexpr int CH = D / 16;
                for (int r = w; r < 16; r += NW) {
                    const int n = 16 * j + r;
                    for (int c = lane; c < 16 * (j + 1); c += 64) s.s[0][r * SS + WC + c] = s.s[1][r * SS + WC + c] = 0.0f;
                    if (!((here >> n) & 1u)) continue;
                    const size_t at = ((size_t)n * heads + head) * D + CH * li;
                    float qn[CH], kn[CH], gn[CH];
#pragma unroll
                    for (int u = 0; u < CH; ++u) {
                        qn[u] = tok_ld<TI>(a.q, at + u);
                        kn[u] = tok_ld<TI>(a.k, at + u);
                    }
                    load_floats<CH>(&s.gk[n * D + CH * li], gn);
                    const float nb = -s.beta[n];
                    uint64_t left = s.t.mask[n] | (1ull << n);
                    left = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(left >> 32)) << 32) |
                           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)left);
                    while (left) {
                        int i = -1;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (left) {
                                const int f = __builtin_ctzll(left);
                                left &= left - 1;
                                if (lg == u) i = f;
                            }
                        }
                        float xq = 0.0f, xk = 0.0f;
                        if (i >= 0) {
                            float gi[CH];
                            load_floats<CH>(&s.gk[i * D + CH * li], gi);
#pragma unroll
                            for (int u = 0; u < CH; ++u) {
                                float ki = tok_ld<TI>(a.k, ((size_t)i * heads + head) * D + CH * li + u);
                                if (i != n) ki *= __expf(gn[u] - gi[u]);
                                xq += qn[u] * ki;
                                xk += kn[u] * ki;
                            }
                        }
                        xq = group_sum<16>(xq);
                        xk = group_sum<16>(xk);
                        if (li == 0 && i >= 0) {
                            s.s[0][r * SS + WC + i] = xq;
                            if (i != n) s.s[1][r * SS + WC + i] = nb * xk;
                        }
                    }
                }
            }
        }
        __syncthreads();
        // ---- 3. (I + A)^{-1}, lane c < 16 its column c ----
        if (DELTA && w == NW - 1 && lane < 16) {
            float tc[16];
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                float ar[16];
                load_floats<16>(&s.s[1][n * SS + WC + 16 * j], ar);
                float x0 = n == lane ? 1.0f : 0.0f, x1 = 0.0f;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    if (i & 1) x1 = __builtin_fmaf(ar[i], tc[i], x1);
                    else x0 = __builtin_fmaf(ar[i], tc[i], x0);
                }
                tc[n] = x0 + x1;
                s.inv[n * 20 + lane] = tc[n];
            }
        }
        // ---- 4. products with the state ----
        v4f acc[NX][2], cmp[NX][2];
#pragma unroll
        for (int x = 0; x < NX; ++x) {
            const uint16_t* arow = x ? &s.k[0][((KB > 1 ? 16 * j : 0) + li) * QS] : &s.q[0][li * QS];
            const size_t plane = x ? sizeof(s.k[0]) / 2 : sizeof(s.q[0]) / 2;
            acc[x][0] = acc[x][1] = cmp[x][0] = cmp[x][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    u32x4 ar[NP];
#pragma unroll
                    for (int m = 0; m < NP; ++m)
                        ar[m] = *reinterpret_cast<const u32x4*>(arow + m * plane + 64 * ks + 16 * lg + 8 * hf);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) acc[x][ct] = mfma_parts<NP>(ar, st[ks][hf][ct], acc[x][ct]);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float y = 0.0f;
#pragma unroll
                for (int m = NP - 1; m >= 0; --m) y += bf16_to_f32(arow[m * plane + ci[u]]);
                if (C > 4 * u)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) cmp[x][ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(y, cb[u][ct], cmp[x][ct], 0, 0, 0);
            }
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                acc[x][ct] = acc[x][ct] * sj[ct] + cmp[x][ct];
                if constexpr (!KDA) acc[x][ct] *= *reinterpret_cast<const v4f*>(&s.e[16 * j + 4 * lg]);
            }
        }
        __syncthreads();                                   // the inverse; the rows may be overwritten
        // ---- 5. m and o ----
        auto context = [&](int x, v4f (&y)[2]) {           // y += scores x context
#pragma unroll
            for (int c = 0; c < WT + NB; ++c) {
                if (c < WT ? c >= wt : c - WT >= j) continue;
                const int cc = c < WT ? 16 * c : WC + 16 * (c - WT);
                const v4f sr = *reinterpret_cast<const v4f*>(&s.s[x][li * SS + cc + 4 * lg]);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        y[ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(sr[v], c < WT ? WM[c < WT ? c : 0][ct][v] : M[c < WT ? 0 : c - WT][ct][v],
                                                                     y[ct], 0, 0, 0);
            }
        };
        if constexpr (DELTA) {
            const v4f be = *reinterpret_cast<const v4f*>(&s.beta[16 * j + 4 * lg]);
            v4f R[2];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                for (int v = 0; v < 4; ++v) R[ct][v] = be[v] * (vr[v][ct] - acc[1][ct][v]);
            context(1, R);
            const v4f ti = *reinterpret_cast<const v4f*>(&s.inv[li * 20 + 4 * lg]);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                M[j][ct] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < 4; ++v) M[j][ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(ti[v], R[ct][v], M[j][ct], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                M[j][0][v] = vr[v][0];
                M[j][1][v] = vr[v][1];
            }
        }
        context(0, acc[0]);
        {
            const v4f sr = *reinterpret_cast<const v4f*>(&s.s[0][li * SS + WC + 16 * j + 4 * lg]);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[0][ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(sr[v], M[j][ct][v], acc[0][ct], 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = 16 * j + 4 * lg + v;
            odd |= !finite_f32(M[j][0][v]) | !finite_f32(M[j][1][v]);
            if (!((here >> n) & 1u)) continue;
            const size_t at = ((size_t)n * heads + head) * D + col;
            if constexpr (sizeof(TI) == 4) *reinterpret_cast<f32x2*>(static_cast<float*>(a.o) + at) = f32x2{acc[0][0][v], acc[0][1][v]};
            else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + at) = pack_bf16(acc[0][0][v], acc[0][1][v]);
            *reinterpret_cast<f32x2*>(a.tm + (head * N + n) * (size_t)D + col) = f32x2{M[j][0][v], M[j][1][v]};
        }
    }
    if (__syncthreads_or(odd)) tree_simple<D, RULE, TI, NT>(a, pos, sp.f.t.mask, sp.f.t.par, here, sp.f.s);
}

template <int D, int RULE, typename TI>
hipError_t tree_mfma(const lq_dims& d, const TreeArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)args.heads);
    if (args.N <= 32)
        return d.W <= 16 ? launch_kernel(LQ_KERNEL_TREE, tree_mfma_kernel<D, 2, 1, RULE, TI>, grid, dim3(2 * D), s, args)
                         : launch_kernel(LQ_KERNEL_TREE, tree_mfma_kernel<D, 2, 2, RULE, TI>, grid, dim3(2 * D), s, args);
    return d.W <= 16 ? launch_kernel(LQ_KERNEL_TREE, tree_mfma_kernel<D, 4, 1, RULE, TI>, grid, dim3(2 * D), s, args)
                     : launch_kernel(LQ_KERNEL_TREE, tree_mfma_kernel<D, 4, 2, RULE, TI>, grid, dim3(2 * D), s, args);
}

template <int RULE, typename TI>
hipError_t tree_io(const lq_dims& d, const TreeArgs& args, hipStream_t s) {
    if (d.dk == 16) return launch_kernel(LQ_KERNEL_TREE, tree_kernel<16, RULE, TI>, dim3((unsigned)args.heads), dim3(64), s, args);
    return d.dk == 64 ? tree_mfma<64, RULE, TI>(d, args, s) : tree_mfma<128, RULE, TI>(d, args, s);
}

}  // namespace

template <int RULE>
hipError_t launch_tree_rule(const lq_dims& d, const TreeArgs& args, hipStream_t s) {
    return d.io_dtype == LQ_IO_BF16 ? tree_io<RULE, uint16_t>(d, args, s) : tree_io<RULE, float>(d, args, s);
}
#endif

}  // namespace lq

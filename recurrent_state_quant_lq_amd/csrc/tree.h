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

#include "la.h"
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

// Presence and ancestors of a row's nodes, lane n = node n with parent entry p (-2: no such node): own = whether the
// entry is valid (-1 or an earlier node), mask = its ancestors while every
// entry on the way up is valid.  A node is present if its own entry and all its
// ancestors' are; no index depends on an unchecked value.  sum: of x over the path
// (the node included), by pointer doubling.
template <typename F>
struct TreeNode {
    uint64_t mask;
    F sum;
    int parent;               // -1: the last committed token
    bool here;
};
template <typename F>
__device__ __forceinline__ TreeNode<F> tree_node(int p, int lane, F x) {
    const bool own = p == -1 || (p >= 0 && p < lane);
    int jump = own ? p : -1;
    TreeNode<F> t;
    t.parent = jump;
    t.mask = jump >= 0 ? 1ull << jump : 0;
    t.sum = x;
    while (__any(jump >= 0)) {                             // paths of doubling length: at most 6 rounds for 64 nodes
        const int from = jump >= 0 ? jump : lane;
        const uint64_t m = __shfl(t.mask, from, 64);
        const F y = __shfl(t.sum, from, 64);
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
// node after node: rows that hold a value that is not finite
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

// ---------------------------------------------------------------------------
// d >= 64: blocks of 16 nodes on matrix products
// ---------------------------------------------------------------------------
// Wave w owns the 32 value columns 32 w + 2 li + ct (a lane's two columns are neighbours:
// one dword of bf16 values, one 8-byte pair of fp32 ones).  Per group of GB blocks:
//   1. the q and k rows to LDS as bf16 parts (one for bf16 tokens with a decay per
//      head; else three; per-key decay: rows scaled by e^{g_n - g_pos}, at most 1);
//   2. scores against the window's keys (in parts in LDS; per-key decay: scaled by
//      e^{g_pos - g_c}) and the nodes' keys, times E and the ancestor mask; those of
//      k times -beta.  Per-key decay takes the nodes' scores pair by pair, with the
//      exponential of each channel's difference: a product of two factors could
//      overflow;
//   3. the products with the state: r o sq in bf16 parts formed on the way, or, for rows in
//      three parts, the int8 values as they are and the rows formed again, scaled by r;
//   4. block after block, without barriers: R = beta (v - Hb^T k) - A_ctx M_ctx,
//      M = (I + A)^{-1} R with A_{n,i} = beta_n <k_n, E k_i> (strictly lower triangular in
//      node order, solved four rows at a time), O = Hb^T q + S M, on the fp32 matrix
//      instruction: accumulators are its B operand as they are, so M never leaves the
//      registers.
// A head's work is a chain of short phases, so what counts is that few of them wait
// for memory: everything that needs no table is requested at once (state, scales,
// rows and values of the first group), the window as soon as pos is known, the next
// group's rows while a group is computed; rows past the end are read from a row that
// exists, so that no load sits behind a branch.
// Bound by the issue of these phases and, with two workgroups a CU (per-key decay: LDS), by
// their latencies; 64 nodes of the delta rule in fp32 and of per-key decay leave room in LDS for one
// workgroup a CU.  d = 128, 2048 heads, bf16 (fp32): delta rule, 32 nodes 52 us (73; bf16: vector
// unit 23, matrix unit 15; 3.0 TB/s), 64 nodes 114 us (205), without it 74 us (136); 1024 heads,
// per-key decay, 21 nodes, fp32 48 us, 64 nodes 145 us (148).
// A product of a masked zero with a value that is not finite would spread it: if any
// m is not finite, the row is computed again node after node.
template <int D, int NB, int WT, int RULE, typename TI>
struct TM {
    static constexpr int NW = D / 32, NT = 64 * NW;
    static constexpr bool KDA = RULE == TREE_KDA, DELTA = RULE != TREE_LA;
    static constexpr int NP = sizeof(TI) == 2 && !KDA ? 1 : 3;     // parts of a token row
    // parts of the window's keys and of the scaled state: three, all 24 bits (plain linear attention, bf16,
    // 2048 heads: with these and the nodes' scores in two parts 36 us, not 41, for 32 nodes and 68, not 74,
    // for 64, but 0.3% of the outputs, not 0.02%, then round to a neighbour of what fp32 sums round to)
    static constexpr int NS = 3;
    // parts of the state: where rows have three parts, the int8 values are kept as they are (exact
    // in bf16) and the rows are formed again after the scores, scaled by r (per-key decay: by
    // r o e^{g_n}): half the products of the state in three parts, and no splits of it for each
    // block (per-key decay, 1024 heads, 21 nodes, fp32: 46 us, not 52; delta rule, 2048 heads,
    // 32 nodes, fp32: 68 us, not 75)
    static constexpr bool FOLD = NP == 3;
    static constexpr int NT8 = FOLD ? 1 : NS;
    static constexpr int GB = NP == 1 ? 2 : 1;                     // blocks per group
    static constexpr int KB = KDA ? GB : NB;                       // blocks whose keys stay in LDS
    static constexpr bool RK = KDA && 16 * NB * D * sizeof(TI) <= 16384;   // (else they are read from memory)
    static constexpr int QS = D + 8;                               // shorts per row
    static constexpr int WC = 16 * WT;                             // window columns of the scores
    // plain linear attention, bf16: m = v is exact in bf16, so the nodes' scores are kept in three
    // bf16 parts and meet the values of two blocks in one bf16 matrix instruction a part
    static constexpr bool VB = !DELTA && sizeof(TI) == 2;
    static constexpr int SS = WC + (VB ? 0 : 16 * NB) + 4;         // floats per score row
    static constexpr int SB = VB ? 16 * NB + 8 : 8;                // shorts per row of the nodes' scores in parts
    struct Shared {
        TreeTables t;
        __align__(16) float g[kTreeMax];                           // scalar decay: g_n (absent nodes: that of slot pos - 1)
        __align__(16) float e[kTreeMax];                           // scalar decay: e^{g_n}
        __align__(16) float beta[kTreeMax];
        float wg[32];                                              // scalar decay: the window's g
        __align__(16) float r[D];                                  // row scales (per-key decay: e^{g_pos} r)
        __align__(16) uint16_t q[NP][16 * GB * QS];
        __align__(16) uint16_t k[NP][16 * KB * QS];
        __align__(16) uint16_t wk[NS][WC * QS];
        __align__(16) float s[DELTA ? 2 : 1][16 * GB * SS];        // scores of q; -beta times those of k
        __align__(16) uint16_t sb[3][VB ? 16 * GB * SB : 8];
        __align__(16) float gk[KDA ? 16 * NB * D : 4];             // per-key decay: g_n
        __align__(16) float gp[KDA ? D : 4];                       // per-key decay: g of slot pos - 1
        __align__(16) TI kr[RK ? 16 * NB * D : 8];                 // per-key decay: the nodes' keys as they are
    };
    union Space {
        Shared m;
        struct {
            TreeTables t;
            TreeSimple<D> s;
        } f;
    };
    // waves per SIMD the registers are sized for: the workgroups that fit the LDS of a CU, 3 at
    // most (2 with 64 nodes, whose registers would spill: a third slower, plain rule)
    static constexpr int FIT = 160 * 1024 / (int)sizeof(Space) * NW / 4;
    static constexpr int WPE = FIT >= 3 && NB == 2 ? 3 : FIT >= 2 ? 2 : 1;
};

// c += a b with a in NP parts, b in NQ parts; small products first.
template <int NP, int NQ>
__device__ __forceinline__ v4f mfma_parts(const u32x4 (&a)[NP], const u32x4 (&b)[NQ], v4f c) {
    if constexpr (NP == 3 && NQ == 3) return mfma_split(a, b, c);
    if constexpr (NP == 3 && NQ == 1) {
        c = mfma_bf16(a[2], b[0], c);
        c = mfma_bf16(a[1], b[0], c);
    }
    if constexpr (NQ >= 3) c = mfma_bf16(a[0], b[2], c);
    if constexpr (NQ >= 2) c = mfma_bf16(a[0], b[1], c);
    return mfma_bf16(a[0], b[0], c);
}

// Eight consecutive token values, and two, as loaded.
template <typename TI> struct Raw8 { u32x4 x[sizeof(TI) / 2]; };
template <typename TI>
__device__ __forceinline__ Raw8<TI> raw8(const void* base, size_t at) {
    Raw8<TI> r;
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const TI*>(base) + at);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(TI) / 2); ++i) r.x[i] = p[i];
    return r;
}
template <typename TI>
__device__ __forceinline__ void widen8(const Raw8<TI>& r, float (&y)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if constexpr (sizeof(TI) == 4) y[u] = __uint_as_float(r.x[u / 4][u % 4]);
        else y[u] = u & 1 ? hi_f32(r.x[0][u / 2]) : lo_f32(r.x[0][u / 2]);
    }
}
template <typename TI> struct Pair;
template <> struct Pair<float> { typedef f32x2 T; };
template <> struct Pair<uint16_t> { typedef uint32_t T; };
__device__ __forceinline__ f32x2 widen2(f32x2 x) { return x; }
__device__ __forceinline__ f32x2 widen2(uint32_t x) { return f32x2{lo_f32(x), hi_f32(x)}; }

// ---------------------------------------------------------------------------
// d = 16: one wave a head
// ---------------------------------------------------------------------------
// Every product is one 16 x 16 x 16 of the fp32 matrix instruction, its operands loaded in the
// layout that the instruction takes (lane (lg, li), step v: row or column li, index 4 lg + v).
// The scores are formed transposed (K Q^T), so that their accumulators are the A operand of S M,
// and M's are its B operand: only A's diagonal block goes through LDS.  Per-key decay forms the
// scores of node pairs channel by channel (lane: one node, four ancestors), as the larger kernel
// does.  Bound by the latency of a wave's phases: 32 nodes, 2048 heads, delta rule 16 us (372
// node after node).
template <int RULE>
struct TreeSmall {
    static constexpr int ND = RULE == TREE_KDA ? 20 * kTreeMax : 4;   // rows of 20 floats (bank spread)
    __align__(16) float g[ND];                             // per-key decay: g_n
    __align__(16) float k[ND];                             // per-key decay: the nodes' keys
    __align__(16) float q[RULE == TREE_KDA ? 20 * 16 : 4]; // per-key decay: the block's queries
    __align__(16) float a[20 * 16];                        // -A of the block
};

template <int NB, int RULE, typename TI>
__global__ __launch_bounds__(64) void tree_small_kernel(TreeArgs a) {
    constexpr int D = 16, LR = 20;
    constexpr bool KDA = RULE == TREE_KDA, DELTA = RULE != TREE_LA;
    __shared__ TreeTables s_t;
    __shared__ union {
        TreeSmall<RULE> m;
        TreeSimple<D> f;
    } sp;
    auto& s = sp.m;
    const int lane = threadIdx.x, li = lane & 15, lg = lane >> 4;
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int W = a.W, C = a.C, N = a.N;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    // ---- requests (rows past the end: the last node's, zeroed below) ----
    const int pos = a.pos[b];
    const int npar = lane < N ? a.parent[(size_t)b * N + lane] : -2;
    const size_t node = (size_t)min(lane, N - 1);
    float nal = 1.0f, nbeta = 0.0f;
    if constexpr (!KDA) nal = a.alpha[a.alpha_tok ? node * a.alpha_tok + head : head % (unsigned)a.H];
    if constexpr (DELTA) nbeta = a.beta[node * heads + head];
    float q[NB][4], k[NB][4], vv[NB][4], lal[KDA ? NB : 1][4];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (16 * j >= N) break;
        const size_t at = ((size_t)min(16 * j + li, N - 1) * heads + head) * D + 4 * lg;
        Row4<TI> rq, rk;
        rq.load(a.q, at);
        rk.load(a.k, at);
        rq.widen4(q[j]);
        rk.widen4(k[j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const size_t to = ((size_t)min(16 * j + 4 * lg + v, N - 1) * heads + head) * D + li;
            vv[j][v] = tok_ld<TI>(a.v, to);
            if constexpr (KDA) lal[j][v] = a.alpha[to];
        }
    }
    const uint32_t raw = *reinterpret_cast<const uint32_t*>(a.sq + head * (size_t)(D * D) + sq_off<D>(0, li) + 4 * lg);
    float rs[4], hb[4];
    load_floats<4>(a.r + head * D + 4 * lg, rs);
    const float sj = a.s[head * D + li];
    if (pos < 0 || pos > W) return;                        // a row outside its window: untouched
    const int last = max(pos - 1, 0);
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W * (KDA ? D : 1);
    float wk[2][4], wm[2][4], wg[2][4], gp[4] = {0.f, 0.f, 0.f, 0.f}, gpos = 0.0f;   // gpos: per-key decay: of channel li
    if (pos > 0) {
        gpos = bg[(size_t)last * (KDA ? D : 1) + (KDA ? li : 0)];
        if constexpr (KDA) load_floats<4>(bg + (size_t)last * D + 4 * lg, gp);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (16 * c < pos) {
                const size_t at = (size_t)min(16 * c + li, last) * D + 4 * lg;
                load_floats<4>(bk + at, wk[c]);
                if constexpr (KDA) load_floats<4>(bg + at, wg[c]);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = min(16 * c + 4 * lg + v, last);
                    wm[c][v] = bm[(size_t)i * D + li];
                    if constexpr (!KDA) wg[c][v] = bg[i];
                }
            }
    }
    // ---- the state: Hb[4 lg + v][li] ----
#pragma unroll
    for (int v = 0; v < 4; ++v) hb[v] = sbyte(raw, v) * rs[v] * sj;
    for (int c = 0; c < C; ++c) {
        const int ic = a.idx[head * C + c] & (D - 1);
        const float y = a.cv[(head * C + c) * D + li];
#pragma unroll
        for (int v = 0; v < 4; ++v) hb[v] += ic == 4 * lg + v ? y : 0.0f;
    }
    // ---- tables: lane n = node n ----
    // (path sums in 64 bits: differences of strong decays keep fp32's precision)
    const TreeNode<double> nd = tree_node(npar, lane, KDA ? 0.0 : (double)(DELTA ? logf(nal) : log_decay(nal)));
    const uint64_t here = __ballot(nd.here);
    const uint64_t mask = nd.here ? nd.mask : 0;
    s_t.mask[lane] = mask;                                 // (for rows that are not finite)
    s_t.par[lane] = (int8_t)nd.parent;
    const float beta = nd.here ? nbeta : 0.0f;
    const double G = KDA ? 0.0 : nd.here ? nd.sum + gpos : gpos;
    if constexpr (!KDA)
        if (nd.here) a.tg[head * N + lane] = (float)G;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (16 * j >= N) break;
        const bool row = (here >> (16 * j + li)) & 1u;     // absent nodes: zeros
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const bool on = (here >> (16 * j + 4 * lg + v)) & 1u;
            q[j][v] = row ? q[j][v] : 0.0f;
            k[j][v] = row ? k[j][v] : 0.0f;
            vv[j][v] = on ? vv[j][v] : 0.0f;
            if constexpr (KDA) lal[j][v] = on ? logf(lal[j][v]) : 0.0f;
        }
        if constexpr (KDA) {
            // path sums of the logarithms, rows 4 lg + v, channel li
            const int n = 16 * j + li;
            const uint64_t path = __shfl(mask, n, 64) | (1ull << n);
            v4f y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c <= j; ++c)
#pragma unroll
                for (int v = 0; v < 4; ++v) y = mfma4((path >> (16 * c + 4 * lg + v)) & 1u ? 1.0f : 0.0f, lal[c][v], y);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = 16 * j + 4 * lg + v;
                s.g[m * LR + li] = y[v] + gpos;
                if ((here >> m) & 1u) a.tg[(head * N + m) * D + li] = y[v] + gpos;
            }
            *reinterpret_cast<v4f*>(&s.k[n * LR + 4 * lg]) = v4f{k[j][0], k[j][1], k[j][2], k[j][3]};
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (16 * c < pos)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if constexpr (KDA) wk[c][v] *= expf(gp[v] - wg[c][v]);
                wk[c][v] = 16 * c + li < pos ? wk[c][v] : 0.0f;
                wm[c][v] = 16 * c + 4 * lg + v < pos ? wm[c][v] : 0.0f;
            }

    v4f M[NB];
    bool odd = false;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (16 * j >= N) break;
        const int n = 16 * j + li;
        const uint64_t anc = __shfl(mask, n, 64);
        const double gn = KDA ? 0.0 : __shfl(G, n, 64);
        const float bn = DELTA ? __shfl(beta, n, 64) : 0.0f;
        if constexpr (KDA) {
            *reinterpret_cast<v4f*>(&s.q[li * LR + 4 * lg]) = v4f{q[j][0], q[j][1], q[j][2], q[j][3]};
            __syncthreads();
        }
        float en[4], ew[4];                                // e^{g_n} of the row's channels; per-key decay: e^{g_n - g_pos}
        if constexpr (KDA) {
            float gr[4];
            load_floats<4>(&s.g[n * LR + 4 * lg], gr);
#pragma unroll
            for (int v = 0; v < 4; ++v) en[v] = expf(gr[v]), ew[v] = expf(gr[v] - gp[v]);
        } else {
            en[0] = en[1] = en[2] = en[3] = expf((float)gn);
        }
        // y += S x context, S^T = K Q^T; x: 0 the queries, 1 the keys
        v4f O = {0.f, 0.f, 0.f, 0.f}, R = O, dq = O, dk = O;   // dq, dk: the block's own scores, transposed
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            O = mfma4(en[v] * q[j][v], hb[v], O);
            if constexpr (DELTA) R = mfma4(en[v] * k[j][v], hb[v], R);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (16 * c < pos) {
                v4f sq = {0.f, 0.f, 0.f, 0.f}, sk = sq;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    sq = mfma4(wk[c][v], KDA ? ew[v] * q[j][v] : q[j][v], sq);
                    if constexpr (DELTA) sk = mfma4(wk[c][v], KDA ? ew[v] * k[j][v] : k[j][v], sk);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float e = KDA ? 1.0f : __expf((float)(gn - wg[c][v]));
                    O = mfma4(sq[v] * e, wm[c][v], O);
                    if constexpr (DELTA) R = mfma4(sk[v] * e, wm[c][v], R);
                }
            }
        [[maybe_unused]] float qn[KDA ? D : 1], kn[KDA ? D : 1], gr[KDA ? D : 1];
        if constexpr (KDA) {
            load_floats<D>(&s.q[li * LR], qn);
            load_floats<D>(&s.k[n * LR], kn);
            load_floats<D>(&s.g[n * LR], gr);
        }
#pragma unroll
        for (int c = 0; c <= j; ++c) {
            v4f sq = {0.f, 0.f, 0.f, 0.f}, sk = sq;
            if constexpr (!KDA) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    sq = mfma4(k[c][v], q[j][v], sq);
                    if constexpr (DELTA) sk = mfma4(k[c][v], k[j][v], sk);
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int i = 16 * c + 4 * lg + v;
                const bool up = (anc >> i) & 1u, on = up || i == n;   // (i = n: <q_n, k_n>; its exponential is 1)
                if constexpr (KDA) {
                    if (__any(on)) {
                        float ki[D], gi[D], xq = 0.0f, xk = 0.0f;
                        load_floats<D>(&s.k[i * LR], ki);
                        load_floats<D>(&s.g[i * LR], gi);
#pragma unroll
                        for (int u = 0; u < D; ++u) {
                            const float y = i == n ? ki[u] : ki[u] * __expf(gr[u] - gi[u]);
                            xq += qn[u] * y;
                            xk += kn[u] * y;
                        }
                        sq[v] = on ? xq : 0.0f;
                        sk[v] = up ? xk : 0.0f;
                    }
                } else {
                    const float e = __expf((float)(gn - __shfl(G, i, 64)));
                    sq[v] = on ? sq[v] * (i == n ? 1.0f : e) : 0.0f;
                    sk[v] = up ? sk[v] * e : 0.0f;
                }
            }
            if (c < j) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    O = mfma4(sq[v], M[c][v], O);
                    if constexpr (DELTA) R = mfma4(sk[v], M[c][v], R);
                }
            } else {
                dq = sq;
                dk = sk;
            }
        }
        if constexpr (DELTA) {
            v4f X[1], own[3];
            float below[3];
            *reinterpret_cast<v4f*>(&s.a[li * LR + 4 * lg]) = dk * -bn;
#pragma unroll
            for (int v = 0; v < 4; ++v) X[0][v] = __shfl(beta, 16 * j + 4 * lg + v, 64) * (vv[j][v] - R[v]);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 3; ++i) own[i] = *reinterpret_cast<const v4f*>(&s.a[(4 * lg + 1 + i) * LR + 4 * lg]);
#pragma unroll
            for (int p = 0; p < 3; ++p) below[p] = (li >> 2) > p ? s.a[li * LR + 4 * p + lg] : 0.0f;
            block_solve(own, below, lg, X);
            M[j] = X[0];
            __syncthreads();                               // (s.a and s.q are rewritten by the next block)
        } else {
            M[j] = v4f{vv[j][0], vv[j][1], vv[j][2], vv[j][3]};
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) O = mfma4(dq[v], M[j][v], O);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int m = 16 * j + 4 * lg + v;
            odd |= !finite_f32(M[j][v]);
            if (!((here >> m) & 1u)) continue;
            tok_st<TI>(a.o, ((size_t)m * heads + head) * D + li, O[v]);
            a.tm[(head * N + m) * D + li] = M[j][v];
        }
    }
    if (__syncthreads_or(odd)) {
        all_loads_barrier();                               // (this pass's stores are done: the rows are written again)
        tree_simple<D, RULE, TI, 64>(a, pos, s_t.mask, s_t.par, here, sp.f);
    }
}

template <int D, int NB, int WT, int RULE, typename TI>
__global__ __launch_bounds__((TM<D, NB, WT, RULE, TI>::NT), (TM<D, NB, WT, RULE, TI>::WPE)) void tree_mfma_kernel(TreeArgs a) {
    using X = TM<D, NB, WT, RULE, TI>;
    constexpr int NW = X::NW, NT = X::NT, NP = X::NP, GB = X::GB, KB = X::KB, QS = X::QS, WC = X::WC, SS = X::SS;
    constexpr bool KDA = X::KDA, DELTA = X::DELTA;
    constexpr int NS = X::NS, SB = X::SB;
    constexpr bool VB = X::VB, FOLD = X::FOLD;
    constexpr int NX = DELTA ? 2 : 1, GD = KDA ? D : 1, KS = D / 64, NG = NB / GB;
    __shared__ typename X::Space sp;
    auto& s = sp.m;

    const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const unsigned b = blockIdx.x / (unsigned)a.H;
    const int W = a.W, C = a.C, N = a.N;
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W * GD;
    const int col = 32 * w + 2 * li;                       // and col + 1

    // ---- requests that depend on nothing ----
    const int pos = a.pos[b];
    float nal = 0.0f, nbeta = 0.0f;                        // wave 0: node `lane`
    int npar = -2;
    if (w == 0) {
        const int n = min(lane, N - 1);
        npar = a.parent[(size_t)b * N + n];
        if constexpr (!KDA) nal = a.alpha[a.alpha_tok ? (size_t)n * a.alpha_tok + head : head % (unsigned)a.H];
        if constexpr (DELTA) nbeta = a.beta[(size_t)n * heads + head];
    }
    // of each block of a group: one 8-channel piece of one of its 16 q rows and k rows, and the lane's values
    constexpr int CPR = D / 8;
    static_assert(NT == 16 * CPR, "one piece of one row per lane");
    const int row = t / CPR, c8 = 8 * (t % CPR);
    Raw8<TI> rq[GB], rk[GB];
    typename Pair<TI>::T vr[GB][4];
    auto request = [&](int g) {
#pragma unroll
        for (int e = 0; e < GB; ++e) {
            const size_t at = ((size_t)min(16 * (GB * g + e) + row, N - 1) * heads + head) * D + c8;
            rq[e] = raw8<TI>(a.q, at);
            rk[e] = raw8<TI>(a.k, at);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = min(16 * (GB * g + e) + 4 * lg + v, N - 1);
                vr[e][v] = *reinterpret_cast<const typename Pair<TI>::T*>(static_cast<const TI*>(a.v) + ((size_t)m * heads + head) * D + col);
            }
        }
    };
    request(0);
    f32x2 na[KDA ? NB / 2 : 1][8];                         // per-key decay: alpha of nodes 32 g + 8 lg .. + 7, columns col, col + 1
    if constexpr (KDA)
#pragma unroll
        for (int g = 0; g < NB / 2; ++g)
#pragma unroll
            for (int u = 0; u < 8; ++u)
                na[g][u] = *reinterpret_cast<const f32x2*>(a.alpha + ((size_t)min(32 * g + 8 * lg + u, N - 1) * heads + head) * D + col);
    v4i raw[KS][2];                                        // columns col + ct, channels 64 ks + 16 lg .. + 15
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
            raw[ks][ct] = *reinterpret_cast<const v4i*>(a.sq + head * (size_t)(D * D) + sq_off<D>(64 * ks + 16 * lg, col + ct));
    float rs = a.r[head * D + (t & (D - 1))];
    const f32x2 sj = *reinterpret_cast<const f32x2*>(a.s + head * D + col);
    // compensator rows: B operand of two k = 4 steps, row 4 u + lg
    f32x2 cb[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    int ci[2] = {0, 0};
    if (C > 0)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const size_t c = head * C + min(4 * u + lg, C - 1);
            ci[u] = a.idx[c];
            cb[u] = *reinterpret_cast<const f32x2*>(a.cv + c * D + col);
        }
    if (pos < 0 || pos > W) return;                        // a row outside its window: untouched

    // ---- the window's requests: one 8-channel piece of a key row per lane and tile, the columns' m rows ----
    const int wt = max(1, (pos + 15) >> 4);                // window tiles in use (the first always: zeros if empty)
    const int last = max(pos - 1, 0);
    float wx[WT][8], wgc[KDA ? WT : 1][8];
    float gpos = 0.0f, gw = 0.0f;                          // g of slot pos - 1 (per-key decay: channel t); of slot `lane`
    v4f WM[WT][2];
    if (pos > 0) {
#pragma unroll
        for (int c = 0; c < WT; ++c) {
            const size_t at = (size_t)min(16 * c + row, last) * D + c8;
            load_floats<8>(bk + at, wx[c]);
            if constexpr (KDA) load_floats<8>(bg + at, wgc[c]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const f32x2 x = *reinterpret_cast<const f32x2*>(bm + (size_t)min(16 * c + 4 * lg + v, last) * D + col);
                WM[c][0][v] = x[0];
                WM[c][1][v] = x[1];
            }
        }
        if constexpr (KDA) gpos = bg[(size_t)last * D + (t & (D - 1))];
        else if (w == 0) {
            gpos = bg[last];
            gw = bg[min(lane, last)];
        }
    }
    // ---- tables ----
    if (w == 0) {
        const TreeNode<float> nd = tree_node(lane < N ? npar : -2, lane, KDA ? 0.0f : DELTA ? logf(nal) : log_decay(nal));
        s.t.mask[lane] = nd.here ? nd.mask : 0;
        s.t.par[lane] = (int8_t)nd.parent;
        const uint64_t here = __ballot(nd.here);
        if (lane == 0) s.t.here = here;
        if constexpr (DELTA) s.beta[lane] = nd.here ? nbeta : 0.0f;
        if constexpr (!KDA) {
            const float g = nd.here ? nd.sum + gpos : gpos;
            s.g[lane] = g;
            s.e[lane] = expf(g);
            if (nd.here) a.tg[head * N + lane] = g;
            if (lane < 32) s.wg[lane] = gw;
        }
    }
    if constexpr (KDA)
        if (t < D) {
            s.gp[t] = gpos;
            rs *= expf(gpos);
        }
    if (t < D) s.r[t] = rs;
    // ---- window keys in three parts ----
    if constexpr (KDA) __syncthreads();                    // gp
#pragma unroll
    for (int c = 0; c < WT; ++c) {
        if (c > 0 && c >= wt) break;
        const bool on = 16 * c + row < pos;
        uint32_t p[NS][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if constexpr (KDA) wx[c][u] *= expf(s.gp[c8 + u] - wgc[c][u]);
            wx[c][u] = on ? wx[c][u] : 0.0f;
        }
        split3<8>(wx[c], p);
#pragma unroll
        for (int m = 0; m < NS; ++m)
            *reinterpret_cast<u32x4*>(&s.wk[m][(16 * c + row) * QS + c8]) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
    }
#pragma unroll
    for (int c = 0; c < WT; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const bool on = 16 * c + 4 * lg + v < pos;
            WM[c][0][v] = on ? WM[c][0][v] : 0.0f;
            WM[c][1][v] = on ? WM[c][1][v] : 0.0f;
        }
    __syncthreads();
    const uint64_t here = s.t.here;
    if constexpr (KDA) {
        // g of every node, channels col and col + 1: the path sums of log alpha as the product of the
        // 0/1 matrix of paths (exact in bf16) and the logarithms in three parts, plus g of slot pos - 1
        const f32x2 g0 = *reinterpret_cast<const f32x2*>(&s.gp[col]);
        u32x4 lp[2][NB / 2][3];
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
            for (int g = 0; g < NB / 2; ++g) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = (here >> (32 * g + 8 * lg + u)) & 1u ? logf(na[g][u][ct]) : 0.0f;
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) lp[ct][g][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            if (16 * j >= N) break;
            const int n = 16 * j + li;
            const uint64_t path = s.t.mask[n] | (1ull << n);
            v4f y[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int g = 0; g <= j / 2; ++g) {
                u32x4 ar[1];
                const uint32_t bits = (uint32_t)(path >> (32 * g)) >> (8 * lg);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    ar[0][u] = ((bits >> (2 * u)) & 1u ? 0x3f80u : 0u) | ((bits >> (2 * u + 1)) & 1u ? 0x3f800000u : 0u);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) y[ct] = mfma_parts<1, 3>(ar, lp[ct][g], y[ct]);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int m = 16 * j + 4 * lg + v;
                const f32x2 x = f32x2{y[0][v], y[1][v]} + g0;
                *reinterpret_cast<f32x2*>(&s.gk[m * D + col]) = x;
                if ((here >> m) & 1u) *reinterpret_cast<f32x2*>(a.tg + (head * N + m) * (size_t)D + col) = x;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        ci[u] &= D - 1;
        if constexpr (KDA) cb[u] *= expf(s.gp[ci[u]]);
        cb[u] = 4 * u + lg < C ? cb[u] : f32x2{0.0f, 0.0f};
    }

    v4f M[VB ? 1 : NB][2];
    u32x2 V[VB ? NB : 1][2];                               // VB: values of the blocks, nodes 4 lg .. + 3, as bf16
    bool odd = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (16 * GB * g >= N) break;
        const int nb = 16 * GB * g + 16 < N ? GB : 1;      // blocks of this group
        uint16_t* kbase = &s.k[0][KB > GB ? 16 * GB * g * QS : 0];
        constexpr size_t QP = sizeof(s.q[0]) / 2, KP = sizeof(s.k[0]) / 2, WP = sizeof(s.wk[0]) / 2;   // shorts per part
        // ---- 1. rows ----
        f32x2 vv[GB][4];
        [[maybe_unused]] float sc[8];                      // per-key decay: the row's scales
#pragma unroll
        for (int e = 0; e < GB; ++e) {
            const int r = 16 * e + row, n = 16 * GB * g + r;
            const bool on = (here >> n) & 1u;              // absent nodes: zeros
            if constexpr (X::RK)
#pragma unroll
                for (int i = 0; i < (int)(sizeof(TI) / 2); ++i)
                    *reinterpret_cast<u32x4*>(&s.kr[n * D + c8 + i * (16 / (int)sizeof(TI))]) = rk[e].x[i];
            if constexpr (NP == 1) {
                *reinterpret_cast<u32x4*>(&s.q[0][r * QS + c8]) = on ? rq[e].x[0] : u32x4{0, 0, 0, 0};
                *reinterpret_cast<u32x4*>(kbase + r * QS + c8) = on ? rk[e].x[0] : u32x4{0, 0, 0, 0};
            } else {
                if constexpr (KDA)
#pragma unroll
                    for (int u = 0; u < 8; ++u) sc[u] = __expf(s.gk[n * D + c8 + u] - s.gp[c8 + u]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y[8];
                    uint32_t p[3][4];
                    widen8<TI>(x ? rk[e] : rq[e], y);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        if constexpr (KDA) y[u] *= sc[u];
                        y[u] = on ? y[u] : 0.0f;
                    }
                    split3<8>(y, p);
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        *reinterpret_cast<u32x4*>((x ? kbase + m * KP : &s.q[m][0]) + r * QS + c8) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
                vv[e][v] = (here >> (16 * (GB * g + e) + 4 * lg + v)) & 1u ? widen2(vr[e][v]) : f32x2{0.f, 0.f};
        }
        __syncthreads();
        // ---- 2. scores: tile (x, e, c) = rows of block e, context tile c (window tiles, then node blocks) ----
        // per-key decay, node pairs: 16 lanes a row (lane li: channels 4 li .. + 3 and 64 + 4 li .. + 3), the
        // row's q on its way meanwhile
        constexpr int CH = D / 16, PP = 16 / (4 * NW);       // passes over the group's rows
        static_assert(!KDA || GB == 1, "one block of rows");
        TI qraw[PP][KDA ? CH : 1];
        if constexpr (KDA)
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                const size_t at = ((size_t)min(16 * g + w + NW * (lg + 4 * p), N - 1) * heads + head) * D + 4 * li;
#pragma unroll
                for (int u = 0; u < CH; ++u) qraw[p][u] = static_cast<const TI*>(a.q)[at + 64 * (u / 4) + u % 4];
            }
        {
            const int nt0 = wt + (KDA ? 0 : GB * g + 1), per = nb == 1 ? nt0 : 2 * nt0 + (KDA ? 0 : 1);   // tiles of block 0, of the group
#pragma unroll 1
            for (int it = w; it < NX * per; it += NW) {
                const int x = it >= per, y0 = x ? it - per : it, e = y0 >= nt0, c = e ? y0 - nt0 : y0;
                const size_t plane = x ? KP : QP;
                const uint16_t* arow = (x ? kbase : &s.q[0][0]) + (16 * e + li) * QS + 8 * lg;
                const int n0 = 16 * (GB * g + e) + 4 * lg;
                const v4f gn = KDA ? v4f{0.f, 0.f, 0.f, 0.f} : *reinterpret_cast<const v4f*>(&s.g[n0]);
                const v4f bn = DELTA && x ? -*reinterpret_cast<const v4f*>(&s.beta[n0]) : v4f{1.f, 1.f, 1.f, 1.f};
                float* dst = &s.s[x][(16 * e + 4 * lg) * SS + li];
                v4f acc = {0.f, 0.f, 0.f, 0.f}, acc2 = acc;
                // (an exponent is at most 0: off by 2^-24 of it, weighted by its exponential)
                if (c < wt) {
                    const uint16_t* brow = &s.wk[0][(16 * c + li) * QS + 8 * lg];
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks) {
                        u32x4 ar[NP], br[NS];
#pragma unroll
                        for (int m = 0; m < NP; ++m) ar[m] = *reinterpret_cast<const u32x4*>(arow + m * plane + 32 * ks);
#pragma unroll
                        for (int m = 0; m < NS; ++m) br[m] = *reinterpret_cast<const u32x4*>(brow + m * WP + 32 * ks);
                        if (ks & 1) acc2 = mfma_parts<NP, NS>(ar, br, acc2);
                        else acc = mfma_parts<NP, NS>(ar, br, acc);
                    }
                    acc += acc2;
                    const float gc = KDA ? 0.0f : s.wg[(16 * c + li) & 31];
#pragma unroll
                    for (int v = 0; v < 4; ++v) dst[v * SS + 16 * c] = acc[v] * (KDA ? 1.0f : __expf(gn[v] - gc)) * bn[v];
                } else if constexpr (!KDA) {
                    const int i = 16 * (c - wt) + li;      // node of this lane's column
                    const uint16_t* brow = &s.k[0][i * QS + 8 * lg];
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks) {
                        u32x4 ar[NP], br[NP];
#pragma unroll
                        for (int m = 0; m < NP; ++m) {
                            ar[m] = *reinterpret_cast<const u32x4*>(arow + m * plane + 32 * ks);
                            br[m] = *reinterpret_cast<const u32x4*>(brow + m * KP + 32 * ks);
                        }
                        if (ks & 1) acc2 = mfma_parts<NP, NP>(ar, br, acc2);
                        else acc = mfma_parts<NP, NP>(ar, br, acc);
                    }
                    acc += acc2;
                    const float gc = s.g[i];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint64_t anc = s.t.mask[n0 + v];
                        const float y = acc[v] * __expf(gn[v] - gc) * bn[v];
                        // (the diagonal of the q scores: <q_n, k_n>; its exponential is 1)
                        const float z = ((anc >> i) & 1u) || (!x && i == n0 + v) ? y : 0.0f;
                        if constexpr (VB) {
                            const int to = (16 * e + 4 * lg + v) * SB + i;
                            const float z1 = z - top_f32(z);
                            s.sb[0][to] = (uint16_t)(__float_as_uint(z) >> 16);
                            s.sb[1][to] = (uint16_t)(__float_as_uint(z1) >> 16);
                            s.sb[2][to] = (uint16_t)(__float_as_uint(z1 - top_f32(z1)) >> 16);
                        } else {
                            dst[v * SS + WC + 16 * (c - wt)] = z;
                        }
                    }
                }
            }
            if constexpr (KDA) {
                // the row's ancestors two at a time
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const int r = w + NW * (lg + 4 * p), n = 16 * GB * g + r;
                    for (int c = li; c < 16 * (GB * g + nb); c += 16) s.s[0][r * SS + WC + c] = s.s[1][r * SS + WC + c] = 0.0f;
                    auto key = [&](int i, float (&y)[CH]) {
#pragma unroll
                        for (int u = 0; u < CH; ++u) {
                            const int ch = 64 * (u / 4) + 4 * li + u % 4;
                            y[u] = X::RK ? widen(s.kr[X::RK ? i * D + ch : 0]) : tok_ld<TI>(a.k, ((size_t)min(i, N - 1) * heads + head) * D + ch);
                        }
                    };
                    auto decay = [&](int i, float (&y)[CH]) {
#pragma unroll
                        for (int u = 0; u < CH; ++u) y[u] = s.gk[i * D + 64 * (u / 4) + 4 * li + u % 4];
                    };
                    float kn[CH], gn[CH];
                    key(n, kn);
                    decay(n, gn);
                    const float nbt = -s.beta[n];
                    uint64_t left = (here >> n) & 1u ? s.t.mask[n] | (1ull << n) : 0;
                    while (__any(left != 0)) {
                        int i[2];
                        float ki[2][CH], gi[2][CH], xq[2] = {0.0f, 0.0f}, xk[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            i[h] = left ? __builtin_ctzll(left) : -1;
                            left &= left - 1;
                            key(max(i[h], 0), ki[h]);      // (none left: node 0's, unused)
                            decay(max(i[h], 0), gi[h]);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int u = 0; u < CH; ++u) {
                                const float y = i[h] == n ? ki[h][u] : ki[h][u] * __expf(gn[u] - gi[h][u]);
                                xq[h] += widen(qraw[p][u]) * y;
                                xk[h] += kn[u] * y;
                            }
                            xq[h] = group_sum<16>(xq[h]);
                            xk[h] = group_sum<16>(xk[h]);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (li == 0 && i[h] >= 0) {
                                s.s[0][r * SS + WC + i[h]] = xq[h];
                                if (i[h] != n) s.s[1][r * SS + WC + i[h]] = nbt * xk[h];
                            }
                    }
                }
            }
        }
        auto compensators = [&](int e, int x, v4f (&cmp)[2]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float z = 0.0f;
#pragma unroll
                for (int m = NP - 1; m >= 0; --m) z += bf16_to_f32((x ? kbase + m * KP : &s.q[m][0])[(16 * e + li) * QS + ci[u]]);
                if (C > 4 * u) {
                    cmp[0] = mfma4(z, cb[u][0], cmp[0]);
                    cmp[1] = mfma4(z, cb[u][1], cmp[1]);
                }
            }
        };
        [[maybe_unused]] v4f kcmp[NX][2];
        if constexpr (FOLD)
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                kcmp[x][0] = kcmp[x][1] = v4f{0.f, 0.f, 0.f, 0.f};
                compensators(0, x, kcmp[x]);
            }
        __syncthreads();
        // ---- 3. products with the state ----
        // where the keys must stay for the next groups' scores, q and k take turns in the rows of q
        constexpr bool TURNS = FOLD && DELTA && !KDA;
        auto scaled_rows = [&](int x0, int x1) {
            const bool on = (here >> (16 * g + row)) & 1u;
#pragma unroll
            for (int x = x0; x < x1; ++x) {
                float y[8];
                uint32_t p[3][4];
                widen8<TI>(x ? rk[0] : rq[0], y);
#pragma unroll
                for (int u = 0; u < 8; ++u) y[u] = on ? y[u] * sc[u] : 0.0f;
                split3<8>(y, p);
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    *reinterpret_cast<u32x4*>((x && !TURNS ? kbase + m * KP : &s.q[m][0]) + row * QS + c8) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
            __syncthreads();
        };
        if constexpr (FOLD) {
#pragma unroll
            for (int u = 0; u < 8; ++u) sc[u] = KDA ? sc[u] * s.r[c8 + u] : s.r[c8 + u];
            scaled_rows(0, TURNS ? 1 : NX);
        }
        v4f acc[GB][NX][2];
#pragma unroll
        for (int e = 0; e < GB; ++e)
#pragma unroll
            for (int x = 0; x < NX; ++x) acc[e][x][0] = acc[e][x][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int turn = 0; turn < (TURNS ? 2 : 1); ++turn) {
            if constexpr (TURNS)
                if (turn) {
                    __syncthreads();                           // q's rows are read
                    scaled_rows(1, 2);
                }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    // B operands: channels 64 ks + 16 lg + 8 hf .. + 7 of columns col + ct
                    const int ch = 64 * ks + 16 * lg + 8 * hf;
                    constexpr int NT8 = X::NT8;
                    u32x4 st[2][NT8];
                    if constexpr (FOLD) {
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint32_t y = (uint32_t)raw[ks][ct][2 * hf + u / 2];
                                st[ct][0][u] = top_halves(sbyte(y, 2 * (u % 2)), sbyte(y, 2 * (u % 2) + 1));
                            }
                    } else {
                        float r[8];
                        load_floats<8>(&s.r[ch], r);
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct) {
                            float x8[8];
                            uint32_t p[NT8][4];
#pragma unroll
                            for (int u = 0; u < 8; ++u) x8[u] = sbyte((uint32_t)raw[ks][ct][2 * hf + u / 4], u % 4) * r[u];
                            split3<8>(x8, p);
#pragma unroll
                            for (int m = 0; m < NT8; ++m) st[ct][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
                        }
                    }
#pragma unroll
                    for (int e = 0; e < GB; ++e) {
                        if (e >= nb) break;
#pragma unroll
                        for (int x = 0; x < NX; ++x) {
                            if (TURNS && x != turn) continue;
                            u32x4 ar[NP];
#pragma unroll
                            for (int m = 0; m < NP; ++m)
                                ar[m] = *reinterpret_cast<const u32x4*>((x && !TURNS ? kbase + m * KP : &s.q[m][0]) + (16 * e + li) * QS + ch);
#pragma unroll
                            for (int ct = 0; ct < 2; ++ct) acc[e][x][ct] = mfma_parts<NP, NT8>(ar, st[ct], acc[e][x][ct]);
                        }
                    }
                }
        }
#pragma unroll
        for (int e = 0; e < GB; ++e) {
            if (e >= nb) break;
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                v4f cmp[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                if constexpr (FOLD) cmp[0] = kcmp[x][0], cmp[1] = kcmp[x][1];
                else compensators(e, x, cmp);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    acc[e][x][ct] = acc[e][x][ct] * sj[ct] + cmp[ct];
                    if constexpr (!KDA) acc[e][x][ct] *= *reinterpret_cast<const v4f*>(&s.e[16 * (GB * g + e) + 4 * lg]);
                }
            }
        }
        if (g + 1 < NG && 16 * GB * (g + 1) < N) {
            request(g + 1);
            __syncthreads();                               // the rows are overwritten by the next group
        }
        // ---- 4. m and o ----
#pragma unroll
        for (int e = 0; e < GB; ++e) {
            if (e >= nb) break;
            const int j = GB * g + e;
            auto context = [&](int x, v4f (&y)[2]) {       // y += scores x context
#pragma unroll
                for (int c = 0; c < WT + (VB ? 0 : NB); ++c) {
                    if (c < WT ? c > 0 && c >= wt : c - WT >= j) continue;
                    const int cc = c < WT ? 16 * c : WC + 16 * (c - WT);
                    const v4f sr = *reinterpret_cast<const v4f*>(&s.s[x][(16 * e + li) * SS + cc + 4 * lg]);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct)
                            y[ct] = mfma4(sr[v], c < WT ? WM[c < WT ? c : 0][ct][v] : M[c < WT || VB ? 0 : c - WT][ct][v], y[ct]);
                }
            };
            if constexpr (DELTA) {
                const v4f be = *reinterpret_cast<const v4f*>(&s.beta[16 * j + 4 * lg]);
                v4f R[2];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int v = 0; v < 4; ++v) R[ct][v] = be[v] * (vv[e][v][ct] - acc[e][NX - 1][ct][v]);
                context(1, R);
                const float* ab = &s.s[1][16 * e * SS + WC + 16 * j];
                v4f own[3];                                                               // -A[4 lg + 1 + i][4 lg + v]
#pragma unroll
                for (int i = 0; i < 3; ++i) own[i] = *reinterpret_cast<const v4f*>(ab + (4 * lg + 1 + i) * SS + 4 * lg);
                float below[3];                                                           // -A[li][4 p + lg]
#pragma unroll
                for (int p = 0; p < 3; ++p) below[p] = (li >> 2) > p ? ab[li * SS + 4 * p + lg] : 0.0f;
                block_solve(own, below, lg, R);
                M[j][0] = R[0];
                M[j][1] = R[1];
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    M[VB ? 0 : j][0][v] = vv[e][v][0];
                    M[VB ? 0 : j][1][v] = vv[e][v][1];
                }
            }
            context(0, acc[e][0]);
            if constexpr (VB) {
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
                    V[VB ? j : 0][ct] = u32x2{top_halves(vv[e][0][ct], vv[e][1][ct]), top_halves(vv[e][2][ct], vv[e][3][ct])};
#pragma unroll
                for (int c = 0; c <= j / 2; ++c) {         // blocks 2 c and 2 c + 1 (none past j: zeros)
                    const bool two = 2 * c + 1 <= j;
                    u32x4 vb[2];
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) {
                        const u32x2 lo = V[VB ? 2 * c : 0][ct], hi = two ? V[VB && two ? 2 * c + 1 : 0][ct] : u32x2{0, 0};
                        vb[ct] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                    }
#pragma unroll
                    for (int part = 2; part >= 0; --part) {
                        const uint16_t* sr = &s.sb[part][(16 * e + li) * SB + 32 * c + 4 * lg];
                        const u32x2 lo = *reinterpret_cast<const u32x2*>(sr), hi = two ? *reinterpret_cast<const u32x2*>(sr + 16) : u32x2{0, 0};
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct) acc[e][0][ct] = mfma_bf16(u32x4{lo[0], lo[1], hi[0], hi[1]}, vb[ct], acc[e][0][ct]);
                    }
                }
            } else {
                const v4f sr = *reinterpret_cast<const v4f*>(&s.s[0][(16 * e + li) * SS + WC + 16 * j + 4 * lg]);
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) acc[e][0][ct] = mfma4(sr[v], M[VB ? 0 : j][ct][v], acc[e][0][ct]);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int n = 16 * j + 4 * lg + v;
                const f32x2 m = {M[VB ? 0 : j][0][v], M[VB ? 0 : j][1][v]};
                odd |= !finite_f32(m[0]) || !finite_f32(m[1]);
                if (!((here >> n) & 1u)) continue;
                const size_t at = ((size_t)n * heads + head) * D + col;
                if constexpr (sizeof(TI) == 4)
                    __builtin_nontemporal_store(f32x2{acc[e][0][0][v], acc[e][0][1][v]}, reinterpret_cast<f32x2*>(static_cast<float*>(a.o) + at));
                else
                    st_nt(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + at), pack_bf16(acc[e][0][0][v], acc[e][0][1][v]));
                __builtin_nontemporal_store(m, reinterpret_cast<f32x2*>(a.tm + (head * N + n) * (size_t)D + col));
            }
        }
    }
    if (__syncthreads_or(odd)) {
        all_loads_barrier();                               // (this pass's stores are done: the rows are written again)
        tree_simple<D, RULE, TI, NT>(a, pos, sp.f.t.mask, sp.f.t.par, here, sp.f.s);
    }
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
    if (d.dk == 16)
        return args.N <= 16 ? launch_kernel(LQ_KERNEL_TREE, tree_small_kernel<1, RULE, TI>, dim3((unsigned)args.heads), dim3(64), s, args)
                            : launch_kernel(LQ_KERNEL_TREE, tree_small_kernel<4, RULE, TI>, dim3((unsigned)args.heads), dim3(64), s, args);
    return d.dk == 64 ? tree_mfma<64, RULE, TI>(d, args, s) : tree_mfma<128, RULE, TI>(d, args, s);
}

}  // namespace

template <int RULE>
hipError_t launch_tree_rule(const lq_dims& d, const TreeArgs& args, hipStream_t s) {
    return d.io_dtype == LQ_IO_BF16 ? tree_io<RULE, uint16_t>(d, args, s) : tree_io<RULE, float>(d, args, s);
}
#endif

}  // namespace lq

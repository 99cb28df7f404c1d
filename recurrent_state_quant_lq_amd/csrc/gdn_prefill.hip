// gdn_prefill.hip -- the gated delta rule over a padded batch of prompts (gfx950).
//
//     H <- (I - beta k k^T) D H + beta k v^T,   o = H^T q  (after the update),
// D = alpha I or diag(alpha).
#include "gdn.h"
#include "la.h"
#include "lq_split.h"

namespace lq {
namespace {

struct GdnPrefillArgs {
    const float* h0;          // or null: zeros
    float* h;
    const void* q;            // q, k, v, o: fp32 or bf16 (the kernel's TI)
    const void* k;
    const void* v;
    const float* alpha;
    const float* beta;
    const int32_t* lens;      // per batch row, or null: T
    void* o;                  // or null
    int T;
    int H;
    int heads;                // B*H: stride between tokens, in heads
};

// ---------------------------------------------------------------------------
// the recurrence itself
// ---------------------------------------------------------------------------
// Per token p = (D H)^T k, z = (D H)^T q, u = beta (v - p), H <- D H + k u^T,
// o = z + (k . q) u: one pass over the state for both sums and one for the update.  Lane t
// holds the columns 4 (t % (D/4)) .. +3 of the rows t / (D/4) + RPP p; tokens come through
// LDS, kGdnStepTokens at a time, requested with the state.
template <int D, bool KDA, typename TI>
__global__ __launch_bounds__(256) void gdn_step_kernel(GdnPrefillArgs a) {
    constexpr int CP = D / 4, NT = D >= 64 ? 256 : 64, RPP = NT / CP, NP = D / RPP, NW = NT / 64, ST = kGdnStepTokens;
    constexpr int NX = ST * D / NT;                                // values of each kind per thread
    constexpr int KINDS = KDA ? 4 : 3;
    __shared__ __align__(16) float sx[KINDS][ST * D];              // q, k, v [, alpha]
    __shared__ float s_al[ST], s_be[ST];
    __shared__ __align__(16) float sp[2][2][NW][D];                // [token parity][p, z]
    __shared__ float s_kq[2][NW];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int T = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int rg = t / CP, c0 = 4 * (t % CP);
    const float* h0 = a.h0 + head * (size_t)(D * D);
    v4f H[NP];
    for (int n0 = 0; n0 < max(T, 1); n0 += ST) {
        TI x[3][NX];
        float xa[NX];
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            const int e = t + NT * u, n = n0 + e / D;
            if (n >= T) break;
            const size_t at = ((size_t)n * heads + head) * D + e % D;
            x[0][u] = static_cast<const TI*>(a.q)[at];
            x[1][u] = static_cast<const TI*>(a.k)[at];
            x[2][u] = static_cast<const TI*>(a.v)[at];
            if (KDA) xa[u] = a.alpha[at];
        }
        float al = 1.0f, be = 0.0f;
        if (t < ST && n0 + t < T) {
            be = a.beta[(size_t)(n0 + t) * heads + head];
            if (!KDA) al = a.alpha[(size_t)(n0 + t) * heads + head];
        }
        if (n0 == 0)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                H[p] = v4f{0.f, 0.f, 0.f, 0.f};
                if (a.h0) H[p] = ld_nt(reinterpret_cast<const v4f*>(h0 + (size_t)(p * RPP + rg) * D + c0));
            }
        else
            __syncthreads();                                       // the tokens before are read
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            const int e = t + NT * u;
            if (n0 + e / D >= T) break;
#pragma unroll
            for (int y = 0; y < 3; ++y) sx[y][e] = widen(x[y][u]);
            if (KDA) sx[KINDS - 1][e] = xa[u];
        }
        if (t < ST) {
            s_al[t] = al;
            s_be[t] = be;
        }
        __syncthreads();
        for (int n = n0; n < min(T, n0 + ST); ++n) {
            const int i = n - n0, par = n & 1;
            const float *q = sx[0] + i * D, *k = sx[1] + i * D, *av = sx[KINDS - 1] + i * D;
            const v4f vv = *reinterpret_cast<const v4f*>(&sx[2][i * D + c0]);
            const float alpha = s_al[i], beta = s_be[i];
            v4f pp = {0.f, 0.f, 0.f, 0.f}, zz = pp;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int row = p * RPP + rg;
                H[p] *= KDA ? av[row] : alpha;
                pp += H[p] * k[row];
                zz += H[p] * q[row];
            }
#pragma unroll
            for (int m = CP; m < 64; m <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pp[e] += __shfl_xor(pp[e], m, 64);
                    zz[e] += __shfl_xor(zz[e], m, 64);
                }
            const float kq = group_sum<64>(t < D ? q[t] * k[t] : 0.0f);
            if (lane < CP) {
                *reinterpret_cast<v4f*>(&sp[par][0][w][c0]) = pp;
                *reinterpret_cast<v4f*>(&sp[par][1][w][c0]) = zz;
            }
            if (lane == 0) s_kq[par][w] = kq;
            __syncthreads();                                       // (the other half is written meanwhile)
            v4f P = {0.f, 0.f, 0.f, 0.f}, Z = P;
            float KQ = 0.0f;
#pragma unroll
            for (int y = 0; y < NW; ++y) {
                P += *reinterpret_cast<const v4f*>(&sp[par][0][y][c0]);
                Z += *reinterpret_cast<const v4f*>(&sp[par][1][y][c0]);
                KQ += s_kq[par][y];
            }
            const v4f u = beta * (vv - P);
#pragma unroll
            for (int p = 0; p < NP; ++p) H[p] += u * k[p * RPP + rg];
            if (a.o && rg == 0)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tok_st<TI>(a.o, ((size_t)n * heads + head) * D + c0 + e, Z[e] + u[e] * KQ);
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
        __builtin_nontemporal_store(H[p], reinterpret_cast<v4f*>(a.h + head * (size_t)(D * D) + (size_t)(p * RPP + rg) * D + c0));
}

// ---------------------------------------------------------------------------
// bf16 tokens, one decay per head, d >= 64: chunks of 64 tokens on bf16 matrix products
// ---------------------------------------------------------------------------
// A workgroup owns a head's state in matrix-instruction accumulators (tile (rt, ct): rows
// 16 rt + 4 (lane / 16) + v, columns 32 w + 2 (lane % 16) + ct of wave w) from the first load
// to the final store.  Per chunk, with g the prefix sums of log alpha (64 bits),
//     A_{n,i} = beta_n e^{g_n - g_i} <k_n, k_i> (i < n),   P_{n,i} = e^{g_n - g_i} <q_n, k_i> (i <= n),
//     R = beta (V - e^g o (K H)),   (I + A) M = R,   O = e^g o (Q H) + P M,
//     H = e^{g_L} H + K^T (e^{g_L - g} o M).
// Tokens enter the products as they are (K^T by transposed LDS reads); H, M, A and P are split into three bf16 parts (all
// their 24 bits).  The accumulator layout is the B operand of the next products, with the rows of
// a 32-block in the order (4 lg + e, 16 + 4 lg + e): K, Q, A and P are stored in that order,
// and H, R and M never leave the registers.  (I + A) M = R runs block after block of 16 tokens:
// the blocks before it on bf16 products, then the inverse of the block itself, which one wave
// forms for all columns (block_solve against the identity), on the fp32 instruction.
// A product of a masked zero with a value that is not finite would spread it to earlier tokens: a
// chunk ends before such a token, which is then the first of its chunk.
constexpr int GL = 64;        // tokens per chunk

struct GdnSegArgs {
    const float* start;       // states before each segment, or null: zeros
    float* end;               // states after each segment, or null: not needed
    float* map;               // maps of each segment, or null (grid.z = 2: the second computes them)
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const float* beta;
    const int32_t* lens;
    void* o;
    size_t seg_stride;        // floats between the states of consecutive segments
    int T, H, heads;
    int seg;                  // tokens per segment
};

template <int L>
struct GdnGates {
    double g[L];
    __align__(16) float e[L], w[L], b[L];
};
// Formed by one wave, lane n = token n; tokens from `left` on decay nothing and change nothing.
// *cut: the first token after the chunk's first one whose gates are not finite.
template <int L>
__device__ __forceinline__ void make_gates(float alpha, float beta, int left, int lane, GdnGates<L>& s, int* cut) {
    const bool on = lane < min(left, L);
    const float la = on ? log_decay(alpha) : 0.0f, be = on ? beta : 0.0f;
    const uint64_t odd = __ballot(lane > 0 && (!finite_f32(la) || !finite_f32(be)));
    if (lane == 0) *cut = odd ? __ffsll((unsigned long long)odd) - 1 : L;
    const double g = wave_scan((double)la);
    const uint64_t bits = __double_as_longlong(g);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)bits, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(bits >> 32), 63);
    const double gl = __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
    // (an exponent is at most 0: off by 2^-24 of it, weighted by its exponential)
    if (lane < L) {
        s.g[lane] = g;
        s.e[lane] = __expf((float)g);
        s.w[lane] = __expf((float)(gl - g));
        s.b[lane] = be;
    }
}

// (n, i) of a 16 x 32 operand block, and block (r, j) of a part of P (j <= r / 2) and of A (r >= 1).
__device__ __forceinline__ constexpr int blk(int row, int i) { return pm<16>(row, (i & 15) >> 2) + 4 * ((i >> 4) & 1) + (i & 3); }
constexpr int kBlk = pm_shorts<16>(4);
__device__ __forceinline__ constexpr int p_blk(int r, int j) { return r < 2 ? r : 2 * r - 2 + j; }
__device__ __forceinline__ constexpr int a_blk(int r, int j) { return r - 1 + j; }
__device__ __forceinline__ constexpr int tile_row(int x) { return x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3; }   // r of x = r (r + 1) / 2 + c

template <int D>
struct GB {
    static constexpr int NW = D / 32, NT = 64 * NW;
    static constexpr int RT = D / 16;
    static constexpr int QP = D / 8;                // pieces per Q / K row
    static constexpr int VS = D / 2 + 4;            // dwords per V row: four rows' columns 16 banks apart
    static constexpr int QROWS = pm_shorts<GL>(QP), PALL = 3 * 6 * kBlk;
};

template <int D, bool OUT>
__global__ __launch_bounds__(GB<D>::NT, 2) void gdn_chunk_kernel(GdnSegArgs a) {
    using P = GB<D>;
    constexpr int NW = P::NW, NT = P::NT, RT = P::RT, QP = P::QP;
    constexpr int LA = 20;                                         // floats per row of A's diagonal blocks
    __shared__ __align__(16) uint16_t sK[pm_shorts<GL>(QP)];
    __shared__ __align__(16) uint32_t sV[GL * P::VS];
    __shared__ __align__(16) uint16_t sA[3][4 * kBlk];             // -A left of the diagonal blocks, in parts
    __shared__ __align__(16) float sD[4][16 * LA];                 // inverses of the diagonal blocks of I + A
    __shared__ __align__(16) uint16_t sQ[OUT ? (P::QROWS > P::PALL ? P::QROWS : P::PALL) : 8];   // Q, then P in parts
    __shared__ GdnGates<GL> s_gate[2];                             // of this chunk and the next
    __shared__ int s_cut[2];

    const int t = threadIdx.x, lane = t & 63;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg;
    const int te = min(len, t0 + a.seg);
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);
    const bool map = !OUT && blockIdx.z;                           // the segment's map: from the identity, without values

    // H[rt][ct][v] = H[16 rt + 4 lg + v][32 w + 2 li + ct]
    v4f H[RT][2];
    if (!map && a.start) {
        const int lg = lane >> 4, band = 16 * w + (lane & 15);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const f32x2 x = *reinterpret_cast<const f32x2*>(a.start + soff + (size_t)(16 * rt + 4 * lg + v) * D + 2 * band);
                H[rt][0][v] = x[0];
                H[rt][1][v] = x[1];
            }
    } else {
        const int diag = map ? 2 * (16 * w + (lane & 15)) - 4 * (lane >> 4) : 1 << 20;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                H[rt][0][v] = 16 * rt + v == diag ? 1.0f : 0.0f;
                H[rt][1][v] = 16 * rt + v == diag + 1 ? 1.0f : 0.0f;
            }
    }
    // columns of A's blocks (1, 0) and (3, 1) that belong to the diagonal blocks: zeros, never written again
    for (int e = t; e < 3 * 2 * 16 * 16; e += NT) sA[e >> 9][((e >> 8) & 1) * (a_blk(3, 1) - a_blk(1, 0)) * kBlk + blk((e >> 4) & 15, 16 + (e & 15))] = 0;

    // chunk loads in registers, one chunk ahead; tokens past `end` read as zeros: pieces of 16 bytes
    constexpr int CPR = D / 8, RPP = NT / CPR;                     // pieces per row, rows per pass
    static_assert(4 * RPP == GL, "four pieces of each kind per thread");
    const uint32_t rb = (uint32_t)heads * (2 * D);                 // bytes between tokens (heads <= chunk_heads(D))
    u32x4 kd[4], vd[4], qd[4];
    auto rows = [&](const void* x, int c0, int end) {              // tokens c0 .. min(c0 + GL, end) - 1 of this head
        return make_rows(static_cast<const char*>(x) + ((size_t)c0 * heads + head) * (2 * D),
                         end > c0 ? (uint32_t)(min(end - c0, GL) - 1) * rb + 2 * D : 0);
    };
    auto load = [&](int c0, int end) {
        const uint32_t tt = fresh(t), off = (tt / CPR) * rb + 16 * (tt % CPR);
        const rsrc_t rk = rows(a.k, c0, end), rv = rows(a.v, c0, end), rq = rows(OUT ? a.q : a.k, c0, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            kd[j] = row_ld4(rk, off + j * RPP * rb);
            if constexpr (OUT) qd[j] = row_ld4(rq, off + j * RPP * rb);
            vd[j] = map ? u32x4{0, 0, 0, 0} : row_ld4(rv, off + j * RPP * rb);
        }
    };
    float al = 1.0f, be = 0.0f;                                    // gates of the next chunk: the last wave's
    auto load_gates = [&](int c0) {
        const size_t at = (size_t)min(c0 + lane, te - 1) * heads + head;
        al = a.alpha[at];
        be = a.beta[at];
    };
    if (t0 < te) {
        load(t0, te);
        if (w == NW - 1) {
            load_gates(t0);
            make_gates<GL>(al, be, te - t0, lane, s_gate[0], &s_cut[0]);
        }
    }
    // registers -> LDS; cut: the first token after the chunk's first one with a value that is not finite
    auto store = [&](int cur) {
        const uint32_t tt = fresh(t), row = tt / CPR, c = 8 * (tt % CPR);
        const int u = (c & 31) >> 2, p0 = (c >> 5) * 4;            // two groups of 4 channels, in operand order
        const int at0 = pm<GL>(row, p0 + (u & 3)) + 4 * (u >> 2), at1 = pm<GL>(row, p0 + ((u + 1) & 3)) + 4 * (u >> 2);
        uint32_t odd = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<u32x2*>(&sK[at0 + pm<GL>(j * RPP, 0)]) = u32x2{kd[j][0], kd[j][1]};
            *reinterpret_cast<u32x2*>(&sK[at1 + pm<GL>(j * RPP, 0)]) = u32x2{kd[j][2], kd[j][3]};
            if constexpr (OUT) {
                *reinterpret_cast<u32x2*>(&sQ[at0 + pm<GL>(j * RPP, 0)]) = u32x2{qd[j][0], qd[j][1]};
                *reinterpret_cast<u32x2*>(&sQ[at1 + pm<GL>(j * RPP, 0)]) = u32x2{qd[j][2], qd[j][3]};
            }
            *reinterpret_cast<u32x4*>(&sV[(row + j * RPP) * P::VS + c / 2]) = vd[j];
            if (j > 0 || row > 0)
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= odd_bf16(kd[j][e]) | odd_bf16(vd[j][e]);
        }
        if (odd) {
            int first = GL;
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                uint32_t x = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) x |= odd_bf16(kd[j][e]) | odd_bf16(vd[j][e]);
                if (x && (j > 0 || row > 0)) first = row + j * RPP;
            }
            atomicMin(&s_cut[cur], first);
        }
    };
    __syncthreads();                                               // the first gates (and s_cut) are written

    int cur = 0, next;
    for (int c0 = t0; c0 < te; c0 = next, cur ^= 1) {
        int ce = min(c0 + GL, te);
        if (w == NW - 1 && ce < te) load_gates(ce);
        store(cur);
        __syncthreads();
        const int cut = s_cut[cur];
        if (cut < ce - c0) {                                       // the chunk again, up to that token
            ce = c0 + cut;
            __syncthreads();
            load(c0, ce);
            if (w == NW - 1) {
                int dummy;
                load_gates(c0);
                make_gates<GL>(al, be, cut, lane, s_gate[cur], &dummy);
                load_gates(ce);
            }
            store(cur);
            __syncthreads();
        }
        next = ce;
        const double* sG = s_gate[cur].g;
        const float *sE = s_gate[cur].e, *sW = s_gate[cur].w, *sB = s_gate[cur].b;
        const float egl = sE[GL - 1];
        const bool more = ce < te;

        // ---- scores: the 10 tiles on and below the diagonal of K K^T and of Q K^T, over the waves ----
        // (tile x = r (r + 1) / 2 + c; its indices are scalars of the wave, so that no code is repeated per tile)
        constexpr int KD = 4 / NW, KT = KD + (6 + NW - 1) / NW, QT = 12 / NW;   // (tiles 10, 11 of Q K^T: zeros right of the diagonal)
        v4f pr[OUT ? QT : 1];
        const int lo = fresh(lane), li = lo & 15, lg = lo >> 4;
        const int at = pm<GL>(li, lg);                             // operand reads: row li, piece lg
#pragma unroll
        for (int y = 0; y < KT; ++y) {
            const bool diag = y < KD;
            const int x = diag ? w + NW * y : min(w + NW * (y - KD), 5);   // block, or tile x = r (r - 1) / 2 + c
            const int r = diag ? x : tile_row(x) + 1, c = diag ? x : x - r * (r - 1) / 2;
            const int ar = at + pm<GL>(16 * r, 0), ac = at + pm<GL>(16 * c, 0);
            const double gi = sG[16 * c + li];
            v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
                acc = mfma_bf16(*reinterpret_cast<const u32x4*>(&sK[ar + pm<GL>(0, 4 * ks)]),
                                *reinterpret_cast<const u32x4*>(&sK[ac + pm<GL>(0, 4 * ks)]), acc);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[v] *= -sB[16 * r + 4 * lg + v] * __expf((float)(sG[16 * r + 4 * lg + v] - gi));
            if (diag) {
                // the block's inverse (I + A)^{-1}: solved against the identity, then an A operand of k = 4 steps
                float* sd = sD[r];
#pragma unroll
                for (int v = 0; v < 4; ++v) sd[(4 * lg + v) * LA + li] = li < 4 * lg + v ? acc[v] : 0.0f;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                v4f own[3], inv[1];
                float below[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) own[i] = *reinterpret_cast<const v4f*>(&sd[(4 * lg + 1 + i) * LA + 4 * lg]);
#pragma unroll
                for (int p = 0; p < 3; ++p) below[p] = (li >> 2) > p ? sd[li * LA + 4 * p + lg] : 0.0f;
#pragma unroll
                for (int v = 0; v < 4; ++v) inv[0][v] = 4 * lg + v == li ? 1.0f : 0.0f;
                block_solve<1>(own, below, lg, inv);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int v = 0; v < 4; ++v) sd[(4 * lg + v) * LA + li] = inv[0][v];
            } else {
                const int to = a_blk(r, c >> 1) * kBlk + 4 * (c & 1) + blk(4 * lg, li);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float p = acc[v], p1 = p - top_f32(p);
                    sA[0][to + 8 * v] = (uint16_t)(__float_as_uint(p) >> 16);
                    sA[1][to + 8 * v] = (uint16_t)(__float_as_uint(p1) >> 16);
                    sA[2][to + 8 * v] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (OUT)
#pragma unroll
            for (int y = 0; y < QT; ++y) {
                const int x = w + NW * y;
                const int r = x < 10 ? tile_row(x) : 2 * (x - 10), c = x < 10 ? x - r * (r + 1) / 2 : r + 1;
                const int ar = at + pm<GL>(16 * r, 0), ac = at + pm<GL>(16 * c, 0);
                const double gi = sG[16 * c + li];
                v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                    acc = mfma_bf16(*reinterpret_cast<const u32x4*>(&sQ[ar + pm<GL>(0, 4 * ks)]),
                                    *reinterpret_cast<const u32x4*>(&sK[ac + pm<GL>(0, 4 * ks)]), acc);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float p = __expf((float)(sG[16 * r + 4 * lg + v] - gi)) * acc[v];
                    pr[y][v] = 16 * (r - c) + 4 * lg + v >= li ? p : 0.0f;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        // ---- K H and Q H ----
        v4f R[4][2], O[OUT ? 4 : 1][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            R[r][0] = R[r][1] = v4f{0.f, 0.f, 0.f, 0.f};
            if constexpr (OUT) O[r][0] = O[r][1] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        auto split_h = [&](int ks, u32x4 (&b)[2][3]) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = H[2 * ks + e / 4][ct][e % 4];
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) b[ct][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
        };
        u32x4 hb[2][2][3];                                         // (the next step's parts are formed during a step)
        split_h(0, hb[0]);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            const u32x4 (&b)[2][3] = hb[ks & 1];
            if (ks + 1 < D / 32) split_h(ks + 1, hb[(ks + 1) & 1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const u32x4 ak = *reinterpret_cast<const u32x4*>(&sK[at + pm<GL>(16 * r, 4 * ks)]);
#pragma unroll
                for (int m = 2; m >= 0; --m)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) R[r][ct] = mfma_bf16(ak, b[ct][m], R[r][ct]);
                if constexpr (OUT) {
                    const u32x4 aq = *reinterpret_cast<const u32x4*>(&sQ[at + pm<GL>(16 * r, 4 * ks)]);
#pragma unroll
                    for (int m = 2; m >= 0; --m)
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct) O[r][ct] = mfma_bf16(aq, b[ct][m], O[r][ct]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const v4f e = *reinterpret_cast<const v4f*>(&sE[16 * r + 4 * lg]);
            const v4f bt = *reinterpret_cast<const v4f*>(&sB[16 * r + 4 * lg]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint32_t x = sV[(16 * r + 4 * lg + v) * P::VS + 16 * w + li];
                R[r][0][v] = bt[v] * (lo_f32(x) - e[v] * R[r][0][v]);
                R[r][1][v] = bt[v] * (hi_f32(x) - e[v] * R[r][1][v]);
            }
            if constexpr (OUT) {
                O[r][0] *= e;
                O[r][1] *= e;
            }
        }
        if (w == NW - 1 && more) make_gates<GL>(al, be, te - ce, lane, s_gate[cur ^ 1], &s_cut[cur ^ 1]);
        __syncthreads();                                           // A is written, Q is read
        if constexpr (OUT) {
            // P in parts, in Q's place; right of the diagonal zeros
#pragma unroll
            for (int y = 0; y < QT; ++y) {
                const int x = w + NW * y;
                const int r = x < 10 ? tile_row(x) : 2 * (x - 10), c = x < 10 ? x - r * (r + 1) / 2 : r + 1;
                const int to = p_blk(r, c >> 1) * kBlk + 4 * (c & 1) + blk(4 * lg, li);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float p = pr[y][v], p1 = p - top_f32(p);
                    sQ[to + 8 * v] = (uint16_t)(__float_as_uint(p) >> 16);
                    sQ[6 * kBlk + to + 8 * v] = (uint16_t)(__float_as_uint(p1) >> 16);
                    sQ[12 * kBlk + to + 8 * v] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
                }
            }
        }
        // ---- (I + A) M = R ----
        u32x4 mp[2][2][3];                                         // M in parts: [32 tokens][ct][part]
        const int ab = blk(li, 4 * lg);                            // operand reads: row li, piece lg
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < (r + 1) / 2; ++j) {
                u32x4 x[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sA[m][a_blk(r, j) * kBlk + ab]);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) R[r][ct] = mfma_split(x, mp[j][ct], R[r][ct]);
            }
            const v4f ti = *reinterpret_cast<const v4f*>(&sD[r][li * LA + 4 * lg]);
            v4f m[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) m[ct] = mfma4(ti[v], R[r][ct][v], m[ct]);
            R[r][0] = m[0];
            R[r][1] = m[1];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const float y[4] = {R[r][ct][0], R[r][ct][1], R[r][ct][2], R[r][ct][3]};
                uint32_t p[3][2];
                split3<4>(y, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    mp[r / 2][ct][m][2 * (r & 1)] = p[m][0];
                    mp[r / 2][ct][m][2 * (r & 1) + 1] = p[m][1];
                    if (!(r & 1)) mp[r / 2][ct][m][2] = mp[r / 2][ct][m][3] = 0;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (OUT) {
            __syncthreads();                                       // P is written
            // ---- O += P M ----
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j <= r / 2; ++j) {
                    u32x4 x[3];
#pragma unroll
                    for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sQ[(6 * m + p_blk(r, j)) * kBlk + ab]);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) O[r][ct] = mfma_split(x, mp[j][ct], O[r][ct]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            const rsrc_t ro = rows(a.o, c0, ce);                   // rows past the end are left as they were
            const uint32_t ooff = 4 * lg * rb + 4 * (16 * w + li);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v) row_st(ro, ooff + (16 * r + v) * rb, pack_bf16(O[r][0][v], O[r][1][v]));
        }
        __builtin_amdgcn_sched_barrier(0);
        load(ce, te);                                              // (none left: zeros; a branch would keep the old rows alive)
        __builtin_amdgcn_sched_barrier(0);
        // ---- H = e^{g_L} H + K^T (w o M) ----
        const int kt = pm<GL>(4 * lg + (li >> 2), li & 3);         // transposed reads: 4 tokens of 16 channels a lane group
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const v4f w0 = *reinterpret_cast<const v4f*>(&sW[32 * j + 4 * lg]);
            const v4f w1 = *reinterpret_cast<const v4f*>(&sW[32 * j + 16 + 4 * lg]);
            u32x4 b[2][3];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = (e < 4 ? w0[e & 3] : w1[e & 3]) * R[2 * j + e / 4][ct][e % 4];
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) b[ct][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint16_t* from = &sK[kt + pm<GL>(32 * j, 4 * (rt >> 1)) + 4 * (rt & 1)];
                const u32x2 k0 = lds_tr(from), k1 = lds_tr(from + pm<GL>(16, 0));
                const u32x4 ak = {k0[0], k0[1], k1[0], k1[1]};
                if (j == 0) {
                    H[rt][0] *= egl;
                    H[rt][1] *= egl;
                }
#pragma unroll
                for (int m = 2; m >= 0; --m)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) H[rt][ct] = mfma_bf16(ak, b[ct][m], H[rt][ct]);
                if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();                                           // LDS is rewritten by the next chunk
    }
    float* end = map ? a.map : a.end;
    if (!end) return;
    const int lf = fresh(lane), lg = lf >> 4, band = 16 * w + (lf & 15);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            *reinterpret_cast<f32x2*>(end + soff + (size_t)(16 * rt + 4 * lg + v) * D + 2 * band) = f32x2{H[rt][0][v], H[rt][1][v]};
}

// Heads that the chunk kernels take: a chunk's rows lie within 32-bit byte offsets.
constexpr size_t chunk_heads(int d) { return (size_t)(1 << 24) / d; }

template <int D, bool KDA, typename TI>
hipError_t gdn_prefill_t(const lq_dims& d, const GdnPrefillArgs& args, void* workspace, hipStream_t s) {
    const dim3 grid((unsigned)args.heads);
    if constexpr (D >= 64 && !KDA && sizeof(TI) == 2)
        if (args.T > kGdnStepTokens && (size_t)args.heads <= chunk_heads(D)) {
            GdnSegArgs sa{args.h0, args.h, nullptr, args.q, args.k, args.v, args.alpha, args.beta, args.lens, args.o, 0,
                          args.T, args.H, args.heads, args.T};
            return args.o ? launch_kernel(LQ_KERNEL_PREFILL, gdn_chunk_kernel<D, true>, grid, dim3(GB<D>::NT), s, sa)
                          : launch_kernel(LQ_KERNEL_PREFILL, gdn_chunk_kernel<D, false>, grid, dim3(GB<D>::NT), s, sa);
        }
    return launch_kernel(LQ_KERNEL_PREFILL, gdn_step_kernel<D, KDA, TI>, grid, dim3(D >= 64 ? 256 : 64), s, args);
}

template <int D>
hipError_t gdn_prefill_d(const lq_dims& d, const GdnPrefillArgs& args, void* workspace, hipStream_t s) {
    const bool bf16 = d.io_dtype == LQ_IO_BF16;
    if (d.decay_mode == LQ_DECAY_PER_KEY)
        return bf16 ? gdn_prefill_t<D, true, uint16_t>(d, args, workspace, s)
                    : gdn_prefill_t<D, true, float>(d, args, workspace, s);
    return bf16 ? gdn_prefill_t<D, false, uint16_t>(d, args, workspace, s)
                : gdn_prefill_t<D, false, float>(d, args, workspace, s);
}

}  // namespace

size_t gdn_workspace_bytes(const lq_dims& d, int T) { return 0; }

hipError_t launch_gdn_prefill(const lq_dims& d, const float* h0, float* h, int T, const void* q, const void* k,
                              const void* v, const float* alpha, const float* beta, const int32_t* lens, void* o,
                              void* workspace, hipStream_t s) {
    GdnPrefillArgs args{h0, h, q, k, v, alpha, beta, lens, o, T, d.H, d.B * d.H};
    switch (d.dk) {
        case 16: return gdn_prefill_d<16>(d, args, workspace, s);
        case 64: return gdn_prefill_d<64>(d, args, workspace, s);
        default: return gdn_prefill_d<128>(d, args, workspace, s);
    }
}

}  // namespace lq

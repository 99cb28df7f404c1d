// gdn_prefill.hip -- the gated delta rule over a padded batch of prompts (gfx950).
//
//     H <- (I - beta k k^T) D H + beta k v^T,   o = H^T q  (after the update),
// D = alpha I or diag(alpha).
#include "gdn.h"
#include "la.h"
#include "lq_split.h"

#include <algorithm>
#include <type_traits>

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
// LDS, kGdnStepTokens at a time, requested with the state.  Bound by memory: one token of 2048 heads
// (d = 128, bf16) 50 us, 5.4 TB/s of the states read and written.  Up to four tokens take it: its token costs
// one pass over registers, a chunk's products the same whatever it holds.
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
// 16 rt + 4 (lane / 16) + v, columns CT (16 w + lane % 16) + ct of wave w, CT = d / 64) from the first load
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
// Bound by the two issue ports of a SIMD in turn: 2048 heads of 512 tokens (d = 128) 512 to 565 us, vector 0.56 and
// matrix 0.53 of the waves' time (two waves a SIMD; 0.96 PFLOP/s of matrix work, a large product of the library
// 1.22, both with the clock that the power leaves); LDS 0.42.  Four waves of 32 columns, since each wave reads
// all of K and Q: eight of 16 took 588 us.  Not kept: the parts of H formed in between the products by
// the scheduler's groups (577), the inverses' steps in between K H (544 to 615), the halves of every second
// piece swapped as in the kernel of 32 tokens (the same at d = 128; 164, not 141, for 512 heads of 1024 tokens
// at d = 64).
constexpr int GL = 64;        // tokens per chunk

struct GdnSegArgs {
    const float* first;       // state before the first segment, or null: zeros
    const float* start;       // states before the segments after it, or null: zeros (their own parts alone)
    float* end;               // states after each segment, or null: not needed
    float* map;               // maps of the segments after the first (grid.z = 2: the second computes them)
    float* fin;               // state after the last segment, or null: not needed
    float* keep;              // null, or where the state before the first segment is copied (h0 is h)
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

// A segment after the first without tokens: what the row holds stays, and only the last one has to write it.
template <bool OUT>
__device__ __forceinline__ bool past_end(int t0, int len) { return t0 >= len && !(OUT && blockIdx.y == gridDim.y - 1); }

template <int L>
struct GdnGates {
    double g[L];
    __align__(16) float e[L], w[L], b[L];
};
template <int L>
struct GdnSteps {             // per key: the decays are in the rows
    __align__(16) float b[L];
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

// What the scan reads is kept (d >= 64) in the tiles of 16 x 16 that its lanes hold, each load a run of 1 KB: a
// segment's states as the accumulators of this file's kernels hold them (whichever columns those are: the scan's
// are independent), its map as the scan's operand, row li, columns 4 lg .. 4 lg + 3 of a tile.  (With both as
// rows of the matrix, four runs of 64 bytes a load, a step of the scan took 2.4 us at d = 128, not 1.5.)
__device__ __forceinline__ v4f* state_at(float* x, int tiles, int row_tile, int col_tile, int lane) {
    return reinterpret_cast<v4f*>(x) + (size_t)(row_tile * tiles + col_tile) * 64 + lane;
}
template <int D>
__device__ __forceinline__ v4f* map_at(float* map, int row, int col) {
    return reinterpret_cast<v4f*>(map) + (size_t)((row >> 4) * (D / 16) + (col >> 4)) * 64 + ((col >> 2) & 3) * 16 + (row & 15);
}
// Accumulators (rows 4 lg + v, column li) as row 4 lg + li % 4, columns 4 (li / 4) + v.
__device__ __forceinline__ v4f quad_rows(const v4f& x, int li) {
    const bool odd = li & 1, up = li & 2;
    const float a = dpp<DPP_XOR1>(odd ? x[0] : x[1]), b = dpp<DPP_XOR1>(odd ? x[2] : x[3]);
    const float a0 = odd ? a : x[0], a1 = odd ? x[1] : a, b0 = odd ? b : x[2], b1 = odd ? x[3] : b;
    const float c = dpp<DPP_XOR2>(up ? a0 : b0), e = dpp<DPP_XOR2>(up ? a1 : b1);
    return up ? v4f{c, e, b0, b1} : v4f{a0, a1, c, e};
}

// (n, i) of a 16 x 32 operand block, and block (r, j) of a part of P (j <= r / 2) and of A (r >= 1).
__device__ __forceinline__ constexpr int blk(int row, int i) { return pm<16>(row, (i & 15) >> 2) + 4 * ((i >> 4) & 1) + (i & 3); }
constexpr int kBlk = pm_shorts<16>(4);
__device__ __forceinline__ constexpr int p_blk(int r, int j) { return r < 2 ? r : 2 * r - 2 + j; }
__device__ __forceinline__ constexpr int a_blk(int r, int j) { return r - 1 + j; }
__device__ __forceinline__ constexpr int tile_row(int x) { return x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3; }   // r of x = r (r + 1) / 2 + c

template <int D>
struct GB {
    static constexpr int NW = 4, NT = 64 * NW;
    static constexpr int CT = D / 64;               // column tiles per wave
    static constexpr int RT = D / 16;
    static constexpr int QP = D / 8;                // pieces per Q / K row
    static constexpr int VS = D + 8;                // values per V row: four rows' columns 16 banks apart
    static constexpr int QROWS = pm_shorts<GL>(QP), PALL = 3 * 6 * kBlk;
    static constexpr int QV(bool out) { return !out ? GL * VS : QROWS + GL * VS > PALL ? QROWS + GL * VS : PALL; }
    static constexpr int WPE = CT == 1 ? 3 : 2;     // workgroups per CU: registers at d = 128, LDS at d = 64
};

template <int D, bool OUT>
__global__ __launch_bounds__(GB<D>::NT, GB<D>::WPE) void gdn_chunk_kernel(GdnSegArgs a) {
    using P = GB<D>;
    constexpr int NW = P::NW, NT = P::NT, RT = P::RT, QP = P::QP, CT = P::CT;
    constexpr int LA = 20;                                         // floats per row of A's diagonal blocks
    __shared__ __align__(16) uint16_t sK[pm_shorts<GL>(QP)];
    __shared__ __align__(16) uint16_t sA[3][4 * kBlk];             // -A left of the diagonal blocks, in parts
    __shared__ __align__(16) float sD[4][16 * LA];                 // inverses of the diagonal blocks of I + A
    __shared__ __align__(16) uint16_t sQV[P::QV(OUT)];             // V and Q, then P in parts
    uint16_t *sV = sQV, *sQ = sQV + GL * P::VS;
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
    if (blockIdx.y ? past_end<OUT>(t0, len) : map) return;
    const float* start = blockIdx.y == 0 ? a.first : a.start;

    // H[rt][ct][v] = H[16 rt + 4 lg + v][CT (16 w + li) + ct]
    typedef float cols __attribute__((ext_vector_type(CT)));
    v4f H[RT][CT];
    if (!map && start && blockIdx.y > 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) H[rt][ct] = *state_at(const_cast<float*>(start) + soff, D / 16, rt, CT * w + ct, lane);
    } else if (!map && start) {
        const float* x = start + head * (size_t)(D * D) + (size_t)(4 * (lane >> 4)) * D + CT * (16 * w + (lane & 15));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const cols y = *reinterpret_cast<const cols*>(x + (size_t)(16 * rt + v) * D);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) H[rt][ct][v] = y[ct];
            }
    } else {
        const int diag = map ? CT * (16 * w + (lane & 15)) - 4 * (lane >> 4) : 1 << 20;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) H[rt][ct][v] = 16 * rt + v == diag + ct ? 1.0f : 0.0f;
    }
    auto write_state = [&](float* to) {
        const int lf = fresh(lane);
        to += (size_t)(4 * (lf >> 4)) * D + CT * (16 * w + (lf & 15));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                cols y;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[ct] = H[rt][ct][v];
                *reinterpret_cast<cols*>(to + (size_t)(16 * rt + v) * D) = y;
            }
    };
    if (!OUT && a.keep && !map && blockIdx.y == 0) write_state(a.keep + head * (size_t)(D * D));
    // columns of A's blocks (1, 0) and (3, 1) that belong to the diagonal blocks: zeros, never written again
    for (int e = t; e < 3 * 2 * 16 * 16; e += NT) sA[e >> 9][((e >> 8) & 1) * (a_blk(3, 1) - a_blk(1, 0)) * kBlk + blk((e >> 4) & 15, 16 + (e & 15))] = 0;

    // chunk loads in registers, one chunk ahead; tokens past `end` read as zeros: pieces of 16 bytes
    constexpr int CPR = D / 8, RPP = NT / CPR, PT = GL / RPP;      // pieces per row, rows per pass, pieces of each kind per thread
    const uint32_t rb = (uint32_t)heads * (2 * D);                 // bytes between tokens (heads <= chunk_heads(D))
    u32x4 kd[PT], vd[PT], qd[PT];
    auto rows = [&](const void* x, int c0, int end) {              // tokens c0 .. min(c0 + GL, end) - 1 of this head
        return make_rows(static_cast<const char*>(x) + ((size_t)c0 * heads + head) * (2 * D),
                         end > c0 ? (uint32_t)(min(end - c0, GL) - 1) * rb + 2 * D : 0);
    };
    auto load = [&](int c0, int end) {
        const uint32_t tt = fresh(t), off = (tt / CPR) * rb + 16 * (tt % CPR);
        const rsrc_t rk = rows(a.k, c0, end), rv = rows(a.v, c0, end), rq = rows(OUT ? a.q : a.k, c0, end);
#pragma unroll
        for (int j = 0; j < PT; ++j) {
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
        for (int j = 0; j < PT; ++j) {
            *reinterpret_cast<u32x2*>(&sK[at0 + pm<GL>(j * RPP, 0)]) = u32x2{kd[j][0], kd[j][1]};
            *reinterpret_cast<u32x2*>(&sK[at1 + pm<GL>(j * RPP, 0)]) = u32x2{kd[j][2], kd[j][3]};
            if constexpr (OUT) {
                *reinterpret_cast<u32x2*>(&sQ[at0 + pm<GL>(j * RPP, 0)]) = u32x2{qd[j][0], qd[j][1]};
                *reinterpret_cast<u32x2*>(&sQ[at1 + pm<GL>(j * RPP, 0)]) = u32x2{qd[j][2], qd[j][3]};
            }
            *reinterpret_cast<u32x4*>(&sV[(row + j * RPP) * P::VS + c]) = vd[j];
            if (j > 0 || row > 0)
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= odd_bf16(kd[j][e]) | odd_bf16(vd[j][e]);
        }
        if (odd) {
            int first = GL;
#pragma unroll
            for (int j = PT - 1; j >= 0; --j) {
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
        constexpr int QT = 3;                                      // (tiles 10, 11 of Q K^T: zeros right of the diagonal)
        v4f pr[OUT ? QT : 1];
        const int lo = fresh(lane), li = lo & 15, lg = lo >> 4;
        const int at = pm<GL>(li, lg);                             // operand reads: row li, piece lg
#pragma unroll
        for (int y = 0; y < 3; ++y) {
            const bool diag = y == 0;
            const int x = diag ? w : min(w + NW * (y - 1), 5);     // block, or tile x = r (r - 1) / 2 + c (the last one again where none is left)
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
        v4f R[4][CT], O[OUT ? 4 : 1][CT];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                R[r][ct] = v4f{0.f, 0.f, 0.f, 0.f};
                if constexpr (OUT) O[r][ct] = v4f{0.f, 0.f, 0.f, 0.f};
            }
        auto split_h = [&](int ks, u32x4 (&b)[CT][3]) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = H[2 * ks + e / 4][ct][e % 4];
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) b[ct][m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
        };
        u32x4 hb[2][CT][3];                                         // (the next step's parts are formed during a step)
        split_h(0, hb[0]);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            const u32x4 (&b)[CT][3] = hb[ks & 1];
            if (ks + 1 < D / 32) split_h(ks + 1, hb[(ks + 1) & 1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const u32x4 ak = *reinterpret_cast<const u32x4*>(&sK[at + pm<GL>(16 * r, 4 * ks)]);
#pragma unroll
                for (int m = 2; m >= 0; --m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) R[r][ct] = mfma_bf16(ak, b[ct][m], R[r][ct]);
                if constexpr (OUT) {
                    const u32x4 aq = *reinterpret_cast<const u32x4*>(&sQ[at + pm<GL>(16 * r, 4 * ks)]);
#pragma unroll
                    for (int m = 2; m >= 0; --m)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) O[r][ct] = mfma_bf16(aq, b[ct][m], O[r][ct]);
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
                const uint16_t* x = &sV[(16 * r + 4 * lg + v) * P::VS + CT * (16 * w + li)];
                if constexpr (CT == 2) {
                    const uint32_t y = *reinterpret_cast<const uint32_t*>(x);
                    R[r][0][v] = bt[v] * (lo_f32(y) - e[v] * R[r][0][v]);
                    R[r][CT - 1][v] = bt[v] * (hi_f32(y) - e[v] * R[r][CT - 1][v]);
                } else {
                    R[r][0][v] = bt[v] * (bf16_to_f32(*x) - e[v] * R[r][0][v]);
                }
            }
            if constexpr (OUT)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) O[r][ct] *= e;
        }
        if (w == NW - 1 && more) make_gates<GL>(al, be, te - ce, lane, s_gate[cur ^ 1], &s_cut[cur ^ 1]);
        __syncthreads();                                           // A is written, Q and V are read
        if constexpr (OUT) {
            // P in parts, in the place of V and Q; right of the diagonal zeros
#pragma unroll
            for (int y = 0; y < QT; ++y) {
                const int x = w + NW * y;
                const int r = x < 10 ? tile_row(x) : 2 * (x - 10), c = x < 10 ? x - r * (r + 1) / 2 : r + 1;
                const int to = p_blk(r, c >> 1) * kBlk + 4 * (c & 1) + blk(4 * lg, li);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float p = pr[y][v], p1 = p - top_f32(p);
                    sQV[to + 8 * v] = (uint16_t)(__float_as_uint(p) >> 16);
                    sQV[6 * kBlk + to + 8 * v] = (uint16_t)(__float_as_uint(p1) >> 16);
                    sQV[12 * kBlk + to + 8 * v] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
                }
            }
        }
        // ---- (I + A) M = R ----
        u32x4 mp[2][CT][3];                                        // M in parts: [32 tokens][ct][part]
        const int ab = blk(li, 4 * lg);                            // operand reads: row li, piece lg
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < (r + 1) / 2; ++j) {
                u32x4 x[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sA[m][a_blk(r, j) * kBlk + ab]);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) R[r][ct] = mfma_split(x, mp[j][ct], R[r][ct]);
            }
            const v4f ti = *reinterpret_cast<const v4f*>(&sD[r][li * LA + 4 * lg]);
            v4f m[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) m[ct] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) m[ct] = mfma4(ti[v], R[r][ct][v], m[ct]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) R[r][ct] = m[ct];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
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
                    for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sQV[(6 * m + p_blk(r, j)) * kBlk + ab]);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) O[r][ct] = mfma_split(x, mp[j][ct], O[r][ct]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            const rsrc_t ro = rows(a.o, c0, ce);                   // rows past the end are left as they were
            if constexpr (CT == 2) {
                const uint32_t ooff = 4 * lg * rb + 4 * (16 * w + li);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int v = 0; v < 4; ++v) row_st(ro, ooff + (16 * r + v) * rb, pack_bf16(O[r][0][v], O[r][CT - 1][v]));
            } else {
                // lanes in pairs: the even one stores both columns of the rows v, the odd one those of v + 1
                const bool up = li & 1;
                const uint32_t ooff = (4 * lg + (li & 1)) * rb + 2 * (16 * w + (li & 14));
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int v = 0; v < 4; v += 2) {
                        const float x = dpp<DPP_XOR1>(up ? O[r][0][v] : O[r][0][v + 1]);
                        row_st(ro, ooff + (16 * r + v) * rb, up ? pack_bf16(x, O[r][0][v + 1]) : pack_bf16(O[r][0][v], x));
                    }
            }
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
            u32x4 b[CT][3];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
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
                if (j == 0)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) H[rt][ct] *= egl;
#pragma unroll
                for (int m = 2; m >= 0; --m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) H[rt][ct] = mfma_bf16(ak, b[ct][m], H[rt][ct]);
                if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();                                           // LDS is rewritten by the next chunk
    }
    if (map) {
        const int lo = fresh(lane), li = lo & 15, lg = lo >> 4;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if constexpr (CT == 1) {
                *map_at<D>(a.map + soff, 16 * rt + 4 * lg + (li & 3), 16 * w + (li & 12)) = quad_rows(H[rt][0], li);
            } else {                                               // two columns a lane: the even lane the rows v = 0, 1
                const bool odd = li & 1;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const float x0 = H[rt][0][v], x1 = H[rt][1][v], y0 = H[rt][0][2 + v], y1 = H[rt][1][2 + v];
                    const float r0 = dpp<DPP_XOR1>(odd ? x0 : y0), r1 = dpp<DPP_XOR1>(odd ? x1 : y1);
                    *map_at<D>(a.map + soff, 16 * rt + 4 * lg + 2 * (li & 1) + v, 32 * w + 2 * (li & 14)) =
                        odd ? v4f{r0, r1, y0, y1} : v4f{x0, x1, r0, r1};
                }
            }
        }
        return;
    }
    if (a.end) {
        const int lo = fresh(lane);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) *state_at(a.end + soff, D / 16, rt, CT * w + ct, lo) = H[rt][ct];
    }
    if (a.fin && blockIdx.y == gridDim.y - 1) write_state(a.fin + head * (size_t)(D * D));
}

// ---------------------------------------------------------------------------
// fp32 tokens, or a decay per key channel, d >= 64: chunks of 32 tokens, every operand in parts
// ---------------------------------------------------------------------------
// The same algebra with all operands in three bf16 parts (six products of nine: the others are at
// most 2^-21 of a product, 2^-24.7 on average).  Wave w owns the 16 columns 16 w + li.
// A decay per key channel: with f the prefix products (per channel) of the decays after the
// chunk's first token,
//     H' = diag(alpha_0) H,  x_n = f_n o k_n (and q_n),  y_i = k_i / f_i,
//     A_{n,i} = beta_n <x_n, y_i>,  P_{n,i} = <f_n o q_n, y_i>,  R = beta (V - X H'),
//     O = (f o Q) H' + P M,  H = diag(f_L) (H' + Y^T M),
// so neither logarithms nor exponentials are formed.  f_n / f_i holds the roundings of the factors
// between the two tokens, as the recurrence's own products do (one of 2^-24 a factor), and those of
// at most one product and one reciprocal more.  1 / f grows: a chunk ends before a token whose f
// leaves [kMinDecay, 1 / kMinDecay] in a channel (the parts are in range there), which is then the
// first of the next chunk, and whose own decay goes to H as it is.  Y^T M stands before f_L: rows x carry a
// power of two s near f_L^(-3/8) besides, y and H' its inverse (exact, and 1 down to f_L = 2^-2), so that M may be
// up to 2^64 / |k| and H' down to 2^-68 at the border (without s 2^30 / |k|: values of 10^13 overflowed).
// Every second piece of an operand row has its halves swapped, in LDS and in H's order on its way to the
// products: the transposed reads, half a piece each, then use all banks (1024 heads of 512 tokens, per key,
// 458, not 474 us).
// bf16 values are loaded by lanes in pairs, two columns of every second row each (512 heads of 1024 tokens at
// d = 64, per key, 206, not 214 us, with a load a value).
// Bound by vector, matrix and LDS time in turn.  Per key, 1024 heads of 512 tokens 465 to 485 us (bf16): two workgroups
// a CU, vector 0.70, matrix 0.48, LDS 0.56 of the time; a quarter of a chunk's is the forming of the rows'
// parts.  That is with decays of down to 2^-2.9 a token, whole chunks; if one channel of a head decays faster, a chunk
// holds the 92 / -log2(alpha) tokens after its first one, each cut one is loaded and split twice, and the time grows: 730 us at
// 2^-4, 1220 at 2^-8, 2370 at 2^-16, 14000 where a channel forgets every token (chunks of one).  fp32, 192 heads of
// up to 1021 tokens 209 us: one workgroup a CU, the longest row's 32 chunks, 6.6 us each
// (0.45, 0.39, 0.39); 512 heads of 512 tokens 216 to 226 us (0.67, 0.59, 0.58).  Six bf16 products
// take 96 cycles where the fp32 instruction takes 256.
constexpr int GF = 32;        // tokens per chunk
constexpr float kMinDecay = 0x1p-92f;

// A prefix product leaves the range, or is no number.
__device__ __forceinline__ bool decays_far(float f) { return !(f >= kMinDecay && f <= 1.0f / kMinDecay); }

// The exponent of a channel's s, from f_L.
__device__ __forceinline__ int scale_exp(float f) { return (3 * (127 - (int)((__float_as_uint(f) >> 23) & 255u))) >> 3; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // -127 < e < 128

template <typename TI> struct Two;                                 // two neighbouring channels of a token
template <> struct Two<float> { typedef u32x2 T; };
template <> struct Two<uint16_t> { typedef uint32_t T; };
__device__ __forceinline__ f32x2 two(u32x2 x) { return f32x2{__uint_as_float(x[0]), __uint_as_float(x[1])}; }
__device__ __forceinline__ f32x2 two(uint32_t x) { return f32x2{lo_f32(x), hi_f32(x)}; }
__device__ __forceinline__ u32x2 row_ld2(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}

template <int D, bool KDA>
struct GF32 {
    static constexpr int NW = D / 16, NT = 64 * NW;
    static constexpr int RT = D / 16, QP = D / 8;
    static constexpr int ROWS = pm_shorts<GF>(QP);  // shorts of one part of 32 rows
};

template <int D, bool KDA, typename TI, bool OUT>
__global__ __launch_bounds__((GF32<D, KDA>::NT), 4) void gdn_chunk32_kernel(GdnSegArgs a) {
    using P = GF32<D, KDA>;
    constexpr int NW = P::NW, NT = P::NT, RT = P::RT, QP = P::QP, ROWS = P::ROWS;
    constexpr int LA = 20, ES = sizeof(TI);
    __shared__ __align__(16) uint16_t sK[3][ROWS];                 // K (per key: f o K) in parts
    __shared__ __align__(16) uint16_t sY[3][KDA ? ROWS : 8];       // per key: K / f in parts
    __shared__ __align__(16) uint16_t sQ[3 * (OUT ? ROWS : 8)];    // Q (per key: f o Q), then P, in parts
    __shared__ __align__(16) uint16_t sA[3][kBlk];                 // -A left of the second diagonal block, in parts
    __shared__ __align__(16) float sD[2][16 * LA];                 // inverses of the diagonal blocks of I + A
    __shared__ std::conditional_t<KDA, GdnSteps<GF>, GdnGates<GF>> s_gate[KDA ? 1 : 2];   // of this chunk (and the next)
    __shared__ __align__(16) float s_first[KDA ? D : 4], s_last[KDA ? D : 4];   // per key: the first token's decay / s, f_L s
    __shared__ int s_cut[2];

    const int t = threadIdx.x, lane = t & 63;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg;
    const int te = min(len, t0 + a.seg);
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);
    const bool map = !OUT && blockIdx.z;
    if (blockIdx.y ? past_end<OUT>(t0, len) : map) return;
    const float* start = blockIdx.y == 0 ? a.first : a.start;

    v4f H[RT];                                                     // H[rt][v] = H[16 rt + 4 lg + v][16 w + li]
    if (!map && start && blockIdx.y > 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) H[rt] = *state_at(const_cast<float*>(start) + soff, D / 16, rt, w, lane);
    } else if (!map && start) {
        const float* from = start + head * (size_t)(D * D) + (size_t)(4 * (lane >> 4)) * D + 16 * w + (lane & 15);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) H[rt][v] = from[(size_t)(16 * rt + v) * D];
    } else {
        const int diag = map ? 16 * w + (lane & 15) - 4 * (lane >> 4) : -(1 << 20);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) H[rt][v] = 16 * rt + v == diag ? 1.0f : 0.0f;
    }
    if (!OUT && a.keep && !map && blockIdx.y == 0) {
        float* to = a.keep + head * (size_t)(D * D) + (size_t)(4 * (lane >> 4)) * D + 16 * w + (lane & 15);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) to[(size_t)(16 * rt + v) * D] = H[rt][v];
    }
    // columns of A's block that belong to the diagonal block: zeros, never written again
    for (int e = t; e < 3 * 16 * 16; e += NT) sA[e >> 8][blk((e >> 4) & 15, 16 + (e & 15))] = 0;

    // chunk loads in registers, one chunk ahead; tokens past `end` read as zeros.  Thread: two channels
    // of four tokens; the values' columns as accumulators hold them
    constexpr int PR = D / 2;                                      // channel pairs
    static_assert(NT == 8 * PR, "four tokens per thread");
    const uint32_t rb = (uint32_t)heads * (ES * D);                // bytes between tokens (heads <= chunk_heads(D))
    typename Two<TI>::T kd[4], qd[4];
    f32x2 ad[KDA ? 4 : 1];
    uint32_t vd[ES == 4 ? 8 : 4];                                  // bf16: lanes in pairs, two columns of every second row
    auto rows = [&](const void* x, int c0, int end, uint32_t es) { // tokens c0 .. min(c0 + GF, end) - 1 of this head
        return make_rows(static_cast<const char*>(x) + ((size_t)c0 * heads + head) * (es * D),
                         end > c0 ? (uint32_t)(min(end - c0, GF) - 1) * (uint32_t)heads * (es * D) + es * D : 0);
    };
    auto load = [&](int c0, int end) {
        const uint32_t tt = fresh(t), pair = tt % PR, n0 = 4 * (tt / PR), off = n0 * rb + 2 * ES * pair;
        const rsrc_t rk = rows(a.k, c0, end, ES), rv = rows(a.v, c0, end, ES), rq = rows(OUT ? a.q : a.k, c0, end, ES);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (ES == 4) {
                kd[e] = row_ld2(rk, off + e * rb);
                if constexpr (OUT) qd[e] = row_ld2(rq, off + e * rb);
            } else {
                kd[e] = row_ld(rk, off + e * rb);
                if constexpr (OUT) qd[e] = row_ld(rq, off + e * rb);
            }
        }
        if constexpr (KDA) {
            const rsrc_t ra = rows(a.alpha, c0, end, 4);
            const uint32_t rba = (uint32_t)heads * (4 * D);
#pragma unroll
            for (int e = 0; e < 4; ++e) ad[e] = __builtin_bit_cast(f32x2, row_ld2(ra, (n0 + e) * rba + 8 * pair));
        }
        const uint32_t ln = tt & 63;
        const uint32_t voff = ES == 4 ? 4 * (ln >> 4) * rb + 4 * (16 * w + (ln & 15))
                                      : (4 * (ln >> 4) + (ln & 1)) * rb + 2 * (16 * w + (ln & 14));
        constexpr int VR = ES == 4 ? 4 : 2;                        // loads per block of 16 tokens
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int v = 0; v < VR; ++v) vd[VR * r + v] = map ? 0u : row_ld(rv, voff + (16 * r + 4 / VR * v) * rb);
    };
    auto values = [&](int r, float (&x)[4]) {                      // as accumulators hold them: tokens 16 r + 4 lg + v
        if constexpr (ES == 4) {
#pragma unroll
            for (int v = 0; v < 4; ++v) x[v] = __uint_as_float(vd[4 * r + v]);
        } else {
            const bool up = lane & 1;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float l = lo_f32(vd[2 * r + j]), h = hi_f32(vd[2 * r + j]);
                const float other = dpp<DPP_XOR1>(up ? l : h);
                x[2 * j] = up ? other : l;
                x[2 * j + 1] = up ? h : other;
            }
        }
    };
    float al = 1.0f, be = 0.0f;                                    // gates of the next chunk: the last wave's
    auto load_gates = [&](int c0) {
        const size_t at = (size_t)min(c0 + (lane & (GF - 1)), te - 1) * heads + head;
        if constexpr (!KDA) al = a.alpha[at];
        be = a.beta[at];
    };
    if (t0 < te) {
        load(t0, te);
        if (w == NW - 1) {
            load_gates(t0);
            if constexpr (!KDA) make_gates<GF>(al, be, te - t0, lane, s_gate[0], &s_cut[0]);
        }
    }
    if (KDA && t == 0) s_cut[0] = s_cut[1] = GF;
    // registers -> LDS, in parts.  s_cut: the first token after the chunk's first one with a value that
    // is not finite, or past which a channel decays too far
    auto store = [&](int cur, int L) {
        const uint32_t tt = fresh(t), pair = tt % PR, quad = tt / PR, n0 = 4 * quad;
        const int c = 2 * pair, u = (c & 31) >> 2;                 // operand order of the channel's 32-block
        const int at = pm<GF>(n0, (c >> 5) * 4 + (u & 3)) + 4 * ((u >> 2) ^ (u & 1)) + (c & 3);   // (odd pieces: halves swapped)
        int first = GF;
        [[maybe_unused]] f32x2 f[4];
        if constexpr (KDA) {
            f32x2 run = {1.0f, 1.0f}, before = run, all = run, own = run;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool on = (int)n0 + e < L;
                const f32x2 x = {on ? ad[e][0] : 1.0f, on ? ad[e][1] : 1.0f};
                if (n0 + e > 0) run *= x;                          // (the first token's own decay is H's)
                else own = x;
                f[e] = run;
            }
            float* s_tot = reinterpret_cast<float*>(sY[0]);        // products of four tokens, in Y's place
            static_assert(sizeof(sY) >= 8 * D * sizeof(float) || !KDA, "a total per channel and four tokens");
            *reinterpret_cast<f32x2*>(&s_tot[quad * D + c]) = run;
            if (w == NW - 1 && lane < GF) {
                const float b = lane < L ? be : 0.0f;
                s_gate[0].b[lane] = b;
                if (lane > 0 && !finite_f32(b)) atomicMin(&s_cut[cur], lane);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i == (int)quad) before = all;
                all *= *reinterpret_cast<const f32x2*>(&s_tot[i * D + c]);
            }
            __syncthreads();                                       // the totals are read
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] *= before;
                if (n0 + e > 0 && (decays_far(f[e][0]) || decays_far(f[e][1]))) first = min(first, (int)n0 + e);
            }
            const int s0 = scale_exp(all[0]), s1 = scale_exp(all[1]);
            const f32x2 scale = {pow2(s0), pow2(s1)};
            if (quad == 0) {
                *reinterpret_cast<f32x2*>(&s_first[c]) = own * f32x2{pow2(-s0), pow2(-s1)};
                *reinterpret_cast<f32x2*>(&s_last[c]) = all * scale;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= scale;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x2 k = two(kd[e]), q = OUT ? two(qd[e]) : f32x2{0.f, 0.f};
            if (n0 + e > 0 && (!finite_f32(k[0]) || !finite_f32(k[1]))) first = min(first, (int)n0 + e);
            float x[6] = {k[0], k[1], q[0], q[1], 0.f, 0.f};
            if constexpr (KDA) {
                x[4] = __builtin_amdgcn_rcpf(f[e][0]) * k[0], x[5] = __builtin_amdgcn_rcpf(f[e][1]) * k[1];
                x[0] *= f[e][0], x[1] *= f[e][1], x[2] *= f[e][0], x[3] *= f[e][1];
            }
            uint32_t p[3][3];
            split3<6>(x, p);
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                *reinterpret_cast<uint32_t*>(&sK[m][at + 8 * e]) = p[m][0];
                if constexpr (OUT) *reinterpret_cast<uint32_t*>(&sQ[m * ROWS + at + 8 * e]) = p[m][1];
                if constexpr (KDA) *reinterpret_cast<uint32_t*>(&sY[m][at + 8 * e]) = p[m][2];
            }
        }
        if constexpr (ES == 4) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int n = 16 * r + 4 * ((int)(tt & 63) >> 4) + v;
                    if (n > 0 && !finite_f32(__uint_as_float(vd[4 * r + v]))) first = min(first, n);
                }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = 16 * r + 4 * ((int)(tt & 63) >> 4) + 2 * j + (int)(tt & 1);
                    if (n > 0 && odd_bf16(vd[2 * r + j])) first = min(first, n);
                }
        }
        if (first < GF) atomicMin(&s_cut[cur], first);
    };
    __syncthreads();                                               // the first gates (and s_cut) are written

    int cur = 0, next;
    for (int c0 = t0; c0 < te; c0 = next, cur ^= 1) {
        int ce = min(c0 + GF, te);
        if (!KDA && w == NW - 1) load_gates(ce);                   // (none left: the last token's again)
        store(cur, ce - c0);
        __syncthreads();
        const int cut = s_cut[cur];
        if (cut < ce - c0) {                                       // the chunk again, up to that token
            ce = c0 + cut;
            __syncthreads();
            load(c0, ce);
            if (w == NW - 1) {
                load_gates(c0);
                if constexpr (!KDA) {
                    int dummy;
                    make_gates<GF>(al, be, cut, lane, s_gate[cur], &dummy);
                    load_gates(ce);
                }
            }
            store(cur, cut);
            __syncthreads();
        }
        if (KDA && t == 0) s_cut[cur] = GF;                        // (read by all; for the chunk after the next)
        next = ce;
        const auto& G = s_gate[KDA ? 0 : cur];

        const int lo = fresh(lane), li = lo & 15, lg = lo >> 4;
        const int at = pm<GF>(li, lg);                             // operand reads: row li, piece lg
        if constexpr (KDA)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) H[rt] *= *reinterpret_cast<const v4f*>(&s_first[16 * rt + 4 * lg]);
        // ---- scores: the three tiles on and below the diagonal, of K K^T and of Q K^T, a wave each ----
        const uint16_t(*sC)[ROWS] = reinterpret_cast<const uint16_t(*)[ROWS]>(KDA ? &sY[0][0] : &sK[0][0]);
        auto scores = [&](const uint16_t* x, int r, int c) {
            v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                u32x4 y[3], z[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    y[m] = *reinterpret_cast<const u32x4*>(&x[m * ROWS + at + pm<GF>(16 * r, 4 * ks)]);
                    z[m] = *reinterpret_cast<const u32x4*>(&sC[m][at + pm<GF>(16 * c, 4 * ks)]);
                }
                acc = mfma_split(y, z, acc);
            }
            if constexpr (!KDA) {
                const double gi = G.g[16 * c + li];
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[v] *= __expf((float)(G.g[16 * r + 4 * lg + v] - gi));
            }
            return acc;
        };
        auto put = [&](uint16_t* p0, int part, int to, const v4f& x) {   // a tile in parts
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float p = x[v], p1 = p - top_f32(p);
                p0[to + 8 * v] = (uint16_t)(__float_as_uint(p) >> 16);
                p0[part + to + 8 * v] = (uint16_t)(__float_as_uint(p1) >> 16);
                p0[2 * part + to + 8 * v] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
            }
        };
        auto invert = [&](int r) {
            const v4f x = scores(sK[0], r, r);
            float* sd = sD[r];
#pragma unroll
            for (int v = 0; v < 4; ++v) sd[(4 * lg + v) * LA + li] = li < 4 * lg + v ? -G.b[16 * r + 4 * lg + v] * x[v] : 0.0f;
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
        };
        // tiles of P: (0, 0), (1, 0), (1, 1), by the last three waves (eight waves; of four: by waves 1 to 3)
        constexpr int PW = NW - 3;
        v4f pr = {0.f, 0.f, 0.f, 0.f};
        if (w < 2) invert(w);
        if (w == (NW == 8 ? 2 : 0)) {
            v4f y = scores(sK[0], 1, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) y[v] *= -G.b[16 + 4 * lg + v];
            put(sA[0], kBlk, blk(4 * lg, li), y);
        }
        if (OUT && w >= PW) {
            const int r = (w - PW + 1) >> 1, c = (w - PW) >> 1;
            pr = scores(sQ, r, c);
#pragma unroll
            for (int v = 0; v < 4; ++v) pr[v] = 16 * (r - c) + 4 * lg + v >= li ? pr[v] : 0.0f;
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- K H and Q H ----
        v4f R[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, O[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            float x[8];
            uint32_t p[3][4];
            u32x4 b[3];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = lg & 1 ? H[2 * ks + (e < 4)][e % 4] : H[2 * ks + e / 4][e % 4];
            split3<8>(x, p);
#pragma unroll
            for (int m = 0; m < 3; ++m) b[m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                u32x4 y[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) y[m] = *reinterpret_cast<const u32x4*>(&sK[m][at + pm<GF>(16 * r, 4 * ks)]);
                R[r] = mfma_split(y, b, R[r]);
                if constexpr (OUT) {
#pragma unroll
                    for (int m = 0; m < 3; ++m) y[m] = *reinterpret_cast<const u32x4*>(&sQ[m * ROWS + at + pm<GF>(16 * r, 4 * ks)]);
                    O[r] = mfma_split(y, b, O[r]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const v4f bt = *reinterpret_cast<const v4f*>(&G.b[16 * r + 4 * lg]);
            if constexpr (!KDA) {
                const v4f e = *reinterpret_cast<const v4f*>(&G.e[16 * r + 4 * lg]);
                R[r] *= e;
                O[r] *= e;
            }
            float x[4];
            values(r, x);
#pragma unroll
            for (int v = 0; v < 4; ++v) R[r][v] = bt[v] * (x[v] - R[r][v]);
        }
        if (w == NW - 1) {
            if constexpr (KDA) load_gates(ce);
            else make_gates<GF>(al, be, te - ce, lane, s_gate[cur ^ 1], &s_cut[cur ^ 1]);
        }
        __syncthreads();                                           // A is written, Q is read
        if (OUT && w >= PW) {                                      // P in parts, in Q's place; right of the diagonal zeros
            const int r = (w - PW + 1) >> 1, c = (w - PW) >> 1;
            put(sQ, 2 * kBlk, r * kBlk + 4 * c + blk(4 * lg, li), pr);
            if (w == PW) put(sQ, 2 * kBlk, 4 + blk(4 * lg, li), v4f{0.f, 0.f, 0.f, 0.f});
        }
        // ---- (I + A) M = R ----
        u32x4 mp[3];                                               // M in parts
        const int ab = blk(li, 4 * lg);                            // operand reads: row li, piece lg
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (r == 1) {
                u32x4 x[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sA[m][ab]);
                R[1] = mfma_split(x, mp, R[1]);
            }
            const v4f ti = *reinterpret_cast<const v4f*>(&sD[r][li * LA + 4 * lg]);
            v4f m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < 4; ++v) m = mfma4(ti[v], R[r][v], m);
            R[r] = m;
            const float y[4] = {m[0], m[1], m[2], m[3]};
            uint32_t p[3][2];
            split3<4>(y, p);
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                mp[u][2 * r] = p[u][0];
                mp[u][2 * r + 1] = p[u][1];
                if (r == 0) mp[u][2] = mp[u][3] = 0;
            }
        }
        if constexpr (OUT) {
            __syncthreads();                                       // P is written
            // ---- O += P M ----
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                u32x4 x[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) x[m] = *reinterpret_cast<const u32x4*>(&sQ[(2 * m + r) * kBlk + ab]);
                O[r] = mfma_split(x, mp, O[r]);
            }
            const rsrc_t ro = rows(a.o, c0, ce, ES);               // rows past the end are left as they were
            if constexpr (ES == 4) {
                const uint32_t ooff = 4 * lg * rb + 4 * (16 * w + li);
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int v = 0; v < 4; ++v) row_st(ro, ooff + (16 * r + v) * rb, __float_as_uint(O[r][v]));
            } else {
                // lanes in pairs: the even one stores both columns of the rows v, the odd one those of v + 1
                const bool up = li & 1;
                const uint32_t ooff = (4 * lg + (li & 1)) * rb + 2 * (16 * w + (li & 14));
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int v = 0; v < 4; v += 2) {
                        const float x = dpp<DPP_XOR1>(up ? O[r][v] : O[r][v + 1]);
                        row_st(ro, ooff + (16 * r + v) * rb, up ? pack_bf16(x, O[r][v + 1]) : pack_bf16(O[r][v], x));
                    }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        load(ce, te);                                              // (none left: zeros)
        __builtin_amdgcn_sched_barrier(0);
        // ---- H = e^{g_L} H + K^T (w o M); per key: f_L o (H + Y^T M) ----
        // transposed reads: 4 tokens of 16 channels a lane group, one half of each piece
        const int kt = pm<GF>(4 * lg + (li >> 2), li & 3), kh[2] = {kt + 4 * (li & 1), kt + 4 * (~li & 1)};
        if constexpr (!KDA) {
            const v4f w0 = *reinterpret_cast<const v4f*>(&G.w[4 * lg]), w1 = *reinterpret_cast<const v4f*>(&G.w[16 + 4 * lg]);
            float x[8];
            uint32_t p[3][4];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (e < 4 ? w0[e & 3] : w1[e & 3]) * R[e / 4][e % 4];
            split3<8>(x, p);
#pragma unroll
            for (int m = 0; m < 3; ++m) mp[m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
        }
        float egl = 1.0f;
        if constexpr (!KDA) egl = G.e[GF - 1];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            u32x4 y[3];
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                const uint16_t* from = &sC[m][kh[rt & 1] + pm<GF>(0, 4 * (rt >> 1))];
                const u32x2 k0 = lds_tr(from), k1 = lds_tr(from + pm<GF>(16, 0));
                y[m] = u32x4{k0[0], k0[1], k1[0], k1[1]};
            }
            if constexpr (!KDA) H[rt] *= egl;
            H[rt] = mfma_split(y, mp, H[rt]);
            if constexpr (KDA) H[rt] *= *reinterpret_cast<const v4f*>(&s_last[16 * rt + 4 * lg]);
            if (rt % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();                                           // LDS is rewritten by the next chunk
    }
    const int lf = fresh(lane);
    if (map) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            *map_at<D>(a.map + soff, 16 * rt + 4 * (lf >> 4) + (lf & 3), 16 * w + (lf & 12)) = quad_rows(H[rt], lf & 15);
        return;
    }
    if (a.end)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) *state_at(a.end + soff, D / 16, rt, w, lf) = H[rt];
    if (!a.fin || blockIdx.y < gridDim.y - 1) return;
    float* end = a.fin + head * (size_t)(D * D);
    end += (size_t)(4 * (lf >> 4)) * D + 16 * w + (lf & 15);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int v = 0; v < 4; ++v) end[(size_t)(16 * rt + v) * D] = H[rt][v];
}

// ---------------------------------------------------------------------------
// d = 16: chunks of 16 tokens, one wave a head and segment
// ---------------------------------------------------------------------------
// Every product is one 16 x 16 x 16 of the fp32 matrix instruction, each operand loaded in the
// layout that the instruction takes (lane (lg, li), step v: row or column li, index 4 lg + v).  The
// scores are formed transposed, so that their accumulators are the A operand of P M as they are;
// only A goes through LDS, for block_solve.  Per key: the same factors as the larger kernel's.
// Bound by a wave's chain of dependent products, two waves a SIMD (vector 0.53, matrix 0.25): 2048 heads of
// 512 tokens 106 us, per key 107 (142 if a channel takes 2^-8 a token, 273 at 2^-16, 1400 where one forgets every token).
// The value of the lane that far before in the row of 16, 1 where there is none.
template <int CTRL>
__device__ __forceinline__ float dpp_one(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(1.0f), __float_as_int(x), CTRL, 0xf, 0xf, false));
}

template <bool KDA, typename TI, bool OUT>
__global__ __launch_bounds__(256) void gdn_small_kernel(GdnSegArgs a) {
    constexpr int D = 16, CS = 16, LR = 20;
    __shared__ __align__(16) float s_a[4][CS * LR];
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4, wv = threadIdx.x >> 6;
    const size_t heads = (size_t)a.heads;
    const size_t head = (size_t)blockIdx.x * 4 + wv;               // one head a wave (waves share nothing)
    if (head >= heads) return;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg, te = min(len, t0 + a.seg);
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);
    const bool map = !OUT && blockIdx.z;
    if (blockIdx.y ? past_end<OUT>(t0, len) : map) return;
    const float* start = blockIdx.y == 0 ? a.first : a.start;
    v4f H = {0.f, 0.f, 0.f, 0.f};                                  // H[4 lg + v][li]
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (map) H[v] = 4 * lg + v == li ? 1.0f : 0.0f;
        else if (start) H[v] = start[(blockIdx.y == 0 ? head * (size_t)(D * D) : soff) + (4 * lg + v) * D + li];
    }
    if (!OUT && a.keep && !map && blockIdx.y == 0)
#pragma unroll
        for (int v = 0; v < 4; ++v) a.keep[head * (size_t)(D * D) + (4 * lg + v) * D + li] = H[v];
    // token li: q, k channels 4 lg + v; tokens 4 lg + v: k, v channel li
    struct Chunk {                                                 // (as loaded: widened on use)
        Row4<TI> q, k;
        Row4<float> ar;
        TI kt[4], vt[4];
        float at[4], al, be;
    };
    auto load = [&](int c0, Chunk& x) {                            // (past the end: the last token, zeroed on use)
        const size_t th = (size_t)min(c0 + li, te - 1) * heads + head;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const size_t to = ((size_t)min(c0 + 4 * lg + v, te - 1) * heads + head) * D + li;
            x.kt[v] = static_cast<const TI*>(a.k)[to];
            x.vt[v] = static_cast<const TI*>(a.v)[to];
            if constexpr (KDA) x.at[v] = a.alpha[to];
        }
        if (OUT) x.q.load(a.q, th * D + 4 * lg);
        x.k.load(a.k, th * D + 4 * lg);
        if constexpr (KDA) x.ar.load(a.alpha, th * D + 4 * lg);
        else x.al = a.alpha[th];
        x.be = a.beta[th];
    };
    auto fold = [](uint64_t m) { return (uint32_t)(m | m >> 16 | m >> 32 | m >> 48) & 0xffffu; };   // over the lane groups
    Chunk cur, nxt;
    if (t0 < te) load(t0, cur);
    for (int c0 = t0; c0 < te;) {
        int L = min(CS, te - c0);
        float kr[4], qr[4] = {0.f, 0.f, 0.f, 0.f}, kt[4], vt[4];
        cur.k.widen4(kr);
        if (OUT) cur.q.widen4(qr);
        // the chunk ends before a later token that is not finite
        const bool oddk = !finite_f32(kr[0]) || !finite_f32(kr[1]) || !finite_f32(kr[2]) || !finite_f32(kr[3]) || !finite_f32(cur.be);
        uint32_t cut = fold(__ballot(oddk));
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            kt[v] = widen(cur.kt[v]);
            vt[v] = map ? 0.0f : widen(cur.vt[v]);
            uint64_t m = __ballot(!finite_f32(vt[v]));             // lane group lg: token 4 lg + v
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((m >> (16 * i)) & 0xffffu) cut |= 1u << (4 * i + v);
        }
        // decays: scalar g of token li, gi of tokens 4 lg + v; per key the products fr of token li, channels
        // 4 lg + v, and fc of tokens 4 lg + v, channel li, after the first token
        double g = 0.0, gl = 0.0, gi[4];
        float fr[4], fc[4], e0[4], el[4];                          // per key: the first decay and f_L of channels 4 lg + v
        if constexpr (!KDA) {
            const float la = log_decay(cur.al);
            cut |= fold(__ballot(!finite_f32(la)));
            cut &= ~1u;
            if (cut) L = min(L, __ffs(cut) - 1);
            g = li < L ? (double)la : 0.0;
            g = scan_step<0x111, 0xf>(g);
            g = scan_step<0x112, 0xf>(g);
            g = scan_step<0x114, 0xf>(g);
            g = scan_step<0x118, 0xf>(g);
            gl = __shfl(g, 15, 16);
#pragma unroll
            for (int v = 0; v < 4; ++v) gi[v] = __shfl(g, 4 * lg + v, 16);
        } else {
            float ar[4];
            cur.ar.widen4(ar);
            cut &= ~1u;
            if (cut) L = min(L, __ffs(cut) - 1);
            bool far = false;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float x = li > 0 && li < L ? ar[v] : 1.0f;
                x *= dpp_one<0x111>(x);
                x *= dpp_one<0x112>(x);
                x *= dpp_one<0x114>(x);
                fr[v] = x * dpp_one<0x118>(x);
                far |= decays_far(fr[v]);
            }
            cut = fold(__ballot(far)) & ~1u;
            if (cut) L = min(L, __ffs(cut) - 1);                   // (products before it stand)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                e0[v] = __shfl(ar[v], 0, 16);
                el[v] = __shfl(fr[v], L - 1, 16);
            }
            float run = 1.0f;                                      // this lane's four tokens, then those of the groups before
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int n = 4 * lg + v;
                run *= n > 0 && n < L ? cur.at[v] : 1.0f;
                fc[v] = run;
            }
            const float s0 = __shfl(run, li, 64), s1 = __shfl(run, 16 + li, 64), s2 = __shfl(run, 32 + li, 64);
            float before = lg == 0 ? 1.0f : lg == 1 ? s0 : lg == 2 ? s0 * s1 : s0 * s1 * s2;
            // the powers of two s only where they are needed (for every chunk: 110 us, not 106)
            if (__any(min(min(el[0], el[1]), min(el[2], el[3])) < 0x1p-56f)) {
                uint32_t exps = 0;                                 // channels 4 lg + v: a byte each
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int x = scale_exp(el[v]);
                    exps |= (uint32_t)(x & 255) << (8 * v);
                    fr[v] *= pow2(x);
                    e0[v] *= pow2(-x);
                    el[v] *= pow2(x);
                }
                before *= pow2((int8_t)(__shfl((int)exps, 4 * (li & 12), 64) >> (8 * (li & 3))));
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) fc[v] *= before;
        }
        const int next = c0 + L;
        if (next < te) load(next, nxt);
        const float beta = li < L ? cur.be : 0.0f;
        // rows x (of K and Q) and y, token li; y of tokens 4 lg + v
        float xk[4], xq[4], yr[4], yc[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const bool on = 4 * lg + v < L;
            const float k0 = li < L ? kr[v] : 0.0f, q0 = li < L ? qr[v] : 0.0f;
            vt[v] = on ? vt[v] : 0.0f;
            kt[v] = on ? kt[v] : 0.0f;
            if constexpr (KDA) {
                xk[v] = li < L ? fr[v] * k0 : 0.0f;
                xq[v] = li < L ? fr[v] * q0 : 0.0f;
                yr[v] = li < L ? __builtin_amdgcn_rcpf(fr[v]) * k0 : 0.0f;
                yc[v] = on ? __builtin_amdgcn_rcpf(fc[v]) * kt[v] : 0.0f;
                H[v] *= e0[v];
            } else {
                xk[v] = k0, xq[v] = q0, yr[v] = k0;
                yc[v] = on ? __expf((float)(gl - gi[v])) * kt[v] : 0.0f;
            }
        }
        // transposed scores: [i = 4 lg + v][n = li]
        v4f p = {0.f, 0.f, 0.f, 0.f}, s = p;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            s = mfma4(yr[v], xk[v], s);
            if (OUT) p = mfma4(yr[v], xq[v], p);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = 4 * lg + v;
            const float e = KDA ? 1.0f : __expf((float)(g - gi[v]));
            s[v] = i < li ? -beta * (e * s[v]) : 0.0f;
            p[v] = i <= li ? e * p[v] : 0.0f;
        }
        float* sa = s_a[wv];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        *reinterpret_cast<v4f*>(&sa[li * LR + 4 * lg]) = s;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        v4f own[3], R[1], O = {0.f, 0.f, 0.f, 0.f}, kh = O;
        float below[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) own[i] = *reinterpret_cast<const v4f*>(&sa[(4 * lg + 1 + i) * LR + 4 * lg]);
#pragma unroll
        for (int i = 0; i < 3; ++i) below[i] = (li >> 2) > i ? sa[li * LR + 4 * i + lg] : 0.0f;
        const float en = KDA ? 1.0f : __expf((float)g);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            kh = mfma4(en * xk[v], H[v], kh);
            if (OUT) O = mfma4(en * xq[v], H[v], O);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) R[0][v] = __shfl(beta, 4 * lg + v, 16) * (vt[v] - kh[v]);
        block_solve<1>(own, below, lg, R);
        if constexpr (OUT) {
#pragma unroll
            for (int v = 0; v < 4; ++v) O = mfma4(p[v], R[0][v], O);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (4 * lg + v < L) tok_st<TI>(a.o, ((size_t)(c0 + 4 * lg + v) * heads + head) * D + li, O[v]);
        }
        if (!KDA) H *= __expf((float)gl);
#pragma unroll
        for (int v = 0; v < 4; ++v) H = mfma4(yc[v], R[0][v], H);
        if constexpr (KDA)
#pragma unroll
            for (int v = 0; v < 4; ++v) H[v] *= el[v];
        cur = nxt;
        c0 = next;
    }
    float* end = map ? a.map + soff : a.end ? a.end + soff : nullptr;
    if (!map && a.fin && blockIdx.y == gridDim.y - 1) end = a.fin + head * (size_t)(D * D);
    if (end)
#pragma unroll
        for (int v = 0; v < 4; ++v) end[(4 * lg + v) * D + li] = H[v];
}

// ---------------------------------------------------------------------------
// few heads: segments of a prompt at once
// ---------------------------------------------------------------------------
// A segment is a linear map of the state before it: X' = G X + E, E the state that it leaves from
// zeros, G the one that it leaves from the identity with every v = 0.  One launch computes E and
// G of all segments, the scan joins them (X_{s+1} = G_s X_s + E_s, in E's place), and the last one
// computes every segment's outputs from the state before it.  A workgroup of the scan owns 16
// columns of a head's state, wave w its rows 16 w ..; both factors in three bf16 parts: G's rows are
// split from registers, loaded four steps ahead, X's columns go through LDS.  A step takes 1.5 us whatever the heads:
// every workgroup of a head splits the same G, so that the two waves a SIMD fill 0.59 of the vector port, and the chain of
// barrier, LDS and twelve products waits for 0.28 of it.  16 heads at d = 128: 8 segments 12 us, 16 segments 24.
struct GdnScanArgs {
    float* x;                 // [segments][heads][d*d]: E_s at s + 1, then the states before the segments
    const float* map;         // G_s at s
    float* fin;               // state after the last segment, or null: formed with the outputs
    const int32_t* lens;      // per batch row, or null: T
    size_t stride;            // floats between segments
    int T, H, seg;
    int n;                    // states to form: x[2] .. x[n]

    // The last state that tokens change: it stays for the segments after it (a product with the identity would
    // lose infinities, NaN and the sign of zeros).
    __device__ __forceinline__ int last(size_t head) const {
        const int len = lens ? min(max(lens[head / (unsigned)H], 0), T) : T;
        return min(n, max(1, (len + seg - 1) / seg));
    }
};
constexpr int kScanAhead = 4;
template <int D, int CT>                                           // CT: neighbouring columns in a lane's tiles
__global__ __launch_bounds__(4 * D) void gdn_scan_kernel(GdnScanArgs a) {
    constexpr int KS = D / 32;
    __shared__ __align__(16) uint16_t s_x[2][3][pm_shorts<16>(D / 8)];   // [column][channel], in parts
    const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t at = blockIdx.x * (size_t)(D * D);
    // G: row 16 w + li, channels 16 c + 4 lg + e; X: rows 16 w + 4 lg + v of the tile's column li
    const float* g0 = a.map + at + (size_t)w * (16 * D) + 4 * lane;
    float* x0 = reinterpret_cast<float*>(state_at(a.x + at, D / 16, w, blockIdx.y, lane));
    const int last = a.last(blockIdx.x);
    struct Step {
        v4f g[KS][2], e;
    };
    auto load = [&](int s, Step& y) {                              // kScanAhead steps before their use
        if (s > last) return;
        const float* g = g0 + (s - 1) * a.stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            y.g[ks][0] = *reinterpret_cast<const v4f*>(g + 512 * ks);
            y.g[ks][1] = *reinterpret_cast<const v4f*>(g + 512 * ks + 256);
        }
        y.e = *reinterpret_cast<const v4f*>(x0 + s * a.stride);
    };
    v4f x;
    auto step = [&](int s, Step& y) {
        const float z[4] = {x[0], x[1], x[2], x[3]};
        uint32_t p[3][2];
        split3<4>(z, p);
#pragma unroll
        for (int m = 0; m < 3; ++m) *reinterpret_cast<u32x2*>(&s_x[s & 1][m][pm<16>(li, 4 * (w >> 1) + lg) + 4 * (w & 1)]) = u32x2{p[m][0], p[m][1]};
        u32x4 g[KS][3];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const float f[8] = {y.g[ks][0][0], y.g[ks][0][1], y.g[ks][0][2], y.g[ks][0][3],
                                y.g[ks][1][0], y.g[ks][1][1], y.g[ks][1][2], y.g[ks][1][3]};
            uint32_t q[3][4];
            split3<8>(f, q);
#pragma unroll
            for (int m = 0; m < 3; ++m) g[ks][m] = u32x4{q[m][0], q[m][1], q[m][2], q[m][3]};
        }
        lds_barrier();                                             // (loads stay in flight; the other half is written meanwhile)
        v4f u[2] = {y.e, {0.f, 0.f, 0.f, 0.f}};                    // two chains
        load(s + kScanAhead, y);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            u32x4 b[3];
#pragma unroll
            for (int m = 0; m < 3; ++m) b[m] = *reinterpret_cast<const u32x4*>(&s_x[s & 1][m][pm<16>(li, 4 * ks + lg)]);
            u[ks & 1] = mfma_split(g[ks], b, u[ks & 1]);
        }
        x = u[0] + u[1];
        *reinterpret_cast<v4f*>(x0 + s * a.stride) = x;
    };
    Step y[kScanAhead];
    x = *reinterpret_cast<const v4f*>(x0 + a.stride);
#pragma unroll
    for (int i = 0; i < kScanAhead; ++i) load(2 + i, y[i]);
    for (int s = 2; s <= last; s += kScanAhead)
#pragma unroll
        for (int i = 0; i < kScanAhead; ++i)
            if (s + i <= last) step(s + i, y[i]);
    if (last < a.n) *reinterpret_cast<v4f*>(x0 + a.n * a.stride) = x;
    if (a.fin)
#pragma unroll
        for (int v = 0; v < 4; ++v) a.fin[at + (size_t)(16 * w + 4 * lg + v) * D + CT * (16 * (blockIdx.y / CT) + li) + blockIdx.y % CT] = x[v];
}

// d = 16: one wave a head.
__global__ __launch_bounds__(256) void gdn_scan16_kernel(GdnScanArgs a, int heads) {
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    const int head = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (head >= heads) return;
    float* x0 = a.x + (size_t)head * 256 + 64 * lg + li;           // X: rows 4 lg + v of column li
    const float* g0 = a.map + (size_t)head * 256 + 16 * li + 4 * lg;   // G: row li, channels 4 lg + v
    v4f x;
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = x0[a.stride + 16 * v];
    const int last = a.last(head);
    for (int s = 2; s <= last; ++s) {
        const v4f g = *reinterpret_cast<const v4f*>(g0 + (s - 1) * a.stride);
        v4f u;
#pragma unroll
        for (int v = 0; v < 4; ++v) u[v] = x0[s * a.stride + 16 * v];
#pragma unroll
        for (int v = 0; v < 4; ++v) u = mfma4(g[v], x[v], u);
        x = u;
#pragma unroll
        for (int v = 0; v < 4; ++v) x0[s * a.stride + 16 * v] = x[v];
    }
    if (last < a.n)
#pragma unroll
        for (int v = 0; v < 4; ++v) x0[a.n * a.stride + 16 * v] = x[v];
    if (a.fin)
#pragma unroll
        for (int v = 0; v < 4; ++v) a.fin[(size_t)head * 256 + (4 * lg + v) * 16 + li] = x[v];
}

// Heads that the chunk kernels take: at d >= 64 a chunk's rows lie within 32-bit byte offsets (d = 16:
// 64-bit ones).  More heads take the recurrence itself.
constexpr size_t chunk_heads(int d) { return d == 16 ? (size_t)INT32_MAX : (size_t)(1 << 24) / d; }
// Tokens per segment, a multiple of 64.  Segments cost the prompt a second time (twice: states and
// maps) and the scan, so they pay where the heads alone leave most CUs idle: up to `heads` heads,
// enough segments for `want` workgroups (d = 16: waves).  Measured, bf16, replayed in a graph:
//   d = 128: 16 heads, 16384 tokens 2429 us whole, 534, 340, 378 and 328-337 for 128, 256, 384 and 512
//   workgroups (fp32: 3235; 741, 486, 559, 501; per key 4232; 1052, 544, 703, 585); 2048 tokens: 32 heads
//   302; 142, 103, 115, 110; 64 heads 310; 266, 175, 201, 183; 128 heads 312 whole, 272 for 256, 296
//   for 512; 64 heads, 512 tokens 79; 72, 62, 61, 79; 300 tokens 51; 55, 49, 52, 52; 128 heads, 130
//   tokens 34, 41 for 256;
//   d = 64: 16 heads, 16384 tokens 1528 whole, 199, 170, 180 and 185 for 256, 512, 768 and 1024; 64 heads,
//   2048 tokens 189; 101, 81, 84, 88; 256 heads, 1024 tokens 110; 108, 108, 115, 126;
//   d = 16: 16 heads, 16384 tokens 2014 whole, 133, 99, 111 and 142 for 512, 1024, 2048 and 4096;
//   64 heads, 4096 tokens 515, 125, 79, 71, 77; 512 heads, 2048 tokens (fp32, per key) 332, 332, 315,
//   266, 264; 1024 heads, 1024 tokens 156, 156, 155, 164, 157.
struct GdnSplit {
    size_t heads, want;
};
constexpr GdnSplit kGdnSplit128{128, 256}, kGdnSplit64{256, 512}, kGdnSplit16{512, 2048};
constexpr int kGdnWhole = 192;
size_t segments_wanted(const lq_dims& d, int T) {
    const size_t heads = (size_t)d.B * d.H;
    const GdnSplit x = d.dk == 16 ? kGdnSplit16 : d.dk == 64 ? kGdnSplit64 : kGdnSplit128;
    return T <= kGdnWhole || heads > x.heads ? 1 : x.want / heads;
}
int segment_tokens(const lq_dims& d, int T) {
    const size_t chunks = ((size_t)T + 63) / 64, want = segments_wanted(d, T);
    return (int)((chunks + want - 1) / want * 64);
}

template <int D, bool KDA, typename TI, bool OUT>
hipError_t chunk_launch(dim3 grid, const GdnSegArgs& sa, hipStream_t s) {
    if constexpr (D == 16)
        return launch_kernel(LQ_KERNEL_PREFILL, gdn_small_kernel<KDA, TI, OUT>, dim3((grid.x + 3) / 4, grid.y, grid.z), dim3(256), s, sa);
    else if constexpr (!KDA && sizeof(TI) == 2)
        return launch_kernel(LQ_KERNEL_PREFILL, gdn_chunk_kernel<D, OUT>, grid, dim3(GB<D>::NT), s, sa);
    else
        return launch_kernel(LQ_KERNEL_PREFILL, gdn_chunk32_kernel<D, KDA, TI, OUT>, grid, dim3(GF32<D, KDA>::NT), s, sa);
}

template <int D, bool KDA, typename TI>
hipError_t gdn_chunks(const lq_dims& d, const GdnPrefillArgs& args, void* workspace, hipStream_t s) {
    const size_t heads = (size_t)args.heads;
    const int seg = segment_tokens(d, args.T), segs = (int)(((size_t)args.T + seg - 1) / seg);
    GdnSegArgs sa{args.h0, nullptr, nullptr, nullptr, args.h, nullptr, args.q, args.k, args.v, args.alpha, args.beta,
                  args.lens, args.o, 0, args.T, args.H, args.heads, seg};
    if (segs == 1) {
        const dim3 grid((unsigned)heads);
        return args.o ? chunk_launch<D, KDA, TI, true>(grid, sa, s) : chunk_launch<D, KDA, TI, false>(grid, sa, s);
    }
    // x[s]: the state before segment s (x[0]: of h0, where h is written over it), maps behind them
    float* x = static_cast<float*>(workspace);
    const size_t stride = heads * D * D;
    const int n = args.o ? segs - 1 : segs;                        // states that the first pass and the scan form
    float* map = x + (size_t)(segs + 1) * stride;
    sa.seg_stride = stride;
    sa.start = nullptr;
    sa.end = x + stride;
    sa.map = map;
    sa.fin = nullptr;
    if (args.o && args.h0 == args.h) sa.keep = x;
    hipError_t e = chunk_launch<D, KDA, TI, false>(dim3((unsigned)heads, (unsigned)n, n > 1 ? 2 : 1), sa, s);
    if (e != hipSuccess) return e;
    if (n > 1 || !args.o) {
        const GdnScanArgs sc{x, map, args.o ? nullptr : args.h, args.lens, stride, args.T, args.H, seg, n};
        if constexpr (D == 16)
            e = launch_kernel(LQ_KERNEL_PREFILL, gdn_scan16_kernel, dim3((unsigned)(heads + 3) / 4), dim3(256), s, sc, (int)heads);
        else
            e = launch_kernel(LQ_KERNEL_PREFILL, gdn_scan_kernel<D, !KDA && sizeof(TI) == 2 ? D / 64 : 1>, dim3((unsigned)heads, D / 16), dim3(4 * D), s, sc);
        if (e != hipSuccess || !args.o) return e;
    }
    if (sa.keep) sa.first = x;
    sa.start = x;
    sa.end = sa.map = sa.keep = nullptr;
    sa.fin = args.h;
    return chunk_launch<D, KDA, TI, true>(dim3((unsigned)heads, (unsigned)segs), sa, s);
}

template <int D, bool KDA, typename TI>
hipError_t gdn_prefill_t(const lq_dims& d, const GdnPrefillArgs& args, void* workspace, hipStream_t s) {
    if (args.T > kGdnStepTokens && (size_t)args.heads <= chunk_heads(D)) return gdn_chunks<D, KDA, TI>(d, args, workspace, s);
    return launch_kernel(LQ_KERNEL_PREFILL, gdn_step_kernel<D, KDA, TI>, dim3((unsigned)args.heads), dim3(D >= 64 ? 256 : 64), s, args);
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

size_t gdn_workspace_bytes(const lq_dims& d, int T) {
    const size_t heads = (size_t)d.B * d.H;
    if (T <= kGdnStepTokens || heads > chunk_heads(d.dk)) return 0;
    // segment_tokens gives at most min(want, chunks of 64) segments; that bound grows with T
    const size_t segs = std::min(segments_wanted(d, T), ((size_t)T + 63) / 64);
    return segs <= 1 ? 0 : (2 * segs + 1) * heads * d.dk * d.dv * sizeof(float);
}

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

// la_prefill.hip -- linear attention with a decay for each head over a prompt (gfx950).
//
//     H <- alpha H + k v^T,   o = H^T q  (after the update).
// Chunk form: for L tokens from state H0, with log-decay prefix sums g_n of the
// chunk's log alpha and E_{n,i} = exp(g_n - g_i) for i <= n, 0 otherwise,
//     o_n = e^{g_n} H0^T q_n + sum_i E_{n,i} <q_n, k_i> v_i,
//     H   = e^{g_L} H0 + sum_i e^{g_L - g_i} k_i v_i^T.
// Every exponent is <= 0, so no factor overflows however strong the decay.
// The prefix sums are kept in 64 bits: tokens after a strong decay (or a
// forget) still see differences g_n - g_i exact to fp32.
//
// Four kernels: chunks of 64 bf16 tokens, chunks of 32 fp32 tokens (d = 64, 128), chunks of
// 16 tokens (d = 16), and the recurrence itself for a few tokens.  In the first two a
// workgroup owns a head's state in matrix-instruction accumulators (tile (rt, ct): rows
// 16 rt + 4 (lane / 16) + v, column lane % 16) from the first load to the final store; the
// accumulator layout is the B operand of the next products with the K index in register
// order, so no value of H or V moves between lanes.  Where the heads alone leave most of
// the GPU idle, a prompt is cut into segments: their states alone, a scan over the
// segments, then their outputs from the states before them.
#include "la.h"
#include "lq_split.h"

namespace lq {
namespace {

struct LaPrefillArgs {
    const float* h0;          // or null: zeros
    float* h;
    const void* q;            // q, k, v, o: fp32 or bf16 (the kernel's TI)
    const void* k;
    const void* v;
    const float* alpha;
    const int32_t* lens;      // per batch row, or null: T
    void* o;                  // or null
    int T;
    int H;
    int heads;                // B*H: stride between tokens, in heads
    int alpha_tok;            // token stride of alpha: heads, or 0 for one decay per head
};

// ---------------------------------------------------------------------------
// bf16 tokens, d >= 64: chunks of 64 tokens on bf16 matrix products
// ---------------------------------------------------------------------------
// q, k and v enter the products as they are.  Every other operand is an fp32
// value split into three bf16 parts (all its 24 bits), whose products with a bf16
// token are exact and accumulate in fp32:
//   state update   K^T (w o V), w_t = e^{g_L - g_t}: w v in parts;
//   outputs        Q H with H in parts and (E o Q K^T) V with the scores in parts.
// (H and the scores in two parts, 16 bits: 302 us, not 331, for 2048 heads of 512 tokens,
// and 124, not 132, for 16 heads of 16384; but 0.6% of the outputs, not 0.02%, then round to
// a neighbour of the value that fp32 sums round to.)
// The wave's D/NW = 32 columns are 2 column tiles; tile ct holds the columns
// 2 li + ct, so a lane's two columns are one dword of a token row: V is loaded
// straight into operand order (lane group lg: tokens 8 lg .. 8 lg + 7 of 32),
// and outputs and the state leave as whole dwords and 8-byte pairs.
// H tiles are the B operand of Q H with the channels of each 32-block in the
// order (4 lg + e, 16 + 4 lg + e); Q and K rows are stored in that order.
// 64 tokens: a chunk's fixed work (the splits of H, three barriers) is shared by as many
// tokens as the LDS of two workgroups a CU holds.  Measured at d = 128: 2048 heads, 512
// tokens 331 us (3.7 TB/s; vector unit busy for 0.62 of the time, matrix unit for 0.43); 16
// heads, 16384 tokens 132 us, of it 43 for the segments' states (0.54, 0.36) and about 80 for the
// outputs (0.60, 0.41).
constexpr int BL = 64;        // tokens per chunk

struct LaSegArgs {
    const float* start;       // states before each segment, or null: zeros
    float* end;               // states after each segment, or null: not needed
    float* decay;             // e^{g} over each segment, or null
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const int32_t* lens;
    void* o;
    size_t seg_stride;        // floats between the states of consecutive segments
    int T, H, heads, alpha_tok;
    int seg;                  // tokens per segment (a multiple of BL)
};

template <int D>
struct LB {
    static constexpr int NW = D / 32, NT = 64 * NW;
    static constexpr int RT = D / 16;
    static constexpr int QP = D / 8, TP = BL / 8;   // pieces per Q / K row, per K^T / score row
};

// Gates of a chunk: prefix sums of log alpha, e^{g_n}, e^{g_L - g_n}.
template <int L>
struct Gates {
    double g[L];
    __align__(16) float e[L], w[L];
};
// Formed by one wave, lane n = token n; tokens from `left` on decay nothing.  Returns g_L.
template <int L>
__device__ __forceinline__ double make_gates(float alpha, int left, int lane, Gates<L>& s) {
    const double g = wave_scan(lane < min(left, L) ? (double)log_decay(alpha) : 0.0);
    const double gl = __shfl(g, 63, 64);
    if (lane < L) {
        s.g[lane] = g;
        s.e[lane] = expf((float)g);
        s.w[lane] = expf((float)(gl - g));
    }
    return gl;
}

template <int D, bool OUT>
__global__ __launch_bounds__(LB<D>::NT, 2) void la_chunk_kernel(LaSegArgs a) {
    using P = LB<D>;
    constexpr int NW = P::NW, NT = P::NT, RT = P::RT, QP = P::QP, TP = P::TP;
    __shared__ __align__(16) uint16_t sQ[OUT ? pm_shorts<BL>(QP) : 8];
    __shared__ __align__(16) uint16_t sK[OUT ? pm_shorts<BL>(QP) : 8];
    __shared__ __align__(16) uint16_t sT[pm_shorts<D>(TP)];        // K^T: [channel][token]
    __shared__ __align__(16) uint16_t sP[3][OUT ? pm_shorts<BL>(TP) : 8];   // scores in parts
    __shared__ Gates<BL> s_gate[2];                                // of this chunk and the next

    const int t = threadIdx.x, lane = t & 63;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg;                        // < T: one segment per started seg tokens
    const int te = min(len, t0 + a.seg);
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);

    // H[rt][ct][v] = H[16 rt + 4 lg + v][32 w + 2 li + ct]
    v4f H[RT][2];
    if (a.start) {
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
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) H[rt][0] = H[rt][1] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (OUT) {
        // score tiles right of the diagonal inside a 32-token step: zeros, never written again
        for (int e = t; e < 3 * 2 * 16 * 8; e += NT) {
            const int part = e >> 8, blk = (e >> 7) & 1, row = (e >> 3) & 15, c = e & 7;
            *reinterpret_cast<uint32_t*>(&sP[part][pm<BL>(32 * blk + row, 4 * blk + 2 + (c >> 2)) + 2 * (c & 3)]) = 0;
        }
    }

    // chunk loads in registers, one chunk ahead; tokens past the end read as zeros
    // (each phase of the chunk loop forms its lane indices anew: addresses kept across the
    // phases would spill, and a reload waits for the loads in flight)
    constexpr int OPW = 128 / D;                                   // octets per wave and pass (D = 64: 2)
    const uint32_t rb = (uint32_t)heads * (2 * D);                 // bytes between tokens (heads <= chunk_heads(D))
    uint32_t kd[2][8], vd[2][8];
    u32x4 qd[4];
    auto rows = [&](const void* x, int c0) {                       // tokens c0 .. min(c0 + BL, te) - 1 of this head
        return make_rows(static_cast<const char*>(x) + ((size_t)c0 * heads + head) * (2 * D),
                         (uint32_t)(min(te - c0, BL) - 1) * rb + 2 * D);
    };
    auto load_v = [&](int c0) {
        const rsrc_t rv = rows(a.v, c0);
        const uint32_t ln = fresh(lane), voff = 8 * (ln >> 4) * rb + 4 * (16 * w + (ln & 15));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) vd[j][e] = row_ld(rv, voff + (32 * j + e) * rb);
    };
    auto load_kq = [&](int c0) {
        const rsrc_t rk = rows(a.k, c0);
        const uint32_t ln = fresh(lane), koff = 8 * (2 * w * OPW + ln / (D / 2)) * rb + 4 * (ln % (D / 2));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) kd[j][e] = row_ld(rk, koff + (8 * j * OPW + e) * rb);
        if constexpr (OUT) {
            const rsrc_t rq = rows(a.q, c0);
            const uint32_t tt = 64 * w + ln, qoff = (tt / (D / 8)) * rb + 16 * (tt % (D / 8));
#pragma unroll
            for (int j = 0; j < 4; ++j) qd[j] = row_ld4(rq, qoff + (j * (NT / (D / 8))) * rb);
        }
    };
    // the chunk's gates: formed by the last wave, one chunk ahead, off the other waves' path
    auto load_gates = [&](int c0) {
        return a.alpha[a.alpha_tok ? (size_t)min(c0 + lane, te - 1) * a.alpha_tok + head : head % (unsigned)a.H];
    };
    if (t0 < te) {
        load_kq(t0);
        load_v(t0);
    }
    double gtot = 0.0;                                             // (last wave) log decay of the segment so far
    if (w == NW - 1 && t0 < te) gtot = make_gates<BL>(load_gates(t0), te - t0, lane, s_gate[0]);

    int cur = 0;
    for (int c0 = t0; c0 < te; c0 += BL, cur ^= 1) {
        const int L = min(BL, te - c0);
        const double* sG = s_gate[cur].g;
        const float *sE = s_gate[cur].e, *sW = s_gate[cur].w;
        const bool ahead = w == NW - 1 && c0 + BL < te;
        float al = 0.0f;
        if (ahead) al = load_gates(c0 + BL);
        // ---- registers -> LDS ----
        const int ln = fresh(lane), kpair = ln % (D / 2), ksub = ln / (D / 2);   // channel pair; octet within a wave's pass
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int oct = (2 * w + j) * OPW + ksub;
            u32x4 x0, x1;                                          // 8 tokens of the pair's two channels
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x0[e] = __builtin_amdgcn_perm(kd[j][2 * e + 1], kd[j][2 * e], 0x05040100u);
                x1[e] = __builtin_amdgcn_perm(kd[j][2 * e + 1], kd[j][2 * e], 0x07060302u);
            }
            *reinterpret_cast<u32x4*>(&sT[pm<D>(2 * kpair, oct)]) = x0;
            *reinterpret_cast<u32x4*>(&sT[pm<D>(2 * kpair + 1, oct)]) = x1;
            if constexpr (OUT) {
                // channels (c, c + 1), c = 2 kpair, in the operand order of their 32-block
                const int u = (2 * kpair & 31) >> 2;
                const int piece = (kpair >> 4) * 4 + (u & 3), in = 4 * (u >> 2) + (2 * kpair & 3);
#pragma unroll
                for (int e = 0; e < 8; ++e) *reinterpret_cast<uint32_t*>(&sK[pm<BL>(8 * oct + e, piece) + in]) = kd[j][e];
            }
        }
        if constexpr (OUT)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = 64 * w + ln + NT * j, row = e / (D / 8), c = 8 * (e % (D / 8));
                const int u = (c & 31) >> 2;                       // two groups of 4 channels: u, u + 1
                const int p0 = (c >> 5) * 4, in = 4 * (u >> 2);
                *reinterpret_cast<u32x2*>(&sQ[pm<BL>(row, p0 + (u & 3)) + in]) = u32x2{qd[j][0], qd[j][1]};
                *reinterpret_cast<u32x2*>(&sQ[pm<BL>(row, p0 + ((u + 1) & 3)) + in]) = u32x2{qd[j][2], qd[j][3]};
            }
        u32x4 V[2][2];                                             // B operands: [32-token step][ct]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                V[j][0][e] = __builtin_amdgcn_perm(vd[j][2 * e + 1], vd[j][2 * e], 0x05040100u);
                V[j][1][e] = __builtin_amdgcn_perm(vd[j][2 * e + 1], vd[j][2 * e], 0x07060302u);
            }
        __syncthreads();

        const float egl = sE[BL - 1];
        if (!OUT && ahead) gtot += make_gates<BL>(al, te - c0 - BL, lane, s_gate[cur ^ 1]);
        if constexpr (OUT) {
            const int lo = fresh(lane), li = lo & 15, lg = lo >> 4;
            const int at = pm<BL>(li, lg);                         // operand reads: row li, piece lg
            // ---- scores: the 10 tiles on and below the diagonal, over the waves ----
            // (one branch per tile on the wave's index, so that every LDS address is a constant
            // away from the lane's)
#pragma unroll
            for (int x = 0; x < 10; ++x) {
                if (x % NW != w) continue;
                const int r = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, c = x - r * (r + 1) / 2;
                v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                    acc = mfma_bf16(*reinterpret_cast<const u32x4*>(&sQ[at + pm<BL>(16 * r, 4 * ks)]),
                                    *reinterpret_cast<const u32x4*>(&sK[at + pm<BL>(16 * c, 4 * ks)]), acc);
                const double gi = sG[16 * c + li];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int n = 16 * r + 4 * lg + v;
                    float p = __expf((float)(sG[n] - gi)) * acc[v];
                    if (r == c) p = li <= 4 * lg + v ? p : 0.0f;
                    const int to = pm<BL>(n, 2 * c) + pm<BL>(0, li >> 3) + (li & 7);
                    const float p1 = p - top_f32(p);
                    sP[0][to] = (uint16_t)(__float_as_uint(p) >> 16);
                    sP[1][to] = (uint16_t)(__float_as_uint(p1) >> 16);
                    sP[2][to] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // ---- O = e^g o (Q H) ----
            v4f O[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) O[r][0] = O[r][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                u32x4 b[2][3];
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
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const u32x4 aq = *reinterpret_cast<const u32x4*>(&sQ[at + pm<BL>(16 * r, 4 * ks)]);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                        for (int m = 2; m >= 0; --m) O[r][ct] = mfma_bf16(aq, b[ct][m], O[r][ct]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const v4f e = *reinterpret_cast<const v4f*>(&sE[16 * r + 4 * lg]);
                O[r][0] *= e;
                O[r][1] *= e;
            }
            if (ahead) gtot += make_gates<BL>(al, te - c0 - BL, lane, s_gate[cur ^ 1]);
            __syncthreads();                                       // the scores are written
            // ---- O += (E o Q K^T) V ----
            // a column's plain sum over the chunk is finite unless one of its values is not
            // (or they overflow: then the careful path is taken for nothing)
            v4f sum[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
                    sum[ct] = mfma_bf16(u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}, V[j][ct], sum[ct]);
            const bool any_odd = __any(!finite_f32(sum[0][0]) || !finite_f32(sum[1][0]));
            if (any_odd)                                           // finite values first: 0 * v must stay 0
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t x = odd_bf16(V[j][ct][e]);
                            V[j][ct][e] &= ((x & 0x8000u) ? 0u : 0xffffu) | ((x & 0x80000000u) ? 0u : 0xffff0000u);
                        }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j <= r / 2; ++j)
#pragma unroll
                    for (int part = 2; part >= 0; --part) {
                        const u32x4 ap = *reinterpret_cast<const u32x4*>(&sP[part][at + pm<BL>(16 * r, 4 * j)]);
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct) O[r][ct] = mfma_bf16(ap, V[j][ct], O[r][ct]);
                    }
            if (any_odd) {
                const rsrc_t rv = rows(a.v, c0);
                const int lq = fresh(4 * lg), vband = fresh(4 * (16 * w + li));
#pragma unroll 1
                for (int i = 0; i < L; ++i) {                      // then the others, from their own token on
                    const uint32_t x = row_ld(rv, i * rb + vband);
                    const uint32_t od = odd_bf16(x);
                    if (od)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const int n = 16 * r + lq + v;
                                const int from = pm<BL>(n, i >> 3) + (i & 7);
                                const float p = n < i ? 0.0f : bf16_to_f32(sP[0][from]) + bf16_to_f32(sP[1][from]) + bf16_to_f32(sP[2][from]);
                                if (n >= i && (od & 0x8000u)) O[r][0][v] += p * lo_f32(x);
                                if (n >= i && (od & 0x80000000u)) O[r][1][v] += p * hi_f32(x);
                            }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)                        // the state takes them all
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x0 = row_ld(rv, (32 * j + 2 * lq + 2 * e) * rb + vband);
                        const uint32_t x1 = row_ld(rv, (32 * j + 2 * lq + 2 * e + 1) * rb + vband);
                        V[j][0][e] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                        V[j][1][e] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                    }
            }
            const rsrc_t ro = rows(a.o, c0);                       // rows past the end are left as they were
            const uint32_t ooff = 4 * lg * rb + 4 * (16 * w + li);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v) row_st(ro, ooff + (16 * r + v) * rb, pack_bf16(O[r][0][v], O[r][1][v]));
        }
        if (c0 + BL < te) {                                        // (here and not earlier: the registers of O are free)
            load_kq(c0 + BL);
            load_v(c0 + BL);
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- H = e^{g_L} H + K^T (w o V) ----
        const int lk = fresh(lane), li = lk & 15, lg = lk >> 4;
        if (a.end || c0 + BL < te) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                H[rt][0] *= egl;
                H[rt][1] *= egl;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const v4f w0 = *reinterpret_cast<const v4f*>(&sW[32 * j + 8 * lg]);
                const v4f w1 = *reinterpret_cast<const v4f*>(&sW[32 * j + 8 * lg + 4]);
                u32x4 b[3][2];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = (e < 2 ? w0[2 * e] : w1[2 * e - 4]) * lo_f32(V[j][ct][e]);
                        const float x1 = (e < 2 ? w0[2 * e + 1] : w1[2 * e - 3]) * hi_f32(V[j][ct][e]);
                        b[0][ct][e] = top_halves(x0, x1);
                        const float y0 = x0 - top_f32(x0), y1 = x1 - top_f32(x1);
                        b[1][ct][e] = top_halves(y0, y1);
                        b[2][ct][e] = top_halves(y0 - top_f32(y0), y1 - top_f32(y1));
                    }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const u32x4 ak = *reinterpret_cast<const u32x4*>(&sT[pm<D>(li, lg) + pm<D>(16 * rt, 4 * j)]);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                        for (int part = 0; part < 3; ++part) H[rt][ct] = mfma_bf16(ak, b[part][ct], H[rt][ct]);
                    if (rt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __syncthreads();                                           // LDS is rewritten by the next chunk
    }
    if (!a.end && !a.decay) return;
    const int lf = fresh(lane), lg = lf >> 4, band = 16 * w + (lf & 15);
    if (a.end)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                *reinterpret_cast<f32x2*>(a.end + soff + (size_t)(16 * rt + 4 * lg + v) * D + 2 * band) =
                    f32x2{H[rt][0][v], H[rt][1][v]};
    if (a.decay && t == NT - 64) a.decay[blockIdx.y * heads + head] = expf((float)gtot);
}

// ---------------------------------------------------------------------------
// fp32 tokens, d >= 64: chunks of 32 tokens, every operand in three bf16 parts
// ---------------------------------------------------------------------------
// An fp32 value is the exact sum of three bf16 parts (its 24 bits cut in three), so a
// product is six bf16 products (of nine: the three left out are at most 2^-21 of it, 2^-24.7
// on average) summed in fp32: 6 x 16 cycles for 16x16x32 against 8 x 32 on the fp32 matrix
// instruction.
// Wave w owns the 16 columns 16 w + li; otherwise as la_chunk_kernel.  32 tokens: three parts
// of three operands fill half a CU's LDS.  Bound by phases that take turns on the vector unit (splits)
// and the matrix unit, two waves a SIMD:
// d = 128, 192 heads of up to 1021 tokens 140 us (4.4 us a chunk; vector unit busy for
// 0.50 of the waves' time, matrix unit for 0.35), 512 heads of 512 tokens 200 us (2.9 TB/s).
// Workgroups of half the columns fill more CUs but form the rows' parts
// twice: 512 heads of 512 tokens 213 us, not 198; 1024 heads of 300 tokens 296 us, not 261.
constexpr int FL = 32;        // tokens per chunk

template <int D>
struct LF {
    static constexpr int NW = D / 16, NT = 64 * NW;
    static constexpr int RT = D / 16;
    static constexpr int QP = D / 8, TP = FL / 8;   // pieces per Q / K row, per K^T / score row
};

template <int D, bool OUT>
__global__ __launch_bounds__(LF<D>::NT, 2) void la_chunk32_kernel(LaSegArgs a) {
    using P = LF<D>;
    constexpr int NW = P::NW, NT = P::NT, RT = P::RT, QP = P::QP, TP = P::TP;
    __shared__ __align__(16) uint16_t sQ[3][OUT ? pm_shorts<FL>(QP) : 8];
    __shared__ __align__(16) uint16_t sK[3][OUT ? pm_shorts<FL>(QP) : 8];
    __shared__ __align__(16) uint16_t sT[3][pm_shorts<D>(TP)];               // (w o K)^T: [channel][token]
    __shared__ __align__(16) uint16_t sP[3][OUT ? pm_shorts<FL>(TP) : 8];    // scores
    __shared__ Gates<FL> s_gate[2];                                // of this chunk and the next

    const int t = threadIdx.x, lane = t & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg;
    const int te = min(len, t0 + a.seg);
    const int col = 16 * w + li;
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);

    v4f H[RT];                                                     // H[rt][v] = H[16 rt + 4 lg + v][col]
    if (a.start) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) H[rt][v] = a.start[soff + (size_t)(16 * rt + 4 * lg + v) * D + col];
    } else {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) H[rt] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (OUT)
        for (int e = t; e < 3 * 16 * 16; e += NT) sP[e >> 8][pm<FL>((e >> 4) & 15, 2 + ((e >> 3) & 1)) + (e & 7)] = 0;   // right of the diagonal

    // chunk loads, one chunk ahead; tokens past the end read as zeros
    constexpr int CPR = D / 8;                                     // 8-channel pieces per row
    static_assert(NT / CPR == FL && NT / D == FL / 8, "one piece and one octet per thread");
    const uint32_t rb = (uint32_t)heads * (4 * D);                 // bytes between tokens (heads <= chunk_heads(D))
    uint32_t kt[8], vr[8];
    u32x4 qr[2], kr[2];
    auto rows = [&](const void* x, int c0) {                       // tokens c0 .. min(c0 + FL, te) - 1 of this head
        return make_rows(static_cast<const char*>(x) + ((size_t)c0 * heads + head) * (4 * D),
                         (uint32_t)(min(te - c0, FL) - 1) * rb + 4 * D);
    };
    auto load = [&](int c0) {
        const uint32_t tt = fresh(t), ln = tt & 63;
        const rsrc_t rk = rows(a.k, c0), rv = rows(a.v, c0);
        const uint32_t koff = 8 * (tt / D) * rb + 4 * (tt % D), voff = 8 * (ln >> 4) * rb + 4 * (16 * w + (ln & 15));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            kt[e] = row_ld(rk, koff + e * rb);
            vr[e] = row_ld(rv, voff + e * rb);
        }
        if constexpr (OUT) {
            const rsrc_t rq = rows(a.q, c0);
            const uint32_t off = (tt / CPR) * rb + 32 * (tt % CPR);
            qr[0] = row_ld4(rq, off);
            qr[1] = row_ld4(rq, off + 16);
            kr[0] = row_ld4(rk, off);
            kr[1] = row_ld4(rk, off + 16);
        }
    };
    auto load_gates = [&](int c0) {
        return a.alpha[a.alpha_tok ? (size_t)min(c0 + (lane & (FL - 1)), te - 1) * a.alpha_tok + head : head % (unsigned)a.H];
    };
    if (t0 < te) load(t0);
    double gtot = 0.0;                                             // (last wave) log decay of the segment so far
    if (w == NW - 1 && t0 < te) gtot = make_gates<FL>(load_gates(t0), te - t0, lane, s_gate[0]);
    __syncthreads();

    int cur = 0;
    for (int c0 = t0; c0 < te; c0 += FL, cur ^= 1) {
        const int L = min(FL, te - c0);
        const double* sG = s_gate[cur].g;
        const float *sE = s_gate[cur].e, *sW = s_gate[cur].w;
        const bool ahead = w == NW - 1 && c0 + FL < te;
        float al = 0.0f;
        if (ahead) al = load_gates(c0 + FL);
        {
            const int tt = fresh(t), kc = tt % D, koct = tt / D;   // K^T: channel, 8 tokens
            float x[8], wt[8];
            uint32_t p[3][4];
            load_floats<8>(sW + 8 * koct, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = wt[e] * __uint_as_float(kt[e]);
            split3<8>(x, p);
#pragma unroll
            for (int m = 0; m < 3; ++m)
                *reinterpret_cast<u32x4*>(&sT[m][pm<D>(kc, koct)]) = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            if constexpr (OUT) {
                const int row = tt / CPR, c8 = 8 * (tt % CPR);
                const int u = (c8 & 31) >> 2;                      // two groups of 4 channels, in operand order
                const int at0 = pm<FL>(row, (c8 >> 5) * 4 + (u & 3)) + 4 * (u >> 2);
                const int at1 = pm<FL>(row, (c8 >> 5) * 4 + ((u + 1) & 3)) + 4 * (u >> 2);
#pragma unroll
                for (int which = 0; which < 2; ++which) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(which ? kr[e / 4][e % 4] : qr[e / 4][e % 4]);
                    split3<8>(x, p);
#pragma unroll
                    for (int m = 0; m < 3; ++m) {
                        uint16_t* dst = which ? sK[m] : sQ[m];
                        *reinterpret_cast<u32x2*>(dst + at0) = u32x2{p[m][0], p[m][1]};
                        *reinterpret_cast<u32x2*>(dst + at1) = u32x2{p[m][2], p[m][3]};
                    }
                }
            }
        }
        float V[8];
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            V[e] = __uint_as_float(vr[e]);
            odd |= !finite_f32(V[e]);
        }
        __syncthreads();
        if (c0 + FL < te) load(c0 + FL);

        const float egl = sE[FL - 1];
        if (!OUT && ahead) gtot += make_gates<FL>(al, te - c0 - FL, lane, s_gate[cur ^ 1]);
        u32x4 vp[3];                                               // B operand: the values in parts
        {
            uint32_t p[3][4];
            split3<8>(V, p);
#pragma unroll
            for (int m = 0; m < 3; ++m) vp[m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
        }
        if constexpr (OUT) {
            // scores: tiles (0,0), (1,0), (1,1), one wave each
            if (w < 3) {
                const int r = (w + 1) >> 1, c = w >> 1;
                v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks) {
                    u32x4 x[3], y[3];
#pragma unroll
                    for (int m = 0; m < 3; ++m) {
                        x[m] = *reinterpret_cast<const u32x4*>(&sQ[m][pm<FL>(li, lg) + pm<FL>(16 * r, 4 * ks)]);
                        y[m] = *reinterpret_cast<const u32x4*>(&sK[m][pm<FL>(li, lg) + pm<FL>(16 * c, 4 * ks)]);
                    }
                    acc = mfma_split(x, y, acc);
                }
                const int i = 16 * c + li;
                const double gi = sG[i];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int n = 16 * r + 4 * lg + v;
                    const float p = i <= n ? __expf((float)(sG[n] - gi)) * acc[v] : 0.0f;
                    const float p1 = p - top_f32(p);
                    const int at = pm<FL>(n, i >> 3) + (i & 7);
                    sP[0][at] = (uint16_t)(__float_as_uint(p) >> 16);
                    sP[1][at] = (uint16_t)(__float_as_uint(p1) >> 16);
                    sP[2][at] = (uint16_t)(__float_as_uint(p1 - top_f32(p1)) >> 16);
                }
            }
            v4f O[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = H[2 * ks + e / 4][e % 4];
                split3<8>(x, p);
                u32x4 b[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) b[m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    u32x4 q[3];
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        q[m] = *reinterpret_cast<const u32x4*>(&sQ[m][pm<FL>(li, lg) + pm<FL>(16 * r, 4 * ks)]);
                    O[r] = mfma_split(q, b, O[r]);
                }
            }
            O[0] *= *reinterpret_cast<const v4f*>(&sE[4 * lg]);
            O[1] *= *reinterpret_cast<const v4f*>(&sE[16 + 4 * lg]);
            if (ahead) gtot += make_gates<FL>(al, te - c0 - FL, lane, s_gate[cur ^ 1]);
            __syncthreads();                                       // the scores are written
            u32x4 fp[3] = {vp[0], vp[1], vp[2]};                   // finite values: 0 * v must stay 0
            if (__any(odd)) {
                float x[8];
                uint32_t p[3][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = finite_f32(V[e]) ? V[e] : 0.0f;
                split3<8>(x, p);
#pragma unroll
                for (int m = 0; m < 3; ++m) fp[m] = u32x4{p[m][0], p[m][1], p[m][2], p[m][3]};
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                u32x4 x3[3];
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    x3[m] = *reinterpret_cast<const u32x4*>(&sP[m][pm<FL>(li, lg) + pm<FL>(16 * r, 0)]);
                O[r] = mfma_split(x3, fp, O[r]);
            }
            if (__any(odd))
#pragma unroll 1
                for (int i = 0; i < L; ++i) {
                    const float x = __uint_as_float(row_ld(rows(a.v, c0), i * rb + 4 * col));
                    if (!finite_f32(x))
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const int n = 16 * r + 4 * lg + v;
                                const int at = pm<FL>(n, i >> 3) + (i & 7);
                                if (n >= i)
                                    O[r][v] += (bf16_to_f32(sP[0][at]) + bf16_to_f32(sP[1][at]) + bf16_to_f32(sP[2][at])) * x;
                            }
                }
            const rsrc_t ro = rows(a.o, c0);                       // rows past the end are left as they were
            const uint32_t ln = fresh(lane), ooff = 4 * (ln >> 4) * rb + 4 * (16 * w + (ln & 15));
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v) row_st(ro, ooff + (16 * r + v) * rb, __float_as_uint(O[r][v]));
        }
        if (a.end || c0 + FL < te) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                H[rt] *= egl;
                u32x4 k3[3];
#pragma unroll
                for (int m = 0; m < 3; ++m) k3[m] = *reinterpret_cast<const u32x4*>(&sT[m][pm<D>(li, lg) + pm<D>(16 * rt, 0)]);
                H[rt] = mfma_split(k3, vp, H[rt]);
            }
        }
        __syncthreads();                                           // LDS is rewritten by the next chunk
    }
    if (a.end)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int v = 0; v < 4; ++v) a.end[soff + (size_t)(16 * rt + 4 * lg + v) * D + col] = H[rt][v];
    if (a.decay && t == NT - 64) a.decay[blockIdx.y * heads + head] = expf((float)gtot);
}

// ---------------------------------------------------------------------------
// a few tokens: the recurrence itself
// ---------------------------------------------------------------------------
// Reads the state once and writes it once; per token the decay, the rank-one update
// and the column sums of H o q.  Lane t holds the columns 4 (t % (D/4)) .. +3 of the
// rows t / (D/4) + RPP p.  The tokens come through LDS, kStepTokens at a time, requested
// with the state.  Bound by memory: one token of 2048 heads at d = 128 in 49 us (5.5 TB/s), four in 58 us.  Against a chunk of 64 (32) tokens, four tokens:
// 2048 heads 58 us, not 60 (76); 16 heads 10.5 us, not 8.7 (7.6); two tokens: 6.5 us, not 8.7 (7.5).
constexpr int kStepTokens = 4;
template <int D, typename TI>
__global__ __launch_bounds__(256) void la_step_kernel(LaPrefillArgs a) {
    constexpr int CP = D / 4, NT = D >= 64 ? 256 : 64, RPP = NT / CP, NP = D / RPP, NW = NT / 64, ST = kStepTokens;
    constexpr int NX = ST * D / NT;                                // values of each kind per thread
    __shared__ __align__(16) float sx[3][ST * D];                  // q, k, v
    __shared__ __align__(16) float so[2][NW][D];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int T = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int rg = t / CP, c0 = 4 * (t % CP);
    const float* h0 = a.h0 + head * (size_t)(D * D);
    v4f H[NP];
    for (int n0 = 0; n0 < max(T, 1); n0 += ST) {
        TI x[3][NX];
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            const int e = t + NT * u, n = n0 + e / D;
            if (n >= T) break;
            const size_t at = ((size_t)n * heads + head) * D + e % D;
            if (a.o) x[0][u] = static_cast<const TI*>(a.q)[at];
            x[1][u] = static_cast<const TI*>(a.k)[at];
            x[2][u] = static_cast<const TI*>(a.v)[at];
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
            for (int y = 0; y < 3; ++y)
                if (y || a.o) sx[y][e] = widen(x[y][u]);
        }
        __syncthreads();
        for (int n = n0; n < min(T, n0 + ST); ++n) {
            const float al = a.alpha_tok ? a.alpha[(size_t)n * a.alpha_tok + head] : a.alpha[head % (unsigned)a.H];
            const float *q = sx[0] + (n - n0) * D, *k = sx[1] + (n - n0) * D;
            const v4f vv = *reinterpret_cast<const v4f*>(&sx[2][(n - n0) * D + c0]);
            v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                H[p] = H[p] * al + vv * k[p * RPP + rg];
                if (a.o) o += H[p] * q[p * RPP + rg];
            }
            if (!a.o) continue;
#pragma unroll
            for (int m = CP; m < 64; m <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], m, 64);
            if (lane < CP) *reinterpret_cast<v4f*>(&so[n & 1][w][c0]) = o;
            __syncthreads();                                       // (the other half is written meanwhile)
            if (t < D) {
                float y = 0.0f;
#pragma unroll
                for (int i = 0; i < NW; ++i) y += so[n & 1][i][t];
                tok_st<TI>(a.o, ((size_t)n * heads + head) * D + t, y);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
        __builtin_nontemporal_store(H[p], reinterpret_cast<v4f*>(a.h + head * (size_t)(D * D) + (size_t)(p * RPP + rg) * D + c0));
}
// Heads that the chunk kernels take: at d >= 64 a chunk's rows lie within 32-bit byte offsets (64 rows of
// 2 d bytes a head, 32 of 4 d); d = 16 has offsets in 64 bits.  More heads take the recurrence itself:
// 131200 heads of 64 (512) tokens, bf16, 1.6 (5.7) ms by chunks, 5.9 (13.4) ms token after token at d = 64 (16).
constexpr size_t chunk_heads(int d) { return d == 16 ? (size_t)INT32_MAX : (size_t)(1 << 24) / d; }

// ---------------------------------------------------------------------------
// d = 16: chunks of 16 tokens, one wave a segment, no LDS
// ---------------------------------------------------------------------------
// With d = 16 every product is one 16 x 16 x 16 of the fp32 matrix instruction, and each
// operand is loaded in the layout that the instruction takes (lane (lg, li), step v: row or
// column li, index 4 lg + v): 80 us for 2048 heads of 512 tokens, bf16 (1.8 TB/s) or fp32
// (3.5 TB/s); 65 and 62 with the tokens in the Infinity Cache.  Bound by the waves' issue (two
// waves a SIMD: vector unit busy for 0.53 of the time, matrix unit for 0.22).  The scores are formed transposed (K Q^T): their accumulators
// are then the A operand of P V as they are.  Everything stays in registers, so waves need
// no barrier and many fit; the next chunk's loads are in flight during a chunk.
template <typename TI, bool OUT>
__global__ __launch_bounds__(256) void la_small_kernel(LaSegArgs a) {
    constexpr int D = 16, CS = 16;
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
    const size_t heads = (size_t)a.heads;
    const size_t head = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);      // one head a wave
    if (head >= heads) return;
    const int len = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;
    const int t0 = (int)blockIdx.y * a.seg, te = min(len, t0 + a.seg);
    const size_t soff = blockIdx.y * a.seg_stride + head * (size_t)(D * D);
    v4f H = {0.f, 0.f, 0.f, 0.f};                                         // H[4 lg + v][li]
    if (a.start)
#pragma unroll
        for (int v = 0; v < 4; ++v) H[v] = a.start[soff + (4 * lg + v) * D + li];
    // token li: q, k channels 4 lg + v; tokens 4 lg + v: k, v channel li
    struct Chunk {                                                        // (as loaded: widened on use)
        Row4<TI> q, k;
        TI kt[4], vt[4];
        float al;
    };
    auto load = [&](int c0, Chunk& x) {                                   // (past the end: the last token, zeroed on use)
        const int n = min(c0 + li, te - 1);
        const size_t at = ((size_t)n * heads + head) * D + 4 * lg;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const size_t to = ((size_t)min(c0 + 4 * lg + v, te - 1) * heads + head) * D + li;
            x.kt[v] = static_cast<const TI*>(a.k)[to];
            x.vt[v] = static_cast<const TI*>(a.v)[to];
        }
        if (OUT) {
            x.q.load(a.q, at);
            x.k.load(a.k, at);
        }
        x.al = a.alpha[a.alpha_tok ? (size_t)n * a.alpha_tok + head : head % (unsigned)a.H];
    };
    Chunk cur, nxt;
    if (t0 < te) load(t0, cur);
    double gtot = 0.0;
    for (int c0 = t0; c0 < te; c0 += CS) {
        const int L = min(CS, te - c0);
        if (c0 + CS < te) load(c0 + CS, nxt);
        // every 16 lanes hold the chunk's prefix sums
        double g = li < L ? (double)log_decay(cur.al) : 0.0;
        g = scan_step<0x111, 0xf>(g);
        g = scan_step<0x112, 0xf>(g);
        g = scan_step<0x114, 0xf>(g);
        g = scan_step<0x118, 0xf>(g);
        const double gl = __shfl(g, 15, 16);
        double gi[4];                                                     // of tokens 4 lg + v
#pragma unroll
        for (int v = 0; v < 4; ++v) gi[v] = __shfl(g, 4 * lg + v, 16);
        // (an exponent is at most 0: off by 2^-24 of it, weighted by its exponential)
        float vt[4], kw[4];
        bool odd = false;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const bool on = 4 * lg + v < L;
            vt[v] = on ? widen(cur.vt[v]) : 0.0f;
            kw[v] = on ? __expf((float)(gl - gi[v])) * widen(cur.kt[v]) : 0.0f;
            odd |= !finite_f32(vt[v]);
        }
        if constexpr (OUT) {
            // P^T[i = 4 lg + v][n = li]
            v4f p = {0.f, 0.f, 0.f, 0.f};
            float qr[4], kr[4];
            cur.q.widen4(qr);
            cur.k.widen4(kr);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float x = li < L ? kr[v] : 0.0f, y = li < L ? qr[v] : 0.0f;
                p = __builtin_amdgcn_mfma_f32_16x16x4f32(x, y, p, 0, 0, 0);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) p[v] = 4 * lg + v <= li ? __expf((float)(g - gi[v])) * p[v] : 0.0f;
            const float en = expf((float)g);
            v4f o = {0.f, 0.f, 0.f, 0.f};                                 // o[n = 4 lg + v][li]
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                o = __builtin_amdgcn_mfma_f32_16x16x4f32(li < L ? en * qr[v] : 0.0f, H[v], o, 0, 0, 0);
                o = __builtin_amdgcn_mfma_f32_16x16x4f32(p[v], finite_f32(vt[v]) ? vt[v] : 0.0f, o, 0, 0, 0);
            }
            if (__any(odd))                                               // the others, from their own token on
#pragma unroll 1
                for (int i = 0; i < L; ++i) {
                    const float x = tok_ld<TI>(a.v, ((size_t)(c0 + i) * heads + head) * D + li);
                    const float p0 = i & 2 ? (i & 1 ? p[3] : p[2]) : (i & 1 ? p[1] : p[0]);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float pn = __shfl(p0, 16 * (i >> 2) + 4 * lg + v, 64);   // P[4 lg + v][i]
                        if (!finite_f32(x) && 4 * lg + v >= i) o[v] += pn * x;
                    }
                }
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (4 * lg + v < L) tok_st<TI>(a.o, ((size_t)(c0 + 4 * lg + v) * heads + head) * D + li, o[v]);
        }
        H *= expf((float)gl);
#pragma unroll
        for (int v = 0; v < 4; ++v) H = __builtin_amdgcn_mfma_f32_16x16x4f32(kw[v], vt[v], H, 0, 0, 0);
        gtot += gl;
        cur = nxt;
    }
    if (a.end)
#pragma unroll
        for (int v = 0; v < 4; ++v) a.end[soff + (4 * lg + v) * D + li] = H[v];
    if (a.decay && lane == 0) a.decay[blockIdx.y * heads + head] = expf((float)gtot);
}

// States before each segment from the states of each segment alone, in place, and the
// state after the last one: S_s = X, X <- decay_s X + S_s.  Four values per lane; bound by
// memory and, with few heads, by the latency of one group of loads (16 heads at d = 128: 5.1 us
// for 8 segments, 12.5 us for 32, 5.4 TB/s).
struct LaScanArgs {
    const float* h0;          // or null: zeros
    float* h;
    float* ws;                // [segments][heads][d*d]
    const float* decay;       // [segments][heads]
    size_t heads;
    int dd4;                  // d*d / 4
    int segs;
};
constexpr int kScanAhead = 8;
__global__ __launch_bounds__(256) void la_scan_kernel(LaScanArgs a) {
    const size_t e = blockIdx.x * 256 + threadIdx.x, head = blockIdx.y;
    if (e >= (size_t)a.dd4) return;
    const size_t at = head * a.dd4 + e, stride = a.heads * a.dd4;
    v4f x = {0.f, 0.f, 0.f, 0.f};
    if (a.h0) x = reinterpret_cast<const v4f*>(a.h0)[at];
    v4f* ws = reinterpret_cast<v4f*>(a.ws);
    for (int s0 = 0; s0 < a.segs; s0 += kScanAhead) {      // (the loads of a group before its first store)
        v4f y[kScanAhead];
        float d[kScanAhead];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u) {
            const int s = min(s0 + u, a.segs - 1);
            y[u] = ws[s * stride + at];
            d[u] = a.decay[s * a.heads + head];
        }
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (s0 + u < a.segs) {
                ws[(s0 + u) * stride + at] = x;
                x = x * d[u] + y[u];
            }
    }
    reinterpret_cast<v4f*>(a.h)[at] = x;
}

// Tokens per segment (a multiple of the chunk).  Segments cost a second read of k and v and
// the states between them, so they pay where the heads alone leave most CUs idle: up to
// `heads` heads, enough segments for `want` workgroups (as many as fit the GPU: two a CU at
// d = 128, three at d = 64; d = 16: waves), and from three chunks on (the whole prompt is one
// launch, segments are three).  Measured, bf16 (fp32), replayed in a graph:
//   d = 128, 2048 tokens: 96 heads 109 us (187) split, 181 (271) whole; 1024 tokens: 192 heads
//   110 us (210) split, 101 (148) whole; 16 heads and 16384 tokens: 161, 131, 139 us
//   (253, 252, 272) for 256, 512 and 768 workgroups;
//   d = 64, 2048 tokens: 128 heads 67 us (92) split, 146 (161) whole; 256 heads 107 us (186)
//   split, 147 (177) whole, 134 (192) for 512 workgroups; 512 heads, 1024 tokens: 96 us (127)
//   in two segments, 104 (127) whole;
//   two chunks (65 tokens): 16 heads at d = 128 16.4 us (16.1) split, 14.3 (15.7) whole, 128
//   heads 27 (33) split, 16 (17) whole; 16 heads at d = 64 13.2 (11.4) split, 12.0 (10.7) whole;
//   three chunks (130 tokens) of 16 heads: 17.6 us (18.3) split, 19.8 (23.6) whole;
//   (many heads lose by it: 128 heads of 130 tokens 31 us (40) split, 21 (25) whole, 512
//   tokens 50 (80) split, 51 (72) whole; 256 heads of 130 tokens at d = 64 28 (26), 18 (17))
//   d = 16, 512 tokens (segments of 8 chunks at least): 768 heads 41 us (43) split, 47 (44)
//   whole; 1024 heads 51 (53) split, 48 (45) whole; 2048 heads 87 (94) split, 65 (62) whole,
//   2.2 (4.4) TB/s.
struct Split {
    size_t heads, want;
};
constexpr Split kSplit128{128, 512}, kSplit64{256, 768}, kSplit16{768, 4096};
constexpr size_t kMinSmall = 128;
size_t segments_wanted(size_t heads, size_t chunks, int d) {
    const Split x = d == 16 ? kSplit16 : d == 64 ? kSplit64 : kSplit128;
    if (heads > x.heads || (d >= 64 && chunks <= 2)) return 1;
    return x.want / heads;                                        // (one round of workgroups)
}
int chunk_tokens(const lq_dims& d) { return d.dk == 16 ? (int)kMinSmall : d.io_dtype == LQ_IO_BF16 ? BL : FL; }
int segment_tokens(const lq_dims& d, int T) {
    const size_t chunk = chunk_tokens(d), chunks = ((size_t)T + chunk - 1) / chunk;
    const size_t want = segments_wanted((size_t)d.B * d.H, chunks, d.dk);
    return (int)((chunks + want - 1) / want * chunk);
}

template <int D, typename TI, bool OUT>
hipError_t chunk_launch(dim3 grid, const LaSegArgs& sa, hipStream_t s) {
    if constexpr (D == 16)
        return launch_kernel(LQ_KERNEL_LA_PREFILL, la_small_kernel<TI, OUT>, dim3((grid.x + 3) / 4, grid.y), dim3(256), s, sa);
    else if constexpr (sizeof(TI) == 2)
        return launch_kernel(LQ_KERNEL_LA_PREFILL, la_chunk_kernel<D, OUT>, grid, dim3(LB<D>::NT), s, sa);
    else
        return launch_kernel(LQ_KERNEL_LA_PREFILL, la_chunk32_kernel<D, OUT>, grid, dim3(LF<D>::NT), s, sa);
}

template <int D, typename TI>
hipError_t la_chunks(const lq_dims& d, const LaPrefillArgs& args, void* workspace, hipStream_t s) {
    const size_t heads = (size_t)args.heads;
    const int seg = segment_tokens(d, args.T), segs = (int)(((size_t)args.T + seg - 1) / seg);
    LaSegArgs sa{args.h0, args.h, nullptr, args.q, args.k, args.v, args.alpha, args.lens, args.o, 0,
                 args.T, args.H, args.heads, args.alpha_tok, seg};
    const dim3 grid((unsigned)heads, (unsigned)segs);
    if (segs == 1) return args.o ? chunk_launch<D, TI, true>(grid, sa, s) : chunk_launch<D, TI, false>(grid, sa, s);
    float* ws = static_cast<float*>(workspace);
    float* decay = ws + (size_t)segs * heads * D * D;
    sa.seg_stride = heads * D * D;
    sa.start = nullptr;
    sa.end = ws;
    sa.decay = decay;
    hipError_t e = chunk_launch<D, TI, false>(grid, sa, s);
    if (e != hipSuccess) return e;
    LaScanArgs sc{args.h0, args.h, ws, decay, heads, D * D / 4, segs};
    e = launch_kernel(LQ_KERNEL_LA_PREFILL, la_scan_kernel, dim3((D * D / 4 + 255) / 256, (unsigned)heads), dim3(256), s, sc);
    if (e != hipSuccess || !args.o) return e;
    sa.start = ws;
    sa.end = nullptr;
    sa.decay = nullptr;
    return chunk_launch<D, TI, true>(grid, sa, s);
}

template <int D, typename TI>
hipError_t la_prefill_t(const lq_dims& d, const LaPrefillArgs& args, void* workspace, hipStream_t s) {
    const dim3 grid((unsigned)args.heads);
    if (args.T <= kStepTokens || (size_t)args.heads > chunk_heads(D))
        return launch_kernel(LQ_KERNEL_LA_PREFILL, la_step_kernel<D, TI>, grid, dim3(D >= 64 ? 256 : 64), s, args);
    return la_chunks<D, TI>(d, args, workspace, s);
}

template <int D>
hipError_t la_prefill_d(const lq_dims& d, const LaPrefillArgs& args, void* workspace, hipStream_t s) {
    return d.io_dtype == LQ_IO_BF16 ? la_prefill_t<D, uint16_t>(d, args, workspace, s)
                                    : la_prefill_t<D, float>(d, args, workspace, s);
}

}  // namespace

size_t la_workspace_bytes(const lq_dims& d, int T) {
    const size_t heads = (size_t)d.B * d.H, chunk = chunk_tokens(d), chunks = ((size_t)T + chunk - 1) / chunk;
    if (T <= kStepTokens || heads > chunk_heads(d.dk)) return 0;
    // segment_tokens gives at most min(want, chunks) segments; that bound grows with T
    const size_t segs = min(segments_wanted(heads, chunks, d.dk), chunks);
    return segs <= 1 ? 0 : segs * heads * ((size_t)d.dk * d.dv + 4) * sizeof(float);
}

hipError_t launch_la_prefill(const lq_dims& d, const float* h0, float* h, int T, const void* q, const void* k,
                             const void* v, const float* alpha, bool alpha_heads, const int32_t* lens, void* o,
                             void* workspace, hipStream_t s) {
    LaPrefillArgs args{h0, h, q, k, v, alpha, lens, o, T, d.H, d.B * d.H, alpha_heads ? 0 : d.B * d.H};
    switch (d.dk) {
        case 16: return la_prefill_d<16>(d, args, workspace, s);
        case 64: return la_prefill_d<64>(d, args, workspace, s);
        default: return la_prefill_d<128>(d, args, workspace, s);
    }
}

}  // namespace lq

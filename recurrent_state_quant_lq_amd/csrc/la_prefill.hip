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
// One workgroup per (b, h); NW waves, wave w owns the columns
// [w*DV/NW, (w+1)*DV/NW) of H in v_mfma_f32_16x16x4_f32 accumulator tiles
// (tile (rt, ct): rows rt*16 + 4*(lane/16) + v, column lane%16), so the state
// stays in registers from the first load to the final store.  Its accumulator
// layout is the B operand of the next products with the K index in register
// order, so no value of H or V moves between lanes.
#include "lq_internal.h"

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

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

constexpr int CL = 16;        // tokens per chunk (the MFMA tile)

template <int D>
struct LP {
    static constexpr int NW = D / 16 < 4 ? D / 16 : 4;     // waves
    static constexpr int NT = 64 * NW;
    static constexpr int RT = D / 16;                      // row tiles
    static constexpr int CTW = D / 16 / NW;                // column tiles per wave
    static constexpr int DP = D + 4;                       // padded LDS row (banks 4n + c)
};

template <int D, typename TI>
__global__ __launch_bounds__(LP<D>::NT) void la_prefill_kernel(LaPrefillArgs a) {
    using P = LP<D>;
    constexpr int NT = P::NT, RT = P::RT, CTW = P::CTW, DP = P::DP;
    __shared__ __align__(16) float sQ[CL * DP];
    __shared__ __align__(16) float sK[CL * DP];
    __shared__ __align__(16) float sV[CL * DP];
    __shared__ __align__(16) float sP[CL * CL];            // E o (Q K^T), lower triangle
    __shared__ double sG[CL];                              // chunk-local log-decay prefix

    const int t = threadIdx.x;
    const int lane = t & 63, li = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const size_t head = blockIdx.x, heads = (size_t)a.heads;
    const int hh = (int)(head % (unsigned)a.H);
    const int T = a.lens ? min(max(a.lens[head / (unsigned)a.H], 0), a.T) : a.T;

    const size_t hoff = head * (size_t)D * D;
    v4f H[RT][CTW];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CTW; ++ct)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                H[rt][ct][v] = a.h0 ? a.h0[hoff + (size_t)(rt * 16 + 4 * lg + v) * D + (w * CTW + ct) * 16 + li] : 0.0f;

    for (int c0 = 0; c0 < T; c0 += CL) {
        const int L = min(CL, T - c0);                     // tokens of this chunk; the rows past it are zeros
        for (int e = t; e < CL * D; e += NT) {
            const int n = e / D, c = e % D;
            const size_t at = ((size_t)(c0 + n) * heads + head) * D + c;
            sQ[n * DP + c] = n < L ? tok_ld<TI>(a.q, at) : 0.0f;
            sK[n * DP + c] = n < L ? tok_ld<TI>(a.k, at) : 0.0f;
            sV[n * DP + c] = n < L ? tok_ld<TI>(a.v, at) : 0.0f;
        }
        if (t == 0) {
            double g = 0.0;
            for (int n = 0; n < CL; ++n) {
                if (n < L) g += (double)log_decay(a.alpha_tok ? a.alpha[(size_t)(c0 + n) * a.alpha_tok + head] : a.alpha[hh]);
                sG[n] = g;
            }
        }
        __syncthreads();
        if (w == 0 && a.o) {
            // P[n][i] = E_{n,i} <q_n, k_i>
            v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int ks = 0; ks < D / 4; ++ks)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(sQ[li * DP + 4 * ks + lg], sK[li * DP + 4 * ks + lg], acc, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int n = 4 * lg + v, i = li;
                sP[n * CL + i] = i <= n ? expf((float)(sG[n] - sG[i])) * acc[v] : 0.0f;
            }
        }
        __syncthreads();
        const float eg = expf((float)sG[li]);              // rows of HQ: token li
        const float egl = expf((float)sG[CL - 1]);
        float ekt[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) ekt[v] = expf((float)(sG[CL - 1] - sG[4 * lg + v]));
#pragma unroll
        for (int ct = 0; ct < CTW; ++ct) {
            const int col = (w * CTW + ct) * 16 + li;
            float vv[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) vv[v] = sV[(4 * lg + v) * DP + col];
            if (a.o) {
                v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    float aq[4];
                    load_floats<4>(sQ + li * DP + rt * 16 + 4 * lg, aq);
#pragma unroll
                    for (int v = 0; v < 4; ++v) o = __builtin_amdgcn_mfma_f32_16x16x4f32(aq[v] * eg, H[rt][ct][v], o, 0, 0, 0);
                }
                // a non-finite v would reach earlier tokens as 0 * v: left out here, added below
                bool odd = false;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    odd |= !finite_f32(vv[v]);
                    o = __builtin_amdgcn_mfma_f32_16x16x4f32(sP[li * CL + 4 * lg + v], finite_f32(vv[v]) ? vv[v] : 0.0f, o, 0, 0, 0);
                }
                if (__any(odd))
                    for (int i = 0; i < L; ++i) {
                        const float x = sV[i * DP + col];
                        if (!finite_f32(x))
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                if (4 * lg + v >= i) o[v] += sP[(4 * lg + v) * CL + i] * x;
                    }
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (4 * lg + v < L) tok_st<TI>(a.o, ((size_t)(c0 + 4 * lg + v) * heads + head) * D + col, o[v]);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                H[rt][ct] *= egl;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    H[rt][ct] = __builtin_amdgcn_mfma_f32_16x16x4f32(sK[(4 * lg + v) * DP + rt * 16 + li] * ekt[v], vv[v],
                                                                     H[rt][ct], 0, 0, 0);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CTW; ++ct)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                a.h[hoff + (size_t)(rt * 16 + 4 * lg + v) * D + (w * CTW + ct) * 16 + li] = H[rt][ct][v];
}

template <int D>
hipError_t la_prefill_t(const lq_dims& d, const LaPrefillArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H);
    if (d.io_dtype == LQ_IO_BF16)
        return launch_kernel(LQ_KERNEL_LA_PREFILL, la_prefill_kernel<D, uint16_t>, grid, dim3(LP<D>::NT), s, args);
    return launch_kernel(LQ_KERNEL_LA_PREFILL, la_prefill_kernel<D, float>, grid, dim3(LP<D>::NT), s, args);
}

}  // namespace

size_t la_workspace_bytes(const lq_dims& d, int T) {
    (void)d;
    (void)T;
    return 0;
}

hipError_t launch_la_prefill(const lq_dims& d, const float* h0, float* h, int T, const void* q, const void* k,
                             const void* v, const float* alpha, bool alpha_heads, const int32_t* lens, void* o,
                             void* workspace, hipStream_t s) {
    (void)workspace;
    LaPrefillArgs args{h0, h, q, k, v, alpha, lens, o, T, d.H, d.B * d.H, alpha_heads ? 0 : d.B * d.H};
    switch (d.dk) {
        case 16: return la_prefill_t<16>(d, args, s);
        case 64: return la_prefill_t<64>(d, args, s);
        default: return la_prefill_t<128>(d, args, s);
    }
}

}  // namespace lq

// gdn_prefill.hip -- the gated delta rule over a padded batch of prompts (gfx950).
//
//     H <- (I - beta k k^T) D H + beta k v^T,   o = H^T q  (after the update),
// D = alpha I or diag(alpha).
#include "gdn.h"
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

template <int D, bool KDA, typename TI>
hipError_t gdn_prefill_t(const lq_dims& d, const GdnPrefillArgs& args, void* workspace, hipStream_t s) {
    const dim3 grid((unsigned)args.heads);
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

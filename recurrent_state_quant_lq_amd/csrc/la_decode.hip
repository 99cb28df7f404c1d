// la_decode.hip -- one token of linear attention over the int8 state (gfx950).
//
// Slot n = pos of the window becomes (k, g_n, v), g_n = g_{n-1} + log alpha, and
//     o = Hb^T (e^{g_n} q) + sum_{i<n} exp(g_n - g_i) <q, k_i> m_i + <q, k> v,
// Hb^T x = s o (sq^T (r o x)) + sum_c x[idx_c] cv_c, with the window-base state Hb
// fixed for the window.  The window's slots have the form the delta rule leaves
// (m_i = v_i here), so the flush is shared.
//
// One workgroup per (b, h), lane j = channel j = value column j.
#include "lq_internal.h"

namespace lq {
namespace {

struct LaDecodeArgs {
    const int8_t* sq;
    const float* r;
    const float* s;
    const int32_t* idx;
    const float* cv;
    float* bk;
    float* bm;
    float* bg;
    const void* q;            // q, k, v, o: fp32 or bf16 (the kernel's TI)
    const void* k;
    const void* v;
    const float* alpha;
    void* o;
    const int32_t* pos_dev;   // per batch row, or null: pos
    int alpha_heads;          // alpha is [H]
    int W, C, H, pos;
};

template <int D, typename TI>
__global__ __launch_bounds__((D < 64 ? 64 : D)) void la_decode_kernel(LaDecodeArgs a) {
    constexpr int NT = D < 64 ? 64 : D, NW = NT / 64;
    __shared__ __align__(16) float sx[D];                  // r o e^{g_n} o q
    __shared__ float sq_[D], sk_[D];
    __shared__ float sa[33];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    const size_t head = blockIdx.x;
    const int W = a.W, C = a.C;
    const int n = a.pos_dev ? a.pos_dev[head / (unsigned)a.H] : a.pos;
    if (n < 0 || n >= W) return;                           // a row outside its window: untouched
    const float g = (n > 0 ? a.bg[head * W + n - 1] : 0.0f) + log_decay(a.alpha[a.alpha_heads ? head % (unsigned)a.H : head]);
    const float e = expf(g);
    if (t < D) {
        sq_[t] = tok_ld<TI>(a.q, head * D + t);
        sk_[t] = tok_ld<TI>(a.k, head * D + t);
        sx[t] = a.r[head * D + t] * (e * sq_[t]);
    }
    __syncthreads();
    for (int i = w; i <= n; i += NW) {
        float x = 0.0f;
        for (int c = lane; c < D; c += 64) x += sq_[c] * (i < n ? a.bk[(head * W + i) * D + c] : sk_[c]);
        x = group_sum<64>(x);
        if (lane == 0) sa[i] = i < n ? x * expf(g - a.bg[head * W + i]) : x;
    }
    __syncthreads();
    if (t < D) {
        float o = 0.0f;
        for (int c = 0; c < D; c += 16) {
            const v4i b = *reinterpret_cast<const v4i*>(a.sq + head * (size_t)(D * D) + sq_off<D>(c, t));
#pragma unroll
            for (int u = 0; u < 16; ++u) o += sbyte((uint32_t)b[u / 4], u % 4) * sx[c + u];
        }
        o *= a.s[head * D + t];
        for (int c = 0; c < C; ++c) o += e * sq_[a.idx[head * C + c] & (D - 1)] * a.cv[(head * C + c) * D + t];
        for (int i = 0; i < n; ++i) o += sa[i] * a.bm[(head * W + i) * D + t];
        const float v = tok_ld<TI>(a.v, head * D + t);
        tok_st<TI>(a.o, head * D + t, o + sa[n] * v);
        a.bk[(head * W + n) * D + t] = sk_[t];
        a.bm[(head * W + n) * D + t] = v;
        if (t == 0) a.bg[head * W + n] = g;
    }
}

template <int D>
hipError_t la_decode_t(const lq_dims& d, const LaDecodeArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H), block(D < 64 ? 64 : D);
    if (d.io_dtype == LQ_IO_BF16) return launch_kernel(LQ_KERNEL_LA_DECODE, la_decode_kernel<D, uint16_t>, grid, block, s, args);
    return launch_kernel(LQ_KERNEL_LA_DECODE, la_decode_kernel<D, float>, grid, block, s, args);
}

}  // namespace

hipError_t launch_la_decode(const lq_dims& d, const lq_state& st, int pos, const int32_t* pos_dev, const void* q,
                            const void* k, const void* v, const float* alpha, bool alpha_heads, void* o,
                            hipStream_t s) {
    LaDecodeArgs args{st.sq, st.row_scale, st.col_scale, st.comp_idx, st.comp_val, st.buf_k, st.buf_m, st.buf_g,
                      q, k, v, alpha, o, pos_dev, alpha_heads, d.W, d.C, d.H, pos};
    switch (d.dk) {
        case 16: return la_decode_t<16>(d, args, s);
        case 64: return la_decode_t<64>(d, args, s);
        default: return la_decode_t<128>(d, args, s);
    }
}

}  // namespace lq

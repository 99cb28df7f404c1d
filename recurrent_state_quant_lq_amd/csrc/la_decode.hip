// la_decode.hip -- one token of linear attention over the int8 state (gfx950).
//
// Slot n = pos of the window becomes (k, g_n, v), g_n = g_{n-1} + log alpha, and
//     o = Hb^T (e^{g_n} q) + sum_{i<n} exp(g_n - g_i) <q, k_i> m_i + <q, k> v,
// Hb^T x = s o (sq^T (r o x)) + sum_c x[idx_c] cv_c, with the window-base state Hb
// fixed for the window.  The window's slots have the form the delta rule leaves
// (m_i = v_i here), so the flush is shared.
//
// One workgroup per (b, h), lane j = channel j = value column j (two waves at d = 128).
// A launch reads about 1.2 bytes of state per element once and does two operations on
// each, so it is bound by memory: every load is requested before the first is used (the
// state and scales at once, the window as soon as pos is known), and a workgroup holds
// few registers and little LDS, so that ten of them share a CU.  The products with the
// state run on the vector unit: a lane's column times the query in LDS (broadcast reads).
// d = 128, 8192 heads, bf16: 39 us, 6.2 TB/s (a plain read of as many bytes: 6.1); 67 us with
// the loads where they are used.
#include "la.h"

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

template <int D, int WM, typename TI>
__global__ __launch_bounds__((D < 64 ? 64 : D)) void la_decode_kernel(LaDecodeArgs a) {
    constexpr int NT = D < 64 ? 64 : D, NW = NT / 64;
    constexpr int LPS = D < 64 ? D : 64, CPL = D / LPS;    // lanes per slot of the dot products, channels per lane
    constexpr int SPR = NT / LPS, ROUNDS = (WM + SPR - 1) / SPR;   // slots per round
    __shared__ __align__(16) float sx[D];                  // r o e^{g_n} o q
    __shared__ __align__(16) float s_q[D], s_k[D];
    __shared__ float sa[WM + 1];
    const int t = threadIdx.x;
    const size_t head = blockIdx.x;
    const int W = a.W, C = a.C, ch = t & (D - 1);
    // requests that depend on nothing
    const int n = a.pos_dev ? a.pos_dev[head / (unsigned)a.H] : a.pos;
    const float al = a.alpha[a.alpha_heads ? head % (unsigned)a.H : head];
    const TI q_raw = static_cast<const TI*>(a.q)[head * D + ch], k_raw = static_cast<const TI*>(a.k)[head * D + ch];
    const TI v_raw = static_cast<const TI*>(a.v)[head * D + ch];
    const float r = a.r[head * D + ch], sj = a.s[head * D + ch];
    v4i raw[D / 16];                                       // the column's bytes
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
        raw[c] = ld_nt(reinterpret_cast<const v4i*>(a.sq + head * (size_t)(D * D) + sq_off<D>(16 * c, ch)));
    float cv[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c < C) cv[c] = a.cv[(head * C + c) * D + ch];
    if (n < 0 || n >= W) return;                           // a row outside its window: untouched
    const float* bk = a.bk + head * (size_t)W * D;
    const float* bm = a.bm + head * (size_t)W * D;
    const float* bg = a.bg + head * (size_t)W;
    const int slot0 = t / LPS, c0 = CPL * (t % LPS), last = max(n - 1, 0);
    float kk[ROUNDS][CPL], gs[ROUNDS], m[WM];
#pragma unroll
    for (int rd = 0; rd < ROUNDS; ++rd)
        if (rd * SPR < n) {
            const int i = min(rd * SPR + slot0, last);     // (past the last slot: that slot again, unused)
            gs[rd] = bg[i];
#pragma unroll
            for (int c = 0; c < CPL; ++c) kk[rd][c] = bk[(size_t)i * D + c0 + c];
        }
#pragma unroll
    for (int i = 0; i < WM; ++i)
        if (i < n) m[i] = ld_nt(bm + (size_t)i * D + ch);
    const float g = (n > 0 ? bg[last] : 0.0f) + log_decay(al), e = expf(g);
    const auto widen = [](TI x) { if constexpr (sizeof(TI) == 4) return x; else return bf16_to_f32(x); };
    const float q = widen(q_raw), k = widen(k_raw), v = widen(v_raw);
    if (t < D) {
        s_q[t] = q;
        s_k[t] = k;
        sx[t] = r * (e * q);
    }
    __syncthreads();
    // a_i = exp(g_n - g_i) <q, k_i>, a_n = <q, k>
    {
        float ql[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) ql[c] = s_q[c0 + c];
#pragma unroll
        for (int rd = 0; rd < ROUNDS; ++rd)
            if (rd * SPR <= n) {
                const int i = rd * SPR + slot0;
                float x = 0.0f;
#pragma unroll
                for (int c = 0; c < CPL; ++c) x += ql[c] * (i < n ? kk[rd][c] : s_k[c0 + c]);
                x = group_sum<LPS>(x);
                if (t % LPS == 0 && i <= n) sa[i] = i < n ? x * expf(g - gs[rd]) : x;
            }
    }
    float o = 0.0f, o2 = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        float x[16];
        load_floats<16>(sx + 16 * c, x);
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
            o = __builtin_fmaf(sbyte((uint32_t)raw[c][u / 4], u % 4), x[u], o);
            o2 = __builtin_fmaf(sbyte((uint32_t)raw[c][u / 4], u % 4 + 1), x[u + 1], o2);
        }
    }
    o = (o + o2) * sj;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c < C) o = __builtin_fmaf(e * s_q[a.idx[head * C + c] & (D - 1)], cv[c], o);
    __syncthreads();
    float y = sa[n] * v;
#pragma unroll
    for (int i = 0; i < WM; ++i)
        if (i < n) y = __builtin_fmaf(sa[i], m[i], y);
    if (t < D) {
        tok_st<TI>(a.o, head * D + t, o + y);
        st_nt(a.bk + (head * W + n) * D + t, k);
        st_nt(a.bm + (head * W + n) * D + t, v);
        if (t == 0) a.bg[head * W + n] = g;
    }
}

template <int D, int WM>
hipError_t la_decode_w(const lq_dims& d, const LaDecodeArgs& args, hipStream_t s) {
    const dim3 grid((unsigned)d.B * (unsigned)d.H), block(D < 64 ? 64 : D);
    if (d.io_dtype == LQ_IO_BF16) return launch_kernel(LQ_KERNEL_LA_DECODE, la_decode_kernel<D, WM, uint16_t>, grid, block, s, args);
    return launch_kernel(LQ_KERNEL_LA_DECODE, la_decode_kernel<D, WM, float>, grid, block, s, args);
}
template <int D>
hipError_t la_decode_t(const lq_dims& d, const LaDecodeArgs& args, hipStream_t s) {
    return d.W <= 8 ? la_decode_w<D, 8>(d, args, s) : d.W <= 16 ? la_decode_w<D, 16>(d, args, s) : la_decode_w<D, 32>(d, args, s);
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

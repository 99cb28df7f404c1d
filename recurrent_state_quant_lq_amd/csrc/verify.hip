// verify.hip -- drafted trees against the target's probabilities (gfx950).
//
// For a row, from the root on: the children of the current node x are tested in the order of
// their indices.  With p the target's and q the draft's distribution after x, and after r
// rejections
//     p_r(t) = max(p(t) - c_r q(t), 0) / S_r,   S_r = sum_t max(p(t) - c_r q(t), 0),
//     q_r(t) = q(t) / Z_r on the tokens that were not rejected,
//     c_0 = 0, S_0 = Z_0 = 1,   c_{r+1} = c_r + S_r / Z_r,   Z_{r+1} = Z_r - q(rejected)
// (drafted with replacement: Z_r = 1), child token t is accepted if u q_r(t) < p_r(t).  This
// is the recursion p_{r+1} = max(p_r - q_r, 0) / its sum, since max(max(a, 0) - b, 0) =
// max(a - b, 0) for b >= 0; a rejected token has p_r(t) < q_r(t), so it drops out of every later
// p by itself.  Without draft probabilities q is 1 at the child's token: u S < p(t), and a
// rejection takes t out of p.  Where the walk ends, the next token is drawn from p_r by its
// distribution function.
//
// Everything after the loads is in 64 bits: the sums' order then moves a border by 2^-50 of it,
// and the nodes' numbers are compared as they are.
//
// A row of p (and q) is read where a sum is needed: after a rejection (S of the next test, or
// the total of the draw) and for the draw.  Each launch of verify_sum_kernel covers the next
// sum of every row, a tile of a row per workgroup, and walks on from the sums before it (the walk
// is a few comparisons, so every wave repeats it); verify_pick_kernel, one workgroup a row, forms
// what sums are left by itself, finds the tile and the token.
#include "gdn.h"

#pragma clang fp contract(off)

namespace lq {
namespace {

constexpr int VT = 256;                  // threads
constexpr int VQ = 4;                    // quads of values per thread
constexpr int TV = VT * VQ * 4;          // values per tile

int verify_tiles(int V) { return (V + TV - 1) / TV; }
constexpr int kVerifyRounds = 1;

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

struct Walk {
    double c, S, Z;
    uint64_t rej;             // children of cur rejected so far
    int cur, len, last;
    bool summed;              // S is the sum over the current residual
};

// One row's nodes, lane n = node n, as every wave holds them.
struct Nodes {
    int parent, token;        // parent -2: no such node
    double u, p, q;
    uint64_t line;            // accepted nodes
    int limit;
    int lane;
    bool with_draft, with_root, replace;
};

__device__ __forceinline__ int rl(int x, int n) { return __builtin_amdgcn_readlane(x, n); }
__device__ __forceinline__ double rl(double x, int n) {
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = rl((int)(uint32_t)b, n), hi = rl((int)(uint32_t)(b >> 32), n);
    return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ const float* row_of(const float* x, const float* x0, int node, int b, const VerifyArgs& a) {
    return node < 0 ? x0 + (size_t)b * a.V : x + ((size_t)node * a.B + b) * a.V;
}

__device__ __forceinline__ Nodes load_nodes(const VerifyArgs& a, int b, int lane) {
    Nodes s;
    s.lane = lane;
    s.line = 0;
    s.with_draft = a.draft != nullptr;
    s.with_root = a.target0 != nullptr;
    s.replace = a.replace != 0;
    s.limit = min(a.P, a.W - a.pos[b]);
    s.parent = -2;
    s.token = 0;
    s.u = s.p = s.q = 0.0;
    if (lane < a.N) {
        const int par = a.parent[(size_t)b * a.N + lane], t = a.token[(size_t)b * a.N + lane];
        if (par >= -1 && par < lane && t >= 0 && t < a.V) {
            s.parent = par;
            s.token = t;
            s.u = (double)a.u[(size_t)lane * a.B + b];
            if (par >= 0 || s.with_root) {
                s.p = (double)row_of(a.target, a.target0, par, b, a)[t];
                if (s.with_draft) s.q = (double)row_of(a.draft, a.draft0, par, b, a)[t];
            }
        }
    }
    return s;
}

__device__ __forceinline__ Walk start_walk() { return Walk{0.0, 1.0, 1.0, 0, -1, 0, -1, false}; }

// Walks on until a sum over the current residual is needed for the next test (true) or no
// child is left to test (false).
__device__ __forceinline__ bool walk_on(Nodes& s, Walk& x) {
    for (;;) {
        const bool chosen = x.cur < 0 && !s.with_root;
        uint64_t kids = 0;
        if (x.len < s.limit && x.S > 0.0 && x.Z > 0.0) {
            kids = __ballot(s.parent == x.cur);
            kids &= x.last < 0 ? ~0ull : x.last >= 63 ? 0ull : ~0ull << (x.last + 1);
        }
        if (!kids) return false;
        if (s.with_draft && x.rej && !x.summed) return true;
        const int n = __ffsll((unsigned long long)kids) - 1;
        x.last = n;
        const int t = rl(s.token, n);
        const double u = rl(s.u, n);
        double p = rl(s.p, n);
        const double q = rl(s.q, n);
        const bool again = (__ballot(s.token == t) & x.rej) != 0;    // a token rejected here before
        bool ok = chosen;
        if (!chosen) {
            if (s.with_draft) {
                const double y = p - x.c * q;
                ok = u * q * x.S < (y > 0.0 ? y : 0.0) * x.Z;
            } else {
                if (again) p = 0.0;
                ok = u * x.S < p;
            }
        }
        if (ok) {
            s.line |= 1ull << n;
            x = Walk{0.0, 1.0, 1.0, 0, n, x.len + 1, n, false};
            continue;
        }
        x.rej |= 1ull << n;
        if (s.with_draft) {
            x.c = x.c + x.S / x.Z;
            if (!s.replace && !again) x.Z = x.Z - q;
            x.summed = false;
        } else {
            x.S = x.S - p;
        }
    }
}

// What the sum that the walk needs next runs over.
struct Residual {
    const float* p;
    const float* q;           // null: c = 0
    double c;
    uint64_t out;             // nodes whose tokens are left out
};
__device__ __forceinline__ Residual residual(const VerifyArgs& a, const Nodes& s, const Walk& x, int b) {
    Residual r;
    const bool left = x.S > 0.0;                           // (nothing left: the target as it is)
    r.p = row_of(a.target, a.target0, x.cur, b, a);
    r.q = s.with_draft && left && x.rej ? row_of(a.draft, a.draft0, x.cur, b, a) : nullptr;
    r.c = x.c;
    r.out = !s.with_draft && left ? x.rej : 0;
    return r;
}

// The residual's values of this thread in a tile.
__device__ __forceinline__ void tile_values(const Residual& r, const Nodes& s, int V, int tile, int t, double (&w)[VQ * 4]) {
    const int base = tile * TV;
#pragma unroll
    for (int j = 0; j < VQ; ++j) {
        const int at = base + (j * VT + t) * 4;
        float p[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
        if (at + 4 <= V) {
            const f4u x = *reinterpret_cast<const f4u*>(r.p + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = x[e];
            if (r.q) {
                const f4u y = *reinterpret_cast<const f4u*>(r.q + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + e < V) {
                    p[e] = r.p[at + e];
                    if (r.q) q[e] = r.q[at + e];
                }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double y = r.q ? (double)p[e] - r.c * (double)q[e] : (double)p[e];
            w[4 * j + e] = y > 0.0 ? y : 0.0;              // (NaN: nothing)
        }
    }
    for (uint64_t m = r.out; m; m &= m - 1) {
        const int off = rl(s.token, __ffsll((unsigned long long)m) - 1) - base;
        if (off < 0 || off >= TV) continue;
#pragma unroll
        for (int j = 0; j < VQ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (off == (j * VT + t) * 4 + e) w[4 * j + e] = 0.0;
    }
}

// Sum over the workgroup, the same in every thread; s_x: one value a wave.
__device__ __forceinline__ double block_sum(double x, double* s_x) {
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
    if ((threadIdx.x & 63) == 0) s_x[threadIdx.x >> 6] = x;
    __syncthreads();
    double y = 0.0;
#pragma unroll
    for (int i = 0; i < VT / 64; ++i) y += s_x[i];
    __syncthreads();
    return y;
}

__device__ __forceinline__ double tile_sum(const Residual& r, const Nodes& s, int V, int tile, double* s_x) {
    double w[VQ * 4], x = 0.0;
    tile_values(r, s, V, tile, threadIdx.x, w);
#pragma unroll
    for (int e = 0; e < VQ * 4; ++e) x += w[e];
    return block_sum(x, s_x);
}

// Sum of a row's tiles, the same in every wave.
__device__ __forceinline__ double row_sum(const double* tiles, int n, int lane) {
    double x = 0.0;
    for (int i = lane; i < n; i += 64) x += tiles[i];
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
    return x;
}

// Walks through the sums of the rounds before `rounds`.  Returns whether the walk needs another
// sum: for a test, or (done) for the draw.
__device__ __forceinline__ bool replay(const VerifyArgs& a, Nodes& s, Walk& x, int b, int rounds, int& used, bool& done) {
    const int tiles = (a.V + TV - 1) / TV;
    for (used = 0;;) {
        done = !walk_on(s, x);
        if (done && ((x.summed && x.S > 0.0) || (x.cur < 0 && !s.with_root))) return false;
        if (used == rounds) return true;
        const double S = row_sum(a.sums + ((size_t)used * a.B + b) * tiles, tiles, s.lane);
        ++used;
        if (done) {                                        // the draw's total
            x.summed = true;
            return false;
        }
        x.S = S;
        x.summed = true;
    }
}

__global__ __launch_bounds__(VT) void verify_sum_kernel(VerifyArgs a, int round) {
    __shared__ double s_x[VT / 64];
    const int tiles = (a.V + TV - 1) / TV;
    const int b = blockIdx.x / (unsigned)tiles, tile = blockIdx.x % (unsigned)tiles, lane = threadIdx.x & 63;
    const int pos = a.pos[b];
    if (pos < 0 || pos > a.W) return;
    Nodes s = load_nodes(a, b, lane);
    Walk x = start_walk();
    int used;
    bool done;
    if (!replay(a, s, x, b, round, used, done)) return;
    const double y = tile_sum(residual(a, s, x, b), s, a.V, tile, s_x);
    if (threadIdx.x == 0) a.sums[((size_t)round * a.B + b) * tiles + tile] = y;
}

__global__ __launch_bounds__(VT) void verify_pick_kernel(VerifyArgs a) {
    __shared__ double s_x[VT / 64];
    __shared__ int s_tile;
    __shared__ double s_base;
    __shared__ int s_pick[VT / 64], s_pos[VT / 64];
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 63, w = t >> 6;
    const int pos = a.pos[b];
    if (pos < 0 || pos > a.W) return;
    const int tiles = (a.V + TV - 1) / TV;
    Nodes s = load_nodes(a, b, lane);
    Walk x = start_walk();
    int used;
    bool done;
    const bool more = replay(a, s, x, b, kVerifyRounds, used, done);
    double* sums = a.sums + ((size_t)(used > 0 ? used - 1 : 0) * a.B + b) * tiles;
    if (more) {                                            // sums beyond the rounds: this workgroup alone
        sums = a.sums + ((size_t)(kVerifyRounds - 1) * a.B + b) * tiles;
        for (;;) {
            const Residual r = residual(a, s, x, b);
            for (int i = 0; i < tiles; ++i) {
                const double y = tile_sum(r, s, a.V, i, s_x);
                if (t == 0) sums[i] = y;
            }
            __threadfence_block();
            __syncthreads();
            if (done) break;
            x.S = row_sum(sums, tiles, lane);
            x.summed = true;
            __syncthreads();
            done = !walk_on(s, x);
            if (done && x.summed && x.S > 0.0) break;
        }
    }
    // the accepted nodes' indices grow along the path
    if (t < a.P) {
        int n = -1;
        uint64_t m = s.line;
        for (int i = 0; m; ++i, m &= m - 1)
            if (i == t) n = __ffsll((unsigned long long)m) - 1;
        a.path[(size_t)b * a.P + t] = n;
    }
    if (t == 0) a.n_path[b] = x.len;
    if (x.cur < 0 && !s.with_root) {
        if (t == 0) a.next[b] = -1;
        return;
    }
    // ---- the draw: the tile, then the token ----
    if (w == 0) {
        const double total = row_sum(sums, tiles, lane);
        const double theta = (double)a.u[(size_t)a.N * a.B + b] * total;
        double before = 0.0;
        int tile = -1, last = -1;
        double base = 0.0, lbase = 0.0;
        for (int i0 = 0; i0 < tiles && tile < 0; i0 += 64) {
            const int i = i0 + lane;
            const double y = i < tiles ? sums[i] : 0.0;
            double c = y;                                   // inclusive prefix sums
            for (int m = 1; m < 64; m <<= 1) {
                const double z = __shfl_up(c, m, 64);
                if (lane >= m) c += z;
            }
            c += before;
            const uint64_t over = __ballot(c > theta && y > 0.0), some = __ballot(y > 0.0);
            if (some) {
                const int n = 63 - __clzll((long long)some);
                last = i0 + n;
                lbase = rl(c, n) - rl(y, n);
            }
            if (over) {
                const int n = __ffsll((unsigned long long)over) - 1;
                tile = i0 + n;
                base = rl(c, n) - rl(y, n);
            }
            before = rl(c, 63);
        }
        if (tile < 0) {                                     // (rounding, or a number of 1 and more)
            tile = last;
            base = lbase;
        }
        if (lane == 0) {
            s_tile = total > 0.0 ? tile : -1;
            s_base = theta - base;
        }
    }
    __syncthreads();
    if (s_tile < 0) {
        if (t == 0) a.next[b] = -1;
        return;
    }
    // values of the tile in index order: quad j of thread t holds 4 (256 j + t) ..
    double v[VQ * 4];
    tile_values(residual(a, s, x, b), s, a.V, s_tile, t, v);
    double before = 0.0;
    const double theta = s_base;
    int pick = -1, last = -1;
#pragma unroll
    for (int j = 0; j < VQ; ++j) {
        const double mine = ((v[4 * j] + v[4 * j + 1]) + v[4 * j + 2]) + v[4 * j + 3];
        double c = mine;
        for (int m = 1; m < 64; m <<= 1) {
            const double z = __shfl_up(c, m, 64);
            if (lane >= m) c += z;
        }
        if (lane == 63) s_x[w] = c;
        __syncthreads();
        double wave0 = before, all = before;
#pragma unroll
        for (int i = 0; i < VT / 64; ++i) {
            if (i < w) wave0 += s_x[i];
            all += s_x[i];
        }
        __syncthreads();
        double y = wave0 + (c - mine);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y += v[4 * j + e];
            if (v[4 * j + e] > 0.0) {
                const int at = s_tile * TV + (j * VT + t) * 4 + e;
                if (pick < 0 && y > theta) pick = at;
                last = at;
            }
        }
        before = all;
    }
    // the smallest index past theta, or the largest one that has a share
    int lo = pick < 0 ? INT32_MAX : pick;
    for (int m = 1; m < 64; m <<= 1) {
        lo = min(lo, __shfl_xor(lo, m, 64));
        last = max(last, __shfl_xor(last, m, 64));
    }
    if (lane == 0) {
        s_pick[w] = lo;
        s_pos[w] = last;
    }
    __syncthreads();
    if (t == 0) {
#pragma unroll
        for (int i = 1; i < VT / 64; ++i) {
            lo = min(lo, s_pick[i]);
            last = max(last, s_pos[i]);
        }
        a.next[b] = lo == INT32_MAX ? last : lo;
    }
}

}  // namespace

size_t verify_workspace_bytes(int B, int N, int V) {
    return (size_t)kVerifyRounds * B * verify_tiles(V) * sizeof(double);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
    for (int r = 0; r < kVerifyRounds; ++r) {
        const hipError_t e = launch_kernel(LQ_KERNEL_VERIFY, verify_sum_kernel, dim3((unsigned)verify_tiles(a.V) * (unsigned)a.B),
                                           dim3(VT), s, a, r);
        if (e != hipSuccess) return e;
    }
    return launch_kernel(LQ_KERNEL_VERIFY, verify_pick_kernel, dim3(a.B), dim3(VT), s, a);
}

}  // namespace lq

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
// rejection takes t out of p and of S.  Where the walk ends, the next token is drawn from p_r by its
// distribution function; if no value of p_r is positive, from p (without draft probabilities S is 1 less
// the rejected values, so that where a row sums to less than 1 it stays above 0 when all of them are).
//
// Everything after the loads is in 64 bits: the sums' order then moves a border by 2^-50 of it,
// and the nodes' numbers are compared as they are.
//
// A row of p (and q) is read where a sum is needed: after a rejection (S of the next test, or
// the total of the draw) and for the draw.  verify_sum_kernel walks every row to its first sum and
// forms it, a tile of the row per wave (the walk is a few comparisons, so every wave repeats it).
// verify_pick_kernel, one workgroup a row, forms what sums are left, finds the tile and the token; with many
// or small rows it does all of it (kAloneRows).
// Bound by the sum's reads and by the latencies before them (positions and nodes, the nodes'
// values, the row): 64 rows of 131072 values with a draft 11 us and 7 for the pick (the rows partly in the
// Infinity Cache), one row of 32000 5.5 and 6.3; alone, 256 rows of 50021 without a draft 18 (two
// launches: 14 and 7), 51 MB in all, waits 0.6 of the waves' time.  Nodes with several children need a sum for each
// rejection, one after the other, on one CU: both rows at its 64 bytes a cycle, and as long again eight vector
// operations a value beside that.  Trees of 32 nodes, 64 rows, 28 to 55 us by what is rejected (drafted without
// replacement; the first sum 11 of them), 57 to 91 (with).  One and two further launches of the sum kernel before the pick took 66 and 75 us, not 61,
// there (102 and 105, not 95), and the pick's sums with 256 threads 127, not 105.  A quad of a row is loaded
// without a bounds test where its whole tile is inside (24 us, not 9, with one per quad).
#include "gdn.h"

#pragma clang fp contract(off)

namespace lq {
namespace {

constexpr int VT = 256;                  // threads of a sum's workgroup
constexpr int PT = 1024;                 // of a pick's: its own sums need as many loads in flight as a CU takes
constexpr int VQ = 8;                    // quads of values per lane and tile
constexpr int TV = 64 * VQ * 4;          // values per tile: one wave's

// verify_pick_kernel alone: one launch less, a row's first sum by one workgroup.  It pays with a workgroup for every
// CU, and with rows so small that a workgroup's reads take no longer than a launch.  Calls with two launches and
// with one, us, 8 nodes with a draft / 5 without: 1 row of 4000 values 13.2, 11.6 / 13.1, 11.4; of 16000 13.5,
// 12.2 / 12.8, 11.1; of 32000 13.1, 13.4 / 13.7, 11.8; of 65536 14.4, 14.5 / 14.1, 12.4; of 131072 14.5, 20.0 /
// 14.2, 16.6; 64 rows of 32000 16.5, 16.7 / 15.6, 14.6; of 65536 16.9, 18.8 / 15.8, 14.5; of 131072 21.3, 23.3 /
// 17.7, 19.1; 256 rows of 32000 23.0, 19.9 / 19.9, 18.3; of 65536 31.1, 26.3 / 25.2, 20.1; of 131072 51.8,
// 49.2 / 34.4, 29.1.
constexpr int kAloneRows = 256, kAloneValues = 1 << 16;     // values of a row; with a draft a quarter
int verify_tiles(int V) { return (V + TV - 1) / TV; }
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

struct Walk {
    double c, S, Z;
    uint64_t rej;             // children of cur rejected so far
    uint64_t line;            // accepted nodes
    int cur, len, last;
    bool summed;              // S is the sum over the current residual
};
// A row's walk between the launches.
enum WalkState { W_TEST, W_DRAW, W_NONE, W_SKIP };   // waits for a sum for a test, for the draw; no draw; not a row
struct Saved {
    Walk x;
    int state, pad;
};

// One row's nodes, lane n = node n, as every wave holds them.
struct Nodes {
    int parent, token;        // parent -2: no such node
    double u, p, q;
    int limit;
    int lane;
    bool with_draft, with_root, replace;
    bool live;                // the row's position is one of the window's
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

// A probability: NaN and what is below 0 count as 0 (a median with NaN is the minimum of the other two).
__device__ __forceinline__ float prob(float x) { return __builtin_amdgcn_fmed3f(x, 0.0f, __builtin_inff()); }

__device__ __forceinline__ Nodes load_nodes(const VerifyArgs& a, int b, int lane) {
    Nodes s;
    s.lane = lane;
    s.with_draft = a.draft != nullptr;
    s.with_root = a.target0 != nullptr;
    s.replace = a.replace != 0;
    const int n = min(lane, a.N - 1);                      // (requested together)
    const int pos = a.pos[b], par = a.parent[(size_t)b * a.N + n], t = a.token[(size_t)b * a.N + n];
    const float u = a.u[(size_t)n * a.B + b];
    s.limit = min(a.P, a.W - pos);
    s.live = pos >= 0 && pos <= a.W;
    const bool here = lane < a.N && par >= -1 && par < lane && t >= 0 && t < a.V && s.live;
    s.parent = here ? par : -2;
    s.token = here ? t : 0;
    s.u = (double)u;
    s.p = s.q = 0.0;
    if (here && (par >= 0 || s.with_root)) {
        const float p = row_of(a.target, a.target0, par, b, a)[t];
        const float q = s.with_draft ? row_of(a.draft, a.draft0, par, b, a)[t] : 0.0f;
        s.p = (double)prob(p);
        s.q = (double)prob(q);
    }
    return s;
}

__device__ __forceinline__ Walk start_walk() { return Walk{0.0, 1.0, 1.0, 0, 0, -1, 0, -1, false}; }

// Walks on until a sum over the current residual is needed for the next test (true) or no
// child is left to test (false).
__device__ __forceinline__ bool walk_on(const Nodes& s, Walk& x) {
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
            x = Walk{0.0, 1.0, 1.0, 0, x.line | 1ull << n, n, x.len + 1, n, false};
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
    r.c = r.q ? x.c : 0.0;
    r.out = !s.with_draft && left ? x.rej : 0;
    return r;
}

// Value i of quad j of a lane in a tile: rounds of whole lines, or (RUN) a run of neighbours a lane.
template <bool RUN>
__device__ __forceinline__ int value_at(int tile, int j, int lane) { return tile * TV + (RUN ? lane * VQ + j : j * 64 + lane) * 4; }

// p (0 where a token is left out) and q of this lane in a tile.
template <bool RUN>
__device__ __forceinline__ void load_tile(const Residual& r, const Nodes& s, int V, int tile, f4u (&p)[VQ], f4u (&q)[VQ]) {
#pragma unroll
    for (int j = 0; j < VQ; ++j) p[j] = q[j] = f4u{0.f, 0.f, 0.f, 0.f};
    if (tile * TV + TV <= V) {
#pragma unroll
        for (int j = 0; j < VQ; ++j) p[j] = *reinterpret_cast<const f4u*>(r.p + value_at<RUN>(tile, j, s.lane));
        if (r.q)
#pragma unroll
            for (int j = 0; j < VQ; ++j) q[j] = *reinterpret_cast<const f4u*>(r.q + value_at<RUN>(tile, j, s.lane));
    } else {
#pragma unroll
        for (int i = 0; i < VQ * 4; ++i) {
            const int at = value_at<RUN>(tile, i / 4, s.lane) + i % 4;
            if (at < V) p[i / 4][i % 4] = r.p[at];
            if (at < V && r.q) q[i / 4][i % 4] = r.q[at];
        }
    }
    if (r.q)
#pragma unroll
        for (int i = 0; i < VQ * 4; ++i) q[i / 4][i % 4] = prob(q[i / 4][i % 4]);
    uint32_t out = 0;                                      // bit 4 j + e: left out
    for (uint64_t m = r.out; m; m &= m - 1) {
        const int off = rl(s.token, __ffsll((unsigned long long)m) - 1) - tile * TV;
        if (off < 0 || off >= TV) continue;
        const int at = RUN ? off / (4 * VQ) : (off >> 2) & 63, bit = RUN ? off % (4 * VQ) : 4 * (off >> 8) + (off & 3);
        if (s.lane == at) out |= 1u << bit;
    }
    static_assert(VQ * 4 <= 32, "a bit for every value");
    if (__any(out != 0))
#pragma unroll
        for (int i = 0; i < VQ * 4; ++i) p[i / 4][i % 4] = (out >> i) & 1u ? 0.0f : p[i / 4][i % 4];
}
// A value's share, q a probability (load_tile).  One rounding: the sums of several rejections are bound by these
// operations (trees 40.2 us, 41.7 with a product and a difference).
__device__ __forceinline__ double share(const Residual& r, float p, float q) {
    const double y = __builtin_fma(-r.c, (double)q, (double)p);
    return y > 0.0 ? y : 0.0;                              // (p that is NaN: nothing)
}

__device__ __forceinline__ double wave_sum(double x) {
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
    return x;
}

__device__ __forceinline__ double tile_sum(const Residual& r, const Nodes& s, int V, int tile) {
    f4u p[VQ], q[VQ];
    load_tile<false>(r, s, V, tile, p, q);
    double x = 0.0;
#pragma unroll
    for (int j = 0; j < VQ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x += share(r, p[j][e], q[j][e]);
    return wave_sum(x);
}

// Sum of a row's tiles, the same in every wave.
__device__ __forceinline__ double row_sum(const double* tiles, int n, int lane) {
    double x = 0.0;
    for (int i = lane; i < n; i += 64) x += tiles[i];
    return wave_sum(x);
}

__device__ __forceinline__ WalkState state_of(bool test, const Nodes& s, const Walk& x) {
    return test ? W_TEST : x.cur < 0 && !s.with_root ? W_NONE : W_DRAW;
}

// The accepted nodes' indices grow along the path.
__device__ __forceinline__ void write_path(const VerifyArgs& a, const Walk& x, int b, int t) {
    if (t < a.P) {
        uint64_t m = x.line;
        for (int i = 0; i < t; ++i) m &= m - 1;
        a.path[(size_t)b * a.P + t] = m ? __ffsll((unsigned long long)m) - 1 : -1;
    }
    if (t == 0) a.n_path[b] = x.len;
}

__device__ __forceinline__ Saved* saved(const VerifyArgs& a, int tiles, int b) {
    return reinterpret_cast<Saved*>(a.sums + (size_t)a.B * tiles) + b;
}

__global__ __launch_bounds__(VT) void verify_sum_kernel(VerifyArgs a) {
    const int tiles = (a.V + TV - 1) / TV, groups = (tiles + VT / 64 - 1) / (VT / 64);
    const int b = blockIdx.x / (unsigned)groups, group = blockIdx.x % (unsigned)groups;
    const int t = threadIdx.x, lane = t & 63;
    Saved* to = saved(a, tiles, b);
    const bool first = group == 0 && t == 0;
    Walk x = start_walk();
    const Nodes s = load_nodes(a, b, lane);
    if (!s.live) {
        if (first) to->state = W_SKIP;
        return;
    }
    const WalkState state = state_of(walk_on(s, x), s, x);
    if (first) {
        to->x = x;
        to->state = state;
    }
    if (group == 0 && state != W_TEST) write_path(a, x, b, t);
    if (state == W_NONE) return;
    const int tile = group * (VT / 64) + __builtin_amdgcn_readfirstlane(t >> 6);
    if (tile >= tiles) return;
    const double y = tile_sum(residual(a, s, x, b), s, a.V, tile);
    if (lane == 0) a.sums[(size_t)b * tiles + tile] = y;
}

// ALONE: without verify_sum_kernel before it.
template <bool ALONE>
__global__ __launch_bounds__(PT) void verify_pick_kernel(VerifyArgs a) {
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 63;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tiles = (a.V + TV - 1) / TV;
    const Saved* from = saved(a, tiles, b);
    int state = ALONE ? W_SKIP : from->state;
    if (!ALONE && state == W_SKIP) return;
    Walk x = start_walk();
    Nodes s;
    if (ALONE) {
        s = load_nodes(a, b, lane);
        if (!s.live) return;
        state = state_of(walk_on(s, x), s, x);
        if (w == 0 && state != W_TEST) write_path(a, x, b, lane);
    }
    if (state == W_NONE) {
        if (t == 0) a.next[b] = -1;
        return;
    }
    double* sums = a.sums + (size_t)b * tiles;
    if (ALONE) {
        const Residual r = residual(a, s, x, b);
        for (int i = w; i < tiles; i += PT / 64) {
            const double y = tile_sum(r, s, a.V, i);
            if (lane == 0) sums[i] = y;
        }
        __syncthreads();
    } else {
        x = from->x;
        s = load_nodes(a, b, lane);
    }
    double total = row_sum(sums, tiles, lane);
    const bool later = state == W_TEST;
    // further sums: this workgroup alone.  A draw from nothing is one from the target as it is.
    while (state == W_TEST || (!(total > 0.0) && x.rej && x.S > 0.0)) {
        x.S = total;
        x.summed = true;
        if (state == W_TEST) state = walk_on(s, x) ? W_TEST : W_DRAW;
        __syncthreads();                                           // (the sums before are read)
        const Residual r = residual(a, s, x, b);
        for (int i = w; i < tiles; i += PT / 64) {
            const double y = tile_sum(r, s, a.V, i);
            if (lane == 0) sums[i] = y;
        }
        __syncthreads();
        total = row_sum(sums, tiles, lane);
    }
    if (w != 0) return;
    if (later) write_path(a, x, b, lane);
    if (!(total > 0.0)) {
        if (lane == 0) a.next[b] = -1;
        return;
    }
    // ---- the draw: the tile, then the token ----
    const double theta = (double)a.u[(size_t)a.N * a.B + b] * total;
    double before = 0.0, base = 0.0, lbase = 0.0;
    int tile = -1, last = -1;
    for (int i0 = 0; i0 < tiles && tile < 0; i0 += 64) {
        const int i = i0 + lane;
        const double y = i < tiles ? sums[i] : 0.0;
        double c = y;                                      // inclusive prefix sums
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
    if (tile < 0) {                                        // (rounding, or a number of 1 and more)
        tile = last;
        base = lbase;
    }
    // a run of neighbours a lane: the lanes' prefix sums, then the values'
    double v[VQ * 4], mine = 0.0;
    {
        const Residual r = residual(a, s, x, b);
        f4u p[VQ], q[VQ];
        load_tile<true>(r, s, a.V, tile, p, q);
#pragma unroll
        for (int e = 0; e < VQ * 4; ++e) {
            v[e] = share(r, p[e / 4][e % 4], q[e / 4][e % 4]);
            mine += v[e];
        }
    }
    double c = mine;
    for (int m = 1; m < 64; m <<= 1) {
        const double z = __shfl_up(c, m, 64);
        if (lane >= m) c += z;
    }
    double y = base + (c - mine);
    int pick = INT32_MAX, end = -1;
#pragma unroll
    for (int e = 0; e < VQ * 4; ++e) {
        y += v[e];
        if (v[e] > 0.0) {
            end = value_at<true>(tile, 0, lane) + e;
            if (pick == INT32_MAX && y > theta) pick = end;
        }
    }
    for (int m = 1; m < 64; m <<= 1) {                     // the smallest index past theta, or the largest that has a share
        pick = min(pick, __shfl_xor(pick, m, 64));
        end = max(end, __shfl_xor(end, m, 64));
    }
    if (lane == 0) a.next[b] = pick == INT32_MAX ? end : pick;
}

}  // namespace

size_t verify_workspace_bytes(int B, int N, int V) {
    return (size_t)B * (verify_tiles(V) * sizeof(double) + sizeof(Saved));
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
    if (a.B >= kAloneRows || (int64_t)a.V * (a.draft ? 4 : 1) <= kAloneValues)
        return launch_kernel(LQ_KERNEL_VERIFY, verify_pick_kernel<true>, dim3(a.B), dim3(PT), s, a);
    const int groups = (verify_tiles(a.V) + VT / 64 - 1) / (VT / 64);
    const hipError_t e = launch_kernel(LQ_KERNEL_VERIFY, verify_sum_kernel, dim3((unsigned)groups * (unsigned)a.B), dim3(VT), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(LQ_KERNEL_VERIFY, verify_pick_kernel<false>, dim3(a.B), dim3(PT), s, a);
}

}  // namespace lq

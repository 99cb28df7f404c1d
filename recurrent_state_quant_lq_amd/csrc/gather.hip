// gather.hip -- rows of the layers' states moved by an index per row (gfx950): sequences that
// are admitted, fork, move together or end.
//
// Row b of dst becomes row index[b] of src: the codec, and the window's slots before that row's
// position.  In place the rows may depend on each other in any way (chains, swaps, one row read
// by many): the columns of a state's rows are independent of each other, so a workgroup takes a
// slab of columns for every row, and per step loads the pieces of all the moved rows into
// registers, passes a barrier, and only then stores.  The step's width follows from the number
// of moved rows, which only the device knows: as many columns as the registers take.  Bound by memory:
// 56 of 64 rows of two layers (32 heads, d = 128) 25 us (4.5 TB/s), a third of 256 rows 23 us one call at a time and 31
// through six states in turn, which no cache holds.  Stores pass by the caches (kept there they push out what
// other workgroups are about to read: 38 and 35 us); loads do not (many rows may read one).
#include "gdn.h"

namespace lq {
namespace {

constexpr int GT = 256;                  // threads
constexpr int GP = 8;                    // pieces of 16 bytes per thread and step: eight waves a SIMD
constexpr int kCap = GT * GP;            // pieces per step
static_assert(kGatherInPlace == kCap, "an in-place gather holds a piece of every row");
constexpr int kLayers = 24;              // layers per launch (their pointers are kernel arguments: 3 KB)
constexpr int kFields = 8;
constexpr uint64_t kSlabs = 4096;

struct GatherArgs {
    void* dst[kLayers][kFields];
    const void* src[kLayers][kFields];
    const int32_t* index;
    const int32_t* pos;       // or null: no window slots
    int32_t* pos_out;         // or null
    uint32_t units[kFields];  // per row: pieces of 16 bytes (numbers of 4: comp_idx, one log decay a slot)
    uint32_t slab0[kFields + 1];         // first slab of each field (a workgroup each)
    int B, src_rows, W, C;
    uint32_t slot[kFields];   // units per window slot, 0: codec
    bool small[kFields];      // units of 4 bytes
    int shift;                // units per slab: 1 << shift
};

enum Field { F_SQ, F_ROW, F_COL, F_IDX, F_VAL, F_K, F_M, F_G };

template <typename U>
__device__ __forceinline__ void move_rows(const GatherArgs& a, int layer, int f, uint32_t slab, const int2* list, int n) {
    const U* src = static_cast<const U*>(a.src[layer][f]);
    U* dst = static_cast<U*>(a.dst[layer][f]);
    const uint32_t units = a.units[f], slot = a.slot[f], W = a.W;
    const uint32_t first = slab << a.shift, end = min(first + (1u << a.shift), units);
    // columns per step: a power of two, so that a step's pieces divide among the threads by shifts
    int shift = a.shift;
    while (shift > 0 && (n << shift) > kCap) --shift;
    for (uint32_t c0 = first; c0 < end; c0 += 1u << shift) {
        const uint32_t at = c0 + (threadIdx.x & ((1u << shift) - 1));   // (GT is a multiple of the columns: the same for all pieces)
        const int row0 = threadIdx.x >> shift, rows = GT >> shift;
        const int window = slot ? (int)(at / slot % W) : -1;
        U x[GP];
        uint32_t on = 0;
#pragma unroll
        for (int u = 0; u < GP; ++u) {
            const int e = row0 + rows * u;
            if (e >= n || at >= end) continue;
            const int i = list[e].y;                       // (dst row, src row; -2: cleared)
            if (window >= 0 && window >= a.pos[i]) continue;
            on |= 1u << u;
            if (i >= 0) {
                x[u] = src[(size_t)i * units + at];
            } else {
                // an empty state: zeros, column factors of 1, the first C rows as compensators
                const uint32_t z = f == F_COL ? 0x3f800000u : f == F_IDX ? at % (uint32_t)a.C : 0u;
                if constexpr (sizeof(U) == 4) x[u] = z;
                else x[u] = U{z, z, z, z};
            }
        }
        __syncthreads();                                   // every row's columns are read
#pragma unroll
        for (int u = 0; u < GP; ++u)
            if ((on >> u) & 1u) __builtin_nontemporal_store(x[u], &dst[(size_t)list[row0 + rows * u].x * units + at]);
    }
}

typedef uint32_t piece __attribute__((ext_vector_type(4)));

__global__ __launch_bounds__(GT) void gather_kernel(GatherArgs a) {
    __shared__ int2 s_list[kCap];
    __shared__ int s_n;
    const int t = threadIdx.x, layer = blockIdx.y;
    int f = 0;
    while (f + 1 < kFields && blockIdx.x >= a.slab0[f + 1]) ++f;
    const uint32_t slab = blockIdx.x - a.slab0[f];
    const bool same = a.dst[layer][F_SQ] == a.src[layer][F_SQ];
    const bool window = a.slot[f] != 0;
    // (more rows than a step holds: out of place only, in groups)
    for (int b0 = 0; b0 < a.B; b0 += kCap) {
        if (t == 0) s_n = 0;
        __syncthreads();
        for (int b = b0 + t; b < min(a.B, b0 + kCap); b += GT) {
            const int i = a.index[b];
            const bool clear = i == -2 && !window;
            const bool move = i >= 0 && i < a.src_rows && !(same && i == b) && !(window && a.pos[i] <= 0);
            if (clear || move) s_list[atomicAdd(&s_n, 1)] = make_int2(b, i);
            if (a.pos_out && blockIdx.x == 0 && layer == 0) {
                if (i == -2) a.pos_out[b] = 0;
                else if (i >= 0 && i < a.src_rows) a.pos_out[b] = a.pos ? a.pos[i] : 0;
            }
        }
        __syncthreads();
        const int n = s_n;
        if (n) {
            if (a.small[f]) move_rows<uint32_t>(a, layer, f, slab, s_list, n);
            else move_rows<piece>(a, layer, f, slab, s_list, n);
        }
        __syncthreads();                                   // the list is rewritten
    }
}

}  // namespace

hipError_t launch_gather(const lq_dims& d, int n_layers, const lq_state* dst, const lq_state* src, int src_rows,
                         const int32_t* index, const int32_t* pos, int32_t* pos_out, hipStream_t s) {
    GatherArgs a;
    const uint32_t H = d.H, dk = d.dk, C = d.C, W = d.W;
    const bool per_key = d.decay_mode == LQ_DECAY_PER_KEY;
    const uint32_t units[kFields] = {H * dk * dk / 16, H * dk / 4, H * dk / 4, H * C, H * C * dk / 4,
                                     H * W * dk / 4, H * W * dk / 4, per_key ? H * W * dk / 4 : H * W};
    // slabs: runs of 256 bytes to 4 KB of a row, as long as there are kSlabs of them.  Few rows that move cost a
    // slab's latencies, many its steps.  Measured (stores through the caches) for 1024, 2048, 4096 and 8192 slabs: 24 layers, 64 rows of 16
    // heads, 4 moved 20, 16, 17, 23 us; one layer, 256 rows of 32 heads, a third moved 29, 26, 26, 26; two
    // layers, 64 rows, 56 moved 29, 28, 26, 28.
    uint64_t all = 0;
    for (int f = 0; f < kFields; ++f) all += f >= F_K && !pos ? 0 : units[f];
    a.shift = 8;
    while (a.shift > 4 && (all * n_layers >> a.shift) < kSlabs) --a.shift;
    a.slab0[0] = 0;
    for (int f = 0; f < kFields; ++f) {
        const bool window = f >= F_K;
        a.units[f] = window && !pos ? 0 : units[f];
        a.slot[f] = !window ? 0 : f == F_G && !per_key ? 1 : dk / 4;
        a.small[f] = f == F_IDX || (f == F_G && !per_key);
        a.slab0[f + 1] = a.slab0[f] + (uint32_t)(((uint64_t)a.units[f] + (1u << a.shift) - 1) >> a.shift);
    }
    a.index = index;
    a.pos = pos;
    a.B = d.B;
    a.src_rows = src_rows;
    a.W = d.W;
    a.C = d.C;
    for (int l0 = 0; l0 < n_layers; l0 += kLayers) {
        const int n = n_layers - l0 < kLayers ? n_layers - l0 : kLayers;
        a.pos_out = l0 == 0 ? pos_out : nullptr;
        for (int l = 0; l < n; ++l) {
            const lq_state &x = dst[l0 + l], &y = src[l0 + l];
            void* const px[kFields] = {x.sq, x.row_scale, x.col_scale, x.comp_idx, x.comp_val, x.buf_k, x.buf_m, x.buf_g};
            const void* const py[kFields] = {y.sq, y.row_scale, y.col_scale, y.comp_idx, y.comp_val, y.buf_k, y.buf_m, y.buf_g};
            for (int f = 0; f < kFields; ++f) {
                a.dst[l][f] = px[f];
                a.src[l][f] = py[f];
            }
        }
        const hipError_t e = launch_kernel(LQ_KERNEL_GATHER, gather_kernel, dim3(a.slab0[kFields], n), dim3(GT), s, a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lq

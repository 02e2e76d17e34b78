// Linear layers with one weight per group of a packed batch, on gfx950:
//     y_r = W_n x_r + b_n   for the rows r of group n,
// and the backward pass grad_x_r = W_n^T g_r, grad_W_n = sum_r g_r x_r^T,
// grad_b_n = sum_r g_r.
//
// The group sizes are device data, so a launch covers the largest number of
// row tiles that any split of R rows into N groups can have, and every
// workgroup finds its own group from the offsets (64 groups at a time, one
// lane each); workgroups beyond the last tile leave.
#include "dmr_internal.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

// A run of rows of one group.
struct RowTile {
    int64_t group, first;   // group < 0: no such tile
    int rows;
};

// Bounds of group n, held inside [0, R] whatever the offsets say.
__device__ __forceinline__ void group_bounds(const int64_t* __restrict__ off, int64_t N, int64_t R, int64_t n,
                                             int64_t& lo, int64_t& hi) {
    lo = hi = 0;
    if (n < N) {
        lo = off[n];
        hi = off[n + 1];
        lo = lo < 0 ? 0 : lo > R ? R : lo;
        hi = hi < lo ? lo : hi > R ? R : hi;
    }
}

__device__ __forceinline__ int64_t wave_inclusive_sum(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Row tile t of all groups' tiles of `per` rows in order. Every wave does
// the same work.
__device__ __forceinline__ RowTile find_row_tile(const int64_t* __restrict__ off, int64_t N, int64_t R, int per,
                                                 int64_t t) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int64_t base = 0; base < N; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        const int64_t tiles = (hi - lo + per - 1) / per;
        const int64_t upto = before + wave_inclusive_sum(tiles, lane);
        const uint64_t hit = __ballot(upto > t);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t first = lo + (t - (upto - tiles)) * per;
            const int64_t left = hi - first;
            RowTile r;
            r.group = uniform64(base + src);
            r.first = uniform64(__shfl(first, src, 64));
            r.rows = __builtin_amdgcn_readfirstlane(__shfl((int)(left < per ? left : per), src, 64));
            return r;
        }
        before = __shfl(upto, 63, 64);
    }
    return {-1, 0, 0};
}

// Stores four consecutive n of row m.
template <class T>
__device__ __forceinline__ void store4(T* __restrict__ row, int n, int N, f32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < N) row[n + i] = (T)v[i];
}

template <class T, int COUNT>
struct alignas(16) Packed {
    T v[COUNT];
};

// Writes a workgroup's tile: rows [0, rows) of `out` (leading dimension ld),
// columns [n0, N), plus bias[n] if given. VEC as in OperandTile::stage.
template <class T, class Tile, bool VEC>
__device__ __forceinline__ void store_tile(const Tile& t, T* __restrict__ out, int64_t ld, int rows, int n0, int N,
                                           const T* __restrict__ bias, int tid) {
    constexpr int STEP = Tile::PAIRED ? 2 : 1;
#pragma unroll
    for (int a = 0; a < Tile::NT; a += STEP) {
        const int n = n0 + Tile::n_of(tid, a);
        f32x4 add[STEP];
#pragma unroll
        for (int s = 0; s < STEP; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = n + 4 * s + i;   // past the end: any value, not stored
                add[s][i] = bias ? (float)bias[at < N ? at : N - 1] : 0.0f;
            }
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
            if (m >= rows) continue;
            T* row = out + (int64_t)m * ld;
            if constexpr (VEC && (Tile::PAIRED || sizeof(T) == 4)) {
                if (n < N) {
                    Packed<T, 4 * STEP> w;
#pragma unroll
                    for (int s = 0; s < STEP; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w.v[4 * s + i] = (T)(t.acc[a + s][b][i] + add[s][i]);
                    *reinterpret_cast<Packed<T, 4 * STEP>*>(row + n) = w;
                }
            } else {
#pragma unroll
                for (int s = 0; s < STEP; ++s) store4<T>(row, n + 4 * s, N, t.acc[a + s][b] + add[s]);
            }
        }
    }
}

// y = x W^T + b (WK: the weight's contiguous direction is summed over) or
// grad_x = g W (!WK), row tile by row tile. `n_out` is the width of `out`,
// `k_in` that of `rows_in`; the weight of a group is [n_out][k_in] if WK and
// [k_in][n_out] if not.
template <class T, int BN, int BM, int WN, int WM, bool WK, bool VEC>
__global__ __launch_bounds__(WN * WM * 64) void grouped_rows(const T* __restrict__ rows_in, int64_t R, int k_in,
                                                             const int64_t* __restrict__ off, int64_t N,
                                                             const T* __restrict__ weight, int n_out,
                                                             const T* __restrict__ bias, T* __restrict__ out,
                                                             int64_t tiles, int n_tiles) {
    using Tile = TileProduct<T, BN, BM, WN, WM, WK, true>;
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    // consecutive workgroups go to the 8 dies in turn: each die takes a run
    // of consecutive tiles, which share rows and weights in its L2
    const int64_t per = (tiles + 7) / 8;
    const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= tiles) return;
    const RowTile at = find_row_tile(off, N, R, BM, id / n_tiles);
    if (at.group < 0) return;
    const int n0 = (int)(id % n_tiles) * BN;
    const int tid = threadIdx.x;
    const T* w = weight + at.group * (int64_t)n_out * k_in + (WK ? (int64_t)n0 * k_in : (int64_t)n0);
    Tile t;
    t.template run<VEC, false>(lds, w, WK ? k_in : n_out, n_out - n0, rows_in + at.first * (int64_t)k_in, k_in, at.rows,
                               k_in, tid, false);
    store_tile<T, Tile, VEC>(t, out + at.first * (int64_t)n_out, n_out, at.rows, n0, n_out,
                             bias ? bias + at.group * (int64_t)n_out : nullptr, tid);
}

// ---------------------------------------------------------------------------
// gradient of the weights: a product over each group's rows
// ---------------------------------------------------------------------------
// A group's rows are cut into pieces of `per` rows. A group of one piece (or
// none) is written directly; the pieces of longer groups go to the workspace
// in float32, each to a slot of its own, and are added in order afterwards:
// no atomics, so the result does not depend on timing.

struct Piece {
    int64_t group, first;   // group < 0: no such piece
    int rows;
    int64_t slot;           // < 0: the group's only piece
};

__device__ __forceinline__ int64_t pieces_of(int64_t rows, int per) { return rows > per ? (rows + per - 1) / per : 1; }

__device__ __forceinline__ Piece find_piece(const int64_t* __restrict__ off, int64_t N, int64_t R, int per, int64_t t) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0, slots_before = 0;
    for (int64_t base = 0; base < N; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        const int64_t pieces = base + lane < N ? pieces_of(hi - lo, per) : 0;
        const int64_t slots = pieces > 1 ? pieces : 0;
        const int64_t upto = before + wave_inclusive_sum(pieces, lane);
        const int64_t slots_upto = slots_before + wave_inclusive_sum(slots, lane);
        const uint64_t hit = __ballot(upto > t);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t k = t - (upto - pieces);
            const int64_t first = lo + k * per;
            const int64_t left = hi - first;
            Piece r;
            r.group = uniform64(base + src);
            r.first = uniform64(__shfl(first, src, 64));
            r.rows = __builtin_amdgcn_readfirstlane(__shfl((int)(left < per ? left : per), src, 64));
            r.slot = uniform64(__shfl(pieces > 1 ? slots_upto - slots + k : (int64_t)-1, src, 64));
            return r;
        }
        before = __shfl(upto, 63, 64);
        slots_before = __shfl(slots_upto, 63, 64);
    }
    return {-1, 0, 0, -1};
}

template <class T, int BN, int BM, int WN, int WM, bool VEC>
__global__ __launch_bounds__(WN * WM * 64) void grouped_weight_grad(
    const T* __restrict__ x, const T* __restrict__ g, int64_t R, int cin, int cout, const int64_t* __restrict__ off,
    int64_t N, int per, T* __restrict__ grad_weight, T* __restrict__ grad_bias, float* __restrict__ slots,
    int64_t slot_count, int64_t items, int n_tiles, int m_tiles) {
    using Tile = TileProduct<T, BN, BM, WN, WM, false, false>;
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    const int64_t each = (items + 7) / 8;
    const int64_t id = (int64_t)(blockIdx.x & 7) * each + (blockIdx.x >> 3);
    if (id >= items) return;
    const int tiles = n_tiles * m_tiles;
    const Piece at = find_piece(off, N, R, per, id / tiles);
    if (at.group < 0 || at.slot >= slot_count) return;
    const int tile = (int)(id % tiles);
    const int n0 = (tile % n_tiles) * BN, m0 = (tile / n_tiles) * BM;
    const int tid = threadIdx.x;
    const bool sums = n0 == 0 && grad_bias != nullptr;
    if (!grad_weight && !sums) return;
    Tile t;
    t.template run<VEC, true>(lds, x + at.first * cin + n0, cin, cin - n0, g + at.first * cout + m0, cout, cout - m0,
                              at.rows, tid, sums);
    const int rows = cout - m0 < BM ? cout - m0 : BM;
    const int lane = tid & 63;
    const bool first_n = (tid >> 6) % WN == 0 && lane < 16;   // one lane per m holds the row's sum
    if (at.slot < 0) {
        if (grad_weight)
            store_tile<T, Tile, VEC>(t, grad_weight + (at.group * cout + m0) * (int64_t)cin, cin, rows, n0, cin,
                                     (const T*)nullptr, tid);
        if (sums && first_n)
#pragma unroll
            for (int b = 0; b < Tile::MT; ++b) {
                const int m = Tile::m_of(tid, b);
                if (m < rows) grad_bias[at.group * cout + m0 + m] = (T)t.ones[b][0];
            }
        return;
    }
    float* slot = slots + at.slot * ((int64_t)cout * cin + cout);
    if (grad_weight) {
#pragma unroll
        for (int a = 0; a < Tile::NT; ++a)
#pragma unroll
            for (int b = 0; b < Tile::MT; ++b) {
                const int m = Tile::m_of(tid, b);
                if (m < rows) store4<float>(slot + (int64_t)(m0 + m) * cin, n0 + Tile::n_of(tid, a), cin, t.acc[a][b]);
            }
    }
    if (sums && first_n)
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
            if (m < rows) slot[(int64_t)cout * cin + m0 + m] = t.ones[b][0];
        }
}

// Adds the pieces of the groups that have more than one, in order.
template <class T>
__global__ __launch_bounds__(256) void grouped_add_pieces(const int64_t* __restrict__ off, int64_t N, int64_t R, int per,
                                                          int64_t values, int64_t weights, const float* __restrict__ slots,
                                                          int64_t slot_count, unsigned blocks, T* __restrict__ grad_weight,
                                                          T* __restrict__ grad_bias) {
    const int lane = threadIdx.x & 63;
    const int64_t group = blockIdx.x / blocks;
    int64_t slot = 0, mine = 0;
    for (int64_t base = 0; base <= group; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        const int64_t pieces = base + lane <= group ? pieces_of(hi - lo, per) : 0;
        const int64_t upto = wave_inclusive_sum(base + lane < group && pieces > 1 ? pieces : 0, lane);
        slot += __shfl(upto, 63, 64);
        if (group < base + 64) mine = __shfl(pieces, (int)(group - base), 64);
    }
    if (mine <= 1 || slot + mine > slot_count) return;
    const int64_t width = values;   // weights, then the bias
    for (int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x; i < width; i += (int64_t)blocks * 256) {
        const bool is_weight = i < weights;
        if (is_weight ? grad_weight == nullptr : grad_bias == nullptr) continue;
        const float* from = slots + slot * width + i;
        float s = from[0];
        for (int64_t k = 1; k < mine; ++k) s += from[k * width];
        if (is_weight) grad_weight[group * weights + i] = (T)s;
        else grad_bias[group * (width - weights) + i - weights] = (T)s;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The most row tiles of `per` rows that R rows in N groups can make.
int64_t most_row_tiles(int64_t R, int64_t N, int per) { return R / per + (N < R ? N : R); }

template <class T, int BN, int BM, int WN, int WM, bool WK>
hipError_t launch_rows_tile(const GroupedLinearArgs& a, const T* in, int k_in, const T* bias, T* out, int n_out, bool vec) {
    const int n_tiles = ceil_div(n_out, BN);
    const int64_t tiles = most_row_tiles(a.R, a.N, BM) * n_tiles;
    const int64_t grid = (tiles + 7) / 8 * 8;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    const T* w = static_cast<const T*>(a.weight);
    if (vec)
        grouped_rows<T, BN, BM, WN, WM, WK, true><<<(unsigned)grid, WN * WM * 64, 0, a.stream>>>(
            in, a.R, k_in, a.off, a.N, w, n_out, bias, out, tiles, n_tiles);
    else
        grouped_rows<T, BN, BM, WN, WM, WK, false><<<(unsigned)grid, WN * WM * 64, 0, a.stream>>>(
            in, a.R, k_in, a.off, a.N, w, n_out, bias, out, tiles, n_tiles);
    return hipGetLastError();
}

template <class T, bool WK>
hipError_t launch_rows(const GroupedLinearArgs& a, const T* in, int k_in, const T* bias, T* out, int n_out, bool vec) {
    if (a.R <= 16 * a.N) return launch_rows_tile<T, 64, 16, 4, 1, WK>(a, in, k_in, bias, out, n_out, vec);
    if (n_out <= 16) return launch_rows_tile<T, 16, 256, 1, 4, WK>(a, in, k_in, bias, out, n_out, vec);
    if (n_out <= 64) return launch_rows_tile<T, 64, 128, 1, 4, WK>(a, in, k_in, bias, out, n_out, vec);
    return launch_rows_tile<T, 128, 128, 2, 2, WK>(a, in, k_in, bias, out, n_out, vec);
}

template <class T, int BN, int BM, int WN, int WM>
hipError_t launch_weight_tile(const GroupedLinearArgs& a, int per, int64_t slot_count, bool vec) {
    const int n_tiles = ceil_div(a.cin, BN), m_tiles = ceil_div(a.cout, BM);
    const int64_t items = (a.R / per + a.N) * n_tiles * m_tiles;
    const int64_t grid = (items + 7) / 8 * 8;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    const T *x = static_cast<const T*>(a.x), *g = static_cast<const T*>(a.grad_y);
    T *gw = static_cast<T*>(a.grad_weight), *gb = static_cast<T*>(a.grad_bias);
    if (vec)
        grouped_weight_grad<T, BN, BM, WN, WM, true><<<(unsigned)grid, WN * WM * 64, 0, a.stream>>>(
            x, g, a.R, a.cin, a.cout, a.off, a.N, per, gw, gb, a.workspace, slot_count, items, n_tiles, m_tiles);
    else
        grouped_weight_grad<T, BN, BM, WN, WM, false><<<(unsigned)grid, WN * WM * 64, 0, a.stream>>>(
            x, g, a.R, a.cin, a.cout, a.off, a.N, per, gw, gb, a.workspace, slot_count, items, n_tiles, m_tiles);
    return hipGetLastError();
}

template <class T>
hipError_t launch_all(const GroupedLinearArgs& a, bool backward) {
    const T* bias = static_cast<const T*>(a.bias);
    const bool widths = a.cin % (16 / sizeof(T)) == 0 && a.cout % (16 / sizeof(T)) == 0;
    if (!backward) {
        const bool vec = widths && aligned16(a.x) && aligned16(a.weight) && aligned16(a.y);
        if (a.R == 0) return hipSuccess;
        timing_begin(kKGroupedLinearFwd, a.stream);
        const hipError_t err = launch_rows<T, true>(a, static_cast<const T*>(a.x), a.cin, bias, static_cast<T*>(a.y), a.cout, vec);
        timing_end(kKGroupedLinearFwd, a.stream);
        return err;
    }
    timing_begin(kKGroupedLinearBwd, a.stream);
    hipError_t err = hipSuccess;
    if (a.grad_x && a.R > 0) {
        const bool vec = widths && aligned16(a.grad_y) && aligned16(a.weight) && aligned16(a.grad_x);
        err = launch_rows<T, false>(a, static_cast<const T*>(a.grad_y), a.cout, (const T*)nullptr, static_cast<T*>(a.grad_x),
                                    a.cin, vec);
    }
    if (err == hipSuccess && (a.grad_weight || a.grad_bias) && a.N > 0) {
        const bool vec = widths && aligned16(a.x) && aligned16(a.grad_y) && aligned16(a.grad_weight);
        const GroupedPieces p = grouped_pieces(a.R, a.N, a.cin, a.cout);
        if (a.cin <= 64 && a.cout <= 64) err = launch_weight_tile<T, 64, 64, 2, 2>(a, p.rows, p.slots, vec);
        else err = launch_weight_tile<T, 128, 128, 2, 2>(a, p.rows, p.slots, vec);
        if (err == hipSuccess && p.slots > 0) {
            const int64_t weights = (int64_t)a.cin * a.cout, values = weights + a.cout;
            const unsigned blocks = (unsigned)(values < 64 * 256 ? (values + 255) / 256 : 64);
            grouped_add_pieces<T><<<(unsigned)(blocks * a.N), 256, 0, a.stream>>>(
                a.off, a.N, a.R, p.rows, values, weights, a.workspace, p.slots, blocks, static_cast<T*>(a.grad_weight),
                static_cast<T*>(a.grad_bias));
            err = hipGetLastError();
        }
    }
    timing_end(kKGroupedLinearBwd, a.stream);
    return err;
}

hipError_t launch_typed(const GroupedLinearArgs& a, bool backward) {
    switch (a.dtype) {
        case DMR_FLOAT32: return launch_all<float>(a, backward);
        case DMR_FLOAT16: return launch_all<_Float16>(a, backward);
        case DMR_BFLOAT16: return launch_all<__bf16>(a, backward);
    }
    return hipErrorInvalidValue;
}

}  // namespace

// Rows of a piece of the weight gradient, and the slots that the pieces of
// groups longer than one piece can take: a group of r > rows has at most
// 2 r / rows of them.
GroupedPieces grouped_pieces(int64_t R, int64_t N, int32_t cin, int32_t cout) {
    const bool small = cin <= 64 && cout <= 64;
    const int64_t side = small ? 64 : 128;
    const int64_t tiles = ((cin + side - 1) / side) * ((cout + side - 1) / side);
    const int64_t want = tiles >= 512 ? 1 : 512 / tiles;   // pieces that fill the device
    int64_t rows = (R + want - 1) / want;
    rows = (rows + 127) / 128 * 128;
    rows = rows < 512 ? 512 : rows > 8192 ? 8192 : rows;
    return {(int)rows, R > rows ? 2 * (R / rows) : 0};
}

hipError_t launch_grouped_linear_forward(const GroupedLinearArgs& a) { return launch_typed(a, false); }
hipError_t launch_grouped_linear_backward(const GroupedLinearArgs& a) { return launch_typed(a, true); }

}  // namespace dmr

// Kernels and launches of the linear layers of packed batches.
//
// T: the type of the products' operands; PT: of x and of the weight, which is T
// but where they are split as they are read; OUT: of the results. TERMS (backward
// only): the upstream gradient is a pair of arrays of T, whose sum it is (2), and
// x and the weight are pairs too (3).
#pragma once

#include "dmr_internal.h"
#include "grouped_tiles.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

template <class V>
struct TypeOf {
    typedef V type;
};

// y = x W^T + b (WK: the weight's contiguous direction is summed over) or
// grad_x = g W (!WK), row tile by row tile. `n_out` is the width of `out`,
// `k_in` that of `rows_in`; the weight of a group is [n_out][k_in] if WK and
// [k_in][n_out] if not.
template <class T, class Tile, bool WK, bool VEC>
__device__ __forceinline__ void rows_of_workgroup(char* lds, uint32_t block, uint32_t blocks,
                                                  const T* __restrict__ rows_in, const T* __restrict__ rows_low, int64_t R,
                                                  int k_in, const int64_t* __restrict__ off, int64_t N,
                                                  const typename Tile::PType* __restrict__ weight,
                                                  const typename Tile::PType* __restrict__ weight_low, int n_out,
                                                  const typename Tile::Out* __restrict__ bias,
                                                  typename Tile::Out* __restrict__ out, bool wide, int64_t tiles,
                                                  int n_tiles, uint32_t places) {
    const int tid = threadIdx.x;
    walk_row_tiles<T, Tile, VEC>(
        lds, block, blocks, rows_in, R, k_in, off, N, tiles, n_tiles, places,
        [&](const RowTile& at, int n0) {
            const int64_t w = at.group * (int64_t)n_out * k_in + (WK ? (int64_t)n0 * k_in : (int64_t)n0);
            return typename Tile::PSource{weight + w, WK ? k_in : n_out, n_out - n0, weight_low ? weight_low + w : nullptr};
        },
        [](const RowTile&, int) { return typename Tile::Zero(); },
        [](const RowTile&, int) { return 0; },
        [&](Tile& t, const RowTile& at, int n0, int) {
            store_tile<typename Tile::Out, Tile>(
                                 t, out + at.first * (int64_t)n_out, n_out, at.rows, n0, n_out,
                                 bias ? bias + at.group * (int64_t)n_out : nullptr, wide, tid);
        },
        false, rows_low);
}

template <class T, class Tile, bool WK, bool VEC>
__global__ __launch_bounds__(Tile::THREADS) void grouped_rows(const T* __restrict__ rows_in, const T* __restrict__ rows_low,
                                                              int64_t R, int k_in, const int64_t* __restrict__ off, int64_t N,
                                                              const typename Tile::PType* __restrict__ weight,
                                                              const typename Tile::PType* __restrict__ weight_low, int n_out,
                                                              const typename Tile::Out* __restrict__ bias,
                                                              typename Tile::Out* __restrict__ out, bool wide,
                                                              int64_t tiles, int n_tiles, uint32_t places) {
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    rows_of_workgroup<T, Tile, WK, VEC>(lds, blockIdx.x, gridDim.x, rows_in, rows_low, R, k_in, off, N, weight, weight_low, n_out,
                                        bias, out, wide, tiles, n_tiles, places);
}

// ---------------------------------------------------------------------------
// gradient of the weights: a product over each group's rows
// ---------------------------------------------------------------------------
template <class T, class Tile, bool VEC>
__device__ __forceinline__ void weight_grad_of_workgroup(
    char* lds, uint32_t block, const typename Tile::PType* __restrict__ x, const typename Tile::PType* __restrict__ x_low,
    const T* __restrict__ g, const T* __restrict__ g_low, int64_t R, int cin, int cout, const int64_t* __restrict__ off,
    int64_t N, int per, typename Tile::Out* __restrict__ grad_weight, typename Tile::Out* __restrict__ grad_bias, bool wide,
    float* __restrict__ slots, int64_t slot_count, int64_t items, int n_tiles, int m_tiles, int shortest = -1) {
    typedef typename Tile::Out Out;
    const int64_t id = tile_of_workgroup<kPieceRun>(block);
    if (id >= items) return;
    const int tiles = n_tiles * m_tiles;
    const Piece at = shortest < 0 ? find_piece(off, N, R, per, (int)(id / tiles)) : find_long(off, N, R, shortest, id / tiles);
    if (at.group < 0 || at.slot >= slot_count) return;
    const int tile = (int)(id % tiles);
    const int n0 = (tile % n_tiles) * Tile::BN, m0 = (tile / n_tiles) * Tile::BM;
    const int tid = threadIdx.x;
    const bool sums = n0 == 0 && grad_bias != nullptr;
    if (!grad_weight && !sums) return;
    Tile t;
    t.template run<VEC>(lds, typename Tile::PSource{x + at.first * cin + n0, cin, cin - n0,
                                                    x_low ? x_low + at.first * cin + n0 : nullptr},
                        {g + at.first * cout + m0, cout, cout - m0, g_low ? g_low + at.first * cout + m0 : nullptr}, at.rows,
                        tid, sums);
    const int rows = cout - m0 < Tile::BM ? cout - m0 : Tile::BM;
    const int lane = tid & 63;
    const bool first_n = Tile::n_of(tid, 0) == 0 && lane < 16;   // one lane per m holds the row's sum
    if (at.slot < 0) {
        if (grad_weight)
            store_tile<Out, Tile>(t, grad_weight + (at.group * cout + m0) * (int64_t)cin, cin, rows, n0, cin,
                                  (const Out*)nullptr, wide, tid);
        if (sums && first_n)
#pragma unroll
            for (int b = 0; b < Tile::MT; ++b) {
                const int m = Tile::m_of(tid, b);
                if (m < rows) grad_bias[at.group * cout + m0 + m] = (Out)t.ones[b][0];
            }
        return;
    }
    float* slot = slots + at.slot * grouped_piece_values(cin, cout);
    if (grad_weight) {
        const bool whole = cin % 4 == 0;
#pragma unroll
        for (int a = 0; a < Tile::NT; ++a)
#pragma unroll
            for (int b = 0; b < Tile::MT; ++b) {
                const int m = Tile::m_of(tid, b), n = n0 + Tile::n_of(tid, a);
                if (m >= rows) continue;
                float* row = slot + (int64_t)(m0 + m) * cin;
                if (!whole) store4<float>(row, n, cin, t.acc[a][b]);
                else if (n < cin) *reinterpret_cast<f32x4*>(row + n) = t.acc[a][b];
            }
    }
    if (sums && first_n)
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
            if (m < rows) slot[(int64_t)cout * cin + m0 + m] = t.ones[b][0];
        }
}

template <class T, class Tile, bool VEC>
__global__ __launch_bounds__(Tile::THREADS) void grouped_weight_grad(
    const typename Tile::PType* __restrict__ x, const typename Tile::PType* __restrict__ x_low, const T* __restrict__ g,
    const T* __restrict__ g_low, int64_t R, int cin, int cout, const int64_t* __restrict__ off, int64_t N, int per,
    typename Tile::Out* __restrict__ grad_weight, typename Tile::Out* __restrict__ grad_bias, bool wide,
    float* __restrict__ slots, int64_t slot_count, int64_t items, int n_tiles, int m_tiles, int shortest) {
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    weight_grad_of_workgroup<T, Tile, VEC>(lds, blockIdx.x, x, x_low, g, g_low, R, cin, cout, off, N, per, grad_weight, grad_bias, wide,
                                           slots, slot_count, items, n_tiles, m_tiles, shortest);
}

// Both gradients in one launch: the workgroups of the weight's, whose chains
// are the longer ones, and then the rows'.
template <class T, class RowTile, class WeightTile, bool VEC>
__global__ __launch_bounds__(RowTile::THREADS) void grouped_both_grads(
    const typename RowTile::PType* __restrict__ x, const typename RowTile::PType* __restrict__ x_low, const T* __restrict__ g,
    const T* __restrict__ g_low, int64_t R, int cin, int cout, const int64_t* __restrict__ off, int64_t N,
    const typename RowTile::PType* __restrict__ weight, const typename RowTile::PType* __restrict__ weight_low,
    typename RowTile::Out* __restrict__ grad_x, bool wide_x, int64_t row_tiles, int row_n_tiles, uint32_t row_places,
    uint32_t weight_places, int per, typename RowTile::Out* __restrict__ grad_weight,
    typename RowTile::Out* __restrict__ grad_bias, bool wide_w, float* __restrict__ slots, int64_t slot_count, int64_t items, int n_tiles, int m_tiles) {
    static_assert(RowTile::THREADS == WeightTile::THREADS, "");
    __shared__ alignas(16) char lds[RowTile::kLdsBytes > WeightTile::kLdsBytes ? RowTile::kLdsBytes : WeightTile::kLdsBytes];
    if (blockIdx.x < weight_places)
        weight_grad_of_workgroup<T, WeightTile, VEC>(lds, blockIdx.x, x, x_low, g, g_low, R, cin, cout, off, N, per,
                                                     grad_weight, grad_bias, wide_w, slots, slot_count, items, n_tiles, m_tiles);
    else
        rows_of_workgroup<T, RowTile, false, VEC>(lds, blockIdx.x - weight_places, row_places, g, g_low, R, cout, off, N, weight,
                                                  weight_low, cin, (const typename RowTile::Out*)nullptr, grad_x, wide_x, row_tiles,
                                                  row_n_tiles, row_places);
}

// Adds the pieces of the groups that have more than one, in a fixed order,
// eight loads in flight a lane. SPLIT: a workgroup takes 256 values of a group
// and its four waves a quarter of the pieces each (small weights, whose long
// groups have many pieces); otherwise it takes 4096 values.
template <bool SPLIT>
constexpr int kAddValues = SPLIT ? 256 : 4096;

template <class T, bool SPLIT>
__global__ __launch_bounds__(256) void grouped_add_pieces(const int64_t* __restrict__ off, int64_t N, int64_t R, int per,
                                                          int64_t values, int64_t width, int64_t weights,
                                                          const float* __restrict__ slots, int64_t slot_count,
                                                          unsigned blocks, T* __restrict__ grad_weight,
                                                          T* __restrict__ grad_bias) {
    __shared__ f32x4 part[SPLIT ? 4 : 1][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t group = blockIdx.x / blocks;
    int64_t slot = 0;
    int mine = 0;
    for (int64_t base = 0; base <= group; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        int length;
        const int pieces = base + lane <= group ? pieces_of(hi - lo, per, length) : 0;
        const int upto = wave_inclusive_sum(base + lane < group && pieces > 1 ? pieces : 0, lane);
        slot += __builtin_amdgcn_readlane(upto, 63);
        if (group < base + 64) mine = __builtin_amdgcn_readlane(pieces, (int)(group - base));
    }
    if (mine <= 1 || slot + mine > slot_count) return;
    // the sum of pieces first, first + 4, .. at value i
    const auto sum = [&](int64_t i, int first) {
        const float* from = slots + (slot + first) * width + i;   // slots are padded to whole vectors
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = first; k < mine; k += 32) {
            f32x4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)   // past the end: this one again, not added
                v[j] = *reinterpret_cast<const f32x4*>(from + (k + 4 * j < mine ? (int64_t)(4 * j) * width : 0));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + 4 * j < mine) s += v[j];
            from += 32 * width;
        }
        return s;
    };
    const auto write = [&](int64_t i0, f32x4 s) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = i0 + j;
            if (i < weights) {
                if (grad_weight) grad_weight[group * weights + i] = (T)s[j];
            } else if (i < values && grad_bias) {
                grad_bias[group * (values - weights) + i - weights] = (T)s[j];
            }
        }
    };
    int64_t begin = (int64_t)(blockIdx.x % blocks) * kAddValues<SPLIT>;
    if constexpr (SPLIT) {
        const int64_t i = begin + lane * 4;
        if (i < values && wave < mine) part[wave][lane] = sum(i, wave);
        __syncthreads();
        if (wave > 0 || i >= values) return;
        f32x4 s = part[0][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w)
            if (w < mine) s += part[w][lane];
        write(i, s);
    } else {
        // four vectors a lane, 1024 values apart, all in flight
        const float* from = slots + slot * width;
        for (; begin < values; begin += (int64_t)blocks * kAddValues<SPLIT>) {
            f32x4 s[4];
            int64_t at[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t i = begin + j * 1024 + tid * 4;
                at[j] = i < values ? i : 0;   // past the end: not written
                s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            for (int k = 0; k < mine; k += 2) {
                f32x4 v[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[u][j] = *reinterpret_cast<const f32x4*>(from + (k + (k + u < mine ? u : 0)) * width + at[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j] += v[0][j];
                    if (k + 1 < mine) s[j] += v[1][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (begin + j * 1024 + tid * 4 < values) write(at[j], s[j]);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <class T, class Tile, bool WK>
hipError_t launch_rows_tile(const GroupedLinearArgs& a, const T* in, int k_in, const typename Tile::Out* bias,
                            typename Tile::Out* out, int n_out, bool vec, bool wide) {
    const int n_tiles = ceil_div(n_out, Tile::BN);
    const int64_t tiles = most_row_tiles(a.R, a.N, Tile::BM) * n_tiles;
    const unsigned places = run_grid<kRun>(tiles);
    if (places == 0) return hipErrorInvalidValue;
    // as many workgroups as the device holds at a time (a multiple of 8 kRun)
    constexpr unsigned kHeld = 256 * (160 * 1024 / Tile::kLdsBytes);
    const unsigned grid = places > kHeld ? kHeld : places;
    const auto w = static_cast<const typename Tile::PType*>(a.weight), w_low = static_cast<const typename Tile::PType*>(a.weight_low);
    const T* low = static_cast<const T*>(a.grad_y_low);
    if (vec)
        grouped_rows<T, Tile, WK, true><<<grid, Tile::THREADS, 0, a.stream>>>(in, low, a.R, k_in, a.off, a.N, w, w_low, n_out,
                                                                              bias, out, wide, tiles, n_tiles, places);
    else if constexpr (Tile::BN < 256)   // the largest tiles have no form for unaligned arrays
        grouped_rows<T, Tile, WK, false><<<grid, Tile::THREADS, 0, a.stream>>>(in, low, a.R, k_in, a.off, a.N, w, w_low, n_out,
                                                                               bias, out, wide, tiles, n_tiles, places);
    return hipGetLastError();
}

// Tiles of rows and of the weight's gradient.
template <class T, class PT, class OUT, int TERMS, bool WK, int BN, int BM, int WN, int WM, int S>
using RowsProduct = TileProduct<T, BN, BM, WN, WM, WK, true, S, false, 1, PT, TERMS, OUT>;
template <class T, class PT, class OUT, int TERMS, int SIDE, int WN, int WM>
using WeightProduct = TileProduct<T, SIDE, SIDE, WN, WM, false, false, 2, true, 1, PT, TERMS, OUT>;
template <class T, class PT, class OUT, int TERMS>
using SmallWeightTile = WeightProduct<T, PT, OUT, TERMS, 64, 2, 2>;

// Operands that are split as they are multiplied have few rows for a group: one
// tile each.
template <class T, class PT, class OUT, int TERMS, bool WK>
hipError_t launch_rows(const GroupedLinearArgs& a, const T* in, int k_in, const OUT* bias, OUT* out, int n_out, bool vec,
                       bool wide) {
    const RowsTile t = grouped_rows_tile(a.R, a.N, n_out, sizeof(T) == 2, !WK, vec);
    const auto launch = [&](auto tile) {
        return launch_rows_tile<T, typename decltype(tile)::type, WK>(a, in, k_in, bias, out, n_out, vec, wide);
    };
    if (t.rows == 16) return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 64, 16, 4, 1, 4>>{});
    if constexpr (!__is_same(T, PT)) {
        return hipErrorInvalidValue;
    } else {
        if (t.columns == 16) return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 16, 128, 1, 4, 2>>{});
        if constexpr (sizeof(T) == 2) {
            if (t.columns == 64 && t.rows == 256) return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 64, 256, 1, 8, 2>>{});
            if (t.columns == 256) return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 256, 256, 4, 2, 2>>{});
        }
        if (t.columns == 64) return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 64, 128, 1, 4, 2>>{});
        return launch(TypeOf<RowsProduct<T, PT, OUT, TERMS, WK, 128, 128, 2, 4, 2>>{});
    }
}

template <class T, class Tile>
hipError_t launch_weight_tile(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide) {
    const int n_tiles = ceil_div(a.cin, Tile::BN), m_tiles = ceil_div(a.cout, Tile::BM);
    const int64_t pieces = a.long_only ? (a.R + a.long_only) / (a.long_only + 1) : a.R / p.rows + a.N;   // at most
    const int64_t items = pieces * n_tiles * m_tiles;
    const int shortest = a.long_only ? a.long_only : -1;
    const unsigned grid = run_grid<kPieceRun>(items);
    if (grid == 0) return hipErrorInvalidValue;
    typedef typename Tile::PType PT;
    typedef typename Tile::Out Out;
    const PT *x = static_cast<const PT*>(a.x), *x_low = static_cast<const PT*>(a.x_low);
    const T *g = static_cast<const T*>(a.grad_y), *g_low = static_cast<const T*>(a.grad_y_low);
    Out *gw = static_cast<Out*>(a.grad_weight), *gb = static_cast<Out*>(a.grad_bias);
    if (vec)
        grouped_weight_grad<T, Tile, true><<<grid, Tile::THREADS, 0, a.stream>>>(
            x, x_low, g, g_low, a.R, a.cin, a.cout, a.off, a.N, p.rows, gw, gb, wide, a.workspace, p.slots, items, n_tiles, m_tiles, shortest);
    else if constexpr (Tile::BN < 256)
        grouped_weight_grad<T, Tile, false><<<grid, Tile::THREADS, 0, a.stream>>>(
            x, x_low, g, g_low, a.R, a.cin, a.cout, a.off, a.N, p.rows, gw, gb, wide, a.workspace, p.slots, items, n_tiles, m_tiles, shortest);
    return hipGetLastError();
}

template <class T, class PT, class OUT, int TERMS, class RowTile>
hipError_t launch_both(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide_x, bool wide_w,
                       int64_t row_tiles, int64_t items) {
    using WeightTile = SmallWeightTile<T, PT, OUT, TERMS>;
    const int n_tiles = ceil_div(a.cin, WeightTile::BN), m_tiles = ceil_div(a.cout, WeightTile::BM);
    const unsigned weights = run_grid<kPieceRun>(items), rows = run_grid<kRun>(row_tiles);
    const auto both = vec ? grouped_both_grads<T, RowTile, WeightTile, true> : grouped_both_grads<T, RowTile, WeightTile, false>;
    both<<<weights + rows, RowTile::THREADS, 0, a.stream>>>(
        static_cast<const PT*>(a.x), static_cast<const PT*>(a.x_low), static_cast<const T*>(a.grad_y),
        static_cast<const T*>(a.grad_y_low), a.R, a.cin, a.cout, a.off, a.N, static_cast<const PT*>(a.weight),
        static_cast<const PT*>(a.weight_low), static_cast<OUT*>(a.grad_x), wide_x, row_tiles, ceil_div(a.cin, RowTile::BN), rows,
        weights, p.rows, static_cast<OUT*>(a.grad_weight), static_cast<OUT*>(a.grad_bias), wide_w, a.workspace, p.slots, items,
        n_tiles, m_tiles);
    return hipGetLastError();
}

// false: the two are not launched together.
template <class T, class PT, class OUT, int TERMS>
bool launch_together(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide_x, bool wide_w, hipError_t& err) {
    if (!a.grad_x || !grouped_together(a.R, a.N, a.cin, a.cout, sizeof(T) == 2)) return false;
    const bool few_rows = a.R <= 16 * a.N;
    const int side = SmallWeightTile<T, PT, OUT, TERMS>::BN;
    const int64_t row_tiles = most_row_tiles(a.R, a.N, few_rows ? 16 : 128) * ceil_div(a.cin, 64);
    const int64_t items = (a.R / p.rows + a.N) * ceil_div(a.cin, side) * ceil_div(a.cout, side);
    if (few_rows)
        err = launch_both<T, PT, OUT, TERMS, RowsProduct<T, PT, OUT, TERMS, false, 64, 16, 4, 1, 4>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    else if constexpr (!__is_same(T, PT))
        err = hipErrorInvalidValue;
    else if (a.cin <= 16)
        err = launch_both<T, PT, OUT, TERMS, RowsProduct<T, PT, OUT, TERMS, false, 16, 128, 1, 4, 2>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    else
        err = launch_both<T, PT, OUT, TERMS, RowsProduct<T, PT, OUT, TERMS, false, 64, 128, 1, 4, 2>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    return true;
}

// How a group's values are shared out when its pieces are added.
inline bool add_split(int64_t values) { return values <= 65536; }
inline int64_t add_blocks(int64_t values) {
    const int64_t each = add_split(values) ? kAddValues<true> : kAddValues<false>;
    return (values + each - 1) / each;
}

template <class T>
hipError_t add_pieces(const GroupedLinearArgs& a, const GroupedPieces& p) {
    const int64_t size = (int64_t)a.cin * a.cout, values = size + a.cout;
    const int64_t blocks = !add_split(values) && add_blocks(values) > 256 ? 256 : add_blocks(values);
    const auto add = add_split(values) ? grouped_add_pieces<T, true> : grouped_add_pieces<T, false>;
    add<<<(unsigned)(blocks * a.N), 256, 0, a.stream>>>(a.off, a.N, a.R, p.rows, values, grouped_piece_values(a.cin, a.cout), size,
                                                        a.workspace, p.slots, (unsigned)blocks, static_cast<T*>(a.grad_weight),
                                                        static_cast<T*>(a.grad_bias));
    return hipGetLastError();
}

template <class T>
hipError_t launch_forward(const GroupedLinearArgs& a) {
    if (a.R == 0) return hipSuccess;
    const bool in16 = a.cin % (16 / sizeof(T)) == 0, out16 = a.cout % (16 / sizeof(T)) == 0;   // rows of whole 16 bytes
    timing_begin(kKGroupedLinearFwd, a.stream);
    const hipError_t err = launch_rows<T, T, T, 1, true>(a, static_cast<const T*>(a.x), a.cin, static_cast<const T*>(a.bias),
                                                          static_cast<T*>(a.y), a.cout,
                                                          in16 && aligned16(a.x) && aligned16(a.weight),
                                                          out16 && aligned16(a.y));
    timing_end(kKGroupedLinearFwd, a.stream);
    return err;
}

template <class T, class PT, class OUT, int TERMS>
hipError_t launch_backward(const GroupedLinearArgs& a) {
    const bool in16 = a.cin % (16 / sizeof(T)) == 0, out16 = a.cout % (16 / sizeof(T)) == 0;   // rows of whole 16 bytes
    timing_begin(kKGroupedLinearBwd, a.stream);
    hipError_t err = hipSuccess;
    const bool weights = (a.grad_weight || a.grad_bias) && a.N > 0;
    const bool whole = in16 && out16 && aligned16(a.grad_y) && aligned16(a.grad_y_low);
    const bool vec_rows = whole && aligned16(a.weight) && aligned16(a.weight_low);
    const bool vec_weights = whole && aligned16(a.x) && aligned16(a.x_low);
    const bool wide_x = in16 && aligned16(a.grad_x), wide_w = in16 && aligned16(a.grad_weight);
    GroupedPieces p = weights ? grouped_pieces(a.R, a.N, a.cin, a.cout, sizeof(T) == 2) : GroupedPieces{};
    if (a.long_only) p = {1 << 30, p.side, 0};
    const bool together = weights && !a.long_only && launch_together<T, PT, OUT, TERMS>(a, p, vec_rows && vec_weights, wide_x, wide_w, err);
    if (!together && a.grad_x && a.R > 0)
        err = launch_rows<T, PT, OUT, TERMS, false>(a, static_cast<const T*>(a.grad_y), a.cout, (const OUT*)nullptr,
                                                    static_cast<OUT*>(a.grad_x), a.cin, vec_rows, wide_x);
    if (err == hipSuccess && weights) {
        const int side = grouped_weight_side(p, vec_weights);
        bool done = together;
        if constexpr (sizeof(T) == 2 && __is_same(T, PT))
            if (!done && side == 256) {
                err = launch_weight_tile<T, WeightProduct<T, PT, OUT, TERMS, 256, 2, 4>>(a, p, true, wide_w);
                done = true;
            }
        if constexpr (__is_same(T, PT))
            if (!done && side == 128) {
                err = launch_weight_tile<T, WeightProduct<T, PT, OUT, TERMS, 128, 2, 2>>(a, p, vec_weights, wide_w);
                done = true;
            }
        if (!done) err = launch_weight_tile<T, SmallWeightTile<T, PT, OUT, TERMS>>(a, p, vec_weights, wide_w);
        if (err == hipSuccess && p.slots > 0) {
            err = add_pieces<OUT>(a, p);
        }
    }
    timing_end(kKGroupedLinearBwd, a.stream);
    return err;
}

}  // namespace
}  // namespace dmr

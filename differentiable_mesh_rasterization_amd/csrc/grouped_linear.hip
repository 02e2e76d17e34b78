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
#include "grouped_tiles.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

// y = x W^T + b (WK: the weight's contiguous direction is summed over) or
// grad_x = g W (!WK), row tile by row tile. `n_out` is the width of `out`,
// `k_in` that of `rows_in`; the weight of a group is [n_out][k_in] if WK and
// [k_in][n_out] if not.
template <class T, class Tile, bool WK, bool VEC>
__device__ __forceinline__ void rows_of_workgroup(char* lds, uint32_t block, uint32_t blocks,
                                                  const T* __restrict__ rows_in, int64_t R, int k_in,
                                                  const int64_t* __restrict__ off, int64_t N,
                                                  const T* __restrict__ weight, int n_out, const T* __restrict__ bias,
                                                  T* __restrict__ out, bool wide, int64_t tiles, int n_tiles,
                                                  uint32_t places) {
    const int tid = threadIdx.x;
    walk_row_tiles<T, Tile, VEC>(
        lds, block, blocks, rows_in, R, k_in, off, N, tiles, n_tiles, places,
        [&](const RowTile& at, int n0) {
            const T* w = weight + at.group * (int64_t)n_out * k_in + (WK ? (int64_t)n0 * k_in : (int64_t)n0);
            return typename Tile::Source{w, WK ? k_in : n_out, n_out - n0};
        },
        [](const RowTile&, int) { return typename Tile::Zero(); },
        [](const RowTile&, int) { return 0; },
        [&](Tile& t, const RowTile& at, int n0, int) {
            store_tile<T, Tile>(t, out + at.first * (int64_t)n_out, n_out, at.rows, n0, n_out,
                                bias ? bias + at.group * (int64_t)n_out : nullptr, wide, tid);
        });
}

template <class T, class Tile, bool WK, bool VEC>
__global__ __launch_bounds__(Tile::THREADS) void grouped_rows(const T* __restrict__ rows_in, int64_t R, int k_in,
                                                              const int64_t* __restrict__ off, int64_t N,
                                                              const T* __restrict__ weight, int n_out,
                                                              const T* __restrict__ bias, T* __restrict__ out, bool wide,
                                                              int64_t tiles, int n_tiles, uint32_t places) {
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    rows_of_workgroup<T, Tile, WK, VEC>(lds, blockIdx.x, gridDim.x, rows_in, R, k_in, off, N, weight, n_out, bias, out, wide,
                                        tiles, n_tiles, places);
}

// ---------------------------------------------------------------------------
// gradient of the weights: a product over each group's rows
// ---------------------------------------------------------------------------
template <class T, class Tile, bool VEC>
__device__ __forceinline__ void weight_grad_of_workgroup(
    char* lds, uint32_t block, const T* __restrict__ x, const T* __restrict__ g, int64_t R, int cin, int cout,
    const int64_t* __restrict__ off, int64_t N, int per, T* __restrict__ grad_weight, T* __restrict__ grad_bias, bool wide,
    float* __restrict__ slots, int64_t slot_count, int64_t items, int n_tiles, int m_tiles) {
    const int64_t id = tile_of_workgroup<kPieceRun>(block);
    if (id >= items) return;
    const int tiles = n_tiles * m_tiles;
    const Piece at = find_piece(off, N, R, per, (int)(id / tiles));
    if (at.group < 0 || at.slot >= slot_count) return;
    const int tile = (int)(id % tiles);
    const int n0 = (tile % n_tiles) * Tile::BN, m0 = (tile / n_tiles) * Tile::BM;
    const int tid = threadIdx.x;
    const bool sums = n0 == 0 && grad_bias != nullptr;
    if (!grad_weight && !sums) return;
    Tile t;
    t.template run<VEC>(lds, typename Tile::Source{x + at.first * cin + n0, cin, cin - n0},
                        {g + at.first * cout + m0, cout, cout - m0}, at.rows, tid, sums);
    const int rows = cout - m0 < Tile::BM ? cout - m0 : Tile::BM;
    const int lane = tid & 63;
    const bool first_n = Tile::n_of(tid, 0) == 0 && lane < 16;   // one lane per m holds the row's sum
    if (at.slot < 0) {
        if (grad_weight)
            store_tile<T, Tile>(t, grad_weight + (at.group * cout + m0) * (int64_t)cin, cin, rows, n0, cin,
                                (const T*)nullptr, wide, tid);
        if (sums && first_n)
#pragma unroll
            for (int b = 0; b < Tile::MT; ++b) {
                const int m = Tile::m_of(tid, b);
                if (m < rows) grad_bias[at.group * cout + m0 + m] = (T)t.ones[b][0];
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
    const T* __restrict__ x, const T* __restrict__ g, int64_t R, int cin, int cout, const int64_t* __restrict__ off,
    int64_t N, int per, T* __restrict__ grad_weight, T* __restrict__ grad_bias, bool wide, float* __restrict__ slots,
    int64_t slot_count, int64_t items, int n_tiles, int m_tiles) {
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    weight_grad_of_workgroup<T, Tile, VEC>(lds, blockIdx.x, x, g, R, cin, cout, off, N, per, grad_weight, grad_bias, wide,
                                           slots, slot_count, items, n_tiles, m_tiles);
}

// Both gradients in one launch: the workgroups of the weight's, whose chains
// are the longer ones, and then the rows'.
template <class T, class RowTile, class WeightTile, bool VEC>
__global__ __launch_bounds__(RowTile::THREADS) void grouped_both_grads(
    const T* __restrict__ x, const T* __restrict__ g, int64_t R, int cin, int cout, const int64_t* __restrict__ off,
    int64_t N, const T* __restrict__ weight, T* __restrict__ grad_x, bool wide_x, int64_t row_tiles, int row_n_tiles,
    uint32_t row_places, uint32_t weight_places, int per, T* __restrict__ grad_weight, T* __restrict__ grad_bias,
    bool wide_w, float* __restrict__ slots, int64_t slot_count, int64_t items, int n_tiles, int m_tiles) {
    static_assert(RowTile::THREADS == WeightTile::THREADS, "");
    __shared__ alignas(16) char lds[RowTile::kLdsBytes > WeightTile::kLdsBytes ? RowTile::kLdsBytes : WeightTile::kLdsBytes];
    if (blockIdx.x < weight_places)
        weight_grad_of_workgroup<T, WeightTile, VEC>(lds, blockIdx.x, x, g, R, cin, cout, off, N, per, grad_weight, grad_bias,
                                                     wide_w, slots, slot_count, items, n_tiles, m_tiles);
    else
        rows_of_workgroup<T, RowTile, false, VEC>(lds, blockIdx.x - weight_places, row_places, g, R, cout, off, N, weight,
                                                  cin, (const T*)nullptr, grad_x, wide_x, row_tiles, row_n_tiles,
                                                  row_places);
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
hipError_t launch_rows_tile(const GroupedLinearArgs& a, const T* in, int k_in, const T* bias, T* out, int n_out, bool vec,
                            bool wide) {
    const int n_tiles = ceil_div(n_out, Tile::BN);
    const int64_t tiles = most_row_tiles(a.R, a.N, Tile::BM) * n_tiles;
    const unsigned places = run_grid<kRun>(tiles);
    if (places == 0) return hipErrorInvalidValue;
    // as many workgroups as the device holds at a time (a multiple of 8 kRun)
    constexpr unsigned kHeld = 256 * (160 * 1024 / Tile::kLdsBytes);
    const unsigned grid = places > kHeld ? kHeld : places;
    const T* w = static_cast<const T*>(a.weight);
    if (vec)
        grouped_rows<T, Tile, WK, true><<<grid, Tile::THREADS, 0, a.stream>>>(in, a.R, k_in, a.off, a.N, w, n_out, bias, out,
                                                                              wide, tiles, n_tiles, places);
    else if constexpr (Tile::BN < 256)   // the largest tiles have no form for unaligned arrays
        grouped_rows<T, Tile, WK, false><<<grid, Tile::THREADS, 0, a.stream>>>(in, a.R, k_in, a.off, a.N, w, n_out, bias, out,
                                                                               wide, tiles, n_tiles, places);
    return hipGetLastError();
}

template <class T, bool WK>
hipError_t launch_rows(const GroupedLinearArgs& a, const T* in, int k_in, const T* bias, T* out, int n_out, bool vec,
                       bool wide) {
    const RowsTile t = grouped_rows_tile(a.R, a.N, n_out, sizeof(T) == 2, !WK, vec);
    if (t.rows == 16)
        return launch_rows_tile<T, TileProduct<T, 64, 16, 4, 1, WK, true, 4>, WK>(a, in, k_in, bias, out, n_out, vec, wide);
    if (t.columns == 16)
        return launch_rows_tile<T, TileProduct<T, 16, 128, 1, 4, WK, true, 2>, WK>(a, in, k_in, bias, out, n_out, vec, wide);
    if constexpr (sizeof(T) == 2) {
        if (t.columns == 64 && t.rows == 256)
            return launch_rows_tile<T, TileProduct<T, 64, 256, 1, 8, WK, true, 2>, WK>(a, in, k_in, bias, out, n_out, vec,
                                                                                         wide);
        if (t.columns == 256)
            return launch_rows_tile<T, TileProduct<T, 256, 256, 4, 2, WK, true, 2>, WK>(a, in, k_in, bias, out, n_out, vec,
                                                                                           wide);
    }
    if (t.columns == 64)
        return launch_rows_tile<T, TileProduct<T, 64, 128, 1, 4, WK, true, 2>, WK>(a, in, k_in, bias, out, n_out, vec, wide);
    return launch_rows_tile<T, TileProduct<T, 128, 128, 2, 4, WK, true, 2>, WK>(a, in, k_in, bias, out, n_out, vec, wide);
}

template <class T>
using SmallWeightTile = TileProduct<T, 64, 64, 2, 2, false, false, 2, true>;

template <class T, class Tile>
hipError_t launch_weight_tile(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide) {
    const int n_tiles = ceil_div(a.cin, Tile::BN), m_tiles = ceil_div(a.cout, Tile::BM);
    const int64_t items = (a.R / p.rows + a.N) * n_tiles * m_tiles;
    const unsigned grid = run_grid<kPieceRun>(items);
    if (grid == 0) return hipErrorInvalidValue;
    const T *x = static_cast<const T*>(a.x), *g = static_cast<const T*>(a.grad_y);
    T *gw = static_cast<T*>(a.grad_weight), *gb = static_cast<T*>(a.grad_bias);
    if (vec)
        grouped_weight_grad<T, Tile, true><<<grid, Tile::THREADS, 0, a.stream>>>(
            x, g, a.R, a.cin, a.cout, a.off, a.N, p.rows, gw, gb, wide, a.workspace, p.slots, items, n_tiles, m_tiles);
    else if constexpr (Tile::BN < 256)
        grouped_weight_grad<T, Tile, false><<<grid, Tile::THREADS, 0, a.stream>>>(
            x, g, a.R, a.cin, a.cout, a.off, a.N, p.rows, gw, gb, wide, a.workspace, p.slots, items, n_tiles, m_tiles);
    return hipGetLastError();
}

template <class T, class RowTile>
hipError_t launch_both(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide_x, bool wide_w,
                       int64_t row_tiles, int64_t items) {
    using WeightTile = SmallWeightTile<T>;
    const int n_tiles = ceil_div(a.cin, WeightTile::BN), m_tiles = ceil_div(a.cout, WeightTile::BM);
    const unsigned weights = run_grid<kPieceRun>(items), rows = run_grid<kRun>(row_tiles);
    const auto both = vec ? grouped_both_grads<T, RowTile, WeightTile, true> : grouped_both_grads<T, RowTile, WeightTile, false>;
    both<<<weights + rows, RowTile::THREADS, 0, a.stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.grad_y), a.R, a.cin, a.cout, a.off, a.N,
        static_cast<const T*>(a.weight), static_cast<T*>(a.grad_x), wide_x, row_tiles, ceil_div(a.cin, RowTile::BN), rows,
        weights, p.rows, static_cast<T*>(a.grad_weight), static_cast<T*>(a.grad_bias), wide_w, a.workspace, p.slots, items,
        n_tiles, m_tiles);
    return hipGetLastError();
}

// false: the two are not launched together.
template <class T>
bool launch_together(const GroupedLinearArgs& a, const GroupedPieces& p, bool vec, bool wide_x, bool wide_w, hipError_t& err) {
    if (!a.grad_x || !grouped_together(a.R, a.N, a.cin, a.cout, sizeof(T) == 2)) return false;
    const bool few_rows = a.R <= 16 * a.N;
    const int side = SmallWeightTile<T>::BN;
    const int64_t row_tiles = most_row_tiles(a.R, a.N, few_rows ? 16 : 128) * ceil_div(a.cin, 64);
    const int64_t items = (a.R / p.rows + a.N) * ceil_div(a.cin, side) * ceil_div(a.cout, side);
    if (few_rows)
        err = launch_both<T, TileProduct<T, 64, 16, 4, 1, false, true, 4>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    else if (a.cin <= 16)
        err = launch_both<T, TileProduct<T, 16, 128, 1, 4, false, true, 2>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    else
        err = launch_both<T, TileProduct<T, 64, 128, 1, 4, false, true, 2>>(a, p, vec, wide_x, wide_w, row_tiles, items);
    return true;
}

// How a group's values are shared out when its pieces are added.
bool add_split(int64_t values) { return values <= 65536; }
int64_t add_blocks(int64_t values) {
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
hipError_t launch_all(const GroupedLinearArgs& a, bool backward) {
    const T* bias = static_cast<const T*>(a.bias);
    const bool in16 = a.cin % (16 / sizeof(T)) == 0, out16 = a.cout % (16 / sizeof(T)) == 0;   // rows of whole 16 bytes
    if (!backward) {
        if (a.R == 0) return hipSuccess;
        timing_begin(kKGroupedLinearFwd, a.stream);
        const hipError_t err = launch_rows<T, true>(a, static_cast<const T*>(a.x), a.cin, bias, static_cast<T*>(a.y), a.cout,
                                                    in16 && aligned16(a.x) && aligned16(a.weight), out16 && aligned16(a.y));
        timing_end(kKGroupedLinearFwd, a.stream);
        return err;
    }
    timing_begin(kKGroupedLinearBwd, a.stream);
    hipError_t err = hipSuccess;
    const bool weights = (a.grad_weight || a.grad_bias) && a.N > 0;
    const bool whole = in16 && out16 && aligned16(a.grad_y);
    const bool vec_rows = whole && aligned16(a.weight), vec_weights = whole && aligned16(a.x);
    const bool wide_x = in16 && aligned16(a.grad_x), wide_w = in16 && aligned16(a.grad_weight);
    const GroupedPieces p = weights ? grouped_pieces(a.R, a.N, a.cin, a.cout, sizeof(T) == 2) : GroupedPieces{};
    const bool together = weights && launch_together<T>(a, p, vec_rows && vec_weights, wide_x, wide_w, err);
    if (!together && a.grad_x && a.R > 0)
        err = launch_rows<T, false>(a, static_cast<const T*>(a.grad_y), a.cout, (const T*)nullptr, static_cast<T*>(a.grad_x),
                                    a.cin, vec_rows, wide_x);
    if (err == hipSuccess && weights) {
        const int side = grouped_weight_side(p, vec_weights);
        bool done = together;
        if constexpr (sizeof(T) == 2)
            if (!done && side == 256) {
                err = launch_weight_tile<T, TileProduct<T, 256, 256, 2, 4, false, false, 2, true>>(a, p, true, wide_w);
                done = true;
            }
        if (!done)
            err = side == 64 ? launch_weight_tile<T, SmallWeightTile<T>>(a, p, vec_weights, wide_w)
                             : launch_weight_tile<T, TileProduct<T, 128, 128, 2, 2, false, false, 2, true>>(a, p, vec_weights,
                                                                                                           wide_w);
        if (err == hipSuccess && p.slots > 0) {
            err = add_pieces<T>(a, p);
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

// The tile side, the rows of a piece of the weight gradient, and the slots
// that the pieces of groups longer than one piece can take: a group of
// r > rows has at most 2 floor(r / rows) of them.
GroupedPieces grouped_pieces(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    // 256 only where the groups' tiles are many before any piece is cut (2
    // groups of 256 to 512, 16384 rows in bfloat16: 59 us with, 50 without)
    const int64_t weights256 = N * ((cin + 255) / 256) * ((cout + 255) / 256);
    const bool large = half && cin > 128 && cout > 128 && R >= 512 * N && weights256 >= 64;
    const int64_t side = cin <= 64 && cout <= 64 ? 64 : large ? 256 : 128;
    const int64_t tiles = ((cin + side - 1) / side) * ((cout + side - 1) / side);
    // a piece is at most one of the places' shares of the work: 256 compute
    // units with one workgroup of the largest tiles, two or four of the others
    const int64_t want = (side == 256 ? 256 : side == 128 ? 512 : 1024) / tiles;
    int64_t rows = want > 0 ? (R + want - 1) / want : R;
    rows = (rows + 127) / 128 * 128;
    rows = rows < 512 ? 512 : rows > 8192 ? 8192 : rows;
    if (R <= 1024) rows = 1024;   // short enough to need no second launch
    return {(int)rows, (int)side, R > rows ? 2 * (R / rows) : 0};
}

// The largest tiles have no form for arrays that are not aligned.
int grouped_weight_side(const GroupedPieces& p, bool vec) { return p.side == 256 && !vec ? 128 : p.side; }

// The tile by the widths and by how many there are: the larger, the fewer
// bytes for a product, but they have to fill 256 compute units. (bfloat16,
// forward: 2048 rows of 512 to 512, 19.3 us with 256 x 256 tiles, 11.0 with
// 128 x 128, 9.4 with 64 x 128; 8192 of 1024 to 1024, 128 tiles of 256 x 256,
// 35.3 and 31.5 with 128 x 128, but the backward's transposed weight 103 and
// 117. 2^20 rows of 64 to 64: 60 us with 64 x 256, 63 with 64 x 128. 217632 rows
// of 64 to 3 in float32: 17.7 us with 16 x 256, 14.3 with 16 x 128.)
RowsTile grouped_rows_tile(int64_t R, int64_t N, int32_t n_out, bool half, bool backward, bool vec) {
    const auto tiles = [&](int bn, int bm) { return (R / bm + 1) * ceil_div(n_out, bn); };
    if (R <= 16 * N) return {64, 16};
    if (n_out <= 16) return {16, 128};
    if (n_out <= 64 || tiles(128, 128) < 256) return half && tiles(64, 256) >= 256 ? RowsTile{64, 256} : RowsTile{64, 128};
    if (half && vec && n_out > 128 && R >= 512 * N && tiles(256, 256) >= (backward ? 112 : 224)) return {256, 256};
    return {128, 128};
}

// Both gradients in one launch where small tiles serve both: narrow layers,
// and calls of so few tiles that one gradient's leave the device unfilled.
// What one waits for, the other fills, and the upstream gradients are read
// while they are near. (One launch against two, us.
// Float32: 217632 rows of 64 to 64, 53 and 64, of 16 to 256, 100 and 172;
// 8192 of 256 to 256, 37 and 70; 2048 of 1024 to 1024, 1552 tiles, 115 and
// 94. 16 bits: 1003 rows of 37 to 19, 15.9 and 20.7; 2^20 of 64 to 64, 120
// and 129; 8192 of 256 to 256, 18.4 and 30.8; 16384 of 256 to 512, 2112
// tiles, 41 and 49; 64 groups of one row, 1024 to 1024, 16384 tiles, 187 and
// 118; 166428 rows of 240 to 64, 61 and 66, but 400000 of 512 to 64, 276 and
// 261.)
bool grouped_together(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    if (R == 0) return false;
    const int64_t few = half ? 2304 : 1536;
    const bool narrow = cin <= 64 || (cin <= 256 && cout <= 64);
    const int64_t row_tiles = most_row_tiles(R, N, R <= 16 * N ? 16 : 128) * ceil_div(cin, 64);
    const int64_t items = (R / grouped_pieces(R, N, cin, cout, half).rows + N) * ceil_div(cin, 64) * ceil_div(cout, 64);
    return (row_tiles + items <= few || narrow) && row_tiles + items <= 1 << 23;
}

bool grouped_add_fits(int64_t N, int32_t cin, int32_t cout) {
    return add_blocks((int64_t)cin * cout + cout) * N <= kMaxWorkItems / 256;
}

bool grouped_sums_fit(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    const GroupedPieces p = grouped_pieces(R, N, cin, cout, half);
    const int side = grouped_weight_side(p, false);   // of the tiles that are more
    const int64_t items = (R / p.rows + N) * ceil_div(cin, side) * ceil_div(cout, side), round = 8 * kPieceRun;
    if ((items + round - 1) / round * round > kMaxWorkItems / 256) return false;
    return p.slots == 0 || grouped_add_fits(N, cin, cout);
}

hipError_t launch_grouped_add_pieces(const GroupedLinearArgs& a, const GroupedPieces& p) {
    switch (a.dtype) {
        case DMR_FLOAT32: return add_pieces<float>(a, p);
        case DMR_FLOAT16: return add_pieces<_Float16>(a, p);
        case DMR_BFLOAT16: return add_pieces<__bf16>(a, p);
    }
    return hipErrorInvalidValue;
}
hipError_t launch_grouped_linear_forward(const GroupedLinearArgs& a) { return launch_typed(a, false); }
hipError_t launch_grouped_linear_backward(const GroupedLinearArgs& a) { return launch_typed(a, true); }

}  // namespace dmr

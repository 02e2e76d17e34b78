// Gated layers with one pair of weights per group of a packed batch, on
// gfx950: for the rows r of group n, with the weight's two planes A and U,
//     a = A_n x_r + a_n,  u = U_n x_r + u_n,  y_r = act(a) u,
// and the backward pass
//     da = g_r u act'(a),  du = g_r act(a),
// of which the gradients of x, of both weights and of both biases are those of
// a linear layer with the outputs [da du] and the weight [A; U].
//
// Forward, a workgroup's tile holds the same columns of both planes (the
// products share the rows' fragments), so a lane has a and u of the same value
// in its accumulators and neither goes to memory. Backward, the same products
// are computed again, with da and du instead of y as their result: only x is
// kept of the forward pass, and act's arguments are float32. (Keeping a and u
// would take 4 F values of traffic for 4 F C operations, even at C of about
// 500 in 16 bits, and round them.) [da du] is rounded to the type, which is
// what the matrix instructions of the two products with it take.
#include "dmr_internal.h"
#include "grouped_tiles.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

// Activation and derivative. 1 / (1 + e^-z) and 1 minus it are formed so that
// neither loses digits to the other; e^-z passes float32's range harmlessly
// (1 / inf = 0).
struct Act {
    float value, slope;
};

__device__ __forceinline__ void logistic(float z, float& s, float& rest) {
    const float t = __builtin_amdgcn_exp2f(z * -1.44269504f);
    s = __builtin_amdgcn_rcpf(1.0f + t);
    rest = z >= 0.0f ? t * s : 1.0f - s;   // t may be infinite below zero
}

template <int KIND>
__device__ __forceinline__ Act activate(float a);
template <>
__device__ __forceinline__ Act activate<DMR_SILU>(float a) {
    float s, rest;
    logistic(a, s, rest);
    return {a * s, __builtin_fmaf(a * s, rest, s)};
}
template <>
__device__ __forceinline__ Act activate<DMR_SIGMOID>(float a) {
    float s, rest;
    logistic(a, s, rest);
    return {s, s * rest};
}
template <>
__device__ __forceinline__ Act activate<DMR_GELU_TANH>(float a) {
    // (1 + tanh z) / 2 is the logistic function of 2 z, z = k (a + c a^3)
    constexpr float k2 = 1.59576912f, c = 0.044715f;   // 2 sqrt(2 / pi)
    const float aa = a * a;
    float s, rest;
    logistic(k2 * a * __builtin_fmaf(c, aa, 1.0f), s, rest);
    return {a * s, __builtin_fmaf(a * s * rest, k2 * __builtin_fmaf(3.0f * c, aa, 1.0f), s)};
}
template <>
__device__ __forceinline__ Act activate<DMR_GELU>(float a) {
    // the normal distribution below a, without cancellation for a < 0
    const float below = 0.5f * erfcf(a * -0.70710678f);
    const float density = 0.39894228f * __builtin_amdgcn_exp2f(a * a * -0.72134752f);
    return {a * below, __builtin_fmaf(a, density, below)};
}

template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    if (act == DMR_SILU) f([](float a) { return activate<DMR_SILU>(a); });
    else if (act == DMR_GELU) f([](float a) { return activate<DMR_GELU>(a); });
    else if (act == DMR_GELU_TANH) f([](float a) { return activate<DMR_GELU_TANH>(a); });
    else f([](float a) { return activate<DMR_SIGMOID>(a); });
}

// One plane's blocks of a tile, for store_tile.
template <class Tile>
struct Plane {
    static constexpr int NT = Tile::PN, MT = Tile::MT;
    static constexpr bool PAIRED = Tile::PAIRED;
    f32x4 acc[NT][MT];
    static __device__ __forceinline__ int n_of(int tid, int a) { return Tile::n_of(tid, a); }
    static __device__ __forceinline__ int m_of(int tid, int b) { return Tile::m_of(tid, b); }
};

// Adds the biases (or nothing) to both planes of a tile.
template <class T, class Tile>
__device__ __forceinline__ void add_biases(Tile& t, const T* __restrict__ bias, int F, int n0, int tid) {
    if (!bias) return;
#pragma unroll
    for (int a = 0; a < Tile::NT; ++a) {
        f32x4 add;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = n0 + Tile::n_of(tid, a) + i;   // past the end: any value, not stored
            add[i] = (float)bias[(a / Tile::PN) * (int64_t)F + (at < F ? at : F - 1)];
        }
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) t.acc[a][b] += add;
    }
}

// Values n .. n + 3 of row m of a [rows, N] array; any value where there is none.
template <class T>
__device__ __forceinline__ f32x4 load4(const T* __restrict__ row, int n, int N, bool exists) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (exists && n + 4 <= N) {
        T t[4];
        __builtin_memcpy(t, row + n, sizeof(t));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)t[i];
    } else if (exists) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) v[i] = (float)row[n + i];
    }
    return v;
}

// GRAD: writes [da du] of the rows to `out` [R, 2 F] from grad_y [R, F];
// otherwise y to `out` [R, F].
template <class T, class Tile, bool VEC, bool GRAD>
__global__ __launch_bounds__(Tile::THREADS) void grouped_gated(const T* __restrict__ x, int64_t R, int C,
                                                               const int64_t* __restrict__ off, int64_t N,
                                                               const T* __restrict__ weight, const T* __restrict__ bias, int F,
                                                               int act, const T* __restrict__ grad_y, T* __restrict__ out,
                                                               bool wide, int64_t tiles, int n_tiles, uint32_t places) {
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    const int tid = threadIdx.x;
    walk_row_tiles<T, Tile, VEC>(
        lds, blockIdx.x, gridDim.x, x, R, C, off, N, tiles, n_tiles, places,
        [&](const RowTile& at, int n0) {
            const T* w = weight + (at.group * 2 * F + n0) * (int64_t)C;
            return typename Tile::Planes(typename Tile::Source{w, C, F - n0},
                                         typename Tile::Source{w + (int64_t)F * C, C, F - n0});
        },
        [&](Tile& t, const RowTile& at, int n0) {
            add_biases<T, Tile>(t, bias ? bias + at.group * 2 * F : nullptr, F, n0, tid);
            Plane<Tile> first, second;
            with_activation(act, [&](auto&& activation) {
#pragma unroll
                for (int b = 0; b < Tile::MT; ++b) {
                    const int m = Tile::m_of(tid, b);
#pragma unroll
                    for (int a = 0; a < Tile::PN; ++a) {
                        f32x4 g;
                        if constexpr (GRAD)
                            g = load4<T>(grad_y + (at.first + m) * F, n0 + Tile::n_of(tid, a), F, m < at.rows);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const Act v = activation(t.acc[a][b][i]);
                            const float u = t.acc[a + Tile::PN][b][i];
                            if constexpr (GRAD) {
                                first.acc[a][b][i] = g[i] * u * v.slope;
                                second.acc[a][b][i] = g[i] * v.value;
                            } else {
                                first.acc[a][b][i] = v.value * u;
                            }
                        }
                    }
                }
            });
            constexpr int WIDTHS = GRAD ? 2 : 1;
            T* rows = out + at.first * (int64_t)F * WIDTHS;
            store_tile<T>(first, rows, (int64_t)F * WIDTHS, at.rows, n0, F, (const T*)nullptr, wide, tid);
            if constexpr (GRAD)
                store_tile<T>(second, rows + F, (int64_t)F * WIDTHS, at.rows, n0, F, (const T*)nullptr, wide, tid);
        });
}

template <class T, class Tile, bool GRAD>
hipError_t launch_tile(const GatedArgs& a, T* out, bool vec, bool wide) {
    const int n_tiles = ceil_div(a.F, Tile::COLUMNS);
    const int64_t tiles = most_row_tiles(a.R, a.N, Tile::BM) * n_tiles;
    const unsigned places = run_grid<kRun>(tiles);
    if (places == 0) return hipErrorInvalidValue;
    // as many workgroups as the device holds at a time (a multiple of 8 kRun)
    constexpr unsigned kHeld = 256 * (160 * 1024 / Tile::kLdsBytes);
    const unsigned grid = places > kHeld ? kHeld : places;
    const T *x = static_cast<const T*>(a.x), *w = static_cast<const T*>(a.weight), *bias = static_cast<const T*>(a.bias);
    const T* g = static_cast<const T*>(a.grad_y);
    if (vec)
        grouped_gated<T, Tile, true, GRAD><<<grid, Tile::THREADS, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, w, bias, a.F, a.act, g,
                                                                                 out, wide, tiles, n_tiles, places);
    else if constexpr (Tile::BN < 256)   // the largest tiles have no form for unaligned arrays
        grouped_gated<T, Tile, false, GRAD><<<grid, Tile::THREADS, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, w, bias, a.F, a.act, g,
                                                                                  out, wide, tiles, n_tiles, places);
    return hipGetLastError();
}

template <class T, int BN, int BM, int WN, int WM, int S>
using GatedTile = TileProduct<T, BN, BM, WN, WM, true, true, S, false, 2>;

template <class T, bool GRAD>
hipError_t launch_products(const GatedArgs& a, T* out) {
    constexpr int each = 16 / (int)sizeof(T);
    const bool vec = a.C % each == 0 && aligned16(a.x) && aligned16(a.weight);
    const bool wide = a.F % each == 0 && aligned16(out);
    const RowsTile t = gated_tile(a.R, a.N, a.F, sizeof(T) == 2, vec);
    if (t.rows == 16) return launch_tile<T, GatedTile<T, 128, 16, 4, 1, 4>, GRAD>(a, out, vec, wide);
    if (t.columns == 16) return launch_tile<T, GatedTile<T, 32, 128, 1, 4, 2>, GRAD>(a, out, vec, wide);
    if constexpr (sizeof(T) == 2)
        if (t.columns == 128) return launch_tile<T, GatedTile<T, 256, 256, 2, 4, 2>, GRAD>(a, out, vec, wide);
    if (t.columns == 32) return launch_tile<T, GatedTile<T, 64, 128, 1, 4, 2>, GRAD>(a, out, vec, wide);
    return launch_tile<T, GatedTile<T, 128, 128, 2, 4, 2>, GRAD>(a, out, vec, wide);
}

template <class T>
hipError_t launch_typed(const GatedArgs& a, bool backward) {
    if (!backward) return launch_products<T, false>(a, static_cast<T*>(a.y));
    if (a.R > 0) {
        const hipError_t err = launch_products<T, true>(a, reinterpret_cast<T*>(a.workspace));
        if (err != hipSuccess) return err;
    }
    // [da du] as the upstream gradient of a linear layer of 2 F outputs
    GroupedLinearArgs b{};
    b.x = a.x; b.R = a.R; b.cin = a.C; b.off = a.off; b.N = a.N; b.weight = a.weight; b.cout = 2 * a.F; b.dtype = a.dtype;
    b.grad_y = a.workspace; b.grad_x = a.grad_x; b.grad_weight = a.grad_weight; b.grad_bias = a.grad_bias;
    b.workspace = reinterpret_cast<float*>(a.workspace + gated_rows_bytes(a.R, a.F, a.dtype));
    b.stream = a.stream;
    return launch_grouped_linear_backward(b);
}

}  // namespace

// The tile by the columns of each plane and by how many there are, as for
// linear layers: the larger, the fewer bytes for a product, but they have to
// fill 256 compute units.
RowsTile gated_tile(int64_t R, int64_t N, int32_t F, bool half, bool vec) {
    const auto tiles = [&](int columns, int rows) { return (R / rows + 1) * ceil_div(F, columns); };
    if (R <= 16 * N) return {64, 16};
    if (F <= 16) return {16, 128};
    if (half && vec && F > 64 && R >= 512 * N && tiles(128, 256) >= 224) return {128, 256};
    if (F <= 32 || tiles(64, 128) < 256) return {32, 128};
    return {64, 128};
}

hipError_t launch_gated(const GatedArgs& a, bool backward) {
    const KernelId id = backward ? kKGatedLinearBwd : kKGatedLinearFwd;
    timing_begin(id, a.stream);
    hipError_t err = hipErrorInvalidValue;
    switch (a.dtype) {
        case DMR_FLOAT32: err = launch_typed<float>(a, backward); break;
        case DMR_FLOAT16: err = launch_typed<_Float16>(a, backward); break;
        case DMR_BFLOAT16: err = launch_typed<__bf16>(a, backward); break;
    }
    timing_end(id, a.stream);
    return err;
}

}  // namespace dmr

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
// 500 in 16 bits, and round them.)
//
// In 16-bit layers [da du] is held as pairs of bfloat16, high + low, which keep
// 16 bits or more of it and float32's range: rounded to the type once, it would
// bring an error of the size of the results' own rounding into them, and in
// float16 gradients below 2^-25 would vanish and products of an upstream
// gradient with u past 65504 become infinite, whatever the sums over them are.
// The two products with it take two matrix instructions for one that way, or
// three with float16 operands, which are pairs of bfloat16 themselves.
#include <type_traits>

#include "dmr_internal.h"
#include "grouped_tiles.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

// Activation and derivative. The exponential's argument is rounded twice, which
// moves it by |z| 2^-23 relatively: so far are negative tails off. With the
// logistic function s of z, e^-z may pass float32's range (1 / inf = 0 then).
// 1 - s is off by 2^-24, which moves the derivative s + a s (1 - s) z' by a s z'
// 2^-24: no more than the rounding of a does. Sigmoid's derivative has no term
// beside s (1 - s), which is e s^2 with s and e = e^-|a| of the magnitude: both
// tails keep their digits (by 1 - s it is 7e-4 off at 10, and zero from 17 on).
struct Act {
    float value, slope;
};

// s of z = -log2(e) z_scaled.
__device__ __forceinline__ float logistic2(float z_scaled) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z_scaled));
}
constexpr float kLog2e = 1.44269504f;

template <int KIND>
__device__ __forceinline__ Act activate(float a);
template <>
__device__ __forceinline__ Act activate<DMR_SILU>(float a) {
    const float s = logistic2(a * -kLog2e), v = a * s;
    return {v, __builtin_fmaf(v, 1.0f - s, s)};
}
template <>
__device__ __forceinline__ Act activate<DMR_SIGMOID>(float a) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(a) * -kLog2e);
    const float s = __builtin_amdgcn_rcpf(1.0f + e), below = e * s;
    return {a < 0.0f ? below : s, below * s};
}
template <>
__device__ __forceinline__ Act activate<DMR_GELU_TANH>(float a) {
    // (1 + tanh z) / 2 is the logistic function of 2 z, z = k (a + c a^3)
    constexpr float k2 = 1.59576912f, c = 0.044715f;   // 2 sqrt(2 / pi)
    const float aa = __builtin_fminf(a * a, 1e8f);   // s is 0 or 1 long before; zero times infinity would be NaN
    const float s = logistic2(a * __builtin_fmaf(-kLog2e * k2 * c, aa, -kLog2e * k2)), v = a * s;
    return {v, __builtin_fmaf(v * (1.0f - s), __builtin_fmaf(3.0f * k2 * c, aa, k2), s)};
}
template <>
__device__ __forceinline__ Act activate<DMR_GELU>(float a) {
    // The normal distribution below -|a| is e^(-a^2 / 2) t Q(t), t = 1 / (1 +
    // 0.27 |a|), with Q of degree 8 fitted for the least relative error over
    // |a| <= 13.5 (2.5e-8, 3.5e-8 with its coefficients in float32, which a test
    // of these nine evaluates; 4e-7 as evaluated here): both tails keep their
    // digits but for the exponential's, and the derivative's density is the same
    // exponential.
    constexpr float q[9] = {0.107719538f, 0.10756075f, 0.101690539f, 0.0724933754f, 0.106836153f,
                            -0.0678442909f, 0.16864185f, -0.1259533f, 0.028855398f};
    const float e = __builtin_amdgcn_exp2f(a * a * -0.72134752f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.27f, __builtin_fabsf(a), 1.0f));
    float p = q[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = __builtin_fmaf(p, t, q[i]);
    const float tail = t * e * p, below = a < 0.0f ? tail : 1.0f - tail;
    return {a * below, __builtin_fmaf(a * 0.39894228f, e, below)};
}

template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    if (act == DMR_SILU) f([](float a) { return activate<DMR_SILU>(a); });
    else if (act == DMR_GELU) f([](float a) { return activate<DMR_GELU>(a); });
    else if (act == DMR_GELU_TANH) f([](float a) { return activate<DMR_GELU_TANH>(a); });
    else f([](float a) { return activate<DMR_SIGMOID>(a); });
}

// Where a lane's values of a tile go: rows [0, rows) of `out` (leading
// dimension ld), columns [n0, N). `wide`: `out` is 16-byte aligned and ld a
// multiple of 16 bytes.
template <class T>
struct TileOut {
    T* out;
    int64_t ld;
    int rows, n0, N;
    bool wide;
};

// Stores block b of a tile's rows, value(a) the four values of block a < NT: as
// soon as they are formed, which keeps them out of scratch memory.
template <class T, class Tile, int NT, class Value>
__device__ __forceinline__ void store_rows(const TileOut<T>& o, int b, int tid, Value&& value) {
    constexpr int STEP = Tile::PAIRED ? 2 : 1;              // blocks of n in a lane's 16 bytes
    constexpr bool CHUNKS = Tile::PAIRED || sizeof(T) == 4;   // a lane holds 16 bytes of a row
    const int m = Tile::m_of(tid, b);
    if (CHUNKS && o.wide) {
        // 32-bit offsets from the tile's corner; stores past the buffer's
        // range are dropped
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(o.out + o.n0, 0, kBufferRange, 0x00020000);
        const uint32_t line = (uint32_t)(o.ld * sizeof(T));
        const int left = o.N - o.n0;
#pragma unroll
        for (int a = 0; a < NT; a += 2 * STEP) {
            const u32x4 c0 = packed<T>(value(a), value(a + STEP - 1));
            const int na = Tile::n_of(tid, a);
            if constexpr (NT % (2 * STEP) == 0) {
                const u32x4 c1 = packed<T>(value(a + STEP), value(a + 2 * STEP - 1));
                const int nb = Tile::n_of(tid, a + STEP);
                store_row_pairs(c0, c1, tid, [&](bool odd, int chunk, u32x4 v) {
                    const int row = (m & ~1) | (odd ? 1 : 0), n = chunk ? nb : na;
                    const uint32_t off = (uint32_t)row * line + (uint32_t)n * (uint32_t)sizeof(T);
                    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, row < o.rows && n < left ? off : kNowhere, 0, 0);
                });
            } else {
                const uint32_t off = (uint32_t)m * line + (uint32_t)na * (uint32_t)sizeof(T);
                __builtin_amdgcn_raw_buffer_store_b128(c0, rsrc, m < o.rows && na < left ? off : kNowhere, 0, 0);
            }
        }
        return;
    }
    if (m >= o.rows) return;
    T* row = o.out + (int64_t)m * o.ld;
#pragma unroll
    for (int a = 0; a < NT; a += STEP) {
        const int n = o.n0 + Tile::n_of(tid, a);
        if (CHUNKS && n + 4 * STEP <= o.N) {
            const u32x4 v = packed<T>(value(a), value(a + STEP - 1));
            __builtin_memcpy(row + n, &v, 16);   // at whatever alignment it has
        } else {
#pragma unroll
            for (int s = 0; s < STEP; ++s) store4<T>(row, n + 4 * s, o.N, value(a + s));
        }
    }
}

// A lane's values of grad_y in a tile, 16 bytes of a row at a time where a
// lane's columns are that many; zero where there are none.
template <class T, class Tile>
struct Upstream {
    static constexpr bool CHUNKS = Tile::PAIRED || sizeof(T) == 4;
    static constexpr int STEP = Tile::PAIRED ? 2 : 1;   // blocks of n in one piece
    static constexpr int BYTES = STEP * 4 * (int)sizeof(T);
    uint32_t raw[Tile::MT][Tile::PN / STEP][BYTES / 4];

    // o: of grad_y
    __device__ __forceinline__ void load(const TileOut<const T>& o, int tid) {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(o.out + o.n0), 0, kBufferRange, 0x00020000);
        const uint32_t line = (uint32_t)(o.ld * sizeof(T));
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
#pragma unroll
            for (int a = 0; a < Tile::PN / STEP; ++a) {
                const int n = Tile::n_of(tid, a * STEP), left = o.N - o.n0 - n;
                if (CHUNKS && o.wide) {
                    const uint32_t off = m < o.rows && left > 0 ? (uint32_t)m * line + (uint32_t)n * (uint32_t)sizeof(T) : kNowhere;
                    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0);
                    __builtin_memcpy(raw[b][a], &v, BYTES);
                } else {
                    const T* at = o.out + (int64_t)m * o.ld + o.n0 + n;
                    T v[4 * STEP];
#pragma unroll
                    for (int i = 0; i < 4 * STEP; ++i) v[i] = (T)0.0f;
                    if (m < o.rows && left >= 4 * STEP) {
                        __builtin_memcpy(v, at, BYTES);
                    } else if (m < o.rows) {
#pragma unroll
                        for (int i = 0; i < 4 * STEP; ++i)
                            if (i < left) v[i] = at[i];
                    }
                    __builtin_memcpy(raw[b][a], v, BYTES);
                }
            }
        }
    }
    __device__ __forceinline__ float value(int b, int a, int i) const {
        T v[4 * STEP];
        __builtin_memcpy(v, raw[b][a / STEP], BYTES);
        return (float)v[a % STEP * 4 + i];
    }
};

// The biases of a lane's columns, which the sums begin with, packed as they
// are in memory.
template <class T, class Tile>
struct Biases {
    static constexpr int WORDS = (int)sizeof(T);   // of four values
    uint32_t raw[Tile::NT][WORDS];
    // bias: of the group's first plane, or null
    __device__ __forceinline__ void load(const T* __restrict__ bias, int F, int n0, int tid) {
#pragma unroll
        for (int a = 0; a < Tile::NT; ++a) {
            const int n = n0 + Tile::n_of(tid, a);
            const T* plane = bias + (a / Tile::PN) * (int64_t)F;
#pragma unroll
            for (int w = 0; w < WORDS; ++w) raw[a][w] = 0;
            if (!bias) continue;
            if (F >= 4) {
                // the last four values shifted down, where there are fewer
                const int at = n < F - 4 ? n : F - 4;
                __builtin_memcpy(raw[a], plane + at, sizeof(raw[a]));
                const int by = n - at;
                if constexpr (WORDS == 2) {
                    const uint64_t v = (uint64_t)raw[a][1] << 32 | raw[a][0];
                    const uint64_t s = by < 4 ? v >> (16 * by) : 0;
                    raw[a][0] = (uint32_t)s;
                    raw[a][1] = (uint32_t)(s >> 32);
                } else if (by > 0) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) raw[a][w] = n + w < F ? __builtin_bit_cast(uint32_t, (float)plane[n + w]) : 0;
                }
            } else {
                T v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = n + i < F ? plane[n + i] : (T)0.0f;
                __builtin_memcpy(raw[a], v, sizeof(v));
            }
        }
    }
    __device__ __forceinline__ f32x4 operator()(int a) const {
        T v[4];
        __builtin_memcpy(v, raw[a], sizeof(v));
        return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
};
struct Nothing {};

// What [da du] is held in, as one array or two.
template <class T>
using Back = typename std::conditional<sizeof(T) == 2, __bf16, float>::type;

// GRAD: writes [da du] of the rows to `out` [R, 2 F] from grad_y [R, F] (and
// its low parts behind it); otherwise y to `out` [R, F].
template <class T, class Tile, bool VEC, bool GRAD>
__global__ __launch_bounds__(Tile::THREADS) void grouped_gated(const T* __restrict__ x, int64_t R, int C,
                                                               const int64_t* __restrict__ off, int64_t N,
                                                               const T* __restrict__ weight, const T* __restrict__ bias, int F,
                                                               int act, const T* __restrict__ grad_y, bool wide_g,
                                                               typename std::conditional<GRAD, Back<T>, T>::type* __restrict__ out,
                                                               bool wide, int64_t tiles, int n_tiles, uint32_t places) {
    typedef typename std::conditional<GRAD, Back<T>, T>::type Out;
    constexpr bool PAIRS = GRAD && sizeof(T) == 2;
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    // Of a thread's number, as it is found anew for every tile: what follows from
    // it would be formed once and kept in scratch memory, for registers are short.
    const auto thread = [] {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        return tid;
    };
    // the 16-byte stores of a wave's part of a tile
    constexpr int kStores = Tile::PAIRED ? Tile::MT * Tile::PN / 2 : Tile::MT * Tile::PN;
    constexpr bool LARGE = sizeof(T) == 2 && Tile::BN == 256;
    walk_row_tiles<T, Tile, VEC, LARGE ? (GRAD ? 4 : 1) * kStores : 0, LARGE>(
        lds, blockIdx.x, gridDim.x, x, R, C, off, N, tiles, n_tiles, places,
        [&](const RowTile& at, int n0) {
            const T* w = weight + (at.group * 2 * F + n0) * (int64_t)C;
            return typename Tile::Planes(typename Tile::PSource{w, C, F - n0, nullptr},
                                         typename Tile::PSource{w + (int64_t)F * C, C, F - n0, nullptr});
        },
        [&](const RowTile& at, int n0) {
            Biases<T, Tile> b;
            b.load(bias && at.group >= 0 ? bias + at.group * 2 * F : nullptr, F, n0, thread());
            return b;
        },
        [&](const RowTile& at, int n0) {
            typename std::conditional<GRAD, Upstream<T, Tile>, Nothing>::type g;
            if constexpr (GRAD) g.load({grad_y + at.first * (int64_t)F, F, at.rows, n0, F, wide_g}, thread());
            return g;
        },
        [&](Tile& t, const RowTile& at, int n0, const auto& g) {
            const int tid = thread();
            constexpr int WIDTHS = GRAD ? 2 : 1;
            const TileOut<Out> first = {out + at.first * (int64_t)F * WIDTHS, (int64_t)F * WIDTHS, at.rows, n0, F, wide};
            TileOut<Out> second = first, first_low = first, second_low = first;
            second.out += F;
            first_low.out += R * F * WIDTHS;
            second_low.out += R * F * WIDTHS + F;
            with_activation(act, [&](auto&& activation) {
#pragma unroll
                for (int b = 0; b < Tile::MT; ++b) {
#pragma unroll
                    for (int a = 0; a < Tile::PN; ++a) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const Act v = activation(t.acc[a][b][i]);
                            const float u = t.acc[a + Tile::PN][b][i];
                            if constexpr (GRAD) {
                                const float up = g.value(b, a, i);
                                t.acc[a][b][i] = up * u * v.slope;
                                t.acc[a + Tile::PN][b][i] = up * v.value;
                            } else {
                                t.acc[a][b][i] = v.value * u;
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);   // registers are short: block after block
                    }
                    store_rows<Out, Tile, Tile::PN>(first, b, tid, [&](int a) { return t.acc[a][b]; });
                    if constexpr (GRAD)
                        store_rows<Out, Tile, Tile::PN>(second, b, tid, [&](int a) { return t.acc[a + Tile::PN][b]; });
                    if constexpr (PAIRS) {
                        store_rows<Out, Tile, Tile::PN>(first_low, b, tid, [&](int a) { return low_of(t.acc[a][b]); });
                        store_rows<Out, Tile, Tile::PN>(second_low, b, tid, [&](int a) { return low_of(t.acc[a + Tile::PN][b]); });
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
        },
        wide);
}

// ---------------------------------------------------------------------------
// narrow layers: the whole backward pass in one kernel
// ---------------------------------------------------------------------------
// With C <= 64 and F <= 128 a workgroup holds both planes of its group's
// weight in LDS and the gradient of the weight in its accumulators, and takes
// a piece of the group's rows, 64 MT rows at a time. 16 MT of them at a time
// give a and u, and da and du from them, which are in a wave's accumulators
// just as the product with the weight takes its operand (row lane & 15, eight
// consecutive f of 16-bit types or four of float32). For the sum over rows,
// [da du] and x go to LDS and each wave takes an equal part of the weight's
// rows. x, grad_y and grad_x pass memory once: 2 C + F values a row where the
// general form, with [da du] in memory, moves 3 C + 7 F.
//
// SPLIT: two waves share 16 MT rows, each with half of the columns: of a and u
// first, of grad_x afterwards, for which they read each other's [da du] from
// LDS. A workgroup has eight waves that way, and a compute unit one workgroup:
// the registers (about 200 a lane) hold no second one in 16 bits, nor does the
// LDS in float32 of more than 64 hidden values. Otherwise a wave has all of its
// rows' [da du] (float32 of at most 64 hidden values, two workgroups).
//
// What bounds it: 2^20 rows of 64 to 64 in bfloat16 take 157 us (memory alone
// 80; LDS, vector and matrix instructions each a part, in turn more than at a
// time), in float16 223, 217632 of 64 to 128 in float32 225 (the float32
// products 139). In bfloat16 of 64 to 64, waves that do not share rows spill
// (306) or have 16 rows each (194); one part of the pairs in LDS after the
// other, for two workgroups on a compute unit, 191; 64 rows at a time 193;
// pieces for 512 workgroups instead of 256, 173.
template <class T, int FP_, int MT_, bool SPLIT_>
struct Narrow {
    static constexpr int FP = FP_, MT = MT_, CP = 64, BM = 64 * MT;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int SHARES = SPLIT ? 2 : 1, THREADS = 256 * SHARES;
    static constexpr bool HALF = sizeof(T) == 2;
    using B = Back<T>;                                // of [da du], in PARTS
    static constexpr int PARTS = HALF ? 2 : 1;
    static constexpr int E = 16 / (int)sizeof(T);     // values of 16 bytes
    static constexpr int XS = CP / (4 * E);           // 64-byte slices of x's row, and of
    static constexpr int PS = FP / (4 * E);           // a plane's
    static constexpr int CB = CP / 16;                // blocks of 16 columns
    // a wave's blocks and slices of a plane's columns, blocks of grad_x's, and
    // of the weight's rows
    static constexpr int PB = FP / 16 / SHARES, PW = PS / SHARES, GB = CB / SHARES, WB = 2 * FP / 64 / SHARES;
    using W = OperandTile<T, FP, true, THREADS, CP * (int)sizeof(T)>;
    using D = OperandTile<B, 2 * FP, false, THREADS>;
    using X = OperandTile<B, CP, false, THREADS>;
    // x and the weight are pairs of B themselves: x is held in LDS as such, the
    // weight's fragments are split as they are read
    static constexpr bool CROSS = HALF && !__is_same(T, B);
    static constexpr int kW = 2 * W::kBytes, kD = BM * 2 * FP * (int)sizeof(T), kX = BM * CP * (int)sizeof(T);
    static constexpr int kLdsBytes = kW + PARTS * kD + (CROSS ? 2 : 1) * kX;
    static_assert(kLdsBytes <= 160 * 1024 && (PARTS == 1 || SPLIT), "");

    // out[m] += the product of a fragment of the weight with the parts q[k][m]
    // of [da du] (low with low is left out).
    static __device__ __forceinline__ void rows_product(u32x4 p, const u32x4 (&q)[PARTS][MT], f32x4 (&out)[MT]) {
        u32x4 high = p;
        if constexpr (CROSS) {
            high = high_bf16<T>(p);
            const u32x4 low = low_bf16<T>(p);
#pragma unroll
            for (int m = 0; m < MT; ++m) out[m] = mma<B>(low, q[0][m], out[m]);
        }
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m) out[m] = mma<B>(high, q[k][m], out[m]);
    }

    // Blocks of a plane, and of grad_x's columns, are paired in 16 bits so
    // that a lane holds eight consecutive values.
    static __device__ __forceinline__ int first_of(int block) { return HALF ? (block >> 1) * 32 + 4 * (block & 1) : block * 16; }
    static constexpr int STRIDE = HALF ? 8 : 4;
    // A lane's first column of slice s of a row.
    static __device__ __forceinline__ int column(int s, int lane) { return s * 4 * E + (lane >> 4) * E; }

    // 16 bytes of line `line` of an image of W, D or X.
    template <class Image>
    static __device__ __forceinline__ char* chunk(char* lds, int line, int chunk, int line_bytes) {
        return lds + line * line_bytes + ((chunk ^ Image::swizzle(line)) << 4);
    }

    // The fragment of the weight's transpose: columns c = first + STRIDE a + i,
    // slice s of a plane's f.
    static __device__ __forceinline__ u32x4 transposed(const char* plane, int s, int first, int lane) {
        constexpr int line_bytes = CP * (int)sizeof(T);
        const int q = lane >> 4, r = lane & 15;
        if constexpr (HALF) {
            s16x4 half[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int f = s * 32 + 8 * q + 4 * h + (r >> 2), c = first + STRIDE * (r & 3);
                const int at = f * line_bytes + (((c >> 3) ^ W::swizzle(f)) << 4) + (c & 7) * 2;
                half[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMR_LDS s16x4*)(plane + at));
            }
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int c = first + STRIDE * (r >> 2) + (r & 3);
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int f = s * 16 + 4 * q + j;
                v[j] = *reinterpret_cast<const uint32_t*>(plane + f * line_bytes + (((c >> 2) ^ W::swizzle(f)) << 4) + (c & 3) * 4);
            }
            return v;
        }
    }
};

// Values n .. n + 3 of N; zero where there are none.
template <class T>
__device__ __forceinline__ f32x4 load4(const T* __restrict__ from, int n, int N) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n + 4 <= N) {
        T t[4];
        __builtin_memcpy(t, from + n, sizeof(t));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) v[i] = (float)from[n + i];
    }
    return v;
}

// 16 bytes of row `row` of a [R, width] array, from value `at` on; zero where
// there are none. VEC: rows are whole 16 bytes, aligned. Others are read past
// the row's end where the array goes on, and what is past it is masked: lanes
// that take different ways would wait for each in turn.
template <class T, bool VEC>
__device__ __forceinline__ u32x4 row_chunk(const T* __restrict__ rows, int64_t R, int64_t row, int at, int width, bool exists) {
    constexpr int E = 16 / (int)sizeof(T);
    const T* from = rows + row * width + at;
    const int left = exists ? width - at : 0;
    u32x4 raw = {0, 0, 0, 0};
    if (VEC) {
        if (left > 0) raw = *reinterpret_cast<const u32x4*>(from);
    } else if (left > 0) {
        if ((R - row) * width - at >= E) {
            __builtin_memcpy(&raw, from, 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // of dword j, the bytes that are the row's
                const int bytes = left * (int)sizeof(T) - 4 * j;
                raw[j] = bytes >= 4 ? raw[j] : bytes <= 0 ? 0u : raw[j] & 0xFFFFu;
            }
        } else {
            T v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = e < left ? from[e] : (T)0.0f;
            __builtin_memcpy(&raw, v, 16);
        }
    }
    return raw;
}

template <class T>
__device__ __forceinline__ float value_of(u32x4 raw, int i) {
    T v[16 / sizeof(T)];
    __builtin_memcpy(v, &raw, 16);
    return (float)v[i];
}

template <class T, class L, bool VEC>
__global__ __launch_bounds__(L::THREADS, 2) void gated_narrow_grads(
    const T* __restrict__ x, int64_t R, int C, const int64_t* __restrict__ off, int64_t N, const T* __restrict__ weight,
    const T* __restrict__ bias, int F, int act, const T* __restrict__ g, T* __restrict__ grad_x, bool wide_x, int per,
    T* __restrict__ grad_weight, T* __restrict__ grad_bias, float* __restrict__ slots, int64_t slot_count) {
    constexpr int MT = L::MT, E = L::E, PB = L::PB, CB = L::CB;
    __shared__ alignas(16) char lds[L::kLdsBytes];
    char *const lds_w = lds, *const lds_d = lds + L::kW, *const lds_x = lds_d + L::PARTS * L::kD;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
    // its 16 MT rows and its share of their columns
    const int first_row = wave % 4 * MT * 16, share = L::SPLIT ? wave / 4 : 0;
    const Piece piece = find_piece(off, N, R, per, (int)blockIdx.x);
    if (piece.group < 0 || piece.slot >= slot_count) return;
    const T* bias_n = bias ? bias + piece.group * 2 * F : nullptr;
    {   // (not for an empty group: without rows the call needs no weight)
        typename L::W::Held held[2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < L::W::kLoads; ++i) {
                const int c = i * L::THREADS + tid, line = c / L::W::kLine;
                held[p].chunk[i] = row_chunk<T, VEC>(weight, N * 2 * F, (piece.group * 2 + p) * F + line,
                                                     ((c % L::W::kLine) ^ L::W::swizzle(line)) * E, C, line < F && piece.rows > 0);
            }
#pragma unroll
        for (int p = 0; p < 2; ++p) L::W::put(lds_w + p * L::W::kBytes, held[p], tid);
    }
    f32x4 sum[L::WB][CB], ones[L::WB];
#pragma unroll
    for (int b = 0; b < L::WB; ++b) {
        ones[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CB; ++c) sum[b][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // This lane's parts of its rows, asked for an iteration ahead, as soon as
    // the last ones are used.
    u32x4 xs[MT][L::XS], gs[MT][L::PW];
    const auto load_x = [&](u32x4 (&to)[MT][L::XS], int from) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = from + first_row + m * 16 + r;
#pragma unroll
            for (int s = 0; s < L::XS; ++s)
                to[m][s] = row_chunk<T, VEC>(x, R, piece.first + row, L::column(s, lane), C, row < piece.rows);
        }
    };
    const auto load_g = [&](u32x4 (&to)[MT][L::PW], int from) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = from + first_row + m * 16 + r;
#pragma unroll
            for (int s = 0; s < L::PW; ++s)
                to[m][s] = row_chunk<T, VEC>(g, R, piece.first + row, L::column(share * L::PW + s, lane), F, row < piece.rows);
        }
    };
    load_x(xs, 0);
    load_g(gs, 0);
    for (int from = 0; from < piece.rows; from += L::BM) {
        const bool more = from + L::BM < piece.rows;
        // Found anew for every iteration in float32 of up to 64 hidden values,
        // whose addresses would else take the registers of its fragments (150
        // and 144 us; of 128 in bfloat16 it costs, 252 and 272).
        int lane = tid & 63;
        if constexpr (!L::HALF && !L::SPLIT) asm volatile("" : "+v"(lane));
        const int r = lane & 15, q = lane >> 4;
        step_barrier<63>();   // the weight is in LDS; the last rows have been summed
        f32x4 acc[2][PB][MT];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int a = 0; a < PB; ++a) {
                const f32x4 add = load4<T>(bias_n + p * F, L::first_of(share * PB + a) + L::STRIDE * q, bias ? F : 0);   // not held: registers are short
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[p][a][m] = add;
#pragma unroll
                for (int s = 0; s < L::XS; ++s) {
                    const u32x4 wf = L::W::fragment(lds_w + p * L::W::kBytes, s, L::first_of(share * PB + a), L::STRIDE, lane);
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[p][a][m] = mma<T>(wf, xs[m][s], acc[p][a][m]);
                }
            }
        if (L::CROSS || share == 0)   // of pairs, each of two waves a part
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < L::XS; ++s) {
                    u32x4 v = xs[m][s];
                    if constexpr (L::CROSS) v = share == 0 ? high_bf16<T>(v) : low_bf16<T>(v);
                    *reinterpret_cast<u32x4*>(L::template chunk<typename L::X>(
                        lds_x + (L::CROSS ? share * L::kX : 0), first_row + m * 16 + r, s * 4 + q, L::CP * (int)sizeof(T))) = v;
                }
        if (more) load_x(xs, from + L::BM);
        // where slice s of plane p of this lane's [da du] goes, and all of a row's are
        const auto place = [&](int k, int m, int p, int s) {
            return reinterpret_cast<u32x4*>(L::template chunk<typename L::D>(
                lds_d + k * L::kD, first_row + m * 16 + r, (p * L::PS + s) * 4 + q, 2 * L::FP * (int)sizeof(T)));
        };
        u32x4 back[MT][2][L::PW];   // used where these are all of a row's
        with_activation(act, [&](auto&& activation) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const bool exists = from + first_row + m * 16 + r < piece.rows;   // nothing comes of rows that do not
#pragma unroll
                for (int s = 0; s < L::PW; ++s) {
                    constexpr int B = L::HALF ? 2 : 1;   // blocks of a slice
                    f32x4 d[2][B];
#pragma unroll
                    for (int h = 0; h < B; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const Act v = activation(acc[0][s * B + h][m][i]);
                            const float up = value_of<T>(gs[m][s], 4 * h + i);
                            d[0][h][i] = exists ? up * acc[1][s * B + h][m][i] * v.slope : 0.0f;
                            d[1][h][i] = exists ? up * v.value : 0.0f;
                        }
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        back[m][p][s] = packed<typename L::B>(d[p][0], d[p][B - 1]);
                        *place(0, m, p, share * L::PW + s) = back[m][p][s];
                        if constexpr (L::PARTS > 1)
                            *place(1, m, p, share * L::PW + s) = packed<typename L::B>(low_of(d[p][0]), low_of(d[p][B - 1]));
                    }
                }
            }
        });
        if (more) load_g(gs, from + L::BM);
        // grad_x of this wave's rows, back_of(part, m, p, s) the operand
        const auto rows_gradient = [&](auto&& back_of) {
            if (!grad_x) return;
            f32x4 out[L::GB][MT];
#pragma unroll
            for (int c = 0; c < L::GB; ++c) {
#pragma unroll
                for (int m = 0; m < MT; ++m) out[c][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int s = 0; s < L::PS; ++s) {
                    u32x4 rows[L::PARTS][MT];
#pragma unroll
                    for (int k = 0; k < L::PARTS; ++k)
#pragma unroll
                        for (int m = 0; m < MT; ++m) rows[k][m] = back_of(k, m, p, s);
#pragma unroll
                    for (int c = 0; c < L::GB; ++c) {
                        const u32x4 wf = L::transposed(lds_w + p * L::W::kBytes, s, L::first_of(share * L::GB + c), lane);
                        L::rows_product(wf, rows, out[c]);
                    }
                }
            constexpr int STEP = L::HALF ? 2 : 1;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int line = from + first_row + m * 16;
                T* rows = grad_x + (piece.first + line) * (int64_t)C;
                const auto put = [&](int row, int n, u32x4 v) {
                    if (line + row >= piece.rows) return;
                    T* to = rows + row * (int64_t)C + n;
                    if (wide_x) {
                        if (n < C) *reinterpret_cast<u32x4*>(to) = v;
                    } else if (n + E <= C) {
                        __builtin_memcpy(to, &v, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (n + e < C) to[e] = (T)value_of<T>(v, e);
                    }
                };
#pragma unroll
                for (int c = 0; c < L::GB; c += 2 * STEP) {
                    const u32x4 c0 = packed<T>(out[c][m], out[c + STEP - 1][m]);
                    const int n0 = (share * L::GB + c) * 16 + q * E;
                    if constexpr (L::GB >= 2 * STEP) {
                        const u32x4 c1 = packed<T>(out[c + STEP][m], out[c + 2 * STEP - 1][m]);
                        store_row_pairs(c0, c1, lane, [&](bool odd, int second, u32x4 v) {
                            put((r & ~1) | (odd ? 1 : 0), second ? n0 + 4 * E : n0, v);
                        });
                    } else {
                        put(r, n0, c0);
                    }
                }
            }
        };
        if constexpr (!L::SPLIT) rows_gradient([&](int, int m, int p, int s) { return back[m][p][s]; });
        step_barrier<63>();   // [da du] and x of all waves are in LDS
        if constexpr (L::SPLIT) rows_gradient([&](int k, int m, int p, int s) { return *place(k, m, p, s); });
#pragma unroll
        for (int s = 0; s < L::BM / (4 * E); ++s) {
            u32x4 xf[CB], xl[CB];
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                xf[c] = L::X::fragment(lds_x, s, c * 16, 4, lane);
                if constexpr (L::CROSS) xl[c] = L::X::fragment(lds_x + L::kX, s, c * 16, 4, lane);
            }
#pragma unroll
            for (int b = 0; b < L::WB; ++b) {
#pragma unroll
                for (int k = 0; k < L::PARTS; ++k) {
                    const u32x4 df = L::D::fragment(lds_d + k * L::kD, s, (wave * L::WB + b) * 16, 4, lane);
                    if constexpr (L::HALF) {
                        constexpr uint32_t bits = one_bits<typename L::B>();
                        ones[b] = mma<typename L::B>(u32x4{bits, bits, bits, bits}, df, ones[b]);
                    } else {
                        ones[b] += __builtin_bit_cast(f32x4, df);
                    }
#pragma unroll
                    for (int c = 0; c < CB; ++c) sum[b][c] = mma<typename L::B>(xf[c], df, sum[b][c]);
                    if constexpr (L::CROSS)
                        if (k == 0)
#pragma unroll
                            for (int c = 0; c < CB; ++c) sum[b][c] = mma<typename L::B>(xl[c], df, sum[b][c]);
                }
            }
        }
    }
    // rows f of the weight's gradient, columns c = 16 block + 4 q + i
    float* slot = piece.slot < 0 ? nullptr : slots + piece.slot * grouped_piece_values(C, 2 * F);
#pragma unroll
    for (int b = 0; b < L::WB; ++b) {
        const int at = (wave * L::WB + b) * 16 + r, p = at / L::FP, f = at % L::FP;
        float total = ones[b][0];
        if constexpr (!L::HALF) {
            total = (ones[b][0] + ones[b][1]) + (ones[b][2] + ones[b][3]);
            total += __shfl_xor(total, 16, 64);
            total += __shfl_xor(total, 32, 64);
        }
        if (f >= F) continue;
        const int64_t row = p * (int64_t)F + f;
        if (grad_weight)
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                const int n = c * 16 + 4 * q;
                if (slot) store4<float>(slot + row * C, n, C, sum[b][c]);
                else store4<T>(grad_weight + (piece.group * 2 * F + row) * C, n, C, sum[b][c]);
            }
        if (grad_bias && q == 0) {
            if (slot) slot[2 * (int64_t)F * C + row] = total;
            else grad_bias[piece.group * 2 * F + row] = (T)total;
        }
    }
}

template <class T, class L>
hipError_t launch_narrow(const GatedArgs& a, const GroupedPieces& p) {
    constexpr int each = 16 / (int)sizeof(T);
    const bool whole = a.C % each == 0, vec = whole && a.F % each == 0 && aligned16(a.x) && aligned16(a.grad_y) && aligned16(a.weight);
    const auto kernel = vec ? gated_narrow_grads<T, L, true> : gated_narrow_grads<T, L, false>;
    kernel<<<(unsigned)(a.R / p.rows + a.N), L::THREADS, 0, a.stream>>>(
        static_cast<const T*>(a.x), a.R, a.C, a.off, a.N, static_cast<const T*>(a.weight), static_cast<const T*>(a.bias), a.F,
        a.act, static_cast<const T*>(a.grad_y), static_cast<T*>(a.grad_x), whole && aligned16(a.grad_x), p.rows,
        static_cast<T*>(a.grad_weight), static_cast<T*>(a.grad_bias), reinterpret_cast<float*>(a.workspace), p.slots);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// few rows for each of many groups: the gradient of the weights
// ---------------------------------------------------------------------------
// The weights of every group are written once, and that is all there is to do:
// a thread takes 16 bytes of columns of eight of the weight's rows and adds
// its group's rows one after another. (Matrix instructions would multiply 64
// rows, of which nearly all are not there.)
constexpr int kShortRows = 8;   // of the weight, a thread's

// The rows of a group that are added that way at most. Few rows on average may
// still be nearly all of one group's: longer groups are left to the linear
// layer's tiles (131072 rows of one group among 32768, 72 to 32 in bfloat16: 4.6 ms
// so, 71 by a thread's loop; 64 groups of four rows, 512 to 512: 45.6 and 42.7 us).
constexpr int kShortMost = 64;

template <class T, bool VEC>
__global__ __launch_bounds__(256) void gated_short_weight_grads(const T* __restrict__ x, int64_t R, int C,
                                                                const int64_t* __restrict__ off, int64_t N,
                                                                const Back<T>* __restrict__ back, int width, bool wide,
                                                                unsigned blocks,
                                                                T* __restrict__ grad_weight, T* __restrict__ grad_bias) {
    constexpr int E = 16 / (int)sizeof(T), PARTS = kShortRows / E;   // 16 bytes of [da du]: eight or four values
    const int64_t n = blockIdx.x / blocks;
    int64_t lo, hi;
    group_bounds(off, N, R, n, lo, hi);
    if (hi - lo > kShortMost) return;
    const unsigned chunks = (unsigned)((C + E - 1) / E);
    const unsigned item = (blockIdx.x % blocks) * 256 + threadIdx.x;
    const int c = (int)(item % chunks) * E;
    const int64_t f = (int64_t)(item / chunks) * kShortRows;
    if (f >= width) return;
    float sum[kShortRows][E], total[kShortRows];
#pragma unroll
    for (int k = 0; k < kShortRows; ++k) {
        total[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) sum[k][e] = 0.0f;
    }
    for (int64_t r = lo; r < hi; ++r) {
        const u32x4 xr = row_chunk<T, VEC>(x, R, r, c, C, true);
        constexpr bool PAIRS = sizeof(T) == 2;
        u32x4 d[PARTS], low[PARTS];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            d[p] = row_chunk<Back<T>, VEC>(back, R, r, (int)f + p * E, width, true);
            if constexpr (PAIRS) low[p] = row_chunk<Back<T>, VEC>(back + R * width, R, r, (int)f + p * E, width, true);
        }
#pragma unroll
        for (int k = 0; k < kShortRows; ++k) {
            float v = value_of<Back<T>>(d[k / E], k % E);
            if constexpr (PAIRS) v += value_of<Back<T>>(low[k / E], k % E);
            total[k] += v;
#pragma unroll
            for (int e = 0; e < E; ++e) sum[k][e] = __builtin_fmaf(v, value_of<T>(xr, e), sum[k][e]);
        }
    }
#pragma unroll
    for (int k = 0; k < kShortRows; ++k) {
        if (f + k >= width) break;
        if (grad_weight) {
            alignas(16) T out[E];
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = (T)sum[k][e];
            T* to = grad_weight + (n * width + f + k) * C + c;
            if (wide) {
                *reinterpret_cast<u32x4*>(to) = *reinterpret_cast<const u32x4*>(out);
            } else if (c + E <= C) {
                __builtin_memcpy(to, out, 16);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c + e < C) to[e] = out[e];
            }
        }
        if (grad_bias && c == 0) grad_bias[n * width + f + k] = (T)total[k];
    }
}

// Workgroups of a group.
int64_t short_blocks(int32_t C, int32_t F, int each) {
    const int64_t items = (int64_t)ceil_div(C, each) * ceil_div(2 * F, kShortRows);
    return (items + 255) / 256;
}

template <class T>
hipError_t launch_short(const GatedArgs& a) {
    constexpr int each = 16 / (int)sizeof(T);
    const int64_t blocks = short_blocks(a.C, a.F, each);
    const bool whole = a.C % each == 0, vec = whole && 2 * a.F % each == 0 && aligned16(a.x);
    const auto kernel = vec ? gated_short_weight_grads<T, true> : gated_short_weight_grads<T, false>;
    kernel<<<(unsigned)(blocks * a.N), 256, 0, a.stream>>>(static_cast<const T*>(a.x), a.R, a.C, a.off, a.N,
                                                           reinterpret_cast<const Back<T>*>(a.workspace), 2 * a.F,
                                                           whole && aligned16(a.grad_weight), (unsigned)blocks,
                                                           static_cast<T*>(a.grad_weight), static_cast<T*>(a.grad_bias));
    return hipGetLastError();
}

template <class T, class Tile, bool GRAD, class Out>
hipError_t launch_tile(const GatedArgs& a, Out* out, bool vec, bool wide_g, bool wide) {
    const int n_tiles = ceil_div(a.F, Tile::COLUMNS);
    // of rows, whole bands of four
    const int64_t tiles = (most_row_tiles(a.R, a.N, Tile::BM) + 3) / 4 * 4 * n_tiles;
    const unsigned places = run_grid<kRun>(tiles);
    if (places == 0) return hipErrorInvalidValue;
    // as many workgroups as the device holds at a time (a multiple of 8 kRun)
    constexpr unsigned kHeld = 256 * (160 * 1024 / Tile::kLdsBytes);
    const unsigned grid = places > kHeld ? kHeld : places;
    const T *x = static_cast<const T*>(a.x), *w = static_cast<const T*>(a.weight), *bias = static_cast<const T*>(a.bias);
    const T* g = static_cast<const T*>(a.grad_y);
    if (vec)
        grouped_gated<T, Tile, true, GRAD><<<grid, Tile::THREADS, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, w, bias, a.F, a.act, g,
                                                                                 wide_g, out, wide, tiles, n_tiles, places);
    else if constexpr (Tile::BN < 256)   // the largest tiles have no form for unaligned arrays
        grouped_gated<T, Tile, false, GRAD><<<grid, Tile::THREADS, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, w, bias, a.F, a.act, g,
                                                                                  wide_g, out, wide, tiles, n_tiles, places);
    return hipGetLastError();
}

template <class T, int BN, int BM, int WN, int WM, int S>
using GatedTile = TileProduct<T, BN, BM, WN, WM, true, true, S, false, 2>;

template <class T, bool GRAD, class Out>
hipError_t launch_products(const GatedArgs& a, Out* out) {
    constexpr int each = 16 / (int)sizeof(T);
    const bool vec = a.C % each == 0 && aligned16(a.x) && aligned16(a.weight);
    const bool whole = a.F % each == 0, wide = whole && aligned16(out), wide_g = whole && aligned16(a.grad_y);
    const RowsTile t = gated_tile(a.R, a.N, a.F, sizeof(T) == 2, vec);
    if (t.rows == 16) return launch_tile<T, GatedTile<T, 128, 16, 4, 1, 4>, GRAD>(a, out, vec, wide_g, wide);
    if (t.columns == 16) return launch_tile<T, GatedTile<T, 32, 128, 1, 4, 2>, GRAD>(a, out, vec, wide_g, wide);
    if constexpr (sizeof(T) == 2)
        if (t.columns == 128) return launch_tile<T, GatedTile<T, 256, 256, 2, 4, 2>, GRAD>(a, out, vec, wide_g, wide);
    if (t.columns == 32) return launch_tile<T, GatedTile<T, 64, 128, 1, 4, 2>, GRAD>(a, out, vec, wide_g, wide);
    return launch_tile<T, GatedTile<T, 128, 128, 2, 4, 2>, GRAD>(a, out, vec, wide_g, wide);
}

// ---------------------------------------------------------------------------
// float16 operands of the products with [da du]
// ---------------------------------------------------------------------------
// Splits n values into pairs of bfloat16, exactly: the high parts and, behind
// them, the low ones. (Splitting fragments as they are read takes more time of
// the vector units than the products take, but where there are few rows, it
// saves the weights' way to memory and back.)
__global__ __launch_bounds__(256) void gated_split(const _Float16* __restrict__ in, int64_t n, __bf16* __restrict__ out) {
    const int64_t step = (int64_t)gridDim.x * 256 * 8;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += step) {
        if (i + 8 <= n) {
            u32x4 raw;
            __builtin_memcpy(&raw, in + i, 16);
            const u32x4 high = high_bf16<_Float16>(raw), low = low_bf16<_Float16>(raw);
            __builtin_memcpy(out + i, &high, 16);
            __builtin_memcpy(out + n + i, &low, 16);
        } else {
            for (int64_t k = i; k < n; ++k) {
                out[k] = (__bf16)(float)in[k];
                out[n + k] = (__bf16)low_of((float)in[k]);
            }
        }
    }
}

const __bf16* launch_split(const void* in, int64_t n, char* to, bool needed, hipStream_t stream) {
    __bf16* out = reinterpret_cast<__bf16*>(to);
    const int64_t blocks = (n + 2047) / 2048;
    if (needed && n > 0)
        gated_split<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(static_cast<const _Float16*>(in), n, out);
    return out;
}

// Whether x and the weight are split in the workspace: where the products take
// more than the smallest tiles.
bool gated_splits(int64_t R, int64_t N, int32_t C, int32_t F, dmr_dtype dtype) {
    return dtype == DMR_FLOAT16 && (R > 16 * N || (double)N * ceil_div(C, 64) * ceil_div(2 * F, 64) > (double)(1 << 22));
}

template <class T>
hipError_t launch_typed(const GatedArgs& a, bool backward) {
    if (!backward) return launch_products<T, false>(a, static_cast<T*>(a.y));
    GroupedLinearArgs b{};
    b.x = a.x; b.R = a.R; b.cin = a.C; b.off = a.off; b.N = a.N; b.weight = a.weight; b.cout = 2 * a.F; b.dtype = a.dtype;
    b.grad_x = a.grad_x; b.grad_weight = a.grad_weight; b.grad_bias = a.grad_bias; b.stream = a.stream;
    if (gated_narrow(a.C, a.F)) {
        const GroupedPieces p = gated_pieces(a.R, a.N, a.C, a.F, sizeof(T) == 2);
        const hipError_t err = a.F <= 64 ? launch_narrow<T, Narrow<T, 64, sizeof(T) == 2 ? 2 : 1, sizeof(T) == 2>>(a, p)
                                         : launch_narrow<T, Narrow<T, 128, 1, true>>(a, p);
        if (err != hipSuccess || p.slots == 0 || !(a.grad_weight || a.grad_bias)) return err;
        b.workspace = reinterpret_cast<float*>(a.workspace);
        return launch_grouped_add_pieces(b, p);
    }
    if (a.R > 0) {
        const hipError_t err = launch_products<T, true>(a, reinterpret_cast<Back<T>*>(a.workspace));
        if (err != hipSuccess) return err;
    }
    if ((a.grad_weight || a.grad_bias) && gated_short(a.R, a.N, a.C, a.F, sizeof(T) == 2)) {
        const hipError_t err = launch_short<T>(a);
        if (err != hipSuccess) return err;
        b.long_only = kShortMost;
        if (a.R <= kShortMost) b.grad_weight = b.grad_bias = nullptr;   // no group is longer
        if (a.R == 0 || !(b.grad_x || b.grad_weight || b.grad_bias)) return hipSuccess;
    }
    // [da du] as the upstream gradient of a linear layer of 2 F outputs
    b.grad_y = a.workspace;
    char* rest = a.workspace + gated_rows_bytes(a.R, a.F);
    if constexpr (sizeof(T) == 4) {
        b.workspace = reinterpret_cast<float*>(rest);
        return launch_grouped_linear_backward(b);
    }
    b.grad_y_low = reinterpret_cast<const __bf16*>(a.workspace) + a.R * 2 * a.F;
    if (gated_splits(a.R, a.N, a.C, a.F, a.dtype)) {
        const int64_t rows = a.R * a.C, weights = a.N * 2 * a.F * a.C;
        const __bf16* x = launch_split(a.x, rows, rest, b.grad_weight || b.grad_bias, a.stream);
        rest += gated_pair_bytes(rows);
        const __bf16* w = launch_split(a.weight, weights, rest, b.grad_x && a.R > 0, a.stream);
        rest += gated_pair_bytes(weights);
        b.x = x;
        b.x_low = x + rows;
        b.weight = w;
        b.weight_low = w + weights;
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    b.workspace = reinterpret_cast<float*>(rest);
    return launch_grouped_linear_backward_pairs(b);
}

}  // namespace

// The tile by the columns of each plane and by how many there are, as for
// linear layers: the larger, the fewer bytes for a product, but they have to
// fill 256 compute units, and rather half of them with tiles of 16 rows than
// fewer with 128. (3204 rows of 664 to 21 in float32: 30 us with 32 x 128, 12.4
// with 64 x 16; 300 of 1024 to 1000 42 and 26; but 10000 of 512 to 48 in
// bfloat16, 158 tiles, 8.1 and 10.4.)
RowsTile gated_tile(int64_t R, int64_t N, int32_t F, bool half, bool vec) {
    const auto tiles = [&](int columns, int rows) { return (R / rows + 1) * ceil_div(F, columns); };
    if (R <= 16 * N || tiles(32, 128) < 128) return {64, 16};
    if (F <= 16) return {16, 128};
    if (half && vec && F > 64 && R >= 512 * N && tiles(128, 256) >= 224) return {128, 256};
    if (F <= 32 || tiles(64, 128) < 256) return {32, 128};
    return {64, 128};
}

bool gated_narrow(int32_t C, int32_t F) { return C <= 64 && F <= 128; }

// Pieces for as many workgroups as the device holds at a time (two on a
// compute unit, or one), of at least 128 rows.
GroupedPieces gated_pieces(int64_t R, int64_t N, int32_t C, int32_t F, bool half) {
    if (!gated_narrow(C, F)) return grouped_pieces(R, N, C, 2 * F, half);
    const int64_t want = F <= 64 && !half ? 512 : 256;
    int64_t rows = (R + want - 1) / want;
    rows = (rows + 127) / 128 * 128;
    rows = rows < 128 ? 128 : rows > 8192 ? 8192 : rows;
    return {(int)rows, 64, R > rows ? 2 * (R / rows) : 0};
}

bool gated_fits(int64_t R, int64_t N, int32_t C, int32_t F, bool half) {
    if (!gated_narrow(C, F)) return grouped_sums_fit(R, N, C, 2 * F, half);
    const GroupedPieces p = gated_pieces(R, N, C, F, half);
    return R / p.rows + N <= kMaxWorkItems / 512 && (p.slots == 0 || grouped_add_fits(N, C, 2 * F));
}

// Whether the weights' gradient is added row by row: where groups have at most
// four rows on average and the weights are many. (bfloat16, the whole backward
// pass: 64 groups of one row, 1024 to 1024, 176 us so and 295 otherwise; 256
// rows in 64 groups, 512 to 512, 51 and 70; but 900 rows 90 and 79, and 200
// rows in 100 groups, 65 to 100, where one launch does both gradients, 28 and 17.)
bool gated_short(int64_t R, int64_t N, int32_t C, int32_t F, bool half) {
    return !gated_narrow(C, F) && R <= 4 * N && (double)N * F * C >= (double)(1 << 21) &&
           short_blocks(C, F, half ? 8 : 4) * N <= kMaxWorkItems / 256;
}

size_t gated_workspace(int64_t R, int64_t N, int32_t C, int32_t F, dmr_dtype dtype) {
    const GroupedPieces p = gated_pieces(R, N, C, F, dtype != DMR_FLOAT32);
    const size_t sums = align_up((size_t)(p.slots * grouped_piece_values(C, 2 * F)) * sizeof(float) + 256, 256);
    if (gated_narrow(C, F)) return sums;
    const size_t pairs = gated_splits(R, N, C, F, dtype) ? gated_pair_bytes(R * C) + gated_pair_bytes(N * 2 * F * C) : 0;
    return sums + gated_rows_bytes(R, F) + pairs;
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

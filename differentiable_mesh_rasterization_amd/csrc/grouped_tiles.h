// What the layers of packed batches share: the tiles of rows that any split
// into groups makes, found on the device, and the stores of their results.
#pragma once

#include "dmr_internal.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

// Consecutive tiles that a die is given at a time: what its 32 compute units
// work on together.
constexpr int kRun = 32;

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

template <class I>
__device__ __forceinline__ I wave_inclusive_sum(I v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const I u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// Workgroup b's place in the order of the tiles. Consecutive workgroups go to
// the 8 dies in turn; this gives each die runs of RUN consecutive tiles (what
// its 32 compute units work on at a time), which share rows and weights in
// its L2, and deals the runs out in turn, so that no die is left with the
// long groups or with the places past the last tile. The grid is a multiple
// of 8 RUN.
template <int RUN>
__device__ __forceinline__ int64_t tile_of_workgroup(uint32_t b) {
    const uint32_t die = b & 7, i = b >> 3;
    return (int64_t)((i / RUN * 8 + die) * RUN + i % RUN);
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Row tile t of all groups' tiles of `per` rows in order. Every wave does
// the same work. (Tile counts fit in 32 bits: a launch holds no more.)
__device__ __forceinline__ RowTile find_row_tile(const int64_t* __restrict__ off, int64_t N, int64_t R, int per, int t) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int64_t base = 0; base < N; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        const int tiles = (int)((hi - lo + per - 1) / per);
        const int upto = before + wave_inclusive_sum(tiles, lane);
        const uint64_t hit = __ballot(upto > t);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t first = lo + (int64_t)(t - (upto - tiles)) * per;
            const int64_t left = hi - first;
            RowTile r;
            r.group = base + src;
            r.first = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)first, src) |
                                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)((uint64_t)first >> 32), src) << 32);
            r.rows = __builtin_amdgcn_readlane((int)(left < per ? left : per), src);
            return r;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
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

// 16 bytes of a row: 8 16-bit or 4 float32 values.
template <class T>
__device__ __forceinline__ u32x4 packed(f32x4 lo, f32x4 hi) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(u32x4, lo);
    } else {
        alignas(16) T v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (T)lo[i];
            v[4 + i] = (T)hi[i];
        }
        return *reinterpret_cast<const u32x4*>(v);
    }
}

// Writes a workgroup's tile: rows [0, rows) of `out` (leading dimension ld),
// columns [n0, N), plus bias[n] if given. `wide`: `out` is 16-byte aligned and
// ld a multiple of 16 bytes.
template <class T, class Tile>
__device__ __forceinline__ void store_tile(const Tile& t, T* __restrict__ out, int64_t ld, int rows, int n0, int N,
                                           const T* __restrict__ bias, bool wide, int tid) {
    constexpr int STEP = Tile::PAIRED ? 2 : 1;              // blocks of n in a lane's 16 bytes
    constexpr bool CHUNKS = Tile::PAIRED || sizeof(T) == 4;   // a lane holds 16 bytes of a row
    f32x4 add[Tile::NT];
#pragma unroll
    for (int a = 0; a < Tile::NT; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = n0 + Tile::n_of(tid, a) + i;   // past the end: any value, not stored
            add[a][i] = bias ? (float)bias[at < N ? at : N - 1] : 0.0f;
        }
    if (CHUNKS && wide) {
        // 32-bit offsets from the tile's corner; stores past the buffer's
        // range are dropped
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(out + n0, 0, kBufferRange, 0x00020000);
        const uint32_t line = (uint32_t)(ld * sizeof(T));
        const int left = N - n0;
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
#pragma unroll
            for (int a = 0; a < Tile::NT; a += 2 * STEP) {
                const u32x4 c0 = packed<T>(t.acc[a][b] + add[a], t.acc[a + STEP - 1][b] + add[a + STEP - 1]);
                const int na = Tile::n_of(tid, a);
                if constexpr (Tile::NT % (2 * STEP) == 0) {
                    const u32x4 c1 = packed<T>(t.acc[a + STEP][b] + add[a + STEP],
                                               t.acc[a + 2 * STEP - 1][b] + add[a + 2 * STEP - 1]);
                    const int nb = Tile::n_of(tid, a + STEP);
                    store_row_pairs(c0, c1, tid, [&](bool odd, int chunk, u32x4 v) {
                        const int row = (m & ~1) | (odd ? 1 : 0), n = chunk ? nb : na;
                        const uint32_t off = (uint32_t)row * line + (uint32_t)n * (uint32_t)sizeof(T);
                        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, row < rows && n < left ? off : kNowhere, 0, 0);
                    });
                } else {
                    const uint32_t off = (uint32_t)m * line + (uint32_t)na * (uint32_t)sizeof(T);
                    __builtin_amdgcn_raw_buffer_store_b128(c0, rsrc, m < rows && na < left ? off : kNowhere, 0, 0);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int a = 0; a < Tile::NT; a += STEP) {
        const int n = n0 + Tile::n_of(tid, a);
#pragma unroll
        for (int b = 0; b < Tile::MT; ++b) {
            const int m = Tile::m_of(tid, b);
            if (m >= rows) continue;
            T* row = out + (int64_t)m * ld;
            if (CHUNKS && n + 4 * STEP <= N) {
                const u32x4 v = packed<T>(t.acc[a][b] + add[a], t.acc[a + STEP - 1][b] + add[a + STEP - 1]);
                __builtin_memcpy(row + n, &v, 16);   // at whatever alignment it has
            } else {
#pragma unroll
                for (int s = 0; s < STEP; ++s) store4<T>(row, n + 4 * s, N, t.acc[a + s][b] + add[a + s]);
            }
        }
    }
}

// Products of the rows of `rows_in` (k_in wide) with weights(tile, column) over
// a workgroup's tiles of rows, each handed to store(product, tile, column,
// held). Asked for ahead of the next tile's loads: held = load(tile, column),
// what a store needs from memory, and start(tile, column), what the next
// tile's sums begin with. YOUNGER: the stores that every wave issues in
// store() at least, if `stores`; the next tile's first steps do not wait for
// them. BANDS: the 32 tiles that a die works on together are four of rows by
// eight of columns, rather than one of rows and the whole of a wide weight,
// which its L2 does not hold. rows_low: the rows' low parts, of tiles of pairs.
template <class T, class Tile, bool VEC, int YOUNGER = 0, bool BANDS = false, class Weights, class Start, class Load, class Store>
__device__ __forceinline__ void walk_row_tiles(char* lds, uint32_t block, uint32_t blocks, const T* __restrict__ rows_in,
                                               int64_t R, int k_in, const int64_t* __restrict__ off, int64_t N,
                                               int64_t tiles, int n_tiles, uint32_t places, Weights&& weights,
                                               Start&& start, Load&& load, Store&& store, bool stores = false,
                                               const T* __restrict__ rows_low = nullptr) {
    const int tid = threadIdx.x;
    bool stored = false;
    // A place's tile of rows; its tile of columns goes to `c`.
    const auto find = [&](uint32_t place, int& c) {
        const int64_t id = tile_of_workgroup<kRun>(place);
        if (id >= tiles) return RowTile{-1, 0, 0};
        if constexpr (BANDS) {
            const int in_band = (int)(id % (4 * n_tiles)), chunk = in_band / 32, in_chunk = in_band % 32;
            const int wide = n_tiles - 8 * chunk < 8 ? n_tiles - 8 * chunk : 8;
            c = 8 * chunk + in_chunk % wide;
            return find_row_tile(off, N, R, Tile::BM, (int)(id / (4 * n_tiles)) * 4 + in_chunk / wide);
        } else {
            c = (int)(id % n_tiles);
            return find_row_tile(off, N, R, Tile::BM, (int)(id / n_tiles));
        }
    };
    // The first tile that exists from a place on, and its first column. (In the
    // order of rows none exists after one that does not.)
    const auto find_from = [&](uint32_t& place, int& n0) {
        int c = 0;
        RowTile r = find(place, c);
        if constexpr (BANDS)
            while (r.group < 0 && place + blocks < places) {
                place += blocks;
                r = find(place, c);
            }
        n0 = c * Tile::COLUMNS;
        return r;
    };
    const auto rows_of = [&](const RowTile& at) {
        return typename Tile::Source{rows_in + at.first * (int64_t)k_in, k_in, at.rows,
                                     rows_low ? rows_low + at.first * (int64_t)k_in : nullptr};
    };
    // A workgroup that takes several tiles finds the next one while a tile is
    // multiplied and issues its first loads before it stores.
    uint32_t place = block;
    int n0 = 0;
    RowTile at = find_from(place, n0);
    auto from = start(at, n0);
    if (at.group >= 0) Tile::template begin<VEC>(lds, weights(at, n0), rows_of(at), k_in, tid);
    while (at.group >= 0) {
        place += blocks;
        int next_n0 = 0;
        const RowTile next = place < places ? find_from(place, next_n0) : RowTile{-1, 0, 0};
        Tile t;
        t.template finish<VEC, YOUNGER>(lds, weights(at, n0), rows_of(at), k_in, tid, false, from, stored);
        stored = stores;
        const auto held = load(at, n0);
        from = start(next, next_n0);
        if (next.group >= 0) Tile::template begin<VEC>(lds, weights(next, next_n0), rows_of(next), k_in, tid);
        store(t, at, n0, held);
        at = next;
        n0 = next_n0;
    }
}

// ---------------------------------------------------------------------------
// sums over a group's rows
// ---------------------------------------------------------------------------
// Of the weight gradient's tiles, whose lengths differ, a die is given shorter
// runs at a time, so that the dies end together.
constexpr int kPieceRun = 8;

// A group of more than `per` rows is cut into equal pieces of at most that
// many. A group of one piece (or none) is written directly; the pieces of
// longer groups go to the workspace in float32, each to a slot of its own, and
// are added in order afterwards: no atomics, so the result does not depend on
// timing.

struct Piece {
    int64_t group, first;   // group < 0: no such piece
    int rows;
    int64_t slot;           // < 0: the group's only piece
};

// The pieces of a group of `rows` rows, and their length (the last may be
// shorter), a multiple of 64 rows.
__device__ __forceinline__ int pieces_of(int64_t rows, int per, int& length) {
    const int64_t n = rows > per ? (rows + per - 1) / per : 1;
    length = (int)((rows + n * 64 - 1) / (n * 64) * 64);
    return rows > per ? (int)((rows + length - 1) / length) : 1;
}

// Piece t of all groups'. Every wave does the same work. Up to 64 groups, the
// pieces are taken longest first, so that what the device finishes with is
// short: lane g compares its group's piece with every other's.
__device__ __forceinline__ Piece find_piece(const int64_t* __restrict__ off, int64_t N, int64_t R, int per, int t) {
    const int lane = threadIdx.x & 63;
    int before = 0, slots_before = 0;
    for (int64_t base = 0; base < N; base += 64) {
        int64_t lo, hi;
        group_bounds(off, N, R, base + lane, lo, hi);
        int length = 0;
        const int pieces = base + lane < N ? pieces_of(hi - lo, per, length) : 0;
        const int slots = pieces > 1 ? pieces : 0;
        const int slots_upto = slots_before + wave_inclusive_sum(slots, lane);
        int first_of;   // this group's first piece in the order
        if (N <= 64) {
            first_of = 0;
            for (int g = 0; g < (int)N; ++g) {
                const int l = __builtin_amdgcn_readlane(length, g), n = __builtin_amdgcn_readlane(pieces, g);
                if (l > length || (l == length && g < lane)) first_of += n;
            }
        } else {
            first_of = before + wave_inclusive_sum(pieces, lane) - pieces;
        }
        const uint64_t hit = __ballot(first_of <= t && t < first_of + pieces);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int k = t - first_of;
            const int64_t first = lo + (int64_t)k * length;
            const int64_t left = hi - first;
            Piece r;
            r.group = base + src;
            r.first = uniform64(__shfl(first, src, 64));
            r.rows = __builtin_amdgcn_readlane((int)(left < length ? left : length), src);
            r.slot = __builtin_amdgcn_readlane(pieces > 1 ? slots_upto - slots + k : -1, src);
            return r;
        }
        before = __builtin_amdgcn_readlane(first_of + pieces, 63);
        slots_before = __builtin_amdgcn_readlane(slots_upto, 63);
    }
    return {-1, 0, 0, -1};
}

// Group t of those of more than `shortest` rows, as one piece. Each of them has a
// multiple of shortest + 1 among its rows: t is the group of the t-th such row,
// if that is its first one. (A search for one row: it takes 15 steps where
// counting 32768 groups takes 512.)
__device__ __forceinline__ Piece find_long(const int64_t* __restrict__ off, int64_t N, int64_t R, int shortest, int64_t t) {
    const int64_t row = t * (shortest + 1);
    int64_t n = 0, past = N;   // the last group that does not begin after the row
    while (past - n > 1) {
        const int64_t mid = (n + past) >> 1;
        if (off[mid] <= row) n = mid;
        else past = mid;
    }
    int64_t lo, hi;
    group_bounds(off, N, R, n, lo, hi);
    if (hi - lo <= shortest || row < lo || row >= hi || row - (shortest + 1) >= lo) return {-1, 0, 0, -1};
    return {n, lo, (int)(hi - lo), -1};
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The most row tiles of `per` rows that R rows in N groups can make.
inline int64_t most_row_tiles(int64_t R, int64_t N, int per) { return R / per + (N < R ? N : R); }

// Workgroups for `tiles` tiles; 0 if a launch cannot hold them.
template <int RUN>
inline unsigned run_grid(int64_t tiles) {
    const int64_t grid = (tiles + 8 * RUN - 1) / (8 * RUN) * (8 * RUN);
    return grid > INT32_MAX ? 0u : (unsigned)grid;
}

}  // namespace
}  // namespace dmr

// Layer norms with one scale and shift per group of a packed batch, on gfx950:
// for every row r of group n, with m and v the mean and variance of its C
// values and s = (v + eps)^-1/2,
//     h_r = s (x_r - m),  y_r = gamma_n h_r + beta_n,
// and the backward pass, with q = gamma_n g_r,
//     grad_x_r = s (q - mean q - h_r mean(q h_r)),
//     grad_gamma_n = sum_r g_r h_r,  grad_beta_n = sum_r g_r.
//
// What bounds it is memory: a row is read once, kept in the registers of the L
// lanes that share it (16 bytes a lane at a time, V times), and written once.
// The backward pass forms m and s again from the row, which it reads anyway,
// so that nothing of the forward pass is kept. (2^20 rows of 64 in bfloat16
// forward: 45 us, 6.0 TB/s with half of the reads from the last cache level;
// backward 65536 of 1024 86 us, 4.7 TB/s, and 9 for its slots; 217632 of 64 in
// float32 29 us, 5.7 TB/s, and 5.)
//
// The mean is rounded and so is off by up to C 2^-24 of the values' size,
// which is much for rows far from zero; the deviations from the rounded mean
// are nearly exact, so their own mean, added up with their squares, corrects
// both mean and variance.
#include "dmr_internal.h"

namespace dmr {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Values in 16 bytes.
template <class T>
constexpr int kVector = 16 / (int)sizeof(T);

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Sums over the aligned blocks of L lanes, the same in every lane of a block.
template <int L, int COUNT>
__device__ __forceinline__ void lane_sums(float (&v)[COUNT]) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        if constexpr (L > 1) v[i] += dpp<0xB1>(v[i]);    // lane ^ 1
        if constexpr (L > 2) v[i] += dpp<0x4E>(v[i]);    // lane ^ 2
        if constexpr (L > 4) v[i] += dpp<0x141>(v[i]);   // the other four of eight, mirrored
        if constexpr (L > 8) v[i] += dpp<0x140>(v[i]);   // the other eight of 16, mirrored
        if constexpr (L > 16) v[i] += __shfl_xor(v[i], 16, 64);
        if constexpr (L > 32) v[i] += __shfl_xor(v[i], 32, 64);
    }
}

// 16 bytes of a row from value `at` on; values that the row does not have are
// zero. WHOLE: a row is a whole number of 16 bytes. Others in 16 bits are read
// past the row's end where the array goes on (`room` values from the row's
// first), and what is past it is masked: lanes that take different ways would
// wait for each in turn (400000 rows of 301 in bfloat16 158 us so, 143 masked;
// 200000 in float32, whose parts are half as long, 120 and 130).
template <class T, bool WHOLE>
__device__ __forceinline__ u32x4 load16(const T* __restrict__ row, int at, int C, int64_t room) {
    u32x4 raw = {0, 0, 0, 0};
    if (WHOLE) {
        if (at < C) __builtin_memcpy(&raw, row + at, 16);
    } else if (at < C) {
        if (sizeof(T) == 2 ? at + kVector<T> <= room : at + kVector<T> <= C) {
            __builtin_memcpy(&raw, row + at, 16);
            if constexpr (sizeof(T) == 2)
#pragma unroll
                for (int j = 0; j < 4; ++j) {   // of dword j, the values that are the row's
                    const int values = C - at - 2 * j;
                    raw[j] = values >= 2 ? raw[j] : values <= 0 ? 0u : raw[j] & 0xFFFFu;
                }
        } else {
            T v[kVector<T>];
#pragma unroll
            for (int e = 0; e < kVector<T>; ++e) v[e] = at + e < C ? row[at + e] : (T)0.0f;
            __builtin_memcpy(&raw, v, 16);
        }
    }
    return raw;
}

template <class T, bool WHOLE>
__device__ __forceinline__ void store16(T* __restrict__ row, int at, int C, const float (&v)[kVector<T>]) {
    T out[kVector<T>];
#pragma unroll
    for (int e = 0; e < kVector<T>; ++e) out[e] = (T)v[e];
    if (at + kVector<T> <= C) {
        __builtin_memcpy(row + at, out, 16);
    } else if (!WHOLE && at < C) {
#pragma unroll
        for (int e = 0; e < kVector<T>; ++e)
            if (at + e < C) row[at + e] = out[e];
    }
}

template <class T>
__device__ __forceinline__ void widen(u32x4 raw, float (&v)[kVector<T>]) {
    T t[kVector<T>];
    __builtin_memcpy(t, &raw, 16);
#pragma unroll
    for (int e = 0; e < kVector<T>; ++e) v[e] = (float)t[e];
}

// Offset i, held inside [0, R] whatever the array says.
__device__ __forceinline__ int64_t bound(const int64_t* __restrict__ off, int64_t i, int64_t R) {
    const int64_t v = off[i];
    return v < 0 ? 0 : v > R ? R : v;
}

// The number of offsets from `lo` on, of N + 1, that are at most r (`below`:
// less than r): r is a row of the last of their groups.
template <bool BELOW = false>
__device__ __forceinline__ int64_t offsets_upto(const int64_t* __restrict__ off, int64_t N, int64_t lo, int64_t r) {
    int64_t hi = N + 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (BELOW ? off[mid] < r : off[mid] <= r) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// (v + eps)^-1/2 from the deviations' squares and mean; NaN stays NaN.
__device__ __forceinline__ float scale_of(float squares, float shift, float each, float eps) {
    const float var = __builtin_fmaf(-shift, shift, squares * each);
    return 1.0f / sqrtf((var > 0.0f ? var : squares * 0.0f) + eps);
}

// A row in the registers of L lanes, and its statistics.
template <class T, int L, int V, bool WHOLE>
struct Row {
    static constexpr int E = kVector<T>;
    float x[V][E];   // h after normalise()
    float scale;

    static __device__ __forceinline__ int column(int part, int v) { return (part + v * L) * E; }

    __device__ __forceinline__ void load(const T* __restrict__ row, int part, int C, int64_t room) {
#pragma unroll
        for (int v = 0; v < V; ++v) widen<T>(load16<T, WHOLE>(row, column(part, v), C, room), x[v]);
    }

    __device__ __forceinline__ void normalise(int part, int C, float eps) {
        const float each = 1.0f / (float)C;
        float sum[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) sum[0] += x[v][e];
        lane_sums<L>(sum);
        const float mean = sum[0] * each;
        float more[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int at = column(part, v) + (WHOLE ? 0 : e);
                const float d = at < C ? x[v][e] - mean : 0.0f;
                x[v][e] = d;
                more[0] += d;
                more[1] = __builtin_fmaf(d, d, more[1]);
            }
        lane_sums<L>(more);
        const float shift = more[0] * each;
        scale = scale_of(more[1], shift, each, eps);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e) x[v][e] = (x[v][e] - shift) * scale;
    }
};

// y of `per` rows a workgroup.
template <class T, int L, int V, bool WHOLE>
__global__ __launch_bounds__(kThreads) void norm_rows(const T* __restrict__ x, int64_t R, int C,
                                                      const int64_t* __restrict__ off, int64_t N,
                                                      const T* __restrict__ gamma, const T* __restrict__ beta, float eps,
                                                      int64_t per, T* __restrict__ y) {
    constexpr int E = kVector<T>, SLOTS = kThreads / L;
    const int part = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int64_t end = begin + per < R ? begin + per : R;
    int64_t group = -1, until = 0;   // the group whose gamma and beta are held, and its end
    float ga[V][E], be[V][E];
    for (int64_t r = begin + slot; r < end; r += SLOTS) {
        if (r >= until || group < 0) {
            const int64_t n = offsets_upto(off, N, group < 0 ? 0 : group + 1, r) - 1;
            if (n < 0 || n >= N) continue;   // a row of no group
            group = n;
            until = off[n + 1];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = Row<T, L, V, WHOLE>::column(part, v);
                if (gamma) widen<T>(load16<T, WHOLE>(gamma + n * C, at, C, (N - n) * C), ga[v]);
                if (beta) widen<T>(load16<T, WHOLE>(beta + n * C, at, C, (N - n) * C), be[v]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!gamma) ga[v][e] = 1.0f;
                    if (!beta) be[v][e] = 0.0f;
                }
            }
        }
        Row<T, L, V, WHOLE> row;
        row.load(x + r * C, part, C, (R - r) * C);
        row.normalise(part, C, eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float out[E];
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = __builtin_fmaf(row.x[v][e], ga[v][e], be[v][e]);
            store16<T, WHOLE>(y + r * C, Row<T, L, V, WHOLE>::column(part, v), C, out);
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A workgroup takes `per` rows, group after group. The sums of a group that
// lies in its rows alone are written directly. Of the others a workgroup has
// at most two: the one that began before its rows (slot 2 w) and the one that
// goes on after them (slot 2 w + 1; slot 2 w if it does both). They are added
// in order afterwards: no atomics, so the result does not depend on timing. A
// slot holds C sums for gamma and C for beta.

__device__ __forceinline__ float* slot_of(float* slots, int C, bool early, bool late) {
    const int64_t w = blockIdx.x;
    return early ? slots + 4 * w * C : late ? slots + (4 * w + 2) * C : nullptr;
}

// Adds the sums that the lanes of a workgroup hold (each of its row's columns)
// over the rows it works on at a time, and hands value (column, sum) to put.
template <int L, int V, int E, class Put>
__device__ __forceinline__ void flush(float (&sums)[2][V][E], float* __restrict__ lds, int C, Put&& put) {
    const int tid = threadIdx.x, part = tid % L, wave = tid >> 6;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int d = L; d < 64; d <<= 1) sums[k][v][e] += __shfl_xor(sums[k][v][e], d, 64);
    constexpr int WIDTH = L * V * E;
    for (int w = 0; w < kThreads / 64; ++w) {
        if (wave == w && (tid & 63) < L) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float* at = lds + k * WIDTH + (part + v * L) * E + e;
                        *at = w == 0 ? sums[k][v][e] : *at + sums[k][v][e];
                    }
        }
        __syncthreads();
    }
    for (int i = tid; i < WIDTH; i += kThreads)
        if (i < C) {
            put(i, 0, lds[i]);
            put(i, 1, lds[WIDTH + i]);
        }
    __syncthreads();
}

template <class T, int L, int V, bool WHOLE>
__global__ __launch_bounds__(kThreads) void norm_grads(const T* __restrict__ x, int64_t R, int C,
                                                       const int64_t* __restrict__ off, int64_t N,
                                                       const T* __restrict__ gamma, float eps, const T* __restrict__ g,
                                                       int64_t per, T* __restrict__ grad_x, T* __restrict__ grad_gamma,
                                                       T* __restrict__ grad_beta, float* __restrict__ slots) {
    constexpr int E = kVector<T>, SLOTS = kThreads / L;
    __shared__ float lds[2 * L * V * E];
    const int part = threadIdx.x % L, slot = threadIdx.x / L;
    const float each = 1.0f / (float)C;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int64_t end = begin + per < R ? begin + per : R;
    const bool sum = grad_gamma || grad_beta;
    int64_t n = 0;
    for (int64_t from = begin; from < end;) {
        // the group of row `from`: the last that begins there or before
        n = offsets_upto(off, N, n, from) - 1;
        if (n < 0) {   // rows before the first group's
            n = 0;
            from = bound(off, 0, R);
            continue;
        }
        if (n >= N) break;
        const int64_t lo = bound(off, n, R), hi = bound(off, n + 1, R);
        const int64_t to = hi < end ? hi : end;
        if (to <= from) break;
        float ga[V][E], sums[2][V][E];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = Row<T, L, V, WHOLE>::column(part, v);
            if (gamma) widen<T>(load16<T, WHOLE>(gamma + n * C, at, C, (N - n) * C), ga[v]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (!gamma) ga[v][e] = 1.0f;
                sums[0][v][e] = sums[1][v][e] = 0.0f;
            }
        }
        for (int64_t r = from + slot; r < to; r += SLOTS) {
            Row<T, L, V, WHOLE> row;
            float q[V][E];
            row.load(x + r * C, part, C, (R - r) * C);
#pragma unroll
            for (int v = 0; v < V; ++v) 
                widen<T>(load16<T, WHOLE>(g + r * C, Row<T, L, V, WHOLE>::column(part, v), C, (R - r) * C), q[v]);
            row.normalise(part, C, eps);
            float means[2] = {0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sums[0][v][e] = __builtin_fmaf(q[v][e], row.x[v][e], sums[0][v][e]);
                    sums[1][v][e] += q[v][e];
                    q[v][e] *= ga[v][e];
                    means[0] += q[v][e];
                    means[1] = __builtin_fmaf(q[v][e], row.x[v][e], means[1]);
                }
            if (!grad_x) continue;
            lane_sums<L>(means);
            const float mq = means[0] * each, mh = means[1] * each;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float out[E];
#pragma unroll
                for (int e = 0; e < E; ++e) out[e] = row.scale * (q[v][e] - mq - row.x[v][e] * mh);
                store16<T, WHOLE>(grad_x + r * C, Row<T, L, V, WHOLE>::column(part, v), C, out);
            }
        }
        from = to;
        if (!sum) continue;
        float* to_slot = slot_of(slots, C, lo < begin, hi > end);
        flush<L, V, E>(sums, lds, C, [&](int i, int k, float v) {
            if (to_slot) to_slot[(int64_t)k * C + i] = v;
            else if (k == 0 && grad_gamma) grad_gamma[n * C + i] = (T)v;
            else if (k == 1 && grad_beta) grad_beta[n * C + i] = (T)v;
        });
    }
}

// Adds the slots of the groups that more than one workgroup has rows of (64 of
// a group's 2 C values a workgroup, each of its waves every WAVESth slot, eight
// loads in flight a lane), and writes the zeros of empty groups.
constexpr int kAddWaves = 16;
template <class T>
__global__ __launch_bounds__(kAddWaves * 64) void norm_add_slots(const int64_t* __restrict__ off, int64_t R, int C, int64_t per,
                                                                 const float* __restrict__ slots, unsigned blocks,
                                                                 T* __restrict__ grad_gamma, T* __restrict__ grad_beta) {
    __shared__ float part[kAddWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = blockIdx.x / blocks;
    const int64_t lo = bound(off, n, R), hi = bound(off, n + 1, R);
    const bool empty = lo >= hi;
    if (!empty && lo / per == (hi - 1) / per) return;
    const int64_t first = lo / per, count = empty ? 0 : (hi - 1) / per - first + 1;
    const int64_t i = (int64_t)(blockIdx.x % blocks) * 64 + lane;   // of 2 C
    float s = 0.0f;
    if (i < 2 * (int64_t)C) {
        // slot 2 first + 1, then 2 w
        const auto at = [&](int64_t k) { return slots + (k == 0 ? 4 * first + 2 : 4 * (first + k)) * C + i; };
        for (int64_t k = wave; k < count; k += 8 * kAddWaves) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = *at(k + kAddWaves * j < count ? k + kAddWaves * j : k);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + kAddWaves * j < count) s += v[j];
        }
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || i >= 2 * (int64_t)C) return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kAddWaves; ++w) s += part[w][lane];
    if (i < C) {
        if (grad_gamma) grad_gamma[n * C + i] = (T)s;
    } else if (grad_beta) {
        grad_beta[n * C + i - C] = (T)s;
    }
}

// ---------------------------------------------------------------------------
// rows that do not fit into a wave's registers
// ---------------------------------------------------------------------------
// A workgroup takes a row at a time and reads it again from the caches for
// every pass; the sums over rows are a kernel of their own, which takes the
// rows' statistics from the workspace.

constexpr int kLongThreads = 1024;

struct Stats {
    float mean, shift, scale, unused;   // h = (x - mean - shift) scale
};

__device__ __forceinline__ void workgroup_sums(float (&v)[2], float* lds) {
    lane_sums<64>(v);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        lds[2 * wave] = v[0];
        lds[2 * wave + 1] = v[1];
    }
    __syncthreads();
    v[0] = v[1] = 0.0f;
#pragma unroll
    for (int w = 0; w < kLongThreads / 64; ++w) {
        v[0] += lds[2 * w];
        v[1] += lds[2 * w + 1];
    }
    __syncthreads();
}

// Calls f(column, values) for the 16-byte parts of a row.
template <class T, class F>
__device__ __forceinline__ void over_row(const T* __restrict__ row, int C, int64_t room, F&& f) {
    for (int at = threadIdx.x * kVector<T>; at < C; at += kLongThreads * kVector<T>) {
        float v[kVector<T>];
        widen<T>(load16<T, false>(row, at, C, room), v);
        f(at, v);
    }
}

template <class T>
__device__ __forceinline__ Stats long_stats(const T* __restrict__ row, int C, int64_t room, float eps, float* lds) {
    const float each = 1.0f / (float)C;
    float sums[2] = {0.0f, 0.0f};
    over_row<T>(row, C, room, [&](int, const float* v) {
#pragma unroll
        for (int e = 0; e < kVector<T>; ++e) sums[0] += v[e];
    });
    workgroup_sums(sums, lds);
    const float mean = sums[0] * each;
    sums[0] = sums[1] = 0.0f;
    over_row<T>(row, C, room, [&](int at, const float* v) {
#pragma unroll
        for (int e = 0; e < kVector<T>; ++e) {
            const float d = at + e < C ? v[e] - mean : 0.0f;
            sums[0] += d;
            sums[1] = __builtin_fmaf(d, d, sums[1]);
        }
    });
    workgroup_sums(sums, lds);
    const float shift = sums[0] * each;
    return {mean, shift, scale_of(sums[1], shift, each, eps), 0.0f};
}

template <class T>
__global__ __launch_bounds__(kLongThreads) void norm_long_rows(const T* __restrict__ x, int64_t R, int C,
                                                               const int64_t* __restrict__ off, int64_t N,
                                                               const T* __restrict__ gamma, const T* __restrict__ beta,
                                                               float eps, T* __restrict__ y) {
    __shared__ float lds[2 * kLongThreads / 64];
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t n = offsets_upto(off, N, 0, r) - 1;
        if (n < 0 || n >= N) continue;
        const T* row = x + r * C;
        const int64_t room = (R - r) * C;
        const Stats s = long_stats<T>(row, C, room, eps, lds);
        over_row<T>(row, C, room, [&](int at, const float* v) {
            float ga[kVector<T>], be[kVector<T>], out[kVector<T>];
            if (gamma) widen<T>(load16<T, false>(gamma + n * C, at, C, (N - n) * C), ga);
            if (beta) widen<T>(load16<T, false>(beta + n * C, at, C, (N - n) * C), be);
#pragma unroll
            for (int e = 0; e < kVector<T>; ++e) {
                const float h = (v[e] - s.mean - s.shift) * s.scale;
                out[e] = __builtin_fmaf(h, gamma ? ga[e] : 1.0f, beta ? be[e] : 0.0f);
            }
            store16<T, false>(y + r * C, at, C, out);
        });
    }
}

template <class T>
__global__ __launch_bounds__(kLongThreads) void norm_long_grad_rows(const T* __restrict__ x, int64_t R, int C,
                                                                    const int64_t* __restrict__ off, int64_t N,
                                                                    const T* __restrict__ gamma, float eps,
                                                                    const T* __restrict__ g, T* __restrict__ grad_x,
                                                                    Stats* __restrict__ stats) {
    __shared__ float lds[2 * kLongThreads / 64];
    const float each = 1.0f / (float)C;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t n = offsets_upto(off, N, 0, r) - 1;
        if (n < 0 || n >= N) continue;
        const T* row = x + r * C;
        const int64_t room = (R - r) * C;
        const Stats s = long_stats<T>(row, C, room, eps, lds);
        if (stats && threadIdx.x == 0) stats[r] = s;
        if (!grad_x) continue;
        const auto q_of = [&](int at, float (&q)[kVector<T>]) {
            float ga[kVector<T>];
            widen<T>(load16<T, false>(g + r * C, at, C, (R - r) * C), q);
            if (!gamma) return;
            widen<T>(load16<T, false>(gamma + n * C, at, C, (N - n) * C), ga);
#pragma unroll
            for (int e = 0; e < kVector<T>; ++e) q[e] *= ga[e];
        };
        float means[2] = {0.0f, 0.0f};
        over_row<T>(row, C, room, [&](int at, const float* v) {
            float q[kVector<T>];
            q_of(at, q);
#pragma unroll
            for (int e = 0; e < kVector<T>; ++e)
                if (at + e < C) {
                    means[0] += q[e];
                    means[1] = __builtin_fmaf(q[e], (v[e] - s.mean - s.shift) * s.scale, means[1]);
                }
        });
        workgroup_sums(means, lds);
        const float mq = means[0] * each, mh = means[1] * each;
        over_row<T>(row, C, room, [&](int at, const float* v) {
            float q[kVector<T>], out[kVector<T>];
            q_of(at, q);
#pragma unroll
            for (int e = 0; e < kVector<T>; ++e) out[e] = s.scale * (q[e] - mq - (v[e] - s.mean - s.shift) * s.scale * mh);
            store16<T, false>(grad_x + r * C, at, C, out);
        });
    }
}

// Sums of `per` rows, 16 bytes of the columns a thread.
template <class T>
__global__ __launch_bounds__(kThreads) void norm_long_sums(const T* __restrict__ x, int64_t R, int C,
                                                           const int64_t* __restrict__ off, int64_t N,
                                                           const T* __restrict__ g, const Stats* __restrict__ stats,
                                                           int64_t per, T* __restrict__ grad_gamma,
                                                           T* __restrict__ grad_beta, float* __restrict__ slots) {
    constexpr int E = kVector<T>;
    const int at = ((int)blockIdx.y * kThreads + (int)threadIdx.x) * E;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int64_t end = begin + per < R ? begin + per : R;
    int64_t n = 0;
    for (int64_t from = begin; from < end;) {
        n = offsets_upto(off, N, n, from) - 1;
        if (n < 0) {   // rows before the first group's
            n = 0;
            from = bound(off, 0, R);
            continue;
        }
        if (n >= N) break;
        const int64_t lo = bound(off, n, R), hi = bound(off, n + 1, R);
        const int64_t to = hi < end ? hi : end;
        if (to <= from) break;
        float sums[2][E];
#pragma unroll
        for (int e = 0; e < E; ++e) sums[0][e] = sums[1][e] = 0.0f;
        for (int64_t r = from; r < to; ++r) {
            const Stats s = stats[r];
            float v[E], q[E];
            widen<T>(load16<T, false>(x + r * C, at, C, (R - r) * C), v);
            widen<T>(load16<T, false>(g + r * C, at, C, (R - r) * C), q);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sums[0][e] = __builtin_fmaf(q[e], (v[e] - s.mean - s.shift) * s.scale, sums[0][e]);
                sums[1][e] += q[e];
            }
        }
        from = to;
        float* to_slot = slot_of(slots, C, lo < begin, hi > end);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (at + e >= C) break;
            if (to_slot) {
                to_slot[at + e] = sums[0][e];
                to_slot[(int64_t)C + at + e] = sums[1][e];
            } else {
                if (grad_gamma) grad_gamma[n * C + at + e] = (T)sums[0][e];
                if (grad_beta) grad_beta[n * C + at + e] = (T)sums[1][e];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Calls f with the kernels' lanes and 16-byte parts of a row as types.
template <int V>
struct Int {
    static constexpr int value = V;
};
template <class F>
void with_row(int lanes, int parts, F&& f) {
    if (parts == 2) f(Int<64>{}, Int<2>{});
    else if (parts == 4) f(Int<64>{}, Int<4>{});
    else if (parts == 8) f(Int<64>{}, Int<8>{});
    else if (lanes == 1) f(Int<1>{}, Int<1>{});
    else if (lanes == 2) f(Int<2>{}, Int<1>{});
    else if (lanes == 4) f(Int<4>{}, Int<1>{});
    else if (lanes == 8) f(Int<8>{}, Int<1>{});
    else if (lanes == 16) f(Int<16>{}, Int<1>{});
    else if (lanes == 32) f(Int<32>{}, Int<1>{});
    else f(Int<64>{}, Int<1>{});
}

template <class T>
hipError_t launch_forward(const LayerNormArgs& a) {
    const T *x = static_cast<const T*>(a.x), *gamma = static_cast<const T*>(a.weight), *beta = static_cast<const T*>(a.bias);
    T* y = static_cast<T*>(a.y);
    const LayerNormPlan p = layer_norm_plan(a.R, a.N, a.C, sizeof(T) == 2, false);
    if (p.lanes == 0) {
        norm_long_rows<T><<<(unsigned)p.workgroups, kLongThreads, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, gamma, beta, a.eps, y);
        return hipGetLastError();
    }
    with_row(p.lanes, p.parts, [&](auto lanes, auto parts) {
        constexpr int L = decltype(lanes)::value, V = decltype(parts)::value;
        const auto kernel = a.C % kVector<T> == 0 ? norm_rows<T, L, V, true> : norm_rows<T, L, V, false>;
        kernel<<<(unsigned)p.workgroups, kThreads, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, gamma, beta, a.eps, p.per, y);
    });
    return hipGetLastError();
}

template <class T>
hipError_t launch_backward(const LayerNormArgs& a) {
    const T *x = static_cast<const T*>(a.x), *gamma = static_cast<const T*>(a.weight), *g = static_cast<const T*>(a.grad_y);
    T *gx = static_cast<T*>(a.grad_x), *gw = static_cast<T*>(a.grad_weight), *gb = static_cast<T*>(a.grad_bias);
    const LayerNormPlan p = layer_norm_plan(a.R, a.N, a.C, sizeof(T) == 2, true);
    const bool sums = gw || gb;
    float* slots = a.workspace;
    if (a.R > 0 && p.lanes == 0) {
        Stats* stats = sums ? reinterpret_cast<Stats*>(a.workspace + p.slot_values) : nullptr;
        const unsigned rows = (unsigned)(a.R < 4096 ? a.R : 4096);
        norm_long_grad_rows<T><<<rows, kLongThreads, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, gamma, a.eps, g, gx, stats);
        if (sums) {
            const unsigned strips = (unsigned)((a.C + kThreads * kVector<T> - 1) / (kThreads * kVector<T>));
            norm_long_sums<T><<<dim3((unsigned)p.workgroups, strips), kThreads, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, g, stats,
                                                                                              p.per, gw, gb, slots);
        }
    } else if (a.R > 0) {
        with_row(p.lanes, p.parts, [&](auto lanes, auto parts) {
            constexpr int L = decltype(lanes)::value, V = decltype(parts)::value;
            const auto kernel = a.C % kVector<T> == 0 ? norm_grads<T, L, V, true> : norm_grads<T, L, V, false>;
            kernel<<<(unsigned)p.workgroups, kThreads, 0, a.stream>>>(x, a.R, a.C, a.off, a.N, gamma, a.eps, g, p.per, gx, gw,
                                                                      gb, slots);
        });
    }
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && sums) {
        const unsigned blocks = (unsigned)((2 * (int64_t)a.C + 63) / 64);
        norm_add_slots<T><<<blocks * (unsigned)a.N, kAddWaves * 64, 0, a.stream>>>(a.off, a.R, a.C, p.per, slots, blocks, gw, gb);
        err = hipGetLastError();
    }
    return err;
}

}  // namespace

// How rows are shared out: the lanes of a row and the 16-byte parts each of
// them holds (0 lanes: a row takes a workgroup), and the rows of a workgroup.
// 2048 workgroups of the backward pass fill the device with the eight that a
// compute unit holds; more would only make more slots. But where groups are
// shorter than the rows that a workgroup works on at a time, it would take
// them one after another: then a workgroup for each of them, as far as slots
// allow (64 groups of one row of 64 in float16: 87 us before, 6.6 so).
LayerNormPlan layer_norm_plan(int64_t R, int64_t N, int32_t C, bool half, bool backward) {
    LayerNormPlan p{};
    const int each = half ? 8 : 4;
    const int64_t parts = ((int64_t)C + each - 1) / each;
    int64_t most = backward ? 2048 : 4096;
    if (parts <= 64) {
        p.parts = 1;
        for (p.lanes = 1; p.lanes < parts;) p.lanes *= 2;
    } else if (parts <= 512) {
        p.lanes = 64;
        p.parts = parts <= 128 ? 2 : parts <= 256 ? 4 : 8;
    } else {
        most = backward ? (most * kThreads + parts - 1) / parts : most;   // strips of columns make the rest
    }
    int64_t slots = p.lanes > 0 ? kThreads / p.lanes : 1;
    if (backward && p.lanes > 0 && N > 0 && R / N < slots) {
        slots = R / N > 1 ? R / N : 1;
        const int64_t room = ((int64_t)1 << 23) / C;
        if (room > most) most = room;
    }
    p.per = (R + most * slots - 1) / (most * slots) * slots;
    p.per = p.per < slots ? slots : p.per;
    p.workgroups = (R + p.per - 1) / p.per;
    p.slot_values = 4 * p.workgroups * C;
    p.workspace = (size_t)p.slot_values * sizeof(float) + (p.lanes == 0 ? (size_t)R * sizeof(Stats) : 0);
    return p;
}

hipError_t launch_layer_norm(const LayerNormArgs& a, bool backward) {
    const KernelId id = backward ? kKLayerNormBwd : kKLayerNormFwd;
    timing_begin(id, a.stream);
    hipError_t err = hipErrorInvalidValue;
    switch (a.dtype) {
        case DMR_FLOAT32: err = backward ? launch_backward<float>(a) : launch_forward<float>(a); break;
        case DMR_FLOAT16: err = backward ? launch_backward<_Float16>(a) : launch_forward<_Float16>(a); break;
        case DMR_BFLOAT16: err = backward ? launch_backward<__bf16>(a) : launch_forward<__bf16>(a); break;
    }
    timing_end(id, a.stream);
    return err;
}

}  // namespace dmr

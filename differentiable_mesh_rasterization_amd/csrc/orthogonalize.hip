// Orthogonalised updates on gfx950: for every matrix U [m, n] of a batch
//     X = U / (|U|_F + eps), then `steps` times
//     A = X X^T,  B = b A + c A A,  X <- a X + B X
// with X [s, l] (s = min(m, n); U is taken transposed when m > n).
//
// The products run on the matrix cores in float16 with float32 sums. All
// values are bounded (the largest singular value of X stays below 1.21), so
// powers of two keep float16 away from its limits (fixed ones, but that an
// update whose norm is far below eps is lifted: see lift_of). Two things keep
// the result exact to more than 11 bits:
//   the diagonals of A and B are kept apart in float32. They are the large
//   entries (A tends to a matrix near the identity, where a X + B X cancels:
//   a + b + c = 0.70 out of 3.44), and with A = D + O, D diagonal,
//       (A A)_ij = (O O)_ij + (d_i + d_j) O_ij,   i != j,
//       (A A)_ii = (O O)_ii + d_i^2,
//       X <- (a + B_ii) X_i + (off-diagonal B) X;
//   X, O and the off-diagonal B are pairs of float16, high + low (22 bits),
// and a product is high high + high low + low high, as exact as float32
// products at three times the cost of one: against the definition in 64 bits
// on matrices of 64 to 2048 that gives 0.6 times the error of float32 products.
// bfloat16 updates take the same products: with the high parts alone the error
// of a 256 x 256 update of 32 strong directions over weak ones is 1.6e-3 of its
// norm, as much as the rounding of the result; with pairs 7e-6.
#include "dmr_internal.h"
#include "mfma_tile.h"

namespace dmr {
namespace {

typedef _Float16 h16;
typedef h16 h16x4 __attribute__((ext_vector_type(4)));

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kLogScaleX = 14;
constexpr float kScaleX = 1 << kLogScaleX, kScaleO = 16384.0f, kScaleB = 8192.0f;

// What U is multiplied by to give X_0 times 2^up. In float64, and the product
// with U too: the norm of finite values may pass float32's range, and so may
// one over a small norm and eps. An infinity or NaN in U gives NaN throughout.
__device__ __forceinline__ double scale_of(double norm, float eps, int up) {
    return __builtin_isfinite(norm) ? __builtin_ldexp(1.0, up) / (norm + (double)eps) : __builtin_nan("");
}

// X_0 has the norm t = |U| / (|U| + eps), which is tiny when |U| is far below
// eps, and a step multiplies it by 3.4445 < 2^1.785 at most. So that float16
// pairs (or float32) do not lose it below their range, X is held times a power
// of two, the largest that keeps this bound below 1 (or 1): 2^lift_of for X_0,
// 2^lift_at after `step` steps, brought down as X grows. A is put back to its
// own scale.
__device__ __forceinline__ int lift_of(double norm, float eps) {
    const double t = norm / (norm + (double)eps);
    if (!(t > 0.0)) return 0;   // zeros, or NaN
    int e = 0;
    (void)__builtin_frexp(t, &e);   // t < 2^e
    return e < 0 ? -e : 0;
}
__device__ __forceinline__ int lift_at(int lift, int step) {
    const int e = lift - (step * 1828 + 1023) / 1024;
    return step > 0 ? (e > 0 ? e : 0) : lift;
}

// ---------------------------------------------------------------------------
// matrices that fit into one workgroup's LDS: one workgroup each, one launch
// ---------------------------------------------------------------------------
// Everything is float32, on the float32 matrix instructions: the whole
// iteration of such a matrix costs less than the launches of the tiled form.

// (1024 threads; 256 if no wave then has more than 4 tiles of X and one of A:
// the barriers of fewer waves are shorter, 12.3 us against 9.6 for 16
// matrices of 3 x 64.)
constexpr int kSmallThreads = 1024;
constexpr int kSmallLds = 150 * 1024;
constexpr int kSmallUpdateTiles = 10;   // 16 x 16 tiles of X a wave holds

struct SmallShape {
    int s, l, sp, lp, ldx, lda;
    size_t bytes;
};
__host__ __device__ __forceinline__ SmallShape small_shape(int m, int n) {
    SmallShape h;
    h.s = m < n ? m : n;
    h.l = m < n ? n : m;
    h.sp = (h.s + 15) / 16 * 16;
    h.lp = (h.l + 15) / 16 * 16;
    h.ldx = h.lp + 4;   // rows 16 bytes past a multiple of 64: fragment reads spread over the banks
    h.lda = h.sp + 4;
    h.bytes = ((size_t)h.sp * h.ldx + (size_t)h.sp * h.lda) * sizeof(float);
    return h;
}

bool is_small(int m, int n) {
    if ((int64_t)m * n > 40000) return false;
    const SmallShape h = small_shape(m, n);
    return h.sp <= 64 && h.bytes <= (size_t)kSmallLds &&
           (h.sp / 16) * (h.lp / 16) <= kSmallUpdateTiles * (kSmallThreads / 64);
}

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS) void orthogonalize_small(const T* __restrict__ update, int m, int n, int steps,
                                                                     float eps, T* __restrict__ out) {
    constexpr int WAVES = THREADS / 64, HELD = THREADS == kSmallThreads ? kSmallUpdateTiles : 4;
    extern __shared__ __align__(16) float lds[];
    __shared__ double part[WAVES];
    const SmallShape h = small_shape(m, n);
    float* x = lds;
    float* a = lds + h.sp * h.ldx;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, q = lane >> 4, r = lane & 15;
    const bool turned = m > n;
    const int64_t base = (int64_t)blockIdx.x * m * n;
    for (int i = tid; i < h.sp * h.ldx; i += THREADS) x[i] = 0.0f;
    __syncthreads();
    double sum = 0.0;
    for (int i = tid; i < m * n; i += THREADS) {
        const float v = (float)update[base + i];
        sum += (double)v * (double)v;
        x[turned ? (i % n) * h.ldx + i / n : (i / n) * h.ldx + i % n] = v;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w];
    sum = sqrt(sum);
    const int lift = __builtin_amdgcn_readfirstlane(lift_of(sum, eps));
    const double inv = scale_of(sum, eps, lift);
    for (int i = tid; i < h.sp * h.ldx; i += THREADS) x[i] = (float)((double)x[i] * inv);
    __syncthreads();

    const int st = h.sp / 16, lt = h.lp / 16, tri = st * (st + 1) / 2;
    // this wave's tile of the lower triangle of A and B
    int ti = 0;
    while ((ti + 1) * (ti + 2) / 2 <= wave) ++ti;
    const int tj = wave - ti * (ti + 1) / 2;
    const bool gram = wave < tri;
    for (int step = 0; step < steps; ++step) {
        const int held = lift_at(lift, step);
        const float back = __builtin_ldexpf(1.0f, -2 * held), down = __builtin_ldexpf(1.0f, lift_at(lift, step + 1) - held);
        f32x4 acc;
        for (int poly = 0; poly < 2; ++poly) {
            const float* from = poly ? a : x;
            const int ld = poly ? h.lda : h.ldx, K = poly ? h.sp : h.lp;
            if (gram) {
                acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                const float* pj = from + (tj * 16 + r) * ld + 4 * q;
                const float* pi = from + (ti * 16 + r) * ld + 4 * q;
                for (int k = 0; k < K; k += 16)
                    acc = mma<float>(*reinterpret_cast<const u32x4*>(pj + k), *reinterpret_cast<const u32x4*>(pi + k), acc);
                if (!poly) acc *= back;
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = kB * a[(ti * 16 + r) * h.lda + tj * 16 + 4 * q + i] + kC * acc[i];
            }
            __syncthreads();   // poly: all of A has been read
            if (gram) {
                // this lane: row ti 16 + r, columns tj 16 + 4 q + i, and the mirrored entries
                *reinterpret_cast<f32x4*>(a + (ti * 16 + r) * h.lda + tj * 16 + 4 * q) = acc;
                if (ti != tj)
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[(tj * 16 + 4 * q + i) * h.lda + ti * 16 + r] = acc[i];
            }
            __syncthreads();
        }
        f32x4 next[HELD];
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int tile = wave + u * WAVES;
            if (tile >= st * lt) continue;
            const int xi = tile % st, xj = tile / st;
            f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < h.sp; k += 16) {
                u32x4 p;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p[j] = __builtin_bit_cast(uint32_t, x[(k + 4 * q + j) * h.ldx + xj * 16 + r]);
                c = mma<float>(p, *reinterpret_cast<const u32x4*>(a + (xi * 16 + r) * h.lda + k + 4 * q), c);
            }
            const f32x4 old = *reinterpret_cast<const f32x4*>(x + (xi * 16 + r) * h.ldx + xj * 16 + 4 * q);
            next[u] = (kA * old + c) * down;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int tile = wave + u * WAVES;
            if (tile >= st * lt) continue;
            *reinterpret_cast<f32x4*>(x + ((tile % st) * 16 + r) * h.ldx + (tile / st) * 16 + 4 * q) = next[u];
        }
        __syncthreads();
    }
    for (int i = tid; i < m * n; i += THREADS)
        out[base + i] = (T)__builtin_ldexpf(x[turned ? (i % n) * h.ldx + i / n : (i / n) * h.ldx + i % n], -lift_at(lift, steps));
}

// ---------------------------------------------------------------------------
// the tiled form
// ---------------------------------------------------------------------------

// Sides are padded to multiples of kPad with zeros, which the iteration
// keeps. X is [sp, lp], the off-diagonal A and B are [sp, sp], held as the
// pairs that PairProduct reads (32 high parts, 32 low parts, ..).
constexpr int kPad = 64;
constexpr int kNormBlocks = 64;

struct Layout {
    int s, l, sp, lp;
    int64_t x[2], o, b, diag, bdiag, norm, lift;   // byte offsets, each for the whole batch
    size_t bytes;
};

Layout layout(int64_t B, int m, int n) {
    Layout w{};
    w.s = m < n ? m : n;
    w.l = m < n ? n : m;
    w.sp = (w.s + kPad - 1) / kPad * kPad;
    w.lp = (w.l + kPad - 1) / kPad * kPad;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const int64_t xs = B * w.sp * w.lp, as = B * w.sp * w.sp;
    for (int k = 0; k < 2; ++k) w.x[k] = take(xs * 4);
    w.o = take(as * 4);
    w.b = take(as * 4);
    w.diag = take(B * w.sp * 4);
    w.bdiag = take(B * w.sp * 4);
    w.norm = take(B * kNormBlocks * 8);
    w.lift = take(B * 4);
    w.bytes = (size_t)at;
    return w;
}

// Where a matrix of rows of `ld` values holds value n of row m: its high
// part, in float16 from the matrix's start, and kLow further its low part.
constexpr int kLow = 32;
__device__ __forceinline__ int64_t place(int64_t m, int ld, int n) { return m * 2 * ld + (n >> 5) * 64 + (n & 31); }

// v as a pair. v is pinned to its float32 value first: the compiler may
// otherwise round the product or sum that gives it straight to float16 for the
// high part, and take the low part from the float32 one, which a tie apart are
// not the same number.
__device__ __forceinline__ void split(float v, h16& hi, h16& lo) {
    asm("" : "+v"(v));
    hi = (h16)v;
    lo = (h16)(v - (float)hi);
}

// Sum of squares of a slice of each matrix (float64: no overflow, and the
// scale is exact).
template <class T>
__global__ __launch_bounds__(256) void orthogonalize_norm(const T* __restrict__ update, int64_t size, bool wide,
                                                          double* __restrict__ norm) {
    __shared__ double part[4];
    constexpr int E = 16 / (int)sizeof(T);
    const T* u = update + (int64_t)(blockIdx.x / kNormBlocks) * size;
    const int64_t at = (int64_t)(blockIdx.x % kNormBlocks) * 256 + threadIdx.x;
    constexpr int64_t stride = kNormBlocks * 256;
    double sum = 0.0;
    if (wide) {
        const int64_t chunks = size / E;
        for (int64_t i = at; i < chunks; i += 4 * stride) {
            alignas(16) T v[4][E];
#pragma unroll
            for (int j = 0; j < 4; ++j)   // past the end: the last chunk again, not added
                *reinterpret_cast<u32x4*>(v[j]) =
                    reinterpret_cast<const u32x4*>(u)[i + j * stride < chunks ? i + j * stride : chunks - 1];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * stride < chunks)
#pragma unroll
                    for (int e = 0; e < E; ++e) sum += (double)(float)v[j][e] * (double)(float)v[j][e];
        }
    } else {
        for (int64_t i = at; i < size; i += stride) sum += (double)(float)u[i] * (double)(float)u[i];
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) norm[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// X_0 as float16 pairs, padded; a 64 x 64 tile a workgroup, through LDS when
// the update is taken transposed.
template <class T>
__global__ __launch_bounds__(256) void orthogonalize_begin(const T* __restrict__ update, int m, int n, float eps,
                                                           const double* __restrict__ norm, int sp, int lp,
                                                           h16* __restrict__ x, int* __restrict__ lift) {
    __shared__ float tile[64][65];
    __shared__ double s_inv;
    const int tiles_l = lp / 64, tiles = tiles_l * (sp / 64);
    const int64_t b = blockIdx.x / tiles;
    const int i0 = (int)(blockIdx.x % tiles) / tiles_l * 64, j0 = (int)(blockIdx.x % tiles) % tiles_l * 64;
    const int tid = threadIdx.x;
    if (tid < 64) {
        double sum = norm[b * kNormBlocks + tid];
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (tid == 0) {
            const double f = sqrt(sum);
            const int up = lift_of(f, eps);
            s_inv = scale_of(f, eps, kLogScaleX + up);
            if (blockIdx.x % tiles == 0) lift[b] = up;
        }
    }
    const bool turned = m > n;
    const T* u = update + b * (int64_t)m * n;
    // rows of U along tid / 64, columns along tid % 64
    const int r0 = turned ? j0 : i0, c0 = turned ? i0 : j0;
    for (int r = tid >> 6; r < 64; r += 4) {
        const int row = r0 + r, col = c0 + (tid & 63);
        const float v = row < m && col < n ? (float)u[(int64_t)row * n + col] : 0.0f;
        if (turned) tile[tid & 63][r] = v;
        else tile[r][tid & 63] = v;
    }
    __syncthreads();
    const double inv = s_inv;
    x += b * sp * (int64_t)lp * 2;
    for (int r = tid >> 3; r < 64; r += 32) {   // 8 values a thread
        const int c = (tid & 7) * 8;
        f16x8 hi, lo;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h16 h, w;
            split((float)((double)tile[r][c + i] * inv), h, w);
            hi[i] = h;
            lo[i] = w;
        }
        h16* at = x + place(i0 + r, lp, j0 + c);
        *reinterpret_cast<f16x8*>(at) = hi;
        *reinterpret_cast<f16x8*>(at + kLow) = lo;
    }
}

// Workgroup b's place in the order of `count` equal tiles: consecutive
// workgroups go to the 8 dies in turn; this gives each die one run, so that
// its L2 holds few matrices (a whole one, of a batch of 8). The grid is
// die_grid(count); places at or past `count` are none.
__device__ __forceinline__ int64_t die_place(int64_t count) {
    return (int64_t)(blockIdx.x & 7) * ((count + 7) / 8) + (blockIdx.x >> 3);
}
__host__ __forceinline__ unsigned die_grid(int64_t count) { return (unsigned)((count + 7) / 8 * 8); }

// (The squares' arguments, and the updates' that come before the last step's
// own, fill one 64-byte line: a second one costs 0.3 us a launch.)

// Tile (ti, tj), ti >= tj, of the lower triangle.
__device__ __forceinline__ void triangle_tile(int id, int& ti, int& tj) {
    ti = (int)((__builtin_sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
    while ((ti + 1) * (ti + 2) / 2 <= id) ++ti;
    while (ti * (ti + 1) / 2 > id) --ti;
    tj = id - ti * (ti + 1) / 2;
}

// Off-diagonal pairs and the diagonal of a symmetric matrix, from the tiles
// of its lower triangle: POLY = false: A = X X^T; true: a + B = a + b A + c A A,
// times what takes X to the next step's lift. The upper triangle is written from the same tiles, transposed in LDS by each
// wave for itself.
template <class Tile, bool POLY>
__global__ __launch_bounds__(Tile::THREADS) void orthogonalize_square(const h16* __restrict__ in, int sp, int K, int tiles,
                                                                      int count, const int* __restrict__ lift,
                                                                      const float* __restrict__ diag, h16* __restrict__ out,
                                                                      float* __restrict__ out_diag, int step) {
    constexpr int BT = Tile::BN;
    // a wave's transposed pair of blocks: 32 rows n of MT 16 columns m
    constexpr int kTurnRow = Tile::MT * 16 + 8, kTurn = 32 * kTurnRow * 2;
    constexpr int kTurnBytes = kTurn * 2 * (Tile::THREADS / 64);
    __shared__ alignas(16) char lds[Tile::kLdsBytes > kTurnBytes ? Tile::kLdsBytes : kTurnBytes];
    int ti, tj;
    const int64_t id = die_place(count);
    if (id >= count) return;
    const int64_t b = id / tiles;
    triangle_tile((int)(id % tiles), ti, tj);
    const int tid = threadIdx.x, lane = tid & 63, m0 = ti * BT, n0 = tj * BT;
    in += b * (int64_t)sp * K * 2;
    out += b * (int64_t)sp * sp * 2;
    out_diag += b * sp;
    if constexpr (POLY) diag += b * sp;
    const int lifted = lift[b];
    asm("" : "+s"(step));   // both are loaded here, not after the product
    Tile t;
    t.run(lds, {in + (int64_t)n0 * K * 2, (int64_t)K * 2, sp - n0}, {in + (int64_t)m0 * K * 2, (int64_t)K * 2, sp - m0}, K, tid);
    const int held = lift_at(lifted, step);
    const float scale = __builtin_ldexpf(1.0f, POLY ? lift_at(lifted, step + 1) - held : -2 * held);
    h16* turn = reinterpret_cast<h16*>(lds) + (tid >> 6) * kTurn;
#pragma unroll
    for (int a = 0; a < Tile::NT; a += 2) {
        const int n = n0 + Tile::n_of(tid, a);
#pragma unroll
        for (int c = 0; c < Tile::MT; ++c) {
            const int m = m0 + Tile::m_of(tid, c);
            const bool inside = n < sp && m < sp;
            f16x8 ohi, olo;
            float dm = 0.0f;
            f32x4 dn[2];
            if constexpr (POLY) {
                const int ms = m < sp ? m : sp - 1, ns = n < sp ? n : sp - 8;   // outside: any value, not stored
                const h16* at = in + place(ms, sp, ns);
                ohi = *reinterpret_cast<const f16x8*>(at);
                olo = *reinterpret_cast<const f16x8*>(at + kLow);
                dm = diag[ms];
                dn[0] = *reinterpret_cast<const f32x4*>(diag + ns);
                dn[1] = *reinterpret_cast<const f32x4*>(diag + ns + 4);
            }
            f16x8 vhi, vlo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = t.acc[a + (i >> 2)][c][i & 3];
                float off;   // the off-diagonal value, scaled
                if constexpr (POLY) {
                    const float o = (float)ohi[i] + (float)olo[i];
                    // v = kScaleO^2 (O O)_mn, o = kScaleO O_mn
                    off = ((kC * kScaleB / (kScaleO * kScaleO)) * v +
                           (kScaleB / kScaleO) * (kB + kC * (dm + dn[i >> 2][i & 3])) * o) * scale;
                    if (m == n + i && inside)
                        out_diag[m] = (kA + (kC * (v * (1.0f / (kScaleO * kScaleO)) + dm * dm) + kB * dm)) * scale;
                } else {
                    off = v * (kScaleO / (kScaleX * kScaleX)) * scale;
                    if (m == n + i && inside) out_diag[m] = v * (1.0f / (kScaleX * kScaleX)) * scale;
                }
                h16 h, l;
                split(m == n + i ? 0.0f : off, h, l);
                vhi[i] = h;
                vlo[i] = l;
                if (ti != tj) {
                    h16* to = turn + (8 * (lane >> 4) + i) * kTurnRow + c * 16 + (lane & 15);
                    to[0] = h;
                    to[32 * kTurnRow] = l;
                }
            }
            if (inside) {
                h16* to = out + place(m, sp, n);
                *reinterpret_cast<f16x8*>(to) = vhi;
                *reinterpret_cast<f16x8*>(to + kLow) = vlo;
            }
        }
        if (ti != tj) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own writes
            constexpr int kRowChunks = Tile::MT * 2;
            const int row0 = n0 + Tile::n_of(tid & ~63, a), col0 = m0 + Tile::m_of(tid & ~63, 0);
#pragma unroll
            for (int k = 0; k < 32 * kRowChunks; k += 64) {
                const int row = (k + lane) / kRowChunks, chunk = (k + lane) % kRowChunks;
                const int rn = row0 + row, cm = col0 + chunk * 8;
                const h16* from = turn + row * kTurnRow + chunk * 8;
                const f16x8 hi = *reinterpret_cast<const f16x8*>(from);
                const f16x8 lo = *reinterpret_cast<const f16x8*>(from + 32 * kTurnRow);
                if (rn < sp && cm < sp) {
                    h16* to = out + place(rn, sp, cm);
                    *reinterpret_cast<f16x8*>(to) = hi;
                    *reinterpret_cast<f16x8*>(to + kLow) = lo;
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    }
}

// X <- (a + B_ii) X_i + (off-diagonal B) X. LAST: the result goes to `out` in
// its own type and orientation ([m, n], transposed if `turned`) instead.
template <class T, class Tile, bool LAST>
__global__ __launch_bounds__(Tile::THREADS) void orthogonalize_update(
    const h16* __restrict__ poly, const float* __restrict__ bdiag, const h16* __restrict__ x, int sp, int lp,
    h16* __restrict__ y, int tiles_n, int tiles, int count, int step, const int* __restrict__ lift,
    T* __restrict__ out, int s, int l, bool turned, bool wide) {
    constexpr int BN = Tile::BN, BM = Tile::BM;
    __shared__ alignas(16) char lds[Tile::kLdsBytes];
    const int64_t id = die_place(count);
    if (id >= count) return;
    const int64_t b = id / tiles;
    const int tile = (int)(id % tiles);
    const int m0 = tile / tiles_n * BM, n0 = tile % tiles_n * BN;
    const int tid = threadIdx.x;
    poly += (b * sp + m0) * (int64_t)sp * 2;
    x += b * sp * (int64_t)lp * 2;
    y += b * sp * (int64_t)lp * 2;
    bdiag += b * sp;
    int lifted = 0;
    if constexpr (LAST) {
        lifted = lift[b];
        asm("" : "+s"(step));   // both are loaded here, not after the product
        out += b * (int64_t)s * l;
    }
    Tile t;
    t.run(lds, {x + n0 * 2, (int64_t)lp * 2, lp - n0}, {poly, (int64_t)sp * 2, sp - m0}, sp, tid);
    const int back = -kLogScaleX - lift_at(lifted, step + 1);
#pragma unroll
    for (int a = 0; a < Tile::NT; a += 2) {
        const int n = n0 + Tile::n_of(tid, a);
        if (n >= lp) continue;
#pragma unroll
        for (int c = 0; c < Tile::MT; ++c) {
            const int m = m0 + Tile::m_of(tid, c);
            if (m >= sp) continue;
            const int64_t at = place(m, lp, n);
            const f16x8 ohi = *reinterpret_cast<const f16x8*>(x + at), olo = *reinterpret_cast<const f16x8*>(x + at + kLow);
            const float scale = bdiag[m];
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = scale * ((float)ohi[i] + (float)olo[i]) + t.acc[a + (i >> 2)][c][i & 3] * (1.0f / kScaleB);
            if constexpr (!LAST) {
                f16x8 vhi, vlo;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h16 h, w;
                    split(v[i], h, w);
                    vhi[i] = h;
                    vlo[i] = w;
                }
                *reinterpret_cast<f16x8*>(y + at) = vhi;
                *reinterpret_cast<f16x8*>(y + at + kLow) = vlo;
            } else if (m < s) {
                if (!turned && wide) {   // rows of whole 16 bytes
                    if (n < l) {
                        struct alignas(16) Row { T v[8]; } row;
#pragma unroll
                        for (int i = 0; i < 8; ++i) row.v[i] = (T)__builtin_ldexpf(v[i], back);
                        T* to = out + (int64_t)m * l + n;
                        if (sizeof(T) == 2 || n + 4 < l) *reinterpret_cast<Row*>(to) = row;
                        else
#pragma unroll
                            for (int i = 0; i < 4; ++i) to[i] = row.v[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (n + i < l)
                            out[turned ? (int64_t)(n + i) * s + m : (int64_t)m * l + n + i] = (T)__builtin_ldexpf(v[i], back);
                }
            }
        }
    }
}

// The side of the tiles of X: larger ones are worth while where about one is
// there for each of the 256 compute units (one 1024 x 2048 in float32, 128 tiles
// of 128 x 128: 549 us with them, 419 with 64 x 64; one 2048 x 2048, 256 of them:
// 814 and 1499), and 256 where they pad X by a quarter more than 128 at most (30
// of 300 x 2000: 735 us with, 635 without). The squares' halves take 128 x 128
// tiles with either (4 of 2048 x 2048: 143 us with 256 x 256, 123 with 128 x 128).
int tile_side(int64_t B, const Layout& w) {
    const auto count = [&](int t) { return B * ((w.sp + t - 1) / t) * ((w.lp + t - 1) / t); };
    if (count(256) >= 224 && count(256) * 16 <= count(128) * 5) return 256;
    return count(128) >= 256 ? 128 : 64;
}

template <class Kernel>
hipError_t allow_lds(Kernel kernel, int bytes) {
    return bytes <= 65536 ? hipSuccess
                          : hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <class T, class Square, class Update>
hipError_t launch_steps(const OrthogonalizeArgs& a, const Layout& w) {
    static_assert(Square::THREADS <= 512 && Update::THREADS <= 512, "orthogonalize_workspace counts on it");
    auto half = [&](int64_t o) { return reinterpret_cast<h16*>(a.workspace + o); };
    auto real = [&](int64_t o) { return reinterpret_cast<float*>(a.workspace + o); };
    const int* lift = reinterpret_cast<const int*>(a.workspace + w.lift);
    const int side = (w.sp + Square::BN - 1) / Square::BN, triangle = side * (side + 1) / 2;
    const int tiles_n = (w.lp + Update::BN - 1) / Update::BN, tiles = tiles_n * ((w.sp + Update::BM - 1) / Update::BM);
    const int squares = (int)a.B * triangle, updates = (int)a.B * tiles;   // no more than 64 x 64 tiles of X
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.n % (16 / (int)sizeof(T)) == 0;
    int cur = 0;
    for (int k = 0; k < a.steps; ++k) {
        orthogonalize_square<Square, false><<<die_grid(squares), Square::THREADS, 0, a.stream>>>(
            half(w.x[cur]), w.sp, w.lp, triangle, squares, lift, nullptr, half(w.o), real(w.diag), k);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        orthogonalize_square<Square, true><<<die_grid(squares), Square::THREADS, 0, a.stream>>>(
            half(w.o), w.sp, w.sp, triangle, squares, lift, real(w.diag), half(w.b), real(w.bdiag), k);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        auto update = [&](auto kernel) {
            kernel<<<die_grid(updates), Update::THREADS, 0, a.stream>>>(
                half(w.b), real(w.bdiag), half(w.x[cur]), w.sp, w.lp, half(w.x[cur ^ 1]), tiles_n, tiles, updates, k,
                lift, static_cast<T*>(a.out), w.s, w.l, a.m > a.n, wide);
        };
        if (k + 1 < a.steps) update(orthogonalize_update<T, Update, false>);
        else update(orthogonalize_update<T, Update, true>);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
        cur ^= 1;
    }
    return hipSuccess;
}

template <class T>
hipError_t launch_tiled(const OrthogonalizeArgs& a) {
    const Layout w = layout(a.B, a.m, a.n);
    const T* u = static_cast<const T*>(a.update);
    double* norm = reinterpret_cast<double*>(a.workspace + w.norm);
    const unsigned tiles64 = (unsigned)(a.B * (w.sp / 64) * (w.lp / 64));
    const int64_t size = (int64_t)a.m * a.n;
    orthogonalize_norm<T><<<(unsigned)(a.B * kNormBlocks), 256, 0, a.stream>>>(
        u, size, (reinterpret_cast<uintptr_t>(u) & 15) == 0 && size * sizeof(T) % 16 == 0, norm);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    orthogonalize_begin<T><<<tiles64, 256, 0, a.stream>>>(
        u, a.m, a.n, a.eps, norm, w.sp, w.lp, reinterpret_cast<h16*>(a.workspace + w.x[0]),
        reinterpret_cast<int*>(a.workspace + w.lift));
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    typedef PairProduct<128, 128, 2, 4, true, 2> Square;
    switch (tile_side(a.B, w)) {
        case 256: return launch_steps<T, Square, PairProduct<256, 256, 4, 2, false, 2>>(a, w);
        case 128: return launch_steps<T, Square, PairProduct<128, 128, 2, 4, false, 2>>(a, w);
        default: return launch_steps<T, PairProduct<64, 64, 2, 4, true, 8>, PairProduct<64, 64, 2, 4, false, 8>>(a, w);
    }
}

// Threads of a small matrix's workgroup.
int small_threads(const SmallShape& h) {
    const int st = h.sp / 16;
    return st * (h.lp / 16) <= 16 && st * (st + 1) / 2 <= 4 ? 256 : kSmallThreads;
}

template <class T>
hipError_t launch_small(const OrthogonalizeArgs& a) {
    const SmallShape h = small_shape(a.m, a.n);
    const int threads = small_threads(h);
    const auto kernel = threads == 256 ? orthogonalize_small<T, 256> : orthogonalize_small<T, kSmallThreads>;
    const hipError_t err = allow_lds(kernel, (int)h.bytes);
    if (err != hipSuccess) return err;
    kernel<<<(unsigned)a.B, threads, h.bytes, a.stream>>>(static_cast<const T*>(a.update), a.m, a.n, a.steps, a.eps,
                                                          static_cast<T*>(a.out));
    return hipGetLastError();
}

}  // namespace

size_t orthogonalize_workspace(int64_t B, int32_t m, int32_t n) {
    if (is_small(m, n)) return B <= kMaxWorkItems / small_threads(small_shape(m, n)) ? 256 : 0;
    const Layout one = layout(1, m, n);
    // the norm takes kNormBlocks workgroups of 256 for a matrix, the products
    // one of 512 for a 64 x 64 tile (of larger tiles there are fewer), their
    // number rounded up to 8
    const int64_t tiles = (int64_t)(one.sp / 64) * (one.lp / 64);
    if (B > kMaxWorkItems / (kNormBlocks * 256) || B > (kMaxWorkItems / 512 - 7) / tiles) return 0;
    return layout(B, m, n).bytes;
}

int orthogonalize_tile(int64_t B, int32_t m, int32_t n) { return is_small(m, n) ? 0 : tile_side(B, layout(B, m, n)); }

hipError_t launch_orthogonalize(const OrthogonalizeArgs& a) {
    timing_begin(kKOrthogonalize, a.stream);
    const bool small = is_small(a.m, a.n);
    hipError_t err = hipErrorInvalidValue;
    switch (a.dtype) {
        case DMR_FLOAT32: err = small ? launch_small<float>(a) : launch_tiled<float>(a); break;
        case DMR_FLOAT16: err = small ? launch_small<_Float16>(a) : launch_tiled<_Float16>(a); break;
        case DMR_BFLOAT16: err = small ? launch_small<__bf16>(a) : launch_tiled<__bf16>(a); break;
    }
    timing_end(kKOrthogonalize, a.stream);
    return err;
}

}  // namespace dmr

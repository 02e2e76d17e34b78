// Matrix-core tiles shared by the layers and the optimiser's products.
//
// A workgroup computes a BM x BN tile of C[m][n] = sum_k Q[m][k] P[n][k] in
// float32 accumulators. Both operands are staged in LDS 128 bytes of k (whole
// cache lines of a row) at a time, in a ring of S stages. A step is two slices
// of 64 bytes of k: while the matrix cores work on one slice's fragments, the
// next slice's are read from LDS into a second set of registers. In the middle
// of a step its last fragments have been read, so its stage is free there:
// that is where the one barrier of a step stands, and where the loads, which
// go straight from memory into LDS, are issued S steps ahead.
//
// What bounds a tile: 256 x 256 16-bit tiles take 64 KB of loads for 2048
// cycles of the matrix cores, and the LDS holds two steps. On 131072 rows of
// 2048 to 2048 the products alone take 752 us, the loads alone 849 and both
// 990 (1.1 PFLOP/s). Steps of 64 bytes (half lines, four stages) are 9%
// slower, 128 x 128 tiles 35%; a ring of three stages for one operand, loads
// into L2 ahead, and a fixed order of loads, reads and products change little.
//
// P is the first operand of the matrix instruction and n its row index, so
// that a lane's four accumulators are four consecutive n of one row m of C:
// C is stored n-contiguous, 16 bytes a lane.
//
// An operand is K-major (row r at base + r ld, k contiguous) or M-major (k at
// base + k ld, rows contiguous), as memory has it; 16-bit M-major tiles are
// transposed on the way from LDS to registers (ds_read_b64_tr_b16: 16 lanes
// read a 4 x 16 block and get its columns). Which k a lane holds does not
// matter as long as both operands agree, so float32 operands take four
// consecutive k of a lane for four successive instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dmr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Bytes of k in a step.
constexpr int kStepBytes = 128;

#define DMR_LDS __attribute__((address_space(3)))

// An offset past every buffer descriptor's range: loads from it give zero.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;
constexpr uint32_t kBufferRange = 0x80000000u;

// The bits of 1, twice.
template <class T>
constexpr uint32_t one_bits();
template <>
constexpr uint32_t one_bits<_Float16>() { return 0x3C003C00u; }
template <>
constexpr uint32_t one_bits<__bf16>() { return 0x3F803F80u; }

// 16 bytes of an operand's fragment: 8 16-bit or 4 float32 elements of k.
template <class T>
__device__ __forceinline__ f32x4 mma(u32x4 p, u32x4 q, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma<_Float16>(u32x4 p, u32x4 q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<__bf16>(u32x4 p, u32x4 q, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<float>(u32x4 p, u32x4 q, f32x4 c) {
    const f32x4 a = __builtin_bit_cast(f32x4, p), b = __builtin_bit_cast(f32x4, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// What is left of v beside its high part in bfloat16 (nothing beside one that
// is not finite).
__device__ __forceinline__ float low_of(float v) {
    const float high = (float)(__bf16)v;
    return __builtin_fabsf(high) < __builtin_inff() ? v - high : 0.0f;
}
__device__ __forceinline__ f32x4 low_of(f32x4 v) { return f32x4{low_of(v[0]), low_of(v[1]), low_of(v[2]), low_of(v[3])}; }

// Both parts of a fragment's eight values as bfloat16.
template <class T>
__device__ __forceinline__ u32x4 high_bf16(u32x4 raw) {
    T v[8];
    __bf16 out[8];
    __builtin_memcpy(v, &raw, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (__bf16)(float)v[i];
    __builtin_memcpy(&raw, out, 16);
    return raw;
}
template <class T>
__device__ __forceinline__ u32x4 low_bf16(u32x4 raw) {
    T v[8];
    __bf16 out[8];
    __builtin_memcpy(v, &raw, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (__bf16)low_of((float)v[i]);
    __builtin_memcpy(&raw, out, 16);
    return raw;
}

// One operand's staged step: ROWS rows of KB bytes of k (K-major: 128).
// SPREAD: M-major fragments of 16-bit rows are paired.
//
// LDS holds it in 16-byte chunks in the order memory has it (the loads write
// LDS linearly, lane after lane), with the chunks of a line exchanged by a
// swizzle so that the 16 lanes of a fragment read hit different banks.
template <class T, int ROWS, bool KMAJOR, int THREADS, int KB = kStepBytes, bool SPREAD = false>
struct OperandTile {
    static constexpr int kElems = 16 / (int)sizeof(T);   // elements of a chunk
    static constexpr int BK = KB / (int)sizeof(T);
    static constexpr int kBytes = ROWS * KB;
    static constexpr int kChunks = kBytes / 16;
    static constexpr int kLoads = (kChunks + THREADS - 1) / THREADS;   // of a thread, at most
    static constexpr int kLoadsLeast = kChunks / THREADS;              // of a wave, at least
    // chunks of a line: a row's k, or the rows of one k
    static constexpr int kLine = KMAJOR ? KB / 16 : ROWS / kElems;

    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KMAJOR) {
            // rows differing in bits 0..3, or in bits 0, 1, 3 and 4, land on
            // 16 different 16-byte slots of 256
            return ((line >> 1) & 1) | (((line >> 2) ^ (line >> 4)) & 1) << 1 | ((line >> 3) & 1) << 2;
        } else if constexpr (sizeof(T) == 2) {
            // paired: the lanes of one k use halves of 4 chunks; not paired: 2
            // whole chunks, and the next 8 of k other ones
            if constexpr (SPREAD) return kLine >= 16 ? (line & 3) << 2 : kLine == 8 ? (line & 2) << 1 : 0;
            else return kLine >= 16 ? ((line & 3) << 1) | (((line >> 3) & 1) << 3) : kLine == 8 ? (line & 2) | ((line >> 3) & 1) << 2 : 0;
        } else {
            return kLine >= 16 ? ((line >> 2) & 3) << 2 : 0;
        }
    }

    // Where a thread's chunks are, from row 0 and the step's first k: byte
    // offsets, past the buffer's range for rows that do not exist.
    struct Offsets {
        uint32_t at[kLoads];
    };
    static __device__ __forceinline__ Offsets offsets(int64_t ld, int rows, int tid) {
        Offsets o;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = i * THREADS + tid;
            const int line = c / kLine, chunk = (c % kLine) ^ swizzle(line);
            const int row = KMAJOR ? line : chunk * kElems;
            o.at[i] = row < rows ? (uint32_t)line * (uint32_t)(ld * sizeof(T)) + (uint32_t)chunk * 16u : kNowhere;
        }
        return o;
    }

    // Loads k in [k0, k0 + BK) of rows [0, ROWS) into LDS: zero where the row
    // is not below `rows` or k not below K. `base` points at row 0 and k = 0;
    // it and ld are multiples of 16 bytes, and so is the extent of the
    // contiguous direction, so that a chunk is inside or outside as a whole.
    static __device__ __forceinline__ void stage(char* lds, const T* base, int64_t ld, const Offsets& o, int k0, int K,
                                                 int tid) {
        const T* at = KMAJOR ? base + k0 : base + (int64_t)k0 * ld;
        const int kleft = K - k0;
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(at), 0, kBufferRange, 0x00020000);
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const bool whole = kleft >= BK;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (kChunks % THREADS != 0 && i * THREADS + wave * 64 >= kChunks) break;
            uint32_t off = o.at[i];
            if (!whole) {
                const int c = i * THREADS + tid, line = c / kLine;
                const int k = KMAJOR ? ((c % kLine) ^ swizzle(line)) * kElems : line;
                if (k >= kleft) off = kNowhere;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (DMR_LDS void*)(lds + (i * THREADS + wave * 64) * 16), 16, off, 0, 0,
                                                     0);
        }
    }

    // The same for arrays that are not so aligned, by way of registers: fetch
    // issues the loads, put writes them to LDS. A chunk that lies inside is
    // one load at whatever alignment it has; one that crosses the end is read
    // element by element.
    struct Held {
        u32x4 chunk[kLoads];
    };
    static __device__ __forceinline__ void fetch(Held& h, const T* base, int64_t ld, int rows, int k0, int K, int tid) {
        const T* at = KMAJOR ? base + k0 : base + (int64_t)k0 * ld;
        const int kleft = K - k0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = i * THREADS + tid;
            const int line = c / kLine, chunk = (c % kLine) ^ swizzle(line);
            // of the contiguous direction, this chunk's elements that exist
            const bool is = c < kChunks && line < (KMAJOR ? rows : kleft);
            const int left = is ? (KMAJOR ? kleft : rows) - chunk * kElems : 0;
            const T* from = at + (int64_t)line * ld + chunk * kElems;
            h.chunk[i] = u32x4{0, 0, 0, 0};
            if (left >= kElems) {
                __builtin_memcpy(&h.chunk[i], from, 16);
            } else if (left > 0) {
                T v[kElems];
#pragma unroll
                for (int e = 0; e < kElems; ++e) v[e] = e < left ? from[e] : (T)0.0f;
                __builtin_memcpy(&h.chunk[i], v, 16);
            }
        }
    }
    static __device__ __forceinline__ void put(char* lds, const Held& h, int tid) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = i * THREADS + tid;
            if (kChunks % THREADS == 0 || c < kChunks) *reinterpret_cast<u32x4*>(lds + c * 16) = h.chunk[i];
        }
    }

    // The fragment of 16 rows for the slice `kk` (64 bytes) of k: lane l
    // holds row row_of(l & 15) and the slice's 16-byte part l >> 4 of k. The
    // rows are given as row_of(4 a + i) = first + stride a + i.
    static __device__ __forceinline__ u32x4 fragment(const char* lds, int kk, int first, int stride, int lane) {
        const int q = lane >> 4, r = lane & 15;
        if constexpr (KMAJOR) {
            const int row = first + stride * (r >> 2) + (r & 3);
            return *reinterpret_cast<const u32x4*>(lds + row * KB + (((kk * 4 + q) ^ swizzle(row)) << 4));
        } else if constexpr (sizeof(T) == 2) {
            s16x4 half[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kk * 32 + 8 * q + 4 * h + (r >> 2);
                const int row = first + stride * (r & 3);
                const int at = k * (ROWS * 2) + (((row >> 3) ^ swizzle(k)) << 4) + (row & 7) * 2;
                half[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DMR_LDS s16x4*)(lds + at));
            }
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int row = first + stride * (r >> 2) + (r & 3);
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = kk * 16 + 4 * q + j;
                v[j] = *reinterpret_cast<const uint32_t*>(lds + k * (ROWS * 4) + (((row >> 2) ^ swizzle(k)) << 4) + (row & 3) * 4);
            }
            return v;
        }
    }
};

// Two M-major fragments of 16-bit rows that are paired (rows first + 8 a + i,
// and 4 further): the lanes of one k read halves of chunks, so lanes of odd q
// read the other fragment's half first, and together they use whole chunks and
// all banks.
template <class Tile>
__device__ __forceinline__ void paired_fragments(const char* lds, int kk, int first, int lane, u32x4& even, u32x4& odd) {
    const int q = lane >> 4;
    const u32x4 a = Tile::fragment(lds, kk, first + 4 * (q & 1), 8, lane);
    const u32x4 b = Tile::fragment(lds, kk, first + 4 - 4 * (q & 1), 8, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        even[j] = q & 1 ? b[j] : a[j];
        odd[j] = q & 1 ? a[j] : b[j];
    }
}

// Waits until at most N of this wave's loads into LDS are outstanding and all
// its reads from LDS are done, then for the other waves. (A barrier alone
// waits for neither.)
template <int N>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The tile product of one workgroup: WN x WM waves, each NT x MT blocks of
// 16 x 16. Of 16-bit types, neighbouring blocks of n are paired so that a lane
// holds eight consecutive n. SUMS: sum over k of Q[m][k] as well.
// PLANES: P is that many matrices, the same COLUMNS = BN / PLANES of n of each:
// a lane holds the same n of them in blocks PN apart.
// TERMS of 2 or 3: Q is a pair of matrices, high + low (which hold twice the
// bits of T's significand), and the sum of the products with each is formed.
// Three where P is a pair as well: the third is P's low part with Q's high one
// (low with low is at most 2^-16 of the product). A step takes all parts where
// the LDS holds two workgroups so (INNER); larger tiles take the terms one after
// another, as one sum over k of TERMS times the steps. P's type PT may be another
// than T = bfloat16: its float16 values are pairs of bfloat16 exactly, and those
// are formed as fragments are multiplied (of INNER tiles). OUT: the results'.
template <class T, int BN_, int BM_, int WN, int WM, bool PK, bool QK, int S, bool SUMS = false, int PLANES = 1, class PT = T,
          int TERMS = 1, class OUT = PT>
struct TileProduct {
    static constexpr int BN = BN_, BM = BM_, THREADS = WN * WM * 64, COLUMNS = BN / PLANES;
    static constexpr int NT = BN / WN / 16, MT = BM / WM / 16, PN = NT / PLANES;
    static constexpr int BK = kStepBytes / (int)sizeof(T);
    static constexpr bool PAIRED = sizeof(T) == 2 && PN % 2 == 0;
    using P = OperandTile<PT, COLUMNS, PK, THREADS, kStepBytes, PAIRED>;
    using Q = OperandTile<T, BM, QK, THREADS>;
    using PType = PT;
    using Out = OUT;
    static constexpr bool SPLIT = !__is_same(T, PT);
    static constexpr bool INNER = TERMS > 1 && S * ((TERMS == 3 && !SPLIT ? 2 : 1) * P::kBytes + 2 * Q::kBytes) <= 80 * 1024;
    static_assert((!SPLIT || (TERMS == 3 && INNER)) && sizeof(T) == sizeof(PT) && (TERMS == 1 || PLANES == 1), "");
    // matrices of a step
    static constexpr int PS = INNER && TERMS == 3 && !SPLIT ? 2 : PLANES, QS = INNER ? 2 : 1;
    static constexpr int kP = PS * P::kBytes, kStage = kP + QS * Q::kBytes, kLdsBytes = S * kStage;
    static_assert(S >= 2 && kLdsBytes <= 160 * 1024 && PN * PLANES == NT, "");

    template <class E>
    struct Operand {   // at row 0 of the tile and k = 0
        const E* at;
        int64_t ld;
        int rows;       // that exist
        const E* low;   // of a pair
    };
    using Source = Operand<T>;
    using PSource = Operand<PT>;
    struct Planes {   // of the same ld and rows
        PSource plane[PLANES];
        __device__ __forceinline__ const PSource& operator[](int i) const { return plane[i]; }
        __device__ __forceinline__ Planes(const PSource& s) : plane{s} {}
        __device__ __forceinline__ Planes(const PSource& s, const PSource& t) : plane{s, t} {}
    };
    struct Fragments {
        u32x4 p[NT], q[MT], p_low[PS > PLANES ? NT : 1], q_low[QS > 1 ? MT : 1];
    };

    f32x4 acc[NT][MT];
    f32x4 ones[SUMS ? MT : 1];

    // First n of this lane's values of block a, and its row m of block b.
    static __device__ __forceinline__ int n_of(int tid, int a) {
        const int wn = (tid >> 6) % WN, q = (tid & 63) >> 4;
        const int c = a % PN;
        return wn * PN * 16 + (PAIRED ? (c >> 1) * 32 + 8 * q + 4 * (c & 1) : c * 16 + 4 * q);
    }
    static __device__ __forceinline__ int m_of(int tid, int b) {
        return ((tid >> 6) / WN) * MT * 16 + b * 16 + (tid & 15);
    }

    // Of step t, of `each` steps a term: its first k, and whose low part it takes.
    struct Step {
        int k0;
        bool p_low, q_low;
    };
    static __device__ __forceinline__ Step step(int t, int each) {
        if constexpr (TERMS == 1 || INNER) return {t * BK, false, false};
        const int term = (t >= each ? 1 : 0) + (TERMS > 2 && t >= 2 * each ? 1 : 0);
        return {(t - term * each) * BK, term == 2, term == 1};
    }
    static __device__ __forceinline__ int all_steps(int each) { return TERMS > 1 && !INNER ? TERMS * each : each; }
    // Matrix i of a step's.
    static __device__ __forceinline__ const PT* p_of(const Planes& p, int i, const Step& s) {
        if constexpr (PS > PLANES) return i == 0 ? p[0].at : p[0].low;
        else return TERMS > 1 && s.p_low ? p[i].low : p[i].at;
    }
    static __device__ __forceinline__ const T* q_of(const Source& q, int i, const Step& s) {
        if constexpr (QS > 1) return i == 0 ? q.at : q.low;
        else return TERMS > 1 && s.q_low ? q.low : q.at;
    }

    template <bool VEC, class Tile, class E>
    static __device__ __forceinline__ void stage(char* lds, const E* at, const Operand<E>& s, const typename Tile::Offsets& o,
                                                 int k0, int K, int tid) {
        if constexpr (VEC) {
            Tile::stage(lds, at, s.ld, o, k0, K, tid);
        } else {
            typename Tile::Held h;
            Tile::fetch(h, at, s.ld, s.rows, k0, K, tid);
            Tile::put(lds, h, tid);
        }
    }

    static __device__ __forceinline__ void read_p(u32x4 (&p)[NT], const char* lds_p, int kk, int tid) {
        const int lane = tid & 63, wn = (tid >> 6) % WN;
#pragma unroll
        for (int a = 0; a < NT; ++a) {
            const char* plane = lds_p + a / PN * P::kBytes;
            const int c = a % PN;
            if constexpr (PAIRED && !PK) {
                if (c % 2 == 0) paired_fragments<P>(plane, kk, wn * PN * 16 + c * 16, lane, p[a], p[a + 1]);
            } else p[a] = P::fragment(plane, kk, wn * PN * 16 + (PAIRED ? (c >> 1) * 32 + 4 * (c & 1) : c * 16), PAIRED ? 8 : 4, lane);
        }
    }
    static __device__ __forceinline__ void read_q(u32x4 (&q)[MT], const char* lds_q, int kk, int tid) {
        const int lane = tid & 63, wm = (tid >> 6) / WN;
#pragma unroll
        for (int b = 0; b < MT; ++b) q[b] = Q::fragment(lds_q, kk, (wm * MT + b) * 16, 4, lane);
    }
    static __device__ __forceinline__ void read(Fragments& f, const char* lds_p, const char* lds_q, int kk, int tid) {
        read_p(f.p, lds_p, kk, tid);
        if constexpr (PS > PLANES) read_p(f.p_low, lds_p + P::kBytes, kk, tid);
        read_q(f.q, lds_q, kk, tid);
        if constexpr (QS > 1) read_q(f.q_low, lds_q + Q::kBytes, kk, tid);
    }

    __device__ __forceinline__ void multiply(const Fragments& f, bool sums) {
#pragma unroll
        for (int a = 0; a < NT; ++a) {
            const u32x4 p = SPLIT ? high_bf16<PT>(f.p[a]) : f.p[a];
#pragma unroll
            for (int b = 0; b < MT; ++b) acc[a][b] = mma<T>(p, f.q[b], acc[a][b]);
            if constexpr (INNER) {
#pragma unroll
                for (int b = 0; b < MT; ++b) acc[a][b] = mma<T>(p, f.q_low[b], acc[a][b]);
                if constexpr (TERMS == 3) {
                    const u32x4 low = SPLIT ? low_bf16<PT>(f.p[a]) : f.p_low[PS > PLANES ? a : 0];
#pragma unroll
                    for (int b = 0; b < MT; ++b) acc[a][b] = mma<T>(low, f.q[b], acc[a][b]);
                }
            }
        }
        if constexpr (SUMS && sizeof(T) == 4) {
            // on the vector units, which are free beside float32 products (a
            // product with ones is half as long again as a 64 x 64 tile's):
            // each lane its k, added over the lanes in the end
            if (sums)
#pragma unroll
                for (int b = 0; b < MT; ++b) ones[b] += __builtin_bit_cast(f32x4, f.q[b]);
        } else if constexpr (SUMS) {
            if (sums) {
                constexpr uint32_t w = one_bits<T>();
                const u32x4 one = {w, w, w, w};
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    ones[b] = mma<T>(one, f.q[b], ones[b]);
                    if constexpr (QS > 1) ones[b] = mma<T>(one, f.q_low[b], ones[b]);
                }
            }
        }
    }

    // Issues the loads of the first steps of a product over k in [0, K).
    template <bool VEC>
    static __device__ __forceinline__ void begin(char* lds, const Planes& p, const Source& q, int K, int tid) {
        const int each = (K + BK - 1) / BK, steps = all_steps(each);
        const typename P::Offsets po = P::offsets(p[0].ld, p[0].rows, tid);
        const typename Q::Offsets qo = Q::offsets(q.ld, q.rows, tid);
#pragma unroll
        for (int t = 0; t < S; ++t)
            if (t < steps) {
                const Step s = step(t, each);
#pragma unroll
                for (int i = 0; i < PS; ++i)
                    stage<VEC, P>(lds + t * kStage + i * P::kBytes, p_of(p, i, s), p[i % PLANES], po, s.k0, K, tid);
#pragma unroll
                for (int i = 0; i < QS; ++i)
                    stage<VEC, Q>(lds + t * kStage + kP + i * Q::kBytes, q_of(q, i, s), q, qo, s.k0, K, tid);
            }
    }

    // What the sums over k begin with: zero, or a value for each block of n.
    struct Zero {
        __device__ __forceinline__ f32x4 operator()(int) const { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    };

    // acc = from(n) + sum over k in [0, K), begun with the same arguments; the
    // LDS is free for other use afterwards. younger: since begin, each wave has
    // issued YOUNGER stores or more, which need not be done when the first
    // steps' loads, which are older, have to be.
    template <bool VEC, int YOUNGER = 0, class From = Zero>
    __device__ __forceinline__ void finish(char* lds, const Planes& p, const Source& q, int K, int tid, bool sums = false,
                                           const From& from = From(), bool younger = false) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int b = 0; b < MT; ++b) acc[a][b] = from(a);
        if constexpr (SUMS)
#pragma unroll
            for (int b = 0; b < MT; ++b) ones[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (K <= 0) return;
        const int each = (K + BK - 1) / BK, steps = all_steps(each);
        const typename P::Offsets po = P::offsets(p[0].ld, p[0].rows, tid);
        const typename Q::Offsets qo = Q::offsets(q.ld, q.rows, tid);
        // a wave's loads of a step; they arrive in the order of their issue
        constexpr int kLoads = VEC ? PS * P::kLoadsLeast + QS * Q::kLoadsLeast : 0;
        static_assert(YOUNGER == 0 || (S == 2 && VEC && kLoads + YOUNGER < 64), "");
        if (YOUNGER > 0 && younger && S <= steps) step_barrier<(S - 1) * kLoads + YOUNGER>();
        else if (S <= steps) step_barrier<(S - 1) * kLoads>();   // step 0 is here
        else step_barrier<0>();
        Fragments first, second;
        read(first, lds, lds + kP, 0, tid);
        int cur = 0;   // this step's stage
        for (int t = 0; t < steps; ++t) {
            char* const here = lds + cur;
            const bool add = sums && !step(t, each).p_low;   // Q's parts are added once
            read(second, here, here + kP, 1, tid);
            multiply(first, add);
            // step t is read, and the loads of step t + 1 have arrived
            if (YOUNGER > 0 && younger && t == 0 && S <= steps) step_barrier<(S - 2) * kLoads + YOUNGER>();
            else if (t - 1 + S < steps) step_barrier<(S - 2) * kLoads>();
            else step_barrier<0>();
            const bool more = t + S < steps;
            typename P::Held held_p[PS];
            typename Q::Held held_q[QS];
            if (more) {
                const Step s = step(t + S, each);
                if constexpr (VEC) {
#pragma unroll
                    for (int i = 0; i < PS; ++i) P::stage(here + i * P::kBytes, p_of(p, i, s), p[0].ld, po, s.k0, K, tid);
#pragma unroll
                    for (int i = 0; i < QS; ++i) Q::stage(here + kP + i * Q::kBytes, q_of(q, i, s), q.ld, qo, s.k0, K, tid);
                } else {
#pragma unroll
                    for (int i = 0; i < PS; ++i) P::fetch(held_p[i], p_of(p, i, s), p[0].ld, p[0].rows, s.k0, K, tid);
#pragma unroll
                    for (int i = 0; i < QS; ++i) Q::fetch(held_q[i], q_of(q, i, s), q.ld, q.rows, s.k0, K, tid);
                }
            }
            cur = cur + kStage == kLdsBytes ? 0 : cur + kStage;
            read(first, lds + cur, lds + cur + kP, 0, tid);   // past the end: not used
            multiply(second, add);
            if constexpr (!VEC)
                if (more) {
#pragma unroll
                    for (int i = 0; i < PS; ++i) P::put(here + i * P::kBytes, held_p[i], tid);
#pragma unroll
                    for (int i = 0; i < QS; ++i) Q::put(here + kP + i * Q::kBytes, held_q[i], tid);
                }
        }
        step_barrier<0>();
        if constexpr (SUMS && sizeof(T) == 4)
            if (sums)
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    float s = (ones[b][0] + ones[b][1]) + (ones[b][2] + ones[b][3]);
                    s += __shfl_xor(s, 16, 64);
                    s += __shfl_xor(s, 32, 64);
                    ones[b][0] = s;
                }
    }

    template <bool VEC>
    __device__ __forceinline__ void run(char* lds, const Planes& p, const Source& q, int K, int tid, bool sums = false) {
        begin<VEC>(lds, p, q, K, tid);
        finish<VEC>(lds, p, q, K, tid, sums);
    }
};

// The same product of operands that are pairs of float16, high + low: high
// high + high low + low high, three matrix instructions for one. In memory the
// 32 high parts of a block of 32 values are followed by their 32 low parts,
// so that a cache line of a row is a step of 32 k with both; row strides
// count float16. The step is long for its bytes (1.5 times that of one plane),
// so a plain ring of S stages feeds it: the loads of step t + S - 1 are issued
// as step t begins.
template <int BN_, int BM_, int WN, int WM, bool PK, int S>
struct PairProduct {
    typedef _Float16 T;
    static constexpr int BN = BN_, BM = BM_, THREADS = WN * WM * 64;
    static constexpr int NT = BN / WN / 16, MT = BM / WM / 16;
    static constexpr bool PAIRED = true;
    static_assert(NT % 2 == 0 && S >= 2, "");
    // M-major, the 2 BN float16 of a line and 32 lines
    using P = OperandTile<T, PK ? BN : 2 * BN, PK, THREADS, PK ? 128 : 64, true>;
    using Q = OperandTile<T, BM, true, THREADS>;
    static constexpr int kStage = P::kBytes + Q::kBytes, kLdsBytes = S * kStage;
    static_assert(kLdsBytes <= 160 * 1024, "");

    struct Source {
        const T* at;
        int64_t ld;
        int rows;   // that exist (M-major: values of a line)
    };

    f32x4 acc[NT][MT];

    static __device__ __forceinline__ int n_of(int tid, int a) {
        return ((tid >> 6) % WN) * NT * 16 + (a >> 1) * 32 + 8 * ((tid & 63) >> 4) + 4 * (a & 1);
    }
    static __device__ __forceinline__ int m_of(int tid, int b) {
        return ((tid >> 6) / WN) * MT * 16 + b * 16 + (tid & 15);
    }

    // acc = sum over k in [0, K), K a multiple of 32; the LDS is free for
    // other use afterwards.
    __device__ __forceinline__ void run(char* lds, const Source& p, const Source& q, int K, int tid) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int b = 0; b < MT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int steps = K / 32;
        const int rows_p = PK ? p.rows : 2 * p.rows;
        const typename P::Offsets po = P::offsets(p.ld, rows_p, tid);
        const typename Q::Offsets qo = Q::offsets(q.ld, q.rows, tid);
        constexpr int kLoads = P::kLoadsLeast + Q::kLoadsLeast;
        const auto stage = [&](char* to, int t) {
            P::stage(to, p.at, p.ld, po, t * P::BK, steps * P::BK, tid);
            Q::stage(to + P::kBytes, q.at, q.ld, qo, t * Q::BK, steps * Q::BK, tid);
        };
#pragma unroll
        for (int t = 0; t < S - 1; ++t)
            if (t < steps) stage(lds + t * kStage, t);
        const int lane = tid & 63, wn = (tid >> 6) % WN, wm = (tid >> 6) / WN;
        int cur = 0;
        for (int t = 0; t < steps; ++t) {
            // step t has arrived, and step t - 1 is multiplied
            if (t + S - 1 <= steps) step_barrier<kLoads * (S - 2)>();
            else step_barrier<0>();
            if (t + S - 1 < steps) stage(lds + (cur == 0 ? kLdsBytes - kStage : cur - kStage), t + S - 1);
            const char* at = lds + cur;
            u32x4 pf[2][NT], qf[2][MT];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const int n = wn * NT * 16 + (a >> 1) * 32, i = 4 * (a & 1);
                    pf[s][a] = PK ? P::fragment(at, s, n + i, 8, lane) : P::fragment(at, 0, 2 * n + 32 * s + i, 8, lane);
                }
#pragma unroll
                for (int b = 0; b < MT; ++b) qf[s][b] = Q::fragment(at + P::kBytes, s, (wm * MT + b) * 16, 4, lane);
            }
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int b = 0; b < MT; ++b) acc[a][b] = mma<T>(pf[0][a], qf[0][b], acc[a][b]);
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    acc[a][b] = mma<T>(pf[0][a], qf[1][b], acc[a][b]);
                    acc[a][b] = mma<T>(pf[1][a], qf[0][b], acc[a][b]);
                }
            cur = cur + kStage == kLdsBytes ? 0 : cur + kStage;
        }
        step_barrier<0>();
    }
};

// Stores two 16-byte chunks of a row that each of a fragment's lanes holds
// (chunk 0 and chunk 1 of its row: 64 bytes apart or more, four lanes to 64
// bytes) as whole 128-byte pieces of a row: neighbouring lanes, of
// neighbouring rows, exchange a chunk, and then store the even row's two and
// the odd row's two. put(odd row?, chunk, value).
template <class Put>
__device__ __forceinline__ void store_row_pairs(u32x4 c0, u32x4 c1, int lane, Put&& put) {
    const bool odd = lane & 1;
    u32x4 got;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t send = odd ? c0[j] : c1[j];
        got[j] = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0xB1, 0xF, 0xF, true);   // lane ^ 1
    }
    put(false, odd ? 1 : 0, odd ? got : c0);
    put(true, odd ? 1 : 0, odd ? c1 : got);
}

}  // namespace dmr

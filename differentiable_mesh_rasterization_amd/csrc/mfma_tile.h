// Matrix-core tiles shared by the layers and the optimiser's products.
//
// A workgroup computes a BM x BN tile of C[m][n] = sum_k Q[m][k] P[n][k] in
// float32 accumulators. Both operands are staged in LDS one K step of 128
// bytes at a time (BK = 64 16-bit or 32 float32 elements), double buffered:
// the loads of step t + 1 go straight from memory into LDS while the waves
// multiply step t.
//
// P is the first operand of the matrix instruction and n its row index, so
// that a lane's four accumulators are four consecutive n of one row m of C:
// C is stored n-contiguous, 16 bytes a lane.
//
// An operand is K-major (row r at base + r ld, k contiguous) or row-major in
// the other sense, "M-major" (k at base + k ld, rows contiguous), as memory
// has it; the transpose of 16-bit M-major tiles happens on the way from LDS
// to registers (ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block and get its
// columns). Which k a lane holds does not matter as long as both operands
// agree, so float32 operands take four consecutive k of a lane for four
// successive instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dmr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define DMR_LDS __attribute__((address_space(3)))

// Bytes of k in a staged step.
constexpr int kStepBytes = 128;

// An offset past every buffer descriptor's range: loads from it give zero.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;
constexpr uint32_t kBufferRange = 0x80000000u;

// The bits of 1 (16-bit types: twice).
template <class T>
constexpr uint32_t one_bits();
template <>
constexpr uint32_t one_bits<float>() { return 0x3F800000u; }
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

// Every wave's loads into LDS have arrived. (A barrier alone does not wait
// for loads from memory.)
__device__ __forceinline__ void staged_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// One operand's staged step: ROWS rows of 128 bytes of k.
//
// LDS holds it in 16-byte chunks in the order memory has it (the loads write
// LDS linearly, lane after lane), with the chunks of a row exchanged by a
// swizzle so that the 16 lanes of a fragment read hit different banks.
template <class T, int ROWS, bool KMAJOR, int THREADS>
struct OperandTile {
    static constexpr int kElems = 16 / (int)sizeof(T);          // elements of a chunk
    static constexpr int BK = kStepBytes / (int)sizeof(T);
    static constexpr int kBytes = ROWS * kStepBytes;
    static constexpr int kChunks = kBytes / 16;
    // chunks of one line: 8 of k of a row, or the rows of one k
    static constexpr int kLine = KMAJOR ? 8 : ROWS / kElems;

    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KMAJOR) {
            // rows differing in bits 0..3, or in bits 0, 1, 3 and 4, land on 16 different 16-byte slots of 256
            return ((line >> 1) & 1) | ((((line >> 2) ^ (line >> 4)) & 1) << 1) | (((line >> 3) & 1) << 2);
        } else if constexpr (sizeof(T) == 2) {
            return kLine >= 16 ? (line & 3) << 2 : kLine == 8 ? (line & 2) << 1 : 0;
        } else {
            return kLine >= 16 ? ((line >> 2) & 3) << 2 : 0;
        }
    }

    // Stages k in [k0, k0 + BK) of rows [0, ROWS): zero where the row is not
    // below `rows` or k not below K. `base` points at row 0 and k = 0.
    // VEC: base and ld are multiples of 16 bytes, and so is the extent of the
    // contiguous direction, so that a chunk is inside or outside as a whole.
    template <bool VEC>
    static __device__ __forceinline__ void stage(char* lds, const T* base, int64_t ld, int rows, int k0, int K, int tid) {
        const T* at = KMAJOR ? base + k0 : base + (int64_t)k0 * ld;
        const int kleft = K - k0;
        if constexpr (VEC) {
            const __amdgpu_buffer_rsrc_t rsrc =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(at), 0, kBufferRange, 0x00020000);
            const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
            for (int i = 0; i * THREADS < kChunks; ++i) {
                if (kChunks % THREADS != 0 && i * THREADS + wave * 64 >= kChunks) break;
                const int c = i * THREADS + tid;
                const int line = c / kLine, chunk = (c % kLine) ^ swizzle(line);
                const int row = KMAJOR ? line : chunk * kElems, k = KMAJOR ? chunk * kElems : line;
                const uint32_t off = (uint32_t)line * (uint32_t)(ld * sizeof(T)) + (uint32_t)chunk * 16u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (DMR_LDS void*)(lds + (i * THREADS + wave * 64) * 16), 16,
                                                         row < rows && k < kleft ? off : kNowhere, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i * THREADS < kChunks; ++i) {
                const int c = i * THREADS + tid;
                if (kChunks % THREADS != 0 && c >= kChunks) break;
                const int line = c / kLine, chunk = (c % kLine) ^ swizzle(line);
                const int row = KMAJOR ? line : chunk * kElems, k = KMAJOR ? chunk * kElems : line;
                const T* from = at + (int64_t)line * ld + chunk * kElems;
                alignas(16) T v[kElems];
#pragma unroll
                for (int e = 0; e < kElems; ++e) {
                    const bool in = KMAJOR ? row < rows && k + e < kleft : row + e < rows && k < kleft;
                    v[e] = in ? from[e] : (T)0.0f;
                }
                *reinterpret_cast<u32x4*>(lds + c * 16) = *reinterpret_cast<const u32x4*>(v);
            }
        }
    }

    // The fragment of 16 rows for k slice `kk` (64 bytes of k): lane l holds
    // row row_of(l & 15) and the slice's 16-byte part l >> 4 of k. The rows
    // are given as row_of(4 a + i) = first + stride a + i.
    static __device__ __forceinline__ u32x4 fragment(const char* lds, int kk, int first, int stride, int lane) {
        const int q = lane >> 4, r = lane & 15;
        if constexpr (KMAJOR) {
            const int row = first + stride * (r >> 2) + (r & 3);
            return *reinterpret_cast<const u32x4*>(lds + row * kStepBytes + (((kk * 4 + q) ^ swizzle(row)) << 4));
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

// The tile product of one workgroup: WN x WM waves, each NT x MT blocks of
// 16 x 16. 16-bit outputs pair neighbouring blocks of n so that a lane holds
// eight consecutive n (16 bytes).
template <class T, int BN_, int BM_, int WN, int WM, bool PK, bool QK>
struct TileProduct {
    static constexpr int BN = BN_, BM = BM_, THREADS = WN * WM * 64;
    static constexpr int NT = BN / WN / 16, MT = BM / WM / 16;
    static constexpr int BK = kStepBytes / (int)sizeof(T);
    static constexpr bool PAIRED = sizeof(T) == 2 && NT % 2 == 0;
    using P = OperandTile<T, BN, PK, THREADS>;
    using Q = OperandTile<T, BM, QK, THREADS>;
    static constexpr int kStage = P::kBytes + Q::kBytes;
    static constexpr int kLdsBytes = 2 * kStage;

    f32x4 acc[NT][MT];
    f32x4 ones[MT];   // SUMS: sum over k of Q[m][k]

    // First n of this lane's values of block a (pairs: of both blocks)
    static __device__ __forceinline__ int n_of(int tid, int a) {
        const int wn = (tid >> 6) % WN, q = (tid & 63) >> 4;
        return wn * NT * 16 + (PAIRED ? (a >> 1) * 32 + 8 * q + 4 * (a & 1) : a * 16 + 4 * q);
    }
    static __device__ __forceinline__ int m_of(int tid, int b) {
        return ((tid >> 6) / WN) * MT * 16 + b * 16 + (tid & 15);
    }

    template <bool SUMS>
    __device__ __forceinline__ void multiply(const char* lds, int tid) {
        const int lane = tid & 63, wn = (tid >> 6) % WN, wm = (tid >> 6) / WN;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            u32x4 p[NT], q[MT];
#pragma unroll
            for (int a = 0; a < NT; ++a)
                p[a] = P::fragment(lds, kk, wn * NT * 16 + (PAIRED ? (a >> 1) * 32 + 4 * (a & 1) : a * 16), PAIRED ? 8 : 4, lane);
#pragma unroll
            for (int b = 0; b < MT; ++b) q[b] = Q::fragment(lds + P::kBytes, kk, (wm * MT + b) * 16, 4, lane);
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int b = 0; b < MT; ++b) acc[a][b] = mma<T>(p[a], q[b], acc[a][b]);
            if constexpr (SUMS) {
                constexpr uint32_t w = one_bits<T>();
                const u32x4 one = {w, w, w, w};
#pragma unroll
                for (int b = 0; b < MT; ++b) ones[b] = mma<T>(one, q[b], ones[b]);
            }
        }
    }

    // acc = sum over k in [0, K). `p` points at (n = 0, k = 0) of the tile,
    // `rows_n` rows of it exist; `q` likewise with m.
    template <bool VEC, bool SUMS>
    __device__ __forceinline__ void run(char* lds, const T* p, int64_t ldp, int rows_n, const T* q, int64_t ldq, int rows_m,
                                        int K, int tid, bool sums) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int b = 0; b < MT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (SUMS)
#pragma unroll
            for (int b = 0; b < MT; ++b) ones[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (K <= 0) return;
        P::template stage<VEC>(lds, p, ldp, rows_n, 0, K, tid);
        Q::template stage<VEC>(lds + P::kBytes, q, ldq, rows_m, 0, K, tid);
        staged_barrier();
        int cur = 0;
        for (int k0 = 0; k0 < K; k0 += BK) {
            if (k0 + BK < K) {
                char* next = lds + (cur ^ 1) * kStage;
                P::template stage<VEC>(next, p, ldp, rows_n, k0 + BK, K, tid);
                Q::template stage<VEC>(next + P::kBytes, q, ldq, rows_m, k0 + BK, K, tid);
            }
            if (SUMS && sums) multiply<true && SUMS>(lds + cur * kStage, tid);
            else multiply<false>(lds + cur * kStage, tid);
            staged_barrier();
            cur ^= 1;
        }
    }
};

}  // namespace dmr

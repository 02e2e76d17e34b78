// Norms of gradients over many tensors, and clipping, on gfx950: with v the
// values of all tensors that belong to group g,
//     n_g = sqrt(sum v^2),   out = v min(1, max_norm / (n_g + eps)).
//
// Squares are added in float64: no value of any type overflows or vanishes,
// and the sum's error is far below the output's rounding whatever the number
// of values. The order of every sum follows from the sizes alone.
#include "dmr_internal.h"

namespace dmr {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // at whatever alignment the values have

constexpr int kThreads = 256;

// What a launch is given: the tensors (values of one group each) and, of
// every group, the first chunk of each tensor.
struct Span {
    const void* in;
    void* out;
    int64_t values;
    int32_t first, dtype;
};
struct Spans {
    Span at[kClipTensors];
    int32_t count, chunks;
};

template <class T>
constexpr int kVector = 16 / (int)sizeof(T);

// Sum over a workgroup, the same in every thread; `part` holds one value a wave.
template <int WAVES>
__device__ __forceinline__ double workgroup_sum(double v, double* part) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += part[w];
    __syncthreads();
    return s;
}

template <class T>
__device__ __forceinline__ double squares_of(u32x4 raw) {
    T v[kVector<T>];
    __builtin_memcpy(v, &raw, 16);
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < kVector<T>; ++e) {
        const double d = (double)(float)v[e];
        s = __builtin_fma(d, d, s);
    }
    return s;
}

// Sum of squares of `n` values by the threads of a workgroup, each its share.
template <class T, int THREADS>
__device__ __forceinline__ double squares(const T* __restrict__ in, int64_t n) {
    const int64_t whole = n / kVector<T>;
    double s = 0.0;
    int64_t i = threadIdx.x;
    for (; i + 3 * THREADS < whole; i += 4 * THREADS) {
        u32x4 raw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) __builtin_memcpy(&raw[u], in + (i + u * THREADS) * kVector<T>, 16);
#pragma unroll
        for (int u = 0; u < 4; ++u) s += squares_of<T>(raw[u]);
    }
    for (; i < whole; i += THREADS) {
        u32x4 raw;
        __builtin_memcpy(&raw, in + i * kVector<T>, 16);
        s += squares_of<T>(raw);
    }
    const int64_t last = whole * kVector<T> + threadIdx.x;
    if (last < n) {
        const double d = (double)(float)in[last];
        s = __builtin_fma(d, d, s);
    }
    return s;
}

// A factor, by 2^exponent: float32 has not the digits of those below its
// normal values, but their products with large values have.
struct Factor {
    float c;
    int exponent;
    __device__ __forceinline__ float operator*(float v) const { return __builtin_ldexpf(v * c, exponent); }
};

// out = in c; the two may be the same array. STREAM: the stores leave the
// caches to what is still to be read.
template <class T, int THREADS, bool STREAM>
__device__ __forceinline__ void scale(const T* in, T* out, int64_t n, Factor c) {
    const int64_t whole = n / kVector<T>;
    const auto put = [&](u32x4 raw, int64_t i) {
        T v[kVector<T>];
        __builtin_memcpy(v, &raw, 16);
#pragma unroll
        for (int e = 0; e < kVector<T>; ++e) v[e] = (T)(c * (float)v[e]);
        if constexpr (STREAM) {
            u32x4_any to;
            __builtin_memcpy(&to, v, 16);
            __builtin_nontemporal_store(to, reinterpret_cast<u32x4_any*>(out + i * kVector<T>));
        } else {
            __builtin_memcpy(out + i * kVector<T>, v, 16);
        }
    };
    int64_t i = threadIdx.x;
    for (; i + 3 * THREADS < whole; i += 4 * THREADS) {
        u32x4 raw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) __builtin_memcpy(&raw[u], in + (i + u * THREADS) * kVector<T>, 16);
#pragma unroll
        for (int u = 0; u < 4; ++u) put(raw[u], i + u * THREADS);
    }
    for (; i < whole; i += THREADS) {
        u32x4 raw;
        __builtin_memcpy(&raw, in + i * kVector<T>, 16);
        put(raw, i);
    }
    const int64_t last = whole * kVector<T> + threadIdx.x;
    if (last < n) out[last] = (T)(c * (float)in[last]);
}

// min(1, max_norm / (norm + eps)); NaN for a norm that is one, and 1 where
// there is nothing to scale (zero by zero).
__device__ __forceinline__ Factor factor(double norm, float max_norm, float eps) {
    const double by = norm + (double)eps;
    if (by == 0.0) return {1.0f, 0};
    double q = (double)max_norm / by;
    if (q >= 1.0) return {1.0f, 0};
    int exponent = 0;
    if (q < 0x1p-126) q = __builtin_frexp(q, &exponent);
    return {(float)q, exponent};
}

template <class F>
__device__ __forceinline__ void typed(int dtype, F&& f) {
    if (dtype == DMR_FLOAT32) f(float{});
    else if (dtype == DMR_FLOAT16) f(_Float16{});
    else f(__bf16{});
}

// Where the values of a workgroup are: its group, its chunk of the launch and
// that chunk's tensor, first value and length.
struct Chunk {
    int64_t group, first, values;
    int32_t index, tensor;
};
__device__ __forceinline__ Chunk find_chunk(const Spans& s, uint32_t id, int64_t length) {
    Chunk c;
    c.group = id / (uint32_t)s.chunks;
    c.index = (int)(id % (uint32_t)s.chunks);
    int lo = 0, hi = s.count;   // the last tensor whose first chunk is not past this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s.at[mid].first <= c.index) lo = mid;
        else hi = mid;
    }
    c.tensor = lo;
    c.first = (int64_t)(c.index - s.at[lo].first) * length;
    const int64_t left = s.at[lo].values - c.first;
    c.values = left < length ? left : length;
    return c;
}

// Every chunk's sum of squares: partial [groups][all chunks of a group].
__global__ __launch_bounds__(kThreads) void clip_squares(const Spans s, int64_t length, int32_t before, int32_t all,
                                                         double* __restrict__ partial) {
    __shared__ double part[kThreads / 64];
    const Chunk c = find_chunk(s, blockIdx.x, length);
    const Span& t = s.at[c.tensor];
    const int64_t at = c.group * t.values + c.first;
    double sum = 0.0;
    typed(t.dtype, [&](auto zero) {
        typedef decltype(zero) T;
        sum = squares<T, kThreads>(static_cast<const T*>(t.in) + at, c.values);
    });
    sum = workgroup_sum<kThreads / 64>(sum, part);
    if (threadIdx.x == 0) partial[c.group * all + before + c.index] = sum;
}

// Scales every chunk by its group's factor, the last chunks first: they were
// read last, and what the caches still hold of them is read from there.
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void clip_scale(const Spans s, int64_t length, int32_t before, int32_t all,
                                                       const double* __restrict__ partial, float max_norm, float eps,
                                                       float* __restrict__ norms) {
    __shared__ double part[kThreads / 64];
    const Chunk c = find_chunk(s, gridDim.x - 1 - blockIdx.x, length);
    double sum = 0.0;
    for (int i = threadIdx.x; i < all; i += kThreads) sum += partial[c.group * all + i];
    const double norm = sqrt(workgroup_sum<kThreads / 64>(sum, part));
    if (before == 0 && c.index == 0 && threadIdx.x == 0) norms[c.group] = (float)norm;
    const Factor by = factor(norm, max_norm, eps);
    const Span& t = s.at[c.tensor];
    const int64_t at = c.group * t.values + c.first;
    typed(t.dtype, [&](auto zero) {
        typedef decltype(zero) T;
        scale<T, kThreads, STREAM>(static_cast<const T*>(t.in) + at, static_cast<T*>(t.out) + at, c.values, by);
    });
}

// Small groups: a workgroup for each does both.
constexpr int kSmallThreads = 1024;
__global__ __launch_bounds__(kSmallThreads) void clip_small(const Spans s, float max_norm, float eps,
                                                            float* __restrict__ norms) {
    __shared__ double part[kSmallThreads / 64];
    const int64_t group = blockIdx.x;
    double sum = 0.0;
    for (int k = 0; k < s.count; ++k) {
        const Span& t = s.at[k];
        typed(t.dtype, [&](auto zero) {
            typedef decltype(zero) T;
            sum += squares<T, kSmallThreads>(static_cast<const T*>(t.in) + group * t.values, t.values);
        });
    }
    const double norm = sqrt(workgroup_sum<kSmallThreads / 64>(sum, part));
    if (threadIdx.x == 0) norms[group] = (float)norm;
    const Factor by = factor(norm, max_norm, eps);
    for (int k = 0; k < s.count; ++k) {
        const Span& t = s.at[k];
        typed(t.dtype, [&](auto zero) {
            typedef decltype(zero) T;
            scale<T, kSmallThreads, false>(static_cast<const T*>(t.in) + group * t.values,
                                           static_cast<T*>(t.out) + group * t.values, t.values, by);
        });
    }
}

}  // namespace

// Chunks are cut so that about 16 workgroups for each compute unit share all
// values, and none below 8192 values, which take as long to start as to read.
// More bytes than half of the last cache level are written past the caches,
// which then hold more of the input when it is read again (402 MB of bfloat16:
// 224 us with ordinary stores, 204 so; no difference up to 25 MB). A pass over
// them reads at 6.4 TB/s, with squares in float32 as in float64.
ClipPlan clip_plan(const dmr_tensor_span* tensors, int32_t count, int64_t groups) {
    ClipPlan p{};
    double all = 0.0, slice = 0.0, bytes = 0.0;
    int32_t used = 0;
    for (int32_t k = 0; k < count; ++k) {
        slice += (double)tensors[k].values;
        bytes += (double)tensors[k].values * (tensors[k].dtype == DMR_FLOAT32 ? 4.0 : 2.0) * (double)groups;
        used += tensors[k].values > 0;
    }
    all = slice * (double)groups;
    p.stream = bytes > (double)(1 << 27);
    p.small = used <= kClipTensors && slice <= 65536.0;
    double length = all / 4096.0;
    length = length < 8192.0 ? 8192.0 : length;
    if (all > 1e18) return p;   // fits: false
    p.length = ((int64_t)length + 2047) / 2048 * 2048;
    int64_t chunks = 0;
    for (int32_t k = 0; k < count; ++k) chunks += (tensors[k].values + p.length - 1) / p.length;
    p.chunks = chunks;
    const int64_t most = kMaxWorkItems / kSmallThreads;
    p.fits = p.small ? groups <= most : chunks <= most / (groups > 0 ? groups : 1);
    return p;
}

hipError_t launch_clip(const ClipArgs& a, const ClipPlan& p) {
    timing_begin(kKClipNorm, a.stream);
    hipError_t err = hipSuccess;
    // every tensor that has values, kClipTensors to a launch
    const auto batches = [&](auto&& launch) {
        int32_t k = 0;
        int64_t before = 0;
        while (k < a.count && err == hipSuccess) {
            Spans s{};
            for (; k < a.count && s.count < kClipTensors; ++k) {
                const dmr_tensor_span& t = a.tensors[k];
                if (t.values == 0) continue;
                s.at[s.count++] = {t.in, t.out, t.values, s.chunks, (int32_t)t.dtype};
                s.chunks += p.small ? 0 : (int32_t)((t.values + p.length - 1) / p.length);
            }
            if (s.count > 0) {
                launch(s, (int32_t)before);
                err = hipGetLastError();
            }
            before += s.chunks;
        }
    };
    if (p.small) {
        Spans s{};
        for (int32_t k = 0; k < a.count; ++k)
            if (a.tensors[k].values > 0)
                s.at[s.count++] = {a.tensors[k].in, a.tensors[k].out, a.tensors[k].values, 0, (int32_t)a.tensors[k].dtype};
        clip_small<<<(unsigned)a.groups, kSmallThreads, 0, a.stream>>>(s, a.max_norm, a.eps, a.norms);
        err = hipGetLastError();
    } else {
        const int32_t all = (int32_t)p.chunks;
        batches([&](const Spans& s, int32_t before) {
            clip_squares<<<(unsigned)(a.groups * s.chunks), kThreads, 0, a.stream>>>(s, p.length, before, all, a.workspace);
        });
        batches([&](const Spans& s, int32_t before) {
            const auto kernel = p.stream ? clip_scale<true> : clip_scale<false>;
            kernel<<<(unsigned)(a.groups * s.chunks), kThreads, 0, a.stream>>>(s, p.length, before, all, a.workspace, a.max_norm,
                                                                               a.eps, a.norms);
        });
    }
    timing_end(kKClipNorm, a.stream);
    return err;
}

}  // namespace dmr

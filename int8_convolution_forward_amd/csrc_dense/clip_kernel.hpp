// The norm of many tensors together, and their scaling by it: two passes over the
// values, bound by HBM.
//
// A launch takes a table of tensors as its argument; its workgroups walk over
// chunks of up to kClipChunk values, numbered through all the table's tensors.  Squares are
// summed in 64 bits, so that no finite value's square overflows or vanishes and the
// sum is exact to about 2^-53 a term; the vector unit has more of that than HBM can
// feed.  Workgroups leave a partial sum each, and every workgroup of the second
// pass adds all of them in the same order: no atomics, and nothing between the
// launches.  Gradients within the limit that stay where they are end the second
// pass there.
//
// 268 million BF16 values in 48 tensors: squares 121 us (537 MB, 4.4 TB/s: reads
// alone), scaling into other memory 183 (1074 MB, 5.9 TB/s); six tensors of 530 000
// FP32 values in all 3.5 and 3.2 us, two launches.  Chunks of one size would leave most
// CUs without one there.
#pragma once

#include "dense_common.hpp"

namespace dense {

constexpr int kClipTensors = 128, kClipThreads = 256;
constexpr int kClipStep = kClipThreads * 8, kClipChunk = 8 * kClipStep;  // values: of a workgroup's load, the most of a chunk
constexpr int kClipWgs = 1024;     // of a launch, at most

struct ClipTable {
    const void *in[kClipTensors];
    void *out[kClipTensors];
    int64_t n[kClipTensors];
    unsigned first[kClipTensors + 1];  // number of a tensor's first chunk; the last: of all
    uint8_t dt[kClipTensors];
    int count;
    int chunk;                         // values: kClipChunk, or less where that would leave CUs without one
};

__device__ __forceinline__ double wave_sum64(double v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o, 64);
    return v;
}

// The sum over the workgroup's threads, in all of them
__device__ __forceinline__ double group_sum64(double v, double *red)
{
    v = wave_sum64(v);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// f(tensor, first value) for each of the workgroup's chunks, in order.  Tensors of no values have no chunks.
template <typename F>
__device__ __forceinline__ void clip_walk(const ClipTable &t, F f)
{
    int i = 0;
    for (unsigned b = blockIdx.x; b < t.first[t.count]; b += gridDim.x) {
        while (b >= t.first[i + 1])
            ++i;
        f(i, (int64_t)(b - t.first[i]) * t.chunk);
    }
}

// The loads of a whole chunk, or of a quarter of its values in 32 bits, go out together, as they lie in memory.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int64_t at, int64_t end)
{
    constexpr int U = 16 / sizeof(T), STEP = kClipStep;
    double s[2] = {0.0, 0.0};
    auto add = [&](const float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s[k & 1] = __builtin_fma((double)v[k], (double)v[k], s[k & 1]);
    };
    int64_t c = at + threadIdx.x * 8;
    for (; c + (U - 1) * STEP + 8 <= end; c += U * STEP) {
        Raw8<T> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            r[u] = __builtin_bit_cast(Raw8<T>, *(const Pack<T, 8> *)(p + c + u * STEP));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen(r[u], v);
            add(v);
        }
    }
    for (; c < end; c += STEP) {
        float v[8];
        load_n(p + c, (int)(end - c), v);
        add(v);
    }
    return s[0] + s[1];
}

__global__ __launch_bounds__(kClipThreads) void clip_squares_kernel(const ClipTable t, double *part)
{
    __shared__ double red[4];
    double s = 0.0;
    clip_walk(t, [&](int i, int64_t at) {
        if (t.dt[i] == DENSE_BF16)
            s += chunk_squares((const bf16 *)t.in[i], at, min(t.n[i], at + t.chunk));
        else if (t.dt[i] == DENSE_FP16)
            s += chunk_squares((const f16 *)t.in[i], at, min(t.n[i], at + t.chunk));
        else
            s += chunk_squares((const float *)t.in[i], at, min(t.n[i], at + t.chunk));
    });
    s = group_sum64(s, red);
    if (threadIdx.x == 0)
        part[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *q, int64_t at, int64_t end, double factor)
{
    constexpr int U = 4;
    // The product is that of 64 bits, rounded to 32 and from there to the type.  A 16-bit value's comes from the
    // factor in two parts, (hi + lo) 2^e: with one of 32 bits, itself off by up to 2^-24, values next to the middle of
    // two 16-bit numbers went to the other side.  (In 64 bits it is the same numbers, by more registers: 268 million
    // BF16 values in 327 us a call, 309 so.)
    const double part = __builtin_amdgcn_frexp_mant(factor);  // at least 1/2, also where the factor is below 2^-126
    const int e = __builtin_amdgcn_frexp_exp(factor);
    const float hi = (float)part, lo = (float)(part - (double)hi);
    auto scale = [&](float v) {
        if constexpr (sizeof(T) == 4)
            return (float)((double)v * factor);
        else  // a factor of 1 takes any value, infinities too
            return __builtin_amdgcn_ldexpf(__builtin_fmaf(v, hi, factor < 1.0 ? v * lo : 0.0f), e);
    };
    int64_t c = at + threadIdx.x * 8;
    for (; c + (U - 1) * kClipThreads * 8 + 8 <= end; c += U * kClipThreads * 8) {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_all(p + c + u * kClipThreads * 8, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[u][k] = scale(v[u][k]);
            store_all(q + c + u * kClipThreads * 8, v[u]);
        }
    }
    for (; c < end; c += kClipThreads * 8) {
        float v[8];
        load_n(p + c, (int)(end - c), v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = scale(v[k]);
        store_n(q + c, (int)(end - c), v);
    }
}

// parts: the partial sums of all launches of the first pass
__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(const ClipTable t, const double *part, int parts,
                                                                  double max_norm, float *norm)
{
    __shared__ double red[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads)
        s += part[i];
    const double size = sqrt(group_sum64(s, red));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = (float)size;
    // a norm that is not finite in 64 bits (an element is not) changes nothing, nor does one within the limit
    const bool clips = size > max_norm && size < INFINITY;
    const double factor = clips ? max_norm / size : 1.0;
    clip_walk(t, [&](int i, int64_t at) {
        if (!clips && t.in[i] == t.out[i])
            return;
        if (t.dt[i] == DENSE_BF16)
            chunk_scale((const bf16 *)t.in[i], (bf16 *)t.out[i], at, min(t.n[i], at + t.chunk), factor);
        else if (t.dt[i] == DENSE_FP16)
            chunk_scale((const f16 *)t.in[i], (f16 *)t.out[i], at, min(t.n[i], at + t.chunk), factor);
        else
            chunk_scale((const float *)t.in[i], (float *)t.out[i], at, min(t.n[i], at + t.chunk), factor);
    });
}

}  // namespace dense

// C entry of the clipping of gradients by their norm: argument checks, launches.
#include <algorithm>
#include <new>
#include <stdlib.h>
#include <string.h>

#include "clip_kernel.hpp"
#include "host_common.hpp"

namespace dense {
namespace {

constexpr int64_t kWsAlign = 256;
// Chunks of a launch are numbered in 32 bits.
constexpr int64_t kMaxChunks = (int64_t)1 << 31;

struct Span {
    uintptr_t from, to;
    bool written;
};

// Memory that is written has to be of one vector alone.
conv_i8_status_t check_overlap(const dense_clip_grads_t &a)
{
    Span *spans = new (std::nothrow) Span[2 * (size_t)a.count + 1];
    if (!spans)
        return CONV_I8_ERR_SCRATCH;
    int64_t count = 1;
    spans[0] = {(uintptr_t)a.norm, (uintptr_t)a.norm + sizeof(float), true};
    for (int64_t i = 0; i < a.count; ++i) {
        const int64_t bytes = a.in[i].n * size_of(a.in[i].dtype);
        if (bytes == 0)
            continue;
        const uintptr_t in = (uintptr_t)a.in[i].ptr, out = (uintptr_t)a.out[i].ptr;
        spans[count++] = {out, out + bytes, true};
        if (in != out)
            spans[count++] = {in, in + bytes, false};
    }
    std::sort(spans, spans + count, [](const Span &x, const Span &y) { return x.from < y.from; });
    bool clash = false;
    uintptr_t end = 0, written = 0;  // ends of what came before, and of what is written of it
    for (int64_t i = 0; i < count; ++i) {
        clash |= spans[i].from < written || (spans[i].written && spans[i].from < end);
        end = std::max(end, spans[i].to);
        if (spans[i].written)
            written = std::max(written, spans[i].to);
    }
    delete[] spans;
    return clash ? CONV_I8_ERR_PARAM : CONV_I8_OK;
}

conv_i8_status_t analyze(const dense_clip_grads_t *a)
{
    if (!a)
        return CONV_I8_ERR_NULL;
    if (a->count < 0 || a->count > kMaxDim)
        return CONV_I8_ERR_DIMS;
    if ((a->count > 0 && (!a->in || !a->out)) || !a->norm)
        return CONV_I8_ERR_NULL;
    if ((uintptr_t)a->norm % 4 || !(a->max_norm >= 0.0))
        return CONV_I8_ERR_PARAM;
    for (int64_t i = 0; i < a->count; ++i) {
        dense_vec_t in = a->in[i], out = a->out[i];
        if (in.dtype == DENSE_NONE || out.dtype != in.dtype)
            return CONV_I8_ERR_DTYPE;
        if (in.n < 0 || in.n > ((int64_t)1 << 40))
            return CONV_I8_ERR_DIMS;
        if (out.n != in.n)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(check_vec(&in, in.n));
        DENSE_TRY(check_vec(&out, in.n));
    }
    return check_overlap(*a);
}

int64_t launches(const dense_clip_grads_t &a) { return a.count > 0 ? ceil_div(a.count, kClipTensors) : 1; }

// Tensors of launch l; returns its chunks.
int64_t table(const dense_clip_grads_t &a, int64_t l, ClipTable *t)
{
    memset(t, 0, sizeof *t);
    const int64_t from = l * kClipTensors;
    t->count = (int)std::min<int64_t>(a.count - from, kClipTensors);
    int64_t total = 0, chunks = 0;
    for (int i = 0; i < t->count; ++i)
        total += std::min(a.in[from + i].n, (int64_t)kClipWgs * kClipChunk);
    t->chunk = (int)std::min<int64_t>(kClipChunk, std::max<int64_t>(1, ceil_div(total, (int64_t)kClipWgs * kClipStep)) * kClipStep);
    for (int i = 0; i < t->count; ++i) {
        t->in[i] = a.in[from + i].ptr;
        t->out[i] = const_cast<void *>(a.out[from + i].ptr);
        t->n[i] = a.in[from + i].n;
        t->dt[i] = (uint8_t)a.in[from + i].dtype;
        t->first[i] = (unsigned)chunks;
        chunks += ceil_div(t->n[i], t->chunk);
        if (chunks >= kMaxChunks)
            return chunks;
    }
    t->first[t->count] = (unsigned)chunks;
    return chunks;
}

}  // namespace
}  // namespace dense

using namespace dense;

extern "C" {

conv_i8_status_t dense_clip_grads_workspace_size(const dense_clip_grads_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    DENSE_TRY(analyze(args));
    *bytes = (size_t)round_up(launches(*args) * kClipWgs * 8, kWsAlign);
    return CONV_I8_OK;
}

conv_i8_status_t dense_clip_grads(const dense_clip_grads_t *args, void *workspace, size_t bytes, void *stream)
{
    DENSE_TRY(analyze(args));
    const int64_t count = launches(*args);
    if (bytes < (size_t)round_up(count * kClipWgs * 8, kWsAlign) || ((uintptr_t)workspace & (kWsAlign - 1)) != 0)
        return CONV_I8_ERR_WORKSPACE;
    if (!workspace)
        return CONV_I8_ERR_NULL;
    ClipTable t;
    for (int64_t l = 0; l < count; ++l)
        if (table(*args, l, &t) >= kMaxChunks)
            return CONV_I8_ERR_UNSUPPORTED;
    double *part = (double *)workspace;
    hipStream_t s = (hipStream_t)stream;
    // every launch of the first pass leaves as many sums as it has workgroups, one at least
    auto wgs = [](int64_t chunks) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(chunks, kClipWgs)); };
    int parts = 0;
    for (int64_t l = 0; l < count; ++l) {
        const unsigned n = wgs(table(*args, l, &t));
        hipLaunchKernelGGL(clip_squares_kernel, dim3(n), dim3(kClipThreads), 0, s, t, part + parts);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
        parts += (int)n;
    }
    for (int64_t l = 0; l < count; ++l) {
        const unsigned n = wgs(table(*args, l, &t));
        hipLaunchKernelGGL(clip_scale_kernel, dim3(n), dim3(kClipThreads), 0, s, t, part, parts, args->max_norm,
                           l == 0 ? args->norm : nullptr);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    return CONV_I8_OK;
}

}  // extern "C"

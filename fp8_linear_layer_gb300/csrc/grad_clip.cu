// grad_clip.cu -- global L2 norm over many gradient tensors, and clipping.
//
//   norm = sqrt(sum_t sum_i g_t[i]^2)
//   out_t[i] = g_t[i] * min(1, max_norm / (norm + 1e-6))
//
// The tensors are cut into chunks of kChunk elements, numbered through all
// tensors of a launch; the table of tensors travels in the kernel's parameters,
// so a call copies nothing to the device.  Pass 1: each CTA sums the squares of
// its chunks in fp32 and leaves one partial.  Pass 2: every CTA adds the
// partials (in the same fixed order everywhere), forms the factor and
// scales its chunks, last chunk first: pass 1 reads the last kClipKeepBytes
// normally and everything before them as evict-first, so that pass 2 finds them
// in L2.  Bound by HBM, which sees most gradients twice: 470 MB of fp32 into other
// buffers 213 us, 0.65 of the floor of one read and one write and 0.92 of the
// copy rate for the 1.33 GB that move.
// Squares are taken in fp32: a gradient beyond 1.8e19 makes the norm infinite.
#include <cuda_runtime.h>

#include "common.cuh"
#include "grad_clip.h"
#include "launch.cuh"

namespace fp8ll {
namespace {

constexpr int kThreadsClip = 256;
constexpr int kSmallTable = 64;   // 2 KB of parameters: the usual call
constexpr int kLargeTable = kClipTensorsPerLaunch;

struct Entry {
    const void* g;
    void* out;
    int64_t n;
    int32_t chunk0;  // number of the tensor's first chunk
    int32_t bf16;
};

template <int CAP>
struct Table {
    int32_t count, chunks;
    int32_t keep_from;  // first chunk whose lines pass 1 leaves in L2 for pass 2
    Entry e[CAP];
};

template <int CAP>
__device__ __forceinline__ int find_entry(const Table<CAP>& t, int chunk) {
    int lo = 0, hi = t.count - 1;  // the last entry whose first chunk is not behind `chunk`
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].chunk0 <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
                : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store1(void* p, int64_t i, int bf16, float v) {
    if (bf16)
        static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    else
        static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ float square_sum(const uint4& w, int bf16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const float a = bf16_lo(u[i]), b = bf16_hi(u[i]);
            s = fmaf(a, a, s);
            s = fmaf(b, b, s);
        } else {
            const float a = __uint_as_float(u[i]);
            s = fmaf(a, a, s);
        }
    }
    return s;
}

__device__ __forceinline__ uint4 scaled(const uint4& w, int bf16, float f) {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = bf16 ? pack_bf16x2(bf16_lo(u[i]) * f, bf16_hi(u[i]) * f) : __float_as_uint(__uint_as_float(u[i]) * f);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// elements from `p + i` up to the next 16-byte boundary, at most n
__device__ __forceinline__ int head_of(const void* p, int bf16, int n) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
    const int h = off == 0 ? 0 : (16 - off) >> (bf16 ? 1 : 2);
    return h < n ? h : n;
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsClip) grad_norm_kernel(const __grid_constant__ Table<CAP> t,
                                                                 float* partials) {
    await_dependency();
    release_dependents();
    __shared__ float part[kThreadsClip / 32];
    float s = 0.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry& e = t.e[find_entry(t, c)];
        const int64_t i0 = static_cast<int64_t>(c - e.chunk0) * kClipChunk;
        const int n = static_cast<int>(e.n - i0 < kClipChunk ? e.n - i0 : kClipChunk);
        const int bf16 = e.bf16;
        const char* g = static_cast<const char*>(e.g) + (bf16 ? 2 : 4) * i0;
        const int per = bf16 ? 8 : 4;
        const int head = head_of(g, bf16, n);
        const int vecs = (n - head) / per;
        const uint4* v = reinterpret_cast<const uint4*>(g + head * (bf16 ? 2 : 4));
        const bool keep = c >= t.keep_from;
        auto load = [&](int j) { return keep ? v[j] : __ldcs(v + j); };
        int i = threadIdx.x;
        for (; i + 3 * kThreadsClip < vecs; i += 4 * kThreadsClip) {
            const uint4 a = load(i), b = load(i + kThreadsClip), d = load(i + 2 * kThreadsClip),
                        f = load(i + 3 * kThreadsClip);
            s += (square_sum(a, bf16) + square_sum(b, bf16)) + (square_sum(d, bf16) + square_sum(f, bf16));
        }
        for (; i < vecs; i += kThreadsClip) s += square_sum(v[i], bf16);
        // the elements before the first and behind the last whole vector
        const int tail = head + vecs * per;
        if (threadIdx.x < head) {
            const float a = load1(g, threadIdx.x, bf16);
            s = fmaf(a, a, s);
        }
        if (tail + static_cast<int>(threadIdx.x) < n) {
            const float a = load1(g, tail + threadIdx.x, bf16);
            s = fmaf(a, a, s);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float total = part[0];
#pragma unroll
        for (int w = 1; w < kThreadsClip / 32; ++w) total += part[w];
        partials[blockIdx.x] = total;
    }
}

// sqrt of the sum of all partials, on every thread, the same bits in every CTA.
// In fp32: the sum is a tree of a few additions per thread and thirteen levels.
// (In fp64 every CTA paid for it at this part's fp64 rate: clipping 67 MB took
// 36.5 us instead of 29.0.)
__device__ __forceinline__ float total_norm(const float* partials, int count) {
    __shared__ float part[kThreadsClip / 32];
    float s = 0.0f;
    for (int i = threadIdx.x; i < count; i += kThreadsClip) s += __ldcg(partials + i);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    float total = part[0];
#pragma unroll
    for (int w = 1; w < kThreadsClip / 32; ++w) total += part[w];
    return sqrtf(total);
}

__global__ void __launch_bounds__(kThreadsClip) grad_norm_finalize_kernel(const float* partials,
                                                                          int count, float* norm) {
    await_dependency();
    const float v = total_norm(partials, count);
    if (threadIdx.x == 0) *norm = v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreadsClip) grad_scale_kernel(const __grid_constant__ Table<CAP> t,
                                                                  const float* partials, int count,
                                                                  float max_norm, float* norm) {
    await_dependency();
    const float v = total_norm(partials, count);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    const float q = __fdiv_rn(max_norm, v + 1e-6f);
    const float f = q > 1.0f ? 1.0f : q;  // a NaN norm stays visible in the gradients
    for (int k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const int c = t.chunks - 1 - k;
        const Entry& e = t.e[find_entry(t, c)];
        if (f == 1.0f && e.out == e.g) continue;  // in place and unchanged
        const int64_t i0 = static_cast<int64_t>(c - e.chunk0) * kClipChunk;
        const int n = static_cast<int>(e.n - i0 < kClipChunk ? e.n - i0 : kClipChunk);
        const int bf16 = e.bf16, size = bf16 ? 2 : 4;
        const char* g = static_cast<const char*>(e.g) + size * i0;
        char* o = static_cast<char*>(e.out) + size * i0;
        if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15u) != 0) {
            // input and output out of step: no vector is aligned in both
            for (int i = threadIdx.x; i < n; i += kThreadsClip) store1(o, i, bf16, load1(g, i, bf16) * f);
            continue;
        }
        const int per = bf16 ? 8 : 4;
        const int head = head_of(g, bf16, n);
        const int vecs = (n - head) / per;
        const uint4* gv = reinterpret_cast<const uint4*>(g + head * size);
        uint4* ov = reinterpret_cast<uint4*>(o + head * size);
        int i = threadIdx.x;
        for (; i + 3 * kThreadsClip < vecs; i += 4 * kThreadsClip) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __ldcs(gv + i + j * kThreadsClip);
#pragma unroll
            for (int j = 0; j < 4; ++j) __stcs(ov + i + j * kThreadsClip, scaled(w[j], bf16, f));
        }
        for (; i < vecs; i += kThreadsClip) ov[i] = scaled(gv[i], bf16, f);
        const int tail = head + vecs * per;
        if (threadIdx.x < head) store1(o, threadIdx.x, bf16, load1(g, threadIdx.x, bf16) * f);
        if (tail + static_cast<int>(threadIdx.x) < n)
            store1(o, tail + threadIdx.x, bf16, load1(g, tail + threadIdx.x, bf16) * f);
    }
}

// tensors first .. of the list that fit one launch; returns the next one
template <int CAP>
int64_t fill(Table<CAP>& t, int64_t count, const fp8ll_grad_t* grads, int64_t first) {
    t.count = 0;
    t.chunks = 0;
    int64_t i = first;
    for (; i < count && t.count < CAP; ++i) {
        if (grads[i].n == 0) continue;
        const int64_t chunks = (grads[i].n + kClipChunk - 1) / kClipChunk;
        t.e[t.count++] = Entry{grads[i].grad, grads[i].out, grads[i].n, t.chunks, grads[i].dtype == FP8LL_BF16};
        t.chunks += static_cast<int32_t>(chunks);
    }
    int64_t bytes = 0;
    t.keep_from = t.chunks;
    for (int k = t.count - 1; k >= 0 && bytes < kClipKeepBytes; --k) {
        const int64_t chunk = static_cast<int64_t>(kClipChunk) * (t.e[k].bf16 ? 2 : 4);
        const int64_t have = t.keep_from - t.e[k].chunk0, room = (kClipKeepBytes - bytes + chunk - 1) / chunk;
        const int64_t take = have < room ? have : room;
        t.keep_from -= static_cast<int32_t>(take);
        bytes += take * chunk;
    }
    return i;
}

int grid_of(int chunks, int num_sms) {
    int g = 8 * num_sms;
    if (g > kClipMaxBlocks) g = kClipMaxBlocks;
    return chunks < g ? chunks : g;
}

template <int CAP>
int run(int64_t count, const fp8ll_grad_t* grads, int scale, float max_norm, float* norm, float* partials,
        cudaStream_t stream, int num_sms) {
    Table<CAP> t;
    int used = 0, launches = 0;
    int held = -1;  // the launch whose tensors t holds
    int64_t starts[kClipMaxTensors / kClipTensorsPerLaunch + 1];
    for (int64_t i = 0; i < count;) {
        const int64_t first = i;
        i = fill(t, count, grads, first);
        held = -1;
        if (t.count == 0) break;  // only empty tensors were left
        held = launches;
        starts[launches++] = first;
        const int g = grid_of(t.chunks, num_sms);
        if (launch_dependent(grad_norm_kernel<CAP>, static_cast<unsigned>(g), kThreadsClip, 0, stream, t,
                             partials + used) != cudaSuccess)
            return -3;
        used += g;
    }
    if (!scale || used == 0) {
        return launch_dependent(grad_norm_finalize_kernel, 1, kThreadsClip, 0, stream, partials, used, norm) ==
                       cudaSuccess
                   ? 0
                   : -3;
    }
    // the launches of pass 1 in reverse order: the last tensors are the ones in L2
    for (int k = launches - 1; k >= 0; --k) {
        if (k != held) fill(t, count, grads, starts[k]);
        if (launch_dependent(grad_scale_kernel<CAP>, static_cast<unsigned>(grid_of(t.chunks, num_sms)), kThreadsClip, 0,
                             stream, t, partials, used, max_norm, k == launches - 1 ? norm : nullptr) != cudaSuccess)
            return -3;
    }
    return 0;
}

}  // namespace

int launch_grad_norm(int64_t count, const fp8ll_grad_t* grads, int scale, float max_norm, float* norm,
                     float* partials, cudaStream_t stream, int num_sms) {
    return count <= kSmallTable
               ? run<kSmallTable>(count, grads, scale, max_norm, norm, partials, stream, num_sms)
               : run<kLargeTable>(count, grads, scale, max_norm, norm, partials, stream, num_sms);
}

}  // namespace fp8ll

// dropout.cu -- dropout whose mask is never stored, added to a residual stream.
//
//   out[i] = residual[i] + (w_i < p 2^32 ? 0 : x[i] / (1 - p))
//
// w_i is word i % 4 of the counter-based generator Philox4x32-10 (Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): key = the
// seed, counter = (i / 4, site, step), i the element's place in the matrix by
// rows, whatever its strides.  So the backward pass draws the same mask again
// from the same numbers: it is this kernel on the gradient.
//
// A word has 32 bits, so an element is dropped with the probability
// floor(p 2^32) / 2^32, and the ten rounds are paid once for four elements.
// Scaling and addition are one fused multiply-add, rounded to bf16 once.
//
// Bound by HBM: 8192 x 4096 with residual 33.1 us, 0.91 of the measured copy rate
// (a mask in memory would cost a byte or a bit an element twice more).  Each thread
// has four 16-byte vectors of both inputs in flight, or one where there are too few
// to give every SM as many: the generator's chain of twenty products per group is
// hidden by other threads.  CTAs are not persistent; in large matrices without gaps each
// asks for the inputs of the CTA half as many behind it as run at once, in L2 (34.1 us
// without; 16384 x 7168 108.7, with it 102.8; as far behind as run at once 34.3, twice as
// far 37.1).  129 x 1001 takes 1.9 us.  Rows with gaps take the same vectors where
// addresses and rows are multiples of 16 bytes; anything else goes element by element.
#include <cuda_runtime.h>

#include "common.cuh"
#include "dropout.h"
#include "l2_prefetch.cuh"
#include "launch.cuh"

namespace fp8ll {
namespace {

__device__ __forceinline__ uint4 philox(uint32_t group, const DropoutParams& p, uint64_t step) {
    uint4 c = make_uint4(group, p.site, static_cast<uint32_t>(step), static_cast<uint32_t>(step >> 32));
    uint32_t k0 = p.key0, k1 = p.key1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c.x, b = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
        c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                       static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

__device__ __forceinline__ uint64_t step_of(const DropoutParams& p) {
    return p.step + (p.step_dev ? static_cast<uint64_t>(*p.step_dev) : 0ull);
}

// a dropped element leaves the residual as it is, whatever x holds there
__device__ __forceinline__ float kept(float x, float res, uint32_t word, const DropoutParams& p) {
    return word >= p.threshold ? fmaf(x, p.scale, res) : res;
}

__device__ __forceinline__ uint32_t kept2(uint32_t x, uint32_t res, uint32_t w0, uint32_t w1, const DropoutParams& p) {
    return pack_bf16x2(kept(bf16_lo(x), bf16_lo(res), w0, p), kept(bf16_hi(x), bf16_hi(res), w1, p));
}

// Elements 4 g .. 4 g + 3 one by one, those below n: any sizes, strides and alignment.
__device__ __forceinline__ void drop_group(const DropoutParams& p, uint64_t step, int64_t g, int64_t n) {
    const uint4 w = philox(static_cast<uint32_t>(g), p, step);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
    int64_t r = 4 * g / p.cols, c = 4 * g - r * p.cols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = 4 * g + j;
        if (i >= n) return;
        const float x = __uint_as_float(static_cast<uint32_t>(p.x[r * p.ldx + c]) << 16);
        const float res = p.res ? __uint_as_float(static_cast<uint32_t>(p.res[r * p.ldr + c]) << 16) : 0.0f;
        p.out[i] = static_cast<uint16_t>(pack_bf16x2(kept(x, res, word[j], p), 0.0f));
        if (++c == p.cols) {
            c = 0;
            ++r;
        }
    }
}

constexpr int kThreads = 256;

// U vectors of eight elements a thread, all loaded before the first is used.
// FLAT: the matrices have no gaps between their rows and count as one row, whose
// last elements beyond the vectors go one by one.
template <int U, bool FLAT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p) {
    await_dependency();
    release_dependents();
    const uint64_t step = step_of(p);
    const int64_t n = p.rows * p.cols, vectors = n / 8;
    const uint32_t per_row = static_cast<uint32_t>(p.cols / 8);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * U) + threadIdx.x;
    if (FLAT && U > 1 && threadIdx.x == 0) {
        const int64_t later = (blockIdx.x + p.ahead) * (kThreads * U);
        if (later + kThreads * U <= vectors) {
            prefetch_l2_rows(p.x + 8 * later, 16 * kThreads * U);
            if (p.res) prefetch_l2_rows(p.res + 8 * later, 16 * kThreads * U);
        }
    }
    uint4 x[U], res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t v = first + u * kThreads;
        if (v >= vectors) continue;
        int64_t ox = 8 * v, orr = 8 * v;
        if (!FLAT) {
            const uint32_t r = static_cast<uint32_t>(v) / per_row;
            const int64_t c = 8 * static_cast<int64_t>(static_cast<uint32_t>(v) - r * per_row);  // from 2^32 on in wide rows
            ox = r * p.ldx + c;
            orr = r * p.ldr + c;
        }
        x[u] = __ldcs(reinterpret_cast<const uint4*>(p.x + ox));
        res[u] = p.res ? __ldcs(reinterpret_cast<const uint4*>(p.res + orr)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t v = first + u * kThreads;
        if (v >= vectors) continue;
        const uint4 a = philox(static_cast<uint32_t>(2 * v), p, step);
        const uint4 b = philox(static_cast<uint32_t>(2 * v + 1), p, step);
        __stcs(reinterpret_cast<uint4*>(p.out + 8 * v),
               make_uint4(kept2(x[u].x, res[u].x, a.x, a.y, p), kept2(x[u].y, res[u].y, a.z, a.w, p),
                          kept2(x[u].z, res[u].z, b.x, b.y, p), kept2(x[u].w, res[u].w, b.z, b.w, p)));
    }
    if (FLAT && blockIdx.x == 0 && threadIdx.x < 2 && 8 * vectors + 4 * threadIdx.x < n)
        drop_group(p, step, 2 * vectors + threadIdx.x, n);
}

__global__ void __launch_bounds__(kThreads) dropout_any_kernel(const __grid_constant__ DropoutParams p) {
    await_dependency();
    release_dependents();
    const uint64_t step = step_of(p);
    const int64_t n = p.rows * p.cols, g = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (4 * g < n) drop_group(p, step, g, n);
}

bool vectors_fit(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

int launch_dropout(const DropoutParams& given, cudaStream_t stream, int num_sms) {
    DropoutParams p = given;
    p.ahead = 2 * static_cast<int64_t>(num_sms);
    const int64_t n = p.rows * p.cols;
    const bool flat = p.rows == 1 || (p.ldx == p.cols && (!p.res || p.ldr == p.cols));
    if (flat) {
        p.rows = 1;
        p.cols = p.ldx = p.ldr = n;
    }
    const bool aligned = vectors_fit(p.x) && vectors_fit(p.out) && vectors_fit(p.res);
    const bool rows = p.cols % 8 == 0 && p.ldx % 8 == 0 && p.ldr % 8 == 0;
    auto blocks = [](int64_t units, int64_t per) { return static_cast<unsigned>((units + per - 1) / per); };
    cudaError_t rc;
    if (!aligned || !(flat || rows)) {
        rc = launch_dependent(dropout_any_kernel, blocks((n + 3) / 4, kThreads), kThreads, 0, stream, p);
    } else {
        const int64_t vectors = n < 8 ? 1 : n / 8;
        if (vectors >= static_cast<int64_t>(num_sms) * kThreads * 16)
            rc = flat ? launch_dependent(dropout_kernel<4, true>, blocks(vectors, 4 * kThreads), kThreads, 0, stream, p)
                      : launch_dependent(dropout_kernel<4, false>, blocks(vectors, 4 * kThreads), kThreads, 0, stream, p);
        else
            rc = flat ? launch_dependent(dropout_kernel<1, true>, blocks(vectors, kThreads), kThreads, 0, stream, p)
                      : launch_dependent(dropout_kernel<1, false>, blocks(vectors, kThreads), kThreads, 0, stream, p);
    }
    return rc == cudaSuccess ? 0 : -3;
}

}  // namespace fp8ll

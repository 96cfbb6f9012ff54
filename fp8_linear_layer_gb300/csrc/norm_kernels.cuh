// norm_kernels.cuh -- the kernels of the root-mean-square norm and of the layer
// norm (CENTER), with the residual's addition and an fp8 output, and of their
// backward passes.  What each computes, and what its launches are measured at,
// stands in rmsnorm.cu and layernorm.cu.
//
// Rows kernel: one row per CTA at a time, T threads with V 16-byte vectors of
// the row each, held as packed bf16 between the sums and the cast; the next row is
// loaded meanwhile, or each row has a CTA of its own (row_alone).  16 neighbouring threads hold one 128-block, so block and MX
// maxima are shuffles, and a lane divides for one of its blocks only.
// Columns kernel: reads h again, while half of it is in L2, and casts it down its
// columns.  (A cluster of CTAs per 128-row band, which formed h and then cast its
// tiles from L2, took 98 us for both at 8192 x 4096: each CTA's chain of loads was
// too long for the CTAs that fit.)
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "l2_prefetch.cuh"
#include "launch.cuh"
#include "mx_rule.cuh"
#include "norm.h"

namespace fp8ll {
namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// The sum of v over the block's threads, on every thread, added in a fixed
// order.  `part` holds one slot per warp; consecutive calls alternate between
// two of them, so that one barrier per call is enough.
__device__ __forceinline__ float block_sum(float v, float* part) {
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

// Two sums at once, each as block_sum makes it.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* part) {
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        v.x = __fadd_rn(v.x, __shfl_xor_sync(0xffffffffu, v.x, off));
        v.y = __fadd_rn(v.y, __shfl_xor_sync(0xffffffffu, v.y, off));
    }
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        s.x = __fadd_rn(s.x, __shfl_xor_sync(0xffffffffu, s.x, off));
        s.y = __fadd_rn(s.y, __shfl_xor_sync(0xffffffffu, s.y, off));
    }
    return s;
}

// y = fl(fl(h rstd) gamma) of eight packed bf16 values, as four pairs
__device__ __forceinline__ void norm8(const uint4& h, const uint4& g, uint64_t rstd2, uint64_t (&y)[4]) {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = mul_f32x2(mul_f32x2(pack_f32x2(bf16_lo(hw[i]), bf16_hi(hw[i])), rstd2),
                         pack_f32x2(bf16_lo(gw[i]), bf16_hi(gw[i])));
}

// y = fma(fl(fl(h - mean) rstd), gamma, beta) likewise
__device__ __forceinline__ void center8(const uint4& h, const uint4& g, const uint4& b, uint64_t minus_mean2,
                                        uint64_t rstd2, uint64_t (&y)[4]) {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = fma_f32x2(
            mul_f32x2(add_f32x2(pack_f32x2(bf16_lo(hw[i]), bf16_hi(hw[i])), minus_mean2), rstd2),
            pack_f32x2(bf16_lo(gw[i]), bf16_hi(gw[i])), pack_f32x2(bf16_lo(bw[i]), bf16_hi(bw[i])));
}

__device__ __forceinline__ float amax8(const uint64_t (&y)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_f32x2(y[i]);
        m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    return m;
}

template <int FMT>
__device__ __forceinline__ uint2 encode8_pairs(const uint64_t (&y)[4], float inv) {
    const uint64_t inv2 = pack_f32x2(inv, inv);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_f32x2(mul_f32x2(y[i], inv2));
        w[i] = Fp8Fmt<FMT>::cvt2(v.x, v.y);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__global__ void zero_word_kernel(float* word) {
    await_dependency();
    release_dependents();
    *word = 0.0f;
}

// max|y| over the block into *amax_out, one atomic per block: non-negative
// floats order like their bits, and a maximum does not depend on the order.  A
// single block stores it; otherwise the word was zeroed before.  LOOK: only where the
// word is smaller yet (a block per row: thousands of atomics in one place are slow).
template <bool LOOK>
__device__ __forceinline__ void fold_amax(float top, float* part, float* amax_out) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    __syncthreads();  // part's last use as sums is over
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, part[w]);
        unsigned* word = reinterpret_cast<unsigned*>(amax_out);
        if (gridDim.x == 1)
            *amax_out = top;
        else if (!LOOK || __float_as_uint(top) > *reinterpret_cast<volatile unsigned*>(word))
            atomicMax(word, __float_as_uint(top));
    }
}

// GREG: gamma (CENTER, V = 1: and beta) stays in registers for all rows of the CTA.
// PRE: the next row is loaded while the current one is reduced and cast (else, where a
// CTA has another one at all, behind it).  MINB: CTAs of MAXT threads that the
// registers leave room for (0: no matter).
template <bool CENTER, int FMT, int RECIPE, int V, int MAXT, bool GREG, bool PRE, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_rows_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[2][32];
    await_dependency();
    // the columns kernel and kernels behind a short one come in early; behind a long
    // one they only get in the way (32768 x 1024 in MXFP8: 54.6 us, else 41.4)
    if (p.qc || p.rows < 2048) release_dependents();
    const int nv = static_cast<int>(p.cols / 8);
    const int T = blockDim.x;
    const int lane = threadIdx.x & 31;
    const int64_t mx_groups = 2 * ((p.rows + 255) / 256);
    float inv_t = 1.0f, s_t = 1.0f, top = 0.0f;
    auto tensor_scale = [&] {
        block_scale<FMT>(*p.amax_in, inv_t, s_t);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s_t;
    };
    if (RECIPE == kRecipeTensor && !CENTER) tensor_scale();
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 xv[V], rv[V];  // the next row, loaded while the current one is reduced and cast
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            const bool in = i < nv && r < p.rows;
            xv[v] = in ? __ldcs(reinterpret_cast<const uint4*>(p.x + r * p.ldx + 8 * i)) : zero;
            rv[v] = in && p.residual ? __ldcs(reinterpret_cast<const uint4*>(p.residual + r * p.ldr + 8 * i)) : zero;
        }
    };
    auto load_weight = [&](const uint16_t* w, int v) {
        const int i = threadIdx.x + v * T;
        return i < nv ? *reinterpret_cast<const uint4*>(w + 8 * i) : zero;
    };
    auto load_beta = [&](int v) { return p.beta ? load_weight(p.beta, v) : zero; };
    int64_t r = blockIdx.x;
    fetch(r);
    if (!PRE && threadIdx.x == 0) {  // row_alone: L2 has the row when its CTA starts
        const int64_t later = r + p.ahead;
        if (p.ahead > 0 && later < p.rows) {
            const uint32_t bytes = static_cast<uint32_t>(2 * p.cols);
            prefetch_l2_rows(p.x + later * p.ldx, bytes);
            if (p.residual) prefetch_l2_rows(p.residual + later * p.ldr, bytes);
        }
    }
    if (RECIPE == kRecipeTensor && CENTER) tensor_scale();  // the row is on its way meanwhile
    constexpr bool BREG = GREG && CENTER && V == 1;
    uint4 gv[GREG ? V : 1], bv[BREG ? V : 1];
    if (GREG) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            gv[v] = load_weight(p.gamma, v);
            if (BREG) bv[BREG ? v : 0] = load_beta(v);
        }
    }
    for (int k = 0; r < p.rows; r += gridDim.x, ++k) {
        uint4 hv[V];
        float sq = 0.0f, mean = 0.0f;
        uint64_t sum2 = 0ull;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            hv[v] = xv[v];
            float f[8];
            unpack8(hv[v], f);
            if (p.residual) {
                float b[8];
                unpack8(rv[v], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += b[e];
                hv[v] = pack8(f);
                unpack8(hv[v], f);
            }
            if (p.h && i < nv) *reinterpret_cast<uint4*>(p.h + r * p.cols + 8 * i) = hv[v];
            if (CENTER) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sum2 = add_f32x2(pack_f32x2(f[2 * e], f[2 * e + 1]), sum2);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
            }
        }
        if (PRE) fetch(r + gridDim.x);
        if (CENTER) {
            const float2 s = unpack_f32x2(sum2);
            mean = __fdiv_rn(block_sum(s.x + s.y, part[0]), static_cast<float>(p.cols));
            if (threadIdx.x == 0) p.mean[r] = mean;
            const uint64_t minus_mean2 = pack_f32x2(-mean, -mean);
            sum2 = 0ull;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (threadIdx.x + v * T >= nv) continue;
                const uint32_t w[4] = {hv[v].x, hv[v].y, hv[v].z, hv[v].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t c = add_f32x2(pack_f32x2(bf16_lo(w[e]), bf16_hi(w[e])), minus_mean2);
                    sum2 = fma_f32x2(c, c, sum2);
                }
            }
            const float2 q = unpack_f32x2(sum2);
            sq = q.x + q.y;
        }
        sq = block_sum(sq, part[CENTER ? 1 : k & 1]);
        // correctly rounded: an ulp here moves every code of the row that lies near a tie
        const float ms = __fdiv_rn(sq, static_cast<float>(p.cols)) + p.eps;
        // a row of zeros without eps stays zeros, here and in the backward pass (a NaN is none)
        const float rstd = ms == 0.0f ? 0.0f : __frsqrt_rn(ms);
        if (threadIdx.x == 0) p.rstd[r] = rstd;
        const uint64_t rstd2 = pack_f32x2(rstd, rstd);
        uint64_t y[V][4];
        float amax[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint4 g = GREG ? gv[GREG ? v : 0] : load_weight(p.gamma, v);
            if (CENTER)
                center8(hv[v], g, BREG ? bv[BREG ? v : 0] : load_beta(v), pack_f32x2(-mean, -mean), rstd2, y[v]);
            else
                norm8(hv[v], g, rstd2, y[v]);
            amax[v] = amax8(y[v]);  // 0 beyond the row
            if (RECIPE == kRecipeTensor) top = fmaxf(top, amax[v]);
        }
        if (p.y) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = threadIdx.x + v * T;
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack_f32x2(y[v][e]);
                    w[e] = pack_bf16x2(f.x, f.y);
                }
                if (i < nv) *reinterpret_cast<uint4*>(p.y + r * p.cols + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (!p.qr) {
            if (!PRE) fetch(r + gridDim.x);
            continue;
        }
        float inv[V];
        if (RECIPE == kRecipeTensor) {
#pragma unroll
            for (int v = 0; v < V; ++v) inv[v] = inv_t;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                amax[v] = fmaxf(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], 1));
                amax[v] = fmaxf(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], 2));
            }
        }
        if (RECIPE == kRecipeMx) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = threadIdx.x + v * T;
                const int e = mx_exponent<FMT>(amax[v]);
                inv[v] = mx_inverse_scale(e);
                if (CENTER) {
                    // the four bytes of a 128-block stand side by side: one store of its first lane
                    uint32_t b = static_cast<uint32_t>(e + 127) << (8 * ((lane >> 2) & 3));
                    b |= __shfl_xor_sync(0xffffffffu, b, 4);
                    b |= __shfl_xor_sync(0xffffffffu, b, 8);
                    if (i < nv && (i & 15) == 0)
                        *reinterpret_cast<uint32_t*>(p.sfr + mx_sf_offset(i >> 4, mx_groups, r, 0)) = b;
                } else if (i < nv && (i & 3) == 0) {
                    p.sfr[mx_sf_offset(i >> 4, mx_groups, r, (i >> 2) & 3)] = static_cast<uint8_t>(e + 127);
                }
            }
        }
        if (RECIPE == kRecipeBlock) {
            // lane j of a 16-lane group divides for vector j % V only, and hands the factor to the others
            float mine = amax[0];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                amax[v] = fmaxf(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], 4));
                amax[v] = fmaxf(amax[v], __shfl_xor_sync(0xffffffffu, amax[v], 8));
                if (v == 0 || (lane & (V - 1)) == v) mine = amax[v];
            }
            float inv_mine, s_mine;
            block_scale<FMT>(mine, inv_mine, s_mine);
            const int vm = lane & (V - 1);
            const int im = threadIdx.x + vm * T;
            if ((lane & 15) < V && im < nv) p.sr[(im >> 4) * p.sldr + r] = s_mine;
#pragma unroll
            for (int v = 0; v < V; ++v) inv[v] = __shfl_sync(0xffffffffu, inv_mine, (lane & 16) + v);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            if (i < nv) __stcs(reinterpret_cast<uint2*>(p.qr + r * p.cols + 8 * i), encode8_pairs<FMT>(y[v], inv[v]));
        }
        if (!PRE) fetch(r + gridDim.x);
    }
    if (RECIPE == kRecipeMx && p.qr) {
        // the scale bytes of rows beyond the matrix hold 127
        for (r = p.rows + blockIdx.x; r < mx_groups * 128; r += gridDim.x)
            for (int64_t i = threadIdx.x; i < p.cols / 128; i += T)
                *reinterpret_cast<uint32_t*>(p.sfr + mx_sf_offset(i, mx_groups, r, 0)) = 0x7F7F7F7Fu;
    }
    if (RECIPE == kRecipeTensor && p.amax_out) fold_amax<!PRE>(top, part[0], p.amax_out);
}

// Column codes of y from h, rstd and gamma, in 128 x 128 tiles of h staged in
// shared memory as the transposed casts do it (each 32-row band rotated by eight
// words): persistent CTAs with two staged tiles, the next one on its way by
// cp.async while one is cast.  Thread t takes the column pair t / 4 and the
// 32-row part t % 4.  |y| = fl(fl(|h| rstd) |gamma|) grows with fl(|h| rstd), so
// a column's maximum needs one product per element and gamma once.  CENTER: y is a
// monotone function of xhat = fl(fl(h - mean) rstd) along a column, so |y| is
// largest at its smallest or its largest xhat.

// CTAs per SM: shared memory has room for three, in which the layer norm's registers
// spill (8192 x 4096, rows and columns, three / two: 63.6 / 61.1 us on 1x128, 69.2 /
// 67.9 in MXFP8, 58.7 / 57.9 per tensor)
template <bool CENTER>
constexpr int cols_ctas() {
    return CENTER ? 2 : 3;
}
struct ColsStage {
    uint32_t tile[128][64];
    float rstd[4][36];  // part p's 32 rows, banks apart
    float mean[4][36];  // CENTER
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool CENTER, int FMT, int RECIPE>
__global__ void __launch_bounds__(256, cols_ctas<CENTER>()) norm_cols_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ __align__(16) uint8_t stage_raw[];
    await_dependency();
    ColsStage* stage = reinterpret_cast<ColsStage*>(stage_raw);
    const uint16_t* h = p.h ? p.h : p.x;
    const int64_t ldh = p.h ? p.cols : p.ldx;
    const int64_t ncb = p.cols / 128, ntiles = (p.rows / 128) * ncb;
    float inv_t = 1.0f, s_t = 1.0f;
    if (RECIPE == kRecipeTensor) block_scale<FMT>(*p.amax_in, inv_t, s_t);
    auto fetch = [&](int64_t t, int buf) {
        const int64_t rb = t / ncb, r0 = rb * 128, c0 = (t - rb * ncb) * 128;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int i = threadIdx.x + it * 256;
            const int rr = i >> 4, ch = i & 15;
            cp_async16(smem_addr(&stage[buf].tile[rr][(ch * 4 + 8 * (rr >> 5)) & 63]), h + (r0 + rr) * ldh + c0 + ch * 8);
        }
        if (threadIdx.x < 128)
            cp_async4(smem_addr(&stage[buf].rstd[threadIdx.x >> 5][threadIdx.x & 31]), p.rstd + r0 + threadIdx.x);
        else if (CENTER)
            cp_async4(smem_addr(&stage[buf].mean[(threadIdx.x >> 5) & 3][threadIdx.x & 31]), p.mean + r0 + (threadIdx.x & 127));
    };
    const int cp = threadIdx.x >> 2, part = threadIdx.x & 3;
    const int wcol = (cp + 8 * part) & 63;
    int64_t t = blockIdx.x;
    if (t < ntiles) fetch(t, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int k = 0; t < ntiles; ++k, t += gridDim.x) {
        const ColsStage& st = stage[k & 1];
        __syncthreads();  // every thread is done with the tile that the next one replaces
        if (t + gridDim.x < ntiles) fetch(t + gridDim.x, (k + 1) & 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const int64_t rb = t / ncb, r0 = rb * 128, c0 = (t - rb * ncb) * 128;
        const int64_t c = c0 + 2 * cp;
        const uint32_t gw = *reinterpret_cast<const uint32_t*>(p.gamma + c);
        const float g_lo = bf16_lo(gw), g_hi = bf16_hi(gw);
        const uint32_t bw = CENTER && p.beta ? *reinterpret_cast<const uint32_t*>(p.beta + c) : 0u;
        const float b_lo = bf16_lo(bw), b_hi = bf16_hi(bw);
        // the thread's i-th pair, scaled (and centred)
        auto xhat = [&](int i) {
            const uint32_t w = st.tile[32 * part + i][wcol];
            const float s = st.rstd[part][i];
            uint64_t v = pack_f32x2(bf16_lo(w), bf16_hi(w));
            if (CENTER) {
                const float m = -st.mean[part][i];
                v = add_f32x2(v, pack_f32x2(m, m));
            }
            return mul_f32x2(v, pack_f32x2(s, s));
        };
        float inv_lo = inv_t, inv_hi = inv_t, s_lo, s_hi;
        if (RECIPE != kRecipeTensor) {
            float a_lo = 0.0f, a_hi = 0.0f;
            if (CENTER) {
                // starting from NaN, which a maximum and a minimum pass over; where all values are NaN, so is the result
                const float none = __int_as_float(0x7FC00000);
                float2 top = make_float2(none, none), low = top;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 v = unpack_f32x2(xhat(i));
                    top = make_float2(fmaxf(top.x, v.x), fmaxf(top.y, v.y));
                    low = make_float2(fminf(low.x, v.x), fminf(low.y, v.y));
                }
                a_lo = fmaxf(fmaxf(fabsf(fmaf(top.x, g_lo, b_lo)), fabsf(fmaf(low.x, g_lo, b_lo))), 0.0f);
                a_hi = fmaxf(fmaxf(fabsf(fmaf(top.y, g_hi, b_hi)), fabsf(fmaf(low.y, g_hi, b_hi))), 0.0f);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 v = unpack_f32x2(xhat(i));
                    a_lo = fmaxf(a_lo, fabsf(v.x));
                    a_hi = fmaxf(a_hi, fabsf(v.y));
                }
                // a maximum over NaN (gamma NaN, or infinite over zeros) is 0, as of the values one by one
                a_lo = fmaxf(__fmul_rn(a_lo, fabsf(g_lo)), 0.0f);
                a_hi = fmaxf(__fmul_rn(a_hi, fabsf(g_hi)), 0.0f);
            }
            if (RECIPE == kRecipeBlock) {
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) {
                    a_lo = fmaxf(a_lo, __shfl_xor_sync(0xffffffffu, a_lo, off));
                    a_hi = fmaxf(a_hi, __shfl_xor_sync(0xffffffffu, a_hi, off));
                }
                // even parts divide for the even column, odd parts for the odd one
                float inv_mine, s_mine;
                block_scale<FMT>(part & 1 ? a_hi : a_lo, inv_mine, s_mine);
                const float other = __shfl_xor_sync(0xffffffffu, inv_mine, 1);
                inv_lo = part & 1 ? other : inv_mine;
                inv_hi = part & 1 ? inv_mine : other;
                if (part < 2) p.sc[rb * p.sldc + c + part] = s_mine;
            } else {
                const int e_lo = mx_exponent<FMT>(a_lo), e_hi = mx_exponent<FMT>(a_hi);
                inv_lo = mx_inverse_scale(e_lo);
                inv_hi = mx_inverse_scale(e_hi);
                const int64_t groups = 2 * ((p.cols + 255) / 256);
                p.sfc[mx_sf_offset(rb, groups, c, part)] = static_cast<uint8_t>(e_lo + 127);
                p.sfc[mx_sf_offset(rb, groups, c + 1, part)] = static_cast<uint8_t>(e_hi + 127);
                // an odd number of 128-column groups: the group beyond the matrix holds 127
                if (c0 + 128 == p.cols && (p.cols & 255) != 0 && threadIdx.x < 128)
                    *reinterpret_cast<uint32_t*>(p.sfc + mx_sf_offset(rb, groups, p.cols + threadIdx.x, 0)) =
                        0x7F7F7F7Fu;
            }
        }
        const uint64_t g2 = pack_f32x2(g_lo, g_hi), inv2 = pack_f32x2(inv_lo, inv_hi);
        const uint64_t b2 = pack_f32x2(b_lo, b_hi);
        uint32_t wl[8], wh[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t x = xhat(4 * i + j);
                v[j] = unpack_f32x2(mul_f32x2(CENTER ? fma_f32x2(x, g2, b2) : mul_f32x2(x, g2), inv2));
            }
            wl[i] = Fp8Fmt<FMT>::cvt2(v[0].x, v[1].x) | (static_cast<uint32_t>(Fp8Fmt<FMT>::cvt2(v[2].x, v[3].x)) << 16);
            wh[i] = Fp8Fmt<FMT>::cvt2(v[0].y, v[1].y) | (static_cast<uint32_t>(Fp8Fmt<FMT>::cvt2(v[2].y, v[3].y)) << 16);
        }
        uint4* dl = reinterpret_cast<uint4*>(p.qc + c * p.rows + r0 + 32 * part);
        uint4* dh = reinterpret_cast<uint4*>(p.qc + (c + 1) * p.rows + r0 + 32 * part);
        __stcs(dl, make_uint4(wl[0], wl[1], wl[2], wl[3]));
        __stcs(dl + 1, make_uint4(wl[4], wl[5], wl[6], wl[7]));
        __stcs(dh, make_uint4(wh[0], wh[1], wh[2], wh[3]));
        __stcs(dh + 1, make_uint4(wh[4], wh[5], wh[6], wh[7]));
    }
}

template <bool CENTER, int FMT, int RECIPE>
int launch_cols(const NormParams& p, cudaStream_t stream, int num_sms) {
    auto kern = norm_cols_kernel<CENTER, FMT, RECIPE>;
    static PerDevice allowed;
    if (allow_shared_memory(allowed, kern, 2 * sizeof(ColsStage)) != 0) return -3;
    const int64_t tiles = p.rows / 128 * (p.cols / 128), cap = static_cast<int64_t>(num_sms) * cols_ctas<CENTER>();
    return launch_dependent(kern, static_cast<unsigned>(tiles < cap ? tiles : cap), 256, 2 * sizeof(ColsStage), stream,
                            p) == cudaSuccess
               ? 0
               : -3;
}

// threads and vectors per thread of a row of nv 16-byte vectors
constexpr int64_t kOneVectorCols = 1024, kTwoVectorCols = 4096;  // most columns with so many
void row_shape(int64_t cols, int& T, int& V) {
    const int64_t nv = cols / 8;
    V = cols <= kOneVectorCols ? 1 : cols <= kTwoVectorCols ? 2 : 4;
    T = static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32);
}

// The layer norm: whether each row has a CTA of its own, of four vectors a thread,
// without a row loaded ahead.  Its 62 to 64 registers let 1024 threads run on an SM
// where the next row's would leave 512, and other rows' CTAs hide what a row waits
// for (its loads, two sums).  us, this / persistent CTAs with the next row ahead
// (rows x cols, with residual; 1x128 | MXFP8 | per tensor; later rows asked for in L2
// by this one, as below, in all its figures):
//   4096 x 8192  41.9 / 55.2 | 46.1 / 61.8 | 42.8 / 54.6
//   777 x 7168   10.5 / 13.3 | 11.8 / 16.0 | 11.9 / 14.2
// where those have two vectors a thread or one, and 768 or more threads on an SM:
//   8192 x 4096  40.5 / 43.9 | 45.1 / 47.5 | 41.5 / 41.1
//   2000 x 4096  13.6 / 14.0 | 14.6 / 15.1 | 14.3 / 12.4
//   400 x 4096    4.3 /  4.1 |  5.8 /  4.6 |  5.6 /  4.7
//   8192 x 2048  23.6 / 23.5 | 25.8 / 25.2 | 24.3 / 22.9
//   777 x 2048    4.3 /  4.3 |  4.9 /  4.7 |  5.9 /  4.6
//   16384 x 1024 23.2 / 24.4 | 24.7 / 27.1 | 23.5 / 23.9
//   2000 x 1024   4.4 /  5.2 |  4.9 /  6.2 |  6.7 /  5.5
// So 1x128 takes it for all of these and per tensor for none.  MXFP8 up to 4096
// columns could go either way: a CTA per row gains 3 to 20% in four of them and
// loses 2 to 25% in three, and the rule is for the short call of wide rows (400 x
// 4096).  The number of rows may not decide: the two forms add a row's sums in
// different orders, and a row's result is to be the same in any batch.
//
// From 128 threads a row on, a CTA asks for the inputs of a later row in L2: the one
// half as many CTAs behind it as run at once, and above 16384 columns, where one CTA
// fits an SM, as many as run at once.  1x128: 16384 x 7168 141 us without, 134 with
// it, 8192 x 4096 41.5 and 40.6 (as far behind as run at once: 135 and 42.2, twice as
// far 140; 8192 x 2048 23.1 either way); 2048 x 24576 83 without, 76.2 with it, half
// as far 75.3, and 4096 x 16512 132, 120.0 and 119.9.
constexpr bool row_alone(int64_t cols, int recipe) {
    return cols > (recipe == kRecipeBlock ? 512 : kTwoVectorCols);
}

template <bool CENTER, int FMT, int RECIPE>
int launch_norm(const NormParams& given, cudaStream_t stream, int num_sms) {
    NormParams p = given;
    int T, V;
    row_shape(p.cols, T, V);
    const bool alone = CENTER && row_alone(p.cols, RECIPE);
    if (alone) {
        V = 4;
        T = static_cast<int>(((p.cols / 8 + V - 1) / V + 31) / 32 * 32);
        p.ahead = T < 128 ? 0 : static_cast<int64_t>(num_sms) * (T > 512 ? 1 : 512 / T);
    }
    // 768 (1024) threads of rows per SM; from 4224 columns on the RMS norm's 118 to 121
    // registers let only 512 run at once (at 7168 columns two CTAs of 224 threads, three
    // launched): the rest start where the first ones end
    int64_t grid = RECIPE == kRecipeMx ? (p.rows + 255) / 256 * 256 : p.rows;
    const int64_t cap = static_cast<int64_t>(num_sms) * ((V == 1 ? 1024 : 768) / T < 1 ? 1 : (V == 1 ? 1024 : 768) / T);
    const int64_t grid_rows = grid;
    if (grid > cap) grid = cap;
    const unsigned g = static_cast<unsigned>(grid);
    // a kernel of one thread: a memset node cost 4 us here
    if (RECIPE == kRecipeTensor && p.amax_out && g > 1 &&
        launch_dependent(zero_word_kernel, 1, 1, 0, stream, p.amax_out) != cudaSuccess)
        return -3;
    cudaError_t rc;
    if constexpr (CENTER) {
        if (alone) {
            const unsigned all = static_cast<unsigned>(grid_rows);
            rc = T <= 512 ? launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 4, 512, false, false, 2>, all, T, 0, stream, p)
                          : launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 4, 1024, false, false, 1>, all, T, 0, stream, p);
        } else if (V == 1) {
            rc = launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 1, 128, true, true, 0>, g, T, 0, stream, p);
        } else if constexpr (!row_alone(kOneVectorCols + 1, RECIPE)) {
            static_assert(row_alone(kTwoVectorCols + 1, RECIPE), "wider rows have a CTA of their own");
            rc = launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 2, 256, true, true, 3>, g, T, 0, stream, p);
        } else {
            return -3;  // not reached: the rule above gives every such row a CTA of its own
        }
    } else {
        switch (V) {
            case 1: rc = launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 1, 128, true, true, 0>, g, T, 0, stream, p); break;
            case 2: rc = launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 2, 256, true, true, 0>, g, T, 0, stream, p); break;
            default:
                rc = T <= 512 ? launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 4, 512, true, true, 0>, g, T, 0, stream, p)
                              : launch_dependent(norm_rows_kernel<CENTER, FMT, RECIPE, 4, 1024, false, true, 0>, g, T, 0, stream, p);
        }
    }
    if (rc != cudaSuccess) return -3;
    return p.qc ? launch_cols<CENTER, FMT, RECIPE>(p, stream, num_sms) : 0;
}

// ---------------------------------------------------------------- backward
//
//   d = dy gamma, xhat = h rstd, m = mean_c (d xhat)
//   dx = rstd (d - xhat m) + dres        dgamma_c = sum_r dy xhat
// and CENTER, with xhat = (h - mean) rstd and m0 = mean_c d:
//   dx = rstd (d - m0 - xhat m) + dres   dbeta_c = sum_r dy
//
// Bound by HBM: 16384 x 7168 with the residual's gradient 159 us (CENTER: 169), 0.87
// (0.83) of the copy rate; the RMS norm's 0.49 at 32768 columns, where a thread holds
// eight vectors and loads nothing ahead.
// T threads walk rows together; a thread keeps the same columns for all of
// them, so dgamma is summed in its registers (SMEM: in shared memory, where a
// row is too wide for them) and written once per CTA as a band of partial sums,
// which the finalize adds in a fixed order.  PRE: the next row's dy and h are
// loaded while the current row is reduced.  LANES: a warp or half a warp per
// row, 256 / LANES rows per CTA, whose sums meet in shared memory at the end
// (0: the whole CTA per row).  Products in packed pairs, each rounded as a
// scalar one would be.
__device__ __forceinline__ void unpack_pairs(const uint4& w, uint64_t (&f)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pack_f32x2(bf16_lo(u[e]), bf16_hi(u[e]));
}

template <bool CENTER, int V, int MAXT, bool SMEM, bool PRE, int LANES, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_grad_kernel(const __grid_constant__ NormGradParams p) {
    static_assert(LANES == 0 || !SMEM, "a warp's sums stay in registers");
    constexpr bool WARP = LANES != 0;
    constexpr int kRowsPerCta = WARP ? 256 / (WARP ? LANES : 1) : 1;
    constexpr int S = CENTER ? 2 : 1;  // sums per column: dgamma, dbeta
    __shared__ float part[2][32];
    __shared__ float2 part2[2][CENTER ? 32 : 1];
    extern __shared__ __align__(16) float acc_smem[];  // SMEM: [S][cols], LANES: [kRowsPerCta][cols]
    await_dependency();
    release_dependents();
    const int nv = static_cast<int>(p.cols / 8);
    const int T = WARP ? LANES : blockDim.x;
    const int tid = WARP ? threadIdx.x % (WARP ? LANES : 1) : threadIdx.x;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint64_t acc[S][SMEM ? 1 : V][4];
    if (SMEM) {
        for (int i = tid; i < S * nv; i += T) {
            reinterpret_cast<uint4*>(acc_smem)[2 * i] = zero;
            reinterpret_cast<uint4*>(acc_smem)[2 * i + 1] = zero;
        }
        if (CENTER) __syncthreads();  // a thread's sums of dbeta may lie where another one wrote zeros
    } else {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[s][SMEM ? 0 : v][e] = 0ull;
    }
    uint4 dn[PRE ? V : 1], hn[PRE ? V : 1];  // the next row
    auto load = [&](const uint16_t* base, int64_t ld, int64_t r, int v) {
        const int i = tid + v * T;
        return i < nv && r < p.rows ? __ldcs(reinterpret_cast<const uint4*>(base + r * ld + 8 * i)) : zero;
    };
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dn[PRE ? v : 0] = load(p.dy, p.lddy, r, v);
            hn[PRE ? v : 0] = load(p.h, p.ldh, r, v);
        }
    };
    auto gamma = [&](int v) {
        const int i = tid + v * T;
        return i < nv ? *reinterpret_cast<const uint4*>(p.gamma + 8 * i) : zero;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsPerCta;
    const int own = WARP ? static_cast<int>(threadIdx.x) / (WARP ? LANES : 1) : 0;  // the row within the CTA
    int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + own;
    // CENTER: the next row's statistics (a load in front of each row is what its chain would begin with)
    float rstd_next = 0.0f, mean_next = 0.0f;
    auto statistics = [&](int64_t row) {
        rstd_next = row < p.rows ? p.rstd[row] : 0.0f;
        mean_next = row < p.rows ? p.mean[row] : 0.0f;
    };
    if (CENTER) statistics(r);
    const int second = LANES == 16 ? own & 1 : 0;  // the halves of a warp leave the loop together
    if (PRE) fetch(r);
    for (int k = 0; r - second < p.rows; r += step, ++k) {
        uint4 dv[V], hv[V], sv[V];
        const float rstd = CENTER ? rstd_next : r < p.rows ? p.rstd[r] : 0.0f;
        const uint64_t rstd2 = pack_f32x2(rstd, rstd);
        const float minus_mean = CENTER ? -mean_next : 0.0f;
        if (CENTER) statistics(r + step);
        const uint64_t minus_mean2 = pack_f32x2(minus_mean, minus_mean);
        uint64_t dot2 = 0ull, sum2 = 0ull;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dv[v] = PRE ? dn[PRE ? v : 0] : load(p.dy, p.lddy, r, v);
            hv[v] = PRE ? hn[PRE ? v : 0] : load(p.h, p.ldh, r, v);
            if (PRE) sv[v] = p.dres ? load(p.dres, p.ldres, r, v) : zero;
        }
        auto xhat = [&](uint64_t h) { return mul_f32x2(CENTER ? add_f32x2(h, minus_mean2) : h, rstd2); };
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = tid + v * T;
            uint64_t d[4], h[4], g[4];
            unpack_pairs(dv[v], d);
            unpack_pairs(hv[v], h);
            unpack_pairs(gamma(v), g);
            if (SMEM && i < nv) {
                ulonglong2* a = reinterpret_cast<ulonglong2*>(acc_smem + 8 * i);
                ulonglong2 a0 = a[0], a1 = a[1];
                a0.x = fma_f32x2(d[0], xhat(h[0]), a0.x);
                a0.y = fma_f32x2(d[1], xhat(h[1]), a0.y);
                a1.x = fma_f32x2(d[2], xhat(h[2]), a1.x);
                a1.y = fma_f32x2(d[3], xhat(h[3]), a1.y);
                a[0] = a0;
                a[1] = a1;
                if (CENTER) {
                    ulonglong2* b = reinterpret_cast<ulonglong2*>(acc_smem + p.cols + 8 * i);
                    ulonglong2 b0 = b[0], b1 = b[1];
                    b0.x = add_f32x2(d[0], b0.x);
                    b0.y = add_f32x2(d[1], b0.y);
                    b1.x = add_f32x2(d[2], b1.x);
                    b1.y = add_f32x2(d[3], b1.y);
                    b[0] = b0;
                    b[1] = b1;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t x = xhat(h[e]);
                if (!SMEM) acc[0][SMEM ? 0 : v][e] = fma_f32x2(d[e], x, acc[0][SMEM ? 0 : v][e]);
                if (!SMEM && CENTER) acc[S - 1][SMEM ? 0 : v][e] = add_f32x2(d[e], acc[S - 1][SMEM ? 0 : v][e]);
                const uint64_t dg = mul_f32x2(d[e], g[e]);
                dot2 = fma_f32x2(dg, x, dot2);
                if (CENTER) sum2 = add_f32x2(dg, sum2);
            }
        }
        if (PRE) fetch(r + step);
        const float2 dot = unpack_f32x2(dot2);
        float sum = dot.x + dot.y, sum0 = 0.0f;
        if (CENTER) {
            const float2 s = unpack_f32x2(sum2);
            sum0 = s.x + s.y;
        }
        if (WARP) {
#pragma unroll
            for (int off = LANES / 2; off >= 1; off >>= 1) {
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
                if (CENTER) sum0 = __fadd_rn(sum0, __shfl_xor_sync(0xffffffffu, sum0, off));
            }
        } else if (CENTER) {
            const float2 s = block_sum2(make_float2(sum, sum0), part2[k & 1]);
            sum = s.x;
            sum0 = s.y;
        } else {
            sum = block_sum(sum, part[k & 1]);
        }
        const float m = -__fdiv_rn(sum, static_cast<float>(p.cols));
        const uint64_t m2 = pack_f32x2(m, m);
        const float m0 = CENTER ? -__fdiv_rn(sum0, static_cast<float>(p.cols)) : 0.0f;
        const uint64_t m02 = pack_f32x2(m0, m0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = tid + v * T;
            if (i >= nv || r >= p.rows) continue;
            uint64_t d[4], h[4], g[4], s[4];
            unpack_pairs(dv[v], d);
            unpack_pairs(hv[v], h);
            unpack_pairs(gamma(v), g);
            if (!PRE) sv[v] = p.dres ? load(p.dres, p.ldres, r, v) : zero;
            unpack_pairs(sv[v], s);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t dg = CENTER ? fma_f32x2(d[e], g[e], m02) : mul_f32x2(d[e], g[e]);
                const uint64_t x = fma_f32x2(rstd2, fma_f32x2(xhat(h[e]), m2, dg), s[e]);
                const float2 f = unpack_f32x2(x);
                w[e] = pack_bf16x2(f.x, f.y);
            }
            __stcs(reinterpret_cast<uint4*>(p.dx + r * p.cols + 8 * i), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float* band = p.partials + (static_cast<int64_t>(blockIdx.x) * S + s) * p.cols;
        if (WARP && s > 0) __syncthreads();  // the sums before have been read
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = tid + v * T;
            if (i >= nv) continue;
            // SMEM: a thread wrote the columns of shared memory that it reads here
            const ulonglong2* a = reinterpret_cast<const ulonglong2*>(acc_smem + s * p.cols + 8 * i);
            ulonglong2* o = reinterpret_cast<ulonglong2*>((WARP ? acc_smem + own * p.cols : band) + 8 * i);
            o[0] = SMEM ? a[0] : make_ulonglong2(acc[s][SMEM ? 0 : v][0], acc[s][SMEM ? 0 : v][1]);
            o[1] = SMEM ? a[1] : make_ulonglong2(acc[s][SMEM ? 0 : v][2], acc[s][SMEM ? 0 : v][3]);
        }
        if (WARP) {
            __syncthreads();
            for (int c = threadIdx.x; c < p.cols; c += 256) {
                float t = acc_smem[c];
#pragma unroll
                for (int w = 1; w < kRowsPerCta; ++w) t = __fadd_rn(t, acc_smem[w * p.cols + c]);
                band[c] = t;
            }
        }
    }
}

// dgamma[c] (+)= sum over the bands: 32 columns per CTA, 32 threads per column
// take every 32nd band, their sums are added in order.  The bands are `ld` apart;
// the grid's second row sums dbeta's, which lie behind dgamma's.
__global__ void __launch_bounds__(1024) norm_grad_finalize_kernel(const float* ws, int bands, int64_t ld,
                                                                  int64_t cols, float* dgamma, float* dbeta,
                                                                  int accumulate) {
    await_dependency();
    ws += blockIdx.y * cols;
    float* out = blockIdx.y ? dbeta : dgamma;
    __shared__ float part[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cl;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int b = sl; b < bands; b += 32) s += __ldcg(ws + b * ld + c);
    }
    part[sl][cl] = s;
    __syncthreads();
    if (sl == 0 && c < cols) {
        float t = part[0][cl];
#pragma unroll
        for (int i = 1; i < 32; ++i) t += part[i][cl];
        out[c] = accumulate ? out[c] + t : t;
    }
}

// the sum of the bands that a gradient's kernel left
template <bool CENTER>
int launch_finalize(const NormGradParams& p, int bands, cudaStream_t stream) {
    constexpr int sums = CENTER ? 2 : 1;
    const dim3 grid(static_cast<unsigned>((p.cols + 31) / 32), CENTER && p.dbeta ? 2 : 1);
    return launch_dependent_clusters(norm_grad_finalize_kernel, grid, 0, 1024, 0, stream, p.partials, bands, sums * p.cols,
                                     p.cols, p.dgamma, p.dbeta, p.accumulate) == cudaSuccess
               ? 0
               : -3;
}

// T threads per CTA (a warp per row: 256), up to `per_sm` CTAs per SM: each leaves
// one band of partial sums.  (They run at once, but for up to 256 columns, where
// registers let two of the four.)
template <bool CENTER, int V, int MAXT, bool SMEM, bool PRE, int LANES, int MINB = 1>
int launch_grad(const NormGradParams& p, int T, int num_sms, int per_sm, cudaStream_t stream) {
    auto kern = norm_grad_kernel<CENTER, V, MAXT, SMEM, PRE, LANES, MINB>;
    constexpr int rows_per_cta = LANES ? 256 / (LANES ? LANES : 1) : 1;
    constexpr int sums = CENTER ? 2 : 1;
    const size_t smem = SMEM || LANES ? static_cast<size_t>(p.cols) * 4 * (SMEM ? sums : rows_per_cta) : 0;
    if (SMEM) {
        static PerDevice allowed;
        if (allow_shared_memory(allowed, kern, CENTER ? kLayerNormMaxCols * 8 : kNormMaxCols * 4) != 0) return -3;
    }
    // Few rows: fewer bands to add up.  Layer norm, us, two CTAs per SM / four (2048 columns) or six
    // (1280): 600 rows 6.8 / 9.0 and 5.8 / 7.8, 1000 rows 8.5 / 9.9 and 7.7 / 8.5, 1400 rows 10.1 / 10.6
    // and 8.9 / 9.9, 2000 rows 11.8 / 12.2 and 10.7 / 10.4, 4000 rows 20.1 / 17.6 and 17.5 / 13.8
    if (CENTER && LANES == 0 && per_sm > 2 && p.rows <= 10 * static_cast<int64_t>(num_sms)) per_sm = 2;
    int64_t cap = static_cast<int64_t>(num_sms) * (per_sm < 1 ? 1 : per_sm);
    if (cap > kGradMaxBands) cap = kGradMaxBands;
    const int64_t want = (p.rows + rows_per_cta - 1) / rows_per_cta;
    const int bands = static_cast<int>(want < cap ? want : cap);
    if (launch_dependent(kern, static_cast<unsigned>(bands), static_cast<unsigned>(T), smem, stream, p) != cudaSuccess)
        return -3;
    return launch_finalize<CENTER>(p, bands, stream);
}

}  // namespace
}  // namespace fp8ll

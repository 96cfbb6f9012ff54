// rmsnorm.cu -- root-mean-square norm with the residual's addition and an fp8
// output, and its backward pass.
//
//   h = bf16(x + r)                     (the residual stream; h = x without r)
//   rstd = 1 / sqrt(mean_c h^2 + eps)
//   y = fl32(fl32(h rstd) gamma)        -> fp8 codes and scales, and / or bf16
//
// The norm is taken of the rounded h, which is what the stream carries on and
// what the backward pass reads.  y is cast from fp32: the cast sees the value
// before any bf16 rounding, so an element is rounded once.
//
// Rows kernel: one row per CTA at a time, T threads with V 16-byte vectors of
// the row each, held as packed bf16 between the sum of squares and the cast.
// 16 neighbouring threads hold one 128-block, so block and MX maxima are
// shuffles.  Columns kernel: 128 x 128 tiles of h staged in shared memory as
// the transposed casts do it, with the row's rstd and the column's gamma
// applied on the way to the codes.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "mx_rule.cuh"
#include "rmsnorm.h"

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

template <int FMT, int RECIPE, int V>
__global__ void __launch_bounds__(1024) rmsnorm_rows_kernel(const __grid_constant__ RmsNormParams p) {
    __shared__ float part[2][32];
    const int nv = static_cast<int>(p.cols / 8);
    const int T = blockDim.x;
    const int64_t mx_groups = 2 * ((p.rows + 255) / 256);
    // MXFP8: the scale bytes of rows beyond the matrix hold 127
    const int64_t all_rows = RECIPE == kRecipeMx && p.qr ? mx_groups * 128 : p.rows;
    float inv_t = 1.0f, s_t = 1.0f, top = 0.0f;
    if (RECIPE == kRecipeTensor) {
        block_scale<FMT>(*p.amax_in, inv_t, s_t);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s_t;
    }
    int k = 0;
    for (int64_t r = blockIdx.x; r < all_rows; r += gridDim.x, ++k) {
        if (RECIPE == kRecipeMx && r >= p.rows) {
            for (int64_t i = threadIdx.x; i < p.cols / 32; i += T)
                p.sfr[mx_sf_offset(i >> 2, mx_groups, r, static_cast<int>(i & 3))] = 127;
            continue;
        }
        uint4 hv[V];
        float sq = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            hv[v] = make_uint4(0, 0, 0, 0);
            if (i < nv) {
                hv[v] = *reinterpret_cast<const uint4*>(p.x + r * p.ldx + 8 * i);
                if (p.residual) {
                    const uint4 rv = *reinterpret_cast<const uint4*>(p.residual + r * p.ldr + 8 * i);
                    float a[8], b[8];
                    unpack8(hv[v], a);
                    unpack8(rv, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] += b[e];
                    hv[v] = pack8(a);
                }
                if (p.h) *reinterpret_cast<uint4*>(p.h + r * p.cols + 8 * i) = hv[v];
            }
            float f[8];
            unpack8(hv[v], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
        }
        sq = block_sum(sq, part[k & 1]);
        const float rstd = rsqrtf(__fdiv_rn(sq, static_cast<float>(p.cols)) + p.eps);
        if (threadIdx.x == 0) p.rstd[r] = rstd;
        if (!p.qr && !p.y && !(RECIPE == kRecipeTensor && p.amax_out)) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            const bool in = i < nv;
            float f[8], g[8];
            unpack8(hv[v], f);
            unpack8(in ? __ldg(reinterpret_cast<const uint4*>(p.gamma + 8 * i)) : make_uint4(0, 0, 0, 0), g);
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = __fmul_rn(__fmul_rn(f[e], rstd), g[e]);
                amax = fmaxf(amax, fabsf(f[e]));
            }
            if (p.y && in) *reinterpret_cast<uint4*>(p.y + r * p.cols + 8 * i) = pack8(f);
            if (RECIPE == kRecipeTensor) {
                if (in) top = fmaxf(top, amax);
                if (p.qr && in) *reinterpret_cast<uint2*>(p.qr + r * p.cols + 8 * i) = encode8<FMT>(f, inv_t);
            } else if (p.qr) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float inv, s;
                if (RECIPE == kRecipeBlock) {
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
                    block_scale<FMT>(amax, inv, s);
                    if (in && (i & 15) == 0) p.sr[(i >> 4) * p.sldr + r] = s;
                } else {
                    const int e = mx_exponent<FMT>(amax);
                    inv = mx_inverse_scale(e);
                    if (in && (i & 3) == 0)
                        p.sfr[mx_sf_offset(i >> 4, mx_groups, r, (i >> 2) & 3)] = static_cast<uint8_t>(e + 127);
                }
                if (in) *reinterpret_cast<uint2*>(p.qr + r * p.cols + 8 * i) = encode8<FMT>(f, inv);
            }
        }
    }
    if (RECIPE == kRecipeTensor && p.amax_out) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        // non-negative floats order like their bits; a maximum does not depend on the order
        if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned*>(p.amax_out), __float_as_uint(top));
    }
}

// Column codes of one 128 x 128 tile of y, as the transposed casts lay them
// out: thread t takes the column pair t / 4 and the 32-row part t % 4.  |y| =
// fl(fl(|h| rstd) |gamma|) grows with fl(|h| rstd), so the block maximum needs
// one product per element and gamma once.
template <int FMT, int RECIPE>
__global__ void __launch_bounds__(256, 4) rmsnorm_cols_kernel(const __grid_constant__ RmsNormParams p) {
    __shared__ __align__(16) uint32_t tile[128][64];
    __shared__ float rs[4][33];
    const uint16_t* h = p.h ? p.h : p.x;
    const int64_t ldh = p.h ? p.cols : p.ldx;
    const int64_t rb = blockIdx.y;
    const int64_t r0 = rb * 128, c0 = static_cast<int64_t>(blockIdx.x) * 128;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
        const int i = threadIdx.x + it * 256;
        const int rr = i >> 4, ch = i & 15;
        *reinterpret_cast<uint4*>(&tile[rr][(ch * 4 + 8 * (rr >> 5)) & 63]) =
            *reinterpret_cast<const uint4*>(h + (r0 + rr) * ldh + c0 + ch * 8);
    }
    if (threadIdx.x < 128) rs[threadIdx.x >> 5][threadIdx.x & 31] = p.rstd[r0 + threadIdx.x];
    __syncthreads();
    const int cp = threadIdx.x >> 2, part = threadIdx.x & 3;
    const int64_t c = c0 + 2 * cp;
    const uint32_t gw = *reinterpret_cast<const uint32_t*>(p.gamma + c);
    const float g_lo = bf16_lo(gw), g_hi = bf16_hi(gw);
    const int wcol = (cp + 8 * part) & 63;
    float inv_lo = 1.0f, inv_hi = 1.0f, s_lo = 1.0f, s_hi = 1.0f;
    if (RECIPE == kRecipeTensor) {
        block_scale<FMT>(*p.amax_in, inv_lo, s_lo);
        inv_hi = inv_lo;
    } else {
        float a_lo = 0.0f, a_hi = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t w = tile[32 * part + i][wcol];
            const float s = rs[part][i];
            a_lo = fmaxf(a_lo, fabsf(__fmul_rn(bf16_lo(w), s)));
            a_hi = fmaxf(a_hi, fabsf(__fmul_rn(bf16_hi(w), s)));
        }
        a_lo = __fmul_rn(a_lo, fabsf(g_lo));
        a_hi = __fmul_rn(a_hi, fabsf(g_hi));
        if (RECIPE == kRecipeBlock) {
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                a_lo = fmaxf(a_lo, __shfl_xor_sync(0xffffffffu, a_lo, off));
                a_hi = fmaxf(a_hi, __shfl_xor_sync(0xffffffffu, a_hi, off));
            }
            block_scale<FMT>(a_lo, inv_lo, s_lo);
            block_scale<FMT>(a_hi, inv_hi, s_hi);
            if (part == 0) {
                p.sc[rb * p.sldc + c] = s_lo;
                p.sc[rb * p.sldc + c + 1] = s_hi;
            }
        } else {
            const int e_lo = mx_exponent<FMT>(a_lo), e_hi = mx_exponent<FMT>(a_hi);
            inv_lo = mx_inverse_scale(e_lo);
            inv_hi = mx_inverse_scale(e_hi);
            const int64_t groups = 2 * ((p.cols + 255) / 256);
            p.sfc[mx_sf_offset(rb, groups, c, part)] = static_cast<uint8_t>(e_lo + 127);
            p.sfc[mx_sf_offset(rb, groups, c + 1, part)] = static_cast<uint8_t>(e_hi + 127);
            // an odd number of 128-column groups: the group beyond the matrix holds 127
            if (c0 + 128 == p.cols && (p.cols & 255) != 0 && threadIdx.x < 128)
                *reinterpret_cast<uint32_t*>(p.sfc + mx_sf_offset(rb, groups, p.cols + threadIdx.x, 0)) = 0x7F7F7F7Fu;
        }
    }
    uint32_t wl[8], wh[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t lo16[2], hi16[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = 4 * i + 2 * j;
            const uint32_t w0 = tile[32 * part + k][wcol], w1 = tile[32 * part + k + 1][wcol];
            const float s0 = rs[part][k], s1 = rs[part][k + 1];
            lo16[j] = encode2<FMT>(__fmul_rn(__fmul_rn(bf16_lo(w0), s0), g_lo),
                                   __fmul_rn(__fmul_rn(bf16_lo(w1), s1), g_lo), inv_lo);
            hi16[j] = encode2<FMT>(__fmul_rn(__fmul_rn(bf16_hi(w0), s0), g_hi),
                                   __fmul_rn(__fmul_rn(bf16_hi(w1), s1), g_hi), inv_hi);
        }
        wl[i] = lo16[0] | (lo16[1] << 16);
        wh[i] = hi16[0] | (hi16[1] << 16);
    }
    uint4* dl = reinterpret_cast<uint4*>(p.qc + c * p.rows + r0 + 32 * part);
    uint4* dh = reinterpret_cast<uint4*>(p.qc + (c + 1) * p.rows + r0 + 32 * part);
    dl[0] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
    dl[1] = make_uint4(wl[4], wl[5], wl[6], wl[7]);
    dh[0] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
    dh[1] = make_uint4(wh[4], wh[5], wh[6], wh[7]);
}

// threads and vectors per thread of a row of nv 16-byte vectors
void row_shape(int64_t cols, int& T, int& V) {
    const int64_t nv = cols / 8;
    V = nv <= 128 ? 1 : nv <= 512 ? 2 : 4;
    T = static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32);
}

template <int FMT, int RECIPE>
int launch_norm(const RmsNormParams& p, cudaStream_t stream, int num_sms) {
    int T, V;
    row_shape(p.cols, T, V);
    if (RECIPE == kRecipeTensor && p.amax_out &&
        cudaMemsetAsync(p.amax_out, 0, sizeof(float), stream) != cudaSuccess)
        return -3;
    int64_t grid = RECIPE == kRecipeMx && p.qr ? (p.rows + 255) / 256 * 256 : p.rows;
    const int64_t cap = static_cast<int64_t>(num_sms) * (2048 / T);
    if (grid > cap) grid = cap;
    const unsigned g = static_cast<unsigned>(grid);
    switch (V) {
        case 1: rmsnorm_rows_kernel<FMT, RECIPE, 1><<<g, T, 0, stream>>>(p); break;
        case 2: rmsnorm_rows_kernel<FMT, RECIPE, 2><<<g, T, 0, stream>>>(p); break;
        default: rmsnorm_rows_kernel<FMT, RECIPE, 4><<<g, T, 0, stream>>>(p); break;
    }
    if (p.qc) {
        const dim3 tiles(static_cast<unsigned>(p.cols / 128), static_cast<unsigned>(p.rows / 128));
        rmsnorm_cols_kernel<FMT, RECIPE><<<tiles, 256, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

// ---------------------------------------------------------------- backward
//
//   d = dy gamma, xhat = h rstd, m = mean_c (d xhat)
//   dx = rstd (d - xhat m) + dres        dgamma_c = sum_r dy xhat
//
// A CTA walks rows; a thread keeps the same columns for all of them, so dgamma
// is summed in its registers and written once per CTA as a band of partial
// sums, which the finalize adds in a fixed order.
template <int V>
__global__ void __launch_bounds__(1024) rmsnorm_grad_kernel(const __grid_constant__ RmsNormGradParams p) {
    __shared__ float part[2][32];
    const int nv = static_cast<int>(p.cols / 8);
    const int T = blockDim.x;
    float acc[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[v][e] = 0.0f;
    int k = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, ++k) {
        uint4 dv[V], hv[V];
        const float rstd = p.rstd[r];
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            dv[v] = hv[v] = make_uint4(0, 0, 0, 0);
            if (i < nv) {
                dv[v] = *reinterpret_cast<const uint4*>(p.dy + r * p.lddy + 8 * i);
                hv[v] = *reinterpret_cast<const uint4*>(p.h + r * p.ldh + 8 * i);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            float d[8], h[8], g[8];
            unpack8(dv[v], d);
            unpack8(hv[v], h);
            unpack8(i < nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma + 8 * i)) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xhat = h[e] * rstd;
                acc[v][e] = fmaf(d[e], xhat, acc[v][e]);
                dot = fmaf(d[e] * g[e], xhat, dot);
            }
        }
        const float m = __fdiv_rn(block_sum(dot, part[k & 1]), static_cast<float>(p.cols));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = threadIdx.x + v * T;
            if (i >= nv) continue;
            float d[8], h[8], g[8], s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            unpack8(dv[v], d);
            unpack8(hv[v], h);
            unpack8(__ldg(reinterpret_cast<const uint4*>(p.gamma + 8 * i)), g);
            if (p.dres) unpack8(*reinterpret_cast<const uint4*>(p.dres + r * p.ldres + 8 * i), s);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(rstd, fmaf(-h[e] * rstd, m, d[e] * g[e]), s[e]);
            *reinterpret_cast<uint4*>(p.dx + r * p.cols + 8 * i) = pack8(d);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = threadIdx.x + v * T;
        if (i >= nv) continue;
        float4* o = reinterpret_cast<float4*>(p.partials + static_cast<int64_t>(blockIdx.x) * p.cols + 8 * i);
        o[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
        o[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
    }
}

// dgamma[c] (+)= sum over the bands: 32 columns per CTA, eight threads per
// column take every eighth band, their sums are added in order
__global__ void __launch_bounds__(256) rmsnorm_grad_finalize_kernel(const float* __restrict__ ws, int64_t bands,
                                                                    int64_t cols, float* __restrict__ out,
                                                                    int accumulate) {
    __shared__ float part[8][32];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cl;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t b = sl; b < bands; b += 8) s += ws[b * cols + c];
    }
    part[sl][cl] = s;
    __syncthreads();
    if (sl == 0 && c < cols) {
        float t = part[0][cl];
#pragma unroll
        for (int i = 1; i < 8; ++i) t += part[i][cl];
        out[c] = accumulate ? out[c] + t : t;
    }
}

}  // namespace

int launch_rmsnorm(const RmsNormParams& p, int recipe, int fmt, cudaStream_t stream, int num_sms) {
    switch (recipe * 2 + fmt) {
        case 0: return launch_norm<0, kRecipeBlock>(p, stream, num_sms);
        case 1: return launch_norm<1, kRecipeBlock>(p, stream, num_sms);
        case 2: return launch_norm<0, kRecipeMx>(p, stream, num_sms);
        case 3: return launch_norm<1, kRecipeMx>(p, stream, num_sms);
        case 4: return launch_norm<0, kRecipeTensor>(p, stream, num_sms);
        case 5: return launch_norm<1, kRecipeTensor>(p, stream, num_sms);
        default: return -3;
    }
}

int launch_rmsnorm_grad(const RmsNormGradParams& p, cudaStream_t stream, int num_sms) {
    int T, V;
    row_shape(p.cols, T, V);
    int64_t cap = static_cast<int64_t>(num_sms) * (1024 / T);
    if (cap > kGradMaxBands) cap = kGradMaxBands;
    const int bands = static_cast<int>(p.rows < cap ? p.rows : cap);
    switch (V) {
        case 1: rmsnorm_grad_kernel<1><<<bands, T, 0, stream>>>(p); break;
        case 2: rmsnorm_grad_kernel<2><<<bands, T, 0, stream>>>(p); break;
        default: rmsnorm_grad_kernel<4><<<bands, T, 0, stream>>>(p); break;
    }
    rmsnorm_grad_finalize_kernel<<<static_cast<unsigned>((p.cols + 31) / 32), 256, 0, stream>>>(
        p.partials, bands, p.cols, p.dgamma, p.accumulate);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace fp8ll

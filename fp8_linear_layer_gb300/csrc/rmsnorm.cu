// rmsnorm.cu -- root-mean-square norm with the residual's addition and an fp8
// output, and its backward pass.
//
//   h = bf16(x + r)                     (the residual stream; h = x without r)
//   rstd = 1 / sqrt(mean_c h^2 + eps)   (0 where that root is 0)
//   y = fl32(fl32(h rstd) gamma)        -> fp8 codes and scales, and / or bf16
//
// The norm is taken of the rounded h, which is what the stream carries on and
// what the backward pass reads.  y is cast from fp32: the cast sees the value
// before any bf16 rounding, so an element is rounded once.
//
// Rows kernel: one row per CTA at a time, T threads with V 16-byte vectors of
// the row each, held as packed bf16 between the sum of squares and the cast;
// the next row is loaded meanwhile.  16 neighbouring threads hold one
// 128-block, so block and MX maxima are shuffles, and a lane divides for one of
// its blocks only.  Bound by HBM: 8192 x 4096 with residual, 1x128: 38 us, 0.91 of
// the measured copy rate (48.9 without the loads ahead and with every lane's own
// divisions).
// Columns kernel: reads h again, while half of it is in L2, and casts it down its
// columns: 20 us more at that size.  (A cluster of CTAs per 128-row band, which
// formed h and then cast its tiles from L2, took 98 us for both: each CTA's chain
// of loads was too long for the CTAs that fit.)
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
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

// y = fl(fl(h rstd) gamma) of eight packed bf16 values, as four pairs
__device__ __forceinline__ void norm8(const uint4& h, const uint4& g, uint64_t rstd2, uint64_t (&y)[4]) {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = mul_f32x2(mul_f32x2(pack_f32x2(bf16_lo(hw[i]), bf16_hi(hw[i])), rstd2),
                         pack_f32x2(bf16_lo(gw[i]), bf16_hi(gw[i])));
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
// single block stores it; otherwise the word was zeroed before.
__device__ __forceinline__ void fold_amax(float top, float* part, float* amax_out) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    __syncthreads();  // part's last use as sums is over
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, part[w]);
        if (gridDim.x == 1)
            *amax_out = top;
        else
            atomicMax(reinterpret_cast<unsigned*>(amax_out), __float_as_uint(top));
    }
}

// GREG: gamma stays in registers for all rows of the CTA
template <int FMT, int RECIPE, int V, int MAXT, bool GREG>
__global__ void __launch_bounds__(MAXT) rmsnorm_rows_kernel(const __grid_constant__ RmsNormParams p) {
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
    if (RECIPE == kRecipeTensor) {
        block_scale<FMT>(*p.amax_in, inv_t, s_t);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s_t;
    }
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
    auto load_gamma = [&](int v) {
        const int i = threadIdx.x + v * T;
        return i < nv ? *reinterpret_cast<const uint4*>(p.gamma + 8 * i) : zero;
    };
    int64_t r = blockIdx.x;
    fetch(r);
    uint4 gv[GREG ? V : 1];
    if (GREG) {
#pragma unroll
        for (int v = 0; v < V; ++v) gv[v] = load_gamma(v);
    }
    for (int k = 0; r < p.rows; r += gridDim.x, ++k) {
        uint4 hv[V];
        float sq = 0.0f;
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
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
        }
        fetch(r + gridDim.x);
        sq = block_sum(sq, part[k & 1]);
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
            norm8(hv[v], GREG ? gv[GREG ? v : 0] : load_gamma(v), rstd2, y[v]);
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
        if (!p.qr) continue;
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
                if (i < nv && (i & 3) == 0)
                    p.sfr[mx_sf_offset(i >> 4, mx_groups, r, (i >> 2) & 3)] = static_cast<uint8_t>(e + 127);
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
    }
    if (RECIPE == kRecipeMx && p.qr) {
        // the scale bytes of rows beyond the matrix hold 127
        for (r = p.rows + blockIdx.x; r < mx_groups * 128; r += gridDim.x)
            for (int64_t i = threadIdx.x; i < p.cols / 128; i += T)
                *reinterpret_cast<uint32_t*>(p.sfr + mx_sf_offset(i, mx_groups, r, 0)) = 0x7F7F7F7Fu;
    }
    if (RECIPE == kRecipeTensor && p.amax_out) fold_amax(top, part[0], p.amax_out);
}

// Column codes of y from h, rstd and gamma, in 128 x 128 tiles of h staged in
// shared memory as the transposed casts do it (each 32-row band rotated by eight
// words): persistent CTAs with two staged tiles, the next one on its way by
// cp.async while one is cast.  Thread t takes the column pair t / 4 and the
// 32-row part t % 4.  |y| = fl(fl(|h| rstd) |gamma|) grows with fl(|h| rstd), so
// a column's maximum needs one product per element and gamma once.
constexpr int kColsCtas = 3;
struct ColsStage {
    uint32_t tile[128][64];
    float rstd[4][36];  // part p's 32 rows, banks apart
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int FMT, int RECIPE>
__global__ void __launch_bounds__(256, kColsCtas) rmsnorm_cols_kernel(const __grid_constant__ RmsNormParams p) {
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
        float inv_lo = inv_t, inv_hi = inv_t, s_lo, s_hi;
        if (RECIPE != kRecipeTensor) {
            float a_lo = 0.0f, a_hi = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t w = st.tile[32 * part + i][wcol];
                const float s = st.rstd[part][i];
                const float2 v = unpack_f32x2(mul_f32x2(pack_f32x2(bf16_lo(w), bf16_hi(w)), pack_f32x2(s, s)));
                a_lo = fmaxf(a_lo, fabsf(v.x));
                a_hi = fmaxf(a_hi, fabsf(v.y));
            }
            // a maximum over NaN (gamma NaN, or infinite over zeros) is 0, as of the values one by one
            a_lo = fmaxf(__fmul_rn(a_lo, fabsf(g_lo)), 0.0f);
            a_hi = fmaxf(__fmul_rn(a_hi, fabsf(g_hi)), 0.0f);
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
        uint32_t wl[8], wh[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = st.tile[32 * part + 4 * i + j][wcol];
                const float s = st.rstd[part][4 * i + j];
                v[j] = unpack_f32x2(mul_f32x2(
                    mul_f32x2(mul_f32x2(pack_f32x2(bf16_lo(w), bf16_hi(w)), pack_f32x2(s, s)), g2), inv2));
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

template <int FMT, int RECIPE>
int launch_cols(const RmsNormParams& p, cudaStream_t stream, int num_sms) {
    auto kern = rmsnorm_cols_kernel<FMT, RECIPE>;
    static PerDevice allowed;
    if (allow_shared_memory(allowed, kern, 2 * sizeof(ColsStage)) != 0) return -3;
    const int64_t tiles = p.rows / 128 * (p.cols / 128), cap = static_cast<int64_t>(num_sms) * kColsCtas;
    return launch_dependent(kern, static_cast<unsigned>(tiles < cap ? tiles : cap), 256, 2 * sizeof(ColsStage), stream,
                            p) == cudaSuccess
               ? 0
               : -3;
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
    // 768 (1024) threads of rows per SM; from 4224 columns on the kernels' 118 to 121
    // registers let only 512 run at once (at 7168 columns two CTAs of 224 threads, three
    // launched): the rest start where the first ones end
    int64_t grid = RECIPE == kRecipeMx ? (p.rows + 255) / 256 * 256 : p.rows;
    const int64_t cap = static_cast<int64_t>(num_sms) * ((V == 1 ? 1024 : 768) / T < 1 ? 1 : (V == 1 ? 1024 : 768) / T);
    if (grid > cap) grid = cap;
    const unsigned g = static_cast<unsigned>(grid);
    // a kernel of one thread: a memset node cost 4 us here
    if (RECIPE == kRecipeTensor && p.amax_out && g > 1 &&
        launch_dependent(zero_word_kernel, 1, 1, 0, stream, p.amax_out) != cudaSuccess)
        return -3;
    cudaError_t rc;
    switch (V) {
        case 1: rc = launch_dependent(rmsnorm_rows_kernel<FMT, RECIPE, 1, 128, true>, g, T, 0, stream, p); break;
        case 2: rc = launch_dependent(rmsnorm_rows_kernel<FMT, RECIPE, 2, 256, true>, g, T, 0, stream, p); break;
        default:
            rc = T <= 512 ? launch_dependent(rmsnorm_rows_kernel<FMT, RECIPE, 4, 512, true>, g, T, 0, stream, p)
                          : launch_dependent(rmsnorm_rows_kernel<FMT, RECIPE, 4, 1024, false>, g, T, 0, stream, p);
    }
    if (rc != cudaSuccess) return -3;
    return p.qc ? launch_cols<FMT, RECIPE>(p, stream, num_sms) : 0;
}

// ---------------------------------------------------------------- backward
//
//   d = dy gamma, xhat = h rstd, m = mean_c (d xhat)
//   dx = rstd (d - xhat m) + dres        dgamma_c = sum_r dy xhat
//
// Bound by HBM: 16384 x 7168 with the residual's gradient 159 us, 0.87 of the copy
// rate; 0.49 at 32768 columns, where a thread holds eight vectors and loads
// nothing ahead.
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

template <int V, int MAXT, bool SMEM, bool PRE, int LANES>
__global__ void __launch_bounds__(MAXT, 1) rmsnorm_grad_kernel(const __grid_constant__ RmsNormGradParams p) {
    static_assert(LANES == 0 || !SMEM, "a warp's sums stay in registers");
    constexpr bool WARP = LANES != 0;
    constexpr int kRowsPerCta = WARP ? 256 / (WARP ? LANES : 1) : 1;
    __shared__ float part[2][32];
    extern __shared__ __align__(16) float acc_smem[];  // SMEM: [cols], LANES: [kRowsPerCta][cols]
    await_dependency();
    release_dependents();
    const int nv = static_cast<int>(p.cols / 8);
    const int T = WARP ? LANES : blockDim.x;
    const int tid = WARP ? threadIdx.x % (WARP ? LANES : 1) : threadIdx.x;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint64_t acc[SMEM ? 1 : V][4];
    if (SMEM) {
        for (int i = tid; i < nv; i += T) {
            reinterpret_cast<uint4*>(acc_smem)[2 * i] = zero;
            reinterpret_cast<uint4*>(acc_smem)[2 * i + 1] = zero;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[SMEM ? 0 : v][e] = 0ull;
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
    const int second = LANES == 16 ? own & 1 : 0;  // the halves of a warp leave the loop together
    if (PRE) fetch(r);
    for (int k = 0; r - second < p.rows; r += step, ++k) {
        uint4 dv[V], hv[V], sv[V];
        const float rstd = r < p.rows ? p.rstd[r] : 0.0f;
        const uint64_t rstd2 = pack_f32x2(rstd, rstd);
        uint64_t dot2 = 0ull;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dv[v] = PRE ? dn[PRE ? v : 0] : load(p.dy, p.lddy, r, v);
            hv[v] = PRE ? hn[PRE ? v : 0] : load(p.h, p.ldh, r, v);
            if (PRE) sv[v] = p.dres ? load(p.dres, p.ldres, r, v) : zero;
        }
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
                a0.x = fma_f32x2(d[0], mul_f32x2(h[0], rstd2), a0.x);
                a0.y = fma_f32x2(d[1], mul_f32x2(h[1], rstd2), a0.y);
                a1.x = fma_f32x2(d[2], mul_f32x2(h[2], rstd2), a1.x);
                a1.y = fma_f32x2(d[3], mul_f32x2(h[3], rstd2), a1.y);
                a[0] = a0;
                a[1] = a1;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t xhat = mul_f32x2(h[e], rstd2);
                if (!SMEM) acc[SMEM ? 0 : v][e] = fma_f32x2(d[e], xhat, acc[SMEM ? 0 : v][e]);
                dot2 = fma_f32x2(mul_f32x2(d[e], g[e]), xhat, dot2);
            }
        }
        if (PRE) fetch(r + step);
        const float2 dot = unpack_f32x2(dot2);
        float sum = dot.x + dot.y;
        if (WARP) {
#pragma unroll
            for (int off = LANES / 2; off >= 1; off >>= 1)
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
        } else {
            sum = block_sum(sum, part[k & 1]);
        }
        const float m = -__fdiv_rn(sum, static_cast<float>(p.cols));
        const uint64_t m2 = pack_f32x2(m, m);
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
                const uint64_t x =
                    fma_f32x2(rstd2, fma_f32x2(mul_f32x2(h[e], rstd2), m2, mul_f32x2(d[e], g[e])), s[e]);
                const float2 f = unpack_f32x2(x);
                w[e] = pack_bf16x2(f.x, f.y);
            }
            __stcs(reinterpret_cast<uint4*>(p.dx + r * p.cols + 8 * i), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
    float* band = p.partials + static_cast<int64_t>(blockIdx.x) * p.cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = tid + v * T;
        if (i >= nv) continue;
        // SMEM: a thread wrote the columns of shared memory that it reads here
        const ulonglong2* a = reinterpret_cast<const ulonglong2*>(acc_smem + 8 * i);
        ulonglong2* o = reinterpret_cast<ulonglong2*>((WARP ? acc_smem + own * p.cols : band) + 8 * i);
        o[0] = SMEM ? a[0] : make_ulonglong2(acc[SMEM ? 0 : v][0], acc[SMEM ? 0 : v][1]);
        o[1] = SMEM ? a[1] : make_ulonglong2(acc[SMEM ? 0 : v][2], acc[SMEM ? 0 : v][3]);
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

// dgamma[c] (+)= sum over the bands: 32 columns per CTA, 32 threads per column
// take every 32nd band, their sums are added in order
__global__ void __launch_bounds__(1024) rmsnorm_grad_finalize_kernel(const float* ws, int bands,
                                                                     int64_t cols, float* out,
                                                                     int accumulate) {
    await_dependency();
    __shared__ float part[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cl;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int b = sl; b < bands; b += 32) s += __ldcg(ws + b * cols + c);
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

// T threads per CTA (a warp per row: 256), up to `per_sm` CTAs per SM: each leaves
// one band of partial sums.  (They run at once, but for up to 256 columns, where
// registers let two of the four.)
template <int V, int MAXT, bool SMEM, bool PRE, int LANES>
int launch_grad(const RmsNormGradParams& p, int T, int num_sms, int per_sm, cudaStream_t stream) {
    auto kern = rmsnorm_grad_kernel<V, MAXT, SMEM, PRE, LANES>;
    constexpr int rows_per_cta = LANES ? 256 / (LANES ? LANES : 1) : 1;
    const size_t smem = SMEM || LANES ? static_cast<size_t>(p.cols) * 4 * rows_per_cta : 0;
    if (SMEM) {
        static PerDevice allowed;
        if (allow_shared_memory(allowed, kern, kNormMaxCols * 4) != 0) return -3;
    }
    int64_t cap = static_cast<int64_t>(num_sms) * (per_sm < 1 ? 1 : per_sm);
    if (cap > kGradMaxBands) cap = kGradMaxBands;
    const int64_t want = (p.rows + rows_per_cta - 1) / rows_per_cta;
    const int bands = static_cast<int>(want < cap ? want : cap);
    if (launch_dependent(kern, static_cast<unsigned>(bands), static_cast<unsigned>(T), smem, stream, p) != cudaSuccess)
        return -3;
    return launch_dependent(rmsnorm_grad_finalize_kernel, static_cast<unsigned>((p.cols + 31) / 32), 1024, 0, stream,
                            p.partials, bands, p.cols, p.dgamma, p.accumulate) == cudaSuccess
               ? 0
               : -3;
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
    const int64_t nv = p.cols / 8;
    auto threads = [nv](int V) { return static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32); };
    // up to 1024 columns a row needs no more than a warp: 25.8 us at 32768 x 512
    // against 35.8 with 64 threads per row and a barrier
    if (nv <= 16) return launch_grad<1, 256, false, true, 16>(p, 256, num_sms, 4, stream);
    if (nv <= 32) return launch_grad<1, 256, false, true, 32>(p, 256, num_sms, 4, stream);
    if (nv <= 64) return launch_grad<2, 256, false, true, 32>(p, 256, num_sms, 2, stream);
    if (nv <= 128) return launch_grad<4, 256, false, true, 32>(p, 256, num_sms, 1, stream);
    // two vectors a thread while the CTA stays within 512 threads, else dgamma
    // moves to shared memory: 102.6 us at 4096 x 14336 against 132.9 with spilled
    // registers
    int T = threads(2);
    if (T <= 512) return launch_grad<2, 512, false, true, 0>(p, T, num_sms, 512 / T, stream);
    T = threads(4);
    if (T <= 512) return launch_grad<4, 512, true, true, 0>(p, T, num_sms, 1, stream);
    return launch_grad<8, 512, true, false, 0>(p, threads(8), num_sms, 1, stream);
}

}  // namespace fp8ll

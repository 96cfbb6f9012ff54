// gemm_rows.cu -- the linear GEMM (bias, activation, residual) for few rows of A.
//
//   Y = act(A B^T + bias) + residual,   A [M][K] a handful of tokens, B [N][K] the weights
//
// Bound by one read of B.  The tile kernels give 256 features to one SM, which
// leaves most SMs idle (56 of them work at N = 14336), and walk all of K there.
// Here the weights are the 128-row side of the MMA and the tokens its N (16, 32
// or 64 columns; 128 where more rows than 64 come here, a tile of them per grid
// row), so little of the tensor core's work is spent on rows that do not exist,
// and K is split over a cluster of up to eight CTAs, which add their fp32 sums
// through distributed shared memory in rank order (deterministic).  Two CTAs per
// SM keep 128 KB or more of B in flight there (at 128 tokens one, 80 KB).  One
// token, 14336 features over 4096: 13.1 us one behind another on 1x128 operands,
// 0.68 of the copy rate; what is left is the launch, the first loads' latency (they
// are asked for only when the kernel before has completed) and the join (4.2 us at
// 7168 x 2048 for 2.2 us of loads).  On the tile kernel 22.1 us, with
// fp8 mma.sync fragments straight from global memory 17.1 (43 at 13 tokens on
// MXFP8: those MMAs take 53 cycles each here).
// Per CTA of 8 warps:
//   warp 0      TMA producer: 128 x 128 bytes of B, the tokens' 128 bytes and,
//               by recipe, their block scales or scale atoms into one ring.
//   warp 1      tensor-memory owner and MMA issuer (M = 128, N = tokens, K = 32,
//               four per 128-deep K block); MXFP8 copies the block's two scale
//               atoms to tensor memory first.
//   warps 4-7   1x128: add sB sA P of each K block into fp32 registers, one row
//               of B per thread, all tokens; otherwise read the accumulator
//               once at the end.
//   all warps   epilogue: a thread takes two neighbouring features.
// GATED: the 128 rows of B are 64 of the gate and the same 64 of the up projection,
// so that a CTA holds both sums of an output.  MXFP8: their scales come from halves
// of two atoms, which warp 3 puts together as a stage lands (a copy to tensor memory
// takes whole atoms, and a TMA box no eight bytes).  One token, 14336 outputs over 4096:
// 22.2 us, 0.81 of the copy rate; 224 CTAs fill 152 SMs unevenly, but with three to an
// SM and K in two parts, which evens that out, it takes as long.
#include <atomic>
#include <cuda_runtime.h>

#include "common.cuh"
#include "gemm_rows.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "norm.h"

namespace fp8ll {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsAcc = 4;  // accumulators of the 1x128 recipe

template <int NT>
constexpr int rows_stages() {
    return NT == 64 ? 4 : 5;
}
template <int NT>
constexpr int rows_ctas_per_sm() {
    return NT == 128 ? 1 : 2;
}

constexpr int kGateRows = kRowsFeatures / 2;  // GATED: output features of a tile

// RAW: room for the two projections' scale atoms
template <int NT, bool RAW>
struct __align__(1024) RowsSmem {
    static constexpr int S = rows_stages<NT>();
    uint8_t w[S][kRowsFeatures * 128];
    uint8_t x[S][NT * 128];
    float sw[S][128];  // 1x128: scales of the block's rows; MXFP8: a 512-byte scale atom
    float sx[S][128];
    float raw[RAW ? S : 1][RAW ? 256 : 4];
    uint64_t sf_ready[S];  // RAW: stage s's atom is put together
    uint64_t full[S];
    uint64_t empty[S];
    uint64_t acc_full[kRowsAcc];
    uint64_t acc_empty[kRowsAcc];
    uint64_t drain;
    uint32_t tmem_base;
    int32_t failed;
};
template <int NT, bool RAW = false>
constexpr size_t rows_smem_bytes() {
    return sizeof(RowsSmem<NT, RAW>) + 1024;
}
// two CTAs per SM; the sums [NT][128] take the place of the weights' stages
static_assert(2 * (rows_smem_bytes<16, true>() + 1024) <= 233472 && 2 * (rows_smem_bytes<32, true>() + 1024) <= 233472 &&
                  2 * (rows_smem_bytes<64, true>() + 1024) <= 233472 && rows_smem_bytes<128, true>() <= 232448,
              "two CTAs per SM, one at 128 tokens");
static_assert(64 * kRowsFeatures * 4 <= rows_stages<64>() * kRowsFeatures * 128 &&
                  128 * kRowsFeatures * 4 <= rows_stages<128>() * kRowsFeatures * 128,
              "sums fit the stages");

template <int RECIPE, int NT>
constexpr uint32_t rows_tmem_cols() {
    // 1x128: four accumulators; MXFP8: one, and eight scale columns per stage
    constexpr uint32_t need = RECIPE == kRecipeBlock ? kRowsAcc * NT
                              : RECIPE == kRecipeMx  ? NT + 8 * rows_stages<NT>()
                                                     : NT;
    return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}

// 16 columns of the 32 tensor-memory lanes of a warp's quadrant: v[i] = column
// addr + i of lane (thread % 32)
__device__ __forceinline__ void tmem_ld_16(uint32_t addr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// no-swizzle shared-memory descriptor of a 32-row x 16-byte scale atom (8-row
// core matrices, 128 bytes apart), and its copy to four tensor-memory columns
__device__ __forceinline__ void copy_scale_atom(uint32_t taddr, uint32_t saddr) {
    const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 16) |
                          (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}

// elements off and off + 1 of a bf16 array where `one` and `two` say they
// exist; `pairs`: every offset is even and the array 4-byte aligned
__device__ __forceinline__ uint32_t load_pair(const uint16_t* p, int64_t off, bool one, bool two, bool pairs) {
    if (pairs) return one ? *reinterpret_cast<const uint32_t*>(p + off) : 0u;
    return (one ? static_cast<uint32_t>(p[off]) : 0u) | (two ? static_cast<uint32_t>(p[off + 1]) << 16 : 0u);
}

__device__ __forceinline__ void store_pair(uint16_t* p, int64_t off, bool one, bool two, bool pairs, uint32_t w) {
    if (pairs) {
        if (one) *reinterpret_cast<uint32_t*>(p + off) = w;
        return;
    }
    if (one) p[off] = static_cast<uint16_t>(w & 0xFFFFu);
    if (two) p[off + 1] = static_cast<uint16_t>(w >> 16);
}

template <int RECIPE, int NT, bool GATED>
__global__ void __launch_bounds__(kRowsThreads, rows_ctas_per_sm<NT>())
    gemm_rows_kernel(const __grid_constant__ RowsMaps maps, const __grid_constant__ RowsParams p) {
    constexpr bool RAW = GATED && RECIPE == kRecipeMx;
    using Smem = RowsSmem<NT, RAW>;
    constexpr int S = Smem::S;
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                        ~static_cast<uintptr_t>(1023));
    float(*sums)[kRowsFeatures] = reinterpret_cast<float(*)[kRowsFeatures]>(sm.w);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cs = p.cluster;
    const int rank = static_cast<int>(blockIdx.x) % cs;
    const int64_t tile = blockIdx.x / cs;
    constexpr int kFeatures = GATED ? kGateRows : kRowsFeatures;
    const int64_t n0 = tile * kFeatures;
    const int m0 = static_cast<int>(blockIdx.y) * NT;  // a multiple of 128 where it is not 0
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / cs);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / cs);
    const uint64_t budget = p.budget_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            if (RAW) mbar_init(smem_addr(&sm.sf_ready[s]), 1);
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), RECIPE == kRecipeBlock ? 5 : 1);  // the MMAs, and the scales' readers
        }
        for (int b = 0; b < kRowsAcc; ++b) {
            mbar_init(smem_addr(&sm.acc_full[b]), 1);
            mbar_init(smem_addr(&sm.acc_empty[b]), 4);
        }
        mbar_init(smem_addr(&sm.drain), 1);
        sm.failed = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&sm.tmem_base), rows_tmem_cols<RECIPE, NT>());
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    await_dependency();
    release_dependents();
    constexpr uint32_t kSfCol = NT;  // MXFP8: scale columns behind the accumulator

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1 && !p.debug_starve; ++kb) {
                ok = mbar_wait(smem_addr(&sm.empty[s]), ph ^ 1u, budget);
                if (!ok) break;
                const uint32_t bar = smem_addr(&sm.full[s]);
                mbar_arrive_expect_tx(bar, (kRowsFeatures + NT) * 128 + (RECIPE == kRecipeBlock  ? 512 + NT * 4
                                                                         : RAW                 ? 1536
                                                                         : RECIPE == kRecipeMx ? 1024
                                                                                               : 0));
                tma_load_2d(smem_addr(sm.w[s]), &maps.w, bar, kb * 128, static_cast<int32_t>(n0));
                if (GATED)
                    tma_load_2d(smem_addr(sm.w[s] + kGateRows * 128), &maps.w, bar, kb * 128,
                                static_cast<int32_t>(p.N + n0));
                tma_load_2d(smem_addr(sm.x[s]), &maps.x, bar, kb * 128, m0);
                if (RECIPE == kRecipeBlock) {
                    tma_load_2d(smem_addr(sm.sw[s]), &maps.sw, bar, static_cast<int32_t>(n0), kb);
                    if (GATED)
                        tma_load_2d(smem_addr(sm.sw[s] + kGateRows), &maps.sw, bar, static_cast<int32_t>(p.N + n0), kb);
                    tma_load_2d(smem_addr(sm.sx[s]), &maps.sx, bar, m0, kb);
                } else if (RECIPE == kRecipeMx) {
                    if (RAW) {
                        const int32_t atom = static_cast<int32_t>(kb * p.groups_w + tile / 2);
                        tma_load_2d(smem_addr(sm.raw[RAW ? s : 0]), &maps.sw, bar, 0, atom);
                        tma_load_2d(smem_addr(sm.raw[RAW ? s : 0] + 128), &maps.sw, bar, 0, atom + p.N / 128);
                    } else {
                        tma_load_2d(smem_addr(sm.sw[s]), &maps.sw, bar, 0, static_cast<int32_t>(kb * p.groups_w + tile));
                    }
                    tma_load_2d(smem_addr(sm.sx[s]), &maps.sx, bar, 0, 
                                static_cast<int32_t>(kb * p.groups_x + m0 / 128));
                }
                ++issued;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            // every load lands before the shared memory goes away
            for (int i = 1; i <= (issued < S ? issued : S); ++i) {
                int si = s - i;
                uint32_t pi = ph;
                if (si < 0) {
                    si += S;
                    pi ^= 1u;
                }
                if (!mbar_wait(smem_addr(&sm.full[si]), pi, budget)) ok = false;
            }
        }
    } else if (warp == 1) {
        int s = 0, ab = 0;
        uint32_t ph = 0, aph = 0;
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(NT >> 3) << 17);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (RECIPE == kRecipeBlock) ok = mbar_wait_warp(smem_addr(&sm.acc_empty[ab]), aph ^ 1u, budget);
            if (ok) ok = mbar_wait_warp(smem_addr(&sm.full[s]), ph, budget);
            if (RAW && ok) ok = mbar_wait_warp(smem_addr(&sm.sf_ready[s]), ph, budget);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                const uint64_t adesc = smem_desc_k_sw128(smem_addr(sm.w[s]));
                const uint64_t bdesc = smem_desc_k_sw128(smem_addr(sm.x[s]));
                if (RECIPE == kRecipeMx) {
                    const uint32_t sf = tmem + kSfCol + 8u * s;
                    copy_scale_atom(sf, smem_addr(sm.sw[s]));
                    copy_scale_atom(sf + 4, smem_addr(sm.sx[s]));
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_mx(tmem, adesc + 2u * k, bdesc + 2u * k, idesc | (k << 4) | (k << 29), sf, sf + 4,
                               kb > kb0 || k > 0);
                } else {
                    const uint32_t d = RECIPE == kRecipeBlock ? tmem + static_cast<uint32_t>(ab * NT) : tmem;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_f8f6f4(d, adesc + 2u * k, bdesc + 2u * k, idesc,
                                   (RECIPE == kRecipeTensor && kb > kb0) || k > 0);
                }
                mma_commit(smem_addr(&sm.empty[s]));
                if (RECIPE == kRecipeBlock || kb == kb1 - 1) mma_commit(smem_addr(&sm.acc_full[ab]));
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
            if (RECIPE == kRecipeBlock && ++ab == kRowsAcc) {
                ab = 0;
                aph ^= 1u;
            }
        }
        // all MMAs complete before tensor memory is released
        if (lane == 0) mma_commit(smem_addr(&sm.drain));
        __syncwarp();
        if (!mbar_wait_warp(smem_addr(&sm.drain), 0, budget)) ok = false;
    } else if (RAW && warp == 3) {
        // a row of an atom is 16 bytes, one word for each 32 rows of the operand: this
        // tile's 64 rows are words 0 and 1 of both atoms, or 2 and 3
        const int first = 2 * static_cast<int>(tile & 1);
        int s = 0;
        uint32_t ph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            ok = mbar_wait_warp(smem_addr(&sm.full[s]), ph, budget);
            if (!ok) break;
            const float* raw = sm.raw[RAW ? s : 0] + 4 * lane + first;
            const float2 gate = *reinterpret_cast<const float2*>(raw), up = *reinterpret_cast<const float2*>(raw + 128);
            *reinterpret_cast<float4*>(sm.sw[s] + 4 * lane) = make_float4(gate.x, gate.y, up.x, up.y);
            // read by the copy to tensor memory, and the raw atoms are refilled by TMA
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_lane0(smem_addr(&sm.sf_ready[s]), lane);
            if (++s == S) {
                s = 0;
                ph ^= 1u;
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
        float acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
        if (RECIPE == kRecipeBlock) {
            int s = 0, ab = 0;
            uint32_t ph = 0, aph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = mbar_wait2_warp(smem_addr(&sm.acc_full[ab]), aph, smem_addr(&sm.full[s]), ph, budget);
                if (!ok) break;
                tc_fence_after();
                const float sw = sm.sw[s][q * 32 + lane];
#pragma unroll
                for (int c = 0; c < NT; c += 16) {
                    float v[16];
                    tmem_ld_16(tq + static_cast<uint32_t>(ab * NT + c), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(v[i], __fmul_rn(sm.sx[s][c + i], sw), acc[c + i]);
                }
                tc_fence_before();
                // the scales were read with ordinary loads and are refilled by TMA
                fence_proxy_async_smem();
                __syncwarp();
                mbar_arrive_lane0(smem_addr(&sm.acc_empty[ab]), lane);
                mbar_arrive_lane0(smem_addr(&sm.empty[s]), lane);
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++ab == kRowsAcc) {
                    ab = 0;
                    aph ^= 1u;
                }
            }
        } else {
            ok = mbar_wait_warp(smem_addr(&sm.acc_full[0]), 0, budget);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < NT; c += 16) {
                    float v[16];
                    tmem_ld_16(tq + static_cast<uint32_t>(c), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c + i] = v[i];
                }
                tc_fence_before();
            }
        }
        // every block's MMAs have read their stages: the sums take their place
        if (ok) {
#pragma unroll
            for (int i = 0; i < NT; ++i) sums[i][q * 32 + lane] = acc[i];
        }
    }
    if (!ok) {
        record_status(p.status, kStatusTimeout);
        sm.failed = 1;
    }
    __syncwarp();
    tc_fence_before();
    if (cs > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, rows_tmem_cols<RECIPE, NT>());

    // thread -> feature; the cluster's CTAs and a CTA's halves share the tokens
    bool write = true;
    for (int r = 0; r < cs; ++r) {
        uint32_t f;
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(f)
                     : "r"(mapa_shared(smem_addr(&sm.failed), static_cast<uint32_t>(r))));
        write = write && f == 0u;
    }
    if (GATED) {
        // a thread takes two neighbouring features, both projections, and every (8 cs)-th
        // token, two tokens at a time so that their loads overlap
        const int nl = 2 * (threadIdx.x & 31);
        const int64_t n = n0 + nl;
        if (write) {
            const uint32_t bg = p.bias ? *reinterpret_cast<const uint32_t*>(p.bias + n) : 0u;
            const uint32_t bu = p.bias ? *reinterpret_cast<const uint32_t*>(p.bias + p.N + n) : 0u;
            const float scale = RECIPE == kRecipeTensor ? __fmul_rn(*p.tsx, *p.tsw) : 1.0f;
            const int rows = p.M - m0 < NT ? p.M - m0 : NT;
            constexpr int U = 2;
            for (int i0 = 8 * rank + warp; i0 < rows; i0 += 8 * U * cs) {
                float2 v[U][2][8];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + 8 * u * cs;
                    if (i >= rows) continue;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float* own = &sums[i][nl + kGateRows * b];
                        if (cs == 1) {
                            v[u][b][0] = *reinterpret_cast<const float2*>(own);
                        } else {
                            const uint32_t a = smem_addr(own);
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                if (r < cs) v[u][b][r] = ld_cluster_f32x2(mapa_shared(a, static_cast<uint32_t>(r)));
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + 8 * u * cs;
                    if (i >= rows) continue;
                    float2 z[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        z[b] = v[u][b][0];
#pragma unroll
                        for (int r = 1; r < 8; ++r) {
                            if (r < cs) {
                                z[b].x = __fadd_rn(z[b].x, v[u][b][r].x);
                                z[b].y = __fadd_rn(z[b].y, v[u][b][r].y);
                            }
                        }
                        if (RECIPE == kRecipeTensor) z[b] = make_float2(__fmul_rn(z[b].x, scale), __fmul_rn(z[b].y, scale));
                        const uint32_t bias = b ? bu : bg;
                        z[b] = make_float2(__fadd_rn(z[b].x, bf16_lo(bias)), __fadd_rn(z[b].y, bf16_hi(bias)));
                    }
                    const float2 a = p.gelu ? gate2<true>(z[0].x, z[0].y) : gate2<false>(z[0].x, z[0].y);
                    const int64_t row = m0 + i;
                    *reinterpret_cast<uint32_t*>(p.out + row * p.N + n) = pack_bf16x2(a.x * z[1].x, a.y * z[1].y);
                    if (p.aux) {
                        uint16_t* aux = p.aux + 2 * row * p.N + n;
                        *reinterpret_cast<uint32_t*>(aux) = pack_bf16x2(z[0].x, z[0].y);
                        *reinterpret_cast<uint32_t*>(aux + p.N) = pack_bf16x2(z[1].x, z[1].y);
                    }
                }
            }
        }
        if (cs > 1) cluster_sync();  // the peers have read this CTA's sums
        return;
    }
    // a thread takes two neighbouring features and every (4 cs)-th token, four
    // tokens at a time so that their loads overlap
    const int nl = 2 * (threadIdx.x & 63);
    const int64_t n = n0 + nl;
    const bool one = n < p.N, two = n + 1 < p.N;
    if (write && one) {
        const bool pairs = (p.N & 1) == 0;
        const bool res_pairs = pairs && (p.ldr & 1) == 0 && (reinterpret_cast<uintptr_t>(p.res) & 3u) == 0;
        const uint32_t bias = p.bias ? load_pair(p.bias, n, true, two, pairs) : 0u;
        const float scale = RECIPE == kRecipeTensor ? __fmul_rn(*p.tsx, *p.tsw) : 1.0f;
        const int rows = p.M - m0 < NT ? p.M - m0 : NT;
        constexpr int U = 4;
        for (int i0 = 4 * rank + static_cast<int>(threadIdx.x >> 6); i0 < rows; i0 += 4 * U * cs) {
            uint32_t res[U];
            float2 v[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 4 * u * cs;
                const bool in = i < rows;
                res[u] = p.res ? load_pair(p.res, (m0 + i) * p.ldr + n, in, in && two, res_pairs) : 0u;
                if (!in) continue;
                const float* own = &sums[i][nl];
                if (cs == 1) {
                    v[u][0] = *reinterpret_cast<const float2*>(own);
                } else {
                    const uint32_t a = smem_addr(own);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (r < cs) v[u][r] = ld_cluster_f32x2(mapa_shared(a, static_cast<uint32_t>(r)));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 4 * u * cs;
                if (i >= rows) continue;
                float z0 = v[u][0].x, z1 = v[u][0].y;
#pragma unroll
                for (int r = 1; r < 8; ++r) {
                    if (r < cs) {
                        z0 = __fadd_rn(z0, v[u][r].x);
                        z1 = __fadd_rn(z1, v[u][r].y);
                    }
                }
                if (RECIPE == kRecipeTensor) {
                    z0 = __fmul_rn(z0, scale);
                    z1 = __fmul_rn(z1, scale);
                }
                z0 = __fadd_rn(z0, bf16_lo(bias));
                z1 = __fadd_rn(z1, bf16_hi(bias));
                const float2 y = p.gelu ? gelu_tanh2(z0, z1) : make_float2(z0, z1);
                const int64_t off = static_cast<int64_t>(m0 + i) * p.N + n;
                store_pair(p.out, off, true, two, pairs,
                           pack_bf16x2(__fadd_rn(y.x, bf16_lo(res[u])), __fadd_rn(y.y, bf16_hi(res[u]))));
                if (p.aux) store_pair(p.aux, off, true, two, pairs, pack_bf16x2(z0, z1));
            }
        }
    }
    if (cs > 1) cluster_sync();  // the peers have read this CTA's sums
}

template <int RECIPE, int NT, bool GATED>
int launch_rows_impl(const RowsMaps& maps, const RowsParams& p, cudaStream_t stream) {
    auto kern = gemm_rows_kernel<RECIPE, NT, GATED>;
    constexpr size_t smem = rows_smem_bytes<NT, GATED && RECIPE == kRecipeMx>();
    static PerDevice allowed;
    if (allow_shared_memory(allowed, kern, smem) != 0) return -3;
    constexpr int features = GATED ? kGateRows : kRowsFeatures;
    const int64_t tiles = (static_cast<int64_t>(p.N) + features - 1) / features;
    const dim3 grid(static_cast<unsigned>(tiles * p.cluster), static_cast<unsigned>((p.M + NT - 1) / NT));
    return launch_dependent_clusters(kern, grid, static_cast<unsigned>(p.cluster), kRowsThreads, smem, stream, maps,
                                     p) == cudaSuccess
               ? 0
               : -3;
}

template <int RECIPE, bool GATED>
int launch_rows_recipe(const RowsMaps& maps, const RowsParams& p, cudaStream_t stream) {
    switch (rows_tokens(p.M)) {
        case 16: return launch_rows_impl<RECIPE, 16, GATED>(maps, p, stream);
        case 32: return launch_rows_impl<RECIPE, 32, GATED>(maps, p, stream);
        case 64: return launch_rows_impl<RECIPE, 64, GATED>(maps, p, stream);
        default: return launch_rows_impl<RECIPE, 128, GATED>(maps, p, stream);
    }
}

}  // namespace

// CTAs of clusters of c, one CTA to an SM, that run at once: the GPCs' sizes leave
// SMs over (of 152, 144 take part in clusters of 4, 120 in clusters of 8)
static int rows_slots(int c) {
    constexpr int NT = 128;  // its shared memory: one CTA fills an SM
    static std::atomic<int> known[64][3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::atomic<int>& slot = known[dev][c == 2 ? 0 : c == 4 ? 1 : 2];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = gemm_rows_kernel<kRecipeBlock, NT, false>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(rows_smem_bytes<NT>())) != cudaSuccess)
            return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(c));
        cfg.blockDim = dim3(kRowsThreads);
        cfg.dynamicSmemBytes = rows_smem_bytes<NT>();
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(c);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n *= c;
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

// A CTA's chain of K blocks halves with every step, as long as its clusters run at
// once.  With one CTA per SM a step needs two blocks for each.  With two (up to 64
// tokens; a cluster of 8 then takes 4 SMs: 36 such clusters run at once, 38 do not)
// the join of the sums, which grows with the tokens, has to be won back.  us, 1x128,
// 1 / 32 / 64 tokens:
//   14336 over 4096  in 1 part  14.9 / 16.1 / 18.7   in 2  13.2 / 14.3 / 16.3
//   14336 over 1024  in 1        6.1 /  7.2 /  8.7   in 2   6.4 /  7.6 /  9.5
//    8192 over 4096  in 2       10.0 / 11.0 / 12.7   in 4   9.4 / 10.4 / 11.5
//    8192 over 1024  in 2        4.8 /  5.6 /  6.8   in 4   4.7 /  5.5 /  6.7
//    4096 over 14336 in 4       14.4 / 15.6 / 17.0   in 8  13.1 / 14.3 / 16.1
//    2112 over 4096  in 4        6.1 /  6.4 /  7.3   in 8   5.1 /  5.8 /  7.5
//    4096 over 5120  in 4        7.8 /  8.4 /  9.4   in 8   7.8 /  9.1 / 10.6
int rows_cluster(int64_t M, int64_t N, int64_t nkb) {
    const int nt = rows_tokens(M);
    const int64_t tiles = (N + kRowsFeatures - 1) / kRowsFeatures * ((M + nt - 1) / nt);
    int c = 1;
    while (c < 8) {
        const int next = 2 * c;
        const bool alone = nkb >= 2 * next && tiles * next <= rows_slots(next);
        const int64_t enough = next == 2 ? 16 : next == 4 ? 8 : nt == 16 ? 32 : nt + 32;
        const bool two_per_sm = nt < 128 && nkb >= enough && tiles * next <= 2 * rows_slots(next < 4 ? next : 4);
        if (!alone && !two_per_sm) break;
        c = next;
    }
    return c;
}

template <bool GATED>
static int launch_rows(const RowsMaps& maps, RowsParams p, int recipe, cudaStream_t stream) {
    p.cluster = rows_cluster(p.M, (GATED ? 2LL : 1LL) * p.N, p.nkb);  // of as many tiles of B
    switch (recipe) {
        case kRecipeBlock: return launch_rows_recipe<kRecipeBlock, GATED>(maps, p, stream);
        case kRecipeMx: return launch_rows_recipe<kRecipeMx, GATED>(maps, p, stream);
        default: return launch_rows_recipe<kRecipeTensor, GATED>(maps, p, stream);
    }
}

int launch_gemm_rows(const RowsMaps& maps, RowsParams p, int recipe, cudaStream_t stream) {
    return launch_rows<false>(maps, p, recipe, stream);
}

int launch_gemm_rows_gated(const RowsMaps& maps, RowsParams p, int recipe, cudaStream_t stream) {
    return launch_rows<true>(maps, p, recipe, stream);
}

}  // namespace fp8ll

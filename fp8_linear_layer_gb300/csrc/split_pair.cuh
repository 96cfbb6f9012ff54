// split_pair.cuh -- splitting a tile's K blocks over the two CTA pairs of a
// cluster of four, for the MXFP8 and per-tensor linear GEMMs.
//
// With few 256 x 256 tiles the pairs leave most SMs idle and each walks all of
// K.  Here pair 0 and pair 1 of a cluster take half of the K blocks each.  Then
// every epilogue thread finishes two of the four rows of its fragment (pair 0
// the first two): it leaves its fp32 sums of the other two in its CTA's shared
// memory (B's stages, whose MMAs have completed) and, behind a cluster barrier,
// adds those that the thread of the same rows in the other pair left there.  The
// two addends commute, so both pairs' rows see the same order.
#pragma once
#include <cstdint>

#include "gemm_kernel.cuh"

namespace fp8ll {

constexpr uint32_t kSplitWords = 2 * kChunks;  // 64-bit words that a thread leaves
constexpr uint32_t kSplitBytes = 32 * kEpiWarps * kSplitWords * 8;

// word j of all threads side by side; part: the pair within the cluster
__device__ __forceinline__ void split_send(const uint64_t (&acc)[4 * kChunks], void* stage, int tid, int part) {
    uint64_t* st = static_cast<uint64_t*>(stage) + tid;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        st[(2 * c) * 32 * kEpiWarps] = part ? acc[4 * c] : acc[4 * c + 2];
        st[(2 * c + 1) * 32 * kEpiWarps] = part ? acc[4 * c + 1] : acc[4 * c + 3];
    }
}

// acc[4 c], acc[4 c + 1]: the finished sums of the thread's two rows
__device__ __forceinline__ void split_add(uint64_t (&acc)[4 * kChunks], const void* stage, int tid, int part,
                                          uint32_t crank) {
    const uint32_t peer = mapa_shared(smem_addr(static_cast<const uint64_t*>(stage) + tid), crank ^ 2u);
    const uint64_t one = pack_f32x2(1.0f, 1.0f);
#pragma unroll
    for (int c0 = 0; c0 < kChunks; c0 += 8) {
        uint64_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            asm volatile("ld.shared::cluster.b64 %0, [%1];"
                         : "=l"(v[j])
                         : "r"(peer + (2 * c0 + j) * 32 * kEpiWarps * 8));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int c = c0 + j / 2, r = j % 2;
            acc[4 * c + r] = fma_f32x2(v[j], one, part ? acc[4 * c + 2 + r] : acc[4 * c + r]);  // exactly the sum
        }
    }
}

// true when a wait of this CTA or of the one it exchanges sums with ran out
__device__ __forceinline__ bool split_failed(const int32_t* failed, uint32_t crank) {
    uint32_t own, peer;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(own) : "r"(mapa_shared(smem_addr(failed), crank)));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(peer) : "r"(mapa_shared(smem_addr(failed), crank ^ 2u)));
    return (own | peer) != 0u;
}

// Whether the split is taken: every tile's cluster of four runs at once, and K
// is long enough to pay for the exchange.  MXFP8, 1000 x 2112 with GELU, residual
// and Z, split / whole: 22.5 / 31.2 us over 7168, 14.9 / 17.0 over 2048; with the
// residual alone 13.1 / 13.6 over 2048, but 11.5 / 10.7 over 1024.
inline bool split_pays(const GemmParams& p, int slots) { return p.total_tiles <= slots && p.groups[0].nkb >= 16; }

}  // namespace fp8ll

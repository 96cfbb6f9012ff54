// split_k.cuh -- splitting a tile's K blocks over the CTAs (1x128: two or four) or
// CTA pairs (MXFP8, per-tensor: two) of a cluster, for the linear GEMMs.
//
// With few tiles the persistent kernels leave most SMs idle and each walks all of
// K.  Here the parts of a cluster take equal shares of a tile's K blocks.  Then
// every epilogue thread finishes 4 / SPLIT of the four rows of its fragment (part 0
// the first): it leaves its fp32 sums of the others in its CTA's shared memory
// (B's stages, whose MMAs have completed) and, behind a cluster barrier, adds those
// that the threads of the same rows in the other parts left there.  All rows add
// the parts in the same order.
#pragma once
#include <cstdint>

#include "gemm_params.h"
#include "ptx.cuh"

namespace fp8ll {

constexpr int kSplitChunks = 16;    // 8-column chunks of an epilogue thread, four rows each
constexpr int kSplitThreads = 256;  // epilogue threads
template <int SPLIT>
constexpr uint32_t kSplitBytes = (SPLIT - 1) * (4 / SPLIT) * kSplitChunks * kSplitThreads * 8;

// the place, among the SPLIT - 1 that a part leaves, of the sums for part `to`
__device__ __forceinline__ int split_slot(int from, int to) { return to - (to > from ? 1 : 0); }

// word j of all threads side by side
template <int SPLIT>
__device__ __forceinline__ void split_send(const uint64_t (&acc)[4 * kSplitChunks], void* stage, int tid, int part) {
    constexpr int R = 4 / SPLIT;
    uint64_t* st = static_cast<uint64_t*>(stage) + tid;
    if (SPLIT == 2) {
#pragma unroll
        for (int c = 0; c < kSplitChunks; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) st[(c * R + r) * kSplitThreads] = part ? acc[4 * c + r] : acc[4 * c + 2 + r];
        return;
    }
#pragma unroll
    for (int to = 0; to < SPLIT; ++to) {
        if (to == part) continue;
        uint64_t* slot = st + split_slot(part, to) * R * kSplitChunks * kSplitThreads;
#pragma unroll
        for (int c = 0; c < kSplitChunks; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) slot[(c * R + r) * kSplitThreads] = acc[4 * c + to * R + r];
    }
}

// acc[4 c + r], r < 4 / SPLIT: the finished sums of the thread's rows.  Part o of
// the cluster is its CTA `first` + `step` o.
template <int SPLIT>
__device__ __forceinline__ void split_add(uint64_t (&acc)[4 * kSplitChunks], const void* stage, int tid, int part,
                                          uint32_t first, uint32_t step) {
    constexpr int R = 4 / SPLIT;
    const uint32_t mine = smem_addr(static_cast<const uint64_t*>(stage) + tid);
    const uint64_t one = pack_f32x2(1.0f, 1.0f);
    uint32_t from[SPLIT];  // where part o left this thread's rows
#pragma unroll
    for (int o = 0; o < SPLIT; ++o)
        from[o] = mapa_shared(mine, first + step * o) + split_slot(o, part) * R * kSplitChunks * kSplitThreads * 8;
    constexpr int B = 8;  // chunks per batch of loads
#pragma unroll
    for (int c0 = 0; c0 < kSplitChunks; c0 += B) {
        uint64_t v[SPLIT - 1][R * B];
        // the others in order: with two parts the addends commute
#pragma unroll
        for (int i = 0; i < SPLIT - 1; ++i) {
            uint32_t addr = from[i + 1];
#pragma unroll
            for (int o = 0; o < SPLIT - 1; ++o)
                if (i == o && o < part) addr = from[o];
#pragma unroll
            for (int j = 0; j < R * B; ++j)
                asm volatile("ld.shared::cluster.b64 %0, [%1];"
                             : "=l"(v[i][j])
                             : "r"(addr + (R * c0 + j) * kSplitThreads * 8));
        }
#pragma unroll
        for (int j = 0; j < R * B; ++j) {
            const int c = c0 + j / R, r = j % R;
            uint64_t own = acc[4 * c + r];
#pragma unroll
            for (int o = 1; o < SPLIT; ++o)
                if (part == o) own = acc[4 * c + o * R + r];
            uint64_t s = part == 0 ? own : v[0][j];
#pragma unroll
            for (int o = 1; o < SPLIT; ++o)  // fma by one: exactly the sum
                s = fma_f32x2(part == o ? own : part < o ? v[o - 1][j] : v[o < SPLIT - 1 ? o : SPLIT - 2][j], one, s);
            acc[4 * c + r] = s;
        }
    }
}

// true when a wait of a CTA that this one exchanges sums with, or its own, ran out
template <int SPLIT>
__device__ __forceinline__ bool split_failed(const int32_t* failed, uint32_t first, uint32_t step) {
    uint32_t any = 0;
#pragma unroll
    for (int o = 0; o < SPLIT; ++o) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_addr(failed), first + step * o)));
        any |= v;
    }
    return any != 0u;
}

// Whether the split in two of the CTA pairs' tiles is taken: every tile's cluster
// of four runs at once, and K is long enough to pay for the exchange, part of which
// is won back because a part's threads store fewer rows: earlier where rows that are
// not 16-byte aligned make each dearer.  It does not depend on what is stored, so
// that a product's sums do not.  MXFP8, us, split / whole, with GELU, residual and Z
// | the residual | neither:
//   1000 x 2112 over 7168  21.6 / 31.2
//                    1536  13.3 / 14.4 | 11.5 / 11.1 | 10.7 / 10.0
//   1000 x 2111 over  768  14.7 / 18.3 | 12.2 / 12.5 | 10.0 /  9.1
//   1000 x 2110 over  768  13.1 / 15.5 | 11.1 / 10.8 |  9.3 /  7.9
//                     512  12.7 / 14.8 | 10.8 / 10.2 |  8.9 /  7.2
inline bool split_pays(const GemmParams& p, int slots) {
    return p.total_tiles <= slots && p.groups[0].nkb >= (p.N % 8 != 0 ? 6 : 16);
}

// The gated gradient, whose rows are dear (two read and two written for one of the
// linear GEMM's), earlier.  us, split / whole, MXFP8 | per tensor:
//   1000 x 2048 over 1024  12.0 / 12.6 | 11.5 / 12.8
//                     512  11.1 / 11.2 | 10.7 / 11.4
//   300 x 1024 over 1024   10.8 / 12.2 | 10.4 / 12.5
// (per tensor with shuffles; without, 11.0 and 10.2 split)
inline constexpr int kGatesSplitBlocks = 8;
inline bool split_gates_pays(const GemmParams& p, int slots) {
    return p.total_tiles <= slots && p.groups[0].nkb >= kGatesSplitBlocks;
}

}  // namespace fp8ll

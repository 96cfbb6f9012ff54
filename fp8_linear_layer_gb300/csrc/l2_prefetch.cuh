// l2_prefetch.cuh -- rows that will be read soon, asked for in L2 by one thread.
#pragma once
#include <cstdint>

namespace fp8ll {

// bytes (a multiple of 16) from ptr (16-byte aligned) on
__device__ __forceinline__ void prefetch_l2_rows(const void* ptr, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

}  // namespace fp8ll

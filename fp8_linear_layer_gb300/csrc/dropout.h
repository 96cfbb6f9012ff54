// dropout.h -- what the dropout kernels receive.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8ll {

// elements of a matrix: their groups of four are numbered in 32 bits
constexpr int64_t kDropoutMaxElements = 1LL << 34;

struct DropoutParams {
    const uint16_t* x;    // bf16 [rows][ldx]
    const uint16_t* res;  // bf16 [rows][ldr] or null
    uint16_t* out;        // bf16 [rows][cols]
    int64_t rows, cols, ldx, ldr;
    int64_t ahead;       // a CTA asks for the inputs of the one so many behind it in L2
    uint32_t threshold;  // words below it drop their element
    float scale;         // of a kept element: 1 / (1 - p)
    uint32_t key0, key1;
    uint32_t site;
    uint64_t step;
    const int64_t* step_dev;  // added to step, or null
};

int launch_dropout(const DropoutParams& p, cudaStream_t stream, int num_sms);

}  // namespace fp8ll

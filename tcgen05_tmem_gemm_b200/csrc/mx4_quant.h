// Launch of the kernels that quantise to 4-bit floats and read them back.
#pragma once

#include "dg_internal.h"

namespace dg {

// A quantised matrix as the kernels see it.
struct Mx4Mem {
    uint8_t *codes, *scales;
    const float *scale;
    int64_t rows, K, code_stride, k_tiles;
    int32_t align;  // rows of codes start at multiples of this many bytes (1, 4 or 16)
};

struct QuantParams {
    Mx4Mem q;
    DevView x;      // rows, k
    int64_t col;    // bytes between neighbouring k, where k is one dim
    int32_t vec;    // k contiguous, rows at multiples of 16 bytes
    int32_t pdl;
};

// back: writes x from q's codes and scales.
cudaError_t launch_quant(const QuantParams &p, int block, bool back, cudaStream_t s);

}  // namespace dg

// Matrix-vector products with 4-bit weights for up to 8 rows of activations:
// y = act(alpha * x W + beta * y + bias), W[k][n] = scale[n][g] (code - zero).
#include "common.cuh"

namespace dg {

namespace {

// One warp per column n: the lanes share a group's bytes (two k each), the
// group's sums are added up across the warp, then scaled.
__global__ void __launch_bounds__(256) gemv_w4_kernel(const GemvW4Params p) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= p.N) return;
    const uint8_t *codes = p.codes + n * p.code_stride;
    const char *scales = p.scales + n * p.scale_stride;
    const uint8_t *zeros = p.zeros ? p.zeros + n * p.zero_stride : nullptr;
    const int ses = elem_bytes(p.scale_dtype);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = 0, g = 0; k0 < p.K; k0 += p.group, ++g) {
        const int k1 = (int)min((int64_t)p.K, k0 + p.group);
        const int z = zeros ? zeros[g] & 15 : 8;
        float part[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k = (int)k0 + lane; k < k1; k += 32) {
            const float w = (float)(((codes[k >> 1] >> (4 * (k & 1))) & 15) - z);
            const int64_t xo = axis_offset(p.x.col, k);
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < p.R)
                    part[r] = fmaf(w, load_elem(p.x.ptr + xo + axis_offset(p.x.row, r), p.x.dtype), part[r]);
        }
        const float s = load_elem(scales + g * ses, p.scale_dtype);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) part[r] += __shfl_xor_sync(0xffffffffu, part[r], off);
            acc[r] = fmaf(s, part[r], acc[r]);
        }
    }
    if (lane != 0) return;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (r >= p.R) break;
        char *yp = const_cast<char *>(p.y.ptr) + axis_offset(p.y.row, r) + axis_offset(p.y.col, n);
        float v = epi_value(acc[r], p.alpha, 1.f, p.beta, yp, p.y.dtype);
        v = epi_fuse(v, p.bias, n, p.act, p.y.dtype != DG_F32);
        store_elem(yp, p.y.dtype, v);
    }
}

}  // namespace

cudaError_t launch_gemv_w4(const GemvW4Params &p, cudaStream_t s) {
    return launch_ex(gemv_w4_kernel, dim3((p.N + 7) / 8), dim3(256), 0, s, dim3(1, 1, 1), p.pdl, p);
}

}  // namespace dg

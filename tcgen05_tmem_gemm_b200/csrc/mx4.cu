// 4-bit floats with block scales: dg_quantize_mx4, dg_dequantize_mx4 and
// dg_gemm_mx4 (its kernel is in mx4_kernel.cuh).
//
// E2M1 has the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4 and 6.  A block of 32 values
// along k has an E8M0 scale, 2^floor(log2(largest) - 2), which brings the
// largest to [4, 8) (above 6 it is cut); a block of 16 an E4M3 scale, a sixth
// of the largest.  Everything is rounded to nearest, ties to even, and every
// division by a block's scale decides as the exact quotient would.
#include <algorithm>
#include <cmath>

#include "mx4_kernel.cuh"

namespace dg {
namespace {

// ------------------------------------------------------------ scales and codes

constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The byte of a block's scale from the largest magnitude's bits (NaN and
// infinities compare above every finite one), and the factor pair (s, r) with
// which mx4_unit makes x / s: for E8M0 the exact 1 / s, for E4M3 s and its
// rounded reciprocal.  A block with a NaN or an infinity has the scale NaN and
// codes of zero.
template <int BLOCK>
__device__ __forceinline__ uint32_t mx4_scale(uint32_t top, float &s, float &r) {
    if (BLOCK == 32) {
        const int e = max((int)(top >> 23) - 2, 0);  // a subnormal has exponent 0
        s = 0.f;
        r = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e): normal for every e up to 252
        if (top >= kInfBits) {
            r = 0.f;
            return 0xff;
        }
        return (uint32_t)e;
    }
    if (top >= kInfBits) {
        s = r = 0.f;
        return 0x7f;
    }
    const float want = __fdiv_rn(__uint_as_float(top), 6.f);
    const uint32_t code = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
    r = s > 0.f ? __frcp_rn(s) : 0.f;
    return code;
}

// x / s.  For E4M3, x times the rounded reciprocal and one correction by the
// remainder, which the fused multiply-add gives exactly: the result differs
// from the exact quotient by little more than half an ulp, is exact where the
// quotient is an FP32 number, and so lies on E2M1's rounding borders exactly
// where the quotient does (s has four significant bits: no other quotient comes
// within half an ulp of a border).
template <int BLOCK>
__device__ __forceinline__ float mx4_unit(float x, float s, float r) {
    if (BLOCK == 32) return r == 0.f ? 0.f : x * r;
    if (r == 0.f) return 0.f;
    const float y = x * r;
    // a zero keeps its sign
    return __uint_as_float(__float_as_uint(fmaf(fmaf(-y, s, x), r, y)) | (__float_as_uint(x) & 0x80000000u));
}

// Eight values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// The value of a scale's byte.
template <int BLOCK>
__device__ __forceinline__ float mx4_scale_value(uint32_t code) {
    if (BLOCK == 32)
        return code == 0xff ? __uint_as_float(0x7fffffffu) : __uint_as_float(code ? code << 23 : 1u << 22);
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(code & 0x7f), __NV_E4M3)));
}

// The magnitudes as FP32: 0, 0.5, then 1.m x 2^(e - 1).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7;
    const uint32_t mag = m < 2 ? (m ? 0x3f000000u : 0u) : ((126u + (m >> 1)) << 23) | (m & 1) << 22;
    return __uint_as_float(mag | (code & 8) << 28);
}

__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t block, int64_t k_tiles) {
    return (row / 128 * k_tiles + block / 4) * 512 + row % 32 * 16 + row % 128 / 32 * 4 + block % 4;
}

// A quantised matrix as the kernels see it.
struct Mx4Mem {
    uint8_t *codes, *scales;
    const float *scale;
    int64_t rows, K, code_stride, k_tiles;
    int32_t words;  // rows of codes start at multiples of 4 bytes
};

struct QuantParams {
    Mx4Mem q;
    DevView x;       // rows, k
    int32_t pdl;
};

// Eight neighbouring k of a row, in FP32; zeros past K.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const char *row, const Axis &col, int64_t k, int64_t K) {
    constexpr int ES = DT == DG_F32 ? 4 : 2;
    if (VEC && k + 8 <= K) {
        uint32_t w[2 * ES];
#pragma unroll
        for (int i = 0; i < ES / 2; ++i) *reinterpret_cast<uint4 *>(w + 4 * i) = *reinterpret_cast<const uint4 *>(row + k * ES + 16 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (DT == DG_F32) v[i] = __uint_as_float(w[i]);
            else if (DT == DG_BF16) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
            else v[i] = __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (i & 1 ? 16 : 0))));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? ld_out<DT>(row + axis_offset(col, k + i)) : 0.f;
}

constexpr int kQuantWarps = 8, kQuantChunks = 4;  // a warp takes 4 x 256 k of a row

// Rows whose k are neighbours: a lane has eight, a block is four (or two) lanes.
template <int DT, int BLOCK, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps) quantize_rows_kernel(const QuantParams p) {
    pdl_wait_then_release();
    constexpr int LANES = BLOCK / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    const bool divide = p.q.scale != nullptr;
    const int64_t K = p.q.K, k0 = (int64_t)blockIdx.x * (kQuantChunks * 256) + lane * 8;
    for (int64_t row = (int64_t)blockIdx.y * kQuantWarps + warp; row < p.q.rows; row += (int64_t)gridDim.y * kQuantWarps) {
        const char *x = p.x.ptr + axis_offset(p.x.row, row);
        float v[kQuantChunks][8];
#pragma unroll
        for (int c = 0; c < kQuantChunks; ++c) load8<DT, VEC>(v[c], x, p.x.col, k0 + c * 256, K);
#pragma unroll
        for (int c = 0; c < kQuantChunks; ++c) {
            const int64_t k = k0 + c * 256;
            if (k - lane * 8 >= K) break;  // the same for the whole warp
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (divide) v[c][i] = __fdiv_rn(v[c][i], factor);
                top = max(top, k + i < K ? abs_bits(v[c][i]) : 0u);
            }
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            float s, r;
            uint32_t code = mx4_scale<BLOCK>(top, s, r);
            // four blocks' scales are one word
            const int64_t block = k / BLOCK;
            code = block * BLOCK < K ? code << (8 * (block & 3)) : 0u;
            code |= __shfl_xor_sync(0xffffffffu, code, LANES);
            code |= __shfl_xor_sync(0xffffffffu, code, 2 * LANES);
            if ((lane & (4 * LANES - 1)) == 0 && k < K)
                *reinterpret_cast<uint32_t *>(p.q.scales + scale_at(row, block, p.q.k_tiles)) = code;
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = k + i < K ? mx4_unit<BLOCK>(v[c][i], s, r) : 0.f;
            const uint32_t e = e2m1x8(u);
            uint8_t *out = p.q.codes + row * p.q.code_stride + k / 2;
            if (p.q.words && k + 8 <= K) *reinterpret_cast<uint32_t *>(out) = e;
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k + 2 * i < K) out[i] = (uint8_t)(e >> (8 * i));
        }
    }
}

constexpr int kTurnK = 64;  // a thread takes 64 k of a row

// Any view, a thread per row and 64 k: made for rows that are neighbours in memory.
template <int DT, int BLOCK>
__global__ void __launch_bounds__(128) quantize_any_kernel(const QuantParams p) {
    pdl_wait_then_release();
    const int64_t row = (int64_t)blockIdx.x * 128 + threadIdx.x, K = p.q.K;
    if (row >= p.q.rows) return;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    const bool divide = p.q.scale != nullptr;
    const char *x = p.x.ptr + axis_offset(p.x.row, row);
    for (int64_t k0 = (int64_t)blockIdx.y * kTurnK; k0 < K; k0 += (int64_t)gridDim.y * kTurnK) {
        float v[kTurnK];
#pragma unroll
        for (int i = 0; i < kTurnK; ++i) v[i] = k0 + i < K ? ld_out<DT>(x + axis_offset(p.x.col, k0 + i)) : 0.f;
        uint32_t scales = 0;
#pragma unroll
        for (int b = 0; b < kTurnK / BLOCK; ++b) {
            if (k0 + b * BLOCK >= K) break;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                float &u = v[b * BLOCK + i];
                if (divide && k0 + b * BLOCK + i < K) u = __fdiv_rn(u, factor);
                top = max(top, abs_bits(u));
            }
            float s, r;
            scales |= mx4_scale<BLOCK>(top, s, r) << (8 * b);
#pragma unroll
            for (int j = 0; j < BLOCK / 8; ++j) {
                const int64_t k = k0 + b * BLOCK + 8 * j;
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = mx4_unit<BLOCK>(v[b * BLOCK + 8 * j + i], s, r);
                const uint32_t e = e2m1x8(u);
                uint8_t *out = p.q.codes + row * p.q.code_stride + k / 2;
                if (p.q.words && k + 8 <= K) *reinterpret_cast<uint32_t *>(out) = e;
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k + 2 * i < K) out[i] = (uint8_t)(e >> (8 * i));
            }
        }
        // blocks past the last one of its tile get a zero
        uint8_t *at = p.q.scales + scale_at(row, k0 / BLOCK, p.q.k_tiles);
        if (BLOCK == 16) {
            *reinterpret_cast<uint32_t *>(at) = scales;
        } else {
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)scales;
            if (k0 + kTurnK >= K && k0 / BLOCK % 4 == 0) *reinterpret_cast<uint16_t *>(at + 2) = 0;
        }
    }
}

// Eight values of a row back.
template <int DT, bool VEC>
__device__ __forceinline__ void store8(const float (&v)[8], char *row, const Axis &col, int64_t k, int64_t K) {
    constexpr int ES = DT == DG_F32 ? 4 : 2;
    if (VEC && k + 8 <= K) {
        uint32_t w[2 * ES];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (DT == DG_F32) {
                w[i] = __float_as_uint(v[i]);
                w[i + 1] = __float_as_uint(v[i + 1]);
            } else {
                w[i / 2] = pack2<DT == DG_BF16>(v[i], v[i + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < ES / 2; ++i) *reinterpret_cast<uint4 *>(row + k * ES + 16 * i) = *reinterpret_cast<uint4 *>(w + 4 * i);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) st_out<DT>(row + axis_offset(col, k + i), v[i]);
}

__device__ __forceinline__ uint32_t codes8(const Mx4Mem &q, int64_t row, int64_t k) {
    const uint8_t *in = q.codes + row * q.code_stride + k / 2;
    if (q.words && k + 8 <= q.K) return *reinterpret_cast<const uint32_t *>(in);
    uint32_t e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k + 2 * i < q.K) e |= (uint32_t)in[i] << (8 * i);
    return e;
}

template <int DT, int BLOCK, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps) dequantize_rows_kernel(const QuantParams p) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    const int64_t K = p.q.K, k0 = (int64_t)blockIdx.x * (kQuantChunks * 256) + lane * 8;
    for (int64_t row = (int64_t)blockIdx.y * kQuantWarps + warp; row < p.q.rows; row += (int64_t)gridDim.y * kQuantWarps) {
        char *y = const_cast<char *>(p.x.ptr) + axis_offset(p.x.row, row);
        uint32_t e[kQuantChunks], s[kQuantChunks];
#pragma unroll
        for (int c = 0; c < kQuantChunks; ++c) {
            const int64_t k = k0 + c * 256;
            e[c] = k < K ? codes8(p.q, row, k) : 0u;
            s[c] = k < K ? p.q.scales[scale_at(row, k / BLOCK, p.q.k_tiles)] : 0u;
        }
#pragma unroll
        for (int c = 0; c < kQuantChunks; ++c) {
            const int64_t k = k0 + c * 256;
            if (k >= K) break;
            const float unit = mx4_scale_value<BLOCK>(s[c]) * factor;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = e2m1_value(e[c] >> (4 * i)) * unit;
            store8<DT, VEC>(v, y, p.x.col, k, K);
        }
    }
}

template <int DT, int BLOCK>
__global__ void __launch_bounds__(128) dequantize_any_kernel(const QuantParams p) {
    pdl_wait_then_release();
    const int64_t row = (int64_t)blockIdx.x * 128 + threadIdx.x, K = p.q.K;
    if (row >= p.q.rows) return;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    char *y = const_cast<char *>(p.x.ptr) + axis_offset(p.x.row, row);
    for (int64_t k0 = (int64_t)blockIdx.y * kTurnK; k0 < K; k0 += (int64_t)gridDim.y * kTurnK) {
        uint32_t e[kTurnK / 8];
#pragma unroll
        for (int j = 0; j < kTurnK / 8; ++j) e[j] = k0 + 8 * j < K ? codes8(p.q, row, k0 + 8 * j) : 0u;
#pragma unroll
        for (int b = 0; b < kTurnK / BLOCK; ++b) {
            if (k0 + b * BLOCK >= K) break;
            const float unit = mx4_scale_value<BLOCK>(p.q.scales[scale_at(row, k0 / BLOCK + b, p.q.k_tiles)]) * factor;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                const int at = b * BLOCK + i;
                if (k0 + at < K)
                    st_out<DT>(y + axis_offset(p.x.col, k0 + at), e2m1_value(e[at / 8] >> (4 * (at % 8))) * unit);
            }
        }
    }
}

// ----------------------------------------------------------------- launches

template <int DT, int BLOCK>
cudaError_t quant_run(const QuantParams &p, bool back, bool rows, bool vec, cudaStream_t s) {
    if (rows) {
        const dim3 grid((unsigned)((p.q.K + kQuantChunks * 256 - 1) / (kQuantChunks * 256)),
                        (unsigned)std::min<int64_t>((p.q.rows + kQuantWarps - 1) / kQuantWarps, 65535));
        auto kern = back ? (vec ? dequantize_rows_kernel<DT, BLOCK, true> : dequantize_rows_kernel<DT, BLOCK, false>)
                         : (vec ? quantize_rows_kernel<DT, BLOCK, true> : quantize_rows_kernel<DT, BLOCK, false>);
        return launch_ex(kern, grid, dim3(32 * kQuantWarps), 0, s, dim3(1, 1, 1), p.pdl, p);
    }
    const dim3 grid((unsigned)((p.q.rows + 127) / 128),
                    (unsigned)std::min<int64_t>((p.q.K + kTurnK - 1) / kTurnK, 65535));
    auto kern = back ? dequantize_any_kernel<DT, BLOCK> : quantize_any_kernel<DT, BLOCK>;
    return launch_ex(kern, grid, dim3(128), 0, s, dim3(1, 1, 1), p.pdl, p);
}

template <int DT>
cudaError_t quant_block(const QuantParams &p, int block, bool back, bool rows, bool vec, cudaStream_t s) {
    return block == 32 ? quant_run<DT, 32>(p, back, rows, vec, s) : quant_run<DT, 16>(p, back, rows, vec, s);
}

constexpr int64_t kMx4Most = (int64_t(1) << 31) - (1 << 13);

int64_t scale_tiles(int64_t K, int block) { return ((K + block - 1) / block + 3) / 4; }

// What every entry point checks of a quantised matrix, before any CUDA call.
dg_status check_mx4(const dg_mx4 *q) {
    if (q->reserved != 0 || (q->block != 16 && q->block != 32)) return DG_ERR_VALUE;
    if (q->rows < 0 || q->K < 0) return DG_ERR_SHAPE;
    if (q->rows > kMx4Most || q->K > kMx4Most) return DG_ERR_UNSUPPORTED;
    if (q->rows == 0 || q->K == 0) return DG_OK;
    if (!q->codes || !q->scales) return DG_ERR_NULL;
    int64_t t;
    if (q->code_stride < 0 || __builtin_mul_overflow(q->rows - 1, q->code_stride, &t) ||
        __builtin_add_overflow(t, (q->K + 1) / 2, &t))
        return DG_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(q->scales) % 16 || reinterpret_cast<uintptr_t>(q->scale) % 4) return DG_ERR_ALIGN;
    return DG_OK;
}

bool mx4_pointers(const dg_mx4 *q) {
    return device_pointer(q->codes) && device_pointer(q->scales) && (!q->scale || device_pointer(q->scale));
}

dg_status quant_call(const dg_view *x, const dg_mx4 *q, bool back, cudaStream_t s) {
    if (!x || !q) return DG_ERR_NULL;
    ViewInfo xi;
    dg_status st;
    if ((st = analyse(x, back, &xi)) != DG_OK || (st = check_mx4(q)) != DG_OK) return st;
    if (xi.rows != q->rows || xi.cols != q->K) return DG_ERR_SHAPE;
    if (x->dtype != DG_F32 && x->dtype != DG_F16 && x->dtype != DG_BF16) return DG_ERR_DTYPE;
    if (q->rows == 0 || q->K == 0) return DG_OK;
    if (!back && q->rows > 1 && q->code_stride < (q->K + 1) / 2) return DG_ERR_STRIDE;
    if (!device_pointer(x->ptr) || !mx4_pointers(q)) return DG_ERR_POINTER;
    int num_sms = 0;
    int *err_word = nullptr;
    if ((st = device_info(&num_sms, &err_word)) != DG_OK) return st;
    QuantParams p{};
    p.q.codes = static_cast<uint8_t *>(const_cast<void *>(q->codes));
    p.q.scales = static_cast<uint8_t *>(const_cast<void *>(q->scales));
    p.q.scale = q->scale;
    p.q.rows = q->rows;
    p.q.K = q->K;
    p.q.code_stride = q->rows > 1 ? q->code_stride : 0;
    p.q.k_tiles = scale_tiles(q->K, q->block);
    p.q.words = reinterpret_cast<uintptr_t>(q->codes) % 4 == 0 && p.q.code_stride % 4 == 0;
    p.x.ptr = static_cast<const char *>(x->ptr);
    p.x.row = xi.row;
    p.x.col = xi.col;
    p.x.dtype = x->dtype;
    p.pdl = early_launch_mode() != 0;
    // neighbours in a row go to neighbouring lanes, unless it is the rows that are neighbours
    const bool rows = !(xi.row.n >= 1 && xi.row.stride[xi.row.n - 1] == xi.es);
    const bool vec = (xi.col.n == 0 || (xi.col.n == 1 && xi.col.stride[0] == xi.es)) &&
                     reinterpret_cast<uintptr_t>(x->ptr) % 16 == 0 &&
                     (xi.row.n == 0 || (xi.row.n == 1 && xi.row.stride[0] % 16 == 0));
    const cudaError_t e = x->dtype == DG_F32   ? quant_block<DG_F32>(p, q->block, back, rows, vec, s)
                          : x->dtype == DG_F16 ? quant_block<DG_F16>(p, q->block, back, rows, vec, s)
                                               : quant_block<DG_BF16>(p, q->block, back, rows, vec, s);
    if (e != cudaSuccess) return DG_ERR_CUDA;
    count_launch();
    return DG_OK;
}

template <int BLOCK>
cudaError_t launch_mx4(Mx4Params p, const CUtensorMap &mp, const CUtensorMap &mq, const CUtensorMap &mq16, int num_sms,
                       cudaStream_t s) {
    static SmemLimit limit;
    const int q_rows = std::min(p.tile_w, (p.M + 15) / 16 * 16);
    const int most = 256 / mx4_scale_cols(BLOCK, p.tile_w);  // stages that TMEM has scale columns for
    int stages = 2;
    while (stages < most && mx4_layout(stages + 1, BLOCK, p.tile_w, q_rows).total <= 227 * 1024) ++stages;
    p.stages = stages;
    const size_t smem = mx4_layout(stages, BLOCK, p.tile_w, q_rows).total;
    const cudaError_t e = limit.ensure(mx4_kernel<BLOCK>, smem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>(num_sms, (int64_t)p.tiles_m * p.tiles_n);
    return launch_ex(mx4_kernel<BLOCK>, dim3(grid), dim3(kMx4Threads), smem, s, dim3(1, 1, 1), p.pdl, mp, mq, mq16, p,
                     q_rows);
}

bool codes_map(CUtensorMap *m, const dg_mx4 *q, int box_rows) {
    const int64_t bytes = (q->K + 1) / 2;
    const int64_t dim[2] = {bytes, q->rows}, stride[1] = {q->rows > 1 ? q->code_stride : (bytes + 15) / 16 * 16};
    const int box[2] = {128, box_rows};
    return encode_map(m, DG_E4M3, 2, q->codes, dim, stride, box, true);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_mx4_scale_bytes(int64_t rows, int64_t K, int32_t block) {
    if (rows < 0 || K < 0 || rows > kMx4Most || K > kMx4Most || (block != 16 && block != 32)) return -1;
    return (rows + 127) / 128 * scale_tiles(K, block) * 512;
}

dg_status dg_quantize_mx4(const dg_view *x, const dg_mx4 *q, void *stream) {
    return quant_call(x, q, false, static_cast<cudaStream_t>(stream));
}

dg_status dg_dequantize_mx4(const dg_mx4 *q, const dg_view *y, void *stream) {
    return quant_call(y, q, true, static_cast<cudaStream_t>(stream));
}

dg_status dg_gemm_mx4(const dg_mx4 *A, const dg_mx4 *B, const dg_view *C, float alpha, float beta,
                      const dg_epilogue *epilogue, void *stream) {
    if (!A || !B || !C) return DG_ERR_NULL;
    if (epilogue && (epilogue->activation < DG_ACT_NONE || epilogue->activation > DG_ACT_GELU_TANH ||
                     epilogue->reserved != 0))
        return DG_ERR_VALUE;
    ViewInfo ci;
    dg_status st;
    if ((st = analyse(C, true, &ci)) != DG_OK || (st = check_mx4(A)) != DG_OK || (st = check_mx4(B)) != DG_OK) return st;
    if (A->block != B->block) return DG_ERR_VALUE;
    if (A->K != B->K || ci.rows != A->rows || ci.cols != B->rows) return DG_ERR_SHAPE;
    if (C->dtype == DG_E4M3) return DG_ERR_DTYPE;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return DG_ERR_VALUE;
    if (ci.row.n > 1 || ci.col.n > 1) return DG_ERR_UNSUPPORTED;
    if (A->rows == 0 || B->rows == 0) return DG_OK;
    const bool product = alpha != 0.f && A->K > 0;
    if (product)
        for (const dg_mx4 *q : {A, B})
            if (reinterpret_cast<uintptr_t>(q->codes) % 16 || (q->rows > 1 && q->code_stride % 16)) return DG_ERR_ALIGN;
    if (product)
        for (const dg_mx4 *q : {A, B})
            if (q->rows > 1 && (q->code_stride == 0 || q->code_stride >= int64_t(1) << 40)) return DG_ERR_UNSUPPORTED;
    const float *bias = epilogue ? epilogue->bias : nullptr;
    if (!device_pointer(C->ptr) || (bias && !device_pointer(bias))) return DG_ERR_POINTER;
    if (product && (!mx4_pointers(A) || !mx4_pointers(B))) return DG_ERR_POINTER;
    int num_sms = 0;
    int *err_word = nullptr;
    if ((st = device_info(&num_sms, &err_word)) != DG_OK) return st;
    Mx4Params p{};
    p.M = (int32_t)A->rows;
    p.N = (int32_t)B->rows;
    p.K = product ? (int32_t)A->K : 0;
    p.tiles_n = (p.N + 127) / 128;
    // 256 rows a tile where that leaves no SM without one
    p.tile_w = p.M > 128 && (int64_t)p.tiles_n * ((p.M + 255) / 256) >= num_sms ? 256 : 128;
    p.tiles_m = (p.M + p.tile_w - 1) / p.tile_w;
    if ((int64_t)p.tiles_m * p.tiles_n > INT32_MAX / 2) return DG_ERR_UNSUPPORTED;
    p.k_tiles = (int32_t)scale_tiles(A->K, A->block);
    p.sa = static_cast<const uint8_t *>(A->scales);
    p.sb = static_cast<const uint8_t *>(B->scales);
    p.fa = product ? A->scale : nullptr;
    p.fb = product ? B->scale : nullptr;
    p.idesc = 1u << 7 | 1u << 10 | (A->block == 32 ? 1u << 23 : 0u) | (128u >> 7) << 27;  // E2M1 twice, M = 128
    p.out.c = static_cast<char *>(C->ptr);
    p.out.rs = ci.row.n ? ci.row.stride[0] : 0;
    p.out.cs = ci.col.n ? ci.col.stride[0] : ci.es;
    p.out.dtype = C->dtype;
    p.out.vec = p.out.cs == ci.es && reinterpret_cast<uintptr_t>(C->ptr) % 16 == 0 && p.out.rs % 16 == 0;
    p.out.alpha = alpha;
    p.out.beta = beta;
    p.out.bias_n = bias;
    p.out.act = epilogue ? epilogue->activation : DG_ACT_NONE;
    p.out.N = p.N;
    p.err_word = err_word;
    p.timeout_ns = wait_timeout_ns();
    p.stall_loader = test_stall();
    p.pdl = early_launch_mode() != 0;
    CUtensorMap mp{}, mq{}, mq16{};
    if (product && (!codes_map(&mp, B, 128) || !codes_map(&mq, A, 64) || !codes_map(&mq16, A, 16)))
        return DG_ERR_UNSUPPORTED;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = A->block == 32 ? launch_mx4<32>(p, mp, mq, mq16, num_sms, s)
                                         : launch_mx4<16>(p, mp, mq, mq16, num_sms, s);
    if (e != cudaSuccess) return DG_ERR_CUDA;
    count_launch();
    return DG_OK;
}

}  // extern "C"

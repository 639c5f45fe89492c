// 4-bit floats with block scales: dg_quantize_mx4, dg_dequantize_mx4 and
// dg_gemm_mx4 (the kernels are in mx4_quant.cu and mx4_kernel.cuh).
#include <algorithm>
#include <cmath>

#include "mx4_kernel.cuh"
#include "mx4_quant.h"

namespace dg {
namespace {

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
    const uintptr_t at = reinterpret_cast<uintptr_t>(q->codes) | (uintptr_t)p.q.code_stride;
    p.q.align = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 1;
    p.x.ptr = static_cast<const char *>(x->ptr);
    p.x.row = xi.row;
    p.x.col = xi.col;
    p.x.dtype = x->dtype;
    p.pdl = early_launch_mode() != 0;
    p.vec = reinterpret_cast<uintptr_t>(x->ptr) % 16 == 0 &&
            (xi.row.n == 0 || (xi.row.n == 1 && xi.row.stride[0] % 16 == 0));
    p.col = xi.col.n == 1 ? xi.col.stride[0] : 0;
    const cudaError_t e = launch_quant(p, q->block, back, s);
    if (e != cudaSuccess) return DG_ERR_CUDA;
    count_launch();
    return DG_OK;
}

template <int BLOCK, bool PAIR>
cudaError_t launch_mx4(Mx4Params p, const CUtensorMap (&m)[4], int q_rows, int num_sms, cudaStream_t s) {
    static SmemLimit limit;
    const int most = 256 / mx4_scale_cols(BLOCK, p.tile_w);  // stages that TMEM has scale columns for
    int stages = 2;
    while (stages < most && mx4_layout(stages + 1, BLOCK, p.tile_w, q_rows).total <= 227 * 1024) ++stages;
    p.stages = stages;
    const size_t smem = mx4_layout(stages, BLOCK, p.tile_w, q_rows).total;
    auto kern = mx4_kernel<BLOCK, PAIR>;
    const cudaError_t e = limit.ensure(kern, smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)p.tiles_m * p.tiles_n;
    const int grid = PAIR ? (int)std::min<int64_t>(num_sms & ~1, 2 * units)
                          : (int)std::min<int64_t>(num_sms, units) * p.split;
    return launch_ex(kern, dim3(grid), dim3(kMx4Threads), smem, s, dim3(PAIR ? 2 : p.split, 1, 1), p.pdl, m[0], m[1], m[2],
                     m[3], p, q_rows);
}

bool codes_map(CUtensorMap *m, const dg_mx4 *q, int box_rows) {
    const int64_t bytes = (q->K + 1) / 2;
    const int64_t dim[2] = {bytes, q->rows}, stride[1] = {q->rows > 1 ? q->code_stride : (bytes + 15) / 16 * 16};
    const int box[2] = {128, box_rows};
    return encode_map(m, DG_E4M3, 2, q->codes, dim, stride, box, true);
}

// Tiles of scales as words: 128 of a tile, tiles along k, tiles along the rows.
bool scales_map(CUtensorMap *m, const dg_mx4 *q, int box_rows) {
    const int64_t tiles = scale_tiles(q->K, q->block);
    const int64_t dim[3] = {128, tiles, (q->rows + 127) / 128}, stride[2] = {512, tiles * 512};
    const int box[3] = {128, 64 / q->block, box_rows};
    return encode_map(m, DG_F32, 3, q->scales, dim, stride, box, false);
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
    const float *bias = epilogue ? epilogue->bias : nullptr;
    if (reinterpret_cast<uintptr_t>(bias) % 4) return DG_ERR_ALIGN;
    if (ci.row.n > 1 || ci.col.n > 1) return DG_ERR_UNSUPPORTED;
    if (A->rows == 0 || B->rows == 0) return DG_OK;
    const bool product = alpha != 0.f && A->K > 0;
    if (product)
        for (const dg_mx4 *q : {A, B})
            if (reinterpret_cast<uintptr_t>(q->codes) % 16 || (q->rows > 1 && q->code_stride % 16)) return DG_ERR_ALIGN;
    if (product)
        for (const dg_mx4 *q : {A, B})
            if (q->rows > 1 && (q->code_stride == 0 || q->code_stride >= int64_t(1) << 40)) return DG_ERR_UNSUPPORTED;
    if (!device_pointer(C->ptr) || (bias && !device_pointer(bias))) return DG_ERR_POINTER;
    if (product && (!mx4_pointers(A) || !mx4_pointers(B))) return DG_ERR_POINTER;
    int num_sms = 0;
    int *err_word = nullptr;
    if ((st = device_info(&num_sms, &err_word)) != DG_OK) return st;
    Mx4Params p{};
    p.M = (int32_t)A->rows;
    p.N = (int32_t)B->rows;
    p.K = product ? (int32_t)A->K : 0;
    // Tiles of 128 x 128 per CTA, or of 256 x 256 per pair of CTAs: whichever takes less time by a model in
    // microseconds per round of the grid, 0.38 a stage and 1 a tile of a CTA, 0.42 and 2.6 of a pair (B200, CTAs
    // and pairs: 777x1000x5003 7.7 and 12.3, 300x512x20000 8.5 and 12.0, 1024x14336x4096 44.5 and 28.9,
    // 2048^3 9.7 and 9.2).
    const int steps = (p.K + kMx4K - 1) / kMx4K;
    auto rounds = [&](int64_t side, int64_t slots) {
        return (double)((((p.N + side - 1) / side) * ((p.M + side - 1) / side) + slots - 1) / slots);
    };
    const bool pair = num_sms >= 2 && p.M > 128 &&
                      rounds(256, num_sms / 2) * (0.42 * steps + 2.6) < rounds(128, num_sms) * (0.38 * steps + 1);
    p.tile_w = pair ? 256 : 128;
    p.tiles_n = pair ? (p.N + 255) / 256 : (p.N + 127) / 128;
    p.tiles_m = (p.M + p.tile_w - 1) / p.tile_w;
    const int q_rows = pair ? 128 : std::min(128, (p.M + 15) / 16 * 16);  // per CTA
    if ((int64_t)p.tiles_m * p.tiles_n > INT32_MAX / 2) return DG_ERR_UNSUPPORTED;
    // Few tiles: k over a cluster of f CTAs.  In microseconds, a stage costs 0.33 and the exchange 0.7 and
    // a tile's rows times (0.02 + 0.09 / f); clusters of eight do not fill every group of SMs.  (B200, f = 1
    // and the chosen one: 8x4096x14336 19.2 -> 10.1, 1x512x2048 4.6 -> 3.6, 128x1024x16384 25.1 -> 9.8;
    // 128x4096x4096 stays at one, 8.6 against 10.3.)
    p.split = 1;
    double least = 0.33 * steps;
    if (!pair)
        for (int f = 2; f <= 8; f *= 2) {
            const int per = (steps + f - 1) / f;
            const double room = (f == 8 ? 0.7 : 0.9) * num_sms;
            if ((double)p.tiles_m * p.tiles_n * f > room || (f - 1) * per >= steps) break;
            const double cost = 0.33 * per + 0.7 + std::min(p.M, 128) * (0.02 + 0.09 / f);
            if (cost < least) {
                least = cost;
                p.split = f;
            }
        }
    p.fa = product ? A->scale : nullptr;
    p.fb = product ? B->scale : nullptr;
    p.idesc = 1u << 7 | 1u << 10 | (A->block == 32 ? 1u << 23 : 0u) | (pair ? 2u : 1u) << 27;  // E2M1 twice, M / 128
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
    CUtensorMap m[4] = {};
    if (product && (!codes_map(&m[0], B, 128) || !codes_map(&m[1], A, q_rows) ||
                    !scales_map(&m[2], B, 1) || !scales_map(&m[3], A, p.tile_w / 128)))
        return DG_ERR_UNSUPPORTED;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // F32 C: no accumulator takes more than kMx4Part of k (the tensor core truncates as it adds); the pieces of a
    // longer sum are added in C, a launch each.  A 16-bit C could not hold them, and its own rounding is larger.
    const TurnedOut out = p.out;
    const int split = p.split;
    const int64_t K = p.K, piece = C->dtype == DG_F32 ? (int64_t)kMx4Part * split : std::max<int64_t>(K, 1);
    for (int64_t k = 0; k == 0 || k < K; k += piece) {
        p.k_from = (int32_t)k;
        p.K = (int32_t)std::min(K, k + piece);
        const int some = (p.K - p.k_from + kMx4K - 1) / kMx4K;
        // every CTA of a cluster has a part of the piece
        for (p.split = split; p.split > 1 && (some + p.split - 1) / p.split * (p.split - 1) >= some;) p.split /= 2;
        p.k_split = (some + p.split - 1) / p.split * kMx4K;
        p.out.beta = k == 0 ? out.beta : 1.f;
        p.out.bias_n = p.K == K ? out.bias_n : nullptr;
        p.out.act = p.K == K ? out.act : DG_ACT_NONE;
        const cudaError_t e =
            A->block == 32 ? (pair ? launch_mx4<32, true>(p, m, q_rows, num_sms, s) : launch_mx4<32, false>(p, m, q_rows, num_sms, s))
                           : (pair ? launch_mx4<16, true>(p, m, q_rows, num_sms, s) : launch_mx4<16, false>(p, m, q_rows, num_sms, s));
        if (e != cudaSuccess) return DG_ERR_CUDA;
        count_launch();
    }
    return DG_OK;
}

}  // extern "C"

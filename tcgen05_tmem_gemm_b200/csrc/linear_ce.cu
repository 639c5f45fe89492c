// Linear cross entropy: the loss of an output layer from its input X and
// weight W without keeping the logits, and its gradient.
//
//   z[t][v] = alpha x_t w_v,   lse[t] = log sum_v exp z[t][v],
//   loss[t] = lse[t] - z[t][target],
//   G[t][v] = dloss[t] (exp(z[t][v] - lse[t]) - (v == target)),
//   dX = alpha G W^T,  dW = alpha X^T G.
//
// The vocabulary is walked in pieces.  A row's logits of one piece are reduced
// to a pair (m, s): their maximum and sum_v exp(z - m); two pairs join as
//   m = max(m1, m2),  s = s1 exp(m1 - m) + s2 exp(m2 - m),
// so one pass over the logits is enough and none of them has to be kept.
//
// In fewer than 32 bits there is G alone: the two products of the gradients
// take it as a tensor-core operand, which is rounded to the type of X (two
// 16-bit parts would double both products).  Its rows are scaled first so that
// the rounding is relative to each entry (ce_norm_kernel, ce_rows_kernel).
// Logits, statistics and all sums are FP32.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "ce.cuh"

namespace dg {

namespace {

constexpr int kStatCols = 2048;                    // logits per block of ce_stats_kernel
constexpr int64_t kForwardPiece = int64_t(256) << 20;  // most bytes of one piece of logits (forward)
constexpr int64_t kGradPiece = int64_t(512) << 20;     // most bytes of one piece of G
constexpr int64_t kShortDim = 1024;
constexpr int kUsualSms = 148;                     // where no device is asked (workspace sizes)

constexpr int64_t kManyPlaneBlocks = 4096;         // from here on ce_planes_kernel takes four rows a block
constexpr int kPieceCols = 256;                    // pieces are whole multiples of this many columns

// One block per row and run of kStatCols columns of a piece of FP32 logits:
// the run's (m, s), and the target's logit if it lies in the run.
__global__ void __launch_bounds__(256)
    ce_stats_kernel(const float *z, int64_t ldz, int64_t T, int64_t V, int v0, int cols, int chunks,
                    const int64_t *target, int64_t ignore_index, float2 *part, float *ztarget) {
    pdl_wait_then_release();
    __shared__ float2 red[8];
    const int64_t t = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x - t * chunks);
    const float *row = z + t * ldz;
    const int c0 = chunk * kStatCols, c1 = min(cols, c0 + kStatCols);
    float v[kStatCols / 256];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kStatCols / 256; ++i) {
        const int c = c0 + threadIdx.x + 256 * i;
        v[i] = c < c1 ? row[c] : -INFINITY;
        m = fmaxf(m, v[i]);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kStatCols / 256; ++i)
        s += v[i] == -INFINITY ? 0.f : exp_fast(v[i] - m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, off), s2 = __shfl_xor_sync(0xffffffffu, s, off);
        join(m, s, m2, s2);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) join(m, s, red[w].x, red[w].y);
        part[(int64_t)chunk * T + t] = make_float2(m, s);
        const int y = read_target(target, ignore_index, V, t);
        if (y >= v0 + c0 && y < v0 + c1) ztarget[t] = row[y - v0];
    }
}

// Joins the `slots` pairs of each row of a piece, in slot order, with the
// row's pair of the earlier pieces; the last piece writes lse and loss.
// 32 rows per block; kJoinWarps warps share the slots, four loads in flight each.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    ce_join_kernel(const float2 *part, int slots, int64_t T, int64_t V, bool first, bool last, float2 *run,
                   const int64_t *target, int64_t ignore_index, const float *ztarget, float *loss, float *lse,
                   int *err_word) {
    pdl_wait_then_release();
    __shared__ float2 red[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f;
    if (t < T)
        for (int i0 = warp; i0 < slots; i0 += 4 * kJoinWarps) {
            float2 q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kJoinWarps;
                q[u] = i < slots ? part[(int64_t)i * T + t] : make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) join(m, s, q[u].x, q[u].y);
        }
    red[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp != 0 || t >= T) return;
    for (int w = 1; w < kJoinWarps; ++w) join(m, s, red[w][lane].x, red[w][lane].y);
    if (!first) join(m, s, run[t].x, run[t].y);
    if (!last) {
        run[t] = make_float2(m, s);
        return;
    }
    const float ls = logf(s);
    lse[t] = m + ls;
    const int y = read_target(target, ignore_index, V, t);
    if (y == kInvalid) {
        loss[t] = NAN;
        if (err_word) atomicCAS(err_word, 0, (int)DG_ERR_VALUE);
    } else {
        // m - z first: exact when the target is near the maximum
        loss[t] = y == kIgnored ? 0.f : (m - ztarget[t]) + ls;
    }
}

// 16-bit pieces of G: dloss is divided by the largest |dloss| of a row that
// counts, so that a gradient that is the same for all rows (a mean) is exactly
// 1 and G's -1 + p at the target is rounded next to 1, where the rounding of
// dloss * (p - 1) would shift a row as a whole.  F16 pieces are also scaled
// towards the top of F16's range (kTop), and rows of a smaller dloss each by a
// power of two more (see ce_rows_kernel): their probabilities would be
// subnormal otherwise.  norm[0] = the largest |dloss|, norm[1] = norm[0] / top,
// which the products multiply their FP32 sums by.
constexpr float kTop = 16384.f;  // |G| <= 1 times this: a factor of four below the largest F16
__device__ __forceinline__ float largest_dloss(const char *dloss, int64_t dloss_stride, const int64_t *target,
                                               int64_t ignore_index, int64_t T, int64_t V, float (&red)[32]) {
    float big = 0.f;
    for (int64_t t = threadIdx.x; t < T; t += blockDim.x) {
        if (read_target(target, ignore_index, V, t) < 0) continue;
        const float g = fabsf(*reinterpret_cast<const float *>(dloss + t * dloss_stride));
        if (g < INFINITY) big = fmaxf(big, g);
    }
    for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    if (threadIdx.x < 32) red[threadIdx.x] = 0.f;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = big;
    __syncthreads();
    big = red[threadIdx.x & 31];
    for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    // below 2^-100 the division would leave FP32's range; such gradients are scaled as far as 2^100 goes
    return big > 0.f ? fmaxf(big, 0x1p-100f) : 1.f;
}

__global__ void __launch_bounds__(1024)
    ce_norm_kernel(const char *dloss, int64_t dloss_stride, const int64_t *target, int64_t ignore_index, int64_t T,
                   int64_t V, float top, float *norm) {
    pdl_wait_then_release();
    __shared__ float red[32];
    const float big = largest_dloss(dloss, dloss_stride, target, ignore_index, T, V, red);
    if (threadIdx.x == 0) {
        norm[0] = big;
        norm[1] = big / top;
    }
}

// Copies a matrix from one pair of strides to another, 256 elements of a row
// per warp and step: a piece of W into rows that start at multiples of 128
// bytes, or a piece of dW out of them.  The products' tensor copies take no
// matrix whose rows start off a multiple of 16 bytes, and their threads' loads
// or stores of single elements cost more than this pass.
template <typename E>
__global__ void __launch_bounds__(256)
    ce_move_kernel(const char *src, int64_t sm, int64_t sn, char *dst, int64_t dm, int64_t dn, int N, int64_t units) {
    pdl_wait_then_release();
    const int64_t per = (N + 255) / 256;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * 8) {
        const int64_t row = u / per;
        const int n0 = (int)(u - row * per) * 256 + (threadIdx.x & 31);
        const char *from = src + row * sm;
        char *to = dst + row * dm;
        E v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = n0 + 32 * j < N ? *reinterpret_cast<const E *>(from + (n0 + 32 * j) * sn) : E(0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (n0 + 32 * j < N) *reinterpret_cast<E *>(to + (n0 + 32 * j) * dn) = v[j];
    }
}

// The same for rows of contiguous 2-byte elements on both sides, in words that
// are aligned in dst: a word of src that lies across two is joined from them,
// each of which holds an element of the row (233 MB in rows of 10862 bytes,
// read and written: 155 us element by element, 77 us in words, 6.1 TB/s).
__global__ void __launch_bounds__(256)
    ce_move_words_kernel(const char *src, int64_t sm, char *dst, int64_t dm, int N, int64_t units) {
    pdl_wait_then_release();
    const int64_t per = (N + 511) / 512;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * 8) {
        const int64_t row = u / per;
        const int part = (int)(u - row * per), lane = threadIdx.x & 31;
        const uint16_t *from = reinterpret_cast<const uint16_t *>(src + row * sm);
        uint16_t *to = reinterpret_cast<uint16_t *>(dst + row * dm);
        const int head = reinterpret_cast<uintptr_t>(to) % 4 ? 1 : 0, words = (N - head) / 2;
        if (part == 0 && lane == 0 && head) to[0] = from[0];
        if (part == 0 && lane == 1 && head + 2 * words < N) to[N - 1] = from[N - 1];
        const bool across = reinterpret_cast<uintptr_t>(from + head) % 4 != 0;
        const uint32_t *fw = reinterpret_cast<const uint32_t *>(from + head - (across ? 1 : 0));
        uint32_t *tw = reinterpret_cast<uint32_t *>(to + head);
        const int w0 = part * 256 + lane;
        uint32_t v[8];
        if (across) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int w = w0 + 32 * j;
                v[j] = w < words ? __funnelshift_r(fw[w], fw[w + 1], 16) : 0u;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = w0 + 32 * j < words ? fw[w0 + 32 * j] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (w0 + 32 * j < words) tw[w0 + 32 * j] = v[j];
    }
}

// One row by one block, or zeros in its place.
template <typename E>
__device__ __forceinline__ void copy_row(const char *src, int64_t step, char *dst, int D, bool zero) {
    int d = threadIdx.x;
    for (; d + 7 * (int)blockDim.x < D; d += 8 * blockDim.x) {
        E v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const E *>(src + (d + j * (int)blockDim.x) * step);
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<E *>(dst)[d + j * (int)blockDim.x] = zero ? E(0) : v[j];
    }
    for (; d < D; d += blockDim.x)
        reinterpret_cast<E *>(dst)[d] = zero ? E(0) : *reinterpret_cast<const E *>(src + d * step);
}

// Up to this many rows every block of ce_rows_kernel finds the largest dloss
// itself, which saves the launch of ce_norm_kernel.
constexpr int64_t kOwnNormRows = 2048;

// An F16 row's finite elements are below 2^(the result) in magnitude; -100 if they are all 0.
__device__ __forceinline__ int row_exponent(const DevView &x, const char *src, int D, int vec, uint32_t (&red)[8]) {
    uint32_t most = 0;
    auto meet = [&](uint32_t h) {
        h &= 0x7fffu;
        if (h < 0x7c00u) most = max(most, h);
    };
    if (vec) {
        for (int d = threadIdx.x; d < D / 8; d += blockDim.x) {
            const uint4 q = reinterpret_cast<const uint4 *>(src)[d];
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) meet(w[i]), meet(w[i] >> 16);
        }
    } else {
        for (int d = threadIdx.x; d < D; d += blockDim.x)
            meet(*reinterpret_cast<const uint16_t *>(src + axis_offset(x.col, d)));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int i = 0; i < (int)blockDim.x / 32; ++i) most = max(most, red[i]);
    int k = -100;
    if (most) frexpf(__half2float(__ushort_as_half((unsigned short)most)), &k);
    return k;
}

// An F16 row times `scale`, a power of two, by one block.
__device__ __forceinline__ void copy_row_scaled(const DevView &x, const char *src, char *dst, int D, int vec,
                                                float scale) {
    auto times = [&](uint32_t h) {
        return (uint32_t)__half_as_ushort(__float2half_rn(__half2float(__ushort_as_half((unsigned short)h)) * scale));
    };
    if (vec) {
        for (int d = threadIdx.x; d < D / 8; d += blockDim.x) {
            uint4 q = reinterpret_cast<const uint4 *>(src)[d];
            uint32_t *w = &q.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = times(w[i] & 0xffffu) | times(w[i] >> 16) << 16;
            reinterpret_cast<uint4 *>(dst)[d] = q;
        }
    } else {
        for (int d = threadIdx.x; d < D; d += blockDim.x)
            reinterpret_cast<uint16_t *>(dst)[d] =
                (uint16_t)times(*reinterpret_cast<const uint16_t *>(src + axis_offset(x.col, d)));
    }
}

// Per row: its RowGrad, and (xc != null) a copy of X's row, zero in rows that
// take no part, so that whatever those rows hold stays out of dW (xl != null:
// another one).
//
// row_undo != null (F16 pieces, a dloss per row): a row whose |dloss| is 2^e
// times the largest would have its probabilities in F16's subnormals, so G's
// row is multiplied by 2^-h, e <= h <= 0, and the factor 2^h goes to dX's row
// (row_undo[t], FP32) and, for dW's sum over the rows, to the copy of X's row
// (scale_copy).  h = e where dW is not asked for.  Else h = e + 10: G's 16 384
// times 2^-10 leaves probabilities above 2^-18 normal, and the rounding of the
// copy's small elements to multiples of 2^-24 moves dW by no more than 2^-35 of
// the largest dloss; and the copy's largest element stays at 2^-10 or above.
__global__ void __launch_bounds__(256)
    ce_rows_kernel(const DevView x, int D, int64_t T, int64_t V, const int64_t *target, int64_t ignore_index,
                   const float *lse, const char *dloss, int64_t dloss_stride, float *norm, int own_norm, float top,
                   RowGrad *rows, float *undo, int64_t undo_n, float *row_undo, int scale_copy, char *xc, char *xl, int64_t ldx, int vec,
                   int *err_word) {
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    const int y = target ? read_target(target, ignore_index, V, t) : 0;
    __shared__ float red[32];
    __shared__ uint32_t red_bits[8];
    const char *src = xc ? x.ptr + axis_offset(x.row, t) : nullptr;
    float big = 1.f;
    if (norm) {
        if (own_norm) {
            big = largest_dloss(dloss, dloss_stride, target, ignore_index, T, V, red);
            if (t == 0 && threadIdx.x == 0) {
                norm[0] = big;
                norm[1] = big / top;
            }
        } else {
            big = norm[0];
        }
    }
    int h = 0;  // the same for the whole block
    float scale = 0.f;
    if (rows && y >= 0) {
        scale = *reinterpret_cast<const float *>(dloss + t * dloss_stride);
        if (row_undo) {
            const float q = fabsf(scale) / big;
            int e = 0;
            if (q > 0.f && q < 1.f) frexpf(q, &e);
            h = max(min(e, 0), -100);
            if (scale_copy) {
                h = min(0, h + 10);
                if (h < 0) h = max(h, min(0, -9 - row_exponent(x, src, D, vec, red_bits)));
            }
        }
    }
    if (rows && threadIdx.x == 0) {
        RowGrad r;
        r.lse = lse[t];
        r.scale = norm ? ldexpf(scale, -h) / big * top : scale;
        r.target = y;
        r.pad_ = 0;
        rows[t] = r;
        if (row_undo) row_undo[t] = ldexpf(big / top, h);
        if (y == kInvalid && err_word) atomicCAS(err_word, 0, (int)DG_ERR_VALUE);
    }
    if (undo)  // the inverse for every row of the products
        for (int64_t i = t * blockDim.x + threadIdx.x; i < undo_n; i += (int64_t)gridDim.x * blockDim.x) undo[i] = big / top;
    if (!xc) return;
    auto copy = [&](char *dst) {
        if (vec) {  // 16 bytes at a time
            const int n = D * elem_bytes(x.dtype) / 16;
#pragma unroll 4
            for (int d = threadIdx.x; d < n; d += blockDim.x)
                reinterpret_cast<uint4 *>(dst)[d] =
                    y < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldcs(reinterpret_cast<const uint4 *>(src) + d);
        } else if (x.col.n == 1) {
            if (x.dtype == DG_F32) copy_row<float>(src, x.col.stride[0], dst, D, y < 0);
            else copy_row<uint16_t>(src, x.col.stride[0], dst, D, y < 0);
        } else if (x.dtype == DG_F32) {
            for (int d = threadIdx.x; d < D; d += blockDim.x)
                reinterpret_cast<float *>(dst)[d] =
                    y < 0 ? 0.f : *reinterpret_cast<const float *>(src + axis_offset(x.col, d));
        } else {
            for (int d = threadIdx.x; d < D; d += blockDim.x)
                reinterpret_cast<uint16_t *>(dst)[d] =
                    y < 0 ? 0 : *reinterpret_cast<const uint16_t *>(src + axis_offset(x.col, d));
        }
    };
    if (xl) copy(xl + t * ldx);
    if (scale_copy && h < 0) copy_row_scaled(x, src, xc + t * ldx, D, vec, ldexpf(1.f, h));
    else copy(xc + t * ldx);
}

// Up to kFewRows rows against a W whose columns are contiguous (a [V x D]
// weight): a dot product per row and column on the CUDA cores, bound by W's
// bytes (the paired tiles multiply 256 rows whatever there are).  A warp takes
// a column at a time, eight 16-byte loads a lane in flight; x is held in shared
// memory as FP32, and after the reduction over the warp lane t owns row t: its
// running (m, s), or its element of G.  Every block leaves one slot of pairs.
// 4096 x 32000 on B200: 49 us for one row (5.3 TB/s), 62 for two, 100 for four;
// the tiles take 75 for any of them.
constexpr int kFewRows = 2;
constexpr int kFewBlocks = 512;        // most blocks: slots of pairs
constexpr int kFewLoads = 8;
template <typename T, int R, bool GRAD>
__global__ void __launch_bounds__(256, 3)
    ce_few_kernel(const DevView x, const char *w, int64_t ldw, int D, int rows, int v0, int cols, float alpha,
                  const CeTile ce, char *g, int64_t ldg) {
    pdl_wait_then_release();
    extern __shared__ float xs[];  // [row][chunk of 256][half][lane][4]
    __shared__ float2 red[8][kFewRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pitch = (D + 255) / 256 * 256;
    for (int r = 0; r < R; ++r) {
        const char *row = x.ptr + axis_offset(x.row, r < rows ? r : 0);
#pragma unroll 4
        for (int d = threadIdx.x; d < pitch; d += 256) {
            const float v = r < rows && d < D ? load_elem(row + axis_offset(x.col, d), x.dtype) : 0.f;
            xs[r * pitch + (d & ~255) + ((d >> 2) & 1) * 128 + ((d >> 3) & 31) * 4 + (d & 3)] = v;
        }
    }
    __syncthreads();
    RowGrad mine{0.f, 0.f, kIgnored, 0};
    int y = kIgnored;
    if (lane < rows) {
        if (GRAD) mine = ce.rows[lane];
        else y = read_target(ce.target, ce.ignore_index, ce.V, lane);
    }
    float m = -INFINITY, s = 0.f;
    const int chunks = pitch / 256;
    for (int c = blockIdx.x * 8 + warp; c < cols; c += gridDim.x * 8) {
        const char *col = w + (int64_t)c * ldw + lane * 16;
        float acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = 0.f;
        for (int q0 = 0; q0 < chunks; q0 += kFewLoads) {
            uint4 v[kFewLoads];
#pragma unroll
            for (int q = 0; q < kFewLoads; ++q) {
                v[q] = make_uint4(0u, 0u, 0u, 0u);
                if ((q0 + q) * 256 + lane * 8 < D) v[q] = __ldcs(reinterpret_cast<const uint4 *>(col + (q0 + q) * 512));
            }
#pragma unroll
            for (int q = 0; q < kFewLoads; ++q) {
                if (q0 + q >= chunks) break;
                float f[8];
                const uint32_t h[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (sizeof(T) == 2 && __is_same(T, __nv_bfloat16)) {
                        f[2 * i] = __uint_as_float(h[i] << 16);
                        f[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
                    } else {
                        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                        f[2 * i] = t.x;
                        f[2 * i + 1] = t.y;
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 *xr = reinterpret_cast<const float4 *>(xs + r * pitch + (q0 + q) * 256) + lane;
                    const float4 a = xr[0], b = xr[32];
                    acc[r] = fmaf(a.x, f[0], acc[r]);
                    acc[r] = fmaf(a.y, f[1], acc[r]);
                    acc[r] = fmaf(a.z, f[2], acc[r]);
                    acc[r] = fmaf(a.w, f[3], acc[r]);
                    acc[r] = fmaf(b.x, f[4], acc[r]);
                    acc[r] = fmaf(b.y, f[5], acc[r]);
                    acc[r] = fmaf(b.z, f[6], acc[r]);
                    acc[r] = fmaf(b.w, f[7], acc[r]);
                }
            }
        }
        float z = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], off);
            if (lane == r) z = alpha * acc[r];
        }
        if (lane < rows) {
            if (GRAD) {
                float v = 0.f;
                if (mine.target >= 0)
                    v = mine.scale * (exp_fast(z - mine.lse) - (v0 + c == mine.target ? 1.f : 0.f));
                store_elem(g + lane * ldg + (int64_t)c * 2, x.dtype, v);
            } else {
                join(m, s, z, 1.f);
                if (y == v0 + c) ce.ztarget[lane] = z;
            }
        }
    }
    if (GRAD) return;
    if (lane < kFewRows) red[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < rows) {
        for (int i = 1; i < 8; ++i) join(m, s, red[i][lane].x, red[i][lane].y);
        ce.part[(int64_t)blockIdx.x * ce.T + lane] = make_float2(m, s);
    }
}

// A piece of FP32 logits to the piece of G.
__global__ void __launch_bounds__(256)
    ce_grad_kernel(const float *z, int64_t ldz, int64_t T, int v0, int cols, const RowGrad *rows, char *g, int64_t ldg,
                   int dtype) {
    pdl_wait_then_release();
    const int chunks = (cols + 1023) / 1024;
    const int64_t t = blockIdx.x / chunks;
    const int c0 = (int)(blockIdx.x - t * chunks) * 1024;
    const RowGrad r = rows[t];
    const int es = elem_bytes(dtype);
    for (int c = c0 + threadIdx.x; c < min(cols, c0 + 1024); c += 256) {
        float v = 0.f;
        if (r.target >= 0) v = r.scale * (exp_fast(z[t * ldz + c] - r.lse) - (v0 + c == r.target ? 1.f : 0.f));
        store_elem(g + t * ldg + (int64_t)c * es, dtype, v);
    }
}

// dX = the FP32 sum over all pieces, rounded once.
__global__ void __launch_bounds__(256) ce_round_kernel(const float *acc, int64_t ld, const DevView out, int D) {
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    char *row = const_cast<char *>(out.ptr) + axis_offset(out.row, t);
    for (int d = threadIdx.x; d < D; d += 256) store_elem(row + axis_offset(out.col, d), out.dtype, acc[t * ld + d]);
}

// dX from the planes of partial sums (FP32, in plane order) and, with several
// pieces of the vocabulary, the sum over the earlier ones: the running sum to
// acc_out, or (acc_out null) alpha * norm[1] (or row_undo) times the whole sum to dX.
// ROWS rows per block: with many rows a block's start takes longer than its loads
// (20000 x 1001, one plane: 99 -> 53 us).
template <int ROWS>
__global__ void __launch_bounds__(256)
    ce_planes_kernel(const float *planes, int64_t ld, int used, int64_t plane_rows, const float *acc_in,
                     float *acc_out, float alpha, const float *norm, const float *row_undo, const DevView out, int64_t M,
                     int D) {
    pdl_wait_then_release();
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    const int d = blockIdx.y * 256 + threadIdx.x;
    if (d >= D) return;
    const float *from = planes + t0 * ld + d;
    const int64_t step = plane_rows * ld;
    float v[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) v[r] = acc_in && t0 + r < M ? acc_in[(t0 + r) * D + d] : 0.f;
#pragma unroll (ROWS == 1 ? 8 : 2)
    for (int c = 0; c < used; ++c, from += step) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v[r] += from[r * ld];  // a plane has whole tiles of rows
    }
    const int rows = (int)(M - t0 < ROWS ? M - t0 : ROWS);
    if (acc_out) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r < rows) acc_out[(t0 + r) * D + d] = v[r];
        return;
    }
    char *to = const_cast<char *>(out.ptr) + axis_offset(out.col, d);
    float scale[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) scale[r] = alpha * (row_undo ? row_undo[t0 + (r < rows ? r : 0)] : norm[1]);
    if (out.row.n == 1) {
        to += t0 * out.row.stride[0];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r < rows) store_elem(to + r * out.row.stride[0], out.dtype, scale[r] * v[r]);
    } else {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r < rows) store_elem(to + axis_offset(out.row, t0 + r), out.dtype, scale[r] * v[r]);
    }
}

// ------------------------------------------------------------------- host side

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

dg_view view2(const void *ptr, int64_t rows, int64_t cols, int64_t rs, int64_t cs, int dtype) {
    dg_view v;
    std::memset(&v, 0, sizeof(v));
    v.ptr = const_cast<void *>(ptr);
    v.ndim = 2;
    v.row_dims = 1;
    v.shape[0] = rows;
    v.shape[1] = cols;
    v.stride[0] = rs;
    v.stride[1] = cs;
    v.dtype = dtype;
    return v;
}

// One merged dim's stride, or any legal one for an extent of 1.
int64_t stride_of(const Axis &a, int es) { return a.n == 1 ? a.stride[0] : es; }

// A matrix given by its two strides: W and dW.
struct Mat {
    char *ptr = nullptr;
    int64_t rs = 0, cs = 0;
    int dtype = 0;
};

struct Problem {
    int64_t T = 0, D = 0, V = 0;
    int es = 0;
    ViewInfo x, w, dx, dw;
    Mat wm, dwm;
    bool tensor = false;   // 16-bit operands
    bool half = false;     // F16
    bool copy_w = false;   // pieces of W are copied to a form that TMA can read
    bool place_dw = false; // pieces of dW are made in the workspace and copied to their place
    int few_slots = kFewBlocks;  // most blocks of ce_few_kernel's statistics: the pairs that the workspace holds
};

dg_status check_problem(const dg_view *X, const dg_view *W, Problem *p) {
    dg_status st;
    if (!X || !W) return DG_ERR_NULL;
    if ((st = analyse(X, false, &p->x)) != DG_OK) return st;
    if ((st = analyse(W, false, &p->w)) != DG_OK) return st;
    p->T = p->x.rows;
    p->D = p->x.cols;
    p->V = p->w.cols;
    if (p->w.rows != p->D || (p->V == 0 && p->T > 0)) return DG_ERR_SHAPE;
    if (X->dtype != W->dtype || X->dtype == DG_E4M3) return DG_ERR_DTYPE;
    p->es = elem_size(X->dtype);
    p->tensor = X->dtype != DG_F32;
    p->half = X->dtype == DG_F16;
    // the products put T and V on a grid dimension of the CUDA-core kernel
    const int64_t most = int64_t(65535) * 64;
    if (p->T > most || p->V > most || p->D > most) return DG_ERR_UNSUPPORTED;
    if (p->w.row.n > 1 || p->w.col.n > 1) return DG_ERR_UNSUPPORTED;
    p->wm = Mat{static_cast<char *>(W->ptr), stride_of(p->w.row, p->es), stride_of(p->w.col, p->es), W->dtype};
    p->copy_w = p->tensor && !p->w.tma_ok && p->D > 0 && p->V > 0;
    return DG_OK;
}

// The workspace's parts, each 256-byte aligned, for pieces of `piece` columns.
struct Layout {
    int64_t xc = 0, part = 0, run = 0, ztarget = 0, z = 0, rows = 0, norm = 0, undo = 0, g = 0, acc = 0, planes = 0;
    int64_t xl = 0, row_undo = 0;
    int64_t wc = 0, oc = 0;
    int64_t ldx = 0, ldz = 0, ldg = 0;
    int64_t total = 0;
};

int64_t take(Layout *l, int64_t bytes) {
    const int64_t at = l->total;
    l->total += align256(bytes);
    return at;
}

// X is copied when the tensor cores could not read it in place through TMA
// (a copy costs T D elements, a gathered operand slows every tile).
bool forward_copies_x(const Problem &p) { return p.tensor && !p.x.tma_ok; }

int64_t undo_count(const Problem &p) { return std::max(p.T, std::max(p.D, p.V)); }
int64_t stat_slots(int64_t piece) { return (piece + kStatCols - 1) / kStatCols; }
int64_t tile_slots(int64_t piece) { return (piece + kSlotCols - 1) / kSlotCols; }

// Whether the CTA-pair kernel makes the logits: operands (or copies of them)
// it can read through TMA, and either enough 256 x 256 tiles for its pairs of SMs, or more rows
// than the thin products' swapped tiles take, or a k so short that a round of
// tiles takes no longer than the launch it saves.  (64 columns: what the
// gradient's tensor stores take; lse and the gradient then come from the same
// logits.)
bool tiles_worth_it(const Problem &p, int num_sms) {
    return p.tensor && (p.w.tma_ok || p.copy_w) && p.V >= 64 &&
           (((p.T + 255) / 256) * ((p.V + 255) / 256) * 2 >= num_sms || p.T > 64 || p.D <= kShortDim);
}

// Whether ce_few_kernel makes the logits.
bool few_rows(const Problem &p) {
    return p.tensor && p.T <= kFewRows && p.D > 0 && p.D % 8 == 0 && p.w.unit_dim == 2 && p.w.tma_ok &&
           p.T * ((p.D + 255) / 256 * 256) * 4 <= 64 * 1024;
}

template <typename T, int R, bool GRAD>
cudaError_t run_few(const Problem &p, const DevView &x, const char *w, int v0, int cols, float alpha, const CeTile &ce,
                    char *g, int64_t ldg, int blocks, int pdl, cudaStream_t s) {
    static SmemLimit limit;
    const size_t smem = (size_t)R * ((p.D + 255) / 256 * 256) * 4;
    const cudaError_t e = limit.ensure(ce_few_kernel<T, R, GRAD>, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(ce_few_kernel<T, R, GRAD>, dim3(blocks), dim3(256), smem, s, dim3(1, 1, 1), pdl, x, w, p.wm.cs,
                     (int)p.D, (int)p.T, v0, cols, alpha, ce, g, ldg);
}

// The blocks of a launch over `cols` columns: three per SM, which is what their registers allow.
int few_blocks(const Problem &p, int64_t cols, int num_sms) {
    return (int)std::min<int64_t>((cols + 7) / 8, std::min<int64_t>(3 * num_sms, p.few_slots));
}

template <bool GRAD>
cudaError_t launch_few(const Problem &p, const DevView &x, const char *w, int v0, int cols, float alpha,
                       const CeTile &ce, char *g, int64_t ldg, int num_sms, int pdl, cudaStream_t s) {
    const int blocks = few_blocks(p, cols, num_sms);
    const bool b = x.dtype == DG_BF16;
    if (p.T == 1)
        return b ? run_few<__nv_bfloat16, 1, GRAD>(p, x, w, v0, cols, alpha, ce, g, ldg, blocks, pdl, s)
                 : run_few<__half, 1, GRAD>(p, x, w, v0, cols, alpha, ce, g, ldg, blocks, pdl, s);
    return b ? run_few<__nv_bfloat16, 2, GRAD>(p, x, w, v0, cols, alpha, ce, g, ldg, blocks, pdl, s)
             : run_few<__half, 2, GRAD>(p, x, w, v0, cols, alpha, ce, g, ldg, blocks, pdl, s);
}

// Threads per row of ce_rows_kernel: with many rows, more of them at once hide
// the chain of loads at a row's start (20000 rows of 1001 elements: 54 -> 28 us with copy_row).
int row_threads(int64_t T) { return T > kOwnNormRows ? 64 : 256; }

// 16-byte rows of X for its copy.
int x_vec(const dg_view *X, const Problem &p) {
    bool ok = p.x.col.n <= 1 && (p.x.col.n == 0 || p.x.col.stride[0] == p.es) && p.D * p.es % 16 == 0 &&
              reinterpret_cast<uintptr_t>(X->ptr) % 16 == 0;
    for (int d = 0; d < p.x.row.n; ++d) ok = ok && p.x.row.stride[d] % 16 == 0;
    return ok;
}

CeTile tile_of(const Problem &p, const int64_t *target, int64_t ignore_index, int64_t v0) {
    CeTile c{};
    c.target = target;
    c.ignore_index = ignore_index;
    c.T = p.T;
    c.V = p.V;
    c.v0 = (int32_t)v0;
    return c;
}

// How the logits are made: FP32 pieces in the workspace, tiles of the CTA-pair
// kernel, or the dot products of a few rows (the whole vocabulary at once).
enum Way { kPieces, kTiles, kFew };

// The copy of a piece of W keeps W's order if the columns are contiguous in it,
// and has each column contiguous otherwise; a single column always is.
bool copy_in_rows(const Problem &p, int64_t cols) { return p.w.unit_dim == 1 && cols > 1; }
int64_t copy_pitch(const Problem &p, int64_t cols) {
    return ((copy_in_rows(p, cols) ? cols : p.D) * p.es + 127) / 128 * 128;
}

void take_w(const Problem &p, int64_t piece, Layout *l) {
    const int64_t cols = std::min(piece, p.V);
    l->wc = take(l, p.copy_w ? (copy_in_rows(p, cols) ? p.D : cols) * copy_pitch(p, cols) : 0);
}

// Columns v0 .. v0 + cols of W, or the place of their copy.
dg_view weight_view(const Problem &p, char *ws, const Layout &l, int64_t v0, int64_t cols) {
    if (!p.copy_w) return view2(p.wm.ptr + v0 * p.wm.cs, p.D, cols, p.wm.rs, p.wm.cs, p.wm.dtype);
    const int64_t pitch = copy_pitch(p, cols);
    return copy_in_rows(p, cols) ? view2(ws + l.wc, p.D, cols, pitch, p.es, p.wm.dtype)
                                 : view2(ws + l.wc, p.D, cols, p.es, pitch, p.wm.dtype);
}

// A row of n elements of dW where its piece is made.
int64_t place_pitch(const Problem &p, int64_t n) { return (n * elem_size(p.dwm.dtype) + 127) / 128 * 128; }

dg_view transposed(dg_view v) {
    std::swap(v.shape[0], v.shape[1]);
    std::swap(v.stride[0], v.stride[1]);
    return v;
}

// An M x N matrix of 2- or 4-byte elements from one pair of strides to another.
cudaError_t launch_move(const char *src, int64_t sm, int64_t sn, char *dst, int64_t dm, int64_t dn, int es, int64_t M,
                        int64_t N, int num_sms, int pdl, cudaStream_t s) {
    const bool in_words = es == 2 && sn == 2 && dn == 2;
    const int64_t units = M * (in_words ? (N + 511) / 512 : (N + 255) / 256);
    const int64_t blocks = std::min<int64_t>((units + 7) / 8, (int64_t)num_sms * 8);
    if (in_words)
        return launch_ex(ce_move_words_kernel, dim3((unsigned)blocks), dim3(256), 0, s, dim3(1, 1, 1), pdl, src, sm, dst,
                         dm, (int)N, units);
    return launch_ex(es == 2 ? ce_move_kernel<uint16_t> : ce_move_kernel<uint32_t>, dim3((unsigned)blocks), dim3(256),
                     0, s, dim3(1, 1, 1), pdl, src, sm, sn, dst, dm, dn, (int)N, units);
}

cudaError_t copy_weight(const Problem &p, char *ws, const Layout &l, int64_t v0, int64_t cols, int num_sms, int pdl,
                        cudaStream_t s) {
    const char *src = p.wm.ptr + v0 * p.wm.cs;
    const int64_t pitch = copy_pitch(p, cols);
    if (copy_in_rows(p, cols))
        return launch_move(src, p.wm.rs, p.wm.cs, ws + l.wc, pitch, p.es, p.es, p.D, cols, num_sms, pdl, s);
    return launch_move(src, p.wm.cs, p.wm.rs, ws + l.wc, pitch, p.es, p.es, cols, p.D, num_sms, pdl, s);
}

Layout forward_layout(const Problem &p, int64_t piece, Way way) {
    Layout l;
    l.ldx = align256(p.D * p.es);
    l.ldz = align256(piece * 4);
    l.xc = take(&l, way != kFew && forward_copies_x(p) ? p.T * l.ldx : 0);
    l.part = take(&l, (way == kFew ? p.few_slots : way == kTiles ? tile_slots(piece) : stat_slots(piece)) * p.T * 8);
    l.run = take(&l, p.T * 8);
    l.ztarget = take(&l, p.T * 4);
    l.z = take(&l, way == kPieces ? p.T * l.ldz : 0);
    take_w(p, piece, &l);
    return l;
}

// The pairs of ce_few_kernel that `bytes` hold beside the rest of its layout.  The least workspace of any
// call holds some, so that its rows always take this way, as their gradient does: lse and the gradient
// come from the same logits.
int few_slots(Problem p, int64_t bytes) {
    p.few_slots = 0;
    const int64_t room = (bytes - forward_layout(p, p.V, kFew).total) / 256 * 256;
    return (int)std::max<int64_t>(0, std::min<int64_t>(kFewBlocks, room / (p.T * 8)));
}

// A product [M x K] [K x N] of few tiles and a long k (dX, whose k is the
// vocabulary, with few rows; dW, whose k is the rows, of a small layer): the
// planes of partial sums that k is split into, so that the tiles times the
// planes fill the pairs of SMs in whole rounds (0: one product without planes).
int plane_count(int64_t M, int64_t N, int64_t K, int num_sms) {
    if (N < 32) return 0;
    const int64_t pairs = num_sms / 2, tiles = ((M + 255) / 256) * ((N + 255) / 256);
    if (tiles >= 2 * num_sms) return 0;
    auto busy = [&](int64_t n) { return (double)(tiles * n) / (double)((tiles * n + pairs - 1) / pairs * pairs); };
    int best = 0;
    double most = busy(1) + 0.1;  // worth it from a tenth on: a plane costs its write and its read
    // the sum walks the planes one after another: more than 16 pay from a k of 65536 on
    // (dX of 3 x 72 from k = 118567: 49 + 5 us with 16 planes, 29 + 11 with 32, 19 + 18 with 64)
    const int limit = K >= 65536 ? 32 : 16;
    for (int n = 2; n <= limit && n * 256 <= K && tiles * n <= 4 * pairs; ++n)
        if (busy(n) - 0.005 * n > most) {
            most = busy(n) - 0.005 * n;
            best = n;
        }
    return best;
}
int64_t plane_bytes(int64_t M, int64_t N, int planes) { return planes * ((M + 255) / 256 * 256) * align256(N * 4); }

// Those of dX (for one row the GEMV over W's rows serves) and of a piece of dW.
struct Planes {
    int dx = 0, dw = 0;
};
Planes plan_planes(const Problem &p, int64_t piece, bool need_dx, bool need_dw, int num_sms) {
    Planes n;
    if (!p.tensor) return n;
    const int64_t cols = std::min(piece, p.V);
    if (need_dx && p.T > 1) n.dx = plane_count(p.T, p.D, cols, num_sms);
    // one plane for a dX whose rows the tensor stores cannot write, up to 256 MB of it
    if (need_dx && p.T > 1 && n.dx == 0 && !p.dx.tma_ok && plane_bytes(p.T, p.D, 1) <= (int64_t(256) << 20)) n.dx = 1;
    if (need_dw) n.dw = p.dw.unit_dim == 2 ? plane_count(cols, p.D, p.T, num_sms) : plane_count(p.D, cols, p.T, num_sms);
    return n;
}

Layout grad_layout(const Problem &p, int64_t piece, bool need_dx, bool need_dw, int dx_dtype, bool tiles,
                   Planes n) {
    Layout l;
    l.ldx = align256(p.D * p.es);
    l.ldz = align256(piece * 4);
    l.ldg = align256(piece * p.es);
    l.xc = take(&l, need_dw || forward_copies_x(p) ? p.T * l.ldx : 0);
    l.rows = take(&l, p.T * (int64_t)sizeof(RowGrad));
    l.norm = take(&l, 256);
    l.undo = take(&l, p.es == 2 ? undo_count(p) * 4 : 0);
    l.row_undo = take(&l, p.half ? p.T * 4 : 0);
    l.xl = take(&l, p.half && need_dw ? p.T * l.ldx : 0);
    l.acc = take(&l, need_dx && piece < p.V && (dx_dtype != DG_F32 || n.dx > 0) ? p.T * p.D * 4 : 0);
    const int64_t cols = std::min(piece, p.V);
    l.planes = take(&l, std::max(plane_bytes(p.T, p.D, n.dx),
                                 p.dw.unit_dim == 2 ? plane_bytes(cols, p.D, n.dw) : plane_bytes(p.D, cols, n.dw)));
    l.g = take(&l, p.T * l.ldg);
    l.z = take(&l, tiles ? 0 : p.T * l.ldz);
    take_w(p, piece, &l);
    if (need_dw && p.place_dw && n.dw == 0)
        l.oc = take(&l, p.dw.unit_dim == 2 ? cols * place_pitch(p, p.D) : p.D * place_pitch(p, cols));
    return l;
}

Problem without_copy(Problem p) {
    p.copy_w = p.place_dw = false;
    return p;
}

int64_t piece_min(const Problem &p) { return std::min<int64_t>(std::max<int64_t>(p.V, 1), kPieceCols); }

// Bytes of workspace that the copy of one column of W or dW takes.
int64_t copied_bytes(const Problem &p) {
    return std::max(p.copy_w ? p.D * p.es + 128 : 0, p.place_dw ? p.D * elem_size(p.dwm.dtype) + 128 : 0);
}

// Pieces of equal size, whole multiples of kPieceCols: as many columns as
// `bytes` of `per_col` bytes each allow.
int64_t piece_for(const Problem &p, int64_t bytes, int64_t per_col) {
    int64_t cols = per_col > 0 ? bytes / per_col : p.V;
    if (cols >= p.V) return std::max<int64_t>(p.V, 1);
    cols = std::max<int64_t>(cols / kPieceCols * kPieceCols, kPieceCols);
    const int64_t n = (p.V + cols - 1) / cols;
    const int64_t even = ((p.V + n - 1) / n + kPieceCols - 1) / kPieceCols * kPieceCols;
    return std::min(cols, even);
}

// The largest useful pieces: of logits, of the tiles' pairs (64 bytes of
// pairs per row and 1024 columns), of G.
int64_t forward_piece(const Problem &p, Way way) {
    if (way == kFew) return p.V;
    if (way == kPieces) return piece_for(p, kForwardPiece, std::max(p.T * 4, copied_bytes(p)));
    if (p.copy_w) return piece_for(p, kForwardPiece, std::max(p.T, copied_bytes(p)));
    const int64_t cols = kForwardPiece / (std::max<int64_t>(p.T, 1) * 8) * kSlotCols;
    return cols >= p.V ? p.V : std::max<int64_t>(cols / kPieceCols * kPieceCols, kPieceCols);
}
int64_t grad_piece(const Problem &p) { return piece_for(p, kGradPiece, std::max(p.T * p.es, copied_bytes(p))); }

dg_status launched(cudaError_t e) {
    if (e != cudaSuccess) return DG_ERR_CUDA;
    count_launch();
    return DG_OK;
}

DevView dev_of(const dg_view *v, const ViewInfo &vi) {
    DevView d{};
    d.ptr = static_cast<const char *>(v->ptr);
    d.row = vi.row;
    d.col = vi.col;
    d.dtype = v->dtype;
    return d;
}

dg_status pair_once(PairCall c, cudaStream_t s) { return pair_call(c, s); }

// The piece, made smaller until the last one has `least` columns or more; 0 or
// less if none does.
int64_t no_sliver(const Problem &p, int64_t piece, int64_t least) {
    while (piece > 0 && piece < p.V && p.V % piece != 0 && p.V % piece < least) piece -= kPieceCols;
    return piece;
}

// The largest piece whose layout fits `bytes` (0: not even the smallest).
template <typename LayoutOf>
int64_t fit_piece(const Problem &p, int64_t bytes, int64_t best, LayoutOf layout_of) {
    int64_t piece = best;
    while (layout_of(piece).total > bytes) {
        if (piece <= piece_min(p)) return 0;
        const int64_t half = (piece / 2 + kPieceCols - 1) / kPieceCols * kPieceCols;
        piece = std::max(piece_min(p), std::min(half, piece - 1));
    }
    return piece;
}

}  // namespace

}  // namespace dg

using namespace dg;

#define DG_TRY(call)                         \
    do {                                     \
        const dg_status st_ = (call);        \
        if (st_ != DG_OK) return st_;        \
    } while (0)

extern "C" {

dg_status dg_linear_ce_workspace(const dg_view *X, const dg_view *W, int64_t *least, int64_t *best) {
    if (!least || !best) return DG_ERR_NULL;
    Problem p;
    DG_TRY(check_problem(X, W, &p));
    const Way way = few_rows(p) ? kFew : tiles_worth_it(p, kUsualSms) ? kTiles : kPieces;
    *least = forward_layout(without_copy(p), piece_min(p), kPieces).total;
    *best = std::max(forward_layout(p, piece_min(p), kPieces).total, forward_layout(p, forward_piece(p, way), way).total);
    return DG_OK;
}

dg_status dg_linear_ce(const dg_view *X, const dg_view *W, const int64_t *target, int64_t ignore_index, float alpha,
                       float *loss, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    Problem p;
    DG_TRY(check_problem(X, W, &p));
    if (!std::isfinite(alpha)) return DG_ERR_VALUE;
    if (p.T == 0) return DG_OK;
    if (!target || !loss || !lse || !workspace) return DG_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(target) % 8 || reinterpret_cast<uintptr_t>(loss) % 4 ||
        reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
        return DG_ERR_ALIGN;
    if (forward_layout(p, piece_min(p), kPieces).total > workspace_bytes) p = without_copy(p);  // no room for it
    if (forward_layout(p, piece_min(p), kPieces).total > workspace_bytes) return DG_ERR_SHAPE;
    int num_sms = 0, *err_word = nullptr;
    DG_TRY(device_info(&num_sms, &err_word));
    if ((p.D > 0 && (!device_pointer(X->ptr) || !device_pointer(W->ptr))) || !device_pointer(target) ||
        !device_pointer(loss) || !device_pointer(lse) || !device_pointer(workspace))
        return DG_ERR_POINTER;
    char *ws = static_cast<char *>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int pdl = early_launch_mode() != 0;
    const dim3 one(1, 1, 1);
    // the copy of X, if there is one, comes first in the workspace
    const dg_view xv = forward_copies_x(p) ? view2(ws, p.T, p.D, align256(p.D * p.es), p.es, X->dtype) : *X;
    Way way = kPieces;
    int64_t tile_piece = 0;
    if (few_rows(p)) p.few_slots = few_slots(p, workspace_bytes);
    if (few_rows(p) && p.few_slots > 0) {
        way = kFew;
    } else if (tiles_worth_it(p, num_sms)) {
        CeTile ce = tile_of(p, target, ignore_index, 0);
        ce.part = reinterpret_cast<float2 *>(ws);
        // TMA reads no single column of a W whose columns are contiguous
        const int64_t cols = no_sliver(
            p, fit_piece(p, workspace_bytes, forward_piece(p, kTiles),
                         [&](int64_t n) { return forward_layout(p, n, kTiles); }), 2);
        if (cols > 0) {
            tile_piece = cols;
            const dg_view wv = weight_view(p, ws, forward_layout(p, cols, kTiles), 0, std::min(cols, p.V));
            if (pair_once(PairCall{&xv, &wv, nullptr, alpha, nullptr, kPairStats, ce, 0, true}, s) == DG_OK) way = kTiles;
        }
    }
    auto layout_of = [&](int64_t piece) { return forward_layout(p, piece, way); };
    const int64_t piece =
        way == kTiles ? tile_piece : fit_piece(p, workspace_bytes, forward_piece(p, way), layout_of);
    if (piece == 0) return DG_ERR_SHAPE;
    const Layout l = layout_of(piece);
    if (way != kFew && forward_copies_x(p)) {
        DG_TRY(launched(launch_ex(ce_rows_kernel, dim3((unsigned)p.T), dim3(row_threads(p.T)), 0, s, one, pdl, dev_of(X, p.x),
                                  (int)p.D, p.T, p.V, (const int64_t *)nullptr, ignore_index, (const float *)nullptr,
                                  (const char *)nullptr, (int64_t)0, (float *)nullptr, 0, 1.f, (RowGrad *)nullptr,
                                  (float *)nullptr, (int64_t)0, (float *)nullptr, 0, ws + l.xc, (char *)nullptr, l.ldx, x_vec(X, p), (int *)nullptr)));
    }
    float2 *part = reinterpret_cast<float2 *>(ws + l.part), *run = reinterpret_cast<float2 *>(ws + l.run);
    float *ztarget = reinterpret_cast<float *>(ws + l.ztarget), *z = reinterpret_cast<float *>(ws + l.z);
    for (int64_t v0 = 0; v0 < p.V; v0 += piece) {
        const int64_t cols = std::min(piece, p.V - v0);
        const dg_view wv = weight_view(p, ws, l, v0, cols);
        if (p.copy_w) DG_TRY(launched(copy_weight(p, ws, l, v0, cols, num_sms, pdl, s)));
        const dg_view zv = view2(z, p.T, cols, l.ldz, 4, DG_F32);
        int slots;
        if (way == kFew) {
            CeTile ce = tile_of(p, target, ignore_index, v0);
            ce.part = part;
            ce.ztarget = ztarget;
            DG_TRY(launched(launch_few<false>(p, dev_of(X, p.x), p.wm.ptr, 0, (int)cols, alpha, ce, nullptr, 0, num_sms,
                                              pdl, s)));
            slots = few_blocks(p, cols, num_sms);
        } else if (way == kTiles) {
            CeTile ce = tile_of(p, target, ignore_index, v0);
            ce.part = part;
            ce.ztarget = ztarget;
            DG_TRY(pair_once(PairCall{&xv, &wv, nullptr, alpha, nullptr, kPairStats, ce, 0, false}, s));
            slots = (int)tile_slots(cols);
        } else {
            DG_TRY(gemm_tiles(&xv, &wv, &zv, alpha, 0.f, nullptr, s));
            slots = (int)stat_slots(cols);
            DG_TRY(launched(launch_ex(ce_stats_kernel, dim3((unsigned)(p.T * slots)), dim3(256), 0, s, one, pdl,
                                      (const float *)z, l.ldz / 4, p.T, p.V, (int)v0, (int)cols, slots, target,
                                      ignore_index, part, ztarget)));
        }
        DG_TRY(launched(launch_ex(ce_join_kernel, dim3((unsigned)((p.T + 31) / 32)), dim3(32 * kJoinWarps), 0, s, one, pdl,
                                  (const float2 *)part, slots, p.T, p.V, v0 == 0, v0 + cols == p.V, run, target,
                                  ignore_index, (const float *)ztarget, loss, lse, err_word)));
    }
    return DG_OK;
}

}  // extern "C"

namespace dg {
namespace {

dg_status check_grad(const dg_view *X, const dg_view *W, const dg_view *dX, const dg_view *dW, Problem *p) {
    DG_TRY(check_problem(X, W, p));
    if (dX) {
        DG_TRY(analyse(dX, true, &p->dx));
        if (p->dx.rows != p->T || p->dx.cols != p->D) return DG_ERR_SHAPE;
        if (dX->dtype == DG_E4M3) return DG_ERR_DTYPE;
    }
    if (dW) {
        DG_TRY(analyse(dW, true, &p->dw));
        if (p->dw.rows != p->D || p->dw.cols != p->V) return DG_ERR_SHAPE;
        if (dW->dtype == DG_E4M3) return DG_ERR_DTYPE;
        if (p->dw.row.n > 1 || p->dw.col.n > 1) return DG_ERR_UNSUPPORTED;
        const int es = elem_size(dW->dtype);
        p->dwm = Mat{static_cast<char *>(dW->ptr), stride_of(p->dw.row, es), stride_of(p->dw.col, es), dW->dtype};
        p->place_dw = p->tensor && !p->dw.tma_ok && p->D > 0 && p->V > 0;
    }
    return DG_OK;
}

// call's product in planes at `planes`; on return call.chunks is the number written.
dg_status in_planes(PairCall &call, char *planes, cudaStream_t s) {
    const int64_t M = call.A->shape[0], N = call.B->shape[1], rows = call.chunks * ((M + 255) / 256 * 256);
    const dg_view pv = view2(planes, rows, N, align256(N * 4), 4, DG_F32);
    call.C = &pv;
    const dg_status st = pair_call(call, s);
    call.C = nullptr;
    return st;
}

// alpha * norm[1] (or row_undo) times the product through planes, to `out` or (acc_out) to the running sum.
dg_status planes_product(PairCall call, char *planes, const DevView &out, const float *acc_in, float *acc_out,
                         float alpha, const float *norm, const float *row_undo, int pdl, cudaStream_t s) {
    const int64_t M = call.A->shape[0], N = call.B->shape[1];
    DG_TRY(in_planes(call, planes, s));
    const int rows = M * ((N + 255) / 256) >= kManyPlaneBlocks ? 4 : 1;
    return launched(launch_ex(rows == 4 ? ce_planes_kernel<4> : ce_planes_kernel<1>,
                              dim3((unsigned)((M + rows - 1) / rows), (unsigned)((N + 255) / 256)), dim3(256), 0, s,
                              dim3(1, 1, 1), pdl, reinterpret_cast<const float *>(planes), align256(N * 4) / 4,
                              call.chunks, (M + 255) / 256 * 256, acc_in, acc_out, alpha, norm, row_undo, out, M, (int)N));
}

// dW's product, k = T.  Few tiles: planes, or the paired tiles all the same
// (the single-CTA kernel's split of k takes 48 us for 120 x 1024 x 4000, a
// round of paired tiles 11).  Many tiles with few rows: the stores of the large
// output take longer than the products, and get twice the epilogue warps
// (32000 x 64 x 4096: 93 -> 85 us; slower from k = 777 on).
dg_status product(const dg_view *A, const dg_view *B, const dg_view *C, const Problem &p, int num_sms, int planes,
                  char *plane_space, float alpha, const float *norm, const float *undo, int pdl, cudaStream_t s) {
    const int64_t tiles = ((A->shape[0] + 255) / 256) * ((B->shape[1] + 255) / 256);
    if (p.tensor && alpha != 0.f) {
        dg_status st = DG_ERR_UNSUPPORTED;
        if (planes > 0 && B->shape[1] < (int64_t)65535 * 256) {
            ViewInfo ci;
            DG_TRY(analyse(C, true, &ci));
            st = planes_product(PairCall{A, B, nullptr, 1.f, nullptr, kPairPartial, {}, planes, false}, plane_space,
                                dev_of(C, ci), nullptr, nullptr, alpha, norm, nullptr, pdl, s);
        }
        if (st == DG_ERR_UNSUPPORTED && (tiles * 2 < num_sms || p.T <= 256)) {
            PairCall call{A, B, C, alpha, undo, kPairWide, {}, 0, false};
            st = pair_call(call, s);
        }
        if (st != DG_ERR_UNSUPPORTED) return st;
    }
    return gemm_tiles(A, B, C, alpha, 0.f, undo, s);
}

}  // namespace
}  // namespace dg

extern "C" {

dg_status dg_linear_ce_grad_workspace(const dg_view *X, const dg_view *W, const dg_view *dX, const dg_view *dW,
                                      int64_t *least, int64_t *best) {
    if (!least || !best) return DG_ERR_NULL;
    Problem p;
    DG_TRY(check_grad(X, W, dX, dW, &p));
    const int dxt = dX ? dX->dtype : DG_F32;
    *least = grad_layout(without_copy(p), piece_min(p), dX != nullptr, dW != nullptr, dxt, false, Planes{}).total;
    *best = std::max(grad_layout(p, piece_min(p), dX != nullptr, dW != nullptr, dxt, false, Planes{}).total,
                     grad_layout(p, grad_piece(p), dX != nullptr, dW != nullptr, dxt,
                                         few_rows(p) || tiles_worth_it(p, kUsualSms),
                                         plan_planes(p, grad_piece(p), dX != nullptr, dW != nullptr, kUsualSms))
                                 .total);
    return DG_OK;
}

dg_status dg_linear_ce_grad(const dg_view *X, const dg_view *W, const int64_t *target, int64_t ignore_index,
                            float alpha, const float *lse, const float *dloss, int64_t dloss_stride, const dg_view *dX,
                            const dg_view *dW, void *workspace, int64_t workspace_bytes, void *stream) {
    Problem p;
    DG_TRY(check_grad(X, W, dX, dW, &p));
    if (!std::isfinite(alpha)) return DG_ERR_VALUE;
    if (!dX && !dW) return DG_ERR_NULL;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int pdl = early_launch_mode() != 0;
    const dim3 one(1, 1, 1);
    int num_sms = 0, *err_word = nullptr;
    if (p.T > 0) {
        if (!target || !lse || !dloss || !workspace) return DG_ERR_NULL;
        if (dloss_stride != 0 && dloss_stride != 4) return DG_ERR_STRIDE;
        if (reinterpret_cast<uintptr_t>(target) % 8 || reinterpret_cast<uintptr_t>(dloss) % 4 ||
            reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
            return DG_ERR_ALIGN;
    }
    const int dxt = dX ? dX->dtype : DG_F32;
    const auto least = [&] {
        return grad_layout(p, piece_min(p), dX != nullptr, dW != nullptr, dxt, false, Planes{}).total;
    };
    if (p.T > 0 && least() > workspace_bytes) p = without_copy(p);  // no room for copies
    if (p.T > 0 && least() > workspace_bytes) return DG_ERR_SHAPE;
    DG_TRY(device_info(&num_sms, &err_word));
    if (p.T > 0 && ((p.D > 0 && (!device_pointer(X->ptr) || !device_pointer(W->ptr))) || !device_pointer(target) ||
                    !device_pointer(lse) || !device_pointer(dloss) || !device_pointer(workspace)))
        return DG_ERR_POINTER;
    if (p.D > 0 && p.T > 0 && dX && !device_pointer(dX->ptr)) return DG_ERR_POINTER;
    if (p.D > 0 && p.V > 0 && dW && !device_pointer(dW->ptr)) return DG_ERR_POINTER;
    if (p.D == 0 || p.V == 0) return DG_OK;  // no gradient has an element
    if (p.T == 0) {
        if (!dW) return DG_OK;
        return launched(launch_scale_c(dev_of(dW, p.dw), p.D, p.V, 0.f, nullptr, DG_ACT_NONE, pdl, s));
    }
    char *ws = static_cast<char *>(workspace);
    // a row that takes no part has no use for its logits, so dW's copy of X serves them too; it
    // comes first in the workspace.  An F16 copy whose rows may be scaled does not: the logits get their own
    const bool copy = dW != nullptr || forward_copies_x(p), own_logits = p.half && dW && dloss_stride != 0;
    const int64_t ldx = align256(p.D * p.es);
    const dg_view xv = copy ? view2(ws, p.T, p.D, ldx, p.es, X->dtype) : *X;
    const dg_view xt = view2(ws, p.D, p.T, p.es, ldx, X->dtype);
    dg_view zx = xv;  // what the logits are made of (its place is known with the layout)
    const bool few = few_rows(p);
    bool tiles = few || tiles_worth_it(p, num_sms);  // no FP32 logits in the workspace
    Planes planes = plan_planes(p, grad_piece(p), dX != nullptr, dW != nullptr, num_sms);
    auto layout_of = [&](int64_t piece) {
        return grad_layout(p, piece, dX != nullptr, dW != nullptr, dxt, tiles, planes);
    };
    if (layout_of(grad_piece(p)).total > workspace_bytes) planes = Planes{};  // a small workspace has room for G only
    int64_t piece = fit_piece(p, workspace_bytes, grad_piece(p), layout_of);
    if (tiles || planes.dx > 0) {
        // the tensor copies of G take pieces of 64 columns or more, the last one too
        piece = no_sliver(p, piece, 64);
        if (piece <= 0) planes = Planes{};
    }
    if (tiles && !few) {
        if (piece > 0) {
            const Layout t = layout_of(piece);
            const dg_view gv = view2(ws + t.g, p.T, std::min(piece, p.V), t.ldg, p.es, X->dtype);
            const dg_view wv = weight_view(p, ws, t, 0, std::min(piece, p.V));
            tiles = pair_once(PairCall{&zx, &wv, &gv, alpha, nullptr, kPairGrad, {}, 0, true}, s) == DG_OK;
        }
        if (piece <= 0 || !tiles) {
            tiles = false;
            piece = planes.dx > 0 ? no_sliver(p, fit_piece(p, workspace_bytes, grad_piece(p), layout_of), 64) : 0;
            if (piece <= 0) planes = Planes{};
        }
    }
    if (piece <= 0) piece = fit_piece(p, workspace_bytes, grad_piece(p), layout_of);
    if (piece == 0) return DG_ERR_SHAPE;
    if (planes.dx > 0) {
        const Layout t = layout_of(piece);
        const int64_t cols = std::min(piece, p.V);
        const dg_view gv = view2(ws + t.g, p.T, cols, t.ldg, p.es, X->dtype);
        const dg_view wt = transposed(weight_view(p, ws, t, 0, cols));
        PairCall call{&gv, &wt, nullptr, 1.f, nullptr, kPairPartial, {}, planes.dx, true};
        if (in_planes(call, ws + t.planes, s) != DG_OK) planes.dx = 0;
    }
    const Layout l = layout_of(piece);
    RowGrad *rows = reinterpret_cast<RowGrad *>(ws + l.rows);
    float *norm = nullptr, *undo = nullptr, *row_undo = nullptr;
    const float top = p.half ? kTop : 1.f;
    if (p.half && dloss_stride != 0) row_undo = reinterpret_cast<float *>(ws + l.row_undo);
    if (own_logits) zx.ptr = ws + l.xl;
    if (p.tensor) {
        norm = reinterpret_cast<float *>(ws + l.norm);
        undo = reinterpret_cast<float *>(ws + l.undo);
        if (p.T > kOwnNormRows)
            DG_TRY(launched(launch_ex(ce_norm_kernel, one, dim3(1024), 0, s, one, pdl,
                                      reinterpret_cast<const char *>(dloss), dloss_stride, target, ignore_index, p.T,
                                      p.V, top, norm)));
    }
    DG_TRY(launched(launch_ex(ce_rows_kernel, dim3((unsigned)p.T), dim3(row_threads(p.T)), 0, s, one, pdl, dev_of(X, p.x), (int)p.D,
                              p.T, p.V, target, ignore_index, lse, reinterpret_cast<const char *>(dloss), dloss_stride,
                              norm, p.T <= kOwnNormRows ? 1 : 0, top, rows, undo, undo_count(p), row_undo,
                              own_logits ? 1 : 0,
                              copy ? ws : (char *)nullptr, own_logits && !few ? ws + l.xl : (char *)nullptr, ldx,
                              x_vec(X, p), err_word)));
    char *g = ws + l.g;
    float *z = reinterpret_cast<float *>(ws + l.z);
    const bool sum = dX && piece < p.V;                        // dX is summed over several pieces
    const bool own_acc = sum && planes.dx == 0 && dxt != DG_F32;  // in the workspace, rounded at the end
    float *acc = reinterpret_cast<float *>(ws + l.acc);
    const dg_view accv = own_acc ? view2(ws + l.acc, p.T, p.D, p.D * 4, 4, DG_F32) : (dX ? *dX : xv);
    for (int64_t v0 = 0; v0 < p.V; v0 += piece) {
        const int64_t cols = std::min(piece, p.V - v0);
        char *wp = p.wm.ptr + v0 * p.wm.cs;
        const dg_view wv = weight_view(p, ws, l, v0, cols);
        const dg_view wt = transposed(wv);
        if (p.copy_w) DG_TRY(launched(copy_weight(p, ws, l, v0, cols, num_sms, pdl, s)));
        const dg_view gv = view2(g, p.T, cols, l.ldg, p.es, X->dtype);
        const dg_view gt = view2(g, cols, p.T, p.es, l.ldg, X->dtype);
        if (few) {
            CeTile ce = tile_of(p, target, ignore_index, v0);
            ce.rows = rows;
            DG_TRY(launched(launch_few<true>(p, dev_of(X, p.x), wp, (int)v0, (int)cols, alpha, ce, g, l.ldg, num_sms,
                                             pdl, s)));
        } else if (tiles) {
            CeTile ce = tile_of(p, target, ignore_index, v0);
            ce.rows = rows;
            DG_TRY(pair_once(PairCall{&zx, &wv, &gv, alpha, nullptr, kPairGrad, ce, 0, false}, s));
        } else {
            const dg_view zv = view2(z, p.T, cols, l.ldz, 4, DG_F32);
            DG_TRY(gemm_tiles(&zx, &wv, &zv, alpha, 0.f, nullptr, s));
            const int64_t blocks = p.T * ((cols + 1023) / 1024);
            DG_TRY(launched(launch_ex(ce_grad_kernel, dim3((unsigned)blocks), dim3(256), 0, s, one, pdl,
                                      (const float *)z, l.ldz / 4, p.T, (int)v0, (int)cols, (const RowGrad *)rows, g,
                                      l.ldg, X->dtype)));
        }
        if (dX && planes.dx > 0) {
            const bool first = v0 == 0, last = v0 + cols == p.V;
            DG_TRY(planes_product(PairCall{&gv, &wt, nullptr, 1.f, nullptr, kPairPartial, {}, planes.dx, false},
                                  ws + l.planes, dev_of(dX, p.dx), first ? nullptr : acc, last ? nullptr : acc, alpha,
                                  norm, row_undo, pdl, s));
        } else if (dX) {
            DG_TRY(gemm_tiles(&gv, &wt, &accv, alpha, v0 == 0 ? 0.f : 1.f, row_undo ? row_undo : undo, s));
        }
        if (dW) {
            // the product in the order that gives dW's unit stride to the columns of the output
            char *op = p.dwm.ptr + v0 * p.dwm.cs;
            const bool cols_first = p.dw.unit_dim == 2;
            const int64_t M = cols_first ? cols : p.D, N = cols_first ? p.D : cols;
            const int64_t sm = cols_first ? p.dwm.cs : p.dwm.rs, sn = cols_first ? p.dwm.rs : p.dwm.cs;
            const int des = elem_size(p.dwm.dtype);
            const bool place = p.place_dw && planes.dw == 0;
            const dg_view ov = place ? view2(ws + l.oc, M, N, place_pitch(p, N), des, p.dwm.dtype)
                                     : view2(op, M, N, sm, sn, p.dwm.dtype);
            DG_TRY(product(cols_first ? &gt : &xt, cols_first ? &xv : &gv, &ov, p, num_sms, planes.dw, ws + l.planes,
                           alpha, norm, undo, pdl, s));
            if (place)
                DG_TRY(launched(launch_move(ws + l.oc, place_pitch(p, N), des, op, sm, sn, des, M, N, num_sms, pdl, s)));
        }
    }
    if (own_acc)
        DG_TRY(launched(launch_ex(ce_round_kernel, dim3((unsigned)p.T), dim3(256), 0, s, one, pdl,
                                  reinterpret_cast<const float *>(ws + l.acc), p.D, dev_of(dX, p.dx), (int)p.D)));
    return DG_OK;
}

}  // extern "C"

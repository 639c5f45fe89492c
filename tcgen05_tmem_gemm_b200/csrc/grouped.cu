// dg_gemm_grouped and dg_gemm_grouped_dw: products of groups of rows whose
// sizes are on the device.  grouped_kernel.cuh has the tensor-core kernel;
// operands that no tensor map describes (FP32, rows at odd addresses, several
// dims) take the CUDA-core kernel here.
#include <algorithm>
#include <climits>
#include <cmath>

#include "grouped_kernel.cuh"

namespace dg {
namespace {

// ------------------------------------------------------------- any operands

// Tiles of 64 x 64, every element addressed through its view.
struct GroupedAnyParams {
    const int64_t *offsets;
    int32_t groups, R, K, Mo, N;
    int32_t tiles_m;            // by k: tiles of C's rows
    DevView a, b, c;
    float alpha, beta;
    const float *scale_r, *scale_n, *bias;
    int32_t act;
    int *err_word;
    int32_t pdl;
};

constexpr int kAnyTile = 64, kAnyK = 16;

template <bool BYK>
__global__ void __launch_bounds__(256) grouped_any_kernel(const GroupedAnyParams p) {
    pdl_wait_then_release();
    extern __shared__ int any_table[];
    int *start = any_table, *size = start + p.groups, *before = size + p.groups;
    __shared__ float As[kAnyK][kAnyTile + 4], Bs[kAnyK][kAnyTile + 4];
    const bool bad = __syncthreads_or(
        group_tables(p.offsets, p.groups, p.R, blockIdx.x == 0 && blockIdx.y == 0 ? p.err_word : nullptr, start, size));
    int g, r0, rows, k0, K;
    if (BYK) {
        g = blockIdx.x / p.tiles_m;
        r0 = (blockIdx.x - g * p.tiles_m) * kAnyTile;
        rows = min(kAnyTile, p.Mo - r0);
        k0 = start[g];
        K = p.K == 0 ? 0 : size[g];
    } else {
        if (threadIdx.x < 32) {
            if (bad) group_disjoint(start, size, p.groups, threadIdx.x);
            group_scan(size, before, p.groups, kAnyTile, threadIdx.x);
        }
        __syncthreads();
        const int u = blockIdx.x;
        if (u >= before[p.groups]) return;
        int lo = 0, hi = p.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= u) lo = mid;
            else hi = mid;
        }
        g = lo;
        r0 = (u - before[g]) * kAnyTile;
        rows = min(kAnyTile, size[g] - r0);
        r0 += start[g];
        k0 = 0;
        K = p.K;
    }
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // 4 x 4 outputs each
    for (int64_t n0 = (int64_t)blockIdx.y * kAnyTile; n0 < p.N; n0 += (int64_t)gridDim.y * kAnyTile) {
        const int cols = (int)min((int64_t)kAnyTile, p.N - n0);
        float acc[4][4] = {};
        for (int k = 0; k < K; k += kAnyK) {
            __syncthreads();
            for (int e = threadIdx.x; e < kAnyK * kAnyTile; e += 256) {
                const int kk = e / kAnyTile, i = e % kAnyTile;
                float a = 0.f, b = 0.f;
                if (k + kk < K) {
                    const int64_t at = (int64_t)k0 + k + kk;
                    if (i < rows)
                        a = load_elem(p.a.ptr + (BYK ? axis_offset(p.a.row, at) + axis_offset(p.a.col, r0 + i)
                                                     : axis_offset(p.a.row, r0 + i) + axis_offset(p.a.col, at)),
                                      p.a.dtype);
                    if (i < cols)
                        b = load_elem(p.b.ptr + axis_offset(p.b.row, BYK ? at : (int64_t)g * p.K + at) +
                                          axis_offset(p.b.col, n0 + i),
                                      p.b.dtype);
                }
                As[kk][i] = a;
                Bs[kk][i] = b;
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kAnyK; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(As[kk][ty * 4 + i], Bs[kk][tx + 16 * j], acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = ty * 4 + i;
            if (row >= rows) continue;
            char *cr = const_cast<char *>(p.c.ptr) +
                       axis_offset(p.c.row, BYK ? (int64_t)g * p.Mo + r0 + row : (int64_t)r0 + row);
            const float sr = p.scale_r ? p.scale_r[r0 + row] : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + tx + 16 * j;
                if (n >= p.N) continue;
                char *cp = cr + axis_offset(p.c.col, n);
                const float sn = p.scale_n ? p.scale_n[(int64_t)g * p.N + n] : 1.f;
                float v = epi_value(acc[i][j], p.alpha * sn, sr, p.beta, cp, p.c.dtype);
                if (p.bias != nullptr || p.act != DG_ACT_NONE)
                    v = epi_fuse(v, p.bias, (int64_t)g * p.N + n, p.act, p.c.dtype != DG_F32);
                store_elem(cp, p.c.dtype, v);
            }
        }
    }
}

// --------------------------------------------------------------- the launches

// What both entry points have in common, after their checks.
struct GroupedCall {
    bool by_k;
    const dg_view *a, *b, *c;  // by rows: A, B, C; by k: X, dY, dW
    ViewInfo ai, bi, ci;
    const int64_t *offsets;
    int32_t groups;
    int64_t R, K, N, Mo;
    float alpha, beta;
    const float *scale_r, *scale_n, *bias;
    int act;
};

DevView dev_of(const dg_view *v, const ViewInfo &vi) {
    DevView d{};
    d.ptr = static_cast<const char *>(v->ptr);
    d.row = vi.row;
    d.col = vi.col;
    d.dtype = v->dtype;
    return d;
}

int64_t one_stride(const Axis &a) { return a.n == 1 ? a.stride[0] : 0; }

constexpr int64_t kMapStride = int64_t(1) << 40;

// A matrix that a tensor map describes along its columns: unit stride along
// them, rows at multiples of 16 bytes.
bool rows_map_ok(const dg_view *v, const ViewInfo &vi) {
    if (vi.row.n > 1 || vi.col.n > 1 || (vi.col.n == 1 && vi.col.stride[0] != vi.es)) return false;
    if (reinterpret_cast<uintptr_t>(v->ptr) % 16) return false;
    return vi.row.n == 0 || (vi.row.stride[0] > 0 && vi.row.stride[0] % 16 == 0 && vi.row.stride[0] < kMapStride);
}

// The stride for a dim of one element: any that a map takes.
int64_t map_stride(int64_t stride, int64_t inner_bytes) { return stride > 0 ? stride : (inner_bytes + 15) / 16 * 16; }

// By rows: B [group, K, N] as a map, along K (mn false) or along N.
bool b_map(const GroupedCall &c, bool mn, int ksub, GroupedParams *p, CUtensorMap *m) {
    const int es = c.ai.es, inner = mn ? 2 : 1, outer = mn ? 1 : 2;  // dims of the view
    const int64_t *shape = c.b->shape, *st = c.b->stride;
    if (reinterpret_cast<uintptr_t>(c.b->ptr) % 16) return false;
    if (shape[inner] > 1 && st[inner] != es) return false;
    const bool many = shape[outer] > 1, groups = shape[0] > 1 && st[0] > 0;
    for (int d : {outer, 0})
        if ((d == 0 ? groups : many) && (st[d] <= 0 || st[d] % 16 || st[d] >= kMapStride)) return false;
    p->p_one_g = groups ? 0 : 1;
    const int64_t os = map_stride(many ? st[outer] : 0, shape[inner] * es);
    const int64_t gs = groups ? st[0] : os * std::max<int64_t>(1, shape[outer]);
    if (gs >= kMapStride) return false;
    // the larger stride last, and a whole number of the smaller one
    p->p_swap_g = gs < os;
    if (std::max(gs, os) % std::min(gs, os)) return false;
    const int box_outer = mn ? ksub * 128 / es : kPRows;
    const int64_t n_groups = groups ? shape[0] : 1;
    const int64_t dim[3] = {shape[inner], p->p_swap_g ? n_groups : shape[outer], p->p_swap_g ? shape[outer] : n_groups};
    const int64_t stride[2] = {std::min(gs, os), std::max(gs, os)};
    const int box[3] = {128 / es, p->p_swap_g ? 1 : box_outer, p->p_swap_g ? box_outer : 1};
    return encode_map(m, c.b->dtype, 3, c.b->ptr, dim, stride, box, true);
}

// By k: rows as two dims of one stride, the inner one as long as a box of h
// rows (see grouped_kernel.cuh); or, for h = 1, plain rows.  Only for R >= h.
bool cut_map(const dg_view *v, const ViewInfo &vi, int64_t R, int h, CUtensorMap *m) {
    if (R < h) return true;  // never used
    const int64_t rs = map_stride(one_stride(vi.row), vi.cols * vi.es);
    const int64_t dim[3] = {vi.cols, h, R - h + 1}, stride[2] = {rs, rs}, dim1[2] = {vi.cols, R};
    const int box[3] = {128 / vi.es, h, 1};
    return encode_map(m, v->dtype, h == 1 ? 2 : 3, v->ptr, h == 1 ? dim1 : dim, stride, box, true);
}

template <bool FP8, int KSUB, bool P_MN, bool BYK>
cudaError_t launch_grouped(GroupedParams p, const GroupedMaps &m, int num_sms, cudaStream_t s) {
    // no more pairs than tiles: by rows each group may end in a narrow one
    const int64_t rows = BYK ? (int64_t)p.groups * ((p.Mo + p.tile_w - 1) / p.tile_w)
                             : std::min(p.groups, p.R) + (int64_t)p.R / 32;
    const int grid = (int)std::min<int64_t>(num_sms & ~1, 2 * rows * p.tiles_n);
    static SmemLimit limit;
    auto kern = grouped_kernel<FP8, KSUB, P_MN, BYK>;
    int stages = 2;
    while (stages < 12 && group_layout(stages + 1, KSUB, p.q_rows, p.groups).total <= 227 * 1024) ++stages;
    p.stages = stages;
    const size_t smem = group_layout(stages, KSUB, p.q_rows, p.groups).total;
    const cudaError_t e = limit.ensure(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3(grid), dim3(kGroupThreads), smem, s, dim3(2, 1, 1), p.pdl, m, p);
}

// The tensor-core kernel; false when the operands do not allow it.
bool tensor_call(const GroupedCall &c, GroupedParams p, int num_sms, cudaStream_t s, cudaError_t *err) {
    const int dt = c.a->dtype;
    if (dt == DG_F32 || !tensor_cores_allowed() || num_sms < 2) return false;
    const bool fp8 = dt == DG_E4M3;
    const bool none = p.K == 0;  // nothing is multiplied: no maps are needed
    GroupedMaps m{};
    if (c.by_k) {
        if (fp8 || c.ci.col.n > 1 || c.c->row_dims != 2) return false;
        // C^T's M side runs along the dim that dW is contiguous along
        const int64_t *cst = c.c->stride, *csh = c.c->shape;
        const bool turned = csh[2] > 1 && cst[2] != elem_size(c.c->dtype) && (csh[1] <= 1 || cst[1] == elem_size(c.c->dtype));
        const dg_view *pv = turned ? c.a : c.b, *qv = turned ? c.b : c.a;
        const ViewInfo &pi = turned ? c.ai : c.bi, &qi = turned ? c.bi : c.ai;
        const int64_t N = pi.cols, Mo = qi.cols;
        constexpr int kd = 128;
        if (!none && (!rows_map_ok(c.a, c.ai) || !rows_map_ok(c.b, c.bi))) return false;
        p.Mo = (int32_t)Mo;
        p.out.N = (int32_t)N;
        p.out.rs = turned ? cst[2] : cst[1];
        p.out.cs = turned ? cst[1] : cst[2];
        p.out_gs = csh[0] > 1 ? cst[0] : 0;
        p.tile_w = Mo > 128 ? 256 : 128;
        p.q_rows = p.tile_w / 2;
        if (!none)
            for (int i = 0; i < 3; ++i) {
                const int h = i == 0 ? kd : i == 1 ? 16 : 1;
                if (!cut_map(pv, pi, c.R, h, &m.m[i]) || !cut_map(qv, qi, c.R, h, &m.m[3 + i])) return false;
            }
        p.idesc |= 3u << 15;  // both operands MN-major
    } else {
        if (c.ci.row.n > 1 || c.ci.col.n > 1) return false;
        p.out.N = (int32_t)c.N;
        p.out.rs = one_stride(c.ci.row);
        p.out.cs = c.ci.col.n ? c.ci.col.stride[0] : c.ci.es;
        // four times the average group, as the most: what a narrower tile saves of the ring holds more stages
        int64_t most = 64;
        while (most < 256 && most * c.groups < 4 * c.R) most *= 2;
        p.tile_w = (int32_t)std::min<int64_t>(most, (c.R + 31) / 32 * 32);
        p.q_rows = p.tile_w <= 32 ? 16 : p.tile_w <= 64 ? 32 : p.tile_w <= 128 ? 64 : 128;
        bool mn = false;
        if (!none) {
            if (!rows_map_ok(c.a, c.ai)) return false;
            if (!b_map(c, false, 1, &p, &m.m[0])) {
                mn = true;
                if (!b_map(c, true, 2, &p, &m.m[0])) return false;
            }
            const int es = c.ai.es;
            const int64_t dim[2] = {c.K, c.R}, stride[1] = {map_stride(one_stride(c.ai.row), c.K * es)};
            for (int i = 0; 16 << i <= p.q_rows; ++i) {
                const int box[2] = {128 / es, 16 << i};
                if (!encode_map(&m.m[1 + i], dt, 2, c.a->ptr, dim, stride, box, true)) return false;
            }
        }
        if (mn) p.idesc |= 1u << 15;
    }
    p.tiles_n = (p.out.N + 255) / 256;
    p.out.c = static_cast<char *>(c.c->ptr);
    const int ces = elem_size(c.c->dtype);
    p.out.vec = p.out.cs == ces && reinterpret_cast<uintptr_t>(c.c->ptr) % 16 == 0 && p.out.rs % 16 == 0 &&
                p.out_gs % 16 == 0;
    if (c.by_k) *err = launch_grouped<false, 2, true, true>(p, m, num_sms, s);
    else if (p.idesc >> 15 & 1)
        *err = fp8 ? launch_grouped<true, 2, true, false>(p, m, num_sms, s)
                   : launch_grouped<false, 2, true, false>(p, m, num_sms, s);
    else
        *err = fp8 ? launch_grouped<true, 1, false, false>(p, m, num_sms, s)
                   : launch_grouped<false, 1, false, false>(p, m, num_sms, s);
    return true;
}

dg_status grouped_call(const GroupedCall &c, cudaStream_t s) {
    int num_sms = 0;
    int *err_word = nullptr;
    const dg_status st = device_info(&num_sms, &err_word);
    if (st != DG_OK) return st;
    const bool product = c.alpha != 0.f && c.K > 0 && c.R > 0;
    GroupedParams p{};
    p.offsets = c.offsets;
    p.groups = c.groups;
    p.R = (int32_t)c.R;
    p.K = product ? (int32_t)c.K : 0;
    p.idesc = 1u << 4 | 256u >> 4 << 24;  // FP32 accumulators, M = 256
    if (c.a->dtype == DG_BF16) p.idesc |= 1u << 7 | 1u << 10;
    p.out.dtype = c.c->dtype;
    p.out.alpha = c.alpha;
    p.out.beta = c.beta;
    p.out.scale_r = product ? c.scale_r : nullptr;
    p.out.scale_n = product ? c.scale_n : nullptr;
    p.out.bias_n = c.bias;
    p.out.act = c.act;
    p.k_chunk = c.a->dtype == DG_E4M3 ? 4096 : 2048;  // 128 steps of the tensor core
    p.scale_n_gs = (int32_t)c.N;
    p.err_word = err_word;
    p.timeout_ns = wait_timeout_ns();
    p.stall_loader = test_stall();
    p.pdl = early_launch_mode() != 0;
    cudaError_t err;
    if (!tensor_call(c, p, num_sms, s, &err)) {
        GroupedAnyParams q{};
        q.offsets = c.offsets;
        q.groups = c.groups;
        q.R = (int32_t)c.R;
        q.K = p.K;
        q.Mo = (int32_t)c.Mo;
        q.N = (int32_t)c.N;
        q.a = dev_of(c.a, c.ai);
        q.b = dev_of(c.b, c.bi);
        q.c = dev_of(c.c, c.ci);
        q.alpha = c.alpha;
        q.beta = c.beta;
        q.scale_r = p.out.scale_r;
        q.scale_n = p.out.scale_n;
        q.bias = c.bias;
        q.act = c.act;
        q.err_word = err_word;
        q.pdl = p.pdl;
        q.tiles_m = (int32_t)((c.Mo + kAnyTile - 1) / kAnyTile);
        const int64_t blocks = c.by_k ? (int64_t)c.groups * q.tiles_m : (c.R + kAnyTile - 1) / kAnyTile + c.groups;
        if (blocks > INT32_MAX) return DG_ERR_UNSUPPORTED;
        const dim3 grid((unsigned)blocks, (unsigned)std::min<int64_t>((c.N + kAnyTile - 1) / kAnyTile, 65535));
        const size_t smem = sizeof(int) * (3 * (size_t)c.groups + 1);
        err = c.by_k ? launch_ex(grouped_any_kernel<true>, grid, dim3(256), smem, s, dim3(1, 1, 1), q.pdl, q)
                     : launch_ex(grouped_any_kernel<false>, grid, dim3(256), smem, s, dim3(1, 1, 1), q.pdl, q);
    }
    if (err != cudaSuccess) return DG_ERR_CUDA;
    count_launch();
    return DG_OK;
}

// Sizes that the kernels count in 32 bits, tiles included.
bool size_ok(int64_t n) { return n <= (int64_t(1) << 31) - (1 << 13); }

// Whether a view is [groups, rows, cols], its first two dims the rows.
dg_status stack_shape(const dg_view *v, int32_t groups) {
    if (v->ndim != 3 || v->row_dims != 2) return DG_ERR_NDIM;
    return v->shape[0] == groups ? DG_OK : DG_ERR_SHAPE;
}

bool in_type(int dt) { return dt == DG_F16 || dt == DG_BF16 || dt == DG_F32 || dt == DG_E4M3; }

dg_status offsets_ok(const int64_t *offsets, int32_t groups) {
    if (groups < 0) return DG_ERR_SHAPE;
    if (groups > 0 && !offsets) return DG_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(offsets) % 8) return DG_ERR_ALIGN;
    return groups > kGroupsMost ? DG_ERR_UNSUPPORTED : DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_gemm_grouped(const dg_view *A, const dg_view *B, const dg_view *C, const int64_t *offsets, int32_t groups,
                          float alpha, float beta, const float *scale_a, const float *scale_b,
                          const dg_epilogue *epilogue, void *stream) {
    if (!A || !B || !C) return DG_ERR_NULL;
    if (epilogue && (epilogue->activation < DG_ACT_NONE || epilogue->activation > DG_ACT_GELU_TANH ||
                     epilogue->reserved != 0))
        return DG_ERR_VALUE;
    GroupedCall c{};
    dg_status st;
    if ((st = analyse(A, false, &c.ai)) != DG_OK || (st = analyse(B, false, &c.bi)) != DG_OK ||
        (st = analyse(C, true, &c.ci)) != DG_OK || (st = stack_shape(B, groups)) != DG_OK)
        return st;
    if (B->shape[1] != c.ai.cols || c.ci.rows != c.ai.rows || c.ci.cols != B->shape[2])
        return DG_ERR_SHAPE;
    if (!in_type(A->dtype) || A->dtype != B->dtype || C->dtype == DG_E4M3) return DG_ERR_DTYPE;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return DG_ERR_VALUE;
    if ((st = offsets_ok(offsets, groups)) != DG_OK) return st;
    for (const float *f : {scale_a, scale_b, epilogue ? epilogue->bias : nullptr})
        if (reinterpret_cast<uintptr_t>(f) % 4) return DG_ERR_ALIGN;
    c.a = A;
    c.b = B;
    c.c = C;
    c.offsets = offsets;
    c.groups = groups;
    c.R = c.ai.rows;
    c.K = c.ai.cols;
    c.N = c.ci.cols;
    c.alpha = alpha;
    c.beta = beta;
    c.scale_r = scale_a;
    c.scale_n = scale_b;
    c.bias = epilogue ? epilogue->bias : nullptr;
    c.act = epilogue ? epilogue->activation : DG_ACT_NONE;
    if (!size_ok(c.R) || !size_ok(c.K) || !size_ok(c.N)) return DG_ERR_UNSUPPORTED;
    if (c.R == 0 || c.N == 0 || groups == 0) return DG_OK;
    const bool product = alpha != 0.f && c.K > 0;
    if (!device_pointer(offsets) || !device_pointer(C->ptr) || (c.bias && !device_pointer(c.bias)))
        return DG_ERR_POINTER;
    if (product && (!device_pointer(A->ptr) || !device_pointer(B->ptr) || (scale_a && !device_pointer(scale_a)) ||
                    (scale_b && !device_pointer(scale_b))))
        return DG_ERR_POINTER;
    return grouped_call(c, static_cast<cudaStream_t>(stream));
}

dg_status dg_gemm_grouped_dw(const dg_view *X, const dg_view *dY, const dg_view *dW, const int64_t *offsets,
                             int32_t groups, float alpha, float beta, void *stream) {
    if (!X || !dY || !dW) return DG_ERR_NULL;
    GroupedCall c{};
    dg_status st;
    if ((st = analyse(X, false, &c.ai)) != DG_OK || (st = analyse(dY, false, &c.bi)) != DG_OK ||
        (st = analyse(dW, true, &c.ci)) != DG_OK || (st = stack_shape(dW, groups)) != DG_OK)
        return st;
    if (c.ai.rows != c.bi.rows || dW->shape[1] != c.ai.cols || dW->shape[2] != c.bi.cols) return DG_ERR_SHAPE;
    if (!in_type(X->dtype) || X->dtype != dY->dtype || dW->dtype == DG_E4M3) return DG_ERR_DTYPE;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return DG_ERR_VALUE;
    if ((st = offsets_ok(offsets, groups)) != DG_OK) return st;
    c.by_k = true;
    c.a = X;
    c.b = dY;
    c.c = dW;
    c.offsets = offsets;
    c.groups = groups;
    c.R = c.ai.rows;
    c.K = 1;  // each group's rows
    c.Mo = c.ai.cols;
    c.N = c.bi.cols;
    c.alpha = alpha;
    c.beta = beta;
    if (!size_ok(c.R) || !size_ok(c.Mo) || !size_ok(c.N)) return DG_ERR_UNSUPPORTED;
    if (c.Mo == 0 || c.N == 0 || groups == 0) return DG_OK;
    if (!device_pointer(offsets) || !device_pointer(dW->ptr)) return DG_ERR_POINTER;
    if (alpha != 0.f && c.R > 0 && (!device_pointer(X->ptr) || !device_pointer(dY->ptr))) return DG_ERR_POINTER;
    return grouped_call(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// The linear cross entropy's arithmetic on logits, shared by its own kernels
// and by the tensor-core kernel's epilogues.
#pragma once

#include "common.cuh"
#include "umma_common.cuh"

namespace dg {

// What a row's target means, besides a column of the vocabulary.
constexpr int kIgnored = -1, kInvalid = -2;

__device__ __forceinline__ int read_target(const int64_t *target, int64_t ignore_index, int64_t V, int64_t t) {
    const int64_t y = target[t];
    if (y == ignore_index) return kIgnored;
    return (y < 0 || y >= V) ? kInvalid : (int)y;
}

// exp(x) = 2^(x log2 e) with the hardware's power of two: relative error about
// 2^-22 + |x| 2^-23 (the product with log2 e is rounded), and 0 for results
// below 2^-126.  In lse's sums the terms next to the maximum count, where x is
// a few units; G's small probabilities are rounded to 16 bits after it.
__device__ __forceinline__ float exp_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// A row's logits as a pair (m, s): their maximum and sum of exp(z - m); m ==
// -infinity means none (or all -infinity).  A NaN or +infinity among the
// logits ends as s = NaN.  join: two pairs as one.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float mx = fmaxf(m, m2);
    const float a = m == -INFINITY ? (s != s ? s : 0.f) : s * exp_fast(m - mx);
    const float b = m2 == -INFINITY ? (s2 != s2 ? s2 : 0.f) : s2 * exp_fast(m2 - mx);
    m = mx;
    s = a + b;
}

// Another N logits: one pass, the running sum rescaled when the maximum moves.
// Four chains for the maximum and eight for the sum, so that few instructions
// wait for one another (a warp has its scheduler almost to itself).  A single
// logit z is the pair (z, 1): join(m, s, z, 1.f).
template <int N>
__device__ __forceinline__ void join_logits(float &m, float &s, const float (&z)[N]) {
    static_assert(N >= 4, "join_logits starts its four chains with a logit each");
    float mx[4] = {m, z[1], z[2], z[3]};
    mx[0] = fmaxf(mx[0], z[0]);
#pragma unroll
    for (int c = 4; c < N; ++c) mx[c & 3] = fmaxf(mx[c & 3], z[c]);
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (top == -INFINITY) {  // nothing but -infinity, and perhaps NaN
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (z[c] != z[c]) s = z[c];
        return;
    }
    float a[8] = {m == -INFINITY ? (s != s ? s : 0.f) : s * exp_fast(m - top), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; ++c) a[c & 7] += exp_fast(z[c] - top);
    m = top;
    s = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

// The logit of column `hit` (relative to the first of the N) if it is one of them.
template <int N>
__device__ __forceinline__ void keep_target(const float (&z)[N], int hit, float *out) {
    if ((unsigned)hit < (unsigned)N) {
#pragma unroll
        for (int c = 0; c < N; ++c)
            if (c == hit) *out = z[c];
    }
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    tmem_ld16(addr, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
    tmem_ld16(addr + 16, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
}

// 32 accumulators as logits alpha * acc of columns j .., -infinity at and past Nj.
__device__ __forceinline__ void logits32(float (&z)[32], float alpha, const uint32_t (&r)[32], int j, int Nj) {
#pragma unroll
    for (int c = 0; c < 32; ++c) z[c] = alpha * __uint_as_float(r[c]);
    if (j + 32 > Nj) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (j + c >= Nj) z[c] = -INFINITY;
    }
}

// Columns of a tile per epilogue warp, and per slot of CeTile::part.
constexpr int kSlotCols = 128;

// One warp's 32 rows (this thread's row i) x 128 columns from j: the row's
// pair goes to the columns' slot.  A thread holds one row, so nothing crosses
// lanes; the TMEM load of the next 32 columns is in flight while 32 are
// reduced.
__device__ __forceinline__ void ce_stats_rows(const CeTile &ce, float alpha, uint32_t t_addr, int i, int Mi, int j,
                                              int Nj) {
    if (j >= Nj) return;
    const bool ok = i < Mi;
    uint32_t r[2][32];
    __syncwarp();
    tmem_ld32(t_addr, r[0]);
    const int y = ok ? read_target(ce.target, ce.ignore_index, ce.V, i) : kIgnored;
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int q = 0; q < kSlotCols / 32; ++q) {
        tmem_ld_wait();
        if (q + 1 < kSlotCols / 32) tmem_ld32(t_addr + 32 * (q + 1), r[(q + 1) & 1]);
        float z[32];
        logits32(z, alpha, r[q & 1], j + 32 * q, Nj);
        join_logits(m, s, z);
        if (y >= 0) keep_target(z, y - ce.v0 - j - 32 * q, ce.ztarget + i);
        __syncwarp();
    }
    if (ok) ce.part[(int64_t)(j / kSlotCols) * ce.T + i] = make_float2(m, s);
}

// The same for a long k.
// The tensor core adds each step's products to the accumulator with
// truncation, so a logit's error grows with the steps (the loss was off by
// 1.4e-6 of itself at k = 4096, the truncations all pointing the same way);
// every chunk of k starts a fresh accumulator, and the chunks are added here,
// rounded to nearest, in registers.
__device__ __forceinline__ void ce_stats_rows_long(float (&sums)[kSlotCols], const CeTile &ce, float alpha,
                                                   uint32_t t_addr, int i, int Mi, int j, int Nj, bool first,
                                                   bool last) {
#pragma unroll
    for (int c0 = 0; c0 < kSlotCols; c0 += 16) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(t_addr + (uint32_t)c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const float v = __uint_as_float(r[c]);
            sums[c0 + c] = first ? v : sums[c0 + c] + v;
        }
    }
    if (!last || j >= Nj) return;
    const bool ok = i < Mi;
    const int y = ok ? read_target(ce.target, ce.ignore_index, ce.V, i) : kIgnored;
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int c0 = 0; c0 < kSlotCols; c0 += 32) {
        float z[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] = j + c0 + c < Nj ? alpha * sums[c0 + c] : -INFINITY;
        join_logits(m, s, z);
        if (y >= 0) keep_target(z, y - ce.v0 - j - c0, ce.ztarget + i);
    }
    if (ok) ce.part[(int64_t)(j / kSlotCols) * ce.T + i] = make_float2(m, s);
}

// One warp's 32 rows x w columns of G = scale (exp(z - lse) - 1[v == target]),
// zero in rows that take no part, through tensor stores in blocks of 32 rows x
// 64 columns (in epilogue_rows_tma's layout).  The two warps of a quarter take
// blocks in turn, each through one staging block of its own.
__device__ __forceinline__ void ce_grad_rows_tma(const CeTile &ce, const EpiParams &e, const CUtensorMap *gmap,
                                                 uint32_t stage, uint32_t t_row, int i_base, int Mi, int j0, int w,
                                                 int Nj, int lane, int first) {
    if (i_base >= Mi) return;  // the whole warp is below G (warp-uniform)
    const bool bf16_out = e.c_dtype == DG_BF16;
    const float alpha = e.alpha;
    RowGrad row{0.f, 0.f, kIgnored, 0};
    if (i_base + lane < Mi) row = ce.rows[i_base + lane];
    for (int c0 = first; c0 < w && j0 + c0 < Nj; c0 += 128) {
        uint32_t r[2][32], p[32];
        tmem_ld32(t_row + (uint32_t)c0, r[0]);
        tmem_ld_wait();
        tmem_ld32(t_row + (uint32_t)c0 + 32, r[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h) tmem_ld_wait();
            float g[32];
            const int hit = row.target - ce.v0 - j0 - c0 - 32 * h;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float q = exp_fast(alpha * __uint_as_float(r[h][c]) - row.lse);
                g[c] = row.target < 0 ? 0.f : row.scale * (c == hit ? q - 1.f : q);
            }
#pragma unroll
            for (int c = 0; c < 16; ++c)
                p[16 * h + c] = bf16_out ? pack2<true>(g[2 * c], g[2 * c + 1]) : pack2<false>(g[2 * c], g[2 * c + 1]);
        }
        if (lane == 0) bulk_wait_read<0>();  // the copy that last read the block is done with it
        __syncwarp();
        const uint32_t rowa = stage + (uint32_t)lane * 128u;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            st_shared_v4(rowa + ((uint32_t)(u ^ (lane & 7)) << 4), p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(gmap, stage, j0 + c0, i_base);
            bulk_commit();
        }
    }
}

// The same for a long k, whose chunks are added in `sums` as in
// ce_stats_rows_long: the logits have to be those that lse was made of, or
// p - 1 at the target of a confident row is nothing but the difference of two
// errors (at k = 4096 and a logit of 30, one accumulator for all of k put it
// off by 3e-4).  The sums hold the warp's two blocks of 64 columns.
__device__ __forceinline__ void ce_grad_rows_long(float (&sums)[kSlotCols], const CeTile &ce, const EpiParams &e,
                                                  const CUtensorMap *gmap, uint32_t stage, uint32_t t_row, int i_base,
                                                  int Mi, int j0, int w, int Nj, int lane, int half, bool first,
                                                  bool last) {
    const int c0 = 64 * half;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (c0 + 128 * b >= w) continue;  // a half-width tile (warp-uniform)
#pragma unroll
        for (int q = 0; q < 64; q += 16) {
            uint32_t r[16];
            __syncwarp();
            tmem_ld16(t_row + (uint32_t)(c0 + 128 * b + q), r);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float v = __uint_as_float(r[c]);
                sums[64 * b + q + c] = first ? v : sums[64 * b + q + c] + v;
            }
        }
    }
    if (!last || i_base >= Mi) return;
    const bool bf16_out = e.c_dtype == DG_BF16;
    const float alpha = e.alpha;
    RowGrad row{0.f, 0.f, kIgnored, 0};
    if (i_base + lane < Mi) row = ce.rows[i_base + lane];
    const uint32_t rowa = stage + (uint32_t)lane * 128u;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int j = j0 + c0 + 128 * b;
        if (c0 + 128 * b >= w || j >= Nj) continue;
        const int hit = row.target - ce.v0 - j;
        if (lane == 0) bulk_wait_read<0>();  // the copy that last read the block is done with it
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float g[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float q = exp_fast(alpha * sums[64 * b + 8 * u + c] - row.lse);
                g[c] = row.target < 0 ? 0.f : row.scale * (8 * u + c == hit ? q - 1.f : q);
            }
            uint32_t p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                p[c] = bf16_out ? pack2<true>(g[2 * c], g[2 * c + 1]) : pack2<false>(g[2 * c], g[2 * c + 1]);
            st_shared_v4(rowa + ((uint32_t)(u ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(gmap, stage, j, i_base);
            bulk_commit();
        }
    }
}

}  // namespace dg

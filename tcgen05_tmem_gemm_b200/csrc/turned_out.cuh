// The epilogue of tiles that compute C^T: TMEM lanes are columns n of C, TMEM
// columns are rows r.  The products of weights with few or a ragged number of
// rows are tiled this way, so that the weight fills the tensor core's fixed
// side and the rows its adjustable one.
//
// After tcgen05.ld a thread holds one n and 32 rows.  A warp turns its 32 x 32
// block through shared memory and stores whole 64- or 128-byte runs of C's
// rows; blocks that a vector store does not fit (an odd N, strided or
// unaligned C) are stored element by element, a warp then writing 32
// neighbouring columns per row.
#pragma once

#include "umma_common.cuh"

namespace dg {

struct TurnedOut {
    char *c;
    int64_t rs, cs;        // bytes between rows and between columns of C
    int32_t dtype;
    int32_t vec;           // columns contiguous, rows at multiples of 16 bytes
    float alpha, beta;
    const float *scale_r;  // per row, or null
    const float *scale_n;  // per column, or null
    const float *bias_n;   // per column, or null
    int32_t act;
    int32_t N;
};

constexpr uint32_t kTurnBytes = 32 * 32 * 4;  // a warp's staging block

// Rows [r0, r0 + rows) of C, whose accumulators are the TMEM columns from
// `taddr` (lane quarter included) on, and columns n0 .. n0 + 31.  `empty`: the
// sums are zero and TMEM is not read.  r0 indexes scale_r and C's rows.
template <int CD, bool FUSED, int ACT>
__device__ __forceinline__ void turned_rows_t(const TurnedOut &o, uint32_t stage, uint32_t taddr, bool empty,
                                              int64_t r0, int rows, int n0, int lane) {
    constexpr int ES = CD == DG_F32 ? 4 : 2;
    const int n = n0 + lane;
    const bool n_ok = n < o.N;
    const float an = o.alpha * (o.scale_n != nullptr && n_ok ? o.scale_n[n] : 1.f);
    const float bn = FUSED && o.bias_n != nullptr && n_ok ? o.bias_n[n] : 0.f;
    const bool vec = o.vec && n0 + 32 <= o.N;
    for (int c0 = 0; c0 < rows; c0 += 32) {
        const int some = min(32, rows - c0);
        uint32_t r[32];
        if (empty) {
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = 0;
        } else {
            __syncwarp();
            tmem_ld16(taddr + (uint32_t)c0, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
            tmem_ld16(taddr + (uint32_t)c0 + 16u, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
            tmem_ld_wait();
        }
        float v[32];
        char *const block = o.c + (r0 + c0) * o.rs + (int64_t)n0 * o.cs;
        if (o.scale_r != nullptr) {
            const float sr = o.scale_r[r0 + c0 + min(lane, some - 1)];  // one row's per lane
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = (an * __shfl_sync(0xffffffffu, sr, c)) * __uint_as_float(r[c]);
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = an * __uint_as_float(r[c]);
        }
        if (o.beta != 0.f) {
#pragma unroll
            for (int h = 0; h < 32; h += 8) {
                float old[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    old[c] = n_ok && h + c < some ? ld_out<CD>(block + (h + c) * o.rs + lane * o.cs) : 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) v[h + c] = fmaf(o.beta, old[c], v[h + c]);
            }
        }
        if (FUSED) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = act_fn<ACT, CD != DG_F32>(v[c] + bn);
        }
        if (!vec) {
            if (n_ok) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < some) st_out<CD>(block + c * o.rs + lane * o.cs, v[c]);
            }
            continue;
        }
        // [row][n] in shared memory, without padding: a warp writes one row's 32
        // values at a time, and reads 512 contiguous bytes per instruction
        __syncwarp();
        const uint32_t at = stage + (uint32_t)lane * ES;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            if (CD == DG_F32) {
                st_shared_f32(at + c * 128u, v[c]);
            } else {
                const uint32_t h = CD == DG_BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v[c]))
                                                 : (uint32_t)__half_as_ushort(__float2half_rn(v[c]));
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + c * 64u), "h"((uint16_t)h) : "memory");
            }
        }
        __syncwarp();
        constexpr int UNITS = 32 * ES / 16;  // 16-byte units per row
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int e = i * 32 + lane, row = e / UNITS;
            const float4 w = ld_shared_v4(stage + (uint32_t)e * 16u);
            if (row < some) *reinterpret_cast<float4 *>(block + row * o.rs + (e % UNITS) * 16) = w;
        }
    }
}

template <bool FUSED, int ACT>
__device__ __forceinline__ void turned_rows_d(const TurnedOut &o, uint32_t stage, uint32_t taddr, bool empty,
                                              int64_t r0, int rows, int n0, int lane) {
    if (o.dtype == DG_F32) turned_rows_t<DG_F32, FUSED, ACT>(o, stage, taddr, empty, r0, rows, n0, lane);
    else if (o.dtype == DG_BF16) turned_rows_t<DG_BF16, FUSED, ACT>(o, stage, taddr, empty, r0, rows, n0, lane);
    else turned_rows_t<DG_F16, FUSED, ACT>(o, stage, taddr, empty, r0, rows, n0, lane);
}

__device__ __forceinline__ void turned_rows(const TurnedOut &o, uint32_t stage, uint32_t taddr, bool empty, int64_t r0,
                                            int rows, int n0, int lane) {
    if (n0 >= o.N) return;
    if (o.act == DG_ACT_GELU_TANH)
        turned_rows_d<true, DG_ACT_GELU_TANH>(o, stage, taddr, empty, r0, rows, n0, lane);
    else if (o.act == DG_ACT_RELU) turned_rows_d<true, DG_ACT_RELU>(o, stage, taddr, empty, r0, rows, n0, lane);
    else if (o.bias_n != nullptr) turned_rows_d<true, DG_ACT_NONE>(o, stage, taddr, empty, r0, rows, n0, lane);
    else turned_rows_d<false, DG_ACT_NONE>(o, stage, taddr, empty, r0, rows, n0, lane);
}

}  // namespace dg

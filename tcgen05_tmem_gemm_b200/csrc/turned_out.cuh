// The epilogue of tiles that compute C^T: TMEM lanes are columns n of C, TMEM
// columns are rows r.  The products of weights with few or a ragged number of
// rows are tiled this way, so that the weight fills the tensor core's fixed
// side and the rows its adjustable one.
//
// Three ways to C, per 32 x 32 block of a warp:
//  - 16-bit C of contiguous columns and aligned rows, beta = 0: TMEM is read in
//    the fragment layout of 8 x 8 matrices (16x256b), whose packed pairs
//    stmatrix turns on their way to shared memory; the warp then stores whole
//    64-byte runs of C's rows, 16 bytes a lane.  About 80 issue slots a block
//    against 130 with the 32 two-byte stores to shared memory of a thread that
//    holds one n, and a third of the latencies.
//  - F32 C: a thread holds one n and 32 rows, and a store of the warp is 128
//    contiguous bytes of a row: no detour.
//  - any other C, and beta != 0: the same, element by element.
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

constexpr uint32_t kTurnBytes = 32 * 32 * 2;  // a warp's staging block
constexpr int kTurnWarps = 8;                 // epilogue warps: two per quarter of the TMEM lanes

// 16 lanes x 32 columns in the fragment layout: r[4 j], r[4 j + 1] are lane
// t / 4, columns 8 j + 2 (t % 4) and the next; r[4 j + 2], r[4 j + 3] lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Four 8 x 8 matrices of 16-bit elements, turned: the eight rows of matrix q
// go to the addresses of lanes 8 q .. 8 q + 7.
__device__ __forceinline__ void stmatrix_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

constexpr int kTurnBlocks = 4;  // a warp's blocks of 32 rows: every other one of a tile of 256
using TurnedWords = uint32_t[kTurnBlocks][4][4];

// Blocks c0 = 32 half, 32 (half + 2), ... of a tile, 16-bit C, beta = 0, columns
// n0 .. n0 + 31 all inside C: read, scaled and packed into registers.
// SR: with a scale per row (a template argument: its registers would spill where
// no call has them).
template <bool SR, bool B16, bool FUSED, int ACT>
__device__ __forceinline__ void turned_read(TurnedWords &w, const TurnedOut &o, uint32_t taddr, int64_t r0, int rows,
                                            int n0, int lane, int half) {
    const int col = 2 * (lane & 3), sub = lane >> 2;
    float an[4], bn[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        an[q] = o.alpha * (o.scale_n != nullptr ? o.scale_n[n0 + 8 * q + sub] : 1.f);
        bn[q] = FUSED && o.bias_n != nullptr ? o.bias_n[n0 + 8 * q + sub] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kTurnBlocks; ++k) {
        const int c0 = 32 * half + 64 * k;
        if (c0 >= rows) continue;
        float sr[8];
        if (SR) {
#pragma unroll
            for (int j = 0; j < 8; ++j)  // rows past the last are not stored: any row's scale will do
                sr[j] = o.scale_r[r0 + min(c0 + 8 * (j >> 1) + col + (j & 1), rows - 1)];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 16 lanes at a time: 32 more registers would spill
            uint32_t r[16];
            __syncwarp();
            tmem_ld_frag(taddr + ((uint32_t)h << 20) + (uint32_t)c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 2 * h; q < 2 * h + 2; ++q) {  // n 8 q .. 8 q + 7
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = SR ? an[q] * sr[2 * j + i] : an[q];
                        v[i] = a * __uint_as_float(r[4 * j + 2 * (q & 1) + i]);
                        if (FUSED) v[i] = act_fn<ACT, true>(v[i] + bn[q]);
                    }
                    w[k][q][j] = pack2<B16>(v[0], v[1]);
                }
            }
        }
    }
}

// 32 columns of TMEM (FP32) added to others, which are there after a tmem_st_wait.
__device__ __forceinline__ void turned_add(uint32_t to, uint32_t from) {
    uint32_t r[32], t[32];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        tmem_ld16(from + (uint32_t)h, *reinterpret_cast<uint32_t(*)[16]>(&r[h]));
        tmem_ld16(to + (uint32_t)h, *reinterpret_cast<uint32_t(*)[16]>(&t[h]));
    }
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) + __uint_as_float(r[i]));
#pragma unroll
    for (int h = 0; h < 32; h += 16) tmem_st16(to + (uint32_t)h, *reinterpret_cast<uint32_t(*)[16]>(&t[h]));
}

// And turned on their way to C.
__device__ __forceinline__ void turned_write(const TurnedWords &w, const TurnedOut &o, uint32_t stage, int64_t r0, int rows,
                                             int n0, int lane, int half) {
    // unit u of row r lies at unit u ^ (r / 2 % 4): neither side has bank conflicts
    const int sub = lane >> 2;
    const uint32_t put = stage + (uint32_t)lane * 64u, swz = (uint32_t)(lane >> 1) & 3u;
    char *at = o.c + (r0 + 32 * half + sub) * o.rs + (int64_t)n0 * 2 + (lane & 3) * 16;
    const int64_t eight = 8 * o.rs;
#pragma unroll
    for (int k = 0; k < kTurnBlocks; ++k) {
        const int c0 = 32 * half + 64 * k;
        if (c0 >= rows) continue;
        __syncwarp();  // the last block has left the staging block
#pragma unroll
        for (int q = 0; q < 4; ++q)
            stmatrix_turned(put + ((uint32_t)q ^ swz) * 16u, w[k][q][0], w[k][q][1], w[k][q][2], w[k][q][3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i, at += eight) {
            const int row = i * 8 + sub;
            const float4 t = ld_shared_v4(stage + (uint32_t)row * 64u + (((uint32_t)lane ^ (uint32_t)(row >> 1)) & 3u) * 16u);
            if (c0 + row < rows) *reinterpret_cast<float4 *>(at) = t;
        }
        at += 4 * eight;
    }
}

// The same for any C: a thread holds column n0 + lane and 32 rows.
template <int CD, bool FUSED, int ACT>
__device__ __forceinline__ void turned_any(const TurnedOut &o, uint32_t taddr, bool empty, int64_t r0, int rows, int n0,
                                           int lane, int half) {
    const int n = n0 + lane;
    const bool n_ok = n < o.N;
    const float an = o.alpha * (o.scale_n != nullptr && n_ok ? o.scale_n[n] : 1.f);
    const float bn = FUSED && o.bias_n != nullptr && n_ok ? o.bias_n[n] : 0.f;
#pragma unroll 1
    for (int c0 = 32 * half; c0 < rows; c0 += 64) {
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
        char *const at = o.c + (r0 + c0) * o.rs + (int64_t)n * o.cs;  // rows are stepped through: 32 kept offsets would spill
        if (o.scale_r != nullptr) {
            const float sr = o.scale_r[r0 + c0 + min(lane, some - 1)];  // one row's per lane
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = (an * __shfl_sync(0xffffffffu, sr, c)) * __uint_as_float(r[c]);
        } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = an * __uint_as_float(r[c]);
        }
        if (o.beta != 0.f) {
            const char *from = at;
#pragma unroll
            for (int h = 0; h < 32; h += 8) {
                float old[8];
#pragma unroll
                for (int c = 0; c < 8; ++c, from += o.rs) old[c] = n_ok && h + c < some ? ld_out<CD>(from) : 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) v[h + c] = fmaf(o.beta, old[c], v[h + c]);
            }
        }
        if (FUSED) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = act_fn<ACT, CD != DG_F32>(v[c] + bn);
        }
        if (n_ok) {
            char *to = at;
#pragma unroll
            for (int c = 0; c < 32; ++c, to += o.rs)
                if (c < some) st_out<CD>(to, v[c]);
        }
    }
}

template <bool SR, bool FUSED, int ACT>
__device__ __forceinline__ void turned_read_d(TurnedWords &w, const TurnedOut &o, uint32_t taddr, int64_t r0, int rows,
                                              int n0, int lane, int half) {
    if (o.dtype == DG_BF16) turned_read<SR, true, FUSED, ACT>(w, o, taddr, r0, rows, n0, lane, half);
    else turned_read<SR, false, FUSED, ACT>(w, o, taddr, r0, rows, n0, lane, half);
}

template <bool FUSED, int ACT>
__device__ __forceinline__ void turned_any_d(const TurnedOut &o, uint32_t taddr, bool empty, int64_t r0, int rows, int n0,
                                             int lane, int half) {
    if (o.dtype == DG_F32) turned_any<DG_F32, FUSED, ACT>(o, taddr, empty, r0, rows, n0, lane, half);
    else if (o.dtype == DG_BF16) turned_any<DG_BF16, FUSED, ACT>(o, taddr, empty, r0, rows, n0, lane, half);
    else turned_any<DG_F16, FUSED, ACT>(o, taddr, empty, r0, rows, n0, lane, half);
}

// One element of a C without scales, from its sum.
__device__ __forceinline__ void turned_store(const TurnedOut &o, float sum, int64_t r, int n) {
    char *const at = o.c + r * o.rs + (int64_t)n * o.cs;
    float v = epi_value(sum, o.alpha, 1.f, o.beta, at, o.dtype);
    if (o.bias_n != nullptr || o.act != DG_ACT_NONE) v = epi_fuse(v, o.bias_n, n, o.act, o.dtype != DG_F32);
    store_elem(at, o.dtype, v);
}

// Rows [r0, r0 + rows) of C (256 at most), whose accumulators are the TMEM
// columns from `taddr` (lane quarter included) on, and columns n0 .. n0 + 31:
// every other block of 32 rows, from block `half` on.  `empty`: the sums are zero
// and TMEM is not read.  r0 indexes scale_r and C's rows.  stage: kTurnBytes of
// the warp's own.  release() is called once, by the whole warp, when the warp has
// done with TMEM.  SR: scales per row take the fast way too.
template <bool SR, typename Release>
__device__ __forceinline__ void turned_rows(const TurnedOut &o, uint32_t stage, uint32_t taddr, bool empty, int64_t r0,
                                            int rows, int n0, int lane, int half, Release release) {
    const bool fused = o.bias_n != nullptr;
    if (n0 >= o.N) {
        release();
    } else if (o.dtype != DG_F32 && o.vec && o.beta == 0.f && n0 + 32 <= o.N && !empty && SR == (o.scale_r != nullptr)) {
        TurnedWords w;
        if (o.act == DG_ACT_GELU_TANH) turned_read_d<SR, true, DG_ACT_GELU_TANH>(w, o, taddr, r0, rows, n0, lane, half);
        else if (o.act == DG_ACT_RELU) turned_read_d<SR, true, DG_ACT_RELU>(w, o, taddr, r0, rows, n0, lane, half);
        else if (fused) turned_read_d<SR, true, DG_ACT_NONE>(w, o, taddr, r0, rows, n0, lane, half);
        else turned_read_d<SR, false, DG_ACT_NONE>(w, o, taddr, r0, rows, n0, lane, half);
        release();
        turned_write(w, o, stage, r0, rows, n0, lane, half);
    } else {
        if (o.act == DG_ACT_GELU_TANH) turned_any_d<true, DG_ACT_GELU_TANH>(o, taddr, empty, r0, rows, n0, lane, half);
        else if (o.act == DG_ACT_RELU) turned_any_d<true, DG_ACT_RELU>(o, taddr, empty, r0, rows, n0, lane, half);
        else if (fused) turned_any_d<true, DG_ACT_NONE>(o, taddr, empty, r0, rows, n0, lane, half);
        else turned_any_d<false, DG_ACT_NONE>(o, taddr, empty, r0, rows, n0, lane, half);
        release();
    }
}

}  // namespace dg

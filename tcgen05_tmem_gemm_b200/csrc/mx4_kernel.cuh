// C = A B^T of 4-bit floats with block scales: tcgen05.mma .block_scale,
// scales in TMEM.
//
// A tile is 128 columns of C by up to 128 of its rows, of a pair of CTAs 256 by
// up to 256, computed as C^T: the tensor core's M side (P) holds rows of B, its
// N side (Q) rows of A, so that a single token costs an N of 16.  In a pair (cta_group::2)
// each CTA has its own 128 rows of P and half of Q's rows; what a stage copies
// per product then falls from 48 to 32 KB per SM, which is what bounds large
// products.  Q's scales are in both CTAs' TMEM, each copied from its own shared
// memory by the same instruction.  A stage of the ring is 256 k: 128 bytes of
// codes per row (tensor copies, 128-byte swizzle) and the scales' tiles as
// they lie in memory (128 rows by 4 blocks, 512 bytes), which one tcgen05.cp
// each spreads over the lanes of TMEM.  Every stage has scale columns of its
// own in TMEM, so a stage's release (its MMAs done) also frees its scales.
//
// Few tiles and a long k: the CTAs of a cluster take a part of k each, leave
// their sums in their rings, and every CTA adds its share of the tile's rows, in
// rank order, from all of them through distributed shared memory.
//
// What bounds it (B200): the copies, about 740 cycles per stage and SM against
// 512 of MMAs, then the power cap (8192 x 4096 x 14336 in blocks of 16: 203 us
// with a cold cache, 222-251 back to back; 4096^3: 52 us cold, 43 from L2); for
// one row the four copies of a stage, 0.3 us (1 x 4096 x 14336 in blocks of 32:
// 7.3 us with its operands in L2, 16.4 from HBM).
#pragma once

#include "common.cuh"
#include "uniform.cuh"
#include "turned_out.cuh"

namespace dg {

struct Mx4Params {
    int32_t M, N;
    int32_t k_from, K;       // the piece of k of this launch, from a multiple of a stage's k up to K
    int32_t tile_w;          // rows of C per tile: 128 or 256 (fewer in the last)
    int32_t tiles_m, tiles_n;
    int32_t stages;
    int32_t split;           // CTAs of a cluster that share a tile's k (not in pairs; each has one tile)
    int32_t k_split;         // k per such CTA, a multiple of a stage's
    const float *fa, *fb;    // their tensors' factors, or null
    uint32_t idesc;          // instruction descriptor without N and scale ids
    TurnedOut out;
    int *err_word;
    uint64_t timeout_ns;
    int32_t stall_loader;
    int32_t pdl;
};

namespace {

// 3-D tiled load (see tma_load_2d).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

constexpr int kMx4Threads = 64 + 32 * kTurnWarps;
constexpr int kMx4K = 256;  // k per stage
// The most k of an accumulator for F32 C: 256 steps of the tensor core, each of which truncates.  Positive products
// under scales that differ came out 5e-6 low; 65536 of them in one accumulator 2.1e-5.
constexpr int kMx4Part = 16384;
constexpr uint32_t kScaleTile = 512;

struct Mx4Layout {
    uint32_t p_bytes, q_bytes, sp_bytes, sq_bytes, stage_bytes, turn_off, bar_off, aux_off, total;
};

// q_rows: rows of Q the ring has room for; scale tiles along k: 256 / (4 block)
__host__ __device__ inline Mx4Layout mx4_layout(int stages, int block, int tile_w, int q_rows) {
    Mx4Layout L;
    const uint32_t t = kMx4K / (4 * block);
    L.p_bytes = 128 * 128;
    L.q_bytes = (uint32_t)q_rows * 128;
    L.sp_bytes = t * kScaleTile;
    L.sq_bytes = (uint32_t)((tile_w + 127) / 128) * t * kScaleTile;
    L.stage_bytes = (L.p_bytes + L.q_bytes + L.sp_bytes + L.sq_bytes + 1023) / 1024 * 1024;
    L.turn_off = L.stage_bytes * stages;
    L.bar_off = L.turn_off + kTurnWarps * kTurnBytes;
    L.aux_off = L.bar_off + 8 * (2 * stages + 5);
    L.total = L.aux_off + 16 + 1024;
    return L;
}

// TMEM: the accumulators (two of 128 columns, or one of 256), then each stage's scales.
__host__ __device__ inline int mx4_scale_cols(int block, int tile_w) {
    return kMx4K / (4 * block) * (4 + 4 * ((tile_w + 127) / 128));
}

template <int BLOCK, bool PAIR>
__device__ __forceinline__ void mma_mx4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    if constexpr (!PAIR) {
        umma_mx4<BLOCK>(d_tmem, a_desc, b_desc, idesc, sfa, sfb, accumulate);
    } else if constexpr (BLOCK == 32) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    }
}

template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else tmem_cp_scales(taddr, desc);
}

template <bool PAIR>
__device__ __forceinline__ void mx4_commit(uint32_t bar) {
    if constexpr (PAIR) tc_commit_pair_mc(bar, 0x3);
    else tc_commit(bar);
}

template <int BLOCK, bool PAIR>
__global__ void __launch_bounds__(kMx4Threads, 1)
    mx4_kernel(const __grid_constant__ CUtensorMap tmap_p, const __grid_constant__ CUtensorMap tmap_q,
               const __grid_constant__ CUtensorMap tmap_sp, const __grid_constant__ CUtensorMap tmap_sq,
               const Mx4Params p, const int q_rows) {
    constexpr int T = kMx4K / (4 * BLOCK);  // scale tiles per stage
    if (threadIdx.x == 64 && p.K > 0) {
        tma_prefetch_desc(&tmap_p);
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_sp);
        tma_prefetch_desc(&tmap_sq);
    }
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Mx4Layout L = mx4_layout(p.stages, BLOCK, p.tile_w, q_rows);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + L.bar_off;
    const uint32_t bar_empty = bar_full + 8 * p.stages;
    const uint32_t bar_tfull = bar_empty + 8 * p.stages;
    const uint32_t bar_tempty = bar_tfull + 16;
    const uint32_t bar_drain = bar_tempty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L.aux_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L.aux_off + 4);

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    const WaitCtl wc{abort_flag, p.err_word, p.timeout_ns};
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int split = PAIR ? 1 : p.split;
    const int first = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x / split;
    const int stride = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x / split;
    const int part = split > 1 ? (int)cluster_ctarank() : 0;
    const int kb = p.k_from + part * p.k_split, ke = split > 1 ? min(p.K, kb + p.k_split) : p.K;  // this CTA's k
    const int units = p.tiles_m * p.tiles_n;
    const int buffers = p.tile_w <= 128 ? 2 : 1;  // accumulators
    const int q_tiles = (p.tile_w + 127) / 128;   // scale tiles along a tile's rows of C

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, (PAIR ? 2 : 1) * kTurnWarps);  // in a pair the even CTA's counts both
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), 512u);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), 512u);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem_base = uniform(*tmem_slot);
    pdl_wait();  // what comes before touches this CTA's own memory only

    // the tile of unit u: m inner, so that CTAs that run at the same time share B's rows
    auto tile_rows = [&](int u, int &m0, int &n0) {
        const int tn = u / p.tiles_m;
        m0 = (u - tn * p.tiles_m) * p.tile_w;
        n0 = tn * (PAIR ? 256 : 128);
        return min(p.tile_w, p.M - m0);
    };

    if (warp == 0) {
        // ------------------------------------------------------- producer
        const int stages = p.stages;
        const bool stall = p.stall_loader == 1;
        int it = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = first; ok && u < units; u += stride) {
            int m0, n0;
            const int rows = tile_rows(u, m0, n0), h = ((rows + 31) & ~31) / 2;  // a pair: Q's rows per CTA
            n0 += (int)rank * 128;
            for (int k = kb; k < ke; k += kMx4K, ++it) {
                if (!warp_wait(bar_empty + 8 * s, ph ^ 1u, wc)) {
                    ok = false;
                    break;
                }
                if (!stall && elect_one()) {
                    const uint32_t full = PAIR ? dsmem_map(bar_full + 8 * s, 0) : bar_full + 8 * s;
                    const uint32_t ps = sbase + s * L.stage_bytes, qs = ps + L.p_bytes;
                    const uint32_t sp = qs + L.q_bytes, sq = sp + L.sp_bytes;
                    const int t0 = k / (4 * BLOCK);
                    const uint32_t bytes = L.p_bytes + L.q_bytes + L.sp_bytes + L.sq_bytes;
                    if (leader) mbar_arrive_expect_tx(bar_full + 8 * s, PAIR ? 2u * bytes : bytes);
                    if (PAIR) {
                        tma_load_2d_pair(ps, &tmap_p, full, k / 2, n0);
                        tma_load_2d_pair(qs, &tmap_q, full, k / 2, m0 + (int)rank * h);
                        tma_load_3d_pair(sp, &tmap_sp, full, 0, t0, n0 / 128);
                        tma_load_3d_pair(sq, &tmap_sq, full, 0, t0, m0 / 128);
                    } else {
                        tma_load_2d(ps, &tmap_p, full, k / 2, n0);
                        tma_load_2d(qs, &tmap_q, full, k / 2, m0);
                        tma_load_3d(sp, &tmap_sp, full, 0, t0, n0 / 128);
                        tma_load_3d(sq, &tmap_sq, full, 0, t0, m0 / 128);
                    }
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!leader) pdl_release();
        // full[] of a pair's even CTA counts both CTAs' bytes
        if (leader && !stall)
            for (int d = 1; d <= stages && it - d >= 0; ++d) {
                const int j = it - d;
                mbar_wait_drain(bar_full + 8 * (j % stages), (uint32_t)(j / stages) & 1u, p.timeout_ns);
            }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        if (leader) {
        const int stages = p.stages;
        const uint32_t scale_cols = (uint32_t)mx4_scale_cols(BLOCK, p.tile_w);
        const uint64_t da0 = make_sw128_desc(sbase, 16u, 1024);
        const uint64_t db0 = make_sw128_desc(sbase + L.p_bytes, 16u, 1024);
        const uint64_t ds0 = make_scales_desc(sbase + L.p_bytes + L.q_bytes);
        int local = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = first; ok && p.K > 0 && u < units; u += stride, ++local) {
            int m0, n0;
            const int rows = tile_rows(u, m0, n0), w = PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15;
            const bool two = rows > 128;  // tiles of Q's scales
            const uint32_t idesc = p.idesc | (uint32_t)(w >> 3) << 17;
            const int b = buffers == 2 ? local & 1 : 0, turn = buffers == 2 ? local >> 1 : local;
            if (!warp_wait(bar_tempty + 8 * b, ((uint32_t)turn & 1u) ^ 1u, wc)) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + (uint32_t)(b * 128);
            for (int k = kb; k < ke; k += kMx4K) {
                if (!warp_wait(bar_full + 8 * s, ph, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t soff = (uint64_t)((s * L.stage_bytes) >> 4);
                const uint32_t sfa = tmem_base + 256u + (uint32_t)s * scale_cols, sfb = sfa + 4u * T;
                const int left = ke - k;
                if (elect_one()) {
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        if (t * 4 * BLOCK >= left) continue;
                        const uint64_t ds = ds0 + soff + (uint64_t)((t * kScaleTile) >> 4);
                        const uint32_t to = sfb + (uint32_t)(4 * t * q_tiles);
                        cp_scales<PAIR>(sfa + 4u * t, ds);
                        cp_scales<PAIR>(to, ds + (uint64_t)((T * kScaleTile) >> 4));
                        if (two) cp_scales<PAIR>(to + 4u, ds + (uint64_t)((2 * T * kScaleTile) >> 4));
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {  // 64 k each
                        if (kk * 64 >= left) continue;
                        // blocks of 16: a tile of scales per instruction; of 32: its lower or upper half
                        const int t = BLOCK == 16 ? kk : kk >> 1;
                        const uint32_t id = BLOCK == 16 ? 0u : 2u * (uint32_t)(kk & 1);
                        const uint64_t off = soff + (uint64_t)((kk * 32) >> 4);
                        mma_mx4<BLOCK, PAIR>(d_tmem, da0 + off, db0 + off, idesc | id << 4 | id << 29, sfa + 4u * t,
                                             sfb + (uint32_t)(4 * t * q_tiles), k > kb || kk > 0 ? 1u : 0u);
                    }
                    mx4_commit<PAIR>(bar_empty + 8 * s);
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if (elect_one()) mx4_commit<PAIR>(bar_tfull + 8 * b);
        }
        pdl_release();
        if (elect_one()) {
            if (PAIR) tc_commit_pair_mc(bar_drain, 0x1);
            else tc_commit(bar_drain);
        }
        mbar_wait_drain(bar_drain, 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------------------ epilogue
        const int quarter = warp & 3, half = warp >= 6 ? 1 : 0;  // the two warps of a quarter take turns
        const uint32_t turn_at = sbase + L.turn_off + (uint32_t)(warp - 2) * kTurnBytes;
        TurnedOut o = p.out;
        if (p.fa != nullptr) o.alpha *= *p.fa;
        if (p.fb != nullptr) o.alpha *= *p.fb;
        int local = 0;
        for (int u = first; u < units; u += stride, ++local) {
            int m0, n0;
            const int rows = tile_rows(u, m0, n0);
            const int b = buffers == 2 ? local & 1 : 0, turn = buffers == 2 ? local >> 1 : local;
            if (p.K > 0) {
                if (!mbar_wait(bar_tfull + 8 * b, (uint32_t)turn & 1u, wc)) break;
                tc_fence_after();
            }
            const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * 128);
            if (split > 1) {  // [row][128 columns] of sums, over the idle ring
                for (int c0 = 32 * half; c0 < rows; c0 += 64) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld16(lanes + (uint32_t)c0, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
                    tmem_ld16(lanes + (uint32_t)c0 + 16u, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c0 + c < rows)
                            st_shared_f32(sbase + (uint32_t)(c0 + c) * 512u + (uint32_t)(quarter * 32 + lane) * 4u,
                                          __uint_as_float(r[c]));
                }
                continue;
            }
            turned_rows<false>(o, turn_at, lanes, p.K == 0, m0, rows, n0 + (int)rank * 128 + quarter * 32, lane, half, [&] {
                            if (p.K == 0) return;
                            tc_fence_before();
                            __syncwarp();
                            if (lane != 0) return;
                            if (PAIR) mbar_arrive_tmem(dsmem_map(bar_tempty + 8 * b, 0));
                            else mbar_arrive(bar_tempty + 8 * b);
                        });
        }
    }

    // ---------------------------------------------------------- teardown
    if (!PAIR && split > 1) {
        __syncwarp();
        cluster_sync();  // every part's sums are there
        int m0, n0;
        const int rows = tile_rows(first, m0, n0);
        TurnedOut o = p.out;
        if (p.fa != nullptr) o.alpha *= *p.fa;
        if (p.fb != nullptr) o.alpha *= *p.fb;
        // a warp takes 32 columns of a row at a time
        for (int i = part * (kMx4Threads / 32) + warp; i < rows * 4; i += split * (kMx4Threads / 32)) {
            const int row = i >> 2, c = (i & 3) * 32 + lane, n = n0 + c;
            const uint32_t at = sbase + (uint32_t)row * 512u + (uint32_t)c * 4u;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = q < split ? dsmem_ld_f32(dsmem_map(at, (uint32_t)q)) : 0.f;
            float sum = v[0];
#pragma unroll
            for (int q = 1; q < 8; ++q) sum += v[q];
            if (n < o.N) turned_store(o, sum, m0 + row, n);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while others read its sums
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA frees TMEM or exits while the pair still uses it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, 512u);
        else tmem_dealloc(tmem_base, 512u);
    }
}

}  // namespace

}  // namespace dg

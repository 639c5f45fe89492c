// Products of groups of rows (the experts of a layer) on CTA pairs:
// tcgen05.mma.cta_group::2, TMA rings, accumulators in TMEM.
//
//   by rows   C[r] = A[r] B[g]            for the rows r of group g
//   by k      C[g] = sum_r X[r]^T Y[r]    over the rows r of group g
//
// The groups' rows are known on the device only, so every CTA reads the
// offsets, and all of them derive the same schedule: one launch, whatever the
// sizes, and no word of memory shared between CTAs.
//
// A tile is 256 columns of C by up to 256 of its rows, computed as C^T: the
// tensor core's M side (P) runs along C's columns, its N side (Q) along the
// rows.  N is a run-time field of the instruction, in steps of 32: a group of
// seven rows costs a 32-wide MMA and not a 256-row tile, which matters when a
// weight is read for a few rows (the copy of P then bounds the kernel), and
// the ragged ends of large groups cost 16 rows on average instead of 128.
//
// By k, both operands are MN-major and the last rows of a group are followed
// by the next group's.  Their copies are cut by the tensor map itself: the map
// has the rows as two dims of the same stride, the inner one as long as the
// box (H rows).  A box that starts at inner coordinate H - v has v rows inside
// and the others out of bounds, which arrive as zeros; the outer coordinate,
// the row behind the last one minus H, makes up for it.  Nothing is masked by
// threads, and a NaN in the next group's rows is never multiplied.  Every
// coordinate inside such a map is an element of the operand, so the row behind
// the last one has to be H at least: boxes that end in the first 128 rows are
// loaded 16 rows at a time, and those that end in the first 16 row by row
// (rows past the group are then asked for past the operand's end).
//
// What bounds it (B200): HBM where a weight meets few rows (64 rows over 8
// groups of 4096 x 14336 BF16 in 155-165 us, 5.7-6.1 TB/s); the tensor core and
// the power cap in large products (8192 rows, K = 14336, N = 4096: 705 us with a
// cold cache, 805-873 back to back); the copies by k, whose operands both arrive
// as 128-byte columns (8192 rows, 8 dW of 4096 x 4096: 204 us cold, 207-250 back
// to back, 1268 cycles per 1024 of MMAs).
//
// The tensor core truncates when it adds to an accumulator: a sum of 14336
// products of BF16 normal values came out 1.6e-5 low, of 4096 4.4e-6, and 65536
// positive products of F16 4.3e-4, twice F16's own rounding.  A sum therefore
// starts a fresh accumulator every 2048 k (E4M3, whose steps are 32 k: 4096; 65536
// positive products in one came out 5.9e-5 low), whatever the type of C, and the
// epilogue adds them up: the first part's accumulator holds the sum, the others
// are made in the other one, one after the other.  Each part after the first
// costs a pause of some 1700 cycles, in which nothing is multiplied (2048 rows
// over 4 groups with a cold cache, N = 4096, BF16: 75 -> 78 us at K = 4096, 217 ->
// 231 at 14336; in calls back to back, at the power cap, up to 3.5 %).  Sums kept
// in registers, which would need no pause, spilled and slowed calls of one part.
#pragma once

#include <climits>

#include "common.cuh"
#include "turned_out.cuh"
#include "uniform.cuh"

namespace dg {

constexpr int kGroupsMost = 1024;

struct GroupedParams {
    const int64_t *offsets;  // groups + 1
    int32_t groups;
    int32_t R;               // rows of all groups: the offsets' upper bound
    int32_t K;               // by rows: depth; by k: 0 where the product is left out, else anything
    int32_t Mo;              // by k: C's rows per group
    int32_t tile_w;          // by k: tile's rows of C; by rows: the most
    int32_t tiles_n;         // 256-column tiles of C
    int32_t stages;
    int32_t q_rows;          // ring space of Q: rows per CTA and sub-block, 16 to 128, a power of two
    int32_t p_swap_g;        // by rows: P's map has the group before its second dim
    int32_t p_one_g;         // by rows: all groups share one B
    int32_t k_chunk;         // k per accumulator (a multiple of a stage's)
    uint32_t idesc;          // instruction descriptor without N
    TurnedOut out;           // of group 0
    int64_t out_gs;          // by k: bytes between groups of C
    int32_t scale_n_gs;      // elements between groups of scale_n and of the bias
    int *err_word;
    uint64_t timeout_ns;
    int32_t stall_loader;    // test hook: the loaders issue nothing
    int32_t pdl;
};

// By rows: B as {K or N, N or K, group}, then A in boxes of 16, 32, 64 and 128
// rows.  By k: Y (P), cut, in boxes of a stage's rows, 16 rows and one, then X
// (Q) likewise.
struct GroupedMaps {
    CUtensorMap m[6];
};

namespace {

constexpr int kGroupThreads = 64 + 32 * kTurnWarps;
constexpr int kPRows = 128;  // P's rows (columns of C) per CTA

struct GroupLayout {
    uint32_t a_sub, a_bytes, b_sub, b_bytes, stage_bytes, turn_off, bar_off, aux_off, table_off, total;
};

__host__ __device__ inline GroupLayout group_layout(int stages, int ksub, int q_rows, int groups) {
    GroupLayout L;
    L.a_sub = kPRows * 128;
    L.a_bytes = (uint32_t)ksub * L.a_sub;
    L.b_sub = (uint32_t)q_rows * 128;
    L.b_bytes = (uint32_t)ksub * L.b_sub;
    L.stage_bytes = L.a_bytes + L.b_bytes;
    L.turn_off = L.stage_bytes * stages;
    L.bar_off = L.turn_off + kTurnWarps * kTurnBytes;
    L.aux_off = L.bar_off + 8 * (2 * stages + 5);
    L.table_off = L.aux_off + 16;  // start, size, tiles before
    L.total = L.table_off + 4 * (3 * (uint32_t)groups + 1) + 1024;
    return L;
}

struct GroupTables {
    const int *start, *size, *before;
};

// One tile: rows [r0, r0 + rows) of C (of group g's C, by k) and columns from n0.
struct GroupUnit {
    int g, r0, rows, w, n0;
    int k0, k;  // by k: first row of the sum; both: its length
};

template <bool BYK>
__device__ __forceinline__ bool group_unit(const GroupedParams &p, const GroupTables &t, int u, GroupUnit &x) {
    if (BYK) {
        const int tiles_m = (p.Mo + p.tile_w - 1) / p.tile_w, per = tiles_m * p.tiles_n;
        if (u >= p.groups * per) return false;
        x.g = u / per;
        const int i = u - x.g * per;
        x.n0 = i / tiles_m * 256;
        x.r0 = i % tiles_m * p.tile_w;
        x.w = p.tile_w;
        x.rows = min(p.tile_w, p.Mo - x.r0);
        x.k0 = t.start[x.g];
        x.k = p.K == 0 ? 0 : t.size[x.g];
        return true;
    }
    const int q = u / p.tiles_n;
    if (q >= t.before[p.groups]) return false;
    int lo = 0, hi = p.groups;  // before[lo] <= q < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.before[mid] <= q) lo = mid;
        else hi = mid;
    }
    // a group's row tiles are neighbours: pairs that run at the same time share P's tile
    const int tiles = t.before[lo + 1] - t.before[lo], i = u - t.before[lo] * p.tiles_n;
    const int tile = i % tiles, size = t.size[lo];
    const int w = ((size + tiles - 1) / tiles + 31) & ~31;  // tiles of one width: none is a sliver
    x.g = lo;
    x.n0 = i / tiles * 256;
    x.w = w;
    x.r0 = t.start[lo] + tile * w;
    x.rows = min(w, size - tile * w);
    x.k0 = 0;
    x.k = p.K;
    return true;
}

// group_unit by a whole warp, in uniform registers.
template <bool BYK>
__device__ __forceinline__ bool warp_unit(const GroupedParams &p, const GroupTables &t, int u, GroupUnit &x) {
    const bool any = group_unit<BYK>(p, t, u, x);
    if (!__any_sync(0xffffffffu, any)) return false;
    x.g = uniform(x.g);
    x.r0 = uniform(x.r0);
    x.w = uniform(x.w);
    x.n0 = uniform(x.n0);
    x.k0 = uniform(x.k0);
    x.k = uniform(x.k);
    return true;
}

// The groups' rows from the offsets, checked: a group whose offsets decrease
// or leave [0, R] has no rows and is reported.  Returns whether the calling
// thread met one.
__device__ __forceinline__ bool group_tables(const int64_t *offsets, int groups, int R, int *err_word, int *start,
                                             int *size) {
    bool bad = false;
    for (int g = threadIdx.x; g < groups; g += blockDim.x) {
        const int64_t a = offsets[g], b = offsets[g + 1];
        const bool ok = a >= 0 && a <= b && b <= R;
        if (!ok && err_word) atomicExch(err_word, (int)DG_ERR_VALUE);
        bad |= !ok;
        start[g] = ok ? (int)a : 0;
        size[g] = ok ? (int)(b - a) : 0;
    }
    return bad;
}

// By rows, one warp, after a bad group: groups that begin in front of the end
// of an earlier one have no rows either.  No row then belongs to two groups, and
// all groups together have at most R rows, which the grid and the counts of tiles
// rely on.  (Offsets that nowhere decrease have no such groups.)
__device__ __forceinline__ void group_disjoint(const int *start, int *size, int groups, int lane) {
    int end = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
        const int g = g0 + lane, n = g < groups ? size[g] : 0, from = g < groups ? start[g] : 0;
        int m = n > 0 ? from + n : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, m, d);
            if (lane >= d) m = max(m, v);
        }
        const int left = __shfl_up_sync(0xffffffffu, m, 1), before = lane > 0 ? max(end, left) : end;
        if (n > 0 && from < before) size[g] = 0;
        end = max(end, __shfl_sync(0xffffffffu, m, 31));
    }
    __syncwarp();
}

// One warp: the tiles of at most w rows before each group.
__device__ __forceinline__ void group_scan(const int *size, int *before, int groups, int w, int lane) {
    int sum = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
        const int n = g0 + lane < groups ? (size[g0 + lane] + w - 1) / w : 0;
        int s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += v;
        }
        if (g0 + lane < groups) before[g0 + lane] = sum + s - n;
        sum += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) before[groups] = sum;
}

// By rows, one warp: the width of tiles, and the tiles before each group.
// A pair takes a k block of 64 in about 295 + 1.15 w cycles (its copies, at
// some 57 bytes per cycle and SM), and the grid runs in whole rounds: narrower
// tiles are worth it where they fill the last round.
__device__ __forceinline__ void group_tiles(const GroupedParams &p, const int *size, int *before, int lane, int pairs) {
    int best = p.tile_w;
    float least = 0.f;
    for (int w = p.tile_w; w >= 32; w -= 32) {
        int n = 0;
        for (int g = lane; g < p.groups; g += 32) n += (size[g] + w - 1) / w;
        n = __reduce_add_sync(0xffffffffu, n);
        const int64_t units = (int64_t)n * p.tiles_n;
        const float cost = (float)((units + pairs - 1) / pairs) * (295.f + 1.15f * (float)w);
        if (w == p.tile_w || cost < least) {
            least = cost;
            best = w;
        }
    }
    group_scan(size, before, p.groups, best, lane);
}

// By k: rows [row, row + v) of one operand, columns c0 .. c0 + cols - 1, to
// MN-major boxes of KD rows; the rest of v's last 16 rows becomes zeros.
template <int KD, int BK>
__device__ __forceinline__ void load_cut(uint32_t dst, const CUtensorMap *m, uint32_t full, int c0, int cols, int row,
                                         int v, int R) {
    const int end = row + v;
    for (int c = 0; c < cols; c += BK, dst += KD * 128) {
        if (end >= KD) {
            tma_load_3d_pair(dst, m, full, c0 + c, KD - v, end - KD);
            continue;
        }
        for (int i = 0; i < v; i += 16) {
            const int some = min(16, v - i), last = row + i + some;
            if (last >= 16) {
                tma_load_3d_pair(dst + i * 128, m + 1, full, c0 + c, 16 - some, last - 16);
            } else {
                for (int j = 0; j < 16; ++j)
                    tma_load_2d_pair(dst + (i + j) * 128, m + 2, full, c0 + c, j < some ? row + i + j : R);
            }
        }
    }
}

template <bool FP8, int KSUB, bool P_MN, bool BYK>
__global__ void __launch_bounds__(kGroupThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps maps, const GroupedParams p) {
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int BK = 128 / ES;         // elements of a 128-byte row
    constexpr int KD = KSUB * BK;        // k per stage
    constexpr int UK = FP8 ? 32 : 16;    // k per instruction
    constexpr uint32_t kMnBox = (uint32_t)KD * 128;  // an MN-major box: KD rows of k, 128 bytes each

    if (threadIdx.x == 64 && p.K > 0 && (!BYK || p.R >= KD)) {
        tma_prefetch_desc(&maps.m[0]);
        if (BYK) tma_prefetch_desc(&maps.m[3]);
    }
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const GroupLayout L = group_layout(p.stages, KSUB, p.q_rows, p.groups);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + L.bar_off;
    const uint32_t bar_empty = bar_full + 8 * p.stages;
    const uint32_t bar_tfull = bar_empty + 8 * p.stages;
    const uint32_t bar_tempty = bar_tfull + 16;
    const uint32_t bar_drain = bar_tempty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L.aux_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L.aux_off + 4);
    int *start = reinterpret_cast<int *>(smem + L.table_off), *size = start + p.groups, *before = size + p.groups;

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const WaitCtl wc{abort_flag, p.err_word, p.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 2 * kTurnWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512u);
        tmem_relinquish_pair();
    }
    // everything above touches this pair's own memory only; what follows reads
    // what the previous kernel may have written
    pdl_wait();
    bool bad = group_tables(p.offsets, p.groups, p.R, p.err_word, start, size);
    tc_fence_before();
    bad = __syncthreads_or(bad);
    if (!BYK) {
        if (warp == 0) {
            if (bad) group_disjoint(start, size, p.groups, lane);
            group_tiles(p, size, before, lane, pairs);
        }
        __syncthreads();
    }
    __syncwarp();
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem_base = uniform(*tmem_slot);
    const GroupTables tables{start, size, before};

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        const int stages = p.stages;
        const bool stall = p.stall_loader == 1;
        int it = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        GroupUnit x, next;
        int u = pair;
        bool more = warp_unit<BYK>(p, tables, u, x);
        for (; ok && more; x = next) {
            const int h = x.w / 2;  // this CTA's rows of the tile
            const int n0 = x.n0 + (int)rank * kPRows, r0 = x.r0 + (int)rank * h;
            // by rows, one copy per sub-block: its fixed cost is that of some 55 rows
            const int size_at = h <= 16 ? 0 : h <= 32 ? 1 : h <= 64 ? 2 : 3, box = BYK ? h : 16 << size_at;
            const CUtensorMap *const mq = &maps.m[BYK ? 3 : 1 + size_at];
            const uint32_t tx_full = 2u * (L.a_bytes + (uint32_t)(KSUB * box) * 128u);
            const int g = p.p_one_g ? 0 : x.g;
            for (int k = 0; k < x.k; k += KD, ++it) {
                if (!warp_wait(bar_empty + 8 * s, ph ^ 1u, wc)) {
                    ok = false;
                    break;
                }
                if (!stall && elect_one()) {
                    const uint32_t full = dsmem_map(bar_full + 8 * s, 0);
                    uint32_t tx = tx_full;
                    if (BYK && x.k0 + min(k + KD, x.k) < KD)  // in boxes of 16 rows, as many as there are
                        tx = 2u * (uint32_t)((kPRows + h) / BK * ((min(KD, x.k - k) + 15) / 16)) * 2048u;
                    if (leader) mbar_arrive_expect_tx(bar_full + 8 * s, tx);
                    const uint32_t as = sbase + s * L.stage_bytes, bs = as + L.a_bytes;
                    if (BYK) {
                        const int v = min(KD, x.k - k), row = x.k0 + k;
                        load_cut<KD, BK>(as, &maps.m[0], full, n0, kPRows, row, v, p.R);
                        load_cut<KD, BK>(bs, mq, full, r0, h, row, v, p.R);
                    } else {
                        if (P_MN) {
#pragma unroll
                            for (int c = 0; c < kPRows / BK; ++c)
                                tma_load_3d_pair(as + c * kMnBox, &maps.m[0], full, n0 + c * BK, p.p_swap_g ? g : k,
                                                 p.p_swap_g ? k : g);
                        } else {
#pragma unroll
                            for (int j = 0; j < KSUB; ++j)
                                tma_load_3d_pair(as + j * L.a_sub, &maps.m[0], full, k + j * BK, p.p_swap_g ? g : n0,
                                                 p.p_swap_g ? n0 : g);
                        }
#pragma unroll
                        for (int j = 0; j < KSUB; ++j) tma_load_2d_pair(bs + j * L.b_sub, mq, full, k + j * BK, r0);
                    }
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
                // finding a unit takes some 1000 cycles: while the first copies of this one are on their way
                if (k == 0) more = warp_unit<BYK>(p, tables, u += pairs, next);
            }
            if (x.k == 0) more = warp_unit<BYK>(p, tables, u += pairs, next);
        }
        if (!leader) pdl_release();
        // full[] of the even CTA counts both CTAs' bytes: once its last
        // phases complete, every copy of the pair has landed
        if (leader && !stall)
            for (int d = 1; d <= stages && it - d >= 0; ++d) {
                const int j = it - d;
                mbar_wait_drain(bar_full + 8 * (j % stages), (uint32_t)(j / stages) & 1u, p.timeout_ns);
            }
    } else if (warp == 1) {
        // ----------------------------------------- MMA issuer (even CTA only)
        if (leader) {
            const int stages = p.stages;
            const uint32_t stage_bytes = L.stage_bytes;
            constexpr bool Q_MN = BYK;
            constexpr uint32_t p_kstep = P_MN ? UK * 128 : UK * ES, q_kstep = Q_MN ? UK * 128 : UK * ES;
            constexpr int kSteps = 128 / (UK * ES);  // instructions per sub-block
            const uint32_t p_sstep = P_MN ? kSteps * p_kstep : L.a_sub, q_sstep = Q_MN ? kSteps * q_kstep : L.b_sub;
            const uint64_t da0 = make_sw128_desc(sbase, P_MN ? kMnBox : 16u, 1024);
            const uint64_t db0 = make_sw128_desc(sbase + L.a_bytes, Q_MN ? kMnBox : 16u, 1024);
            int s = 0, b = 0, uses[2] = {0, 0};  // the accumulator in turn, and the uses of each
            uint32_t ph = 0;
            bool ok = true;
            GroupUnit x, next;
            int u = pair;
            bool more = warp_unit<BYK>(p, tables, u, x);
            for (; ok && more; x = next) {
                if (x.k == 0) {
                    more = warp_unit<BYK>(p, tables, u += pairs, next);
                    continue;
                }
                const uint32_t idesc = p.idesc | (uint32_t)(x.w >> 3) << 17;
                int at = b;  // a sum's first part is made in this accumulator, the others in the other one
                uint32_t d_tmem = tmem_base;
                for (int k = 0, kc = 0; k < x.k; k += KD, kc += KD) {
                    if (kc == p.k_chunk) {
                        if (elect_one()) tc_commit_pair_mc(bar_tfull + 8 * at, 0x3);
                        at = b ^ 1;
                        kc = 0;
                    }
                    if (kc == 0) {
                        if (!warp_wait(bar_tempty + 8 * at, ((uint32_t)(at ? uses[1] : uses[0]) & 1u) ^ 1u, wc)) {
                            ok = false;
                            break;
                        }
                        if (at) ++uses[1];
                        else ++uses[0];
                        tc_fence_after();
                        d_tmem = tmem_base + (uint32_t)(at * 256);
                    }
                    if (!warp_wait(bar_full + 8 * s, ph, wc)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t soff = (uint64_t)((s * stage_bytes) >> 4);
                    const int some = x.k - k;
                    if (elect_one()) {
#pragma unroll
                        for (int sub = 0; sub < KSUB; ++sub) {
#pragma unroll
                            for (int kk = 0; kk < kSteps; ++kk) {
                                if (sub * BK + kk * UK >= some) continue;  // zeros past the end of k
                                const uint64_t da = da0 + soff + (uint64_t)((sub * p_sstep + kk * p_kstep) >> 4);
                                const uint64_t db = db0 + soff + (uint64_t)((sub * q_sstep + kk * q_kstep) >> 4);
                                const uint32_t acc = (kc > 0 || sub > 0 || kk > 0) ? 1u : 0u;
                                if (FP8) umma_f8_pair(d_tmem, da, db, idesc, acc);
                                else umma_f16_pair(d_tmem, da, db, idesc, acc);
                            }
                        }
                        tc_commit_pair_mc(bar_empty + 8 * s, 0x3);  // the stage is free in both CTAs
                    }
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (k == 0) more = warp_unit<BYK>(p, tables, u += pairs, next);  // beside the first MMAs
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair_mc(bar_tfull + 8 * at, 0x3);
                b ^= 1;  // free before the sum is, if that had several parts
            }
            pdl_release();
            if (elect_one()) tc_commit_pair_mc(bar_drain, 0x1);
            mbar_wait_drain(bar_drain, 0, p.timeout_ns);
        }
    } else {
        // ------------------------------------------- epilogue (both CTAs)
        const int quarter = warp & 3, half = warp >= 6 ? 1 : 0;  // the two warps of a quarter take turns
        const uint32_t turn = sbase + L.turn_off + (uint32_t)(warp - 2) * kTurnBytes;
        int b = 0, uses[2] = {0, 0};
        GroupUnit x;
        for (int u = pair; group_unit<BYK>(p, tables, u, x); u += pairs) {
            TurnedOut o = p.out;
            if (BYK) o.c += x.g * p.out_gs;
            const int64_t gs = (int64_t)x.g * p.scale_n_gs;
            if (o.scale_n != nullptr) o.scale_n += gs;
            if (o.bias_n != nullptr) o.bias_n += gs;
            const int n0 = x.n0 + (int)rank * kPRows + quarter * 32;
            const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
            const uint32_t acc = lanes + (uint32_t)(b * 256), part = lanes + (uint32_t)((b ^ 1) * 256);
            const uint32_t empty_bar = dsmem_map(bar_tempty + 8 * b, 0), part_empty = dsmem_map(bar_tempty + 8 * (b ^ 1), 0);
            bool ok = true;
            for (int k = 0; k < x.k; k += min(p.k_chunk, x.k - k)) {
                const int at = k > 0 ? b ^ 1 : b;
                if (!mbar_wait(bar_tfull + 8 * at, (uint32_t)(at ? uses[1] : uses[0]) & 1u, wc)) {
                    ok = false;
                    break;
                }
                if (at) ++uses[1];
                else ++uses[0];
                tc_fence_after();
                if (x.k <= p.k_chunk) break;
                if (k == 0) continue;
                // a further part: added to the first one's accumulator
                for (int c0 = 32 * half; c0 < x.rows; c0 += 64) turned_add(acc + (uint32_t)c0, part + (uint32_t)c0);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_tmem(part_empty);
                tmem_st_wait();
            }
            if (!ok) break;
            turned_rows<FP8>(o, turn, acc, x.k == 0, x.r0, x.rows, n0, lane, half, [&] {
                if (x.k == 0) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_tmem(empty_bar);
            });
            if (x.k > 0) b ^= 1;
        }
    }

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA frees TMEM or exits while the pair still uses it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512u);
    }
}

}  // namespace

}  // namespace dg

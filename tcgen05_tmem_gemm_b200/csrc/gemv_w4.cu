// Matrix-vector products with 4-bit weights for up to 8 rows of activations:
// y = act(alpha * x W + beta * y + bias), W[k][n] = scale[n][g] (code - zero).
//
// Mathematics.  Inside a group, sum_k x (code - zero) scale = scale * sum_k x
// (code - zero), and code - zero is an integer of at most 5 bits, exact in
// BF16 and F16.  So the warp-level tensor instruction (m16n8k16) multiplies
// 16 columns of W (its M side) with up to 8 rows of x (its N side) in FP32,
// and a group's FP32 sum is scaled once: per weight there is only the
// unpacking (11 instructions per 8 codes), whatever the number of rows.  On
// CUDA cores eight rows would cost eight multiply-adds per weight more.  The
// tensor core is idle otherwise (an 8-row tile wastes nothing that counts),
// so m16n8k16 straight from registers serves where tcgen05's 128-row tiles
// with operands in shared memory would need the unpacked weights written
// there first.
//
// Unpacking.  A 32-bit word w holds the codes of k .. k+7; (w >> 4j) &
// 0x000F000F are the codes of k+j and k+j+4 in the low bits of two 16-bit
// halves.  OR-ed into the significand of 128 (BF16) or 1024 (F16) they read
// as 128 + code or 1024 + code, and one packed add of -(128 + zero) leaves
// code - zero exactly (the usual conversion of small integers through a
// floating-point number's significand).  F16's longer significand also takes
// the codes of odd j four bits higher (1024 + 16 code), where a packed
// multiply-add by 1/16 leaves the same and saves the shift.  The pairs
// (k+j, k+j+4) fix the order in which a thread meets k; x is staged in shared
// memory in the same order.
//
// What bounds it.  1 x 4096 x 128000 (BF16, groups of 128, zero points): 73 us,
// 3.7 TB/s.  No unit is full: HBM 44 %, issue slots 56 %, the pipe of the
// shifts and masks 51 %.  Fourteen warps per SM (registers) run chains of
// dependent instructions: a warp waits 1.6 cycles per instruction for the one
// before it, 0.7 for the integer pipe, 0.6 for memory and 0.5 at barriers.
// Small products are bound by their start: about 6 us until the first codes
// have come and x is staged.
//
// Work split.  It streams W once, so what counts is bytes in flight and few
// instructions per byte.  A warp owns 16 columns and a share of k, in steps of
// 128 k; every lane copies the 16 bytes of each of its two columns that it will
// itself unpack into a ring of two batches of steps in shared memory (cp.async:
// no registers, no synchronisation between lanes, bytes past a column's end
// arrive as zeros).  A block is column tiles x warps along k
// over one staged slice of x; blocks of a cluster share k further where there
// are few columns.  Partial sums meet in shared memory and, across a cluster,
// in distributed shared memory, in a fixed order.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "sm100.cuh"

namespace dg {

namespace {

constexpr int kBlockK = 128;   // k per step of a warp: 16 bytes of codes per lane and column
// A batch of steps of a warp in the ring: per step, lane and column 16 bytes
// or, where the columns do not start at multiples of 16 (VEC false), per column
// the aligned 16-byte chunks that hold the batch's 256 bytes.
constexpr uint32_t kLooseColumn = (256 + 16) + 16;
constexpr int kBatch = 4;      // steps between waits
constexpr int kMaxWarps = 16;  // per block; at 128 registers a thread also per SM
constexpr int kMostX = 48 * 1024;  // most bytes of x staged by a block
__host__ __device__ constexpr uint32_t batch_bytes(bool vec) { return vec ? kBatch * 32 * 2 * 16 : 16 * kLooseColumn; }

// (w & mask) | bits in one instruction (two literals would take two).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

template <typename T>
struct Pair;  // packed 16-bit arithmetic of x's type

template <>
struct Pair<__nv_bfloat16> {
    struct Zero {  // -(128 + zero), twice
        uint32_t lo;
        __device__ __forceinline__ Zero from(int src) const { return Zero{__shfl_sync(0xffffffffu, lo, src)}; }
    };
    static __device__ __forceinline__ Zero zero(uint32_t z) { return Zero{z * 0x00010001u | 0xC300C300u}; }
    static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %3, %2;" : "=r"(r) : "r"(a), "r"(b), "r"(0x3F803F80u));
        return r;
    }
    // the pairs j = 0..3 of code - zero
    static __device__ __forceinline__ void unpack(uint32_t (&a)[4], uint32_t w, Zero z) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = add(and_or(w >> (4 * j), 0x000F000Fu, 0x43004300u), z.lo);
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1, const float (&c)[4]) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }
};

template <>
struct Pair<__half> {
    struct Zero {  // -(1024 + zero) and -(64 + zero), twice each
        uint32_t lo, hi;
        __device__ __forceinline__ Zero from(int src) const {
            return Zero{__shfl_sync(0xffffffffu, lo, src), __shfl_sync(0xffffffffu, hi, src)};
        }
    };
    static __device__ __forceinline__ Zero zero(uint32_t z) {
        return Zero{z * 0x00010001u | 0xE400E400u, z * 0x00100010u | 0xD400D400u};
    }
    static __device__ __forceinline__ void unpack(uint32_t (&a)[4], uint32_t w, Zero z) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = w >> (8 * h);
            const uint32_t even = and_or(v, 0x000F000Fu, 0x64006400u), odd = and_or(v, 0x00F000F0u, 0x64006400u);
            asm("fma.rn.f16x2 %0, %1, %3, %2;" : "=r"(a[2 * h]) : "r"(even), "r"(z.lo), "r"(0x3C003C00u));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[2 * h + 1]) : "r"(odd), "r"(0x2C002C00u), "r"(z.hi));
        }
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1, const float (&c)[4]) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }
};

// Copies the lane's 16 bytes of one column from byte b into its place, zeros
// past the column's `nbytes`.  The column starts at a multiple of 16.
__device__ __forceinline__ void copy_codes(uint32_t to, const uint8_t *row, int b, int nbytes) {
    const int n = min(max(nbytes - b, 0), 16);
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(row + (n > 0 ? b : 0)), "r"(n)
                 : "memory");
}

__device__ __forceinline__ void copy16(uint32_t slot, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(slot), "l"(src) : "memory");
}
// A batch's codes of 16 columns at any alignment: `bytes` bytes of each column
// from byte b on, as the aligned 16-byte chunks that hold them (17 for a whole
// batch; half a warp copies a column's first 16).  Bytes before a column or
// past its end are not read: the copy of a last chunk is cut short, a first
// chunk that the column starts inside of is put together byte by byte.
__device__ __forceinline__ void copy_loose(uint32_t to, uint8_t *to_ptr, const uint8_t *codes, int64_t stride, int n0,
                                           int N, int b, int bytes, int nbytes, int lane) {
    if (b >= 16 && bytes == kBatch * (kBlockK / 2) && b + bytes + 16 <= nbytes && n0 + 16 <= N) {  // all chunks whole
        const uint8_t *row = codes + (int64_t)(n0 + (lane >> 4)) * stride;
        const int64_t step = 2 * stride, off = b + 16 * (lane & 15);
        uint32_t at = to + (lane >> 4) * kLooseColumn + 16 * (lane & 15);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            copy16(at, reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(row) & ~uintptr_t(15)) + off);
            row += step;
            at += 2 * kLooseColumn;
        }
        if (lane < 16) {
            const uint8_t *last = codes + (int64_t)(n0 + lane) * stride;
            copy16(to + lane * kLooseColumn + 256,
                   reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(last) & ~uintptr_t(15)) + b + 256);
        }
        return;
    }
    auto chunk = [&](int col, int c) {
        const uint8_t *row = codes + (int64_t)min(n0 + col, N - 1) * stride;
        const int d = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        if (16 * c >= d + bytes) return;
        const int at = b - d + 16 * c;  // the chunk's first byte in the column
        if (at < 0) {
            for (int q = d; q < 16; ++q)
                if (q - d < nbytes) to_ptr[col * kLooseColumn + q] = row[q - d];
        } else {
            const int n = min(max(nbytes - at, 0), 16);
            if (n > 0)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + col * kLooseColumn + 16 * c),
                             "l"(row + at), "r"(n)
                             : "memory");
            else
                *reinterpret_cast<uint4 *>(to_ptr + col * kLooseColumn + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
    };
#pragma unroll 1
    for (int j = 0; j < 8; ++j) chunk(2 * j + (lane >> 4), lane & 15);
    if (lane < 16) chunk(lane, 16);
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Eight 16-bit x, h = k .. k+7, as the four pairs (k+j, k+j+4).
__device__ __forceinline__ uint4 x_pairs(const uint4 &h) {
    return make_uint4(__byte_perm(h.x, h.z, 0x5410), __byte_perm(h.x, h.z, 0x7632), __byte_perm(h.y, h.w, 0x5410),
                      __byte_perm(h.y, h.w, 0x7632));
}

// x of k .. k+7 of row r, element by element (eight loads in flight), zeros at
// and past K.
__device__ __noinline__ uint4 x_elements(const DevView &x, int r, int k, int K) {
    const char *row = x.ptr + axis_offset(x.row, r);
    uint32_t e[8];
    if (x.col.n <= 1) {
        const int64_t cs = x.col.stride[0];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = k + i < K ? *reinterpret_cast<const uint16_t *>(row + (k + i) * cs) : (uint16_t)0;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = k + i < K ? *reinterpret_cast<const uint16_t *>(row + axis_offset(x.col, k + i)) : (uint16_t)0;
    }
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// The raw bits of a scale, converted where it is used, so that the load can
// be in flight until then.
__device__ __forceinline__ uint32_t scale_bits(const char *row, int grp, int dtype) {
    if (dtype == DG_F32) return __ldg(reinterpret_cast<const uint32_t *>(row) + grp);
    return __ldg(reinterpret_cast<const uint16_t *>(row) + grp);
}
__device__ __forceinline__ float scale_value(uint32_t bits, int dtype) {
    if (dtype == DG_F32) return __uint_as_float(bits);
    if (dtype == DG_BF16) return __uint_as_float(bits << 16);
    return __half2float(__ushort_as_half((unsigned short)bits));
}

// How the runs of 32 k that the four lanes of a quad hold in one step share
// scales: SETS = 1, all four (groups that are multiples of 128); 2, lanes 0-1
// and 2-3 (multiples of 64); 4, each has its own.  A tensor instruction sums
// over the quad, so with several sets the sums are kept apart through x: a
// column of the N side whose x is zero in the other sets' lanes sums one set
// only.  PACKED: the columns hold 8 / SETS rows of x for every set at once;
// else one pass of instructions per set, over the same unpacked codes.
//
// Scales and zero points of this lane's two columns for one batch of steps, as
// loaded: SETS = 1, lane t holds those of the t-th step and the quad shares
// them by shuffles; else those of its own set in every step.
template <int SETS>
struct Scales {
    static constexpr int kN = SETS == 1 ? 1 : kBatch;
    uint32_t s0[kN], s1[kN], z0[kN], z1[kN];
};

struct W4Layout {
    uint32_t pitch, zero, ring, red, part, total;  // x: pitch bytes per row, then a step of zeros; the ring;
                                                    // red: the warps' sums; part: the block's
};

// A block of `tiles` column tiles and `kw` warps along k, each taking `steps`
// steps per round.
__host__ __device__ inline W4Layout w4_layout(int R, int tiles, int kw, int steps, bool vec) {
    W4Layout L;
    L.pitch = (uint32_t)(kw * steps * kBlockK * 2 + 64);  // rows 64 bytes apart modulo 128: no bank conflicts
    L.zero = (uint32_t)R * L.pitch;
    L.ring = (L.zero + 256 + 127) / 128 * 128;
    const uint32_t ring_bytes = (uint32_t)(tiles * kw) * 2 * batch_bytes(vec);
    L.red = L.ring;  // the sums take the ring's place after the last step
    L.part = L.ring + ring_bytes;
    L.total = L.part + (uint32_t)(tiles * 128 * 4);
    return L;
}

template <typename T, bool VEC, int SETS, bool PACKED>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) gemv_w4_kernel(const __grid_constant__ GemvW4Params p) {
    constexpr int kRows = PACKED ? 8 / SETS : 8;    // rows of x per set of columns
    constexpr int kPasses = PACKED ? 1 : SETS;
    pdl_wait();
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr uint32_t kStageBytes = 32 * 2 * 16, kColumn = kStageBytes / 2, kBatchBytes = batch_bytes(VEC);
    const W4Layout L = w4_layout(p.R, p.tiles, p.kw, p.steps, VEC);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = warp / p.kw, kw = warp - tile * p.kw;
    const int g = lane >> 2, t = lane & 3;
    const int n0 = (blockIdx.x * p.tiles + tile) * 16;
    const int nbytes = (p.K + 1) / 2;
    const int blocks_k = (p.K + kBlockK - 1) / kBlockK;
    const int per_round = p.kw * p.steps, stride = gridDim.y * per_round;

    // this lane's columns, g and g + 8 of the tile (clamped; the extra ones are not stored)
    const int64_t c0 = min(n0 + g, p.N - 1), c1 = min(n0 + g + 8, p.N - 1);
    const uint8_t *row0 = p.codes + c0 * p.code_stride, *row1 = p.codes + c1 * p.code_stride;
    const uint32_t shift0 = 8 * (uint32_t)(reinterpret_cast<uintptr_t>(row0) & 3);
    const uint32_t shift1 = 8 * (uint32_t)(reinterpret_cast<uintptr_t>(row1) & 3);
    // where this lane's words of the batch's first step lie (VEC false)
    const uint32_t loose0 = g * kLooseColumn + (uint32_t)(reinterpret_cast<uintptr_t>(row0) & 12) + 16 * t;
    const uint32_t loose1 = (g + 8) * kLooseColumn + (uint32_t)(reinterpret_cast<uintptr_t>(row1) & 12) + 16 * t;
    (void)shift0, (void)shift1, (void)loose0, (void)loose1;
    const char *srow0 = p.scales + c0 * p.scale_stride, *srow1 = p.scales + c1 * p.scale_stride;
    const uint8_t *zrow0 = p.zeros + c0 * p.zero_stride, *zrow1 = p.zeros + c1 * p.zero_stride;
    auto fetch = [&](int kb, int left) {
        Scales<SETS> q;
#pragma unroll
        for (int u = 0; u < Scales<SETS>::kN; ++u) {
            // (with two sets the first of the set's two runs, which may be the only one before K)
            const int k = SETS == 1 ? (kb + t) * kBlockK : (kb + u) * kBlockK + 128 / SETS * (t * SETS / 4);
            q.s0[u] = q.s1[u] = 0u;
            q.z0[u] = q.z1[u] = 8u;
            if ((SETS == 1 ? t : u) < left && k < p.K) {  // a run past the end has the scale 0 and the sum 0
                const int grp = p.group_shift >= 0 ? k >> p.group_shift : k / p.group;
                q.s0[u] = scale_bits(srow0, grp, p.scale_dtype);
                q.s1[u] = scale_bits(srow1, grp, p.scale_dtype);
                if (p.zeros) {
                    q.z0[u] = __ldg(zrow0 + grp);
                    q.z1[u] = __ldg(zrow1 + grp);
                }
            }
        }
        return q;
    };

    // This warp's batches of steps: in each round of per_round blocks of k (a cluster's blocks
    // take rounds in turn) p.steps consecutive steps.  The copies walk two batches ahead.
    uint8_t *const mine = smem + L.ring + (uint32_t)warp * 2 * kBatchBytes + (VEC ? (uint32_t)lane * 16 : 0u);
    const uint32_t ring = smem_u32(mine);
    int next_kb = blockIdx.y * per_round + kw * p.steps, next_left = p.steps;
    auto copy_batch = [&](uint32_t half) {
        const int n = min(min(next_left, kBatch), blocks_k - next_kb);
        if (n == kBatch && (next_kb + kBatch) * (kBlockK / 2) <= nbytes && VEC) {
            const uint8_t *a = row0 + next_kb * (kBlockK / 2) + 16 * t, *b = row1 + next_kb * (kBlockK / 2) + 16 * t;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                copy16(half + u * kStageBytes, a + u * (kBlockK / 2));
                copy16(half + u * kStageBytes + kColumn, b + u * (kBlockK / 2));
            }
        } else if (VEC) {
#pragma unroll 1
            for (int u = 0; u < n; ++u) {
                const int b = (next_kb + u) * (kBlockK / 2) + 16 * t;
                copy_codes(half + u * kStageBytes, row0, b, nbytes);
                copy_codes(half + u * kStageBytes + kColumn, row1, b, nbytes);
            }
        } else if (n > 0) {
            __syncwarp();  // every lane has read what lay here
            copy_loose(half, mine + (half - ring), p.codes, p.code_stride, n0, p.N, next_kb * (kBlockK / 2),
                       n * (kBlockK / 2), nbytes, lane);
        }
        copy_commit();
        next_kb += kBatch;
        next_left -= kBatch;
        if (next_left <= 0) {
            next_kb += next_left + stride - p.steps;
            next_left = p.steps;
        }
    };
    copy_batch(ring);
    copy_batch(ring + kBatchBytes);

    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t half = 0;
    // (a block of one column tile and one warp along k has 32 threads)
    for (int i = threadIdx.x; i < 64; i += blockDim.x) *reinterpret_cast<uint32_t *>(smem + L.zero + i * 4) = 0u;
    for (int kb_round = blockIdx.y * per_round; kb_round < blocks_k; kb_round += stride) {
        const int kb0 = kb_round + kw * p.steps;
        const int nst = min(p.steps, blocks_k - kb0);  // may be negative: nothing for this warp
        Scales<SETS> ahead = fetch(kb0, nst);
        if (kb_round != (int)blockIdx.y * per_round) __syncthreads();  // the previous round's x is read
        // x of this round, in the order the words meet it
        {
            const int chunks = min(per_round, blocks_k - kb_round) * 16;
            for (int r = 0; r < p.R; ++r)
                for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
                    // position [step][word c][lane t] holds k = 32 t + 8 c ..
                    const int k = (kb_round + (i >> 4)) * kBlockK + 32 * (i & 3) + 8 * ((i >> 2) & 3);
                    const uint4 h = p.x_vec16 && k + 8 <= p.K
                                        ? *reinterpret_cast<const uint4 *>(p.x.ptr + r * p.x_ld + (int64_t)k * 2)
                                        : x_elements(p.x, r, k, p.K);
                    *reinterpret_cast<uint4 *>(smem + r * L.pitch + i * 16) = x_pairs(h);
                }
        }
        __syncthreads();
        // this lane's x, column g of the N side; zeros where the column has no row or, with several
        // sets, not this lane's
        const uint32_t xrow = t * 16 + (g % kRows) * L.pitch + kw * p.steps * 256, xzero = t * 16 + L.zero;
        uint32_t xs[kPasses], xstep[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const bool real = g % kRows < p.R && (SETS == 1 || t * SETS / 4 == (PACKED ? g / kRows : i));
            xs[i] = real ? xrow : xzero;
            xstep[i] = real ? 256 : 0;
        }
        for (int st = 0; st < p.steps; st += kBatch) {
            const Scales<SETS> q = ahead;
            if (st + kBatch < nst) ahead = fetch(kb0 + st + kBatch, nst - st - kBatch);
            copy_wait<1>();
            if (!VEC) __syncwarp();  // the lanes copied for one another
            // plain loads: the compiler may move a step's loads over the step before
            auto step = [&](int u) {
                uint32_t w0[4], w1[4];
                if (VEC) {
                    const uint4 v0 = *reinterpret_cast<const uint4 *>(mine + half + u * kStageBytes);
                    const uint4 v1 = *reinterpret_cast<const uint4 *>(mine + half + u * kStageBytes + kColumn);
                    w0[0] = v0.x, w0[1] = v0.y, w0[2] = v0.z, w0[3] = v0.w;
                    w1[0] = v1.x, w1[1] = v1.y, w1[2] = v1.z, w1[3] = v1.w;
                } else {
                    const uint32_t *v0 = reinterpret_cast<const uint32_t *>(mine + half + loose0 + u * 64);
                    const uint32_t *v1 = reinterpret_cast<const uint32_t *>(mine + half + loose1 + u * 64);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w0[c] = __funnelshift_r(v0[c], v0[c + 1], shift0);
                        w1[c] = __funnelshift_r(v1[c], v1[c + 1], shift1);
                    }
                }
                const int at = SETS == 1 ? 0 : u;
                typename Pair<T>::Zero z0 = Pair<T>::zero(q.z0[at] & 15u), z1 = Pair<T>::zero(q.z1[at] & 15u);
                float s0 = scale_value(q.s0[at], p.scale_dtype), s1 = scale_value(q.s1[at], p.scale_dtype);
                if (SETS == 1) {  // lane u of the quad has this step's
                    z0 = z0.from((lane & ~3) | u);
                    z1 = z1.from((lane & ~3) | u);
                    s0 = __shfl_sync(0xffffffffu, s0, (lane & ~3) | u);
                    s1 = __shfl_sync(0xffffffffu, s1, (lane & ~3) | u);
                }
                const float none[4] = {0.f, 0.f, 0.f, 0.f};
                float d[kPasses][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t a[4], b[4];
                    Pair<T>::unpack(a, w0[c], z0);
                    Pair<T>::unpack(b, w1[c], z1);
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(smem + xs[i] + u * xstep[i] + c * 64);
                        if (c == 0) Pair<T>::mma(d[i], a[0], b[0], a[1], b[1], x.x, x.y, none);
                        else Pair<T>::mma(d[i], a[0], b[0], a[1], b[1], x.x, x.y, d[i]);
                        Pair<T>::mma(d[i], a[2], b[2], a[3], b[3], x.z, x.w, d[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    float f0 = s0, f1 = s1;
                    if (kPasses > 1) {  // the lane of this set
                        f0 = __shfl_sync(0xffffffffu, s0, (lane & ~3) | (4 / SETS * i));
                        f1 = __shfl_sync(0xffffffffu, s1, (lane & ~3) | (4 / SETS * i));
                    }
                    acc[0] = fmaf(f0, d[i][0], acc[0]);
                    acc[1] = fmaf(f0, d[i][1], acc[1]);
                    acc[2] = fmaf(f1, d[i][2], acc[2]);
                    acc[3] = fmaf(f1, d[i][3], acc[3]);
                }
            };
            if (st + kBatch <= nst) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) step(u);
            } else {
#pragma unroll
                for (int u = 0; u < kBatch - 1; ++u)
                    if (st + u < nst) step(u);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) xs[i] += kBatch * xstep[i];
            copy_batch(ring + half);
            half = kBatchBytes - half;
        }
    }
    copy_wait<0>();
    pdl_release();

    // The warps' sums: [tile][warp along k][column of the N side][16 columns of W], in the ring's place.
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem + L.red), *part = reinterpret_cast<float *>(smem + L.part);
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(warp * 8 + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[i];
    __syncthreads();
    const bool single = gridDim.y == 1;
    auto store = [&](int e, float sum) {
        const int n = (blockIdx.x * p.tiles + (e >> 7)) * 16 + (e & 15), r = (e >> 4) & 7;
        if (r >= p.R || n >= p.N) return;
        char *yp = const_cast<char *>(p.y.ptr);
        if (p.y_plain) yp += r * p.y_rs + n * p.y_cs;
        else yp += axis_offset(p.y.row, r) + axis_offset(p.y.col, n);
        float v = epi_value(sum, p.alpha, 1.f, p.beta, yp, p.y.dtype);
        if (p.bias != nullptr || p.act != DG_ACT_NONE) v = epi_fuse(v, p.bias, n, p.act, p.y.dtype != DG_F32);
        store_elem(yp, p.y.dtype, v);
    };
    for (int e = threadIdx.x; e < p.tiles * 128; e += blockDim.x) {
        if (((e >> 4) & 7) >= p.R) continue;
        float sum = 0.f;
        for (int i = 0; i < p.kw; ++i)
#pragma unroll
            for (int q = 0; q < (PACKED ? SETS : 1); ++q)  // a row's columns of the N side, one per set
                sum += red[((e >> 7) * p.kw + i) * 128 + (e & 127) + q * kRows * 16];
        if (single) store(e, sum);
        else part[e] = sum;
    }
    if (single) return;
    // each block of the cluster finishes its share of the outputs, adding in rank order
    __syncthreads();
    cluster_sync();
    const int ranks = gridDim.y;
    for (int e = (int)cluster_ctarank() + ranks * threadIdx.x; e < p.tiles * 128; e += ranks * blockDim.x) {
        if (((e >> 4) & 7) >= p.R) continue;
        float sum = 0.f;
        for (int q = 0; q < ranks; ++q) sum += dsmem_ld_f32(dsmem_map(smem_u32(part + e), q));
        store(e, sum);
    }
    cluster_sync();  // keep every block's sums alive until all remote reads are done
}

template <typename T, bool VEC, int SETS, bool PACKED>
cudaError_t run(const GemvW4Params &p, int split, cudaStream_t s) {
    static SmemLimit limit;
    auto kern = gemv_w4_kernel<T, VEC, SETS, PACKED>;
    const size_t smem = w4_layout(p.R, p.tiles, p.kw, p.steps, VEC).total;
    const cudaError_t e = limit.ensure(kern, smem, true);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3((p.N + 16 * p.tiles - 1) / (16 * p.tiles), split), dim3(32 * p.kw * p.tiles), smem, s,
                     dim3(1, split, 1), p.pdl, p);
}

template <typename T, bool VEC>
cudaError_t run_sets(const GemvW4Params &p, int split, cudaStream_t s) {
    if (p.group % 128 == 0) return run<T, VEC, 1, false>(p, split, s);
    if (p.group % 64 == 0) return p.R <= 4 ? run<T, VEC, 2, true>(p, split, s) : run<T, VEC, 2, false>(p, split, s);
    return p.R <= 2 ? run<T, VEC, 4, true>(p, split, s) : run<T, VEC, 4, false>(p, split, s);
}

// The shape of the launch: kw warps of a block share k, and `split` blocks of a cluster (which then stage
// a smaller slice of x each); a block has `tiles` tiles of columns.  The cheapest by a model in units
// of a warp's step: an SM's warps take turns, a warp costs about five steps besides its own, staging a
// chunk of x a third of one, a round of x behind the first eight, a cluster's exchange two; fourteen
// warps or fewer wait on latencies and take the same time.  Blocks that do not fit at once cost whole
// waves while there are few (B200: 1 x 10293 x 31689 121 us in 1.1 waves, 70 in one; 8 x 10240 x 31689
// 80 us with two blocks of eight warps per SM, 62 with one of sixteen; 1 x 4096 x 128000 73 us with
// four of four, 85 with one of sixteen).
struct Shape {
    int kw = 1, tiles = 1, steps = 1, split = 1;
};
Shape best_shape(const GemvW4Params &p, bool vec, int num_sms) {
    const int blocks_k = (p.K + kBlockK - 1) / kBlockK;
    const int64_t col_tiles = (p.N + 15) / 16;
    Shape best;
    double least = 0;
    for (int i = 0; i < 16 * kMaxWarps; ++i) {
        const int kw = 1 << (i & 3), split = 1 << (i >> 2 & 3), tiles = (i >> 4) + 1;
        if ((kw > 1 || split > 1) && kw * split > blocks_k) continue;
        if (tiles * kw > kMaxWarps || (tiles > 1 && tiles > col_tiles)) continue;
        if (tiles * kw < 4 && tiles < col_tiles) continue;  // blocks of four warps and more
        const int most = std::max(1, kMostX / (p.R * kBlockK * 2 * kw));  // steps whose x fits
        const int per_warp = (blocks_k + kw * split - 1) / (kw * split);
        const int rounds = (per_warp + most - 1) / most, steps = (per_warp + rounds - 1) / rounds;
        const int64_t blocks = (col_tiles + tiles - 1) / tiles * split;
        const int64_t smem = w4_layout(p.R, tiles, kw, steps, vec).total + 1024;
        const int64_t fit = std::min<int64_t>(kMaxWarps / (kw * tiles), 228 * 1024 / smem);
        if (fit == 0) continue;
        const int64_t resident = std::min<int64_t>(fit, (blocks + num_sms - 1) / num_sms);
        // a cluster's blocks lie in one group of some 18 SMs, not all of which are filled
        const double spread = split < 4 ? 1 : resident > 1 ? 0.9 : split == 4 ? 0.85 : 0.75;
        double waves = (double)blocks / (spread * (double)(resident * num_sms));
        waves = waves <= 3 ? std::ceil(waves) : waves + 0.3;
        const double chunks = (double)p.R * kw * steps * 16 / (32 * kw * tiles);
        const double alone = waves > 1 ? 8.0 / (double)(resident * resident) : 0;  // little runs while a block starts
        const double work = rounds * (steps + chunks / 3) + 5 + alone + 8 * (rounds - 1) + (split > 1 ? 2 : 0);
        const double cost = waves * work * std::max<double>(14, (double)(resident * kw * tiles));
        if (least == 0 || cost < least) {
            least = cost;
            best = Shape{kw, tiles, steps, split};
        }
    }
    return best;
}

// A thread's latest shapes, by the sizes they depend on (finding one takes
// as long as launching).
struct ShapeKey {
    int R, K, N, vec, num_sms;
};
Shape shape_of(const GemvW4Params &p, bool vec, int num_sms) {
    constexpr int kKept = 16;
    static thread_local ShapeKey keys[kKept] = {};
    static thread_local Shape shapes[kKept];
    static thread_local int next = 0;
    const ShapeKey key{p.R, p.K, p.N, vec ? 1 : 0, num_sms};
    for (int i = 0; i < kKept; ++i)
        if (keys[i].R == key.R && keys[i].K == key.K && keys[i].N == key.N && keys[i].vec == key.vec &&
            keys[i].num_sms == key.num_sms)
            return shapes[i];
    const Shape s = best_shape(p, vec, num_sms);
    keys[next] = key;
    shapes[next] = s;
    next = (next + 1) % kKept;
    return s;
}

}  // namespace

cudaError_t launch_gemv_w4(GemvW4Params p, int num_sms, cudaStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.codes) | (p.N > 1 ? (uintptr_t)p.code_stride : 0);
    const bool vec = at % 16 == 0;
    const Shape shape = shape_of(p, vec, num_sms);
    p.kw = shape.kw;
    p.tiles = shape.tiles;
    p.steps = shape.steps;
    p.group_shift = (p.group & (p.group - 1)) == 0 ? __builtin_ctz((unsigned)p.group) : -1;
    if (p.in_dtype == DG_BF16)
        return vec ? run_sets<__nv_bfloat16, true>(p, shape.split, s)
                   : run_sets<__nv_bfloat16, false>(p, shape.split, s);
    return vec ? run_sets<__half, true>(p, shape.split, s) : run_sets<__half, false>(p, shape.split, s);
}

}  // namespace dg

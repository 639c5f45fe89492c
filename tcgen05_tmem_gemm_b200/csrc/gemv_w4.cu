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
// code - zero exactly.  The pairs (k+j, k+j+4) fix the order in which a
// thread meets k; x is staged in shared memory in the same order.
//
// Work split.  It streams W once and is bound by HBM, so what counts is bytes
// in flight.  A block owns 16 * MT columns; its eight warps (and the blocks of
// its cluster) share k in blocks of 128.  A lane loads 16 bytes of a column's
// codes at a time, all loads of up to kBatch blocks of k at once, before x is
// staged, so the two trips to memory overlap.  Partial sums meet in shared
// memory and, across a cluster, in distributed shared memory, in a fixed
// order.
#include <atomic>

#include "common.cuh"
#include "sm100.cuh"

namespace dg {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockK = 128;   // k per step of a warp: 16 bytes of codes per lane and column
constexpr int kBatch = 4;      // steps whose loads are in flight together

template <typename T>
struct Pair;  // packed 16-bit arithmetic of x's type

template <>
struct Pair<__nv_bfloat16> {
    static constexpr uint32_t kMagic = 0x43004300u;     // 128, 128
    static constexpr uint32_t kNegMagic = 0xC300C300u;  // -128, -128
    static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <>
struct Pair<__half> {
    static constexpr uint32_t kMagic = 0x64006400u;     // 1024, 1024
    static constexpr uint32_t kNegMagic = 0xE400E400u;  // -1024, -1024
    static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// The four words a lane multiplies in one step.  Word c of lane t (t = lane %
// 4) holds k = 32 t + 8 c (kLaneMajor: a lane's 16 bytes as loaded) or
// k = 32 c + 8 t (kWordMajor: word c of all four lanes lies in one run of 32
// k, so groups of 32 can be scaled one by one).
enum Order { kLaneMajor, kWordMajor };

__device__ __forceinline__ int order_k(Order o, int c, int t) { return o == kLaneMajor ? 32 * t + 8 * c : 32 * c + 8 * t; }

// Lane-major to word-major: a 4 x 4 transpose among the four lanes of a quad.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
#pragma unroll
    for (int step = 1; step <= 2; ++step) {
        const bool hi = t & step;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int a = step == 1 ? 2 * p : p, b = a + step;  // the pair of words that trade places
            const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? w[a] : w[b], step);
            if (hi) w[a] = got;
            else w[b] = got;
        }
    }
}

// The codes of k .. k+7 (k a multiple of 8) of a column, bytes at or past
// `nbytes` as zero.
__device__ __forceinline__ uint32_t load_word_bytes(const uint8_t *row, int k, int nbytes) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k / 2 + i < nbytes) w |= (uint32_t)__ldg(row + k / 2 + i) << (8 * i);
    return w;
}

// One step's words of one column.  VEC: the alignment of every column's codes.
template <int VEC, Order O>
__device__ __forceinline__ void load_codes(uint32_t (&w)[4], const uint8_t *row, int k0, int t, int nbytes) {
    if (VEC == 16) {  // as the lane's 16 bytes; a word-major kernel transposes them before use
        const int b = k0 / 2 + 16 * t;
        if (b + 16 <= nbytes) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + b));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = load_word_bytes(row, k0 + 32 * t + 8 * c, nbytes);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = k0 + order_k(O, c, t);
            if (VEC == 4 && k / 2 + 4 <= nbytes) w[c] = __ldcs(reinterpret_cast<const uint32_t *>(row + k / 2));
            else w[c] = load_word_bytes(row, k, nbytes);
        }
    }
}

// One word's eight codes of two columns (16-row halves of the M side) times
// x: two tensor instructions.
template <typename T>
__device__ __forceinline__ void word_mma(float (&d)[4], uint32_t lo, uint32_t hi, uint32_t zlo, uint32_t zhi,
                                         const uint4 &x) {
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            a[2 * q] = Pair<T>::add(((lo >> (4 * (j + q))) & 0x000F000Fu) | Pair<T>::kMagic, zlo);
            a[2 * q + 1] = Pair<T>::add(((hi >> (4 * (j + q))) & 0x000F000Fu) | Pair<T>::kMagic, zhi);
        }
        Pair<T>::mma(d, a, j == 0 ? x.x : x.z, j == 0 ? x.y : x.w);
    }
}

// Eight consecutive x of one row as the four pairs (k+j, k+j+4).
__device__ __forceinline__ uint4 x_pairs(const GemvW4Params &p, int r, int k, bool vec) {
    uint32_t h[4];
    if (vec && k + 8 <= p.K) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p.x.ptr + axis_offset(p.x.row, r) + (int64_t)k * 2);
        h[0] = v.x;
        h[1] = v.y;
        h[2] = v.z;
        h[3] = v.w;
    } else {
        const char *row = p.x.ptr + axis_offset(p.x.row, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t e[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int kk = k + 2 * i + q;
                e[q] = kk < p.K ? *reinterpret_cast<const uint16_t *>(row + axis_offset(p.x.col, kk)) : 0u;
            }
            h[i] = e[0] | (e[1] << 16);
        }
    }
    return make_uint4(__byte_perm(h[0], h[2], 0x5410), __byte_perm(h[0], h[2], 0x7632),
                      __byte_perm(h[1], h[3], 0x5410), __byte_perm(h[1], h[3], 0x7632));
}

struct W4Layout {
    uint32_t pitch, red, part, total;  // x: pitch bytes per row; red: the warps' sums; part: the block's
};

// steps: the most steps of k any warp takes in one round.
__host__ __device__ inline W4Layout w4_layout(int R, int steps, int mt) {
    W4Layout L;
    L.pitch = (uint32_t)(kWarps * steps * kBlockK * 2 + 64);  // rows 64 bytes apart modulo 128: no bank conflicts
    L.red = (uint32_t)R * L.pitch;
    const uint32_t red_bytes = (uint32_t)(kWarps * mt * 128 * 4);
    L.part = L.red + red_bytes;
    L.total = L.part + (uint32_t)(mt * 128 * 4);
    return L;
}

// FINE: groups that are not whole multiples of 128 (word-major, one scale per
// 32 k), else one scale per step.
template <typename T, int MT, int VEC, bool FINE>
__global__ void __launch_bounds__(kThreads) gemv_w4_kernel(const GemvW4Params p) {
    constexpr Order O = (FINE || VEC != 16) ? kWordMajor : kLaneMajor;
    pdl_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    const W4Layout L = w4_layout(p.R, p.steps, MT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16 * MT;
    const int nbytes = (p.K + 1) / 2;
    const int blocks_k = (p.K + kBlockK - 1) / kBlockK;

    // this lane's columns: g and g + 8 of each 16 (clamped; the extra ones are not stored)
    const uint8_t *row[MT][2];
    int64_t col[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            col[m][h] = min(n0 + 16 * m + 8 * h + g, p.N - 1);
            row[m][h] = p.codes + col[m][h] * p.code_stride;
        }
    const int ses = elem_bytes(p.scale_dtype);

    float acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;

    // Rounds: kWarps * steps blocks of k at a time, a cluster's blocks taking
    // turns; warp w takes `steps` consecutive ones.
    const int per_round = kWarps * p.steps;
    for (int kb_round = blockIdx.y * per_round; kb_round < blocks_k; kb_round += gridDim.y * per_round) {
        const int kb0 = kb_round + warp * p.steps;
        const int nst = min(p.steps, blocks_k - kb0);  // may be negative: nothing for this warp
        uint32_t w[kBatch][MT][2][4];
        float sc[FINE ? kBatch : 1][MT][2];
        uint32_t zc[FINE ? kBatch : 1][MT][2];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (u < nst)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        load_codes<VEC, O>(w[u][m][h], row[m][h], (kb0 + u) * kBlockK, t, nbytes);
        // scales and zero points: lane t of a quad fetches step t's (or run t's of each
        // step, FINE) and the quad shares them by shuffles
#pragma unroll
        for (int u = 0; u < (FINE ? kBatch : 1); ++u) {
            const int k = FINE ? (kb0 + u) * kBlockK + 32 * t : (kb0 + t) * kBlockK;
            const bool ok = k < p.K && (FINE ? u : t) < nst;
            const int grp = ok ? k / p.group : 0;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sc[u][m][h] = ok ? load_elem(p.scales + col[m][h] * p.scale_stride + (int64_t)grp * ses,
                                                 p.scale_dtype)
                                     : 0.f;
                    const uint32_t z = !p.zeros ? 8u : ok ? p.zeros[col[m][h] * p.zero_stride + grp] & 15u : 0u;
                    zc[u][m][h] = Pair<T>::kNegMagic | (z * 0x00010001u);
                }
        }
        if (kb_round != (int)blockIdx.y * per_round) __syncthreads();  // the previous round's x is read
        // x of this round, in the order the words meet it
        for (int e = threadIdx.x; e < p.R * per_round * 16; e += kThreads) {
            const int r = e / (per_round * 16), i = e - r * (per_round * 16);
            const int kb = i >> 4, c = (i >> 2) & 3, q = i & 3;
            *reinterpret_cast<uint4 *>(smem + r * L.pitch + i * 16) =
                x_pairs(p, r, (kb_round + kb) * kBlockK + order_k(O, c, q), p.x_vec16);
        }
        __syncthreads();
        const uint8_t *xs = smem + g * L.pitch + warp * p.steps * 256 + t * 16;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (u >= nst) break;
            float d[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[m][i] = 0.f;
                if (O == kWordMajor && VEC == 16) {
                    quad_transpose(w[u][m][0], t);
                    quad_transpose(w[u][m][1], t);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (g < p.R) x = *reinterpret_cast<const uint4 *>(xs + u * 256 + c * 64);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int su = FINE ? u : 0, src = FINE ? c : u;  // who holds this run's scale
                    const uint32_t z0 = __shfl_sync(0xffffffffu, zc[su][m][0], (lane & ~3) | src);
                    const uint32_t z1 = __shfl_sync(0xffffffffu, zc[su][m][1], (lane & ~3) | src);
                    word_mma<T>(d[m], w[u][m][0][c], w[u][m][1][c], z0, z1, x);
                    if (FINE || c == 3) {
                        const float s0 = __shfl_sync(0xffffffffu, sc[su][m][0], (lane & ~3) | src);
                        const float s1 = __shfl_sync(0xffffffffu, sc[su][m][1], (lane & ~3) | src);
                        acc[m][0] = fmaf(s0, d[m][0], acc[m][0]);
                        acc[m][1] = fmaf(s0, d[m][1], acc[m][1]);
                        acc[m][2] = fmaf(s1, d[m][2], acc[m][2]);
                        acc[m][3] = fmaf(s1, d[m][3], acc[m][3]);
                        if (FINE)
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[m][i] = 0.f;
                    }
                }
            }
        }
    }
    pdl_release();

    // The warps' sums: [warp][m][row r of x][16 columns].
    float *red = reinterpret_cast<float *>(smem + L.red), *part = reinterpret_cast<float *>(smem + L.part);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[((warp * MT + m) * 8 + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[m][i];
    __syncthreads();
    const bool single = gridDim.y == 1;
    auto store = [&](int e, float sum) {
        const int n = n0 + (e >> 7) * 16 + (e & 15), r = (e >> 4) & 7;
        if (r >= p.R || n >= p.N) return;
        char *yp = const_cast<char *>(p.y.ptr) + axis_offset(p.y.row, r) + axis_offset(p.y.col, n);
        const float v = epi_value(sum, p.alpha, 1.f, p.beta, yp, p.y.dtype);
        store_elem(yp, p.y.dtype, epi_fuse(v, p.bias, n, p.act, p.y.dtype != DG_F32));
    };
    for (int e = threadIdx.x; e < MT * 128; e += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += red[i * MT * 128 + e];
        if (single) store(e, sum);
        else part[e] = sum;
    }
    if (single) return;
    // each block of the cluster finishes its share of the outputs, adding in rank order
    __syncthreads();
    cluster_sync();
    const int ranks = gridDim.y;
    for (int e = (int)cluster_ctarank() + ranks * threadIdx.x; e < MT * 128; e += ranks * kThreads) {
        float sum = 0.f;
        for (int q = 0; q < ranks; ++q) sum += dsmem_ld_f32(dsmem_map(smem_u32(part + e), q));
        store(e, sum);
    }
    cluster_sync();  // keep every block's sums alive until all remote reads are done
}

template <typename T, int MT, int VEC, bool FINE>
cudaError_t run(const GemvW4Params &p, int split, cudaStream_t s) {
    static SmemLimit limit;
    auto kern = gemv_w4_kernel<T, MT, VEC, FINE>;
    const size_t smem = w4_layout(p.R, p.steps, MT).total;
    const cudaError_t e = limit.ensure(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, dim3((p.N + 16 * MT - 1) / (16 * MT), split), dim3(kThreads), smem, s, dim3(1, split, 1),
                     p.pdl, p);
}

template <typename T, int MT, int VEC>
cudaError_t run_fine(const GemvW4Params &p, int split, cudaStream_t s) {
    return p.group % kBlockK ? run<T, MT, VEC, true>(p, split, s) : run<T, MT, VEC, false>(p, split, s);
}

template <typename T>
cudaError_t run_vec(const GemvW4Params &p, int mt, int vec, int split, cudaStream_t s) {
    if (vec == 16) return mt == 2 ? run_fine<T, 2, 16>(p, split, s) : run_fine<T, 1, 16>(p, split, s);
    if (vec == 4) return run_fine<T, 1, 4>(p, split, s);
    return run_fine<T, 1, 1>(p, split, s);
}

}  // namespace

cudaError_t launch_gemv_w4(GemvW4Params p, int num_sms, cudaStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.codes) | (p.N > 1 ? (uintptr_t)p.code_stride : 0);
    const int vec = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 1;
    const int mt = (vec == 16 && p.R > 4) ? 2 : 1;
    const int tiles = (p.N + 16 * mt - 1) / (16 * mt);
    const int blocks_k = (p.K + kBlockK - 1) / kBlockK;
    // k split over a cluster while there are too few column tiles for three blocks per SM and every
    // warp keeps at least one block of k
    int split = 1;
    while (split < 8 && tiles * split * 2 <= num_sms * 3 && blocks_k >= kWarps * split * 2) split *= 2;
    const int per_warp = (blocks_k + kWarps * split - 1) / (kWarps * split);
    const int rounds = (per_warp + kBatch - 1) / kBatch;
    p.steps = (per_warp + rounds - 1) / rounds;
    if (p.in_dtype == DG_BF16) return run_vec<__nv_bfloat16>(p, mt, vec, split, s);
    if (p.in_dtype == DG_F16) return run_vec<__half>(p, mt, vec, split, s);
    return cudaErrorInvalidValue;
}

}  // namespace dg

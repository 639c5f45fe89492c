// Kernels of dg_quantize_mx4 and dg_dequantize_mx4.
//
// E2M1 has the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4 and 6.  A block of 32 values
// along k has an E8M0 scale, 2^floor(log2(largest) - 2), which brings the
// largest to [4, 8) (above 6 it is cut); a block of 16 an E4M3 scale, a sixth
// of the largest.  Everything is rounded to nearest, ties to even, and every
// division by a block's scale decides as the exact quotient would.
//
// They should be bound by HBM and no unit is full (8192 x 14336 BF16 on B200, 300
// MB: quantised in blocks of 32 in 59 us, of 16 in 70, with a factor 88; read back
// in 53; the bytes take 46).  With a factor 53 % of the issue slots and 32 % of
// DRAM are used, reading back 46 % and 41 %, and waiting for loads is the largest
// stall: 8 to 16 instructions per value, a third of the warps an SM holds, and
// a row loaded one row ahead of its use.
#include <algorithm>

#include "mx4_quant.h"
#include "umma_common.cuh"

namespace dg {
namespace {

// ------------------------------------------------------------ scales and codes

constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The byte of a block's scale from the largest magnitude's bits (NaN and
// infinities compare above every finite one), and the pair (s, r) with which
// mx4_unit makes x / s: for E8M0 the exact 1 / s, for E4M3 s and its rounded
// reciprocal.  A block with a NaN or an infinity has the scale NaN and
// codes of zero.
template <int BLOCK>
__device__ __forceinline__ uint32_t mx4_scale(uint32_t top, float &s, float &r) {
    if (BLOCK == 32) {
        const int e = max((int)(top >> 23) - 2, 0);  // a subnormal has exponent 0
        s = 0.f;
        r = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e): normal for every e up to 252
        if (top >= kInfBits) {
            r = 0.f;
            return 0xff;
        }
        return (uint32_t)e;
    }
    if (top >= kInfBits) {
        s = r = 0.f;
        return 0x7f;
    }
    // top / 6, rounded once (as quotient2 does; where the remainder underflows the scale is 0 in any case)
    const float x = __uint_as_float(top), sixth = 1.f / 6.f, y = x * sixth;
    const float want = fmaf(fmaf(-y, 6.f, x), sixth, y);
    const uint32_t code = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
    r = s > 0.f ? __frcp_rn(s) : 0.f;
    return code;
}

// Two FP32 values in one register pair, and the instructions that take two at
// a time.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// x / s but for the sign of a zero, from the rounded reciprocal r of s and -s:
// one correction of x r by the remainder, which the fused multiply-add gives
// exactly.  The result differs from the exact quotient by little more than half
// an ulp and is exact where the quotient is an FP32 number.
__device__ __forceinline__ Two quotient2(Two x, Two minus_s, Two r) {
    const Two y = mul2(x, r);
    return fma2(fma2(y, minus_s, x), r, y);
}

// Two values under their block's scale.  The quotient by an E4M3 number lies on
// E2M1's rounding borders exactly where the exact quotient does: with four
// significant bits in s no other comes within half an ulp of a border.
template <int BLOCK>
__device__ __forceinline__ Two mx4_unit(Two x, Two minus_s, Two r) {
    return BLOCK == 32 ? mul2(x, r) : quotient2(x, minus_s, r);
}

__device__ __forceinline__ float with_sign(float v, float x) {
    return __uint_as_float((__float_as_uint(v) & 0x7fffffffu) | (__float_as_uint(x) & 0x80000000u));
}

// Eight values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// And back.
__device__ __forceinline__ void e2m1x8_values(uint32_t e, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(e));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = t.x;
        v[2 * i + 1] = t.y;
    }
}

// The value of a scale's byte.
template <int BLOCK>
__device__ __forceinline__ float mx4_scale_value(uint32_t code) {
    if (BLOCK == 32)
        return code == 0xff ? __uint_as_float(0x7fffffffu) : __uint_as_float(code ? code << 23 : 1u << 22);
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(code & 0x7f), __NV_E4M3)));
}

// A division out of line: inlined at every use its code no longer fits the
// instruction cache.
__device__ __noinline__ float divided(float x, float t) { return __fdiv_rn(x, t); }

// The division by the matrix's factor: u = x / t, rounded once.
struct Factor {
    float t, size, r;       // t, |t| and its rounded reciprocal
    uint32_t flip;          // the codes' sign bits where t is negative
    bool divide, plain;     // plain: t is of a size for which quotient() holds
    __device__ explicit Factor(const float *scale) {
        divide = scale != nullptr;
        t = divide ? *scale : 1.f;
        size = fabsf(t);
        flip = t < 0.f ? 0x88888888u : 0u;
        plain = size >= 0x1p-60f && size <= 0x1p60f;
        r = plain ? __frcp_rn(size) : 0.f;
    }
    // x / |t|, but for the sign of a zero: correctly rounded, while nothing
    // underflows, because a second correction starts from a quotient within an
    // ulp (Markstein 1990, "Computation of elementary functions on the IBM RISC
    // System/6000 processor").
    __device__ __forceinline__ Two quotient(Two x) const {
        const Two ms(-size, -size), rr(r, r), q = quotient2(x, ms, rr);
        return fma2(fma2(q, ms, x), rr, q);
    }
};

// Below this magnitude of a block's largest value, or of its quotient, the
// quotients are divided one by one; above it a value whose remainder or quotient
// underflows is so small a part of the largest that its code is 0 in any case.
constexpr float kLeastPlain = 0x1p-90f;
constexpr float kMostPlain = 0x1p126f;  // and no quotient of the block is near the end of FP32

// 32 neighbouring k of a row as they lie in memory (zeros past K).
template <int DT>
struct Lot {
    static constexpr int ES = DT == DG_F32 ? 4 : 2;
    static constexpr int W = 8 * ES;  // words
    uint32_t w[W];
    __device__ __forceinline__ float operator[](int i) const {
        if (DT == DG_F32) return __uint_as_float(w[i]);
        if (DT == DG_BF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        return __half2float(__ushort_as_half((unsigned short)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu)));
    }
    // the largest magnitude of block b, as FP32; NaN if there is one (16-bit magnitudes order as integers)
    template <int BLOCK>
    __device__ __forceinline__ uint32_t top(int b) const {
        constexpr int N = W * BLOCK / 32;
        uint32_t m = 0;
        if constexpr (DT == DG_F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) m = max(m, w[b * N + i] & 0x7fffffffu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[b * N + i] & 0x7fff7fffu));
            m = max(m & 0xffffu, m >> 16);
            if (DT == DG_BF16) return m << 16;
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) & 0x7fffffffu;
        }
    }
};

// The codes of a lot's 32 values (the first n of them, n >= 32 for all) and, in
// the low bytes of the result, its 32 / BLOCK scales.
template <int DT, int BLOCK>
__device__ __forceinline__ uint32_t encode(const Lot<DT> &x, int n, const Factor &f, uint32_t (&e)[4]) {
    uint32_t scales = 0;
#pragma unroll
    for (int b = 0; b < 32 / BLOCK; ++b) {
        const uint32_t top = x.template top<BLOCK>(b);
        const float most = __uint_as_float(top);
        const bool plain = f.plain && (top == 0 || (most >= kLeastPlain && most * f.r >= kLeastPlain &&
                                                    most * f.r <= kMostPlain));  // zeros: lanes past K among them
        // the largest |x / t| is that of the largest |x|: rounding keeps the order
        uint32_t under = top;
        if (f.divide) {
            float q, unused;
            if (plain) f.quotient(Two(most, 0.f)).get(q, unused);
            else q = divided(most, f.size);
            under = abs_bits(q);
        }
        float s, r;
        const uint32_t code = mx4_scale<BLOCK>(under, s, r);
        if (b * BLOCK < n) scales |= code << (8 * b);
        const Two ms(-s, -s), rr(r, r);
        // each way a loop of its own: a branch per pair costs as much as the arithmetic
        if (!f.divide) {
#pragma unroll
            for (int j = 0; j < BLOCK / 8; ++j) {
                float u[8];
                const int at = b * BLOCK + 8 * j;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float x0 = x[at + i], x1 = x[at + i + 1];
                    mx4_unit<BLOCK>(Two(x0, x1), ms, rr).get(u[i], u[i + 1]);
                    if (BLOCK == 16) {
                        u[i] = with_sign(u[i], x0);
                        u[i + 1] = with_sign(u[i + 1], x1);
                    }
                }
                e[at / 8] = e2m1x8(u);
            }
        } else if (plain) {
#pragma unroll
            for (int j = 0; j < BLOCK / 8; ++j) {
                float u[8];
                const int at = b * BLOCK + 8 * j;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float x0 = x[at + i], x1 = x[at + i + 1];
                    mx4_unit<BLOCK>(f.quotient(Two(x0, x1)), ms, rr).get(u[i], u[i + 1]);
                    u[i] = with_sign(u[i], x0);
                    u[i + 1] = with_sign(u[i + 1], x1);
                }
                e[at / 8] = e2m1x8(u) ^ f.flip;
            }
        } else {
#pragma unroll
            for (int j = 0; j < BLOCK / 8; ++j) {
                float u[8];
                const int at = b * BLOCK + 8 * j;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float x0 = x[at + i], x1 = x[at + i + 1];
                    mx4_unit<BLOCK>(Two(divided(x0, f.size), divided(x1, f.size)), ms, rr).get(u[i], u[i + 1]);
                    u[i] = with_sign(u[i], x0);
                    u[i + 1] = with_sign(u[i + 1], x1);
                }
                e[at / 8] = e2m1x8(u) ^ f.flip;
            }
        }
        if (r == 0.f) {
#pragma unroll
            for (int j = 0; j < BLOCK / 8; ++j) e[b * BLOCK / 8 + j] = 0u;
        }
    }
    if (n < 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i + 8 > n) e[i] &= 8 * i >= n ? 0u : (1u << (4 * (n - 8 * i))) - 1u;
    }
    return scales;
}

// The 16 bytes of 32 codes, of which the first n exist.
__device__ __forceinline__ void store_codes(uint8_t *out, int align, const uint32_t (&e)[4], int n) {
    if (align == 16 && n >= 32) {
        *reinterpret_cast<uint4 *>(out) = make_uint4(e[0], e[1], e[2], e[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (align >= 4 && 8 * i + 8 <= n) {
            *reinterpret_cast<uint32_t *>(out + 4 * i) = e[i];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (8 * i + 2 * j < n) out[4 * i + j] = (uint8_t)(e[i] >> (8 * j));
        }
    }
}

// Four bytes of codes, of which the first n codes exist.
__device__ __forceinline__ uint32_t load_codes8(const uint8_t *in, int align, int n) {
    if (align >= 4 && n >= 8) return *reinterpret_cast<const uint32_t *>(in);
    uint32_t e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (2 * i < n) e |= (uint32_t)in[i] << (8 * i);
    return e;
}

// ------------------------------------------------------------- k contiguous

constexpr int kQuantWarps = 8;
constexpr int kSpan = 1024;  // k per warp

// Words a warp has in shared memory for `kSpan` elements that start anywhere,
// one word of padding per lane's 32 elements.
template <int DT>
constexpr int kStageWords = (DT == DG_F32 ? kSpan : kSpan / 2) + 33 + 4;

// The words of a row's 1024 k that start at x, whatever the address: whole
// 128-byte lines per load, kept in registers; then, through a warp's part of
// shared memory, lane l's 32 elements, from element 32 l on.
template <int DT>
struct Raw {
    static constexpr int W = Lot<DT>::W, N = DT == DG_F32 ? W : W + 1, per = 4 / Lot<DT>::ES;  // elements per word
    uint32_t w[N];
    uint32_t odd;  // the first word's lower half is not the row's
    __device__ __forceinline__ void load(const char *x, int elems, int lane) {
        odd = DT == DG_F32 ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(x) >> 1) & 1u;
        const char *at = x - 2 * odd + 4 * lane;
        const int count = (elems + (int)odd + per - 1) / per;
#pragma unroll
        for (int i = 0; i < N; ++i, at += 128) {
            const int j = 32 * i + lane;
            w[i] = 0;
            if (j >= count) continue;
            if (DT == DG_F32 || (!(odd && j == 0) && per * j + 1 - (int)odd < elems)) {
                w[i] = *reinterpret_cast<const uint32_t *>(at);
            } else {  // a word that is half the row's
                const bool low = !(odd && j == 0);
                w[i] = (uint32_t)*reinterpret_cast<const uint16_t *>(at + (low ? 0 : 2)) << (low ? 0 : 16);
            }
        }
    }
    __device__ __forceinline__ void turn(Lot<DT> &v, uint32_t *mine, int lane) const {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = 32 * i + lane;
            if (i < W || j < 32 * W + 1) mine[j + j / W] = w[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t b = mine[lane * (W + 1) + i];
            v.w[i] = DT == DG_F32
                         ? b
                         : __funnelshift_r(b, mine[i + 1 < W ? lane * (W + 1) + i + 1 : (lane + 1) * (W + 1)], 16u * odd);
        }
    }
};

// A lane's 32 elements at an address that is a multiple of 16, n of which exist.
template <int DT>
__device__ __forceinline__ void load_lot(Lot<DT> &v, const char *x, int n) {
    constexpr int W = Lot<DT>::W;
    if (n >= 32) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            *reinterpret_cast<uint4 *>(v.w + 4 * i) = *reinterpret_cast<const uint4 *>(x + 16 * i);
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const char *at = x + 4 * i;
        if (DT == DG_F32) {
            v.w[i] = i < n ? *reinterpret_cast<const uint32_t *>(at) : 0u;
        } else {
            const uint32_t lo = 2 * i < n ? *reinterpret_cast<const uint16_t *>(at) : 0u;
            const uint32_t hi = 2 * i + 1 < n ? *reinterpret_cast<const uint16_t *>(at + 2) : 0u;
            v.w[i] = lo | hi << 16;
        }
    }
}

// A warp takes 1024 k of four rows that are 32 apart, whose scales are
// neighbours; a lane has 32 k of each: one block of 32 or two of 16, so that no
// maximum crosses lanes.  VEC: a lane loads its own 64 (or 128) bytes, 16 at a
// time (the warp's four loads share their lines in L1), a row ahead of the one
// it works on.  Otherwise (rows at any address) the warp copies the row through
// shared memory; there a third block per SM is worth a few spilled registers
// (8192 x 14337 BF16 119 -> 100 us), while the compiler's own choice, three as
// well, is best for the rest.
template <int DT, int BLOCK, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps, VEC || DT == DG_F32 ? 0 : 3) quantize_rows_kernel(const QuantParams p) {
    pdl_wait_then_release();
    constexpr int ES = Lot<DT>::ES;
    __shared__ uint32_t stage[VEC ? 1 : kQuantWarps * kStageWords<DT>];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Factor f(p.q.scale);
    const int K = (int)p.q.K, k0 = (int)blockIdx.x * kSpan, k = k0 + lane * 32, n = max(0, K - k);
    const uint32_t tile = blockIdx.x * (uint32_t)(kSpan / BLOCK / 4) + (uint32_t)lane / (BLOCK / 8);  // of scales, along k
    const int64_t quarters = (p.q.rows + 127) / 128 * 4;
    for (int64_t quarter = blockIdx.y; quarter < quarters; quarter += gridDim.y) {
        const int64_t row0 = quarter / 4 * 128 + quarter % 4 * 8 + warp;
        const int rows = (int)min((int64_t)4, (p.q.rows - row0 + 31) / 32);
        if (rows <= 0) continue;
        Lot<DT> v, next;
        Raw<DT> raw;
        auto load = [&](int i) {
            const char *x = p.x.ptr + axis_offset(p.x.row, row0 + 32 * i) + (int64_t)k0 * ES;
            if (VEC) load_lot(next, x + lane * 32 * ES, n);
            else raw.load(x, min(kSpan, K - k0), lane);
        };
        load(0);
        uint4 scales = make_uint4(0, 0, 0, 0);
        uint8_t *codes = p.q.codes + row0 * p.q.code_stride + k / 2;
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
            if (VEC) v = next;
            else raw.turn(v, stage + warp * kStageWords<DT>, lane);
            if (i + 1 < rows) load(i + 1);
            uint32_t e[4];
            uint32_t s = encode<DT, BLOCK>(v, n, f, e);
            // four blocks' scales are one word
            if (BLOCK == 32) {
                s <<= 8 * (lane & 3);
                s |= __shfl_xor_sync(0xffffffffu, s, 1);
                s |= __shfl_xor_sync(0xffffffffu, s, 2);
            } else {
                s <<= 16 * (lane & 1);
                s |= __shfl_xor_sync(0xffffffffu, s, 1);
            }
            scales = make_uint4(scales.y, scales.z, scales.w, s);  // the last four
            if (n > 0) store_codes(codes + 32 * i * p.q.code_stride, p.q.align, e, n);
        }
        if (n == 0 || (lane & (BLOCK / 8 - 1)) != 0) continue;
        uint32_t *const out = reinterpret_cast<uint32_t *>(p.q.scales + (row0 / 128 * p.q.k_tiles + tile) * 512 + row0 % 32 * 16);
        if (rows == 4) {
            *reinterpret_cast<uint4 *>(out) = scales;
        } else {
            if (rows == 3) out[rows - 3] = scales.y;
            if (rows >= 2) out[rows - 2] = scales.z;
            out[rows - 1] = scales.w;
        }
    }
}

// A warp reads 1024 k of four rows back that are 32 apart, a lane eight k at a
// time: its stores are whole 512-byte runs.  Rows at any address go through
// shared memory, as above.
template <int DT, int BLOCK, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps) dequantize_rows_kernel(const QuantParams p) {
    pdl_wait_then_release();
    constexpr int ES = Lot<DT>::ES, W = 2 * ES;  // words of eight values
    __shared__ uint32_t stage[VEC ? 1 : kQuantWarps * kStageWords<DT>];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    const int K = (int)p.q.K, k0 = (int)blockIdx.x * kSpan, n0 = K - k0 - lane * 8;
    const int block = lane * 8 / BLOCK;  // of the first chunk
    const int64_t quarters = (p.q.rows + 127) / 128 * 4;
    for (int64_t quarter = blockIdx.y; quarter < quarters; quarter += gridDim.y) {
        const int64_t row0 = quarter / 4 * 128 + quarter % 4 * 8 + warp;
        const int rows = (int)min((int64_t)4, (p.q.rows - row0 + 31) / 32);
        if (rows <= 0) continue;
        // the scales of all four rows are 16 bytes
        const uint8_t *scales = p.q.scales + row0 % 32 * 16 +
                                (row0 / 128 * p.q.k_tiles + blockIdx.x * (uint32_t)(kSpan / BLOCK / 4) + block / 4) * 512;
        uint4 s[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            s[c] = n0 > c * 256 ? *reinterpret_cast<const uint4 *>(scales + c * (64 / BLOCK) * 512) : make_uint4(0, 0, 0, 0);
        const uint8_t *codes = p.q.codes + row0 * p.q.code_stride + k0 / 2 + lane * 4;
        uint32_t *const mine = stage + warp * kStageWords<DT>;
        uint32_t e[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                e[i][c] = i < rows && n0 > c * 256
                              ? load_codes8(codes + 32 * i * p.q.code_stride + c * 128, p.q.align, n0 - c * 256)
                              : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= rows) break;
            char *const y = const_cast<char *>(p.x.ptr) + axis_offset(p.x.row, row0 + 32 * i) + (int64_t)k0 * ES;
            if (!VEC) __syncwarp();  // the last row's words have been stored
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int n = n0 - c * 256;
                if (n <= 0) continue;
                const uint32_t word = i == 0 ? s[c].x : i == 1 ? s[c].y : i == 2 ? s[c].z : s[c].w;
                const float unit = mx4_scale_value<BLOCK>(word >> (8 * (block & 3)) & 0xff) * factor;
                float v[8];
                e2m1x8_values(e[i][c], v);
#pragma unroll
                for (int j = 0; j < 8; j += 2) mul2(Two(v[j], v[j + 1]), Two(unit, unit)).get(v[j], v[j + 1]);
                uint32_t w[W];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    w[j] = DT == DG_F32 ? __float_as_uint(v[j]) : pack2<DT == DG_BF16>(v[2 * j & 7], v[(2 * j + 1) & 7]);
                char *const at = y + (c * 256 + lane * 8) * ES;
                if (VEC && n >= 8) {
#pragma unroll
                    for (int j = 0; j < W / 4; ++j)
                        *reinterpret_cast<uint4 *>(at + 16 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                } else if (VEC) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < n) {
                            if (DT == DG_F32) *reinterpret_cast<uint32_t *>(at + 4 * j) = w[j & (W - 1)];
                            else *reinterpret_cast<uint16_t *>(at + 2 * j) = (uint16_t)(w[j / 2 & (W - 1)] >> (j & 1 ? 16 : 0));
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) mine[(c * 32 + lane) * W + j] = w[j];
                }
            }
            if (VEC) continue;
            __syncwarp();
            const uint32_t odd = DT == DG_F32 ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(y) >> 1) & 1u;
            char *const words = y - 2 * odd;
            const int elems = min(kSpan, K - k0), per = 4 / ES, count = (elems + (int)odd + per - 1) / per;
#pragma unroll 4
            for (int j = lane; j < count; j += 32) {
                char *at = words + (int64_t)j * 4;
                const uint32_t here = mine[j], b = odd ? __funnelshift_r(j > 0 ? mine[j - 1] : 0u, here, 16) : here;
                if (DT == DG_F32 || (!(odd && j == 0) && per * j + 1 - (int)odd < elems)) {
                    *reinterpret_cast<uint32_t *>(at) = b;
                } else {
                    const bool low = !(odd && j == 0);
                    *reinterpret_cast<uint16_t *>(at + (low ? 0 : 2)) = (uint16_t)(b >> (low ? 0 : 16));
                }
            }
        }
    }
}

// ------------------------------------------------------------------ any view

constexpr int kTurnK = 32;  // a thread takes 32 k

// Any view, a thread per row and 32 k: made for rows that are neighbours in
// memory (a weight along its other dim), whose loads are then whole sectors.
// ONE: k is one dim.  (Two neighbouring 16-bit rows per thread and 4-byte load
// were slower: 8192 x 14336 BF16 in blocks of 16 131 -> 157 us.)
template <int DT, int BLOCK, bool ONE>
__global__ void __launch_bounds__(128) quantize_any_kernel(const QuantParams p) {
    pdl_wait_then_release();
    const int64_t row = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (row >= p.q.rows) return;
    const int K = (int)p.q.K;
    const Factor f(p.q.scale);
    const char *x = p.x.ptr + axis_offset(p.x.row, row);
    uint8_t *scales_row = p.q.scales + row / 128 * p.q.k_tiles * 512 + row % 32 * 16 + row % 128 / 32 * 4;
    for (int64_t k64 = (int64_t)blockIdx.y * kTurnK; k64 < K; k64 += (int64_t)gridDim.y * kTurnK) {
        const int k0 = (int)k64, n = K - k0;
        Lot<DT> v;
        auto put = [&](int i, const char *at) {
            uint32_t b = 0;
            if (i < n) {
                if (DT == DG_F32) b = *reinterpret_cast<const uint32_t *>(at);
                else b = *reinterpret_cast<const uint16_t *>(at);
            }
            if (DT == DG_F32) v.w[i & (Lot<DT>::W - 1)] = b;
            else if (i & 1) v.w[i / 2] |= b << 16;
            else v.w[i / 2] = b;
        };
        if (ONE) {
            const char *at = x + k0 * p.col;
#pragma unroll
            for (int i = 0; i < 32; ++i, at += p.col) put(i, at);
        } else {
#pragma unroll 1
            for (int i = 0; i < 32; ++i) put(i, x + axis_offset(p.x.col, min(k0 + i, K - 1)));
        }
        uint32_t e[4];
        const uint32_t scales = encode<DT, BLOCK>(v, n, f, e);
        store_codes(p.q.codes + row * p.q.code_stride + k0 / 2, p.q.align, e, n);
        // the blocks past the last one of their tile get a zero
        const int block = k0 / BLOCK;
        uint8_t *out = scales_row + (int64_t)(block / 4) * 512 + block % 4;
        if (BLOCK == 16) {
            *reinterpret_cast<uint16_t *>(out) = (uint16_t)scales;
            if (n <= 32 && block % 4 == 0) *reinterpret_cast<uint16_t *>(out + 2) = 0;
        } else {
            *out = (uint8_t)scales;
            if (n <= 32)
                for (int i = block % 4 + 1; i < 4; ++i) out[i - block % 4] = 0;
        }
    }
}

// The reverse.  ROWS 2: pairs of neighbouring 16-bit rows, stored four bytes at
// a time (8192 x 14336 BF16 from blocks of 16: 115 -> 67 us).
template <int DT, int BLOCK, bool ONE, int ROWS>
__global__ void __launch_bounds__(128) dequantize_any_kernel(const QuantParams p) {
    pdl_wait_then_release();
    const int64_t row0 = ((int64_t)blockIdx.x * 128 + threadIdx.x) * ROWS;
    if (row0 >= p.q.rows) return;
    const bool two = ROWS == 2 && row0 + 1 < p.q.rows;
    const int K = (int)p.q.K;
    const float factor = p.q.scale != nullptr ? *p.q.scale : 1.f;
    char *y = const_cast<char *>(p.x.ptr) + axis_offset(p.x.row, row0);
    for (int64_t k64 = (int64_t)blockIdx.y * kTurnK; k64 < K; k64 += (int64_t)gridDim.y * kTurnK) {
        const int k0 = (int)k64;
        uint32_t e[ROWS][kTurnK / 8];
        float unit[ROWS][kTurnK / BLOCK];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int64_t row = q == 1 && !two ? row0 : row0 + q;
            const uint8_t *codes = p.q.codes + row * p.q.code_stride + k0 / 2;
            if (p.q.align == 16 && k0 + kTurnK <= K) {
                *reinterpret_cast<uint4 *>(e[q]) = *reinterpret_cast<const uint4 *>(codes);
            } else {
#pragma unroll
                for (int j = 0; j < kTurnK / 8; ++j)
                    e[q][j] = k0 + 8 * j < K ? load_codes8(codes + 4 * j, p.q.align, K - k0 - 8 * j) : 0u;
            }
            const int block = k0 / BLOCK;
            const uint8_t *s = p.q.scales + (row / 128 * p.q.k_tiles + block / 4) * 512 + row % 32 * 16 +
                               row % 128 / 32 * 4 + block % 4;
#pragma unroll
            for (int b = 0; b < kTurnK / BLOCK; ++b)
                unit[q][b] = k0 + b * BLOCK < K ? mx4_scale_value<BLOCK>(s[b]) * factor : 0.f;
        }
        char *at = y + (ONE ? k0 * p.col : 0);
#pragma unroll
        for (int j = 0; j < kTurnK / 8; ++j) {
            const int k = k0 + 8 * j;
            if (k >= K) break;
            float v[ROWS][8];
#pragma unroll
            for (int q = 0; q < ROWS; ++q) e2m1x8_values(e[q][j], v[q]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (k + i < K) {
                    char *const to = ONE ? at : y + axis_offset(p.x.col, k + i);
                    const float first = v[0][i] * unit[0][8 * j / BLOCK];
                    if (ROWS == 2 && two)
                        *reinterpret_cast<uint32_t *>(to) =
                            pack2<DT == DG_BF16>(first, v[ROWS - 1][i] * unit[ROWS - 1][8 * j / BLOCK]);
                    else st_out<DT>(to, first);
                }
                at += ONE ? p.col : 0;
            }
        }
    }
}

template <int DT, int BLOCK, bool ONE, int ROWS>
cudaError_t run_any(const QuantParams &p, bool back, cudaStream_t s) {
    const int rows = back ? 128 * ROWS : 128;
    const dim3 grid((unsigned)((p.q.rows + rows - 1) / rows),
                    (unsigned)std::min<int64_t>((p.q.K + kTurnK - 1) / kTurnK, 65535));
    auto kern = back ? dequantize_any_kernel<DT, BLOCK, ONE, ROWS> : quantize_any_kernel<DT, BLOCK, ONE>;
    return launch_ex(kern, grid, dim3(128), 0, s, dim3(1, 1, 1), p.pdl, p);
}

template <int DT, int BLOCK>
cudaError_t run(const QuantParams &p, bool back, cudaStream_t s) {
    // neighbours in a row go to neighbouring lanes; otherwise neighbouring rows do
    if (p.x.col.n == 0 || (p.x.col.n == 1 && p.col == Lot<DT>::ES)) {
        const dim3 grid((unsigned)((p.q.K + kSpan - 1) / kSpan),
                        (unsigned)std::min<int64_t>((p.q.rows + 127) / 128 * 4, 65532));
        auto kern = back ? (p.vec ? dequantize_rows_kernel<DT, BLOCK, true> : dequantize_rows_kernel<DT, BLOCK, false>)
                         : (p.vec ? quantize_rows_kernel<DT, BLOCK, true> : quantize_rows_kernel<DT, BLOCK, false>);
        return launch_ex(kern, grid, dim3(32 * kQuantWarps), 0, s, dim3(1, 1, 1), p.pdl, p);
    }
    if (p.x.col.n != 1) return run_any<DT, BLOCK, false, 1>(p, back, s);
    // pairs of neighbouring 16-bit rows, each at a multiple of four bytes
    if constexpr (DT != DG_F32) {
        if (p.q.rows > 1 && p.x.row.n == 1 && p.x.row.stride[0] == 2 && p.col % 4 == 0 &&
            reinterpret_cast<uintptr_t>(p.x.ptr) % 4 == 0)
            return run_any<DT, BLOCK, true, 2>(p, back, s);
    }
    return run_any<DT, BLOCK, true, 1>(p, back, s);
}

}  // namespace

cudaError_t launch_quant(const QuantParams &p, int block, bool back, cudaStream_t s) {
    if (p.x.dtype == DG_F32) return block == 32 ? run<DG_F32, 32>(p, back, s) : run<DG_F32, 16>(p, back, s);
    if (p.x.dtype == DG_F16) return block == 32 ? run<DG_F16, 32>(p, back, s) : run<DG_F16, 16>(p, back, s);
    return block == 32 ? run<DG_BF16, 32>(p, back, s) : run<DG_BF16, 16>(p, back, s);
}

}  // namespace dg

// mma_planes.cuh -- warp-level products of fp32 matrices on the tensor cores at fp32 accuracy.
//
// A matrix in shared memory is kept as one or two fp16 planes and a power-of-two scale s:
//   x = s * (hi + lo),  hi = fp16(x / s),  lo = fp16(x / s - hi).
// s puts the largest magnitude of the scaled set (a tile, or a row) into [2^9, 2^10), so hi + lo holds
// 22 bits of every element down to 2^-13 of that maximum and an absolute 2^-35 of it below: the step of
// fp32 where it matters.  A bf16 set (8 bits) is exact in the hi plane alone down to 2^-26 of its maximum, with
// an absolute 2^-34 of it below.  Maxima below 2^-100 count as 2^-100.  A product takes the
// terms hi hi, hi lo and lo hi (lo lo is below 2^-22 of the result), each an m16n8k16 fp16 tensor-core
// instruction with fp32 accumulation: three for two split matrices, two where one is exact.  bf16 planes
// would need three each (six terms) for the same accuracy, tf32 planes run at half the rate (measured
// here: 600 TFLOP/s for fp16 and bf16, 300 for tf32, 75 for packed fp32 FMA).
//
// Planes are laid out in blocks of 64 columns: rows of 128 bytes whose 16-byte chunks are XORed by the row
// (mod 8), so that the eight rows an ldmatrix phase reads lie in different banks, and so do the pairs an
// accumulator writes.  It is the 128-byte swizzle of tcgen05 operands too (blocks start at multiples of
// 1024 bytes), so one tile serves both.
#pragma once

#include <cuda_fp16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace planes {

// Byte offset of element (row, col) in a plane with COLS columns (64 or 128), blocks of 64 columns HS apart.
template <int COLS, int HS>
__device__ __forceinline__ uint32_t offset(int row, int col) {
    if constexpr (COLS == 64) return (uint32_t)(row * 128 + ((col * 2) ^ ((row & 7) << 4)));
    else return (uint32_t)((col >> 6) * HS + row * 128 + (((col & 63) * 2) ^ ((row & 7) << 4)));
}

// A matrix of P planes of COLS columns in shared memory: planes LO bytes apart, blocks of 64 columns HS.
template <int COLS, int P, int LO, int HS>
struct Mat {
    static constexpr int lo = LO;
    uint32_t at;
    __device__ __forceinline__ uint32_t operator()(int row, int col) const { return at + offset<COLS, HS>(row, col); }
};

template <int O>
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(O));
}
template <int O>
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(O));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Left operand, 16 x 16 blocks: stored [m][k] (T false) or [k][m] (T true).  lane_a is this lane's
// address in block (m0, 0); load_a adds k0.
template <bool T, int COLS, int P, int LO, int HS>
__device__ __forceinline__ uint32_t lane_a(Mat<COLS, P, LO, HS> A, int m0, int lane) {
    if constexpr (T) return A((lane & 7) + ((lane >> 4) << 3), m0 + (lane & 8));
    else return A(m0 + (lane & 15), (lane >> 4) << 3);
}
template <bool T, int O, int HS>
__device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t lane_at, int k0) {
    if constexpr (T) ldsm_t<O>(r, lane_at + k0 * 128);
    else ldsm<O>(r, (lane_at ^ ((k0 & 63) * 2)) + (k0 >> 6) * HS);
}
// Right operand, 16 x 16 blocks (r[0], r[1]: columns n0 .. n0 + 7; r[2], r[3]: the next eight): stored
// [n][k] (T false) or [k][n] (T true).  lane_b is this lane's address in block (0, 0).
template <bool T, int COLS, int P, int LO, int HS>
__device__ __forceinline__ uint32_t lane_b(Mat<COLS, P, LO, HS> B, int lane) {
    if constexpr (T) return B(lane & 15, (lane >> 4) << 3);
    else return B((lane & 7) + ((lane >> 4) << 3), lane & 8);
}
template <bool T, int O, int HS>
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t lane_at, int n0, int k0) {
    if constexpr (T) ldsm_t<O>(r, (lane_at ^ ((n0 & 63) * 2)) + (n0 >> 6) * HS + k0 * 128);
    else ldsm<O>(r, ((lane_at + n0 * 128) ^ ((k0 & 63) * 2)) + (k0 >> 6) * HS);
}

// Which 16-blocks of A's inner dimension can be non-zero: all, j <= i (A lower triangular), or j >= i.
enum Fill { kFull, kLower, kUpper };

// acc += A B for this warp's row tiles m[] and the columns n0 .. n0 + 8 NT; TA, TB: stored transposed
// (see lane_a, lane_b); K: inner dimension.
template <int K, bool TA, bool TB, Fill F = kFull, int MT, int NT, int CA, int PA, int LA, int HA, int CB, int PB, int LB,
          int HB>
__device__ __forceinline__ void product(float (&acc)[MT][NT][4], Mat<CA, PA, LA, HA> A, const int (&m)[MT],
                                        Mat<CB, PB, LB, HB> B, int n0, int lane) {
    uint32_t la[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) la[i] = lane_a<TA>(A, m[i], lane);
    const uint32_t lb = lane_b<TB>(B, lane);
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t a[PA][MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if ((F == kLower && k > m[i]) || (F == kUpper && k < m[i])) continue;
            load_a<TA, 0, HA>(a[0][i], la[i], k);
            if constexpr (PA == 2) load_a<TA, LA, HA>(a[1][i], la[i], k);
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            if (F != kFull && MT == 1 && ((F == kLower && k > m[0]) || (F == kUpper && k < m[0]))) continue;
            uint32_t b[PB][4];
            load_b<TB, 0, HB>(b[0], lb, n0 + 8 * j, k);
            if constexpr (PB == 2) load_b<TB, LB, HB>(b[1], lb, n0 + 8 * j, k);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if ((F == kLower && k > m[i]) || (F == kUpper && k < m[i])) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) mma(acc[i][j + h], a[0][i], b[0][2 * h], b[0][2 * h + 1]);
                if constexpr (PB == 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma(acc[i][j + h], a[0][i], b[1][2 * h], b[1][2 * h + 1]);
                }
                if constexpr (PA == 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma(acc[i][j + h], a[1][i], b[0][2 * h], b[0][2 * h + 1]);
                }
            }
        }
    }
}

template <int MT, int NT>
__device__ __forceinline__ void clear(float (&acc)[MT][NT][4]) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
}

// Calls f(i, j, h, row, column) for every pair acc[i][j][2 h], acc[i][j][2 h + 1] of this warp.
template <int MT, int NT, class Fn>
__device__ __forceinline__ void pairs(const int (&m)[MT], int n0, int lane, Fn f) {
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j) f(i, j, h, m[i] + g + 8 * h, n0 + 8 * j + t);
}

// The scale of a set whose largest magnitude has the given fp32 bits: mul = 2^(9 - e), back = 1 / mul.
struct Scale {
    float mul, back;
};
__device__ __forceinline__ Scale scale_of(uint32_t max_bits) {
    int e = (int)(max_bits >> 23) - 127;
    e = e < -100 ? -100 : (e > 127 ? 127 : e);
    Scale s;
    s.mul = __int_as_float((136 - e) << 23);
    s.back = __int_as_float((118 + e) << 23);
    return s;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// hi and lo planes of a scaled pair.
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&x)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Address of the pair (i, j, h) of pairs() in a plane: n0 is a multiple of 8 NT, which divides 64.
template <int NT, int COLS, int P, int LO, int HS>
__device__ __forceinline__ uint32_t pair_at(Mat<COLS, P, LO, HS> a, int m, int n0, int j, int h, int lane) {
    const int g = lane >> 2;
    const uint32_t first = a.at + (n0 >> 6) * HS + (m + g) * 128 + (((n0 & 63) * 2) ^ (g << 4)) + (lane & 3) * 4;
    return (first ^ (16 * j)) + 8 * h * 128;
}

// Writes this warp's accumulators, times mul, into two planes.
template <int COLS, int LO, int HS, int MT, int NT>
__device__ __forceinline__ void write(Mat<COLS, 2, LO, HS> dst, const float (&acc)[MT][NT][4], const int (&m)[MT], int n0,
                                      int lane, float mul) {
    pairs<MT, NT>(m, n0, lane, [&](int i, int j, int h, int, int) {
        uint32_t hi, lo;
        split(acc[i][j][2 * h] * mul, acc[i][j][2 * h + 1] * mul, hi, lo);
        const uint32_t at = pair_at<NT>(dst, m[i], n0, j, h, lane);
        sts32(at, hi);
        sts32(at + LO, lo);
    });
}

// The same with a factor for each row.
template <int COLS, int LO, int HS, int MT, int NT>
__device__ __forceinline__ void write(Mat<COLS, 2, LO, HS> dst, const float (&acc)[MT][NT][4], const int (&m)[MT], int n0,
                                      int lane, const float (&mul)[MT][2]) {
    pairs<MT, NT>(m, n0, lane, [&](int i, int j, int h, int, int) {
        uint32_t hi, lo;
        split(acc[i][j][2 * h] * mul[i][h], acc[i][j][2 * h + 1] * mul[i][h], hi, lo);
        const uint32_t at = pair_at<NT>(dst, m[i], n0, j, h, lane);
        sts32(at, hi);
        sts32(at + LO, lo);
    });
}

// The pair (i, j, h) of a matrix, without its scale.
template <int NT, int COLS, int P, int LO, int HS>
__device__ __forceinline__ float2 read(Mat<COLS, P, LO, HS> a, int m, int n0, int j, int h, int lane) {
    const uint32_t at = pair_at<NT>(a, m, n0, j, h, lane);
    float2 x = halves(lds32(at));
    if constexpr (P == 2) {
        const float2 y = halves(lds32(at + LO));
        x.x += y.x;
        x.y += y.y;
    }
    return x;
}

// Eight consecutive elements of a row, from column col (a multiple of eight).
template <int COLS, int P, int LO, int HS>
__device__ __forceinline__ void read8(Mat<COLS, P, LO, HS> a, int row, int col, float (&x)[8]) {
    const uint32_t at = a(row, col);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint32_t u[4];
        lds128(at + p * LO, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = halves(u[i]);
            x[2 * i] = p ? x[2 * i] + y.x : y.x;
            x[2 * i + 1] = p ? x[2 * i + 1] + y.y : y.y;
        }
    }
}

template <int MT, int NT>
__device__ __forceinline__ uint32_t max_bits(const float (&acc)[MT][NT][4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = max(m, abs_bits(acc[i][j][e]));
    return __reduce_max_sync(0xffffffffu, m);
}

// The largest of W warps' maxima (W a power of two up to 32; a barrier lies between their writes and this).
template <int W>
__device__ __forceinline__ uint32_t top_of(const uint32_t* red, int lane) {
    return __reduce_max_sync(0xffffffffu, red[lane & (W - 1)]);
}

}  // namespace planes
}  // namespace gdn

// mma_planes.cuh -- warp-level products of fp32 matrices on the tensor cores at fp32 accuracy.
//
// A matrix in shared memory is kept as one or two fp16 planes and a power-of-two scale s:
//   x = s * (hi + lo),  hi = fp16(x / s),  lo = fp16(x / s - hi).
// s puts the largest magnitude of the scaled set (a tile, or a row) into [2^9, 2^10), so hi + lo holds
// 22 bits of every element down to 2^-13 of that maximum and an absolute 2^-35 of it below: the step of
// fp32 where it matters.  A bf16 matrix (8 bits) is exact in the hi plane alone.  A product takes the
// terms hi hi, hi lo and lo hi (lo lo is below 2^-22 of the result), each an m16n8k16 fp16 tensor-core
// instruction with fp32 accumulation: three for two split matrices, two where one is exact.  bf16 planes
// would need three each (six terms) for the same accuracy, tf32 planes run at half the rate.
//
// Planes are row-major with their 16-byte chunks XORed by the row (mod 8), so that the eight rows an
// ldmatrix phase reads lie in different banks, and so do the pairs an accumulator writes.
#pragma once

#include <cuda_fp16.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace planes {

// Byte offset of element (row, col) in a plane with COLS columns (64 or 128).
template <int COLS>
__device__ __forceinline__ uint32_t offset(int row, int col) {
    return (uint32_t)(row * COLS * 2 + ((((col >> 3) ^ (row & 7)) << 4) | ((col & 7) << 1)));
}

// A matrix of planes in shared memory: shared address of the hi plane, distance to the lo plane.
struct Mat {
    uint32_t at, lo;
};

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 16 x 16 block of A at rows m0, columns k0: stored [m][k] (T false) or [k][m] (T true).
template <int COLS, bool T>
__device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t base, int m0, int k0, int lane) {
    if constexpr (T) ldsm_t(r, base + offset<COLS>(k0 + (lane & 7) + ((lane >> 4) << 3), m0 + (lane & 8)));
    else ldsm(r, base + offset<COLS>(m0 + (lane & 15), k0 + ((lane >> 4) << 3)));
}
// The 16 x 16 block of B at k0, n0 (r[0], r[1]: columns n0 .. n0 + 7; r[2], r[3]: the next eight):
// stored [n][k] (T false) or [k][n] (T true).
template <int COLS, bool T>
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
    if constexpr (T) ldsm_t(r, base + offset<COLS>(k0 + (lane & 15), n0 + ((lane >> 4) << 3)));
    else ldsm(r, base + offset<COLS>(n0 + (lane & 7) + ((lane >> 4) << 3), k0 + (lane & 8)));
}

// Which 16-blocks of A's inner dimension can be non-zero: all, j <= i (A lower triangular), or j >= i.
enum Fill { kFull, kLower, kUpper };

// acc += A B for this warp's row tiles m[] and the columns n0 .. n0 + 8 NT.  CA, CB: columns of the
// stored matrices; TA, TB: stored transposed (see load_a, load_b); PA, PB: planes; K: inner dimension.
template <int MT, int NT, int K, int CA, bool TA, int PA, int CB, bool TB, int PB, Fill F = kFull>
__device__ __forceinline__ void product(float (&acc)[MT][NT][4], Mat A, const int (&m)[MT], Mat B, int n0, int lane) {
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t a[PA][MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if ((F == kLower && k > m[i]) || (F == kUpper && k < m[i])) continue;
#pragma unroll
            for (int p = 0; p < PA; ++p) load_a<CA, TA>(a[p][i], A.at + p * A.lo, m[i], k, lane);
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            uint32_t b[PB][4];
#pragma unroll
            for (int p = 0; p < PB; ++p) load_b<CB, TB>(b[p], B.at + p * B.lo, n0 + 8 * j, k, lane);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if ((F == kLower && k > m[i]) || (F == kUpper && k < m[i])) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma(acc[i][j + h], a[0][i], b[0][2 * h], b[0][2 * h + 1]);
                    if constexpr (PB == 2) mma(acc[i][j + h], a[0][i], b[1][2 * h], b[1][2 * h + 1]);
                    if constexpr (PA == 2) mma(acc[i][j + h], a[1][i], b[0][2 * h], b[0][2 * h + 1]);
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

// Calls f(value, row, column) for every accumulator element of this warp.
template <int MT, int NT, class Fn>
__device__ __forceinline__ void each(float (&acc)[MT][NT][4], const int (&m)[MT], int n0, int lane, Fn f) {
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(acc[i][j][e], m[i] + g + (e >> 1) * 8, n0 + 8 * j + t + (e & 1));
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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& x, uint32_t& y) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Writes this warp's accumulators, times mul, into planes of COLS columns.
template <int COLS, int MT, int NT>
__device__ __forceinline__ void write(Mat dst, const float (&acc)[MT][NT][4], const int (&m)[MT], int n0, int lane,
                                      float mul) {
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi, lo;
                split(acc[i][j][2 * h] * mul, acc[i][j][2 * h + 1] * mul, hi, lo);
                const uint32_t at = dst.at + offset<COLS>(m[i] + g + 8 * h, n0 + 8 * j + t);
                sts32(at, hi);
                sts32(at + dst.lo, lo);
            }
}

// The pair of elements (row, col), (row, col + 1) of a matrix of P planes, without its scale.
template <int COLS, int P>
__device__ __forceinline__ float2 read(Mat a, int row, int col) {
    const uint32_t at = a.at + offset<COLS>(row, col);
    float2 x = halves(lds32(at));
    if constexpr (P == 2) {
        const float2 y = halves(lds32(at + a.lo));
        x.x += y.x;
        x.y += y.y;
    }
    return x;
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

}  // namespace planes
}  // namespace gdn

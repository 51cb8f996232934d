// bf16_planes.cuh -- products of fp32 matrices on the tensor cores as sums of bf16 products.
//
// A fp32 matrix is three bf16 planes, x = hi + mid + lo (8 bits each, fp32's whole range, no scales); a bf16 input
// is one plane as it lies in memory.  A product takes the terms of planes i and j with i + j <= 2, each an m16n8k16
// instruction with fp32 accumulation: three for an input times a fp32 matrix, six for two fp32 matrices; what is
// left out is below 2^-24 of a term.  Two planes (2^-17) are enough in front of an output that is rounded to bf16.
// The alternative, two fp16 planes with scales (mma_planes.cuh), takes three instructions for six and scales by rows
// that have to follow every operand; bf16 inputs, exact in one plane without conversion, make up for it on tcgen05.
//
// Tiles, addresses and fragments are those of mma_planes.cuh: blocks of 64 columns, rows of 128 bytes, 16-byte chunks
// XORed by the row.
#pragma once

#include "mma_planes.cuh"
#include "ssm_internal.cuh"

namespace gdn {
namespace bfp {

using planes::Fill;
using planes::kFull;
using planes::kLower;
using planes::kUpper;
using planes::lane_a;
using planes::lane_b;
using planes::load_a;
using planes::load_b;
using planes::Mat;
using gdn::F2;
using gdn::fma2;
using gdn::widen;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(F2 a) {
    float x, y;
    a.get(x, y);
    return pack_bf16(x, y);
}
// The next plane of a pair, and what is left of the pair.
__device__ __forceinline__ uint32_t peel(F2& a) {
    const uint32_t u = pack(a);
    a = fma2(widen(u), F2(-1.f, -1.f), a);
    return u;
}
// The next plane of a pair, and what is left of the pair.
__device__ __forceinline__ uint32_t peel(float& x, float& y) {
    const uint32_t u = pack_bf16(x, y);
    x -= __uint_as_float(u << 16);
    y -= __uint_as_float(u & 0xffff0000u);
    return u;
}
template <int P>
__device__ __forceinline__ void split(float x, float y, uint32_t (&u)[P]) {
#pragma unroll
    for (int i = 0; i + 1 < P; ++i) u[i] = peel(x, y);
    u[P - 1] = pack_bf16(x, y);
}

// Matrix of ROWS x COLS in P planes at shared address `at`.
template <int ROWS, int COLS, int P>
using Tile = Mat<COLS, P, ROWS * COLS * 2, ROWS * 128>;
template <int ROWS, int COLS, int P>
constexpr int kTileBytes = ROWS * COLS * 2 * P;

// Eight consecutive elements into their planes.
template <int COLS, int P, int LO, int HS>
__device__ __forceinline__ void put8(Mat<COLS, P, LO, HS> m, int row, int col, const float (&x)[8]) {
    uint32_t u[P][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[P];
        split<P>(x[2 * i], x[2 * i + 1], v);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p][i] = v[p];
    }
    const uint32_t at = m(row, col);
#pragma unroll
    for (int p = 0; p < P; ++p) planes::sts128(at + p * LO, u[p]);
}

// The value at (row, col), col even, and its neighbour.
template <int COLS, int P, int LO, int HS>
__device__ __forceinline__ float2 get2(Mat<COLS, P, LO, HS> m, int row, int col) {
    const uint32_t at = m(row, col);
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = P - 1; p >= 0; --p) {
        const uint32_t u = planes::lds32(at + p * LO);
        r.x += __uint_as_float(u << 16);
        r.y += __uint_as_float(u & 0xffff0000u);
    }
    return r;
}

// Terms of one 16 x 8 block and one k step: planes a of the left, b (pairs of registers from `h`) of the right operand.
template <int PA, int PB>
__device__ __forceinline__ void terms(float (&acc)[4], const uint32_t (&a)[PA][4], const uint32_t (&b)[PB][4], int h) {
    // smallest terms first
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < PA; ++i)
#pragma unroll
            for (int j = 0; j < PB; ++j)
                if (i + j == s) mma(acc, a[i], b[j][2 * h], b[j][2 * h + 1]);
}

// acc += A B for this warp's 16 rows from m and columns n0 .. n0 + 8 NT; TA, TB: stored transposed; K: inner dimension.
// The tensor cores cut a sum off where fp32 would round it, which leaves every long sum too near to zero: with all
// of K summed there, 24 cuts, sums of gradients over 8192 tokens were 4e-6 off.  So a k step's terms are summed on
// their own, the smallest first, and added to acc by a rounded addition (2.5e-7).
template <int K, bool TA, bool TB, Fill F = kFull, int NT, int CA, int PA, int LA, int HA, int CB, int PB, int LB, int HB>
__device__ __forceinline__ void product(float (&acc)[NT][4], Mat<CA, PA, LA, HA> A, int m, Mat<CB, PB, LB, HB> B, int n0,
                                        int lane) {
    const uint32_t la = lane_a<TA>(A, m, lane), lb = lane_b<TB>(B, lane);
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        if ((F == kLower && k > m) || (F == kUpper && k < m)) continue;
        uint32_t a[PA][4];
        load_a<TA, 0, HA>(a[0], la, k);
        if constexpr (PA > 1) load_a<TA, LA, HA>(a[1], la, k);
        if constexpr (PA > 2) load_a<TA, 2 * LA, HA>(a[2], la, k);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            uint32_t b[PB][4];
            load_b<TB, 0, HB>(b[0], lb, n0 + 8 * j, k);
            if constexpr (PB > 1) load_b<TB, LB, HB>(b[1], lb, n0 + 8 * j, k);
            if constexpr (PB > 2) load_b<TB, 2 * LB, HB>(b[2], lb, n0 + 8 * j, k);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                terms<PA, PB>(sum, a, b, h);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j + h][e] += sum[e];
            }
        }
    }
}

template <int NT>
__device__ __forceinline__ void clear(float (&acc)[NT][4]) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
}

// Calls f(j, h, row, column) for every pair acc[j][2 h], acc[j][2 h + 1] of this warp.
template <int NT, class Fn>
__device__ __forceinline__ void pairs(int m, int n0, int lane, Fn f) {
    const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j) f(j, h, m + g + 8 * h, n0 + 8 * j + t);
}

// Writes a pair into its planes.
template <int COLS, int P, int LO, int HS>
__device__ __forceinline__ void put2(Mat<COLS, P, LO, HS> m, int row, int col, float x, float y) {
    uint32_t u[P];
    split<P>(x, y, u);
    const uint32_t at = m(row, col);
#pragma unroll
    for (int p = 0; p < P; ++p) planes::sts32(at + p * LO, u[p]);
}

// Eight consecutive inputs as they are loaded; zeros where `on` is false.
struct Raw8 {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, bool on) {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
            a = reinterpret_cast<const float4*>(p)[0];
            b = reinterpret_cast<const float4*>(p)[1];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    template <int COLS, int P, int LO, int HS>
    __device__ __forceinline__ void put(Mat<COLS, P, LO, HS> m, int row, int col) const {
        float x[8];
        get(x);
        put8(m, row, col, x);
    }
};

}  // namespace bfp
}  // namespace gdn

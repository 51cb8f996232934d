// ssm_tc.cuh -- what the tcgen05 kernels of the selective scan share.
#pragma once

#include <cudaTypedefs.h>

#include "sm100_ptx.cuh"
#include "ssm_chunk.cuh"

namespace gdn {
namespace ssm {
namespace tc {

using namespace ptx;

constexpr int kT = 128;                    // tokens of a chunk
constexpr int kBlock = kT * 128;           // bytes of a tile of 128 rows and 64 columns
constexpr uint64_t kLimit = 2000000000ull;  // ns, bound on any wait
constexpr float kLog2e = 1.4426950408889634f;

// MMAs issued by the elected thread of a warp that runs as one (its operands stay in uniform registers): left operand
// from shared memory, or from TMEM.
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t on, uint64_t* bar) {
    if (on) mma_commit(bar);
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on;
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
// 16 and eight consecutive columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Polls until the phase completes; false when another role has given up, or the bound has passed (recorded).
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead, int* err) {
    const long long limit = static_cast<long long>(kLimit) * 21 / 10, t0 = clock64();
    while (!mbar_try_wait(bar, parity, 100000u)) {
        if (*dead) return false;
        if (clock64() - t0 > limit) {
            record_error(err, GDN_ERR_TIMEOUT);
            *dead = 1;
            return false;
        }
    }
    return true;
}
// 16-byte chunk c of row r of a tile
__device__ __forceinline__ uint32_t at16(uint32_t tile, int r, int c) { return tile + r * 128 + ((c ^ (r & 7)) << 4); }

// The gates of four consecutive tokens of a chunk of 128 (lane l of a warp holds tokens 4 l ..), `left` of them inside
// the sequence, from their logits z (bias added).  Sums of log decays inside the token's run of 32 (eight lanes) from its
// start in two floats, in units of log2; exponentials of those, of the sums to the run's end, to the chunk's end and
// from its start.  Sums to an end are taken from that end, so that they lose nothing to cancellation.
struct LaneGates {
    float dt[4], ph[4], pl[4], from_run[4], to_run[4], to_end[4], from_start[4];
    float tot[4], all;  // sums over the runs, and over the chunk
};
__device__ __forceinline__ void lane_gates(const float (&z)[4], int left, float rate, int lane, LaneGates& o) {
    float gl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o.dt[e] = e < left ? ssm_softplus(z[e]) : 0.f;
        gl[e] = e < left ? log_decay(rate, o.dt[e]) : 0.f;
    }
    Two pre[4];
    pre[0] = Two{gl[0], 0.f};
#pragma unroll
    for (int e = 1; e < 4; ++e) pre[e] = two_add(pre[e - 1], Two{gl[e], 0.f});
    Two run = pre[3];
    float suf = (gl[0] + gl[1]) + (gl[2] + gl[3]);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
        const Two up{__shfl_up_sync(0xffffffffu, run.h, d, 8), __shfl_up_sync(0xffffffffu, run.l, d, 8)};
        const float down = __shfl_down_sync(0xffffffffu, suf, d, 8);
        if ((lane & 7) >= d) run = two_add(up, run);
        if ((lane & 7) + d < 8) suf += down;
    }
    Two before{__shfl_up_sync(0xffffffffu, run.h, 1, 8), __shfl_up_sync(0xffffffffu, run.l, 1, 8)};
    if ((lane & 7) == 0) before = Two{0.f, 0.f};
    float behind = __shfl_down_sync(0xffffffffu, suf, 1, 8);
    if ((lane & 7) == 7) behind = 0.f;
    float head = 0.f, tail = 0.f;
    o.all = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        o.tot[u] = __shfl_sync(0xffffffffu, run.h, 8 * u + 7);
        if (u < lane >> 3) head += o.tot[u];
        if (u > lane >> 3) tail += o.tot[u];
        o.all += o.tot[u];
    }
#pragma unroll
    for (int e = 3; e >= 0; --e) {
        const Two p = two_add(before, pre[e]);
        o.ph[e] = p.h * kLog2e;
        // the product's rounding, and the low part
        o.pl[e] = fmaf(p.h, kLog2e, -o.ph[e]) + p.l * kLog2e + p.h * 1.9259629911266175e-8f;
        o.from_run[e] = expf(p.h);
        o.to_run[e] = expf(behind);
        o.to_end[e] = expf(behind + tail);
        o.from_start[e] = expf(head + p.h);
        behind += gl[e];
    }
}

// Rows of the gates of a chunk and head, and behind them e^{total} of the four runs and of the chunk.
enum Row { rPh, rPl, rFromRun, rToRun, rDt, rToEnd, rFromStart, kRows };
constexpr int kGates = kRows * kT + 8;

// ---- host ------------------------------------------------------------------------------------------

inline long slots128(int num_seqs, int total_T) { return (long)total_T / kT + num_seqs; }

// ssm_tc_scan.cu: the segments of a bf16 call; the gates of all chunks; the states that the segments begin with (no gates
// given: forwards).
inline size_t segments128(int num_seqs, int total_T, int H, int P, int N, int directions, bool varied, Segments* g, unsigned char* at) {
    const SegmentCost cost = directions == 1 ? SegmentCost{2.7, 1.7, 10.} : SegmentCost{1.8, 1.7, 8.};
    return segments_layout(num_seqs, total_T, H, P, N, kT, directions, varied, cost, g, at);
}
cudaError_t launch_gates128(const SsmArgs& a, float* gates, cudaStream_t s);
cudaError_t launch_starts(const SsmArgs& a, const float* gates, const Segments& g, int directions, cudaStream_t s);
// The images of the states at the chunks' starts and of their gradients at the chunks' ends: [slots][H][P / 64] of N x 64
// numbers each: row n, 16-byte vector c at place c ^ (n & 7).
cudaError_t launch_states(const SsmArgs& a, const float* gates, const Segments& g, float* states, float* dstates, cudaStream_t s);

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        const bool got = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                         q == cudaDriverEntryPointSuccess;
        return got ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// Rows of `width` bf16 elements, `stride` apart, in boxes of 128 rows and 64 columns; rows past the last read as zeros.
inline bool map_rows(CUtensorMap* m, const void* base, long rows, long width, long stride) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, kT}, es[2] = {1, 1};
    return encoder() && encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace ssm
}  // namespace gdn

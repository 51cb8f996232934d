// ssm_tc_scan.cu -- what lies between the chunks of 128 tokens of a bf16 scan: gates, states, and segments of long
// sequences.
//
// The states along a sequence, and their gradients backwards, are one product a chunk (U = B^T V, or C^T (b dy)) and
//   S <- e^{G_last} S + U.
// A walk along a sequence takes a block 1.7 us a chunk, the latency of its phases (tensor pipe 20%, issue slots 44%); two
// sequences of 4096 tokens, 32 heads of 64, d_state 128, in both directions: 54 us with 134 MB of images written, 2.5
// TB/s.  Both directions in one launch take as long as one.  Segments: see ssm_fwd.cu.
#include "ssm_tc.cuh"

namespace gdn {
namespace ssm {
namespace {

using namespace ptx;
using namespace tc;

// ---- gates ---------------------------------------------------------------------------------------

constexpr int kGateWarps = 8;
__global__ void __launch_bounds__(kGateWarps * 32) ssm_gates128_kernel(SsmArgs a, float* gates) {
    dependency_start();
    Chunk c;
    if (!find_chunk<kT>(a.seqs, blockIdx.x, a.err, c)) return;
    const int lane = threadIdx.x & 31, h = blockIdx.y * kGateWarps + (threadIdx.x >> 5);
    if (h >= a.H) return;
    const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = 4 * lane + e;
        z[e] = t < c.len ? a.a[(long)(c.t0 + t) * a.H + h] + bias : 0.f;
    }
    LaneGates o;
    lane_gates(z, c.len - 4 * lane, rate, lane, o);
    float* gt = gates + ((long)blockIdx.x * a.H + h) * kGates;
    const auto put = [&](int row, const float (&x)[4]) {
        *reinterpret_cast<float4*>(gt + row * kT + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
    };
    put(rPh, o.ph);
    put(rPl, o.pl);
    put(rFromRun, o.from_run);
    put(rToRun, o.to_run);
    put(rDt, o.dt);
    put(rToEnd, o.to_end);
    put(rFromStart, o.from_start);
    if (lane < 4) gt[kRows * kT + lane] = expf(lane == 0 ? o.tot[0] : (lane == 1 ? o.tot[1] : (lane == 2 ? o.tot[2] : o.tot[3])));
    if (lane == 4) gt[kRows * kT + 4] = expf(o.all);
}

// ---- states --------------------------------------------------------------------------------------

// Warps 0 - 7 form the factors (V, or b dy: three planes), 8 - 15 take the state on and lay its image out, 16 issues the
// MMAs, 17 the loads, 18 brings the gates.  Blocks with blockIdx.y = 1 go backwards, from dfinal_state.  With `own` the
// blocks leave their segments' states from zero, and nothing of the way.
struct ScanOut {
    const float* gates;  // or null: the blocks form them
    Segments g;
    bool own;
    float* images[2];
};
constexpr int kWorkers = 256, kScanThreads = 2 * kWorkers + 96;
enum ScanBar { KF0, KF1, KE0, KE1, XF0, XF1, XE0, XE1, GF0, GF1, GE0, GE1, VR, UD, SR, DR, kScanBars };
template <int N>
struct ScanLay {
    static constexpr int nb = N / 64, image = N * 256;
    static constexpr int k = 0, x = k + 2 * nb * kBlock, v = x + 2 * kBlock, st = v + 3 * kBlock, gates = st + 2 * image,
                         gate_bytes = (kT + 8) * 4, bars = gates + 2 * gate_bytes, bytes = bars + kScanBars * 8 + 16;
};

template <int N>
__global__ void __launch_bounds__(kScanThreads, 1)
ssm_scan_tc_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mY, const __grid_constant__ CUtensorMap mB,
                   const __grid_constant__ CUtensorMap mC, SsmArgs a, ScanOut w) {
    using L = ScanLay<N>;
    constexpr int NB = L::nb;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sm = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(smem + L::bars + kScanBars * 8);
    volatile int* dead = reinterpret_cast<volatile int*>(smem + L::bars + kScanBars * 8 + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const bool back = blockIdx.y;
    dependency_start();
    const int slices = a.P / 64, s = blockIdx.x % slices, h = blockIdx.x / slices % a.H, index = blockIdx.x / slices / a.H;
    Run run;
    // what a segment leaves goes to the next one: the last of a sequence has none
    if (!find_run(a.seqs, w.g.each, kT, index, a.err, run) || (w.own && (back ? run.first : run.last))) {
        dependency_wait();
        return;
    }
    const int bos = __shfl_sync(0xffffffffu, run.t0, 0), eos = __shfl_sync(0xffffffffu, run.end, 0);
    const int chunks = (eos - bos + kT - 1) / kT;
    const int g = h / (a.H / a.G);
    const long row0 = (((long)run.n * a.H + h) * a.P + s * 64) * N, own0 = (((long)index * a.H + h) * a.P + s * 64) * N;
    const long slot0 = run.slot0;
    const auto chunk_of = [&](int c) { return back ? chunks - 1 - c : c; };

    if (tid == 0) {
        for (int i = 0; i < kScanBars; ++i)
            mbar_init(&bars[i], i == VR || i == SR || i == XE0 || i == XE1 ? kWorkers : (i == GE0 || i == GE1 ? 2 * kWorkers : (i == GF0 || i == GF1 ? 32 : 1)));
        *dead = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tbase, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependency_wait();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tbase, 0);
    const uint32_t tU = tm, tS = tm + 192;  // U: the three planes' sums
    const auto wait = [&](int bar, int index) -> bool {
        bool ok = mbar_try_wait(&bars[bar], index & 1, 100000u);
        if (!ok) ok = wait_slow(&bars[bar], index & 1, dead, a.err);
        return __all_sync(0xffffffffu, ok);
    };
    const auto gates_of = [&](int c) { return reinterpret_cast<float*>(smem + L::gates + (c & 1) * L::gate_bytes); };

    if (warp < 8) {
        // ================= factors =================
        const int q = warp & 3, half = warp >> 2, i = q * 32 + lane;
        for (int c = 0; c < chunks; ++c) {
            if (!wait(GF0 + (c & 1), c >> 1)) break;
            const float f = gates_of(c)[i];
            mbar_arrive(&bars[GE0 + (c & 1)]);
            const int left = eos - bos - chunk_of(c) * kT;
            if (!wait(XF0 + (c & 1), c >> 1)) break;
            if (left < kT && !wait(KF0 + (c & 1), c >> 1)) break;
            if (c > 0 && !wait(UD, c - 1)) break;
            const uint32_t xt = sm + L::x + (c & 1) * kBlock;
            const bool live = i < left;
#pragma unroll 2
            for (int k = half * 4; k < half * 4 + 4; ++k) {
                uint32_t u[4] = {0, 0, 0, 0}, v[3][4];
                if (live) planes::lds128(at16(xt, i, k), u);
                else
                    for (int b = 0; b < NB; ++b) planes::sts128(at16(sm + L::k + ((c & 1) * NB + b) * kBlock, i, k), u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bfp::F2 t = bfp::widen(u[e]) * bfp::F2(f, f);
                    v[0][e] = bfp::peel(t);
                    v[1][e] = bfp::peel(t);
                    v[2][e] = bfp::pack(t);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) planes::sts128(at16(sm + L::v + p * kBlock, i, k), v[p]);
            }
            fence_async_smem();
            mbar_arrive(&bars[XE0 + (c & 1)]);
            mbar_arrive(&bars[VR]);
        }
    } else if (warp < 16) {
        // ================= state =================
        const int q = warp & 3, half = (warp >> 2) & 1, r = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const bool holds = r < N, leader = tid == kWorkers;
        const float* init = nullptr;
        float* last = nullptr;
        if (w.own) {
            last = (back ? w.g.own[1] : w.g.own[0]) + own0;
        } else if (w.g.each) {
            init = (back ? w.g.start[1] : w.g.start[0]) + own0;
        } else {
            const float* given = back ? a.dfinal_state : a.initial_state;
            init = given ? given + row0 : nullptr;
        }
        if (!w.own && back && run.first && a.dinitial_state) last = a.dinitial_state + row0;
        float decay = 0.f, total = 1.f;
        for (int c = 0; c <= chunks; ++c) {
            bool ok = c == 0 || wait(UD, c - 1);
            tc_fence_after();
            if (c < chunks) {  // the image before the last one has been read by its copy
                if (leader) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                if (bar_sync_or(1, kWorkers, !ok)) break;
            } else if (!ok) {
                break;
            }
            const uint32_t st = sm + L::st + (c & 1) * L::image;
#pragma unroll 2
            for (int k = 0; k < 4; ++k) {
                const int col = half * 32 + 8 * k;
                bfp::F2 S[4];
                if (c == 0) {
#pragma unroll
                    for (int p = 0; p < 8; p += 2) {
                        const float* from = init + (long)(col + p) * N + r;
                        S[p / 2] = holds && init ? bfp::F2(from[0], from[N]) : bfp::F2(0.f, 0.f);
                    }
                } else {
                    uint32_t old[8], hi[8], mid[8], lo[8];
                    tmem_ld8(tS + lanes + col, old);
                    tmem_ld8(tU + lanes + col, hi);
                    tmem_ld8(tU + lanes + 64 + col, mid);
                    tmem_ld8(tU + lanes + 128 + col, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int p = 0; p < 8; p += 2)
                        S[p / 2] = bfp::fma2(bfp::F2(decay, decay), bfp::F2::of(old[p], old[p + 1]),
                                             bfp::F2::of(hi[p], hi[p + 1]) + (bfp::F2::of(mid[p], mid[p + 1]) + bfp::F2::of(lo[p], lo[p + 1])));
                }
                float v[8];
#pragma unroll
                for (int p = 0; p < 4; ++p) S[p].get(v[2 * p], v[2 * p + 1]);
                if (c == chunks) {
                    if (holds && last) {
#pragma unroll
                        for (int p = 0; p < 8; ++p) last[(long)(col + p) * N + r] = v[p];
                    }
                    continue;
                }
                uint32_t u[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) u[p] = __float_as_uint(v[p]);
                tmem_st8(tS + lanes + col, u);
                if (holds && !w.own) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t part[4] = {u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]};
                        planes::sts128(st + r * 256 + (((half * 8 + 2 * k + e) ^ (r & 7)) << 4), part);
                    }
                }
            }
            if (c == chunks) break;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars[SR]);
            fence_async_smem();
            ok = wait(GF0 + (c & 1), c >> 1);
            decay = gates_of(c)[kT];
            total *= decay;
            mbar_arrive(&bars[GE0 + (c & 1)]);
            if (bar_sync_or(1, kWorkers, !ok)) break;
            if (leader && !w.own) {
                float* to = (back ? w.images[1] : w.images[0]) + (((slot0 + chunk_of(c)) * a.H + h) * slices + s) * (long)(N * 64);
                bulk_store(to, smem + L::st + (c & 1) * L::image, L::image);
                bulk_commit();
            }
        }
        if (leader && w.own && s == 0) (back ? w.g.decay[1] : w.g.decay[0])[(long)index * a.H + h] = total;
        if (leader) bulk_wait_all();
    } else if (warp == 16) {
        // ================= MMAs =================
        constexpr uint32_t idU = idesc_bf16(128, 192, 1, 1);
        const uint32_t on = elect();
        const uint64_t dV = sdesc_sw128(sm + L::v, kBlock, 1024);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const uint64_t dK = sdesc_sw128(sm + L::k + st * NB * kBlock, kBlock, 1024);
            if (!wait(KF0 + st, c >> 1) || !wait(SR, c) || !wait(VR, c)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kT / 16; ++k) mma_ss(on, tU, dK + k * 128, dV + k * 128, idU, k > 0);
            commit(on, &bars[UD]);
            commit(on, &bars[KE0 + st]);
        }
        if (chunks > 0) {
            commit(on, &bars[DR]);
            mbar_wait(&bars[DR], 0, kLimit);
        }
    } else if (warp == 17) {
        // ================= loads =================
        const uint32_t on = elect();
        int nk = 0, nx = 0;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, t0 = bos + chunk_of(c) * kT;
            if (c >= 2 && !wait(XE0 + st, (c >> 1) - 1)) break;
            if (on) {
                mbar_arrive_expect_tx(&bars[XF0 + st], kBlock);
                tma_load_2d(smem + L::x + st * kBlock, back ? &mY : &mX, &bars[XF0 + st], h * a.P + s * 64, t0);
            }
            ++nx;
            if (c >= 2 && !wait(KE0 + st, (c >> 1) - 1)) break;
            if (on) {
                mbar_arrive_expect_tx(&bars[KF0 + st], NB * kBlock);
                for (int q = 0; q < NB; ++q)
                    tma_load_2d(smem + L::k + (st * NB + q) * kBlock, back ? &mC : &mB, &bars[KF0 + st], g * N + 64 * q, t0);
            }
            ++nk;
        }
        for (int k = max(0, nk - 2); k < nk; ++k) mbar_wait(&bars[KF0 + (k & 1)], (k >> 1) & 1, kLimit);
        for (int k = max(0, nx - 2); k < nx; ++k) mbar_wait(&bars[XF0 + (k & 1)], (k >> 1) & 1, kLimit);
    } else {
        // ================= gates =================
        const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        for (int c = 0; c < chunks; ++c) {
            float4 f;
            float all;
            if (w.gates) {
                const float* gt = w.gates + ((slot0 + chunk_of(c)) * a.H + h) * (long)kGates;
                f = *reinterpret_cast<const float4*>(gt + (back ? rFromStart : rToEnd) * kT + 4 * lane);
                if (!back) {
                    const float4 d = *reinterpret_cast<const float4*>(gt + rDt * kT + 4 * lane);
                    f = make_float4(f.x * d.x, f.y * d.y, f.z * d.z, f.w * d.w);
                }
                all = gt[kRows * kT + 4];
            } else {  // forwards
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = bos + c * kT + 4 * lane + e;
                    z[e] = t < eos ? a.a[(long)t * a.H + h] + bias : 0.f;
                }
                LaneGates o;
                lane_gates(z, eos - bos - c * kT - 4 * lane, rate, lane, o);
                f = make_float4(o.to_end[0] * o.dt[0], o.to_end[1] * o.dt[1], o.to_end[2] * o.dt[2], o.to_end[3] * o.dt[3]);
                all = expf(o.all);
            }
            if (c >= 2 && !wait(GE0 + (c & 1), (c >> 1) - 1)) break;
            float* to = gates_of(c);
            *reinterpret_cast<float4*>(to + 4 * lane) = f;
            if (lane == 0) to[kT] = all;
            mbar_arrive(&bars[GF0 + (c & 1)]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tm, 256);
    }
}

template <int N>
cudaError_t launch_scan128(const SsmArgs& a, const ScanOut& w, int directions, cudaStream_t s) {
    CUtensorMap mX, mY{}, mB, mC{};
    const long T = a.seqs.total_T;
    if (!map_rows(&mX, a.x, T, (long)a.H * a.P, a.x_stride) || !map_rows(&mB, a.B, T, (long)a.G * N, a.B_stride)) return cudaErrorInvalidValue;
    if (directions == 2 && (!map_rows(&mY, a.dout, T, (long)a.H * a.P, (long)a.H * a.P) || !map_rows(&mC, a.C, T, (long)a.G * N, a.C_stride)))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(ssm_scan_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, ScanLay<N>::bytes);
    if (e != cudaSuccess) return e;
    const long runs = w.g.each ? segment_slots(a.seqs.num_seqs, a.seqs.total_T, w.g) : a.seqs.num_seqs;
    const dim3 grid((unsigned)(runs * a.H * (a.P / 64)), directions);
    if (w.gates) return launch_after(ssm_scan_tc_kernel<N>, grid, kScanThreads, ScanLay<N>::bytes, s, mX, mY, mB, mC, a, w);
    // the call's first kernel
    ssm_scan_tc_kernel<N><<<grid, kScanThreads, ScanLay<N>::bytes, s>>>(mX, mY, mB, mC, a, w);
    return cudaGetLastError();
}

}  // namespace

namespace tc {

cudaError_t launch_gates128(const SsmArgs& a, float* gates, cudaStream_t s) {
    const dim3 grid((unsigned)slots128(a.seqs.num_seqs, a.seqs.total_T), (unsigned)((a.H + kGateWarps - 1) / kGateWarps));
    ssm_gates128_kernel<<<grid, kGateWarps * 32, 0, s>>>(a, gates);
    return cudaGetLastError();
}

cudaError_t launch_starts(const SsmArgs& a, const float* gates, const Segments& g, int directions, cudaStream_t s) {
    const ScanOut w{gates, g, true, {nullptr, nullptr}};
    const cudaError_t e = a.N == 128 ? launch_scan128<128>(a, w, directions, s) : launch_scan128<64>(a, w, directions, s);
    if (e != cudaSuccess) return e;
    return launch_join(a, g, directions, s);
}

cudaError_t launch_states(const SsmArgs& a, const float* gates, const Segments& g, float* states, float* dstates, cudaStream_t s) {
    const ScanOut w{gates, g, false, {states, dstates}};
    return a.N == 128 ? launch_scan128<128>(a, w, 2, s) : launch_scan128<64>(a, w, 2, s);
}

}  // namespace tc
}  // namespace ssm
}  // namespace gdn

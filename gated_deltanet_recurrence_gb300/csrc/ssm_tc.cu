// ssm_tc.cu -- the selective state space scan over packed bf16 prompts on the tensor cores (tcgen05), in one kernel.
//
// The chunked form (see ssm_fwd.cu) with chunks of 128 tokens.  A block takes one (sequence, head, 64 rows of the
// state) and walks along its chunks; nothing but inputs, outputs and the states at both ends touches memory.  Per
// chunk four products, accumulated in TMEM:
//   CB = C B^T                         [128 tokens x 128 tokens], exact inputs
//   CS = C [S hi | S mid]              [128 tokens x 64 | 64], the state at the chunk's start in two bf16 planes
//   U  = B^T [V hi | V mid + V lo]     [N x 64 | 64], V_j = e^{G_last - G_j} dt_j x_j in three planes
//   MX = (CB o decays dt) X            [128 tokens x 64], its left side in two planes, from TMEM
// The planes of a factor lie side by side, so that the other one is read once for all of them (an instruction with
// N = 64 is bound by reading the left operand); their results are added in registers.  The state itself stays in TMEM in
// fp32 and is taken through registers once a chunk: S <- e^{G_last} S + U with rounded additions (the tensor cores
// cut sums off, which a state carried through many chunks would keep).
//
// Warps: 0 - 7 form the masked products M of a chunk and, while M X and the next C B^T run, the V of the next chunk (a
// thread is a token and half of what its row needs); 8 - 15 take the state on (a thread is a state column [the N side]
// and half of its 64 rows) and the outputs out (a token and half its row); 16 issues the MMAs, 17 the loads, 18 forms
// the gates.  Decays of pairs of tokens in different runs of 32 are products of two factors that are at most 1; inside a
// run they are exponentials of differences of sums in two floats.
// The bodies of all loops are a few dozen instructions: nineteen warps in five roles share the instruction caches,
// and straight code was fetched no faster than an instruction in four cycles.
//
// What bounds it is a chunk's chain of phases: 2.7 us whatever the number of blocks (shared memory about 3900 of a
// chunk's 5200 cycles, the tensor pipe 34%, issue slots 54%).  Two sequences of 4096 tokens, 64 heads of 64, d_state 128:
// 90 us, 1.6 TB/s, 190 TFLOP/s of the recurrence in chunks; 32768 tokens of 16 heads in segments (ssm_fwd.cu) 136 us.  Three
// kernels on mma.sync with chunks of 64, as for fp32, took 360 us.
//
// Every mbarrier wait is bounded; when one runs out the kernel records GDN_ERR_TIMEOUT, every role leaves its loop,
// copies and MMAs in flight are waited for (bounded), TMEM is freed.
#include "ssm_tc.cuh"

namespace gdn {
namespace ssm {
namespace {

using namespace ptx;
using namespace tc;

constexpr int kWorkers = 256;              // threads of a role's two sets of four warps
constexpr int kThreads = 2 * kWorkers + 3 * 32;

enum Bar { FB, EB, FC0, FC1, EC0, EC1, FX0, FX1, EX0, EX1, GF0, GF1, GE0, GE1, VR, UA, UD, SR, CSD, CBD, MR, YD, YE, DR, kBars };

template <int N>
struct Lay {
    static constexpr int nb = N / 64;  // tiles of B and of C
    static constexpr int b = 0, c = b + nb * kBlock, x = c + 2 * nb * kBlock, v = x + 2 * kBlock, s = v + 3 * kBlock,
                         gates = s + 2 * kBlock, gate_rows = 6, gate_bytes = (gate_rows * kT + 8) * 4,
                         bars = gates + 2 * gate_bytes, bytes = bars + kBars * 8 + 16;
};
// rows of the gates of a chunk: sums from the start of the token's run of 32 in two floats (log2), the second less log2
// dt, e^{sums to the run's end} dt, e^{sums to the chunk's end} dt, e^{sums from the chunk's start}; then e^{total} of
// the runs and of the chunk
enum Gate { kPh, kPl, kPd, kQ, kW, kB };

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
ssm_tc_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mC,
              SsmArgs a, Segments w) {
    using L = Lay<N>;
    constexpr int NB = L::nb;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sm = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(smem + L::bars + kBars * 8);
    volatile int* dead = reinterpret_cast<volatile int*>(smem + L::bars + kBars * 8 + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int slices = a.P / 64, s = blockIdx.x % slices, h = blockIdx.x / slices % a.H, index = blockIdx.x / slices / a.H;
    Run run;
    if (!find_run(a.seqs, w.each, kT, index, a.err, run)) {
        dependency_wait();
        return;
    }
    const int bos = __shfl_sync(0xffffffffu, run.t0, 0), eos = __shfl_sync(0xffffffffu, run.end, 0);
    const int chunks = (eos - bos + kT - 1) / kT;
    const int g = h / (a.H / a.G);
    const long row0 = (((long)run.n * a.H + h) * a.P + s * 64) * N;
    const float* init = a.initial_state ? a.initial_state + row0 : nullptr;
    if (w.each) init = w.start[0] + (((long)index * a.H + h) * a.P + s * 64) * N;
    float* last = run.last && a.final_state ? a.final_state + row0 : nullptr;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            const bool all = i == VR || i == SR || i == MR || i == YE || i == EX0 || i == EX1;
            mbar_init(&bars[i], all ? kWorkers : (i == GE0 || i == GE1 ? 2 * kWorkers : (i == GF0 || i == GF1 ? 32 : 1)));
        }
        *dead = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tbase, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependency_wait();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tbase, 0);
    const uint32_t tU = tm, tS = tm + 128, tCS = tm + 192, tMX = tm + 320, tCB = tm + 384;

    // the completion number `index` of a barrier; false once a wait has run out here or elsewhere.  A whole warp goes on
    // or none of it.
    const auto wait = [&](int bar, int index) -> bool {
        bool ok = mbar_try_wait(&bars[bar], index & 1, 100000u);
        if (!ok) ok = wait_slow(&bars[bar], index & 1, dead, a.err);
        return __all_sync(0xffffffffu, ok);
    };
    const auto gates_of = [&](int c) { return reinterpret_cast<float*>(smem + L::gates + (c & 1) * L::gate_bytes); };

    if (warp < 8) {
        // ================= masked products and V =================
        const int q = warp & 3, half = warp >> 2, i = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        // which runs of columns this warp masks: of the rows' q + 1 and the zeros behind them, about half each
        const uint32_t mine = half ? (q == 0 ? 14u : (q == 1 ? 10u : 12u)) : (q == 0 ? 1u : (q == 1 ? 5u : 3u));
        // V of this token; rows past the sequence's end become zeros wherever they are summed over
        const auto form_v = [&](int c) -> bool {
            if (!wait(GF0 + (c & 1), c >> 1)) return false;
            const float w = gates_of(c)[kW * kT + i];
            if (!wait(FX0 + (c & 1), c >> 1)) return false;
            if (c + 1 == chunks && !wait(FB, c)) return false;
            if (c > 0 && !wait(UD, c - 1)) return false;
            const uint32_t xt = sm + L::x + (c & 1) * kBlock;
            const bool live = i < eos - bos - c * kT;
#pragma unroll 2
            for (int k = half * 4; k < half * 4 + 4; ++k) {
                uint32_t u[4] = {0, 0, 0, 0}, v[3][4];
                if (live) planes::lds128(at16(xt, i, k), u);
                else {
                    planes::sts128(at16(xt, i, k), u);
                    for (int b = 0; b < NB; ++b) planes::sts128(at16(sm + L::b + b * kBlock, i, k), u);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bfp::F2 t = bfp::widen(u[e]) * bfp::F2(w, w);
                    v[0][e] = bfp::peel(t);
                    v[1][e] = bfp::peel(t);
                    v[2][e] = bfp::pack(t);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) planes::sts128(at16(sm + L::v + p * kBlock, i, k), v[p]);
            }
            fence_async_smem();
            mbar_arrive(&bars[VR]);
            return true;
        };
        for (int c = 0; c < chunks; ++c) {
            if (c == 0 && !form_v(0)) break;
            const float* gt = gates_of(c);
            const float ph = gt[kPh * kT + i], pl = gt[kPl * kT + i];
            // e^{sums from the end of run u to this token} for this warp's runs before the token's
            float f0 = exp2_hw(ph + pl), f1 = f0;
            if (q == 3 && half == 0) {
                f1 = f0 * gt[L::gate_rows * kT + 2];
                f0 = f1 * gt[L::gate_rows * kT + 1];
            } else if (q == 2 && half == 0) {
                f0 *= gt[L::gate_rows * kT + 1];
            }
            if (!wait(CBD, c)) break;
            tc_fence_after();
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                if (!(mine >> u & 1)) continue;
                const uint32_t at = tCB + lanes + 32 * u;
                if (u > q) {
                    const uint32_t zero[8] = {};
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) tmem_st8(at + 8 * k, zero);
                    continue;
                }
                const float f = u & 1 ? f1 : f0;
                // the two planes of sixteen columns, eight words each, take those columns' place
                uint32_t next[16];
                tmem_ld16(at, next);
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t r[16], hi[8], lo[8];
                    bfp::F2 m[8];
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = next[j];
                    if (k == 0) tmem_ld16(at + 16, next);
                    const float* base = gt + 32 * u + 16 * k;
                    if (u == q) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 th = *reinterpret_cast<const float4*>(base + kPh * kT + j);
                            const float4 td = *reinterpret_cast<const float4*>(base + kPd * kT + j);
                            const bfp::F2 one(-1.f, -1.f);
                            bfp::F2 d[2] = {bfp::fma2(bfp::F2(th.x, th.y), one, bfp::F2(ph, ph)) + bfp::fma2(bfp::F2(td.x, td.y), one, bfp::F2(pl, pl)),
                                            bfp::fma2(bfp::F2(th.z, th.w), one, bfp::F2(ph, ph)) + bfp::fma2(bfp::F2(td.z, td.w), one, bfp::F2(pl, pl))};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x, y;
                                d[e].get(x, y);
                                (bfp::F2::of(r[j + 2 * e], r[j + 2 * e + 1]) * bfp::F2(exp2_hw(x), exp2_hw(y))).get(x, y);
                                // what lies behind the token is selected away
                                x = 16 * k + j + 2 * e <= lane ? x : 0.f;
                                y = 16 * k + j + 2 * e + 1 <= lane ? y : 0.f;
                                m[j / 2 + e] = bfp::F2(x, y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(base + kQ * kT + j);
                            m[j / 2] = bfp::F2::of(r[j], r[j + 1]) * bfp::F2(t.x, t.y) * bfp::F2(f, f);
                            m[j / 2 + 1] = bfp::F2::of(r[j + 2], r[j + 3]) * bfp::F2(t.z, t.w) * bfp::F2(f, f);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        hi[j] = bfp::peel(m[j]);
                        lo[j] = bfp::pack(m[j]);
                    }
                    tmem_st8(at + 16 * k, hi);
                    tmem_st8(at + 16 * k + 8, lo);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars[MR]);
            mbar_arrive(&bars[GE0 + (c & 1)]);
            if (c + 1 < chunks && !form_v(c + 1)) break;
        }
    } else if (warp < 16) {
        // ================= state and outputs =================
        const int q = warp & 3, half = (warp >> 2) & 1, r = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const bool holds = r < N;
        const float D = a.D ? a.D[h] : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((long)bos * a.H + h) * a.P + s * 64 + half * 32;
        const long out_stride = (long)a.H * a.P;
        float decay = 0.f;
        for (int c = 0; c <= chunks; ++c) {
            // the state at the start of chunk c
            if (c > 0) {
                if (!wait(UD, c - 1)) break;
                if (c < chunks && !wait(CSD, c - 1)) break;
                tc_fence_after();
            }
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
                    uint32_t old[8], hi[8], mid[8];
                    tmem_ld8(tS + lanes + col, old);
                    tmem_ld8(tU + lanes + col, hi);
                    tmem_ld8(tU + lanes + 64 + col, mid);
                    tmem_wait_ld();
#pragma unroll
                    for (int p = 0; p < 8; p += 2)
                        S[p / 2] = bfp::fma2(bfp::F2(decay, decay), bfp::F2::of(old[p], old[p + 1]),
                                             bfp::F2::of(hi[p], hi[p + 1]) + bfp::F2::of(mid[p], mid[p + 1]));
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
                uint32_t w[8], hi[4], mid[4];
#pragma unroll
                for (int p = 0; p < 8; ++p) w[p] = __float_as_uint(v[p]);
                tmem_st8(tS + lanes + col, w);
                if (holds) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        hi[e] = bfp::peel(S[e]);
                        mid[e] = bfp::pack(S[e]);
                    }
                    planes::sts128(at16(sm + L::s, r, half * 4 + k), hi);
                    planes::sts128(at16(sm + L::s + kBlock, r, half * 4 + k), mid);
                }
            }
            if (c < chunks) {
                tmem_wait_st();
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&bars[SR]);
                if (!wait(GF0 + (c & 1), c >> 1)) break;
                decay = gates_of(c)[L::gate_rows * kT + 4];
            }
            if (c == 0) continue;
            // the outputs of chunk c - 1: token r
            const int d = c - 1;
            const float bi = gates_of(d)[kB * kT + r];
            if (!wait(YD, d)) break;
            tc_fence_after();
            const uint32_t xt = sm + L::x + (d & 1) * kBlock;
#pragma unroll 2
            for (int k = 0; k < 4; ++k) {
                uint32_t hi[8], mid[8], mx[8], u[4];
                const int col = half * 32 + 8 * k;
                tmem_ld8(tCS + lanes + col, hi);
                tmem_ld8(tCS + lanes + 64 + col, mid);
                tmem_ld8(tMX + lanes + col, mx);
                const uint32_t at = at16(xt, r, half * 4 + k);
                planes::lds128(at, u);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bfp::F2 y = bfp::fma2(bfp::F2(bi, bi), bfp::F2::of(hi[2 * e], hi[2 * e + 1]) + bfp::F2::of(mid[2 * e], mid[2 * e + 1]),
                                                bfp::F2::of(mx[2 * e], mx[2 * e + 1]));
                    u[e] = bfp::pack(bfp::fma2(bfp::F2(D, D), bfp::widen(u[e]), y));
                }
                planes::sts128(at, u);  // y takes x's place
            }
            tc_fence_before();
            mbar_arrive(&bars[YE]);
            mbar_arrive(&bars[GE0 + (d & 1)]);
            __syncwarp();
            const int len = min(eos - bos - d * kT, kT);
            // eight rows of 64 bytes at a time
            uint32_t u[4][4];
            const int t = q * 32 + (lane >> 2), col = lane & 3;
#pragma unroll
            for (int k = 0; k < 4; ++k) planes::lds128(at16(xt, t + 8 * k, half * 4 + col), u[k]);
            __nv_bfloat16* to = out + ((long)d * kT + t) * out_stride + col * 8;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t + 8 * k < len) *reinterpret_cast<uint4*>(to + 8 * k * out_stride) = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
            fence_async_smem();
            mbar_arrive(&bars[EX0 + (d & 1)]);
        }
    } else if (warp == 16) {
        // ================= MMAs =================
        constexpr uint32_t idCB = idesc_bf16(128, 128, 0, 0), idCS = idesc_bf16(128, 128, 0, 1), idU = idesc_bf16(128, 128, 1, 1),
                           idUl = idesc_bf16(128, 64, 1, 1), idMX = idesc_bf16(128, 64, 0, 1);
        const uint32_t on = elect();
        const uint64_t dBk = sdesc_sw128(sm + L::b, 16, 1024), dBm = sdesc_sw128(sm + L::b, kBlock, 1024),
                       dS = sdesc_sw128(sm + L::s, kBlock, 1024), dV = sdesc_sw128(sm + L::v, kBlock, 1024);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const uint64_t dCk = sdesc_sw128(sm + L::c + st * NB * kBlock, 16, 1024),
                           dX = sdesc_sw128(sm + L::x + st * kBlock, kBlock, 1024);
            if (!wait(FB, c) || !wait(FC0 + st, c >> 1)) break;
            if (c > 0 && !wait(YD, c - 1)) break;  // MX has read the masked products that CB overwrites
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < N / 16; ++k) {
                const uint64_t off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
                mma_ss(on, tCB, dCk + off, dBk + off, idCB, k > 0);
            }
            commit(on, &bars[CBD]);
            if (!wait(SR, c) || !wait(VR, c)) break;  // (SR: the state has taken the former U in)
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kT / 16; ++k) mma_ss(on, tU, dBm + k * 128, dV + k * 128, idU, k > 0);
            commit(on, &bars[UA]);
            if (c > 0 && !wait(YE, c - 1)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < N / 16; ++k)
                mma_ss(on, tCS, dCk + (((k >> 2) * kBlock + (k & 3) * 32) >> 4), dS + k * 128, idCS, k > 0);
            commit(on, &bars[CSD]);
            commit(on, &bars[EC0 + st]);
            // the low plane's sums go into the middle one's columns; MMAs of two shapes on the same columns are not
            // ordered by themselves
            if (!wait(UA, c)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kT / 16; ++k) mma_ss(on, tU + 64, dBm + k * 128, dV + 2 * (kBlock >> 4) + k * 128, idUl, 1);
            commit(on, &bars[UD]);
            commit(on, &bars[EB]);
            if (!wait(FX0 + st, c >> 1) || !wait(MR, c)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 1; p >= 0; --p)
#pragma unroll
                for (int k = 0; k < kT / 16; ++k) mma_ts(on, tMX, tCB + 16 * k + 8 * p, dX + k * 128, idMX, p == 0 || k > 0);
            commit(on, &bars[YD]);
        }
        if (chunks > 0) {  // MMAs in flight, after a wait that ran out, end before TMEM is freed
            commit(on, &bars[DR]);
            mbar_wait(&bars[DR], 0, kLimit);
        }
    } else if (warp == 17) {
        // ================= loads =================
        const uint32_t on = elect();
        int nb = 0, nc = 0, nx = 0;  // loads issued
        const int xc = h * a.P + s * 64, gc = g * N;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, t0 = bos + c * kT;
            if (c >= 2 && !wait(EX0 + st, (c >> 1) - 1)) break;
            if (on) {
                mbar_arrive_expect_tx(&bars[FX0 + st], kBlock);
                tma_load_2d(smem + L::x + st * kBlock, &mX, &bars[FX0 + st], xc, t0);
                if (c + 1 < chunks) prefetch_2d(&mX, xc, t0 + kT);
            }
            ++nx;
            if (c >= 2 && !wait(EC0 + st, (c >> 1) - 1)) break;
            if (on) {
                mbar_arrive_expect_tx(&bars[FC0 + st], NB * kBlock);
                for (int q = 0; q < NB; ++q) tma_load_2d(smem + L::c + (st * NB + q) * kBlock, &mC, &bars[FC0 + st], gc + 64 * q, t0);
                // B has one place only: its next tile waits in L2
                if (c + 1 < chunks)
                    for (int q = 0; q < NB; ++q) prefetch_2d(&mB, gc + 64 * q, t0 + kT);
            }
            ++nc;
            if (c >= 1 && !wait(EB, c - 1)) break;
            if (on) {
                mbar_arrive_expect_tx(&bars[FB], NB * kBlock);
                for (int q = 0; q < NB; ++q) tma_load_2d(smem + L::b + q * kBlock, &mB, &bars[FB], gc + 64 * q, t0);
            }
            ++nb;
        }
        // the last loads have landed before the block may leave
        for (int k = max(0, nc - 2); k < nc; ++k) mbar_wait(&bars[FC0 + (k & 1)], (k >> 1) & 1, kLimit);
        for (int k = max(0, nx - 2); k < nx; ++k) mbar_wait(&bars[FX0 + (k & 1)], (k >> 1) & 1, kLimit);
        if (nb > 0) mbar_wait(&bars[FB], (nb - 1) & 1, kLimit);
    } else {
        // ================= gates =================
        const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        float z[4];
        const auto fetch = [&](int c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = bos + c * kT + 4 * lane + e;
                z[e] = t < eos ? a.a[(long)t * a.H + h] : 0.f;
            }
        };
        if (chunks > 0) fetch(0);
        for (int c = 0; c < chunks; ++c) {
            LaneGates o;
            float zb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) zb[e] = z[e] + bias;
            lane_gates(zb, eos - bos - c * kT - 4 * lane, rate, lane, o);
            if (c + 1 < chunks) fetch(c + 1);
            if (c >= 2 && !wait(GE0 + (c & 1), (c >> 1) - 1)) break;
            float* gt = gates_of(c);
            float pd[4], q[4], w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pd[e] = o.pl[e] - log2f(o.dt[e]);  // no step: an exponential of -inf
                q[e] = o.to_run[e] * o.dt[e];
                w[e] = o.to_end[e] * o.dt[e];
            }
            const auto put = [&](int row, const float (&x)[4]) {
                *reinterpret_cast<float4*>(gt + row * kT + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
            };
            put(kPh, o.ph);
            put(kPl, o.pl);
            put(kPd, pd);
            put(kQ, q);
            put(kW, w);
            put(kB, o.from_start);
            if (lane < 4) gt[L::gate_rows * kT + lane] = expf(lane == 0 ? o.tot[0] : (lane == 1 ? o.tot[1] : (lane == 2 ? o.tot[2] : o.tot[3])));
            if (lane == 4) gt[L::gate_rows * kT + 4] = expf(o.all);
            mbar_arrive(&bars[GF0 + (c & 1)]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

template <int N>
cudaError_t launch(const SsmArgs& a, const Segments& w, cudaStream_t s) {
    CUtensorMap mX, mB, mC;
    const long T = a.seqs.total_T;
    if (!encoder() || !map_rows(&mX, a.x, T, (long)a.H * a.P, a.x_stride) || !map_rows(&mB, a.B, T, (long)a.G * N, a.B_stride) ||
        !map_rows(&mC, a.C, T, (long)a.G * N, a.C_stride))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(ssm_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::bytes);
    if (e != cudaSuccess) return e;
    const long runs = w.each ? segment_slots(a.seqs.num_seqs, a.seqs.total_T, w) : a.seqs.num_seqs;
    const dim3 grid((unsigned)(runs * a.H * (a.P / 64)));
    if (w.each) return launch_after(ssm_tc_kernel<N>, grid, kThreads, Lay<N>::bytes, s, mX, mB, mC, a, w);
    ssm_tc_kernel<N><<<grid, kThreads, Lay<N>::bytes, s>>>(mX, mB, mC, a, w);
    return cudaGetLastError();
}

}  // namespace

size_t tc_workspace_bytes(int num_seqs, int total_T, int H, int P, int N) {
    size_t most = 0;
    for (int varied = 0; varied < 2; ++varied) {
        const size_t segments = segments128(num_seqs, total_T, H, P, N, 1, varied, nullptr, nullptr);
        if (segments > most) most = segments;
    }
    return most;
}

cudaError_t launch_tc(const SsmArgs& a, cudaStream_t s) {
    Segments w{};
    const Packed& q = a.seqs;
    segments128(q.num_seqs, q.total_T, a.H, a.P, a.N, 1, q.cu && q.num_seqs > 1, &w, static_cast<unsigned char*>(a.workspace));
    if (w.each) {
        const cudaError_t e = launch_starts(a, nullptr, w, 1, s);
        if (e != cudaSuccess) return e;
    }
    return a.N == 128 ? launch<128>(a, w, s) : launch<64>(a, w, s);
}

}  // namespace ssm
}  // namespace gdn

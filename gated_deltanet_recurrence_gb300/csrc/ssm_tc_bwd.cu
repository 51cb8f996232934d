// ssm_tc_bwd.cu -- the gradients of the selective scan of bf16 prompts on the tensor cores (tcgen05).
//
// The formulas are those of ssm_bwd.cu, with chunks of 128 tokens.  The gates of all chunks and the states at the chunks'
// starts, with their gradients at the chunks' ends, come from ssm_tc_scan.cu; here the gradients, one block per chunk and
// subset of a group's heads.
//
// A head's step is a chain of phases, about 19000 cycles, one block an SM for its tiles: planes of dS (2100), products
// with it (2200), their results (1000 - 2400), planes of S_0 and dy . x (1500), masks and planes of M (4000), products
// with those (2100), dx and dC (2500); the tensor pipe is busy 13% of it.  All of a chunk is on the way through
// registers, whose 64,000 the accumulators of dB, dC and E fill, so that steps do not overlap.  Tried, and no faster: 256
// threads, rolled loops for the masks (260 us for 255 of the call below), tiles of both states at once with their
// conversion beside the products (254). Two sequences of 4096 tokens, 32 heads of 64 in two groups, d_state 128: 171 us
// of the call's 236 (with states 54, gates 4, sums 4; kernels on mma.sync took 735).
//
// Every fp32 factor is three bf16 planes, exact beside the bf16 inputs; where a factor's planes lie side by side, the
// input is read once for all of them.  All matrices of pairs of tokens are held with row j (the earlier token) and
// column i >= j, as they are needed: (C B^T)^T once a block; per head dy . x; the masked decays' products M^T as the left
// operand of M^T dy from TMEM; E^T summed over the heads in registers.
//   dg_t = sum over pairs i >= t > j of T_ij + sum_{i >= t} b_i dy_i . S_0 C_i + b_last <dS_1, S_0>
//          + sum_{j < t} r_j v_j . dS_1 B_j
// is taken as it stands, without subtractions: suffix sums of T along a row, added over the rows before t.
#include <type_traits>

#include "ssm_tc.cuh"

namespace gdn {
namespace ssm {
namespace {

using namespace ptx;
using namespace tc;

struct TcWork {
    float* gates;    // [slots][H][kGates]
    float* states;   // images, see launch_states
    float* dstates;
    float* sums;
    float* parts;
    int subsets;
    Segments g;
};

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kSums = 5 * 4 * kT + 2 * kGradWarps;  // numbers that the steps of a head leave for its dg
enum GradBar { LB, LX0, LX1, LS, MM, kGradBars };
template <int N>
struct GradLay {
    static constexpr int nb = N / 64, image = N * 256;
    static constexpr int b = 0, c = b + nb * kBlock, x = c + nb * kBlock, y = x + 2 * kBlock, sp = y + 2 * kBlock, st = sp + 3 * kBlock,
                         gates = st + image, sums = gates + 2 * kGates * 4, bars = sums + kSums * 4,
                         bytes = bars + kGradBars * 8 + 16;
};

// TMEM: (C B^T)^T | results of 128 columns in turn | results with three planes, then M^T | M^T dy
constexpr uint32_t kCB = 0, kRes = 128, kPlane = 256, kDv = 448;

// Thread: token (row) 32 q + lane of the warp's quarter q, and its quarter cg of a result's columns.
template <int N>
__global__ void __launch_bounds__(kGradThreads, 1)
ssm_grad_tc_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mY, const __grid_constant__ CUtensorMap mB,
                   const __grid_constant__ CUtensorMap mC, SsmArgs a, TcWork w) {
    using L = GradLay<N>;
    constexpr int NB = L::nb, NV = N * 8 / kGradThreads;  // NV: vectors of eight of a state that a thread converts
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sm = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint32_t* tbase = reinterpret_cast<uint32_t*>(smem + L::bars + kGradBars * 8);
    volatile int* dead = reinterpret_cast<volatile int*>(smem + L::bars + kGradBars * 8 + 4);
    float* sums = reinterpret_cast<float*>(smem + L::sums);
    // by quarter of the rows (colS) or of the columns: [4][128] each
    float *colS = sums, *rowT = sums + 4 * kT, *in1 = sums + 8 * kT, *in2 = sums + 12 * kT, *ddt = sums + 16 * kT, *part = sums + 20 * kT;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), q = warp & 3, cg = warp >> 2;
    const int g = blockIdx.y % a.G, subset = blockIdx.y / a.G, per = a.H / a.G;
    const int h0 = g * per + per * subset / w.subsets, h1 = g * per + per * (subset + 1) / w.subsets;
    Chunk c;
    if (!find_chunk<kT>(a.seqs, blockIdx.x, a.err, c)) {
        const long all = (long)gridDim.x * a.H;
        for (int i = tid; i < h1 - h0; i += kGradThreads) {
            const long at = (long)blockIdx.x * a.H + h0 + i;
            w.sums[at] = w.sums[all + at] = w.sums[2 * all + at] = 0.f;
        }
        dependency_wait();
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kGradBars; ++i) mbar_init(&bars[i], 1);
        *dead = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tbase, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependency_wait();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tbase, 0), lanes = (uint32_t)(q * 32) << 16, on = elect();
    const auto wait = [&](int bar, int index) -> bool {
        bool there = mbar_try_wait(&bars[bar], index & 1, 100000u);
        if (!there) there = wait_slow(&bars[bar], index & 1, dead, a.err);
        return __all_sync(0xffffffffu, there);
    };
    const int slices = a.P / 64, steps = (h1 - h0) * slices, j = q * 32 + lane;
    const auto image = [&](const float* all, int step) {
        return all + (((long)blockIdx.x * a.H + h0) * slices + step) * (long)(N * 64);
    };
    const auto load_xy = [&](int step) {  // one thread
        const int pl = step & 1, col = (h0 + step / slices) * a.P + step % slices * 64;
        mbar_arrive_expect_tx(&bars[LX0 + pl], 2 * kBlock);
        tma_load_2d(smem + L::x + pl * kBlock, &mX, &bars[LX0 + pl], col, c.t0);
        tma_load_2d(smem + L::y + pl * kBlock, &mY, &bars[LX0 + pl], col, c.t0);
    };
    const auto load_image = [&](const float* from) {
        mbar_arrive_expect_tx(&bars[LS], L::image);
        bulk_load(smem + L::st, from, L::image, &bars[LS]);
    };
    const auto gates_of = [&](int h) { return reinterpret_cast<float*>(smem + L::gates) + ((h - h0) & 1) * kGates; };
    const auto ask_gates = [&](int h) {  // asynchronous copies of each thread's own
        if (tid < kGates / 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(gates_of(h) + 4 * tid)),
                         "l"(w.gates + ((long)blockIdx.x * a.H + h) * kGates + 4 * tid)
                         : "memory");
        ring_commit();
    };
    if (warp == 0 && on) {
        mbar_arrive_expect_tx(&bars[LB], 2 * NB * kBlock);
        for (int k = 0; k < NB; ++k) {
            tma_load_2d(smem + L::b + k * kBlock, &mB, &bars[LB], g * N + 64 * k, c.t0);
            tma_load_2d(smem + L::c + k * kBlock, &mC, &bars[LB], g * N + 64 * k, c.t0);
        }
        if (steps > 0) {
            load_xy(0);
            load_image(image(w.dstates, 0));
        }
    }
    int images = steps > 0 ? 1 : 0, tiles = images, seen = 0, mm = 0;  // loads asked for; images waited for; MMAs waited for
    if (steps > 0) ask_gates(h0);
    // rows past the chunk's end, which other sequences may have filled, are zeros in every tile
    const auto zero_rows = [&](uint32_t tile) {
        const uint32_t zero[4] = {0, 0, 0, 0};
        const int r = tid >> 2;
        if (r >= c.len) {
            planes::sts128(at16(tile, r, (tid & 3) * 2), zero);
            planes::sts128(at16(tile, r, (tid & 3) * 2 + 1), zero);
        }
    };
    bool ok = wait(LB, 0);
    if (ok && c.len < kT)
        for (int k = 0; k < 2 * NB; ++k) zero_rows(sm + L::b + k * kBlock);
    fence_async_smem();
    const uint64_t dBk = sdesc_sw128(sm + L::b, 16, 1024), dBm = sdesc_sw128(sm + L::b, kBlock, 1024),
                   dCk = sdesc_sw128(sm + L::c, 16, 1024), dCm = sdesc_sw128(sm + L::c, kBlock, 1024),
                   dSk = sdesc_sw128(sm + L::sp, 16, 1024), dSm = sdesc_sw128(sm + L::sp, kBlock, 1024);
    constexpr uint32_t id128 = idesc_bf16(128, 128, 0, 0), idN = idesc_bf16(128, N, 0, 0), id192 = idesc_bf16(128, 192, 0, 1),
                       id64 = idesc_bf16(128, 64, 0, 1);
    const auto kstep = [](int k) { return (uint64_t)(((k >> 2) * kBlock + (k & 3) * 32) >> 4); };  // of a K-major tile
    bfp::F2 Es[16], dB[16], dC[16];  // pairs of columns
#pragma unroll
    for (int i = 0; i < 16; ++i) Es[i] = dB[i] = dC[i] = bfp::F2(0.f, 0.f);
    bfp::F2 ss2(0.f, 0.f), sd2(0.f, 0.f);

    // dg, da and the sums of a head whose parts are all there, in `from`: one warp, four tokens a lane
    const auto finish_head = [&](int h, const float* from) {
        const float* gt = gates_of(h);
        const float *colS = from, *rowT = from + 4 * kT, *in1 = from + 8 * kT, *in2 = from + 12 * kT, *ddt = from + 16 * kT,
                    *part = from + 20 * kT;
        const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = 4 * lane + e < c.len ? a.a[(long)(c.t0 + 4 * lane + e) * a.H + h] + bias : 0.f;
        const int u = lane >> 3;
        const auto four = [&](const float* from, float (&x)[4]) { load_row<4>(from + 4 * lane, x); };
        float u1[4] = {}, u2[4] = {}, dd[4] = {}, dg[4] = {}, cols[4] = {}, own[3][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float x[5][4];
            four(in1 + k * kT, x[0]);
            four(in2 + k * kT, x[1]);
            four(ddt + k * kT, x[2]);
            four(colS + k * kT, x[3]);
            four(rowT + k * kT, x[4]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u1[e] += x[0][e];
                u2[e] += x[1][e];
                dd[e] += x[2][e];
                if (k == u) dg[e] += x[3][e];
                if (k < u) cols[e] += x[3][e];
#pragma unroll
                for (int run = 0; run < 3; ++run)  // what a row in run `run` or before has in the runs behind it
                    if (run < k && u <= run) own[run][e] += x[4][e];
            }
        }
        float dot = lane < kGradWarps ? part[lane] : 0.f, dD = lane < kGradWarps ? part[kGradWarps + lane] : 0.f;
        // sums over the rows before t of those, and of u2; over the rows from t on of u1
        float pre[4], suf = (u1[0] + u1[1]) + (u1[2] + u1[3]);
#pragma unroll
        for (int k = 0; k < 3; ++k) pre[k] = (own[k][0] + own[k][1]) + (own[k][2] + own[k][3]);
        pre[3] = (u2[0] + u2[1]) + (u2[2] + u2[3]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            float up[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) up[k] = __shfl_up_sync(0xffffffffu, pre[k], d);
            const float down = __shfl_down_sync(0xffffffffu, suf, d);
            dot += __shfl_xor_sync(0xffffffffu, dot, d);
            dD += __shfl_xor_sync(0xffffffffu, dD, d);
            if (lane >= d) {
#pragma unroll
                for (int k = 0; k < 4; ++k) pre[k] += up[k];
            }
            if (lane + d < 32) suf += down;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pre[k] = __shfl_up_sync(0xffffffffu, pre[k], 1);
            if (lane == 0) pre[k] = 0.f;
        }
        suf = __shfl_down_sync(0xffffffffu, suf, 1);
        if (lane == 31) suf = 0.f;
        float run = (cols[0] + cols[1]) + (cols[2] + cols[3]);  // over the columns from t on of t's run
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const float down = __shfl_down_sync(0xffffffffu, run, d, 8);
            if ((lane & 7) + d < 8) run += down;
        }
        run = __shfl_down_sync(0xffffffffu, run, 1, 8);
        if ((lane & 7) == 7) run = 0.f;
        dot *= gt[kRows * kT + 4];
        float before = u == 0 ? pre[0] : (u == 1 ? pre[1] : (u == 2 ? pre[2] : 0.f));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dg[e] += (before + pre[3]) + dot;
            before += u == 0 ? own[0][e] : (u == 1 ? own[1][e] : (u == 2 ? own[2][e] : 0.f));
            pre[3] += u2[e];
        }
        float sA = 0.f, sb = 0.f;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
            suf += u1[e];
            run += cols[e];
            dg[e] += suf + run;
            const int t = 4 * lane + e;
            if (t >= c.len) continue;
            const float da = fmaf(-rate, dg[e], dd[e]) * sigmoidf_(z[e]);
            a.da[(long)(c.t0 + t) * a.H + h] = da;
            sA = fmaf(dg[e], -rate * gt[rDt * kT + t], sA);
            sb += da;
        }
        sA = warp_sum(sA);
        sb = warp_sum(sb);
        if (lane == 0) {
            const long all = (long)gridDim.x * a.H, sh = (long)blockIdx.x * a.H + h;
            w.sums[sh] = sA;
            w.sums[all + sh] = sb;
            w.sums[2 * all + sh] = dD;
        }
    };
    // dx of a step lies in its x's place until the next step, when whole rows are written
    const auto store_dx = [&](int step) {
        __nv_bfloat16* dx = static_cast<__nv_bfloat16*>(a.dx) + ((long)c.t0 * a.H + h0 + step / slices) * a.P + step % slices * 64;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 64 + (tid >> 3), k = tid & 7;
            uint32_t u[4];
            planes::lds128(at16(sm + L::x + (step & 1) * kBlock, r, k), u);
            if (r < c.len) reinterpret_cast<uint4*>(dx + (long)r * a.H * a.P)[k] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    };

    bool failed = __syncthreads_or(!ok);
    if (!failed && warp == 0) {  // (C B^T)^T: row j of B, column i of C
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < N / 16; ++k) mma_ss(on, tm + kCB, dBk + kstep(k), dCk + kstep(k), id128, k > 0);
        commit(on, &bars[MM]);
    }
    if (!failed) failed = __syncthreads_or(!wait(MM, mm++));
    for (int step = 0; step < steps && !failed; ++step) {
        const int h = h0 + step / slices, s = step % slices, place = step & 1;
        const uint32_t xt = sm + L::x + place * kBlock, yt = sm + L::y + place * kBlock;
        const uint64_t dX = sdesc_sw128(xt, 16, 1024), dYk = sdesc_sw128(yt, 16, 1024), dYm = sdesc_sw128(yt, kBlock, 1024);
        const float* gt = gates_of(h);
        // ---- dS into its planes
        asm volatile("cp.async.wait_all;" ::: "memory");
        // a finished head's parts wait in the former dy's place for a warp that has nothing to mask
        float* parts = reinterpret_cast<float*>(smem + L::y + (place ^ 1) * kBlock);
        if (s == 0 && step > 0)
            for (int i = tid; i < kSums; i += kGradThreads) parts[i] = sums[i];
        ok = wait(LX0 + place, step >> 1) && wait(LS, seen++);
        if (ok && c.len < kT) {
            zero_rows(xt);
            zero_rows(yt);
        }
        const auto convert = [&](bool second) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * kGradThreads + tid, n = v >> 3, k = v & 7;
                const uint32_t at = at16(sm + L::sp, n, k);
                uint32_t u[2][4], pl[3][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) planes::lds128(sm + L::st + n * 256 + (((2 * k + e) ^ (n & 7)) << 4), u[e]);
                if (second) {  // dS is the sum of the planes that S0 replaces
#pragma unroll
                    for (int p = 0; p < 3; ++p) planes::lds128(at + p * kBlock, pl[p]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ss2 = bfp::fma2(bfp::F2::of(u[e >> 1][2 * (e & 1)], u[e >> 1][2 * (e & 1) + 1]),
                                        bfp::widen(pl[0][e]) + (bfp::widen(pl[1][e]) + bfp::widen(pl[2][e])), ss2);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bfp::F2 t = bfp::F2::of(u[e >> 1][2 * (e & 1)], u[e >> 1][2 * (e & 1) + 1]);
                    pl[0][e] = bfp::peel(t);
                    pl[1][e] = bfp::peel(t);
                    pl[2][e] = bfp::pack(t);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) planes::sts128(at + p * kBlock, pl[p]);
            }
        };
        convert(false);
        fence_async_smem();
        if ((failed = __syncthreads_or(!ok))) break;
        if (warp == 0) {
            if (on) {
                load_image(image(w.states, step));
            }
            tc_fence_after();
            // X dS: [token, n], the smallest plane first; B dS^T: [token, p] of the three planes
#pragma unroll
            for (int p = 2; p >= 0; --p)
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(on, tm + kRes, dX + 2 * k, dSk + p * (kBlock >> 4) + 2 * k, idN, p < 2 || k > 0);
#pragma unroll
            for (int k = 0; k < N / 16; ++k) mma_ss(on, tm + kPlane, dBk + kstep(k), dSm + k * 128, id192, k > 0);
            commit(on, &bars[MM]);
        }
        ++images;
        if (step > 0) store_dx(step - 1);
        ok = wait(MM, mm++);
        tc_fence_after();
        const float dt = gt[rDt * kT + j], r_end = gt[rToEnd * kT + j];
        {
            const bfp::F2 f(dt * r_end, dt * r_end), re(r_end, r_end);
            bfp::F2 sum(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t hi[8], mid[8], lo[8], x[4];
                tmem_ld8(tm + kPlane + lanes + cg * 16 + 8 * p, hi);
                tmem_ld8(tm + kPlane + lanes + 64 + cg * 16 + 8 * p, mid);
                tmem_ld8(tm + kPlane + lanes + 128 + cg * 16 + 8 * p, lo);
                planes::lds128(at16(xt, j, cg * 2 + p), x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bfp::F2 v = re * (bfp::F2::of(hi[2 * e], hi[2 * e + 1]) + (bfp::F2::of(mid[2 * e], mid[2 * e + 1]) + bfp::F2::of(lo[2 * e], lo[2 * e + 1])));
                    sum = bfp::fma2(v, bfp::widen(x[e]), sum);
                    float v0, v1;
                    v.get(v0, v1);
                    hi[2 * e] = __float_as_uint(v0);
                    hi[2 * e + 1] = __float_as_uint(v1);
                }
                tmem_st8(tm + kDv + lanes + cg * 16 + 8 * p, hi);  // M^T dy is added to it there
            }
            float q2, odd;
            sum.get(q2, odd);
            q2 += odd;
            if (cg * 32 < N) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t r[8];
                    tmem_ld8(tm + kRes + lanes + cg * 32 + 8 * p, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e) dB[4 * p + e] = bfp::fma2(f, bfp::F2::of(r[2 * e], r[2 * e + 1]), dB[4 * p + e]);
                }
            }
            float* to = in2 + cg * kT + j;
            *to = (s ? *to : 0.f) + dt * q2;
            tmem_wait_st();
        }
        tc_fence_before();
        if ((failed = __syncthreads_or(!ok))) break;
        if (warp == 0) {  // x_j . dy_i
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(on, tm + kRes, dX + 2 * k, dYk + 2 * k, id128, k > 0);
            commit(on, &bars[MM]);
        }
        // ---- S0 into the planes' place
        ok = wait(LS, seen++);
        convert(true);
        fence_async_smem();
        ok = wait(MM, mm++) && ok;
        tc_fence_after();
        // ---- E, T and M^T of this thread's row and run of columns
        {
            const int u = cg;
            float acc = 0.f;
            if (u < q) {
                const uint32_t zero[8] = {};
#pragma unroll
                for (int p = 0; p < 6; ++p) tmem_st8(tm + kPlane + lanes + 48 * u + 8 * p, zero);
                if (s == 0 && step > 0 && warp == 3) finish_head(h - 1, parts);
            } else {
                float f = gt[rToRun * kT + j];
                for (int v = q + 1; v < u; ++v) f *= gt[kRows * kT + v];
                const float ph = gt[rPh * kT + j], pl = gt[rPl * kT + j];
                const bfp::F2 f2(f, f), dt2(dt, dt);
                // eight columns at a time, from the last; the run on the diagonal keeps its upper triangle
                const auto columns = [&](auto diagonal) {
                    constexpr bool kDiagonal = decltype(diagonal)::value;
#pragma unroll
                    for (int p = 3; p >= 0; --p) {
                        uint32_t re[8], rc[8], hi[4], mid[4], lo[4];
                        tmem_ld8(tm + kRes + lanes + 32 * u + 8 * p, re);
                        tmem_ld8(tm + kCB + lanes + 32 * u + 8 * p, rc);
                        bfp::F2 d[4];
                        float x[8], y[8];
                        if constexpr (kDiagonal) {
                            load_row<8>(gt + rPh * kT + 32 * u + 8 * p, x);
                            load_row<8>(gt + rPl * kT + 32 * u + 8 * p, y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = exp2_hw((x[e] - ph) + (y[e] - pl));
#pragma unroll
                            for (int e = 0; e < 4; ++e) d[e] = bfp::F2(x[2 * e], x[2 * e + 1]);
                        } else {
                            load_row<8>(gt + rFromRun * kT + 32 * u + 8 * p, x);
#pragma unroll
                            for (int e = 0; e < 4; ++e) d[e] = bfp::F2(x[2 * e], x[2 * e + 1]) * f2;
                        }
                        tmem_wait_ld();
                        float t[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bfp::F2 cb = bfp::F2::of(rc[2 * e], rc[2 * e + 1]);
                            bfp::F2 E = d[e] * dt2 * bfp::F2::of(re[2 * e], re[2 * e + 1]), M = d[e] * cb;
                            if constexpr (kDiagonal) {
                                float v0, v1;
                                E.get(v0, v1);
                                E = bfp::F2(8 * p + 2 * e >= lane ? v0 : 0.f, 8 * p + 2 * e + 1 >= lane ? v1 : 0.f);
                                M.get(v0, v1);
                                M = bfp::F2(8 * p + 2 * e >= lane ? v0 : 0.f, 8 * p + 2 * e + 1 >= lane ? v1 : 0.f);
                            }
                            Es[4 * p + e] = Es[4 * p + e] + E;
                            (E * cb).get(t[2 * e], t[2 * e + 1]);
                            hi[e] = bfp::peel(M);
                            mid[e] = bfp::peel(M);
                            lo[e] = bfp::pack(M);
                        }
                        const uint32_t at = tm + kPlane + lanes + 24 * (2 * u + (p >> 1)) + 4 * (p & 1);
                        tmem_st4(at, hi);
                        tmem_st4(at + 8, mid);
                        tmem_st4(at + 16, lo);
#pragma unroll
                        for (int e = 7; e >= 0; --e) {
                            if constexpr (kDiagonal) {  // sum over i >= t of row j < t
                                const bool below = 8 * p + e > lane;
                                acc += below ? t[e] : 0.f;
                                t[e] = below ? acc : 0.f;
                            } else {  // all rows lie before t: the sums over i >= t are taken of the columns' sums
                                acc += t[e];
                            }
                        }
                        const float col = sum_rows<8, 32>(t, lane);
                        if (lane < 8) {
                            float* to = colS + q * kT + 32 * u + 8 * p + lane;
                            *to = (s ? *to : 0.f) + col;
                        }
                    }
                };
                if (u == q) columns(std::true_type{});
                else columns(std::false_type{});
            }
            float* to = rowT + u * kT + j;
            *to = (s ? *to : 0.f) + acc;
            tmem_wait_st();
        }
        fence_async_smem();  // the finished head's parts have been read: the next dy may come
        tc_fence_before();
        if ((failed = __syncthreads_or(!ok))) break;
        if (warp == 0) {
            if (on && step + 1 < steps) {
                load_image(image(w.dstates, step + 1));
                load_xy(step + 1);
            }
            tc_fence_after();
            // M^T dy, and dy S0
#pragma unroll
            for (int p = 2; p >= 0; --p)
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ts(on, tm + kDv, tm + kPlane + 24 * k + 8 * p, dYm + k * 128, id64, 1);
#pragma unroll
            for (int p = 2; p >= 0; --p)
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ss(on, tm + kRes, dYk + 2 * k, dSk + p * (kBlock >> 4) + 2 * k, idN, p < 2 || k > 0);
            commit(on, &bars[MM]);
        }
        if (step + 1 < steps) {
            ++images;
            ++tiles;
            if (s == slices - 1) ask_gates(h + 1);
        }
        ok = wait(MM, mm++);
        tc_fence_after();
        {
            const float D = a.D ? a.D[h] : 0.f, b = gt[rFromStart * kT + j];
            const bfp::F2 dt2(dt, dt), D2(D, D), b2(b, b);
            bfp::F2 qd2(0.f, 0.f), q12(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t r[8], x[4], y[4];
                tmem_ld8(tm + kDv + lanes + cg * 16 + 8 * p, r);
                planes::lds128(at16(xt, j, cg * 2 + p), x);
                planes::lds128(at16(yt, j, cg * 2 + p), y);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bfp::F2 v = bfp::F2::of(r[2 * e], r[2 * e + 1]), xe = bfp::widen(x[e]), ye = bfp::widen(y[e]);
                    qd2 = bfp::fma2(v, xe, qd2);
                    sd2 = bfp::fma2(ye, xe, sd2);
                    x[e] = bfp::pack(bfp::fma2(dt2, v, D2 * ye));
                }
                planes::sts128(at16(xt, j, cg * 2 + p), x);  // dx takes x's place
            }
            if (cg * 32 < N) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t r[8], x[4];
                    tmem_ld8(tm + kRes + lanes + cg * 32 + 8 * p, r);
                    planes::lds128(at16(sm + L::c + (cg >> 1) * kBlock, j, (cg & 1) * 4 + p), x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bfp::F2 v = b2 * bfp::F2::of(r[2 * e], r[2 * e + 1]);
                        q12 = bfp::fma2(v, bfp::widen(x[e]), q12);
                        dC[4 * p + e] = dC[4 * p + e] + v;
                    }
                }
            }
            float qd, q1, odd;
            qd2.get(qd, odd);
            qd += odd;
            q12.get(q1, odd);
            q1 += odd;
            float* to = in1 + cg * kT + j;
            *to = (s ? *to : 0.f) + q1;
            to = ddt + cg * kT + j;
            *to = (s ? *to : 0.f) + qd;
            if (s == slices - 1) {
                float x0, x1, y0, y1;
                ss2.get(x0, x1);
                sd2.get(y0, y1);
                x0 = warp_sum(x0 + x1);
                y0 = warp_sum(y0 + y1);
                if (lane == 0) {
                    part[warp] = x0;
                    part[kGradWarps + warp] = y0;
                }
                ss2 = sd2 = bfp::F2(0.f, 0.f);
            }
        }
        tc_fence_before();
        failed = __syncthreads_or(!ok);
    }
    if (!failed && warp == 3) finish_head(h1 - 1, sums);
    if (!failed) {
        store_dx(steps - 1);
        // dB += E^T C, dC += E B with the heads' sum of E in three planes, the last in dy's place: rows j, columns i.  (With
        // two, 2^-17, ten times as many of the bf16 outputs lie beside the nearest value: 0.17% for 0.02%.)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[e] = bfp::peel(Es[4 * p + e]);
                mid[e] = bfp::peel(Es[4 * p + e]);
                lo[e] = bfp::pack(Es[4 * p + e]);
            }
            const uint32_t tile = sm + L::sp + (cg >> 1) * kBlock;
            planes::sts128(at16(tile, j, (cg & 1) * 4 + p), hi);
            planes::sts128(at16(tile + 2 * kBlock, j, (cg & 1) * 4 + p), mid);
            planes::sts128(at16(sm + L::y + (cg >> 1) * kBlock, j, (cg & 1) * 4 + p), lo);
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            constexpr uint32_t idB = idesc_bf16(128, N, 0, 1), idC = idesc_bf16(128, N, 1, 1);
#pragma unroll
            for (int p = 2; p >= 0; --p) {
                const uint32_t tile = sm + (p == 2 ? L::y : L::sp + 2 * p * kBlock);
                const uint64_t dEk = sdesc_sw128(tile, 16, 1024), dEm = sdesc_sw128(tile, kBlock, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    mma_ss(on, tm + kRes, dEk + kstep(k), dCm + k * 128, idB, p < 2 || k > 0);
                    mma_ss(on, tm + kPlane, dEm + k * 128, dBm + k * 128, idC, p < 2 || k > 0);
                }
            }
            commit(on, &bars[MM]);
        }
        ok = wait(MM, mm++);
        failed = __syncthreads_or(!ok);
        tc_fence_after();
        if (!failed && cg * 32 < N) {
            const long at = ((long)(c.t0 + j) * a.G + g) * N + cg * 32, all = (long)a.seqs.total_T * a.G * N;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t rb[8], rc[8];
                tmem_ld8(tm + kRes + lanes + cg * 32 + 8 * p, rb);
                tmem_ld8(tm + kPlane + lanes + cg * 32 + 8 * p, rc);
                tmem_wait_ld();
                float vb[8], vc[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    (dB[4 * p + e] + bfp::F2::of(rb[2 * e], rb[2 * e + 1])).get(vb[2 * e], vb[2 * e + 1]);
                    (dC[4 * p + e] + bfp::F2::of(rc[2 * e], rc[2 * e + 1])).get(vc[2 * e], vc[2 * e + 1]);
                }
                if (j >= c.len) continue;
                if (w.subsets > 1) {
                    store_row<8>(w.parts + subset * all + at + 8 * p, vb);
                    store_row<8>(w.parts + (w.subsets + subset) * all + at + 8 * p, vc);
                } else {
                    store_row<8>(static_cast<__nv_bfloat16*>(a.dB) + at + 8 * p, vb);
                    store_row<8>(static_cast<__nv_bfloat16*>(a.dC) + at + 8 * p, vc);
                }
            }
        }
    }
    // loads and MMAs in flight, after a wait that ran out, end before the block leaves
    if (failed && warp == 0 && on) {
        mbar_wait(&bars[LB], 0, kLimit);
        for (int k = max(0, tiles - 2); k < tiles; ++k) mbar_wait(&bars[LX0 + (k & 1)], (k >> 1) & 1, kLimit);
        if (images > 0) mbar_wait(&bars[LS], (images - 1) & 1, kLimit);
        mbar_wait(&bars[MM], (mm - 1) & 1, kLimit);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// Subsets of a group's heads: more blocks fill more SMs, but each loads B and C, ends with two products of its own, and
// writes dB and dC in fp32 for another kernel to add.  Counted in steps of a head.  In us, for 1, 2, 4 and 8 subsets and
// the choice made here: 8192 tokens of 32 heads in two groups 233, 262, 302, 348, 233; 2048 of 32 in one 341, 197, 126,
// 94, 94; 1024 of 16 180, 111, 74, 56, 50; 4096 of 64 684, 387, 237, 260, 237.
int subsets_of(int num_seqs, int total_T, int H, int G, int N) {
    const long blocks = slots128(num_seqs, total_T) * G, per = H / G;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= per && s <= 16; ++s) {
        const double rounds = (double)((blocks * s + kSMs - 1) / kSMs), heads = (double)((per + s - 1) / s) + 0.7;
        const double parts = s > 1 ? 0.8 + (2.0 * s + 1) * 2 * total_T * G * N * 4 / 5e12 / 5e-6 : 0.0;
        if (rounds * heads + parts < least) {
            least = rounds * heads + parts;
            best = s;
        }
    }
    return best;
}

size_t layout(int num_seqs, int total_T, int H, int G, int P, int N, bool varied, TcWork* w, unsigned char* at) {
    const size_t slots = (size_t)slots128(num_seqs, total_T);
    const size_t gates = up256(slots * H * kGates * sizeof(float)), states = slots * H * P * N * sizeof(float),
                 sums = up256(slots * H * 3 * sizeof(float));
    const int subsets = subsets_of(num_seqs, total_T, H, G, N);
    const size_t parts = subsets > 1 ? (size_t)subsets * 2 * total_T * G * N * sizeof(float) : 0;
    if (w) {
        w->gates = reinterpret_cast<float*>(at);
        w->states = reinterpret_cast<float*>(at + gates);
        w->dstates = reinterpret_cast<float*>(at + gates + states);
        w->sums = reinterpret_cast<float*>(at + gates + 2 * states);
        w->parts = reinterpret_cast<float*>(at + gates + 2 * states + sums);
        w->subsets = subsets;
    }
    const size_t used = gates + 2 * states + sums + up256(parts);
    return used + segments128(num_seqs, total_T, H, P, N, 2, varied, w ? &w->g : nullptr, w ? at + used : nullptr);
}

template <int N>
cudaError_t launch(const SsmArgs& a, const TcWork& w, cudaStream_t s) {
    CUtensorMap mX, mY, mB, mC;
    const long T = a.seqs.total_T;
    if (!map_rows(&mX, a.x, T, (long)a.H * a.P, a.x_stride) || !map_rows(&mY, a.dout, T, (long)a.H * a.P, (long)a.H * a.P) ||
        !map_rows(&mB, a.B, T, (long)a.G * N, a.B_stride) || !map_rows(&mC, a.C, T, (long)a.G * N, a.C_stride))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(ssm_grad_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, GradLay<N>::bytes);
    if (e == cudaSuccess) e = launch_gates128(a, w.gates, s);
    if (e == cudaSuccess && w.g.each) e = launch_starts(a, w.gates, w.g, 2, s);
    if (e == cudaSuccess) e = launch_states(a, w.gates, w.g, w.states, w.dstates, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)slots128(a.seqs.num_seqs, a.seqs.total_T), (unsigned)(a.G * w.subsets));
    return launch_after(ssm_grad_tc_kernel<N>, grid, kGradThreads, GradLay<N>::bytes, s, mX, mY, mB, mC, a, w);
}

}  // namespace

size_t tc_bwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N) {
    const size_t equal = layout(num_seqs, total_T, H, G, P, N, false, nullptr, nullptr),
                 varied = layout(num_seqs, total_T, H, G, P, N, true, nullptr, nullptr);
    return equal > varied ? equal : varied;
}

cudaError_t launch_tc_bwd(const SsmArgs& a, cudaStream_t s) {
    TcWork w{};
    layout(a.seqs.num_seqs, a.seqs.total_T, a.H, a.G, a.P, a.N, a.seqs.cu && a.seqs.num_seqs > 1, &w, static_cast<unsigned char*>(a.workspace));
    const cudaError_t e = a.N == 128 ? launch<128>(a, w, s) : launch<64>(a, w, s);
    if (e != cudaSuccess) return e;
    Work f{};
    f.sums = w.sums;
    f.parts = w.parts;
    f.subsets = w.subsets;
    return launch_finish(a, f, slots128(a.seqs.num_seqs, a.seqs.total_T), s);
}

}  // namespace ssm
}  // namespace gdn

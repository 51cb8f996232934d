// ssm_bwd.cu -- the gradients of the selective state space scan.
//
// Inside a chunk, with v = dt x, b_i = e^{G_i}, r_j = e^{G_last - G_j}, S_0 the state at its start and dS_1 the
// gradient of the state at its end, and for j <= i
//   M_ij = e^{G_i - G_j} C_i . B_j,   E_ij = e^{G_i - G_j} dy_i . v_j,   T_ij = M_ij dy_i . v_j:
//   dv_j = sum_i M_ij dy_i + r_j dS_1 B_j,
//   dC_i = sum_j E_ij B_j + b_i S_0^T dy_i,        dB_j = sum_i E_ij C_i + r_j dS_1^T v_j,
//   dS_0 = b_last dS_1 + sum_i b_i dy_i C_i^T,
//   dG_i = sum_{j < i} T_ij - sum_{m > i} T_mi + b_i dy_i . S_0 C_i - r_i v_i . dS_1 B_i,
//   dg_t = sum_{i >= t} dG_i + b_last <dS_1, S_0> + sum_j r_j v_j . dS_1 B_j
// (the diagonal of T leaves dG; T's sums over rows and over columns are held in two floats up to dg, where what lies
// behind t cancels: in fp32 dA_log of 8192 tokens was 3e-6 off), and with z = a + dt_bias, rate = exp(A_log):
//   ddt = dv . x - rate dg,  da = ddt sigmoid(z),  dx = dt dv + D dy,
//   dA_log = sum dg g,  ddt_bias = sum da,  dD = sum dy . x.
// The states and their gradients come from the scan kernels of the forward pass, run in both directions.  The
// gradient kernel's block takes one chunk and a subset of the heads of one group, so that C B^T is formed once and
// dB, dC of the group's heads are summed before they are written.  This is the fp32 form (bf16: ssm_tc_bwd.cu), on three
// planes a factor; a head's step is a chain of seven products with barriers between them, and its latency bounds short
// batches (493 tokens of six heads: 36 us), the tensor instructions and the splits long ones
// (6144 tokens of 24 heads, d_state 128, in three sequences: 485 us).
#include "ssm_chunk.cuh"

namespace gdn {
namespace ssm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// 16 warps: warp w holds rows 16 (w % 4) .. and a quarter of the columns.
template <int N>
struct Smem {
    static constexpr int k = 0, c = k + bfp::kTileBytes<kC, N, 3>, x = c + bfp::kTileBytes<kC, N, 3>,
                         y = x + bfp::kTileBytes<kC, 64, 3>, s = y + bfp::kTileBytes<kC, 64, 3>,
                         m = s + bfp::kTileBytes<64, N, 3>, bytes = m + bfp::kTileBytes<kC, 64, 3>;
};

// Sums over the four lanes that share a row of an accumulator.
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int N>
__global__ void __launch_bounds__(kThreads) ssm_grad_kernel(SsmArgs a, Work w) {
    using L = Smem<N>;
    constexpr int NT = N / 32;  // NT: 8-column tiles of a warp in a 64 x N result
    constexpr int KV = kC * N / 8 / kThreads;  // vectors of a 64 x N tile a thread loads
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const bfp::Tile<kC, N, 3> Kt{base + L::k}, Ct{base + L::c};
    const bfp::Tile<kC, 64, 3> Xt{base + L::x}, Yt{base + L::y};
    const bfp::Tile<64, N, 3> St{base + L::s};
    const bfp::Tile<kC, 64, 3> Mt{base + L::m};
    __shared__ float gate[kGateRows][kC];
    __shared__ Two rowT[4][kC], colT[4][kC];
    __shared__ float in1[4][kC], in2[4][kC], ddt4[4][kC];  // by column (row) of warps
    __shared__ float part[2][kWarps];  // <dS, S0>, dD
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.y % a.G, subset = blockIdx.y / a.G, per = a.H / a.G;
    const int lo = per * subset / w.subsets, hi = per * (subset + 1) / w.subsets;
    Chunk c;
    const bool found = find_chunk(a.seqs, blockIdx.x, a.err, c);
    dependency_wait();
    if (!found) {
        const long all = (long)gridDim.x * a.H;
        for (int i = tid; i < hi - lo; i += kThreads) {
            const long at = (long)blockIdx.x * a.H + g * per + lo + i;
            w.sums[at] = w.sums[all + at] = w.sums[2 * all + at] = 0.f;
        }
        return;
    }
    const int m = (warp & 3) * 16, cw = warp >> 2, n0 = cw * (N / 4), p0 = cw * 16;
    {
        const float* B = static_cast<const float*>(a.B) + (long)c.t0 * a.B_stride + (long)g * N;
        const float* C = static_cast<const float*>(a.C) + (long)c.t0 * a.C_stride + (long)g * N;
#pragma unroll
        for (int i = 0; i < KV; ++i) {
            const int v = i * kThreads + tid, r = v / (N / 8), col = v % (N / 8) * 8;
            bfp::Raw8 k, q;
            k.load(B + (long)r * a.B_stride + col, r < c.len);
            q.load(C + (long)r * a.C_stride + col, r < c.len);
            k.put(Kt, r, col);
            q.put(Ct, r, col);
        }
    }
    __syncthreads();
    float CK[2][4], Es[2][4], dB[NT][4], dC[NT][4];
    bfp::clear(CK);
    bfp::clear(Es);
    bfp::clear(dB);
    bfp::clear(dC);
    bfp::product<N, false, false>(CK, Ct, m, Kt, p0, lane);
    const int slices = a.P / 64;
    for (int h = g * per + lo; h < g * per + hi; ++h) {
        const long sh = (long)blockIdx.x * a.H + h;
        const float D = a.D ? a.D[h] : 0.f;
        float E[2][4];
        bfp::clear(E);
        float ss = 0.f, sd = 0.f;
        for (int s = 0; s < slices; ++s) {
            __syncthreads();  // what was in the tiles and sums has been read
            if (s == 0) {
                for (int i = tid; i < kGateRows * kC; i += kThreads)
                    (&gate[0][0])[i] = w.gates[sh * (kGateRows * kC) + i];
            }
            {
                const int r = tid / 8, col = tid % 8 * 8;
                const long ch = (long)h * a.P + s * 64 + col;
                bfp::Raw8 x, y;
                x.load(static_cast<const float*>(a.x) + (long)(c.t0 + r) * a.x_stride + ch, r < c.len);
                y.load(static_cast<const float*>(a.dout) + (long)(c.t0 + r) * a.H * a.P + ch, r < c.len);
                x.put(Xt, r, col);
                y.put(Yt, r, col);
            }
            const float* S0 = w.states + (sh * a.P + s * 64) * N;
            const float* S1 = w.dstates + (sh * a.P + s * 64) * N;
#pragma unroll
            for (int i = 0; i < KV; ++i) {
                const int v = i * kThreads + tid, r = v / (N / 8), col = v % (N / 8) * 8;
                float x[8], z[8];
                load_row<8>(S1 + (long)r * N + col, x);
                load_row<8>(S0 + (long)r * N + col, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], z[e], ss);
                bfp::put8(St, r, col, x);
            }
            __syncthreads();
            if (s == 0) {
                bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int t) {
                    float v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float d = (gate[1][i] - gate[1][t + e]) + (gate[2][i] - gate[2][t + e]);
                        v[e] = t + e <= i ? CK[j][2 * hh + e] * expf(d) : 0.f;
                    }
                    bfp::put2(Mt, i, t, v[0], v[1]);
                });
            }
            bfp::product<64, false, false>(E, Yt, m, Xt, p0, lane);
            // dB: rows r_j dt_j times x dS
            {
                float acc[NT][4];
                bfp::clear(acc);
                bfp::product<64, false, true>(acc, Xt, m, St, n0, lane);
                bfp::pairs<NT>(m, n0, lane, [&](int j, int hh, int i, int) {
                    const float f = gate[0][i] * gate[4][i];
                    dB[j][2 * hh] = fmaf(f, acc[j][2 * hh], dB[j][2 * hh]);
                    dB[j][2 * hh + 1] = fmaf(f, acc[j][2 * hh + 1], dB[j][2 * hh + 1]);
                });
            }
            __syncthreads();  // M is in place
            // dv: B dS^T and M^T dy
            {
                float acc[2][4], q2[2] = {0.f, 0.f}, qd[2] = {0.f, 0.f};
                bfp::clear(acc);
                bfp::product<N, false, false>(acc, Kt, m, St, p0, lane);
                bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int p) {
                    const float2 x = bfp::get2(Xt, i, p);
                    acc[j][2 * hh] *= gate[4][i];
                    acc[j][2 * hh + 1] *= gate[4][i];
                    q2[hh] = fmaf(acc[j][2 * hh], x.x, fmaf(acc[j][2 * hh + 1], x.y, q2[hh]));
                });
                bfp::product<kC, true, true, bfp::kUpper>(acc, Mt, m, Yt, p0, lane);
                float* dx = static_cast<float*>(a.dx) + ((long)c.t0 * a.H + h) * a.P + s * 64;
                bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int p) {
                    const float2 x = bfp::get2(Xt, i, p), y = bfp::get2(Yt, i, p);
                    const float v0 = acc[j][2 * hh], v1 = acc[j][2 * hh + 1];
                    qd[hh] = fmaf(v0, x.x, fmaf(v1, x.y, qd[hh]));
                    sd = fmaf(y.x, x.x, fmaf(y.y, x.y, sd));
                    const float o0 = fmaf(gate[0][i], v0, D * y.x), o1 = fmaf(gate[0][i], v1, D * y.y);
                    if (i < c.len) *reinterpret_cast<float2*>(dx + (long)i * a.H * a.P + p) = make_float2(o0, o1);
                });
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float u = quad_sum(q2[hh]), v = quad_sum(qd[hh]);
                    const int i = m + (lane >> 2) + 8 * hh;
                    if ((lane & 3) == 0) {  // one warp a row and quarter: plain read and write
                        in2[cw][i] = (s ? in2[cw][i] : 0.f) + gate[0][i] * u;
                        ddt4[cw][i] = (s ? ddt4[cw][i] : 0.f) + v;
                    }
                }
            }
            __syncthreads();  // dS has been read: S0 takes its place
#pragma unroll
            for (int i = 0; i < KV; ++i) {
                const int v = i * kThreads + tid, r = v / (N / 8), col = v % (N / 8) * 8;
                float z[8];
                load_row<8>(S0 + (long)r * N + col, z);
                bfp::put8(St, r, col, z);
            }
            __syncthreads();
            {
                float acc[NT][4], q1[2] = {0.f, 0.f};
                bfp::clear(acc);
                bfp::product<64, false, true>(acc, Yt, m, St, n0, lane);
                bfp::pairs<NT>(m, n0, lane, [&](int j, int hh, int i, int n) {
                    const float2 q = bfp::get2(Ct, i, n);
                    const float u = gate[3][i] * acc[j][2 * hh], v = gate[3][i] * acc[j][2 * hh + 1];
                    q1[hh] = fmaf(u, q.x, fmaf(v, q.y, q1[hh]));
                    dC[j][2 * hh] += u;
                    dC[j][2 * hh + 1] += v;
                });
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float u = quad_sum(q1[hh]);
                    const int i = m + (lane >> 2) + 8 * hh;
                    if ((lane & 3) == 0) in1[cw][i] = (s ? in1[cw][i] : 0.f) + u;
                }
            }
        }
        // E, T and the sums of T's rows and columns below the diagonal
        {
            Two rows[2] = {}, cols[2][2] = {};
            bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int t) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float d = (gate[1][i] - gate[1][t + e]) + (gate[2][i] - gate[2][t + e]);
                    const float v = t + e <= i ? E[j][2 * hh + e] * (gate[0][t + e] * expf(d)) : 0.f;
                    Es[j][2 * hh + e] += v;
                    const float q = t + e < i ? v * CK[j][2 * hh + e] : 0.f;
                    two_add(rows[hh], q);
                    two_add(cols[j][e], q);
                }
            });
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                Two u = two_add(rows[hh], two_shfl(rows[hh], 1));
                u = two_add(u, two_shfl(u, 2));
                if ((lane & 3) == 0) rowT[cw][m + (lane >> 2) + 8 * hh] = u;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    Two u = cols[j][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) u = two_add(u, two_shfl(u, o));
                    if (lane < 4) colT[warp & 3][p0 + 8 * j + 2 * lane + e] = u;
                }
            ss = warp_sum(ss);
            sd = warp_sum(sd);
            if (lane == 0) {
                part[0][warp] = ss;
                part[1][warp] = sd;
            }
        }
        __syncthreads();
        // warp 0: the chunk's tokens, two a lane
        if (warp == 0) {
            float dot = lane < kWarps ? part[0][lane] : 0.f, dD = lane < kWarps ? part[1][lane] : 0.f;
            dot = warp_sum(dot) * gate[3][kC - 1];
            dD = warp_sum(dD);
            Two own[2];
            float ddt[2], tot2 = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                Two d{0.f, 0.f};
                float u1 = 0.f, u2 = 0.f;
                ddt[e] = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    d = two_add(d, two_add(rowT[x][i], Two{-colT[x][i].h, -colT[x][i].l}));
                    u1 += in1[x][i];
                    u2 += in2[x][i];
                    ddt[e] += ddt4[x][i];
                }
                two_add(d, u1);
                two_add(d, -u2);
                own[e] = d;
                tot2 += u2;
            }
            dot += warp_sum(tot2);
            Two suf = two_add(own[0], own[1]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const Two down{__shfl_down_sync(0xffffffffu, suf.h, o), __shfl_down_sync(0xffffffffu, suf.l, o)};
                if (lane + o < 32) suf = two_add(suf, down);
            }
            Two behind{__shfl_down_sync(0xffffffffu, suf.h, 1), __shfl_down_sync(0xffffffffu, suf.l, 1)};
            if (lane == 31) behind = Two{0.f, 0.f};
            behind = two_add(behind, own[1]);
            const float dg[2] = {(suf.h + dot) + suf.l, (behind.h + dot) + behind.l};
            const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
            float sA = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                if (i >= c.len) continue;
                const long at = (long)(c.t0 + i) * a.H + h;
                const float gi = -rate * gate[0][i];
                const float da = fmaf(-rate, dg[e], ddt[e]) * sigmoidf_(a.a[at] + bias);
                a.da[at] = da;
                sA = fmaf(dg[e], gi, sA);
                sb += da;
            }
            sA = warp_sum(sA);
            sb = warp_sum(sb);
            if (lane == 0) {
                const long all = (long)gridDim.x * a.H;
                w.sums[sh] = sA;
                w.sums[all + sh] = sb;
                w.sums[2 * all + sh] = dD;
            }
        }
    }
    __syncthreads();
    bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int t) { bfp::put2(Mt, i, t, Es[j][2 * hh], Es[j][2 * hh + 1]); });
    __syncthreads();
    bfp::product<kC, false, true, bfp::kLower>(dC, Mt, m, Kt, n0, lane);
    bfp::product<kC, true, true, bfp::kUpper>(dB, Mt, m, Ct, n0, lane);
    bfp::pairs<NT>(m, n0, lane, [&](int j, int hh, int i, int n) {
        if (i >= c.len) return;
        const long at = ((long)(c.t0 + i) * a.G + g) * N + n;
        const float2 vb = make_float2(dB[j][2 * hh], dB[j][2 * hh + 1]), vc = make_float2(dC[j][2 * hh], dC[j][2 * hh + 1]);
        if (w.subsets > 1) {
            const long all = (long)a.seqs.total_T * a.G * N;
            *reinterpret_cast<float2*>(w.parts + subset * all + at) = vb;
            *reinterpret_cast<float2*>(w.parts + (w.subsets + subset) * all + at) = vc;
        } else {
            *reinterpret_cast<float2*>(static_cast<float*>(a.dB) + at) = vb;
            *reinterpret_cast<float2*>(static_cast<float*>(a.dC) + at) = vc;
        }
    });
}

// What is left, in one launch of three kinds of blocks: the sums over the slots of dA_log, ddt_bias and dD, 32 heads a
// block; the subsets' dB and dC added up in order, eight elements a thread; zeros for the tokens outside every sequence.
constexpr int kZeroBlocks = kSMs;
template <typename T>
__global__ void __launch_bounds__(256) ssm_finish_kernel(SsmArgs a, Work w, long slots, int sum_blocks, int part_blocks) {
    dependency_wait();
    const int per = (a.H + 31) / 32;
    if ((int)blockIdx.x < sum_blocks) {
        __shared__ Two part[8][32];
        const int which = blockIdx.x / per, lane = threadIdx.x & 31, h = blockIdx.x % per * 32 + lane, k = threadIdx.x >> 5;
        float* out = which == 0 ? a.dA_log : (which == 1 ? a.ddt_bias : a.dD);
        if (!out) return;
        const float* t = w.sums + (long)which * slots * a.H;
        Two sum{0.f, 0.f};
        if (h < a.H) {
            long r = k;
            for (; r + 24 < slots; r += 32) {
                const float x[4] = {t[r * a.H + h], t[(r + 8) * a.H + h], t[(r + 16) * a.H + h], t[(r + 24) * a.H + h]};
#pragma unroll
                for (int i = 0; i < 4; ++i) two_add(sum, x[i]);
            }
            for (; r < slots; r += 8) two_add(sum, t[r * a.H + h]);
        }
        part[k][lane] = sum;
        __syncthreads();
        if (k == 0 && h < a.H) {
            for (int i = 1; i < 8; ++i) sum = two_add(sum, part[i][lane]);
            out[h] = sum.h + sum.l;
        }
        return;
    }
    if (packed_find(a.seqs, 0, 1, 0, a.err) == -2) return;
    const long first = a.seqs.cu ? a.seqs.bos(0) : 0, end = a.seqs.cu ? a.seqs.bos(a.seqs.num_seqs) : a.seqs.total_T;
    const int b = blockIdx.x - sum_blocks;
    const long elems = (long)a.seqs.total_T * a.G * a.N;
    if (b < part_blocks) {
        const bool second = 2 * b >= part_blocks;
        const long at = ((long)(b - (second ? part_blocks / 2 : 0)) * 256 + threadIdx.x) * 8, t = at / ((long)a.G * a.N);
        if (at >= elems || t < first || t >= end) return;
        const float* p = w.parts + (second ? w.subsets * elems : 0) + at;
        float x[8] = {};
        for (int s = 0; s < w.subsets; ++s) {
            float y[8];
            load_row<8>(p + s * elems, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += y[e];
        }
        store_row<8>(static_cast<T*>(second ? a.dC : a.dB) + at, x);
        return;
    }
    // few rows as a rule, walked by all threads
    const float zero[8] = {};
    const long rows = first + (a.seqs.total_T - end), stride = (long)kZeroBlocks * 256;
    const long q0 = (long)(b - part_blocks) * 256 + threadIdx.x;
    const auto clear = [&](void* out, long width) {
        for (long q = q0; q < rows * width; q += stride) {
            const long r = q / width, t = r < first ? r : end + (r - first);
            store_row<8>(static_cast<T*>(out) + (t * width + q % width) * 8, zero);
        }
    };
    clear(a.dx, (long)a.H * a.P / 8);
    clear(a.dB, (long)a.G * a.N / 8);
    clear(a.dC, (long)a.G * a.N / 8);
    for (long q = q0; q < rows * a.H; q += stride) {
        const long r = q / a.H, t = r < first ? r : end + (r - first);
        a.da[t * a.H + q % a.H] = 0.f;
    }
}

template <int N>
cudaError_t grad_one(const SsmArgs& a, const Work& w, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(ssm_grad_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<N>::bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)slots_of(a.seqs.num_seqs, a.seqs.total_T), (unsigned)(a.G * w.subsets));
    return launch_after(ssm_grad_kernel<N>, grid, kThreads, Smem<N>::bytes, s, a, w);
}

// Subsets of a group's heads: blocks for two rounds, at least two heads a block unless that leaves SMs without one (each
// subset writes its dB and dC in fp32 for another kernel to add).  For one, two, three rounds: 2048 tokens of 16 heads
// 202, 155, 155 us; 6144 of 24 in three sequences 583, 485, 509.  One head a block against all three, 493 tokens of six
// heads in two groups: 36 us for 59; one against two, 23 tokens of 15 in three: 36 for 68.
int subsets_of(int num_seqs, int total_T, int H, int G) {
    const long blocks = slots_of(num_seqs, total_T) * G, per = H / G;
    long n = (2 * kSMs + blocks - 1) / blocks;
    const long most = per == 1 || blocks * per <= kSMs ? per : per / 2;
    n = n > most ? most : n;
    return (int)(n < 1 ? 1 : n);
}

size_t layout(int num_seqs, int total_T, int H, int G, int P, int N, bool varied, Work* w, unsigned char* at) {
    const size_t slots = (size_t)slots_of(num_seqs, total_T);
    const size_t gates = up256(slots * H * kGateRows * kC * sizeof(float));
    const size_t states = up256(slots * H * P * N * sizeof(float)), sums = up256(slots * H * 3 * sizeof(float));
    const int subsets = subsets_of(num_seqs, total_T, H, G);
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
    return used + segments64(num_seqs, total_T, H, P, N, 2, varied, w ? &w->g : nullptr, w ? at + used : nullptr);
}

}  // namespace

cudaError_t launch_finish(const SsmArgs& a, const Work& w, long slots, cudaStream_t s) {
    const int sums = a.dA_log || a.ddt_bias || a.dD ? 3 * ((a.H + 31) / 32) : 0;
    const int parts = w.subsets > 1 ? 2 * (int)(((long)a.seqs.total_T * a.G * a.N / 8 + 255) / 256) : 0;
    const int zeros = a.zero_outside && a.seqs.cu && a.seqs.total_T > 0 ? kZeroBlocks : 0;
    if (sums + parts + zeros == 0) return cudaSuccess;
    const dim3 grid((unsigned)(sums + parts + zeros));
    return a.dtype == GDN_BF16 ? launch_after(ssm_finish_kernel<__nv_bfloat16>, grid, 256, 0, s, a, w, slots, sums, parts)
                               : launch_after(ssm_finish_kernel<float>, grid, 256, 0, s, a, w, slots, sums, parts);
}

}  // namespace ssm

size_t ssm_bwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N, gdn_dtype dtype) {
    if (dtype == GDN_BF16 && total_T > 0) return ssm::tc_bwd_workspace_bytes(num_seqs, total_T, H, G, P, N);
    const size_t equal = ssm::layout(num_seqs, total_T, H, G, P, N, false, nullptr, nullptr),
                 varied = ssm::layout(num_seqs, total_T, H, G, P, N, true, nullptr, nullptr);
    return equal > varied ? equal : varied;
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, cudaStream_t s) {
    if (a.dtype == GDN_BF16 && a.seqs.total_T > 0) return ssm::launch_tc_bwd(a, s);
    ssm::Work w{};
    ssm::layout(a.seqs.num_seqs, a.seqs.total_T, a.H, a.G, a.P, a.N, a.seqs.cu && a.seqs.num_seqs > 1, &w, static_cast<unsigned char*>(a.workspace));
    cudaError_t e = ssm::launch_gates(a, w, s);
    if (e == cudaSuccess) e = ssm::launch_scan(a, w, 2, s);
    if (e != cudaSuccess) return e;
    const long slots = ssm::slots_of(a.seqs.num_seqs, a.seqs.total_T);
    e = a.N == 128 ? ssm::grad_one<128>(a, w, s) : ssm::grad_one<64>(a, w, s);
    if (e != cudaSuccess) return e;
    return ssm::launch_finish(a, w, slots, s);
}

}  // namespace gdn

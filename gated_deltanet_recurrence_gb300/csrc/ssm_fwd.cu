// ssm_fwd.cu -- the selective state space scan over packed prompts, in chunks of 64 tokens.
//
// Per head, with v_t = dt_t x_t and G the running sums of the log decays g_t = -exp(A_log) dt_t inside a chunk,
//   y_i = e^{G_i} S_0 C_i + sum_{j <= i} e^{G_i - G_j} (B_j . C_i) v_j + D x_i,
//   S_1 = e^{G_last} S_0 + sum_j e^{G_last - G_j} v_j B_j^T.
// Fp32 inputs (bf16: ssm_tc.cu).  Three kernels: the gates of all chunks; the states at the chunk starts, one block per
// (sequence or segment of it, head, 64 rows) that walks along its chunks with the state in registers; the outputs, one
// block per chunk and share of a group's heads.  All products are fp32 matrices in three bf16 planes, six terms each: the
// tensor instructions and the splits into planes bound the outputs (6144 tokens of 24 heads of 128, d_state 128: 431 us),
// a chunk's latency the walk (3.3 us, d_state 64: 2.1).  A block of four warps for each (chunk, head) took 629 us.
// Smallest calls: 200 tokens of two heads 16 us, three launches that start behind one another.
//
// Long sequences of few heads are cut into segments of `each` chunks: all segments' own states (from zero) at once, then
//   start_{k + 1} = e^{sum of segment k} start_k + own_k
// for all numbers of a state at once, then the walk itself from the segments' starts: the walk's work twice, spread over
// all SMs.  6144 tokens of 8 heads, d_state 128: 403 us whole, 103 in segments.
#include "ssm_chunk.cuh"

namespace gdn {
namespace ssm {
namespace {

// ---- gates ---------------------------------------------------------------------------------------

// One warp per (slot, head): lane l holds tokens 2 l and 2 l + 1.
constexpr int kGateWarps = 8;
__global__ void __launch_bounds__(kGateWarps * 32) ssm_gates_kernel(SsmArgs a, float* gates) {
    dependency_start();
    Chunk c;
    if (!find_chunk(a.seqs, blockIdx.x, a.err, c)) return;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * kGateWarps + (threadIdx.x >> 5);
    if (h >= a.H) return;
    const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    float dt[2], g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        dt[i] = t < c.len ? ssm_softplus(a.a[(long)(c.t0 + t) * a.H + h] + bias) : 0.f;
        g[i] = t < c.len ? log_decay(rate, dt[i]) : 0.f;
    }
    Two pair = two_add(Two{g[0], 0.f}, Two{g[1], 0.f}), sum = pair;
    float suf = g[0] + g[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two up{__shfl_up_sync(0xffffffffu, sum.h, o), __shfl_up_sync(0xffffffffu, sum.l, o)};
        if (lane >= o) sum = two_add(up, sum);
        const float down = __shfl_down_sync(0xffffffffu, suf, o);
        if (lane + o < 32) suf += down;
    }
    // sums before this lane's tokens, and behind them
    Two before{__shfl_up_sync(0xffffffffu, sum.h, 1), __shfl_up_sync(0xffffffffu, sum.l, 1)};
    if (lane == 0) before = Two{0.f, 0.f};
    float behind = __shfl_down_sync(0xffffffffu, suf, 1);
    if (lane == 31) behind = 0.f;
    const Two G0 = two_add(before, Two{g[0], 0.f});
    float* out = gates + ((long)blockIdx.x * a.H + h) * (kGateRows * kC) + 2 * lane;
    *reinterpret_cast<float2*>(out) = make_float2(dt[0], dt[1]);
    *reinterpret_cast<float2*>(out + kC) = make_float2(G0.h, sum.h);
    *reinterpret_cast<float2*>(out + 2 * kC) = make_float2(G0.l, sum.l);
    *reinterpret_cast<float2*>(out + 3 * kC) = make_float2(expf(G0.h) * (1.f + G0.l), expf(sum.h) * (1.f + sum.l));
    *reinterpret_cast<float2*>(out + 4 * kC) = make_float2(expf(behind + g[1]), expf(behind));
}

// ---- states --------------------------------------------------------------------------------------

// Block: 8 warps; warp w holds rows 16 (w % 4) .. of the 64 and half of the N columns.  Blocks with blockIdx.y = 1: the
// states' gradients, from the last chunk to the first.  With `own` the blocks leave their segments' states from zero, and
// nothing of the way.
constexpr int kScanThreads = 256;
template <int N>
__global__ void __launch_bounds__(kScanThreads) ssm_scan_kernel(SsmArgs a, Work w, bool own) {
    constexpr int NT = N / 16, KV = N / 32;  // KV: vectors of B a thread loads
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const bfp::Tile<kC, N, 3> Kt{base};
    const bfp::Tile<kC, 64, 3> Vt{base + bfp::kTileBytes<kC, N, 3>};
    __shared__ float fac[kC];
    const bool REV = blockIdx.y;
    dependency_start();
    const int slices = a.P / 64, s = blockIdx.x % slices, h = blockIdx.x / slices % a.H, index = blockIdx.x / slices / a.H;
    Run run;
    // what a segment leaves goes to the next one: the last of a sequence has none
    if (!find_run(a.seqs, w.g.each, kC, index, a.err, run) || (own && (REV ? run.first : run.last))) {
        dependency_wait();
        return;
    }
    const int bos = run.t0, eos = run.end, chunks = (eos - bos + kC - 1) / kC;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m0 = (warp & 3) * 16, n0 = (warp >> 2) * (N / 2);
    const int g = h / (a.H / a.G);
    const float* K = static_cast<const float*>(REV ? a.C : a.B) + (long)g * N;
    const long k_stride = REV ? a.C_stride : a.B_stride;
    const float* X = static_cast<const float*>(REV ? a.dout : a.x) + (long)h * a.P + s * 64;
    const long x_stride = REV ? (long)a.H * a.P : a.x_stride;
    const long row0 = (((long)run.n * a.H + h) * a.P + s * 64) * N, own0 = (((long)index * a.H + h) * a.P + s * 64) * N;
    const float* init = nullptr;
    float* last = nullptr;
    if (own) {
        last = (REV ? w.g.own[1] : w.g.own[0]) + own0;
    } else {
        const float* given = REV ? a.dfinal_state : a.initial_state;
        init = w.g.each ? (REV ? w.g.start[1] : w.g.start[0]) + own0 : (given ? given + row0 : nullptr);
        float* end = REV ? a.dinitial_state : a.final_state;
        if (end && (REV ? run.first : run.last)) last = end + row0;
    }
    float* keep = REV ? w.dstates : w.states;

    dependency_wait();
    float S[NT][4];
    bfp::pairs<NT>(m0, n0, lane, [&](int j, int hh, int p, int c) {
        const float2 v = init ? *reinterpret_cast<const float2*>(init + (long)p * N + c) : make_float2(0.f, 0.f);
        S[j][2 * hh] = v.x;
        S[j][2 * hh + 1] = v.y;
    });
    bfp::Raw8 kr[KV], xr[2];
    float gd = 0.f, gb = 0.f, gl = 0.f;  // this thread's token: dt, the chunk factor; the whole chunk's decay
    const auto fetch = [&](int k) {
        const int t0 = bos + k * kC, len = min(eos - t0, kC);
#pragma unroll
        for (int i = 0; i < KV; ++i) {
            const int v = i * kScanThreads + tid, r = v / (N / 8), c = v % (N / 8) * 8;
            kr[i].load(K + (long)(t0 + r) * k_stride + c, r < len);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = i * kScanThreads + tid, r = v / 8, c = v % 8 * 8;
            xr[i].load(X + (long)(t0 + r) * x_stride + c, r < len);
        }
        const float* gt = w.gates + ((run.slot0 + k) * a.H + h) * (kGateRows * kC);
        if (tid < kC) {
            gd = REV ? 1.f : gt[tid];
            gb = gt[(REV ? 3 : 4) * kC + tid];
        }
        gl = gt[3 * kC + kC - 1];
    };
    float total = 1.f;
    if (chunks > 0) fetch(REV ? chunks - 1 : 0);
    for (int q = 0; q < chunks; ++q) {
        const int k = REV ? chunks - 1 - q : q;
        const float decay = gl;
        total *= decay;
        if (tid < kC) fac[tid] = gd * gb;
#pragma unroll
        for (int i = 0; i < KV; ++i) {
            const int v = i * kScanThreads + tid;
            kr[i].put(Kt, v / (N / 8), v % (N / 8) * 8);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = i * kScanThreads + tid, r = v / 8;
            float x[8];
            xr[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= fac[r];
            bfp::put8(Vt, r, v % 8 * 8, x);
        }
        float* to = keep + (((run.slot0 + k) * a.H + h) * a.P + s * 64) * N;
        bfp::pairs<NT>(m0, n0, lane, [&](int j, int hh, int p, int c) {
            if (!own) *reinterpret_cast<float2*>(to + (long)p * N + c) = make_float2(S[j][2 * hh], S[j][2 * hh + 1]);
            S[j][2 * hh] *= decay;
            S[j][2 * hh + 1] *= decay;
        });
        if (q + 1 < chunks) fetch(REV ? k - 1 : k + 1);
        __syncthreads();
        bfp::product<kC, true, true>(S, Vt, m0, Kt, n0, lane);
        __syncthreads();
    }
    if (last)
        bfp::pairs<NT>(m0, n0, lane, [&](int j, int hh, int p, int c) {
            *reinterpret_cast<float2*>(last + (long)p * N + c) = make_float2(S[j][2 * hh], S[j][2 * hh + 1]);
        });
    if (own && s == 0 && tid == 0) (REV ? w.g.decay[1] : w.g.decay[0])[(long)index * a.H + h] = total;
}

template <int N>
cudaError_t scan_one(const SsmArgs& a, const Work& w, bool own, int directions, cudaStream_t s) {
    constexpr int smem = bfp::kTileBytes<kC, N, 3> + bfp::kTileBytes<kC, 64, 3>;
    const cudaError_t e = cudaFuncSetAttribute(ssm_scan_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long runs = w.g.each ? segment_slots(a.seqs.num_seqs, a.seqs.total_T, w.g) : a.seqs.num_seqs;
    return launch_after(ssm_scan_kernel<N>, dim3((unsigned)(runs * a.H * (a.P / 64)), directions), kScanThreads, smem, s, a, w, own);
}

// ---- segments ------------------------------------------------------------------------------------

// One thread: four numbers of the states of a (sequence, head), in one direction, along its segments; loads of four
// segments at a time.  About 3 us.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) ssm_join_kernel(SsmArgs a, Segments g) {
    const int n = blockIdx.z, back = blockIdx.y / a.H, h = blockIdx.y % a.H, unit = g.each * g.unit;
    dependency_start();
    const bool bad = packed_find(a.seqs, 0, 1, 0, a.err) == -2;
    dependency_wait();
    if (bad) return;
    const int bos = a.seqs.bos(n), count = max((a.seqs.bos(n + 1) - bos + unit - 1) / unit, 1);
    const long size = (long)a.P * a.N, at = ((long)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (at >= size) return;
    const float* given = back ? a.dfinal_state : a.initial_state;
    float4 S = given ? *reinterpret_cast<const float4*>(given + ((long)n * a.H + h) * size + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    const long first = bos / unit + n;
    const auto row = [&](int k) { return (first + (back ? count - 1 - k : k)) * a.H + h; };  // of the k-th segment on the way
    // the first one's too: the given states may be overwritten by the last segment's block
    *reinterpret_cast<float4*>((back ? g.start[1] : g.start[0]) + row(0) * size + at) = S;
    for (int k0 = 0; k0 + 1 < count; k0 += 4) {
        float4 own[4];
        float decay[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k0 + e + 1 >= count) continue;
            own[e] = *reinterpret_cast<const float4*>((back ? g.own[1] : g.own[0]) + row(k0 + e) * size + at);
            decay[e] = (back ? g.decay[1] : g.decay[0])[row(k0 + e)];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k0 + e + 1 >= count) continue;
            S.x = fmaf(decay[e], S.x, own[e].x);
            S.y = fmaf(decay[e], S.y, own[e].y);
            S.z = fmaf(decay[e], S.z, own[e].z);
            S.w = fmaf(decay[e], S.w, own[e].w);
            *reinterpret_cast<float4*>((back ? g.start[1] : g.start[0]) + row(k0 + e + 1) * size + at) = S;
        }
    }
}

// ---- outputs -------------------------------------------------------------------------------------

// Block: a chunk and a share of one group's (head, 64 rows of its state); C B^T is formed once for them.  16 warps of 16
// tokens and 16 columns each.  What the next head brings is loaded beside the products of this one.
constexpr int kOutThreads = 512;
template <int N>
constexpr int kOutSmem = 2 * bfp::kTileBytes<kC, N, 3> + bfp::kTileBytes<kC, 64, 3> + bfp::kTileBytes<64, N, 3>;
template <int N>
__global__ void __launch_bounds__(kOutThreads) ssm_out_kernel(SsmArgs a, Work w, int shares) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const bfp::Tile<kC, N, 3> Kt{base}, Ct{base + bfp::kTileBytes<kC, N, 3>};
    const bfp::Tile<kC, 64, 3> Xt{base + 2 * bfp::kTileBytes<kC, N, 3>}, Mt{base};  // the masked products take B's place
    const bfp::Tile<64, N, 3> St{base + 2 * bfp::kTileBytes<kC, N, 3> + bfp::kTileBytes<kC, 64, 3>};
    __shared__ float gate[kGateRows][kC];
    Chunk c;
    if (!find_chunk(a.seqs, blockIdx.x, a.err, c)) {
        dependency_wait();
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, m = (tid >> 5 & 3) * 16, p0 = (tid >> 7) * 16;
    const int slices = a.P / 64, g = blockIdx.y % a.G, share = blockIdx.y / a.G, units = a.H / a.G * slices;
    const int u0 = (int)((long)units * share / shares), u1 = (int)((long)units * (share + 1) / shares);
    {
        const float* B = static_cast<const float*>(a.B) + (long)c.t0 * a.B_stride + (long)g * N;
        const float* C = static_cast<const float*>(a.C) + (long)c.t0 * a.C_stride + (long)g * N;
#pragma unroll
        for (int v = tid; v < kC * N / 8; v += kOutThreads) {
            const int r = v / (N / 8), col = v % (N / 8) * 8;
            bfp::Raw8 k, q;
            k.load(B + (long)r * a.B_stride + col, r < c.len);
            q.load(C + (long)r * a.C_stride + col, r < c.len);
            k.put(Kt, r, col);
            q.put(Ct, r, col);
        }
    }
    __syncthreads();
    float CB[2][4];
    bfp::clear(CB);
    if (p0 <= m) bfp::product<N, false, false>(CB, Ct, m, Kt, p0, lane);
    constexpr int NV = N / 64;  // vectors of a state that a thread loads
    bfp::Raw8 xr, sr[NV];
    float gr = 0.f;
    const auto fetch = [&](int u) {
        const int h = g * (a.H / a.G) + u / slices, s = u % slices;
        const float* X = static_cast<const float*>(a.x) + (long)c.t0 * a.x_stride + (long)h * a.P + s * 64;
        xr.load(X + (long)(tid / 8) * a.x_stride + tid % 8 * 8, tid / 8 < c.len);
        const float* S0 = w.states + (((long)blockIdx.x * a.H + h) * a.P + s * 64) * N;
#pragma unroll
        for (int i = 0; i < NV; ++i) sr[i].load(S0 + (long)(i * kOutThreads + tid) * 8, true);
        if (tid < kGateRows * kC) gr = w.gates[((long)blockIdx.x * a.H + h) * (kGateRows * kC) + tid];
    };
    dependency_wait();  // gates and states
    if (u0 < u1) fetch(u0);
    for (int u = u0; u < u1; ++u) {
        __syncthreads();  // what was in the tiles has been read
        xr.put(Xt, tid / 8, tid % 8 * 8);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * kOutThreads + tid;
            sr[i].put(St, v / (N / 8), v % (N / 8) * 8);
        }
        if (tid < kGateRows * kC) (&gate[0][0])[tid] = gr;
        __syncthreads();
        const int h = g * (a.H / a.G) + u / slices, s = u % slices;
        if (p0 <= m)
            bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int col) {
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = col + e;
                    const float d = (gate[1][i] - gate[1][t]) + (gate[2][i] - gate[2][t]);
                    v[e] = t <= i ? CB[j][2 * hh + e] * gate[0][t] * expf(d) : 0.f;
                }
                bfp::put2(Mt, i, col, v[0], v[1]);
            });
        if (u + 1 < u1) fetch(u + 1);
        float Y[2][4];
        bfp::clear(Y);
        bfp::product<N, false, false>(Y, Ct, m, St, p0, lane);
        bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int) {
            Y[j][2 * hh] *= gate[3][i];
            Y[j][2 * hh + 1] *= gate[3][i];
        });
        __syncthreads();
        bfp::product<kC, false, true, bfp::kLower>(Y, Mt, m, Xt, p0, lane);
        const float D = a.D ? a.D[h] : 0.f;
        float* out = static_cast<float*>(a.out) + ((long)c.t0 * a.H + h) * a.P + s * 64;
        bfp::pairs<2>(m, p0, lane, [&](int j, int hh, int i, int col) {
            if (i >= c.len) return;
            const float2 x = bfp::get2(Xt, i, col);
            const float y0 = fmaf(D, x.x, Y[j][2 * hh]), y1 = fmaf(D, x.y, Y[j][2 * hh + 1]);
            *reinterpret_cast<float2*>(out + (long)i * a.H * a.P + col) = make_float2(y0, y1);
        });
    }
}

template <int N>
cudaError_t out_one(const SsmArgs& a, const Work& w, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(ssm_out_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutSmem<N>);
    if (e != cudaSuccess) return e;
    // shares for two rounds of blocks: each brings B and C again (for one, two, three rounds: 2048 tokens of 16 heads 80,
    // 70, 78 us; 6144 of 24 in three sequences 251, 224, 232)
    const long slots = slots_of(a.seqs.num_seqs, a.seqs.total_T), blocks = slots * a.G, units = (long)(a.H / a.G) * (a.P / 64);
    const long fill = (2 * kSMs + blocks - 1) / blocks, shares = fill < units ? fill : units;
    return launch_after(ssm_out_kernel<N>, dim3((unsigned)slots, (unsigned)(a.G * shares)), kOutThreads, kOutSmem<N>, s, a, w, (int)shares);
}

}  // namespace

cudaError_t launch_gates(const SsmArgs& a, const Work& w, cudaStream_t s) {
    const dim3 grid((unsigned)slots_of(a.seqs.num_seqs, a.seqs.total_T), (unsigned)((a.H + kGateWarps - 1) / kGateWarps));
    ssm_gates_kernel<<<grid, kGateWarps * 32, 0, s>>>(a, w.gates);
    return cudaGetLastError();
}

cudaError_t launch_join(const SsmArgs& a, const Segments& g, int directions, cudaStream_t s) {
    const dim3 grid((unsigned)(a.P * a.N / (4 * kJoinThreads)), (unsigned)(a.H * directions), (unsigned)a.seqs.num_seqs);
    return launch_after(ssm_join_kernel, grid, kJoinThreads, 0, s, a, g);
}

cudaError_t launch_scan(const SsmArgs& a, const Work& w, int directions, cudaStream_t s) {
    const auto scan = [&](bool own) {
        return a.N == 128 ? scan_one<128>(a, w, own, directions, s) : scan_one<64>(a, w, own, directions, s);
    };
    if (w.g.each) {
        cudaError_t e = scan(true);
        if (e == cudaSuccess) e = launch_join(a, w.g, directions, s);
        if (e != cudaSuccess) return e;
    }
    return scan(false);
}

// Chunks of a segment, or 0.  Blocks are counted against the SMs.  Few rows: as many segments as fill the SMs, where that
// pays for sequences of one length, or, where the lengths may differ, for the longest of n, taken as 1 + 1/2 + ... + 1/n
// times the average.  A packed batch of up to two rounds of blocks, forwards: segments a little longer than the average,
// where they pay for that longest one. In us, whole and in segments, bf16, d_state 128, 64 rows a head: 1536 tokens of 8
// heads 36, 27; 6144 of 8 128, 30; 6144 of 24 129, 48; 32768 of 16 657, 136; 8192 in 4 sequences of 16 heads 47, 56
// (stays whole).  Packed: lengths 1, 37, 513, 3001, 64, 1333, 700 of 24 rows 71, 60 (seven of 807: 47, 52); 8000, 3 x
// 2000, 4 x 500 of 24 170, 118 (eight of 2048: 95, 105).  Segments of 0.75, 1, 1.25 times the average:
// the first of these 65, 61, 60, the third 129, 129, 118.
static int segment_chunks(int num_seqs, int total_T, int H, int P, int unit, int directions, bool varied, SegmentCost cost) {
    const long rows = (long)H * (P / 64) * directions * num_seqs, chunks = ((long)total_T + unit - 1) / unit,
               avg = (chunks + num_seqs - 1) / num_seqs;
    const auto split = [&](long each) { return each * (cost.whole + cost.own) + cost.more; };
    if (rows > 2 * kSMs || total_T > 1 << 29) return 0;  // a segment's tokens are an int
    double longest = (double)avg;
    for (int n = 2; varied && n <= num_seqs; ++n) longest += (double)avg / n;
    if (rows <= kSMs) {
        const long count = kSMs / rows, fill = (avg + count - 1) / count, each = fill < 4 ? 4 : fill;
        if (longest * cost.whole > split(each)) return (int)each;
    }
    if (directions > 1 || !varied) return 0;
    const long each = avg + avg / 4 < 8 ? 8 : avg + avg / 4;
    return longest * cost.whole > split(each) ? (int)each : 0;
}

size_t segments_layout(int num_seqs, int total_T, int H, int P, int N, int unit, int directions, bool varied, SegmentCost cost,
                       Segments* g, unsigned char* at) {
    Segments w{};
    w.unit = unit;
    w.each = segment_chunks(num_seqs, total_T, H, P, unit, directions, varied, cost);
    size_t bytes = 0;
    if (w.each) {
        const size_t slots = (size_t)segment_slots(num_seqs, total_T, w), states = slots * H * P * N * sizeof(float),
                     decays = up256(slots * H * sizeof(float));
        for (int i = 0; i < directions && g; ++i) {
            w.own[i] = reinterpret_cast<float*>(at + 2 * i * states);
            w.start[i] = reinterpret_cast<float*>(at + (2 * i + 1) * states);
            w.decay[i] = reinterpret_cast<float*>(at + 2 * directions * states + i * decays);
        }
        bytes = directions * (2 * states + decays);
    }
    if (g) *g = w;
    return bytes;
}

}  // namespace ssm

size_t ssm_fwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N, gdn_dtype dtype) {
    if (dtype == GDN_BF16) return total_T > 0 ? ssm::tc_workspace_bytes(num_seqs, total_T, H, P, N) : 0;
    const size_t slots = (size_t)ssm::slots_of(num_seqs, total_T);
    const size_t used = ssm::up256(slots * H * ssm::kGateRows * ssm::kC * sizeof(float)) + slots * H * P * N * sizeof(float);
    const size_t equal = ssm::segments64(num_seqs, total_T, H, P, N, 1, false, nullptr, nullptr),
                 varied = ssm::segments64(num_seqs, total_T, H, P, N, 1, true, nullptr, nullptr);
    return used + (equal > varied ? equal : varied);
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t s) {
    if (a.dtype == GDN_BF16 && a.seqs.total_T > 0) return ssm::launch_tc(a, s);
    ssm::Work w{};
    const size_t slots = (size_t)ssm::slots_of(a.seqs.num_seqs, a.seqs.total_T);
    w.gates = static_cast<float*>(a.workspace);
    w.states = w.gates + ssm::up256(slots * a.H * ssm::kGateRows * ssm::kC * sizeof(float)) / sizeof(float);
    ssm::segments64(a.seqs.num_seqs, a.seqs.total_T, a.H, a.P, a.N, 1, a.seqs.cu && a.seqs.num_seqs > 1, &w.g,
                    reinterpret_cast<unsigned char*>(w.states + slots * a.H * a.P * a.N));
    cudaError_t e = ssm::launch_gates(a, w, s);
    if (e == cudaSuccess) e = ssm::launch_scan(a, w, 1, s);
    if (e != cudaSuccess || a.seqs.total_T == 0) return e;
    return a.N == 128 ? ssm::out_one<128>(a, w, s) : ssm::out_one<64>(a, w, s);
}

}  // namespace gdn

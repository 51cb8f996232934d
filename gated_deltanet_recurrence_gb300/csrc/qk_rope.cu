// qk_rope.cu -- queries and keys normalised per head and rotated by their position, in one pass.
//
// "6.6 Gated DeltaNet", 6.6.4, normalises q and k per head before they meet the state; layers that also carry the
// token's position in them rotate pairs of channels.  With n = x / sqrt(mean x^2 + eps) (RMS norm) or
// x / sqrt(sum x^2 + eps) (length one), m = w n, and for pair i of the first d_rot channels
//   (u, v) -> (u cos_i - v sin_i, v cos_i + u sin_i),
// with cos_i, sin_i of the token's position from a table; the other channels pass.  Gradients: the rotation
// backwards, then dw = sum dm n, dn = dm w, dx = r (dn - n mean(dn n)) (or the sum's, for length one).
//
// Memory would bound it; 8192 tokens of 16 + 4 heads of 128 (bf16) take 16.4 us, 5.2 TB/s (77% of a copy's rate),
// gradients of 3001 tokens of 16 + 16 heads of 64 8.9 us with the launch behind.  What is left are instructions (43% of the
// issue slots; 58% and 17.5 us before arithmetic went in pairs of channels) and, at two blocks an SM, their latency.  Two
// blocks with all values in registers; three, with spills, 17.8 for 17.0 on another machine.
//
// Rows come through rings of asynchronous copies, as in short_conv.cu.  A row (one head of one
// token) is d / 8 lanes of 8 channels; a set of lanes takes one token and several heads, so that the token's cosines and
// sines and the weights are loaded once.  Pairs of channels m = d_rot / 2 apart are exchanged by shuffles where they lie
// in the same place of another lane (m a multiple of 8), through shared memory otherwise.
#include "ssm_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kV = 8;
enum Pairs { kNeighbours, kLanes, kShared };
// Rows worked on together, and groups of them on their way; the rings that hold them (of x; backwards of the gradient
// too).
template <bool BWD>
constexpr int kTogether = BWD ? 2 : 4;
constexpr int kAhead = 2;
template <typename T, bool BWD>
using Rows = Ring<T, kV, kTogether<BWD> * kAhead, kThreads>;

// Lanes of a row: the power of two that holds d / 8 vectors.
int lanes_of(int d) {
    int l = 1;
    while (l * kV < d) l *= 2;
    return l;
}

// Heads a set of lanes takes: all of a token's when there are tokens enough for a block an SM, fewer in small calls.  In
// us, with sets for half a block, one, two, four and eight blocks an SM: 8192 tokens of 16 + 4 heads of 128 (bf16) 18.2,
// 18.3, 18.3, 19.6, 23.8; 3001 of 16 + 16 of 64: 9.6, 7.6, 6.8, 8.4, 11.7; 1000 of 8 + 8 of 256: 8.0, 6.7, 8.4, 11.3,
// 16.6.
int heads_per_set(int T, int heads, int L) {
    const long sets = (long)kSMs * (kThreads / L);
    int per = heads;
    while (per > 1 && (long)T * ((heads + per - 1) / per) < sets) per = (per + 1) / 2;
    return per;
}

template <int L>
__device__ __forceinline__ float set_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One lane's eight channels x and their partners y, as they lie in memory (so that bf16 pairs move in one exchange).
constexpr int kPairsOf = kV / 2;
template <typename T, int L, Pairs PAIRS>
__device__ __forceinline__ void partners(const RawRow<T, kV>& r, const F2 (&x)[kPairsOf], F2 (&y)[kPairsOf], int lane, int from, int m,
                                         float* row) {
    if constexpr (PAIRS == kNeighbours) {
#pragma unroll
        for (int j = 0; j < kPairsOf; ++j) {
            float u, v;
            x[j].get(u, v);
            y[j] = F2(v, u);
        }
    } else if constexpr (PAIRS == kLanes) {
        RawRow<T, kV> p;
#pragma unroll
        for (int j = 0; j < RawRow<T, kV>::W; ++j) p.u[j] = __shfl_sync(0xffffffffu, r.u[j], from, L);
        p.get(y);
    } else {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kPairsOf; ++j) x[j].get(row[lane * kV + 2 * j], row[lane * kV + 2 * j + 1]);
        __syncwarp();
        float o[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = lane * kV + j;
            o[j] = row[c < m ? c + m : (c < 2 * m ? c - m : c)];
        }
        pair_up<kV>(o, y);
    }
}
__device__ __forceinline__ float sum_of(F2 x) {
    float u, v;
    x.get(u, v);
    return u + v;
}

// One block: kThreads / L sets; a set: one token, `per` heads of the q and k heads taken together.  Sets are numbered
// part by part, each part's tokens rounded up to whole warps, so that all sets of a warp have the same heads.
template <typename T, int L, Pairs PAIRS, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) qk_kernel(QkArgs a, int per, long tokens, long sets) {
    constexpr int U = kTogether<BWD>;
    extern __shared__ __align__(16) unsigned char smem[];
    Rows<T, BWD> rx(smem), rg(smem + (BWD ? Rows<T, BWD>::kSmem : 0));
    __shared__ float stage[PAIRS == kShared ? kThreads * kV : 1];
    const int lane = threadIdx.x % L;
    const int c0 = lane * kV, d = a.d, m = a.rot / 2;
    const bool in = c0 < d;
    const float inv = a.l2 ? 1.0f : 1.0f / (float)d;
    float* row = stage + (PAIRS == kShared ? threadIdx.x / L * L * kV : 0);
    const int off = m / kV, from = lane >= 2 * off ? lane : (lane < off ? lane + off : lane - off);
    F2 dw[2][kPairsOf];
#pragma unroll
    for (int j = 0; j < kPairsOf; ++j) dw[0][j] = dw[1][j] = F2(0.f, 0.f);
    const long stride = (long)gridDim.x * (kThreads / L);
    for (long base = (long)blockIdx.x * (kThreads / L); base < sets; base += stride) {
        const long set = base + threadIdx.x / L;
        const long t = set % tokens;
        const int part = (int)(set / tokens);
        bool live = set < sets && t < a.T;
        float cs[kV], sn[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) { cs[j] = 1.f; sn[j] = 0.f; }
        if (live) {
            const long pos = a.positions ? (long)a.positions[t] : t;
            if (pos < 0 || pos >= a.max_positions) {
                if (lane == 0) record_error(a.err, GDN_ERR_ARG);
                live = false;
            } else {
                const float* tab = a.cos_sin + pos * a.rot;
                if (PAIRS == kLanes) {
                    if (c0 < 2 * m) {
                        load_row<kV>(tab + (c0 < m ? c0 : c0 - m), cs);
                        load_row<kV>(tab + (c0 < m ? c0 + m : c0), sn);
                        if ((c0 >= m) == BWD) {
#pragma unroll
                            for (int j = 0; j < kV; ++j) sn[j] = -sn[j];
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        const int c = c0 + j;
                        if (c >= 2 * m) continue;
                        const int i = PAIRS == kNeighbours ? c >> 1 : (c < m ? c : c - m);
                        const bool second = PAIRS == kNeighbours ? c & 1 : c >= m;
                        cs[j] = tab[i];
                        sn[j] = second != BWD ? tab[m + i] : -tab[m + i];
                    }
                }
            }
        }
        const bool on = live && in;
        if (!on) {  // a set without a row reads zeros, whatever an earlier one has left
            for (int i = 0; i < U * kAhead; ++i) {
                rx.clear(i);
                if (BWD) rg.clear(i);
            }
        }
        // this set's heads of q, then of k
        const int lo = part * per, hi = min(a.heads[0] + a.heads[1], lo + per);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h0 = i ? max(lo - a.heads[0], 0) : lo, h1 = i ? hi - a.heads[0] : min(hi, a.heads[0]);
            if (h0 >= h1) continue;
            // forward: the weights go into the rotation's factors, w of the channel and of its partner
            F2 w[kPairsOf], fc[kPairsOf], fs[kPairsOf];
            {
                float own[kV], wc[kV], ws[kV];
#pragma unroll
                for (int j = 0; j < kV; ++j) own[j] = 1.f;
                if (in && a.w[i]) load_row<kV>(a.w[i] + c0, own);
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const int c = c0 + j;
                    const int other = PAIRS == kNeighbours ? c ^ 1 : (c < m ? c + m : (c < 2 * m ? c - m : c));
                    wc[j] = BWD ? cs[j] : own[j] * cs[j];
                    ws[j] = !BWD && in && a.w[i] ? a.w[i][other] * sn[j] : sn[j];
                }
                pair_up<kV>(own, w);
                pair_up<kV>(wc, fc);
                pair_up<kV>(ws, fs);
            }
            const T* src = static_cast<const T*>(a.x[i]) + t * a.x_stride[i] + h0 * d + c0;
            const T* grad = BWD ? static_cast<const T*>(a.dout[i]) + (t * a.heads[i] + h0) * d + c0 : nullptr;
            T* out = static_cast<T*>(a.out[i]) + t * a.out_stride[i] + h0 * d + c0;
            int asked = h0;
            const auto ask = [&](int q) {
                if (on) {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (asked + u < h1) {
                            rx.ask(U * q + u, src + u * d);
                            if (BWD) rg.ask(U * q + u, grad + u * d);
                        }
                }
                ring_commit();
                asked += U;
                src += U * d;
                if (BWD) grad += U * d;
            };
#pragma unroll
            for (int q = 0; q < kAhead; ++q) ask(q);
            int group = 0;
            for (int h = h0; h < h1; h += U) {
                RawRow<T, kV> xr[U], gr[BWD ? U : 1];
                ring_wait<kAhead - 1>();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rx.read(U * group + u, xr[u]);
                    if constexpr (BWD) rg.read(U * group + u, gr[u]);
                }
                ask(group);
                group = group + 1 == kAhead ? 0 : group + 1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h + u >= h1) break;
                    F2 x[kPairsOf], y[kPairsOf], s2(0.f, 0.f);
                    xr[u].get(x);
#pragma unroll
                    for (int j = 0; j < kPairsOf; ++j) s2 = fma2(x[j], x[j], s2);
                    const float ms = set_sum<L>(sum_of(s2)) * inv + a.eps;
                    // a set without a row has a sum of zero, whose factor with eps = 0 is infinite, and adds to dw
                    const float r = BWD && !live ? 0.f : rsqrtf(ms);
                    const F2 r2(r, r);
                    if constexpr (!BWD) {
                        partners<T, L, PAIRS>(xr[u], x, y, lane, from, m, row);
#pragma unroll
                        for (int j = 0; j < kPairsOf; ++j) x[j] = r2 * fma2(y[j], fs[j], x[j] * fc[j]);
                        if (on) store_pairs<kV>(out + u * d, x);
                    } else {
                        F2 g[kPairsOf], d2(0.f, 0.f);
                        gr[u].get(g);
                        partners<T, L, PAIRS>(gr[u], g, y, lane, from, m, row);
#pragma unroll
                        for (int j = 0; j < kPairsOf; ++j) {
                            g[j] = fma2(y[j], fs[j], g[j] * fc[j]);
                            x[j] = x[j] * r2;
                            dw[i][j] = fma2(g[j], x[j], dw[i][j]);
                            g[j] = g[j] * w[j];
                            d2 = fma2(g[j], x[j], d2);
                        }
                        const float dot = -set_sum<L>(sum_of(d2)) * inv;
#pragma unroll
                        for (int j = 0; j < kPairsOf; ++j) g[j] = r2 * fma2(x[j], F2(dot, dot), g[j]);
                        if (on) store_pairs<kV>(out + u * d, g);
                    }
                }
                out += U * d;
            }
            ring_wait<0>();
        }
    }
    if constexpr (BWD) {
        if (!a.partial) return;
        // the block's sets are added in order; its row of the table is [q's d, k's d]
        __shared__ float sums[kThreads / L][2][L * kV];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kPairsOf; ++j) dw[i][j].get(sums[threadIdx.x / L][i][c0 + 2 * j], sums[threadIdx.x / L][i][c0 + 2 * j + 1]);
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * d; e += kThreads) {
            const int i = e >= d, c = i ? e - d : e;
            float s = 0.f;
            for (int q = 0; q < kThreads / L; ++q) s += sums[q][i][c];
            a.partial[((long)i * gridDim.x + blockIdx.x) * d + c] = s;
        }
    }
}

struct Plan {
    int L, per;
    long tokens, sets, blocks;
};
Plan plan(int T, int H, int H_k, int d, bool bwd) {
    Plan p;
    p.L = lanes_of(d);
    p.per = heads_per_set(T, H + H_k, p.L);
    const int warp = 32 / p.L;
    p.tokens = ((long)T + warp - 1) / warp * warp;
    p.sets = p.tokens * ((H + H_k + p.per - 1) / p.per);
    p.blocks = (p.sets + kThreads / p.L - 1) / (kThreads / p.L);
    // the sums over rows go into one row of a table per block: the blocks stay and walk on
    if (bwd && p.blocks > 4 * kSMs) p.blocks = 4 * kSMs;
    return p;
}

template <typename T, int L, bool BWD>
cudaError_t launch_pairs(const QkArgs& a, const Plan& p, cudaStream_t s) {
    const auto kernel = a.interleaved ? qk_kernel<T, L, kNeighbours, BWD>
                        : (a.rot / 2) % kV == 0 ? qk_kernel<T, L, kLanes, BWD>
                                                : qk_kernel<T, L, kShared, BWD>;
    constexpr int smem = (BWD ? 2 : 1) * Rows<T, BWD>::kSmem;
    const cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)p.blocks, kThreads, smem, s>>>(a, p.per, p.tokens, p.sets);
    return cudaGetLastError();
}

template <bool BWD>
cudaError_t launch(const QkArgs& a, const Plan& p, cudaStream_t s) {
    if (p.blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    const bool bf = a.dtype == GDN_BF16;
    switch (p.L) {
        case 1: return bf ? launch_pairs<__nv_bfloat16, 1, BWD>(a, p, s) : launch_pairs<float, 1, BWD>(a, p, s);
        case 2: return bf ? launch_pairs<__nv_bfloat16, 2, BWD>(a, p, s) : launch_pairs<float, 2, BWD>(a, p, s);
        case 4: return bf ? launch_pairs<__nv_bfloat16, 4, BWD>(a, p, s) : launch_pairs<float, 4, BWD>(a, p, s);
        case 8: return bf ? launch_pairs<__nv_bfloat16, 8, BWD>(a, p, s) : launch_pairs<float, 8, BWD>(a, p, s);
        case 16: return bf ? launch_pairs<__nv_bfloat16, 16, BWD>(a, p, s) : launch_pairs<float, 16, BWD>(a, p, s);
        case 32: return bf ? launch_pairs<__nv_bfloat16, 32, BWD>(a, p, s) : launch_pairs<float, 32, BWD>(a, p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t s) {
    return launch<false>(a, plan(a.T, a.heads[0], a.heads[1], a.d, false), s);
}

size_t qk_bwd_workspace_bytes(int T, int H, int H_k, int d) {
    return (size_t)plan(T, H, H_k, d, true).blocks * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t s) {
    const Plan p = plan(a.T, a.heads[0], a.heads[1], a.d, true);
    if (p.blocks > 0) {
        const cudaError_t e = launch<true>(a, p, s);
        if (e != cudaSuccess) return e;
    }
    return a.dw[0] || a.dw[1] ? launch_column_sum(a.partial, p.blocks, a.d, a.dw[0], a.dw[1], s) : cudaSuccess;
}

}  // namespace gdn

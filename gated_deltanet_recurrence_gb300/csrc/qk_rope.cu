// qk_rope.cu -- queries and keys normalised per head and rotated by their position, in one pass.
//
// "6.6 Gated DeltaNet", 6.6.4, normalises q and k per head before they meet the state; layers that also carry the
// token's position in them rotate pairs of channels.  With n = x / sqrt(mean x^2 + eps) (RMS norm) or
// x / sqrt(sum x^2 + eps) (length one), m = w n, and for pair i of the first d_rot channels
//   (u, v) -> (u cos_i - v sin_i, v cos_i + u sin_i),
// with cos_i, sin_i of the token's position from a table; the other channels pass.  Gradients: the rotation
// backwards, then dw = sum dm n, dn = dm w, dx = r (dn - n mean(dn n)) (or the sum's, for length one).
//
// Bound by memory.  A row (one head of one token) is d / 8 lanes of 8 channels; a set of lanes takes one token
// and several heads, so that the token's cosines and sines and the weights are loaded once.  Pairs of channels
// m = d_rot / 2 apart are exchanged by shuffles where they lie in the same place of another lane (m a multiple
// of 8), through shared memory otherwise.
#include "ssm_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kV = 8;
enum Pairs { kNeighbours, kLanes, kShared };

// Lanes of a row: the power of two that holds d / 8 vectors.
int lanes_of(int d) {
    int l = 1;
    while (l * kV < d) l *= 2;
    return l;
}

// Heads a set of lanes takes: all of a token's when there are tokens enough, fewer in small calls.
int heads_per_set(int T, int heads, int L) {
    const long sets = (long)kSMs * 4 * (kThreads / L);
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

// The rotation of one lane's eight channels; `sign` is -1 for the rotation backwards.  cs, sn: this lane's cosines and
// sines by channel (1 and 0 past d_rot), where sn has the sign with which the partner's value enters.
template <int L, Pairs PAIRS>
__device__ __forceinline__ void rotate(float (&x)[kV], const float (&cs)[kV], const float (&sn)[kV], int lane, int d, int m,
                                       float* row) {
    float y[kV];
    if constexpr (PAIRS == kNeighbours) {
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = x[j ^ 1];
    } else if constexpr (PAIRS == kLanes) {
        const int off = m / kV;
        const int from = lane < off ? lane + off : lane - off;  // lanes past d_rot get a value they do not use
#pragma unroll
        for (int j = 0; j < kV; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], from & (L - 1), L);
    } else {
        __syncwarp();
        if (lane * kV < d) {
#pragma unroll
            for (int j = 0; j < kV; ++j) row[lane * kV + j] = x[j];
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = lane * kV + j;
            y[j] = c < m ? row[c + m] : (c < 2 * m ? row[c - m] : 0.f);
        }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) x[j] = sn[j] == 0.f ? x[j] * cs[j] : fmaf(y[j], sn[j], x[j] * cs[j]);
}

// One block: kThreads / L sets; a set: one token, `per` heads of the q and k heads taken together.
template <typename T, int L, Pairs PAIRS, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_kernel(QkArgs a, int per, int parts, long sets) {
    __shared__ float stage[PAIRS == kShared ? kThreads * kV : 1];
    const int lane = threadIdx.x % L;
    const int c0 = lane * kV, d = a.d, m = a.rot / 2;
    const bool in = c0 < d;
    const float inv = a.l2 ? 1.0f : 1.0f / (float)d;
    float* row = stage + (PAIRS == kShared ? threadIdx.x / L * L * kV : 0);
    float w[2][kV], dw[2][kV];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < kV; ++j) { w[i][j] = 1.f; dw[i][j] = 0.f; }
        if (in && a.w[i]) load_row<kV>(a.w[i] + c0, w[i]);
    }
    // every set of a block makes the same number of passes: the shuffles and barriers of a warp stay together
    const long stride = (long)gridDim.x * (kThreads / L);
    for (long base = (long)blockIdx.x * (kThreads / L); base < sets; base += stride) {
        const long set = base + threadIdx.x / L;
        const int t = (int)(set / parts), part = (int)(set % parts);
        bool live = set < sets;
        float cs[kV], sn[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) { cs[j] = 1.f; sn[j] = 0.f; }
        if (live) {
            const long pos = a.positions ? (long)a.positions[t] : (long)t;
            if (pos < 0 || pos >= a.max_positions) {
                live = false;
                if (lane == 0) record_error(a.err, GDN_ERR_ARG);
            } else {
                const float* tab = a.cos_sin + pos * a.rot;
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
        const int h1 = min(a.heads[0] + a.heads[1], (part + 1) * per);
#pragma unroll 2
        for (int p = 0; p < per; ++p) {
            const int hh = part * per + p, i = hh >= a.heads[0], h = i ? hh - a.heads[0] : hh;
            const bool on = live && in && hh < h1;
            float x[kV], g[kV];
#pragma unroll
            for (int j = 0; j < kV; ++j) x[j] = g[j] = 0.f;
            if (on) {
                load_row<kV>(static_cast<const T*>(i ? a.x[1] : a.x[0]) + (long)t * (i ? a.x_stride[1] : a.x_stride[0]) + (long)h * d + c0, x);
                if (BWD) load_row<kV>(static_cast<const T*>(i ? a.dout[1] : a.dout[0]) + ((long)t * (i ? a.heads[1] : a.heads[0]) + h) * d + c0, g);
            }
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < kV; ++j) ss = fmaf(x[j], x[j], ss);
            const float r = rsqrtf(set_sum<L>(ss) * inv + a.eps);
            T* out = static_cast<T*>(i ? a.out[1] : a.out[0]) + (long)t * (i ? a.out_stride[1] : a.out_stride[0]) + (long)h * d + c0;
            if constexpr (!BWD) {
#pragma unroll
                for (int j = 0; j < kV; ++j) x[j] *= r * (i ? w[1][j] : w[0][j]);
                rotate<L, PAIRS>(x, cs, sn, lane, d, m, row);
                if (on) store_row<kV>(out, x);
            } else {
                rotate<L, PAIRS>(g, cs, sn, lane, d, m, row);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    x[j] *= r;
                    const float gn = on ? g[j] * x[j] : 0.f;
                    dw[0][j] += i ? 0.f : gn;
                    dw[1][j] += i ? gn : 0.f;
                    g[j] *= i ? w[1][j] : w[0][j];
                    dot = fmaf(g[j], x[j], dot);
                }
                dot = set_sum<L>(dot) * inv;
#pragma unroll
                for (int j = 0; j < kV; ++j) g[j] = r * (g[j] - x[j] * dot);
                if (on) store_row<kV>(out, g);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.partial) return;
        // the block's sets are added in order; its row of the table is [q's d, k's d]
        __shared__ float sums[kThreads / L][2][L * kV];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) sums[threadIdx.x / L][i][c0 + j] = dw[i][j];
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
    int L, per, parts;
    long sets, blocks;
};
Plan plan(int T, int H, int H_k, int d, bool bwd) {
    Plan p;
    p.L = lanes_of(d);
    p.per = heads_per_set(T, H + H_k, p.L);
    p.parts = (H + H_k + p.per - 1) / p.per;
    p.sets = (long)T * p.parts;
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
    kernel<<<(unsigned)p.blocks, kThreads, 0, s>>>(a, p.per, p.parts, p.sets);
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

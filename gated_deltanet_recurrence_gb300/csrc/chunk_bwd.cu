// chunk_bwd.cu -- gradients of the chunked gated delta rule (gdn_chunk_bwd).
//
// Forward, per chunk of C = 64 tokens (chunk form of "5. 线性注意力", "Delta Rule 的 Chunk 实现"), with
// G the inclusive sum of g in the chunk, b = e^G, D_ij = e^(G_i - G_j) for j <= i and 0 above, q and k
// normalised (q scaled), S0 the state at the chunk's start:
//   A = strictly lower part of diag(beta) (K K^T * D),   T = (I + A)^-1,
//   W = T diag(beta b) K,   U = T diag(beta) V - W S0^T,   P = Q K^T * D,
//   Y = diag(b) Q S0^T + P U,   S1 = b_C S0 + U^T Kd   with Kd = diag(b_C / b) K.
// Put together, a chunk maps its start state affinely, and the adjoint maps dS1 back the same way:
//   S1  = S0 M + B,       M = b_C I - W^T Kd,   B = (T diag(beta) V)^T Kd,
//   dS0 = dS1 M^T + X,    X = dY^T (diag(b) Q - P W).
// Adjoint inside a chunk, given S0 and dS1:
//   dR = T^T (P^T dY + Kd dS1^T),       dV = diag(beta) dR,
//   dP = (dY U^T) * D,                  Z = -strictly lower part of (dR U^T) * D,
//   dQ  = diag(b) dY S0 + dP K,
//   dK+ = diag(beta) E,  E = Z K - diag(b) dR S0,
//   dK- = H + dP^T Q + Z^T diag(beta) K,  H = diag(b_C / b) U dS1,    dK = dK+ + dK-,
//   dbeta_i = dR_i . v_i + E_i . k_i,
//   dg_i = sum over j >= i of (dQ_j . q_j + dK+_j . k_j - (dK- - H)_j . k_j)
//          + sum over j < i of H_j . k_j + b_C <S0, dS1>.
// (Each row dot with q or k collects the terms in which that row's e^G or e^-G enters.  The diagonal
// of P carries e^0: its two contributions cancel, so it is kept out of these dots and a token that
// decays nothing gets dg = 0 exactly.)
//
// Three kernels: the chunks' own quantities (T, M, B, X), all chunks at once; the two affine
// recurrences over the chunks of a sequence, forwards for S0 and backwards for dS1, which replace B
// and X; the chunks' gradients, all chunks at once.  With grouped heads the gradients of q and k go to
// fp32 scratch per value head, and a fourth kernel adds the heads of a group in order.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kC = 64;
constexpr int kThreads = 256;

// ---- the chunk slots ---------------------------------------------------------------------------
// Chunk c of sequence n has slot base(n) + c.  With lengths from cu_seqlens base(n) = cu[n] / 64 + n
// leaves every sequence at least as many slots as it has chunks; unused slots do nothing.  With equal
// lengths base(n) = n * chunks per sequence.
struct Span {
    long bos, eos;   // the sequence's tokens
    int n, c;        // sequence and chunk; n < 0: an unused slot or a malformed cu_seqlens
    int chunks;      // of the sequence
};

__host__ __device__ __forceinline__ long slot_count(int num_seqs, int total_T) {
    return (long)total_T / kC + num_seqs;
}

// Whether cu_seqlens is monotone and inside [0, total_T] (all threads; contains a block barrier).
__device__ bool cu_valid(const ChunkBwdArgs& a) {
    if (!a.cu_seqlens) return true;
    bool bad = false;
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) {
        const int lo = a.cu_seqlens[i], hi = a.cu_seqlens[i + 1];
        bad |= lo < 0 || hi < lo || hi > a.total_T;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) record_error(a.err, GDN_ERR_CU_SEQLENS);
        return false;
    }
    return true;
}

__device__ __forceinline__ void seq_span(const ChunkBwdArgs& a, int n, Span& s, long& base) {
    if (a.cu_seqlens) {
        s.bos = a.cu_seqlens[n];
        s.eos = a.cu_seqlens[n + 1];
        base = s.bos / kC + n;
    } else {
        const long len = a.total_T / a.num_seqs;
        s.bos = n * len;
        s.eos = s.bos + len;
        base = n * ((len + kC - 1) / kC);
    }
    s.n = n;
    s.chunks = (int)((s.eos - s.bos + kC - 1) / kC);
}

// The span of a slot; needs a valid cu_seqlens.
__device__ Span find_span(const ChunkBwdArgs& a, long slot) {
    Span s;
    long base;
    int lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {  // the last sequence whose base is <= slot
        const int mid = (lo + hi + 1) / 2;
        seq_span(a, mid, s, base);
        if (base <= slot) lo = mid;
        else hi = mid - 1;
    }
    seq_span(a, lo, s, base);
    s.c = (int)(slot - base);
    if (s.c < 0 || s.c >= s.chunks) s.n = -1;
    return s;
}

// ---- workspace ---------------------------------------------------------------------------------
// Per (slot, head): T [64, 64], M [d, d], B then S0 [d, d], X then dS1 [d, d], fp32.
struct Work {
    float *T, *M, *S, *dS;   // arrays over (slot, head)
    float *dq, *dk;          // [total_T, H, d] each, grouped heads only
};

__host__ __device__ __forceinline__ Work work_of(void* ws, long units, long tokens, int d) {
    Work w;
    w.T = static_cast<float*>(ws);
    w.M = w.T + units * kC * kC;
    w.S = w.M + units * d * d;
    w.dS = w.S + units * d * d;
    w.dq = w.dS + units * d * d;
    w.dk = w.dq + tokens * d;
    return w;
}

__device__ __forceinline__ float load_elem(const void* p, gdn_dtype dt, long i) {
    return dt == GDN_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// The chunk's cumulative log-decays and the factors made of them, in shared memory.
struct Gates {
    float G[kC], b[kC], tail[kC], beta[kC];  // tail = b_C / b
};

__device__ void load_gates(const ChunkBwdArgs& a, Gates& t, long t0, int len, int h) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, i0 = 2 * lane, i1 = i0 + 1;
        const float g0 = i0 < len ? a.g[(t0 + i0) * a.H + h] : 0.f;
        const float g1 = i1 < len ? a.g[(t0 + i1) * a.H + h] : 0.f;
        float s = g0 + g1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        const float last = __shfl_sync(0xffffffffu, s, 31), c0 = s - g1;
        t.G[i0] = c0; t.G[i1] = s;
        t.b[i0] = expf(c0); t.b[i1] = expf(s);
        t.tail[i0] = expf(last - c0); t.tail[i1] = expf(last - s);
        t.beta[i0] = i0 < len ? a.beta[(t0 + i0) * a.H + h] : 0.f;
        t.beta[i1] = i1 < len ? a.beta[(t0 + i1) * a.H + h] : 0.f;
    }
}

// A chunk of a token tensor [T, heads, D] as fp32 rows of D words; zeros past the sequence's end.
template <int D>
__device__ void load_tile(float* dst, const void* src, gdn_dtype dt, long t0, int len, int heads, int h) {
    for (int i = threadIdx.x; i < kC * D; i += kThreads) {
        const int r = i / D, x = i % D;
        dst[i] = r < len ? load_elem(src, dt, ((t0 + r) * heads + h) * D + x) : 0.f;
    }
}

// Normalises the rows of a tile; inv receives each row's factor (without the scale).
template <int D>
__device__ void normalise(float* tile, float* inv, int use_l2, float scale) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < kC; r += kThreads / 32) {
        float ss = 0.f;
        for (int x = lane; x < D; x += 32) ss += tile[r * D + x] * tile[r * D + x];
        ss = warp_sum(ss);
        const float f = use_l2 ? rsqrtf(ss + kL2Eps) : 1.f;
        for (int x = lane; x < D; x += 32) tile[r * D + x] *= f * scale;
        if (lane == 0) inv[r] = f;
    }
}

// Entry (i, j) of a 64 x 64 product of rows: x_i . y_j over D.
template <int D>
__device__ __forceinline__ float dot_rows(const float* x, int i, const float* y, int j) {
    float s = 0.f;
    for (int e = 0; e < D; ++e) s = fmaf(x[i * D + e], y[j * D + e], s);
    return s;
}

// ---- chunk quantities ----------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_bwd_prep_kernel(ChunkBwdArgs a, Work w) {
    extern __shared__ float sm[];
    __shared__ Gates t;
    __shared__ float inv[kC];
    float *Q = sm, *K = Q + kC * D, *V = K + kC * D, *Y = V + kC * D, *W = Y + kC * D, *U = W + kC * D;
    float *A = U + kC * D, *T = A + kC * kC;
    if (!cu_valid(a)) return;
    const long slot = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hk), tid = threadIdx.x;
    const Span s = find_span(a, slot);
    if (s.n < 0) return;
    const long t0 = s.bos + (long)s.c * kC;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    load_gates(a, t, t0, len, h);
    load_tile<D>(Q, a.q, a.qkv_dtype, t0, len, a.Hk, hk);
    load_tile<D>(K, a.k, a.qkv_dtype, t0, len, a.Hk, hk);
    load_tile<D>(V, a.v, a.qkv_dtype, t0, len, a.H, h);
    load_tile<D>(Y, a.dout, a.dout_dtype, t0, len, a.H, h);
    __syncthreads();
    normalise<D>(Q, inv, a.use_l2, a.scale);
    normalise<D>(K, inv, a.use_l2, 1.f);
    __syncthreads();
    for (int e = tid; e < kC * kC; e += kThreads) {
        const int i = e / kC, j = e % kC;
        A[e] = j < i ? t.beta[i] * dot_rows<D>(K, i, K, j) * expf(t.G[i] - t.G[j]) : 0.f;
        T[e] = i == j ? 1.f : 0.f;
    }
    __syncthreads();
    // rows of T by substitution: T_ij = -A_ij - sum over j < m < i of A_im T_mj
    for (int i = 1; i < kC; ++i) {
        if (tid < i) {
            float acc = A[i * kC + tid];
            for (int m = tid + 1; m < i; ++m) acc = fmaf(A[i * kC + m], T[m * kC + tid], acc);
            T[i * kC + tid] = -acc;
        }
        __syncthreads();
    }
    const long unit = slot * a.H + h;
    for (int e = tid; e < kC * kC; e += kThreads) {
        const int i = e / kC, j = e % kC;
        w.T[unit * kC * kC + e] = T[e];
        A[e] = j <= i ? dot_rows<D>(Q, i, K, j) * expf(t.G[i] - t.G[j]) : 0.f;  // P from here on
    }
    for (int e = tid; e < kC * D; e += kThreads) {
        const int i = e / D, x = e % D;
        float sw = 0.f, su = 0.f;
        for (int j = 0; j <= i; ++j) {
            const float f = T[i * kC + j] * t.beta[j];
            sw = fmaf(f * t.b[j], K[j * D + x], sw);
            su = fmaf(f, V[j * D + x], su);
        }
        W[e] = sw;
        U[e] = su;
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // Q becomes diag(b) Q - P W
        const int i = e / D, x = e % D;
        float acc = t.b[i] * Q[e];
        for (int j = 0; j <= i; ++j) acc = fmaf(-A[i * kC + j], W[j * D + x], acc);
        Q[e] = acc;
    }
    __syncthreads();
    for (int e = tid; e < D * D; e += kThreads) {
        const int r = e / D, x = e % D;
        float m = r == x ? t.b[kC - 1] : 0.f, b = 0.f, g = 0.f;
        for (int j = 0; j < kC; ++j) {
            const float kd = t.tail[j] * K[j * D + x];
            m = fmaf(-W[j * D + r], kd, m);
            b = fmaf(U[j * D + r], kd, b);
            g = fmaf(Y[j * D + r], Q[j * D + x], g);
        }
        w.M[unit * D * D + e] = m;
        w.S[unit * D * D + e] = b;
        w.dS[unit * D * D + e] = g;
    }
}

// ---- the two recurrences over a sequence's chunks ----------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_bwd_scan_kernel(ChunkBwdArgs a, Work w) {
    extern __shared__ float sm[];
    float *S = sm, *N = sm + D * D;
    if (!cu_valid(a)) return;
    const int n = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
    const bool back = blockIdx.y != 0;
    Span s;
    long base;
    seq_span(a, n, s, base);
    const long state = ((long)n * a.H + h) * D * D;
    const float* from = back ? a.dfinal_state : a.initial_state;
    for (int e = tid; e < D * D; e += kThreads) S[e] = from ? from[state + e] : 0.f;
    __syncthreads();
    for (int i = 0; i < s.chunks; ++i) {
        const long unit = (base + (back ? s.chunks - 1 - i : i)) * a.H + h;
        const float* M = w.M + unit * D * D;
        float* add = (back ? w.dS : w.S) + unit * D * D;
        for (int e = tid; e < D * D; e += kThreads) {
            const int r = e / D, x = e % D;
            float acc = add[e];
            for (int y = 0; y < D; ++y) acc = fmaf(S[r * D + y], back ? M[x * D + y] : M[y * D + x], acc);
            N[e] = acc;
        }
        __syncthreads();
        for (int e = tid; e < D * D; e += kThreads) {
            add[e] = S[e];
            S[e] = N[e];
        }
        __syncthreads();
    }
    if (back && a.dinitial_state)
        for (int e = tid; e < D * D; e += kThreads) a.dinitial_state[state + e] = S[e];
}

// ---- gradients -----------------------------------------------------------------------------------

// Gradient of one row through x -> scale * x * inv: dx = scale * inv * (d - n (n . d)), n = x * inv.
// xh = scale * n is the forward row, dot = d . xh.
__device__ __forceinline__ float unnormalise(float d, float xh, float dot, float inv, float scale, int use_l2) {
    return use_l2 ? scale * inv * (d - xh * (dot / (scale * scale))) : scale * d;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_bwd_grad_kernel(ChunkBwdArgs a, Work w) {
    extern __shared__ float sm[];
    __shared__ Gates t;
    __shared__ float qinv[kC], kinv[kC], qdot[kC], kpos[kC], kneg[kC], hdot[kC], dpp[kC], diag[kC];
    float *Q = sm, *K = Q + kC * D, *Y = K + kC * D, *U = Y + kC * D, *R = U + kC * D, *X = R + kC * D;
    float *P = X + kC * D, *Z = P + kC * kC;
    if (!cu_valid(a)) return;
    const long slot = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, rep = a.H / a.Hk, hk = h / rep, tid = threadIdx.x;
    const Span s = find_span(a, slot);
    if (s.n < 0) return;
    const long t0 = s.bos + (long)s.c * kC;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const long unit = slot * a.H + h;
    const float* T = w.T + unit * kC * kC;
    const float* S0 = w.S + unit * D * D;
    const float* dS1 = w.dS + unit * D * D;
    load_gates(a, t, t0, len, h);
    load_tile<D>(Q, a.q, a.qkv_dtype, t0, len, a.Hk, hk);
    load_tile<D>(K, a.k, a.qkv_dtype, t0, len, a.Hk, hk);
    load_tile<D>(Y, a.dout, a.dout_dtype, t0, len, a.H, h);
    __syncthreads();
    normalise<D>(Q, qinv, a.use_l2, a.scale);
    normalise<D>(K, kinv, a.use_l2, 1.f);
    __syncthreads();
    for (int e = tid; e < kC * kC; e += kThreads) {
        const int i = e / kC, j = e % kC;
        P[e] = j <= i ? dot_rows<D>(Q, i, K, j) * expf(t.G[i] - t.G[j]) : 0.f;
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // X = P^T dY + Kd dS1^T
        const int i = e / D, r = e % D;
        float acc = 0.f;
        for (int x = 0; x < D; ++x) acc = fmaf(K[i * D + x], dS1[r * D + x], acc);
        acc *= t.tail[i];
        for (int j = i; j < kC; ++j) acc = fmaf(P[j * kC + i], Y[j * D + r], acc);
        X[e] = acc;
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // dR = T^T X
        const int i = e / D, r = e % D;
        float acc = 0.f;
        for (int j = i; j < kC; ++j) acc = fmaf(T[j * kC + i], X[j * D + r], acc);
        R[e] = acc;
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // X = diag(beta) (V - diag(b) K S0^T)
        const int i = e / D, r = e % D;
        float acc = 0.f;
        for (int x = 0; x < D; ++x) acc = fmaf(K[i * D + x], S0[r * D + x], acc);
        const float v = i < len ? load_elem(a.v, a.qkv_dtype, ((t0 + i) * a.H + h) * D + r) : 0.f;
        X[e] = t.beta[i] * (v - t.b[i] * acc);
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // U = T X
        const int i = e / D, r = e % D;
        float acc = 0.f;
        for (int j = 0; j <= i; ++j) acc = fmaf(T[i * kC + j], X[j * D + r], acc);
        U[e] = acc;
    }
    __syncthreads();
    for (int e = tid; e < kC * kC; e += kThreads) {  // P becomes dP
        const int i = e / kC, j = e % kC;
        const float dec = j <= i ? expf(t.G[i] - t.G[j]) : 0.f;
        const float n = j <= i ? dot_rows<D>(Y, i, U, j) * dec : 0.f;
        if (i == j) {
            dpp[i] = n;
            diag[i] = n * P[e];  // dP_ii q_i . k_i
        }
        P[e] = j < i ? n : 0.f;
        Z[e] = j < i ? -dot_rows<D>(R, i, U, j) * dec : 0.f;
    }
    // X: the row dots need whole rows of dQ, dK+ / beta, dK-, H: four passes through one buffer
    const int warp = tid >> 5, lane = tid & 31;
    float state_dot = 0.f;
    for (int e = tid; e < D * D; e += kThreads) state_dot = fmaf(S0[e], dS1[e], state_dot);
    state_dot = warp_sum(state_dot);
    __syncthreads();
    float* red = Z + 1;  // in the part of Z's first row that is above the diagonal, which nothing reads
    if (lane == 0) red[warp] = state_dot;
    __syncthreads();
    auto row_dots = [&](const float* x, const float* y, float* out) {
        for (int r = warp; r < kC; r += kThreads / 32) {
            float v = 0.f;
            for (int e = lane; e < D; e += 32) v = fmaf(x[r * D + e], y[r * D + e], v);
            v = warp_sum(v);
            if (lane == 0) out[r] = v;
        }
    };
    for (int r = warp; r < kC; r += kThreads / 32) {  // dV, and dR . v
        float v = 0.f;
        for (int e = lane; e < D && r < len; e += 32) {
            const long at = ((t0 + r) * a.H + h) * D + e;
            const float x = R[r * D + e];
            v = fmaf(x, load_elem(a.v, a.qkv_dtype, at), v);
            store_out(a.dv, at, a.qkv_dtype, t.beta[r] * x);
        }
        v = warp_sum(v);
        if (lane == 0) hdot[r] = v;  // kept until dbeta below
    }
    for (int e = tid; e < kC * D; e += kThreads) {  // dQ
        const int i = e / D, x = e % D;
        float acc = 0.f;
        for (int r = 0; r < D; ++r) acc = fmaf(Y[i * D + r], S0[r * D + x], acc);
        acc *= t.b[i];
        for (int j = 0; j < i; ++j) acc = fmaf(P[i * kC + j], K[j * D + x], acc);
        X[e] = acc;
    }
    __syncthreads();
    row_dots(X, Q, qdot);
    __syncthreads();
    for (int e = tid; e < len * D; e += kThreads) {
        const int i = e / D, x = e % D;
        const float d = unnormalise(fmaf(dpp[i], K[e], X[e]), Q[e], qdot[i] + diag[i], qinv[i], a.scale, a.use_l2);
        if (rep > 1) w.dq[((t0 + i) * a.H + h) * D + x] = d;
        else store_out(a.dq, ((t0 + i) * a.Hk + hk) * D + x, a.qkv_dtype, d);
    }
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // E
        const int i = e / D, x = e % D;
        float acc = 0.f;
        for (int r = 0; r < D; ++r) acc = fmaf(R[i * D + r], S0[r * D + x], acc);
        acc *= -t.b[i];
        for (int j = 0; j < i; ++j) acc = fmaf(Z[i * kC + j], K[j * D + x], acc);
        X[e] = acc;
    }
    __syncthreads();
    row_dots(X, K, kpos);
    __syncthreads();
    if (tid < kC && tid < len) a.dbeta[(t0 + tid) * a.H + h] = hdot[tid] + kpos[tid];
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // R = H
        const int i = e / D, x = e % D;
        float acc = 0.f;
        for (int r = 0; r < D; ++r) acc = fmaf(U[i * D + r], dS1[r * D + x], acc);
        R[e] = acc * t.tail[i];
    }
    __syncthreads();
    row_dots(R, K, hdot);
    __syncthreads();
    for (int e = tid; e < kC * D; e += kThreads) {  // U = dK- - H without P's diagonal
        const int i = e / D, x = e % D;
        float acc = 0.f;
        for (int j = i + 1; j < kC; ++j) acc = fmaf(P[j * kC + i], Q[j * D + x], acc);
        for (int j = i + 1; j < kC; ++j) acc = fmaf(Z[j * kC + i] * t.beta[j], K[j * D + x], acc);
        U[e] = acc;
    }
    __syncthreads();
    row_dots(U, K, kneg);
    __syncthreads();
    for (int e = tid; e < len * D; e += kThreads) {
        const int i = e / D, x = e % D;
        const float dot = t.beta[i] * kpos[i] + kneg[i] + hdot[i] + diag[i];
        const float sum = t.beta[i] * X[e] + U[e] + R[e] + dpp[i] * Q[e];
        const float d = unnormalise(sum, K[e], dot, kinv[i], 1.f, a.use_l2);
        if (rep > 1) w.dk[((t0 + i) * a.H + h) * D + x] = d;
        else store_out(a.dk, ((t0 + i) * a.Hk + hk) * D + x, a.qkv_dtype, d);
    }
    if (tid == 0) {
        float acc = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) acc += red[i];
        acc *= t.b[kC - 1];
        for (int i = kC - 1; i >= 0; --i) {
            acc += qdot[i] + t.beta[i] * kpos[i] - kneg[i];
            qdot[i] = acc;
        }
        float before = 0.f;
        for (int i = 0; i < len; ++i) {
            a.dg[(t0 + i) * a.H + h] = qdot[i] + before;
            before += hdot[i];
        }
    }
}

// dq, dk of grouped heads: the sum over the group's value heads, in order.  Tokens outside every
// sequence are left as they were.
__global__ void __launch_bounds__(kThreads) chunk_bwd_heads_kernel(ChunkBwdArgs a, Work w) {
    if (!cu_valid(a)) return;
    const int rep = a.H / a.Hk;
    const long first = a.cu_seqlens ? a.cu_seqlens[0] : 0;
    const long end = a.cu_seqlens ? a.cu_seqlens[a.num_seqs] : a.total_T;
    const long per = (long)a.Hk * a.d;
    for (long i = first * per + (long)blockIdx.x * kThreads + threadIdx.x; i < end * per;
         i += (long)gridDim.x * kThreads) {
        const long row = i / a.d;  // token * Hk + hk
        const long at = row * rep * a.d + i % a.d;
        float sq = 0.f, sk = 0.f;
        for (int j = 0; j < rep; ++j) {
            sq += w.dq[at + (long)j * a.d];
            sk += w.dk[at + (long)j * a.d];
        }
        store_out(a.dq, i, a.qkv_dtype, sq);
        store_out(a.dk, i, a.qkv_dtype, sk);
    }
}

template <int D>
cudaError_t launch(const ChunkBwdArgs& a, cudaStream_t s) {
    const long units = slot_count(a.num_seqs, a.total_T) * a.H;
    const Work w = work_of(a.workspace, units, (long)a.total_T * a.H, D);
    const int tile = (6 * kC * D + 2 * kC * kC) * (int)sizeof(float);
    const int states = 2 * D * D * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(chunk_bwd_prep_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, tile);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_bwd_grad_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, tile);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_bwd_scan_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, states);
    if (e != cudaSuccess) return e;
    if (a.total_T > 0) {
        chunk_bwd_prep_kernel<D><<<(unsigned)units, kThreads, tile, s>>>(a, w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    chunk_bwd_scan_kernel<D><<<dim3((unsigned)(a.num_seqs * a.H), 2), kThreads, states, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess || a.total_T == 0) return e;
    chunk_bwd_grad_kernel<D><<<(unsigned)units, kThreads, tile, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess || a.H == a.Hk) return e;
    chunk_bwd_heads_kernel<<<152 * 8, kThreads, 0, s>>>(a, w);
    return cudaGetLastError();
}

}  // namespace

size_t chunk_bwd_workspace_bytes(int num_seqs, int total_T, int H, int Hk, int d) {
    const size_t units = (size_t)slot_count(num_seqs, total_T) * H;
    const size_t words = units * (kC * kC + 3 * (size_t)d * d) + (H > Hk ? 2 * (size_t)total_T * H * d : 0);
    return words * sizeof(float);
}

cudaError_t launch_chunk_bwd(const ChunkBwdArgs& a, cudaStream_t s) {
    return a.d == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace gdn

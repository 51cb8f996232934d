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
// Every product is taken on the tensor cores from fp16 planes at fp32 accuracy (mma_planes.cuh); what is
// between the products is fp32.
//
// Three kernels: the chunks' own quantities (T, M, B, X), all chunks at once; the two affine
// recurrences over the chunks of a sequence, forwards for S0 and backwards for dS1, which replace B
// and X; the chunks' gradients, all chunks at once.  With grouped heads the gradients of q and k go to
// fp32 scratch per value head, and a fourth kernel adds the heads of a group in order.
#include "gdn_internal.cuh"
#include "mma_planes.cuh"

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

using planes::Mat;
using planes::Scale;

// ---- workspace ---------------------------------------------------------------------------------
// Per (slot, head): the planes of T (64 x 64) and of M (d x d) as they lie in shared memory, B then S0
// and X then dS1 (d x d, fp32), and a few words beside them.
struct Meta {
    float t_scale, m_scale;
    uint32_t s_max[8], ds_max[8];  // bits of the largest magnitude in each 16 rows of S0 and dS1
    uint32_t pad[14];
};
static_assert(sizeof(Meta) == 128, "");

struct Work {
    unsigned char *T, *M;
    float *S, *dS;
    Meta* meta;
    float *dq, *dk;  // [total_T, H, d] each, grouped heads only
};

constexpr size_t kTBytes = 2 * kC * kC * sizeof(__half);
__host__ __device__ constexpr size_t m_bytes(int d) { return 2 * (size_t)d * d * sizeof(__half); }

__host__ __device__ __forceinline__ Work work_of(void* ws, long units, long tokens, int d) {
    Work w;
    w.T = static_cast<unsigned char*>(ws);
    w.M = w.T + units * kTBytes;
    w.S = reinterpret_cast<float*>(w.M + units * m_bytes(d));
    w.dS = w.S + units * d * d;
    w.meta = reinterpret_cast<Meta*>(w.dS + units * d * d);
    w.dq = reinterpret_cast<float*>(w.meta + units);
    w.dk = w.dq + tokens * d;
    return w;
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

// Four consecutive elements of a q/k/v-like tensor.
__device__ __forceinline__ void load4(const void* src, gdn_dtype dt, long i, float (&x)[4]) {
    if (dt == GDN_BF16) load_vec<4>(static_cast<const __nv_bfloat16*>(src) + i, x);
    else load_vec<4>(static_cast<const float*>(src) + i, x);
}

// A chunk of a token tensor [T, heads, D] as P planes (P = 1 takes bf16 only, which one plane holds
// exactly), each row with a power of two of its own; zeros past the sequence's end.  factor[r] takes
// row r of the planes to x (norm false), or to scale * x / |x| (norm and use_l2) and scale * x (norm,
// not use_l2); inv[r] receives 1 / |x| (1 without).  Rows of a factor that later products fold into a
// contraction must not differ by much: with use_l2 their size is set by the norm, without it (common)
// all rows share the largest row's power of two, in which case the block synchronises on *top.
template <int D, int P>
__device__ void load_rows(Mat dst, const void* src, gdn_dtype dt, long t0, int len, int heads, int h, float* factor,
                          float* inv, bool norm, bool use_l2, float scale, uint32_t* top) {
    constexpr int LPR = D / 4, RPP = 32 / LPR, N = kC / (kThreads / 32) / RPP;  // lanes a row, rows a pass, passes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR;
    float x[N][4];
    uint32_t big[N];
    float ss[N];
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const int r = (p * (kThreads / 32) + warp) * RPP + lane / LPR;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[p][e] = 0.f;
        if (r < len) load4(src, dt, ((t0 + r) * heads + h) * D + 4 * l, x[p]);
    }
    uint32_t all = 0;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        ss[p] = 0.f;
        big[p] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ss[p] = fmaf(x[p][e], x[p][e], ss[p]);
            big[p] = max(big[p], planes::abs_bits(x[p][e]));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            ss[p] += __shfl_xor_sync(0xffffffffu, ss[p], o);
            big[p] = max(big[p], __shfl_xor_sync(0xffffffffu, big[p], o));
        }
        all = max(all, big[p]);
    }
    const bool common = norm && !use_l2;
    if (common) {
        atomicMax(top, all);
        __syncthreads();
        all = *top;
    }
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const int r = (p * (kThreads / 32) + warp) * RPP + lane / LPR;
        const Scale s = planes::scale_of(common ? all : big[p]);
        uint32_t hi[2], lo[2];
        planes::split(x[p][0] * s.mul, x[p][1] * s.mul, hi[0], lo[0]);
        planes::split(x[p][2] * s.mul, x[p][3] * s.mul, hi[1], lo[1]);
        const uint32_t at = dst.at + planes::offset<D>(r, 4 * l);
        planes::sts64(at, hi[0], hi[1]);
        if constexpr (P == 2) planes::sts64(at + dst.lo, lo[0], lo[1]);
        if (l == 0) {
            const float f = norm && use_l2 ? rsqrtf(ss[p] + kL2Eps) : 1.f;
            factor[r] = (norm ? f * scale : 1.f) * s.back;
            if (inv) inv[r] = f;
        }
    }
}

// Largest of the block's eight warp maxima (a barrier lies between their writes and this).
__device__ __forceinline__ uint32_t top_of(const uint32_t* red) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, red[i]);
    return m;
}

// ---- chunk quantities ----------------------------------------------------------------------------

// Index of (i, j) in a 64 x 64 fp32 matrix whose columns are XORed by the row: rows and columns are
// both read without bank conflicts.
__device__ __forceinline__ int at64(int i, int j) { return i * kC + (j ^ (i & 31)); }

// X = (I + A)^-1 for strictly lower triangular A (both at64; X's upper triangle is scratch): the four
// 16 x 16 diagonal blocks by substitution, a warp each and a column a lane, then twice the block below
// two inverted neighbours, X21 = -X22 (A21 X11).
__device__ void unit_lower_inverse(const float* A, float* X) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp < 4 && lane < 16) {
        const int o = 16 * warp;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) acc = fmaf(-A[at64(o + i, o + m)], x[m], acc);
            x[i] = acc;
            if (i >= lane) X[at64(o + i, o + lane)] = acc;
        }
    }
    __syncthreads();
    for (int e = tid; e < 512; e += kThreads) {  // two pairs of 16-blocks
        const int o = (e >> 8) * 32, r = (e >> 4) & 15, c = e & 15;
        float acc = 0.f;
        for (int m = c; m < 16; ++m) acc = fmaf(A[at64(o + 16 + r, o + m)], X[at64(o + m, o + c)], acc);
        X[at64(o + r, o + 16 + c)] = acc;
    }
    __syncthreads();
    for (int e = tid; e < 512; e += kThreads) {
        const int o = (e >> 8) * 32, r = (e >> 4) & 15, c = e & 15;
        float acc = 0.f;
        for (int m = 0; m <= r; ++m) acc = fmaf(-X[at64(o + 16 + r, o + 16 + m)], X[at64(o + m, o + 16 + c)], acc);
        X[at64(o + 16 + r, o + c)] = acc;
    }
    __syncthreads();
    for (int e = tid; e < 1024; e += kThreads) {  // the pair of 32-blocks
        const int r = e >> 5, c = e & 31;
        float acc = 0.f;
        for (int m = 0; m < 32; ++m) {
            const float x = X[at64(m, c)];
            acc = fmaf(A[at64(32 + r, m)], m >= c ? x : 0.f, acc);
        }
        X[at64(r, 32 + c)] = acc;
    }
    __syncthreads();
    for (int e = tid; e < 1024; e += kThreads) {
        const int r = e >> 5, c = e & 31;
        float acc = 0.f;
        for (int m = 0; m <= r; ++m) acc = fmaf(-X[at64(32 + r, 32 + m)], X[at64(m, 32 + c)], acc);
        X[at64(32 + r, c)] = acc;
    }
    __syncthreads();
}

// Sixteen consecutive elements of row r from column c, times mul and the factors of the columns, into
// the planes of a 64 x 64 matrix in shared memory and, if given, into its image in global memory.
__device__ __forceinline__ void put16(Mat dst, unsigned char* image, int r, int c, const float (&x)[16]) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) planes::split(x[2 * i], x[2 * i + 1], hi[i], lo[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t o = planes::offset<kC>(r, c + 8 * i);
        if (image) {
            *reinterpret_cast<uint4*>(image + o) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
            *reinterpret_cast<uint4*>(image + kTBytes / 2 + o) =
                make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        } else {
            planes::sts64(dst.at + o, hi[4 * i], hi[4 * i + 1]);
            planes::sts64(dst.at + o + 8, hi[4 * i + 2], hi[4 * i + 3]);
            planes::sts64(dst.at + dst.lo + o, lo[4 * i], lo[4 * i + 1]);
            planes::sts64(dst.at + dst.lo + o + 8, lo[4 * i + 2], lo[4 * i + 3]);
        }
    }
}

// Shared memory of the preparation: K, dY, V, Q (P planes each; the planes of Q' replace V and Q), P and
// one 64 x 64 matrix made of T, then W and U (two planes each; before, A and T in fp32).
template <int D, int P>
struct PrepSmem {
    static constexpr uint32_t plane = kC * D * 2, square = kC * kC * 2;
    static constexpr uint32_t K = 0, Y = P * plane, V = 2 * P * plane, Q = 3 * P * plane;
    static constexpr uint32_t Pm = 4 * P * plane, TX = Pm + 2 * square, W = TX + 2 * square, U = W + 2 * plane;
    static constexpr uint32_t bytes = U + 2 * plane;
};

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1) chunk_bwd_prep_kernel(ChunkBwdArgs a, Work w) {
    using L = PrepSmem<D, P>;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ Gates t;
    __shared__ float fK[kC], fQ[kC], fY[kC], fV[kC];
    __shared__ uint32_t red[9][8], tops[2];
    if (!cu_valid(a)) return;
    const long slot = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hk), tid = threadIdx.x;
    const Span s = find_span(a, slot);
    if (s.n < 0) return;
    const long t0 = s.bos + (long)s.c * kC, unit = slot * a.H + h;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const Mat K{base + L::K, L::plane}, Y{base + L::Y, L::plane}, V{base + L::V, L::plane}, Q{base + L::Q, L::plane};
    const Mat Qp{base + L::V, L::plane}, Pm{base + L::Pm, L::square}, TX{base + L::TX, L::square};
    const Mat W{base + L::W, L::plane}, U{base + L::U, L::plane};
    float *Af = reinterpret_cast<float*>(sm + L::W), *Tf = reinterpret_cast<float*>(sm + L::U);

    if (tid < 2) tops[tid] = 0;
    load_gates(a, t, t0, len, h);
    __syncthreads();
    load_rows<D, P>(K, a.k, a.qkv_dtype, t0, len, a.Hk, hk, fK, nullptr, true, a.use_l2, 1.f, &tops[0]);
    load_rows<D, P>(Q, a.q, a.qkv_dtype, t0, len, a.Hk, hk, fQ, nullptr, true, a.use_l2, a.scale, &tops[1]);
    load_rows<D, P>(V, a.v, a.qkv_dtype, t0, len, a.H, h, fV, nullptr, false, false, 1.f, nullptr);
    load_rows<D, P>(Y, a.dout, a.dout_dtype, t0, len, a.H, h, fY, nullptr, false, false, 1.f, nullptr);
    __syncthreads();

    // Warps 2 x 4 over a 64-row result.  A warp's two row tiles are mw and 3 - mw, which gives both rows
    // of warps the same share of a triangular product.
    const int warp = tid >> 5, lane = tid & 31, mw = warp >> 2, nw = warp & 3;
    const int m[2] = {16 * mw, 16 * (3 - mw)};
    constexpr int NT = D / 32;
    const int nd = nw * (D / 4), nc = nw * 16;
    {
        float kk[2][2][4], qk[2][2][4];
        planes::clear(kk);
        planes::clear(qk);
        planes::product<2, 2, D, D, false, P, D, false, P>(kk, K, m, K, nc, lane);
        planes::product<2, 2, D, D, false, P, D, false, P>(qk, Q, m, K, nc, lane);
        planes::each(kk, m, nc, lane, [&](float& x, int i, int j) {
            Af[at64(i, j)] = j < i ? x * (t.beta[i] * fK[i] * fK[j] * expf(t.G[i] - t.G[j])) : 0.f;
        });
        planes::each(qk, m, nc, lane, [&](float& x, int i, int j) {
            x = j <= i ? x * (fQ[i] * fK[j] * expf(t.G[i] - t.G[j])) : 0.f;
        });
        const uint32_t top = planes::max_bits(qk);
        if (lane == 0) red[0][warp] = top;
        __syncthreads();
        const Scale sp = planes::scale_of(top_of(red[0]));
        planes::write<kC>(Pm, qk, m, nc, lane, sp.mul);
    }
    const float p_back = planes::scale_of(top_of(red[0])).back;
    unit_lower_inverse(Af, Tf);

    // T's planes to the workspace; T diag(beta b) and T diag(beta) (with the rows' factors of K and V) as
    // the left sides of W and U
    float tr[16];
    const int rr = tid >> 2, rc = (tid & 3) * 16;
    {
        uint32_t m0 = 0, m1 = 0, m2 = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = rc + i;
            tr[i] = j <= rr ? Tf[at64(rr, j)] : 0.f;
            const float x = tr[i] * t.beta[j];
            m0 = max(m0, planes::abs_bits(tr[i]));
            m1 = max(m1, planes::abs_bits(x * t.b[j] * fK[j]));
            m2 = max(m2, planes::abs_bits(x * fV[j]));
        }
        m0 = __reduce_max_sync(0xffffffffu, m0);
        m1 = __reduce_max_sync(0xffffffffu, m1);
        m2 = __reduce_max_sync(0xffffffffu, m2);
        if (lane == 0) { red[1][warp] = m0; red[2][warp] = m1; red[3][warp] = m2; }
    }
    __syncthreads();
    const Scale st = planes::scale_of(top_of(red[1])), sw1 = planes::scale_of(top_of(red[2]));
    const Scale su1 = planes::scale_of(top_of(red[3]));
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = tr[i] * st.mul;
        put16(TX, w.T + unit * kTBytes, rr, rc, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = tr[i] * t.beta[rc + i] * t.b[rc + i] * fK[rc + i] * sw1.mul;
        put16(TX, nullptr, rr, rc, x);
    }
    __syncthreads();
    float acc_w[2][NT][4];
    planes::clear(acc_w);
    planes::product<2, NT, kC, kC, false, 2, D, true, P, planes::kLower>(acc_w, TX, m, K, nd, lane);
    planes::each(acc_w, m, nd, lane, [&](float& x, int, int) { x *= sw1.back; });
    {
        const uint32_t top = planes::max_bits(acc_w);
        if (lane == 0) red[4][warp] = top;
    }
    __syncthreads();
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = tr[i] * t.beta[rc + i] * fV[rc + i] * su1.mul;
        put16(TX, nullptr, rr, rc, x);
    }
    const Scale sw = planes::scale_of(top_of(red[4]));
    planes::write<D>(W, acc_w, m, nd, lane, sw.mul);
    __syncthreads();
    {
        float acc[2][NT][4];
        planes::clear(acc);
        planes::product<2, NT, kC, kC, false, 2, D, true, P, planes::kLower>(acc, TX, m, V, nd, lane);
        planes::each(acc, m, nd, lane, [&](float& x, int i, int) { x *= su1.back * t.tail[i] * fK[i]; });
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[5][warp] = top;
        __syncthreads();
        planes::write<D>(U, acc, m, nd, lane, planes::scale_of(top_of(red[5])).mul);
    }
    {
        float acc[2][NT][4];  // Q' = diag(b) Q - P W, with the rows' factors of dY
        planes::clear(acc);
        planes::product<2, NT, kC, kC, false, 2, D, true, 2, planes::kLower>(acc, Pm, m, W, nd, lane);
        const int g = lane >> 2, c = (lane & 3) * 2;
        const float back = p_back * sw.back;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int r = m[i] + g + 8 * hh;
                    const float2 q = planes::read<D, P>(Q, r, nd + 8 * j + c);
                    const float f = t.b[r] * fQ[r];
                    acc[i][j][2 * hh] = fY[r] * (f * q.x - back * acc[i][j][2 * hh]);
                    acc[i][j][2 * hh + 1] = fY[r] * (f * q.y - back * acc[i][j][2 * hh + 1]);
                }
        planes::each(acc_w, m, nd, lane, [&](float& x, int i, int) { x *= t.tail[i] * fK[i]; });
        const uint32_t top = planes::max_bits(acc), top_w = planes::max_bits(acc_w);
        if (lane == 0) { red[6][warp] = top; red[7][warp] = top_w; }
        __syncthreads();  // also: Q, V and W have been read
        planes::write<D>(Qp, acc, m, nd, lane, planes::scale_of(top_of(red[6])).mul);
        planes::write<D>(W, acc_w, m, nd, lane, planes::scale_of(top_of(red[7])).mul);
    }
    __syncthreads();

    constexpr int MT = D / 32;
    int md[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) md[i] = mw * (D / 2) + 16 * i;
    auto to_global = [&](float (&acc)[MT][NT][4], float* dst, float back) {
        const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    *reinterpret_cast<float2*>(dst + (md[i] + g + 8 * hh) * D + nd + 8 * j + c) =
                        make_float2(acc[i][j][2 * hh] * back, acc[i][j][2 * hh + 1] * back);
    };
    {
        float acc[MT][NT][4];
        planes::clear(acc);
        planes::product<MT, NT, kC, D, true, 2, D, true, P>(acc, U, md, K, nd, lane);
        to_global(acc, w.S + unit * D * D, planes::scale_of(top_of(red[5])).back);
        planes::clear(acc);
        planes::product<MT, NT, kC, D, true, P, D, true, 2>(acc, Y, md, Qp, nd, lane);
        to_global(acc, w.dS + unit * D * D, planes::scale_of(top_of(red[6])).back);
        planes::clear(acc);
        planes::product<MT, NT, kC, D, true, 2, D, true, P>(acc, W, md, K, nd, lane);
        const float back = planes::scale_of(top_of(red[7])).back;
        planes::each(acc, md, nd, lane, [&](float& x, int i, int j) { x = (i == j ? t.b[kC - 1] : 0.f) - back * x; });
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[8][warp] = top;
        __syncthreads();
        const Scale sc = planes::scale_of(top_of(red[8]));
        unsigned char* M = w.M + unit * m_bytes(D);
        const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t hi, lo;
                    planes::split(acc[i][j][2 * hh] * sc.mul, acc[i][j][2 * hh + 1] * sc.mul, hi, lo);
                    const uint32_t o = planes::offset<D>(md[i] + g + 8 * hh, nd + 8 * j + c);
                    *reinterpret_cast<uint32_t*>(M + o) = hi;
                    *reinterpret_cast<uint32_t*>(M + m_bytes(D) / 2 + o) = lo;
                }
        if (tid == 0) {
            w.meta[unit].t_scale = st.back;
            w.meta[unit].m_scale = sc.back;
        }
    }
}

// ---- the two recurrences over a sequence's chunks ----------------------------------------------
// A warp keeps 16 rows of the state in its accumulators for the whole sequence: the accumulator layout
// of the state is the left operand's layout of the next product, so the rows never pass through shared
// memory, and rows do not depend on one another.  M's planes arrive by asynchronous copies, two stages.

constexpr int kScanThreads = 128;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// N = S M (TB true) or S M^T, for the rows' scaled planes hi, lo.
template <int D, bool TB>
__device__ __forceinline__ void scan_product(float (&N)[D / 8][4], const uint32_t (&hi)[D / 16][4],
                                             const uint32_t (&lo)[D / 16][4], uint32_t M, int lane) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
            uint32_t b[2][4];
            planes::load_b<D, TB>(b[0], M, 8 * j, 16 * k, lane);
            planes::load_b<D, TB>(b[1], M + m_bytes(D) / 2, 8 * j, 16 * k, lane);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                planes::mma(N[j + h], hi[k], b[0][2 * h], b[0][2 * h + 1]);
                planes::mma(N[j + h], hi[k], b[1][2 * h], b[1][2 * h + 1]);
                planes::mma(N[j + h], lo[k], b[0][2 * h], b[0][2 * h + 1]);
            }
        }
}

template <int D>
__global__ void __launch_bounds__(kScanThreads, 1) chunk_bwd_scan_kernel(ChunkBwdArgs a, Work w) {
    extern __shared__ __align__(128) unsigned char sm[];
    constexpr int NT = D / 8, KT = D / 16, slices = D / 64;
    if (!cu_valid(a)) return;
    const int pair = blockIdx.x / slices, n = pair / a.H, h = pair % a.H;
    const bool back = blockIdx.y != 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x % slices) * 64 + warp * 16, row = r0 + (lane >> 2), col = (lane & 3) * 2;
    Span s;
    long base;
    seq_span(a, n, s, base);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const long state = ((long)n * a.H + h) * D * D + row * D + col;
    const float* from = back ? a.dfinal_state : a.initial_state;
    auto unit_of = [&](int i) { return (base + (back ? s.chunks - 1 - i : i)) * a.H + h; };
    auto fetch = [&](int i) {
        const unsigned char* src = w.M + unit_of(i) * m_bytes(D);
        const uint32_t dst = smem + (i & 1) * (uint32_t)m_bytes(D);
        for (uint32_t o = threadIdx.x * 16; o < m_bytes(D); o += kScanThreads * 16) copy16(dst + o, src + o);
    };
    if (s.chunks > 0) fetch(0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    float S[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const float2 x = from ? *reinterpret_cast<const float2*>(from + state + 8 * j) : make_float2(0.f, 0.f);
        const float2 y = from ? *reinterpret_cast<const float2*>(from + state + 8 * D + 8 * j) : make_float2(0.f, 0.f);
        S[j][0] = x.x; S[j][1] = x.y; S[j][2] = y.x; S[j][3] = y.y;
    }
    // what follows the last chunk is wanted only as the gradient of the initial state
    const int steps = back && a.dinitial_state ? s.chunks : s.chunks - 1;
    for (int i = 0; i < s.chunks; ++i) {
        const long unit = unit_of(i);
        float* at = (back ? w.dS : w.S) + unit * D * D + row * D + col;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // stage i is here, and every warp has left the stage before it
        if (i + 1 < s.chunks) fetch(i + 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        float add[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float2 x = *reinterpret_cast<const float2*>(at + 8 * j);
            const float2 y = *reinterpret_cast<const float2*>(at + 8 * D + 8 * j);
            add[j][0] = x.x; add[j][1] = x.y; add[j][2] = y.x; add[j][3] = y.y;
        }
        const float m_scale = w.meta[unit].m_scale;
        uint32_t top0 = 0, top1 = 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2*>(at + 8 * j) = make_float2(S[j][0], S[j][1]);
            *reinterpret_cast<float2*>(at + 8 * D + 8 * j) = make_float2(S[j][2], S[j][3]);
            top0 = max(top0, max(planes::abs_bits(S[j][0]), planes::abs_bits(S[j][1])));
            top1 = max(top1, max(planes::abs_bits(S[j][2]), planes::abs_bits(S[j][3])));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            top0 = max(top0, __shfl_xor_sync(0xffffffffu, top0, o));
            top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, o));
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(top0, top1));
        if (lane == 0) (back ? w.meta[unit].ds_max : w.meta[unit].s_max)[r0 / 16] = top;
        if (i >= steps) break;
        const Scale s0 = planes::scale_of(top0), s1 = planes::scale_of(top1);
        uint32_t hi[KT][4], lo[KT][4];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                planes::split(S[2 * k + e][0] * s0.mul, S[2 * k + e][1] * s0.mul, hi[k][2 * e], lo[k][2 * e]);
                planes::split(S[2 * k + e][2] * s1.mul, S[2 * k + e][3] * s1.mul, hi[k][2 * e + 1], lo[k][2 * e + 1]);
            }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[j][e] = 0.f;
        const uint32_t M = smem + (i & 1) * (uint32_t)m_bytes(D);
        if (back) scan_product<D, false>(S, hi, lo, M, lane);
        else scan_product<D, true>(S, hi, lo, M, lane);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[j][e] = fmaf(S[j][e], (e < 2 ? s0.back : s1.back) * m_scale, add[j][e]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (back && a.dinitial_state) {
        float* out = a.dinitial_state + state;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2*>(out + 8 * j) = make_float2(S[j][0], S[j][1]);
            *reinterpret_cast<float2*>(out + 8 * D + 8 * j) = make_float2(S[j][2], S[j][3]);
        }
    }
}

// ---- gradients -----------------------------------------------------------------------------------

// Shared memory of the gradient kernel: K, Q, dY (P planes each; with two planes at d = 128 Q and dY
// share one place, in turn), a state (dS1, S0, dS1 in turn), P then dP, T then Z, and two 64 x d buffers.
template <int D, int P>
struct GradSmem {
    static constexpr bool share = P == 2;
    static constexpr uint32_t plane = kC * D * 2, square = kC * kC * 2, state = D * D * 2;
    static constexpr uint32_t K = 0, Q = P * plane, Y = share ? Q : 2 * P * plane;
    static constexpr uint32_t ST = Y + P * plane, Pm = ST + 2 * state, Tm = Pm + 2 * square;
    static constexpr uint32_t B1 = Tm + 2 * square, B2 = B1 + 2 * plane, bytes = B2 + 2 * plane;
};

// A d x d fp32 state as planes with the given scale.  DOT: returns also this thread's part of the dot
// product with what the planes held before (old_back takes them to values).
template <int D, bool DOT>
__device__ float load_state(Mat dst, const float* src, Scale s, float old_back) {
    constexpr int N = D * D / 4 / kThreads, H = N < 8 ? N : 8;
    float dot = 0.f;
#pragma unroll
    for (int b = 0; b < N; b += H) {
        float x[H][4];
#pragma unroll
        for (int p = 0; p < H; ++p) load_vec<4>(src + ((b + p) * kThreads + threadIdx.x) * 4, x[p]);
#pragma unroll
        for (int p = 0; p < H; ++p) {
            const int e = ((b + p) * kThreads + threadIdx.x) * 4;
            const uint32_t at = dst.at + planes::offset<D>(e / D, e % D);
            if constexpr (DOT) {
                uint32_t u[2], v[2];
                planes::lds64(at, u[0], u[1]);
                planes::lds64(at + dst.lo, v[0], v[1]);
                const float2 u0 = planes::halves(u[0]), u1 = planes::halves(u[1]);
                const float2 v0 = planes::halves(v[0]), v1 = planes::halves(v[1]);
                dot = fmaf(u0.x + v0.x, x[p][0], dot);
                dot = fmaf(u0.y + v0.y, x[p][1], dot);
                dot = fmaf(u1.x + v1.x, x[p][2], dot);
                dot = fmaf(u1.y + v1.y, x[p][3], dot);
            }
            uint32_t hi[2], lo[2];
            planes::split(x[p][0] * s.mul, x[p][1] * s.mul, hi[0], lo[0]);
            planes::split(x[p][2] * s.mul, x[p][3] * s.mul, hi[1], lo[1]);
            planes::sts64(at, hi[0], hi[1]);
            planes::sts64(at + dst.lo, lo[0], lo[1]);
        }
    }
    return dot * old_back;
}

// A pair of elements of a q/k/v-like tensor.
__device__ __forceinline__ float2 load2(const void* src, gdn_dtype dt, long i) {
    float x[2];
    if (dt == GDN_BF16) load_vec<2>(static_cast<const __nv_bfloat16*>(src) + i, x);
    else load_vec<2>(static_cast<const float*>(src) + i, x);
    return make_float2(x[0], x[1]);
}
__device__ __forceinline__ void store2(void* dst, gdn_dtype dt, long i, float x, float y) {
    if (dt == GDN_BF16)
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(dst) + i) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<float2*>(static_cast<float*>(dst) + i) = make_float2(x, y);
}

// Gradient of one element through xh = scale * x * inv: with n = x * inv,
// dx = scale * inv * (d - n (n . d)); dot = d . xh.
__device__ __forceinline__ float unnormalise(float d, float xh, float dot, float inv, float scale, int use_l2) {
    return use_l2 ? scale * inv * (d - xh * (dot / (scale * scale))) : scale * d;
}

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1) chunk_bwd_grad_kernel(ChunkBwdArgs a, Work w) {
    using L = GradSmem<D, P>;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ Gates t;
    __shared__ float fK[kC], fQ[kC], fY[kC], kinv[kC], qinv[kC], dpp[kC], diag[kC];
    __shared__ uint32_t red[2][8], tops[2];
    if (!cu_valid(a)) return;
    const long slot = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, rep = a.H / a.Hk, hk = h / rep, tid = threadIdx.x;
    const Span s = find_span(a, slot);
    if (s.n < 0) return;
    const long t0 = s.bos + (long)s.c * kC, unit = slot * a.H + h;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const Mat K{base + L::K, L::plane}, Q{base + L::Q, L::plane}, Y{base + L::Y, L::plane};
    const Mat ST{base + L::ST, L::state}, Pm{base + L::Pm, L::square}, Tm{base + L::Tm, L::square};
    const Mat B1{base + L::B1, L::plane}, B2{base + L::B2, L::plane};
    const int warp = tid >> 5, lane = tid & 31, mw = warp >> 2, nw = warp & 3;
    const int m[2] = {16 * mw, 16 * (3 - mw)};  // see the preparation
    constexpr int NT = D / 32;
    const int nd = nw * (D / 4), nc = nw * 16, g = lane >> 2, c2 = (lane & 3) * 2;
    const Meta& meta = w.meta[unit];

    uint32_t s_top = 0, ds_top = 0;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        s_top = max(s_top, meta.s_max[i]);
        ds_top = max(ds_top, meta.ds_max[i]);
    }
    const Scale ss = planes::scale_of(s_top), sds = planes::scale_of(ds_top);
    const float t_back = meta.t_scale;
    const float* S0 = w.S + unit * D * D;
    const float* dS1 = w.dS + unit * D * D;

    if (tid < 2) tops[tid] = 0;
    load_gates(a, t, t0, len, h);
    __syncthreads();
    load_rows<D, P>(K, a.k, a.qkv_dtype, t0, len, a.Hk, hk, fK, kinv, true, a.use_l2, 1.f, &tops[0]);
    load_rows<D, P>(Q, a.q, a.qkv_dtype, t0, len, a.Hk, hk, fQ, qinv, true, a.use_l2, a.scale, &tops[1]);
    if constexpr (!L::share)
        load_rows<D, P>(Y, a.dout, a.dout_dtype, t0, len, a.H, h, fY, nullptr, false, false, 1.f, nullptr);
    load_state<D, false>(ST, dS1, sds, 0.f);
    {
        const uint4* src = reinterpret_cast<const uint4*>(w.T + unit * kTBytes);
        uint4* dst = reinterpret_cast<uint4*>(sm + L::Tm);
#pragma unroll
        for (int i = 0; i < (int)(kTBytes / 16 / kThreads); ++i) dst[i * kThreads + tid] = src[i * kThreads + tid];
    }
    __syncthreads();

    // Row reductions of accumulators: f(value, row, column pair's first column)
    auto pairs = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) f(i, j, hh, m[i] + g + 8 * hh, nd + 8 * j + c2);
    };

    float qk[2][2][4];  // Q K^T * D
    planes::clear(qk);
    planes::product<2, 2, D, D, false, P, D, false, P>(qk, Q, m, K, nc, lane);
    planes::each(qk, m, nc, lane, [&](float& x, int i, int j) {
        x = j <= i ? x * (fQ[i] * fK[j] * expf(t.G[i] - t.G[j])) : 0.f;
    });
    planes::each(qk, m, nc, lane, [&](float& x, int i, int j) {
        if (i == j) diag[i] = x;  // q_i . k_i for now
    });
    if constexpr (L::share) {
        __syncthreads();
        load_rows<D, P>(Y, a.dout, a.dout_dtype, t0, len, a.H, h, fY, nullptr, false, false, 1.f, nullptr);
        __syncthreads();
    }
    // P with the rows' factors of dY, for P^T dY
    planes::each(qk, m, nc, lane, [&](float& x, int i, int) { x *= fY[i]; });
    {
        const uint32_t top = planes::max_bits(qk);
        if (lane == 0) red[0][warp] = top;
    }
    __syncthreads();
    const Scale sp = planes::scale_of(top_of(red[0]));
    planes::write<kC>(Pm, qk, m, nc, lane, sp.mul);
    float acc[2][NT][4], dR[2][NT][4];
    planes::clear(dR);  // Kd dS1^T first, in dR's registers
    planes::product<2, NT, D, D, false, P, D, false, 2>(dR, K, m, ST, nd, lane);
    __syncthreads();
    planes::clear(acc);
    planes::product<2, NT, kC, kC, true, 2, D, true, P, planes::kUpper>(acc, Pm, m, Y, nd, lane);
    pairs([&](int i, int j, int hh, int r, int) {
        const float f = t.tail[r] * fK[r] * sds.back;
#pragma unroll
        for (int e = 2 * hh; e < 2 * hh + 2; ++e) acc[i][j][e] = fmaf(acc[i][j][e], sp.back, dR[i][j][e] * f);
    });
    {
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[1][warp] = top;
    }
    __syncthreads();  // also: dS1's planes have been read
    const Scale sdu = planes::scale_of(top_of(red[1]));
    planes::write<D>(B1, acc, m, nd, lane, sdu.mul);
    load_state<D, false>(ST, S0, ss, 0.f);
    __syncthreads();

    float2 v[2][NT][2];
    pairs([&](int i, int j, int hh, int r, int x) {
        v[i][j][hh] = r < len ? load2(a.v, a.qkv_dtype, ((t0 + r) * a.H + h) * D + x) : make_float2(0.f, 0.f);
    });
    planes::clear(dR);  // dR = T^T (P^T dY + Kd dS1^T)
    planes::product<2, NT, kC, kC, true, 2, D, true, 2, planes::kUpper>(dR, Tm, m, B1, nd, lane);
    float vdot[2][2] = {};
    pairs([&](int i, int j, int hh, int r, int x) {
        float &x0 = dR[i][j][2 * hh], &x1 = dR[i][j][2 * hh + 1];
        x0 *= t_back * sdu.back;
        x1 *= t_back * sdu.back;
        vdot[i][hh] = fmaf(x0, v[i][j][hh].x, fmaf(x1, v[i][j][hh].y, vdot[i][hh]));
        if (r < len) store2(a.dv, a.qkv_dtype, ((t0 + r) * a.H + h) * D + x, t.beta[r] * x0, t.beta[r] * x1);
    });
    {
        const uint32_t top = planes::max_bits(dR);
        if (lane == 0) red[0][warp] = top;
    }
    planes::clear(acc);  // diag(beta) (V - diag(b) K S0^T)
    planes::product<2, NT, D, D, false, P, D, false, 2>(acc, K, m, ST, nd, lane);
    pairs([&](int i, int j, int hh, int r, int) {
        const float f = t.b[r] * fK[r] * ss.back;
        acc[i][j][2 * hh] = t.beta[r] * (v[i][j][hh].x - f * acc[i][j][2 * hh]);
        acc[i][j][2 * hh + 1] = t.beta[r] * (v[i][j][hh].y - f * acc[i][j][2 * hh + 1]);
    });
    __syncthreads();  // red[0]; B1 has been read, red[1] too
    const Scale sr = planes::scale_of(top_of(red[0]));
    planes::write<D>(B2, dR, m, nd, lane, sr.mul);
    {
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[1][warp] = top;
    }
    __syncthreads();
    const Scale sv = planes::scale_of(top_of(red[1]));
    planes::write<D>(B1, acc, m, nd, lane, sv.mul);

    float dQ[2][NT][4], E[2][NT][4];
    planes::clear(dQ);
    planes::product<2, NT, D, D, false, P, D, true, 2>(dQ, Y, m, ST, nd, lane);
    planes::clear(E);
    planes::product<2, NT, D, D, false, 2, D, true, 2>(E, B2, m, ST, nd, lane);
    pairs([&](int i, int j, int hh, int r, int) {
        const float fq = t.b[r] * fY[r] * ss.back, fe = -t.b[r] * sr.back * ss.back;
#pragma unroll
        for (int e = 2 * hh; e < 2 * hh + 2; ++e) {
            dQ[i][j][e] *= fq;
            E[i][j][e] *= fe;
        }
    });
    __syncthreads();  // B1 is written; S0's planes have been read
    planes::clear(acc);  // U = T diag(beta) (V - ...)
    planes::product<2, NT, kC, kC, false, 2, D, true, 2, planes::kLower>(acc, Tm, m, B1, nd, lane);
    planes::each(acc, m, nd, lane, [&](float& x, int, int) { x *= t_back * sv.back; });
    {
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[0][warp] = top;
    }
    const float state_dot = load_state<D, true>(ST, dS1, sds, ss.back);  // and <S0, dS1>
    __syncthreads();
    const Scale su = planes::scale_of(top_of(red[0]));
    planes::write<D>(B1, acc, m, nd, lane, su.mul);
    __syncthreads();

    float H[2][NT][4];
    planes::clear(H);
    planes::product<2, NT, D, D, false, 2, D, true, 2>(H, B1, m, ST, nd, lane);
    pairs([&](int i, int j, int hh, int r, int) {
        const float f = t.tail[r] * su.back * sds.back;
        H[i][j][2 * hh] *= f;
        H[i][j][2 * hh + 1] *= f;
    });
    // dP and Z, each twice: with the factors of K's rows on the columns (for the products with K) and
    // with the factors of the left rows (for the transposed products)
    float dP[2][2][4], Z[2][2][4];
    planes::clear(dP);
    planes::product<2, 2, D, D, false, P, D, false, 2>(dP, Y, m, B1, nc, lane);
    planes::clear(Z);
    planes::product<2, 2, D, D, false, 2, D, false, 2>(Z, B2, m, B1, nc, lane);
    planes::each(dP, m, nc, lane, [&](float& x, int i, int j) {
        const float y = j <= i ? x * (fY[i] * su.back * expf(t.G[i] - t.G[j])) : 0.f;
        if (i == j) {
            dpp[i] = y;
            diag[i] *= y;  // the thread that wrote q_i . k_i
        }
        x = j < i ? y : 0.f;
    });
    planes::each(Z, m, nc, lane, [&](float& x, int i, int j) {
        x = j < i ? -x * (sr.back * su.back * expf(t.G[i] - t.G[j])) : 0.f;
    });
    uint32_t tp[4] = {0, 0, 0, 0};
    planes::each(dP, m, nc, lane, [&](float& x, int i, int j) {
        tp[0] = max(tp[0], planes::abs_bits(x * fK[j]));
        tp[1] = max(tp[1], planes::abs_bits(x * fQ[i]));
    });
    planes::each(Z, m, nc, lane, [&](float& x, int i, int j) {
        tp[2] = max(tp[2], planes::abs_bits(x * fK[j]));
        tp[3] = max(tp[3], planes::abs_bits(x * t.beta[i] * fK[i]));
    });
    __syncthreads();  // B1, B2, ST, P and T have been read
    // the state's place now holds the four maxima of each warp, then row sums and the state dot
    uint32_t* tops4 = reinterpret_cast<uint32_t*>(sm + L::ST);
    float* sums = reinterpret_cast<float*>(sm + L::ST) + 64;  // [5][4][64]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, tp[i]);
        if (lane == 0) tops4[i * 8 + warp] = top;
    }
    {
        const float x = warp_sum(state_dot);
        if (lane == 0) reinterpret_cast<float*>(tops4)[32 + warp] = x;
    }
    if constexpr (L::share)
        load_rows<D, P>(Q, a.q, a.qkv_dtype, t0, len, a.Hk, hk, fQ, qinv, true, a.use_l2, a.scale, &tops[1]);
    __syncthreads();
    const Mat dPk{Pm.at, L::square}, Zk{Tm.at, L::square}, dPq{B1.at, L::square}, Zb{B2.at, L::square};
    Scale sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = planes::scale_of(top_of(tops4 + i * 8));
    auto put = [&](Mat dst, float (&x)[2][2][4], float mul, auto&& factor) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int r = m[i] + g + 8 * hh, c = nc + 8 * j + c2;
                    uint32_t hi, lo;
                    planes::split(x[i][j][2 * hh] * factor(r, c) * mul, x[i][j][2 * hh + 1] * factor(r, c + 1) * mul, hi, lo);
                    const uint32_t at = dst.at + planes::offset<kC>(r, c);
                    planes::sts32(at, hi);
                    planes::sts32(at + dst.lo, lo);
                }
    };
    put(dPk, dP, sc[0].mul, [&](int, int j) { return fK[j]; });
    put(dPq, dP, sc[1].mul, [&](int i, int) { return fQ[i]; });
    put(Zk, Z, sc[2].mul, [&](int, int j) { return fK[j]; });
    put(Zb, Z, sc[3].mul, [&](int i, int) { return t.beta[i] * fK[i]; });
    __syncthreads();

    float qdot[2][2] = {}, kpos[2][2] = {}, kneg[2][2] = {}, hdot[2][2] = {};
    planes::clear(acc);
    planes::product<2, NT, kC, kC, false, 2, D, true, P, planes::kLower>(acc, dPk, m, K, nd, lane);
    pairs([&](int i, int j, int hh, int r, int x) {
        const float2 q = planes::read<D, P>(Q, r, x);
        float &x0 = dQ[i][j][2 * hh], &x1 = dQ[i][j][2 * hh + 1];
        x0 = fmaf(acc[i][j][2 * hh], sc[0].back, x0);
        x1 = fmaf(acc[i][j][2 * hh + 1], sc[0].back, x1);
        qdot[i][hh] = fmaf(x0, q.x, fmaf(x1, q.y, qdot[i][hh]));
    });
    planes::clear(acc);
    planes::product<2, NT, kC, kC, false, 2, D, true, P, planes::kLower>(acc, Zk, m, K, nd, lane);
    pairs([&](int i, int j, int hh, int r, int x) {
        const float2 k = planes::read<D, P>(K, r, x);
        float &x0 = E[i][j][2 * hh], &x1 = E[i][j][2 * hh + 1];
        x0 = fmaf(acc[i][j][2 * hh], sc[2].back, x0);
        x1 = fmaf(acc[i][j][2 * hh + 1], sc[2].back, x1);
        kpos[i][hh] = fmaf(x0, k.x, fmaf(x1, k.y, kpos[i][hh]));
        hdot[i][hh] = fmaf(H[i][j][2 * hh], k.x, fmaf(H[i][j][2 * hh + 1], k.y, hdot[i][hh]));
    });
    planes::clear(acc);
    planes::product<2, NT, kC, kC, true, 2, D, true, P, planes::kUpper>(acc, dPq, m, Q, nd, lane);
    planes::each(acc, m, nd, lane, [&](float& x, int, int) { x *= sc[1].back; });
    {
        float x[2][NT][4];
        planes::clear(x);
        planes::product<2, NT, kC, kC, true, 2, D, true, P, planes::kUpper>(x, Zb, m, K, nd, lane);
        pairs([&](int i, int j, int hh, int r, int col) {
            const float2 k = planes::read<D, P>(K, r, col);
            const float x0 = fmaf(x[i][j][2 * hh], sc[3].back, acc[i][j][2 * hh]);
            const float x1 = fmaf(x[i][j][2 * hh + 1], sc[3].back, acc[i][j][2 * hh + 1]);
            kneg[i][hh] = fmaf(x0, k.x, fmaf(x1, k.y, kneg[i][hh]));
            H[i][j][2 * hh] += x0;  // dK- without P's diagonal
            H[i][j][2 * hh + 1] += x1;
        });
    }
    // each warp's part of the row sums, then the rows' sums over the four warps beside it
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float x[5] = {qdot[i][hh], kpos[i][hh], kneg[i][hh], hdot[i][hh], vdot[i][hh]};
            const int r = m[i] + g + 8 * hh;
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                x[k] += __shfl_xor_sync(0xffffffffu, x[k], 1);
                x[k] += __shfl_xor_sync(0xffffffffu, x[k], 2);
                if ((lane & 3) == 0) sums[(k * 4 + nw) * kC + r] = x[k];
            }
        }
    __syncthreads();
    auto sum_of = [&](int k, int r) {
        const float* x = sums + k * 4 * kC + r;
        return (x[0] + x[kC]) + (x[2 * kC] + x[3 * kC]);
    };
    const long q_row = rep > 1 ? a.H : a.Hk;
    const int q_head = rep > 1 ? h : hk;
    void* dq = rep > 1 ? w.dq : a.dq;
    void* dk = rep > 1 ? w.dk : a.dk;
    const gdn_dtype qk_type = rep > 1 ? GDN_F32 : a.qkv_dtype;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = m[i] + g + 8 * hh;
            if (r >= len) continue;
            const float qd = fmaf(sum_of(0, r), fQ[r], diag[r]);
            const float kd = fmaf(t.beta[r] * sum_of(1, r) + sum_of(2, r) + sum_of(3, r), fK[r], diag[r]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int x = nd + 8 * j + c2;
                const float2 q = planes::read<D, P>(Q, r, x), k = planes::read<D, P>(K, r, x);
                const float q0 = q.x * fQ[r], q1 = q.y * fQ[r], k0 = k.x * fK[r], k1 = k.y * fK[r];
                const long at = ((t0 + r) * q_row + q_head) * D + x;
                store2(dq, qk_type, at,
                       unnormalise(fmaf(dpp[r], k0, dQ[i][j][2 * hh]), q0, qd, qinv[r], a.scale, a.use_l2),
                       unnormalise(fmaf(dpp[r], k1, dQ[i][j][2 * hh + 1]), q1, qd, qinv[r], a.scale, a.use_l2));
                const float d0 = fmaf(t.beta[r], E[i][j][2 * hh], fmaf(dpp[r], q0, H[i][j][2 * hh]));
                const float d1 = fmaf(t.beta[r], E[i][j][2 * hh + 1], fmaf(dpp[r], q1, H[i][j][2 * hh + 1]));
                store2(dk, qk_type, at, unnormalise(d0, k0, kd, kinv[r], 1.f, a.use_l2),
                       unnormalise(d1, k1, kd, kinv[r], 1.f, a.use_l2));
            }
        }
    // dbeta; dg by a scan from the chunk's end and one from its start, two rows a lane
    if (warp == 0) {
        float d[2], hd[2], x = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            const float kp = sum_of(1, r) * fK[r];
            if (r < len) a.dbeta[(t0 + r) * a.H + h] = sum_of(4, r) + kp;
            d[e] = sum_of(0, r) * fQ[r] + t.beta[r] * kp - sum_of(2, r) * fK[r];
            hd[e] = sum_of(3, r) * fK[r];
        }
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x += reinterpret_cast<const float*>(tops4)[32 + i];
        float after = d[0] + d[1], before = hd[0] + hd[1];  // inclusive sums over the later, the earlier lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, after, o), z = __shfl_up_sync(0xffffffffu, before, o);
            if (lane + o < 32) after += y;
            if (lane >= o) before += z;
        }
        float later = __shfl_down_sync(0xffffffffu, after, 1), earlier = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 31) later = 0.f;
        if (lane == 0) earlier = 0.f;
        const float carried = t.b[kC - 1] * x;
        const int r = 2 * lane;
        if (r < len) a.dg[(t0 + r) * a.H + h] = (later + d[1] + d[0]) + earlier + carried;
        if (r + 1 < len) a.dg[(t0 + r + 1) * a.H + h] = (later + d[1]) + (earlier + hd[0]) + carried;
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

template <int D, int P>
cudaError_t launch(const ChunkBwdArgs& a, cudaStream_t s) {
    const long units = slot_count(a.num_seqs, a.total_T) * a.H;
    const Work w = work_of(a.workspace, units, (long)a.total_T * a.H, D);
    const int prep = PrepSmem<D, P>::bytes, grad = GradSmem<D, P>::bytes, scan = 2 * (int)m_bytes(D);
    cudaError_t e = cudaFuncSetAttribute(chunk_bwd_prep_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, prep);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_bwd_grad_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, grad);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(chunk_bwd_scan_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, scan);
    if (e != cudaSuccess) return e;
    if (a.total_T > 0) {
        chunk_bwd_prep_kernel<D, P><<<(unsigned)units, kThreads, prep, s>>>(a, w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    chunk_bwd_scan_kernel<D><<<dim3((unsigned)(a.num_seqs * a.H * (D / 64)), 2), kScanThreads, scan, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess || a.total_T == 0) return e;
    chunk_bwd_grad_kernel<D, P><<<(unsigned)units, kThreads, grad, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess || a.H == a.Hk) return e;
    chunk_bwd_heads_kernel<<<152 * 8, kThreads, 0, s>>>(a, w);
    return cudaGetLastError();
}

}  // namespace

size_t chunk_bwd_workspace_bytes(int num_seqs, int total_T, int H, int Hk, int d) {
    const size_t units = (size_t)slot_count(num_seqs, total_T) * H;
    return units * (kTBytes + m_bytes(d) + 2 * sizeof(float) * d * d + sizeof(Meta)) +
           (H > Hk ? 2 * sizeof(float) * total_T * H * d : 0);
}

cudaError_t launch_chunk_bwd(const ChunkBwdArgs& a, cudaStream_t s) {
    // bf16 throughout: one plane holds an input exactly
    const bool one = a.qkv_dtype == GDN_BF16 && a.dout_dtype == GDN_BF16;
    if (a.d == 128) return one ? launch<128, 1>(a, s) : launch<128, 2>(a, s);
    return one ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
}

}  // namespace gdn

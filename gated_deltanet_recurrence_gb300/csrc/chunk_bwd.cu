// chunk_bwd.cu -- gradients of the chunked gated delta rule (gdn_chunk_bwd).
//
// Forward, per chunk of C = 64 tokens (chunk form of "5. 线性注意力", "Delta Rule 的 Chunk 实现"), with
// G the inclusive sum of g in the chunk, b = e^G, D_ij = e^(G_i - G_j) for j <= i and 0 above, q and k
// normalised (q scaled), S0 the state at the chunk's start:
//   A = strictly lower part of diag(beta) (K K^T * D),   T = (I + A)^-1,
//   W = T diag(beta b) K,   U = T diag(beta) V - W S0^T,   P = Q K^T * D,
//   Y = diag(b) Q S0^T + P U,   S1 = b_C S0 + U^T Kd   with Kd = diag(b_C / b) K.
// Given dY and dS1, backwards through the chunk:
//   E  = Kd dS1^T,   dR = T^T (P^T dY + E),   dV = diag(beta) dR,
//   dS0 = b_C dS1 + X - E^T W   with X = dY^T (diag(b) Q - P W),
//   dP = (dY U^T) * D,   Z = -strictly lower part of (dR U^T) * D,
//   dQ  = diag(b) dY S0 + dP K,
//   dK+ = diag(beta) F,  F = Z K - diag(b) dR S0,
//   dK- = H + dP^T Q + Z^T diag(beta) K,  H = diag(b_C / b) U dS1,    dK = dK+ + dK-,
//   dbeta_i = dR_i . v_i + F_i . k_i,
//   dg_i = sum over j >= i of (dQ_j . q_j + dK+_j . k_j - (dK- - H)_j . k_j)
//          + sum over j < i of H_j . k_j + b_C <S0, dS1>.
// (Each row dot with q or k collects the terms in which that row's e^G or e^-G enters.  The diagonal
// of P carries e^0: its two contributions cancel, so it is kept out of these dots and a token that
// decays nothing gets dg = 0 exactly.)
//
// Three kernels:
//   prep  all chunks at once: T, W, T diag(beta) V, P, X, and K as it is used below;
//   scan  the two recurrences over the chunks of a sequence, S0 -> S1 forwards and dS1 -> dS0 backwards.
//         In each the state meets only W and K: on the way it leaves S0, U and dS1, E for every chunk;
//   grad  all chunks at once: the gradients.
// With grouped heads the gradients of q and k go to fp32 scratch per value head, and a fourth kernel
// adds the heads of a group in order.
//
// Every product is taken on the tensor cores from fp16 planes at fp32 accuracy (mma_planes.cuh); what is
// between the products is fp32.  What has a row a token is scaled row by row, so that a token's gradients keep
// that accuracy beside tokens of the chunk whose q, k, v or dY are larger by any factor; the states and X have one
// scale a matrix (or, in the scan, one a row of theirs).
//
// The chain over the chunks is the only serial part, so it is kept to what the state meets, and the rest
// runs over all chunks at once; the price is what the kernels hand over, 296 KB a chunk and head at d = 128.
// Measured on 2 x 4096 tokens, 16 heads, d = 128, bf16: 0.70 ms in all (inputs and outputs alone would take
// 35 us at the copy rate), prep 185, scan 217 - 220, grad 304 us; 16384 tokens, 32 heads: 2.62 ms.  (With one scale
// a chunk where there is one a row now: 0.68 ms and 2.52 ms.)
#include "mma_planes.cuh"
#include "sm100_ptx.cuh"
#include "train_internal.cuh"

namespace gdn {
namespace {

using planes::Mat;
using planes::Scale;

constexpr int kC = 64;

// Division of numbers below 2^31 by a divisor that the host knows, as a product with its scaled reciprocal
// (Granlund and Montgomery, "Division by Invariant Integers using Multiplication", 1994): with
// 2^(l - 1) < d <= 2^l and mul = floor(2^(31 + l) / d) + 1, n / d = floor(n mul / 2^(31 + l)).  (The half
// dozen divisions a block begins with were 2.5k cycles before its first load.)
struct Divisor {
    uint32_t mul, shift;
    static __host__ Divisor of(uint32_t d) {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;
        return {(uint32_t)((1ull << (31 + l)) / d + 1), 31 + l};
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)((uint64_t)(uint32_t)n * mul >> shift); }
};

// ---- the chunk slots ---------------------------------------------------------------------------
// Chunk c of sequence n has slot base(n) + c.  With lengths from cu_seqlens base(n) = cu[n] / 64 + n
// leaves every sequence at least as many slots as it has chunks; unused slots do nothing.  With equal
// lengths base(n) = n * chunks per sequence.
struct Span {
    long bos, eos, base;   // the sequence's tokens and first slot
    int n, chunks, c;      // sequence, its chunks, this chunk
};

__host__ __device__ __forceinline__ long slot_count(int num_seqs, int total_T) {
    return (long)total_T / kC + num_seqs;
}

__device__ __forceinline__ Span seq_span(const ChunkBwdArgs& a, int n) {
    Span s;
    if (a.cu_seqlens) {
        s.bos = a.cu_seqlens[n];
        s.eos = a.cu_seqlens[n + 1];
        s.base = s.bos / kC + n;
    } else {
        const long len = a.total_T / a.num_seqs;
        s.bos = n * len;
        s.eos = s.bos + len;
        s.base = n * ((len + kC - 1) / kC);
    }
    s.n = n;
    s.chunks = (int)((s.eos - s.bos + kC - 1) / kC);
    s.c = 0;
    return s;
}

// Above this many sequences a kernel of its own looks cu_seqlens over and writes down each slot's sequence;
// up to it every block does so for itself, which saves the launch (four loads a thread at most).
constexpr int kScanSeqs = 1024;

// index[0]: whether cu_seqlens is well formed; index[1 + slot]: the slot's sequence, or -1.  One block.
__global__ void __launch_bounds__(1024) chunk_bwd_index_kernel(ChunkBwdArgs a, int* index, int slots) {
    bool bad = false;
    for (int i = threadIdx.x; i < a.num_seqs; i += 1024) {
        const int lo = a.cu_seqlens[i], hi = a.cu_seqlens[i + 1];
        bad |= lo < 0 || hi < lo || hi > a.total_T;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        index[0] = !bad;
        if (bad) record_error(a.err, GDN_ERR_CU_SEQLENS);
    }
    if (bad) return;
    for (int i = threadIdx.x; i < slots; i += 1024) index[1 + i] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.num_seqs; i += 1024) {
        const int lo = a.cu_seqlens[i], hi = a.cu_seqlens[i + 1];
        for (int c = 0; c * kC < hi - lo; ++c) index[1 + lo / kC + i + c] = i;
    }
}

// ---- workspace ---------------------------------------------------------------------------------
// Per (slot, head):
//   link   what the scan needs of a chunk: planes of W (two) and K (one or two), then c, w, b_last
//   T, P   T^T and P^T (fp32 [64, 64], on and above the diagonal): the gradient kernel's planes of them carry
//          factors of dY's and of other rows, which have to go in before the rounding
//   U      (T diag(beta) V)^T, then U^T (fp32 [d, 64])  E   E^T (fp32 [d, 64])
//   S      S0 (fp32 [d, d])                             dS  X, then dS1 (fp32 [d, d])
//   meta   scales and maxima
struct LinkTail {
    float c[kC];  // takes row j of K's planes to Kd: tail_j and the row's factor
    float w[kC];  // takes row j of W's planes to W
    float b_last, pad[63];
};  // 768 bytes, so that a link's planes, at any of its places, start at a multiple of 256
static_assert(sizeof(LinkTail) == 768, "");

struct Meta {
    uint32_t s_max[16], ds_max[16];  // bits of the largest magnitudes of parts of S0, dS1
    float pad[32];
    float p_diag[kC];  // P's diagonal, q_i . k_i
};
static_assert(sizeof(Meta) == 512, "");

constexpr size_t kTBytes = kC * kC * sizeof(float);
__host__ __device__ constexpr size_t link_bytes(int d, int p) {
    return (2 + (size_t)p) * kC * d * sizeof(__half) + sizeof(LinkTail);
}

struct Work {
    unsigned char* link;
    float *T, *P, *U, *E, *S, *dS;
    Meta* meta;
    float *dq, *dk;  // [total_T, H, d] each, grouped heads only
    int* index;      // 1 + slots, many sequences only (else null)
    Divisor heads, rep, chunks;  // H, H / Hk, and with equal lengths the chunks of a sequence
    int len, per;                // with equal lengths: a sequence's tokens and chunks (0: no tokens)
};

// K's planes in the link: one where the inputs are bf16 throughout (it holds them exactly), else two.
__host__ __forceinline__ int input_planes(gdn_dtype qkv, gdn_dtype dout) {
    return qkv == GDN_BF16 && dout == GDN_BF16 ? 1 : 2;
}

__host__ __forceinline__ size_t index_bytes(size_t slots) { return ((1 + slots) * sizeof(int) + 255) / 256 * 256; }

__host__ __forceinline__ Work work_of(void* ws, size_t slots, size_t units, size_t tokens, int d, int p, bool index) {
    Work w;
    w.index = index ? static_cast<int*>(ws) : nullptr;
    w.link = static_cast<unsigned char*>(ws) + index_bytes(slots);
    w.T = reinterpret_cast<float*>(w.link + units * link_bytes(d, p));
    w.P = w.T + units * kC * kC;
    w.U = w.P + units * kC * kC;
    w.E = w.U + units * kC * d;
    w.S = w.E + units * kC * d;
    w.dS = w.S + units * d * d;
    w.meta = reinterpret_cast<Meta*>(w.dS + units * d * d);
    w.dq = reinterpret_cast<float*>(w.meta + units);
    w.dk = w.dq + tokens * d;
    return w;
}

// Whether cu_seqlens is monotone and inside [0, total_T]; finds the spans of N slots, whose n is -1 for an
// unused slot.  All threads take part; contains block barriers.
template <int N>
__device__ bool find_spans(const ChunkBwdArgs& a, const Work& w, const int (&slot)[N], Span (&s)[N]) {
    __shared__ int found[N];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k].n = -1;
    if (!a.cu_seqlens) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (slot[k] >= 0 && w.per > 0) {
                const int n = w.chunks(slot[k]);
                if (n >= a.num_seqs) continue;
                s[k].n = n;
                s[k].bos = (long)n * w.len;
                s[k].eos = s[k].bos + w.len;
                s[k].base = (long)n * w.per;
                s[k].chunks = w.per;
                s[k].c = slot[k] - n * w.per;
            }
        return true;
    }
    int n[N];
    if (const int* index = w.index) {
        if (!index[0]) return false;
#pragma unroll
        for (int k = 0; k < N; ++k) n[k] = slot[k] >= 0 ? index[1 + slot[k]] : -1;
    } else {
        if (threadIdx.x < N) found[threadIdx.x] = -1;
        __syncthreads();
        bool bad = false;
        for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) {
            const int lo = a.cu_seqlens[i], hi = a.cu_seqlens[i + 1];
            bad |= lo < 0 || hi < lo || hi > a.total_T;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const long c = slot[k] - (lo / kC + i);
                if (slot[k] >= 0 && c >= 0 && c * kC < (long)hi - lo) found[k] = i;  // one i at most, where none is bad
            }
        }
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0) record_error(a.err, GDN_ERR_CU_SEQLENS);
            return false;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) n[k] = found[k];
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (n[k] >= 0) {
            s[k] = seq_span(a, n[k]);
            s[k].c = (int)(slot[k] - s[k].base);
        }
    return true;
}

__device__ bool cu_valid(const ChunkBwdArgs& a, const Work& w) {
    const int none[1] = {-1};
    Span s[1];
    return find_spans<1>(a, w, none, s);
}

// ---- decays ------------------------------------------------------------------------------------

// The chunk's cumulative log2-decays and the factors made of them, in shared memory.  The sums are kept
// in two floats: their differences are small beside them, and a rounding of the sum (1e-5 of a difference
// where decays are fast) would be an error of e^(G_i - G_j) itself.
struct Gates {
    float2 G[kC];                         // G log2(e) = x + y
    float b[kC], beta[kC];                // e^G
};

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float decay(float2 gi, float2 gj) { return exp2_approx((gi.x - gj.x) + (gi.y - gj.y)); }

// (x + y) + (u + v) as a pair whose second part is the rounding of the first.
__device__ __forceinline__ float2 add2(float2 p, float2 q) {
    const float s = p.x + q.x, d = s - p.x;
    const float e = ((p.x - (s - d)) + (q.x - d)) + (p.y + q.y);
    const float x = s + e;
    return make_float2(x, e - (x - s));
}

// By one warp, two tokens a lane: raw between fetch and put, as for Rows.
struct GateRows {
    float g[2], beta[2];

    // A log-decay below -128 is taken as -128: e^-128 is zero in fp32 either way, and the sums keep their
    // precision for the tokens behind one that forgets everything (g = -inf included).
    __device__ __forceinline__ void fetch(const ChunkBwdArgs& a, long t0, int len, int h, int lane) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = 2 * lane + e < len;
            g[e] = in ? a.g[(t0 + 2 * lane + e) * a.H + h] : 0.f;
            g[e] = g[e] < -128.f ? -128.f : g[e];
            beta[e] = in ? a.beta[(t0 + 2 * lane + e) * a.H + h] : 0.f;
        }
    }
    __device__ __forceinline__ void put(Gates& t, int lane) const {
        const float2 first = make_float2(g[0], 0.f);
        float2 s = add2(first, make_float2(g[1], 0.f));  // inclusive sums over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float2 x = make_float2(__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o));
            if (lane >= o) s = add2(x, s);
        }
        float2 before = make_float2(__shfl_up_sync(0xffffffffu, s.x, 1), __shfl_up_sync(0xffffffffu, s.y, 1));
        if (lane == 0) before = make_float2(0.f, 0.f);
        const float2 G[2] = {add2(before, first), s};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // times log2(e) = hi + lo
            const float hi = 1.44269502f, lo = 1.92596299e-8f, x = G[e].x * hi;
            const float y = fmaf(G[e].x, hi, -x) + fmaf(G[e].x, lo, G[e].y * hi);
            t.G[2 * lane + e] = make_float2(x, y);
            t.b[2 * lane + e] = expf(G[e].x) * (1.f + G[e].y);
            t.beta[2 * lane + e] = beta[e];
        }
    }
};

// ---- loads -------------------------------------------------------------------------------------

// Four consecutive elements of a q/k/v-like tensor.
__device__ __forceinline__ void load4(const void* src, gdn_dtype dt, long i, float (&x)[4]) {
    if (dt == GDN_BF16) load_vec<4>(static_cast<const __nv_bfloat16*>(src) + i, x);
    else load_vec<4>(static_cast<const float*>(src) + i, x);
}

// A chunk of a token tensor [T, heads, D]: raw in registers between fetch (which only loads) and put, so
// that the loads of several tensors are under way together.  With P = 1 the tensor is bf16.  NW warps take
// part, LPR lanes a row and every row at once, so that a row's norm and maximum are a few shuffles and its
// factors are worked out by its own lanes.  (A warp's 32 lanes on one row after another took 5.4k cycles
// for a 64 x 128 tile, most of them waiting for shuffles.)
template <int NW, int D, int P>
struct Rows {
    static constexpr int LPR = NW / 2, V = P == 1 ? 8 : 4, N = D / LPR / V;  // lanes a row; elements, vectors a lane
    uint4 raw[P == 1 ? N : 1];
    float x[P == 2 ? N : 1][4];

    static __device__ __forceinline__ int row(int warp, int lane) { return warp * (kC / NW) + lane / LPR; }
    // Column of a lane's vector i; odd rows of four lanes take the vectors in another order, so that the
    // eight lanes of a store phase lie in different banks.
    static __device__ __forceinline__ int col(int i, int lane) {
        const int k = LPR == 4 ? i ^ ((lane / LPR) & 1) : i;
        return V * (lane % LPR + LPR * k);
    }

    __device__ __forceinline__ void fetch(const void* src, gdn_dtype dt, long t0, int len, int heads, int h, int warp,
                                          int lane) {
        const int r = row(warp, lane);
        const long at = ((t0 + r) * heads + h) * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (P == 1) {
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < len) raw[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + at + col(i, lane));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
                if (r < len) load4(src, dt, at + col(i, lane), x[i]);
            }
        }
    }

    static __device__ __forceinline__ float2 wide(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }

    // As planes, each row with a power of two of its own (one plane holds bf16 exactly, down to 2^-26 of the
    // row's largest).  factor[r] takes row r of the planes to x (NORM false), or to scale * x / |x| (NORM,
    // use_l2) and scale * x (NORM, not use_l2); inv[r], if given, receives 1 / |x| (1 without).
    // STORE false: the factors only.
    template <bool NORM, bool STORE = true, int LO, int HS>
    __device__ __forceinline__ void put(Mat<D, P, LO, HS> dst, float* factor, float* inv, bool use_l2, float scale,
                                        int warp, int lane) const {
        const int r = row(warp, lane);
        float ss = 0.f;
        uint32_t top = 0;
        if constexpr (P == 1) {
            __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t v = u[e] & 0x7fff7fffu;
                    m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&v));
                    if constexpr (NORM) {
                        const float2 y = wide(u[e]);
                        ss = fmaf(y.x, y.x, fmaf(y.y, y.y, ss));
                    }
                }
            }
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
            top = max(w & 0xffff0000u, w << 16);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    top = max(top, planes::abs_bits(x[i][e]));
                    if constexpr (NORM) ss = fmaf(x[i][e], x[i][e], ss);
                }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if constexpr (NORM) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        const Scale s = planes::scale_of(top);
#pragma unroll
        for (int i = 0; STORE && i < N; ++i) {
            const uint32_t at = dst(r, col(i, lane));
            if constexpr (P == 1) {
                const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = wide(u[e]);
                    const __half2 z = __floats2half2_rn(y.x * s.mul, y.y * s.mul);
                    h[e] = *reinterpret_cast<const uint32_t*>(&z);
                }
                planes::sts128(at, h);
            } else {
                uint32_t hi[2], lo[2];
                planes::split(x[i][0] * s.mul, x[i][1] * s.mul, hi[0], lo[0]);
                planes::split(x[i][2] * s.mul, x[i][3] * s.mul, hi[1], lo[1]);
                planes::sts64(at, hi[0], hi[1]);
                planes::sts64(at + LO, lo[0], lo[1]);
            }
        }
        if (lane % LPR == 0) {
            const float f = NORM && use_l2 ? rsqrtf(ss + kL2Eps) : 1.f;
            factor[r] = (NORM ? f * scale : 1.f) * s.back;
            if (inv) inv[r] = f;
        }
    }
};

// Asks for a stretch of global memory (a multiple of 16 bytes) to be brought into L2.
__device__ __forceinline__ void prefetch(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Asks for the rows of a chunk of one token tensor that a later block will read, LINES of 128 bytes each;
// all T threads.
template <int T, int LINES>
__device__ __forceinline__ void prefetch_lines(const char* src, const Span& s, int heads, int h, int tid) {
    const long t0 = s.bos + (long)s.c * kC;
    const int rows = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const char* first = src + (t0 * heads + h) * (LINES * 128);
#pragma unroll
    for (int i = tid; i < kC * LINES; i += T)
        if (i / LINES < rows)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(first + (long)(i / LINES) * heads * (LINES * 128) + i % LINES * 128));
}
template <int T, int D>
__device__ __forceinline__ void prefetch_rows(const void* src, gdn_dtype dt, const Span& s, int heads, int h, int tid) {
    if (dt == GDN_BF16) prefetch_lines<T, D / 64>(static_cast<const char*>(src), s, heads, h, tid);
    else prefetch_lines<T, D / 32>(static_cast<const char*>(src), s, heads, h, tid);
}

// The same of its g and beta, a token a thread.
__device__ __forceinline__ void prefetch_gates(const ChunkBwdArgs& a, const Span& s, int h, int tid) {
    const long t = s.bos + (long)s.c * kC + tid;
    if (tid < kC && t < s.eos) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.g + t * a.H + h));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.beta + t * a.H + h));
    }
}

// Blocks of one chunk each run for tens of microseconds with few loads of their own under way, so each
// asks for the inputs of the block that will follow it on its SM (about kSMs x blocks an SM later).
constexpr int kSMs = 152;

// ---- prep ----------------------------------------------------------------------------------------

constexpr int kPrepThreads = 256;

constexpr int kLd = kC + 4;  // row of a 64 x 64 fp32 matrix in shared memory (16-byte aligned rows)

// X = (I + A)^-1 for strictly lower triangular A (X's upper triangle is scratch): the four 16 x 16
// diagonal blocks by substitution, a warp each and a column a lane, then twice the block below two
// inverted neighbours, X21 = -X22 (A21 X11).  Warps 4 .. 7, idle during the substitution, call `meanwhile`.
template <class Fn>
__device__ __forceinline__ void unit_lower_inverse(const float* A, float* X, Fn meanwhile) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto row4 = [](const float* p, int i, int j) { return *reinterpret_cast<const float4*>(p + i * kLd + j); };
    if (warp < 4) {
        const int o = 16 * warp, c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc[2] = {i == c ? 1.f : 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 v = row4(A, o + i, o + m);
                const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4 && m + k < i; ++k) acc[k & 1] = fmaf(-r[k], x[m + k], acc[k & 1]);
            }
            x[i] = acc[0] + acc[1];
            if (lane < 16) X[(o + i) * kLd + o + c] = x[i];  // zero above the diagonal
        }
    } else {
        meanwhile();
    }
    __syncthreads();
#pragma unroll
    for (int e = tid; e < 512; e += kPrepThreads) {  // two pairs of 16-blocks
        const int o = (e >> 8) * 32, r = (e >> 4) & 15, c = e & 15;
        float acc = 0.f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 v = row4(A, o + 16 + r, o + m);
            const float* x = X + (o + m) * kLd + o + c;
            acc = fmaf(v.x, x[0], fmaf(v.y, x[kLd], fmaf(v.z, x[2 * kLd], fmaf(v.w, x[3 * kLd], acc))));
        }
        X[(o + r) * kLd + o + 16 + c] = acc;
    }
    __syncthreads();
#pragma unroll
    for (int e = tid; e < 512; e += kPrepThreads) {
        const int o = (e >> 8) * 32, r = (e >> 4) & 15, c = e & 15;
        float acc = 0.f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 v = row4(X, o + 16 + r, o + 16 + m);
            const float* y = X + (o + m) * kLd + o + 16 + c;
            acc = fmaf(v.x, y[0], fmaf(v.y, y[kLd], fmaf(v.z, y[2 * kLd], fmaf(v.w, y[3 * kLd], acc))));
        }
        X[(o + 16 + r) * kLd + o + c] = -acc;
    }
    __syncthreads();
    // the pair of 32-blocks: a warp four rows, a lane a column; scratch above X11's diagonal blocks is skipped
    const int c = lane, r0 = 4 * warp;
    {
        float acc[4] = {};
#pragma unroll
        for (int m = 0; m < 32; m += 4) {
            const float* p = X + m * kLd + c;
            const bool in = m >= 16 || c < 16;
            const float x[4] = {in ? p[0] : 0.f, in ? p[kLd] : 0.f, in ? p[2 * kLd] : 0.f, in ? p[3 * kLd] : 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = row4(A, 32 + r0 + i, m);
                acc[i] = fmaf(v.x, x[0], fmaf(v.y, x[1], fmaf(v.z, x[2], fmaf(v.w, x[3], acc[i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[(r0 + i) * kLd + 32 + c] = acc[i];
    }
    __syncthreads();
    {
        float acc[4] = {};
#pragma unroll
        for (int m = 0; m < 32; m += 4) {
            if (m >= 16 && r0 < 16) break;  // X22's scratch block
            const float* p = X + m * kLd + 32 + c;
            const float y[4] = {p[0], p[kLd], p[2 * kLd], p[3 * kLd]};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = row4(X, 32 + r0 + i, 32 + m);
                acc[i] = fmaf(v.x, y[0], fmaf(v.y, y[1], fmaf(v.z, y[2], fmaf(v.w, y[3], acc[i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[(32 + r0 + i) * kLd + c] = -acc[i];
    }
    __syncthreads();
}

// N scaled elements of row r from column c (both multiples of eight) into the planes of a 64 x 64 matrix.
template <int N, int LO>
__device__ __forceinline__ void put_part(Mat<kC, 2, LO, 0> dst, int r, int c, const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) planes::split(x[i + 2 * j], x[i + 2 * j + 1], hi[j], lo[j]);
        planes::sts128(dst(r, c + i), hi);
        planes::sts128(dst(r, c + i) + LO, lo);
    }
}

// Copies N * 16 bytes from shared to global memory, T threads.
template <int N, int T>
__device__ __forceinline__ void copy_out(unsigned char* dst, const unsigned char* src, int tid) {
    static_assert(N % T == 0, "");
#pragma unroll
    for (int i = 0; i < N / T; ++i)
        reinterpret_cast<uint4*>(dst)[i * T + tid] = reinterpret_cast<const uint4*>(src)[i * T + tid];
}

// The largest magnitudes of a warp's part of its rows into tops[column of warps][row].
template <int MT, int NT>
__device__ __forceinline__ void row_tops(uint32_t* tops, const float (&acc)[MT][NT][4], const int (&m)[MT], int nw, int lane) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) top = max(top, planes::abs_bits(acc[i][j][2 * h + e]));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if ((lane & 3) == 0) tops[nw * kC + m[i] + (lane >> 2) + 8 * h] = top;
        }
}
__device__ __forceinline__ Scale row_scale(const uint32_t* tops, int r) {
    return planes::scale_of(max(max(tops[r], tops[kC + r]), max(tops[2 * kC + r], tops[3 * kC + r])));
}

// Shared memory: K, V, Q (P planes each; the two planes of Q' go over V and Q), a 64 x 64 matrix (T with
// factors, then P) and a 64 x d buffer (W, then dY); before them, over both, A and T in fp32.  d = 128 in
// bf16 takes 96 KB, so two blocks share an SM and one works while the other waits at a barrier.
// No pipe is full (185 us at the sizes above: tensor pipe 26%, shared memory 50%, issue slots 38%, DRAM
// 2.5 TB/s): what is left is the latency of a chunk's dependent steps.  Blocks that stay on their SM took
// 210 us (what the loop keeps in registers spills).
template <int D, int P>
struct PrepSmem {
    static constexpr int plane = kC * D * 2, square = kC * kC * 2, fp32 = 2 * kC * kLd * 4 - 2 * square;
    static constexpr int K = 0, V = P * plane, Q = 2 * P * plane, TX = 3 * P * plane, W = TX + 2 * square;
    static constexpr int bytes = W + (2 * plane > fp32 ? 2 * plane : fp32);
};

template <int D, int P>
__global__ void __launch_bounds__(kPrepThreads, P == 1 ? 2 : 1) chunk_bwd_prep_kernel(ChunkBwdArgs a, Work w) {
    using L = PrepSmem<D, P>;
    constexpr int NW = kPrepThreads / 32, PL = L::plane, SQ = L::square, HS = kC * 128;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ Gates t;
    __shared__ float fK[kC], fQ[kC], fY[kC], fV[kC];
    __shared__ float back_u[kC], back_w[kC];
    __shared__ uint32_t red[2][NW], w_tops[4 * kC];
    const int ahead = blockIdx.x + 2 * kSMs, next = ahead < (int)gridDim.x ? ahead : -1;
    const int slots[2] = {w.heads(blockIdx.x), next < 0 ? -1 : w.heads(next)};
    const long slot = slots[0];
    Span spans[2];
    if (!find_spans<2>(a, w, slots, spans) || spans[0].n < 0) return;
    const Span& s = spans[0];
    const int h = blockIdx.x - slots[0] * a.H, hk = w.rep(h), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long t0 = s.bos + (long)s.c * kC, unit = slot * a.H + h;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    const Mat<D, P, PL, HS> K{base + L::K}, V{base + L::V}, Q{base + L::Q}, Y{base + L::W};
    const Mat<D, 2, PL, HS> Qp{base + L::V}, W{base + L::W};
    const Mat<kC, 2, SQ, 0> TX{base + L::TX};
    float *Af = reinterpret_cast<float*>(sm + L::TX), *Tf = Af + kC * kLd;
    unsigned char* link = w.link + unit * link_bytes(D, P);
    LinkTail& tail = *reinterpret_cast<LinkTail*>(link + (2 + P) * PL);

    {
        GateRows gates;
        if (warp == NW - 1) gates.fetch(a, t0, len, h, lane);
        Rows<NW, D, P> k, v, q;
        k.fetch(a.k, a.qkv_dtype, t0, len, a.Hk, hk, warp, lane);
        q.fetch(a.q, a.qkv_dtype, t0, len, a.Hk, hk, warp, lane);
        v.fetch(a.v, a.qkv_dtype, t0, len, a.H, h, warp, lane);
        if (warp == NW - 1) gates.put(t, lane);
        k.template put<true>(K, fK, nullptr, a.use_l2, 1.f, warp, lane);
        q.template put<true>(Q, fQ, nullptr, a.use_l2, a.scale, warp, lane);
        v.template put<false>(V, fV, nullptr, false, 1.f, warp, lane);
    }
    __syncthreads();

    // Warps 2 x 4 over a 64-row result.  A warp's two row tiles are mw and 3 - mw, which gives both rows
    // of warps the same share of a triangular product.
    const int mw = warp >> 2, nw = warp & 3;
    const int m[2] = {16 * mw, 16 * (3 - mw)};
    constexpr int NT = D / 32;
    const int nd = nw * (D / 4), nc = nw * 16;
    {
        float kk[2][2][4];
        planes::clear(kk);
        planes::product<D, false, false>(kk, K, m, K, nc, lane);
        planes::pairs<2, 2>(m, nc, lane, [&](int i, int j, int hh, int r, int c) {
            const float f = t.beta[r] * fK[r];
            const float2 gr = t.G[r];
            *reinterpret_cast<float2*>(Af + r * kLd + c) =
                make_float2(c < r ? kk[i][j][2 * hh] * (f * fK[c]) * decay(gr, t.G[c]) : 0.f,
                            c + 1 < r ? kk[i][j][2 * hh + 1] * (f * fK[c + 1]) * decay(gr, t.G[c + 1]) : 0.f);
        });
    }
    __syncthreads();
    unit_lower_inverse(Af, Tf, [&] {
        constexpr int half = kPrepThreads / 2;
        const int th = tid - half;
        copy_out<P * PL / 16, half>(link + 2 * PL, sm + L::K, th);
        if (th < kC) tail.c[th] = decay(t.G[kC - 1], t.G[th]) * fK[th];
        if (spans[1].n < 0) return;
        const int h2 = next - slots[1] * a.H, hk2 = w.rep(h2);
        prefetch_rows<half, D>(a.k, a.qkv_dtype, spans[1], a.Hk, hk2, th);
        prefetch_rows<half, D>(a.q, a.qkv_dtype, spans[1], a.Hk, hk2, th);
        prefetch_rows<half, D>(a.v, a.qkv_dtype, spans[1], a.H, h2, th);
        prefetch_rows<half, D>(a.dout, a.dout_dtype, spans[1], a.H, h2, th);
        prefetch_gates(a, spans[1], h2, th);
    });

    // T to the workspace; T diag(beta) and T diag(beta b) (with the rows' factors of V and K) as the left
    // sides of U and W, each row with a power of two of its own: a row contracts over its own and earlier
    // tokens, and keeps its accuracy beside later ones whose v is larger
    float tr[16];
    const int rr = tid >> 2, rc = (tid & 3) * 16;
    float mul_u, mul_w;
    {
        uint32_t m1 = 0, m2 = 0;
#pragma unroll
        for (int i = 0; i < 16; i += 4) load_vec<4>(Tf + rr * kLd + rc + i, tr + i);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int j = rc + i;
            tr[i] = j <= rr ? tr[i] : 0.f;
            if (j <= rr) w.T[(unit * kC + j) * kC + rr] = tr[i];
            tr[i] *= t.beta[j];
            m1 = max(m1, planes::abs_bits(tr[i] * fV[j]));
            m2 = max(m2, planes::abs_bits(tr[i] * (t.b[j] * fK[j])));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {  // a row's four lanes
            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        }
        const Scale su = planes::scale_of(m1), sk = planes::scale_of(m2);
        mul_u = su.mul;
        mul_w = sk.mul;
        if (rc == 0) {
            back_u[rr] = su.back;
            back_w[rr] = sk.back;
        }
    }
    __syncthreads();
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = tr[i] * fV[rc + i] * mul_u;
        put_part(TX, rr, rc, x);
    }
    __syncthreads();
    float acc[2][NT][4];
    planes::clear(acc);
    planes::product<kC, false, true, planes::kLower>(acc, TX, m, V, nd, lane);
    planes::pairs<2, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int c) {
        w.U[(unit * D + c) * kC + r] = acc[i][j][2 * hh] * back_u[r];
        w.U[(unit * D + c + 1) * kC + r] = acc[i][j][2 * hh + 1] * back_u[r];
    });
    __syncthreads();
    {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = tr[i] * (t.b[rc + i] * fK[rc + i]) * mul_w;
        put_part(TX, rr, rc, x);
    }
    __syncthreads();
    planes::clear(acc);
    planes::product<kC, false, true, planes::kLower>(acc, TX, m, K, nd, lane);
    planes::pairs<2, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int) {
        acc[i][j][2 * hh] *= back_w[r];
        acc[i][j][2 * hh + 1] *= back_w[r];
    });
    row_tops(w_tops, acc, m, nw, lane);
    float qk[2][2][4];  // P
    planes::clear(qk);
    planes::product<D, false, false>(qk, Q, m, K, nc, lane);
    planes::pairs<2, 2>(m, nc, lane, [&](int i, int j, int hh, int r, int c) {
        const float2 gr = t.G[r];
        float &x = qk[i][j][2 * hh], &y = qk[i][j][2 * hh + 1];
        x = c <= r ? x * (fQ[r] * fK[c]) * decay(gr, t.G[c]) : 0.f;
        y = c + 1 <= r ? y * (fQ[r] * fK[c + 1]) * decay(gr, t.G[c + 1]) : 0.f;
        if (c == r) w.meta[unit].p_diag[r] = x;
        if (c + 1 == r) w.meta[unit].p_diag[r] = y;
        if (c <= r) w.P[(unit * kC + c) * kC + r] = x;
        if (c + 1 <= r) w.P[(unit * kC + c + 1) * kC + r] = y;
    });
    {
        const uint32_t top = planes::max_bits(qk);
        if (lane == 0) red[0][warp] = top;
    }
    __syncthreads();
    const Scale sp = planes::scale_of(planes::top_of<NW>(red[0], lane));
    // W's rows have powers of two of their own: beside the first rows' the later ones' decays may be anything.
    // P W contracts over them, so they go into P's columns (as shares of the largest).
    const float w0 = row_scale(w_tops, lane).back, w1 = row_scale(w_tops, lane + 32).back;
    const float w_top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(w0, w1))));
    {
        float mul[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) mul[i][hh] = row_scale(w_tops, m[i] + (lane >> 2) + 8 * hh).mul;
        planes::write(W, acc, m, nd, lane, mul);
        if (warp == 0) {
            tail.w[lane] = w0;
            tail.w[lane + 32] = w1;
        }
        const float share = (nw < 2 ? w0 : w1) * (1.f / w_top);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = __shfl_sync(0xffffffffu, share, (nc + 8 * j + (lane & 3) * 2 + e) & 31) * sp.mul;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qk[i][j][e] *= f;
                    qk[i][j][2 + e] *= f;
                }
            }
        planes::write(TX, qk, m, nc, lane, 1.f);
    }
    Rows<NW, D, P> y;
    y.fetch(a.dout, a.dout_dtype, t0, len, a.H, h, warp, lane);
    __syncthreads();
    planes::clear(acc);  // Q' = diag(b) Q - P W
    planes::product<kC, false, true, planes::kLower>(acc, TX, m, W, nd, lane);
    planes::pairs<2, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int) {
        const float2 q = planes::read<NT>(Q, m[i], nd, j, hh, lane);
        const float f = t.b[r] * fQ[r], p = w_top * sp.back;
        acc[i][j][2 * hh] = f * q.x - p * acc[i][j][2 * hh];
        acc[i][j][2 * hh + 1] = f * q.y - p * acc[i][j][2 * hh + 1];
    });
    copy_out<2 * PL / 16, kPrepThreads>(link, sm + L::W, tid);
    if (tid == 0) {
        tail.b_last = t.b[kC - 1];
    }
    __syncthreads();  // W, V and Q have been read
    y.template put<false>(Y, fY, nullptr, false, 1.f, warp, lane);
    __syncthreads();
    planes::pairs<2, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int) {
        acc[i][j][2 * hh] *= fY[r];
        acc[i][j][2 * hh + 1] *= fY[r];
    });
    {
        const uint32_t top = planes::max_bits(acc);
        if (lane == 0) red[1][warp] = top;
    }
    __syncthreads();
    const Scale sq = planes::scale_of(planes::top_of<NW>(red[1], lane));
    planes::write(Qp, acc, m, nd, lane, sq.mul);
    __syncthreads();
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {  // X = dY^T Q', 32 rows of a warp at a time
        const int mx[2] = {mw * (D / 2) + 32 * half, mw * (D / 2) + 32 * half + 16};
        planes::clear(acc);
        planes::product<kC, true, true>(acc, Y, mx, Qp, nd, lane);
        planes::pairs<2, NT>(mx, nd, lane, [&](int i, int j, int hh, int r, int c) {
            *reinterpret_cast<float2*>(w.dS + (unit * D + r) * D + c) =
                make_float2(acc[i][j][2 * hh] * sq.back, acc[i][j][2 * hh + 1] * sq.back);
        });
    }
}

// ---- scan ----------------------------------------------------------------------------------------
// Two warps keep 16 rows of the state in their accumulators for the whole sequence, half the columns each:
// an accumulator's layout is the left operand's layout of the next product, so the state never passes
// through shared memory, and rows do not depend on one another.  Per chunk, forwards:
// U^T = (T diag(beta) V)^T - S W^T, then S <- b_C S + U^T Kd; backwards: E^T = dS Kd^T, then
// dS <- b_C dS + X - E^T W.  The first product is split over the inner dimension, each warp taking its own
// columns of the state, and the two parts meet through shared memory; both warps then hold the whole of
// U^T or E^T (16 x 64) and take the second product for their own columns.  A pair has one barrier a step,
// between its writes of the parts and their reads, and two places for the parts, used in turn: a warp that
// writes a place again has met the next step's barrier, which its partner reaches only after reading it.
// The chunks' links arrive by bulk copies; each pair of warps waits for a link and gives it back by itself, so
// that pairs drift apart and one sub-partition's two warps (of two pairs) are not in the same phase.
// At the sizes above 128 blocks take 64 steps of 3.4 us (6.4k cycles); MMAs fill 41% of it, the rest is the
// splitting of S and Z into planes and the wait for the other half.  With the links copied by all warps
// between block barriers it took 252 us; with the transposed state on tcgen05, 250 us: its products have
// N = 64 and are bound by reading the left side from shared memory (56 cycles each).

constexpr int kScanThreads = 256;
constexpr int scan_stages(int d, int p) { return d == 128 && p == 2 ? 2 : 3; }
constexpr int kParts = 8 * 16 * kC * 4;  // one part of Z of each warp
constexpr int scan_bytes(int d, int p) { return scan_stages(d, p) * (int)link_bytes(d, p) + 2 * kParts + 64; }
constexpr uint64_t kWaitNs = 2000000000ull;  // bound on one barrier wait

// N[j] += rows (16 x 16 KT, in the accumulator layout) times B from column n0 and inner index k0: the
// rows' planes are made here, scaled by mul (one power of two for each of this thread's two rows).  An SM
// sub-partition has two warps only: the blocks of B for the next step are loaded before this step's
// products, and the terms of one accumulator lie NT products apart.
template <bool TB, int KT, int NT, int CB, int PB, int LB, int HB>
__device__ __forceinline__ void row_product(float (&N)[NT][4], const float (&rows)[2 * KT][4], const float (&mul)[2],
                                            Mat<CB, PB, LB, HB> B, int n0, int k0, int lane) {
    const uint32_t lb = planes::lane_b<TB>(B, lane);
    uint32_t b[2][PB][NT / 2][4];
    auto load = [&](uint32_t (&x)[PB][NT / 2][4], int k) {
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
            planes::load_b<TB, 0, HB>(x[0][j], lb, n0 + 16 * j, k0 + 16 * k);
            if constexpr (PB == 2) planes::load_b<TB, LB, HB>(x[1][j], lb, n0 + 16 * j, k0 + 16 * k);
        }
    };
    load(b[0], 0);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        if (k + 1 < KT) load(b[(k + 1) & 1], k + 1);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            planes::split(rows[2 * k + e][0] * mul[0], rows[2 * k + e][1] * mul[0], hi[2 * e], lo[2 * e]);
            planes::split(rows[2 * k + e][2] * mul[1], rows[2 * k + e][3] * mul[1], hi[2 * e + 1], lo[2 * e + 1]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) planes::mma(N[j], hi, b[k & 1][0][j / 2][2 * (j & 1)], b[k & 1][0][j / 2][2 * (j & 1) + 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) planes::mma(N[j], lo, b[k & 1][0][j / 2][2 * (j & 1)], b[k & 1][0][j / 2][2 * (j & 1) + 1]);
        if constexpr (PB == 2) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                planes::mma(N[j], hi, b[k & 1][1][j / 2][2 * (j & 1)], b[k & 1][1][j / 2][2 * (j & 1) + 1]);
        }
    }
}

// The scales of this thread's two rows (spread over the four lanes of a quad) and the largest magnitude
// of the warp's sixteen.
template <int NT>
__device__ __forceinline__ uint32_t row_scales(const float (&x)[NT][4], Scale (&s)[2]) {
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = max(top[e >> 1], planes::abs_bits(x[j][e]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        s[i] = planes::scale_of(top[i]);
    }
    return __reduce_max_sync(0xffffffffu, max(top[0], top[1]));
}

template <int D, int P, bool BACK>
__device__ __forceinline__ void scan(const ChunkBwdArgs& a, const Work& w, const Span& s, int h, int slice,
                                     unsigned char* sm) {
    constexpr int NT = D / 16, ZT = kC / 8, PL = kC * D * 2, LINK = (int)link_bytes(D, P), ST = scan_stages(D, P);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pair = warp >> 1, half = warp & 1;
    const int block = slice * 4 + pair, row = block * 16 + (lane >> 2), c2 = (lane & 3) * 2, n0 = half * (D / 2);
    const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    // parts of Z, [2][warps][ZT][32]: even steps, odd steps
    float4* parts = reinterpret_cast<float4*>(sm + ST * LINK) + (warp * ZT) * 32 + lane;
    const int to_other = (warp & 1 ? -1 : 1) * ZT * 32;
    const long state = ((long)s.n * a.H + h) * D * D + row * D + n0 + c2;
    const float* from = BACK ? a.dfinal_state : a.initial_state;
    auto unit_of = [&](int i) { return (s.base + (BACK ? s.chunks - 1 - i : i)) * a.H + h; };
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + ST * LINK + 2 * kParts);
    uint64_t* empty = full + ST;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], kScanThreads / 32);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    // A wait that gives up is recorded, and this thread waits no more: what it computes from then on is
    // meaningless but stays in its own places, and the kernel ends.
    bool ok = true;
    auto wait = [&](uint64_t* bar, int use) {
        if (ok && !ptx::mbar_wait(bar, use & 1, kWaitNs)) {
            ok = false;
            record_error(a.err, GDN_ERR_TIMEOUT);
        }
    };
    auto fetch = [&](int i) {  // one thread: the link of chunk i, once chunk i - ST has given its place back
        if (i >= s.chunks) return;
        if (i >= ST) wait(&empty[i % ST], i / ST - 1);
        ptx::mbar_arrive_expect_tx(&full[i % ST], LINK);
        ptx::bulk_load(sm + (i % ST) * LINK, w.link + unit_of(i) * LINK, LINK, &full[i % ST]);
    };
    if (threadIdx.x == 0) fetch(0);
    float S[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const float2 x = from ? *reinterpret_cast<const float2*>(from + state + hh * 8 * D + 8 * j) : make_float2(0.f, 0.f);
            S[j][2 * hh] = x.x;
            S[j][2 * hh + 1] = x.y;
        }
    // what follows the last chunk is wanted only as the gradient of the initial state
    const int steps = BACK && a.dinitial_state ? s.chunks : s.chunks - 1;
    // X of a chunk (backwards), or (T diag(beta) V)^T (forwards): loaded while the chunk before is worked on
    float x[BACK ? NT : ZT][4];
    auto load_x = [&](int i) {
        if (i >= s.chunks) return;
        const float* p = BACK ? w.dS + unit_of(i) * D * D + row * D + n0 + c2 : w.U + (unit_of(i) * D + row) * kC + c2;
#pragma unroll
        for (int j = 0; j < (BACK ? NT : ZT); ++j)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) load_vec<2>(p + hh * 8 * (BACK ? D : kC) + 8 * j, x[j] + 2 * hh);
    };
    // this block's rows of them, and its half or whole of a link, in L2 some steps before
    constexpr int AHEAD = 4;
    auto ask = [&](int i) {
        if (i >= s.chunks) return;
        if (BACK) prefetch(w.dS + (unit_of(i) * D + slice * 64) * D, 64 * D * 4);
        else prefetch(w.U + (unit_of(i) * D + slice * 64) * kC, 64 * kC * 4);
        prefetch(w.link + unit_of(i) * LINK + slice * (LINK / (D / 64) / 16 * 16), LINK / (D / 64) / 16 * 16);
    };
    if (threadIdx.x == 32)
        for (int i = 1; i < AHEAD; ++i) ask(i);
    load_x(0);
    for (int i = 0; i < s.chunks; ++i) {
        if (threadIdx.x == 32) ask(i + AHEAD);
        const long unit = unit_of(i);
        float4* mine = parts + (i & 1) * (kParts / 16);
        const float4* other = mine + to_other;
        float* kept = (BACK ? w.dS : w.S) + unit * D * D + row * D + n0 + c2;
        float* side = (BACK ? w.E : w.U) + (unit * D + row) * kC + c2;
        if (threadIdx.x == 0) fetch(i + 1);
        __syncwarp();
        wait(&full[i % ST], i / ST);
        const uint32_t at = smem + (i % ST) * LINK;
        const LinkTail& tail = *reinterpret_cast<const LinkTail*>(sm + (i % ST) * LINK + (2 + P) * PL);
        const Mat<D, 2, PL, kC * 128> W{at};
        const Mat<D, P, PL, kC * 128> K{at + 2 * PL};
        Scale rs[2], zs[2];
        const uint32_t top = row_scales(S, rs);
        if (lane == 0) (BACK ? w.meta[unit].ds_max : w.meta[unit].s_max)[block * 2 + half] = top;
        const float mul[2] = {rs[0].mul, rs[1].mul};
        float Z[ZT][4];
#pragma unroll
        for (int j = 0; j < ZT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) Z[j][e] = 0.f;
        if constexpr (BACK) row_product<false, NT / 2>(Z, S, mul, K, 0, n0, lane);
        else row_product<false, NT / 2>(Z, S, mul, W, 0, n0, lane);
        const float f[2] = {rs[0].back, rs[1].back};
#pragma unroll
        for (int j = 0; j < ZT; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) Z[j][e] *= f[e >> 1];
            mine[j * 32] = make_float4(Z[j][0], Z[j][1], Z[j][2], Z[j][3]);
        }
        asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
#pragma unroll
        for (int j = 0; j < ZT; ++j) {
            const float4 o = other[j * 32];
            const float2 c = *reinterpret_cast<const float2*>(tail.c + 8 * j + c2);
            const float2 wf = *reinterpret_cast<const float2*>(tail.w + 8 * j + c2);
            const float y[4] = {o.x, o.y, o.z, o.w};
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float cj = e & 1 ? c.y : c.x, wj = e & 1 ? wf.y : wf.x;
                if constexpr (BACK) {
                    v[e] = (Z[j][e] + y[e]) * cj;
                    Z[j][e] = -v[e] * wj;
                } else {
                    v[e] = fmaf(Z[j][e] + y[e], -wj, x[j][e]);
                    Z[j][e] = v[e] * cj;
                }
            }
            if ((j < ZT / 2) == (half == 0)) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    *reinterpret_cast<float2*>(side + hh * 8 * kC + 8 * j) = make_float2(v[2 * hh], v[2 * hh + 1]);
            }
        }
        if constexpr (!BACK) load_x(i + 1);
        float N[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) N[j][e] = 0.f;
        float zb[2] = {0.f, 0.f};
        if (i < steps) {
            row_scales(Z, zs);
            const float zmul[2] = {zs[0].mul, zs[1].mul};
            zb[0] = zs[0].back;
            zb[1] = zs[1].back;
            if constexpr (BACK) row_product<true, ZT / 2>(N, Z, zmul, W, n0, 0, lane);
            else row_product<true, ZT / 2>(N, Z, zmul, K, n0, 0, lane);
        }
        const float b_last = tail.b_last;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&empty[i % ST]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
                *reinterpret_cast<float2*>(kept + hh * 8 * D + 8 * j) = make_float2(S[j][2 * hh], S[j][2 * hh + 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[j][e] = fmaf(N[j][e], zb[e >> 1], BACK ? fmaf(b_last, S[j][e], x[j][e]) : b_last * S[j][e]);
        }
        if constexpr (BACK) load_x(i + 1);
    }
    if (threadIdx.x == 0 && !ok)  // no copy may still be on its way when the block ends
        for (int i = s.chunks > ST ? s.chunks - ST : 0; i < s.chunks; ++i) ptx::mbar_wait(&full[i % ST], (i / ST) & 1, kWaitNs);
    if (BACK && a.dinitial_state) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
                *reinterpret_cast<float2*>(a.dinitial_state + state + hh * 8 * D + 8 * j) =
                    make_float2(S[j][2 * hh], S[j][2 * hh + 1]);
    }
}

template <int D, int P>
__global__ void __launch_bounds__(kScanThreads, 1) chunk_bwd_scan_kernel(ChunkBwdArgs a, Work w) {
    extern __shared__ __align__(1024) unsigned char sm[];
    constexpr int slices = D / 64;
    if (!cu_valid(a, w)) return;
    dependency_wait();
    const int unit = blockIdx.x / slices, slice = blockIdx.x % slices;
    const Span s = seq_span(a, unit / a.H);
    if (blockIdx.y) scan<D, P, true>(a, w, s, unit % a.H, slice, sm);
    else scan<D, P, false>(a, w, s, unit % a.H, slice, sm);
}

// ---- grad ----------------------------------------------------------------------------------------
// P comes from the preparation.  The small products up to dR run on warp-level MMAs; those with the states,
// with U and with K and Q on tcgen05, whose accumulators (TMEM) leave the registers, and whose operands are read from shared memory
// once per block instead of once per warp.  They are stacked so that M = 128 is full:
//   D1 = [dY; dR] S0            rows 0 .. 63: dQ's, rows 64 .. 127: F's part from the state
//   NZ = [dY; dR] U^T           dP and Z before their decays
//   D2 = [dP; Z] K              with K's row factors folded into dP's and Z's columns
//   D3 = dP^T Q + (diag(beta) Z)^T K,  HH = U dS1:  the hi plane of the left side in rows 0 .. 63, its lo
//        plane in rows 64 .. 127, to be added up
// A thread then has one token's row: of dQ (TMEM lanes 0 .. 63) or of F and dK (lanes 64 .. 127), and 32
// columns of it.
// 304 us at the sizes above: some 38k cycles a chunk, 10k of them until its first tiles are in place; tensor
// pipe 14%, issue slots 39%, DRAM 2.5 TB/s.  What brought it there, from 398 us: the products on tcgen05 (351),
// P from the preparation (320), E's and v's loads a phase earlier (314), T, P, E and S0 by bulk copies instead
// of through registers (302), no divisions, and no wait for TMEM or v, at a block's start (289);
// scales by rows and columns instead of one a tile took it to 304.  Blocks that
// stay on their SM took 382 against 320 us with the chunk in the loop (spills) and 447 as a function of its own.

constexpr uint64_t kMmaWaitNs = 2000000000ull;

// Shared memory.  YR holds dY (rows 0 .. 63) above dR (rows 64 .. 127), two planes; later dP^T's and Z^T's
// left sides go where dR was, and with `share` Q comes and goes in dY's place.  ST holds S0, then dS1, then
// the rows that pass from one half of the lanes to the other.  SQ holds P^T's planes, then T^T's, beside T^T
// in fp32 (P^T comes in fp32 to dR's place), then maxima and scales (at SQ + TMP), then dP above Z.  B1 holds
// E, then P^T dY + E, then U^T, then the row sums.
//
// A token's results have to hold beside those of any other token of the chunk, whose dY may be larger by any
// factor, and so may v (and U): what has a row a token gets a power of two a row.  dY_i, dR_i and
// (P^T dY + E)_i carry theirs where they are right sides too: there the other side's column i is multiplied by
// it in fp32, before its own rows are scaled and split (tri_planes; dP^T Q and Z^T K have their scales by
// columns for the same reason).
template <int D, int P>
struct GradSmem {
    // d = 64: two blocks share an SM, which takes Q out; d = 128 in fp32 needs the room as well
    static constexpr bool share = P == 2 || D == 64;
    // room for diag(beta) Z beside dP^T's left side, or only after U has been used
    static constexpr bool late = D == 64;
    static constexpr int H2 = D / 64, half = kC * 128, plane = half * H2, yr = 2 * plane, st = D * 128 * H2;
    static constexpr int K = 0, Q = P * plane, YR = share ? Q : 2 * P * plane;
    static constexpr int ST = YR + 2 * yr, SQ = ST + 2 * st, B1 = SQ + 4 * half, bytes = B1 + 2 * plane;
    // at TMP: maxima of dR's rows [4][64], scales of dR and of U [2][64], maxima of dP's and Z's rows [column
    // group][128] and columns [4][64]
    static constexpr int TMP = 2 * half, tRows = TMP, tScale = TMP + 1024, tPZ = TMP + 2048, tCols = TMP + 4096;
    static constexpr int WM = D / 32, threads = WM * 128;
    // TMEM columns: D1, D2, D3, then NZ and HH in turn
    static constexpr int tD1 = 0, tD2 = D, tD3 = 2 * D, tNZ = 3 * D, tmem = 4 * D;
};

// An fp32 matrix of ROWS x COLS, raw in registers between fetch and put.  put writes its planes with the
// given scale; with DOT it returns this thread's part of the dot product with what the planes held before,
// without its scale.
template <int T, int ROWS, int COLS>
struct Flat {
    static constexpr int N = ROWS * COLS / 4 / T;
    float x[N][4];

    __device__ __forceinline__ void fetch(const float* src) {
#pragma unroll
        for (int p = 0; p < N; ++p) load_vec<4>(src + (p * T + threadIdx.x) * 4, x[p]);
    }
    template <bool DOT, int LO, int HS>
    __device__ __forceinline__ float put(Mat<COLS, 2, LO, HS> dst, float mul) const {
        const float by[4] = {mul, mul, mul, mul};
        return put<DOT>(dst, by);
    }
    template <bool DOT, int LO, int HS>  // a scale for each of this thread's four columns (the same in every row)
    __device__ __forceinline__ float put(Mat<COLS, 2, LO, HS> dst, const float (&mul)[4]) const {
        static_assert(T * 4 % COLS == 0, "");
        float dot = 0.f;
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int e = (p * T + threadIdx.x) * 4;
            const uint32_t at = dst(e / COLS, e % COLS);
            if constexpr (DOT) {
                uint32_t u[2], v[2];
                planes::lds64(at, u[0], u[1]);
                planes::lds64(at + LO, v[0], v[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 hi = planes::halves(u[i]), lo = planes::halves(v[i]);
                    dot = fmaf(hi.x + lo.x, x[p][2 * i], dot);
                    dot = fmaf(hi.y + lo.y, x[p][2 * i + 1], dot);
                }
            }
            uint32_t hi[2], lo[2];
            planes::split(x[p][0] * mul[0], x[p][1] * mul[1], hi[0], lo[0]);
            planes::split(x[p][2] * mul[2], x[p][3] * mul[3], hi[1], lo[1]);
            planes::sts64(at, hi[0], hi[1]);
            planes::sts64(at + LO, lo[0], lo[1]);
        }
        return dot;
    }
};

// A pair of elements of a q/k/v-like tensor, kept as it is in memory until it is wanted (with P = 1 the tensor
// is bf16): a conversion behind the load would wait for it.
template <int P>
struct Pair {
    uint32_t raw;
    __device__ __forceinline__ void load(const void* src, gdn_dtype, long i, bool in) {
        raw = in ? *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(src) + i) : 0u;
    }
    __device__ __forceinline__ float2 value() const {
        return make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u));
    }
};
template <>
struct Pair<2> {
    float x[2];
    __device__ __forceinline__ void load(const void* src, gdn_dtype dt, long i, bool in) {
        x[0] = x[1] = 0.f;
        if (!in) return;
        if (dt == GDN_BF16) load_vec<2>(static_cast<const __nv_bfloat16*>(src) + i, x);
        else load_vec<2>(static_cast<const float*>(src) + i, x);
    }
    __device__ __forceinline__ float2 value() const { return make_float2(x[0], x[1]); }
};
__device__ __forceinline__ void store2(void* dst, gdn_dtype dt, long i, float x, float y) {
    if (dt == GDN_BF16)
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(dst) + i) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<float2*>(static_cast<float*>(dst) + i) = make_float2(x, y);
}
// Eight consecutive elements.
__device__ __forceinline__ void store8(void* dst, gdn_dtype dt, long i, const float (&x)[8]) {
    if (dt == GDN_BF16) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + i) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float* p = static_cast<float*>(dst) + i;
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// f16 x f16 -> f32, dense; a_mn / b_mn select MN-major operands
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 16 consecutive 32-bit TMEM columns of this thread's lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// One pass of tcgen05 MMAs over an inner dimension of 16 STEPS, by one thread: D (+)= A B.  A and B are
// shared addresses of 128-byte-swizzled tiles; MN: stored [inner][outer], blocks of 64 outer elements
// `block` bytes apart; otherwise stored [outer][inner], blocks of 64 inner elements `block` bytes apart.
template <int STEPS, int N, bool AMN, bool BMN>
__device__ __forceinline__ void issue(uint32_t d, uint32_t A, int a_block, uint32_t B, int b_block, bool accumulate) {
    constexpr uint32_t id = idesc_f16(128, N, AMN, BMN);
    // a step adds to the descriptors' start addresses (in units of 16 bytes), which never carry out
    const uint64_t da = ptx::sdesc_sw128(A, AMN ? a_block : 16, 1024), db = ptx::sdesc_sw128(B, BMN ? b_block : 16, 1024);
    const uint32_t a_hi = (uint32_t)(da >> 32), b_hi = (uint32_t)(db >> 32), a_lo = (uint32_t)da, b_lo = (uint32_t)db;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const uint32_t ao = AMN ? k * 2048 : (k >> 2) * a_block + (k & 3) * 32;
        const uint32_t bo = BMN ? k * 2048 : (k >> 2) * b_block + (k & 3) * 32;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
            "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d), "r"(a_lo + (ao >> 4)), "r"(a_hi),
            "r"(b_lo + (bo >> 4)), "r"(b_hi), "r"(id), "r"((uint32_t)(accumulate || k > 0))
            : "memory");
    }
}

// The planes of X diag(f) for an upper triangular X (rows of fp32 at x), each row with a power of two of its
// own: T threads, N elements each (a row's lanes are neighbours), f of this thread's columns.  back[r] takes
// row r of the planes to X diag(f).
template <int T, int LO, int N>
__device__ __forceinline__ void tri_planes(Mat<kC, 2, LO, 0> dst, const float* x, const float (&f)[N], float* back) {
    static_assert(N == kC * kC / T, "");
    constexpr int LPR = kC / N;
    const int r = threadIdx.x / LPR, c = (threadIdx.x % LPR) * N;
    float y[N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; i += 4) load_vec<4>(x + i, y + i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        y[i] = c + i >= r ? y[i] * f[i] : 0.f;  // below the diagonal nothing was written
        top = max(top, planes::abs_bits(y[i]));
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Scale s = planes::scale_of(top);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] *= s.mul;
    put_part(dst, r, c, y);
    if (c == 0) back[r] = s.back;
}

template <int D, int P>
__global__ void __launch_bounds__(GradSmem<D, P>::threads, D == 64 && P == 1 ? 2 : 1)
    chunk_bwd_grad_kernel(ChunkBwdArgs a, Work w) {
    using L = GradSmem<D, P>;
    constexpr int T = L::threads, NW = T / 32, WM = L::WM, MT = 4 / WM, HF = L::half, PL = L::plane, CG = NW / 4;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ Gates t;
    __shared__ __align__(16) float fY[kC];
    __shared__ float fK[kC], fQ[kC], kinv[kC], qinv[kC], dpp[kC], diag[kC];
    uint32_t* u_tops = reinterpret_cast<uint32_t*>(diag);  // of U's tokens, before diag is written
    __shared__ uint32_t tmem_at;
    __shared__ float dots[NW];
    __shared__ uint64_t bars[5];  // of the MMAs; of the copies of T, P and E; of S0's
    const int ahead = blockIdx.x + kSMs, next = ahead < (int)gridDim.x ? ahead : -1;
    const int slots[2] = {w.heads(blockIdx.x), next < 0 ? -1 : w.heads(next)};
    const long slot = slots[0];
    Span spans[2];
    if (!find_spans<2>(a, w, slots, spans) || spans[0].n < 0) return;
    dependency_wait();
    const Span& s = spans[0];
    const int h = blockIdx.x - slots[0] * a.H, hk = w.rep(h), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long t0 = s.bos + (long)s.c * kC, unit = slot * a.H + h;
    const int len = s.eos - t0 < kC ? (int)(s.eos - t0) : kC;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
    constexpr int QHS = L::share ? 2 * HF : HF, QLO = L::share ? L::yr : PL;
    const Mat<D, P, PL, HF> K{base + L::K};
    const Mat<D, P, QLO, QHS> Q{base + L::Q};
    const Mat<D, P, L::yr, 2 * HF> Y{base + L::YR};
    const Mat<D, 2, L::yr, 2 * HF> R{base + L::YR + HF};
    const Mat<D, 2, L::st, D * 128> ST{base + L::ST};
    const Mat<kC, 2, HF, 0> Tri{base + L::SQ};                              // of P^T, then of T^T
    const Mat<kC, 2, 2 * HF, 0> dP{base + L::SQ}, Zm{base + L::SQ + HF};
    const Mat<D, 2, PL, HF> B1{base + L::B1};
    const Mat<kC, 2, PL, 0> UT{base + L::B1};  // U^T
    // the left sides of D3: planes two blocks apart in dR's place; diag(beta) Z in dY's place or, later, in U's
    const Mat<kC, 2, 2 * HF, 0> Pt{base + L::YR + HF};
    constexpr int ZLO = L::late ? HF : 2 * HF;
    const Mat<kC, 2, ZLO, 0> Zt{base + (L::late ? L::B1 : L::YR + 5 * HF)};
    // Warps WM x 4.  With two row tiles a warp's are mw and 3 - mw; with one, the four warps of an SM
    // sub-partition (warp mod 4) are the four row tiles of a column block: either way the shares of a
    // triangular product are even.
    const int mw = warp >> 2, nw = warp & 3;
    int m[MT];
    m[0] = 16 * mw;
    if constexpr (MT == 2) m[1] = 16 * (3 - mw);
    constexpr int NT = D / 32;
    const int nd = nw * (D / 4);
    const Meta& meta = w.meta[unit];
    const float* dS1 = w.dS + unit * D * D;
    auto prefetch_states = [&](long u) {
        prefetch(w.S + u * D * D, D * D * 4);
        prefetch(w.E + u * kC * D, kC * D * 4);
        prefetch(w.U + u * kC * D, kC * D * 4);
        prefetch(w.dS + u * D * D, D * D * 4);
    };
    if (tid == 0) {
        if (blockIdx.x < kSMs) prefetch_states(unit);
        for (int i = 0; i < 5; ++i) ptx::mbar_init(&bars[i], 1);
        ptx::fence_mbar_init();
        ptx::mbar_arrive_expect_tx(&bars[3], 2 * (uint32_t)kTBytes + kC * D * 4);
        for (int i = 0; i < 2; ++i)
            ptx::bulk_load(sm + L::YR + (2 * i + 1) * HF, w.P + unit * kC * kC + i * (HF / 4), HF, &bars[3]);
        ptx::bulk_load(sm + L::SQ + 2 * HF, w.T + unit * kC * kC, (uint32_t)kTBytes, &bars[3]);
        ptx::bulk_load(sm + L::B1, w.E + unit * kC * D, kC * D * 4, &bars[3]);
        ptx::mbar_arrive_expect_tx(&bars[4], D * D * 4);
        ptx::bulk_load(sm + L::ST, w.S + unit * D * D, D * D * 4, &bars[4]);
    }
    // A wait that gives up is recorded; what follows is then meaningless, but ends.
    bool ok = true;
    auto wait = [&](int i, int use) {
        if (ok && !ptx::mbar_wait(&bars[i], use, kMmaWaitNs)) {
            ok = false;
            record_error(a.err, GDN_ERR_TIMEOUT);
        }
        ptx::tc_fence_after();
    };
    Flat<T, D, D> state;
    Flat<T, D, kC> u;
    Scale ss, sds;
    {
        GateRows gates;
        if (warp == NW - 1) gates.fetch(a, t0, len, h, lane);
        Rows<NW, D, P> k, q, y;
        k.fetch(a.k, a.qkv_dtype, t0, len, a.Hk, hk, warp, lane);
        q.fetch(a.q, a.qkv_dtype, t0, len, a.Hk, hk, warp, lane);
        y.fetch(a.dout, a.dout_dtype, t0, len, a.H, h, warp, lane);
        if (warp == 1) {  // takes thousands of cycles, while the loads are under way
            ptx::tmem_alloc(&tmem_at, L::tmem);
            ptx::tmem_relinquish();
        }
        if (tid < kC) u_tops[tid] = 0;
        const int part = lane & (D / 8 - 1);  // one of the scan's warps
        const uint32_t top[2] = {meta.s_max[part], meta.ds_max[part]};
        if (warp == NW - 1) gates.put(t, lane);
        k.template put<true>(K, fK, kinv, a.use_l2, 1.f, warp, lane);
        q.template put<true, !L::share>(Q, fQ, qinv, a.use_l2, a.scale, warp, lane);
        y.template put<false>(Y, fY, nullptr, false, 1.f, warp, lane);
        if constexpr (P == 1) {  // dY's lo plane is zero (below dR's, rows of 8 KB)
#pragma unroll
            for (int i = 0; i < PL / 16 / T; ++i) {
                const int e = i * T + tid;
                *reinterpret_cast<uint4*>(sm + L::YR + L::yr + (e >> 9) * 2 * HF + (e & 511) * 16) = make_uint4(0, 0, 0, 0);
            }
        }
        ss = planes::scale_of(__reduce_max_sync(0xffffffffu, top[0]));
        sds = planes::scale_of(__reduce_max_sync(0xffffffffu, top[1]));
    }
    Pair<P> v[MT][NT][2];
    planes::pairs<MT, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int c) {
        v[i][j][hh].load(a.v, a.qkv_dtype, ((t0 + r) * a.H + h) * D + c, r < len);
    });
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tm = tmem_at;
    if (spans[1].n >= 0) {
        const int h2 = next - slots[1] * a.H, hk2 = w.rep(h2);
        prefetch_rows<T, D>(a.k, a.qkv_dtype, spans[1], a.Hk, hk2, tid);
        prefetch_rows<T, D>(a.q, a.qkv_dtype, spans[1], a.Hk, hk2, tid);
        prefetch_rows<T, D>(a.v, a.qkv_dtype, spans[1], a.H, h2, tid);
        prefetch_rows<T, D>(a.dout, a.dout_dtype, spans[1], a.H, h2, tid);
        prefetch_gates(a, spans[1], h2, tid);
        if (tid == 0) {
            prefetch(w.T + (long)next * kC * kC, kTBytes);
            prefetch(w.P + (long)next * kC * kC, kTBytes);
            prefetch(w.meta + next, sizeof(Meta));
            prefetch_states(next);
        }
    }

    constexpr int EL = kC * kC / T, LPR = kC / EL;  // a thread's elements of a 64 x 64 matrix, lanes a row
    const int er = tid / LPR, ec = (tid % LPR) * EL;
    uint32_t* b1_tops = reinterpret_cast<uint32_t*>(sm + L::YR + HF);  // once P^T has been read
    {
        wait(3, 0);
        float f[EL];
#pragma unroll
        for (int i = 0; i < EL; i += 4) load_vec<4>(fY + ec + i, f + i);
        tri_planes<T>(Tri, reinterpret_cast<const float*>(sm + L::YR + HF + (er >> 5) * 2 * HF) + (er & 31) * kC + ec, f, dpp);
        wait(4, 0);
        state.fetch(reinterpret_cast<const float*>(sm + L::ST));
        __syncthreads();
        state.template put<false>(ST, ss.mul);
        float acc[MT][NT][4];  // P^T dY + E
        planes::clear(acc);
        planes::product<kC, false, true, planes::kUpper>(acc, Tri, m, Y, nd, lane);
        const float* E = reinterpret_cast<const float*>(sm + L::B1);
        planes::pairs<MT, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int c) {
            acc[i][j][2 * hh] = fmaf(acc[i][j][2 * hh], dpp[r], E[c * kC + r]);
            acc[i][j][2 * hh + 1] = fmaf(acc[i][j][2 * hh + 1], dpp[r], E[(c + 1) * kC + r]);
        });
        row_tops(b1_tops, acc, m, nw, lane);
        __syncthreads();
        float mul[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) mul[i][hh] = row_scale(b1_tops, m[i] + (lane >> 2) + 8 * hh).mul;
        planes::write(B1, acc, m, nd, lane, mul);
    }
    {
        float f[EL];  // T^T takes the scales of B1's rows
#pragma unroll
        for (int i = 0; i < EL; ++i) f[i] = row_scale(b1_tops, ec + i).back;
        tri_planes<T>(Tri, reinterpret_cast<const float*>(sm + L::SQ + 2 * HF) + er * kC + ec, f, dpp);
    }
    __syncthreads();
    float vdot[MT][2] = {};
    float* fR = reinterpret_cast<float*>(sm + L::SQ + L::tScale);  // takes a row of R to dR,
    float* fU = fR + kC;                                           // a column of U^T's planes to U^T
    {
        uint32_t* dr_tops = reinterpret_cast<uint32_t*>(sm + L::SQ + L::tRows);
        u.fetch(w.U + unit * kC * D);
        float dR[MT][NT][4];
        planes::clear(dR);
        planes::product<kC, false, true, planes::kUpper>(dR, Tri, m, B1, nd, lane);
        planes::pairs<MT, NT>(m, nd, lane, [&](int i, int j, int hh, int r, int c) {
            float &x = dR[i][j][2 * hh], &y = dR[i][j][2 * hh + 1];
            x *= dpp[r];
            y *= dpp[r];
            const float2 vv = v[i][j][hh].value();
            vdot[i][hh] = fmaf(x, vv.x, fmaf(y, vv.y, vdot[i][hh]));
            if (r < len) store2(a.dv, a.qkv_dtype, ((t0 + r) * a.H + h) * D + c, t.beta[r] * x, t.beta[r] * y);
        });
        row_tops(dr_tops, dR, m, nw, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // a thread's four tokens of U; lanes 16 apart have the same
            uint32_t top = 0;
#pragma unroll
            for (int p = 0; p < u.N; ++p) top = max(top, planes::abs_bits(u.x[p][e]));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (lane < 16) atomicMax(&u_tops[4 * lane + e], top);
        }
        __syncthreads();  // also: B1, P^T and T^T have been read
        float mul[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = m[i] + (lane >> 2) + 8 * hh;
                const Scale sr = row_scale(dr_tops, r);
                mul[i][hh] = sr.mul;
                if (nw == 0 && (lane & 3) == 0) fR[r] = sr.back;
            }
        planes::write(R, dR, m, nd, lane, mul);
        float mul_u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Scale su = planes::scale_of(u_tops[4 * (lane & 15) + e]);
            mul_u[e] = su.mul;
            if (tid < 16) fU[4 * lane + e] = su.back;
        }
        u.template put<false>(UT, mul_u);
    }
    // D1 and NZ
    ptx::fence_async_smem();
    __syncthreads();
    if (tid == 0) {
        ptx::tc_fence_after();
        constexpr int KS = D / 16;
        const uint32_t yr = base + L::YR, ut = base + L::B1, st = base + L::ST;
        issue<KS, 64, false, true>(tm + L::tNZ, yr, 2 * HF, ut, 16, false);
        issue<KS, 64, false, true>(tm + L::tNZ, yr, 2 * HF, ut + PL, 16, true);
        issue<KS, 64, false, true>(tm + L::tNZ, yr + L::yr, 2 * HF, ut, 16, true);
        ptx::mma_commit(&bars[0]);
        issue<KS, D, false, true>(tm + L::tD1, yr, 2 * HF, st, D * 128, false);
        issue<KS, D, false, true>(tm + L::tD1, yr, 2 * HF, st + L::st, D * 128, true);
        issue<KS, D, false, true>(tm + L::tD1, yr + L::yr, 2 * HF, st, D * 128, true);
        ptx::mma_commit(&bars[1]);
    }
    state.fetch(dS1);
    // This thread's token, which half of the lanes, and its columns of a 64-wide and of a d-wide result
    const int part = (warp & 3) >> 1, row = (warp & 1) * 32 + lane, cg = warp >> 2;
    const float p_diag = meta.p_diag[row];
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    constexpr int NC = kC / CG;
    float x[NC];
    wait(0, 0);
    {
        const float2 gr = t.G[row];
        const float f = part ? -fR[row] : fY[row], f2 = part ? t.beta[row] * fK[row] : fQ[row];
        uint32_t top = 0, mine = 0;
#pragma unroll
        for (int p = 0; p < NC; p += 16) {
            const int c0 = cg * NC + p;
            if (c0 > (row | 31)) {  // above the diagonal in every row of this warp
#pragma unroll
                for (int i = 0; i < 16; ++i) x[p + i] = 0.f;
                continue;
            }
            uint32_t raw[16];
            tmem_ld16(lanes + L::tNZ + c0, raw);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = c0 + i;
                const float y = __uint_as_float(raw[i]) * f * (decay(gr, t.G[c]) * fU[c]);
                if (c == row && part == 0) {
                    dpp[row] = y;
                    diag[row] = p_diag * y;  // dP_ii q_i . k_i
                }
                x[p + i] = c < row ? y : 0.f;
                top = max(top, planes::abs_bits(x[p + i] * fK[c]));
                const uint32_t col = __reduce_max_sync(0xffffffffu, planes::abs_bits(x[p + i] * f2));
                if (lane == p + i) mine = col;
            }
        }
        reinterpret_cast<uint32_t*>(sm + L::SQ + L::tPZ)[cg * 128 + part * kC + row] = top;
        if (lane < NC) reinterpret_cast<uint32_t*>(sm + L::SQ + L::tCols)[(warp & 3) * kC + cg * NC + lane] = mine;
    }
    wait(1, 0);  // S0's planes, dY and dR have been read
    const float state_dot = warp_sum(state.template put<true>(ST, sds.mul));  // and <S0, dS1>
    const float f1 = (part ? -t.b[row] * fR[row] : t.b[row] * fY[row]) * ss.back;
    const float fh = decay(t.G[kC - 1], t.G[row]) * fU[row] * sds.back;
    if (lane == 0) dots[warp] = state_dot;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // scales: dP's and Z's rows their own for D2; one for a column of both for D3, where they are added: it
    // goes where dY's row factors were
    float* fC = fY;
    if (tid < kC) fC[tid] = row_scale(reinterpret_cast<const uint32_t*>(sm + L::SQ + L::tCols), tid).mul;
    Scale sk;
    {
        const uint32_t* tops_pz = reinterpret_cast<const uint32_t*>(sm + L::SQ + L::tPZ) + part * kC + row;
        uint32_t top = max(tops_pz[0], tops_pz[128]);
        if constexpr (CG == 4) top = max(top, max(tops_pz[256], tops_pz[384]));
        sk = planes::scale_of(top);
    }
    if constexpr (L::share) {
        Rows<NW, D, P> q;
        q.fetch(a.q, a.qkv_dtype, t0, len, a.Hk, hk, warp, lane);
        q.template put<true>(Q, fQ, qinv, a.use_l2, a.scale, warp, lane);
    }
    __syncthreads();
    auto put_row = [&](auto dst, auto&& value) {
#pragma unroll
        for (int i = 0; i < NC; i += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) planes::split(value(i + 2 * j), value(i + 2 * j + 1), hi[j], lo[j]);
            const uint32_t at = dst(row, cg * NC + i);
            planes::sts128(at, hi);
            planes::sts128(at + decltype(dst)::lo, lo);
        }
    };
    put_row(part ? Zm : dP, [&](int i) { return x[i] * fK[cg * NC + i] * sk.mul; });
    const float fq = part ? t.beta[row] * fK[row] : fQ[row];
    if (part == 0) put_row(Pt, [&](int i) { return x[i] * fq * fC[cg * NC + i]; });
    else if (!L::late) put_row(Zt, [&](int i) { return x[i] * fq * fC[cg * NC + i]; });
    ptx::fence_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        ptx::tc_fence_after();
        constexpr int KS = D / 16;
        const uint32_t ut = base + L::B1, st = base + L::ST, sq_at = base + L::SQ;
        issue<KS, D, true, true>(tm + L::tNZ, ut, PL, st, D * 128, false);          // HH
        issue<KS, D, true, true>(tm + L::tNZ, ut, PL, st + L::st, D * 128, true);
        if constexpr (L::late) ptx::mma_commit(&bars[0]);
        issue<4, D, false, true>(tm + L::tD2, sq_at, 0, K.at, HF, false);
        issue<4, D, false, true>(tm + L::tD2, sq_at + 2 * HF, 0, K.at, HF, true);
        issue<4, D, true, true>(tm + L::tD3, Pt.at, 2 * HF, Q.at, QHS, false);
        if constexpr (P == 2) {
            issue<4, D, false, true>(tm + L::tD2, sq_at, 0, K.at + PL, HF, true);
            issue<4, D, true, true>(tm + L::tD3, Pt.at, 2 * HF, Q.at + QLO, QHS, true);
        }
    }
    if constexpr (L::late) {
        wait(0, 1);  // U has been read
        if (part) put_row(Zt, [&](int i) { return x[i] * fq * fC[cg * NC + i]; });
        ptx::fence_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
    }
    if (tid == 0) {
        ptx::tc_fence_after();
        issue<4, D, true, true>(tm + L::tD3, Zt.at, ZLO, K.at, HF, true);
        if constexpr (P == 2) issue<4, D, true, true>(tm + L::tD3, Zt.at, ZLO, K.at + PL, HF, true);
        ptx::mma_commit(&bars[2]);
    }
    wait(2, 0);

    // 32 columns of this token's row: dQ or F in y; dK- + H (this half's planes) in z
    const int c0 = cg * 32;
    float y[32], z[32];
    float dot0 = 0.f, dot1 = 0.f, dot2 = 0.f;  // dQ . q or F . k; H . k; (dK- - H) . k
    {
        const float fd = __uint_as_float((254u << 23) - __float_as_uint(fC[row]));  // 1 / fC, a power of two
        uint32_t r1[32], r2[32];
        ptx::tmem_ld32(lanes + L::tD1 + c0, r1);
        ptx::tmem_ld32(lanes + L::tD2 + c0, r2);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = fmaf(__uint_as_float(r2[i]), sk.back, __uint_as_float(r1[i]) * f1);
        ptx::tmem_ld32(lanes + L::tD3 + c0, r1);
        ptx::tmem_ld32(lanes + L::tNZ + c0, r2);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            float k[8], q[8];
            planes::read8(K, row, c0 + i, k);
            if (part == 0) planes::read8(Q, row, c0 + i, q);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float hx = __uint_as_float(r2[i + j]) * fh, dx = __uint_as_float(r1[i + j]) * fd;
                dot0 = fmaf(y[i + j], part ? k[j] : q[j], dot0);
                dot1 = fmaf(hx, k[j], dot1);
                dot2 = fmaf(dx, k[j], dot2);
                z[i + j] = hx + dx;
            }
        }
    }
    // row sums, each by column group: [0] dQ . q, [1] F . k, [2, 3] H . k, [4, 5] (dK- - H) . k of the two
    // halves, [6] dR . v of the four columns of warps
    float(*sums)[4][kC] = reinterpret_cast<float(*)[4][kC]>(sm + L::B1);
    sums[part][cg][row] = dot0;
    sums[2 + part][cg][row] = dot1;
    sums[4 + part][cg][row] = dot2;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float e = vdot[i][hh];
            e += __shfl_xor_sync(0xffffffffu, e, 1);
            e += __shfl_xor_sync(0xffffffffu, e, 2);
            if ((lane & 3) == 0) sums[6][nw][m[i] + (lane >> 2) + 8 * hh] = e;
        }
    // the first half of the lanes hands its part of dK's rows over
    auto pass = [&](int c) {
        return reinterpret_cast<float4*>(sm + L::ST + row * D * 4 + (((c >> 2) ^ (row & 7)) << 4));
    };
    if (part == 0) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) *pass(c0 + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, L::tmem);
    }
    auto sum_of = [&](int k, int r, int n) {
        float e = sums[k][0][r] + sums[k][1][r];
        if (n == 4) e += sums[k][2][r] + sums[k][3][r];
        return e;
    };
    // through the normalisation: with xh = scale * x * inv and n = x * inv, dx = scale * inv * (d - n (n . d))
    const bool grouped = a.H > a.Hk;
    if (row < len) {
        const gdn_dtype type = grouped ? GDN_F32 : a.qkv_dtype;
        const long at = ((t0 + row) * (grouped ? a.H : a.Hk) + (grouped ? h : hk)) * D + c0;
        const float dp = dpp[row], fq_row = fQ[row], fk_row = fK[row];
        if (part == 0) {
            const float qd = a.use_l2 ? fmaf(sum_of(0, row, CG), fq_row, diag[row]) / (a.scale * a.scale) * fq_row : 0.f;
            const float o = a.scale * qinv[row], dk_row = dp * fk_row;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                float k[8], q[8], out[8];
                planes::read8(K, row, c0 + i, k);
                planes::read8(Q, row, c0 + i, q);
#pragma unroll
                for (int j = 0; j < 8; ++j) out[j] = o * (fmaf(dk_row, k[j], y[i + j]) - q[j] * qd);
                store8(grouped ? w.dq : a.dq, type, at + i, out);
            }
        } else {
            const float beta = t.beta[row], o = kinv[row], dq_row = dp * fq_row;
            const float other = sum_of(2, row, CG) + sum_of(3, row, CG) + sum_of(4, row, CG) + sum_of(5, row, CG);
            const float kd = a.use_l2 ? fmaf(beta * sum_of(1, row, CG) + other, fk_row, diag[row]) * fk_row : 0.f;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                float k[8], q[8], out[8];
                planes::read8(K, row, c0 + i, k);
                planes::read8(Q, row, c0 + i, q);
                const float4 z0 = *pass(c0 + i), z1 = *pass(c0 + i + 4);
                const float zz[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = fmaf(beta, y[i + j], fmaf(dq_row, q[j], z[i + j] + zz[j]));
                    out[j] = o * (d - k[j] * kd);
                }
                store8(grouped ? w.dk : a.dk, type, at + i, out);
            }
        }
    }
    // dbeta; dg by a scan from the chunk's end and one from its start, two rows a lane
    if (warp == NW - 1) {
        float d[2], hd[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            const float kp = sum_of(1, r, CG) * fK[r];
            if (r < len) a.dbeta[(t0 + r) * a.H + h] = sum_of(6, r, 4) + kp;
            d[e] = sum_of(0, r, CG) * fQ[r] + t.beta[r] * kp - (sum_of(4, r, CG) + sum_of(5, r, CG)) * fK[r];
            hd[e] = (sum_of(2, r, CG) + sum_of(3, r, CG)) * fK[r];
        }
        const float carried = t.b[kC - 1] * ss.back * warp_sum(lane < NW ? dots[lane] : 0.f);
        float after = d[0] + d[1], before = hd[0] + hd[1];  // inclusive sums over the later, the earlier lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float p = __shfl_down_sync(0xffffffffu, after, o), q = __shfl_up_sync(0xffffffffu, before, o);
            if (lane + o < 32) after += p;
            if (lane >= o) before += q;
        }
        float later = __shfl_down_sync(0xffffffffu, after, 1), earlier = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 31) later = 0.f;
        if (lane == 0) earlier = 0.f;
        const int r = 2 * lane;
        const float dg[2] = {(later + d[1] + d[0]) + earlier + carried, (later + d[1]) + (earlier + hd[0]) + carried};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (r + e < len) {  // nothing passes a decay to zero: no gradient, where the sums leave a rounding
                const long at = (t0 + r + e) * a.H + h;
                a.dg[at] = a.g[at] < -128.f ? 0.f : dg[e];
            }
    }
    if (tid == 0 && !ok)  // no copy may still be on its way when the block ends
        for (int i = 3; i < 5; ++i) ptx::mbar_wait(&bars[i], 0, kMmaWaitNs);
}

// dq, dk of grouped heads: the sum over the group's value heads, in order.  Tokens outside every
// sequence are left as they were.
__global__ void __launch_bounds__(kPrepThreads) chunk_bwd_heads_kernel(ChunkBwdArgs a, Work w) {
    if (!cu_valid(a, w)) return;
    dependency_wait();
    const int rep = a.H / a.Hk;
    const long first = a.cu_seqlens ? a.cu_seqlens[0] : 0;
    const long end = a.cu_seqlens ? a.cu_seqlens[a.num_seqs] : a.total_T;
    const long per = (long)a.Hk * a.d;
    for (long i = first * per + (long)blockIdx.x * kPrepThreads + threadIdx.x; i < end * per;
         i += (long)gridDim.x * kPrepThreads) {
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

// Zeros to the rows of tokens before the first and behind the last sequence, of those gradients that are given:
// blockIdx.y is the gradient, a word of four bytes a thread (a row of every one is a multiple of them).
__global__ void __launch_bounds__(kPrepThreads) chunk_bwd_zero_outside_kernel(ChunkBwdArgs a) {
    const int first = a.cu_seqlens[0], end = a.cu_seqlens[a.num_seqs];
    if (first < 0 || end < first || end > a.total_T) return;  // gdn_chunk_bwd records it
    void* const outs[5] = {a.dq, a.dk, a.dv, a.dg, a.dbeta};
    uint32_t* out = static_cast<uint32_t*>(outs[blockIdx.y]);
    if (!out) return;
    const long words = blockIdx.y > 2 ? a.H : (long)(blockIdx.y == 2 ? a.H : a.Hk) * a.d / (a.qkv_dtype == GDN_BF16 ? 2 : 1);
    const long before = first * words, skip = (end - first) * words, all = a.total_T * words - skip;
    for (long i = (long)blockIdx.x * kPrepThreads + threadIdx.x; i < all; i += (long)gridDim.x * kPrepThreads)
        out[i < before ? i : i + skip] = 0u;
}

template <int D, int P>
cudaError_t launch(const ChunkBwdArgs& a, cudaStream_t s) {
    const size_t slots = (size_t)slot_count(a.num_seqs, a.total_T), units = slots * a.H;
    const bool index = a.cu_seqlens && a.num_seqs > kScanSeqs;
    Work w = work_of(a.workspace, slots, units, (size_t)a.total_T * a.H, D, P, index);
    w.heads = Divisor::of(a.H);
    w.rep = Divisor::of(a.H / a.Hk);
    w.len = a.cu_seqlens ? 0 : a.total_T / a.num_seqs;
    w.per = (w.len + kC - 1) / kC;
    w.chunks = Divisor::of(w.per > 0 ? w.per : 1);
    const int prep = PrepSmem<D, P>::bytes, grad = GradSmem<D, P>::bytes, scan = scan_bytes(D, P);
    auto allow = [](const void* f, int bytes) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        return e != cudaSuccess ? e : cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    };
    cudaError_t e = allow(reinterpret_cast<const void*>(chunk_bwd_prep_kernel<D, P>), prep);
    if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(chunk_bwd_scan_kernel<D, P>), scan);
    if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(chunk_bwd_grad_kernel<D, P>), grad);
    if (e != cudaSuccess) return e;
    if (index) {
        chunk_bwd_index_kernel<<<1, 1024, 0, s>>>(a, w.index, (int)slots);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    // The first kernel is launched plainly: what it reads may come from the kernel before it.  Those behind
    // it may read the inputs and the index (both complete before it) ahead of dependency_wait(), but nothing else.
    const dim3 chains((unsigned)(a.num_seqs * a.H * (D / 64)), 2);
    if (a.total_T == 0) {
        chunk_bwd_scan_kernel<D, P><<<chains, kScanThreads, scan, s>>>(a, w);
        return cudaGetLastError();
    }
    chunk_bwd_prep_kernel<D, P><<<(unsigned)units, kPrepThreads, prep, s>>>(a, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(chunk_bwd_scan_kernel<D, P>, chains, kScanThreads, scan, s, a, w);
    if (e != cudaSuccess) return e;
    e = launch_after(chunk_bwd_grad_kernel<D, P>, dim3((unsigned)units), GradSmem<D, P>::threads, grad, s, a, w);
    if (e != cudaSuccess || a.H == a.Hk) return e;
    return launch_after(chunk_bwd_heads_kernel, dim3(kSMs * 8), kPrepThreads, 0, s, a, w);
}

}  // namespace

size_t chunk_bwd_workspace_bytes(int num_seqs, int total_T, int H, int Hk, int d) {
    const size_t slots = (size_t)slot_count(num_seqs, total_T), units = slots * H;
    const size_t unit = link_bytes(d, 2) + 2 * kTBytes + sizeof(float) * (2 * kC * d + 2 * d * d) + sizeof(Meta);
    return index_bytes(slots) + units * unit + (H > Hk ? 2 * sizeof(float) * total_T * H * d : 0);
}

cudaError_t launch_chunk_bwd_zero_outside(const ChunkBwdArgs& a, cudaStream_t s) {
    chunk_bwd_zero_outside_kernel<<<dim3(kSMs / 4, 5), kPrepThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_chunk_bwd(const ChunkBwdArgs& a, cudaStream_t s) {
    const bool one = input_planes(a.qkv_dtype, a.dout_dtype) == 1;
    if (a.d == 128) return one ? launch<128, 1>(a, s) : launch<128, 2>(a, s);
    return one ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
}

}  // namespace gdn

// short_conv.cu -- the causal short convolution as a call of its own: prompts, tokens and gradients.
//
// "5. 线性注意力", "因果卷积(Causal Conv1d)": four taps per channel and a SiLU,
//   c_t = bias + sum_j w_j x_{t-3+j},   out_t = silu(c_t),
// with the three inputs before a sequence's first token in its history.  Gradients: dc = dout silu'(c),
//   dx_t = sum_j w_j dc_{t+3-j},  dw_j = sum_t dc_t x_{t-3+j},  dbias = sum_t dc_t.
//
// Every input is read once and every output written once but for the three rows in front of (and, for gradients, behind)
// the run of tokens that a thread walks along with the window of four inputs in registers.  Arithmetic and sums are fp32;
// an output is rounded once, at its store. Memory would bound all three calls; what does is the issue of instructions
// (65% and 53% of the slots, at the three blocks an SM that the registers leave room for) and the start and end of a run.
// So a thread asks for its rows by asynchronous copies into a ring of its own in shared memory, four groups of four rows
// ahead, which takes neither registers nor waits, has few channels (four forward, two backward: eight and four were slower, for their
// registers), and takes its sigmoid from the hardware's exponential and reciprocal.  Gradients' arithmetic goes in pairs
// of channels (8192 x 4352: 69 -> 66 us; forward that spilled, 33 -> 36 us).  Measured, bf16: 8192 tokens of 4352
// channels 27.5 us, 5.2 TB/s (77% of a copy's rate; 32768 tokens 93 us, 6.1 TB/s); gradients of 4132 tokens of 2304
// channels 22 us, four of them the sums behind, 2.6 TB/s; a token of five sequences of 384 channels 1.9 us.  Fp32: gradients
// of 8192 tokens of 4352 channels 81 us, 5.3 TB/s; of 4132 of 2304 25.8 (with two blocks an SM 29.8).
#include "ssm_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTaps = GDN_CONV_KERNEL;
constexpr int kVec = 4;     // channels of a thread, forward
constexpr int kVecB = 2;    // and in the backward pass, whose taps, windows and sums take 30 registers a channel
constexpr int kSMs = 152;
constexpr int kGroups = 4;  // groups of four rows that a thread has on their way
constexpr int kSums = kVecB * 5 + 1;  // sums of a thread of the backward pass, and a word between them
template <typename T>
constexpr int kRingsB = 2 * Ring<T, kVecB, 4 * kGroups, kThreads>::kSmem;
static_assert(kRingsB<__nv_bfloat16> >= 8 * 32 * kSums * 4, "the sums take the rings' place");
static_assert(3 * (kRingsB<float> + 1024 + 256) <= 228 * 1024, "three blocks an SM, with what the system and packed_find keep");

template <bool SILU>
__device__ __forceinline__ float silu_or(float c) {
    return SILU ? c * sigmoid_hw(c) : c;
}

// The input at position p (token index t0 + p of the batch) of a sequence whose first token is t0: its history
// for p < 0, zeros without one.
template <typename T, int VEC>
__device__ __forceinline__ void input_at(const ShortConvArgs& a, int n, int bos, int p, int c0, float (&x)[VEC]) {
    if (p >= 0) {
        load_row<VEC>(static_cast<const T*>(a.x) + (long)(bos + p) * a.x_stride + c0, x);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            x[j] = a.state_in ? a.state_in[((long)n * a.dim + c0 + j) * 3 + 3 + p] : 0.f;
    }
}

template <int VEC>
__device__ __forceinline__ void load_taps(const ShortConvArgs& a, int c0, float (&w)[VEC][kTaps], float (&b)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        load_vec<4>(a.w + (long)(c0 + j) * kTaps, w[j]);
        b[j] = a.bias ? a.bias[c0 + j] : 0.f;
    }
}

// A vector's taps and bias in pairs of channels.
template <int VEC>
__device__ __forceinline__ void load_taps(const ShortConvArgs& a, int c0, F2 (&w)[kTaps][VEC / 2], F2 (&b)[VEC / 2]) {
    float x[VEC][kTaps], y[VEC];
    load_taps<VEC>(a, c0, x, y);
    pair_up<VEC>(y, b);
#pragma unroll
    for (int i = 0; i < kTaps; ++i)
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) w[i][j] = F2(x[2 * j][i], x[2 * j + 1][i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void input_at(const ShortConvArgs& a, int n, int bos, int p, int c0, F2 (&x)[VEC / 2]) {
    float y[VEC];
    input_at<T, VEC>(a, n, bos, p, c0, y);
    pair_up<VEC>(y, x);
}
// The sum of the taps' products with the inputs of four tokens, the newest first.
__device__ __forceinline__ F2 taps(const F2& w0, const F2& w1, const F2& w2, const F2& w3, F2 b, F2 x, F2 h2, F2 h1, F2 h0) {
    return fma2(w3, x, fma2(w2, h2, fma2(w1, h1, fma2(w0, h0, b))));
}

// The last three inputs of sequence n, for one vector of channels.
template <typename T, int VEC>
__device__ void final_history(const ShortConvArgs& a, int n, int bos, int len, int c0) {
    float h[3][VEC];
#pragma unroll
    for (int j = 0; j < 3; ++j) input_at<T, VEC>(a, n, bos, len - 3 + j, c0, h[j]);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int k = 0; k < 3; ++k) a.state_out[((long)n * a.dim + c0 + j) * 3 + k] = h[k][j];
}

// A thread: one channel vector along one run of `run` tokens; threads are numbered through the vectors of a run, then
// through the runs.  The blocks behind `blocks` write the final histories (num_seqs * vectors threads).
template <typename T, bool SILU>
__global__ void __launch_bounds__(kThreads, 3) conv_fwd_kernel(ShortConvArgs a, int run, unsigned blocks) {
    extern __shared__ __align__(16) unsigned char smem[];
    Ring<T, kVec, 4 * kGroups, kThreads> ring(smem);
    const int vecs = a.dim / kVec;
    if (blockIdx.x >= blocks) {
        if (packed_find(a.seqs, 0, 1, 0, a.err) == -2) return;
        const long q = (long)(blockIdx.x - blocks) * kThreads + threadIdx.x;
        if (q >= (long)a.seqs.num_seqs * vecs) return;
        const int n = (int)(q / vecs), bos = a.seqs.bos(n);
        final_history<T, kVec>(a, n, bos, a.seqs.bos(n + 1) - bos, (int)(q % vecs) * kVec);
        return;
    }
    const long q = (long)blockIdx.x * kThreads;
    const int skip = (int)(q % vecs) + (int)threadIdx.x, v = skip % vecs;
    const long first = q / vecs * run;  // of the block's first thread
    const long start = first + (long)(skip / vecs) * run;
    const bool on = start < a.seqs.total_T;
    const int c0 = v * kVec;
    float w[kVec][kTaps], b[kVec], h[3][kVec];
    if (on) load_taps<kVec>(a, c0, w, b);
    int n = packed_find(a.seqs, (int)first, 1, 0, a.err);
    if (n == -2 || !on) return;
    int t = (int)start;
    const int end = (int)min(start + run, (long)a.seqs.total_T), N = a.seqs.num_seqs;
    if (n < 0) {  // tokens before the first sequence stay as they are
        n = 0;
        t = max(t, a.seqs.bos(0));
    }
    if (t >= end) return;
    T* out = static_cast<T*>(a.out);
    while (n < N && t < end) {
        const int bos = a.seqs.bos(n), eos = a.seqs.bos(n + 1);
        if (t >= eos) { ++n; continue; }
        const int stop = min(end, eos);
        const long xs = a.x_stride, os = a.dim;
        const T* src = static_cast<const T*>(a.x) + (long)t * xs + c0;
        T* dst = out + (long)t * os + c0;
        const auto one = [&](const float (&x)[kVec], const float (&h2)[kVec], const float (&h1)[kVec], const float (&h0)[kVec], T* to) {
            float o[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                o[j] = silu_or<SILU>(fmaf(w[j][3], x[j], fmaf(w[j][2], h2[j], fmaf(w[j][1], h1[j], fmaf(w[j][0], h0[j], b[j])))));
            store_row<kVec>(to, o);
        };
        // four rows at a time; the rows of the groups behind them are on their way
        int asked = t;
        const T* next = src;
        const auto ask = [&](int group) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (asked + i < stop) ring.ask(4 * group + i, next + i * xs);
            ring_commit();
            asked += 4;
            next += 4 * xs;
        };
#pragma unroll
        for (int q = 0; q < kGroups; ++q) ask(q);
#pragma unroll
        for (int j = 0; j < 3; ++j) input_at<T, kVec>(a, n, bos, t - bos - 3 + j, c0, h[j]);
        int group = 0;
        for (; t < stop; t += 4) {
            float x[4][kVec];
            ring_wait<kGroups - 1>();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < stop) ring.read(4 * group + i, x[i]);
            one(x[0], h[2], h[1], h[0], dst);
            if (t + 1 < stop) one(x[1], x[0], h[2], h[1], dst + os);
            if (t + 2 < stop) one(x[2], x[1], x[0], h[2], dst + 2 * os);
            if (t + 3 < stop) one(x[3], x[2], x[1], x[0], dst + 3 * os);
            ask(group);
            group = group + 1 == kGroups ? 0 : group + 1;
            dst += 4 * os;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                h[0][j] = x[1][j];
                h[1][j] = x[2][j];
                h[2][j] = x[3][j];
            }
        }
        ring_wait<0>();
        t = stop;
    }
}

// One thread: four channels of one sequence, its history read, moved on by T tokens and written back.
template <typename T, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(ShortConvArgs a) {
    const int vecs = a.dim / 4;
    const long q = (long)blockIdx.x * 128 + threadIdx.x;
    if (q >= (long)a.N * vecs) return;
    const int n = (int)(q / vecs), c0 = (int)(q % vecs) * 4;
    const int slot = a.idx ? a.idx[n] : n;
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        record_error(a.err, GDN_ERR_ARG);
        return;
    }
    float4* st = reinterpret_cast<float4*>(a.pool + ((long)slot * a.dim + c0) * 3);
    const T* src = static_cast<const T*>(a.x) + (long)n * a.T * a.x_stride + c0;
    T* out = static_cast<T*>(a.out) + (long)n * a.T * a.dim + c0;
    float w[4][kTaps], b[4], x[4], h[12];  // h: channel by channel, oldest first
    load_row<4>(src, x);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const float4 f = st[i];
        h[4 * i] = f.x; h[4 * i + 1] = f.y; h[4 * i + 2] = f.z; h[4 * i + 3] = f.w;
    }
    load_taps<4>(a, c0, w, b);
    for (int t = 0; t < a.T; ++t) {
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = fmaf(w[j][3], x[j], fmaf(w[j][2], h[3 * j + 2], fmaf(w[j][1], h[3 * j + 1], fmaf(w[j][0], h[3 * j], b[j]))));
            o[j] = silu_or<SILU>(c);
            h[3 * j] = h[3 * j + 1];
            h[3 * j + 1] = h[3 * j + 2];
            h[3 * j + 2] = x[j];
        }
        store_row<4>(out + (long)t * a.dim, o);
        if (t + 1 < a.T) load_row<4>(src + (long)(t + 1) * a.x_stride, x);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) st[i] = make_float4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

// dc of one token: the slope of the SiLU at c, times dout.
template <bool SILU>
__device__ __forceinline__ F2 dc_of(F2 c, F2 d) {
    if (!SILU) return d;
    const F2 sg = sigmoid_hw(c), one(1.f, 1.f);
    return d * sg * fma2(c, fma2(sg, F2(-1.f, -1.f), one), one);
}

// A block is 32 channel vectors (of two) x 8 runs of tokens; the sums over its runs are added in order and go to
// row blockIdx.x of the table of partial sums [rows][dim * 4], with the biases' [rows][dim] behind it.  The blocks
// with blockIdx.x = rows give the gradients of the carried histories, one thread per (sequence, vector).
template <typename T, bool SILU>
__global__ void __launch_bounds__(kThreads, 3) conv_bwd_kernel(ShortConvArgs a, int run, int rows) {
    extern __shared__ __align__(16) unsigned char smem[];
    Ring<T, kVecB, 4 * kGroups, kThreads> rx(smem), rd(smem + Ring<T, kVecB, 4 * kGroups, kThreads>::kSmem);
    const int vecs = a.dim / kVecB;
    const int v = blockIdx.y * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    const int c0 = v * kVecB, N = a.seqs.num_seqs;
    const bool on = v < vecs;
    const T* src = static_cast<const T*>(a.x) + c0;
    const T* dout = static_cast<const T*>(a.dout) + c0;
    T* dx = static_cast<T*>(a.dx) + c0;
    const bool state_block = (int)blockIdx.x == rows;
    const int first = state_block ? 0 : (int)blockIdx.x * 8 * run;
    constexpr int kPairs = kVecB / 2;
    F2 w[kTaps][kPairs], b[kPairs], dw[kTaps][kPairs], db[kPairs];
    const F2 zero2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        db[j] = zero2;
#pragma unroll
        for (int i = 0; i < kTaps; ++i) dw[i][j] = zero2;
    }
    if (on) load_taps<kVecB>(a, c0, w, b);
    int n = packed_find(a.seqs, first, 1, 0, a.err);
    if (state_block) {
        if (n == -2 || !on) return;
        for (int m = k; m < N; m += 8) {
            const int bos = a.seqs.bos(m), len = a.seqs.bos(m + 1) - bos;
            F2 x[6][kPairs], g[3][kPairs];
#pragma unroll
            for (int p = 0; p < 6; ++p) {
                if (p - 3 < len) input_at<T, kVecB>(a, m, bos, p - 3, c0, x[p]);
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) {  // dc of the first three tokens
#pragma unroll
                for (int j = 0; j < kPairs; ++j) g[p][j] = zero2;
                if (p >= len) continue;
                float y[kVecB];
                load_row<kVecB>(dout + (long)(bos + p) * a.dim, y);
                F2 d[kPairs];
                pair_up<kVecB>(y, d);
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    g[p][j] = dc_of<SILU>(taps(w[0][j], w[1][j], w[2][j], w[3][j], b[j], x[p + 3][j], x[p + 2][j], x[p + 1][j], x[p][j]), d[j]);
            }
            float two[3][kVecB];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                // position p - 3 meets token q through tap p - q (of the taps 0 .. 2)
                (w[0][j] * g[0][j]).get(two[0][2 * j], two[0][2 * j + 1]);
                fma2(w[0][j], g[1][j], w[1][j] * g[0][j]).get(two[1][2 * j], two[1][2 * j + 1]);
                fma2(w[0][j], g[2][j], fma2(w[1][j], g[1][j], w[2][j] * g[0][j])).get(two[2][2 * j], two[2][2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < kVecB; ++j) {
                const long at = ((long)m * a.dim + c0 + j) * 3;
                float o[3] = {two[0][j], two[1][j], two[2][j]};
                float s[3] = {0.f, 0.f, 0.f};
                if (a.dstate_out) {
#pragma unroll
                    for (int p = 0; p < 3; ++p) s[p] = a.dstate_out[at + p];
                }
                // entry p of the final history is position len - 3 + p: a carried one where that is negative
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const int e = p - len;  // entry of the final history at position p - 3
                    if (e >= 0) o[p] += e == 0 ? s[0] : (e == 1 ? s[1] : s[2]);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) a.dstate_in[at + p] = o[p];
            }
        }
        return;
    }
    const bool sound = n != -2;  // without sound offsets nothing is written but zeros to the sums
    int t = first + k * run;
    const int end = min(t + run, a.seqs.total_T);
    if (n < 0) n = sound ? 0 : N;
    const int head = sound ? a.seqs.bos(0) : 0, tail = sound ? a.seqs.bos(N) : 0;
    if (on && sound && a.zero_outside) {
        const float zero[kVecB] = {};
        for (int u = t; u < min(end, head); ++u) store_row<kVecB>(dx + (long)u * a.dim, zero);
        for (int u = max(t, tail); u < end; ++u) store_row<kVecB>(dx + (long)u * a.dim, zero);
    }
    t = max(t, head);
    while (on && n < N && t < end) {
        const int bos = a.seqs.bos(n), eos = a.seqs.bos(n + 1);
        if (t >= eos) { ++n; continue; }
        const int stop = min(end, eos);
        F2 h[3][kPairs], g[3][kPairs];  // the inputs and the dc of the three tokens before
        const int from = t;
        const long xs = a.x_stride, os = a.dim;
        const T* px = src + (long)t * xs;
        const T* pd = dout + (long)t * os;
        T* po = dx + (long)(t - 3) * os;
        // dc of a token of the run (its sums too, where `sums`), from its input and the three before it
        const auto dc = [&](const F2 (&x)[kPairs], const F2 (&h2)[kPairs], const F2 (&h1)[kPairs], const F2 (&h0)[kPairs],
                            const F2 (&d)[kPairs], bool sums, F2 (&gc)[kPairs]) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                gc[j] = dc_of<SILU>(taps(w[0][j], w[1][j], w[2][j], w[3][j], b[j], x[j], h2[j], h1[j], h0[j]), d[j]);
                if (sums) {
                    dw[0][j] = fma2(gc[j], h0[j], dw[0][j]);
                    dw[1][j] = fma2(gc[j], h1[j], dw[1][j]);
                    dw[2][j] = fma2(gc[j], h2[j], dw[2][j]);
                    dw[3][j] = fma2(gc[j], x[j], dw[3][j]);
                    db[j] = db[j] + gc[j];
                }
            }
        };
        // the gradient that is complete with g3, the dc of three tokens later
        const auto gradient = [&](const F2 (&g3)[kPairs], const F2 (&g2)[kPairs], const F2 (&g1)[kPairs], const F2 (&g0)[kPairs],
                                  const F2 (&more)[kPairs], T* to) {
            F2 o[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) o[j] = taps(w[3][j], w[2][j], w[1][j], w[0][j], more[j], g3[j], g2[j], g1[j], g0[j]);
            store_pairs<kVecB>(to, o);
        };
        F2 none[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) none[j] = zero2;
        const int last = min(stop + 3, eos);
        int asked = t, group = 0;
        const auto ask = [&](int q) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (asked + i < last) {
                    rx.ask(4 * q + i, px + i * xs);
                    rd.ask(4 * q + i, pd + i * os);
                }
            ring_commit();
            asked += 4;
            px += 4 * xs;
            pd += 4 * os;
        };
#pragma unroll
        for (int q = 0; q < kGroups; ++q) ask(q);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            input_at<T, kVecB>(a, n, bos, t - bos - 3 + j, c0, h[j]);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) g[j][i] = zero2;
        }
        for (; t + 4 <= stop; t += 4) {
            F2 x[4][kPairs], d[4][kPairs], n4[4][kPairs];
            ring_wait<kGroups - 1>();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rx.read(4 * group + i, x[i]);
                rd.read(4 * group + i, d[i]);
            }
            ask(group);
            group = group + 1 == kGroups ? 0 : group + 1;
            dc(x[0], h[2], h[1], h[0], d[0], true, n4[0]);
            dc(x[1], x[0], h[2], h[1], d[1], true, n4[1]);
            dc(x[2], x[1], x[0], h[2], d[2], true, n4[2]);
            dc(x[3], x[2], x[1], x[0], d[3], true, n4[3]);
            if (t != from) {  // the three tokens before the run are another thread's
                gradient(n4[0], g[2], g[1], g[0], none, po);
                gradient(n4[1], n4[0], g[2], g[1], none, po + os);
                gradient(n4[2], n4[1], n4[0], g[2], none, po + 2 * os);
            }
            gradient(n4[3], n4[2], n4[1], n4[0], none, po + 3 * os);
            po += 4 * os;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                h[0][j] = x[1][j]; h[1][j] = x[2][j]; h[2][j] = x[3][j];
                g[0][j] = n4[1][j]; g[1][j] = n4[2][j]; g[2][j] = n4[3][j];
            }
        }
        // what is left of the run, and the three tokens behind it, which give their dc to its last tokens
        const int rest = stop + 3 - t, live = eos - t;
        ring_wait<0>();
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            if (i >= rest) break;
            const int u = t + i - 3;
            F2 x[kPairs], d[kPairs], gc[kPairs], more[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) x[j] = gc[j] = more[j] = zero2;
            if (i < live) {
                const int slot = 4 * (i < 4 ? group : (group + 1 == kGroups ? 0 : group + 1)) + (i & 3);
                rx.read(slot, x);
                rd.read(slot, d);
                dc(x, h[2], h[1], h[0], d, t + i < stop, gc);
            }
            if (a.dstate_out && u >= eos - 3 && u < eos) {
                float y[kVecB];
#pragma unroll
                for (int j = 0; j < kVecB; ++j) y[j] = a.dstate_out[((long)n * a.dim + c0 + j) * 3 + u - (eos - 3)];
                pair_up<kVecB>(y, more);
            }
            if (u >= from) gradient(gc, g[2], g[1], g[0], more, dx + (long)u * os);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                h[0][j] = h[1][j]; h[1][j] = h[2][j]; h[2][j] = x[j];
                g[0][j] = g[1][j]; g[1][j] = g[2][j]; g[2][j] = gc[j];
            }
        }
        t = stop;
    }
    if (!a.partial) return;
    // in the rings' place, once every thread has read its rows
    ring_wait<0>();
    __syncthreads();
    float(*sh)[32][kSums] = reinterpret_cast<float(*)[32][kSums]>(smem);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        float* to = sh[k][threadIdx.x & 31];
#pragma unroll
        for (int i = 0; i < kTaps; ++i) dw[i][j].get(to[2 * j * kTaps + i], to[(2 * j + 1) * kTaps + i]);
        db[j].get(to[kVecB * kTaps + 2 * j], to[kVecB * kTaps + 2 * j + 1]);
    }
    __syncthreads();
    float* pw = a.partial + (long)blockIdx.x * a.dim * kTaps;
    float* pb = a.partial + (long)rows * a.dim * kTaps + (long)blockIdx.x * a.dim;
    for (int i = threadIdx.x; i < 32 * kVecB * 5; i += kThreads) {
        const int l = i / (kVecB * 5), e = i % (kVecB * 5), vv = blockIdx.y * 32 + l;
        if (vv >= vecs) break;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += sh[r][l][e];
        if (e < kVecB * kTaps) pw[(long)vv * kVecB * kTaps + e] = s;
        else pb[(long)vv * kVecB + e - kVecB * kTaps] = s;
    }
}

// Tokens a thread walks, of a call whose runs find room `at_once` by three blocks an SM: whole rounds of those, few and
// long runs, which start and end seldom.  In us, forward, 8192 tokens x 4352 channels (bf16) with runs of 21, 26, 32, 39,
// 77 (a round): 36, 33, 33, 30, 28; 4132 x 2304 with 21 (a round), 26, 32, 39: 10.1, 11.3, 12.0, 10.9; 500 x 2304 with 2,
// 4, 16: 5.6, 5.1, 5.5; 32768 x 4352 with runs of at most 64, 96, 128, 192: 95, 95, 93, 92.  Gradients, 8192 x 4352 with
// 19, 27, 36: 79, 69, 64, with 58, 72, 86 (two rounds), 103, 128: 63, 61.5, 62, 61, 59; 500 x 2304 with 4, 8, 16: 11.8, 9.3,
// 8.8; 100 x 384: 6.4, 6.6, 7.4.  Their places are whole blocks for each 32 vectors: with the fractions counted too,
// 4132 x 2304 takes 23.2 for 19.8 (a second round), 32768 x 4352 197 for 200.
int run_length(long total_T, long at_once, int least) {
    const long longest = 128, most = at_once > 0 ? at_once : 1, whole = (total_T + most - 1) / most;
    const long rounds = whole > longest ? (whole + longest - 1) / longest : 1, run = (total_T + most * rounds - 1) / (most * rounds);
    return (int)(run < least ? least : run);
}

}  // namespace

cudaError_t launch_short_conv_fwd(const ShortConvArgs& a, cudaStream_t s) {
    const int vecs = a.dim / kVec;
    const int run = run_length(a.seqs.total_T, 3L * kSMs * kThreads / vecs, 4);
    const long runs = ((long)a.seqs.total_T + run - 1) / run, blocks = (runs * vecs + kThreads - 1) / kThreads;
    const long tail = a.state_out ? ((long)a.seqs.num_seqs * vecs + kThreads - 1) / kThreads : 0;
    using B = __nv_bfloat16;
    const auto kernel = a.dtype == GDN_BF16 ? (a.silu ? conv_fwd_kernel<B, true> : conv_fwd_kernel<B, false>)
                                            : (a.silu ? conv_fwd_kernel<float, true> : conv_fwd_kernel<float, false>);
    const int smem = a.dtype == GDN_BF16 ? Ring<__nv_bfloat16, kVec, 4 * kGroups, kThreads>::kSmem : Ring<float, kVec, 4 * kGroups, kThreads>::kSmem;
    cudaError_t set = allow_smem(kernel, smem);
    if (set != cudaSuccess) return set;
    // histories that are carried in place are written behind everything that reads them
    const bool apart = a.state_out && a.state_out == a.state_in;
    if (blocks + tail > 0x7fffffffL) return cudaErrorInvalidValue;
    if (blocks > 0 || (tail > 0 && !apart)) {
        kernel<<<(unsigned)(blocks + (apart ? 0 : tail)), kThreads, smem, s>>>(a, run, (unsigned)blocks);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (apart) {
        kernel<<<(unsigned)tail, kThreads, smem, s>>>(a, run, 0);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

cudaError_t launch_short_conv_step(const ShortConvArgs& a, cudaStream_t s) {
    const long blocks = ((long)a.N * (a.dim / 4) + 127) / 128;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    using B = __nv_bfloat16;
    const auto kernel = a.dtype == GDN_BF16 ? (a.silu ? conv_step_kernel<B, true> : conv_step_kernel<B, false>)
                                            : (a.silu ? conv_step_kernel<float, true> : conv_step_kernel<float, false>);
    kernel<<<(unsigned)blocks, 128, 0, s>>>(a);
    return cudaGetLastError();
}

static void bwd_plan(int total_T, int dim, int& run, int& rows) {
    run = run_length(total_T, 3 * kSMs / ((dim / kVecB + 31) / 32) * 8, 8);
    rows = (int)(((long)total_T + 8L * run - 1) / (8L * run));
}

size_t short_conv_bwd_workspace_bytes(int total_T, int dim) {
    int run, rows;
    bwd_plan(total_T, dim, run, rows);
    return (size_t)rows * dim * 5 * sizeof(float);
}

cudaError_t launch_short_conv_bwd(const ShortConvArgs& a, cudaStream_t s) {
    int run, rows;
    bwd_plan(a.seqs.total_T, a.dim, run, rows);
    const dim3 grid((unsigned)(rows + (a.dstate_in ? 1 : 0)), (unsigned)((a.dim / kVecB + 31) / 32));
    if (grid.x > 0) {
        const bool bf = a.dtype == GDN_BF16;
        using B = __nv_bfloat16;
        const auto kernel = bf ? (a.silu ? conv_bwd_kernel<B, true> : conv_bwd_kernel<B, false>)
                               : (a.silu ? conv_bwd_kernel<float, true> : conv_bwd_kernel<float, false>);
        const int smem = bf ? kRingsB<B> : kRingsB<float>;
        cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<grid, kThreads, smem, s>>>(a, run, rows);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!a.dw && !a.dbias) return cudaSuccess;
    const long cols = (long)a.dim * kTaps;
    return launch_column_sums(ColumnSum{a.partial, cols, a.dw}, ColumnSum{a.partial + rows * cols, a.dim, a.dbias}, rows, s);
}

}  // namespace gdn

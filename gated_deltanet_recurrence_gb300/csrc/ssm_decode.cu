// ssm_decode.cu -- tokens of the selective state space scan on states kept in a pool.
//
//   dt = softplus(a + dt_bias),  S <- exp(-exp(A_log) dt) S + dt x B^T,  y = S C + D x,
// applied T times in order to each sequence's state.  Bound by memory (256 sequences, 32 heads, 64 x 128: 82.7 us, 6.5
// TB/s, 96% of a copy's rate; one to eight sequences are bound by latency, 5 us): a state is read once, stays in
// registers for the T tokens and is written once.  A block takes 64 rows of one (sequence, head) state: a warp eight rows
// (N = 128; a row is 32 lanes of four elements) or four pairs of rows (N = 64), so that a warp has eight (four) 512-byte
// loads in flight before the first token's arithmetic.  The products with C are summed over the lanes for all rows of a
// warp together.  Arithmetic is fp32; y is rounded once, at its store.
#include "ssm_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmArgs a) {
    constexpr int L = N / 4;             // lanes of a row
    constexpr int PW = 32 / L;           // rows a warp load covers
    constexpr int R = kRows / 8 / PW;    // loads of a warp
    const int parts = a.P / kRows;
    const long unit = blockIdx.x;
    const int part = (int)(unit % parts), h = (int)(unit / parts % a.H);
    const long n = unit / parts / a.H;
    int slot = (int)n;
    if (a.idx) {
        slot = a.idx[n];
        if (slot < 0) return;
    }
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) record_error(a.err, GDN_ERR_ARG);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / L, l = lane % L;
    const int p0 = part * kRows + warp * 8 + sub;  // row r of this lane: p0 + r * PW
    float* st = a.pool + (((long)slot * a.H + h) * a.P + p0) * N + l * 4;
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) load_vec<4>(st + (long)r * PW * N, S[r]);
    const int g = h / (a.H / a.G);
    const float rate = expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;
    for (int t = 0; t < a.T; ++t) {
        const long tok = n * a.T + t;
        float B[4], C[4], x[R];
        load_row<4>(static_cast<const T*>(a.B) + tok * a.B_stride + (long)g * N + l * 4, B);
        load_row<4>(static_cast<const T*>(a.C) + tok * a.C_stride + (long)g * N + l * 4, C);
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = to_f32(static_cast<const T*>(a.x)[tok * a.x_stride + (long)h * a.P + p0 + r * PW]);
        const float dt = ssm_softplus(a.a[tok * a.H + h] + bias), alpha = expf(-rate * dt);
        float y[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float v = dt * x[r];
            y[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[r][i] = fmaf(v, B[i], alpha * S[r][i]);
                y[r] = fmaf(S[r][i], C[i], y[r]);
            }
        }
        const float sum = sum_rows<R, L>(y, l);
        if (l < R) {
            const int p = p0 + l * PW;
            const float xr = to_f32(static_cast<const T*>(a.x)[tok * a.x_stride + (long)h * a.P + p]);
            static_cast<T*>(a.out)[(tok * a.H + h) * a.P + p] = from_f32<T>(fmaf(D, xr, sum));
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        *reinterpret_cast<float4*>(st + (long)r * PW * N) = make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
}

template <typename T>
cudaError_t launch(const SsmArgs& a, unsigned blocks, cudaStream_t s) {
    if (a.N == 128) ssm_step_kernel<T, 128><<<blocks, kThreads, 0, s>>>(a);
    else ssm_step_kernel<T, 64><<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t s) {
    const long blocks = (long)a.n_seq * a.H * (a.P / kRows);
    if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, (unsigned)blocks, s) : launch<float>(a, (unsigned)blocks, s);
}

}  // namespace gdn

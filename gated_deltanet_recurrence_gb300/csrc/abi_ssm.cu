// abi_ssm.cu -- the extern "C" entry points of the state space layer: argument checks and dispatch.
// Declarations and the meaning of every argument are in include/gdn.h.
#include <math.h>

#include "ssm_internal.cuh"

namespace {

constexpr long kMaxElements = 1L << 42;  // leaves room for the index arithmetic

bool valid_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }
template <class... P>
bool aligned(P... p) {
    const void* ptrs[] = {p...};
    for (const void* q : ptrs)
        if (q && (reinterpret_cast<uintptr_t>(q) & 15u) != 0) return false;
    return true;
}
// What is read and written one number at a time: logits, the vectors over heads, and their gradients.
template <class... P>
bool aligned4(P... p) {
    const void* ptrs[] = {p...};
    for (const void* q : ptrs)
        if (q && (reinterpret_cast<uintptr_t>(q) & 3u) != 0) return false;
    return true;
}
// Rows of `width` elements, `stride` apart: none overlap, each starts on a 16-byte boundary.
bool rows_ok(long stride, long width) { return stride >= width && stride % 8 == 0 && stride <= (1L << 31); }
int status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH; }
bool packed_ok(const int32_t* cu, int num_seqs, int total_T) {
    return num_seqs > 0 && total_T >= 0 && num_seqs <= (1 << 24) && (cu || total_T % num_seqs == 0);
}
bool elements_ok(long rows, long width) { return width <= 0 || rows <= kMaxElements / width; }

// Tokens of a packed convolution: its kernels count in 32 bits up to eight runs of 128 tokens past the last one, and
// the rows that they ask for ahead.
constexpr int kMaxConvTokens = 0x7fffffff - 2048;

// The sizes of a convolution call; GDN_ERR_UNSUPPORTED for channels that are no whole vectors.
int conv_sizes(long tokens, int dim) {
    if (dim <= 0 || !elements_ok(tokens, dim)) return GDN_ERR_ARG;
    return dim % 8 == 0 && dim <= (1 << 20) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

int ssm_sizes(long tokens, long sequences, int H, int G, int P, int N) {
    if (H <= 0 || G <= 0 || G > H || H % G != 0) return GDN_ERR_ARG;
    if ((P != 64 && P != 128) || (N != 64 && N != 128)) return GDN_ERR_UNSUPPORTED;
    if (H > 16384 || !elements_ok(tokens, (long)H * P) || !elements_ok(sequences, (long)H * P * N)) return GDN_ERR_ARG;
    if (sequences * H * (P / 64) > 0x7fffffffL) return GDN_ERR_ARG;
    return GDN_OK;
}

bool ssm_strides(const gdn::SsmArgs& a) {
    return rows_ok(a.x_stride, (long)a.H * a.P) && rows_ok(a.B_stride, (long)a.G * a.N) &&
           rows_ok(a.C_stride, (long)a.G * a.N);
}

int qk_args(gdn::QkArgs& a, const void* q, long q_stride, const void* k, long k_stride, const float* cos_sin,
            const int32_t* positions, long max_positions, const float* q_weight, const float* k_weight, gdn_norm norm,
            float eps, int interleaved, int T, int H, int H_k, int d, int d_rot, gdn_dtype dtype) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (T < 0 || H <= 0 || H_k < 0 || H > 65536 || H_k > 65536 || d <= 0 || d_rot < 0 || d_rot > d || d_rot % 2 ||
        !(eps >= 0.0f) || (norm != GDN_NORM_RMS && norm != GDN_NORM_L2) || max_positions < 0)
        return GDN_ERR_ARG;
    if (d % 8 != 0 || d > 256) return GDN_ERR_UNSUPPORTED;
    if (!rows_ok(q_stride, (long)H * d) || (H_k && !rows_ok(k_stride, (long)H_k * d))) return GDN_ERR_ARG;
    if (!positions && (long)T > max_positions && d_rot) return GDN_ERR_ARG;
    if (T > 0 && (!q || (H_k && !k) || (d_rot && !cos_sin))) return GDN_ERR_ARG;
    if (!aligned(q, k, cos_sin, q_weight, k_weight)) return GDN_ERR_ARG;
    a.x[0] = q; a.x[1] = k; a.x_stride[0] = q_stride; a.x_stride[1] = k_stride;
    a.w[0] = q_weight; a.w[1] = k_weight; a.heads[0] = H; a.heads[1] = H_k;
    // without a rotation positions say nothing
    a.cos_sin = cos_sin; a.positions = d_rot ? positions : nullptr; a.max_positions = d_rot ? max_positions : (long)T;
    a.l2 = norm == GDN_NORM_L2; a.eps = eps; a.interleaved = interleaved ? 1 : 0;
    a.T = T; a.d = d; a.rot = d_rot; a.dtype = dtype;
    return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_short_conv_fwd(const void* x, long x_stride, const float* weight, const float* bias, const int32_t* cu_seqlens,
                       int num_seqs, int total_T, int dim, gdn_dtype dtype, int silu, const float* conv_state_in,
                       float* conv_state_out, void* out, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (!packed_ok(cu_seqlens, num_seqs, total_T) || total_T > kMaxConvTokens) return GDN_ERR_ARG;
    const int rc = conv_sizes((long)total_T + 3L * num_seqs, dim);
    if (rc != GDN_OK) return rc;
    if (!rows_ok(x_stride, dim)) return GDN_ERR_ARG;
    if (total_T == 0 && !conv_state_out) return GDN_OK;
    if (!weight || (total_T > 0 && (!x || !out))) return GDN_ERR_ARG;
    if (!aligned(x, weight, bias, conv_state_in, conv_state_out, out)) return GDN_ERR_ARG;
    gdn::ShortConvArgs a{};
    a.x = x; a.x_stride = x_stride; a.w = weight; a.bias = bias; a.seqs = gdn::Packed{cu_seqlens, num_seqs, total_T};
    a.dim = dim; a.dtype = dtype; a.silu = silu ? 1 : 0; a.state_in = conv_state_in; a.state_out = conv_state_out;
    a.out = out;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_short_conv_fwd(a, static_cast<cudaStream_t>(stream)));
}

int gdn_short_conv_step(const void* x, long x_stride, const float* weight, const float* bias, float* conv_state_pool,
                        int num_slots, const int32_t* state_indices, int N, int T, int dim, gdn_dtype dtype, int silu,
                        void* out, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (N < 0 || T <= 0 || num_slots <= 0 || (!state_indices && num_slots < N)) return GDN_ERR_ARG;
    if ((long)N * T > (1L << 40)) return GDN_ERR_ARG;
    int rc = conv_sizes((long)N * T, dim);
    if (rc == GDN_OK) rc = conv_sizes(3L * num_slots, dim);
    if (rc != GDN_OK) return rc;
    if (!rows_ok(x_stride, dim)) return GDN_ERR_ARG;
    if (N == 0) return GDN_OK;
    if (!x || !weight || !conv_state_pool || !out) return GDN_ERR_ARG;
    if (!aligned(x, weight, bias, conv_state_pool, out)) return GDN_ERR_ARG;
    gdn::ShortConvArgs a{};
    a.x = x; a.x_stride = x_stride; a.w = weight; a.bias = bias; a.dim = dim; a.dtype = dtype; a.silu = silu ? 1 : 0;
    a.pool = conv_state_pool; a.num_slots = num_slots; a.idx = state_indices; a.N = N; a.T = T; a.out = out;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_short_conv_step(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_short_conv_bwd_workspace_size(int num_seqs, int total_T, int dim) {
    if (num_seqs <= 0 || total_T < 0 || total_T > kMaxConvTokens || conv_sizes((long)total_T + 3L * num_seqs, dim) != GDN_OK) return 0;
    return gdn::short_conv_bwd_workspace_bytes(total_T, dim);
}

int gdn_short_conv_bwd(const void* dout, const void* x, long x_stride, const float* weight, const float* bias,
                       const int32_t* cu_seqlens, int num_seqs, int total_T, int dim, gdn_dtype dtype, int silu,
                       const float* conv_state_in, const float* dconv_state_out, void* dx, float* dweight, float* dbias,
                       float* dconv_state_in, int zero_outside, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (!packed_ok(cu_seqlens, num_seqs, total_T) || total_T > kMaxConvTokens) return GDN_ERR_ARG;
    const int rc = conv_sizes((long)total_T + 3L * num_seqs, dim);
    if (rc != GDN_OK) return rc;
    if (!rows_ok(x_stride, dim)) return GDN_ERR_ARG;
    if (!weight || (total_T > 0 && (!dout || !x || !dx))) return GDN_ERR_ARG;
    if (!aligned(dout, x, weight, bias, conv_state_in, dconv_state_out, dx, dweight, dbias, dconv_state_in)) return GDN_ERR_ARG;
    gdn::ShortConvArgs a{};
    if (dweight || dbias) {
        const size_t need = gdn::short_conv_bwd_workspace_bytes(total_T, dim);
        if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace))) return GDN_ERR_WORKSPACE;
        a.partial = static_cast<float*>(workspace);
    }
    if (total_T == 0 && !dweight && !dbias && !dconv_state_in) return GDN_OK;
    a.x = x; a.x_stride = x_stride; a.w = weight; a.bias = bias; a.seqs = gdn::Packed{cu_seqlens, num_seqs, total_T};
    a.dim = dim; a.dtype = dtype; a.silu = silu ? 1 : 0; a.state_in = conv_state_in;
    a.dout = dout; a.dstate_out = dconv_state_out; a.dx = dx; a.dw = dweight; a.dbias = dbias;
    a.dstate_in = dconv_state_in; a.zero_outside = zero_outside ? 1 : 0;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_short_conv_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_ssm_chunk_fwd_workspace_size(int num_seqs, int total_T, int H, int G, int d_head, int d_state, gdn_dtype dtype) {
    if (!valid_dtype(dtype) || num_seqs <= 0 || total_T < 0 || num_seqs > (1 << 24) ||
        ssm_sizes((long)total_T + 64L * num_seqs, num_seqs + total_T / 64L, H, G, d_head, d_state) != GDN_OK)
        return 0;
    return gdn::ssm_fwd_workspace_bytes(num_seqs, total_T, H, G, d_head, d_state, dtype);
}

int gdn_ssm_chunk_fwd(const void* x, long x_stride, const void* B, long B_stride, const void* C, long C_stride,
                      const float* a_logits, const float* A_log, const float* dt_bias, const float* D,
                      const int32_t* cu_seqlens, int num_seqs, int total_T, int H, int G, int d_head, int d_state,
                      gdn_dtype dtype, const float* initial_state, float* final_state, void* out, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (!packed_ok(cu_seqlens, num_seqs, total_T)) return GDN_ERR_ARG;
    const int rc = ssm_sizes((long)total_T + 64L * num_seqs, num_seqs + total_T / 64L, H, G, d_head, d_state);
    if (rc != GDN_OK) return rc;
    gdn::SsmArgs a{};
    a.x = x; a.x_stride = x_stride; a.B = B; a.B_stride = B_stride; a.C = C; a.C_stride = C_stride;
    a.a = a_logits; a.A_log = A_log; a.dt_bias = dt_bias; a.D = D;
    a.seqs = gdn::Packed{cu_seqlens, num_seqs, total_T}; a.H = H; a.G = G; a.P = d_head; a.N = d_state; a.dtype = dtype;
    if (!ssm_strides(a)) return GDN_ERR_ARG;
    if (total_T == 0 && !final_state) return GDN_OK;
    if (!A_log || (total_T > 0 && (!x || !B || !C || !a_logits || !out))) return GDN_ERR_ARG;
    if (!aligned(x, B, C, initial_state, final_state, out) || !aligned4(a_logits, A_log, dt_bias, D)) return GDN_ERR_ARG;
    const size_t need = gdn::ssm_fwd_workspace_bytes(num_seqs, total_T, H, G, d_head, d_state, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return GDN_ERR_WORKSPACE;
    a.initial_state = initial_state; a.final_state = final_state; a.out = out; a.workspace = workspace;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_ssm_fwd(a, static_cast<cudaStream_t>(stream)));
}

int gdn_ssm_step(const void* x, long x_stride, const void* B, long B_stride, const void* C, long C_stride,
                 const float* a_logits, const float* A_log, const float* dt_bias, const float* D, float* state_pool,
                 int num_slots, const int32_t* state_indices, int N, int T, int H, int G, int d_head, int d_state,
                 gdn_dtype dtype, void* out, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (N < 0 || T <= 0 || num_slots <= 0 || (!state_indices && num_slots < N)) return GDN_ERR_ARG;
    if ((long)N * T > (1L << 40)) return GDN_ERR_ARG;
    int rc = ssm_sizes((long)N * T, N, H, G, d_head, d_state);
    if (rc == GDN_OK && !elements_ok(num_slots, (long)H * d_head * d_state)) rc = GDN_ERR_ARG;
    if (rc != GDN_OK) return rc;
    gdn::SsmArgs a{};
    a.x = x; a.x_stride = x_stride; a.B = B; a.B_stride = B_stride; a.C = C; a.C_stride = C_stride;
    a.a = a_logits; a.A_log = A_log; a.dt_bias = dt_bias; a.D = D; a.H = H; a.G = G; a.P = d_head; a.N = d_state;
    a.dtype = dtype;
    if (!ssm_strides(a)) return GDN_ERR_ARG;
    if (N == 0) return GDN_OK;
    if (!x || !B || !C || !a_logits || !A_log || !state_pool || !out) return GDN_ERR_ARG;
    if (!aligned(x, B, C, state_pool, out) || !aligned4(a_logits, A_log, dt_bias, D)) return GDN_ERR_ARG;
    a.pool = state_pool; a.num_slots = num_slots; a.idx = state_indices; a.n_seq = N; a.T = T; a.out = out;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_ssm_step(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_ssm_chunk_bwd_workspace_size(int num_seqs, int total_T, int H, int G, int d_head, int d_state, gdn_dtype dtype) {
    if (!valid_dtype(dtype) || num_seqs <= 0 || total_T < 0 || num_seqs > (1 << 24) ||
        ssm_sizes((long)total_T + 64L * num_seqs, num_seqs + total_T / 64L, H, G, d_head, d_state) != GDN_OK)
        return 0;
    return gdn::ssm_bwd_workspace_bytes(num_seqs, total_T, H, G, d_head, d_state, dtype);
}

int gdn_ssm_chunk_bwd(const void* dout, const void* x, long x_stride, const void* B, long B_stride, const void* C,
                      long C_stride, const float* a_logits, const float* A_log, const float* dt_bias, const float* D,
                      const int32_t* cu_seqlens, int num_seqs, int total_T, int H, int G, int d_head, int d_state,
                      gdn_dtype dtype, const float* initial_state, const float* dfinal_state, void* dx, void* dB, void* dC,
                      float* da, float* dA_log, float* ddt_bias, float* dD, float* dinitial_state, int zero_outside,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dtype)) return GDN_ERR_DTYPE;
    if (!packed_ok(cu_seqlens, num_seqs, total_T)) return GDN_ERR_ARG;
    const int rc = ssm_sizes((long)total_T + 64L * num_seqs, num_seqs + total_T / 64L, H, G, d_head, d_state);
    if (rc != GDN_OK) return rc;
    gdn::SsmArgs a{};
    a.x = x; a.x_stride = x_stride; a.B = B; a.B_stride = B_stride; a.C = C; a.C_stride = C_stride;
    a.a = a_logits; a.A_log = A_log; a.dt_bias = dt_bias; a.D = D;
    a.seqs = gdn::Packed{cu_seqlens, num_seqs, total_T}; a.H = H; a.G = G; a.P = d_head; a.N = d_state; a.dtype = dtype;
    if (!ssm_strides(a)) return GDN_ERR_ARG;
    if (!A_log || (total_T > 0 && (!dout || !x || !B || !C || !a_logits || !dx || !dB || !dC || !da))) return GDN_ERR_ARG;
    if (!aligned(dout, x, B, C, initial_state, dfinal_state, dx, dB, dC, dinitial_state) ||
        !aligned4(a_logits, A_log, dt_bias, D, da, dA_log, ddt_bias, dD))
        return GDN_ERR_ARG;
    const size_t need = gdn::ssm_bwd_workspace_bytes(num_seqs, total_T, H, G, d_head, d_state, dtype);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return GDN_ERR_WORKSPACE;
    a.initial_state = initial_state; a.dout = dout; a.dfinal_state = dfinal_state; a.dx = dx; a.dB = dB; a.dC = dC;
    a.da = da; a.dA_log = dA_log; a.ddt_bias = ddt_bias; a.dD = dD; a.dinitial_state = dinitial_state;
    a.zero_outside = zero_outside ? 1 : 0; a.workspace = workspace;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_ssm_bwd(a, static_cast<cudaStream_t>(stream)));
}

int gdn_qk_norm_rope(const void* q, long q_stride, const void* k, long k_stride, const float* cos_sin,
                     const int32_t* positions, long max_positions, const float* q_weight, const float* k_weight,
                     gdn_norm norm, float eps, int interleaved, int T, int H, int H_k, int d, int d_rot, gdn_dtype dtype,
                     void* q_out, long q_out_stride, void* k_out, long k_out_stride, void* stream) {
    gdn::QkArgs a{};
    const int rc = qk_args(a, q, q_stride, k, k_stride, cos_sin, positions, max_positions, q_weight, k_weight, norm, eps,
                           interleaved, T, H, H_k, d, d_rot, dtype);
    if (rc != GDN_OK) return rc;
    if (!rows_ok(q_out_stride, (long)H * d) || (H_k && !rows_ok(k_out_stride, (long)H_k * d))) return GDN_ERR_ARG;
    if (T == 0) return GDN_OK;
    if (!q_out || (H_k && !k_out) || !aligned(q_out, k_out)) return GDN_ERR_ARG;
    a.out[0] = q_out; a.out[1] = k_out; a.out_stride[0] = q_out_stride; a.out_stride[1] = k_out_stride;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_qk_norm_rope_bwd_workspace_size(int T, int H, int H_k, int d) {
    if (T < 0 || H <= 0 || H_k < 0 || H > 65536 || H_k > 65536 || d <= 0 || d % 8 != 0 || d > 256) return 0;
    return gdn::qk_bwd_workspace_bytes(T, H, H_k, d);
}

int gdn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, long q_stride, const void* k, long k_stride,
                         const float* cos_sin, const int32_t* positions, long max_positions, const float* q_weight,
                         const float* k_weight, gdn_norm norm, float eps, int interleaved, int T, int H, int H_k, int d,
                         int d_rot, gdn_dtype dtype, void* dq, long dq_stride, void* dk, long dk_stride, float* dq_weight,
                         float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::QkArgs a{};
    const int rc = qk_args(a, q, q_stride, k, k_stride, cos_sin, positions, max_positions, q_weight, k_weight, norm, eps,
                           interleaved, T, H, H_k, d, d_rot, dtype);
    if (rc != GDN_OK) return rc;
    if (!rows_ok(dq_stride, (long)H * d) || (H_k && !rows_ok(dk_stride, (long)H_k * d)) || (!H_k && dk_weight)) return GDN_ERR_ARG;
    if (T == 0 && !dq_weight && !dk_weight) return GDN_OK;
    if (T > 0 && (!dq_out || !dq || (H_k && (!dk_out || !dk)))) return GDN_ERR_ARG;
    if (!aligned(dq_out, dk_out, dq, dk, dq_weight, dk_weight)) return GDN_ERR_ARG;
    if (dq_weight || dk_weight) {
        const size_t need = gdn::qk_bwd_workspace_bytes(T, H, H_k, d);
        if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace))) return GDN_ERR_WORKSPACE;
        a.partial = static_cast<float*>(workspace);
    }
    a.dout[0] = dq_out; a.dout[1] = dk_out; a.out[0] = dq; a.out[1] = dk; a.out_stride[0] = dq_stride; a.out_stride[1] = dk_stride;
    a.dw[0] = dq_weight; a.dw[1] = dk_weight;
    a.err = gdn::device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    return status(gdn::launch_qk_norm_rope_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

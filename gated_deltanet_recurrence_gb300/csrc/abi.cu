// abi.cu -- the extern "C" entry points of libgdn.so: argument checks, dispatch, error word.
// Declarations and the meaning of every argument are in include/gdn.h.
#include <math.h>
#include <atomic>
#include <mutex>

#include "gdn_internal.cuh"
#include "ssm_internal.cuh"

namespace {

// Device-side status word: kernels record the first error they see (atomicCAS from 0).
__device__ int g_gdn_device_error;

constexpr int kMaxDevices = 64;
int* g_err_ptr[kMaxDevices] = {};
std::mutex g_err_mu;

// Address of the error word on the current device (looked up once per device).
int* device_error_ptr() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_err_mu);
    if (!g_err_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_gdn_device_error) != cudaSuccess) {
            cudaGetLastError();  // do not leave the failure for a later launch check to report
            return nullptr;
        }
        g_err_ptr[dev] = static_cast<int*>(p);
    }
    return g_err_ptr[dev];
}

bool valid_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool head_size_ok(int d_k, int d_v) { return d_k == d_v && (d_k == 64 || d_k == 128); }
bool heads_ok(int H, int H_k) { return H > 0 && H_k >= 1 && H_k <= H && H % H_k == 0; }
bool valid_decay(int d) { return d == GDN_DECAY_PER_HEAD || d == GDN_DECAY_PER_KEY_CHANNEL; }

// Checks the short-convolution arguments and fills c; `rows` is the number of state rows (sequences
// or pool slots).  Decode updates may be in place only without grouped heads.
int conv_args(const float* w, const float* st_in, float* st_out, int H, int H_k, int d, long rows,
              bool decode, gdn::ConvArgs& c) {
    c = gdn::ConvArgs{};
    if (!w) return (st_in || st_out) ? GDN_ERR_ARG : GDN_OK;
    const long long dim = 2LL * H_k * d + (long long)H * d;
    if (dim > 0x7fffffffLL / 4 || (long long)rows * dim * 3 > (1LL << 40)) return GDN_ERR_ARG;
    if (decode && st_in && st_in == st_out && H_k != H) return GDN_ERR_ARG;
    c.w = w; c.state_in = st_in; c.state_out = st_out; c.dim = (int)dim;
    return GDN_OK;
}

int launch_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

std::atomic<int> g_prefill_fused_form{GDN_FORM_AUTO};
std::atomic<int> g_decode_blocks_form{GDN_FORM_AUTO};

bool valid_form(int f) { return f == GDN_FORM_AUTO || f == GDN_FORM_OFF || f == GDN_FORM_ON; }

}  // namespace

namespace gdn {
int prefill_fused_form() { return g_prefill_fused_form.load(std::memory_order_relaxed); }
int decode_blocks_form() { return g_decode_blocks_form.load(std::memory_order_relaxed); }
int* device_error_word() { return device_error_ptr(); }
}  // namespace gdn

extern "C" {

const char* gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "GDN_OK";
        case GDN_ERR_ARG: return "GDN_ERR_ARG: invalid argument (null pointer, size or alignment)";
        case GDN_ERR_DTYPE: return "GDN_ERR_DTYPE: unknown element type";
        case GDN_ERR_CU_SEQLENS: return "GDN_ERR_CU_SEQLENS: cu_seqlens not monotone or outside [0, total_T]";
        case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE: workspace missing or too small";
        case GDN_ERR_LAUNCH: return "GDN_ERR_LAUNCH: kernel launch failed";
        case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT: a bounded device wait gave up";
        case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED: head size or option not supported";
        case GDN_ERR_CUDA: return "GDN_ERR_CUDA: CUDA runtime call failed";
        default: return "unknown gdn_status";
    }
}

int gdn_set_kernel_forms(int prefill_fused, int decode_blocks) {
    if (!valid_form(prefill_fused) || !valid_form(decode_blocks)) return GDN_ERR_ARG;
    g_prefill_fused_form.store(prefill_fused, std::memory_order_relaxed);
    g_decode_blocks_form.store(decode_blocks, std::memory_order_relaxed);
    return GDN_OK;
}

int gdn_get_device_error(void* stream, int* device_status) {
    if (!device_status) return GDN_ERR_ARG;
    *device_status = GDN_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
    int* p = device_error_ptr();
    if (!p) return GDN_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyAsync(&v, p, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return GDN_ERR_CUDA;
    if (cudaMemsetAsync(p, 0, sizeof(int), s) != cudaSuccess) return GDN_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
    *device_status = v;
    return GDN_OK;
}

// The tensor-core path (bf16 q/k/v; d = 128, or d = 64 run as 128-wide tiles whose extra columns
// are zeros) keeps per-chunk intermediates (W, U^T, the decayed Q K^T, Q~, K~ and decay factors,
// about 75 KB per chunk and head) in the caller's workspace; the fp32 CUDA-core path needs none.
static bool uses_tc_path(int num_seqs, int total_T, int H, int d_k, int d_v, int qkv_dtype) {
    return qkv_dtype == GDN_BF16 && d_k == d_v && (d_k == 128 || d_k == 64) && total_T > 0 &&
           num_seqs > 0 && H > 0;
}

size_t gdn_chunk_fwd_workspace_size(int num_seqs, int total_T, int H, int d_k, int d_v,
                                    gdn_dtype qkv_dtype) {
    if (!uses_tc_path(num_seqs, total_T, H, d_k, d_v, qkv_dtype)) return 0;
    return gdn::prefill_tc_workspace_bytes(num_seqs, total_T, H);
}

int gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const int32_t* cu_seqlens, int num_seqs, int total_T, int H, int H_k,
                  int d_k, int d_v, gdn_dtype qkv_dtype, gdn_decay decay, float scale,
                  int use_qk_l2norm, const float* conv_weight, const float* conv_state_in,
                  float* conv_state_out, const float* initial_state, float* final_state,
                  const float* gate_z, const float* norm_weight, float norm_eps,
                  void* out, gdn_dtype out_dtype,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(qkv_dtype) || !valid_dtype(out_dtype)) return GDN_ERR_DTYPE;
    if (num_seqs <= 0 || total_T < 0 || !heads_ok(H, H_k) || !valid_decay(decay)) return GDN_ERR_ARG;
    if (!head_size_ok(d_k, d_v)) return GDN_ERR_UNSUPPORTED;
    if ((long long)num_seqs * H > 0x7fffffffLL) return GDN_ERR_ARG;
    if (!cu_seqlens && total_T % num_seqs != 0) return GDN_ERR_ARG;
    if (total_T > 0 && (!q || !k || !v || !g || !beta || !out)) return GDN_ERR_ARG;
    if (!(norm_eps >= 0.0f) || (gate_z == nullptr && norm_weight != nullptr)) return GDN_ERR_ARG;
    const void* ptrs[] = {q, k, v, g, beta, initial_state, final_state, gate_z, norm_weight, out,
                          conv_weight, conv_state_in, conv_state_out};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    gdn::ConvArgs conv;
    const int crc = conv_args(conv_weight, conv_state_in, conv_state_out, H, H_k, d_k, num_seqs, false, conv);
    if (crc != GDN_OK) return crc;
    const size_t need = gdn_chunk_fwd_workspace_size(num_seqs, total_T, H, d_k, d_v, qkv_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (total_T == 0 && !final_state && !conv_state_out) return GDN_OK;

    gdn::PrefillArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.cu_seqlens = cu_seqlens; a.num_seqs = num_seqs; a.total_T = total_T; a.H = H; a.Hk = H_k;
    a.d = d_k; a.qkv_dtype = qkv_dtype; a.g_per_channel = decay == GDN_DECAY_PER_KEY_CHANNEL;
    a.conv = conv;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)d_k);
    a.use_l2 = use_qk_l2norm ? 1 : 0;
    a.initial_state = initial_state; a.final_state = final_state;
    a.z = gate_z; a.w = norm_weight; a.eps = norm_eps; a.out = out; a.out_dtype = out_dtype;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    a.err = device_error_ptr();
    if (!a.err) return GDN_ERR_CUDA;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return GDN_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (total_T > 0 || final_state) {
        if (uses_tc_path(num_seqs, total_T, H, d_k, d_v, qkv_dtype) && gdn::prefill_tc_supported(a))
            e = gdn::launch_prefill_tc(a, st);
        else
            e = gdn::launch_prefill_simt(a, st);
    }
    // the final convolution state is written after every kernel that reads the input state
    if (e == cudaSuccess && conv.state_out) e = gdn::launch_conv_state(a, st);
    return launch_status(e);
}

static bool chunk_bwd_sizes_ok(int num_seqs, int total_T, int H, int H_k, int d_k, int d_v) {
    return num_seqs > 0 && total_T >= 0 && heads_ok(H, H_k) && head_size_ok(d_k, d_v) &&
           ((long long)total_T / 64 + num_seqs) * H <= 0x7fffffffLL &&
           (long long)total_T * H <= 0x7fffffffLL;
}

size_t gdn_chunk_bwd_workspace_size(int num_seqs, int total_T, int H, int H_k, int d_k, int d_v) {
    if (!chunk_bwd_sizes_ok(num_seqs, total_T, H, H_k, d_k, d_v)) return 0;
    return gdn::chunk_bwd_workspace_bytes(num_seqs, total_T, H, H_k, d_k);
}

int gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const int32_t* cu_seqlens, int num_seqs, int total_T, int H, int H_k,
                  int d_k, int d_v, gdn_dtype qkv_dtype, gdn_decay decay, float scale,
                  int use_qk_l2norm, const float* initial_state,
                  const void* dout, gdn_dtype dout_dtype, const float* dfinal_state,
                  void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dinitial_state,
                  void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_dtype(qkv_dtype) || !valid_dtype(dout_dtype)) return GDN_ERR_DTYPE;
    if (num_seqs <= 0 || total_T < 0 || !heads_ok(H, H_k) || !valid_decay(decay)) return GDN_ERR_ARG;
    if (!head_size_ok(d_k, d_v) || decay != GDN_DECAY_PER_HEAD) return GDN_ERR_UNSUPPORTED;
    if (!chunk_bwd_sizes_ok(num_seqs, total_T, H, H_k, d_k, d_v)) return GDN_ERR_ARG;
    if (!cu_seqlens && total_T % num_seqs != 0) return GDN_ERR_ARG;
    if (total_T > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
        return GDN_ERR_ARG;
    const void* ptrs[] = {q, k, v, g, beta, initial_state, dout, dfinal_state, dq, dk, dv, dg, dbeta,
                          dinitial_state};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    const size_t need = gdn_chunk_bwd_workspace_size(num_seqs, total_T, H, H_k, d_k, d_v);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return GDN_ERR_WORKSPACE;
    if (total_T == 0 && !dinitial_state) return GDN_OK;
    gdn::ChunkBwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.cu_seqlens = cu_seqlens; a.num_seqs = num_seqs; a.total_T = total_T; a.H = H; a.Hk = H_k;
    a.d = d_k; a.qkv_dtype = qkv_dtype;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)d_k);
    a.use_l2 = use_qk_l2norm ? 1 : 0;
    a.initial_state = initial_state; a.dout = dout; a.dout_dtype = dout_dtype;
    a.dfinal_state = dfinal_state; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta;
    a.dinitial_state = dinitial_state; a.workspace = workspace;
    a.err = device_error_ptr();
    if (!a.err) return GDN_ERR_CUDA;
    return launch_status(gdn::launch_chunk_bwd(a, static_cast<cudaStream_t>(stream)));
}

int gdn_chunk_bwd_zero_outside(const int32_t* cu_seqlens, int num_seqs, int total_T, int H, int H_k, int d_k,
                               int d_v, gdn_dtype qkv_dtype, void* dq, void* dk, void* dv, float* dg,
                               float* dbeta, void* stream) {
    if (!valid_dtype(qkv_dtype)) return GDN_ERR_DTYPE;
    if (num_seqs <= 0 || total_T < 0 || !heads_ok(H, H_k)) return GDN_ERR_ARG;
    if (!head_size_ok(d_k, d_v)) return GDN_ERR_UNSUPPORTED;
    if (!chunk_bwd_sizes_ok(num_seqs, total_T, H, H_k, d_k, d_v)) return GDN_ERR_ARG;
    const void* ptrs[] = {dq, dk, dv, dg, dbeta};
    bool any = false;
    for (const void* p : ptrs) {
        if (p && !aligned16(p)) return GDN_ERR_ARG;
        any |= p != nullptr;
    }
    if (!cu_seqlens || total_T == 0 || !any) return GDN_OK;
    gdn::ChunkBwdArgs a{};
    a.cu_seqlens = cu_seqlens; a.num_seqs = num_seqs; a.total_T = total_T; a.H = H; a.Hk = H_k;
    a.d = d_k; a.qkv_dtype = qkv_dtype;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta;
    return launch_status(gdn::launch_chunk_bwd_zero_outside(a, static_cast<cudaStream_t>(stream)));
}

static int decode_entry(const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float* state, int num_slots, const int32_t* idx, int N,
                        int T, int H, int H_k, int d_k, int d_v, gdn_dtype qkv_dtype,
                        gdn_decay decay, float scale, int use_qk_l2norm, const float* conv_weight,
                        const float* conv_state_in, float* conv_state_out, const float* gate_z,
                        const float* norm_weight, float norm_eps, void* out, gdn_dtype out_dtype,
                        void* stream) {
    if (!valid_dtype(qkv_dtype) || !valid_dtype(out_dtype)) return GDN_ERR_DTYPE;
    if (N < 0 || T <= 0 || !heads_ok(H, H_k) || num_slots <= 0 || !valid_decay(decay)) return GDN_ERR_ARG;
    if (!head_size_ok(d_k, d_v)) return GDN_ERR_UNSUPPORTED;
    if ((long long)N * H > 0x7fffffffLL || (long long)N * T * H * d_k > (1LL << 40)) return GDN_ERR_ARG;
    if (!idx && num_slots < N) return GDN_ERR_ARG;
    if (N == 0) return GDN_OK;
    if (!q || !k || !v || !g || !beta || !state || !out) return GDN_ERR_ARG;
    if (!(norm_eps >= 0.0f) || (gate_z == nullptr && norm_weight != nullptr)) return GDN_ERR_ARG;
    const void* ptrs[] = {q, k, v, g, beta, state, gate_z, norm_weight, out, conv_weight,
                          conv_state_in, conv_state_out};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    gdn::DecodeArgs a{};
    const int crc = conv_args(conv_weight, conv_state_in, conv_state_out, H, H_k, d_k, num_slots, true, a.conv);
    if (crc != GDN_OK) return crc;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.num_slots = num_slots;
    a.idx = idx; a.N = N; a.T = T; a.H = H; a.Hk = H_k; a.d = d_k; a.qkv_dtype = qkv_dtype;
    a.g_per_channel = decay == GDN_DECAY_PER_KEY_CHANNEL;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)d_k);
    a.use_l2 = use_qk_l2norm ? 1 : 0;
    a.z = gate_z; a.w = norm_weight; a.eps = norm_eps; a.out = out; a.out_dtype = out_dtype;
    a.err = device_error_ptr();
    if (!a.err) return GDN_ERR_CUDA;
    return launch_status(gdn::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

int gdn_recurrent_step(const void* q, const void* k, const void* v, const float* g,
                       const float* beta, float* state, int N, int H, int H_k, int d_k, int d_v,
                       gdn_dtype qkv_dtype, gdn_decay decay, float scale, int use_qk_l2norm,
                       const float* conv_weight, const float* conv_state_in, float* conv_state_out,
                       const float* gate_z, const float* norm_weight, float norm_eps,
                       void* out, gdn_dtype out_dtype, void* stream) {
    return decode_entry(q, k, v, g, beta, state, N > 0 ? N : 1, nullptr, N, 1, H, H_k, d_k, d_v,
                        qkv_dtype, decay, scale, use_qk_l2norm, conv_weight, conv_state_in,
                        conv_state_out, gate_z, norm_weight, norm_eps, out, out_dtype, stream);
}

int gdn_recurrent_multi_step(const void* q, const void* k, const void* v, const float* g,
                             const float* beta, float* state_pool, int num_slots,
                             const int32_t* state_indices, int N, int T, int H, int H_k, int d_k,
                             int d_v, gdn_dtype qkv_dtype, gdn_decay decay, float scale,
                             int use_qk_l2norm, const float* conv_weight,
                             const float* conv_state_in, float* conv_state_out,
                             const float* gate_z, const float* norm_weight, float norm_eps,
                             void* out, gdn_dtype out_dtype, void* stream) {
    return decode_entry(q, k, v, g, beta, state_pool, num_slots, state_indices, N, T, H, H_k, d_k,
                        d_v, qkv_dtype, decay, scale, use_qk_l2norm, conv_weight, conv_state_in,
                        conv_state_out, gate_z, norm_weight, norm_eps, out, out_dtype, stream);
}

int gdn_gate_rmsnorm_silu(const void* y, gdn_dtype y_dtype, const float* z,
                          const float* norm_weight, float eps, void* out, gdn_dtype out_dtype,
                          long rows, int d_v, void* stream) {
    if (!valid_dtype(y_dtype) || !valid_dtype(out_dtype)) return GDN_ERR_DTYPE;
    if (rows < 0 || d_v <= 0 || d_v % 32 != 0 || d_v > 1024 || !(eps >= 0.0f)) return GDN_ERR_ARG;
    if ((rows + 7) / 8 > 0x7fffffffL) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    if (!y || !z || !out) return GDN_ERR_ARG;
    gdn::GateArgs a{};
    a.y = y; a.y_dtype = y_dtype; a.z = z; a.w = norm_weight; a.eps = eps;
    a.out = out; a.out_dtype = out_dtype; a.rows = rows; a.d_v = d_v;
    return launch_status(gdn::launch_gate(a, static_cast<cudaStream_t>(stream)));
}

int gdn_decay_from_logits(const float* a_logits, const float* A_log, const float* dt_bias,
                          const float* b, float* g_out, float* beta_out, long total_T, int H,
                          void* stream) {
    if (total_T < 0 || H <= 0) return GDN_ERR_ARG;
    if (total_T == 0) return GDN_OK;
    if (!a_logits || !A_log || !g_out || (b && !beta_out)) return GDN_ERR_ARG;
    gdn::GatePrepArgs a{};
    a.a = a_logits; a.A_log = A_log; a.dt_bias = dt_bias; a.b = b;
    a.g = g_out; a.beta = beta_out; a.total_T = total_T; a.H = H;
    return launch_status(gdn::launch_gate_prep(a, static_cast<cudaStream_t>(stream)));
}

// Sizes of the norms' training form: a group of at most 1024 channels, at most 2^20 channels a row,
// and element counts that leave room for the index arithmetic.
static bool norm_sizes_ok(long rows, int groups, int size) {
    return rows >= 0 && groups >= 1 && size >= 1 && size <= 1024 && (long long)groups * size <= (1 << 20) &&
           rows <= (1L << 42) / ((long)groups * size);
}

size_t gdn_gate_bwd_workspace_size(long rows, int groups, int group_size) {
    return norm_sizes_ok(rows, groups, group_size) ? gdn::norm_bwd_workspace_bytes(rows, groups, group_size) : 0;
}

static int norm_bwd_entry(const gdn::NormArgs& in, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::NormArgs a = in;
    const void* ptrs[] = {a.dout, a.y, a.z, a.w, a.b, a.dy, a.dz, a.dw, a.db};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    if (a.dw || a.db) {
        const size_t need = gdn::norm_bwd_workspace_bytes(a.rows, a.groups, a.size);
        if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDN_ERR_WORKSPACE;
        a.partial = static_cast<float*>(workspace);
    }
    return launch_status(gdn::launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

int gdn_gate_rmsnorm_silu_bwd(const void* dout, gdn_dtype dout_dtype, const void* y, gdn_dtype y_dtype,
                              const float* z, const float* norm_weight, float eps, void* dy, float* dz,
                              float* dnorm_weight, long rows, int d_v, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (!valid_dtype(dout_dtype) || !valid_dtype(y_dtype)) return GDN_ERR_DTYPE;
    if (d_v <= 0 || d_v % 32 != 0 || !norm_sizes_ok(rows, 1, d_v) || !(eps >= 0.0f)) return GDN_ERR_ARG;
    if (rows == 0 && !dnorm_weight) return GDN_OK;
    if (rows > 0 && (!dout || !y || !z || !dy || !dz)) return GDN_ERR_ARG;
    gdn::NormArgs a{};
    a.y = y; a.y_dtype = y_dtype; a.z = z; a.w = norm_weight; a.eps = eps;
    a.dout = dout; a.dout_dtype = dout_dtype; a.dy = dy; a.dz = dz; a.dw = dnorm_weight;
    a.rows = rows; a.groups = 1; a.size = d_v; a.rms = 1;
    return norm_bwd_entry(a, workspace, workspace_bytes, stream);
}

int gdn_gate_groupnorm_silu(const void* y, gdn_dtype y_dtype, const float* z, const float* weight,
                            const float* bias, float eps, void* out, gdn_dtype out_dtype, long rows,
                            int groups, int group_size, void* stream) {
    if (!valid_dtype(y_dtype) || !valid_dtype(out_dtype)) return GDN_ERR_DTYPE;
    if (!norm_sizes_ok(rows, groups, group_size) || !(eps >= 0.0f)) return GDN_ERR_ARG;
    if (rows == 0) return GDN_OK;
    if (!y || !out) return GDN_ERR_ARG;
    const void* ptrs[] = {y, z, weight, bias, out};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    gdn::NormArgs a{};
    a.y = y; a.y_dtype = y_dtype; a.z = z; a.w = weight; a.b = bias; a.eps = eps;
    a.out = out; a.out_dtype = out_dtype; a.rows = rows; a.groups = groups; a.size = group_size;
    return launch_status(gdn::launch_groupnorm(a, static_cast<cudaStream_t>(stream)));
}

int gdn_gate_groupnorm_silu_bwd(const void* dout, gdn_dtype dout_dtype, const void* y, gdn_dtype y_dtype,
                                const float* z, const float* weight, const float* bias, float eps,
                                void* dy, float* dz, float* dweight, float* dbias, long rows,
                                int groups, int group_size, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (!valid_dtype(dout_dtype) || !valid_dtype(y_dtype)) return GDN_ERR_DTYPE;
    if (!norm_sizes_ok(rows, groups, group_size) || !(eps >= 0.0f)) return GDN_ERR_ARG;
    if (rows == 0 && !dweight && !dbias) return GDN_OK;
    if (rows > 0 && (!dout || !y || !dy || !z != !dz)) return GDN_ERR_ARG;
    gdn::NormArgs a{};
    a.y = y; a.y_dtype = y_dtype; a.z = z; a.w = weight; a.b = bias; a.eps = eps;
    a.dout = dout; a.dout_dtype = dout_dtype; a.dy = dy; a.dz = dz; a.dw = dweight; a.db = dbias;
    a.rows = rows; a.groups = groups; a.size = group_size;
    return norm_bwd_entry(a, workspace, workspace_bytes, stream);
}

static bool decay_bwd_sizes_ok(long total_T, int H) {
    return total_T >= 0 && H > 0 && H <= (1 << 20) && total_T <= (1L << 42) / H;
}

size_t gdn_decay_bwd_workspace_size(long total_T, int H) {
    return decay_bwd_sizes_ok(total_T, H) ? gdn::gate_prep_bwd_workspace_bytes(total_T, H) : 0;
}

int gdn_decay_from_logits_bwd(const float* a_logits, const float* A_log, const float* dt_bias, const float* b,
                              const float* dg, const float* dbeta, float* da, float* dA_log,
                              float* ddt_bias, float* db, long total_T, int H, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (!decay_bwd_sizes_ok(total_T, H)) return GDN_ERR_ARG;
    if (total_T == 0 && !dA_log && !ddt_bias) return GDN_OK;
    if (!A_log || (total_T > 0 && (!a_logits || !dg || !da || !b != !dbeta || !b != !db))) return GDN_ERR_ARG;
    const void* ptrs[] = {a_logits, A_log, dt_bias, b, dg, dbeta, da, dA_log, ddt_bias, db};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ARG;
    gdn::GatePrepBwdArgs a{};
    if (dA_log || ddt_bias) {
        const size_t need = gdn::gate_prep_bwd_workspace_bytes(total_T, H);
        if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDN_ERR_WORKSPACE;
        a.partial = static_cast<float*>(workspace);
    }
    a.a = a_logits; a.A_log = A_log; a.dt_bias = dt_bias; a.b = b; a.dg = dg; a.dbeta = dbeta;
    a.da = da; a.dA_log = dA_log; a.ddt = ddt_bias; a.db = db; a.total_T = total_T; a.H = H;
    return launch_status(gdn::launch_gate_prep_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

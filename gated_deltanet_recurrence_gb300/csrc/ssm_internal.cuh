// ssm_internal.cuh -- what the kernels of the state space layer share: the short convolution as a call of its
// own, the selective scan, the norm and rotation of queries and keys (not part of the ABI).
#pragma once

#include "train_internal.cuh"

namespace gdn {

// ---- packed sequences --------------------------------------------------------------------------

// cu_seqlens of `num_seqs` sequences in a batch of total_T tokens; null cu: equal lengths.
struct Packed {
    const int32_t* cu;
    int num_seqs, total_T;
    __device__ __forceinline__ int bos(int n) const { return cu ? cu[n] : n * (total_T / num_seqs); }
};

// The whole block looks through cu_seqlens once: the number of n in [0, num_seqs] whose bos(n) / unit + n * pad
// is at most `at` (unit = 1, pad = 0: tokens; unit = chunk, pad = 1: chunk slots), minus one, or -2 and a record
// in the error word where the array is malformed.  Every thread gets the answer.
__device__ __forceinline__ int packed_find(const Packed& s, int at, int unit, int pad, int* err) {
    if (!s.cu) {
        const int T = s.total_T / s.num_seqs;
        if (!T) return -1;
        const int per = pad ? 0 : T;
        if (!pad) return min(at / per, s.num_seqs);
    }
    int count = 0;
    bool bad = false;
    for (int n = threadIdx.x; n <= s.num_seqs; n += blockDim.x) {
        const int c = s.bos(n);
        if (s.cu) bad |= c < 0 || c > s.total_T || (n > 0 && s.cu[n - 1] > c);
        count += c / unit + n * pad <= at;
    }
    __shared__ int total;
    if (threadIdx.x == 0) total = 0;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) record_error(err, GDN_ERR_CU_SEQLENS);
        return -2;
    }
    count = __reduce_add_sync(0xffffffffu, count);
    if ((threadIdx.x & 31) == 0 && count) atomicAdd(&total, count);
    __syncthreads();
    return total - 1;
}

// ---- vectors of VEC consecutive elements, converted to fp32 (16-byte aligned for 8 bf16 and 4 fp32) ---------

template <int VEC>
__device__ __forceinline__ void load_row(const float* p, float (&out)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) load_vec<4>(p + i, out + i);
}
template <int VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&out)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = __uint_as_float(u[i] << 16);
            out[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        load_vec<4>(p, out);
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&t);
}
template <int VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[VEC]) {
    uint32_t u[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) u[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}

// The step and the log decay of one token: dt = softplus(a + bias), g = -rate dt with rate = exp(A_log).
__device__ __forceinline__ float ssm_softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// ---- launchers (called from abi_ssm.cu after argument checks) -------------------------------------

// Device error word of the current device, or null (abi.cu).
int* device_error_word();

// out0[c] (out1[c]) = sum over rows of table[r][c] (of the second table behind it), in a fixed order; a kernel that
// begins behind the one before it on the stream.
cudaError_t launch_column_sum(const float* table, long rows, long cols, float* out0, float* out1, cudaStream_t s);

struct ShortConvArgs {
    const void* x; long x_stride; const float* w; const float* bias; Packed seqs; int dim; gdn_dtype dtype; int silu;
    const float* state_in; float* state_out; void* out;
    // tokens
    float* pool; int num_slots; const int32_t* idx; int N, T;
    // gradients
    const void* dout; const float* dstate_out; void* dx; float* dw; float* dbias; float* dstate_in; int zero_outside;
    float* partial; int* err;
};
cudaError_t launch_short_conv_fwd(const ShortConvArgs& a, cudaStream_t s);
cudaError_t launch_short_conv_step(const ShortConvArgs& a, cudaStream_t s);
cudaError_t launch_short_conv_bwd(const ShortConvArgs& a, cudaStream_t s);
size_t short_conv_bwd_workspace_bytes(int total_T, int dim);

struct QkArgs {
    const void* x[2]; long x_stride[2]; const float* w[2]; void* out[2]; long out_stride[2]; int heads[2];  // q, k
    const void* dout[2]; float* dw[2];                                       // gradients: out is dx, dout contiguous
    const float* cos_sin; const int32_t* positions; long max_positions; int l2; float eps; int interleaved;
    int T, d, rot; gdn_dtype dtype; float* partial; int* err;
};
cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t s);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t s);
size_t qk_bwd_workspace_bytes(int T, int H, int H_k, int d);

struct SsmArgs {
    const void* x; long x_stride; const void* B; long B_stride; const void* C; long C_stride;
    const float* a; const float* A_log; const float* dt_bias; const float* D;
    Packed seqs; int H, G, P, N; gdn_dtype dtype;
    const float* initial_state; float* final_state; void* out;
    // tokens
    float* pool; int num_slots; const int32_t* idx; int n_seq, T;
    // gradients
    const void* dout; const float* dfinal_state; void* dx; void* dB; void* dC; float* da; float* dA_log; float* ddt_bias;
    float* dD; float* dinitial_state; int zero_outside;
    void* workspace; int* err;
};
cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_ssm_bwd(const SsmArgs& a, cudaStream_t s);
size_t ssm_fwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N, gdn_dtype dtype);
size_t ssm_bwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N, gdn_dtype dtype);

}  // namespace gdn

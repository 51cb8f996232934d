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
    if constexpr (VEC == 2) load_vec<2>(p, out);
    else
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
        load_vec<VEC>(p, out);
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float (&x)[VEC]) {
    if constexpr (VEC == 2) *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    else
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
    else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t*>(p) = u[0];
}

// Two floats in one 64-bit register: additions, products and sums of both at once.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ static F2 of(uint32_t x, uint32_t y) { return F2(__uint_as_float(x), __uint_as_float(y)); }
    __device__ __forceinline__ void get(float& x, float& y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// The two values of a bf16 pair.
__device__ __forceinline__ F2 widen(uint32_t u) { return F2::of(u << 16, u & 0xffff0000u); }
template <int VEC>
__device__ __forceinline__ void pair_up(const float (&x)[VEC], F2 (&y)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) y[i] = F2(x[2 * i], x[2 * i + 1]);
}
template <int VEC, typename T>
__device__ __forceinline__ void store_pairs(T* p, const F2 (&y)[VEC / 2]) {
    float x[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) y[i].get(x[2 * i], x[2 * i + 1]);
    store_row<VEC>(p, x);
}

// VEC consecutive elements as they lie in memory.
template <typename T, int VEC>
struct RawRow {
    static constexpr int W = VEC * (int)sizeof(T) / 4;
    uint32_t u[W];
    __device__ __forceinline__ void get(F2 (&x)[VEC / 2]) const {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            if constexpr (sizeof(T) == 4) x[i] = F2::of(u[2 * i], u[2 * i + 1]);
            else x[i] = widen(u[i]);
        }
    }
    __device__ __forceinline__ void get(float (&x)[VEC]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float(u[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    }
};

// A thread's own ring of rows on their way from global memory: SLOTS rows of VEC elements, each asked for by the
// thread itself and read by it alone, so that no barrier is needed and a row in flight takes no registers.  Slots of
// the block's threads lie side by side.  Rows are asked for in groups; wait<P>() returns when all groups but the
// last P are there.
template <typename T, int VEC, int SLOTS, int THREADS>
struct Ring {
    static constexpr int BYTES = VEC * (int)sizeof(T);
    static constexpr int kSmem = SLOTS * BYTES * THREADS;
    uint32_t at;
    __device__ __forceinline__ explicit Ring(void* smem)
        : at(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * (BYTES < 16 ? BYTES : 16)) {}
    __device__ __forceinline__ void ask(int slot, const T* p) {
        const uint32_t to = at + slot * (BYTES * THREADS);
        if constexpr (BYTES == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
        else if constexpr (BYTES == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(p) : "memory");
        else
#pragma unroll
            for (int i = 0; i < BYTES; i += 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * THREADS),
                             "l"(reinterpret_cast<const char*>(p) + i)
                             : "memory");
    }
    __device__ __forceinline__ void clear(int slot) const {
        const uint32_t to = at + slot * (BYTES * THREADS);
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + (i / 4) * 16 * THREADS + (i % 4) * 4), "r"(0) : "memory");
    }
    template <class V, int C>  // floats, or pairs
    __device__ __forceinline__ void read(int slot, V (&x)[C]) const {
        RawRow<T, VEC> r;
        read(slot, r);
        r.get(x);
    }
    __device__ __forceinline__ void read(int slot, RawRow<T, VEC>& r) const {
        const uint32_t from = at + slot * (BYTES * THREADS);
        if constexpr (BYTES == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r.u[0]) : "r"(from) : "memory");
        else if constexpr (BYTES == 8)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.u[0]), "=r"(r.u[1]) : "r"(from) : "memory");
        else
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r.u[4 * i]), "=r"(r.u[4 * i + 1]), "=r"(r.u[4 * i + 2]), "=r"(r.u[4 * i + 3])
                             : "r"(from + i * 16 * THREADS)
                             : "memory");
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int P>
__device__ __forceinline__ void ring_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(P) : "memory"); }

__device__ __forceinline__ float exp2_hw(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x) from the hardware exponential and reciprocal (six instructions with its product): an absolute 1e-7, and
// relative (4 + 1.16 max(-x, 0)) 2^-23.  Where e^-x overflows the reciprocal is 0, as it should be.
__device__ __forceinline__ float sigmoid_hw(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + exp2_hw(x * -1.4426950408889634f)));
    return y;
}

__device__ __forceinline__ F2 sigmoid_hw(F2 x) {
    float u, v, y, z;
    (x * F2(-1.4426950408889634f, -1.4426950408889634f)).get(u, v);
    (F2(exp2_hw(u), exp2_hw(v)) + F2(1.f, 1.f)).get(u, v);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(u));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(v));
    return F2(y, z);
}

// Sums of R values over groups of L lanes; value r's sum ends in the lanes with (lane % L) % R == r (R <= L).
template <int R, int L>
__device__ __forceinline__ float sum_rows(float (&y)[R], int lane) {
#pragma unroll
    for (int o = R / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int r = 0; r < o; ++r) {
            const bool up = lane & o;
            const float give = up ? y[r] : y[r + o], keep = up ? y[r + o] : y[r];
            y[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
#pragma unroll
    for (int o = R; o < L; o <<= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
    return y[0];
}

// The step and the log decay of one token: dt = softplus(a + bias), g = -rate dt with rate = exp(A_log).
__device__ __forceinline__ float ssm_softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// Lets a kernel have `smem` bytes of dynamic shared memory, where that is more than any kernel may have unasked.
template <class K>
cudaError_t allow_smem(K kernel, int smem) {
    if (smem <= 20 * 1024) return cudaSuccess;  // beside 28 KB of static arrays at most
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

// ---- launchers (called from abi_ssm.cu after argument checks) -------------------------------------

// Device error word of the current device, or null (abi.cu).
int* device_error_word();

// The column sums of two tables of as many rows, in a fixed order, by a kernel that begins behind the one before it on
// the stream; and those of a table and of the one that lies behind it.
cudaError_t launch_column_sums(const ColumnSum& sum0, const ColumnSum& sum1, long rows, cudaStream_t s);
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

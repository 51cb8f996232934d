// gate_bwd.cu -- the training form of the gates: the output norm as a group norm (forward), the
// gradients of both output norms, and the gradients of the gate preparation.
//
// All four are one pass over the data (HBM-bound): a row's statistics are taken from values that
// stay in registers, every input is read once and every output written once.  Arithmetic and sums
// are fp32; an output is rounded once, at its store.
//
// Norms.  A group of `size` channels is shared by L lanes of a warp (a power of two), each holding
// NV vectors of VEC consecutive channels: vector i of lane l covers channels (i L + l) VEC ....
// Lane sets walk the rows with a stride that keeps their group index, so the weight and bias of a
// set's channels are loaded once, and the sums over rows (dweight, dbias) stay in its registers.
//
// The mean of a group is taken twice: what is left of it after the first subtraction (a rounding of
// the sum, which 1 / sqrt(var + eps) would magnify where a group is nearly constant) is its own mean
// and is taken off as well.
//
// Sums over rows end in a table of partial sums in the workspace, which a second kernel adds up
// column by column in a fixed order: no atomics, so the same call gives the same bits.  A small call's
// blocks are one cluster instead and add their sums up through distributed shared memory, without
// the table and the second launch.
#include <cooperative_groups.h>

#include "train_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kCluster = 8;  // blocks of a small call's cluster
// A call that wants sums over rows is small up to this many blocks of one vector a lane.  us a call, one
// cluster against a grid and column_sum_kernel, as a replayed graph and called from the binding:
//   blocks                             4                8               16               32               64
//   RMS norm, d = 64           4.2/29  5.1/33   4.2/28  5.1/31   5.1/28  5.5/32   6.6/27  5.6/31   9.7/30  5.9/31
//   gate preparation, H = 6    3.0/31  3.9/33   3.1/31  4.1/32   3.4/30  4.1/34   4.1/30  4.6/33   5.4/31  4.5/35
// and the RMS norm of d = 1024 (four vectors a lane) 8.0/30 against 9.2/31 at 8 blocks, 11.8/32 against 9.2/32
// at 16.
constexpr int kNormClusterBlocks = 16, kDecayClusterBlocks = 32;
constexpr int kClusterChannels = 4096;  // whose two sums fit beside the kernel's shared memory

// Launches one cluster of `blocks` blocks.
template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), int blocks, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return launch_config(cfg, kernel, args...);
}

// out[c] = the sum over the cluster's blocks, in order, of element at(c) of each block's `table`; the
// blocks share the columns.  Every thread of the cluster takes part, and tables may be reused after it.
template <class At, class Out>
__device__ __forceinline__ void cluster_sum(float* table, int cols, At at, Out out) {
    const auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    const int n = gridDim.x;
    for (int c = blockIdx.x * kThreads + threadIdx.x; c < cols; c += n * kThreads) {
        float x[kCluster], sum = 0.f;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) x[r] = r < n ? cluster.map_shared_rank(table, r)[at(c)] : 0.f;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) sum += x[r];
        out(c, sum);
    }
    cluster.sync();
}

template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float* out) {
    if constexpr (VEC == 1) out[0] = p[0];
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 4) load_vec<4>(p + i, out + i);
}
template <int VEC>
__device__ __forceinline__ void load_any(const void* base, gdn_dtype dt, long idx, float* out) {
    if (dt == GDN_BF16) {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + idx;
        if constexpr (VEC == 8) {
            const uint4 t = *reinterpret_cast<const uint4*>(p);
            const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                out[2 * i] = __uint_as_float(u[i] << 16);
                out[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else if constexpr (VEC == 4) {
            load_vec<4>(p, out);
        } else {
            out[0] = to_f32(p[0]);
        }
    } else {
        load_f32<VEC>(static_cast<const float*>(base) + idx, out);
    }
}
template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float* x) {
    if constexpr (VEC == 1) p[0] = x[0];
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int VEC>
__device__ __forceinline__ void store_any(void* base, gdn_dtype dt, long idx, const float* x) {
    if (dt == GDN_BF16) {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + idx;
        if constexpr (VEC == 1) {
            p[0] = __float2bfloat16_rn(x[0]);
        } else {
            uint32_t u[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&t);
            }
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
            else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
        }
    } else {
        store_f32<VEC>(static_cast<float*>(base) + idx, x);
    }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 1 / (1 + e^-x) from the hardware exponential and reciprocal: an absolute 1e-7, and relative
// (4 + 1.16 max(-x, 0)) 2^-23 (__expf's error grows with its argument; 6e-7 at x = -1, 2e-6 at -12).  Taking what
// the argument's rounding leaves off back into the exponential, 7e-7 for every x, is six instructions more: group
// norm forward of 8192 x 16 x 128 28.8 us against 26.7, its backward 50.1 against 47.7.  With expf and a division
// the norms were bound by their instructions.
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// How the lane sets cover rows x groups: `stride` sets (a multiple of the groups) work, set s on
// group s % groups and rows s / groups, s / groups + stride / groups, ...
struct NormPlan {
    int L, nv, vec, blocks;
    bool cluster;        // the blocks are one cluster, which adds the sums over rows up itself
    long stride, prows;  // prows: rows of the table of partial sums
};

// sums: sums over rows are wanted.
NormPlan norm_plan(long rows, int groups, int size, bool bwd, bool sums) {
    NormPlan p;
    p.vec = size % 8 == 0 ? 8 : size % 4 == 0 ? 4 : 1;
    const int vecs = size / p.vec;
    p.L = 1;
    while (p.L < 32 && p.L < vecs) p.L *= 2;
    p.nv = (vecs + p.L - 1) / p.L;
    const long per_block = kThreads / p.L;
    const long all = (rows * groups + per_block - 1) / per_block;      // one row a set
    const long least = (groups + per_block - 1) / per_block;           // every group has a set
    // blocks an SM, measured on 8192 x 16 x 128 bf16: forward 3 (27 us; 2: 31, 4: 28), backward 2 (RMS norm
    // 44 us, group norm 52; 3: 48 and 57, 4: 55 and 68)
    const long most = (bwd ? 2 : 3) * kSMs;
    long b = all < most ? all : most;
    if (b < least) b = least;
    p.cluster = sums && all * p.nv <= kNormClusterBlocks && groups <= per_block && groups * size <= kClusterChannels;
    if (p.cluster && b > kCluster) b = kCluster;
    p.blocks = (int)b;
    p.stride = b * per_block / groups * groups;
    // a block whose sets cover every group adds its own sets up first
    p.prows = groups <= per_block ? b : p.stride / groups;
    return p;
}

// Asks for a lane's part of the row its set takes next (the first vector of each row; rows longer than a
// warp's vectors have enough loads of their own under way).
template <int VEC>
__device__ __forceinline__ void prefetch_row(const void* p, gdn_dtype dt, long at) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + at * (dt == GDN_BF16 ? 2 : 4)));
}

// 8192 x 16 x 128 bf16, gated: 26.7 us (plain form 396), 5.0 TB/s, 74% of the copy rate; 0.68 of the issue
// slots are taken, so instructions stand close behind DRAM.
template <int L, int NV, int VEC>
__global__ void __launch_bounds__(kThreads, VEC == 8 && NV == 1 ? 3 : 1) groupnorm_kernel(NormArgs a, long stride) {
    const long set = (long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    const int grp = (int)(set % a.groups);
    const long rstep = stride / a.groups;
    const float inv = 1.0f / (float)a.size;
    float w[NV][VEC], b[NV][VEC];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * L + lane) * VEC;
        in[i] = c < a.size && set < stride;
#pragma unroll
        for (int j = 0; j < VEC; ++j) { w[i][j] = 1.f; b[i][j] = 0.f; }
        if (in[i] && a.w) load_f32<VEC>(a.w + (long)grp * a.size + c, w[i]);
        if (in[i] && a.b) load_f32<VEC>(a.b + (long)grp * a.size + c, b[i]);
    }
    // every lane of a warp runs the same number of passes (the sums below are warp-wide shuffles)
    const long passes = (a.rows + rstep - 1) / rstep;
    long row = set / a.groups;
    for (long p = 0; p < passes; ++p, row += rstep) {
        const bool live = row < a.rows;
        const long base = (row * a.groups + grp) * a.size;
        if (in[0] && row + rstep < a.rows) {
            const long at = base + rstep * a.groups * a.size + lane * VEC;
            prefetch_row<VEC>(a.y, a.y_dtype, at);
            if (a.z) prefetch_row<VEC>(a.z, GDN_F32, at);
        }
        float y[NV][VEC], z[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * L + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[i][j] = z[i][j] = 0.f;
            if (!in[i] || !live) continue;
            load_any<VEC>(a.y, a.y_dtype, base + c, y[i]);
            if (a.z) load_f32<VEC>(a.z + base + c, z[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += y[i][j];
        }
        const float mean = lanes_sum<L>(sum) / (float)a.size;
        float rest = 0.f, ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                y[i][j] -= mean;
                rest += y[i][j];
                ss += y[i][j] * y[i][j];
            }
        }
        const float off = lanes_sum<L>(rest) * inv;
        const float r = rsqrtf(fmaxf(lanes_sum<L>(ss) * inv - off * off, 0.f) + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i] || !live) continue;
            const int c = (i * L + lane) * VEC;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float m = fmaf(w[i][j], (y[i][j] - off) * r, b[i][j]);
                const float t = a.z ? z[i][j] : m;
                o[j] = (a.z ? m : 1.f) * t * sigmoid_fast(t);
            }
            store_any<VEC>(a.out, a.out_dtype, base + c, o);
        }
    }
}

// 8192 x 16 x 128 bf16 with the sums over rows: RMS norm 42.9 us (plain form 892), 81% of the copy rate; group
// norm 47.2 us (986), 73%.  DRAM bounds both (issue slots 0.53 and 0.61); about 5 us of it are column_sum_kernel.
// prows: rows of the table of partial sums.  ONE: the grid is one cluster and writes dw and db itself.
template <int L, int NV, int VEC, bool RMS, bool ONE>
__global__ void __launch_bounds__(kThreads, VEC == 8 && NV == 1 ? 2 : 1) norm_bwd_kernel(NormArgs a, long stride, long prows) {
    const long set = (long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int lane = threadIdx.x % L;
    const int grp = (int)(set % a.groups);
    const long rstep = stride / a.groups;
    const float inv = 1.0f / (float)a.size;
    const bool gated = RMS || a.z;
    float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * L + lane) * VEC;
        in[i] = c < a.size && set < stride;
#pragma unroll
        for (int j = 0; j < VEC; ++j) { w[i][j] = 1.f; b[i][j] = 0.f; dw[i][j] = 0.f; db[i][j] = 0.f; }
        if (in[i] && a.w) load_f32<VEC>(a.w + (long)grp * a.size + c, w[i]);
        if (!RMS && in[i] && a.b) load_f32<VEC>(a.b + (long)grp * a.size + c, b[i]);
    }
    const long passes = (a.rows + rstep - 1) / rstep;
    long row = set / a.groups;
    for (long p = 0; p < passes; ++p, row += rstep) {
        const bool live = row < a.rows;
        const long base = (row * a.groups + grp) * a.size;
        if (in[0] && row + rstep < a.rows) {
            const long at = base + rstep * a.groups * a.size + lane * VEC;
            prefetch_row<VEC>(a.y, a.y_dtype, at);
            prefetch_row<VEC>(a.dout, a.dout_dtype, at);
            if (a.z) prefetch_row<VEC>(a.z, GDN_F32, at);
        }
        float y[NV][VEC], z[NV][VEC], d[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * L + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[i][j] = z[i][j] = d[i][j] = 0.f;
            if (!in[i] || !live) continue;
            load_any<VEC>(a.y, a.y_dtype, base + c, y[i]);
            load_any<VEC>(a.dout, a.dout_dtype, base + c, d[i]);
            if (gated) load_f32<VEC>(a.z + base + c, z[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += y[i][j];
        }
        const float mean = RMS ? 0.f : lanes_sum<L>(sum) / (float)a.size;
        float rest = 0.f, ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                y[i][j] -= mean;
                rest += y[i][j];
                ss += y[i][j] * y[i][j];
            }
        }
        const float off = RMS ? 0.f : lanes_sum<L>(rest) * inv;
        const float var = fmaxf(lanes_sum<L>(ss) * inv - off * off, 0.f);
        const float r = live ? rsqrtf(var + a.eps) : 0.f;  // rows past the end add nothing to dw, db
        // y becomes n; d becomes dn; z becomes dz
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = (y[i][j] - off) * r, g = d[i][j];
                const float m = RMS ? w[i][j] * n : fmaf(w[i][j], n, b[i][j]);
                const float t = gated ? z[i][j] : m;
                const float sg = sigmoid_fast(t), act = t * sg, slope = fmaf(act, 1.0f - sg, sg);
                const float dm = g * (gated ? act : slope);
                z[i][j] = g * m * slope;
                dw[i][j] = fmaf(dm, n, dw[i][j]);
                if (!RMS) db[i][j] += dm;
                const float dn = dm * w[i][j];
                y[i][j] = n;
                d[i][j] = dn;
                s1 += dn;
                s2 = fmaf(dn, n, s2);
            }
        }
        const float m1 = RMS ? 0.f : lanes_sum<L>(s1) * inv;
        const float m2 = lanes_sum<L>(s2) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i] || !live) continue;
            const int c = (i * L + lane) * VEC;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = r * (d[i][j] - m1 - y[i][j] * m2);
            store_any<VEC>(a.dy, a.y_dtype, base + c, o);
            if (gated) store_f32<VEC>(a.dz + base + c, z[i]);
        }
    }
    if (!ONE && !a.partial) return;
    const long channels = (long)a.groups * a.size;
    constexpr int PER = kThreads / L;
    if (!ONE && a.groups > PER) {
        if (set >= stride) return;
        float* pw = a.partial + (set / a.groups) * channels + (long)grp * a.size;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
            const int c = (i * L + lane) * VEC;
            if (a.dw) store_f32<VEC>(pw + c, dw[i]);
            if (!RMS && a.db) store_f32<VEC>(pw + prows * channels + c, db[i]);
        }
        return;
    }
    // the block's sets of one group are added in order (idle sets hold zeros)
    __shared__ float sh[kThreads * VEC];
    extern __shared__ __align__(16) float sums[];  // [2, channels], in a cluster
    const int k = threadIdx.x / L;
    float* pw = (ONE ? sums : a.partial + blockIdx.x * channels) + (long)grp * a.size;
#pragma unroll
    for (int part = 0; part < (RMS ? 1 : 2); ++part) {
        if (!(part ? a.db : a.dw)) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float(&x)[VEC] = part ? db[i] : dw[i];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < VEC; ++j) sh[j * kThreads + threadIdx.x] = x[j];
            __syncthreads();
            const int c = (i * L + lane) * VEC;
            if (k < a.groups && c < a.size) {
                for (int q = k + a.groups; q < PER; q += a.groups)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[j] += sh[j * kThreads + q * L + lane];
                store_f32<VEC>(pw + part * (ONE ? 1 : prows) * channels + c, x);
            }
        }
    }
    if constexpr (ONE) {
        const int n = (int)channels;
        cluster_sum(sums, a.db ? 2 * n : n, [](int c) { return c; }, [&](int c, float x) {
            if (c >= n) a.db[c - n] = x;
            else if (a.dw) a.dw[c] = x;
        });
    }
}

// out[c] = sum over r of table[r][c] for both tables (the second may be absent): 32 columns and 32
// interleaved row ranges per block, each range added in order, the ranges then in order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) column_sum_kernel(const float* table, long rows, long cols, float* out0,
                                                                 float* out1) {
    dependency_wait();
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, k = threadIdx.x >> 5;
    const long c = (long)blockIdx.x * 32 + x;
    const float* t = table + (blockIdx.y ? rows * cols : 0);
    float* out = blockIdx.y ? out1 : out0;
    if (!out) return;
    float s = 0.f;
    if (c < cols) {
        long r = k;
        for (; r + 96 < rows; r += 128) {
            const float v[4] = {t[r * cols + c], t[(r + 32) * cols + c], t[(r + 64) * cols + c], t[(r + 96) * cols + c]};
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; r < rows; r += 32) s += t[r * cols + c];
    }
    part[k][x] = s;
    __syncthreads();
    // warp k adds column k's 32 parts
    const long ck = (long)blockIdx.x * 32 + k;
    const float sum = warp_sum(part[x][k]);
    if (x == 0 && ck < cols) out[ck] = sum;
}

template <int L, int NV, int VEC>
cudaError_t launch_norm_one(const NormArgs& a, const NormPlan& p, bool bwd, cudaStream_t s) {
    if (!bwd) {
        groupnorm_kernel<L, NV, VEC><<<p.blocks, kThreads, 0, s>>>(a, p.stride);
    } else if (p.cluster) {
        const auto kernel = a.rms ? norm_bwd_kernel<L, NV, VEC, true, true> : norm_bwd_kernel<L, NV, VEC, false, true>;
        return launch_cluster(kernel, p.blocks, 2 * sizeof(float) * a.groups * a.size, s, a, p.stride, 0);
    } else {
        const auto kernel = a.rms ? norm_bwd_kernel<L, NV, VEC, true, false> : norm_bwd_kernel<L, NV, VEC, false, false>;
        kernel<<<p.blocks, kThreads, 0, s>>>(a, p.stride, p.prows);
    }
    return cudaGetLastError();
}

template <int VEC>
cudaError_t launch_norm_vec(const NormArgs& a, const NormPlan& p, bool bwd, cudaStream_t s) {
    switch (p.L) {
        case 1: return launch_norm_one<1, 1, VEC>(a, p, bwd, s);
        case 2: return launch_norm_one<2, 1, VEC>(a, p, bwd, s);
        case 4: return launch_norm_one<4, 1, VEC>(a, p, bwd, s);
        case 8: return launch_norm_one<8, 1, VEC>(a, p, bwd, s);
        case 16: return launch_norm_one<16, 1, VEC>(a, p, bwd, s);
        default: break;
    }
    if (p.nv == 1) return launch_norm_one<32, 1, VEC>(a, p, bwd, s);
    if (p.nv == 2) return launch_norm_one<32, 2, VEC>(a, p, bwd, s);
    if (p.nv <= 4) return launch_norm_one<32, 4, VEC>(a, p, bwd, s);
    if constexpr (VEC < 8) {
        if (p.nv <= 8) return launch_norm_one<32, 8, VEC>(a, p, bwd, s);
    }
    if constexpr (VEC == 1) return launch_norm_one<32, 32, VEC>(a, p, bwd, s);
    return cudaErrorInvalidValue;  // groups of more than 1024 channels are refused before
}

cudaError_t launch_norm(const NormArgs& a, const NormPlan& p, bool bwd, cudaStream_t s) {
    if (p.vec == 8) return launch_norm_vec<8>(a, p, bwd, s);
    if (p.vec == 4) return launch_norm_vec<4>(a, p, bwd, s);
    return launch_norm_vec<1>(a, p, bwd, s);
}

// ---- gate preparation --------------------------------------------------------------------------

// Thread q of the grid works on column vector q % (H / VEC) of rows q / (H / VEC), ..., with a
// stride that keeps its column, so the column sums stay in registers.
struct DecayPlan {
    int vec, blocks;
    bool cluster;  // as in NormPlan
    long cols, stride, prows;  // column vectors; working threads; rows of the partial table
};

DecayPlan decay_plan(long total_T, int H, bool sums) {
    DecayPlan p;
    p.vec = H % 4 == 0 ? 4 : 1;
    p.cols = H / p.vec;
    const long all = (total_T * p.cols + kThreads - 1) / kThreads;
    const long least = (p.cols + kThreads - 1) / kThreads;
    long b = all < 4 * kSMs ? all : 4 * kSMs;
    if (b < least) b = least;
    p.cluster = sums && all <= kDecayClusterBlocks && p.cols <= kThreads;
    if (p.cluster && b > kCluster) b = kCluster;
    p.blocks = (int)b;
    p.stride = b * kThreads / p.cols * p.cols;
    p.prows = p.cols <= kThreads ? b : p.stride / p.cols;
    return p;
}

// 131072 x 32: 21 us as a replayed graph (plain form 181 us; 15 us at the copy rate), 27 - 34 us called from the
// binding, whose checks and allocations take that long.
template <int VEC>
__global__ void __launch_bounds__(kThreads) gate_prep_bwd_kernel(GatePrepBwdArgs a, long cols, long stride,
                                                                 long prows) {
    const long q = (long)blockIdx.x * kThreads + threadIdx.x;
    const long h = (q % cols) * VEC;
    float A[VEC], bias[VEC], sA[VEC], sd[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        A[j] = expf(a.A_log[h + j]);
        bias[j] = a.dt_bias ? a.dt_bias[h + j] : 0.f;
        sA[j] = sd[j] = 0.f;
    }
    if (q < stride) {
        const long n = a.total_T * cols;
        for (long i = q; i < n; i += stride) {
            float x[VEC], dg[VEC], o[VEC];
            load_f32<VEC>(a.a + i * VEC, x);
            load_f32<VEC>(a.dg + i * VEC, dg);
            if (a.b) {
                float b[VEC], dbeta[VEC];
                load_f32<VEC>(a.b + i * VEC, b);
                load_f32<VEC>(a.dbeta + i * VEC, dbeta);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {  // beta (1 - beta) = e / (1 + e)^2; __expf as in sigmoid_fast
                    const float e = __expf(-fabsf(b[j])), q = __fdividef(1.0f, 1.0f + e);
                    b[j] = dbeta[j] * (e * q * q);
                }
                store_f32<VEC>(a.db + i * VEC, b);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {  // softplus(t) = max(t, 0) + log(1 + e), sigmoid(t) from the same e
                const float t = x[j] + bias[j];
                const float e = __expf(-fabsf(t)), q = __fdividef(1.0f, 1.0f + e);
                const float sp = fmaxf(t, 0.f) + log1pf(e), gA = dg[j] * A[j];
                o[j] = -gA * (t >= 0.f ? q : e * q);
                sA[j] -= gA * sp;
                sd[j] += o[j];
            }
            store_f32<VEC>(a.da + i * VEC, o);
        }
    }
    if (!a.dA_log && !a.ddt) return;
    // threads of the block that hold the same columns are added in order (cols <= kThreads); idle
    // threads hold zeros
    __shared__ float sh[2][kThreads][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) { sh[0][threadIdx.x][j] = sA[j]; sh[1][threadIdx.x][j] = sd[j]; }
    __syncthreads();
    const long H = cols * VEC;
    if (threadIdx.x < cols)
        for (long t = threadIdx.x + cols; t < kThreads; t += cols)
#pragma unroll
            for (int j = 0; j < VEC; ++j) { sA[j] += sh[0][t][j]; sd[j] += sh[1][t][j]; }
    if (!prows) {
        if (threadIdx.x < cols)
#pragma unroll
            for (int j = 0; j < VEC; ++j) { sh[0][q % cols][j] = sA[j]; sh[1][q % cols][j] = sd[j]; }  // read by no thread above
        const int n = (int)H;
        cluster_sum(&sh[0][0][0], 2 * n, [&](int c) { return c < n ? c : c - n + kThreads * VEC; }, [&](int c, float x) {
            float* out = c < n ? a.dA_log : a.ddt;
            if (out) out[c < n ? c : c - n] = x;
        });
        return;
    }
    long prow = blockIdx.x;
    if (cols <= kThreads) {
        if (threadIdx.x >= cols) return;
    } else {
        if (q >= stride) return;
        prow = q / cols;
    }
    store_f32<VEC>(a.partial + prow * H + h, sA);
    store_f32<VEC>(a.partial + (prows + prow) * H + h, sd);
}

}  // namespace

size_t norm_bwd_workspace_bytes(long rows, int groups, int size) {
    const NormPlan p = norm_plan(rows, groups, size, true, false);  // small calls do not use it
    return (size_t)p.prows * groups * size * 2 * sizeof(float);
}

cudaError_t launch_groupnorm(const NormArgs& a, cudaStream_t s) {
    return launch_norm(a, norm_plan(a.rows, a.groups, a.size, false, false), false, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s) {
    const bool sums = a.dw || a.db;
    const NormPlan p = norm_plan(a.rows, a.groups, a.size, true, sums);
    cudaError_t e = launch_norm(a, p, true, s);
    if (e != cudaSuccess || !sums || p.cluster) return e;
    const long cols = (long)a.groups * a.size;
    return launch_after(column_sum_kernel, dim3((unsigned)((cols + 31) / 32), a.db ? 2 : 1), kSumThreads, 0, s,
                        a.partial, p.prows, cols, a.dw, a.db);
}

size_t gate_prep_bwd_workspace_bytes(long total_T, int H) {
    return (size_t)decay_plan(total_T, H, false).prows * H * 2 * sizeof(float);
}

cudaError_t launch_gate_prep_bwd(const GatePrepBwdArgs& a, cudaStream_t s) {
    const bool sums = a.dA_log || a.ddt;
    const DecayPlan p = decay_plan(a.total_T, a.H, sums);
    const auto kernel = p.vec == 4 ? gate_prep_bwd_kernel<4> : gate_prep_bwd_kernel<1>;
    if (p.cluster) return launch_cluster(kernel, p.blocks, 0, s, a, p.cols, p.stride, 0);
    kernel<<<p.blocks, kThreads, 0, s>>>(a, p.cols, p.stride, p.prows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !sums) return e;
    return launch_after(column_sum_kernel, dim3((unsigned)((a.H + 31) / 32), a.ddt ? 2 : 1), kSumThreads, 0, s,
                        a.partial, p.prows, a.H, a.dA_log, a.ddt);
}

}  // namespace gdn

// ssm_chunk.cuh -- what the chunked kernels of the selective scan share: chunks, gates, the states at chunk starts.
//
// A chunk is 64 tokens of one sequence; its slot is bos / 64 + n + k for chunk k of sequence n, so that slots do not
// overlap for any lengths and number at most total_T / 64 + num_seqs.  For each slot and head the gates kernel
// leaves five rows of 64 numbers: dt, the running sums G of the log decays in two floats (hi, lo), b = e^G, and
// r = e^(G_last - G), whose exponent is summed from the end so that it loses nothing to cancellation.
#pragma once

#include "bf16_planes.cuh"

namespace gdn {
namespace ssm {

constexpr int kC = 64;          // tokens of a chunk
constexpr int kGateRows = 5;    // dt, G hi, G lo, b, r
constexpr float kMinLog = -128.f;  // a log decay below it is a decay to zero

// A sum in two floats, h + l.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {
    const float s = a.h + b.h, z = s - a.h;
    const float e = (a.h - (s - z)) + (b.h - z) + (a.l + b.l);
    Two r;
    r.h = s + e;
    r.l = e - (r.h - s);
    return r;
}
__device__ __forceinline__ void two_add(Two& a, float x) {
    const float s = a.h + x, z = s - a.h;
    a.l += (a.h - (s - z)) + (x - z);
    a.h = s;
}
__device__ __forceinline__ Two two_shfl(Two a, int mask) {
    return Two{__shfl_xor_sync(0xffffffffu, a.h, mask), __shfl_xor_sync(0xffffffffu, a.l, mask)};
}

struct Chunk {
    int n, k, bos, eos, t0, len;  // sequence, chunk of it, its tokens, the chunk's first token, tokens in it
};
// The chunk of a slot; false where the slot holds none.  The whole block takes part.
__device__ __forceinline__ bool find_chunk(const Packed& s, int slot, int* err, Chunk& c) {
    c.n = packed_find(s, slot, kC, 1, err);
    if (c.n < 0 || c.n >= s.num_seqs) return false;
    c.bos = s.bos(c.n);
    c.eos = s.bos(c.n + 1);
    c.k = slot - (c.bos / kC + c.n);
    c.t0 = c.bos + c.k * kC;
    c.len = min(c.eos - c.t0, kC);
    return c.len > 0;
}
inline long slots_of(int num_seqs, int total_T) { return (long)total_T / kC + num_seqs; }

struct Work {
    float* gates;     // [slots][H][kGateRows][64]
    float* states;    // [slots][H][P][N], at the chunks' starts
    float* dstates;   // [slots][H][P][N], at the chunks' ends
    float* sums;      // [3][slots][H]: dA_log, ddt_bias, dD of each chunk
    float* parts;     // [subsets][total_T][G][N] twice (dB, dC), with more than one subset of a group's heads
    int subsets;
};

// Launches the gates, and the states at the chunks' starts; `both`: also their gradients at the chunks' ends.
cudaError_t launch_gates(const SsmArgs& a, const Work& w, cudaStream_t s);
cudaError_t launch_scan(const SsmArgs& a, const Work& w, bool both, cudaStream_t s);
// The whole forward pass of bf16 prompts (ssm_tc.cu), for total_T > 0.
size_t tc_workspace_bytes(int num_seqs, int total_T, int H, int P, int N);
cudaError_t launch_tc(const SsmArgs& a, cudaStream_t s);
// The gradients of bf16 prompts (ssm_tc_bwd.cu), for total_T > 0, and what every backward pass ends with: dB and dC added
// up, zeros outside the sequences, sums over the slots.
size_t tc_bwd_workspace_bytes(int num_seqs, int total_T, int H, int G, int P, int N);
cudaError_t launch_tc_bwd(const SsmArgs& a, cudaStream_t s);
cudaError_t launch_finish(const SsmArgs& a, const Work& w, long slots, cudaStream_t s);

}  // namespace ssm
}  // namespace gdn

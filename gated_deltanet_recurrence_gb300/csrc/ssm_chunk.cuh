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

constexpr int kSMs = 152;
constexpr int kC = 64;          // tokens of a chunk
constexpr int kGateRows = 5;    // dt, G hi, G lo, b, r
constexpr float kMinLog = -128.f;  // a log decay below it is a decay to zero
// fmaxf would make a decay to zero of a NaN.
__device__ __forceinline__ float log_decay(float rate, float dt) {
    const float g = -rate * dt;
    return g < kMinLog ? kMinLog : g;
}

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
// The chunk (of TOKENS) of a slot; false where the slot holds none.  The whole block takes part.
template <int TOKENS = kC>
__device__ __forceinline__ bool find_chunk(const Packed& s, int slot, int* err, Chunk& c) {
    c.n = packed_find(s, slot, TOKENS, 1, err);
    if (c.n < 0 || c.n >= s.num_seqs) return false;
    c.bos = s.bos(c.n);
    c.eos = s.bos(c.n + 1);
    c.k = slot - (c.bos / TOKENS + c.n);
    c.t0 = c.bos + c.k * TOKENS;
    c.len = min(c.eos - c.t0, TOKENS);
    return c.len > 0;
}
inline long slots_of(int num_seqs, int total_T) { return (long)total_T / kC + num_seqs; }

// Sequences are walked along whole, or, where that leaves SMs idle, in segments of `each` chunks at once: first every
// segment's own end state (from zero), then those joined into the states that the segments begin with.  Segments have
// slots as chunks have; an empty sequence has one segment.  Index 1 of a pair: backwards, gradients of states.
struct Segments {
    int each, unit;   // chunks of a segment (0: whole sequences), tokens of a chunk
    float* decay[2];  // [slots][H]: e^{sum of the segment's log decays}
    float* own[2];    // [slots][H][P][N]
    float* start[2];
};
struct Run {
    int n, t0, end;     // sequence, tokens
    bool first, last;   // of its sequence
    long slot0;         // of its first chunk
};
// The segment of slot `index`, or sequence `index`; false where there is none.  The whole block takes part.
__device__ __forceinline__ bool find_run(const Packed& s, int each, int chunk, int index, int* err, Run& r) {
    const int unit = each * chunk, found = each ? packed_find(s, index, unit, 1, err) : packed_find(s, 0, 1, 0, err);
    if (each ? found < 0 || found >= s.num_seqs : found == -2) return false;
    r.n = each ? found : index;
    const int bos = s.bos(r.n), eos = s.bos(r.n + 1), k = each ? index - (bos / unit + r.n) : 0;
    r.t0 = bos + k * unit;
    r.first = k == 0;
    if (!r.first && r.t0 >= eos) return false;
    r.last = !each || eos - r.t0 <= unit;
    r.end = r.last ? eos : r.t0 + unit;
    r.slot0 = bos / chunk + r.n + (long)k * each;
    return true;
}
inline long segment_slots(int num_seqs, int total_T, const Segments& g) { return (long)total_T / (g.each * g.unit) + num_seqs; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// ssm_fwd.cu: the segments of a call and the workspace that they need, laid out from `at` (`varied`: the lengths may
// differ).  The cost of a chunk, in us: along whole sequences, for a segment's own state; of what segments need besides.
struct SegmentCost {
    double whole, own, more;
};
size_t segments_layout(int num_seqs, int total_T, int H, int P, int N, int unit, int directions, bool varied, SegmentCost cost,
                       Segments* g, unsigned char* at);
cudaError_t launch_join(const SsmArgs& a, const Segments& g, int directions, cudaStream_t s);

struct Work {
    float* gates;     // [slots][H][kGateRows][64]
    float* states;    // [slots][H][P][N], at the chunks' starts
    float* dstates;   // [slots][H][P][N], at the chunks' ends
    float* sums;      // [3][slots][H]: dA_log, ddt_bias, dD of each chunk
    float* parts;     // [subsets][total_T][G][N] twice (dB, dC), with more than one subset of a group's heads
    int subsets;
    Segments g;
};

// The segments of a fp32 call.  Launches the gates, and the states at the chunks' starts; with two directions also their
// gradients at the chunks' ends.
inline size_t segments64(int num_seqs, int total_T, int H, int P, int N, int directions, bool varied, Segments* g, unsigned char* at) {
    const double chunk = N == 128 ? 3.3 : 2.1;
    return segments_layout(num_seqs, total_T, H, P, N, kC, directions, varied, SegmentCost{chunk, chunk, 8.}, g, at);
}
cudaError_t launch_gates(const SsmArgs& a, const Work& w, cudaStream_t s);
cudaError_t launch_scan(const SsmArgs& a, const Work& w, int directions, cudaStream_t s);
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

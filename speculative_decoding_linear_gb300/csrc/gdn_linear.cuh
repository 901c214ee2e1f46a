// gdn_linear.cuh -- segments, layouts and gates shared by the kernels of decay-gated linear
// attention over sequences (gdn_linear_seq_forward / gdn_linear_seq_backward).
//
// Without the delta rule's erasure a segment of tokens adds to the state what does not depend on
// the state before it:
//   S_end = e^G S + sum_s e^{G - g_s} beta_s v_s k_s^T,      g the running sum of log_alpha, G its end
//   o_t   = e^{g_t} S q_t + sum_{s <= t} e^{g_t - g_s} beta_s (q_t.k_s) v_s
// so every segment's sum is formed at once, a scan over the segments (one multiply and add for each
// element of the state) gives the states between them, and every segment's rows are formed at once.
// The gradients have the same shape, with the scan from the end.
#pragma once

#include "gdn_seq.cuh"

namespace gdn {

// Segment c of sequence s has the slot offset_s / L + s + c (see seq_slots: those of different
// sequences never meet).
__host__ __device__ inline int seg_slots(int nseq, int total, int L) { return total / L + nseq; }
__device__ __forceinline__ int seg_slot0(int first, int s, int L) { return first / L + s; }

// Sequence, first token and tokens of a slot's segment, and its number in the sequence: false for
// an empty slot.  The search ends for any content of the offsets; seq_range checks the sequence found.
__device__ __forceinline__ bool slot_segment(const SeqShape& a, int L, int slot, int& s, int& c, int& first, int& rows, int* err) {
    int lo = 0, hi = a.nseq - 1;
    const int len = a.total / a.nseq;
    while (lo < hi) {
        const int m = lo + ((hi - lo + 1) >> 1);
        const int o = a.offsets == nullptr ? m * len : min(max(a.offsets[m], 0), a.total);
        if (o / L + m <= slot) lo = m; else hi = m - 1;
    }
    s = lo;
    int b, n;
    if (!seq_range(a, s, b, n, err)) return false;
    c = slot - seg_slot0(b, s, L);
    if (c < 0 || (long long)c * L >= n) return false;
    first = b + c * L;
    rows = min(L, n - c * L);
    return true;
}

// Places in the record (kept from the forward pass to the backward one) and in the workspace.
//   start   states at the segments' starts, for the rows' kernels: fp32, or bf16 terms (in the record, if there is one)
//   gates   what the gates of each (slot, head) give, and where each slot's segment lies (likewise)
//   end     gradients of the states at the segments' ends
//   local   what each segment adds to the state (or to its gradient), fp32
//   gend    e^G of each (slot, head)
//   phi     e^G <dS_end, S_start> by pieces of the state
//   part    per token: sums that the gates' gradients are made of
struct LinLayout {
    size_t rec_gates, rec_total;
    size_t ws_local, ws_gend, ws_start, ws_gates, ws_forward, ws_end, ws_phi, ws_part, ws_heads, ws_total;
};
LinLayout lin_layout(const SeqShape& s, int dtype);
LinLayout lin_layout_tc(const SeqShape& s);
constexpr int kLinSegment = 512;                     // tokens of a segment with bf16 inputs

constexpr int kScanThreads = 256;
constexpr int kScanTile = kScanThreads * 4;          // elements of a state that one CTA of the scan takes
inline int scan_tiles(const SeqShape& s) { return (s.dk * s.dv + kScanTile - 1) / kScanTile; }

// A sum of log decays as two floats (48 bits: differences of long sums stay exact; doubles would take sixteen cycles
// an operation of a warp), added with the error of each addition kept.
struct LogSum {
    float hi, lo;
};
__device__ __forceinline__ LogSum operator+(LogSum a, LogSum b) {
    const float s = a.hi + b.hi, y = s - a.hi;
    const float e = ((a.hi - (s - y)) + (b.hi - y)) + (a.lo + b.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}
__device__ __forceinline__ LogSum operator-(LogSum a, LogSum b) { return a + LogSum{-b.hi, -b.lo}; }
// e^(hi + lo): an exponent rounded to one float would cost |hi| 2^-24 of the decay
__device__ __forceinline__ float decay_of(LogSum a) {
    const float e = expf(a.hi);
    return fmaf(e, a.lo, e);
}

// Inclusive sums over a warp's lanes.
__device__ __forceinline__ LogSum warp_scan(LogSum x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const LogSum y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if ((int)(threadIdx.x & 31) >= o) x = x + y;
    }
    return x;
}

cudaError_t launch_linear_forward_tc(const SeqArgs& a, cudaStream_t st);
cudaError_t launch_linear_backward_tc(const SeqArgs& a, cudaStream_t st);
cudaError_t launch_linear_scan(const SeqShape& sh, int L, int terms, bool back, const float* local, const float* gend, int gend_apart, const float* S0,
                               void* out, size_t apart, const void* start, float* phi, float* last, int* err, cudaStream_t st);

}  // namespace gdn

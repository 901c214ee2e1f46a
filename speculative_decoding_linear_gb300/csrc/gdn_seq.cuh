// gdn_seq.cuh -- argument blocks, chunk slots and layouts shared by the sequence
// operators' kernels (gdn_seq_forward / gdn_seq_backward).
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr int kChunk = 64;        // tokens per chunk of the sequence operators
constexpr int kSMs = 152;

struct SeqShape {
    int nseq, total, H, Hk, dk, dv;
    const int32_t* offsets;       // [nseq + 1], or nullptr: total / nseq tokens each
    int ldq, ldk, ldv;            // elements from one token to the next
};

// Chunk c of sequence s has the slot offset_s / 64 + s + c.  A sequence of n tokens takes
// ceil(n / 64) <= n / 64 + 1 slots, so the slots of different sequences never meet, and a
// chunk's place needs no table of chunk counts.  Some slots stay empty.
__host__ __device__ inline int seq_slots(int nseq, int total) { return total / kChunk + nseq; }

// First token and length of sequence s.  Returns false, and records GDN_ERR_INDEX, where the
// offsets are not nondecreasing inside [0, total]; nothing of that sequence is touched then.
__device__ __forceinline__ bool seq_range(const SeqShape& a, int s, int& first, int& len, int* err) {
    if (a.offsets == nullptr) {
        len = a.total / a.nseq;
        first = s * len;
        return true;
    }
    const int b = a.offsets[s], e = a.offsets[s + 1];
    first = b;
    len = e - b;
    if (b < 0 || e < b || e > a.total) {
        set_error(err, GDN_ERR_INDEX);
        first = len = 0;
        return false;
    }
    return true;
}

__device__ __forceinline__ int seq_slot0(const SeqShape& a, int s) {
    return (a.offsets == nullptr ? s * (a.total / a.nseq) : a.offsets[s]) / kChunk + s;
}

__device__ __forceinline__ int seq_end(const SeqShape& a, int s) {
    return a.offsets == nullptr ? (s + 1) * (a.total / a.nseq) : a.offsets[s + 1];
}

// Tokens of no sequence lie before `b`, the first offset, and from `e`, the last, on (a batch padded to a fixed
// number of tokens).  False where there are none.
__device__ __forceinline__ bool seq_outside(const SeqShape& a, int& b, int& e) {
    if (a.offsets == nullptr) return false;
    b = min(max(a.offsets[0], 0), a.total);
    e = min(max(a.offsets[a.nseq], b), a.total);
    return b > 0 || e < a.total;
}

// Those tokens' rows of `row` elements become zero, by all threads of the grid from `skip` of a CTA on.
template <typename T>
static __device__ __noinline__ void zero_rows(void* p, size_t row, int b, int e, int total, int skip = 0) {
    const int each = blockDim.x - skip;
    const size_t i0 = (size_t)blockIdx.x * each + (threadIdx.x - skip), n = (size_t)gridDim.x * each;
    for (size_t i = i0; i < b * row; i += n) static_cast<T*>(p)[i] = T{};
    for (size_t i = e * row + i0; i < total * row; i += n) static_cast<T*>(p)[i] = T{};
}

// Sequence and chunk of a slot: false for an empty slot.  The search is for the last
// sequence whose first slot is not behind `slot`; it ends for any content of the offsets,
// and seq_range checks the one that it finds.
__device__ __forceinline__ bool slot_chunk(const SeqShape& a, int slot, int& s, int& first, int& rows, int* err) {
    if (a.offsets == nullptr) {
        // the same search by bisection on s * len / 64 + s
        const int len = a.total / a.nseq;
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (m * len / kChunk + m <= slot) lo = m; else hi = m - 1;
        }
        s = lo;
    } else {
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int m = lo + ((hi - lo + 1) >> 1);
            const int o = min(max(a.offsets[m], 0), a.total);
            if (o / kChunk + m <= slot) lo = m; else hi = m - 1;
        }
        s = lo;
    }
    int b, n;
    if (!seq_range(a, s, b, n, err)) return false;
    const int c = slot - (b / kChunk + s);
    if (c < 0 || c * kChunk >= n) return false;
    first = b + c * kChunk;
    rows = min(kChunk, n - c * kChunk);
    return true;
}

struct SeqArgs {
    SeqShape sh;
    const void *q, *k, *v;
    const float *la, *beta;
    const float* S0;              // nullptr: zero
    void* out;
    float* S_T;                   // nullptr: not wanted
    // backward
    const void* dout;
    const float* dS_T;            // nullptr: zero
    void *dq, *dk, *dv;
    float *dla, *dbeta;
    float* dS0;                   // nullptr: not wanted
    char* ws;
    char* rec;                    // nullptr: forward without a record
    int* err;
};

// Record (kept from the forward pass to the backward one) and workspace of the path that a
// call's sizes and type take.
struct SeqLayout {
    size_t rec_S, rec_eps, rec_o, rec_op, rec_total;     // record: chunk start states, errors, outputs, chunk operands
    size_t ws_dS, ws_dV, ws_dq, ws_dk, ws_op, ws_part, ws_phi, ws_total;   // workspace
    size_t ws_forward() const { return ws_part; }        // what a forward pass takes of it: the chunk operands
};

SeqLayout seq_layout(const SeqShape& s, int dtype);

// log decay as the kernels use it: a log_alpha of -inf (the state forgotten) is e^{-200} = 0 in
// fp32, and stays finite in differences; a NaN stays one.
__device__ __forceinline__ float gate_log(float la) { return la < -200.f ? -200.f : la; }

cudaError_t launch_seq_forward_f32(const SeqArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_seq_backward_f32(const SeqArgs& a, int dtype, cudaStream_t st);

}  // namespace gdn

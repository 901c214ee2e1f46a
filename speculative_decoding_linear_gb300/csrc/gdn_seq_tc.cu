// gdn_seq_tc.cu -- the gated delta rule over packed sequences on the tensor core (bf16 inputs;
// d_k is taken up to 64, 128, 192 or 256 with columns of zero): forward and backward pass.
//
// In a chunk of C = 64 tokens with start state S (here d_k x d_v), g the cumulative log gate,
// G_tj = e^{g_t - g_j}, L = strictly lower G (.) K K^T, P = lower G (.) Q K^T:
//   r = V - e^g K S,  eps = That r,  That = (I + L diag(beta))^{-1},  delta = beta eps
//   O = e^g Q S + Phat r,  Phat = P diag(beta) That
//   S+ = e^{g_end} S + K^T (e^{g_end - g} delta)
// That and Phat need no state: seq_prep_kernel forms them for all chunks at once.  The chunks
// of a sequence then follow one another in seq_fwd_kernel, one CTA for each NV value columns of
// a (sequence, head), which are independent.  A chunk is three dependent products,
//   [K; Q] S  ->  [That; Phat] r  ->  K^T (bt eps),
// and what bounds a long sequence is their latency: a chain of T / 64 chunks.  S stays in
// registers in fp32 (a row of d_k for each thread, NV columns of it) and goes to shared memory as
// two bf16 terms for the first product; That and Phat have two as well, r and bt eps three.  A pass that
// keeps a record takes three of all: the gates' gradients are differences of dots with o and eps.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_seq_tc.cuh"

namespace gdn {

using namespace seqtc;

namespace {

// ---------------------------------------------------------------------------
// seq_prep_kernel: the operands and gates of one (chunk, head)
// ---------------------------------------------------------------------------
// K K^T and Q K^T are one product [K; Q] K^T.  (I + A)^-1 of a strictly lower A is found in two
// blocks of 32, each by substitution, a column for each thread in registers, row after row: no step
// waits for another thread, and what a row adds to those below it is independent of one another.
// Phat then is a second product.  With a record T = (I + diag(beta) L)^-1 is found beside That by other
// warps, Ptil = P T, and Phat = Ptil diag(beta) since diag(beta) That = T diag(beta).
// Bound by the instructions of the exponentials, substitutions and splits: 8192 tokens of 8 heads of 256 36 us
// (100 MB: 2.8 TB/s), with a record 58; one chunk alone 10 us, a chain of its stages.
constexpr int kPrepThreads = 256;
constexpr int kLd = kChunk + 4;          // fp32 rows on 16 bytes

template <int DK, bool REC>
struct PrepGeom {
    static constexpr int kSides = REC ? 2 : 1;
    static constexpr uint32_t kTile = 128 * 128;                 // [K; Q], 64 columns
    static constexpr uint32_t kKQ = (DK / 64) * kTile;
    // over them: A^T (with a record diag(beta) L behind it), in its place That and T; the images of P
    // (later of Phat), of That, and of T; Ptil's image takes the place of That and T
    static constexpr uint32_t kMat = kChunk * kLd * 4;
    static constexpr uint32_t kImage = 3 * 64 * 128;             // 64 rows of 64, three terms
    static constexpr uint32_t kP = (kSides * kMat + 1023) & ~1023u;
    static constexpr uint32_t kT = kP + kImage;
    static constexpr uint32_t kMats = kT + kSides * kImage;
    static constexpr uint32_t kBuf = kKQ > kMats ? kKQ : kMats;
    static constexpr uint32_t kSmem = kBuf + 2048 + 1024;
    static_assert(kP >= (REC ? kImage : 0) && kBuf % 1024 == 0, "images");
};

// (h, l) += (yh, yl), each pair the sum of a float and the rounding error of it (Knuth's two-sum)
__device__ __forceinline__ void add2(float& h, float& l, float yh, float yl) {
    const float s = __fadd_rn(h, yh), z = __fsub_rn(s, h);
    const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(s, z)), __fsub_rn(yh, z));
    const float t = __fadd_rn(e, __fadd_rn(l, yl));
    h = __fadd_rn(s, t);
    l = __fsub_rn(t, __fsub_rn(h, s));
}

template <int DK, bool REC>
__global__ void __launch_bounds__(kPrepThreads, REC ? 2 : 3)
    seq_prep_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, SeqArgs a, char* ops) {
    using G = PrepGeom<DK, REC>;
    constexpr uint32_t kHalf = 64 * 128;                  // one term of an image
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    float* M = reinterpret_cast<float*>(sm);              // A^T, then That; behind it diag(beta) L, then T
    float* ghi = reinterpret_cast<float*>(sm + G::kBuf);
    float* glo = ghi + kChunk;
    float* bt = glo + kChunk;
    uint32_t* holder = reinterpret_cast<uint32_t*>(bt + kChunk);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const uint32_t bar = base + G::kBuf + 1024, bar2 = bar + 8, bar3 = bar + 16;

    const SeqShape& sh = a.sh;
    const int h = blockIdx.x % sh.H, slot = blockIdx.x / sh.H, hk = h / (sh.H / sh.Hk);
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    int s, first, rows;
    // by warps that have nothing to do before the product
    const auto zero_outside = [&] {
        int b, e;
        if (tid >= 128 && seq_outside(sh, b, e)) zero_rows<uint4>(a.out, (size_t)sh.H * sh.dv / 8, b, e, sh.total, 128);
    };
    if (!slot_chunk(sh, slot, s, first, rows, a.err)) {
        zero_outside();
        griddep_launch();
        return;
    }
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar2, 1);
        mbar_init(bar3, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        fence_proxy_async_smem();
        mbar_expect_tx(bar, G::kKQ);
#pragma unroll
        for (int b = 0; b < DK / 64; ++b) {
            tma_3d(base + b * G::kTile, &tmK, 64 * b, hk, first, bar);
            tma_3d(base + b * G::kTile + 8192, &tmQ, 64 * b, hk, first, bar);
        }
    }
    zero_outside();
    if (warp == 1) tmem_alloc(smem_u32(holder), 128);
    if (warp == 2) {
        // inclusive sum of the log gates as two floats, their difference exact to 2^-48 of the sum: the
        // exponents are differences of far tokens.  (In 64 bits this took 5 us, longer than all the rest.)
        float xh[2], xl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i;
            xh[i] = t < rows ? gate_log(a.la[((size_t)first + t) * sh.H + h]) : 0.f;
            xl[i] = 0.f;
            bt[t] = t < rows ? a.beta[((size_t)first + t) * sh.H + h] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float yh = __shfl_up_sync(0xffffffffu, xh[i], o), yl = __shfl_up_sync(0xffffffffu, xl[i], o);
                if (lane >= o) add2(xh[i], xl[i], yh, yl);
            }
        }
        add2(xh[1], xl[1], __shfl_sync(0xffffffffu, xh[0], 31), __shfl_sync(0xffffffffu, xl[0], 31));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ghi[lane + 32 * i] = xh[i];
            glo[lane + 32 * i] = xl[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(*holder);
    if (warp == 0) {
        wait_or_dead(bar, 0, a.err, dead);
        __syncwarp();
        if (elect_one()) {
            const uint64_t d = k_desc<128>(base);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const uint64_t t = d + (((k / 4) * G::kTile + 32 * (k % 4)) >> 4);
                mma_bf16(tmem, t, t, idesc_bf16(128, 64), k != 0);
            }
            mma_commit(bar2);
        }
    }
    // the gates, while the product runs
    char* op = ops + (size_t)blockIdx.x * (REC ? kOpRecord : kOpBytes);
    if (tid >= 64 && tid < 128) {
        const int t = tid - 64;
        float* gates = reinterpret_cast<float*>(op);
        const float eh = ghi[rows - 1], el = glo[rows - 1], tail = expf((eh - ghi[t]) + (el - glo[t]));
        gates[kGBt + t] = bt[t] * tail;
        gates[kGEg + t] = expf(ghi[t] + glo[t]);
        gates[kGTail + t] = tail;
        gates[kGBeta + t] = bt[t];
        if (t < 4) gates[kGEnd + t] = expf(eh + el);
        gates[kGHi + t] = ghi[t];
        gates[kGLo + t] = glo[t];
    }
    wait_or_dead(bar2, 0, a.err, dead);
    __syncwarp();
    tc_fence_after();
    // row t of K K^T (lanes 0..63) and of Q K^T (lanes 64..127); 32 columns for each half of the warps,
    // eight at a time (a loop: code that runs once a chunk costs its fetches)
    {
        const int t = 32 * (warp & 1) + lane, c0 = 32 * (warp >> 2);
        const bool strict = !(warp & 2);
        const float gh = ghi[t], gl = glo[t], bb = bt[t];
        // rows 0..31 see no column of the second half; a token past the sequence's end sees none, whatever
        // lies in its q and k
        const int seen = t < rows ? t + (strict ? 0 : 1) : 0;
        const bool none = (warp & 1) == 0 && c0 != 0;
#pragma unroll 1
        for (int j = c0; j < c0 + 32; j += 8) {
            float x[8] = {};
            if (!none) {
                uint32_t d[8];
                tmem_ld_n(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + j, d);
                const float4 h0 = *reinterpret_cast<const float4*>(ghi + j), h1 = *reinterpret_cast<const float4*>(ghi + j + 4),
                             l0 = *reinterpret_cast<const float4*>(glo + j), l1 = *reinterpret_cast<const float4*>(glo + j + 4);
                const float hh[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w}, ll[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // outside the mask the exponent may be large: it is not evaluated there
                    const bool in = j + e < seen;
                    const float ex = expf(in ? (gh - hh[e]) + (gl - ll[e]) : 0.f);
                    x[e] = in ? __uint_as_float(d[e]) * ex : 0.f;
                }
            }
            const float4 b0 = *reinterpret_cast<const float4*>(bt + j), b1 = *reinterpret_cast<const float4*>(bt + j + 4);
            const float be[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
            if (strict) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    M[(j + e) * kLd + t] = x[e] * be[e];
                    if (REC) M[kChunk * kLd + (j + e) * kLd + t] = x[e] * bb;
                }
            } else {
                if (!REC)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= be[e];
                put_terms<128, 3>(base + G::kP, kHalf, t, j, x);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // (I + A)^-1 in two steps: by substitution the blocks of 32 on the diagonal, a column of one for each
    // of 64 threads (128 with a record), two rows an instruction ...
    const bool solves = warp < 2 * G::kSides;
    float* mine = M + (warp >> 1) * kChunk * kLd;
    {
        const int o = warp & 1 ? 32 : 0;
        float2 x[16];
        if (solves) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = make_float2(2 * i == lane ? 1.f : 0.f, 2 * i + 1 == lane ? 1.f : 0.f);
            const float* m = mine + o * kLd + o;
#pragma unroll
            for (int k = 0; k < 31; ++k) {
                const float xk = k & 1 ? x[k / 2].y : x[k / 2].x;
                const float2 nx = make_float2(-xk, -xk);
#pragma unroll
                for (int i = (k + 1) & ~3; i < 32; i += 4) {      // rows up to k in the first four meet zeros
                    const float4 w = *reinterpret_cast<const float4*>(m + k * kLd + i);
                    if (i + 1 > k) x[i / 2] = ffma2(make_float2(w.x, w.y), nx, x[i / 2]);
                    x[i / 2 + 1] = ffma2(make_float2(w.z, w.w), nx, x[i / 2 + 1]);
                }
            }
        }
        // ... each into its place (in rows now; the transposed A21 in the upper right stays) ...
        __syncwarp();
        if (solves)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                mine[(o + 2 * i) * kLd + o + lane] = x[i].x;
                mine[(o + 2 * i + 1) * kLd + o + lane] = x[i].y;
            }
    }
    __syncthreads();
    // ... then T21 = - T22 (A21 T11), four columns of a row for each thread
    {
        const int t = (tid >> 3) & 31, c = 4 * (tid & 7);
        float2 y[G::kSides][2] = {};
#pragma unroll
        for (int z = 0; z < G::kSides; ++z) {
            float* m = M + z * kChunk * kLd;
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const float u = m[k * kLd + 32 + t];              // A21[t][k], transposed
                const float4 w = *reinterpret_cast<const float4*>(m + k * kLd + c);
                y[z][0] = ffma2(make_float2(u, u), make_float2(w.x, w.y), y[z][0]);
                y[z][1] = ffma2(make_float2(u, u), make_float2(w.z, w.w), y[z][1]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int z = 0; z < G::kSides; ++z)
            *reinterpret_cast<float4*>(M + z * kChunk * kLd + t * kLd + 32 + c) = make_float4(y[z][0].x, y[z][0].y, y[z][1].x, y[z][1].y);
        __syncthreads();
#pragma unroll
        for (int z = 0; z < G::kSides; ++z) {
            float* m = M + z * kChunk * kLd;
            y[z][0] = y[z][1] = make_float2(0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const float u = -m[(32 + t) * kLd + 32 + k];
                const float4 w = *reinterpret_cast<const float4*>(m + k * kLd + 32 + c);
                y[z][0] = ffma2(make_float2(u, u), make_float2(w.x, w.y), y[z][0]);
                y[z][1] = ffma2(make_float2(u, u), make_float2(w.z, w.w), y[z][1]);
            }
            *reinterpret_cast<float4*>(m + (32 + t) * kLd + c) = make_float4(y[z][0].x, y[z][0].y, y[z][1].x, y[z][1].y);
        }
    }
    __syncthreads();
    // That (and T) as operands
#pragma unroll 1
    for (int i = 0; i < 2 * G::kSides; ++i) {
        const int r = (tid >> 3) + 32 * (i & 1), c = tid & 7;
        const float* m = M + (i >> 1) * kChunk * kLd + r * kLd + 8 * c;
        const float4 u = *reinterpret_cast<const float4*>(m), w = *reinterpret_cast<const float4*>(m + 4);
        float v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
        if (r < 32 && c >= 4)                             // above the diagonal blocks
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        put_terms<128, 3>(base + G::kT + (i >> 1) * G::kImage, kHalf, r, 8 * c, v);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int odd = (slot - seq_slot0(sh, s)) & 1;
    if (warp == 0) {
        if (elect_one()) {
            // P's 64 rows and whatever lies behind (lanes that nothing reads), term t with the first 3 - t
            // of the other, the small products first
            const uint64_t dP = k_desc<128>(base + G::kP), dT = mn_desc<128>(base + G::kT + (REC ? G::kImage : 0), 0);
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                for (int t = 0; t <= sum; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + 64, dP + ((t * kHalf + 32 * k) >> 4), dT + (((sum - t) * kHalf + k * 2048) >> 4),
                                 idesc_bf16(128, 64) | kBMn, sum != 2 || t + k != 0);
            mma_commit(bar3);
            // the operands' halves are 64 rows of each term
#pragma unroll
            for (int z = 0; z < (REC ? 3 : 2); ++z) bulk_s2g(op + kOpGates + z * kOpTerm + (odd ? kHalf : 0), base + G::kT + z * kHalf, kHalf);
            if (REC)
#pragma unroll
                for (int z = 0; z < 3; ++z) bulk_s2g(op + kOpBack + z * kOpTerm, base + G::kT + G::kImage + z * kHalf, kHalf);
        }
        __syncwarp();
    }
    wait_or_dead(bar3, 0, a.err, dead);
    __syncwarp();
    tc_fence_after();
    if (tid == 0 && *dead) {                              // copies and products in flight end before the CTA does
        mbar_wait(bar, 0, a.err);
        mbar_wait(bar2, 0, a.err);
        mbar_wait(bar3, 0, a.err);
    }
    __syncwarp();
    if ((warp & 2) == 0) {
        const int t = 32 * (warp & 1) + lane, c0 = 32 * (warp >> 2);
        float y[32];
        tmem_sum<32, 1>(tmem + 64 + ((uint32_t)(32 * (warp & 3)) << 16) + c0, 0, y);
        if (REC) {
            put_terms<128, 3>(base, kHalf, t, c0, y);     // over That and T, which the images hold
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] *= bt[c0 + j];
        }
        put_terms<128, REC ? 3 : 2>(base + G::kP, kHalf, t, c0, y);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && elect_one()) {
#pragma unroll
        for (int z = 0; z < (REC ? 3 : 2); ++z) bulk_s2g(op + kOpGates + z * kOpTerm + (odd ? 0 : kHalf), base + G::kP + z * kHalf, kHalf);
        if (REC)
#pragma unroll
            for (int z = 0; z < 3; ++z) bulk_s2g(op + kOpBack + z * kOpTerm + kHalf, base + z * kHalf, kHalf);
        bulk_all_done();
    }
    __syncwarp();
    griddep_launch();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
}

// ---------------------------------------------------------------------------
// seq_fwd_kernel
// ---------------------------------------------------------------------------
// Ten warps.  Eight compute: a thread owns a row of the state, and a token's row of K (warps
// 0, 1, 4, 5; in odd chunks the others) or of Q in the token steps, columns halved between warps 0-3
// and 4-7.  One starts the copies of K, Q, V, the gates and [That; Phat], one issues the products.
//
// Bound by a chunk's chain: some 1.5 us with 16 columns and heads of 256, of which the three products and their
// handovers between warps are the larger part.  1 x 8192, 8 heads of 256 (16 columns, 128 CTAs): 196 us.
// 4 x 2048 (32 columns, 256 CTAs): 142 us, with a record 188.
template <int DK, int NV, int ST>
struct FwdGeom {
    static constexpr int kMH = DK > 128 ? 2 : 1;                  // halves of 128 rows of d_k
    static constexpr int kW = NV * 2;                             // bytes of an operand row
    // 64 columns of d_k: 64 rows of an even chunk's K, of Q, of an odd chunk's K.  [K; Q] and [Q; K] are
    // 128 rows behind one another, K is there for two chunks and Q for one
    static constexpr uint32_t kTile = 192 * 128;
    static constexpr uint32_t kTP = 2 * kMH * kTile;              // filled up to 128 or 256 columns
    static constexpr uint32_t kS = kTP + ST * kOpTerm;            // ST terms
    static constexpr uint32_t kSTerm = DK * kW;
    static constexpr uint32_t kR = kS + ST * kSTerm;              // three terms
    static constexpr uint32_t kRTerm = 64 * kW;
    static constexpr uint32_t kV = kR + 3 * kRTerm;               // one V; gates of two chunks
    static constexpr uint32_t kG = kV + 64 * kW;
    static constexpr uint32_t kBar = kG + 2 * kGateFwd;
    static constexpr uint32_t kSmem = kBar + 256 + 1024;
    static constexpr int kD1 = 0, kD2 = ST * NV, kD3 = kD2 + 3 * NV, kCols = kD3 + kMH * 3 * NV;
    static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kSmem <= 227 * 1024, "tile");
};
constexpr int kFwdThreads = 320;

// More than one CTA per SM must not ask for more than the 512 columns of its TMEM.
template <int DK, int NV, int ST>
constexpr size_t fwd_smem() {
    using G = FwdGeom<DK, NV, ST>;
    const size_t least = G::kAlloc == 512 ? 116 * 1024 : G::kAlloc == 256 ? 78 * 1024 : 58 * 1024;
    return G::kSmem > least ? G::kSmem : least;
}

// The sequence of the r-th place by length, the longest first: a long one that begins when others have ended would
// work on alone.  In the order given where all CTAs begin at once, lengths are equal or there are too many to count
// (many sequences even out by themselves).  buf: 1028 bytes of shared memory.  Prep and scan of
// 24 prompts, 16000 tokens, 8 heads of 128: 169 to 171 us, in the order given 182 to 194; 9 sequences with the
// longest, of 2000, at the end, 8 heads of 256: 142 against 169.
constexpr int kMaxRanked = 256;
__device__ __forceinline__ int seq_by_length(const SeqShape& sh, int r, int* buf) {
    if (sh.offsets == nullptr || sh.nseq > kMaxRanked || gridDim.x <= kSMs) return r;
    const int t = threadIdx.x;
    int n = 0;
    if (t < sh.nseq) buf[t] = n = (int)((uint32_t)sh.offsets[t + 1] - (uint32_t)sh.offsets[t]);
    __syncthreads();
    if (t < sh.nseq) {
        int rank = 0;
        for (int j = 0; j < sh.nseq; ++j) rank += buf[j] > n || (buf[j] == n && j < t);
        if (rank == r) buf[kMaxRanked] = t;
    }
    __syncthreads();
    return warp_uniform(buf[kMaxRanked]);
}

template <int DK, int NV, int ST>
__global__ void __launch_bounds__(kFwdThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, SeqArgs a, const char* ops, uint32_t op_bytes, char* recS, char* recE, float* recO) {
    using G = FwdGeom<DK, NV, ST>;
    constexpr int W = G::kW, NH = NV / 2;                 // NH: value columns of a thread in the token steps
    constexpr int SC = G::kMH == 2 ? NV : NH;             // value columns of a thread's state row
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    // copies landed (two stages; operands), their places free; products done; operands written
    const uint32_t full0 = base + G::kBar, empty0 = full0 + 16, tpf = full0 + 32, tpe = full0 + 40, b1 = full0 + 48,
                   b2 = full0 + 56, b3 = full0 + 64, drain = full0 + 72, vf = full0 + 80, ve = full0 + 88, qf = full0 + 96, qe = full0 + 104, ge0 = full0 + 112;
    uint32_t* holder = reinterpret_cast<uint32_t*>(sm + G::kBar + 160);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / NV;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H;
    const int s = seq_by_length(sh, blockIdx.x / (tiles * sh.H), reinterpret_cast<int*>(sm + G::kS));
    const int hk = h / (sh.H / sh.Hk), v0 = tile * NV;
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) {           // the whole CTA
        griddep_wait();                                   // the operands' kernel ends before this one
        return;
    }
    first = warp_uniform(first);
    len = warp_uniform(len);
    const int chunks = (len + kChunk - 1) / kChunk;
    const size_t slot0 = (size_t)(first / kChunk + s);

    if (tid == 0) {
        init_barriers(full0, 16, [&](uint32_t bar) { return bar == ve ? 4 : bar >= ge0 ? 8 : 1; });
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (DK % 128 != 0) {                                  // columns of d_k that no copy fills
        for (uint32_t o = tid * 16; o < G::kTile; o += kFwdThreads * 16) st_shared16(base + (DK / 64) * G::kTile + o, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 9) tmem_alloc(smem_u32(holder), G::kAlloc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(*holder);

    if (warp == 8) {
        griddep_wait();
        if (elect_one()) {
            int issued = 0, q_issued = 0, v_issued = 0, ops_issued = 0;
            // to L2 ahead of time: a copy that has to go to memory takes longer than a chunk
            auto prefetch = [&](int c) {
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) {
                    tma_prefetch_3d(&tmK, 64 * b, hk, first + c * kChunk);
                    tma_prefetch_3d(&tmQ, 64 * b, hk, first + c * kChunk);
                }
                tma_prefetch_2d(&tmV, h * sh.dv + v0, first + c * kChunk);
            };
            for (int c = 0; c < chunks; ++c) {
                if (c + 2 < chunks) prefetch(c + 2);
                if (c >= 2 && !(wait_or_dead(empty0 + 8 * (c & 1), ((c >> 1) & 1) ^ 1, a.err, dead) &&
                                wait_or_dead(ge0 + 8 * (c & 1), ((c >> 1) & 1) ^ 1, a.err, dead)))
                    break;
                const uint32_t f = full0 + 8 * (c & 1);
                const char* op = ops + ((slot0 + c) * sh.H + h) * op_bytes;
                mbar_expect_tx(f, DK * 128 + kGateFwd);
#pragma unroll
                for (int b = 0; b < DK / 64; ++b)
                    tma_3d(base + (c & 1) * 16384 + b * G::kTile, &tmK, 64 * b, hk, first + c * kChunk, f);
                bulk_copy_g2s(base + G::kG + (c & 1) * kGateFwd, op, kGateFwd, f);
                issued = c + 1;
                if (c >= 1 && !wait_or_dead(qe, (c - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(qf, DK * 128);
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) tma_3d(base + 8192 + b * G::kTile, &tmQ, 64 * b, hk, first + c * kChunk, qf);
                q_issued = c + 1;
                if (c >= 1 && !wait_or_dead(ve, (c - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(vf, 64 * W);
                tma_2d(base + G::kV, &tmV, h * sh.dv + v0, first + c * kChunk, vf);
                v_issued = c + 1;
                if (c >= 1 && !wait_or_dead(tpe, (c - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(tpf, ST * kOpTerm);
                bulk_copy_g2s(base + G::kTP, op + kOpGates, ST * kOpTerm, tpf);
                ops_issued = c + 1;
            }
            // copies in flight land before the CTA ends, though a warp that waits for them may give up
            for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) mbar_wait(full0 + 8 * (c & 1), (c >> 1) & 1, a.err);
            if (q_issued > 0) mbar_wait(qf, (q_issued - 1) & 1, a.err);
            if (v_issued > 0) mbar_wait(vf, (v_issued - 1) & 1, a.err);
            if (ops_issued > 0) mbar_wait(tpf, (ops_issued - 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 9) {
        // after a wait that gave up, products run on what is there: the result is void, the error recorded
        const uint64_t dS = mn_desc<W>(base + G::kS, G::kSTerm), dR = mn_desc<W>(base + G::kR, G::kRTerm), dTP = k_desc<128>(base + G::kTP);
        const bool leader = elect_one();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = c & 1;
            wait_or_dead(full0 + 8 * (c & 1), (c >> 1) & 1, a.err, dead);
            wait_or_dead(qf, ph, a.err, dead);
            __syncwarp();
            named_sync(1, 288);
            tc_fence_after();
            if (leader) {
                const uint64_t dKQ = k_desc<128>(base + (c & 1) * 8192);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(tmem + G::kD1, dKQ + (((k / 4) * G::kTile + 32 * (k % 4)) >> 4), dS + (k * 16 * W >> 4),
                             idesc_bf16(128, ST * NV) | kBMn, k != 0);
                mma_commit(b1);
                mma_commit(qe);
                if (ST == 3)
                    bulk_s2g(recS + (((slot0 + c) * sh.H + h) * tiles + tile) * (ST * G::kSTerm), base + G::kS, ST * G::kSTerm);
            }
            __syncwarp();
            wait_or_dead(tpf, ph, a.err, dead);
            __syncwarp();
            named_sync(2, 160);
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int t = 0; t < ST; ++t)              // term t with the first 3 - t of r
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + G::kD2, dTP + t * (kOpTerm >> 4) + 2 * k, dR + (k * 16 * W >> 4),
                                 idesc_bf16(128, (3 - t) * NV) | kBMn, t + k != 0);
                mma_commit(b2);
                mma_commit(tpe);
                if (ST == 3) bulk_read_done();    // S's image may be written again once b3 is through
            }
            __syncwarp();
            named_sync(3, 160);
            tc_fence_after();
            if (leader) {
                const uint64_t dK = mn_desc<128>(base + (c & 1) * 16384, G::kTile);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int m = 0; m < G::kMH; ++m)
                        mma_bf16(tmem + G::kD3 + m * 3 * NV, dK + ((2 * m * G::kTile + k * 2048) >> 4), dR + (k * 16 * W >> 4),
                                 idesc_bf16(128, 3 * NV) | kAMn | kBMn, k != 0);
                mma_commit(b3);
                mma_commit(empty0 + 8 * (c & 1));
            }
            __syncwarp();
        }
        if (leader) {
            if (ST == 3) bulk_all_done();
            mma_commit(drain);                            // products in flight end before their TMEM is freed, as above
            mbar_wait(drain, 0, a.err);
        }
        __syncwarp();
    } else {
        const int wg = warp >> 2, w4 = warp & 3;
        const int tok = 32 * (w4 & 1) + lane, vc = wg * NH;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const int srow = (G::kMH == 2 ? 128 * wg : 0) + 32 * w4 + lane, scol = G::kMH == 2 ? 0 : wg * NH;
        const bool owns = srow < DK;
        const bool whole = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;      // 32-byte rows of columns
        float S[SC];
        {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * sh.dk + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) S[j] = srow < sh.dk && a.S0 != nullptr ? a.S0[at + (size_t)j * sh.dk] : 0.f;
        }
        griddep_wait();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = c & 1;
            const bool reads_k = (w4 < 2) == ((c & 1) == 0);      // token rows of K, else of Q
            const int rows = min(kChunk, len - c * kChunk);
            // the state as the first product's operand: rows of d_k, value columns along the row
            if (owns) put_terms<W, ST>(base + G::kS, G::kSTerm, srow, scol, S);
            if (rows < kChunk) {
                // the copy brought tokens of what lies behind: rows of zero instead
                wait_or_dead(full0 + 8 * (c & 1), (c >> 1) & 1, a.err, dead);
                wait_or_dead(qf, ph, a.err, dead);
                for (int i = tid; i < (DK / 64) * 2 * (kChunk - rows) * 8; i += 256) {
                    const int p = i & 7, r = rows + (i >> 3) % (kChunk - rows), b = (i >> 3) / (kChunk - rows);
                    st_shared16(base + (b >> 1) * G::kTile + (b & 1 ? 8192 : (c & 1) * 16384) + r * 128 + p * 16, 0, 0, 0, 0);
                }
            }
            operand_ready(1, 288);
            wait_or_dead(full0 + 8 * (c & 1), (c >> 1) & 1, a.err, dead);
            const float* gates = reinterpret_cast<const float*>(sm + G::kG + (c & 1) * kGateFwd);
            const float eg = gates[kGEg + tok], bt = gates[kGBt + tok], ee = gates[kGEnd];
            __syncwarp();
            if (lane == 0) mbar_arrive(ge0 + 8 * (c & 1));
            uint4 vr[NH / 8];
            if (reads_k) {
                wait_or_dead(vf, ph, a.err, dead);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NH / 8; ++i) {
                    vr[i] = reinterpret_cast<const uint4*>(sm + G::kV + tok * W + vc * 2)[i];
                    if (tok >= rows) vr[i] = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(ve);
            }
            wait_or_dead(b1, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            float x[NH];
            tmem_sum<NH, ST>(tmem + G::kD1 + lanes + vc, NV, x);
            if (reads_k) {
#pragma unroll
                for (int i = 0; i < NH / 8; ++i) {
                    const uint32_t u[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[8 * i + 2 * j] = fmaf(-eg, x[8 * i + 2 * j], __uint_as_float(u[j] << 16));
                        x[8 * i + 2 * j + 1] = fmaf(-eg, x[8 * i + 2 * j + 1], __uint_as_float(u[j] & 0xffff0000u));
                    }
                }
                put_terms<W, 3>(base + G::kR, G::kRTerm, tok, vc, x);
                operand_ready(2, 160);
            }
            wait_or_dead(b2, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            float y[NH];
            tmem_sum<NH, 3>(tmem + G::kD2 + lanes + vc, NV, y);
            if (reads_k) {
#pragma unroll
                for (int j = 0; j < NH; ++j) x[j] = bt * y[j];
                put_terms<W, 3>(base + G::kR, G::kRTerm, tok, vc, x);
                operand_ready(3, 160);
                if constexpr (ST == 3) {                  // eps as three bf16 terms, operands of 64 rows
                    bool swap;
                    char* e = recE + (((slot0 + c) * sh.H + h) * tiles + tile) * (size_t)(3 * kChunk * W) + pieces_at<W, NH>(tok, vc, swap);
                    uint32_t p[NH / 2][3];
#pragma unroll
                    for (int j = 0; j < NH / 2; ++j) split_pair<3>(y[2 * j], y[2 * j + 1], p[j]);
#pragma unroll
                    for (int t = 0; t < 3; ++t) {
                        uint4 u[NH / 8];
#pragma unroll
                        for (int i = 0; i < NH / 8; ++i) u[i] = make_uint4(p[4 * i][t], p[4 * i + 1][t], p[4 * i + 2][t], p[4 * i + 3][t]);
                        stg_pieces(e + t * kChunk * W, u, swap, true);
                    }
                }
            } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (((size_t)first + c * kChunk + tok) * sh.H + h) * sh.dv + v0 + vc;
                float* e = recO + (((slot0 + c) * sh.H + h) * tiles + tile) * (size_t)(kChunk * NV) + tok * NV + vc;
#pragma unroll
                for (int j = 0; j < NH; ++j) y[j] = fmaf(eg, x[j], y[j]);
                uint4 u[NH / 8], f[NH / 4];
#pragma unroll
                for (int i = 0; i < NH / 8; ++i)
                    u[i] = make_uint4(pack_bf16(y[8 * i], y[8 * i + 1]), pack_bf16(y[8 * i + 2], y[8 * i + 3]), pack_bf16(y[8 * i + 4], y[8 * i + 5]),
                                      pack_bf16(y[8 * i + 6], y[8 * i + 7]));
                if (tok < rows) stg_pieces(o, u, false, whole);
                if constexpr (ST == 3) {                  // unrounded, for the gates' gradient
#pragma unroll
                    for (int i = 0; i < NH / 4; ++i)
                        f[i] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
                    stg_pieces(e, f, false, true);
                }
            }
            __syncwarp();
            wait_or_dead(b3, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            constexpr int kStep = SC < 16 ? SC : 16;      // columns read at a time: registers
#pragma unroll
            for (int g = 0; g < SC; g += kStep) {
                float d[kStep];
                tmem_sum<kStep, 3>(tmem + G::kD3 + (G::kMH == 2 ? wg * 3 * NV : 0) + lanes + scol + g, NV, d);
#pragma unroll
                for (int j = 0; j < kStep; ++j) S[g + j] = fmaf(ee, S[g + j], d[j]);
            }
        }
        if (a.S_T != nullptr && srow < sh.dk) {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * sh.dk + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) a.S_T[at + (size_t)j * sh.dk] = S[j];
        }
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kAlloc);
    }
}

// ---------------------------------------------------------------------------
// seq_bwd_kernel: the chunks of a sequence from its end
// ---------------------------------------------------------------------------
// With dS+ the gradient at a chunk's end (d_k x d_v, in registers like the state), x = tail (K dS+),
//   w = T^T x + Ptil^T dO,  dV = beta w,  dS = e^{g_end} dS+ + Q^T (e^g dO) - K^T (e^g dV).
// w is the gradient of beta eps: T takes That's place so that it comes without beta, which may be
// zero.  Three dependent products again: K dS+ -> T^T x -> K^T (-e^g dV); Ptil^T dO and
// Q^T (e^g dO) run behind the first.  dS+ goes to the workspace as the operand that it is in shared
// memory, dV as two bf16 terms; seq_grad_kernel takes both.
//
// The gates' gradients are dots over d_v and come from here, where w and dS are fp32:
//   dbeta_t = w_t.eps_t,   dlog_alpha_t = dlog_alpha_{t+1} + dO_t.o_t - dV_t.v_t,
// the second since <S_t, dS_t> changes from token to token by just these; its value at a chunk's
// first token is <S, dS>, S the chunk's start state.  Each CTA writes its columns' parts.
//
// Bound like the forward scan by a chunk's chain, 2.3 us with 16 columns and heads of 256: 1 x 8192, 8 heads of 256
// 288 us, 4 x 2048 (32 columns) 283 us.  <S, dS> at every fourth chunk, with sums of the steps between, took 45 us less
// of 4 x 2048 and left dlog_alpha 1.5e-6 of its size off instead of 8e-7.
template <int DK, int NV>
struct BwdGeom {
    static constexpr int kMH = DK > 128 ? 2 : 1;
    static constexpr int kW = NV * 2;
    static constexpr uint32_t kTile = 64 * 128;                   // K or Q, 64 columns of d_k
    static constexpr uint32_t kQK = 2 * kMH * kTile;              // filled up to 128 or 256 columns
    static constexpr uint32_t kO = kQK;                           // a stage: K, dO as an operand, gates
    static constexpr uint32_t kG = kO + 64 * kW;
    static constexpr uint32_t kStage = (kG + kGateBwd + 1023) & ~1023u;
    static constexpr uint32_t kBar = kG + kGateBwd;               // barriers behind the first stage's gates
    static_assert(kBar + 192 <= kStage, "gates and barriers share the end of a stage");
    static constexpr uint32_t kQ = 2 * kStage;                    // one Q
    static constexpr uint32_t kTP = kQ + kQK;
    static constexpr uint32_t kS = kTP + 3 * kOpTerm;             // three terms
    static constexpr uint32_t kSTerm = DK * kW;
    static constexpr uint32_t kR = kS + 3 * kSTerm;               // three terms of x, then of -e^g dV
    static constexpr uint32_t kRTerm = 64 * kW;
    static constexpr uint32_t kE = kR + 3 * kRTerm;               // three terms of e^g dO
    static constexpr uint32_t kSmem = kE + 3 * kRTerm + 1024;
    static constexpr int kD1 = 0, kD2 = 3 * NV, kDP = kD2 + 3 * NV, kD3 = kDP + NV, kCols = kD3 + kMH * 3 * NV;
    static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kSmem <= 227 * 1024, "tile");
};

template <int DK, int NV>
constexpr size_t bwd_smem() {
    using G = BwdGeom<DK, NV>;
    const size_t least = G::kAlloc == 512 ? 116 * 1024 : G::kAlloc == 256 ? 78 * 1024 : 58 * 1024;
    return G::kSmem > least ? G::kSmem : least;
}

// Twelve warps: eight that compute, one for the copies, one that issues products, two for the outputs and
// the gates' dots (lanes 64 .. 127 of the second product repeat dV for them).
constexpr int kBwdThreads = 384;

template <int DK, int NV>
__global__ void __launch_bounds__(kBwdThreads, 1)
    seq_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmO, SeqArgs a, const char* ops, const char* recS, const char* recE, const float* recO,
                   char* wsS, char* wsV, float* part, float* phi) {
    using G = BwdGeom<DK, NV>;
    constexpr int W = G::kW, NH = NV / 2;
    constexpr int SC = G::kMH == 2 ? NV : NH;
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    const uint32_t full0 = base + G::kBar, empty0 = full0 + 16, tpf = full0 + 32, tpe = full0 + 40, b1 = full0 + 48,
                   b2 = full0 + 56, b3 = full0 + 64, drain = full0 + 72, qf = full0 + 80, qe = full0 + 88, he0 = full0 + 96;
    uint32_t* holder = reinterpret_cast<uint32_t*>(sm + G::kBar + 128);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const SeqShape& sh = a.sh;
    {
        int b, e;
        if (seq_outside(sh, b, e)) {
            for (void* p : {a.dq, a.dk}) zero_rows<uint4>(p, (size_t)sh.Hk * sh.dk / 8, b, e, sh.total);
            zero_rows<uint4>(a.dv, (size_t)sh.H * sh.dv / 8, b, e, sh.total);
            for (float* p : {a.dla, a.dbeta}) zero_rows<float>(p, sh.H, b, e, sh.total);
        }
    }
    const int tiles = sh.dv / NV;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H;
    const int s = seq_by_length(sh, blockIdx.x / (tiles * sh.H), reinterpret_cast<int*>(sm + G::kS));
    const int hk = h / (sh.H / sh.Hk), v0 = tile * NV;
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;     // the whole CTA
    first = warp_uniform(first);
    len = warp_uniform(len);
    const int chunks = (len + kChunk - 1) / kChunk;
    const size_t slot0 = (size_t)(first / kChunk + s);

    if (tid == 0) {
        init_barriers(full0, 14, [&](uint32_t bar) { return bar >= he0 ? 2 : 1; });
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (DK % 128 != 0) {                                  // columns of d_k that no copy fills
        for (int st = 0; st < 3; ++st)
            for (uint32_t o = tid * 16; o < G::kTile; o += kBwdThreads * 16)
                st_shared16(base + (st < 2 ? st * G::kStage : G::kQ) + (DK / 64) * G::kTile + o, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 9) tmem_alloc(smem_u32(holder), G::kAlloc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(*holder);

    // eight columns of w: T^T x (three terms) and, in the columns behind, Ptil^T dO
    auto read_w = [&](int col, uint32_t lanes, float* x) {
        uint32_t u[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t) tmem_ld_n(tmem + G::kD2 + lanes + col + t * NV, u[t]);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = ((__uint_as_float(u[2][j]) + __uint_as_float(u[1][j])) + __uint_as_float(u[3][j])) + __uint_as_float(u[0][j]);
    };
    // i counts the chunks as they are taken, c = chunks - 1 - i is the chunk
    if (warp >= 10) {
        // a token's dV and its dots, NH columns at a time
        const int w4 = warp & 3, tok = 32 * (w4 & 1) + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const bool whole = (reinterpret_cast<uintptr_t>(a.dv) & 31u) == 0;      // 32-byte rows of columns
        const bool ws_whole = (reinterpret_cast<uintptr_t>(wsV) & 31u) == 0;
        if (chunks > 0) asm volatile("bar.arrive 1, 352;\n" ::: "memory");
        for (int i = 0; i < chunks; ++i) {
            const int c = chunks - 1 - i;
            const uint32_t ph = i & 1, st = (i & 1) * G::kStage;
            const int rows = min(kChunk, len - c * kChunk);
            const size_t at = ((slot0 + c) * sh.H + h) * tiles + tile;
            const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + ((size_t)first + c * kChunk + tok) * sh.ldv + (size_t)h * sh.dv + v0;
            uint4 te[3][NH / 8], to[NH / 4], tv[NH / 8];
            bool swap = false;
            auto load = [&](int vc) {                     // eps (three terms), o and v
                const char* e = recE + at * (3 * kChunk * W) + pieces_at<W, NH>(tok, vc, swap);
#pragma unroll
                for (int t = 0; t < 3; ++t) ldg_pieces(e + t * kChunk * W, te[t]);
                ldg_pieces(recO + at * (kChunk * NV) + tok * NV + vc, to);
#pragma unroll
                for (int p = 0; p < NH / 8; ++p) {
                    tv[p] = make_uint4(0, 0, 0, 0);
                    if (tok < rows) tv[p] = *reinterpret_cast<const uint4*>(vp + vc + 8 * p);
                }
            };
            load(0);
            wait_or_dead(full0 + 8 * (i & 1), (i >> 1) & 1, a.err, dead);
            const float beta = reinterpret_cast<const float*>(sm + st + G::kG)[kGBeta - kGEg + tok];
            wait_or_dead(b2, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            float all[NV];
#pragma unroll
            for (int g = 0; g < NV; g += 8) read_w(g, lanes, all + g);
            tc_fence_before();
            __syncwarp();
            // read: the next chunk's products may come
            if (i + 1 < chunks) asm volatile("bar.arrive 1, 352;\n" ::: "memory");
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int vc = half * NH;
                if (half > 0) load(vc);
                float *x = all + vc, db = 0.f, dl = 0.f;
                uint4 hi[NH / 8], lo[NH / 8];
#pragma unroll
                for (int p = 0; p < NH / 8; ++p) {
                    const int q = NH == 16 ? p ^ 1 : p;   // where the pieces changed places
                    uint4 td = *reinterpret_cast<const uint4*>(sm + st + G::kO + sw_piece<W>(tok, vc / 8 + p));
                    if (tok >= rows) td = make_uint4(0, 0, 0, 0);
                    const uint4 ea = swap ? te[0][q] : te[0][p], eb = swap ? te[1][q] : te[1][p], ec = swap ? te[2][q] : te[2][p];
                    const uint32_t *e0 = &ea.x, *e1 = &eb.x, *e2 = &ec.x, *o4 = &to[2 * p].x, *v4 = &tv[p].x, *d4 = &td.x;
                    uint32_t u[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            auto part16 = [&](uint32_t w) { return __uint_as_float(z ? w & 0xffff0000u : w << 16); };
                            float& w = x[8 * p + 2 * j + z];
                            db = fmaf(w, part16(e0[j]) + (part16(e1[j]) + part16(e2[j])), db);
                            w *= beta;
                            dl = fmaf(part16(d4[j]), __uint_as_float(o4[2 * j + z]), fmaf(-w, part16(v4[j]), dl));
                        }
                        split_pair<2>(x[8 * p + 2 * j], x[8 * p + 2 * j + 1], u[j]);
                    }
                    hi[p] = make_uint4(u[0][0], u[1][0], u[2][0], u[3][0]);
                    lo[p] = make_uint4(u[0][1], u[1][1], u[2][1], u[3][1]);
                }
                bool turn;
                char* e = wsV + at * (size_t)(2 * kChunk * W) + pieces_at<W, NH>(tok, vc, turn);
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.dv) + (((size_t)first + c * kChunk + tok) * sh.H + h) * sh.dv + v0 + vc;
                stg_pieces(e, hi, turn, ws_whole);
                stg_pieces(e + kChunk * W, lo, turn, ws_whole);
                if (tok < rows) stg_pieces(o, hi, false, whole);
                float* q = part + (at * 2 + half) * (2 * kChunk) + tok;
                q[0] = db;
                q[kChunk] = dl;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(he0 + 8 * (i & 1));               // dO and the gates may be overwritten
            __syncwarp();
        }
    } else if (warp == 8) {
        if (elect_one()) {
            int issued = 0, q_issued = 0, ops_issued = 0;
            for (int i = 0; i < chunks; ++i) {
                const int c = chunks - 1 - i;
                if (i >= 2 && !(wait_or_dead(empty0 + 8 * (i & 1), ((i >> 1) & 1) ^ 1, a.err, dead) &&
                                wait_or_dead(he0 + 8 * (i & 1), ((i >> 1) & 1) ^ 1, a.err, dead)))
                    break;
                const uint32_t st = base + (i & 1) * G::kStage, f = full0 + 8 * (i & 1);
                const char* op = ops + ((slot0 + c) * sh.H + h) * kOpRecord;
                mbar_expect_tx(f, DK * 128 + 64 * W + kGateBwd);
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) tma_3d(st + b * G::kTile, &tmK, 64 * b, hk, first + c * kChunk, f);
                tma_2d(st + G::kO, &tmO, h * sh.dv + v0, first + c * kChunk, f);
                bulk_copy_g2s(st + G::kG, op + 4 * kGEg, kGateBwd, f);
                const size_t at = ((slot0 + c) * sh.H + h) * tiles + tile;     // what the compute warps will read themselves
                bulk_prefetch_l2(recE + at * (3 * kChunk * W), 3 * kChunk * W);
                bulk_prefetch_l2(recO + at * (kChunk * NV), kChunk * NV * 4);
                bulk_prefetch_l2(recS + at * (3 * G::kSTerm), 3 * G::kSTerm);
                issued = i + 1;
                if (i >= 1 && !wait_or_dead(qe, (i - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(qf, DK * 128);
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) tma_3d(base + G::kQ + b * G::kTile, &tmQ, 64 * b, hk, first + c * kChunk, qf);
                q_issued = i + 1;
                if (i >= 1 && !wait_or_dead(tpe, (i - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(tpf, 3 * kOpTerm);
                bulk_copy_g2s(base + G::kTP, op + kOpBack, 3 * kOpTerm, tpf);
                ops_issued = i + 1;
            }
            // copies in flight land before the CTA ends, though a warp that waits for them may give up
            for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) mbar_wait(full0 + 8 * (i & 1), (i >> 1) & 1, a.err);
            if (q_issued > 0) mbar_wait(qf, (q_issued - 1) & 1, a.err);
            if (ops_issued > 0) mbar_wait(tpf, (ops_issued - 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 9) {
        const uint64_t dS = mn_desc<W>(base + G::kS, G::kSTerm), dR = mn_desc<W>(base + G::kR, G::kRTerm),
                       dE = mn_desc<W>(base + G::kE, G::kRTerm);
        // [T; Ptil]^T: the index of M runs along the 64 columns of a row, and its second 64 are the
        // first again, so that lanes 64 .. 127 of the result repeat lanes 0 .. 63
        const uint64_t dTP = mn_desc<128>(base + G::kTP, 0);
        const bool leader = elect_one();
        for (int i = 0; i < chunks; ++i) {
            const uint32_t ph = i & 1, st = base + (i & 1) * G::kStage;
            wait_or_dead(full0 + 8 * (i & 1), (i >> 1) & 1, a.err, dead);
            wait_or_dead(tpf, ph, a.err, dead);
            wait_or_dead(qf, ph, a.err, dead);
            __syncwarp();
            named_sync(1, 352);
            tc_fence_after();
            const uint64_t dK = mn_desc<128>(st, G::kTile), dQ = mn_desc<128>(base + G::kQ, G::kTile);
            if (leader) {
                // 128 rows: K's 64 and whatever lies behind, lanes that nothing reads
                const uint64_t dKr = k_desc<128>(st), dO = mn_desc<W>(st + G::kO, 0);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_bf16(tmem + G::kD1, dKr + (((k / 4) * G::kTile + 32 * (k % 4)) >> 4), dS + (k * 16 * W >> 4),
                             idesc_bf16(128, 3 * NV) | kBMn, k != 0);
                mma_commit(b1);
                bulk_s2g(wsS + (((slot0 + chunks - 1 - i) * sh.H + h) * tiles + tile) * (2 * G::kSTerm), base + G::kS, 2 * G::kSTerm);
#pragma unroll
                for (int k = 0; k < 12; ++k)
                    mma_bf16(tmem + G::kDP, dTP + (k / 4) * (kOpTerm >> 4) + (8192 + (k % 4) * 2048 >> 4), dO + ((k % 4) * 16 * W >> 4),
                             idesc_bf16(128, NV) | kAMn | kBMn, k != 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int m = 0; m < G::kMH; ++m)
                        mma_bf16(tmem + G::kD3 + m * 3 * NV, dQ + ((2 * m * G::kTile + k * 2048) >> 4), dE + (k * 16 * W >> 4),
                                 idesc_bf16(128, 3 * NV) | kAMn | kBMn, k != 0);
                mma_commit(qe);
            }
            __syncwarp();
            named_sync(2, 160);
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int t = 0; t < 3; ++t)               // term t with the first 3 - t of x
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + G::kD2, dTP + t * (kOpTerm >> 4) + (k * 2048 >> 4), dR + (k * 16 * W >> 4),
                                 idesc_bf16(128, (3 - t) * NV) | kAMn | kBMn, t + k != 0);
                mma_commit(b2);
                mma_commit(tpe);
                bulk_read_done();                         // dS's image may be written again once b3 is through
            }
            __syncwarp();
            named_sync(3, 160);
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int m = 0; m < G::kMH; ++m)
                        mma_bf16(tmem + G::kD3 + m * 3 * NV, dK + ((2 * m * G::kTile + k * 2048) >> 4), dR + (k * 16 * W >> 4),
                                 idesc_bf16(128, 3 * NV) | kAMn | kBMn, 1);
                mma_commit(b3);
                mma_commit(empty0 + 8 * (i & 1));
            }
            __syncwarp();
        }
        if (leader) {
            bulk_all_done();
            mma_commit(drain);                            // products in flight end before their TMEM is freed, as above
            mbar_wait(drain, 0, a.err);
        }
        __syncwarp();
    } else {
        const int wg = warp >> 2, w4 = warp & 3;
        const bool reads_k = w4 < 2;                      // x and -e^g dV of a token, else e^g dO
        const int tok = 32 * (w4 & 1) + lane, vc = wg * NH;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const int srow = (G::kMH == 2 ? 128 * wg : 0) + 32 * w4 + lane, scol = G::kMH == 2 ? 0 : wg * NH;
        const bool owns = srow < DK;
        float S[SC];
        {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * sh.dk + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) S[j] = srow < sh.dk && a.dS_T != nullptr ? a.dS_T[at + (size_t)j * sh.dk] : 0.f;
        }
        // This CTA's part of <S, dS> at the start of chunk c: N columns from g on of the thread's row, three
        // terms, in S's image, swizzled as it was in shared memory.
        constexpr int N = SC < 16 ? SC : 16;
        auto load_state = [&](int c, int g, uint4 (&u)[3][N / 8]) {
            bool swap;
            const char* p = recS + (((slot0 + c) * sh.H + h) * tiles + tile) * (3 * G::kSTerm) + pieces_at<W, N>(srow, scol + g, swap);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                if (owns) ldg_pieces(p + t * G::kSTerm, u[t]);
                else
#pragma unroll
                    for (int k = 0; k < N / 8; ++k) u[t][k] = make_uint4(0, 0, 0, 0);
            }
        };
        auto dot_state = [&](int g, const uint4 (&u)[3][N / 8]) {
            bool swap;
            pieces_at<W, N>(srow, scol + g, swap);
            float d = 0.f;
#pragma unroll
            for (int j = 0; j < N / 8; ++j) {
                const int z = N == 16 ? j ^ 1 : j;
                const uint4 a0 = swap ? u[0][z] : u[0][j], a1 = swap ? u[1][z] : u[1][j], a2 = swap ? u[2][z] : u[2][j];
                const uint32_t uu[4] = {a0.x, a0.y, a0.z, a0.w}, mm[4] = {a1.x, a1.y, a1.z, a1.w}, ll[4] = {a2.x, a2.y, a2.z, a2.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d = fmaf(__uint_as_float(uu[e] << 16) + (__uint_as_float(mm[e] << 16) + __uint_as_float(ll[e] << 16)), S[g + 8 * j + 2 * e], d);
                    d = fmaf(__uint_as_float(uu[e] & 0xffff0000u) + (__uint_as_float(mm[e] & 0xffff0000u) + __uint_as_float(ll[e] & 0xffff0000u)),
                             S[g + 8 * j + 2 * e + 1], d);
                }
            }
            return d;
        };
        auto store_phi = [&](int c, float d) {
            d = warp_sum(d);
            if (lane == 0) phi[(((slot0 + c) * sh.H + h) * tiles + tile) * 8 + warp] = d;
        };
        auto state_dot = [&](int c) {
            float d = 0.f;
#pragma unroll
            for (int g = 0; g < SC; g += N) {
                uint4 u[3][N / 8];
                load_state(c, g, u);
                d += dot_state(g, u);
            }
            store_phi(c, d);
        };
        for (int i = 0; i < chunks; ++i) {
            const int c = chunks - 1 - i;
            const uint32_t ph = i & 1, st = (i & 1) * G::kStage;
            const int rows = min(kChunk, len - c * kChunk);
            if (owns) put_terms<W, 3>(base + G::kS, G::kSTerm, srow, scol, S);
            wait_or_dead(full0 + 8 * (i & 1), (i >> 1) & 1, a.err, dead);
            __syncwarp();
            if (rows < kChunk) {
                // the copies brought tokens of what lies behind: rows of zero instead
                wait_or_dead(qf, ph, a.err, dead);
                for (int j = tid; j < (DK / 64) * 2 * (kChunk - rows) * 8; j += 256) {
                    const int p = j & 7, r = rows + (j >> 3) % (kChunk - rows), b = (j >> 3) / (kChunk - rows);
                    st_shared16(base + (b & 1 ? G::kQ : st) + (b >> 1) * G::kTile + r * 128 + p * 16, 0, 0, 0, 0);
                }
            }
            const float* gates = reinterpret_cast<const float*>(sm + st + G::kG);
            const float eg = gates[tok], tail = gates[kGTail - kGEg + tok], beta = gates[kGBeta - kGEg + tok], ee = gates[kGEnd - kGEg];
            float x[NH];
            if (!reads_k) {
#pragma unroll
                for (int p = 0; p < NH / 8; ++p) {
                    uint4* at = reinterpret_cast<uint4*>(sm + st + G::kO + sw_piece<W>(tok, vc / 8 + p));
                    uint4 u = *at;
                    if (tok >= rows) *at = u = make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[8 * p + 2 * j] = eg * __uint_as_float(w[j] << 16);
                        x[8 * p + 2 * j + 1] = eg * __uint_as_float(w[j] & 0xffff0000u);
                    }
                }
                put_terms<W, 3>(base + G::kE, G::kRTerm, tok, vc, x);
            }
            operand_ready(1, 352);
            // All load the state that belongs to dS now; the warps that read K form its dot behind the third
            // product's start, the others at once.
            uint4 pre[SC / N][3][N / 8];
            if (i > 0)
#pragma unroll
                for (int g = 0; g < SC / N; ++g) load_state(c + 1, g * N, pre[g]);
            if (i > 0 && !reads_k) {
                float d = 0.f;
#pragma unroll
                for (int g = 0; g < SC / N; ++g) d += dot_state(g * N, pre[g]);
                store_phi(c + 1, d);
            }
            if (reads_k) {
                wait_or_dead(b1, ph, a.err, dead);
                __syncwarp();
                tc_fence_after();
                tmem_sum<NH, 3>(tmem + G::kD1 + lanes + vc, NV, x);
#pragma unroll
                for (int j = 0; j < NH; ++j) x[j] *= tail;
                put_terms<W, 3>(base + G::kR, G::kRTerm, tok, vc, x);
                operand_ready(2, 160);
                wait_or_dead(b2, ph, a.err, dead);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < NH; g += 8) read_w(vc + g, lanes, x + g);
#pragma unroll
                for (int j = 0; j < NH; ++j) x[j] *= -eg * beta;
                put_terms<W, 3>(base + G::kR, G::kRTerm, tok, vc, x);
                operand_ready(3, 160);
                if (i > 0) {
                    float d = 0.f;
#pragma unroll
                    for (int g = 0; g < SC / N; ++g) d += dot_state(g * N, pre[g]);
                    store_phi(c + 1, d);
                }
            }
            __syncwarp();
            wait_or_dead(b3, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            constexpr int kStep = SC < 16 ? SC : 16;      // columns read at a time: registers
#pragma unroll
            for (int g = 0; g < SC; g += kStep) {
                float d[kStep];
                tmem_sum<kStep, 3>(tmem + G::kD3 + (G::kMH == 2 ? wg * 3 * NV : 0) + lanes + scol + g, NV, d);
#pragma unroll
                for (int j = 0; j < kStep; ++j) S[g + j] = fmaf(ee, S[g + j], d[j]);
            }
        }
        if (chunks > 0) state_dot(0);
        if (a.dS0 != nullptr && srow < sh.dk) {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * sh.dk + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) a.dS0[at + (size_t)j * sh.dk] = S[j];
        }
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kAlloc);
    }
}

// ---------------------------------------------------------------------------
// seq_grad_kernel: dq and dk of one (chunk, head) after another
// ---------------------------------------------------------------------------
// With S the chunk's start state and dS+ the gradient at its end (d_k x d_v), both as the scans
// left them, E = dO eps^T, F = dV eps^T, MP = lower G E beta, ME = strictly lower G F beta:
//   dq      = e^g dO S^T + MP K                     lanes 0..63 of one accumulator, rows dO and MP,
//   k_read  = -e^g dV S^T - ME K                    lanes 64..127, rows dV and -ME
//   k_write = bt eps dS+^T + MP^T Q - ME^T K        lanes 64..127 of another, whose others nobody reads
// and dk their sum.  The rows' factors e^g and bt are applied in place between the products over
// d_v and those over the chunk's tokens: the operands stay what the scans stored, dO exact.
// The gates' gradients are added up here from the parts that the backward scan left.
//
// Bound by its reads, 4 bytes for each element of S and dS+ of every chunk, and by what an item does after them.
// 4 x 1024 tokens, 8 heads of 256: 106 us, 405 MB read (3.8 TB/s); 1 x 8192 174 us, 4 x 2048 182 us; 16 x 1024, heads
// of 128: 161 us.  One CTA per SM (two for d_k up to 128) goes through the chunks.  Slots of shared memory take NV
// columns of d_v at a time: with 32 columns two of 28 KB (d_k 64), one of 36 (128), two of 44 or 52 (192, 256), with 16
// four of 14, two of 18, four of 22 or 26.  The single slot is no ring: there a copy waits for the products before it,
// and the SM's other CTA works meanwhile.
template <int DK, int NV>
struct GradGeom {
    static constexpr int kW = NV * 2;
    static constexpr uint32_t kTile = 128 * 128;                  // [Q; K], 64 columns of d_k
    static constexpr uint32_t kBlk = 64 * kW;                     // 64 rows of an operand over d_v
    static constexpr uint32_t kM = (DK / 64) * kTile;             // [MP; -ME], two terms
    static constexpr uint32_t kSlot0 = kM + 2 * 16384;
    // blocks of a slot: dO, dV hi, zero, dV lo, -, or what was there, eps hi, zero, what was there, eps lo; then S or
    // dS+, or eps hi, lo
    static constexpr uint32_t kImg = 5 * kBlk;
    static constexpr uint32_t kSlot = kImg + 2 * DK * kW;
    // two CTAs on an SM where d_k leaves room for their TMEM: one streams while the other scales and writes
    static constexpr int kCtas = DK <= 128 ? 2 : 1;
    static constexpr int kSlots = (NV == 16 ? 4 : 2) / (DK == 128 ? 2 : 1);
    static constexpr uint32_t kGates = kSlot0 + kSlots * kSlot;
    static constexpr uint32_t kMisc = kGates + kOpGates;          // four floats
    static constexpr uint32_t kBar = kMisc + 16;
    static constexpr uint32_t kUsed = kBar + 256 + 1024;
    static constexpr uint32_t kSmem = kCtas == 2 || kUsed > 116 * 1024 ? kUsed : 116 * 1024;      // no more CTAs than TMEM
    static constexpr int kDa = 0, kDw = DK, kE = 0;       // E and F are read before the others begin
    static constexpr int kAlloc = 2 * DK <= 128 ? 128 : 2 * DK <= 256 ? 256 : 512;
    static_assert(kSmem <= (kCtas == 2 ? 113 : 227) * 1024 && (kCtas == 1 || 3 * kSmem > 227 * 1024), "CTAs");
    static_assert(kSmem <= 227 * 1024 && kSlot % 1024 == 0, "slots");
};

template <int DK, int NV>
__global__ void __launch_bounds__(kFwdThreads, GradGeom<DK, NV>::kCtas)
    seq_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmO, SeqArgs a, const char* ops, const char* recS, const char* recE,
                    const char* wsS, const char* wsV, const float* part, const float* phi, float* dqf, float* dkf) {
    using G = GradGeom<DK, NV>;
    constexpr int W = G::kW, HC = DK / 2;                 // HC: columns of d_k of a thread
    constexpr int CS = G::kCtas == 2 ? 16 : 32;           // columns at a time
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    const uint32_t kqf = base + G::kBar, kqe = kqf + 8, ef = kqf + 16, p2 = kqf + 24, fin = kqf + 32,
                   drain = kqf + 40, p3 = kqf + 48, full0 = kqf + 56, empty0 = full0 + 8 * G::kSlots;
    uint32_t* holder = reinterpret_cast<uint32_t*>(sm + G::kBar + 128);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / NV, rep = sh.H / sh.Hk;
    const int tid = threadIdx.x, warp = warp_uniform(tid >> 5), lane = tid & 31;
    const int items = seq_slots(sh.nseq, sh.total) * sh.Hk;

    if (tid == 0) {
        init_barriers(kqf, 7 + 2 * G::kSlots, [&](uint32_t bar) { return bar == kqe ? 8 : 1; });
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    for (int sl = 0; sl < G::kSlots; ++sl)
        for (uint32_t o = tid * 16; o < G::kBlk; o += kFwdThreads * 16)
            st_shared16(base + G::kSlot0 + sl * G::kSlot + 2 * G::kBlk + o, 0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 9) tmem_alloc(smem_u32(holder), G::kAlloc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(*holder);
    griddep_wait();

    if (warp == 8) {
        if (elect_one()) {
            int n = 0, it = 0, kq_issued = 0;
            bool ok = true;
            for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
                int s, first, rows;
                if (!slot_chunk(sh, item / sh.Hk, s, first, rows, a.err)) continue;
                const int hk = item % sh.Hk;
                for (int r = 0; r < rep && ok; ++r, ++n) {
                    const int h = hk * rep + r;
                    const size_t sh_at = (size_t)(item / sh.Hk) * sh.H + h;
                    // Q, K and the gates behind the first slots: their place is free only when the item before has ended
                    const int kq_at = min(G::kSlots, 3 * tiles - 1);
                    for (int j = 0; j < 3 * tiles; ++j, ++it) {
                        if (j == kq_at) {
                            if (n >= 1 && !(ok = wait_or_dead(kqe, (n - 1) & 1, a.err, dead))) break;
                            mbar_expect_tx(kqf, 2 * DK * 128 + kOpGates);
                            ++kq_issued;
#pragma unroll
                            for (int b = 0; b < DK / 64; ++b) {
                                tma_3d(base + b * G::kTile, &tmQ, 64 * b, hk, first, kqf);
                                tma_3d(base + b * G::kTile + 8192, &tmK, 64 * b, hk, first, kqf);
                            }
                            bulk_copy_g2s(base + G::kGates, ops + sh_at * kOpRecord, kOpGates, kqf);
                        }
                        const uint32_t sl = base + G::kSlot0 + (it % G::kSlots) * G::kSlot, f = full0 + 8 * (it % G::kSlots);
                        if (it >= G::kSlots && !(ok = wait_or_dead(empty0 + 8 * (it % G::kSlots), ((it / G::kSlots) & 1) ^ 1, a.err, dead))) break;
                        const int v = j % tiles, v0 = v * NV;
                        const char *e = recE + (sh_at * tiles + v) * (3 * G::kBlk), *w = wsV + (sh_at * tiles + v) * (2 * G::kBlk);
                        if (j < tiles || j >= 2 * tiles) {
                            mbar_expect_tx(f, 3 * G::kBlk + (j < tiles ? 2 * G::kBlk : 2 * DK * W));
                            tma_2d(sl, &tmO, h * sh.dv + v0, first, f);
                            bulk_copy_g2s(sl + G::kBlk, w, G::kBlk, f);
                            bulk_copy_g2s(sl + 3 * G::kBlk, w + G::kBlk, G::kBlk, f);
                            if (j < tiles) {
                                bulk_copy_g2s(sl + G::kImg, e, 2 * G::kBlk, f);
                            } else {
                                bulk_copy_g2s(sl + G::kImg, recS + (sh_at * tiles + v) * (3 * DK * W), 2 * DK * W, f);
                            }
                        } else {
                            mbar_expect_tx(f, 2 * G::kBlk + 2 * DK * W);
                            bulk_copy_g2s(sl + G::kBlk, e, G::kBlk, f);
                            bulk_copy_g2s(sl + 4 * G::kBlk, e + G::kBlk, G::kBlk, f);
                            bulk_copy_g2s(sl + G::kImg, wsS + (sh_at * tiles + v) * (2 * DK * W), 2 * DK * W, f);
                        }
                    }
                }
            }
            // copies in flight land before the CTA ends, though a warp that waits for them may give up
            if (kq_issued > 0) mbar_wait(kqf, (kq_issued - 1) & 1, a.err);
            for (int j = it > G::kSlots ? it - G::kSlots : 0; j < it; ++j)
                mbar_wait(full0 + 8 * (j % G::kSlots), (j / G::kSlots) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == 9) {
        const bool leader = elect_one();
        const uint64_t dM = k_desc<128>(base + G::kM), dMt = mn_desc<128>(base + G::kM, 0),
                       dQKt = mn_desc<128>(base, G::kTile);
        int n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int s, first, rows;
            if (!slot_chunk(sh, item / sh.Hk, s, first, rows, a.err)) continue;
            for (int r = 0; r < rep; ++r, ++n) {
                for (int j = 0; j < tiles; ++j, ++it) {
                    const uint32_t sl = base + G::kSlot0 + (it % G::kSlots) * G::kSlot;
                    wait_or_dead(full0 + 8 * (it % G::kSlots), (it / G::kSlots) & 1, a.err, dead);
                    __syncwarp();
                    if (leader) {
                        const uint64_t dA = k_desc<W>(sl), dB = k_desc<W>(sl + G::kImg);
#pragma unroll
                        for (int k = 0; k < NV / 16; ++k) {
                            mma_bf16(tmem + G::kE, dA + 2 * k, dB + 2 * k, idesc_bf16(128, 128), j + k != 0);
                            mma_bf16(tmem + G::kE, dA + (2 * G::kBlk >> 4) + 2 * k, dB + 2 * k, idesc_bf16(128, 64), 1);
                        }
                        mma_commit(empty0 + 8 * (it % G::kSlots));
                    }
                    __syncwarp();
                }
                if (leader) mma_commit(ef);
                __syncwarp();
                if constexpr (DK < 128) named_sync(1, 288);                       // E and F are read
                tc_fence_after();
                for (int j = 0; j < 2 * tiles; ++j, ++it) {
                    const int second = j < tiles;         // k_write's product over d_v first: its rows are scaled meanwhile
                    if (DK >= 128 && j == tiles) {
                        named_sync(1, 288);
                        tc_fence_after();
                    }
                    const uint32_t sl = base + G::kSlot0 + (it % G::kSlots) * G::kSlot, d = tmem + (second ? G::kDw : G::kDa);
                    wait_or_dead(full0 + 8 * (it % G::kSlots), (it / G::kSlots) & 1, a.err, dead);
                    __syncwarp();
                    if (leader) {
                        const uint64_t dA = k_desc<W>(sl), dB = k_desc<W>(sl + G::kImg),
                                       dA2 = dA + ((second ? 3 : 2) * G::kBlk >> 4);
#pragma unroll
                        for (int k = 0; k < NV / 16; ++k) {
                            mma_bf16(d, dA + 2 * k, dB + 2 * k, idesc_bf16(128, DK), (second ? j : j - tiles) + k != 0);
                            mma_bf16(d, dA + 2 * k, dB + (DK * W >> 4) + 2 * k, idesc_bf16(128, DK), 1);
                            mma_bf16(d, dA2 + 2 * k, dB + 2 * k, idesc_bf16(128, DK), 1);
                        }
                        mma_commit(empty0 + 8 * (it % G::kSlots));
                        if (j + 1 == tiles) mma_commit(p2);
                    }
                    __syncwarp();
                }
                if (leader) mma_commit(p3);
                __syncwarp();
                wait_or_dead(kqf, n & 1, a.err, dead);
                __syncwarp();
                named_sync(2, 288);                       // k_write's rows scaled, [MP; -ME] written
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)          // [MP; -ME]^T [Q; K]
                        mma_bf16(tmem + G::kDw, dMt + (k / 8) * 1024 + ((k % 8) * 2048 >> 4), dQKt + ((k % 8) * 2048 >> 4),
                                 idesc_bf16(128, DK) | kAMn | kBMn, 1);
                }
                __syncwarp();
                named_sync(5, 288);                       // the others' rows scaled
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)           // [MP; -ME] K
                        mma_bf16(tmem + G::kDa, dM + (k / 4) * 1024 + 2 * (k % 4), dQKt + (8192 + (k % 4) * 2048 >> 4),
                                 idesc_bf16(128, DK) | kBMn, 1);
                    mma_commit(fin);
                }
                __syncwarp();
                named_sync(3, 288);                       // results read
                tc_fence_after();
            }
        }
        if (leader && *dead) {                            // products in flight end before their TMEM is freed
            mma_commit(drain);
            mbar_wait(drain, 0, a.err);
        }
        __syncwarp();
    } else {
        const int wg = warp >> 2, w4 = warp & 3, L = 32 * w4 + lane, t = L & 63;
        const bool is_k = w4 >= 2;                        // this thread's row: of dV, ME, dk, else of dO, MP, dq
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const float* gates = reinterpret_cast<const float*>(sm + G::kGates);
        float* ys = reinterpret_cast<float*>(sm + G::kMisc);
        int n = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int s, first, rows;
            if (!slot_chunk(sh, item / sh.Hk, s, first, rows, a.err)) continue;
            const bool more = seq_end(sh, s) - first > kChunk;
            const int hk = item % sh.Hk;
            for (int r = 0; r < rep; ++r, ++n) {
                const int h = hk * rep + r;
                const size_t sh_at = (size_t)(item / sh.Hk) * sh.H + h;
                if (warp == 7) {
                    // <S, dS> at this chunk's first token and at the next one's
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float* p = phi + (sh_at + (size_t)i * sh.H) * tiles * 8;
                        float ph = 0.f, pl = 0.f;
                        if (i == 0 || more)
                            for (int j = lane; j < 8 * tiles; j += 32) add2(ph, pl, p[j], 0.f);
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) {
                            const float qh = __shfl_xor_sync(0xffffffffu, ph, o), ql = __shfl_xor_sync(0xffffffffu, pl, o);
                            add2(ph, pl, qh, ql);
                        }
                        if (lane == 0) {
                            ys[2 * i] = ph;
                            ys[2 * i + 1] = pl;
                        }
                    }
                }
                named_sync(4, 256);
                if (warp == 0) {
                    // dbeta; dlog_alpha from the nearer end of the chunk: the sums' errors grow with their length
                    float yh[2], yl[2], zh[2], zl[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = lane + 32 * i;
                        const float* q = part + sh_at * tiles * (4 * kChunk) + t;
                        float db = 0.f;
                        yh[i] = yl[i] = 0.f;
#pragma unroll 8
                        for (int j = 0; j < 2 * tiles; ++j) {
                            db += q[j * 2 * kChunk];
                            add2(yh[i], yl[i], q[j * 2 * kChunk + kChunk], 0.f);
                        }
                        if (t < rows) a.dbeta[((size_t)first + t) * sh.H + h] = db;
                        zh[i] = yh[i];                    // sums up to and with this token, of each half
                        zl[i] = yl[i];
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const float uh = __shfl_up_sync(0xffffffffu, zh[i], o), ul = __shfl_up_sync(0xffffffffu, zl[i], o);
                            if (lane >= o) add2(zh[i], zl[i], uh, ul);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // - (the sum before this token) from the start, + the sum from it on from the end
                        const bool end = i == 1 && more;
                        float bh = ys[end ? 2 : 0], bl = ys[end ? 3 : 1];
                        add2(bh, bl, yh[i], yl[i]);
                        add2(bh, bl, -zh[i], -zl[i]);
                        const float th = __shfl_sync(0xffffffffu, zh[i], 31), tl = __shfl_sync(0xffffffffu, zl[i], 31);
                        if (end) add2(bh, bl, th, tl);
                        if (i == 1 && !more) add2(bh, bl, -__shfl_sync(0xffffffffu, zh[0], 31), -__shfl_sync(0xffffffffu, zl[0], 31));
                        if (lane + 32 * i < rows) a.dla[((size_t)first + lane + 32 * i) * sh.H + h] = bh + bl;
                    }
                }
                wait_or_dead(kqf, n & 1, a.err, dead);
                wait_or_dead(ef, n & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                const float eg = gates[kGEg + t], bt = gates[kGBt + t];
                {
                    float m[32];
#pragma unroll
                    for (int g = 0; g < 32; g += CS) {
                        uint32_t e0[CS], e1[CS];
                        tmem_ld_n(tmem + G::kE + lanes + 32 * wg + g, e0);
                        tmem_ld_n(tmem + G::kE + lanes + 64 + 32 * wg + g, e1);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < CS; ++j) m[g + j] = __uint_as_float(e0[j]) + __uint_as_float(e1[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    asm volatile("bar.arrive 1, 288;\n" ::: "memory");
                    const float gh = gates[kGHi + t], gl = gates[kGLo + t];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int c = 32 * wg + j;
                        m[j] = t < rows && (is_k ? c < t : c <= t)
                                   ? (is_k ? -m[j] : m[j]) * expf((gh - gates[kGHi + c]) + (gl - gates[kGLo + c])) * gates[kGBeta + c]
                                   : 0.f;
                    }
                    put_terms<128, 2>(base + G::kM, 16384, L, 32 * wg, m);
                }
                if (rows < kChunk)                        // tokens of what lies behind: rows of zero instead
                    for (int j = tid; j < (DK / 64) * 2 * (kChunk - rows) * 8; j += 256) {
                        const int p = j & 7, q = rows + (j >> 3) % (kChunk - rows), b = (j >> 3) / (kChunk - rows);
                        st_shared16(base + b * 8192 + q * 128 + p * 16, 0, 0, 0, 0);
                    }
                auto scale = [&](uint32_t col, float f) {
#pragma unroll 1
                    for (int g = 0; g < HC / CS; ++g) {
                        uint32_t x[CS];
                        tmem_ld_n(tmem + col + lanes + HC * wg + CS * g, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < CS; ++j) x[j] = __float_as_uint(f * __uint_as_float(x[j]));
                        tmem_st_n(tmem + col + lanes + HC * wg + CS * g, x);
                    }
                    tmem_wait_st();
                };
                wait_or_dead(p2, n & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                if (is_k) scale(G::kDw, bt);
                operand_ready(2, 288);
                wait_or_dead(p3, n & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                scale(G::kDa, is_k ? -eg : eg);
                operand_ready(5, 288);
                wait_or_dead(fin, n & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                const size_t at = ((size_t)(first + t) * sh.Hk + hk) * sh.dk;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_k ? a.dk : a.dq) + at;
                float* acc = (is_k ? dkf : dqf) + at;
#pragma unroll 1
                for (int g = 0; g < HC / CS; ++g) {
                    const int c0 = HC * wg + CS * g;
                    uint32_t x[CS], y[CS];
                    tmem_ld_n(tmem + G::kDa + lanes + c0, x);
                    if (is_k) tmem_ld_n(tmem + G::kDw + lanes + c0, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int p = 0; p < CS / 8; ++p) {
                        const int c = c0 + 8 * p;
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(x[8 * p + e]) + (is_k ? __uint_as_float(y[8 * p + e]) : 0.f);
                        if (t < rows && c < sh.dk) {
                            if (rep > 1) {                // the group's heads in their order
                                float4* f = reinterpret_cast<float4*>(acc + c);
                                if (r > 0) {
                                    const float4 f0 = f[0], f1 = f[1];
                                    o[0] += f0.x; o[1] += f0.y; o[2] += f0.z; o[3] += f0.w;
                                    o[4] += f1.x; o[5] += f1.y; o[6] += f1.z; o[7] += f1.w;
                                }
                                if (r + 1 < rep) {
                                    f[0] = make_float4(o[0], o[1], o[2], o[3]);
                                    f[1] = make_float4(o[4], o[5], o[6], o[7]);
                                }
                            }
                            if (r + 1 == rep)
                                *reinterpret_cast<uint4*>(out + c) = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                                                pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(kqe);          // Q, K, the gates and ys may be overwritten
                __syncwarp();
                asm volatile("bar.arrive 3, 288;\n" ::: "memory");
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, G::kAlloc);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// Rows of tokens, 64 a box, of `cols` columns; swizzled by 128, 64 or 32 bytes, or (0) as they are.
bool token_map(CUtensorMap* m, const void* p, long long total, int width, long long ld, int cols, int swizzle) {
    const auto enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)total}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)kChunk}, estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
               : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
               : swizzle == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                               : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of tokens of one q/k head, 64 a box, in boxes of 64 columns: those behind d_k come as zeros, so that
// a d_k between the kernels' widths is one whose last columns are zero.
bool head_map(CUtensorMap* m, const void* p, const SeqShape& sh, long long ld) {
    const auto enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)sh.dk, (cuuint64_t)sh.Hk, (cuuint64_t)sh.total},
                     strides[2] = {(cuuint64_t)sh.dk * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kChunk}, estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool qk_maps(const SeqArgs& a, CUtensorMap* q, CUtensorMap* k) {
    return head_map(q, a.q, a.sh, a.sh.ldq) && head_map(k, a.k, a.sh, a.sh.ldk);
}

template <int DK, bool REC>
cudaError_t prep_go(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, char* ops, cudaStream_t st) {
    static bool done[64];
    constexpr size_t smem = PrepGeom<DK, REC>::kSmem;
    cudaError_t e = ensure_smem(seq_prep_kernel<DK, REC>, smem, done);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)seq_slots(a.sh.nseq, a.sh.total) * a.sh.H);
    return launch_kernel(seq_prep_kernel<DK, REC>, dim3(grid), dim3(kPrepThreads), smem, st, false, q, k, a, ops);
}

template <int DK, int NV, int ST>
cudaError_t fwd_go(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, cudaStream_t st) {
    static bool done[64];
    cudaError_t e = ensure_smem(seq_fwd_kernel<DK, NV, ST>, fwd_smem<DK, NV, ST>(), done);
    if (e != cudaSuccess) return e;
    CUtensorMap v;
    if (!token_map(&v, a.v, a.sh.total, a.sh.H * a.sh.dv, a.sh.ldv, NV, 0)) return cudaErrorInvalidValue;
    const SeqLayout L = seq_layout(a.sh, GDN_DTYPE_BF16);
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / NV));
    return launch_kernel(seq_fwd_kernel<DK, NV, ST>, dim3(grid), dim3(kFwdThreads), fwd_smem<DK, NV, ST>(), st, true, q, k, v, a,
                         (const char*)(ST == 3 ? a.rec + L.rec_op : a.ws + L.ws_op), ST == 3 ? kOpRecord : kOpBytes,
                         ST == 3 ? a.rec + L.rec_S : nullptr, ST == 3 ? a.rec + L.rec_eps : nullptr,
                         ST == 3 ? reinterpret_cast<float*>(a.rec + L.rec_o) : nullptr);
}

template <int DK>
cudaError_t forward_dk(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, GDN_DTYPE_BF16);
    const cudaError_t e = a.rec != nullptr ? prep_go<DK, true>(q, k, a, a.rec + L.rec_op, st)
                                           : prep_go<DK, false>(q, k, a, a.ws + L.ws_op, st);
    if (e != cudaSuccess) return e;
    if (a.rec != nullptr) return seq_tc_cols(a.sh) == 32 ? fwd_go<DK, 32, 3>(q, k, a, st) : fwd_go<DK, 16, 3>(q, k, a, st);
    // without a record two CTAs of 16 columns fit an SM where d_k is no more than 128, and what one waits the other
    // works.  Prep and scan with 16 and with 32 columns, us: 8 heads of 128, 16 x 1024 175 and 188, 64 x 256 192 and
    // 204; 16 heads of 128, 32 x 1024 594 and 642; 8 heads of 64, 16 x 1024 115 and 121, 64 x 1024 397 and 414; d_k 64 and
    // d_v 128, 16 x 1024 162 and 176; d_k 128 and d_v 256, 8 x 2048 268 and 297
    if constexpr (DK <= 128)
        return fwd_go<DK, 16, 2>(q, k, a, st);
    else
        return seq_tc_cols(a.sh) == 32 ? fwd_go<DK, 32, 2>(q, k, a, st) : fwd_go<DK, 16, 2>(q, k, a, st);
}

template <int DK, int NV>
cudaError_t bwd_go(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    static bool done_scan[64], done_grad[64];
    cudaError_t e = ensure_smem(seq_bwd_kernel<DK, NV>, bwd_smem<DK, NV>(), done_scan);
    if (e == cudaSuccess) e = ensure_smem(seq_grad_kernel<DK, NV>, GradGeom<DK, NV>::kSmem, done_grad);
    if (e != cudaSuccess) return e;
    const SeqShape& sh = a.sh;
    CUtensorMap o;
    if (!token_map(&o, a.dout, sh.total, sh.H * sh.dv, sh.H * sh.dv, NV, 2 * NV)) return cudaErrorInvalidValue;
    const char* ops = a.rec + L.rec_op;
    float *part = reinterpret_cast<float*>(a.ws + L.ws_part), *phi = reinterpret_cast<float*>(a.ws + L.ws_phi);
    e = launch_kernel(seq_bwd_kernel<DK, NV>, dim3((unsigned)((size_t)sh.nseq * sh.H * (sh.dv / NV))), dim3(kBwdThreads),
                      bwd_smem<DK, NV>(), st, false, q, k, o, a, ops, (const char*)(a.rec + L.rec_S), (const char*)(a.rec + L.rec_eps),
                      (const float*)(a.rec + L.rec_o), a.ws + L.ws_dS, a.ws + L.ws_dV, part, phi);
    if (e != cudaSuccess) return e;
    const long long items = (long long)seq_slots(sh.nseq, sh.total) * sh.Hk, ctas = GradGeom<DK, NV>::kCtas * kSMs;
    return launch_kernel(seq_grad_kernel<DK, NV>, dim3((unsigned)(items < ctas ? items : ctas)), dim3(kFwdThreads),
                         GradGeom<DK, NV>::kSmem, st, true, q, k, o, a, ops, (const char*)(a.rec + L.rec_S),
                         (const char*)(a.rec + L.rec_eps), (const char*)(a.ws + L.ws_dS), (const char*)(a.ws + L.ws_dV),
                         (const float*)part, (const float*)phi, reinterpret_cast<float*>(a.ws + L.ws_dq),
                         reinterpret_cast<float*>(a.ws + L.ws_dk));
}

template <int DK>
cudaError_t backward_dk(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    return seq_tc_cols(a.sh) == 32 ? bwd_go<DK, 32>(q, k, a, L, st) : bwd_go<DK, 16>(q, k, a, L, st);
}

}  // namespace

bool seq_tc_takes(int dtype) { return dtype == GDN_DTYPE_BF16; }

// Value columns of a scan's CTA.  A chunk takes some 1.4 times as long with 32 as with 16, so 16 where they all
// run at once, one CTA an SM, and 32 where 16 would take another turn.  Prep and scan of 8 heads of 256, with a record
// and then backward: 1 x 8192 314 and 468 us with 16, 442 and 694 with 32; 4 x 2048 321 and 493 with 16, 259 and
// 470 with 32.
int seq_tc_cols(const SeqShape& s) {
    return s.dv % 32 == 0 && (size_t)s.nseq * s.H * (s.dv / 16) > kSMs ? 32 : 16;
}

cudaError_t launch_seq_forward_tc(const SeqArgs& a, cudaStream_t st) {
    CUtensorMap q, k;
    if (!qk_maps(a, &q, &k)) return cudaErrorInvalidValue;
    switch (seq_tc_dk(a.sh.dk)) {
        case 64: return forward_dk<64>(q, k, a, st);
        case 128: return forward_dk<128>(q, k, a, st);
        case 192: return forward_dk<192>(q, k, a, st);
        default: return forward_dk<256>(q, k, a, st);
    }
}

cudaError_t launch_seq_backward_tc(const SeqArgs& a, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, GDN_DTYPE_BF16);
    CUtensorMap q, k;
    if (!qk_maps(a, &q, &k)) return cudaErrorInvalidValue;
    switch (seq_tc_dk(a.sh.dk)) {
        case 64: return backward_dk<64>(q, k, a, L, st);
        case 128: return backward_dk<128>(q, k, a, L, st);
        case 192: return backward_dk<192>(q, k, a, L, st);
        default: return backward_dk<256>(q, k, a, L, st);
    }
}

}  // namespace gdn

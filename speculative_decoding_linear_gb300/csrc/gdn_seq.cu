// gdn_seq.cu -- the gated delta rule over packed sequences: entry points, layouts, and the
// CUDA-core kernels that serve fp32 inputs.
//
//   S' = e^{la_t} S_{t-1},  eps_t = v_t - S' k_t,  S_t = S' + beta_t eps_t k_t^T,  o_t = S_t q_t
//
// Forward, token by token: each row of S (one value index) is independent, so lanes keep
// rows in registers and need one dot product with k_t, one with q_t for each row and token.
//
// Backward: with dS the gradient of S_t (dO_t q_t^T added), w_t = dS k_t, the gradient of eps_t
// is dV_t = beta_t w_t and dS_{t-1} = e^{la_t} (dS - dV_t k_t^T): the rows stay independent, and
// S is not needed.  dq, dk and the gates' gradients need S and dS against each other: they are
// formed for each chunk of 64 tokens from the state at its start (S, kept by the forward pass),
// the gradient at its end (dS+), eps and dV.  With g the cumulative log gate within the chunk
// and G_tj = e^{g_t - g_j} (j <= t):
//   dq_t  = e^{g_t} S^T dO_t + sum_{j<=t} G_tj beta_j (dO_t.eps_j) k_j
//   dk_t  = - e^{g_t} S^T dV_t - sum_{j<t} G_tj beta_j (dV_t.eps_j) k_j                 ("read")
//           + sum_{s>=t} G_st beta_t (dO_s.eps_t) q_s - sum_{s>t} G_st beta_t (dV_s.eps_t) k_s
//           + beta_t w2_t,  w2_t = e^{g_end - g_t} dS+^T eps_t                           ("write")
//   dbeta_j = sum_t G_tj ((q_t.k_j)(dO_t.eps_j) - [t>j] (k_t.k_j)(dV_t.eps_j)) + k_j.w2_j
//   dla_t = e^{g_end} <S, dS+> + sum_{s<t} beta_s k_s.w2_s + sum_{s>=t} (q_s.dq_s + k_s.read_s - k_s.write'_s)
// (write' without the w2 term).  No division by beta or alpha: both may be zero.
#include "gdn_seq_tc.cuh"

namespace gdn {

namespace {

// A row of S is kept by LPR lanes, eight columns each in pairs: LPR 8, 16 or 32 for a d_k of up to 64, 128 or 256.
// A token costs a warp its chain, the dot products and log2(LPR) shuffles, and little else: a warp of its own brings
// the CTA's tokens into a ring in shared memory, kGroup at a time.  R rows for a lane: one is quicker where a
// scheduler has few warps (600 tokens, 8 heads of 128: 160 us against 214), two where it has many (3 x 200 tokens,
// 8 heads of 256: 186 against 275).  301 tokens, 4 heads of 64: 84 us, 0.28 us a token.
constexpr int kGroup = 8, kRing = 4;

template <int LPR, int R>
struct Scan {
    static constexpr int kThreads = 128, kAll = kThreads + 32;
    static constexpr int kRows = kThreads / LPR * R;                 // value rows of a CTA
    static constexpr int kK = 0, kQ = 8 * LPR, kV = kQ + 8 * LPR, kLa = kV + kRows, kBeta = kLa + 1, kToken = kLa + 4;   // floats
    static constexpr size_t kSmem = (size_t)kRing * kGroup * kToken * 4;
};

__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Group g's tokens into its place of the ring, by a warp: 8 g, 8 g + 1, ... from the sequence's first token on, or from
// its last one back.
template <int LPR, int R, bool BACK>
__device__ __forceinline__ void copy_group(const SeqArgs& a, float* ring, const float* v, size_t ldv, int first, int len, int g, int h,
                                           int hk) {
    using C = Scan<LPR, R>;
    const SeqShape& sh = a.sh;
    const int n = min(kGroup, len - g * kGroup), lane = threadIdx.x & 31;
    float* dst = ring + (size_t)(g % kRing) * kGroup * C::kToken;
    for (int j = 0; j < n; ++j) {
        const int at = g * kGroup + j;
        const size_t t = (size_t)first + (BACK ? len - 1 - at : at);
        float* x = dst + j * C::kToken;
        const float* k = static_cast<const float*>(a.k) + t * sh.ldk + (size_t)hk * sh.dk;
        const float* q = static_cast<const float*>(a.q) + t * sh.ldq + (size_t)hk * sh.dk;
        for (int p = 4 * lane; p < sh.dk; p += 128) {
            cp_async16(x + C::kK + p, k + p);
            cp_async16(x + C::kQ + p, q + p);
        }
        if (4 * lane < C::kRows)
            cp_async16(x + C::kV + 4 * lane, v + t * ldv + 4 * lane);
        else if (lane >= 30)
            cp_async4(x + (lane == 30 ? C::kLa : C::kBeta), (lane == 30 ? a.la : a.beta) + t * sh.H + h);
    }
}

// step(token in the ring, its number in the sequence) for all tokens in their order
template <int LPR, int R, bool BACK, class Step>
__device__ __forceinline__ void for_tokens(const SeqArgs& a, const float* v, size_t ldv, int first, int len, int h, int hk, Step&& step) {
    using C = Scan<LPR, R>;
    extern __shared__ float4 ring4[];
    float* ring = reinterpret_cast<float*>(ring4);
    const bool copies = threadIdx.x >= C::kThreads;
    // columns behind d_k, which no copy fills
    for (int i = threadIdx.x; i < kRing * kGroup * C::kToken; i += C::kAll) ring[i] = 0.f;
    __syncthreads();
    const int groups = (len + kGroup - 1) / kGroup;
    if (copies)
        for (int g = 0; g < kRing - 1; ++g) {
            if (g < groups) copy_group<LPR, R, BACK>(a, ring, v, ldv, first, len, g, h, hk);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        }
    for (int g = 0; g < groups; ++g) {
        if (copies) asm volatile("cp.async.wait_group %0;\n" ::"n"(kRing - 2) : "memory");
        __syncthreads();                       // group g is there, group g - 1 read
        if (copies) {
            if (g + kRing - 1 < groups) copy_group<LPR, R, BACK>(a, ring, v, ldv, first, len, g + kRing - 1, h, hk);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            continue;
        }
        const float* x = ring + (size_t)(g % kRing) * kGroup * C::kToken;
        const int n = min(kGroup, len - g * kGroup), i0 = BACK ? len - 1 - g * kGroup : g * kGroup;
        if (n == kGroup) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) step(x + j * C::kToken, BACK ? i0 - j : i0 + j);
        } else {
            for (int j = 0; j < n; ++j) step(x + j * C::kToken, BACK ? i0 - j : i0 + j);
        }
    }
}

// One lane's eight columns of a row of n: 4 l + {0..3}, and 4 LPR more.
template <int LPR>
__device__ __forceinline__ void ld_cols(const float* p, int n, int l, float2 (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 4 * LPR * j + 4 * l;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < n) u = *reinterpret_cast<const float4*>(p + c);
        x[2 * j] = make_float2(u.x, u.y);
        x[2 * j + 1] = make_float2(u.z, u.w);
    }
}
template <int LPR>
__device__ __forceinline__ void st_cols(float* p, int n, int l, const float2 (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 4 * LPR * j + 4 * l;
        if (c < n) *reinterpret_cast<float4*>(p + c) = make_float4(x[2 * j].x, x[2 * j].y, x[2 * j + 1].x, x[2 * j + 1].y);
    }
}
// a lane's part of a dot product, and N of them summed over the lanes of a row at once
__device__ __forceinline__ float part(const float2 (&a)[4], const float2 (&b)[4]) {
    const float2 s = ffma2(a[1], b[1], fmul2(a[0], b[0])), u = ffma2(a[3], b[3], fmul2(a[2], b[2]));
    return (s.x + s.y) + (u.x + u.y);
}
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&x)[N]) {
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) {
        float y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __shfl_xor_sync(0xffffffffu, x[i], m);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += y[i];
    }
}

// What a thread of a scan works on.
template <int LPR, int R>
struct Place {
    int s, h, hk, l, rl, row0, first, len;
    size_t head;                               // its row of the state, of the heads' rows
    __device__ __forceinline__ bool find(const SeqArgs& a) {
        const SeqShape& sh = a.sh;
        const int tiles = sh.dv / Scan<LPR, R>::kRows;
        s = blockIdx.x / (tiles * sh.H);
        h = blockIdx.x / tiles % sh.H;
        hk = h / (sh.H / sh.Hk);
        l = threadIdx.x % LPR;
        rl = threadIdx.x % Scan<LPR, R>::kThreads / LPR * R;
        row0 = blockIdx.x % tiles * Scan<LPR, R>::kRows;
        head = ((size_t)s * sh.H + h) * sh.dv + row0 + rl;
        return seq_range(sh, s, first, len, a.err);
    }
    // the row of a chunk's kept state
    __device__ __forceinline__ float* kept(float* p, const SeqShape& sh, int i) const {
        return p + (((size_t)(first / kChunk + s + i / kChunk) * sh.H + h) * sh.dv + row0 + rl) * sh.dk;
    }
};

template <int LPR, int R>
__global__ void __launch_bounds__(Scan<LPR, R>::kAll, 4) seq_scan_kernel(SeqArgs a, float* recS, float* eps) {
    using C = Scan<LPR, R>;
    const SeqShape& sh = a.sh;
    int out_b, out_e;
    if (seq_outside(sh, out_b, out_e)) zero_rows<float4>(a.out, (size_t)sh.H * sh.dv / 4, out_b, out_e, sh.total);
    Place<LPR, R> at;
    if (!at.find(a)) return;
    const int l = at.l;
    const bool computes = threadIdx.x < C::kThreads;
    float2 S[R][4] = {};
    if (computes && a.S0 != nullptr)
#pragma unroll
        for (int r = 0; r < R; ++r) ld_cols<LPR>(a.S0 + (at.head + r) * sh.dk, sh.dk, l, S[r]);
    const size_t ldo = (size_t)sh.H * sh.dv, o0 = at.first * ldo + (size_t)at.h * sh.dv + at.row0 + at.rl;
    float *out = static_cast<float*>(a.out) + o0, *ep = eps == nullptr ? nullptr : eps + o0;
    const float* v = static_cast<const float*>(a.v) + (size_t)at.h * sh.dv + at.row0;
    for_tokens<LPR, R, false>(a, v, sh.ldv, at.first, at.len, at.h, at.hk, [&](const float* x, int i) {
        if (recS != nullptr && i % kChunk == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) st_cols<LPR>(at.kept(recS, sh, i) + r * sh.dk, sh.dk, l, S[r]);
        float2 k[4], q[4];
        ld_cols<LPR>(x + C::kK, 8 * LPR, l, k);
        ld_cols<LPR>(x + C::kQ, 8 * LPR, l, q);
        const float ea = expf(gate_log(x[C::kLa]));
        // with S' = e^la S: e = v - S' k and o = S' q + delta (k.q), one round of sums for a token
        float d[2 * R + 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            d[2 * r] = part(S[r], k);
            d[2 * r + 1] = part(S[r], q);
        }
        d[2 * R] = part(k, q);
        row_sums<LPR>(d);
        const float2 ea2 = make_float2(ea, ea);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float e = fmaf(-ea, d[2 * r], x[C::kV + at.rl + r]), de = x[C::kBeta] * e;
            const float2 de2 = make_float2(de, de);
#pragma unroll
            for (int j = 0; j < 4; ++j) S[r][j] = ffma2(de2, k[j], fmul2(ea2, S[r][j]));
            if (l == 0) {
                out[r] = fmaf(de, d[2 * R], ea * d[2 * r + 1]);
                if (ep != nullptr) ep[r] = e;
            }
        }
        out += ldo;
        if (ep != nullptr) ep += ldo;
    });
    if (computes && a.S_T != nullptr)
#pragma unroll
        for (int r = 0; r < R; ++r) st_cols<LPR>(a.S_T + (at.head + r) * sh.dk, sh.dk, l, S[r]);
}

template <int LPR, int R>
__global__ void __launch_bounds__(Scan<LPR, R>::kAll, 4) seq_scan_back_kernel(SeqArgs a, float* dSc, float* dVf) {
    using C = Scan<LPR, R>;
    const SeqShape& sh = a.sh;
    Place<LPR, R> at;
    if (!at.find(a)) return;
    const int l = at.l;
    const bool computes = threadIdx.x < C::kThreads;
    float2 S[R][4] = {};
    if (computes && a.dS_T != nullptr)
#pragma unroll
        for (int r = 0; r < R; ++r) ld_cols<LPR>(a.dS_T + (at.head + r) * sh.dk, sh.dk, l, S[r]);
    const size_t ldo = (size_t)sh.H * sh.dv;
    size_t o = ((size_t)at.first + at.len - 1) * ldo + (size_t)at.h * sh.dv + at.row0 + at.rl;
    const float* dout = static_cast<const float*>(a.dout) + (size_t)at.h * sh.dv + at.row0;
    for_tokens<LPR, R, true>(a, dout, ldo, at.first, at.len, at.h, at.hk, [&](const float* x, int i) {
        if (i == at.len - 1 || i % kChunk == kChunk - 1)
#pragma unroll
            for (int r = 0; r < R; ++r) st_cols<LPR>(at.kept(dSc, sh, i) + r * sh.dk, sh.dk, l, S[r]);
        float2 k[4], q[4];
        ld_cols<LPR>(x + C::kK, 8 * LPR, l, k);
        ld_cols<LPR>(x + C::kQ, 8 * LPR, l, q);
        const float ea = expf(gate_log(x[C::kLa]));
        // w = beta (dS + dO q^T) k
        float d[R + 1];
#pragma unroll
        for (int r = 0; r < R; ++r) d[r] = part(S[r], k);
        d[R] = part(k, q);
        row_sums<LPR>(d);
        const float2 ea2 = make_float2(ea, ea);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float ot = x[C::kV + at.rl + r], w = x[C::kBeta] * fmaf(ot, d[R], d[r]);
            const float2 ot2 = make_float2(ot, ot), w2 = make_float2(-w, -w);
#pragma unroll
            for (int j = 0; j < 4; ++j) S[r][j] = fmul2(ea2, ffma2(w2, k[j], ffma2(ot2, q[j], S[r][j])));
            if (l == 0) {
                dVf[o + r] = w;
                static_cast<float*>(a.dv)[o + r] = w;
            }
        }
        o -= ldo;
    });
    if (computes && a.dS0 != nullptr)
#pragma unroll
        for (int r = 0; r < R; ++r) st_cols<LPR>(a.dS0 + (at.head + r) * sh.dk, sh.dk, l, S[r]);
}

// One CTA per (chunk, head): products of 64 x 64 tiles in slices of 32 that go through shared memory, the next
// slice on its way meanwhile; a thread keeps four rows and four columns of each product.  Where heads share q and k,
// each writes its own dq and dk, and seq_heads_kernel adds them.
constexpr int kGradThreads = 256;
constexpr int kLdm = kChunk + 1;
constexpr int kSlice = 32, kLds = kChunk + 4;
constexpr int kSliceFloats = kSlice * kLds;
constexpr size_t kGradSmem = (5 * kSliceFloats + 3 * kChunk * kLdm + 6 * kChunk) * 4;

// A slice in a thread's registers, on its way to shared memory: two pieces of four columns.
struct Slice {
    float4 x[2];
};
// 64 rows of `n` (at most 32) columns, zeros behind `rows` and `n`
__device__ __forceinline__ void ld_turned(Slice& z, const float* src, size_t ld, int rows, int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * kGradThreads, r = i % kChunk, c = i / kChunk * 4;
        z.x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < n) z.x[u] = *reinterpret_cast<const float4*>(src + r * ld + c);
    }
}
__device__ __forceinline__ void st_turned(float* dst, const Slice& z) {       // dst[column][row]
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * kGradThreads, r = i % kChunk, c = i / kChunk * 4;
        dst[c * kLds + r] = z.x[u].x;
        dst[(c + 1) * kLds + r] = z.x[u].y;
        dst[(c + 2) * kLds + r] = z.x[u].z;
        dst[(c + 3) * kLds + r] = z.x[u].w;
    }
}
// `rows` (at most 32) rows of n (at most 64) columns as they are, zeros behind both
__device__ __forceinline__ void ld_rows(Slice& z, const float* src, size_t ld, int rows, int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * kGradThreads, r = i / 16, c = i % 16 * 4;
        z.x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < n) z.x[u] = *reinterpret_cast<const float4*>(src + r * ld + c);
    }
}
__device__ __forceinline__ void st_rows(float* dst, const Slice& z) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * kGradThreads, r = i / 16, c = i % 16 * 4;
        *reinterpret_cast<float4*>(dst + r * kLds + c) = z.x[u];
    }
}
__device__ __forceinline__ void outer(const float (&x)[4], const float4& y, float (&c)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i][0] = fmaf(x[i], y.x, c[i][0]);
        c[i][1] = fmaf(x[i], y.y, c[i][1]);
        c[i][2] = fmaf(x[i], y.z, c[i][2]);
        c[i][3] = fmaf(x[i], y.w, c[i][3]);
    }
}
__device__ __forceinline__ void outer(const float4& x, const float4& y, float (&c)[4][4]) {
    const float z[4] = {x.x, x.y, x.z, x.w};
    outer(z, y, c);
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// hi + lo += x, the sum's rounding kept in lo
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
}

__global__ void __launch_bounds__(kGradThreads)
    seq_grad_kernel(SeqArgs a, const float* recS, const float* eps, const float* dSc, const float* dVf, float* dqo,
                    float* dko) {
    extern __shared__ float4 sm4[];
    float* X = reinterpret_cast<float*>(sm4);
    float *Y = X + kSliceFloats, *Z = Y + kSliceFloats, *U = Z + kSliceFloats, *V = U + kSliceFloats;
    float* MP = V + kSliceFloats;            // G beta (dO.eps)
    float* ME = MP + kChunk * kLdm;          // G beta (dV.eps), t > j
    float* MB = ME + kChunk * kLdm;          // dbeta's terms
    float* ghi = MB + kChunk * kLdm;         // cumulative log gate, two floats
    float* glo = ghi + kChunk;
    float* bt = glo + kChunk;
    float* xs = bt + kChunk;
    float* us = xs + kChunk;
    float* red = us + kChunk;
    const SeqShape& sh = a.sh;
    const int h = blockIdx.x % sh.H, slot = blockIdx.x / sh.H, hk = h / (sh.H / sh.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ty = tid / 16 * 4, tx = tid % 16 * 4;
    int s, first, rows, out_b, out_e;
    if (seq_outside(sh, out_b, out_e)) {
        for (float* p : {dqo, dko}) zero_rows<float4>(p, (size_t)sh.H * sh.dk / 4, out_b, out_e, sh.total);
        zero_rows<float4>(a.dv, (size_t)sh.H * sh.dv / 4, out_b, out_e, sh.total);
        for (float* p : {a.dla, a.dbeta}) zero_rows<float>(p, sh.H, out_b, out_e, sh.total);
    }
    if (!slot_chunk(sh, slot, s, first, rows, a.err)) return;
    const float* q = static_cast<const float*>(a.q) + (size_t)first * sh.ldq + (size_t)hk * sh.dk;
    const float* k = static_cast<const float*>(a.k) + (size_t)first * sh.ldk + (size_t)hk * sh.dk;
    const size_t ldo = (size_t)sh.H * sh.dv;
    const float* dout = static_cast<const float*>(a.dout) + (size_t)first * ldo + (size_t)h * sh.dv;
    const float* e = eps + (size_t)first * ldo + (size_t)h * sh.dv;
    const float* dV = dVf + (size_t)first * ldo + (size_t)h * sh.dv;
    const float* S = recS + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
    const float* dS = dSc + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
    if (tid < kChunk) {
        xs[tid] = us[tid] = 0.f;
        bt[tid] = tid < rows ? a.beta[((size_t)first + tid) * sh.H + h] : 0.f;
        red[tid] = tid < rows ? gate_log(a.la[((size_t)first + tid) * sh.H + h]) : 0.f;
    }
    __syncthreads();
    if (tid == 0) {
        float hi = 0.f, lo = 0.f;
        for (int t = 0; t < kChunk; ++t) {           // tokens behind the last keep the last one's
            add_exact(hi, lo, red[t]);
            const float g = hi + lo;
            ghi[t] = g;
            glo[t] = lo - (g - hi);
        }
    }
    {
        float e1[4][4] = {}, e2[4][4] = {}, qk[4][4] = {}, kk[4][4] = {};
        Slice x, y, z;
        const auto ld_dv = [&](int c) {
            const int n = sh.dv - c;
            ld_turned(x, dout + c, ldo, rows, n);
            ld_turned(y, dV + c, ldo, rows, n);
            ld_turned(z, e + c, ldo, rows, n);
        };
        const auto ld_dk = [&](int c) {
            const int n = sh.dk - c;
            ld_turned(x, q + c, sh.ldq, rows, n);
            ld_turned(y, k + c, sh.ldk, rows, n);
        };
        ld_dv(0);
        for (int c = 0; c < sh.dv; c += kSlice) {
            __syncthreads();
            st_turned(X, x);
            st_turned(Y, y);
            st_turned(Z, z);
            __syncthreads();
            if (c + kSlice < sh.dv) ld_dv(c + kSlice); else ld_dk(0);
#pragma unroll 8
            for (int j = 0; j < kSlice; ++j) {
                const float4 w = at4(Z + j * kLds + tx);
                outer(at4(X + j * kLds + ty), w, e1);
                outer(at4(Y + j * kLds + ty), w, e2);
            }
        }
        for (int c = 0; c < sh.dk; c += kSlice) {
            __syncthreads();
            st_turned(X, x);
            st_turned(Y, y);
            __syncthreads();
            if (c + kSlice < sh.dk) ld_dk(c + kSlice);
#pragma unroll 8
            for (int j = 0; j < kSlice; ++j) {
                const float4 w = at4(Y + j * kLds + tx);
                outer(at4(X + j * kLds + ty), w, qk);
                outer(at4(Y + j * kLds + ty), w, kk);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int t = ty + i, j = tx + m;
                float mp = 0.f, me = 0.f, mb = 0.f;
                if (t < rows && j <= t) {
                    const float G = expf((ghi[t] - ghi[j]) + (glo[t] - glo[j]));
                    mp = G * bt[j] * e1[i][m];
                    mb = G * qk[i][m] * e1[i][m];
                    if (j < t) {
                        me = G * bt[j] * e2[i][m];
                        mb -= G * kk[i][m] * e2[i][m];
                    }
                }
                MP[t * kLdm + j] = mp;
                ME[t * kLdm + j] = me;
                MB[t * kLdm + j] = mb;
            }
    }
    __syncthreads();
    const float gend_hi = ghi[kChunk - 1], gend_lo = glo[kChunk - 1];
    float dot = 0.f;
    for (int cb = 0; cb < sh.dk; cb += kChunk) {
        const int n = min(kChunk, sh.dk - cb);
        float dq[4][4] = {}, dr[4][4] = {}, dw[4][4] = {}, w2[4][4] = {};
        Slice x, y, z, u, w;
        const auto ld_v = [&](int v) {
            const int nv = sh.dv - v;
            ld_turned(x, dout + v, ldo, rows, nv);
            ld_turned(y, dV + v, ldo, rows, nv);
            ld_turned(z, e + v, ldo, rows, nv);
            ld_rows(u, S + (size_t)v * sh.dk + cb, sh.dk, nv, n);
            ld_rows(w, dS + (size_t)v * sh.dk + cb, sh.dk, nv, n);
        };
        const auto ld_j = [&](int j0) {
            ld_rows(u, q + (size_t)j0 * sh.ldq + cb, sh.ldq, rows - j0, n);
            ld_rows(w, k + (size_t)j0 * sh.ldk + cb, sh.ldk, rows - j0, n);
        };
        ld_v(0);
        for (int v = 0; v < sh.dv; v += kSlice) {
            __syncthreads();
            st_turned(X, x);
            st_turned(Y, y);
            st_turned(Z, z);
            st_rows(U, u);
            st_rows(V, w);
#pragma unroll
            for (int m = 0; m < 2; ++m)
                dot += u.x[m].x * w.x[m].x + u.x[m].y * w.x[m].y + u.x[m].z * w.x[m].z + u.x[m].w * w.x[m].w;
            __syncthreads();
            if (v + kSlice < sh.dv) ld_v(v + kSlice); else ld_j(0);
#pragma unroll 4
            for (int j = 0; j < kSlice; ++j) {
                const float4 f = at4(U + j * kLds + tx), g = at4(V + j * kLds + tx);
                outer(at4(X + j * kLds + ty), f, dq);
                outer(at4(Y + j * kLds + ty), f, dr);
                outer(at4(Z + j * kLds + ty), g, w2);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = ty + i;
            const float eg = expf(ghi[t] + glo[t]), et = expf((gend_hi - ghi[t]) + (gend_lo - glo[t]));
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                dq[i][m] *= eg;
                dr[i][m] *= -eg;
                w2[i][m] *= et;
            }
        }
        for (int j0 = 0; j0 < rows; j0 += kSlice) {
            __syncthreads();
            st_rows(U, u);
            st_rows(V, w);
            __syncthreads();
            if (j0 + kSlice < rows) ld_j(j0 + kSlice);
#pragma unroll 4
            for (int j = 0; j < kSlice; ++j) {
                const float4 f = at4(U + j * kLds + tx), g = at4(V + j * kLds + tx);
                float p[4], m[4], pt[4], mt[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = MP[(ty + i) * kLdm + j0 + j];
                    m[i] = -ME[(ty + i) * kLdm + j0 + j];
                    pt[i] = MP[(j0 + j) * kLdm + ty + i];
                    mt[i] = -ME[(j0 + j) * kLdm + ty + i];
                }
                outer(p, g, dq);
                outer(m, g, dr);
                outer(pt, f, dw);
                outer(mt, g, dw);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = ty + i;
            float xq = 0.f, xu = 0.f;
            if (t < rows && tx < n) {
                const float4 qv = at4(q + (size_t)t * sh.ldq + cb + tx), kv = at4(k + (size_t)t * sh.ldk + cb + tx);
                const float qc[4] = {qv.x, qv.y, qv.z, qv.w}, kc[4] = {kv.x, kv.y, kv.z, kv.w};
                float gq[4], gk[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    xq += qc[m] * dq[i][m] + kc[m] * (dr[i][m] - dw[i][m]);
                    xu = fmaf(kc[m], w2[i][m], xu);
                    gq[m] = dq[i][m];
                    gk[m] = dr[i][m] + dw[i][m] + bt[t] * w2[i][m];
                }
                const size_t at = ((size_t)(first + t) * sh.H + h) * sh.dk + cb + tx;
                *reinterpret_cast<float4*>(dqo + at) = make_float4(gq[0], gq[1], gq[2], gq[3]);
                *reinterpret_cast<float4*>(dko + at) = make_float4(gk[0], gk[1], gk[2], gk[3]);
            }
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) {
                xq += __shfl_xor_sync(0xffffffffu, xq, m);
                xu += __shfl_xor_sync(0xffffffffu, xu, m);
            }
            if (tx == 0) {
                xs[t] += xq;
                us[t] += xu;
            }
        }
    }
    dot = warp_sum(dot);
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    if (tid < rows) {
        const size_t at = ((size_t)first + tid) * sh.H + h;
        float hi = 0.f, lo = 0.f;
        for (int w = 0; w < kGradThreads / 32; ++w) hi += red[w];
        hi *= expf(gend_hi + gend_lo);
        for (int t = 0; t < rows; ++t) add_exact(hi, lo, t < tid ? bt[t] * us[t] : xs[t]);
        a.dla[at] = hi + lo;
        hi = us[tid];
        lo = 0.f;
        for (int t = tid; t < rows; ++t) add_exact(hi, lo, MB[t * kLdm + tid]);
        a.dbeta[at] = hi + lo;
    }
}

// dq and dk of a q/k head: the sum over the heads that share it, in their order.
__global__ void __launch_bounds__(256) seq_heads_kernel(const float* dqo, const float* dko, float* dq, float* dk, size_t n4, int rep, int dk4) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const size_t at = i / dk4 * rep * dk4 + i % dk4;
    const float4 *p = reinterpret_cast<const float4*>(dqo) + at, *u = reinterpret_cast<const float4*>(dko) + at;
    float4 x = p[0], y = u[0];
    for (int r = 1; r < rep; ++r) {
        const float4 z = p[(size_t)r * dk4], w = u[(size_t)r * dk4];
        x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
        y = make_float4(y.x + w.x, y.y + w.y, y.z + w.z, y.w + w.w);
    }
    reinterpret_cast<float4*>(dq)[i] = x;
    reinterpret_cast<float4*>(dk)[i] = y;
}

template <int LPR, int R>
cudaError_t forward_go(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    static bool done[64];
    const cudaError_t rc = ensure_smem(seq_scan_kernel<LPR, R>, Scan<LPR, R>::kSmem, done);
    if (rc != cudaSuccess) return rc;
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / Scan<LPR, R>::kRows));
    float* S = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_S) : nullptr;
    float* e = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_eps) : nullptr;
    return launch_kernel(seq_scan_kernel<LPR, R>, dim3(grid), dim3(Scan<LPR, R>::kAll), Scan<LPR, R>::kSmem, st, false, a, S, e);
}

template <int LPR, int R>
cudaError_t backward_go(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    static bool done_scan[64], done[64];
    cudaError_t rc = ensure_smem(seq_scan_back_kernel<LPR, R>, Scan<LPR, R>::kSmem, done_scan);
    if (rc == cudaSuccess) rc = ensure_smem(seq_grad_kernel, kGradSmem, done);
    if (rc != cudaSuccess) return rc;
    const SeqShape& sh = a.sh;
    const unsigned grid = (unsigned)((size_t)sh.nseq * sh.H * (sh.dv / Scan<LPR, R>::kRows));
    float* dS = reinterpret_cast<float*>(a.ws + L.ws_dS);
    float* dV = reinterpret_cast<float*>(a.ws + L.ws_dV);
    rc = launch_kernel(seq_scan_back_kernel<LPR, R>, dim3(grid), dim3(Scan<LPR, R>::kAll), Scan<LPR, R>::kSmem, st, false, a, dS, dV);
    if (rc != cudaSuccess || sh.total == 0) return rc;
    const bool shared = sh.H > sh.Hk;
    float *dq = static_cast<float*>(a.dq), *dk = static_cast<float*>(a.dk);
    float *dqo = shared ? reinterpret_cast<float*>(a.ws + L.ws_dq) : dq, *dko = shared ? reinterpret_cast<float*>(a.ws + L.ws_dk) : dk;
    rc = launch_kernel(seq_grad_kernel, dim3((unsigned)((size_t)seq_slots(sh.nseq, sh.total) * sh.H)), dim3(kGradThreads), kGradSmem, st,
                       false, a, (const float*)(a.rec + L.rec_S), (const float*)(a.rec + L.rec_eps), (const float*)dS, (const float*)dV,
                       dqo, dko);
    if (rc != cudaSuccess || !shared) return rc;
    const size_t n4 = (size_t)sh.total * sh.Hk * sh.dk / 4;
    return launch_kernel(seq_heads_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st, false, (const float*)dqo,
                         (const float*)dko, dq, dk, n4, sh.H / sh.Hk, sh.dk / 4);
}

// Two rows for a lane where a scheduler has more than three warps with one (four schedulers an SM; LPR lanes a row),
// and the CTA's rows divide d_v.
bool two_rows(const SeqShape& s, int lpr) {
    return s.dv % (256 / lpr) == 0 && (long long)s.nseq * s.H * s.dv * lpr / 32 > 3LL * 4 * kSMs;
}

}  // namespace

// also a bf16 call without tokens, which copies the state and reads nothing of bf16
cudaError_t launch_seq_forward_f32(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    if (a.sh.dk <= 64) return two_rows(a.sh, 8) ? forward_go<8, 2>(a, L, st) : forward_go<8, 1>(a, L, st);
    if (a.sh.dk <= 128) return two_rows(a.sh, 16) ? forward_go<16, 2>(a, L, st) : forward_go<16, 1>(a, L, st);
    return two_rows(a.sh, 32) ? forward_go<32, 2>(a, L, st) : forward_go<32, 1>(a, L, st);
}

cudaError_t launch_seq_backward_f32(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    if (a.sh.dk <= 64) return two_rows(a.sh, 8) ? backward_go<8, 2>(a, L, st) : backward_go<8, 1>(a, L, st);
    if (a.sh.dk <= 128) return two_rows(a.sh, 16) ? backward_go<16, 2>(a, L, st) : backward_go<16, 1>(a, L, st);
    return two_rows(a.sh, 32) ? backward_go<32, 2>(a, L, st) : backward_go<32, 1>(a, L, st);
}

SeqLayout seq_layout(const SeqShape& s, int dtype) {
    SeqLayout L = {};
    const bool tc = seq_tc_takes(dtype);
    const size_t slots = seq_slots(s.nseq, s.total), state = slots * s.H * (tc ? seq_tc_dk(s.dk) : s.dk) * s.dv * 4;
    // the tensor-core kernels keep rows of tokens for whole chunks
    const size_t rows = (tc ? slots * kChunk : (size_t)s.total) * s.H * s.dv * 4;
    // heads that share q and k: their sum so far, or (fp32) all of them
    const size_t heads = s.H > s.Hk ? (size_t)s.total * (tc ? s.Hk : s.H) * s.dk * 4 : 0;
    const size_t tiles = slots * s.H * (s.dv / 16);        // of 16 value columns at least
    L.rec_S = 0;
    // three bf16 terms of the tensor-core kernels' operands, or fp32
    L.rec_eps = align_up(L.rec_S + (tc ? state / 2 * 3 : state), kSectionAlign);
    L.rec_o = align_up(L.rec_eps + (tc ? rows / 2 * 3 : rows), kSectionAlign);
    L.rec_op = align_up(L.rec_o + (tc ? rows : 0), kSectionAlign);
    L.rec_total = align_up(L.rec_op + (tc ? slots * s.H * seqtc::kOpRecord : 0), kSectionAlign);
    L.ws_op = 0;
    L.ws_part = align_up(L.ws_op + (tc ? slots * s.H * seqtc::kOpBytes : 0), kSectionAlign);
    L.ws_phi = align_up(L.ws_part + (tc ? tiles * 4 * kChunk * 4 : 0), kSectionAlign);
    L.ws_dS = align_up(L.ws_phi + (tc ? tiles * 8 * 4 : 0), kSectionAlign);
    L.ws_dV = align_up(L.ws_dS + state, kSectionAlign);
    L.ws_dq = align_up(L.ws_dV + rows, kSectionAlign);
    L.ws_dk = align_up(L.ws_dq + heads, kSectionAlign);
    L.ws_total = align_up(L.ws_dk + heads, kSectionAlign);
    return L;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p != nullptr && aligned16(p); }
// the tensor-core kernels write and read a record by 32 bytes
bool record_ok(const void* p, bool tc) { return (reinterpret_cast<uintptr_t>(p) & (tc ? 31u : 15u)) == 0; }
// gates and offsets are read one by one: any row of a larger tensor will do
bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dim_ok(int d) { return d >= 16 && d <= kMaxDim && d % 16 == 0; }

bool shape_ok(const SeqShape& s) {
    if (s.nseq < 1 || s.total < 0 || s.H < 1 || s.Hk < 1 || s.H % s.Hk != 0 || !dim_ok(s.dk) || !dim_ok(s.dv)) return false;
    if ((long long)s.nseq + s.total > (1LL << 30)) return false;
    // grid sizes: (sequence, head, 4 value rows) and (chunk slot, head)
    return (long long)s.nseq * s.H * (s.dv / 4) <= 0x7fffffffLL &&
           (long long)seq_slots(s.nseq, s.total) * s.H <= 0x7fffffffLL;
}

bool strides_ok(const SeqShape& s, int dtype) {
    const int unit = 16 / elem_bytes(dtype);
    const long long qk = (long long)s.Hk * s.dk, v = (long long)s.H * s.dv;      // a row: what fits a stride fits an int
    return s.ldq >= qk && s.ldk >= qk && s.ldv >= v && s.ldq % unit == 0 && s.ldk % unit == 0 && s.ldv % unit == 0;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (a == nullptr || b == nullptr) return false;
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return x < y + nb && y < x + na;
}

struct Span {
    const void* p;
    size_t n;
};

// No written span may meet a read one or another written one.
bool disjoint(const Span* w, int nw, const Span* r, int nr) {
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(w[i].p, w[i].n, w[j].p, w[j].n)) return false;
        for (int j = 0; j < nr; ++j)
            if (overlap(w[i].p, w[i].n, r[j].p, r[j].n)) return false;
    }
    return true;
}

size_t strided_bytes(int total, int ld, int row, int e) {
    return total == 0 ? 0 : ((size_t)(total - 1) * ld + row) * e;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_seq_workspace_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, nullptr, 0, 0, 0};
    if (bytes == nullptr || !shape_ok(s) || (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32)) return GDN_ERR_ARG;
    *bytes = seq_layout(s, dtype).ws_total;
    return GDN_OK;
}

int gdn_seq_forward_workspace_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, nullptr, 0, 0, 0};
    if (bytes == nullptr || !shape_ok(s) || (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32)) return GDN_ERR_ARG;
    *bytes = seq_layout(s, dtype).ws_forward();
    return GDN_OK;
}

int gdn_seq_record_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, nullptr, 0, 0, 0};
    if (bytes == nullptr || !shape_ok(s) || (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32)) return GDN_ERR_ARG;
    *bytes = seq_layout(s, dtype).rec_total;
    return GDN_OK;
}

int gdn_seq_forward(const void* q, int ldq, const void* k, int ldk, const void* v, int ldv, int dtype,
                    const float* log_alpha, const float* beta, const float* S0, const int32_t* offsets, void* out,
                    float* S_T, void* record, void* workspace, int nseq, int total, int H, int Hk, int dk, int dv,
                    cudaStream_t stream) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, offsets, ldq, ldk, ldv};
    if ((dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32) || !shape_ok(s) || !strides_ok(s, dtype)) return GDN_ERR_ARG;
    if (offsets == nullptr && total % nseq != 0) return GDN_ERR_ARG;
    const bool tc = total > 0 && seq_tc_takes(dtype);
    const SeqLayout L = seq_layout(s, dtype);
    if (L.ws_forward() == 0) workspace = nullptr;          // not touched
    if (!aligned16(S0) || !aligned16(S_T) || !record_ok(record, tc) || !words(offsets) || (L.ws_forward() > 0 && !given(workspace)))
        return GDN_ERR_ARG;
    if (total > 0 && (!given(q) || !given(k) || !given(v) || log_alpha == nullptr || !words(log_alpha) || beta == nullptr || !words(beta) || !given(out)))
        return GDN_ERR_ARG;
    const size_t e = elem_bytes(dtype), vo = (size_t)total * H * dv * e, gb = (size_t)total * H * 4,
                 sb = (size_t)nseq * H * dv * dk * 4;
    const Span w[] = {{out, vo}, {record, L.rec_total}, {workspace, L.ws_forward()}, {S_T, sb}};
    const Span r[] = {{q, strided_bytes(total, ldq, Hk * dk, (int)e)}, {k, strided_bytes(total, ldk, Hk * dk, (int)e)},
                      {v, strided_bytes(total, ldv, H * dv, (int)e)}, {log_alpha, gb}, {beta, gb},
                      {offsets, ((size_t)nseq + 1) * 4}};
    if (!disjoint(w, 4, r, 6)) return GDN_ERR_ARG;
    // S_T may be S0 itself: each element is read before it is written, by the same thread
    if (S_T != S0 && overlap(S0, sb, S_T, sb)) return GDN_ERR_ARG;
    for (int i = 0; i < 3; ++i)
        if (overlap(S0, sb, w[i].p, w[i].n)) return GDN_ERR_ARG;
    SeqArgs a = {};
    int st;
    a.err = current_error_word(&st);
    if (a.err == nullptr) return st;
    a.sh = s;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_alpha;
    a.beta = beta;
    a.S0 = S0;
    a.out = out;
    a.S_T = S_T;
    a.rec = static_cast<char*>(record);
    a.ws = static_cast<char*>(workspace);
    const cudaError_t rc = tc ? launch_seq_forward_tc(a, stream) : launch_seq_forward_f32(a, dtype, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_seq_backward(const void* q, int ldq, const void* k, int ldk, const void* v, int ldv, int dtype,
                     const float* log_alpha, const float* beta, const int32_t* offsets, const void* dout,
                     const float* dS_T, const void* record, void* dq, void* dk_out, void* dv_out, float* dlog_alpha,
                     float* dbeta, float* dS0, void* workspace, int nseq, int total, int H, int Hk, int dk, int dv,
                     cudaStream_t stream) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, offsets, ldq, ldk, ldv};
    if ((dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32) || !shape_ok(s) || !strides_ok(s, dtype)) return GDN_ERR_ARG;
    if (offsets == nullptr && total % nseq != 0) return GDN_ERR_ARG;
    const bool tc = total > 0 && seq_tc_takes(dtype);
    if (!aligned16(dS_T) || !aligned16(dS0) || !words(offsets) || !given(workspace) || record == nullptr || !record_ok(record, tc))
        return GDN_ERR_ARG;
    if (total > 0 && (!given(q) || !given(k) || !given(v) || log_alpha == nullptr || !words(log_alpha) || beta == nullptr || !words(beta) || !given(dout) ||
                      !given(dq) || !given(dk_out) || !given(dv_out) || !given(dlog_alpha) || !given(dbeta)))
        return GDN_ERR_ARG;
    const SeqLayout L = seq_layout(s, dtype);
    const size_t e = elem_bytes(dtype), vo = (size_t)total * H * dv * e, gb = (size_t)total * H * 4,
                 qb = (size_t)total * Hk * dk * e, sb = (size_t)nseq * H * dv * dk * 4;
    const Span w[] = {{dq, qb}, {dk_out, qb}, {dv_out, vo}, {dlog_alpha, gb}, {dbeta, gb}, {workspace, L.ws_total}, {dS0, sb}};
    const Span r[] = {{q, strided_bytes(total, ldq, Hk * dk, (int)e)}, {k, strided_bytes(total, ldk, Hk * dk, (int)e)},
                      {v, strided_bytes(total, ldv, H * dv, (int)e)}, {log_alpha, gb}, {beta, gb},
                      {offsets, ((size_t)nseq + 1) * 4}, {dout, vo}, {record, L.rec_total}};
    if (!disjoint(w, 7, r, 8)) return GDN_ERR_ARG;
    if (dS0 != dS_T && overlap(dS0, sb, dS_T, sb)) return GDN_ERR_ARG;
    for (int i = 0; i < 6; ++i)
        if (overlap(dS_T, sb, w[i].p, w[i].n)) return GDN_ERR_ARG;
    SeqArgs a = {};
    int st;
    a.err = current_error_word(&st);
    if (a.err == nullptr) return st;
    a.sh = s;
    a.q = q;
    a.k = k;
    a.v = v;
    a.la = log_alpha;
    a.beta = beta;
    a.dout = dout;
    a.dS_T = dS_T;
    a.rec = const_cast<char*>(static_cast<const char*>(record));
    a.dq = dq;
    a.dk = dk_out;
    a.dv = dv_out;
    a.dla = dlog_alpha;
    a.dbeta = dbeta;
    a.dS0 = dS0;
    a.ws = static_cast<char*>(workspace);
    const cudaError_t rc = tc ? launch_seq_backward_tc(a, stream) : launch_seq_backward_f32(a, dtype, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

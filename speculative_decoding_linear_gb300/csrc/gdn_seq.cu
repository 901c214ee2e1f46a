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

// A row of S is kept by LPR lanes of a warp, eight columns each: LPR 8, 16 or 32 for a d_k of up to 64, 128 or 256.
// Two rows for a lane, and kAhead tokens read ahead of their use: what is left of a token is its chain, a dot
// product of eight columns and log2(LPR) shuffles.
constexpr int kRowsPerLane = 2, kAhead = 4;

template <int LPR>
struct Scan {
    static constexpr int kThreads = LPR == 8 ? 64 : 128;
    static constexpr int kRows = kThreads / LPR * kRowsPerLane;      // value rows of a CTA: 16, 16 or 8, so it divides d_v
};

// One lane's eight columns of a row of dk: 4 l + {0..3}, and 4 LPR more.
template <int LPR>
__device__ __forceinline__ void ld_cols(const float* p, int dk, int l, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 4 * LPR * j + 4 * l;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < dk) u = *reinterpret_cast<const float4*>(p + c);
        x[4 * j] = u.x; x[4 * j + 1] = u.y; x[4 * j + 2] = u.z; x[4 * j + 3] = u.w;
    }
}
template <int LPR>
__device__ __forceinline__ void st_cols(float* p, int dk, int l, const float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 4 * LPR * j + 4 * l;
        if (c < dk) *reinterpret_cast<float4*>(p + c) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
}
// the dot product of a row, in every lane of it
template <int LPR>
__device__ __forceinline__ float row_dot(const float (&a)[8], const float (&b)[8]) {
    float s = a[0] * b[0], u = a[4] * b[4];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        s = fmaf(a[i], b[i], s);
        u = fmaf(a[4 + i], b[4 + i], u);
    }
    s += u;
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
}

struct Token {
    float k[8], q[8], v[kRowsPerLane], la, beta;
};

template <int LPR>
__device__ __forceinline__ void ld_token(const SeqArgs& a, const float* v, size_t ldv, size_t t, int h, int hk, int l, Token& x) {
    const SeqShape& sh = a.sh;
    ld_cols<LPR>(static_cast<const float*>(a.k) + t * sh.ldk + (size_t)hk * sh.dk, sh.dk, l, x.k);
    ld_cols<LPR>(static_cast<const float*>(a.q) + t * sh.ldq + (size_t)hk * sh.dk, sh.dk, l, x.q);
    const float2 u = *reinterpret_cast<const float2*>(v + t * ldv);
    x.v[0] = u.x;
    x.v[1] = u.y;
    x.la = a.la[t * sh.H + h];
    x.beta = a.beta[t * sh.H + h];
}

template <int LPR>
__global__ void __launch_bounds__(Scan<LPR>::kThreads) seq_scan_kernel(SeqArgs a, float* recS, float* eps) {
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / Scan<LPR>::kRows;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int l = threadIdx.x % LPR, row0 = tile * Scan<LPR>::kRows + threadIdx.x / LPR * kRowsPerLane, hk = h / (sh.H / sh.Hk);
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;
    const size_t head = ((size_t)s * sh.H + h) * sh.dv + row0;
    float S[kRowsPerLane][8];
#pragma unroll
    for (int r = 0; r < kRowsPerLane; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[r][i] = 0.f;
        if (a.S0 != nullptr) ld_cols<LPR>(a.S0 + (head + r) * sh.dk, sh.dk, l, S[r]);
    }
    const float* v = static_cast<const float*>(a.v) + (size_t)h * sh.dv + row0;
    const int slot0 = first / kChunk + s;
    Token x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (u < len) ld_token<LPR>(a, v, sh.ldv, (size_t)first + u, h, hk, l, x[u]);
    for (int i0 = 0; i0 < len; i0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= len) break;
            const size_t t = (size_t)first + i;
            if (recS != nullptr && i % kChunk == 0) {
                float* p = recS + (((size_t)(slot0 + i / kChunk) * sh.H + h) * sh.dv + row0) * sh.dk;
#pragma unroll
                for (int r = 0; r < kRowsPerLane; ++r) st_cols<LPR>(p + (size_t)r * sh.dk, sh.dk, l, S[r]);
            }
            const float ea = expf(gate_log(x[u].la));
            float e[kRowsPerLane], o[kRowsPerLane];
#pragma unroll
            for (int r = 0; r < kRowsPerLane; ++r) {
#pragma unroll
                for (int j = 0; j < 8; ++j) S[r][j] *= ea;
                e[r] = x[u].v[r] - row_dot<LPR>(S[r], x[u].k);
            }
#pragma unroll
            for (int r = 0; r < kRowsPerLane; ++r) {
                const float de = x[u].beta * e[r];
#pragma unroll
                for (int j = 0; j < 8; ++j) S[r][j] = fmaf(de, x[u].k[j], S[r][j]);
                o[r] = row_dot<LPR>(S[r], x[u].q);
            }
            if (l == 0) {
                const size_t at = (t * sh.H + h) * sh.dv + row0;
                *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(o[0], o[1]);
                if (eps != nullptr) *reinterpret_cast<float2*>(eps + at) = make_float2(e[0], e[1]);
            }
            if (i + kAhead < len) ld_token<LPR>(a, v, sh.ldv, t + kAhead, h, hk, l, x[u]);
        }
    }
    if (a.S_T != nullptr)
#pragma unroll
        for (int r = 0; r < kRowsPerLane; ++r) st_cols<LPR>(a.S_T + (head + r) * sh.dk, sh.dk, l, S[r]);
}

template <int LPR>
__global__ void __launch_bounds__(Scan<LPR>::kThreads) seq_scan_back_kernel(SeqArgs a, float* dSc, float* dVf) {
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / Scan<LPR>::kRows;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int l = threadIdx.x % LPR, row0 = tile * Scan<LPR>::kRows + threadIdx.x / LPR * kRowsPerLane, hk = h / (sh.H / sh.Hk);
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;
    const size_t head = ((size_t)s * sh.H + h) * sh.dv + row0, ldo = (size_t)sh.H * sh.dv;
    float S[kRowsPerLane][8];
#pragma unroll
    for (int r = 0; r < kRowsPerLane; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[r][i] = 0.f;
        if (a.dS_T != nullptr) ld_cols<LPR>(a.dS_T + (head + r) * sh.dk, sh.dk, l, S[r]);
    }
    const float* dout = static_cast<const float*>(a.dout) + (size_t)h * sh.dv + row0;
    const int slot0 = first / kChunk + s;
    Token x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (u < len) ld_token<LPR>(a, dout, ldo, (size_t)first + len - 1 - u, h, hk, l, x[u]);
    for (int i0 = len - 1; i0 >= 0; i0 -= kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 - u;
            if (i < 0) break;
            const size_t t = (size_t)first + i;
            if (i == len - 1 || i % kChunk == kChunk - 1) {
                float* p = dSc + (((size_t)(slot0 + i / kChunk) * sh.H + h) * sh.dv + row0) * sh.dk;
#pragma unroll
                for (int r = 0; r < kRowsPerLane; ++r) st_cols<LPR>(p + (size_t)r * sh.dk, sh.dk, l, S[r]);
            }
            const float ea = expf(gate_log(x[u].la));
            float w[kRowsPerLane];
#pragma unroll
            for (int r = 0; r < kRowsPerLane; ++r) {
#pragma unroll
                for (int j = 0; j < 8; ++j) S[r][j] = fmaf(x[u].v[r], x[u].q[j], S[r][j]);
                w[r] = x[u].beta * row_dot<LPR>(S[r], x[u].k);
#pragma unroll
                for (int j = 0; j < 8; ++j) S[r][j] = ea * fmaf(-w[r], x[u].k[j], S[r][j]);
            }
            if (l == 0) {
                const size_t at = (t * sh.H + h) * sh.dv + row0;
                *reinterpret_cast<float2*>(dVf + at) = make_float2(w[0], w[1]);
                *reinterpret_cast<float2*>(static_cast<float*>(a.dv) + at) = make_float2(w[0], w[1]);
            }
            if (i >= kAhead) ld_token<LPR>(a, dout, ldo, t - kAhead, h, hk, l, x[u]);
        }
    }
    if (a.dS0 != nullptr)
#pragma unroll
        for (int r = 0; r < kRowsPerLane; ++r) st_cols<LPR>(a.dS0 + (head + r) * sh.dk, sh.dk, l, S[r]);
}

// One CTA per (chunk, q/k head); the value heads of the group in turn, their dq and dk added in fp32 in that
// order.  All of it is products of 64 x 64 tiles in slices of 32 that go through shared memory; a thread
// keeps four rows and four columns of each product.
constexpr int kGradThreads = 256;
constexpr int kLdm = kChunk + 1;
constexpr int kSlice = 32, kLds = kChunk + 4;
constexpr int kSliceFloats = kSlice * kLds;
constexpr size_t kGradSmem = (5 * kSliceFloats + 3 * kChunk * kLdm + 6 * kChunk) * 4;

// 64 rows of `n` (at most 32) columns, turned: dst[column][row], zeros behind `rows` and `n`
__device__ __forceinline__ void slice_turned(float* dst, const float* src, size_t ld, int rows, int n) {
    for (int i = threadIdx.x; i < kChunk * kSlice / 4; i += kGradThreads) {
        const int r = i % kChunk, c = i / kChunk * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < n) x = *reinterpret_cast<const float4*>(src + r * ld + c);
        dst[c * kLds + r] = x.x;
        dst[(c + 1) * kLds + r] = x.y;
        dst[(c + 2) * kLds + r] = x.z;
        dst[(c + 3) * kLds + r] = x.w;
    }
}
// `rows` (at most 32) rows of n (at most 64) columns as they are, zeros behind both
__device__ __forceinline__ void slice_rows(float* dst, const float* src, size_t ld, int rows, int n) {
    for (int i = threadIdx.x; i < kChunk * kSlice / 4; i += kGradThreads) {
        const int r = i / 16, c = i % 16 * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < n) x = *reinterpret_cast<const float4*>(src + r * ld + c);
        *reinterpret_cast<float4*>(dst + r * kLds + c) = x;
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
    seq_grad_kernel(SeqArgs a, const float* recS, const float* eps, const float* dSc, const float* dVf, float* dqf,
                    float* dkf) {
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
    const int hk = blockIdx.x % sh.Hk, slot = blockIdx.x / sh.Hk, rep = sh.H / sh.Hk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ty = tid / 16 * 4, tx = tid % 16 * 4;
    int s, first, rows;
    if (!slot_chunk(sh, slot, s, first, rows, a.err)) return;
    const float* q = static_cast<const float*>(a.q) + (size_t)first * sh.ldq + (size_t)hk * sh.dk;
    const float* k = static_cast<const float*>(a.k) + (size_t)first * sh.ldk + (size_t)hk * sh.dk;
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const size_t ldo = (size_t)sh.H * sh.dv;
        const float* dout = static_cast<const float*>(a.dout) + (size_t)first * ldo + (size_t)h * sh.dv;
        const float* e = eps + (size_t)first * ldo + (size_t)h * sh.dv;
        const float* dV = dVf + (size_t)first * ldo + (size_t)h * sh.dv;
        const float* S = recS + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
        const float* dS = dSc + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
        __syncthreads();
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
            for (int c = 0; c < sh.dv; c += kSlice) {
                const int n = min(kSlice, sh.dv - c);
                slice_turned(X, dout + c, ldo, rows, n);
                slice_turned(Y, dV + c, ldo, rows, n);
                slice_turned(Z, e + c, ldo, rows, n);
                __syncthreads();
#pragma unroll 8
                for (int j = 0; j < kSlice; ++j) {
                    const float4 z = at4(Z + j * kLds + tx);
                    outer(at4(X + j * kLds + ty), z, e1);
                    outer(at4(Y + j * kLds + ty), z, e2);
                }
                __syncthreads();
            }
            for (int c = 0; c < sh.dk; c += kSlice) {
                const int n = min(kSlice, sh.dk - c);
                slice_turned(X, q + c, sh.ldq, rows, n);
                slice_turned(Y, k + c, sh.ldk, rows, n);
                __syncthreads();
#pragma unroll 8
                for (int j = 0; j < kSlice; ++j) {
                    const float4 z = at4(Y + j * kLds + tx);
                    outer(at4(X + j * kLds + ty), z, qk);
                    outer(at4(Y + j * kLds + ty), z, kk);
                }
                __syncthreads();
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
            for (int v = 0; v < sh.dv; v += kSlice) {
                const int nv = min(kSlice, sh.dv - v);
                slice_turned(X, dout + v, ldo, rows, nv);
                slice_turned(Y, dV + v, ldo, rows, nv);
                slice_turned(Z, e + v, ldo, rows, nv);
                slice_rows(U, S + (size_t)v * sh.dk + cb, sh.dk, nv, n);
                slice_rows(V, dS + (size_t)v * sh.dk + cb, sh.dk, nv, n);
                __syncthreads();
#pragma unroll 4
                for (int j = 0; j < kSlice; ++j) {
                    const float4 x = at4(U + j * kLds + tx), y = at4(V + j * kLds + tx);
                    outer(at4(X + j * kLds + ty), x, dq);
                    outer(at4(Y + j * kLds + ty), x, dr);
                    outer(at4(Z + j * kLds + ty), y, w2);
                }
                for (int j = tid; j < kSlice * kChunk; j += kGradThreads) {
                    const int at = j / kChunk * kLds + j % kChunk;
                    dot = fmaf(U[at], V[at], dot);
                }
                __syncthreads();
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
                slice_rows(U, q + (size_t)j0 * sh.ldq + cb, sh.ldq, rows - j0, n);
                slice_rows(V, k + (size_t)j0 * sh.ldk + cb, sh.ldk, rows - j0, n);
                __syncthreads();
#pragma unroll 4
                for (int j = 0; j < kSlice; ++j) {
                    const float4 x = at4(U + j * kLds + tx), y = at4(V + j * kLds + tx);
                    float p[4], m[4], pt[4], mt[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = MP[(ty + i) * kLdm + j0 + j];
                        m[i] = -ME[(ty + i) * kLdm + j0 + j];
                        pt[i] = MP[(j0 + j) * kLdm + ty + i];
                        mt[i] = -ME[(j0 + j) * kLdm + ty + i];
                    }
                    outer(p, y, dq);
                    outer(m, y, dr);
                    outer(pt, x, dw);
                    outer(mt, y, dw);
                }
                __syncthreads();
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
                    const size_t at = ((size_t)(first + t) * sh.Hk + hk) * sh.dk + cb + tx;
                    float4 oq = make_float4(gq[0], gq[1], gq[2], gq[3]), ok = make_float4(gk[0], gk[1], gk[2], gk[3]);
                    if (r > 0) {
                        const float4 pq = at4(dqf + at), pk = at4(dkf + at);
                        oq = make_float4(oq.x + pq.x, oq.y + pq.y, oq.z + pq.z, oq.w + pq.w);
                        ok = make_float4(ok.x + pk.x, ok.y + pk.y, ok.z + pk.z, ok.w + pk.w);
                    }
                    const bool last = r + 1 == rep;
                    *reinterpret_cast<float4*>((last ? static_cast<float*>(a.dq) : dqf) + at) = oq;
                    *reinterpret_cast<float4*>((last ? static_cast<float*>(a.dk) : dkf) + at) = ok;
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
}

template <int LPR>
cudaError_t forward_go(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / Scan<LPR>::kRows));
    float* S = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_S) : nullptr;
    float* e = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_eps) : nullptr;
    return launch_kernel(seq_scan_kernel<LPR>, dim3(grid), dim3(Scan<LPR>::kThreads), 0, st, false, a, S, e);
}

template <int LPR>
cudaError_t backward_go(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    static bool done[64];
    cudaError_t e = ensure_smem(seq_grad_kernel, kGradSmem, done);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / Scan<LPR>::kRows));
    float* dS = reinterpret_cast<float*>(a.ws + L.ws_dS);
    float* dV = reinterpret_cast<float*>(a.ws + L.ws_dV);
    e = launch_kernel(seq_scan_back_kernel<LPR>, dim3(grid), dim3(Scan<LPR>::kThreads), 0, st, false, a, dS, dV);
    if (e != cudaSuccess || a.sh.total == 0) return e;
    return launch_kernel(seq_grad_kernel, dim3((unsigned)((size_t)seq_slots(a.sh.nseq, a.sh.total) * a.sh.Hk)),
                         dim3(kGradThreads), kGradSmem, st, false, a,
                         (const float*)(a.rec + L.rec_S), (const float*)(a.rec + L.rec_eps), (const float*)dS,
                         (const float*)dV, reinterpret_cast<float*>(a.ws + L.ws_dq),
                         reinterpret_cast<float*>(a.ws + L.ws_dk));
}

}  // namespace

// also a bf16 call without tokens, which copies the state and reads nothing of bf16
cudaError_t launch_seq_forward_simt(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    return a.sh.dk <= 64 ? forward_go<8>(a, L, st) : a.sh.dk <= 128 ? forward_go<16>(a, L, st) : forward_go<32>(a, L, st);
}

cudaError_t launch_seq_backward_simt(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    return a.sh.dk <= 64 ? backward_go<8>(a, L, st) : a.sh.dk <= 128 ? backward_go<16>(a, L, st) : backward_go<32>(a, L, st);
}

SeqLayout seq_layout(const SeqShape& s, int dtype) {
    SeqLayout L = {};
    const bool tc = seq_tc_takes(dtype);
    const size_t slots = seq_slots(s.nseq, s.total), state = slots * s.H * (tc ? seq_tc_dk(s.dk) : s.dk) * s.dv * 4;
    // the tensor-core kernels keep rows of tokens for whole chunks
    const size_t rows = (tc ? slots * kChunk : (size_t)s.total) * s.H * s.dv * 4;
    const size_t heads = s.H > s.Hk ? (size_t)s.total * s.Hk * s.dk * 4 : 0;
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
// gates and offsets are read one by one: any row of a larger tensor will do
bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dim_ok(int d) { return d >= 16 && d <= kMaxDim && d % 16 == 0; }

bool shape_ok(const SeqShape& s) {
    if (s.nseq < 1 || s.total < 0 || s.H < 1 || s.Hk < 1 || s.H % s.Hk != 0 || !dim_ok(s.dk) || !dim_ok(s.dv)) return false;
    if ((long long)s.nseq + s.total > (1LL << 30)) return false;
    // grid sizes: (sequence, head, 8 value rows) and (chunk slot, head)
    return (long long)s.nseq * s.H * (s.dv / 8) <= 0x7fffffffLL &&
           (long long)seq_slots(s.nseq, s.total) * s.H <= 0x7fffffffLL;
}

bool strides_ok(const SeqShape& s, int dtype) {
    const int unit = 16 / elem_bytes(dtype);
    return s.ldq >= s.Hk * s.dk && s.ldk >= s.Hk * s.dk && s.ldv >= s.H * s.dv && s.ldq % unit == 0 &&
           s.ldk % unit == 0 && s.ldv % unit == 0;
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
    if (!aligned16(S0) || !aligned16(S_T) || !aligned16(record) || !words(offsets) || !given(workspace)) return GDN_ERR_ARG;
    if (total > 0 && (!given(q) || !given(k) || !given(v) || log_alpha == nullptr || !words(log_alpha) || beta == nullptr || !words(beta) || !given(out)))
        return GDN_ERR_ARG;
    const SeqLayout L = seq_layout(s, dtype);
    const size_t e = elem_bytes(dtype), vo = (size_t)total * H * dv * e, gb = (size_t)total * H * 4,
                 sb = (size_t)nseq * H * dv * dk * 4;
    const Span w[] = {{out, vo}, {record, L.rec_total}, {workspace, L.ws_total}, {S_T, sb}};
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
    const bool tc = total > 0 && seq_tc_takes(dtype);
    const cudaError_t rc = tc ? launch_seq_forward_tc(a, stream) : launch_seq_forward_simt(a, dtype, stream);
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
    if (!aligned16(dS_T) || !aligned16(dS0) || !words(offsets) || !given(workspace) || !given(record)) return GDN_ERR_ARG;
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
    const bool tc = total > 0 && seq_tc_takes(dtype);
    const cudaError_t rc = tc ? launch_seq_backward_tc(a, stream) : launch_seq_backward_simt(a, dtype, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

// gdn_seq.cu -- the gated delta rule over packed sequences: entry points, layouts, and the
// CUDA-core kernels that serve fp32 inputs and the head sizes that the tensor-core kernels
// do not take.
//
//   S' = e^{la_t} S_{t-1},  eps_t = v_t - S' k_t,  S_t = S' + beta_t eps_t k_t^T,  o_t = S_t q_t
//
// Forward, token by token: each row of S (one value index) is independent, so a warp keeps four
// rows in registers and needs one dot product with k_t, one with q_t for each row and token.
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

constexpr int kScanRows = 16;     // value rows per CTA of the token-serial scans: four warps of four

// One lane's eight columns of a row of dk: 4 lane + {0..3} and 128 more.
template <typename T>
__device__ __forceinline__ void ld_cols(const T* p, int dk, int lane, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 128 * j + 4 * lane;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < dk) u = ld4<T>(p, c);
        x[4 * j] = u.x; x[4 * j + 1] = u.y; x[4 * j + 2] = u.z; x[4 * j + 3] = u.w;
    }
}
__device__ __forceinline__ void st_cols(float* p, int dk, int lane, const float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 128 * j + 4 * lane;
        if (c < dk) *reinterpret_cast<float4*>(p + c) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
}
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
    return s;
}

template <typename T>
__global__ void __launch_bounds__(128) seq_scan_kernel(SeqArgs a, float* recS, float* eps) {
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / kScanRows;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * kScanRows + warp * 4, hk = h / (sh.H / sh.Hk);
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;
    const size_t head = ((size_t)s * sh.H + h) * sh.dv + row0;
    float S[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[r][i] = 0.f;
        if (a.S0 != nullptr) ld_cols(a.S0 + (head + r) * sh.dk, sh.dk, lane, S[r]);
    }
    const T* q = static_cast<const T*>(a.q) + (size_t)hk * sh.dk;
    const T* k = static_cast<const T*>(a.k) + (size_t)hk * sh.dk;
    const T* v = static_cast<const T*>(a.v) + (size_t)h * sh.dv + row0;
    const int slot0 = first / kChunk + s;
    for (int i = 0; i < len; ++i) {
        const size_t t = (size_t)first + i;
        if (recS != nullptr && i % kChunk == 0) {
            float* p = recS + (((size_t)(slot0 + i / kChunk) * sh.H + h) * sh.dv + row0) * sh.dk;
#pragma unroll
            for (int r = 0; r < 4; ++r) st_cols(p + (size_t)r * sh.dk, sh.dk, lane, S[r]);
        }
        float kt[8], qt[8], d[4];
        ld_cols(k + t * sh.ldk, sh.dk, lane, kt);
        ld_cols(q + t * sh.ldq, sh.dk, lane, qt);
        const float4 vt = ld4<T>(v + t * sh.ldv, 0);
        const float ea = expf(gate_log(a.la[t * sh.H + h])), b = a.beta[t * sh.H + h];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < 8; ++j) S[r][j] *= ea;
            d[r] = warp_sum(dot8(S[r], kt));
        }
        const float e[4] = {vt.x - d[0], vt.y - d[1], vt.z - d[2], vt.w - d[3]};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float de = b * e[r];
#pragma unroll
            for (int j = 0; j < 8; ++j) S[r][j] = fmaf(de, kt[j], S[r][j]);
            d[r] = warp_sum(dot8(S[r], qt));
        }
        if (lane < 4) {
            const float o = lane == 0 ? d[0] : lane == 1 ? d[1] : lane == 2 ? d[2] : d[3];
            st_elem<T>(static_cast<T*>(a.out), (t * sh.H + h) * sh.dv + row0 + lane, o);
            if (eps != nullptr)
                eps[(t * sh.H + h) * sh.dv + row0 + lane] = lane == 0 ? e[0] : lane == 1 ? e[1] : lane == 2 ? e[2] : e[3];
        }
    }
    if (a.S_T != nullptr)
#pragma unroll
        for (int r = 0; r < 4; ++r) st_cols(a.S_T + (head + r) * sh.dk, sh.dk, lane, S[r]);
}

template <typename T>
__global__ void __launch_bounds__(128) seq_scan_back_kernel(SeqArgs a, float* dSc, float* dVf) {
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / kScanRows;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * kScanRows + warp * 4, hk = h / (sh.H / sh.Hk);
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;
    const size_t head = ((size_t)s * sh.H + h) * sh.dv + row0;
    float S[4][8];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) S[r][i] = 0.f;
        if (a.dS_T != nullptr) ld_cols(a.dS_T + (head + r) * sh.dk, sh.dk, lane, S[r]);
    }
    const T* q = static_cast<const T*>(a.q) + (size_t)hk * sh.dk;
    const T* k = static_cast<const T*>(a.k) + (size_t)hk * sh.dk;
    const T* dout = static_cast<const T*>(a.dout) + (size_t)h * sh.dv + row0;
    const int slot0 = first / kChunk + s;
    for (int i = len - 1; i >= 0; --i) {
        const size_t t = (size_t)first + i;
        if (i == len - 1 || i % kChunk == kChunk - 1) {
            float* p = dSc + (((size_t)(slot0 + i / kChunk) * sh.H + h) * sh.dv + row0) * sh.dk;
#pragma unroll
            for (int r = 0; r < 4; ++r) st_cols(p + (size_t)r * sh.dk, sh.dk, lane, S[r]);
        }
        float kt[8], qt[8], w[4];
        ld_cols(k + t * sh.ldk, sh.dk, lane, kt);
        ld_cols(q + t * sh.ldq, sh.dk, lane, qt);
        const float4 ot = ld4<T>(dout + t * sh.H * sh.dv, 0);
        const float o4[4] = {ot.x, ot.y, ot.z, ot.w};
        const float ea = expf(gate_log(a.la[t * sh.H + h])), b = a.beta[t * sh.H + h];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < 8; ++j) S[r][j] = fmaf(o4[r], qt[j], S[r][j]);
            w[r] = b * warp_sum(dot8(S[r], kt));
#pragma unroll
            for (int j = 0; j < 8; ++j) S[r][j] = ea * fmaf(-w[r], kt[j], S[r][j]);
        }
        if (lane < 4) {
            const float x = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
            const size_t at = (t * sh.H + h) * sh.dv + row0 + lane;
            dVf[at] = x;
            st_elem<T>(static_cast<T*>(a.dv), at, x);
        }
    }
    if (a.dS0 != nullptr)
#pragma unroll
        for (int r = 0; r < 4; ++r) st_cols(a.dS0 + (head + r) * sh.dk, sh.dk, lane, S[r]);
}

// One CTA per (chunk, q/k head); the value heads of the group in turn, their dq and dk added in
// fp32 in that order.
constexpr int kGradThreads = 256;
constexpr int kLdm = kChunk + 1;
constexpr size_t kGradSmem = (3 * kChunk * kLdm + 6 * kChunk) * 4;

template <typename T>
__global__ void __launch_bounds__(kGradThreads)
    seq_grad_kernel(SeqArgs a, const float* recS, const float* eps, const float* dSc, const float* dVf, float* dqf,
                    float* dkf) {
    extern __shared__ float sm[];
    float* MP = sm;                          // G beta (dO.eps)
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int s, first, rows;
    if (!slot_chunk(sh, slot, s, first, rows, a.err)) return;
    const T* q = static_cast<const T*>(a.q) + (size_t)first * sh.ldq + (size_t)hk * sh.dk;
    const T* k = static_cast<const T*>(a.k) + (size_t)first * sh.ldk + (size_t)hk * sh.dk;
    for (int r = 0; r < rep; ++r) {
        const int h = hk * rep + r;
        const T* dout = static_cast<const T*>(a.dout) + ((size_t)first * sh.H + h) * sh.dv;
        const float* e = eps + ((size_t)first * sh.H + h) * sh.dv;
        const float* dV = dVf + ((size_t)first * sh.H + h) * sh.dv;
        const size_t ldo = (size_t)sh.H * sh.dv;
        const float* S = recS + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
        const float* dS = dSc + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
        __syncthreads();
        if (tid == 0) {
            double g = 0.0;
            for (int t = 0; t < rows; ++t) {
                g += (double)gate_log(a.la[((size_t)first + t) * sh.H + h]);
                ghi[t] = (float)g;
                glo[t] = (float)(g - (double)ghi[t]);
            }
        }
        if (tid < rows) bt[tid] = a.beta[((size_t)first + tid) * sh.H + h];
        __syncthreads();
        for (int i = tid; i < kChunk * kChunk; i += kGradThreads) {
            const int t = i / kChunk, j = i % kChunk;
            float mp = 0.f, me = 0.f, mb = 0.f;
            if (t < rows && j <= t) {
                float e1 = 0.f, e2 = 0.f, qk = 0.f, kk = 0.f;
                for (int c = 0; c < sh.dv; c += 4) {
                    const float4 x = ld4<T>(dout + t * ldo, c), y = ld4<float>(e + j * ldo, c), z = ld4<float>(dV + t * ldo, c);
                    e1 += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
                    e2 += z.x * y.x + z.y * y.y + z.z * y.z + z.w * y.w;
                }
                for (int c = 0; c < sh.dk; c += 4) {
                    const float4 x = ld4<T>(q + (size_t)t * sh.ldq, c), y = ld4<T>(k + (size_t)j * sh.ldk, c),
                                 z = ld4<T>(k + (size_t)t * sh.ldk, c);
                    qk += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
                    kk += z.x * y.x + z.y * y.y + z.z * y.z + z.w * y.w;
                }
                const float G = expf((ghi[t] - ghi[j]) + (glo[t] - glo[j]));
                mp = G * bt[j] * e1;
                mb = G * qk * e1;
                if (j < t) {
                    me = G * bt[j] * e2;
                    mb -= G * kk * e2;
                }
            }
            MP[t * kLdm + j] = mp;
            ME[t * kLdm + j] = me;
            MB[t * kLdm + j] = mb;
        }
        __syncthreads();
        const float gend_hi = ghi[rows - 1], gend_lo = glo[rows - 1];
        for (int t = warp; t < rows; t += kGradThreads / 32) {
            float xq = 0.f, xu = 0.f;
            const float eg = expf(ghi[t] + glo[t]), et = expf((gend_hi - ghi[t]) + (gend_lo - glo[t]));
            for (int c = lane; c < sh.dk; c += 32) {
                float sq = 0.f, sr = 0.f, w2 = 0.f, dq = 0.f, dr = 0.f, dw = 0.f;
                for (int v = 0; v < sh.dv; ++v) {
                    const float Sv = S[(size_t)v * sh.dk + c];
                    sq = fmaf(ld_elem<T>(dout + t * ldo, v), Sv, sq);
                    sr = fmaf(dV[t * ldo + v], Sv, sr);
                    w2 = fmaf(e[t * ldo + v], dS[(size_t)v * sh.dk + c], w2);
                }
                w2 *= et;
                for (int j = 0; j <= t; ++j) {
                    const float kj = ld_elem<T>(k + (size_t)j * sh.ldk, c);
                    dq = fmaf(MP[t * kLdm + j], kj, dq);
                    dr = fmaf(ME[t * kLdm + j], kj, dr);
                }
                for (int j = t; j < rows; ++j) {
                    dw = fmaf(MP[j * kLdm + t], ld_elem<T>(q + (size_t)j * sh.ldq, c), dw);
                    dw = fmaf(-ME[j * kLdm + t], ld_elem<T>(k + (size_t)j * sh.ldk, c), dw);
                }
                dq = fmaf(eg, sq, dq);
                dr = -fmaf(eg, sr, dr);
                const float qc = ld_elem<T>(q + (size_t)t * sh.ldq, c), kc = ld_elem<T>(k + (size_t)t * sh.ldk, c);
                xq += qc * dq + kc * (dr - dw);
                xu = fmaf(kc, w2, xu);
                float dkc = dr + dw + bt[t] * w2;
                const size_t at = ((size_t)(first + t) * sh.Hk + hk) * sh.dk + c;
                if (rep > 1) {
                    if (r > 0) {
                        dq += dqf[at];
                        dkc += dkf[at];
                    }
                    dqf[at] = dq;
                    dkf[at] = dkc;
                }
                if (r == rep - 1) {
                    st_elem<T>(static_cast<T*>(a.dq), at, dq);
                    st_elem<T>(static_cast<T*>(a.dk), at, dkc);
                }
            }
            xq = warp_sum(xq);
            xu = warp_sum(xu);
            if (lane == 0) {
                xs[t] = xq;
                us[t] = xu;
            }
        }
        float dot = 0.f;
        for (int i = tid; i < sh.dv * sh.dk; i += kGradThreads) dot = fmaf(S[i], dS[i], dot);
        dot = warp_sum(dot);
        if (lane == 0) red[warp] = dot;
        __syncthreads();
        if (tid < rows) {
            const size_t at = ((size_t)first + tid) * sh.H + h;
            double z = 0.0;
            for (int w = 0; w < kGradThreads / 32; ++w) z += (double)red[w];
            z *= (double)expf(gend_hi + gend_lo);
            for (int t = 0; t < rows; ++t) z += t < tid ? (double)bt[t] * us[t] : (double)xs[t];
            a.dla[at] = (float)z;
            double db = us[tid];
            for (int t = tid; t < rows; ++t) db += MB[t * kLdm + tid];
            a.dbeta[at] = (float)db;
        }
    }
}

template <typename T>
cudaError_t forward_simt(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / kScanRows));
    float* S = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_S) : nullptr;
    float* e = a.rec ? reinterpret_cast<float*>(a.rec + L.rec_eps) : nullptr;
    return launch_kernel(seq_scan_kernel<T>, dim3(grid), dim3(128), 0, st, false, a, S, e);
}

template <typename T>
cudaError_t backward_simt(const SeqArgs& a, const SeqLayout& L, cudaStream_t st) {
    static bool done[64];
    cudaError_t e = ensure_smem(seq_grad_kernel<T>, kGradSmem, done);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / kScanRows));
    float* dS = reinterpret_cast<float*>(a.ws + L.ws_dS);
    float* dV = reinterpret_cast<float*>(a.ws + L.ws_dV);
    e = launch_kernel(seq_scan_back_kernel<T>, dim3(grid), dim3(128), 0, st, false, a, dS, dV);
    if (e != cudaSuccess || a.sh.total == 0) return e;
    return launch_kernel(seq_grad_kernel<T>, dim3((unsigned)((size_t)seq_slots(a.sh.nseq, a.sh.total) * a.sh.Hk)),
                         dim3(kGradThreads), kGradSmem, st, false, a,
                         (const float*)(a.rec + L.rec_S), (const float*)(a.rec + L.rec_eps), (const float*)dS,
                         (const float*)dV, reinterpret_cast<float*>(a.ws + L.ws_dq),
                         reinterpret_cast<float*>(a.ws + L.ws_dk));
}

}  // namespace

cudaError_t launch_seq_forward_simt(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    return dtype == GDN_DTYPE_F32 ? forward_simt<float>(a, L, st) : forward_simt<__nv_bfloat16>(a, L, st);
}

cudaError_t launch_seq_backward_simt(const SeqArgs& a, int dtype, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, dtype);
    return dtype == GDN_DTYPE_F32 ? backward_simt<float>(a, L, st) : backward_simt<__nv_bfloat16>(a, L, st);
}

SeqLayout seq_layout(const SeqShape& s, int dtype) {
    SeqLayout L = {};
    const bool tc = seq_tc_takes(s, dtype);
    const size_t slots = seq_slots(s.nseq, s.total), state = slots * s.H * s.dk * s.dv * 4;
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
    // grid sizes: (sequence, head, 16 value rows) and (chunk slot, head)
    return (long long)s.nseq * s.H * (s.dv / 16) <= 0x7fffffffLL &&
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
    const bool tc = total > 0 && seq_tc_takes(s, dtype);
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
    const bool tc = total > 0 && seq_tc_takes(s, dtype);
    const cudaError_t rc = tc ? launch_seq_backward_tc(a, stream) : launch_seq_backward_simt(a, dtype, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

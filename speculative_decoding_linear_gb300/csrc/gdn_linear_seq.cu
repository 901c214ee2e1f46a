// gdn_linear_seq.cu -- decay-gated linear attention over packed sequences: entry points, the scan over
// segments, and the kernels of fp32 inputs.
//
// fp32 inputs: segments of 64 tokens, four kinds of kernels
//   lin_local_kernel   C = sum_t c_t a_t b_t^T of a segment, 64 x 64 tiles of the state
//   lin_scan_kernel    the states (or their gradients) between the segments
//   lin_rows_kernel    64 rows of o, dq, dk or dv: the state's product, the masked scores, and their product
//   lin_gates_kernel   dlog_alpha and dbeta
// All products are fp32 on the CUDA cores, in 64 x 64 tiles of four by four values a thread: fp32 inputs carried
// as bf16 terms would take six to nine products on the tensor core for each of these.
// 8192 tokens of 8 heads, 256 x 256: forward 1.13 ms, backward 2.36; 4 x 2048, 64 x 64: 0.10 and 0.29; bound by shared memory's reads,
// two of 16 bytes for 16 multiply-adds.
#include "gdn_checks.cuh"
#include "gdn_linear.cuh"

namespace gdn {
namespace {

constexpr int kSegF = 64;                   // tokens of a segment
constexpr int kT = 256;                     // threads
constexpr int kK = 32;                      // depth of a staged tile
constexpr int kLd = 68;                     // floats from one staged row to the next

struct Mat {                                // element (r, c) is p[r ld + c]; zero outside rows x cols
    const float* p;
    size_t ld;
    int rows, cols;
    __device__ __forceinline__ float4 at(int r, int c) const {        // cols and c are multiples of four
        return r < rows && c < cols ? ld4<float>(p + (size_t)r * ld, c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
};

// A thread's part of a piece of 64 x 32 on its way to shared memory: it is fetched while the piece before it is multiplied.
constexpr int kPart = 64 * kK / 4 / kT;
struct Part {
    float4 x[kPart];
};
// s[k][m] of a piece whose k index runs along the row, from column k0 on
__device__ __forceinline__ Part fetch_k(const Mat& m, int k0) {
    Part p;
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
        const int i = threadIdx.x + j * kT;
        p.x[j] = m.at(i / (kK / 4), k0 + i % (kK / 4) * 4);
    }
    return p;
}
__device__ __forceinline__ void put_k(float (*s)[kLd], const Part& p) {
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
        const int i = threadIdx.x + j * kT, r = i / (kK / 4), k = i % (kK / 4) * 4;
        s[k][r] = p.x[j].x;
        s[k + 1][r] = p.x[j].y;
        s[k + 2][r] = p.x[j].z;
        s[k + 3][r] = p.x[j].w;
    }
}
// s[k][n] of a piece whose n index runs along the row, from row k0 on; its rows scaled
__device__ __forceinline__ Part fetch_n(const Mat& m, int k0) {
    Part p;
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
        const int i = threadIdx.x + j * kT;
        p.x[j] = m.at(k0 + i / 16, i % 16 * 4);
    }
    return p;
}
__device__ __forceinline__ void put_n(float (*s)[kLd], const Part& p, const float* scale = nullptr) {
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
        const int i = threadIdx.x + j * kT, k = i / 16, n = i % 16 * 4;
        const float f = scale != nullptr ? scale[k] : 1.f;
        *reinterpret_cast<float4*>(&s[k][n]) = scale != nullptr ? make_float4(f * p.x[j].x, f * p.x[j].y, f * p.x[j].z, f * p.x[j].w) : p.x[j];
    }
}

using Acc = float[4][4];
__device__ __forceinline__ void clear(Acc& c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i / 4][i % 4] = 0.f;
}
__device__ __forceinline__ void tile_mul(Acc& c, const float (*a)[kLd], const float (*b)[kLd]) {
    const int m = threadIdx.x / 16 * 4, n = threadIdx.x % 16 * 4;
#pragma unroll 8
    for (int k = 0; k < kK; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(&a[k][m]), y = *reinterpret_cast<const float4*>(&b[k][n]);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
    }
}

struct alignas(16) Stage {               // read by 16 bytes
    float a[kK][kLd], b[kK][kLd];
};
// c += A B^T, both with k along the row; A B with `along_n`
template <bool along_n>
__device__ __forceinline__ Part fetch_b(const Mat& B, int k) { return along_n ? fetch_n(B, k) : fetch_k(B, k); }
template <bool along_n>              // a and b: the first pieces
__device__ __forceinline__ void product(Acc& c, Stage& s, const Mat& A, const Mat& B, int K, Part a, Part b) {
    for (int k = 0; k < K; k += kK) {
        __syncthreads();
        put_k(s.a, a);
        if (along_n) put_n(s.b, b); else put_k(s.b, b);
        __syncthreads();
        if (k + kK < K) {
            a = fetch_k(A, k + kK);
            b = fetch_b<along_n>(B, k + kK);
        }
        tile_mul(c, s.a, s.b);
    }
}

// Gates of a segment's tokens, in shared memory.
struct Gates {
    float hi[kSegF], lo[kSegF], beta[kSegF], head[kSegF], tail[kSegF];      // head e^{g_t}, tail e^{G - g_t}
    float end;                                                              // e^G
};
__device__ void load_gates(Gates& g, const SeqArgs& a, int first, int rows, int h) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        LogSum x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 2 * lane + j;
            x[j] = {t < rows ? gate_log(a.la[(size_t)(first + t) * a.sh.H + h]) : 0.f, 0.f};
            g.beta[t] = t < rows ? a.beta[(size_t)(first + t) * a.sh.H + h] : 0.f;
        }
        x[1] = x[1] + x[0];
        const LogSum all = warp_scan(x[1]), upto = all - x[1], end = {__shfl_sync(0xffffffffu, all.hi, 31), __shfl_sync(0xffffffffu, all.lo, 31)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = 2 * lane + j;
            const LogSum p = upto + x[j];
            g.hi[t] = p.hi;
            g.lo[t] = p.lo;
            g.head[t] = decay_of(p);
            g.tail[t] = decay_of(end - p);
        }
        if (lane == 0) g.end = decay_of(end);
    }
    __syncthreads();
}
// e^{g_t - g_s}, s <= t: sums of log decays do not grow, so the larger one's rounding error of their difference is had by two operations
__device__ __forceinline__ float decay(const Gates& g, int t, int s) {
    const float d = g.hi[t] - g.hi[s], off = (d - g.hi[t]) + g.hi[s], e = expf(d);
    return fmaf(e, (g.lo[t] - g.lo[s]) - off, e);
}

__device__ __forceinline__ Mat token_rows(const void* p, size_t ld, int first, int rows, int head, int d) {
    return {static_cast<const float*>(p) + (size_t)first * ld + (size_t)head * d, ld, rows, d};
}
__device__ __forceinline__ Mat columns(const Mat& m, int c0) { return {m.p + c0, m.ld, m.rows, m.cols - c0}; }

// ---------------------------------------------------------------------------
// what a segment adds to the state: sum_t beta_t e^{G - g_t} v_t k_t^T; or, BACK, to the gradient of the
// state: sum_t e^{g_t} dO_t q_t^T.  One CTA a 64 x 64 tile.
// ---------------------------------------------------------------------------
template <bool BACK>
__global__ void __launch_bounds__(kT) lin_local_kernel(SeqArgs a, float* local, float* gend) {
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    const int slot = blockIdx.x / sh.H, h = blockIdx.x % sh.H, hk = h / (sh.H / sh.Hk);
    const int tiles_k = (sh.dk + 63) / 64, r0 = blockIdx.y / tiles_k * 64, c0 = blockIdx.y % tiles_k * 64;
    int s, c, first, rows;
    if (!slot_segment(sh, kSegF, slot, s, c, first, rows, a.err)) return;
    __shared__ Gates g;
    __shared__ Stage st;
    __shared__ float w[kSegF];
    const Mat A = columns(token_rows(BACK ? a.dout : a.v, BACK ? (size_t)sh.H * sh.dv : sh.ldv, first, rows, h, sh.dv), r0);
    const Mat B = columns(token_rows(BACK ? a.q : a.k, BACK ? sh.ldq : sh.ldk, first, rows, hk, sh.dk), c0);
    Part x = fetch_n(A, 0), y = fetch_n(B, 0);            // on their way beside the gates
    load_gates(g, a, first, rows, h);
    if (threadIdx.x < kSegF) w[threadIdx.x] = BACK ? g.head[threadIdx.x] : g.beta[threadIdx.x] * g.tail[threadIdx.x];
    if (threadIdx.x == 0 && blockIdx.y == 0) gend[(size_t)slot * sh.H + h] = g.end;
    Acc acc;
    clear(acc);
    for (int k = 0; k < kSegF; k += kK) {
        __syncthreads();
        put_n(st.a, x, w + k);
        put_n(st.b, y);
        __syncthreads();
        if (k + kK < kSegF) {
            x = fetch_n(A, k + kK);
            y = fetch_n(B, k + kK);
        }
        tile_mul(acc, st.a, st.b);
    }
    const int m = r0 + threadIdx.x / 16 * 4, n = c0 + threadIdx.x % 16 * 4;
    float* out = local + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m + i < sh.dv && n < sh.dk)
            *reinterpret_cast<float4*>(out + (size_t)(m + i) * sh.dk + n) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

// ---------------------------------------------------------------------------
// 64 rows of o, dq, dk or dv, 64 columns a CTA.  Rows and scores:
//   kOut  W_ts = beta_s e^{g_t - g_s} (q_t.k_s)   o_t  = e^{g_t} S q_t + sum_s W_ts v_s
//   kDq   W_ts = beta_s e^{g_t - g_s} (dO_t.v_s)  dq_t = e^{g_t} S^T dO_t + sum_s W_ts k_s
//   kDk   W_st = e^{g_t - g_s} (v_s.dO_t)         dk_s = beta_s (e^{G - g_s} dS^T v_s + sum_t W_st q_t)
//   kDv   W_st = e^{g_t - g_s} (k_s.q_t)          dv_s = beta_s (e^{G - g_s} dS k_s + sum_t W_st dO_t)
// dq and dk are summed over the value heads that share them.  part: this tile's columns of q_t.(e^{g_t} S^T dO_t)
// (kDq) and v_s.(e^{G - g_s} dS k_s) (kDv), [slot][H][tile][64].
// ---------------------------------------------------------------------------
enum { kOut, kDq, kDk, kDv };

template <int MODE>
__global__ void __launch_bounds__(kT) lin_rows_kernel(SeqArgs a, const float* states, float* part) {
    constexpr bool keys = MODE == kDk || MODE == kDv, value_cols = MODE == kOut || MODE == kDv;
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    const int rep = sh.H / sh.Hk, heads = value_cols ? sh.H : sh.Hk, dx = value_cols ? sh.dv : sh.dk, dc = value_cols ? sh.dk : sh.dv;
    const int slot = blockIdx.x / heads, head = blockIdx.x % heads, n0 = blockIdx.y * 64;
    void* out = MODE == kOut ? a.out : MODE == kDq ? a.dq : MODE == kDk ? a.dk : a.dv;
    int ob, oe;
    if (blockIdx.y == 0 && seq_outside(sh, ob, oe)) zero_rows<float>(out, (size_t)heads * dx, ob, oe, sh.total);
    int s, c, first, rows;
    if (!slot_segment(sh, kSegF, slot, s, c, first, rows, a.err)) return;
    __shared__ Gates g;
    __shared__ Stage st;
    __shared__ alignas(16) float w[kSegF][kLd];
    const int m = threadIdx.x / 16 * 4, n = threadIdx.x % 16 * 4;
    const size_t ldo = (size_t)sh.H * sh.dv;
    Acc acc;
    clear(acc);
    for (int r = 0; r < (value_cols ? 1 : rep); ++r) {
        const int h = value_cols ? head : head * rep + r, hk = value_cols ? head / rep : head;
        const Mat q = token_rows(a.q, sh.ldq, first, rows, hk, sh.dk), k = token_rows(a.k, sh.ldk, first, rows, hk, sh.dk),
                  v = token_rows(a.v, sh.ldv, first, rows, h, sh.dv), o = token_rows(a.dout, ldo, first, rows, h, sh.dv);
        const Mat A = MODE == kOut ? q : MODE == kDq ? o : MODE == kDk ? v : k, B = MODE == kOut ? k : MODE == kDq ? v : MODE == kDk ? o : q,
                  X = columns(MODE == kOut ? v : MODE == kDq ? k : MODE == kDk ? q : o, n0);
        const float* S = states + ((size_t)slot * sh.H + h) * sh.dv * sh.dk;
        const Mat M = {S + (value_cols ? (size_t)n0 * sh.dk : (size_t)n0), (size_t)sh.dk, value_cols ? sh.dv - n0 : sh.dv, value_cols ? sh.dk : sh.dk - n0};
        Part pa = fetch_k(A, 0), pb = fetch_b<!value_cols>(M, 0);     // on their way beside the gates
        __syncthreads();
        load_gates(g, a, first, rows, h);
        Acc y;
        clear(y);
        product<!value_cols>(y, st, A, M, dc, pa, pb);
        pa = fetch_k(A, 0);
        pb = fetch_k(B, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = keys ? g.tail[m + i] : g.head[m + i], b = keys ? g.beta[m + i] : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[i][j] *= f;
                acc[i][j] = fmaf(b, y[i][j], acc[i][j]);
            }
        }
        if (MODE == kDq || MODE == kDv) {       // these columns' share of the row's dot with q or v
            const Mat z = columns(MODE == kDq ? q : v, n0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 zi = z.at(m + i, n);
                float d = y[i][0] * zi.x + y[i][1] * zi.y + y[i][2] * zi.z + y[i][3] * zi.w;
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
                if (threadIdx.x % 16 == 0)
                    part[(((size_t)slot * sh.H + h) * gridDim.y + blockIdx.y) * kSegF + m + i] = d;
            }
        }
        clear(y);
        Part x = fetch_n(X, 0);
        product<false>(y, st, A, B, dc, pa, pb);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = m + i, col = n + j;
                float f = 0.f;
                if (row < rows && col < rows && (keys ? col >= row : col <= row))
                    f = y[i][j] * (keys ? g.beta[row] * decay(g, col, row) : g.beta[col] * decay(g, row, col));
                w[col][row] = f;
            }
        for (int k0 = 0; k0 < kSegF; k0 += kK) {
            __syncthreads();
            put_n(st.b, x);
            __syncthreads();
            if (k0 + kK < kSegF) x = fetch_n(X, k0 + kK);
            tile_mul(acc, w + k0, st.b);
        }
    }
    float* p = static_cast<float*>(out) + ((size_t)first * heads + head) * dx;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m + i < rows && n0 + n + j < dx) p[(size_t)(m + i) * heads * dx + n0 + n + j] = acc[i][j];
}

// ---------------------------------------------------------------------------
// Gradients of the gates of one (segment, head).  With E_ts = beta_s e^{g_t - g_s} (q_t.k_s) (dO_t.v_s), s < t:
//   dlog_alpha_u = sum_{s < u <= t} E_ts + sum_{t >= u} q_t.(e^{g_t} S^T dO_t) + sum_{s < u} beta_s v_s.(e^{G - g_s} dS k_s) + e^G <dS, S>
//   dbeta_s      = sum_{t >= s} E_ts / beta_s + v_s.(e^{G - g_s} dS k_s)
// The first sum is taken as it stands, nothing cancels: each row's running sum over s, then the sum over rows t from u on of the
// row's sum before u (rows minus columns from u on: 301 tokens 4.3e-7 of dlog_alpha off, 2.2e-7 so, in the same time).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kT) lin_gates_kernel(SeqArgs a, const float* part_q, int tiles_q, const float* part_k, int tiles_k,
                                                       const float* phi, int tiles_phi) {
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    int ob, oe;
    if (seq_outside(sh, ob, oe)) {
        zero_rows<float>(a.dla, sh.H, ob, oe, sh.total);
        zero_rows<float>(a.dbeta, sh.H, ob, oe, sh.total);
    }
    const int slot = blockIdx.x / sh.H, h = blockIdx.x % sh.H, hk = h / (sh.H / sh.Hk);
    int s, c, first, rows;
    if (!slot_segment(sh, kSegF, slot, s, c, first, rows, a.err)) return;
    __shared__ Gates g;
    __shared__ Stage st;
    __shared__ float col[16][kSegF], diag[kSegF], pairs[4][kSegF];
    const Mat q = token_rows(a.q, sh.ldq, first, rows, hk, sh.dk), k = token_rows(a.k, sh.ldk, first, rows, hk, sh.dk),
              o = token_rows(a.dout, (size_t)sh.H * sh.dv, first, rows, h, sh.dv), v = token_rows(a.v, sh.ldv, first, rows, h, sh.dv);
    const Part pa = fetch_k(q, 0), pb = fetch_k(k, 0);               // on their way beside the gates
    load_gates(g, a, first, rows, h);
    const int m = threadIdx.x / 16 * 4, n = threadIdx.x % 16 * 4;
    Acc x, y;
    clear(x);
    clear(y);
    product<false>(x, st, q, k, sh.dk, pa, pb);
    product<false>(y, st, o, v, sh.dv, fetch_k(o, 0), fetch_k(v, 0));
    // E_ts in the place of the products' pieces, [t][s]
    float (*e)[kLd] = reinterpret_cast<float (*)[kLd]>(&st);
    static_assert(sizeof(Stage) >= sizeof(float) * kSegF * kLd, "they fit");
    __syncthreads();
    float cs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = m + i, u = n + j;
            if (t >= rows || u > t) continue;
            const float f = x[i][j] * y[i][j] * decay(g, t, u);
            if (u == t) {
                diag[t] = f;
            } else {
                r[j] = g.beta[u] * f;
                cs[j] += f;
            }
        }
        *reinterpret_cast<float4*>(&e[m + i][n]) = make_float4(r[0], r[1], r[2], r[3]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) col[threadIdx.x / 16][n + j] = cs[j];
    __syncthreads();
    {                                                     // row t's sum before u in its place, 16 columns a thread
        float* row = &e[threadIdx.x / 4][threadIdx.x % 4 * 16];
        float v[16], all = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) all += v[i] = row[i];
        float before = __shfl_up_sync(0xffffffffu, all, 1, 4);
        if (threadIdx.x % 4 == 0) before = 0.f;
        const float two = __shfl_up_sync(0xffffffffu, before, 1, 4), three = __shfl_up_sync(0xffffffffu, before, 2, 4);
        if (threadIdx.x % 4 >= 2) before = two + before;
        if (threadIdx.x % 4 == 3) before = three + before;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            row[i] = before;
            before += v[i];
        }
    }
    __syncthreads();
    {                                                     // of rows from u on, 16 rows a thread
        const int u = threadIdx.x % kSegF, part = threadIdx.x / kSegF;
        float sum = 0.f;
#pragma unroll
        for (int t = 16 * part; t < 16 * part + 16; ++t) sum += t >= u ? e[t][u] : 0.f;
        pairs[part][u] = sum;
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const size_t at = (size_t)slot * sh.H + h;
    float ph = 0.f;
    for (int i = lane; i < tiles_phi; i += 32) ph += phi[at * tiles_phi + i];
    ph = warp_sum(ph);
    // from the last token on for the queries' part, from the first for the keys': tokens 2 lane and 2 lane + 1
    float own[2], from[2], before[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = 2 * lane + j;
        own[j] = from[j] = before[j] = 0.f;
        if (t >= rows) continue;
        float cc = 0.f, iq = 0.f, ik = 0.f;
        for (int i = 0; i < 16; ++i) cc += col[i][t];
        for (int i = 0; i < tiles_q; ++i) iq += part_q[(at * tiles_q + i) * kSegF + t];
        for (int i = 0; i < tiles_k; ++i) ik += part_k[(at * tiles_k + i) * kSegF + t];
        own[j] = (pairs[0][t] + pairs[1][t]) + (pairs[2][t] + pairs[3][t]);
        from[j] = iq;
        before[j] = g.beta[t] * ik;
        a.dbeta[(size_t)(first + t) * sh.H + h] = cc + diag[t] + ik;
    }
    float f = from[0] + from[1], b = before[0] + before[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float fo = __shfl_down_sync(0xffffffffu, f, o), bo = __shfl_up_sync(0xffffffffu, b, o);
        if (lane + o < 32) f += fo;
        if (lane >= o) b += bo;
    }
    // f: from token 2 lane + 2 on; b: up to token 2 lane - 1.  The neighbour's sums, not this lane's less its own: with fast decays
    // its own terms are far larger than what remains.
    f = __shfl_down_sync(0xffffffffu, f, 1);
    b = __shfl_up_sync(0xffffffffu, b, 1);
    if (lane == 31) f = 0.f;
    if (lane == 0) b = 0.f;
    f += from[1];
    if (2 * lane + 1 < rows) a.dla[(size_t)(first + 2 * lane + 1) * sh.H + h] = (own[1] + f) + (b + before[0]) + ph;
    if (2 * lane < rows) a.dla[(size_t)(first + 2 * lane) * sh.H + h] = (own[0] + (f + from[0])) + b + ph;
}

// ---------------------------------------------------------------------------
// The states between segments: S_0 = first (null: zero), out_c = S_c, S_{c+1} = gend_c S_c + local_c, last = the
// end's (null: not wanted); BACK from the last segment to the first, with phi = gend_c <S_c, start_c>.  One thread
// four neighbouring elements, all segments; the next kAhead segments' values are on their way.
//   TERMS 0: out and start are fp32, out may be local itself; else they are bf16 terms, out_term elements apart
//   (out TERMS of them, start three).
// Bound by memory: 4 bytes read and 4 or 2 TERMS written for each element of a segment's state (backwards 6 more read): 8192 tokens
// of 8 heads, 256 x 256, 12.7 us with two terms, 16.5 with three, 26 backwards, 5.1 to 5.3 TB/s.
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;

template <int TERMS>
__device__ __forceinline__ void put_state(void* out, size_t at, size_t apart, float4 x) {
    if constexpr (TERMS == 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = x;
    } else {
#pragma unroll
        for (int i = 0; i < TERMS; ++i) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + i * apart + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            const float2 l = __bfloat1622float2(lo), u = __bfloat1622float2(hi);
            x = make_float4(x.x - l.x, x.y - l.y, x.z - u.x, x.w - u.y);
        }
    }
}
template <int TERMS>
__device__ __forceinline__ float4 get_state(const void* in, size_t at, size_t apart) {
    if constexpr (TERMS == 0) return ld4<float>(static_cast<const float*>(in), at);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 2; i >= 0; --i) {
        const float4 y = ld4<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(in) + i * apart, at);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    return x;
}

template <int TERMS, bool BACK>
__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(SeqShape sh, int L, const float* local, const float* gend, int gend_apart, const float* S0,
                                                                 void* out, size_t apart, const void* start, float* phi, float* last, int* err) {
    griddep_wait();
    griddep_launch();
    const int state = sh.dv * sh.dk, tiles = (state + kScanTile - 1) / kScanTile;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int e = tile * kScanTile + threadIdx.x * 4;
    const bool mine = e < state;
    int first, len;
    if (!seq_range(sh, s, first, len, err)) return;
    const int n = (len + L - 1) / L, slot0 = seg_slot0(first, s, L);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine && S0 != nullptr) x = ld4<float>(S0, ((size_t)s * sh.H + h) * state + e);
    __shared__ float sums[kScanThreads / 32][kAhead];
    for (int c0 = 0; c0 < n; c0 += kAhead) {
        float4 y[kAhead], z[kAhead];
        float ge[kAhead], dot[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int c = BACK ? n - 1 - (c0 + j) : c0 + j;
            const size_t at = (size_t)(slot0 + c) * sh.H + h;
            const bool live = mine && c0 + j < n;
            y[j] = live ? ld4<float>(local, at * state + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (BACK) z[j] = live ? get_state<TERMS>(start, at * state + e, apart) : make_float4(0.f, 0.f, 0.f, 0.f);
            ge[j] = c0 + j < n ? gend[at * gend_apart] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int c = BACK ? n - 1 - (c0 + j) : c0 + j;
            if (c0 + j >= n) {
                dot[j] = 0.f;
                continue;
            }
            if (mine) put_state<TERMS>(out, ((size_t)(slot0 + c) * sh.H + h) * state + e, apart, x);
            if (BACK) dot[j] = ge[j] * (x.x * z[j].x + x.y * z[j].y + x.z * z[j].z + x.w * z[j].w);
            x = make_float4(fmaf(ge[j], x.x, y[j].x), fmaf(ge[j], x.y, y[j].y), fmaf(ge[j], x.z, y[j].z), fmaf(ge[j], x.w, y[j].w));
        }
        if (BACK) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                dot[j] = warp_sum(dot[j]);
                if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < kAhead && c0 + (int)threadIdx.x < n) {
                float d = 0.f;
                for (int w = 0; w < kScanThreads / 32; ++w) d += sums[w][threadIdx.x];
                phi[((size_t)(slot0 + n - 1 - (c0 + threadIdx.x)) * sh.H + h) * tiles + tile] = d;
            }
            __syncthreads();
        }
    }
    if (mine && last != nullptr) *reinterpret_cast<float4*>(last + ((size_t)s * sh.H + h) * state + e) = x;
}

}  // namespace

cudaError_t launch_linear_scan(const SeqShape& sh, int L, int terms, bool back, const float* local, const float* gend, int gend_apart, const float* S0,
                               void* out, size_t apart, const void* start, float* phi, float* last, int* err, cudaStream_t st) {
    const dim3 grid((unsigned)((size_t)sh.nseq * sh.H * scan_tiles(sh)));
    const auto k = terms == 0 ? (back ? lin_scan_kernel<0, true> : lin_scan_kernel<0, false>)
                   : terms == 2 ? lin_scan_kernel<2, false>
                                : (back ? lin_scan_kernel<3, true> : lin_scan_kernel<3, false>);
    return launch_kernel(k, grid, dim3(kScanThreads), 0, st, sh.total > 0, sh, L, local, gend, gend_apart, S0, out, apart, start, phi, last, err);
}

namespace {

cudaError_t forward_f32(const SeqArgs& a, cudaStream_t st) {
    const SeqShape& sh = a.sh;
    const LinLayout L = lin_layout(sh, GDN_DTYPE_F32);
    float* states = reinterpret_cast<float*>(a.rec != nullptr ? a.rec : a.ws + L.ws_local);
    float* gend = reinterpret_cast<float*>(a.ws + L.ws_gend);
    const unsigned sth = (unsigned)((size_t)seg_slots(sh.nseq, sh.total, kSegF) * sh.H), tk = (sh.dk + 63) / 64, tv = (sh.dv + 63) / 64;
    cudaError_t e = launch_kernel(lin_local_kernel<false>, dim3(sth, tk * tv), dim3(kT), 0, st, false, a, states, gend);
    if (e == cudaSuccess) e = launch_linear_scan(sh, kSegF, 0, false, states, gend, 1, a.S0, states, 0, nullptr, nullptr, a.S_T, a.err, st);
    if (e == cudaSuccess && sh.total > 0)
        e = launch_kernel(lin_rows_kernel<kOut>, dim3(sth, tv), dim3(kT), 0, st, true, a, (const float*)states, (float*)nullptr);
    return e;
}

cudaError_t backward_f32(const SeqArgs& a, cudaStream_t st) {
    const SeqShape& sh = a.sh;
    const LinLayout L = lin_layout(sh, GDN_DTYPE_F32);
    const float* starts = reinterpret_cast<const float*>(a.rec);
    float *ends = reinterpret_cast<float*>(a.ws + L.ws_local), *gend = reinterpret_cast<float*>(a.ws + L.ws_gend),
          *phi = reinterpret_cast<float*>(a.ws + L.ws_phi);
    const size_t slots = seg_slots(sh.nseq, sh.total, kSegF);
    const unsigned sth = (unsigned)(slots * sh.H), stk = (unsigned)(slots * sh.Hk), tk = (sh.dk + 63) / 64, tv = (sh.dv + 63) / 64;
    float *part_q = reinterpret_cast<float*>(a.ws + L.ws_part), *part_k = part_q + slots * sh.H * tk * kSegF;
    cudaError_t e = launch_kernel(lin_local_kernel<true>, dim3(sth, tk * tv), dim3(kT), 0, st, false, a, ends, gend);
    if (e == cudaSuccess) e = launch_linear_scan(sh, kSegF, 0, true, ends, gend, 1, a.dS_T, ends, 0, starts, phi, a.dS0, a.err, st);
    if (e != cudaSuccess || sh.total == 0) return e;
    e = launch_kernel(lin_rows_kernel<kDq>, dim3(stk, tk), dim3(kT), 0, st, true, a, starts, part_q);
    if (e == cudaSuccess) e = launch_kernel(lin_rows_kernel<kDk>, dim3(stk, tk), dim3(kT), 0, st, true, a, (const float*)ends, (float*)nullptr);
    if (e == cudaSuccess) e = launch_kernel(lin_rows_kernel<kDv>, dim3(sth, tv), dim3(kT), 0, st, true, a, (const float*)ends, part_k);
    if (e == cudaSuccess)
        e = launch_kernel(lin_gates_kernel, dim3(sth), dim3(kT), 0, st, true, a, (const float*)part_q, (int)tk, (const float*)part_k,
                          (int)tv, (const float*)phi, scan_tiles(sh));
    return e;
}

}  // namespace

LinLayout lin_layout(const SeqShape& s, int dtype) {
    if (dtype == GDN_DTYPE_BF16) return lin_layout_tc(s);
    LinLayout L = {};
    const size_t slots = seg_slots(s.nseq, s.total, kSegF), sth = slots * s.H, state = sth * s.dv * s.dk * 4;
    L.rec_total = align_up(state, kSectionAlign);
    L.ws_gend = align_up(L.ws_local + state, kSectionAlign);
    L.ws_forward = align_up(L.ws_gend + sth * 4, kSectionAlign);
    L.ws_phi = L.ws_forward;
    L.ws_part = align_up(L.ws_phi + sth * scan_tiles(s) * 4, kSectionAlign);
    L.ws_total = align_up(L.ws_part + sth * ((s.dk + 63) / 64 + (s.dv + 63) / 64) * kSegF * 4, kSectionAlign);
    return L;
}

namespace {

using namespace check;

bool shape_ok(const SeqShape& s) {
    if (s.nseq < 1 || s.total < 0 || s.H < 1 || s.Hk < 1 || s.H % s.Hk != 0 || !dim_ok(s.dk) || !dim_ok(s.dv)) return false;
    if ((long long)s.nseq + s.total > (1LL << 30) || s.Hk > 1 << 18) return false;
    // grid sizes: (sequence, head, piece of the state), and (slot, head) or four blocks of it
    return (long long)s.nseq * s.H * scan_tiles(s) <= 0x7fffffffLL && (long long)seg_slots(s.nseq, s.total, kSegF) * s.H <= 0x7fffffffLL &&
           (long long)seg_slots(s.nseq, s.total, kLinSegment) * s.H * 4 <= 0x7fffffffLL;
}

bool strides_ok(const SeqShape& s, int dtype) {
    const int unit = 16 / elem_bytes(dtype);
    const long long qk = (long long)s.Hk * s.dk, v = (long long)s.H * s.dv;      // a row: what fits a stride fits an int
    return s.ldq >= qk && s.ldk >= qk && s.ldv >= v && s.ldq % unit == 0 && s.ldk % unit == 0 && s.ldv % unit == 0;
}

int sizes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes, size_t LinLayout::*what) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, nullptr, 0, 0, 0};
    if (bytes == nullptr || !shape_ok(s) || !type_ok(dtype)) return GDN_ERR_ARG;
    *bytes = lin_layout(s, dtype).*what;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_linear_seq_workspace_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    return sizes(nseq, total, H, Hk, dk, dv, dtype, bytes, &LinLayout::ws_total);
}
int gdn_linear_seq_forward_workspace_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    return sizes(nseq, total, H, Hk, dk, dv, dtype, bytes, &LinLayout::ws_forward);
}
int gdn_linear_seq_record_bytes(int nseq, int total, int H, int Hk, int dk, int dv, int dtype, size_t* bytes) {
    return sizes(nseq, total, H, Hk, dk, dv, dtype, bytes, &LinLayout::rec_total);
}

int gdn_linear_seq_forward(const void* q, int ldq, const void* k, int ldk, const void* v, int ldv, int dtype, const float* log_alpha,
                           const float* beta, const float* S0, const int32_t* offsets, void* out, float* S_T, void* record, void* workspace,
                           int nseq, int total, int H, int Hk, int dk, int dv, cudaStream_t stream) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, offsets, ldq, ldk, ldv};
    if (!type_ok(dtype) || !shape_ok(s) || !strides_ok(s, dtype) || (offsets == nullptr && total % nseq != 0)) return GDN_ERR_ARG;
    if (!aligned16(S0) || !aligned16(S_T) || !aligned16(record) || !words(offsets) || !given(workspace)) return GDN_ERR_ARG;
    if (total > 0 && (!given(q) || !given(k) || !given(v) || !given_words(log_alpha) || !given_words(beta) || !given(out))) return GDN_ERR_ARG;
    const LinLayout L = lin_layout(s, dtype);
    const int e = elem_bytes(dtype);
    const size_t gb = (size_t)total * H * 4, sb = (size_t)nseq * H * dv * dk * 4;
    const Span w[] = {{out, (size_t)total * H * dv * e}, {record, L.rec_total}, {workspace, L.ws_forward}, {S_T, sb}};
    const Span r[] = {{q, strided_bytes(total, ldq, Hk * dk, e)}, {k, strided_bytes(total, ldk, Hk * dk, e)},
                      {v, strided_bytes(total, ldv, H * dv, e)},  {log_alpha, gb},
                      {beta, gb},                                 {offsets, ((size_t)nseq + 1) * 4}};
    // S_T may be S0 itself: each element is read before it is written, by the same thread
    if (!disjoint(w, 4, r, 6) || (S_T != S0 && overlap({S0, sb}, w[3]))) return GDN_ERR_ARG;
    for (int i = 0; i < 3; ++i)
        if (overlap({S0, sb}, w[i])) return GDN_ERR_ARG;
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
    const cudaError_t rc = dtype == GDN_DTYPE_F32 ? forward_f32(a, stream) : launch_linear_forward_tc(a, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_linear_seq_backward(const void* q, int ldq, const void* k, int ldk, const void* v, int ldv, int dtype, const float* log_alpha,
                            const float* beta, const int32_t* offsets, const void* dout, const float* dS_T, const void* record, void* dq,
                            void* dk_out, void* dv_out, float* dlog_alpha, float* dbeta, float* dS0, void* workspace, int nseq, int total,
                            int H, int Hk, int dk, int dv, cudaStream_t stream) {
    const SeqShape s = {nseq, total, H, Hk, dk, dv, offsets, ldq, ldk, ldv};
    if (!type_ok(dtype) || !shape_ok(s) || !strides_ok(s, dtype) || (offsets == nullptr && total % nseq != 0)) return GDN_ERR_ARG;
    if (!aligned16(dS_T) || !aligned16(dS0) || !words(offsets) || !given(workspace) || !given(record)) return GDN_ERR_ARG;
    if (total > 0 && (!given(q) || !given(k) || !given(v) || !given_words(log_alpha) || !given_words(beta) || !given(dout) || !given(dq) ||
                      !given(dk_out) || !given(dv_out) || !given_words(dlog_alpha) || !given_words(dbeta)))
        return GDN_ERR_ARG;
    const LinLayout L = lin_layout(s, dtype);
    const int e = elem_bytes(dtype);
    const size_t vo = (size_t)total * H * dv * e, gb = (size_t)total * H * 4, qb = (size_t)total * Hk * dk * e, sb = (size_t)nseq * H * dv * dk * 4;
    const Span w[] = {{dq, qb}, {dk_out, qb}, {dv_out, vo}, {dlog_alpha, gb}, {dbeta, gb}, {workspace, L.ws_total}, {dS0, sb}};
    const Span r[] = {{q, strided_bytes(total, ldq, Hk * dk, e)}, {k, strided_bytes(total, ldk, Hk * dk, e)},
                      {v, strided_bytes(total, ldv, H * dv, e)},  {log_alpha, gb},
                      {beta, gb},                                 {offsets, ((size_t)nseq + 1) * 4},
                      {dout, vo},                                 {record, L.rec_total}};
    if (!disjoint(w, 7, r, 8) || (dS0 != dS_T && overlap({dS_T, sb}, w[6]))) return GDN_ERR_ARG;
    for (int i = 0; i < 6; ++i)
        if (overlap({dS_T, sb}, w[i])) return GDN_ERR_ARG;
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
    const cudaError_t rc = dtype == GDN_DTYPE_F32 ? backward_f32(a, stream) : launch_linear_backward_tc(a, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

// gdn_norm.cu -- the norms around a block and their gradients, one pass over the data each.
//
//   gated norm   y = w (o r) silu(z),  r = (mean o^2 + eps)^{-1/2}, for each head's row of d values
//   block norm   x' = rho x + gamma (w_post (z r1)),  h = w (x' r2), for each row of D values
//
// All are bound by their reads and writes.  A row lives in the registers of the lanes that
// read it (eight values each, 16-byte loads), its sums are reduced between those lanes, and it
// is written from there, so that every input is read and every output written once.  Sums and
// statistics are fp32; values are rounded once, on the way out.
//
// The gradients of the weights are sums over all rows.  Each thread adds its own columns' terms
// over the rows that its CTA takes, a CTA's threads are added in shared memory and written as one
// row of partial sums, and a second kernel adds those rows in their order: no atomics, so equal
// inputs give equal bits.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kPartialRows = 304;        // CTAs of a gradient kernel at most: two per SM

template <typename T>
__device__ __forceinline__ void st8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void st8<float>(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void st8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
    uint4 u;
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = u;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// ---------------------------------------------------------------------------
// gated norm: LANES lanes per row of d <= 8 LANES values
// ---------------------------------------------------------------------------
struct GatedArgs {
    const void *o, *z, *w, *dy;
    void *y, *dout, *dz;
    float* part;
    long long rows;
    int d;
    float eps;
};

template <typename TO, typename T, int LANES>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(GatedArgs a) {
    const int c = 8 * (threadIdx.x % LANES);
    const long long row = (long long)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const bool in = row < a.rows && c < a.d;
    float o[8] = {}, z[8] = {}, w[8] = {};
    if (in) {
        ld8<TO>(static_cast<const TO*>(a.o) + row * a.d + c, o);
        ld8<T>(static_cast<const T*>(a.z) + row * a.d + c, z);
        ld8<T>(static_cast<const T*>(a.w) + c, w);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(o[i], o[i], s);
    const float r = rsqrtf(lanes_sum<LANES>(s) / a.d + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * r * w[i] * (z[i] * sigmoid(z[i]));
    if (in) st8<T>(static_cast<T*>(a.y) + row * a.d + c, o);
}

template <typename TO, typename T, int LANES>
__global__ void __launch_bounds__(kThreads) gated_norm_back_kernel(GatedArgs a) {
    __shared__ float sw[kThreads][8];
    const int c = 8 * (threadIdx.x % LANES);
    float w[8] = {}, dw[8] = {};
    if (c < a.d) ld8<T>(static_cast<const T*>(a.w) + c, w);
    const long long step = (long long)gridDim.x * (kThreads / LANES);
    // whole warps stay in the loop together: the bound is the one of the CTA's first row
    for (long long base = (long long)blockIdx.x * (kThreads / LANES); base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LANES;
        const bool in = row < a.rows && c < a.d;
        float o[8] = {}, z[8] = {}, dy[8] = {};
        if (in) {
            ld8<TO>(static_cast<const TO*>(a.o) + row * a.d + c, o);
            ld8<T>(static_cast<const T*>(a.z) + row * a.d + c, z);
            ld8<T>(static_cast<const T*>(a.dy) + row * a.d + c, dy);
        }
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float sg = sigmoid(z[i]), silu = z[i] * sg, wy = dy[i] * w[i];
            s = fmaf(o[i], o[i], s);
            t = fmaf(o[i], wy * silu, t);
            z[i] = sg * fmaf(z[i], 1.f - sg, 1.f);       // silu'
            dy[i] = dy[i] * silu;                        // the norm's own gradient, before w
        }
        const float r = rsqrtf(lanes_sum<LANES>(s) / a.d + a.eps);
        const float m = lanes_sum<LANES>(t) * r / a.d;   // mean of n dn
        float g[8], dz[8];
        if (in) {
            float y[8];
            ld8<T>(static_cast<const T*>(a.dy) + row * a.d + c, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = o[i] * r;
                g[i] = r * (dy[i] * w[i] - n * m);
                dz[i] = y[i] * n * w[i] * z[i];
                dw[i] = fmaf(dy[i], n, dw[i]);
            }
            st8<TO>(static_cast<TO*>(a.dout) + row * a.d + c, g);
            st8<T>(static_cast<T*>(a.dz) + row * a.d + c, dz);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sw[threadIdx.x][i] = dw[i];
    __syncthreads();
    for (int x = threadIdx.x; x < a.d; x += kThreads) {
        float s = 0.f;
        for (int g = 0; g < kThreads / LANES; ++g) s += sw[g * LANES + x / 8][x % 8];
        a.part[(size_t)blockIdx.x * a.d + x] = s;
    }
}

// Column sums of `n` rows of partial sums, up to three arrays of them behind one another.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float* part, int n, int D, float* out0, float* out1, float* out2) {
    __shared__ float sm[8][32];
    const int x = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
    const float* p = part + (size_t)blockIdx.y * n * D;
    float s = 0.f;
    if (x < D)
        for (int i = g; i < n; i += 8) s += p[(size_t)i * D + x];
    sm[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && x < D) {
        for (int i = 1; i < 8; ++i) s += sm[i][threadIdx.x & 31];
        out[x] = s;
    }
}

// ---------------------------------------------------------------------------
// block norm: a row of D values by a warp (D <= 1024) or by the whole CTA
// ---------------------------------------------------------------------------
struct BlockArgs {
    const void *x, *z, *wp, *gate, *w, *dh, *dx2;
    void *x2, *h, *dx, *dz;
    float* part;
    long long rows;
    int D;
    float eps, rho;
};

// Sums of N values over a row's threads (a warp or the CTA); every thread gets them.
template <bool CTA, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*sm)[kThreads / 32]) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = warp_sum(s[i]);
    if constexpr (CTA) {
        __syncthreads();                     // the last reduction's reads are done
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) sm[i][threadIdx.x >> 5] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) t += sm[i][w];
            s[i] = t;
        }
    }
}

template <typename T, bool CTA, int V, bool POST>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(BlockArgs a) {
    __shared__ float sm[3][kThreads / 32];
    constexpr int TPR = CTA ? kThreads : 32, RPC = kThreads / TPR;
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
    if (row >= a.rows) return;               // a whole warp, or nobody
    float x[V][8];
    float s[1] = {0.f};
    const T* xr = static_cast<const T*>(a.x) + row * a.D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + i * TPR);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
        if (c < a.D) ld8<T>(xr + c, x[i]);
    }
    if constexpr (POST) {
        float z[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
            if (c < a.D) ld8<T>(static_cast<const T*>(a.z) + row * a.D + c, z[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] = fmaf(z[i][j], z[i][j], s[0]);
        }
        row_sums<CTA, 1>(s, sm);
        const float r = rsqrtf(s[0] / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            if (c < a.D) {
                float w[8], g[8];
                ld8<T>(static_cast<const T*>(a.wp) + c, w);
                ld8<T>(static_cast<const T*>(a.gate) + c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(g[j], z[i][j] * r * w[j], a.rho * x[i][j]);
                st8<T>(static_cast<T*>(a.x2) + row * a.D + c, x[i]);
            }
        }
        s[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(x[i][j], x[i][j], s[0]);
    row_sums<CTA, 1>(s, sm);
    const float r = rsqrtf(s[0] / a.D + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + i * TPR);
        if (c < a.D) {
            float w[8];
            ld8<T>(static_cast<const T*>(a.w) + c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= r * w[j];
            st8<T>(static_cast<T*>(a.h) + row * a.D + c, x[i]);
        }
    }
}

template <typename T, bool CTA, int V, bool POST>
__global__ void __launch_bounds__(kThreads) block_norm_back_kernel(BlockArgs a) {
    __shared__ float sm[3][kThreads / 32];
    constexpr int TPR = CTA ? kThreads : 32, RPC = kThreads / TPR;
    const int t = threadIdx.x % TPR;
    float dw[V][8] = {}, dwp[POST ? V : 1][8] = {}, dg[POST ? V : 1][8] = {};
    for (long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR; row < a.rows; row += (long long)gridDim.x * RPC) {
        float x[V][8], y[V][8], z[POST ? V : 1][8];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            const size_t at = (size_t)row * a.D + c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = y[i][j] = 0.f;
                if constexpr (POST) z[i][j] = 0.f;
            }
            if (c < a.D) {
                float w[8];
                ld8<T>(static_cast<const T*>(a.x) + at, x[i]);
                ld8<T>(static_cast<const T*>(a.dh) + at, y[i]);
                ld8<T>(static_cast<const T*>(a.w) + c, w);
                if constexpr (POST) ld8<T>(static_cast<const T*>(a.z) + at, z[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[0] = fmaf(x[i][j], x[i][j], s[0]);
                    s[1] = fmaf(x[i][j], y[i][j] * w[j], s[1]);
                    if constexpr (POST) s[2] = fmaf(z[i][j], z[i][j], s[2]);
                }
            }
        }
        row_sums<CTA, 3>(s, sm);
        const float r = rsqrtf(s[0] / a.D + a.eps), m = s[1] * r / a.D;
        const float rz = POST ? rsqrtf(s[2] / a.D + a.eps) : 0.f;
        float u[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            const size_t at = (size_t)row * a.D + c;
            if (c < a.D) {
                float w[8], d[8] = {}, dx[8];
                ld8<T>(static_cast<const T*>(a.w) + c, w);
                if (a.dx2 != nullptr) ld8<T>(static_cast<const T*>(a.dx2) + at, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = x[i][j] * r;
                    dw[i][j] = fmaf(y[i][j], n, dw[i][j]);
                    d[j] += r * (y[i][j] * w[j] - n * m);
                    dx[j] = a.rho * d[j];
                }
                st8<T>(static_cast<T*>(a.dx) + at, dx);
                if constexpr (POST) {
                    float wp[8], g[8];
                    ld8<T>(static_cast<const T*>(a.wp) + c, wp);
                    ld8<T>(static_cast<const T*>(a.gate) + c, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float n = z[i][j] * rz;
                        dwp[i][j] = fmaf(d[j] * g[j], n, dwp[i][j]);
                        dg[i][j] = fmaf(d[j] * wp[j], n, dg[i][j]);
                        x[i][j] = d[j] * g[j] * wp[j];
                        u[0] = fmaf(x[i][j], n, u[0]);
                    }
                }
            }
        }
        if constexpr (POST) {
            row_sums<CTA, 1>(u, sm);
            const float mz = u[0] / a.D;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = 8 * (t + i * TPR);
                if (c < a.D) {
                    float dz[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) dz[j] = rz * (x[i][j] - z[i][j] * rz * mz);
                    st8<T>(static_cast<T*>(a.dz) + (size_t)row * a.D + c, dz);
                }
            }
        }
    }
    // partial sums [3][gridDim.x][D]; the warps of a CTA in their order
    extern __shared__ float acc[];
    for (int p = 0; p < (POST ? 3 : 1); ++p) {
        float* out = a.part + ((size_t)p * gridDim.x + blockIdx.x) * a.D;
        for (int g = 0; g < RPC; ++g) {
            if (threadIdx.x / TPR == g)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = 8 * (t + i * TPR);
                    if (c < a.D)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float v = dw[i][j];
                            if constexpr (POST) v = p == 0 ? v : p == 1 ? dwp[i][j] : dg[i][j];
                            if constexpr (CTA) out[c + j] = v;
                            else if (g == 0) acc[c + j] = v;
                            else if (g < RPC - 1) acc[c + j] += v;
                            else out[c + j] = acc[c + j] + v;
                        }
                }
            if constexpr (!CTA) __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename TO, typename T, int LANES>
cudaError_t gated_go(const GatedArgs& a, float* dw, bool back, cudaStream_t st) {
    const long long per = kThreads / LANES, ctas = (a.rows + per - 1) / per;
    if (!back) return launch_kernel(gated_norm_kernel<TO, T, LANES>, dim3((unsigned)ctas), dim3(kThreads), 0, st, false, a);
    const int n = (int)(ctas < kPartialRows ? ctas : kPartialRows);
    cudaError_t e = launch_kernel(gated_norm_back_kernel<TO, T, LANES>, dim3((unsigned)n), dim3(kThreads), 0, st, false, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(sum_rows_kernel, dim3((a.d + 31) / 32, 1), dim3(256), 0, st, false, (const float*)a.part, n, a.d, dw,
                         (float*)nullptr, (float*)nullptr);
}

template <typename TO, typename T>
cudaError_t gated_lanes(const GatedArgs& a, float* dw, bool back, cudaStream_t st) {
    if (a.d <= 16) return gated_go<TO, T, 2>(a, dw, back, st);
    if (a.d <= 32) return gated_go<TO, T, 4>(a, dw, back, st);
    if (a.d <= 64) return gated_go<TO, T, 8>(a, dw, back, st);
    if (a.d <= 128) return gated_go<TO, T, 16>(a, dw, back, st);
    return gated_go<TO, T, 32>(a, dw, back, st);
}

cudaError_t gated(const GatedArgs& a, float* dw, bool back, int odtype, int dtype, cudaStream_t st) {
    if (odtype == GDN_DTYPE_F32)
        return dtype == GDN_DTYPE_F32 ? gated_lanes<float, float>(a, dw, back, st)
                                      : gated_lanes<float, __nv_bfloat16>(a, dw, back, st);
    return dtype == GDN_DTYPE_F32 ? gated_lanes<__nv_bfloat16, float>(a, dw, back, st)
                                  : gated_lanes<__nv_bfloat16, __nv_bfloat16>(a, dw, back, st);
}

template <typename T, bool CTA, int V, bool POST>
cudaError_t block_go(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, cudaStream_t st) {
    const long long per = CTA ? 1 : kThreads / 32, ctas = (a.rows + per - 1) / per;
    if (!back) return launch_kernel(block_norm_kernel<T, CTA, V, POST>, dim3((unsigned)ctas), dim3(kThreads), 0, st, false, a);
    const int n = (int)(ctas < kPartialRows ? ctas : kPartialRows);
    cudaError_t e = launch_kernel(block_norm_back_kernel<T, CTA, V, POST>, dim3((unsigned)n), dim3(kThreads),
                                  CTA ? 0 : (size_t)a.D * 4, st, false, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(sum_rows_kernel, dim3((a.D + 31) / 32, POST ? 3 : 1), dim3(256), 0, st, false, (const float*)a.part,
                         n, a.D, dw, dwp, dgate);
}

// V vectors of eight values per thread: the fewest that hold the row
template <typename T, bool POST>
cudaError_t block_v(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, cudaStream_t st) {
    if (a.D <= 256) return block_go<T, false, 1, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 512) return block_go<T, false, 2, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 1024) return block_go<T, false, 4, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 2048) return block_go<T, true, 1, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 4096) return block_go<T, true, 2, POST>(a, dw, dwp, dgate, back, st);
    return block_go<T, true, 4, POST>(a, dw, dwp, dgate, back, st);
}

cudaError_t block(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, int dtype, cudaStream_t st) {
    if (dtype == GDN_DTYPE_F32)
        return a.z != nullptr ? block_v<float, true>(a, dw, dwp, dgate, back, st) : block_v<float, false>(a, dw, dwp, dgate, back, st);
    return a.z != nullptr ? block_v<__nv_bfloat16, true>(a, dw, dwp, dgate, back, st)
                          : block_v<__nv_bfloat16, false>(a, dw, dwp, dgate, back, st);
}

constexpr int kMaxWidth = 8192;          // D of the block norm: four vectors for each of 256 threads
constexpr long long kMaxRows = 1LL << 31;

bool given(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(int t) { return t == GDN_DTYPE_BF16 || t == GDN_DTYPE_F32; }
bool gated_ok(long long rows, int d, float eps) {
    return rows >= 1 && rows < kMaxRows && d >= 16 && d <= kMaxDim && d % 16 == 0 && eps > 0.f;
}
bool block_ok(long long rows, int D, float eps) {
    return rows >= 1 && rows < kMaxRows && D >= 8 && D <= kMaxWidth && D % 8 == 0 && eps > 0.f;
}

struct Span {
    const void* p;
    size_t n;
};
bool meet(const Span& a, const Span& b) {
    const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
    return x != nullptr && y != nullptr && x < y + b.n && y < x + a.n;
}
// Written spans are apart from one another and from the read ones; the first `same` of them may
// each be one of the first `rows` read spans itself, of the same size (each element is read before
// it is written, by the same thread).
template <int W, int R>
bool spans_ok(const Span (&w)[W], const Span (&r)[R], int same, int rows) {
    for (int i = 0; i < W; ++i) {
        for (int j = i + 1; j < W; ++j)
            if (meet(w[i], w[j])) return false;
        for (int j = 0; j < R; ++j)
            if (meet(w[i], r[j]) && (i >= same || j >= rows || w[i].p != r[j].p || w[i].n != r[j].n)) return false;
    }
    return true;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_norm_workspace_bytes(long long rows, int width, size_t* bytes) {
    if (bytes == nullptr || !block_ok(rows, width, 1.f)) return GDN_ERR_ARG;
    *bytes = align_up((size_t)(rows < kPartialRows ? rows : kPartialRows) * 3 * width * 4, kSectionAlign);
    return GDN_OK;
}

int gdn_gated_norm(const void* o, int o_dtype, const void* gate, const void* weight, void* out, int dtype, long long rows,
                   int d, float eps, cudaStream_t stream) {
    if (!dtype_ok(o_dtype) || !dtype_ok(dtype) || !gated_ok(rows, d, eps)) return GDN_ERR_ARG;
    if (!given(o) || !given(gate) || !given(weight) || !given(out)) return GDN_ERR_ARG;
    const size_t n = (size_t)rows * d, e = elem_bytes(dtype);
    const Span w[] = {{out, n * e}}, r[] = {{o, n * elem_bytes(o_dtype)}, {gate, n * e}, {weight, d * e}};
    if (!spans_ok(w, r, 1, 2)) return GDN_ERR_ARG;
    int st;
    if (current_error_word(&st) == nullptr) return st;
    GatedArgs a = {o, gate, weight, nullptr, out, nullptr, nullptr, nullptr, rows, d, eps};
    return gated(a, nullptr, false, o_dtype, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_gated_norm_backward(const void* o, int o_dtype, const void* gate, const void* weight, const void* dout_y, void* d_o,
                            void* dgate, float* dweight, void* workspace, int dtype, long long rows, int d, float eps,
                            cudaStream_t stream) {
    if (!dtype_ok(o_dtype) || !dtype_ok(dtype) || !gated_ok(rows, d, eps)) return GDN_ERR_ARG;
    if (!given(o) || !given(gate) || !given(weight) || !given(dout_y) || !given(d_o) || !given(dgate) || !given(dweight) ||
        !given(workspace))
        return GDN_ERR_ARG;
    const size_t n = (size_t)rows * d, e = elem_bytes(dtype), eo = elem_bytes(o_dtype);
    size_t wb;
    if (gdn_norm_workspace_bytes(rows, d, &wb) != GDN_OK) return GDN_ERR_ARG;
    const Span w[] = {{d_o, n * eo}, {dgate, n * e}, {dweight, (size_t)d * 4}, {workspace, wb}};
    const Span r[] = {{o, n * eo}, {gate, n * e}, {weight, d * e}, {dout_y, n * e}};
    if (!spans_ok(w, r, 0, 0)) return GDN_ERR_ARG;
    int st;
    if (current_error_word(&st) == nullptr) return st;
    GatedArgs a = {o, gate, weight, dout_y, nullptr, d_o, dgate, static_cast<float*>(workspace), rows, d, eps};
    return gated(a, dweight, true, o_dtype, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_block_norm(const void* x, const void* z, const void* post_weight, const void* gate, const void* weight, void* x_out,
                   void* h, int dtype, long long rows, int width, float eps, float res_scale, cudaStream_t stream) {
    if (!dtype_ok(dtype) || !block_ok(rows, width, eps)) return GDN_ERR_ARG;
    if (!given(x) || !given(weight) || !given(h)) return GDN_ERR_ARG;
    const bool post = z != nullptr;
    if (post ? (!given(z) || !given(post_weight) || !given(gate) || !given(x_out))
             : (post_weight != nullptr || gate != nullptr || x_out != nullptr || res_scale != 1.f))
        return GDN_ERR_ARG;
    const size_t e = elem_bytes(dtype), n = (size_t)rows * width * e, v = width * e;
    const Span w[] = {{x_out, n}, {h, n}}, r[] = {{x, n}, {z, n}, {weight, v}, {post_weight, v}, {gate, v}};
    if (!spans_ok(w, r, 2, 2)) return GDN_ERR_ARG;
    int st;
    if (current_error_word(&st) == nullptr) return st;
    BlockArgs a = {x, z, post_weight, gate, weight, nullptr, nullptr, x_out, h, nullptr, nullptr, nullptr, rows, width, eps, res_scale};
    return block(a, nullptr, nullptr, nullptr, false, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_block_norm_backward(const void* x_out, const void* z, const void* post_weight, const void* gate, const void* weight,
                            const void* dh, const void* dx_out, void* dx, void* dz, float* dpost_weight, float* dgate,
                            float* dweight, void* workspace, int dtype, long long rows, int width, float eps, float res_scale,
                            cudaStream_t stream) {
    if (!dtype_ok(dtype) || !block_ok(rows, width, eps)) return GDN_ERR_ARG;
    if (!given(x_out) || !given(weight) || !given(dh) || !given(dx) || !given(dweight) || !given(workspace)) return GDN_ERR_ARG;
    if (dx_out != nullptr && !given(dx_out)) return GDN_ERR_ARG;
    const bool post = z != nullptr;
    if (post ? (!given(z) || !given(post_weight) || !given(gate) || !given(dz) || !given(dpost_weight) || !given(dgate))
             : (post_weight != nullptr || gate != nullptr || dz != nullptr || dpost_weight != nullptr || dgate != nullptr ||
                res_scale != 1.f))
        return GDN_ERR_ARG;
    const size_t e = elem_bytes(dtype), n = (size_t)rows * width * e, v = width * e, f = (size_t)width * 4;
    size_t wb;
    if (gdn_norm_workspace_bytes(rows, width, &wb) != GDN_OK) return GDN_ERR_ARG;
    const Span w[] = {{dx, n}, {dz, n}, {dpost_weight, f}, {dgate, f}, {dweight, f}, {workspace, wb}};
    const Span r[] = {{x_out, n}, {z, n}, {dh, n}, {dx_out, n}, {post_weight, v}, {gate, v}, {weight, v}};
    if (!spans_ok(w, r, 0, 0)) return GDN_ERR_ARG;
    int st;
    if (current_error_word(&st) == nullptr) return st;
    BlockArgs a = {x_out, z, post_weight, gate, weight, dh, dx_out, nullptr, nullptr, dx, dz, static_cast<float*>(workspace),
                   rows, width, eps, res_scale};
    return block(a, dweight, dpost_weight, dgate, true, dtype, stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

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
//
// 8192 x 8 rows of 256, bf16: gated norm 19 us (100 MB, 5.2 TB/s), its gradients 35 us (168 MB, 4.8 TB/s).  8192 rows
// of 2048: block norm 28 us (134 MB, 4.8 TB/s), its gradients 47 us (201 MB, 4.3 TB/s).  The gradients' last two
// microseconds are the second kernel's.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
// CTAs of a gradient kernel at most, each a row of partial sums (the block norm: two): in bf16 as many as are
// resident together, so that none begins when others have ended.  The block norm's kernel holds two rows in up
// to 128 registers a thread, 512 threads an SM.  Its fp32 forms take 132 to 151 up to 2048 values: one CTA fewer
// is resident, and the last ones begin when others have ended (8192 x 2048 136 us, 3.0 TB/s).  The gated norm's
// gradients beside fp32 gates spill some 100 bytes at their 80 registers (8192 x 8 rows of 256 in fp32 73 us, 4.6 TB/s).
constexpr int kSMs = 152, kGatedCtas = 3 * kSMs;
constexpr int block_ctas(int threads) { return kSMs * (512 / threads); }

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

// Eight values as they lie in memory: held back a row ahead, and widened where they are used.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float operator[](int i) const {
        const uint32_t w = (&u.x)[i / 2];
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float operator[](int i) const { return i < 4 ? (&a.x)[i] : (&b.x)[i - 4]; }
};

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// For results in types TO and T beside gates in T.  bf16 results are rounded by 2^-8: the hardware's exponential and
// reciprocal do for them (2^-21, and 2^-23 |z| of the exponential), and the exact ones would take as long as the reads.
// An fp32 gradient beside bf16 gates takes the exact exponential, and the reciprocal, 2^-22, from the hardware (8192 x 8
// rows of 256 43 us; with both exact 54, registers spill); fp32 throughout both exact ones.  dweight, fp32 always,
// adds up what its rows were computed with.
template <typename TO, typename T>
__device__ __forceinline__ float sigmoid(float z) {
    const float e = sizeof(TO) == 2 && sizeof(T) == 2 ? __expf(-z) : expf(-z);
    return sizeof(T) == 2 ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
}

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
    for (int i = 0; i < 8; ++i) o[i] = o[i] * r * w[i] * (z[i] * sigmoid<T, T>(z[i]));
    if (in) st8<T>(static_cast<T*>(a.y) + row * a.d + c, o);
}

template <typename TO, typename T, int LANES>
__global__ void __launch_bounds__(kThreads, 3) gated_norm_back_kernel(GatedArgs a) {
    __shared__ float sw[kThreads][8];
    const int c = 8 * (threadIdx.x % LANES);
    const float inv_d = 1.f / a.d;
    Raw8<T> w;
    float dw[8] = {};
    w.zero();
    if (c < a.d) w.load(static_cast<const T*>(a.w) + c);
    const long long step = (long long)gridDim.x * (kThreads / LANES);
    Raw8<TO> on;
    Raw8<T> zn, yn;
    auto load = [&](long long row) {
        on.zero();
        zn.zero();
        yn.zero();
        if (row < a.rows && c < a.d) {
            on.load(static_cast<const TO*>(a.o) + row * a.d + c);
            zn.load(static_cast<const T*>(a.z) + row * a.d + c);
            yn.load(static_cast<const T*>(a.dy) + row * a.d + c);
        }
    };
    // whole warps stay in the loop together: the bound is the one of the CTA's first row
    const long long mine = threadIdx.x / LANES;
    long long base = (long long)blockIdx.x * (kThreads / LANES);
    load(base + mine);
    for (; base < a.rows; base += step) {
        const long long row = base + mine;
        const Raw8<TO> o = on;
        const Raw8<T> z = zn, y = yn;
        load(row + step);                                // the next row's reads, before this one's sums wait
        float s = 0.f, t = 0.f, sg[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sg[i] = sigmoid<TO, T>(z[i]);
            s = fmaf(o[i], o[i], s);
            t = fmaf(o[i], y[i] * w[i] * (z[i] * sg[i]), t);
        }
        const float r = rsqrtf(lanes_sum<LANES>(s) * inv_d + a.eps);
        const float m = lanes_sum<LANES>(t) * r * inv_d;     // mean of n dn
        float g[8], dz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = o[i] * r, silu = z[i] * sg[i], dn = y[i] * silu;     // dn: before w
            g[i] = r * (dn * w[i] - n * m);
            dz[i] = y[i] * n * w[i] * (sg[i] * fmaf(z[i], 1.f - sg[i], 1.f));    // silu' = sg (1 + z (1 - sg))
            dw[i] = fmaf(dn, n, dw[i]);
        }
        if (row < a.rows && c < a.d) {
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
    griddep_launch();
}

// Column sums of `n` rows of partial sums, 32 columns to a CTA, its warps' rows added in their order;
// of a second array behind the first too, times each of two rows of weights.
template <typename T>
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float* part, int n, int D, float* out, const T* f1, float* out1,
                                                        const T* f2, float* out2) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, x = blockIdx.x * 32 + lane;
    const float* p = part + (size_t)blockIdx.y * n * D;
    float s = 0.f;
    griddep_wait();
    if (x < D)
#pragma unroll 8
        for (int i = g; i < n; i += 32) s += p[(size_t)i * D + x];
    sm[g][lane] = s;
    __syncthreads();
    // warp w: column w's 32 sums
    s = warp_sum(sm[lane][g]);
    const int c = blockIdx.x * 32 + g;
    if (lane == 0 && c < D) {
        if (blockIdx.y == 0) {
            out[c] = s;
        } else {
            out1[c] = s * ld_elem<T>(f1, c);
            out2[c] = s * ld_elem<T>(f2, c);
        }
    }
}

// ---------------------------------------------------------------------------
// block norm: a row of D values by the TPR threads of a CTA, or (TPR 32) by one of its eight warps
// ---------------------------------------------------------------------------
struct BlockArgs {
    const void *x, *z, *wp, *gate, *w, *dh, *dx2;
    void *x2, *h, *dx, *dz;
    float* part;
    long long rows;
    int D;
    float eps, rho;
};

template <int TPR>
constexpr int kBlockThreads = TPR == 32 ? 256 : TPR;

// Sums of N values over a row's threads; every thread gets them.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*sm)[16]) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = warp_sum(s[i]);
    if constexpr (TPR > 32) {
        __syncthreads();                     // the last reduction's reads are done
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) sm[i][threadIdx.x >> 5] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) t += sm[i][w];
            s[i] = t;
        }
    }
}

template <typename T, int TPR, int V, bool POST>
__global__ void __launch_bounds__(kBlockThreads<TPR>) block_norm_kernel(BlockArgs a) {
    __shared__ float sm[1][16];
    constexpr int RPC = kBlockThreads<TPR> / TPR;
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
    if (row >= a.rows) return;               // a whole warp, or nobody
    float x[V][8];
    float s[1] = {0.f};
    const T* xr = static_cast<const T*>(a.x) + row * a.D;
    Raw8<T> w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + i * TPR);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
        w[i].zero();
        if (c < a.D) {
            ld8<T>(xr + c, x[i]);
            w[i].load(static_cast<const T*>(a.w) + c);
        }
    }
    if constexpr (POST) {
        Raw8<T> z[V], wp[V], g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            z[i].zero();
            if (c < a.D) {
                z[i].load(static_cast<const T*>(a.z) + row * a.D + c);
                wp[i].load(static_cast<const T*>(a.wp) + c);
                g[i].load(static_cast<const T*>(a.gate) + c);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] = fmaf(z[i][j], z[i][j], s[0]);
        }
        row_sums<TPR, 1>(s, sm);
        const float r = rsqrtf(s[0] / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            if (c < a.D) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = fmaf(g[i][j], z[i][j] * r * wp[i][j], a.rho * x[i][j]);
                st8<T>(static_cast<T*>(a.x2) + row * a.D + c, x[i]);
            }
        }
        s[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(x[i][j], x[i][j], s[0]);
    row_sums<TPR, 1>(s, sm);
    const float r = rsqrtf(s[0] / a.D + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + i * TPR);
        if (c < a.D) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= r * w[i][j];
            st8<T>(static_cast<T*>(a.h) + row * a.D + c, x[i]);
        }
    }
}

// With n = x' r, y = dh w, m = mean(y n), k = gamma w_post and n_z = z r_z:
//   d = dx' + r (y - n m),  dx = rho d,  dz = r_z (d k - n_z mean(d k n_z)).
// The last mean needs d, which needs the sums of the row before: it is put together from sums that
// do not, of dx' k z, y k z and x' k z, so that a row waits for one reduction, not for two.
// The gradients of w_post and gamma are one sum, of d n_z, times the other of the two.
template <typename T, int TPR, int V, bool POST>
__global__ void __launch_bounds__(kBlockThreads<TPR>) block_norm_back_kernel(BlockArgs a) {
    __shared__ float sm[6][16];
    constexpr int RPC = kBlockThreads<TPR> / TPR;
    constexpr int VP = POST ? V : 1;
    const int t = threadIdx.x % TPR;
    const float inv_d = 1.f / a.D;
    float dw[V][8] = {}, de[VP][8] = {};
    Raw8<T> xn[V], yn[V], dn[V], zn[VP], w[V], wp[VP], gt[VP];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (t + i * TPR);
        w[i].zero();
        if (c < a.D) w[i].load(static_cast<const T*>(a.w) + c);
        if constexpr (POST) {
            wp[i].zero();
            gt[i].zero();
            if (c < a.D) {
                wp[i].load(static_cast<const T*>(a.wp) + c);
                gt[i].load(static_cast<const T*>(a.gate) + c);
            }
        }
    }
    auto load = [&](long long row) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            const size_t at = (size_t)row * a.D + c;
            xn[i].zero();
            yn[i].zero();
            dn[i].zero();
            if constexpr (POST) zn[i].zero();
            if (c < a.D && row < a.rows) {
                xn[i].load(static_cast<const T*>(a.x) + at);
                yn[i].load(static_cast<const T*>(a.dh) + at);
                if (a.dx2 != nullptr) dn[i].load(static_cast<const T*>(a.dx2) + at);
                if constexpr (POST) zn[i].load(static_cast<const T*>(a.z) + at);
            }
        }
    };
    const long long step = (long long)gridDim.x * RPC;
    long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
    load(row);
    for (; row < a.rows; row += step) {
        Raw8<T> x[V], y[V], dx2[V], z[VP];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = xn[i];
            y[i] = yn[i];
            dx2[i] = dn[i];
            if constexpr (POST) z[i] = zn[i];
        }
        if (V == 1) load(row + step);                    // the next row's reads, before this one's sums wait
        float s[POST ? 6 : 2] = {};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yw = y[i][j] * w[i][j];
                s[0] = fmaf(x[i][j], x[i][j], s[0]);
                s[1] = fmaf(x[i][j], yw, s[1]);
                if constexpr (POST) {
                    const float kz = gt[i][j] * wp[i][j] * z[i][j];
                    s[2] = fmaf(z[i][j], z[i][j], s[2]);
                    s[3] = fmaf(dx2[i][j], kz, s[3]);
                    s[4] = fmaf(yw, kz, s[4]);
                    s[5] = fmaf(x[i][j], kz, s[5]);
                }
            }
        row_sums<TPR, POST ? 6 : 2>(s, sm);
        const float r = rsqrtf(s[0] * inv_d + a.eps), m = s[1] * r * inv_d;
        float rz = 0.f, mz = 0.f;
        if constexpr (POST) {
            rz = rsqrtf(s[2] * inv_d + a.eps);
            mz = rz * inv_d * (s[3] + r * (s[4] - r * m * s[5]));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (t + i * TPR);
            const size_t at = (size_t)row * a.D + c;
            float dx[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = x[i][j] * r, d = dx2[i][j] + r * (y[i][j] * w[i][j] - n * m);
                dw[i][j] = fmaf(y[i][j], n, dw[i][j]);
                dx[j] = a.rho * d;
                if constexpr (POST) {
                    const float nz = z[i][j] * rz;
                    de[i][j] = fmaf(d, nz, de[i][j]);
                    dz[j] = rz * (d * gt[i][j] * wp[i][j] - nz * mz);
                }
            }
            if (c < a.D) {
                st8<T>(static_cast<T*>(a.dx) + at, dx);
                if constexpr (POST) st8<T>(static_cast<T*>(a.dz) + at, dz);
            }
        }
        if (V > 1) load(row + step);
    }
    // partial sums [2][gridDim.x][D]; the warps of a CTA in their order
    extern __shared__ float acc[];
    for (int p = 0; p < (POST ? 2 : 1); ++p) {
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
                            if constexpr (POST) v = p == 0 ? v : de[i][j];
                            if constexpr (TPR > 32) out[c + j] = v;
                            else if (g == 0) acc[c + j] = v;
                            else if (g < RPC - 1) acc[c + j] += v;
                            else out[c + j] = acc[c + j] + v;
                        }
                }
            if constexpr (TPR == 32) __syncthreads();
        }
    }
    griddep_launch();
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename TO, typename T, int LANES>
cudaError_t gated_go(const GatedArgs& a, float* dw, bool back, cudaStream_t st) {
    const long long per = kThreads / LANES, ctas = (a.rows + per - 1) / per;
    if (!back) return launch_kernel(gated_norm_kernel<TO, T, LANES>, dim3((unsigned)ctas), dim3(kThreads), 0, st, false, a);
    const int n = (int)(ctas < kGatedCtas ? ctas : kGatedCtas);
    cudaError_t e = launch_kernel(gated_norm_back_kernel<TO, T, LANES>, dim3((unsigned)n), dim3(kThreads), 0, st, false, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(sum_rows_kernel<T>, dim3((a.d + 31) / 32, 1), dim3(1024), 0, st, true, (const float*)a.part, n, a.d, dw,
                         (const T*)nullptr, (float*)nullptr, (const T*)nullptr, (float*)nullptr);
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

template <typename T, int TPR, int V, bool POST>
cudaError_t block_go(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, cudaStream_t st) {
    constexpr int threads = kBlockThreads<TPR>;
    const long long per = threads / TPR, ctas = (a.rows + per - 1) / per;
    if (!back) return launch_kernel(block_norm_kernel<T, TPR, V, POST>, dim3((unsigned)ctas), dim3(threads), 0, st, false, a);
    const int n = (int)(ctas < block_ctas(threads) ? ctas : block_ctas(threads));
    cudaError_t e = launch_kernel(block_norm_back_kernel<T, TPR, V, POST>, dim3((unsigned)n), dim3(threads),
                                  TPR == 32 ? (size_t)a.D * 4 : 0, st, false, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(sum_rows_kernel<T>, dim3((a.D + 31) / 32, POST ? 2 : 1), dim3(1024), 0, st, true, (const float*)a.part, n,
                         a.D, dw, static_cast<const T*>(a.gate), dwp, static_cast<const T*>(a.wp), dgate);
}

// The fewest threads that hold a row in one vector of eight values each, past 4096 values in two.  The gradients
// of two spill (with the post-norm bf16 304 bytes of stores a thread, fp32 440) and read no row ahead: 2048 x 8192 97 us (2.1 TB/s)
// in bf16 and 132 (3.1) in fp32, 3200 x 5120, where a quarter of the vectors is past the row's end, 122 and 151;
// 4096 x 4096 in one vector 53 and 110.
template <typename T, bool POST>
cudaError_t block_v(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, cudaStream_t st) {
    if (a.D <= 256) return block_go<T, 32, 1, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 1024) return block_go<T, 128, 1, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 2048) return block_go<T, 256, 1, POST>(a, dw, dwp, dgate, back, st);
    if (a.D <= 4096) return block_go<T, 512, 1, POST>(a, dw, dwp, dgate, back, st);
    return block_go<T, 512, 2, POST>(a, dw, dwp, dgate, back, st);
}

cudaError_t block(const BlockArgs& a, float* dw, float* dwp, float* dgate, bool back, int dtype, cudaStream_t st) {
    if (dtype == GDN_DTYPE_F32)
        return a.z != nullptr ? block_v<float, true>(a, dw, dwp, dgate, back, st) : block_v<float, false>(a, dw, dwp, dgate, back, st);
    return a.z != nullptr ? block_v<__nv_bfloat16, true>(a, dw, dwp, dgate, back, st)
                          : block_v<__nv_bfloat16, false>(a, dw, dwp, dgate, back, st);
}

constexpr int kMaxWidth = 8192;          // D of the block norm: two vectors for each of 512 threads
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
    const long long most = block_ctas(width <= 1024 ? 128 : width <= 2048 ? 256 : 512);
    *bytes = align_up((size_t)(rows < most ? rows : most) * 2 * width * 4, kSectionAlign);
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

// gdn_seq_tc.cu -- the gated delta rule over packed sequences on the tensor core (bf16 inputs,
// d_k a multiple of 64): forward pass.
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
// two bf16 terms for the first product; r and bt eps as three.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_seq_tc.cuh"

namespace gdn {

using namespace seqtc;

namespace {

// ---------------------------------------------------------------------------
// seq_prep_kernel: That, Phat and the gates of one (chunk, head)
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kLd = kChunk + 1;

template <int DK>
struct PrepGeom {
    static constexpr uint32_t kTile = 128 * 128;                 // [K; Q], 64 columns
    static constexpr uint32_t kKQ = (DK / 64) * kTile;
    static constexpr uint32_t kMats = 3 * kChunk * kLd * 4;      // A, T, P in fp32 over the tiles
    static constexpr uint32_t kBuf = kKQ > kMats ? kKQ : ((kMats + 1023) & ~1023u);
    static constexpr uint32_t kSmem = kBuf + 2048 + 1024;
};

template <int DK>
__global__ void __launch_bounds__(kPrepThreads)
    seq_prep_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, SeqArgs a, char* ops) {
    using G = PrepGeom<DK>;
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    float* A = reinterpret_cast<float*>(sm);
    float* T = A + kChunk * kLd;
    float* P = T + kChunk * kLd;
    float* ghi = reinterpret_cast<float*>(sm + G::kBuf);
    float* glo = ghi + kChunk;
    float* bt = glo + kChunk;
    uint32_t* holder = reinterpret_cast<uint32_t*>(bt + kChunk);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const uint32_t bar = base + G::kBuf + 1024, bar2 = bar + 8;

    const SeqShape& sh = a.sh;
    const int h = blockIdx.x % sh.H, slot = blockIdx.x / sh.H, hk = h / (sh.H / sh.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int s, first, rows;
    if (!slot_chunk(sh, slot, s, first, rows, a.err)) {
        griddep_launch();
        return;
    }
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar2, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        fence_proxy_async_smem();
        mbar_expect_tx(bar, G::kKQ);
#pragma unroll
        for (int b = 0; b < DK / 64; ++b) {
            tma_2d(base + b * G::kTile, &tmK, hk * DK + 64 * b, first, bar);
            tma_2d(base + b * G::kTile + 8192, &tmQ, hk * DK + 64 * b, first, bar);
        }
    }
    if (warp == 1) tmem_alloc(smem_u32(holder), 64);
    if (warp == 2) {
        // inclusive sum of the log gates in 64 bits, kept as two floats: differences of far tokens
        double x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i;
            x[i] = t < rows ? (double)gate_log(a.la[((size_t)first + t) * sh.H + h]) : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, x[i], o);
                if (lane >= o) x[i] += y;
            }
        }
        x[1] += __shfl_sync(0xffffffffu, x[0], 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i;
            ghi[t] = (float)x[i];
            glo[t] = (float)(x[i] - (double)(float)x[i]);
            bt[t] = t < rows ? a.beta[((size_t)first + t) * sh.H + h] : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    if (tid == 0) {
        if (wait_or_dead(bar, 0, a.err, dead)) {
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const uint32_t t = base + (k / 4) * G::kTile + 32 * (k % 4);
                mma_bf16(tmem, k_desc<128>(t), k_desc<128>(t), idesc_bf16(128, 64), k != 0);
            }
        }
        mma_commit(bar2);
    }
    wait_or_dead(bar2, 0, a.err, dead);
    __syncwarp();
    tc_fence_after();
    // row t of K K^T (lanes 0..63) and of Q K^T (lanes 64..127); 32 columns for each half of the warps
    {
        const int t = 32 * (warp & 1) + lane, c0 = 32 * (warp >> 2);
        uint32_t d[32];
        tmem_ld_n(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c0, d);
        tmem_wait_ld();
        float* out = (warp & 2) ? P : A;
        const int strict = (warp & 2) ? 0 : 1;
        const float gh = ghi[t], gl = glo[t];
        float* row = out + t * kLd + c0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int c = c0 + j;
            // outside the mask the exponent may be large: it is not evaluated there.  A token past the
            // sequence's end has beta 0 and is selected away, whatever lies in its q and k
            float x = 0.f;
            if (c + strict <= t && t < rows) x = __uint_as_float(d[j]) * expf((gh - ghi[c]) + (gl - glo[c])) * bt[c];
            row[j] = x;
        }
    }
    tc_fence_before();
    __syncthreads();
    // That = (I + A)^-1: blocks of 16 on the diagonal by substitution, a column for each thread
    if (lane < 16 && warp < 4) {
        const int o = 16 * warp;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (k < i) y = fmaf(-A[(o + i) * kLd + o + k], x[k], y);
            x[i] = y;
            T[(o + i) * kLd + o + lane] = y;
        }
    } else if (warp >= 4) {
        // above the diagonal blocks That is zero
        for (int i = tid - 128; i < kChunk * kChunk; i += 128) {
            const int t = i / kChunk, c = i % kChunk;
            if (c / 16 > t / 16) T[t * kLd + c] = 0.f;
        }
    }
    __syncthreads();
    // then blocks of 32 and 64: lower left = - T22 (A21 T11); A21 T11 goes over A21
#pragma unroll
    for (int b = 16; b < kChunk; b *= 2) {
        const int n = (kChunk / (2 * b)) * b * b;
        float y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = tid + u * kPrepThreads;
            y[u] = 0.f;
            if (i < n) {
                const int blk = i / (b * b), t = (i / b) % b, c = i % b, o = blk * 2 * b;
                for (int k = c; k < b; ++k) y[u] = fmaf(A[(o + b + t) * kLd + o + k], T[(o + k) * kLd + o + c], y[u]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = tid + u * kPrepThreads;
            if (i < n) A[(i / (b * b) * 2 * b + b + (i / b) % b) * kLd + i / (b * b) * 2 * b + i % b] = y[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = tid + u * kPrepThreads;
            if (i < n) {
                const int blk = i / (b * b), t = (i / b) % b, c = i % b, o = blk * 2 * b;
                float z = 0.f;
                for (int k = 0; k <= t; ++k) z = fmaf(-T[(o + b + t) * kLd + o + b + k], A[(o + b + k) * kLd + o + c], z);
                T[(o + b + t) * kLd + o + c] = z;
            }
        }
        __syncthreads();
    }
    // Phat = (P diag(beta)) That, four rows and four columns for each thread
    {
        const int t0 = 4 * (tid / 16), c0 = 4 * (tid % 16);
        float y[4][4] = {};
        for (int k = c0; k < t0 + 4; ++k) {
            float u[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = P[(t0 + i) * kLd + k];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = T[k * kLd + c0 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[i][j] = fmaf(u[i], w[j], y[i][j]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) P[(t0 + i) * kLd + c0 + j] = y[i][j];
    }
    __syncthreads();
    char* op = ops + (size_t)blockIdx.x * kOpBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * i, c = tid & 7;
        const float* x = (r < 64 ? T + r * kLd : P + (r - 64) * kLd) + 8 * c;
        uint32_t p[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_pair<2>(x[2 * j], x[2 * j + 1], p[j]);
        char* at = op + sw_piece<128>(r, c);
        *reinterpret_cast<uint4*>(at) = make_uint4(p[0][0], p[1][0], p[2][0], p[3][0]);
        *reinterpret_cast<uint4*>(at + 16384) = make_uint4(p[0][1], p[1][1], p[2][1], p[3][1]);
    }
    float* gates = reinterpret_cast<float*>(op + kOpImage);
    const float eh = ghi[rows - 1], el = glo[rows - 1];
    if (tid < 64) {
        gates[tid] = expf(ghi[tid] + glo[tid]);
        gates[64 + tid] = bt[tid] * expf((eh - ghi[tid]) + (el - glo[tid]));
        if (tid == 0) gates[128] = expf(eh + el);
    }
    griddep_launch();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------------------
// seq_fwd_kernel
// ---------------------------------------------------------------------------
template <int DK, int NV>
struct FwdGeom {
    static constexpr int kMH = DK > 128 ? 2 : 1;                  // halves of 128 rows of d_k
    static constexpr int kW = NV * 2;                             // bytes of an operand row
    static constexpr uint32_t kTile = 128 * 128;                  // [K; Q], 64 columns of d_k
    static constexpr uint32_t kStage = 2 * kMH * kTile;           // d_k filled up to 128 or 256
    static constexpr uint32_t kTP = 2 * kStage;
    static constexpr uint32_t kS = kTP + kOpImage;                // two terms
    static constexpr uint32_t kSTerm = DK * kW;
    static constexpr uint32_t kR = kS + 2 * kSTerm;               // three terms
    static constexpr uint32_t kRTerm = 64 * kW;
    static constexpr uint32_t kBar = kR + 3 * kRTerm;
    static constexpr uint32_t kSmem = kBar + 256 + 1024;
    static constexpr int kD1 = 0, kD2 = 2 * NV, kD3 = kD2 + 3 * NV, kCols = kD3 + kMH * 3 * NV;
    static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kSmem <= 227 * 1024, "tile");
};
constexpr int kFwdThreads = 288;          // eight warps that compute, one that copies

// More than one CTA per SM must not ask for more than the 512 columns of its TMEM.
template <int DK, int NV>
constexpr size_t fwd_smem() {
    using G = FwdGeom<DK, NV>;
    const size_t least = G::kAlloc == 512 ? 116 * 1024 : G::kAlloc == 256 ? 78 * 1024 : 48 * 1024;
    return G::kSmem > least ? G::kSmem : least;
}

template <int DK, int NV>
__global__ void __launch_bounds__(kFwdThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, SeqArgs a, const char* ops,
                   char* recS, char* recE) {
    using G = FwdGeom<DK, NV>;
    constexpr int W = G::kW, NH = NV / 2;                 // NH: value columns of a thread in the token steps
    constexpr int SC = G::kMH == 2 ? NV : NH;             // value columns of a thread's state row
    extern __shared__ unsigned char raw[];
    const uint32_t r0 = smem_u32(raw), base = (r0 + 1023u) & ~1023u;
    unsigned char* sm = raw + (base - r0);
    const uint32_t full0 = base + G::kBar, empty0 = full0 + 16, tpf = full0 + 32, tpe = full0 + 40, b1 = full0 + 48,
                   b2 = full0 + 56, b3 = full0 + 64, drain = full0 + 72;
    uint32_t* holder = reinterpret_cast<uint32_t*>(sm + G::kBar + 128);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const SeqShape& sh = a.sh;
    const int tiles = sh.dv / NV;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % sh.H, s = blockIdx.x / (tiles * sh.H);
    const int hk = h / (sh.H / sh.Hk), v0 = tile * NV;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int first, len;
    if (!seq_range(sh, s, first, len, a.err)) return;     // the whole CTA
    const int chunks = (len + kChunk - 1) / kChunk;
    const size_t slot0 = (size_t)(first / kChunk + s);

    if (tid == 0) {
        for (int i = 0; i < 10; ++i) mbar_init(full0 + 8 * i, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (DK % 128 != 0) {                                  // columns of d_k that no copy fills
        for (int st = 0; st < 2; ++st)
            for (uint32_t o = tid * 16; o < G::kTile; o += kFwdThreads * 16)
                st_shared16(base + st * G::kStage + (DK / 64) * G::kTile + o, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 8) tmem_alloc(smem_u32(holder), G::kAlloc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;

    if (warp == 8) {
        griddep_wait();
        if (lane == 0) {
            int issued = 0, ops_issued = 0;
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                if (c >= 2 && !wait_or_dead(empty0 + 8 * st, ((c >> 1) & 1) ^ 1, a.err, dead)) break;
                const uint32_t kq = base + st * G::kStage, f = full0 + 8 * st;
                mbar_expect_tx(f, 2 * DK * 128);
#pragma unroll
                for (int b = 0; b < DK / 64; ++b) {
                    tma_2d(kq + b * G::kTile, &tmK, hk * DK + 64 * b, first + c * kChunk, f);
                    tma_2d(kq + b * G::kTile + 8192, &tmQ, hk * DK + 64 * b, first + c * kChunk, f);
                }
                issued = c + 1;
                if (c >= 1 && !wait_or_dead(tpe, (c - 1) & 1, a.err, dead)) break;
                mbar_expect_tx(tpf, kOpImage);
                bulk_copy_g2s(base + G::kTP, ops + ((slot0 + c) * sh.H + h) * kOpBytes, kOpImage, tpf);
                ops_issued = c + 1;
            }
            if (*dead) {                                  // copies in flight land before the CTA ends
                for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) mbar_wait(full0 + 8 * (c & 1), (c >> 1) & 1, a.err);
                if (ops_issued > 0) mbar_wait(tpf, (ops_issued - 1) & 1, a.err);
            }
        }
        __syncwarp();
    } else {
        const int wg = warp >> 2, w4 = warp & 3;
        const bool reads_k = w4 < 2;                      // token rows of K, else of Q
        const int tok = 32 * (w4 & 1) + lane, vc = wg * NH;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const int srow = (G::kMH == 2 ? 128 * wg : 0) + 32 * w4 + lane, scol = G::kMH == 2 ? 0 : wg * NH;
        const bool owns = srow < DK;
        const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + (size_t)h * sh.dv + v0 + vc;
        float S[SC];
        {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * DK + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) S[j] = owns && a.S0 != nullptr ? a.S0[at + (size_t)j * DK] : 0.f;
        }
        uint4 vr[NH / 8];
        auto load_v = [&](int c) {
            const int t = c * kChunk + tok;
#pragma unroll
            for (int i = 0; i < NH / 8; ++i)
                vr[i] = reads_k && t < len ? reinterpret_cast<const uint4*>(vp + ((size_t)first + t) * sh.ldv)[i] : make_uint4(0, 0, 0, 0);
        };
        float eg_n = 0.f, bt_n = 0.f, ee_n = 0.f;
        auto load_gates = [&](int c) {
            const float* g = reinterpret_cast<const float*>(ops + ((slot0 + c) * sh.H + h) * kOpBytes + kOpImage);
            eg_n = g[tok];
            bt_n = g[64 + tok];
            ee_n = g[128];
        };
        load_v(0);
        griddep_wait();
        if (chunks > 0) load_gates(0);
        for (int c = 0; c < chunks; ++c) {
            const uint32_t ph = c & 1, kq = base + (c & 1) * G::kStage;
            const int rows = min(kChunk, len - c * kChunk);
            const float eg = eg_n, bt = bt_n, ee = ee_n;
            // the state as the first product's operand: rows of d_k, value columns along the row
            if (owns) put_terms<W, 2>(base + G::kS, G::kSTerm, srow, scol, S);
            if (rows < kChunk) {
                // the copies brought tokens of what lies behind: rows of zero instead
                wait_or_dead(full0 + 8 * (c & 1), (c >> 1) & 1, a.err, dead);
                for (int i = tid; i < (DK / 64) * 2 * (kChunk - rows) * 8; i += 256) {
                    const int p = i & 7, r = rows + (i >> 3) % (kChunk - rows), b = (i >> 3) / (kChunk - rows);
                    st_shared16(kq + b * 8192 + r * 128 + p * 16, 0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            named_sync(1, 256);
            tc_fence_after();
            if (tid == 0) {
                if (wait_or_dead(full0 + 8 * (c & 1), (c >> 1) & 1, a.err, dead))
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_bf16(tmem + G::kD1, k_desc<128>(kq + (k / 4) * G::kTile + 32 * (k % 4)),
                                 mn_desc<W>(base + G::kS + k * 16 * W, G::kSTerm), idesc_bf16(128, 2 * NV) | kBMn, k != 0);
                mma_commit(b1);
                if (recS != nullptr)
                    bulk_s2g(recS + (((slot0 + c) * sh.H + h) * tiles + tile) * (2 * G::kSTerm), base + G::kS, 2 * G::kSTerm);
            }
            wait_or_dead(b1, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            float x[NH];
            tmem_sum<NH, 2>(tmem + G::kD1 + lanes + vc, NV, x);
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
                fence_proxy_async_smem();
                tc_fence_before();
                named_sync(2, 128);
                tc_fence_after();
                if (tid == 0) {
                    if (wait_or_dead(tpf, ph, a.err, dead)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + G::kD2, k_desc<128>(base + G::kTP + 32 * k),
                                     mn_desc<W>(base + G::kR + k * 16 * W, G::kRTerm), idesc_bf16(128, 3 * NV) | kBMn, k != 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + G::kD2, k_desc<128>(base + G::kTP + 16384 + 32 * k),
                                     mn_desc<W>(base + G::kR + k * 16 * W, G::kRTerm), idesc_bf16(128, 2 * NV) | kBMn, 1);
                    }
                    mma_commit(b2);
                    mma_commit(tpe);
                }
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
                fence_proxy_async_smem();
                tc_fence_before();
                if (tid == 0 && recS != nullptr) bulk_read_done();   // S's image is read: it may be written again
                named_sync(2, 128);
                tc_fence_after();
                if (tid == 0) {
                    if (!*dead)
#pragma unroll
                        for (int m = 0; m < G::kMH; ++m)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16(tmem + G::kD3 + m * 3 * NV, mn_desc<128>(kq + 2 * m * G::kTile + k * 2048, G::kTile),
                                         mn_desc<W>(base + G::kR + k * 16 * W, G::kRTerm),
                                         idesc_bf16(128, 3 * NV) | kAMn | kBMn, k != 0);
                    mma_commit(b3);
                    mma_commit(empty0 + 8 * (c & 1));
                }
                __syncwarp();
                if (recE != nullptr) {                    // eps as two bf16 terms [2][64][dv]
                    char* e = recE + ((slot0 + c) * sh.H + h) * (size_t)(2 * kChunk * 2) * sh.dv + ((size_t)tok * sh.dv + v0 + vc) * 2;
#pragma unroll
                    for (int i = 0; i < NH / 8; ++i) {
                        uint32_t p[4][2];
#pragma unroll
                        for (int j = 0; j < 4; ++j) split_pair<2>(y[8 * i + 2 * j], y[8 * i + 2 * j + 1], p[j]);
                        *reinterpret_cast<uint4*>(e + 16 * i) = make_uint4(p[0][0], p[1][0], p[2][0], p[3][0]);
                        *reinterpret_cast<uint4*>(e + (size_t)kChunk * 2 * sh.dv + 16 * i) = make_uint4(p[0][1], p[1][1], p[2][1], p[3][1]);
                    }
                }
                if (c + 1 < chunks) load_v(c + 1);
            } else if (tok < rows) {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (((size_t)first + c * kChunk + tok) * sh.H + h) * sh.dv + v0 + vc;
#pragma unroll
                for (int i = 0; i < NH / 8; ++i) {
                    uint32_t p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[j] = pack_bf16(fmaf(eg, x[8 * i + 2 * j], y[8 * i + 2 * j]), fmaf(eg, x[8 * i + 2 * j + 1], y[8 * i + 2 * j + 1]));
                    *reinterpret_cast<uint4*>(o + 8 * i) = make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
            if (c + 1 < chunks) load_gates(c + 1);
            wait_or_dead(b3, ph, a.err, dead);
            __syncwarp();
            tc_fence_after();
            {
                float d[SC];
                tmem_sum<SC, 3>(tmem + G::kD3 + (G::kMH == 2 ? wg * 3 * NV : 0) + lanes + scol, NV, d);
#pragma unroll
                for (int j = 0; j < SC; ++j) S[j] = fmaf(ee, S[j], d[j]);
            }
        }
        if (a.S_T != nullptr && owns) {
            const size_t at = (((size_t)s * sh.H + h) * sh.dv + v0 + scol) * DK + srow;
#pragma unroll
            for (int j = 0; j < SC; ++j) a.S_T[at + (size_t)j * DK] = S[j];
        }
        if (tid == 0) {
            if (recS != nullptr) bulk_all_done();
            if (*dead) {                                  // products in flight end before their TMEM is freed
                mma_commit(drain);
                mbar_wait(drain, 0, a.err);
            }
        }
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
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

// Rows of tokens, 64 columns (128 bytes, swizzled) x 64 tokens a box.
bool token_map(CUtensorMap* m, const void* p, int total, int width, int ld) {
    const auto enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)total}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)kChunk}, estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK>
cudaError_t prep_go(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, char* ops, cudaStream_t st) {
    static bool done[64];
    cudaError_t e = ensure_smem(seq_prep_kernel<DK>, PrepGeom<DK>::kSmem, done);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)seq_slots(a.sh.nseq, a.sh.total) * a.sh.H);
    return launch_kernel(seq_prep_kernel<DK>, dim3(grid), dim3(kPrepThreads), PrepGeom<DK>::kSmem, st, false, q, k, a, ops);
}

template <int DK, int NV>
cudaError_t fwd_go(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, char* ops, char* recS, char* recE, cudaStream_t st) {
    static bool done[64];
    cudaError_t e = ensure_smem(seq_fwd_kernel<DK, NV>, fwd_smem<DK, NV>(), done);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((size_t)a.sh.nseq * a.sh.H * (a.sh.dv / NV));
    return launch_kernel(seq_fwd_kernel<DK, NV>, dim3(grid), dim3(kFwdThreads), fwd_smem<DK, NV>(), st, true, q, k, a, (const char*)ops,
                         recS, recE);
}

template <int DK>
cudaError_t forward_dk(const CUtensorMap& q, const CUtensorMap& k, const SeqArgs& a, char* ops, char* recS, char* recE, cudaStream_t st) {
    const cudaError_t e = prep_go<DK>(q, k, a, ops, st);
    if (e != cudaSuccess) return e;
    return seq_tc_cols(a.sh) == 32 ? fwd_go<DK, 32>(q, k, a, ops, recS, recE, st) : fwd_go<DK, 16>(q, k, a, ops, recS, recE, st);
}

}  // namespace

bool seq_tc_takes(const SeqShape& s, int dtype) { return dtype == GDN_DTYPE_BF16 && s.dk % 64 == 0; }

int seq_tc_cols(const SeqShape& s) {
    return s.dv % 32 == 0 && (size_t)s.nseq * s.H * (s.dv / 16) > 152 ? 32 : 16;
}

cudaError_t launch_seq_forward_tc(const SeqArgs& a, cudaStream_t st) {
    const SeqLayout L = seq_layout(a.sh, GDN_DTYPE_BF16);
    char* ops = a.rec != nullptr ? a.rec + L.rec_op : a.ws + L.ws_op;
    char* recS = a.rec != nullptr ? a.rec + L.rec_S : nullptr;
    char* recE = a.rec != nullptr ? a.rec + L.rec_eps : nullptr;
    CUtensorMap q, k;
    if (!token_map(&q, a.q, a.sh.total, a.sh.Hk * a.sh.dk, a.sh.ldq) || !token_map(&k, a.k, a.sh.total, a.sh.Hk * a.sh.dk, a.sh.ldk))
        return cudaErrorInvalidValue;
    switch (a.sh.dk) {
        case 64: return forward_dk<64>(q, k, a, ops, recS, recE, st);
        case 128: return forward_dk<128>(q, k, a, ops, recS, recE, st);
        case 192: return forward_dk<192>(q, k, a, ops, recS, recE, st);
        default: return forward_dk<256>(q, k, a, ops, recS, recE, st);
    }
}

}  // namespace gdn

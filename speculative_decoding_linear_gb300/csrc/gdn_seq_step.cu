// gdn_seq_step.cu -- one token of the gated delta rule for each sequence of a batch, the states
// of a pool updated in place (single-token decode):
//   S' = e^{la} S,  eps = v - S' k,  S = S' + beta eps k^T,  o = S q
//
// Bound by the state: 8 bytes of traffic for each of its elements against 7 operations, each
// row of S (one value index) independent.  A warp takes four rows, each lane 16-byte pieces of
// them, so that a row is read and written once, in whole 128-byte lines, and the two dot
// products of a row stay inside the warp.  64 rows of a batch, 56 of them live, 8 heads of 256: 39 us, 6.0 TB/s
// (89 % of a copy); one row 2.4 us.
#include "gdn_seq.cuh"

namespace gdn {
namespace {

constexpr int kRows = 16;        // value rows per CTA: four warps of four

struct StepArgs {
    const void *q, *k, *v;
    const float *la, *beta;
    float* S;
    const int32_t* index;
    void* out;
    int B, slots, H, Hk, dk, dv;
    int* err;
};

template <typename T>
__global__ void __launch_bounds__(128) seq_step_kernel(StepArgs a) {
    const int tiles = a.dv / kRows;
    const int tile = blockIdx.x % tiles, h = (blockIdx.x / tiles) % a.H, b = blockIdx.x / (tiles * a.H);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * kRows + warp * 4, hk = h / (a.H / a.Hk);
    const int at = a.index != nullptr ? a.index[b] : b;
    T* out = static_cast<T*>(a.out) + ((size_t)b * a.H + h) * a.dv + row0;
    if (at < 0 || at >= a.slots) {          // an empty row of the batch, or an index that is none
        if (at != -1 && threadIdx.x == 0) set_error(a.err, GDN_ERR_INDEX);
        if (lane < 4) st_elem<T>(out, lane, 0.f);
        return;
    }
    float* S = a.S + (((size_t)at * a.H + h) * a.dv + row0) * a.dk;
    const T* q = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * a.dk;
    const T* k = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * a.dk;
    float4 x[4][2], kt[2], qt[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 128 * j + 4 * lane;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r][j] = c < a.dk ? *reinterpret_cast<const float4*>(S + (size_t)r * a.dk + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        kt[j] = c < a.dk ? ld4<T>(k, c) : make_float4(0.f, 0.f, 0.f, 0.f);
        qt[j] = c < a.dk ? ld4<T>(q, c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float4 v4 = ld4<T>(static_cast<const T*>(a.v) + ((size_t)b * a.H + h) * a.dv + row0, 0);
    const float vt[4] = {v4.x, v4.y, v4.z, v4.w};
    const float ea = expf(gate_log(a.la[(size_t)b * a.H + h])), bt = a.beta[(size_t)b * a.H + h];
    float o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float4& s = x[r][j];
            s.x *= ea; s.y *= ea; s.z *= ea; s.w *= ea;
            d += s.x * kt[j].x + s.y * kt[j].y + s.z * kt[j].z + s.w * kt[j].w;
        }
        const float de = bt * (vt[r] - warp_sum(d));
        d = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float4& s = x[r][j];
            s.x = fmaf(de, kt[j].x, s.x); s.y = fmaf(de, kt[j].y, s.y);
            s.z = fmaf(de, kt[j].z, s.z); s.w = fmaf(de, kt[j].w, s.w);
            d += s.x * qt[j].x + s.y * qt[j].y + s.z * qt[j].z + s.w * qt[j].w;
            const int c = 128 * j + 4 * lane;
            if (c < a.dk) *reinterpret_cast<float4*>(S + (size_t)r * a.dk + c) = s;
        }
        o[r] = warp_sum(d);
    }
    if (lane < 4) st_elem<T>(out, lane, lane == 0 ? o[0] : lane == 1 ? o[1] : lane == 2 ? o[2] : o[3]);
}

bool given(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// gates and indices are read one by one: any row of a larger tensor will do
bool words(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dim_ok(int d) { return d >= 16 && d <= kMaxDim && d % 16 == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return x != nullptr && y != nullptr && x < y + nb && y < x + na;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int gdn_seq_step(const void* q, const void* k, const void* v, int dtype, const float* log_alpha,
                            const float* beta, float* S, const int32_t* state_index, void* out, int B, int slots,
                            int H, int Hk, int dk, int dv, cudaStream_t stream) {
    if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32) return GDN_ERR_ARG;
    if (B < 1 || slots < 1 || H < 1 || Hk < 1 || H % Hk != 0 || !dim_ok(dk) || !dim_ok(dv)) return GDN_ERR_ARG;
    if ((long long)B * H * (dv / kRows) > 0x7fffffffLL) return GDN_ERR_ARG;
    if (state_index == nullptr && slots < B) return GDN_ERR_ARG;
    if (!given(q) || !given(k) || !given(v) || !words(log_alpha) || !words(beta) || !given(S) || !given(out) ||
        (state_index != nullptr && !words(state_index)))
        return GDN_ERR_ARG;
    const size_t e = elem_bytes(dtype), sb = (size_t)slots * H * dv * dk * 4, vo = (size_t)B * H * dv * e,
                 qb = (size_t)B * Hk * dk * e, gb = (size_t)B * H * 4;
    const struct { const void* p; size_t n; } in[] = {{q, qb}, {k, qb}, {v, vo}, {log_alpha, gb}, {beta, gb},
                                                      {state_index, (size_t)B * 4}};
    for (const auto& x : in)
        if (overlap(S, sb, x.p, x.n) || overlap(out, vo, x.p, x.n)) return GDN_ERR_ARG;
    if (overlap(S, sb, out, vo)) return GDN_ERR_ARG;
    int st;
    StepArgs a = {q, k, v, log_alpha, beta, S, state_index, out, B, slots, H, Hk, dk, dv, current_error_word(&st)};
    if (a.err == nullptr) return st;
    const dim3 grid((unsigned)((size_t)B * H * (dv / kRows)));
    const cudaError_t rc = dtype == GDN_DTYPE_F32
                               ? launch_kernel(seq_step_kernel<float>, grid, dim3(128), 0, stream, false, a)
                               : launch_kernel(seq_step_kernel<__nv_bfloat16>, grid, dim3(128), 0, stream, false, a);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

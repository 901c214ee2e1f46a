// gdn_rotary.cu -- rotary positions of q and k: each pair (x, y) of a head's first `rot` elements turned by
// the angle position * frequency, and scaled:
//   x' = scale (x cos a - y sin a),  y' = scale (x sin a + y cos a)
// The inverse turns by -a, which is the gradient's way back (the turn is orthogonal).
//
// The angle keeps its full accuracy at any int32 position without a reduction: a frequency is kept as a 64-bit
// fraction of a turn, position times fraction wraps modulo one turn by itself, and the upper 32 bits of it (1.5e-9 rad)
// are the angle.  A frequency's fraction is its 24-bit significand times 2^66 / 2 pi, an exact integer product.
//
// Bound by memory: each element is read and written once.  A thread takes V pairs of one token in the registers,
// 16 bytes a load where the sizes allow, and the same pairs of one head after another, so that the angles' sines
// are formed once for several heads.
#include <math.h>

#include "gdn_checks.cuh"

namespace gdn {
namespace {

constexpr int kRotThreads = 256;

struct RotaryArgs {
    const void *q, *k;
    void *q_out, *k_out;
    long long ldq, ldk, ldqo, ldko;
    const int32_t* positions;
    const float* inv_freq;
    float scale;
    int total, H, Hk, d, rot, each;          // each: heads of a thread
    bool inverse, copy_q, copy_k;            // copy: the elements behind `rot` go to another place
};

// A frequency in turns, modulo one turn, times 2^64; NaN, infinities and sizes of 2^26 and more have none.
__device__ __forceinline__ unsigned long long turn_fraction(float f, bool& fine) {
    constexpr unsigned long long kTurn = 0xa2f9836e4e44152aull;      // 2^66 / 2 pi
    const uint32_t u = __float_as_uint(f);
    const int ex = (u >> 23) & 255;
    const unsigned long long m = (u & 0x7fffffu) | (ex > 0 ? 0x800000u : 0u);
    const int shift = 2 - ((ex > 0 ? ex : 1) - 150);                 // of the 88-bit product
    fine = shift >= 0;
    const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
    unsigned long long r = 0;
    if (shift <= 0) r = lo;
    else if (shift < 64) r = (lo >> shift) | (hi << (64 - shift));
    else if (shift < 128) r = hi >> (shift - 64);
    return u >> 31 ? 0ull - r : r;
}

template <typename T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Piece {
    T x[V];
};

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryArgs a) {
    const int units = a.d / (2 * V);
    const long long i = (long long)blockIdx.x * kRotThreads + threadIdx.x;
    const long long t = i / units;
    const int u = (int)(i - t * units);
    if (t >= a.total) return;
    const int heads = a.H + a.Hk, h0 = blockIdx.y * a.each, h1 = min(heads, h0 + a.each);
    const bool turned = u * V * 2 < a.rot;
    float cs[V], sn[V];
    if (turned) {
        const unsigned long long pos = (unsigned long long)(long long)a.positions[t];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bool fine;
            const unsigned long long w = turn_fraction(a.inv_freq[u * V + j], fine) * pos;
            // upper 32 bits as half turns in [-1, 1)
            sincospif((float)(int)(w >> 32) * 0x1p-31f, &sn[j], &cs[j]);
            sn[j] = fine ? (a.inverse ? -a.scale : a.scale) * sn[j] : __int_as_float(0x7fffffff);
            cs[j] = fine ? a.scale * cs[j] : sn[j];
        }
    }
    // the unit's two pieces: pairs side by side, or half of `rot` apart; behind `rot` its 2 V neighbours
    const int first = turned && !INTERLEAVED ? u * V : 2 * V * u, second = turned && !INTERLEAVED ? first + a.rot / 2 : first + V;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool is_q = h < a.H;
        const int hh = is_q ? h : h - a.H;
        const T* in = static_cast<const T*>(is_q ? a.q : a.k) + t * (is_q ? a.ldq : a.ldk) + (long long)hh * a.d;
        T* out = static_cast<T*>(is_q ? a.q_out : a.k_out) + t * (is_q ? a.ldqo : a.ldko) + (long long)hh * a.d;
        if (!turned && !(is_q ? a.copy_q : a.copy_k)) continue;
        const Piece<T, V> x = *reinterpret_cast<const Piece<T, V>*>(in + first), y = *reinterpret_cast<const Piece<T, V>*>(in + second);
        Piece<T, V> p = x, r = y;
        if (turned) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = INTERLEAVED ? 2 * j : j, f = INTERLEAVED ? 2 * j + 1 : j;
                const float b = ld_elem<T>(INTERLEAVED ? (e < V ? &x.x[e % V] : &y.x[e % V]) : &x.x[e], 0),
                            c = ld_elem<T>(INTERLEAVED ? (f < V ? &x.x[f % V] : &y.x[f % V]) : &y.x[f], 0);
                const float lo = b * cs[j] - c * sn[j], hi = b * sn[j] + c * cs[j];
                st_elem<T>(INTERLEAVED ? (e < V ? &p.x[e % V] : &r.x[e % V]) : &p.x[e], 0, lo);
                st_elem<T>(INTERLEAVED ? (f < V ? &p.x[f % V] : &r.x[f % V]) : &r.x[f], 0, hi);
            }
        }
        *reinterpret_cast<Piece<T, V>*>(out + first) = p;
        *reinterpret_cast<Piece<T, V>*>(out + second) = r;
    }
}

template <typename T, int V>
cudaError_t rotary_go(RotaryArgs a, bool interleaved, cudaStream_t st) {
    const long long threads = (long long)a.total * (a.d / (2 * V));
    const int heads = a.H + a.Hk;
    a.each = heads;
    const dim3 grid((unsigned)((threads + kRotThreads - 1) / kRotThreads), (unsigned)((heads + a.each - 1) / a.each));
    return launch_kernel(interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, grid, dim3(kRotThreads), 0, st, false, a);
}

// Rows of `row` elements, ld apart, of both: whether an element of one may be one of the other's.
bool rows_meet(const void* p, long long ldp, long long rowp, const void* q, long long ldq, long long rowq, int total, int e) {
    using namespace check;
    if (!overlap({p, strided_bytes(total, ldp, rowp, e)}, {q, strided_bytes(total, ldq, rowq, e)})) return false;
    if (ldp != ldq) return true;
    const long long ld = ldp * e, at = ((long long)(reinterpret_cast<intptr_t>(q) - reinterpret_cast<intptr_t>(p)) % ld + ld) % ld;
    return at < rowp * e || at + rowq * e > ld;       // columns of one wider tensor lie apart in every row
}

}  // namespace
}  // namespace gdn

using namespace gdn;
using namespace gdn::check;

extern "C" int gdn_rotary_frequencies(int rot, double base, double factor, double original, double low, double high, float* inv_freq) {
    if (rot < 2 || rot % 2 != 0 || rot > kMaxDim || !(base > 0.0) || !(factor > 0.0) || !(original >= 0.0) || inv_freq == nullptr) return GDN_ERR_ARG;
    if (!isfinite(base) || !isfinite(factor) || !isfinite(original) || !isfinite(low) || !isfinite(high)) return GDN_ERR_ARG;
    if (original > 0.0 && !(low < high)) return GDN_ERR_ARG;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot);
        double kept = 0.0;
        if (original > 0.0) kept = fmin(1.0, fmax(0.0, (original * f / 6.283185307179586 - low) / (high - low)));
        inv_freq[i] = (float)(f * kept + f / factor * (1.0 - kept));
    }
    return GDN_OK;
}

extern "C" int gdn_rotary(const void* q, int ldq, const void* k, int ldk, int dtype, const int32_t* positions, const float* inv_freq,
                          float scale, void* q_out, int ldq_out, void* k_out, int ldk_out, int total, int H, int Hk, int d, int rot,
                          int interleaved, int inverse, cudaStream_t stream) {
    if (!type_ok(dtype) || total < 0 || H < 1 || Hk < 0 || !dim_ok(d) || rot < 2 || rot > d || rot % 2 != 0) return GDN_ERR_ARG;
    if (Hk == 0 && (k != nullptr || k_out != nullptr)) return GDN_ERR_ARG;
    const int e = elem_bytes(dtype), unit = 16 / e;
    const long long rq = (long long)H * d, rk = (long long)Hk * d;
    if (ldq < rq || ldq_out < rq || ldq % unit != 0 || ldq_out % unit != 0) return GDN_ERR_ARG;
    if (Hk > 0 && (ldk < rk || ldk_out < rk || ldk % unit != 0 || ldk_out % unit != 0)) return GDN_ERR_ARG;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) || !given_words(inv_freq)) return GDN_ERR_ARG;
    if ((long long)H + Hk > 65535 || (long long)total * (d / 2) / kRotThreads + 1 > 0x7fffffffLL) return GDN_ERR_ARG;
    if (total == 0) return GDN_OK;
    if (!given(q) || !given(q_out) || !given_words(positions) || (Hk > 0 && (!given(k) || !given(k_out)))) return GDN_ERR_ARG;
    const struct { const void* p; long long ld, row; } w[] = {{q_out, ldq_out, rq}, {k_out, ldk_out, rk}}, in[] = {{q, ldq, rq}, {k, ldk, rk}};
    const Span small[] = {{positions, (size_t)total * 4}, {inv_freq, (size_t)rot * 2}};
    const int n = Hk > 0 ? 2 : 1;
    for (int i = 0; i < n; ++i) {
        const Span o = {w[i].p, strided_bytes(total, w[i].ld, w[i].row, e)};
        if (overlap(o, small[0]) || overlap(o, small[1])) return GDN_ERR_ARG;
        for (int j = 0; j < n; ++j) {
            // in place: each element is read before it is written, by the same thread
            if (i == j && w[i].p == in[j].p && w[i].ld == in[j].ld) continue;
            if (rows_meet(w[i].p, w[i].ld, w[i].row, in[j].p, in[j].ld, in[j].row, total, e)) return GDN_ERR_ARG;
        }
    }
    if (n == 2 && rows_meet(q_out, ldq_out, rq, k_out, ldk_out, rk, total, e)) return GDN_ERR_ARG;
    int st;
    if (current_error_word(&st) == nullptr) return st;      // the device is one that the library runs on
    const RotaryArgs a = {q, k, q_out, k_out, ldq, ldk, ldq_out, ldk_out, positions, inv_freq, scale, total, H, Hk, d, rot, 0,
                          inverse != 0, q_out != q, k_out != k};
    // pairs of a thread: as many as 16 bytes hold that divide half of `rot` (and so the rest of the head too)
    const int pairs = rot / 2;
    cudaError_t rc;
    if (dtype == GDN_DTYPE_F32)
        rc = pairs % 4 == 0 ? rotary_go<float, 4>(a, interleaved, stream) : pairs % 2 == 0 ? rotary_go<float, 2>(a, interleaved, stream)
                                                                                           : rotary_go<float, 1>(a, interleaved, stream);
    else
        rc = pairs % 8 == 0   ? rotary_go<__nv_bfloat16, 8>(a, interleaved, stream)
             : pairs % 4 == 0 ? rotary_go<__nv_bfloat16, 4>(a, interleaved, stream)
             : pairs % 2 == 0 ? rotary_go<__nv_bfloat16, 2>(a, interleaved, stream)
                              : rotary_go<__nv_bfloat16, 1>(a, interleaved, stream);
    return rc == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

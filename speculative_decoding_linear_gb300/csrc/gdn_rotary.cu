// gdn_rotary.cu -- rotary positions of q and k: each pair (x, y) of a head's first `rot` elements turned by
// the angle position * frequency, and scaled:
//   x' = scale (x cos a - y sin a),  y' = scale (x sin a + y cos a)
// The inverse turns by -a, which is the gradient's way back (the turn is orthogonal).
//
// The angle keeps its accuracy at any int32 position without a reduction: a frequency is kept as a 64-bit fraction of a
// turn, position times fraction wraps modulo one turn by itself, and the upper 32 bits of it are the angle.  A
// frequency's fraction is its 24-bit significand times 2^66 / 2 pi (96 bits of it), cut off below 2^-64 of a turn: twice that
// times 2^31 is 2.3e-10 turns.  The quarter turn that the angle lies next to is taken off as an integer, so that what is
// rounded to a float is at most an eighth of a turn, off by 3.7e-9 turns (as half turns up to one, 1.5e-8).
//
// Bound by memory: each element is read and written once.  A block of threads takes a few tokens: it forms their sines
// and cosines in shared memory, once for all heads, and then each thread V pairs of a head at a time, 16 bytes a load
// where the sizes allow.  Many small blocks, so that one's sines run beside another's loads: q and k of 8192 tokens, 8
// heads of 256 each, 26.6 us (5.0 TB/s, 74 % of a copy); two pieces of each thread on their way at once 30.7 us (more
// registers, fewer blocks), blocks of 256 threads 26.8 us, every thread its own sines for its 16 heads 30.6 us.
#include <math.h>

#include "gdn_checks.cuh"

namespace gdn {
namespace {

constexpr int kRotThreads = 128, kRotPieces = 2, kRotTokens = 16;      // of a block: threads, pieces of each about, tokens at most

struct RotaryArgs {
    const void *q, *k;
    void *q_out, *k_out;
    long long ldq, ldk, ldqo, ldko;
    const int32_t* positions;
    const float* inv_freq;
    float scale;
    int total, H, Hk, d, rot, tokens;        // tokens: of a block
    uint32_t by_units, by_heads;             // 2^32 / units and / heads, rounded up
    bool inverse, copy_q, copy_k;            // copy: the elements behind `rot` go to another place
};

// A frequency in turns, modulo one turn, times 2^64; NaN, infinities and sizes of 2^26 and more have none.
__device__ __forceinline__ unsigned long long turn_fraction(float f, bool& fine) {
    constexpr unsigned long long kTurn = 0xa2f9836e4e441529ull, kTurnLow = 0xfc2757d2ull;      // 2^66 / 2 pi, and its next 32 bits
    const uint32_t u = __float_as_uint(f);
    const int ex = (u >> 23) & 255;
    const unsigned long long m = (u & 0x7fffffu) | (ex > 0 ? 0x800000u : 0u);
    const int shift = 2 - ((ex > 0 ? ex : 1) - 150);                 // of the 88-bit product
    fine = shift >= 0;
    const unsigned long long low = m * kTurnLow >> 32, lo = m * kTurn + low, hi = __umul64hi(m, kTurn) + (lo < low);
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
    extern __shared__ __align__(16) float turns[];           // cosines of the block's tokens, then their sines: [tokens][rot / 2]
    const int pairs = a.rot / 2, units = a.d / (2 * V), turned_units = pairs / V, heads = a.H + a.Hk;
    const int t0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.total - t0);
    float *cs = turns, *sn = turns + a.tokens * pairs;
    for (int i = threadIdx.x; i < tokens * pairs; i += kRotThreads) {
        const int t = i / pairs, j = i - t * pairs;
        bool fine;
        const unsigned long long w = turn_fraction(a.inv_freq[j], fine) * (unsigned long long)(long long)a.positions[t0 + t];
        const uint32_t turn = (uint32_t)(w >> 32), quarter = (turn + 0x20000000u) >> 30 & 3;      // the nearest quarter
        float s, c;
        sincospif((float)(int)(turn - (quarter << 30)) * 0x1p-31f, &s, &c);      // from it, in [-1 / 4, 1 / 4) half turns
        const float y = quarter & 1 ? c : s, x = quarter & 1 ? s : c;
        sn[i] = !fine ? __int_as_float(0x7fffffff) : y * ((quarter & 2) != 0 != a.inverse ? -a.scale : a.scale);
        cs[i] = !fine ? __int_as_float(0x7fffffff) : x * (quarter + 1 & 2 ? -a.scale : a.scale);
    }
    __syncthreads();
    const int n = tokens * heads * units;
    for (uint32_t i = threadIdx.x; i < (uint32_t)n; i += kRotThreads) {
        // i = (token heads + head) units + unit; the products stay below 2^32
        const uint32_t th = units == 1 ? i : __umulhi(i, a.by_units), t = heads == 1 ? th : __umulhi(th, a.by_heads);
        const int u = i - th * units, h = th - t * heads;
        const bool turned = u < turned_units, is_q = h < a.H;
        if (!turned && !(is_q ? a.copy_q : a.copy_k)) continue;
        // the unit's two pieces: pairs side by side, or half of `rot` apart; behind `rot` its 2 V neighbours
        const int first = turned && !INTERLEAVED ? u * V : 2 * V * u, second = turned && !INTERLEAVED ? pairs : V;
        const long long token = t0 + t, off = (long long)(is_q ? h : h - a.H) * a.d + first;
        const T* in = static_cast<const T*>(is_q ? a.q : a.k) + token * (is_q ? a.ldq : a.ldk) + off;
        T* out = static_cast<T*>(is_q ? a.q_out : a.k_out) + token * (is_q ? a.ldqo : a.ldko) + off;
        const Piece<T, V> x = *reinterpret_cast<const Piece<T, V>*>(in), y = *reinterpret_cast<const Piece<T, V>*>(in + second);
        Piece<T, V> p = x, r = y;
        if (turned) {
            const int at = t * pairs + u * V;
            alignas(16) float c[V], s[V];                    // by 16 bytes, else eight lanes' words share a bank
            if constexpr (V >= 4) {
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    *reinterpret_cast<float4*>(c + j) = *reinterpret_cast<const float4*>(cs + at + j);
                    *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(sn + at + j);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    c[j] = cs[at + j];
                    s[j] = sn[at + j];
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int lo = INTERLEAVED ? 2 * j : j, hi = INTERLEAVED ? 2 * j + 1 : j;
                const float b = ld_elem<T>(INTERLEAVED ? (lo < V ? &x.x[lo % V] : &y.x[lo % V]) : &x.x[lo], 0),
                            d = ld_elem<T>(INTERLEAVED ? (hi < V ? &x.x[hi % V] : &y.x[hi % V]) : &y.x[hi], 0);
                st_elem<T>(INTERLEAVED ? (lo < V ? &p.x[lo % V] : &r.x[lo % V]) : &p.x[lo], 0, b * c[j] - d * s[j]);
                st_elem<T>(INTERLEAVED ? (hi < V ? &p.x[hi % V] : &r.x[hi % V]) : &r.x[hi], 0, b * s[j] + d * c[j]);
            }
        }
        *reinterpret_cast<Piece<T, V>*>(out) = p;
        *reinterpret_cast<Piece<T, V>*>(out + second) = r;
    }
}

template <typename T, int V>
cudaError_t rotary_go(RotaryArgs a, bool interleaved, cudaStream_t st) {
    const int units = a.d / (2 * V), heads = a.H + a.Hk;
    // tokens of a block: two pieces a thread, but one token where there are few
    const long long pieces = (long long)units * heads;
    long long t = kRotPieces * kRotThreads / pieces;
    if (t > kRotTokens) t = kRotTokens;
    if (t < 1 || a.total < 4LL * kSMs * t) t = 1;
    a.tokens = (int)t;
    a.by_units = (uint32_t)(((1ull << 32) + units - 1) / units);
    a.by_heads = (uint32_t)(((1ull << 32) + heads - 1) / heads);
    const dim3 grid((unsigned)((a.total + t - 1) / t));
    return launch_kernel(interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, grid, dim3(kRotThreads), (size_t)t * a.rot * 4, st, false, a);
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
    if ((long long)H + Hk > 65535) return GDN_ERR_ARG;
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
    const RotaryArgs a = {q, k, q_out, k_out, ldq, ldk, ldq_out, ldk_out, positions, inv_freq, scale, total, H, Hk, d, rot, 0, 0, 0,
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

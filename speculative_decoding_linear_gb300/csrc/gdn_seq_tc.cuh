// gdn_seq_tc.cuh -- operand layouts, splits and tcgen05 wrappers shared by the sequence
// operators' tensor-core kernels.
//
// An fp32 operand x enters a product as bf16 terms x = hi + mid (+ low), each the rounding of
// what the terms before it left; q, k, v and dO are bf16 already and exact.  Two terms leave at
// most 2^-16 of x (3e-6 of it in the mean square), three 2^-24.  The terms of the B operand lie
// side by side along N, so that the A operand is read once for all of them, and their products
// are added in fp32 where the accumulator is read.  A product of two split operands leaves out
// those of the small terms, 2^-16 of the whole and below.
#pragma once

#include "gdn_seq.cuh"
#include "gdn_tc_ptx.cuh"

namespace gdn {
namespace seqtc {

using namespace tc;

// N consecutive TMEM columns of this warp's 32 lanes; the caller waits (tmem_wait_ld).
__device__ __forceinline__ void tmem_ld_n(uint32_t t, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_n(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_n(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }

// Sum of T term columns (NT columns apart) of N consecutive columns.
template <int N, int T>
__device__ __forceinline__ void tmem_sum(uint32_t t, int apart, float (&x)[N]) {
    uint32_t r[T][N];
#pragma unroll
    for (int i = 0; i < T; ++i) tmem_ld_n(t + i * apart, r[i]);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        x[j] = __uint_as_float(r[T - 1][j]);        // the small terms first
#pragma unroll
        for (int i = T - 2; i >= 0; --i) x[j] += __uint_as_float(r[i][j]);
    }
}

// Shared-memory operand stored as rows (of K) of W bytes with the hardware's W-byte swizzle.
// Byte offset of 16-byte piece c of row r.
template <int W>
__device__ __forceinline__ uint32_t sw_piece(int r, int c) {
    if constexpr (W == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    if constexpr (W == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}
template <int W>
constexpr uint64_t kSwCode = W == 128 ? 2 : W == 64 ? 4 : 6;

// Descriptor of an operand whose M or N index runs along the row (MN-major): pieces of W bytes
// of it `mn_apart` bytes apart, eight rows of K together, the next eight 8 W bytes on.
template <int W>
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t mn_apart) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((mn_apart >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((8 * W) >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= kSwCode<W> << 61;
    return d;
}
// Descriptor of an operand whose K index runs along the row (K-major), rows of W bytes.
template <int W>
__device__ __forceinline__ uint64_t k_desc(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)((8 * W) >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= kSwCode<W> << 61;
    return d;
}
constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;      // instruction descriptor: operand is MN-major

__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Two values as T packed bf16 terms each; the values become what is left of them.
template <int T>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[T]) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
        p[i] = pack_bf16(a, b);
        a -= __uint_as_float(p[i] << 16);
        b -= __uint_as_float(p[i] & 0xffff0000u);
    }
}

// N values of row `row`, columns col0 .. col0 + N - 1, as T terms of a W-byte-row operand.
template <int W, int T, int N>
__device__ __forceinline__ void put_terms(uint32_t base, uint32_t term_apart, int row, int col0, const float (&x)[N]) {
#pragma unroll
    for (int c = 0; c < N / 8; ++c) {
        uint32_t p[4][T];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_pair<T>(x[8 * c + 2 * i], x[8 * c + 2 * i + 1], p[i]);
        const uint32_t at = base + sw_piece<W>(row, col0 / 8 + c);
#pragma unroll
        for (int i = 0; i < T; ++i) st_shared16(at + i * term_apart, p[0][i], p[1][i], p[2][i], p[3][i]);
    }
}

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_read_done() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_all_done() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

// Bounded wait that gives up at once after any wait of the CTA has given up.  It polls with
// test_wait: a waiting thread that try_wait suspends comes back some 340 cycles late (a product's
// end seen 160 cycles after its last instruction instead of 500), three times in a chunk.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool poll_slow(uint32_t bar, uint32_t parity, int* err, volatile int* dead) {
    const uint64_t t0 = globaltimer_ns(), limit = wait_limit_ns(err);
    while (true) {
        for (int i = 0; i < 256; ++i)
            if (mbar_test(bar, parity)) return true;
        if (*dead) return false;
        if (globaltimer_ns() - t0 > limit) {
            set_error(err, GDN_ERR_TIMEOUT);
            *dead = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_or_dead(uint32_t bar, uint32_t parity, int* err, volatile int* dead) {
#pragma unroll 1
    for (int i = 0; i < 512; ++i)
        if (mbar_test(bar, parity)) return true;
    return poll_slow(bar, parity, err, dead);
}

// A value that is the same in the whole warp, known so to the compiler, and one thread of the warp.
// tcgen05.mma takes its descriptors from uniform registers: built from values that the compiler
// knows to be uniform, an issue takes about 20 cycles, else 80 to 200 (measured), more than the
// product itself at the N of these kernels.
__device__ __forceinline__ int warp_uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
    return e != 0;
}

// n barriers behind one another, each initialised once (again, on a live one, is undefined): arrivals(its address).
template <class Arrivals>
__device__ __forceinline__ void init_barriers(uint32_t first, int n, Arrivals&& arrivals) {
    for (int i = 0; i < n; ++i) {
        const uint32_t bar = first + 8 * i;
        mbar_init(bar, arrivals(bar));
    }
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// A warp's generic writes of an operand are done, told to the warp that issues the products (which
// waits in named_sync with the same id and count).  A barrier of the SM hands over in some 30
// cycles, an mbarrier that is polled in 200 and more.
__device__ __forceinline__ void operand_ready(int id, int n) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(n) : "memory");
}

// 32 consecutive TMEM columns of this warp's 32 lanes; tmem_wait_st before they are used.
__device__ __forceinline__ void tmem_st_n(uint32_t t, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_n(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// N/8 pieces of 16 bytes that are neighbours in memory: whole sectors where there are two, with a
// 32-byte access (a warp's rows lie apart, so that half sectors cost as much as whole ones), unless the
// place is not `wide`, aligned to 16 bytes only.  `swap`: the pieces of a pair change places.
template <int P>
__device__ __forceinline__ void stg_pieces(void* p, const uint4 (&x)[P], bool swap, bool wide) {
    if constexpr (P == 1) {
        *reinterpret_cast<uint4*>(p) = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const uint4 a = swap ? x[i + 1] : x[i], b = swap ? x[i] : x[i + 1];
            if (wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(static_cast<char*>(p) + 16 * i), "r"(a.x),
                             "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                             : "memory");
            } else {
                static_cast<uint4*>(p)[i] = a;
                static_cast<uint4*>(p)[i + 1] = b;
            }
        }
    }
}
// at a 32-byte boundary
template <int P>
__device__ __forceinline__ void ldg_pieces(const void* p, uint4 (&x)[P]) {
    if constexpr (P == 1) {
        x[0] = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                         : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w), "=r"(x[i + 1].x), "=r"(x[i + 1].y), "=r"(x[i + 1].z),
                           "=r"(x[i + 1].w)
                         : "l"(static_cast<const char*>(p) + 16 * i));
        }
    }
}
// Place of a thread's NH columns from vc on in row `tok` of a W-byte operand, as stg_pieces takes them.
template <int W, int NH>
__device__ __forceinline__ uint32_t pieces_at(int tok, int vc, bool& swap) {
    const uint32_t at = sw_piece<W>(tok, vc / 8);
    swap = NH == 16 && (at & 16) != 0;
    return NH == 16 ? at & ~16u : at;
}

// Bring a box into L2; nothing waits for it.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0),
                 "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// ---------------------------------------------------------------------------
// per (slot, head): what a chunk needs of its gates and of K K^T, Q K^T
//   gates   fp32: bt = beta_t e^{g_end - g_t}, eg = e^{g_t}, e^{g_end}, tail = e^{g_end - g_t}, beta,
//           g as two floats
//   tp      [That; Phat] ([Phat; That] for a sequence's odd chunks), 128 rows of 64, 128-byte-swizzled
//           K-major, bf16 terms of 16 KiB: two, or in a record three
//   tpb     in a record: [T; Ptil] of the backward pass, three terms
// ---------------------------------------------------------------------------
constexpr uint32_t kOpGates = 2048, kOpTerm = 16384;
constexpr uint32_t kOpBytes = kOpGates + 2 * kOpTerm;       // without a record
constexpr uint32_t kOpBack = kOpGates + 3 * kOpTerm;        // tpb's place in a record
constexpr uint32_t kOpRecord = kOpBack + 3 * kOpTerm;
constexpr int kGBt = 0, kGEg = 64, kGEnd = 128, kGTail = 132, kGBeta = 196, kGHi = 260, kGLo = 324;
constexpr uint32_t kGateFwd = 528;                          // bytes that the forward scan takes
constexpr uint32_t kGateBwd = 784;                          // and the backward scan, from kGEg

}  // namespace seqtc

bool seq_tc_takes(int dtype);
inline int seq_tc_dk(int dk) { return (dk + 63) / 64 * 64; }      // d_k as the kernels keep it: zeros behind
int seq_tc_cols(const SeqShape& s);      // value columns of a CTA
cudaError_t launch_seq_forward_tc(const SeqArgs& a, cudaStream_t st);
cudaError_t launch_seq_backward_tc(const SeqArgs& a, cudaStream_t st);

}  // namespace gdn

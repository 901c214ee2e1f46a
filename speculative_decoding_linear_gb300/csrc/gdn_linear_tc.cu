// gdn_linear_tc.cu -- decay-gated linear attention over packed sequences with bf16 inputs, on the tensor core.
//
// Segments of 512 tokens, blocks of 128.  Six kinds of kernels a pass:
//   lin_prep_kernel       the decays of each segment's tokens
//   lin_local_tc_kernel   what a segment adds to the state (or to its gradient): one product over its tokens
//   lin_scan_kernel       the states between the segments (gdn_linear_seq.cu), left as bf16 terms
//   lin_rows_tc_kernel    128 rows of o, dq, dk or dv: the state's product, scaled by row, and then for each block of
//                         the segment the scores, masked and decayed, and their product
//   lin_pairs_tc_kernel   the row and column sums of (q.k)(dO.v) that the gates' gradients are made of
//   lin_gates_tc_kernel   dlog_alpha and dbeta from them
//
// Inside a segment the masked scores are formed outright, as an attention without a softmax: at 512 tokens that is
// about the work of carrying the state from block to block (10 of 16 blocks' scores and their products, against four
// products with the state and four updates in two terms), and it leaves no chain: every block of rows is on its own.
//
// Decays enter as products of numbers up to one: e^{g_t - g_s} between blocks is e^{(from t's block's start to t)} times
// e^{(from s to t's block's start)}, and inside a block a difference of sums of two floats each.
#include <cudaTypedefs.h>

#include "gdn_linear.cuh"
#include "gdn_seq_tc.cuh"

namespace gdn {
namespace {

using namespace seqtc;

constexpr int kSeg = kLinSegment, kBlk = 128;

// D (+)= A B with the A operand in TMEM: lane = row, two neighbours of K in each 32-bit column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A bounded wait with nothing called: around a call the compiler saves what a role holds, some 150 instructions a wait, and
// these kernels' roles together have to stay within the instruction cache (70 KB of code ran at a third of its time behind
// misses of it).  Gives up at once after any wait of the CTA has given up; `dead` null: by its own limit only.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, int* err, volatile int* dead) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !mbar_test(bar, parity); ++n)
        if ((n & 1023) == 0) {
            const uint64_t now = globaltimer_ns();
            if (n == 1024) t0 = now;
            if (dead != nullptr && *dead) return false;
            if (now - t0 > wait_limit_ns(err)) {
                set_error(err, GDN_ERR_TIMEOUT);
                if (dead != nullptr) *dead = 1;
                return false;
            }
        }
    return true;
}

// What the gates of a (slot, head) give, floats by token; g the sum of log decays from the segment's start to the token
// and with it, G to the segment's end, b that from the block's start, B to the block's end.
constexpr int kGCoef = 0,                    // beta e^{G - g}: what the token adds to the state at the segment's end
    kGHead = kSeg,                           // e^g
    kGTail = 2 * kSeg,                       // e^{G - g}
    kGPre = 3 * kSeg,                        // e^b
    kGPost = 4 * kSeg,                       // e^{B - b}
    kGHi = 5 * kSeg, kGLo = 6 * kSeg,        // b as two floats
    kGBeta = 7 * kSeg,                       // beta; zero behind the segment, as kGCoef
    kGTot = 8 * kSeg,                        // e^B of the four blocks, e^G
    kGAll = 8 * kSeg + 32;
// Behind the gates of all (slot, head): each slot's first token and its tokens, none for an empty slot.
__device__ __forceinline__ const int2* slot_table(const float* gates, int slots, int H) {
    return reinterpret_cast<const int2*>(gates + (size_t)slots * H * kGAll);
}

// A slot's first token and tokens; none where they are not the call's (a record that is not this call's own).
__device__ __forceinline__ int2 slot_entry(const int2* table, int slot, int total) {
    const int2 e = table[slot];
    return e.x < 0 || e.y < 0 || e.y > kSeg || e.x > total - e.y ? make_int2(0, 0) : e;
}

// Behind the table: how many slots have b blocks or more (b = 1 .. 4), and the slots by blocks, most first.  One warp, 256 slots'
// entries on their way at a time, read twice.  Others of the CTA wait for this warp, and their waits have a limit: with a pass for
// each count, a group's entries behind the stores of the one before it, 300 000 sequences of two tokens took 20.0 ms and not 13.4,
// and 4096 of four (one head of 128) 511 us and not 416.
__device__ __forceinline__ const int* slot_order(const int2* table, int slots) { return reinterpret_cast<const int*>(table + slots); }
__device__ __noinline__ void order_slots(const int2* table, int slots, int total) {
    constexpr int kMost = kSeg / kBlk, kGroups = 8;
    int* order = const_cast<int*>(slot_order(table, slots));
    const int lane = threadIdx.x & 31;
    int blocks[kGroups], n[kMost], at[kMost];             // n: slots with i + 1 blocks or more; at: place of the next with i + 1
    const auto load = [&](int s0) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int s = s0 + 32 * j + lane;
            blocks[j] = s < slots ? (slot_entry(table, s, total).y + kBlk - 1) / kBlk : 0;
        }
    };
#pragma unroll
    for (int i = 0; i < kMost; ++i) n[i] = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < slots; s0 += 32 * kGroups) {
        load(s0);
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
            for (int i = 0; i < kMost; ++i) n[i] += blocks[j] > i;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        n[i] = (int)__reduce_add_sync(0xffffffffu, (unsigned)n[i]);
        if (lane == 0) order[i] = n[i];
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) at[i] = i + 1 < kMost ? n[i + 1] : 0;
#pragma unroll 1
    for (int s0 = 0; s0 < slots; s0 += 32 * kGroups) {
        load(s0);
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                const unsigned m = __ballot_sync(0xffffffffu, blocks[j] == i + 1);
                if (blocks[j] == i + 1) order[kMost + at[i] + __popc(m & ((1u << lane) - 1))] = s0 + 32 * j + lane;
                at[i] += __popc(m);
            }
    }
}

__global__ void __launch_bounds__(kBlk) lin_prep_kernel(SeqArgs a, float* gates) {
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    const int slot = blockIdx.x / sh.H, h = blockIdx.x % sh.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int s, c, first = 0, rows = 0;
    const bool is = slot_segment(sh, kSeg, slot, s, c, first, rows, a.err);
    if (h == 0 && tid == 0) const_cast<int2*>(slot_table(gates, gridDim.x / sh.H, sh.H))[slot] = make_int2(is ? first : 0, is ? rows : 0);
    if (!is) return;
    __shared__ LogSum total[4];
    float la[4], beta[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = 4 * tid + e;
        la[e] = t < rows ? a.la[(size_t)(first + t) * sh.H + h] : 0.f;
        beta[e] = t < rows ? a.beta[(size_t)(first + t) * sh.H + h] : 0.f;
    }
    LogSum pre[4], x = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x = x + LogSum{gate_log(la[e]), 0.f};
        pre[e] = x;
    }
    const LogSum upto = warp_scan(x) - x;
#pragma unroll
    for (int e = 0; e < 4; ++e) pre[e] = pre[e] + upto;
    if (lane == 31) total[warp] = pre[3];
    __syncthreads();
    LogSum before = {0.f, 0.f}, behind = {0.f, 0.f};
    for (int b = 0; b < 4; ++b) {
        if (b < warp) before = before + total[b];
        if (b > warp) behind = behind + total[b];
    }
    float* out = gates + (size_t)blockIdx.x * kGAll;
    float y[8][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const LogSum left = total[warp] - pre[e];
        y[2][e] = decay_of(left + behind);
        y[0][e] = beta[e] * y[2][e];
        y[1][e] = decay_of(before + pre[e]);
        y[3][e] = decay_of(pre[e]);
        y[4][e] = decay_of(left);
        y[5][e] = pre[e].hi;
        y[6][e] = pre[e].lo;
        y[7][e] = beta[e];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(out + i * kSeg + 4 * tid) = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
    if (lane == 31) out[kGTot + warp] = y[3][3];
    if (tid == 0) out[kGTot + 4] = decay_of(total[0] + behind);
}

__device__ __forceinline__ float ex2(float x) {      // 2^x, to 2^-22 of it; below 2^-126 zero
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ void tmem_st_n(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
using seqtc::tmem_st_n;

// Place in a ring of n stages and the parity of its use; products are issued from values that the compiler knows to be
// the same in the whole warp (no division, no early end of a loop).
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++st == n) {
            st = 0;
            ph ^= 1;
        }
    }
};

// Tokens of a head as 64-element by 64-token boxes of shared memory, rows of 128 swizzled bytes.
constexpr uint32_t kBox = 64 * 128;

// ---------------------------------------------------------------------------
// C = sum_t c_t a_t b_t^T over a segment's tokens, in tiles of 128 rows of d_v by 128 columns of d_k; one CTA an SM takes
// tile after tile.   forward  c_t = beta_t e^{G - g_t}, a = v, b = k;   BACK  c_t = e^{g_t}, a = dO, b = q
// c_t a_t is an fp32 operand: three bf16 terms of it (2^-24 of it are left), as the sum is an fp32 output after up to
// 2^17 tokens; the terms go to TMEM, where each thread holds one row of d_v.  b is bf16 and exact.  The tensor core cuts
// off what does not fit 24 bits at each addition, always toward zero, 1.5e-8 of the sum: so a sum is of 192 tokens, and what
// follows is added to it in memory, rounded (with slow decays dS0 is 9.7e-7 off with sums of 256 tokens, 7.0e-7 of 192, 4.6e-7 of
// 128, and was 1.7e-6 in one sum of 512; 8192 tokens forward 98.8, 102 and 108 us with sums of 256, 192 and 128).
// Bound by the products, three for each of the state's, and by forming their operands: 8192 tokens of 8 heads, 256 x 256, 37 us
// (700 TFLOP/s of products, tensor core busy some 38 % of the time; a CTA has 3 or 4 of the 512 tiles).  Warps 0-7 form the terms (four warps 32
// tokens, two buffers each), 8-11 move the sums out (two in TMEM) by way of shared memory, 12 copies, 13 multiplies.
// ---------------------------------------------------------------------------
constexpr int kLocalThreads = 448, kLocalStages = 5, kLocalTok = 64, kLocalSum = 192;
constexpr int kLocalListed = 256;
constexpr uint32_t kLocalStage = 4 * kBox;                       // two boxes of a, two of b
constexpr uint32_t kLocalOut = kLocalStages * kLocalStage, kLocalCoef = kLocalOut + 128 * 128 * 4, kLocalBars = kLocalCoef + kLocalStages * kLocalTok * 4,
                   kLocalNBars = 2 * kLocalStages + 13, kLocalList = kLocalBars + 8 * kLocalNBars + 16, kLocalSmem = kLocalList + kLocalListed;
constexpr uint32_t kLocalA = 256, kLocalABuf = 48;               // TMEM: two sums, then four buffers of three terms of 16

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(reinterpret_cast<uint64_t>(map)),
                     "r"(src), "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src),
                     "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }

// The slots by their blocks of tokens, most first, where a list in shared memory holds them; one warp.
__device__ __noinline__ void list_slots(const int2* table, int slots, int total, unsigned char* list) {
    const int lane = threadIdx.x & 31;
    int blocks[kLocalListed / 32], at = 0;
#pragma unroll
    for (int j = 0; j < kLocalListed / 32; ++j) {
        const int s = 32 * j + lane;
        blocks[j] = s < slots ? (slot_entry(table, s, total).y + kBlk - 1) / kBlk : -1;
    }
#pragma unroll 1
    for (int b = kSeg / kBlk; b >= 0; --b)
#pragma unroll
        for (int j = 0; j < kLocalListed / 32; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, blocks[j] == b);
            if (blocks[j] == b) list[at + __popc(m & ((1u << lane) - 1))] = (unsigned char)(32 * j + lane);
            at += __popc(m);
        }
}
// Tile i of the launch; empty slots have none.  A CTA's tiles: one of each turn of the grid, every other turn backwards.  Where
// lengths differ (offsets are given) and up to 256 slots, the longest come first: 24 prompts of 16 000 tokens 23.8 us, in the
// slots' order 28; one of 8192 tokens 35.3 with the list, 33.8 without (sums of 256 tokens).
struct LocalItems {
    int H, tiles_v, tiles_k, slots, total;
    const int2* table;
    const unsigned char* list;             // null: the slots' order
    __device__ __forceinline__ int count() const { return slots * H * tiles_v * tiles_k; }
    __device__ __forceinline__ int first_of(int turn) const { return turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); }
    __device__ __forceinline__ int slot_of(int at) const { return list != nullptr ? list[at] : at; }
    __device__ __forceinline__ int get(int i, int& slot, int& h, int& r0, int& c0, int& first) const {
        const int tiles = tiles_v * tiles_k, t = i % tiles, sh = i / tiles;
        slot = slot_of(sh / H);
        h = sh % H;
        r0 = t / tiles_k * 128;
        c0 = t % tiles_k * 128;
        const int2 e = slot_entry(table, slot, total);
        first = warp_uniform(e.x);
        return warp_uniform(e.y);
    }
};

template <bool BACK>
__global__ void __launch_bounds__(kLocalThreads, 1)
    lin_local_tc_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mo, SeqArgs a,
                        const float* gates) {
    extern __shared__ __align__(1024) char sm[];
    const SeqShape& sh = a.sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_uniform(tid >> 5), rep = sh.H / sh.Hk;
    const int slots = seg_slots(sh.nseq, sh.total, kSeg);
    const LocalItems items = {sh.H, (sh.dv + 127) / 128, (sh.dk + 127) / 128, slots, sh.total, slot_table(gates, slots, sh.H),
                              sh.offsets != nullptr && slots <= kLocalListed ? reinterpret_cast<const unsigned char*>(sm + kLocalList) : nullptr};
    const int count = items.count();
    const uint32_t base = smem_u32(sm), bars = base + kLocalBars;
    const uint32_t full0 = bars, empty0 = bars + 8 * kLocalStages, a_full = bars + 16 * kLocalStages, a_free = a_full + 32, acc_full = a_full + 64,
                   acc_free = a_full + 80, drain = a_full + 96;
    uint32_t* holder = reinterpret_cast<uint32_t*>(sm + kLocalBars + 8 * kLocalNBars);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    if (tid == 0) {
        // full: the copy; empty: the products and the eight warps that read a; a_full, acc_free: four warps; else products
        init_barriers(bars, kLocalNBars, [&](uint32_t b) { return b >= empty0 && b < a_full ? 9u : (b >= a_full && b < a_free) || (b >= acc_free && b < drain) ? 4u : 1u; });
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 13) tmem_alloc(smem_u32(holder), 512);
    __syncthreads();
    const uint32_t tmem = warp_uniform(*holder);
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    if (items.list != nullptr) {
        if (warp == 0) list_slots(items.table, slots, sh.total, reinterpret_cast<unsigned char*>(sm + kLocalList));
        __syncthreads();
    }
    int slot, h, r0, c0, first;
    Ring ring;
    if (warp == 12) {
        if (elect_one()) {
            int issued = 0;
            bool ok = true;
            for (int turn = 0, i; ok && (i = items.first_of(turn)) < count; ++turn) {
                // one thread: no shuffles here
                const int tiles = items.tiles_v * items.tiles_k, t = i % tiles, s_h = i / tiles;
                slot = items.slot_of(s_h / sh.H);
                h = s_h % sh.H;
                r0 = t / items.tiles_k * 128;
                c0 = t % items.tiles_k * 128;
                const int2 e = slot_entry(items.table, slot, sh.total);
                const int na = (min(128, sh.dv - r0) + 63) / 64, nb = (min(128, sh.dk - c0) + 63) / 64;
                for (int k = 0; ok && k < e.y; k += kLocalTok, ring.next(kLocalStages)) {
                    const uint32_t at = base + ring.st * kLocalStage, bar = full0 + 8 * ring.st;
                    if (issued >= kLocalStages && !(ok = wait_here(empty0 + 8 * ring.st, ring.ph ^ 1, a.err, dead))) break;
                    mbar_expect_tx(bar, (na + nb) * kBox + kLocalTok * 4);
                    bulk_copy_g2s(base + kLocalCoef + ring.st * kLocalTok * 4, gates + ((size_t)slot * sh.H + h) * kGAll + (BACK ? kGHead : kGCoef) + k, kLocalTok * 4, bar);
                    for (int x = 0; x < na; ++x) tma_3d(at + x * kBox, &ma, r0 + 64 * x, h, e.x + k, bar);
                    for (int x = 0; x < nb; ++x) tma_3d(at + (2 + x) * kBox, &mb, c0 + 64 * x, h / rep, e.x + k, bar);
                    ++issued;
                }
            }
            if (*dead)                                    // copies in flight end before the CTA does
                for (int j = max(0, issued - kLocalStages); j < issued; ++j) wait_here(full0 + 8 * (j % kLocalStages), (j / kLocalStages) & 1, a.err, nullptr);
        }
        __syncwarp();
    } else if (warp == 13) {
        const bool leader = elect_one();
        uint32_t unit = 0, step = 0;                      // sums and stages so far
        for (int turn = 0, i; (i = items.first_of(turn)) < count; ++turn) {
            const int rows = items.get(i, slot, h, r0, c0, first);
            const uint32_t id = idesc_bf16(128, min(128, sh.dk - c0)) | kBMn;
            for (int k = 0; k < rows; k += kLocalTok, ring.next(kLocalStages), ++step) {
                const uint32_t acc = tmem + 128 * (unit & 1);
                const int at = k % kLocalSum;
                if (at == 0 && unit >= 2) wait_here(acc_free + 8 * (unit & 1), (unit >> 1 & 1) ^ 1, a.err, dead);
                wait_here(full0 + 8 * ring.st, ring.ph, a.err, dead);
                const uint64_t db = mn_desc<128>(base + ring.st * kLocalStage + 2 * kBox, kBox);
#pragma unroll
                for (int b = 0; b < 2; ++b) {             // 32 tokens
                    const int left = rows - k - 32 * b;
                    const uint32_t buf = 2 * b + (step & 1);
                    wait_here(a_full + 8 * buf, step >> 1 & 1, a.err, dead);
                    __syncwarp();
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            if (16 * y < left)
#pragma unroll
                                for (int t = 2; t >= 0; --t)      // the small terms first
                                    mma_bf16_ts(acc, tmem + kLocalA + buf * kLocalABuf + 16 * t + 8 * y, db + ((b * 4096 + y * 2048) >> 4), id,
                                                at + b + y > 0 || t < 2);
                        mma_commit(a_free + 8 * buf);
                        if (b == 1) mma_commit(empty0 + 8 * ring.st);
                    }
                    __syncwarp();
                }
                if (at + kLocalTok == kLocalSum || k + kLocalTok >= rows) {
                    if (leader) mma_commit(acc_full + 8 * (unit & 1));
                    __syncwarp();
                    ++unit;
                }
            }
        }
        if (leader) {                                     // products in flight end before their TMEM is freed
            mma_commit(drain);
            wait_here(drain, 0, a.err, nullptr);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int g = warp >> 2, w4 = warp & 3, r = 32 * w4 + lane, piece = r >> 3 & 7;      // 32 tokens of a stage; row of the tile
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        uint32_t step = 0;
        for (int turn = 0, i; (i = items.first_of(turn)) < count; ++turn) {
            const int rows = items.get(i, slot, h, r0, c0, first);
            for (int k = 0; k < rows; k += kLocalTok, ring.next(kLocalStages), ++step) {
                const int left = rows - k - 32 * g;
                const uint32_t buf = 2 * g + (step & 1), A = tmem + kLocalA + buf * kLocalABuf + lanes;
                wait_here(full0 + 8 * ring.st, ring.ph, a.err, dead);
                if (step >= 2) wait_here(a_free + 8 * buf, (step >> 1 & 1) ^ 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                if (left > 0 && left < 32 && left % 16 != 0) {        // tokens of what lies behind: rows of zero, up to whole products
                    for (int x = tid & 127; x < (16 - left % 16) * 16; x += 128)
                        st_shared16(base + ring.st * kLocalStage + (2 + (x >> 3 & 1)) * kBox + (32 * g + left + (x >> 4)) * 128 + (x & 7) * 16, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                const char* raw = sm + ring.st * kLocalStage + (r >> 6) * kBox + 32 * g * 128 + (r & 7) * 2;
                const float4* cf = reinterpret_cast<const float4*>(sm + kLocalCoef + ring.st * kLocalTok * 4 + 32 * g * 4);
                if (left > 0) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {            // 16 tokens
                        uint32_t u[16], p[3][8];
#pragma unroll
                        for (int t = 0; t < 16; ++t) u[t] = *reinterpret_cast<const unsigned short*>(raw + (16 * half + t) * 128 + ((piece ^ (t & 7)) << 4));
                        if (left < 32) {                  // nothing of the tokens behind (their factors are zero, they may be NaN)
#pragma unroll
                            for (int t = 0; t < 16; ++t)
                                if (16 * half + t >= left) u[t] = 0;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 f = cf[4 * half + j / 2];
                            float2 x = fmul2(j % 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y), make_float2(__uint_as_float(u[2 * j] << 16), __uint_as_float(u[2 * j + 1] << 16)));
#pragma unroll
                            for (int t = 0; t < 3; ++t) {
                                p[t][j] = pack_bf16(x.x, x.y);
                                if (t < 2) x = ffma2(make_float2(__uint_as_float(p[t][j] << 16), __uint_as_float(p[t][j] & 0xffff0000u)), make_float2(-1.f, -1.f), x);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < 3; ++t) tmem_st_n(A + 16 * t + 8 * half, p[t]);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(a_full + 8 * buf);
                    mbar_arrive(empty0 + 8 * ring.st);
                }
                __syncwarp();
            }
        }
    } else {
        const int w4 = warp & 3, r = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16, mine = base + kLocalOut + r * 128;
        if (!BACK && blockIdx.x == gridDim.x - 1 && warp == 8) order_slots(items.table, slots, sh.total);       // for the rows' kernels
        uint32_t unit = 0;
        for (int turn = 0, i; (i = items.first_of(turn)) < count; ++turn) {
            const int rows = items.get(i, slot, h, r0, c0, first), n = min(128, sh.dk - c0);
            for (int k = 0; k < rows; k += kLocalSum, ++unit) {
                if (unit > 0) {                           // what was there has left shared memory; a tile's sum before this one, arrived
                    if (warp == 8) bulk_all_done();
                    named_sync(1, 128);
                }
                wait_here(acc_full + 8 * (unit & 1), unit >> 1 & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
                for (int x = 0; x < n; x += 16) {         // four pieces of 16 bytes, in images of 32 columns, swizzled
                    uint32_t y[16];
                    tmem_ld_n(tmem + 128 * (unit & 1) + lanes + x, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared16(mine + (x >> 5) * 16384 + ((((x >> 2 & 7) + j) ^ (r & 7)) << 4), y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_free + 8 * (unit & 1));
                named_sync(1, 128);
                if (warp == 8) {
                    if (lane == 0) {
                        for (int x = 0; x < n; x += 32) tma_store_3d(&mo, base + kLocalOut + (x >> 5) * 16384, c0 + x, r0, slot * sh.H + h, k > 0);
                        bulk_commit();
                    }
                    __syncwarp();
                }
            }
        }
        if (warp == 8) bulk_all_done();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// 128 rows of o, dq, dk or dv.
//   kOut  o_t  = e^{g_t} S q_t + sum_{s <= t} beta_s e^{g_t - g_s} (q_t.k_s) v_s
//   kDq   dq_t = e^{g_t} S^T dO_t + sum_{s <= t} beta_s e^{g_t - g_s} (dO_t.v_s) k_s
//   kDk   dk_s = beta_s (e^{G - g_s} dS^T v_s + sum_{t >= s} e^{g_t - g_s} (v_s.dO_t) q_t)
//   kDv   dv_s = beta_s (e^{G - g_s} dS k_s + sum_{t >= s} e^{g_t - g_s} (k_s.q_t) dO_t)
// with S the state at the segment's start, dS the gradient at its end.
//
// The sum of products stays in TMEM: first the state's product, whose rows the workers scale there, then for each
// block of 128 tokens the scores (A and B from shared memory), which the workers read, decay, split into two bf16 terms and
// write back in place as the A operands of the products with X (tokens x columns, from shared memory as it lies).
// Two terms of a score or a state leave 2^-17 of it, so a bf16 output has its own rounding only (with one term of each the
// error against 64 bits was 2.3e-3 for 1.7e-3; 1 x 8192 tokens 46 us, and 54 with two).  kDq and kDv carry the state as three:
// q_t.(e^{g_t} S^T dO_t) and v_s.(e^{G - g_s} dS k_s), which the gates' fp32 gradients need, are taken from those fp32 sums.
//
// A CTA an SM takes block after block of rows; the scores of a block of columns, be it the next rows' first, are formed
// before the product of the one before it, so that the workers' pass over scores runs beside products.  Warps 0-7 work
// (four a half of the columns), 8-11 move finished sums out, 12 copies, 13 multiplies.
// 8192 tokens of 8 heads, 256 x 256, caches cold: kOut 54 us, kDk 56, kDq 75, kDv 72 (900 to 800 TFLOP/s of products; tensor
// core busy 47 and 40 % of an SM's time).  Bound by the chain of a block: scores, the workers' pass (some 1.4 k cycles), and
// the state's product with its scaling (4 k) at the start of each item, which the next item's scores cover in part only: two
// sums of 256 columns do not fit TMEM beside two blocks' scores.
// ---------------------------------------------------------------------------
enum { kOut, kDq, kDk, kDv };
constexpr int kRowThreads = 448, kMaxRing = 8;

struct RowsPlan {              // shared memory of a launch
    int ring, x_log, nr;       // stages; log2 of the tokens of a stage of X; buffers of row operands
    uint32_t stage, r, bars, smem;
};

struct RowsArgs {
    RowsPlan p;
    float* part;               // kDq, kDv: the row's dot by halves of the columns, [slot][H][2][512]
    size_t part_apart;         // floats from one (slot, head) to the next
    float* heads;              // kDq, kDk where heads share q and k: [total][H][d_k], else null
    const float* gates;
    int terms;
};

// What the workers keep of an item's gates, twice: factors of the columns of blocks other than rb; in block rb, by quarters
// of 32 rows, factors of its columns for the quarter's rows (both with beta where rows are queries); its sums as two floats.
struct RowGates {
    float cf[kSeg], quarter[4][kBlk], beta[kBlk], hi[kBlk];
    __nv_bfloat16 lo[kBlk];
};
// behind the barriers
constexpr int kRowNBars = 2 * kMaxRing + 17;
constexpr int kRowItems = 64;  // of a CTA that stand in shared memory
constexpr uint32_t kRowHolder = kRowNBars * 8, kRowGates = (kRowHolder + 8 + 15) / 16 * 16, kRowList = kRowGates + 2 * sizeof(RowGates),
                   kRowTail = kRowList + kRowItems * 16;
static_assert(sizeof(RowGates) % 16 == 0, "read by 16 bytes");

// A CTA's item of a turn: (slot, first token, rows + 1024 x blocks of columns + 8192 x its head of q and k, head), rows 0
// where there is none.  First segments of four blocks, whose four items are neighbours (they read the same tiles), in
// another order each turn, so that a CTA's turns bring long and short ones; then the shorter segments' items from the
// longest to the shortest.  (Everything from the longest to the shortest balances as well but reads all tiles at once:
// 4 x 2048 tokens forward and backward 440 us for 410.  Shorter segments by segment too: packed prompts 99 us for 87.)
// A chain of loads and divisions of some 3 k cycles: a CTA's first items are looked up at once when it starts, each by a
// thread (by each role before its next item, a seventh of the products' issuing went there).  Called, not inlined: four roles
// ask for items, and the instruction cache is small.
__device__ __noinline__ int4 rows_item(int turn, const int* order, const int2* table, int slots, int H, int rep, int total) {
    constexpr int kMost = kSeg / kBlk;
    static_assert(kMost == 4, "counts of slots with one block to four");
    const int2 n12 = reinterpret_cast<const int2*>(order)[0], n34 = reinterpret_cast<const int2*>(order)[1];
    const int i = turn * gridDim.x + blockIdx.x, n_most = min(max(n34.y, 0), slots);
    int m = i / kMost, b = kMost - (i + turn) % kMost, from = 0;
    if (m >= n_most * H) {
        from = n_most;
        const int k3 = (min(max(n34.x, n_most), slots) - n_most) * H, k2 = (min(max(n12.y, n_most), slots) - n_most) * H,
                  k1 = (min(max(n12.x, n_most), slots) - n_most) * H;
        m = i - n_most * H * kMost;
        b = m < k3 ? 3 : m < k3 + k2 ? 2 : 1;
        m -= b == 3 ? 0 : b == 2 ? k3 : k3 + k2;
        if (m >= k1) return make_int4(0, 0, 0, 0);
    }
    const int at = m / H, slot = order[kMost + from + at], h = m - at * H;
    if ((unsigned)slot >= (unsigned)slots) return make_int4(0, 0, 0, 0);
    const int2 e = slot_entry(table, slot, total);
    return (e.y + kBlk - 1) / kBlk < b ? make_int4(0, 0, 0, 0) : make_int4(slot, e.x, e.y + b * 1024 + h / rep * 8192, h);
}
template <int MODE>
struct RowsItem {
    int slot, h, hk, rb, first, rows, row_n, nblk;
    __device__ __forceinline__ void look(int turn, const int4* list, const int2* table, const SeqShape& sh, int slots, int rep) {
        constexpr bool keys = MODE == kDk || MODE == kDv;
        const int4 e = turn < kRowItems ? list[turn] : rows_item(turn, slot_order(table, slots), table, slots, sh.H, rep, sh.total);
        slot = e.x;
        first = e.y;
        rows = e.z & 1023;
        nblk = e.z >> 10 & 7;                             // blocks of columns: rb .. last, or 0 .. rb
        hk = e.z >> 13;
        h = e.w;
        rb = keys ? (rows + kBlk - 1) / kBlk - nblk : nblk - 1;
        row_n = min(kBlk, rows - rb * kBlk);
    }
    __device__ __forceinline__ bool there() const { return rows > 0; }
    __device__ __forceinline__ int col_block(int j) const { return MODE == kDk || MODE == kDv ? rb + j : j; }
    __device__ __forceinline__ int col_rows(int j) const { return min(kBlk, rows - col_block(j) * kBlk); }
};

template <int MODE>
__global__ void __launch_bounds__(kRowThreads, 1)
    lin_rows_tc_kernel(const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ CUtensorMap ms, SeqArgs a, RowsArgs ra) {
    constexpr bool keys = MODE == kDk || MODE == kDv, values = MODE == kOut || MODE == kDv;     // rows are keys; columns d_v
    constexpr uint32_t scores = 256;                      // TMEM: one sum of 256 columns or two of 128, then two blocks' scores
    extern __shared__ __align__(1024) char sm[];
    const SeqShape& sh = a.sh;
    const RowsPlan& p = ra.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_uniform(tid >> 5);
    void* out = MODE == kOut ? a.out : MODE == kDq ? a.dq : MODE == kDk ? a.dk : a.dv;
    const int rep = sh.H / sh.Hk, out_heads = values ? sh.H : sh.Hk;
    const int da = values ? sh.dk : sh.dv, dx = values ? sh.dv : sh.dk;
    const int slots = seg_slots(sh.nseq, sh.total, kSeg);
    const int2* table = slot_table(ra.gates, slots, sh.H);
    const uint32_t base = smem_u32(sm), bars = base + p.bars;
    const uint32_t full0 = bars, empty0 = bars + 8 * kMaxRing, rfull = bars + 16 * kMaxRing, rfree = rfull + 16, acc_free = rfull + 32, acc_done = rfull + 48,
                   s_full = rfull + 64, p_full = rfull + 80, x_done = rfull + 96, inter_done = rfull + 112, acc_ready = rfull + 120, drain = rfull + 128;
    char* tail = sm + p.bars;
    uint32_t* holder = reinterpret_cast<uint32_t*>(tail + kRowHolder);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    const int na = (da + 63) / 64, nb = (da + 127) / 128, nx = (dx + 63) / 64, n_inter = ra.terms * na;
    const int two_sums = dx <= 128;                       // sums in TMEM, less one; the second 128 columns on
    const uint32_t r_bytes = na * 2 * kBox;
    const int rows_x = 1 << p.x_log;
    if (tid == 0) {
#pragma unroll 1
        for (uint32_t b = bars; b < bars + 8 * kRowNBars; b += 8)
            mbar_init(b, (b >= p_full && b < x_done) || b == acc_ready ? 8u : b >= acc_free && b < acc_done ? 4u : 1u);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 13) tmem_alloc(smem_u32(holder), 512);
    __syncthreads();
    const uint32_t tmem = warp_uniform(*holder);
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    {
        int ob, oe;
        if (seq_outside(sh, ob, oe)) zero_rows<__nv_bfloat16>(out, (size_t)out_heads * dx, ob, oe, sh.total);
    }
    int4* list = reinterpret_cast<int4*>(tail + kRowList);
    if (tid < kRowItems) list[tid] = rows_item(tid, slot_order(table, slots), table, slots, sh.H, rep, sh.total);
    __syncthreads();
    // Scores and products of a CTA's blocks of columns, one after another over its items, interleaved: the scores of a
    // block before the product of the one before it, the state's product behind the first scores of its rows.  The rows'
    // operand is used up by its last scores (or the state's product): the next rows' arrives while the workers have those,
    // and with one place for it an item's first scores come behind the last product of the item before (75 k cycles a CTA
    // of 8192 tokens for 70 the other way around).
    RowsItem<MODE> it;
    it.look(0, list, table, sh, slots, rep);
    if (warp == 12) {
        if (elect_one()) {
            const bool whole_a = da % 64 == 0, whole_x = dx % 64 == 0;
            const size_t apart = (size_t)slots * sh.H;
            Ring ring, rr;
            int issued = 0, r_issued = 0;
            bool ok = true;
            RowsItem<MODE> prev, after;
            int turns = 0;
            bool last = false;
            for (int j = 0, pj = -1; ok && !last;) {          // it's block j; the block before it, prev's pj
                last = !it.there();
                const bool x_first = last || (j == 0 && p.nr == 1);
                const int n0 = pj == 0 ? n_inter : 0, nxt = pj >= 0 ? (prev.col_rows(pj) + rows_x - 1) >> p.x_log : 0, ns = last ? 0 : nb;
                // the state's stages, then scores' and X's in their order; new rows' own operand before both (e stays where it is)
                bool row_op = j == 0 && !last;
#pragma unroll 1
                for (int e = 0; e < n0 + ns + nxt;) {
                    const int w = e - n0, s_at = x_first ? w - nxt : w, x_at = x_first ? w : w - ns;
                    const bool state = e < n0, r = !state && row_op, score = r || (!state && s_at >= 0 && s_at < ns);
                    const uint32_t st = r ? rr.st : ring.st, ph = (r ? rr.ph : ring.ph) ^ 1, bar = (r ? rfull : full0) + 8 * st, dst = base + (r ? p.r + st * r_bytes : st * p.stage);
                    if ((r ? r_issued >= p.nr : issued >= p.ring) && !(ok = wait_here((r ? rfree : empty0) + 8 * st, ph, a.err, dead))) break;
                    // boxes of 64 columns (all of them in one where the map has whole boxes: slabs behind the last come as zeros);
                    // tokens that they hold beyond the sequence's are read and never used
                    const bool one = state ? values : score ? whole_a : whole_x;
                    const int slabs = state || !score ? nx : r ? na : whole_a ? min(2, na) : min(2, na - 2 * s_at), rows = state ? 64 : score ? kBlk : rows_x;
                    mbar_expect_tx(bar, state && values ? dx * 128 : slabs * rows * 128);
                    const CUtensorMap* m = state ? &ms : r ? &mr : score ? &mb : &mx;
                    const int head = score ? (values ? it.hk : it.h) : values ? prev.h : prev.hk;
                    const int t0 = r ? it.first + it.rb * kBlk
                                     : score ? it.first + it.col_block(j) * kBlk : prev.first + prev.col_block(pj) * kBlk + x_at * rows_x;
                    const int x0 = score && !r ? 2 * s_at : 0;
                    // the state's, small terms first: rows of d_v by 64 of d_k along the row, or 64 rows of d_v by d_k
                    const int sx = e % na, sz = (int)((ra.terms - 1 - e / na) * apart + (size_t)prev.slot * sh.H + prev.h);
#pragma unroll 1
                    for (int x = 0; x < (one ? 1 : slabs); ++x) {
                        const uint32_t to = dst + x * rows * 128;
                        if (state) tma_3d(to, m, values ? 64 * sx : 64 * x, values ? 0 : 64 * sx, sz, bar);
                        else tma_4d(to, m, one ? 0 : 64 * (x0 + x), head, t0, one ? x0 : 0, bar);
                    }
                    if (r) {
                        rr.next(p.nr);
                        ++r_issued;
                        row_op = false;
                    } else {
                        ring.next(p.ring);
                        ++issued;
                        ++e;
                    }
                }
                if (last) break;
                if (j == 0) after.look(++turns, list, table, sh, slots, rep);
                prev = it;
                pj = j;
                if (++j == it.nblk) {
                    j = 0;
                    it = after;
                }
            }
            if (*dead) {                                  // copies in flight end before the CTA does
#pragma unroll 1
                for (int j = max(0, r_issued - p.nr); j < r_issued; ++j) wait_here(rfull + 8 * (j % p.nr), (j / p.nr) & 1, a.err, nullptr);
#pragma unroll 1
                for (int j = max(0, issued - p.ring); j < issued; ++j) wait_here(full0 + 8 * (j % p.ring), (j / p.ring) & 1, a.err, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 13) {
        const bool leader = elect_one();
        Ring ring, rr;
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            wait_here(bar, parity, a.err, dead);
            __syncwarp();
            tc_fence_after();
        };
        const uint32_t id_x = idesc_bf16(128, dx) | kBMn, id_i = idesc_bf16(128, dx) | (values ? 0u : kBMn);
        const auto free_r = [&]() {                       // the rows' operand is used up
            if (leader) mma_commit(rfree + 8 * rr.st);
            __syncwarp();
            rr.next(p.nr);
        };
        uint32_t items = 0, blocks = 0;                   // sums, and blocks of scores, so far
        RowsItem<MODE> after;
        int turns = 0, p_rows = 0;                        // p_rows: tokens of the block of columns before
        bool p_last = false;
        for (int j = 0, pj = -1;;) {
            const bool last = !warp_uniform(it.there()), x_first = last || (j == 0 && p.nr == 1);
            const uint32_t ab = two_sums ? items & 1 : 0, ap = two_sums ? items >> 1 & 1 : items & 1, acc = tmem + 128 * ab;
            if (pj == 0) {
                if (items > (uint32_t)two_sums) wait(acc_free + 8 * ab, ap ^ 1);
                const uint64_t dR = k_desc<128>(base + p.r + rr.st * r_bytes);
#pragma unroll 1
                for (int e = 0, x = 0; e < n_inter; ++e, ring.next(p.ring)) {
                    wait(full0 + 8 * ring.st, ring.ph);
                    if (leader) {
                        const uint32_t sb = base + ring.st * p.stage;
                        const uint64_t dA = dR + (x * 2 * kBox >> 4), dB = values ? k_desc<128>(sb) : mn_desc<128>(sb, kBox);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (64 * x + 16 * k < da) mma_bf16(acc, dA + 2 * k, dB + (values ? 2 * k : 128 * k), id_i, e + k > 0);
                        mma_commit(empty0 + 8 * ring.st);
                    }
                    __syncwarp();
                    if (++x == na) x = 0;
                }
                if (leader) mma_commit(inter_done);
                __syncwarp();
                if (p_last) free_r();
            }
#pragma unroll 1
            for (int ph = 0; ph < 2; ++ph) {
                if ((ph == 0) != x_first && !last) {      // scores of it's block j
                    const uint32_t u = blocks & 1, D = tmem + scores + 128 * u, id = idesc_bf16(128, (warp_uniform(it.col_rows(j)) + 15) & ~15);
                    if (j == 0) wait(rfull + 8 * rr.st, rr.ph);
                    if (blocks > 1) wait(x_done + 8 * u, (blocks >> 1 & 1) ^ 1);      // the scores before are used up
                    const uint64_t dR = k_desc<128>(base + p.r + rr.st * r_bytes);
#pragma unroll 1
                    for (int x = 0; x < na; ++x) {
                        if ((x & 1) == 0) wait(full0 + 8 * ring.st, ring.ph);
                        const bool more = (x & 1) == 0 && x + 1 < na;
                        if (leader) {
                            const uint64_t dA = dR + (x * 2 * kBox >> 4), dB = k_desc<128>(base + ring.st * p.stage) + ((x & 1) * 2 * kBox >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (64 * x + 16 * k < da) mma_bf16(D, dA + 2 * k, dB + 2 * k, id, x + k > 0);
                            if (!more) mma_commit(empty0 + 8 * ring.st);
                        }
                        __syncwarp();
                        if (!more) ring.next(p.ring);
                    }
                    if (leader) mma_commit(s_full + 8 * u);
                    __syncwarp();
                    if (j > 0 && j + 1 == warp_uniform(it.nblk)) free_r();
                }
                if ((ph == 0) == x_first && pj >= 0) {    // the product of the block before
                    const uint32_t n = blocks - 1, u = n & 1;
                    if (pj == 0) wait(acc_ready, items & 1);
                    wait(p_full + 8 * u, n >> 1 & 1);
#pragma unroll 1
                    for (int x = 0; x < p_rows; x += 64) {            // 64 tokens
                        if ((x & rows_x - 1) == 0) wait(full0 + 8 * ring.st, ring.ph);
                        const bool more = x + 64 < p_rows && (x + 64 & rows_x - 1) != 0;       // of the stage
                        if (leader) {
                            const uint64_t dB = mn_desc<128>(base + ring.st * p.stage, rows_x * 128) + (x & rows_x - 1) * 8;
                            const uint32_t A = tmem + scores + 128 * u + x;           // 16 tokens: 8 columns of first terms, 8 of second
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (x + 16 * k < p_rows) {
                                    mma_bf16_ts(acc, A + 16 * k + 8, dB + 128 * k, id_x, 1);
                                    mma_bf16_ts(acc, A + 16 * k, dB + 128 * k, id_x, 1);
                                }
                            if (!more) mma_commit(empty0 + 8 * ring.st);
                        }
                        __syncwarp();
                        if (!more) ring.next(p.ring);
                    }
                    if (leader) {
                        mma_commit(x_done + 8 * u);
                        if (p_last) mma_commit(acc_done + 8 * ab);
                    }
                    __syncwarp();
                }
            }
            if (pj >= 0 && p_last) ++items;
            if (last) break;
            ++blocks;
            if (j == 0) after.look(++turns, list, table, sh, slots, rep);
            p_rows = warp_uniform(it.col_rows(j));
            p_last = warp_uniform(j + 1 == it.nblk);
            pj = j;
            if (p_last) {
                j = 0;
                it = after;
            } else {
                ++j;
            }
        }
        if (leader) {                                     // products in flight end before their TMEM is freed
            mma_commit(drain);
            wait_here(drain, 0, a.err, nullptr);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int g = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const int chunks = dx / 16, ch0 = g == 0 ? 0 : (chunks + 1) / 2, ch1 = g == 0 ? (chunks + 1) / 2 : chunks;      // of 16 columns
        RowGates* gates = reinterpret_cast<RowGates*>(tail + kRowGates);
        uint32_t items = 0, blocks = 0;
        int turns = 0;
        int at_stage = nb, stage_ph = 0;                  // of the ring, behind this block's scores, and their turn's parity
        const auto turn = [&]() {
#pragma unroll 1
            for (; at_stage >= p.ring; at_stage -= p.ring) stage_ph ^= 1;
        };
        // an item's gates on their way: its row's, two columns', the blocks', block rb's
        float g_row[6], g_col[2][2], g_tot[4], g_blk[3], g_m[2][2];
        const auto load_gates = [&]() {
            const float* gt = ra.gates + ((size_t)it.slot * sh.H + it.h) * kGAll;
            const int r = it.rb * kBlk + row, c = it.rb * kBlk + (tid & 127);
            g_row[0] = gt[kGHi + r];
            g_row[1] = gt[kGLo + r];
            g_row[2] = gt[(keys ? kGPost : kGPre) + r];
            g_row[3] = gt[(keys ? kGTail : kGHead) + r];
            // the sums that a quarter's factors are relative to: at its last key, or before its first query
            const int m = it.rb * kBlk + 32 * w4 + (keys ? 31 : -1);
            g_row[4] = !keys && w4 == 0 ? 0.f : gt[kGHi + m];
            g_row[5] = !keys && w4 == 0 ? 0.f : gt[kGLo + m];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                g_col[e][0] = gt[(keys ? kGPre : kGPost) + tid + 256 * e];
                g_col[e][1] = gt[kGBeta + tid + 256 * e];
                const int w = 2 * (tid >> 7) + e, mw = it.rb * kBlk + 32 * w + (keys ? 31 : -1);
                g_m[e][0] = !keys && w == 0 ? 0.f : gt[kGHi + mw];
                g_m[e][1] = !keys && w == 0 ? 0.f : gt[kGLo + mw];
            }
            const float4 t4 = *reinterpret_cast<const float4*>(gt + kGTot);
            g_tot[0] = t4.x; g_tot[1] = t4.y; g_tot[2] = t4.z; g_tot[3] = t4.w;
            g_blk[0] = gt[kGHi + c];
            g_blk[1] = gt[kGLo + c];
            g_blk[2] = keys ? 1.f : gt[kGBeta + c];
        };
        // An item's gates are loaded while the one before is worked on.
        if (it.there()) load_gates();
        while (it.there()) {
            const RowsItem<MODE> cur = it;
            RowGates& G = gates[items & 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tid + 256 * e, b = t / kBlk, w = 2 * (tid >> 7) + e;
                float f = keys ? g_col[e][0] : g_col[e][0] * g_col[e][1];
#pragma unroll
                for (int m = 1; m < 3; ++m)           // blocks between
                    if (m > min(b, cur.rb) && m < max(b, cur.rb)) f *= g_tot[m];
                G.cf[t] = f;
                const float d = (g_m[e][0] - g_blk[0]) + (g_m[e][1] - g_blk[1]);
                G.quarter[w][tid & 127] = g_blk[2] * ex2(keys ? d * -kLog2e : d * kLog2e);
            }
            if (tid < kBlk) {
                G.beta[tid] = g_blk[2];
                G.hi[tid] = g_blk[0];
                G.lo[tid] = __float2bfloat16_rn(g_blk[1]);
            }
            const float mine = g_row[0], mine_lo = g_row[1], rf = g_row[2], sf = g_row[3];
            const float dm = (mine - g_row[4]) + (mine_lo - g_row[5]), qf = ex2(keys ? dm * -kLog2e : dm * kLog2e);
            const int rb = cur.rb, hk = cur.hk, nblk = cur.nblk;
            const bool live = row < cur.row_n;
            const size_t token = (size_t)cur.first + rb * kBlk + row, at = (size_t)cur.slot * sh.H + cur.h;
            named_sync(2, 256);
            const uint32_t acc = tmem + (two_sums ? 128 * (items & 1) : 0) + lanes;
            for (int j = 0; j < nblk; ++j, ++blocks) {
                const uint32_t u = blocks & 1;
                const int cb = cur.col_block(j), n = cur.col_rows(j);
                const uint32_t S = tmem + lanes + scores + 128 * u + 64 * g;
                wait_here(s_full + 8 * u, blocks >> 1 & 1, a.err, dead);
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {             // 16 columns
                    const int c0 = 64 * g + 16 * q, cq = c0 >> 5;
                    uint32_t x[16], y[16];                // 16 tokens' pairs, first terms and second terms
                    if (c0 >= n || (cb == rb && (keys ? cq < w4 : cq > w4))) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = 0;        // behind the segment, or masked altogether
                    } else {
                        tmem_ld_n(S + 16 * q, x);
                        tmem_wait_ld();
                        if (cb == rb && cq == w4) {       // around the diagonal
#pragma unroll
                            for (int e0 = 0; e0 < 16; e0 += 4) {
                                const float4 h4 = *reinterpret_cast<const float4*>(G.hi + c0 + e0), f4 = *reinterpret_cast<const float4*>(G.beta + c0 + e0);
                                const uint2 l2 = *reinterpret_cast<const uint2*>(G.lo + c0 + e0);
                                const float hs[4] = {h4.x, h4.y, h4.z, h4.w}, fs[4] = {f4.x, f4.y, f4.z, f4.w},
                                            ls[4] = {__uint_as_float(l2.x << 16), __uint_as_float(l2.x & 0xffff0000u), __uint_as_float(l2.y << 16),
                                                     __uint_as_float(l2.y & 0xffff0000u)};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int col = c0 + e0 + e;
                                    const float d = (hs[e] - mine) + (ls[e] - mine_lo);
                                    const float f = fs[e] * ex2(keys ? d * kLog2e : d * -kLog2e);
                                    x[e0 + e] = (keys ? col >= row : col <= row) ? __float_as_uint(f * __uint_as_float(x[e0 + e])) : 0u;
                                }
                            }
                        } else {
                            const float* tab = cb == rb ? G.quarter[w4] + c0 : G.cf + cb * kBlk + c0;
                            const float r1 = cb == rb ? qf : rf;
                            const float2 r2 = make_float2(r1, r1);
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(tab + e);
                                const float2 y0 = fmul2(fmul2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), r2), make_float2(f.x, f.y)),
                                             y1 = fmul2(fmul2(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), r2), make_float2(f.z, f.w));
                                x[e] = __float_as_uint(y0.x);
                                x[e + 1] = __float_as_uint(y0.y);
                                x[e + 2] = __float_as_uint(y1.x);
                                x[e + 3] = __float_as_uint(y1.y);
                            }
                        }
                        if (c0 + 16 > n) {                // a tail
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = c0 + e < n ? x[e] : 0u;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float x0 = __uint_as_float(x[2 * e]), x1 = __uint_as_float(x[2 * e + 1]);
                            y[e] = pack_bf16(x0, x1);
                            y[8 + e] = pack_bf16(x0 - __uint_as_float(y[e] << 16), x1 - __uint_as_float(y[e] & 0xffff0000u));
                        }
                    }
                    tmem_st_n(S + 16 * q, y);             // over the columns just read
                }
                tmem_wait_st();
                if (j == 0) {                             // the next item's gates; the state's product: its rows scaled
                    it.look(++turns, list, table, sh, slots, rep);
                    if (it.there()) load_gates();
                    const __nv_bfloat16* z = MODE == kDq ? static_cast<const __nv_bfloat16*>(a.q) + token * sh.ldq + (size_t)hk * sh.dk
                                                         : static_cast<const __nv_bfloat16*>(a.v) + token * sh.ldv + (size_t)cur.h * sh.dv;
                    constexpr bool dots = MODE == kDq || MODE == kDv;
                    uint4 w[3][2] = {};                   // q's or v's columns, three chunks on their way
                    const auto load = [&](uint4 (&x)[2], int ch) {
                        if (!dots || !live || ch >= ch1) return;
                        x[0] = *reinterpret_cast<const uint4*>(z + 16 * ch);
                        x[1] = *reinterpret_cast<const uint4*>(z + 16 * ch + 8);
                    };
#pragma unroll
                    for (int e = 0; e < 3; ++e) load(w[e], ch0 + e);
                    wait_here(inter_done, items & 1, a.err, dead);
                    __syncwarp();
                    tc_fence_after();
                    float dot = 0.f;
#pragma unroll 1
                    for (int ch = ch0; ch < ch1; ++ch) {
                        uint32_t x[16];
                        tmem_ld_n(acc + 16 * ch, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(sf * __uint_as_float(x[c]));
                        tmem_st_n(acc + 16 * ch, x);
                        if (dots) {
                            const uint32_t y[8] = {w[0][0].x, w[0][0].y, w[0][0].z, w[0][0].w, w[0][1].x, w[0][1].y, w[0][1].z, w[0][1].w};
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                dot = fmaf(__uint_as_float(x[2 * c]), __uint_as_float(y[c] << 16), dot);
                                dot = fmaf(__uint_as_float(x[2 * c + 1]), __uint_as_float(y[c] & 0xffff0000u), dot);
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                w[0][e] = w[1][e];
                                w[1][e] = w[2][e];
                            }
                            load(w[2], ch + 3);
                        }
                        __syncwarp();
                    }
                    if ((MODE == kDq || MODE == kDv) && live) ra.part[at * ra.part_apart + g * kSeg + rb * kBlk + row] = dot;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_ready);
                }
                // the ring's stages: the state's, the next scores', X's
                if (j == 0) at_stage += n_inter;
                if (j + 1 < nblk || (p.nr > 1 && it.there())) at_stage += nb;
                turn();
                if (n % 16 != 0) {                        // X's tokens of what lies behind: rows of zero, up to whole products
                    // not before what was in X's stage is used up: the state's terms, or the X before
                    if (j > 0) wait_here(x_done + 8 * (u ^ 1), (blocks - 1) >> 1 & 1, a.err, dead);
                    const int last = (n - 1) >> p.x_log, over = at_stage + last >= p.ring, st = at_stage + last - (over ? p.ring : 0);
                    wait_here(full0 + 8 * st, stage_ph ^ over, a.err, dead);
                    const int r = (n & 15) + (tid >> 3);
                    if (r < 16)
#pragma unroll 1
                        for (int x = 0; x < nx; ++x) st_shared16(base + st * p.stage + (x * rows_x + (n & rows_x - 16) + r) * 128 + (tid & 7) * 16, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                at_stage += ((n + rows_x - 1) >> p.x_log) + (j + 1 == nblk && p.nr == 1 ? nb : 0);
                turn();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * u);
            }
            ++items;
        }
    } else {
        const int w4 = warp & 3, row = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const bool shared = !values && rep > 1;
        const bool whole = (reinterpret_cast<uintptr_t>(shared ? static_cast<const void*>(ra.heads) : out) & 31u) == 0;      // by 32 bytes: both may start on 16
        for (uint32_t items = 0; it.there(); it.look(++items, list, table, sh, slots, rep)) {
            const uint32_t ab = two_sums ? items & 1 : 0, ap = two_sums ? items >> 1 & 1 : items & 1, acc = tmem + 128 * ab + lanes;
            const bool live = row < it.row_n;
            const size_t token = (size_t)it.first + it.rb * kBlk + row;
            const int head = values ? it.h : it.hk;
            const float of = keys ? ra.gates[((size_t)it.slot * sh.H + it.h) * kGAll + kGBeta + it.rb * kBlk + row] : 1.f;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + token * out_heads * dx + (size_t)head * dx;
            float* o32 = shared ? ra.heads + (token * sh.H + it.h) * dx : nullptr;
            wait_here(acc_done + 8 * ab, ap, a.err, dead);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < dx; c0 += 32) {
                uint32_t vs[2][16];
                tmem_ld_n(acc + c0, vs[0]);
                if (c0 + 16 < dx) tmem_ld_n(acc + c0 + 16, vs[1]);
                tmem_wait_ld();
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int c = c0 + 16 * e2;
                    const uint32_t (&v)[16] = vs[e2];
                    if (!live || c >= dx) break;
                    float y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = of * __uint_as_float(v[e]);
                    if (shared) {
                        uint4 w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = make_uint4(__float_as_uint(y[4 * e]), __float_as_uint(y[4 * e + 1]), __float_as_uint(y[4 * e + 2]), __float_as_uint(y[4 * e + 3]));
                        stg_pieces<4>(o32 + c, w, false, whole);
                    } else {
                        uint4 w[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            w[e] = make_uint4(pack_bf16(y[8 * e], y[8 * e + 1]), pack_bf16(y[8 * e + 2], y[8 * e + 3]), pack_bf16(y[8 * e + 4], y[8 * e + 5]),
                                              pack_bf16(y[8 * e + 6], y[8 * e + 7]));
                        stg_pieces<2>(o + c, w, false, whole);
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_free + 8 * ab);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Sums of F_ts = e^{g_t - g_s} (q_t.k_s) (dO_t.v_s), s < t, of 128 rows t with the segment's blocks up to theirs: by
// rows with beta_s, by columns without, and F_tt.  Both scores are products of bf16 inputs, exact but for fp32 sums.
// Warps 0-7 work, warp 8 copies, warp 9 multiplies; a CTA a block of rows, two an SM where both fit, the longest first.  8192 tokens of 8
// heads, 256 x 256: 47 us, tensor core busy 25 % of the time: bound by the workers' pass over two scores of each pair.
// ---------------------------------------------------------------------------
// floats of a (slot, head): rows with their own block's columns, F_tt, q's and v's dots by halves, columns by block of rows,
// rows with the blocks before
constexpr int kPartRow = 0, kPartDiag = kSeg, kPartQ = 2 * kSeg, kPartK = 4 * kSeg, kPartCol = 6 * kSeg, kPartOff = 10 * kSeg, kPartAll = 11 * kSeg;

constexpr int kPairThreads = 320;
struct PairsPlan {
    int ring;
    bool two;
    uint32_t r2, stages, bars, smem;
};
constexpr uint32_t kPairHolder = 2 * kMaxRing * 8 + 6 * 8, kPairCf = kPairHolder + 16, kPairBeta = kPairCf + kSeg * 4,
                   kPairHi = kPairBeta + kSeg * 4, kPairLo = kPairHi + kBlk * 4, kPairCol = kPairLo + kBlk * 4, kPairTail = kPairCol + 2 * 4 * kBlk * 4;
static_assert(kPairCf % 16 == 0 && kPairBeta % 16 == 0, "read by 16 bytes");

__global__ void __launch_bounds__(kPairThreads, 2)
    lin_pairs_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mk,
                        const __grid_constant__ CUtensorMap mv, SeqArgs a, PairsPlan p, const float* gates, float* part) {
    extern __shared__ __align__(1024) char sm[];
    const SeqShape& sh = a.sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_uniform(tid >> 5);
    const int slots = seg_slots(sh.nseq, sh.total, kSeg);
    const int at = blockIdx.x / 4, rb = 3 - blockIdx.x % 4, slot = at / sh.H, h = at % sh.H, hk = h / (sh.H / sh.Hk);
    griddep_wait();
    griddep_launch();
    const int2 seg = slot_entry(slot_table(gates, slots, sh.H), slot, sh.total);
    const int first = seg.x, rows = warp_uniform(seg.y);
    if (rb * kBlk >= rows) return;
    // the workers' gates, on their way
    const float* gt = gates + ((size_t)slot * sh.H + h) * kGAll;
    float g_col[2][2], g_tot[4], g_hi = 0.f, g_lo = 0.f;
    if (warp < 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            g_col[i][0] = gt[kGPost + tid + 256 * i];
            g_col[i][1] = gt[kGBeta + tid + 256 * i];
        }
        const float4 t4 = *reinterpret_cast<const float4*>(gt + kGTot);
        g_tot[0] = t4.x; g_tot[1] = t4.y; g_tot[2] = t4.z; g_tot[3] = t4.w;
        if (tid < kBlk) {
            g_hi = gt[kGHi + rb * kBlk + tid];
            g_lo = gt[kGLo + rb * kBlk + tid];
        }
    }
    const int row_n = min(kBlk, rows - rb * kBlk), nk = (sh.dk + 63) / 64, nv = (sh.dv + 63) / 64;
    const auto col_rows = [&](int j) { return j == rb ? row_n : kBlk; };
    const uint32_t base = smem_u32(sm), bars = base + p.bars;
    const uint32_t full0 = bars, empty0 = bars + 8 * kMaxRing, rfull = bars + 16 * kMaxRing, s_full = rfull + 8, s_used = rfull + 24, done = rfull + 40;
    char* tail = sm + p.bars;
    uint32_t* holder = reinterpret_cast<uint32_t*>(tail + kPairHolder);
    volatile int* dead = reinterpret_cast<volatile int*>(holder + 1);
    float *cf = reinterpret_cast<float*>(tail + kPairCf), *beta = reinterpret_cast<float*>(tail + kPairBeta),
          *hi = reinterpret_cast<float*>(tail + kPairHi), *lo = reinterpret_cast<float*>(tail + kPairLo), *col = reinterpret_cast<float*>(tail + kPairCol);
    const int G = p.two ? 2 : 1;
    const uint32_t cols = p.two ? 512 : 256;
    if (tid == 0) {
        init_barriers(bars, 2 * kMaxRing + 6, [&](uint32_t b) { return b >= s_used && b < done ? 8u : 1u; });
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 9) tmem_alloc(smem_u32(holder), cols);
    __syncthreads();
    const uint32_t tmem = warp_uniform(*holder);
    tc_fence_after();
    if (warp == 8) {
        if (elect_one()) {
            // slab x of 128 tokens, or (the rows' own) all slabs in one box where the map has whole ones
            const bool whole_k = sh.dk % 64 == 0, whole_v = sh.dv % 64 == 0;
            mbar_expect_tx(rfull, (nk + nv) * 2 * kBox);
#pragma unroll 1
            for (int x = 0; x < (whole_k ? 1 : nk); ++x) tma_4d(base + x * 2 * kBox, &mq, 64 * x, hk, first + rb * kBlk, 0, rfull);
#pragma unroll 1
            for (int x = 0; x < (whole_v ? 1 : nv); ++x) tma_4d(base + p.r2 + x * 2 * kBox, &mo, 64 * x, h, first + rb * kBlk, 0, rfull);
            Ring ring;
            int it = 0;
            bool ok = true;
            for (int j = 0; ok && j <= rb; ++j)
#pragma unroll 1
                for (int x = 0; x < nk + nv; ++x, ++it, ring.next(p.ring)) {
                    if (it >= p.ring && !(ok = wait_here(empty0 + 8 * ring.st, ring.ph ^ 1, a.err, dead))) break;
                    const bool is_k = x < nk, whole = is_k ? whole_k : whole_v;
                    const int sl = is_k ? x : x - nk;
                    mbar_expect_tx(full0 + 8 * ring.st, 2 * kBox);
                    tma_4d(base + p.stages + ring.st * 2 * kBox, is_k ? &mk : &mv, whole ? 0 : 64 * sl, is_k ? hk : h, first + j * kBlk, whole ? sl : 0, full0 + 8 * ring.st);
                }
            if (*dead) {                                  // copies in flight end before the CTA does
                wait_here(rfull, 0, a.err, nullptr);
                for (int j = max(0, it - p.ring); j < it; ++j) wait_here(full0 + 8 * (j % p.ring), (j / p.ring) & 1, a.err, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        const bool leader = elect_one();
        Ring ring;
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            wait_here(bar, parity, a.err, dead);
            __syncwarp();
            tc_fence_after();
        };
        wait(rfull, 0);
        uint32_t use = 0;
        for (int j = 0, u = 0; j <= rb; ++j) {
            if (use > 0) wait(s_used + 8 * u, (use - 1) & 1);
            const uint32_t id = idesc_bf16(128, (col_rows(j) + 15) & ~15);
            for (int half = 0; half < 2; ++half) {
                const int d = half == 0 ? sh.dk : sh.dv;
                const uint32_t D = tmem + 256 * u + 128 * half;
                const uint64_t dR = k_desc<128>(base + (half == 0 ? 0 : p.r2));
                for (int x = 0; 64 * x < d; ++x, ring.next(p.ring)) {
                    wait(full0 + 8 * ring.st, ring.ph);
                    if (leader) {
                        const uint64_t dA = dR + (x * 2 * kBox >> 4), dB = k_desc<128>(base + p.stages + ring.st * 2 * kBox);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (64 * x + 16 * k < d) mma_bf16(D, dA + 2 * k, dB + 2 * k, id, x + k > 0);
                        mma_commit(empty0 + 8 * ring.st);
                    }
                    __syncwarp();
                }
            }
            if (leader) mma_commit(s_full + 8 * u);
            __syncwarp();
            if (++u == G) {
                u = 0;
                ++use;
            }
        }
        if (leader) {
            mma_commit(done);                             // and products in flight end before their TMEM is freed
            wait_here(done, 0, a.err, nullptr);
        }
        __syncwarp();
    } else {
        const int g = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tid + 256 * i, b = t / kBlk;
            float f = g_col[i][0];
#pragma unroll
            for (int m = 1; m < 3; ++m)                   // blocks between
                if (m > b && m < rb) f *= g_tot[m];
            cf[t] = f;
            beta[t] = g_col[i][1];
        }
        if (tid < kBlk) {
            hi[tid] = g_hi;
            lo[tid] = g_lo;
        }
        named_sync(2, 256);
        const float mine = hi[row], mine_lo = lo[row], rf = decay_of(LogSum{mine, mine_lo});
        const bool live = row < row_n;
        float* out = part + ((size_t)slot * sh.H + h) * kPartAll;
        float sum = 0.f, diag = 0.f, off = 0.f;
        for (int j = 0; j <= rb; ++j) {
            if (j == rb) {
                off = sum;
                sum = 0.f;
            }
            const int u = j % G, n = col_rows(j);
            wait_here(s_full + 8 * u, (j / G) & 1, a.err, dead);
            __syncwarp();
            tc_fence_after();
            float* cj = col + (j & 1) * 4 * kBlk + w4 * kBlk;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int c0 = 64 * g + 32 * q;
                float f[32];
                if (c0 >= ((n + 15) & ~15) || (j == rb && c0 > 32 * w4 + 31)) {
                    f[0] = 0.f;
                } else {
                    const uint32_t D = tmem + lanes + 256 * u + c0;
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t x[16], y[16];
                        tmem_ld_n(D + e, x);
                        tmem_ld_n(D + 128 + e, y);
                        tmem_wait_ld();
                        const float* bt = beta + j * kBlk + c0 + e;
                        if (j == rb) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int cc = c0 + e + i;
                                const float w = ex2(((mine - hi[cc]) + (mine_lo - lo[cc])) * kLog2e);
                                const float v = live && cc < n && cc <= row ? w * __uint_as_float(x[i]) * __uint_as_float(y[i]) : 0.f;
                                diag = cc == row ? v : diag;
                                f[e + i] = cc == row ? 0.f : v;
                            }
                        } else {
                            const float* cj4 = cf + j * kBlk + c0 + e;
#pragma unroll
                            for (int i = 0; i < 16; ++i) f[e + i] = live ? rf * cj4[i] * __uint_as_float(x[i]) * __uint_as_float(y[i]) : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum = fmaf(bt[i], f[e + i], sum);
                    }
                    // each lane's column: halves of what is left change places between lanes
#pragma unroll
                    for (int half = 16; half > 0; half >>= 1) {
                        const bool up = (lane & half) != 0;
#pragma unroll
                        for (int i = 0; i < half; ++i) {
                            const float send = up ? f[i] : f[i + half], keep = up ? f[i + half] : f[i];
                            f[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
                        }
                    }
                }
                cj[c0 + lane] = f[0];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_used + 8 * u);
            named_sync(3 + g, 128);
            const int i = tid & 127;
            if (i < 64) {
                const float* q = col + (j & 1) * 4 * kBlk + 64 * g + i;
                out[kPartCol + rb * kSeg + j * kBlk + 64 * g + i] = (q[0] + q[kBlk]) + (q[2 * kBlk] + q[3 * kBlk]);
            }
        }
        // both halves' row sums, one after the other
        named_sync(2, 256);
        if (g == 1) {
            cf[row] = sum;
            cf[kBlk + row] = off;
            hi[row] = diag;
        }
        named_sync(2, 256);
        if (g == 0 && live) {
            out[kPartRow + rb * kBlk + row] = sum + cf[row];
            out[kPartOff + rb * kBlk + row] = off + cf[kBlk + row];
            out[kPartDiag + rb * kBlk + row] = diag + hi[row];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, cols);
    }
}

// ---------------------------------------------------------------------------
// dlog_alpha and dbeta of one (segment, head) from those sums (E_ts = beta_s F_ts), four tokens a thread:
//   dlog_alpha_u = sum_{s < u <= t} E_ts + sum_{t >= u} q_t.(e^{g_t} S^T dO_t) + sum_{s < u} beta_s v_s.(e^{G - g_s} dS k_s) + e^G <dS, S>
//   dbeta_s      = sum_{t >= s} F_ts + v_s.(e^{G - g_s} dS k_s)
// The first sum's pairs (t, s) by blocks: t in u's block and s before it, sums of rows from u on; s in u's block and t behind it,
// sums of columns before u; both elsewhere, whole blocks' sums; both in u's block, rows minus columns from u on.  So what cancels is
// of one block's terms (rows minus columns of the segment left 9.7e-7 of dlog_alpha, 6.2e-7 so).  Latency of a scan over 512 tokens:
// 7.4 us whether 8192 or 6001 tokens.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kBlk) lin_gates_tc_kernel(SeqArgs a, const float* part, const float* phi, int tiles) {
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    int ob, oe;
    if (seq_outside(sh, ob, oe)) {
        zero_rows<float>(a.dla, sh.H, ob, oe, sh.total);
        zero_rows<float>(a.dbeta, sh.H, ob, oe, sh.total);
    }
    const int slot = blockIdx.x / sh.H, h = blockIdx.x % sh.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int s, c, first, rows;
    if (!slot_segment(sh, kSeg, slot, s, c, first, rows, a.err)) return;
    const size_t at = (size_t)slot * sh.H + h;
    const float* p = part + at * kPartAll;
    __shared__ float sums[3][4], whole[4][4];             // whole: rows of a later block with columns of an earlier one
    float from[4], before[4], own[4], pre[4], ph = 0.f;
    for (int i = tid; i < tiles; i += kBlk) ph += phi[at * tiles + i];
    const int last = (rows - 1) / kBlk;                   // a warp has a block's tokens
    float later[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = 4 * tid + e;
        from[e] = before[e] = own[e] = pre[e] = 0.f;
        if (t >= rows) continue;
        const float beta = a.beta[(size_t)(first + t) * sh.H + h], mine = p[kPartCol + warp * kSeg + t];
        float cc = 0.f;
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float x = i > warp && i <= last ? p[kPartCol + i * kSeg + t] : 0.f;
            cc += x;
            later[i] = fmaf(beta, x, later[i]);
        }
        const float ik = p[kPartK + t] + p[kPartK + kSeg + t];
        from[e] = p[kPartQ + t] + p[kPartQ + kSeg + t];
        own[e] = (p[kPartRow + t] - beta * mine) + p[kPartOff + t];
        pre[e] = beta * cc;
        before[e] = beta * ik;
        a.dbeta[(size_t)(first + t) * sh.H + h] = (cc + mine) + p[kPartDiag + t] + ik;
    }
    float f = (from[0] + from[1]) + (from[2] + from[3]), b = (before[0] + before[1]) + (before[2] + before[3]),
          ow = (own[0] + own[1]) + (own[2] + own[3]), pr = (pre[0] + pre[1]) + (pre[2] + pre[3]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float fo = __shfl_down_sync(0xffffffffu, f, o), bo = __shfl_up_sync(0xffffffffu, b, o), oo = __shfl_down_sync(0xffffffffu, ow, o),
                    po = __shfl_up_sync(0xffffffffu, pr, o);
        if (lane + o < 32) {
            f += fo;
            ow += oo;
        }
        if (lane >= o) {
            b += bo;
            pr += po;
        }
    }
    ph = warp_sum(ph);
#pragma unroll
    for (int i = 1; i < 4; ++i) later[i] = warp_sum(later[i]);
    if (lane == 0) {
        sums[0][warp] = f;
        sums[2][warp] = ph;
#pragma unroll
        for (int i = 1; i < 4; ++i) whole[i][warp] = later[i];
    }
    if (lane == 31) sums[1][warp] = b;
    __syncthreads();
    // f, ow: from the first token behind this thread's on; b, pr: up to the token before this thread's.  The neighbour's sums, not this
    // thread's less its own: with fast decays its own terms are far larger than what remains.
    f = __shfl_down_sync(0xffffffffu, f, 1);
    ow = __shfl_down_sync(0xffffffffu, ow, 1);
    b = __shfl_up_sync(0xffffffffu, b, 1);
    pr = __shfl_up_sync(0xffffffffu, pr, 1);
    if (lane == 31) f = ow = 0.f;
    if (lane == 0) b = pr = 0.f;
    ph = (sums[2][0] + sums[2][1]) + (sums[2][2] + sums[2][3]);
    for (int w = 0; w < 4; ++w) {
        if (w > warp) f += sums[0][w];
        if (w < warp) b += sums[1][w];
        for (int i = warp + 1; i < 4 && w < warp; ++i) ph += whole[i][w];
    }
#pragma unroll
    for (int e = 3; e >= 0; --e) {
        f += from[e];
        ow += own[e];
        from[e] = f + ow;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (4 * tid + e < rows) a.dla[(size_t)(first + 4 * tid + e) * sh.H + h] = from[e] + ((b + pr) + ph);
        b += before[e];
        pr += pre[e];
    }
}

// dq (blockIdx.y 0) and dk of heads that share q and k: the sum of theirs, in their order, for the tokens of the slots only (rows of
// a sequence that is not one stay as they were).  A CTA 16 tokens, one thread eight columns.  Bound by memory: 6001 tokens, 8
// heads of 2, 128 columns, 12.0 us (4.6 TB/s; 32 tokens a CTA 13.8).
constexpr int kHeadTok = 16;
__global__ void __launch_bounds__(256) lin_heads_kernel(SeqArgs a, const float* gates, const float* dq, const float* dk) {
    const SeqShape& sh = a.sh;
    griddep_wait();
    griddep_launch();
    const int slots = seg_slots(sh.nseq, sh.total, kSeg), slot = blockIdx.x / (kSeg / kHeadTok), t0 = blockIdx.x % (kSeg / kHeadTok) * kHeadTok;
    const int2 seg = slot_entry(slot_table(gates, slots, sh.H), slot, sh.total);
    const float* in = blockIdx.y == 0 ? dq : dk;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(blockIdx.y == 0 ? a.dq : a.dk);
    const int rep = sh.H / sh.Hk, each = sh.dk / 8;
    const long long row = (long long)sh.Hk * each, n = min(kHeadTok, seg.y - t0) * row;
    for (long long i = threadIdx.x; i < n; i += 256) {
        const int t = (int)(i / row), x = (int)(i - t * row), hk = x / each, d = (x - hk * each) * 8;
        const size_t token = (size_t)seg.x + t0 + t;
        const float* p = in + (token * sh.H + (size_t)hk * rep) * sh.dk + d;
        float y[8], z[8];
        ld8<float>(p, y);
        for (int r = 1; r < rep; ++r) {
            ld8<float>(p + (size_t)r * sh.dk, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += z[j];
        }
        *reinterpret_cast<uint4*>(out + (token * sh.Hk + hk) * sh.dk + d) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
bool map_nd(CUtensorMap* m, int rank, const void* p, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box, bool f32) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    if (enc == nullptr) return false;
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// boxes of 128 bytes by `rows` of the second dimension, or (0) one of it and 64 of the third
bool map_3d(CUtensorMap* m, const void* p, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2], uint32_t rows, bool f32 = false) {
    const cuuint32_t box[3] = {f32 ? 32u : 64u, rows > 0 ? rows : 1u, rows > 0 ? 1u : 64u};
    return map_nd(m, 3, p, dims, strides, box, f32);
}
// Tokens of a head by slabs of 64 columns, `rows` tokens and `slabs` slabs a box: (column, head, token, slab).  Where d is not a
// whole number of slabs, one slab a box, and what lies behind d comes as zeros.
bool slab_map(CUtensorMap* m, const void* p, const SeqShape& sh, int d, int heads, long long ld, int rows, int slabs) {
    const bool whole = d % 64 == 0;
    const cuuint64_t dims[4] = {(cuuint64_t)(whole ? 64 : d), (cuuint64_t)heads, (cuuint64_t)sh.total, (cuuint64_t)(whole ? d / 64 : 1)},
                     strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, 128};
    const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)rows, (cuuint32_t)(whole ? slabs : 1)};
    return map_nd(m, 4, p, dims, strides, box, false);
}
// (d, head, token): what lies behind d comes as zeros, so that any multiple of 16 is one of 64
bool token_map(CUtensorMap* m, const void* p, const SeqShape& sh, int d, int heads, long long ld) {
    return map_3d(m, p, {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)sh.total}, {(cuuint64_t)d * 2, (cuuint64_t)ld * 2}, 0);
}
// (d_k, d_v, term and slot and head)
bool state_map(CUtensorMap* m, const void* p, const SeqShape& sh, int terms, int rows) {
    const cuuint64_t n = (cuuint64_t)terms * seg_slots(sh.nseq, sh.total, kSeg) * sh.H;
    return map_3d(m, p, {(cuuint64_t)sh.dk, (cuuint64_t)sh.dv, n}, {(cuuint64_t)sh.dk * 2, (cuuint64_t)sh.dk * sh.dv * 2}, (uint32_t)rows);
}

// (d_k, d_v, slot and head) of what the segments add
bool local_map(CUtensorMap* m, const float* p, const SeqShape& sh) {
    const cuuint64_t n = (cuuint64_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H;
    return map_3d(m, p, {(cuuint64_t)sh.dk, (cuuint64_t)sh.dv, n}, {(cuuint64_t)sh.dk * 4, (cuuint64_t)sh.dk * sh.dv * 4}, sh.dv < 128 ? sh.dv : 128, true);
}

constexpr uint32_t kSmemMost = 227 * 1024, kSmemHalf = 113 * 1024;      // one CTA an SM, two

RowsPlan rows_plan(int da, int dx) {
    RowsPlan p = {};
    const int na = (da + 63) / 64, nx = (dx + 63) / 64;
    p.x_log = dx > 128 ? 6 : 7;
    p.stage = 2 * kBox * (na > 1 || nx > 1 ? 2 : 1);
    const uint32_t r = na * 2 * kBox, rest = kRowTail;
    // two buffers of row operands where they leave the ring what two blocks' scores and X take
    p.nr = (int)((kSmemMost - rest - 2 * r) / p.stage) >= 2 * ((da + 127) / 128 + (kBlk >> p.x_log)) ? 2 : 1;
    const int room = (int)((kSmemMost - rest - p.nr * r) / p.stage);
    p.ring = room < kMaxRing ? room : kMaxRing;
    p.r = p.ring * p.stage;            // behind the ring
    p.bars = p.r + p.nr * r;
    p.smem = p.bars + kRowTail;
    return p;
}

template <int MODE>
cudaError_t rows_go(const CUtensorMap& ms, const SeqArgs& a, const float* gates, float* part, float* heads, int terms, cudaStream_t st) {
    static bool done[64];
    const SeqShape& sh = a.sh;
    constexpr bool values = MODE == kOut || MODE == kDv;
    const RowsArgs ra = {rows_plan(values ? sh.dk : sh.dv, values ? sh.dv : sh.dk), part, (size_t)kPartAll, heads, gates, terms};
    const cudaError_t e = ensure_smem(lin_rows_tc_kernel<MODE>, kSmemMost, done);
    if (e != cudaSuccess) return e;
    const size_t items = (size_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H * (kSeg / kBlk);      // fours, as the grid's size is
    const dim3 grid((unsigned)(items < kSMs ? items : kSMs));
    struct Operand {
        const void* p;
        int d, heads;
        long long ld;
    } const q = {a.q, sh.dk, sh.Hk, sh.ldq}, k = {a.k, sh.dk, sh.Hk, sh.ldk}, v = {a.v, sh.dv, sh.H, sh.ldv}, o = {a.dout, sh.dv, sh.H, (long long)sh.H * sh.dv},
      r = MODE == kOut ? q : MODE == kDq ? o : MODE == kDk ? v : k, b = MODE == kOut ? k : MODE == kDq ? v : MODE == kDk ? o : q,
      x = MODE == kOut ? v : MODE == kDq ? k : MODE == kDk ? q : o;
    const int na = (r.d + 63) / 64, nx = (x.d + 63) / 64;
    CUtensorMap mr, mb, mx;
    if (!slab_map(&mr, r.p, sh, r.d, r.heads, r.ld, kBlk, na) || !slab_map(&mb, b.p, sh, b.d, b.heads, b.ld, kBlk, na < 2 ? na : 2) ||
        !slab_map(&mx, x.p, sh, x.d, x.heads, x.ld, 1 << ra.p.x_log, nx))
        return cudaErrorInvalidValue;
    return launch_kernel(lin_rows_tc_kernel<MODE>, grid, dim3(kRowThreads), ra.p.smem, st, true, mr, mb, mx, ms, a, ra);
}

cudaError_t prep_go(const SeqArgs& a, float* gates, cudaStream_t st) {
    const unsigned grid = (unsigned)((size_t)seg_slots(a.sh.nseq, a.sh.total, kSeg) * a.sh.H);
    return launch_kernel(lin_prep_kernel, dim3(grid), dim3(kBlk), 0, st, false, a, gates);
}

template <bool BACK>
cudaError_t local_go(const SeqArgs& a, const float* gates, float* local, cudaStream_t st) {
    static bool done[64];
    const SeqShape& sh = a.sh;
    CUtensorMap ma, mb, mo;
    if (!(BACK ? token_map(&ma, a.dout, sh, sh.dv, sh.H, (long long)sh.H * sh.dv) && token_map(&mb, a.q, sh, sh.dk, sh.Hk, sh.ldq)
               : token_map(&ma, a.v, sh, sh.dv, sh.H, sh.ldv) && token_map(&mb, a.k, sh, sh.dk, sh.Hk, sh.ldk)) ||
        !local_map(&mo, local, sh))
        return cudaErrorInvalidValue;
    const cudaError_t e = ensure_smem(lin_local_tc_kernel<BACK>, kLocalSmem, done);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)seg_slots(sh.nseq, sh.total, kSeg) * sh.H * ((sh.dv + 127) / 128) * ((sh.dk + 127) / 128);
    return launch_kernel(lin_local_tc_kernel<BACK>, dim3((unsigned)(tiles < kSMs ? tiles : kSMs)), dim3(kLocalThreads), kLocalSmem, st, !BACK,
                         ma, mb, mo, a, gates);
}

cudaError_t pairs_go(const SeqArgs& a, const float* gates, float* part, cudaStream_t st) {
    static bool done[64];
    const SeqShape& sh = a.sh;
    CUtensorMap q, k, v, o;
    if (!slab_map(&q, a.q, sh, sh.dk, sh.Hk, sh.ldq, kBlk, sh.dk / 64) || !slab_map(&k, a.k, sh, sh.dk, sh.Hk, sh.ldk, kBlk, 1) ||
        !slab_map(&v, a.v, sh, sh.dv, sh.H, sh.ldv, kBlk, 1) || !slab_map(&o, a.dout, sh, sh.dv, sh.H, (long long)sh.H * sh.dv, kBlk, sh.dv / 64))
        return cudaErrorInvalidValue;
    PairsPlan p = {};
    p.r2 = (sh.dk + 63) / 64 * 2 * kBox;
    p.stages = p.r2 + (sh.dv + 63) / 64 * 2 * kBox;
    p.two = p.stages + 2 * 2 * kBox + kPairTail > kSmemHalf;
    const uint32_t room = (p.two ? kSmemMost : kSmemHalf) - p.stages - kPairTail;
    p.ring = (int)(room / (2 * kBox)) < kMaxRing ? (int)(room / (2 * kBox)) : kMaxRing;
    p.bars = p.stages + p.ring * 2 * kBox;
    p.smem = p.bars + kPairTail;
    const cudaError_t e = ensure_smem(lin_pairs_tc_kernel, kSmemMost, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((size_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H * (kSeg / kBlk)));
    return launch_kernel(lin_pairs_tc_kernel, grid, dim3(kPairThreads), p.smem, st, true, q, o, k, v, a, p, gates, part);
}

}  // namespace

LinLayout lin_layout_tc(const SeqShape& s) {
    LinLayout L = {};
    const size_t slots = seg_slots(s.nseq, s.total, kSeg), sth = slots * s.H, state = sth * s.dv * s.dk, gates = sth * kGAll * 4 + slots * 12 + 16;
    L.rec_gates = align_up(3 * state * 2, kSectionAlign);
    L.rec_total = align_up(L.rec_gates + gates, kSectionAlign);
    L.ws_start = align_up(L.ws_local + state * 4, kSectionAlign);
    L.ws_gates = align_up(L.ws_start + 2 * state * 2, kSectionAlign);
    L.ws_forward = align_up(L.ws_gates + gates, kSectionAlign);
    // the backward pass's own, from ws_start on
    L.ws_end = L.ws_start;
    L.ws_phi = align_up(L.ws_end + 3 * state * 2, kSectionAlign);
    L.ws_part = align_up(L.ws_phi + sth * scan_tiles(s) * 4, kSectionAlign);
    L.ws_heads = align_up(L.ws_part + sth * kPartAll * 4, kSectionAlign);
    L.ws_total = align_up(L.ws_heads + (s.H > s.Hk ? 2 * (size_t)s.total * s.H * s.dk * 4 : 0), kSectionAlign);
    if (L.ws_total < L.ws_forward) L.ws_total = L.ws_forward;
    return L;
}

cudaError_t launch_linear_forward_tc(const SeqArgs& a, cudaStream_t st) {
    const SeqShape& sh = a.sh;
    const LinLayout L = lin_layout_tc(sh);
    const bool keep = a.rec != nullptr;
    float *local = reinterpret_cast<float*>(a.ws + L.ws_local), *gates = reinterpret_cast<float*>(keep ? a.rec + L.rec_gates : a.ws + L.ws_gates);
    char* starts = keep ? a.rec : a.ws + L.ws_start;
    const size_t apart = (size_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H * sh.dv * sh.dk;
    const auto scan = [&]() {
        return launch_linear_scan(sh, kSeg, keep ? 3 : 2, false, local, gates + kGTot + 4, kGAll, a.S0, starts, apart, nullptr, nullptr, a.S_T, a.err, st);
    };
    if (sh.total == 0) return scan();            // the states pass through
    CUtensorMap ms;
    if (!state_map(&ms, starts, sh, 2, sh.dv)) return cudaErrorInvalidValue;
    cudaError_t e = prep_go(a, gates, st);
    if (e == cudaSuccess) e = local_go<false>(a, gates, local, st);
    if (e == cudaSuccess) e = scan();
    if (e == cudaSuccess) e = rows_go<kOut>(ms, a, gates, nullptr, nullptr, 2, st);
    return e;
}

cudaError_t launch_linear_backward_tc(const SeqArgs& a, cudaStream_t st) {
    const SeqShape& sh = a.sh;
    const LinLayout L = lin_layout_tc(sh);
    const float* gates = reinterpret_cast<const float*>(a.rec + L.rec_gates);
    float *local = reinterpret_cast<float*>(a.ws + L.ws_local), *phi = reinterpret_cast<float*>(a.ws + L.ws_phi),
          *part = reinterpret_cast<float*>(a.ws + L.ws_part), *dq = nullptr, *dk = nullptr;
    char* ends = a.ws + L.ws_end;
    if (sh.H > sh.Hk) {
        dq = reinterpret_cast<float*>(a.ws + L.ws_heads);
        dk = dq + (size_t)sh.total * sh.H * sh.dk;
    }
    const size_t apart = (size_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H * sh.dv * sh.dk;
    const auto scan = [&]() {
        return launch_linear_scan(sh, kSeg, 3, true, local, gates + kGTot + 4, kGAll, a.dS_T, ends, apart, a.rec, phi, a.dS0, a.err, st);
    };
    if (sh.total == 0) return scan();
    CUtensorMap ms, me_keys, me_values;      // the starts by 64 rows of d_v; the ends so and by all
    if (!state_map(&ms, a.rec, sh, 3, 64) || !state_map(&me_keys, ends, sh, 2, 64) || !state_map(&me_values, ends, sh, 3, sh.dv))
        return cudaErrorInvalidValue;
    cudaError_t e = local_go<true>(a, gates, local, st);
    if (e == cudaSuccess) e = scan();
    if (e == cudaSuccess) e = rows_go<kDq>(ms, a, gates, part + kPartQ, dq, 3, st);
    if (e == cudaSuccess) e = rows_go<kDk>(me_keys, a, gates, nullptr, dk, 2, st);
    if (e == cudaSuccess) e = rows_go<kDv>(me_values, a, gates, part + kPartK, nullptr, 3, st);
    if (e == cudaSuccess) e = pairs_go(a, gates, part, st);
    if (e == cudaSuccess)
        e = launch_kernel(lin_gates_tc_kernel, dim3((unsigned)((size_t)seg_slots(sh.nseq, sh.total, kSeg) * sh.H)), dim3(kBlk), 0, st, true, a,
                          (const float*)part, (const float*)phi, scan_tiles(sh));
    if (e == cudaSuccess && sh.H > sh.Hk)
        e = launch_kernel(lin_heads_kernel, dim3((unsigned)((size_t)seg_slots(sh.nseq, sh.total, kSeg) * (kSeg / kHeadTok)), 2), dim3(256), 0, st, true, a, gates,
                          (const float*)dq, (const float*)dk);
    return e;
}

}  // namespace gdn

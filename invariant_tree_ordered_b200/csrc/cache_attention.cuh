// Attention over the paged 8-bit cache (cache.cuh), with the key reduction in tree order.
//
// Query t of sequence b sits at position i = start[b] + t and sees the keys at positions 0..i.  They are reduced like
// in the other attentions of the library: leaves of 128 consecutive positions, each a (max, sum, weighted value sum)
// summary, combined by the halving tree over the ceil((i + 1) / 128) leaves, so a row's bits depend only on its
// query and the cache's contents, never on the batch or on how the work is split.
//
// The bytes of a page go to the tensor cores as they lie in the cache (tcgen05 kind::f8f6f4, unswizzled operands), so
// nothing is ever widened.  What is not 8 bits wide is given to them as two e4m3 terms of 4 significant bits:
//   query   q 2^x = h + l / 32, x such that the row's largest |q| 2^x lies in [128, 256): exact down to 2^-14 of it, and
//           below that to 2^-22 of it;
//   weight  256 f p = h + l, rounded at 2^-9 relative or 2^-18 of the leaf's largest (f below).
// Why two terms are enough for the weights: the output is rounded to bf16 once, by up to 2^-8, and the weights' roundings do
// not know of one another, so that their mean over the keys is smaller still.  Against 64 bits the chunks below are off by
// 1.666e-3 of the output's norm, and sums in fp32 rounded to bf16 by 1.659e-3.  A third term would make the products of the
// values half as long again.  The sum s takes the weights before they are rounded: a key of a page with a small f keeps its
// share of s in full where its 256 f p is cut, which a sum of the rounded ones would lose.
// With keys as the 128 rows of an MMA and queries as its columns, few queries waste few columns, which suits a decode
// step (G query heads of one token share a kv head):
//   S^T = K [h | l]     M = 128 keys, N = 2 rows, K = head_dim
//   a_j = (S_h + S_l / 32) kscale_j;  m = max over the leaf's visible keys;  p_j = 2^((a_j - m) c), c = 2^-x log2(e) / sqrt(D)
//   f_j = vscale_j / (largest vscale among the row's visible pages of the leaf), a power of two
//   s = sum of p_j in fp32: within 32 keys by halves (16 apart first), then (w0 + w1) + (w2 + w3)
//   O^T = V^T [h | l]   M = 128 dims, N = 2 rows, K = 128 keys, O = O_h + O_l
// The two terms stand side by side in N, not one after the other in K: with few columns an MMA's time is that of reading
// its 128 rows (measured: scores as K h + K l, l in e5m2, took four long contexts from 108 to 154 us).
// Combining two summaries: M = max, e = 2^(m - M) (1 for the side that holds M), s = fma(s', e', s e), o likewise.
//
// A CTA works on tiles of R rows (query, head) that share a kv head and a 128-position block, hence the number of leaves.
// Warp 0 copies pages to shared memory (cp.async.bulk, one copy per page and operand), warp 1 issues the MMAs, and four
// warps do the rest: a thread is a key for the scores and a dim for the values, so its summaries' value parts live in its
// TMEM lane (pending ones too).
//
// Split: the work is cut into units (tile, tree node of at most T leaves) and each CTA takes a contiguous run of them
// by weight; T is chosen on the device such that a CTA has about CATT_UNITS units.  A tile whose tree is cut leaves its
// nodes' summaries in the workspace, and a second kernel evaluates the tree above them.  Nodes are subtrees of the row's
// own tree, so the bits do not depend on the cut.
//
// What bounds it.  Few rows over long contexts: the cache's bytes (4 sequences of 120-131 thousand positions, 32 query and
// 4 kv heads of 128 dims: 111 us with both kernels, 4.7 TB/s; the first one reads the cache's bytes and nothing more at
// 5.0 TB/s, its planning included).  Mixed batches: the chain of a leaf (scores, maximum over four warps, weights, values,
// tree: 4.6 thousand cycles in the long contexts, with three CTAs on an SM) and the 10 us of planning, first loads and the
// second kernel (64 sequences of 1 to 8192 positions: 53 us, 18 us of bytes).  Many rows: the same chain's instructions, 36 per
// row, key and lane over all six warps (chunks of 300-512 queries over 5-8 thousand positions: 0.86 ms, 199 TFLOP/s); issue
// slots are 47 % used, the tensor pipe 3 to 11 %.
#pragma once

#include <cuda_fp16.h>

#include "cache.cuh"

namespace tbik {

constexpr int CATT_LEAF = 128;
// Units per CTA that the split aims at, and the weight of a unit's start in leaves.  Units of 1, 2, 3, 4 per CTA took
// 137, 117, 110, 108 us for four long contexts and 53, 56, 57, 58 us for a mixed batch; starts of 1, 2, 3, 5 leaves 54,
// 52, 56, 54 us for that batch and the same for the others.
constexpr int CATT_UNITS = 3;
constexpr int CATT_START = 2;
constexpr int CATT_JOIN_DEPTH = 4;  // levels above the units that one thread of the second kernel evaluates alone

struct CacheAttParams {
    const uint16_t* q;
    const uint8_t* pages;
    const float* scales;
    const int32_t* table;
    const int32_t* start;
    const int32_t* cu;
    const int32_t* rows;
    uint16_t* out;
    int tokens, batch, slots, max_pages, num_pages, heads, kv_heads, page, max_q, max_keys;
    int group;       // heads / kv_heads
    int page_shift;  // log2(page)
    uint32_t group_inv;  // ceil(2^31 / group)
    float scale;     // log2(e) / sqrt(head_dim)
    // workspace: number of cut tiles, their descriptors, and the nodes' summaries
    int* count;      // [2]: cut tiles, whether a tree was cut deeper than CATT_JOIN_DEPTH
    int4* tiles;     // [max_slots / 2][2]
    float2* ms;      // [max_slots][R]
    float* o;        // [max_slots][R][D]
    int max_slots;
    unsigned long long wait_cycles;
    unsigned debug;
};

template <int D_, int R_>
struct CattCfg {
    static constexpr int D = D_, R = R_;
    static constexpr int NC = 2 * R;                // columns of S and of O
    static constexpr int SBUF = R == 32 ? 1 : 2, OBUF = SBUF;
    static constexpr int PENDING = R == 32 ? 5 : 6;  // summaries that can wait: log2 of the leaves of a unit
    static constexpr int MAX_NODE = 1 << PENDING;
    static constexpr int TPEND = R == 32 ? 4 : 6;   // of them in TMEM; the largest ones may be in shared memory
    static constexpr int S_COL = 0, O_COL = SBUF * NC, ST_COL = O_COL + OBUF * NC;
    static constexpr int COLS = R == 8 ? 128 : 256;
    static constexpr int CTAS = R == 8 ? 3 : 2;      // that an SM holds
    static_assert(ST_COL + TPEND * R <= COLS && COLS * CTAS <= 512, "TMEM columns");
    static constexpr int THREADS = 192;
    static constexpr int TILE = 128 * D;             // bytes of a leaf's keys or values
    static constexpr int STAGES = D == 64 ? 4 : R == 16 ? 3 : 2;
    static constexpr int OFF_K = 0, OFF_V = STAGES * TILE, OFF_Q = 2 * STAGES * TILE;
    static constexpr int QB = NC * D, PB = 128 * NC;
    static constexpr int OFF_P = OFF_Q + QB;
    static constexpr int OFF_ST = OFF_P + PB;  // the pending summaries that TMEM has no room for
    static constexpr int OFF_BAR = OFF_ST + (PENDING - TPEND) * R * 128 * 4;
    static constexpr int OFF_X = OFF_BAR + 512;
    // in floats: maxima [2][4][R], sums [2][4][R], constants [2][R], value scales [2][8],
    // and per warp: factors and rows [4][R], pending (m, s) [PENDING][2][R]
    static constexpr int X_MAX = 0, X_SUM = 8 * R, X_CST = 16 * R, X_PV = 18 * R, X_WARP = X_PV + 16;
    static constexpr int X_PER_WARP = 4 * R + PENDING * 2 * R;
    static constexpr int X_FLOATS = X_WARP + 4 * X_PER_WARP;
    static constexpr int SMEM = OFF_X + X_FLOATS * 4;
    static_assert(SMEM <= 230000, "shared memory");
};

__device__ __forceinline__ uint64_t smem_desc_flat(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46;
}
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// e4m3 operands (format 0), fp32 accumulator; both operands K-major, or both MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int mn_major) {
    return (1u << 4) | ((uint32_t)mn_major << 15) | ((uint32_t)mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float warp_max_f32(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int N>
__device__ __forceinline__ void catt_ld(uint32_t addr, uint32_t (&r)[N]);
template <int N>
__device__ __forceinline__ void catt_st(uint32_t addr, const float (&v)[N]);
template <>
__device__ __forceinline__ void catt_ld<8>(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void catt_ld<16>(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void catt_ld<32>(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void catt_ld<64>(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr)
        : "memory");
}
template <>
__device__ __forceinline__ void catt_st<8>(uint32_t addr, const float (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
        : "memory");
}
template <>
__device__ __forceinline__ void catt_st<16>(uint32_t addr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
        : "memory");
}
template <>
__device__ __forceinline__ void catt_st<32>(uint32_t addr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])), "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
        : "memory");
}

// The bounded waits of device_common.cuh with their loops kept small: the softmax warps run through their whole code
// once per leaf, and unrolled waits (of which there are a dozen) would push it out of the instruction cache
// (measured: 160 KB of code, a leaf took three times as long).
__device__ __forceinline__ bool catt_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    bool ok;
#pragma unroll 1
    while (!(ok = mbar_try_wait(bar, parity))) {
        if (*abort_flag) break;
        if ((uint64_t)(clock64() - t0) > limit) {
            *abort_flag = 1;
            set_error(TBIK_ERR_TIMEOUT);
            break;
        }
    }
    return ok;
}
__device__ __forceinline__ void catt_drain(uint64_t* bar, uint32_t parity, uint64_t limit) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if ((uint64_t)(clock64() - t0) > limit) {
            set_error(TBIK_ERR_TIMEOUT);
            break;
        }
    }
}

// ------------------------------------------------------------------ the split

// Leaves of node v (of 2^d, left to right) at depth d of the tree over L leaves.  Halving gives the left part the odd
// leaf, so the L mod 2^d nodes with one leaf more are those whose index, its d bits reversed, is smallest.  0 where a
// single leaf cannot be cut any further.
__host__ __device__ __forceinline__ int catt_node_size(int L, int d, int v) {
#ifdef __CUDA_ARCH__
    const uint32_t rev = d ? __brev((uint32_t)v) >> (32 - d) : 0u;
#else
    uint32_t rev = 0;
    for (int k = 0; k < d; ++k) rev |= (uint32_t)(v >> k & 1) << (d - 1 - k);
#endif
    return (int)(((uint32_t)L + (1u << d) - 1u - rev) >> d);
}
// The smallest depth whose nodes have at most T leaves.
__host__ __device__ __forceinline__ int catt_depth(int L, int T) {
    int d = 0;
    for (int x = (L + T - 1) / T; (1 << d) < x;) ++d;
    return d;
}
// Number of nodes that leaf j of a tree over n leaves closes.
__host__ __device__ __forceinline__ int catt_pops(int n, int j) {
    int pops = 0;
#pragma unroll 1
    while (n > 1) {
        if (j == n - 1) ++pops;
        else pops = 0;
        const int h = (n + 1) >> 1;
        if (j < h) {
            n = h;
        } else {
            j -= h;
            n -= h;
        }
    }
    return pops;
}

// x / group for x < 2^16 (group <= 64: the error x / 2^31 is below 1 / group).
__device__ __forceinline__ int catt_div(const CacheAttParams& p, int x) { return (int)((uint64_t)(uint32_t)x * p.group_inv >> 31); }

// The new tokens of a sequence within one block of 128 positions.
struct CattItem {
    int b, slot;    // sequence, table row
    int tok0, i0;   // its first token (packed) and that token's position
    int rows, L;    // (token, head) rows per kv head (0: nothing to do), leaves
};

// Sequence b's first packed token and their number (0 if cu makes no sense).
__device__ __forceinline__ int catt_tokens(const CacheAttParams& p, int b, int& n) {
    if (!p.cu) {
        n = 1;
        return b;
    }
    const int a = p.cu[b], e = p.cu[b + 1];
    n = (a < 0 || e < a || e > p.tokens) ? 0 : e - a;
    return a;
}
// How many of a sequence's n tokens (from its first on) have an answer.
__device__ __forceinline__ int catt_usable(const CacheAttParams& p, int s, int slot, int n) {
    if (s < 0 || slot < 0 || slot >= p.slots) return 0;
    long long lim = min((long long)p.max_keys, (long long)p.max_pages * p.page) - s;
    lim = min(min(lim, (long long)n), (long long)p.max_q);
    return lim > 0 ? (int)lim : 0;
}
// What can be answered of sequence b: its first `use` tokens, from packed token `first` and position s on (use = 0: s = 0).
struct CattSeq {
    int b, slot, first, s, use;
    int n;  // its tokens
};
__device__ __forceinline__ CattSeq catt_seq(const CacheAttParams& p, int b, bool& bad) {
    CattSeq q;
    q.b = b;
    q.first = catt_tokens(p, b, q.n);
    q.s = p.start[b];
    q.slot = p.rows ? p.rows[b] : b;
    q.use = catt_usable(p, q.s, q.slot, q.n);
    bad |= q.use < q.n || (p.cu && q.n == 0 && (q.first < 0 || p.cu[b + 1] < q.first || p.cu[b + 1] > p.tokens));
    if (q.use == 0) q.s = 0;
    return q;
}
// Its tokens in block blk of 128 positions.
__device__ __forceinline__ CattItem catt_item(const CacheAttParams& p, const CattSeq& q, int blk) {
    CattItem t;
    const int lo = max(0, blk * CATT_LEAF - q.s), hi = min(q.use, (blk + 1) * CATT_LEAF - q.s);
    t.b = q.b;
    t.slot = q.slot;
    t.L = blk + 1;
    t.tok0 = q.first + lo;
    t.i0 = q.s + lo;
    t.rows = hi > lo ? (hi - lo) * p.group : 0;
    return t;
}

// Where a CTA begins: set by the whole block, read by every role.
struct CattPlan {
    long long x0, x1, at;  // the CTA's run of the weight axis, and the weight before its first item
    CattItem it;           // that item (no rows: none)
    int slot_base, tile_base, T;
};

// A unit: node v of tile `tau` of kv head h of an item (in this order, the nodes of a tile one after the other, so that
// its queries are taken once).
template <int R>
struct CattUnits {
    CattItem it;
    int h, tau, tiles, d, v, lo, size;
    int slot_base, tile_base, T;
    long long at, end;

    __device__ __forceinline__ void enter(const CattItem& i) {
        it = i;
        tiles = (it.rows + R - 1) / R;
        d = catt_depth(it.L, T);
    }
    // Positions of the tile's first and last query.
    __device__ __forceinline__ int imin(const CacheAttParams& p) const { return it.i0 + catt_div(p, tau * R); }
    __device__ __forceinline__ int imax(const CacheAttParams& p) const { return it.i0 + catt_div(p, min(it.rows, (tau + 1) * R) - 1); }
    __device__ __forceinline__ int slot() const { return slot_base + ((h * tiles + tau) << d) + v; }
    __device__ __forceinline__ bool same_tile(const CattUnits& o) const { return it.b == o.it.b && it.L == o.it.L && h == o.h && tau == o.tau; }
    // The first unit that starts at or behind x0.
    __device__ __forceinline__ bool first(const CacheAttParams& p, const CattPlan& pl) {
        slot_base = pl.slot_base;
        tile_base = pl.tile_base;
        T = pl.T;
        end = pl.x1;
        if (pl.it.rows == 0 || pl.x0 >= pl.x1) return false;
        enter(pl.it);
        // a tile weighs its leaves and a start for each node that is not empty; of these there are min(v, lo) before v
        const int cost = it.L + CATT_START * min(it.L, 1 << d);
        const long long y = pl.x0 - pl.at, tile = y < (1ll << 31) ? (long long)((uint32_t)y / (uint32_t)cost) : y / cost;
        const int z = (int)(y - tile * cost);
        h = (int)(tile / tiles);
        tau = (int)(tile - (long long)h * tiles);
        v = lo = 0;
        size = it.L;
#pragma unroll 1
        for (int k = d - 1; k >= 0; --k) {  // down to the last node that starts at or before z
            const int left = (size + 1) >> 1, r = lo + left;
            if (r + CATT_START * min(v + (1 << k), r) <= z) {
                v += 1 << k;
                lo = r;
                size -= left;
            } else {
                size = left;
            }
        }
        at = pl.at + tile * cost + lo + CATT_START * min(v, lo);
        return at < pl.x0 || size == 0 ? next(p) : at < end;
    }
    __device__ __forceinline__ bool next(const CacheAttParams& p) {
        if (size) at += size + CATT_START;
        if (at >= end) return false;
        lo += size;
#pragma unroll 1
        while (++v < (1 << d)) {
            size = catt_node_size(it.L, d, v);
            if (size) return true;
        }
        v = lo = 0;
        size = catt_node_size(it.L, d, 0);
        if (++tau < tiles) return true;
        tau = 0;
        if (++h < p.kv_heads) return true;
        h = 0;
        if (d > 0) {
            slot_base += (p.kv_heads * tiles) << d;
            tile_base += p.kv_heads * tiles;
        }
        // the sequence's next block, or the next sequence that has something to do
        bool bad = false;
        int blk = it.L, b = it.b;
#pragma unroll 1
        for (;;) {
            const CattSeq q = catt_seq(p, b, bad);
            if (blk < 0) blk = q.s / CATT_LEAF;
            if (blk * CATT_LEAF < q.s + q.use) {
                enter(catt_item(p, q, blk));
                break;
            }
            if (++b >= p.batch) return false;
            blk = -1;
        }
        v = lo = 0;
        size = catt_node_size(it.L, d, 0);
        return true;
    }
};

__device__ __forceinline__ long long catt_div_up(long long a, int b) {
    return a < (1ll << 31) ? (long long)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b) : (a + b - 1) / b;
}

// Per warp of the block: sums of a scan step.
struct CattScan {
    long long w, c;
    int flags;
};
// Sums of w and c over lower threads, their totals over the block, and the or of the flags.  Two barriers.
__device__ __forceinline__ void catt_scan(long long& w, long long& c, int& flags, CattScan* buf, long long& wt, long long& ct) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long sw = w, sc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sw, o), z = __shfl_up_sync(0xffffffffu, sc, o);
        if (lane >= o) {
            sw += y;
            sc += z;
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    __syncthreads();
    if (lane == 31) buf[warp] = CattScan{sw, sc, flags};
    __syncthreads();
    long long bw = 0, bc = 0;
    wt = ct = 0;
    flags = 0;
#pragma unroll 1
    for (int k = 0; k < (int)blockDim.x / 32; ++k) {
        const CattScan t = buf[k];
        if (k < warp) {
            bw += t.w;
            bc += t.c;
        }
        wt += t.w;
        ct += t.c;
        flags |= t.flags;
    }
    w = bw + sw - w;
    c = bc + sc - c;
}

// Fills `pl`; true if some token of the call has no answer.  Every thread takes a run of a sequence's blocks of 128
// positions: `per` threads share a sequence when there are fewer sequences than threads, and with as many threads as runs
// (the usual case) every sequence is read once.  Only blocks that hold tokens are looked at, so the work does not depend on
// max_q (a call with 1024 sequences of 8 tokens and max_q left at its default took 931 us with one look per sequence and
// block that max_q allows; it takes 137 us).
template <int R, int MAX_NODE>
__device__ __forceinline__ bool catt_plan_body(const CacheAttParams& p, CattPlan* pl, CattScan* buf) {
    const int tid = threadIdx.x, nt = blockDim.x;
    int shift = 0;
    while (p.cu && (long long)p.batch << (shift + 1) <= nt) ++shift;
    const int runs = p.batch << shift;
    bool bad = false;
    int flags = 0;
    CattSeq q;
    int k0 = 0, k1 = 0;  // blocks of the run
    auto load = [&](int i) {
        q = catt_seq(p, i >> shift, bad);
        const int f = q.s / CATT_LEAF, blocks = q.use ? (q.s + q.use - 1) / CATT_LEAF + 1 - f : 0, sub = i & ((1 << shift) - 1);
        k0 = f + (int)((long long)blocks * sub >> shift);
        k1 = f + (int)((long long)blocks * (sub + 1) >> shift);
    };
    auto tiles = [&](int k) { return (long long)p.kv_heads * ((catt_item(p, q, k).rows + R - 1) / R); };
    long long leaves = 0, tokens = 0, total = 0, t0, t1;
#pragma unroll 1
    for (int i = tid; i < runs; i += nt) {
        load(i);
        if (!(i & ((1 << shift) - 1))) tokens += q.n;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) leaves += tiles(k) * (k + 1);
    }
    catt_scan(leaves, tokens, flags, buf, t0, t1);
    if (t1 > p.tokens) {
        // Ranges that overlap: their work, and the slots that it asks for, are not bounded by the call's sizes.
        if (tid == 0) {
            pl->it.rows = 0;
            pl->x0 = pl->x1 = 0;
            if (blockIdx.x == 0) {
                set_error(TBIK_ERR_POSITION);
                if (p.max_slots) p.count[0] = p.count[1] = 0;
            }
        }
        return false;
    }
    long long unused = 0;
    const long long aim = catt_div_up(t0, (int)gridDim.x * CATT_UNITS);
    const int T = (int)min((long long)MAX_NODE, max(1ll, aim));
    // A block's weight, which is that of its units (their leaves and their start), added to w; its slots and tiles, if its
    // trees are cut, to c: (slots << 32) + tiles.
    auto add = [&](int k, long long& w, long long& c) {
        const long long ht = tiles(k);
        const int L = k + 1, d = catt_depth(L, T);
        w += (L + CATT_START * min(L, 1 << d)) * ht;
        if (d) {
            c += ((ht << d) << 32) + ht;
            if (d > CATT_JOIN_DEPTH) flags |= 2;
        }
    };
    if (runs > nt) {
        long long w = 0;
#pragma unroll 1
        for (int i = tid; i < runs; i += nt) {
            load(i);
#pragma unroll 1
            for (int k = k0; k < k1; ++k) add(k, w, unused);
        }
        unused = 0;
        catt_scan(w, unused, flags, buf, total, t1);
    }
    if (tid == 0) {
        pl->it.rows = 0;
        pl->T = T;
    }
    long long at = 0, cut = 0, step = 0;
    flags = 0;
#pragma unroll 1
    for (int base = 0; base < runs; base += nt) {
        long long w = 0, c = 0, wt, ct;
        if (base + tid < runs) {
            if (runs > nt) load(base + tid);
#pragma unroll 1
            for (int k = k0; k < k1; ++k) add(k, w, c);
        }
        int f = flags | (bad ? 1 : 0);
        const long long mine = w;
        catt_scan(w, c, f, buf, wt, ct);
        flags = f;
        if (base == 0) {
            if (runs <= nt) total = wt;
            step = catt_div_up(total, (int)gridDim.x);
        }
        const long long x0 = step * blockIdx.x;
        if (mine && at + w <= x0 && x0 < at + w + mine) {
            long long a = at + w, e = cut + c, next = a;
            int k = k0;
#pragma unroll 1
            for (; k + 1 < k1; ++k) {
                long long ne = e;
                add(k, next, ne);
                if (x0 < next) break;
                a = next;
                e = ne;
            }
            pl->it = catt_item(p, q, k);
            pl->at = a;
            pl->slot_base = (int)(e >> 32);
            pl->tile_base = (int)(e & 0xffffffff);
        }
        at += wt;
        cut += ct;
    }
    if (tid == 0) {
        pl->x0 = min(total, step * blockIdx.x);
        pl->x1 = min(total, step * (blockIdx.x + 1));
        if (blockIdx.x == 0 && p.max_slots) {
            p.count[0] = (cut >> 32) > p.max_slots ? 0 : (int)(cut & 0xffffffff);
            p.count[1] = flags & 2;
        }
    }
    return flags & 1;
}

// A call of its own in the small tiles' kernels, whose roles' registers are then laid out without it (drafted tokens 41.6 us
// in place of 43.0; one query 13.7 in place of 13.3), part of the kernel for 32 rows (chunks 852 us in place of 856).
template <int R, int MAX_NODE>
__device__ __noinline__ bool catt_plan_call(const CacheAttParams& p, CattPlan* pl, CattScan* buf) {
    return catt_plan_body<R, MAX_NODE>(p, pl, buf);
}
template <int R, int MAX_NODE>
__device__ __forceinline__ bool catt_plan(const CacheAttParams& p, CattPlan* pl, CattScan* buf) {
    if constexpr (R == 32) return catt_plan_body<R, MAX_NODE>(p, pl, buf);
    else return catt_plan_call<R, MAX_NODE>(p, pl, buf);
}

// Tokens without an answer: NaN, and an error unless the sequence was not granted (start < 0).
template <int D>
__device__ __noinline__ void catt_mark(const CacheAttParams& p) {
#pragma unroll 1
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        int n;
        const int first = catt_tokens(p, b, n), s = p.start[b];
        if (n == 0 && p.cu && p.cu[b + 1] != first) {
            if (threadIdx.x == 0) set_error(TBIK_ERR_POSITION);
            continue;
        }
        const int use = catt_usable(p, s, p.rows ? p.rows[b] : b, n);
        if (use >= n) continue;
        if (s >= 0 && threadIdx.x == 0) set_error(TBIK_ERR_PAGE);
        uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)(first + use) * p.heads * D);
        const size_t m = (size_t)(n - use) * p.heads * (D / 8);
#pragma unroll 1
        for (size_t k = threadIdx.x; k < m; k += blockDim.x) o[k] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    }
}

// ------------------------------------------------------------------ the kernel

// Factors of two summaries' parts: 1 for the side that holds the maximum.
__device__ __forceinline__ void catt_factors(float am, float bm, float& M, float& ea, float& eb) {
    M = fmaxf(am, bm);
    ea = am == M ? 1.0f : ex2_hw(am - M);
    eb = bm == M ? 1.0f : ex2_hw(bm - M);
}

template <int D, int R>
__global__ void __launch_bounds__(CattCfg<D, R>::THREADS, CattCfg<D, R>::CTAS) cache_attention_kernel(const __grid_constant__ CacheAttParams p) {
    using C = CattCfg<D, R>;
    constexpr int ST = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ CattPlan plan;
    __shared__ CattScan scan_buf[16];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t *kf = bars, *ke = bars + ST, *vf = bars + 2 * ST, *ve = bars + 3 * ST;  // [ST] landed, MMAs retired
    uint64_t* b = bars + 4 * ST;   // s_full[2] s_empty[2] o_full[2] o_empty[2] p_full q_full
    uint64_t* done = b + 10;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((4 * ST + 12) * 8 <= 512, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t lim = p.wait_cycles;
    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int i = 0; i < 4 * ST; ++i) mbar_init(&bars[i], 1);
#pragma unroll 1
        for (int i = 0; i < 10; ++i) mbar_init(&b[i], i == 2 || i == 3 || i >= 6 ? 4 : 1);  // what four warps report
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::COLS);
        tmem_relinquish();
    }
    const bool marks = catt_plan<R, C::MAX_NODE>(p, &plan, scan_buf);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    CattUnits<R> u;
    const bool any = u.first(p, plan);

    if (warp == 0) {
        // ---------------------------------------------------- page copies
        const int npl = CATT_LEAF >> p.page_shift;
        const uint32_t pbytes = (uint32_t)p.page * D;
        const size_t vplane = (size_t)p.num_pages * p.kv_heads * pbytes;
        uint32_t g = 0, gv = 0;  // leaves whose keys, values were requested
        bool ok = true;
#pragma unroll 1
        for (bool more = any; more && ok; more = u.next(p)) {
            const int32_t* row = p.table + (size_t)u.it.slot * p.max_pages;
            const int pages = (u.imax(p) >> p.page_shift) + 1;  // that the tile sees
            int pg = u.lo * npl + lane;
            int id = lane < npl && pg < pages ? row[pg] : 0;
#pragma unroll 1
            for (int l = 0; l < u.size; ++l) {
                const int here = min(npl, pages - (u.lo + l) * npl);
                const int pn = pg + npl;
                const int idn = l + 1 < u.size && lane < npl && pn < pages ? row[pn] : 0;
                if (id < 0 || id >= p.num_pages) id = 0;  // its keys are marked where the scores are taken
                const uint8_t* src = p.pages + ((size_t)id * p.kv_heads + u.h) * pbytes;
                const int st = g % ST;
                const uint32_t ph = (g / ST) & 1;
                ok = g < ST || catt_wait(&ke[st], ph ^ 1, abort_flag, lim);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&kf[st], here * pbytes);
                __syncwarp();
                if (lane < here) bulk_load(smem_u32(smem + C::OFF_K + st * C::TILE) + lane * pbytes, src, pbytes, smem_u32(&kf[st]));
                ok = g++ < ST || catt_wait(&ve[st], ph ^ 1, abort_flag, lim);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&vf[st], here * pbytes);
                __syncwarp();
                if (lane < here) bulk_load(smem_u32(smem + C::OFF_V + st * C::TILE) + lane * pbytes, src + vplane, pbytes, smem_u32(&vf[st]));
                ++gv;
                pg = pn;
                id = idn;
            }
        }
        if (lane == 0) {
            // what is in flight has to land before the CTA can exit
#pragma unroll 1
            for (uint32_t x = g > (uint32_t)ST ? g - ST : 0; x < g; ++x) catt_drain(&kf[x % ST], (x / ST) & 1, lim);
#pragma unroll 1
            for (uint32_t x = gv > (uint32_t)ST ? gv - ST : 0; x < gv; ++x) catt_drain(&vf[x % ST], (x / ST) & 1, lim);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issue
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_e4m3_f32(128, C::NC, 0), id_o = idesc_e4m3_f32(128, C::NC, 1);
            uint32_t g = 0, nq = 0;
            CattUnits<R> tile = u;
            // O^T of leaf x; D = 64 leaves lanes 64..127 with what lies behind (not read)
            auto values = [&](uint32_t x) -> bool {
                const int st = x % ST;
                if (!catt_wait(&vf[st], (x / ST) & 1, abort_flag, lim)) return false;
                const uint32_t ob = x % C::OBUF, use = x / C::OBUF;
                if (!catt_wait(&b[8], x & 1, abort_flag, lim)) return false;
                if (use > 0 && !catt_wait(&b[6 + ob], (use - 1) & 1, abort_flag, lim)) return false;
                tc_fence_after();
                const uint32_t pa = smem_u32(smem + C::OFF_P);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_f8(tmem + C::O_COL + ob * C::NC,
                              smem_desc_flat(smem_u32(smem + C::OFF_V + st * C::TILE) + k * 32 * D, D * 8, 128),
                              smem_desc_flat(pa + k * 32 * C::NC, 8 * C::NC, 128), id_o, k ? 1u : 0u);
                tc_commit(&b[4 + ob]);
                tc_commit(&ve[st]);
                return true;
            };
#pragma unroll 1
            for (bool more = any; more; more = u.next(p)) {
                const bool fresh = g == 0 || !u.same_tile(tile);
                tile = u;
#pragma unroll 1
                for (int l = 0; l < u.size; ++l, ++g) {
                    const int st = g % ST;
                    if (!catt_wait(&kf[st], (g / ST) & 1, abort_flag, lim)) goto mma_out;
                    const uint32_t sb = g % C::SBUF, use = g / C::SBUF;
                    if (l == 0 && fresh && !catt_wait(&b[9], nq & 1, abort_flag, lim)) goto mma_out;
                    if (use > 0 && !catt_wait(&b[2 + sb], (use - 1) & 1, abort_flag, lim)) goto mma_out;
                    tc_fence_after();
                    const uint32_t qa = smem_u32(smem + C::OFF_Q), ka = smem_u32(smem + C::OFF_K + st * C::TILE);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        tc_mma_f8(tmem + C::S_COL + sb * C::NC, smem_desc_flat(ka + k * 256, 128, D * 8),
                                  smem_desc_flat(qa + k * 256, 128, D * 8), id_s, k ? 1u : 0u);
                    tc_commit(&b[0 + sb]);
                    if (l == 0 && fresh) ++nq;
                    tc_commit(&ke[st]);
                    if (g > 0 && !values(g - 1)) goto mma_out;
                }
            }
            if (g > 0) values(g - 1);
        mma_out:
            tc_commit(done);  // every MMA retires before TMEM is released
            catt_drain(done, 0, lim);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- scores, weights, summaries
        const int qd = warp & 3, tid = qd * 32 + lane;  // tid: TMEM lane = key = dim
        float* x = reinterpret_cast<float*>(smem + C::OFF_X);
        float* xw = x + C::X_WARP + qd * C::X_PER_WARP;   // this warp's own
        float *fac = xw, *ofac = xw + R;                 // [R] factors of a step
        float *rmax = xw + 2 * R, *rval = xw + 3 * R;   // [R] a row's -m c, and 256 / its largest value scale
        float2* pend = reinterpret_cast<float2*>(xw + 4 * R);  // [PENDING][R] (m, s)
        const uint32_t tm = tmem + ((uint32_t)(qd * 32) << 16);
        uint8_t* qs = smem + C::OFF_Q;
        uint8_t* ps = smem + C::OFF_P;
        float* overflow = reinterpret_cast<float*>(smem + C::OFF_ST) + tid;  // [PENDING - TPEND][R][128]
        const bool has_dim = tid < D;
        const int bar = 1;
        bool ab = false;

        // Queries of a unit's rows as two e4m3 terms each, and their constants c.
        auto load_q = [&](const CattUnits<R>& un, uint32_t nq) {
            constexpr int TPR = D / 8, RPP = 128 / TPR;  // threads per row, rows per pass
            float* cst = x + C::X_CST + (nq & 1) * R;
            const int part = tid % TPR;
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += RPP) {
                const int r = r0 + tid / TPR;
                const int fr = un.tau * R + r;
                const bool live = r < R && fr < un.it.rows;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (live) {
                    const int t = catt_div(p, fr), hd = un.h * p.group + fr - t * p.group;
                    w = *reinterpret_cast<const uint4*>(p.q + ((size_t)(un.it.tok0 + t) * p.heads + hd) * D + part * 8);
                }
                const uint32_t a[4] = {w.x, w.y, w.z, w.w};
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(a[k] & 0x7fffu, (a[k] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                // exponents below -119 would take the scale out of range; such a row's scores are zero anyway
                const int e = max((int)(top >> 7) - 127, -119);
                const float sc = cache_pow2(7 - e);
                float f[8];
                unpack8(w, f);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float y0 = __fmul_rn(f[2 * k], sc), y1 = __fmul_rn(f[2 * k + 1], sc);
                    hi[k] = pack_e4m3(y0, y1);
                    const float2 z = unpack_e4m3(hi[k]);
                    lo[k] = pack_e4m3(__fmul_rn(__fsub_rn(y0, z.x), 32.0f), __fmul_rn(__fsub_rn(y1, z.y), 32.0f));
                    if (top >= 0x7f80u) hi[k] = 0x7f7fu;  // not finite: the row's result is NaN
                }
                if (r < R) {
                    const int at = (r & 7) * 16 + (part >> 1) * 128 + (part & 1) * 8;
                    *reinterpret_cast<uint2*>(qs + (r >> 3) * (D * 8) + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                    *reinterpret_cast<uint2*>(qs + ((R + r) >> 3) * (D * 8) + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                    if (part == 0) cst[r] = top >= 0x7f80u ? 1.0f : __fmul_rn(cache_pow2(e - 7), p.scale);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b[9]);
        };
        // The page of this thread's key in leaf l of a unit: what the table holds, if some row of the tile sees the key.
        auto key_page = [&](const CattUnits<R>& un, int imax, int l) -> int {
            const int pos = (un.lo + l) * CATT_LEAF + tid;
            return pos <= imax ? p.table[(size_t)un.it.slot * p.max_pages + (pos >> p.page_shift)] : -1;
        };
        auto key_scales = [&](int h, int id, float& k, float& v) {
            k = v = 0.0f;
            if (id >= 0 && id < p.num_pages) {
                const float* at = p.scales + (size_t)id * p.kv_heads + h;
                k = at[0];
                v = at[(size_t)p.num_pages * p.kv_heads];
            }
        };
        // Lane k: how many nodes leaf k closes (low half), and leaf k + 32 (high half).
        auto pop_codes = [&](int size) { return catt_pops(size, min(lane, size - 1)) | catt_pops(size, min(lane + 32, size - 1)) << 16; };

        uint32_t g = 0, nq = 0;  // leaves, tiles of queries
        float prev_m = 0.0f, prev_o = 0.0f;  // lane = row: its maximum and the scale of its O
        int depth = 0;
        float cks = 0.0f, cvs = 0.0f;
        int cid = -1, imax = 0, codes = 0;
        if (any) {
            imax = u.imax(p);
            cid = key_page(u, imax, 0);
            load_q(u, 0);
            key_scales(u.h, cid, cks, cvs);
            codes = pop_codes(u.size);
        }

        // The summary of leaf l of the unit (the CTA's leaf g1) enters the tree.
        auto tree_step = [&](uint32_t g1, int l) {
            const uint32_t ob = g1 % C::OBUF;
            float* sums = x + C::X_SUM + (g1 & 1) * 4 * R;
            const int row = lane % R;
            float m = prev_m;
            float s = __fadd_rn(__fadd_rn(sums[row], sums[R + row]), __fadd_rn(sums[2 * R + row], sums[3 * R + row]));
            const int code = __shfl_sync(0xffffffffu, codes, l & 31);
            int pops = l < 32 ? code & 0xffff : code >> 16;
            const bool last = l + 1 == u.size;
            if (l == 0) depth = C::PENDING - (32 - __clz(max(u.size - 1, 0)));  // small trees stay in TMEM
            // O is in units of prev_o, a power of two: the first step multiplies it in
            float scale_o = prev_o;
            float o[R];
            if (has_dim) {
                uint32_t raw[C::NC];
                catt_ld<C::NC>(tm + C::O_COL + ob * C::NC, raw);
#pragma unroll
                for (int r = 0; r < R; r += 2)
                    upk2(add2(pk2(__uint_as_float(raw[r]), __uint_as_float(raw[r + 1])),
                              pk2(__uint_as_float(raw[R + r]), __uint_as_float(raw[R + r + 1]))), o[r], o[r + 1]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b[6 + ob]);
            if (pops == 0) {
                if (lane < R) ofac[lane] = scale_o;
                __syncwarp();
                if (has_dim)
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(ofac + r);
                        upk2(mul2(pk2(o[r], o[r + 1]), pk2(f.x, f.y)), o[r], o[r + 1]);
                        upk2(mul2(pk2(o[r + 2], o[r + 3]), pk2(f.z, f.w)), o[r + 2], o[r + 3]);
                    }
            }
#pragma unroll 1
            for (; pops > 0; --pops) {
                --depth;
                const float2 a = pend[depth * R + row];
                float M, ea, eb;
                catt_factors(a.x, m, M, ea, eb);
                s = __fmaf_rn(s, eb, __fmul_rn(a.y, ea));
                m = M;
                if (lane < R) {
                    fac[lane] = ea;
                    ofac[lane] = __fmul_rn(eb, scale_o);
                }
                scale_o = 1.0f;
                __syncwarp();
                if (has_dim) {
                    uint32_t raw[R];
                    if (C::TPEND < C::PENDING && depth < C::PENDING - C::TPEND) {
#pragma unroll
                        for (int r = 0; r < R; ++r) raw[r] = __float_as_uint(overflow[(depth * R + r) * 128]);
                    } else {
                        catt_ld<R>(tm + C::ST_COL + (depth - (C::PENDING - C::TPEND)) * R, raw);
                    }
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 fa = *reinterpret_cast<const float4*>(fac + r), fb = *reinterpret_cast<const float4*>(ofac + r);
                        upk2(fma2(pk2(o[r], o[r + 1]), pk2(fb.x, fb.y),
                                  mul2(pk2(__uint_as_float(raw[r]), __uint_as_float(raw[r + 1])), pk2(fa.x, fa.y))),
                             o[r], o[r + 1]);
                        upk2(fma2(pk2(o[r + 2], o[r + 3]), pk2(fb.z, fb.w),
                                  mul2(pk2(__uint_as_float(raw[r + 2]), __uint_as_float(raw[r + 3])), pk2(fa.z, fa.w))),
                             o[r + 2], o[r + 3]);
                    }
                }
                __syncwarp();
            }
            if (!last) {
                if (lane < R) pend[depth * R + lane] = make_float2(m, s);
                if (has_dim) {
                    if (C::TPEND < C::PENDING && depth < C::PENDING - C::TPEND) {
#pragma unroll
                        for (int r = 0; r < R; ++r) overflow[(depth * R + r) * 128] = o[r];
                    } else {
                        catt_st<R>(tm + C::ST_COL + (depth - (C::PENDING - C::TPEND)) * R, o);
                    }
                }
                ++depth;
                __syncwarp();
                return;
            }
            const int fr0 = u.tau * R, live = min(R, u.it.rows - fr0);
            if (u.d == 0) {
                if (lane < R) ofac[lane] = __frcp_rn(s);
                __syncwarp();
                if (has_dim) {
                    int t = catt_div(p, fr0), hd = fr0 - t * p.group;
                    uint16_t* op = p.out + ((size_t)(u.it.tok0 + t) * p.heads + u.h * p.group) * D + tid;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (r < live) op[hd * D] = f2bf(__fmul_rn(o[r], ofac[r]));
                        if (++hd == p.group) {
                            hd = 0;
                            op += (size_t)p.heads * D;
                        }
                    }
                }
            } else {
                const int slot = u.slot();
                if ((unsigned)slot >= (unsigned)p.max_slots) {
                    set_error(TBIK_ERR_WORKSPACE);
                } else {
                    if (qd == 0 && lane < R) p.ms[(size_t)slot * R + lane] = make_float2(m, s);
                    if (has_dim) {
                        float* op = p.o + ((size_t)slot * R) * D + tid;
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (r < live) op[r * D] = o[r];
                    }
                    if (u.v == 0 && tid == 0) {
                        int4* t = p.tiles + 2 * (size_t)(u.tile_base + u.h * u.tiles + u.tau);
                        t[0] = make_int4(slot, u.d, u.it.L, min(R, u.it.rows - u.tau * R));
                        t[1] = make_int4(u.it.tok0, u.tau * R, u.h, 0);
                    }
                }
            }
            __syncwarp();
        };

#pragma unroll 1
        for (bool more = any; more;) {
            CattUnits<R> nxt = u;
            const bool has_next = nxt.next(p);
            const int fr0 = u.tau * R, i0 = u.it.i0 & 127;
            const int nmax = has_next ? nxt.imax(p) : 0;
            const int row_i = (i0 + catt_div(p, fr0 + lane % R)) & 127;  // lane = row: its position in the block
            const float* cst = x + C::X_CST + (nq & 1) * R;
            const bool fresh = has_next && !nxt.same_tile(u);  // other queries come next
#pragma unroll 1
            for (int l = 0; l <= u.size; ++l) {
                int nid = -1;  // the next leaf's key, its scales, and lane = row: this leaf's maximum and scale of O
                float nks = 0.0f, nvs = 0.0f, nm = 0.0f, no = 0.0f;
                if (l == u.size) {  // nothing but the last leaf's O is left
                    if (named_barrier_or(bar, 128, ab)) goto epi_out;
                    ab = !catt_wait(&b[4 + (g - 1) % C::OBUF], ((g - 1) / C::OBUF) & 1, abort_flag, lim);
                    ab = __any_sync(0xffffffffu, ab);
                } else {
                    const bool last = l + 1 == u.size;
                    const uint32_t sb = g % C::SBUF;
                    float a[R];
                    float* mx = x + C::X_MAX + (g & 1) * 4 * R;
                    float* pv = x + C::X_PV + (g & 1) * 8;
                    const bool diag = u.lo + l == u.it.L - 1;
                    if (!last) nid = key_page(u, imax, l + 1);
                    else if (has_next) nid = key_page(nxt, nmax, 0);
                    if (!ab) ab = !catt_wait(&b[0 + sb], (g / C::SBUF) & 1, abort_flag, lim);
                    ab = __any_sync(0xffffffffu, ab);
                    const bool seen = (u.lo + l) * CATT_LEAF + tid <= imax, no_page = seen && (cid < 0 || cid >= p.num_pages);
                    if (!ab) {
                        tc_fence_after();
                        uint32_t raw[C::NC];
                        catt_ld<C::NC>(tm + C::S_COL + sb * C::NC, raw);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b[2 + sb]);
                        const f2x k2 = pk2(cks, cks), i32 = pk2(0.03125f, 0.03125f);
#pragma unroll
                        for (int r = 0; r < R; r += 2)
                            upk2(mul2(fma2(pk2(__uint_as_float(raw[R + r]), __uint_as_float(raw[R + r + 1])), i32,
                                           pk2(__uint_as_float(raw[r]), __uint_as_float(raw[r + 1]))), k2), a[r], a[r + 1]);
                        if (__any_sync(0xffffffffu, no_page)) {
                            if (no_page) {
#pragma unroll
                                for (int r = 0; r < R; ++r) a[r] = __uint_as_float(0x7fc00000u);
                                set_error(TBIK_ERR_PAGE);
                            }
                        }
                        if (diag) {
                            // row r is at block position i0 + (fr0 + r) / group and does not see this key if that is less
                            // than tid, that is, if fr0 + r < (tid - i0) * group
                            const int hidden = (tid - i0) * p.group - fr0;
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                if (r < hidden) a[r] = -INFINITY;
                        }
#pragma unroll
                        for (int r = 0; r < R; r += 4) {
                            float4 m4;
                            m4.x = warp_max_f32(a[r]);
                            m4.y = warp_max_f32(a[r + 1]);
                            m4.z = warp_max_f32(a[r + 2]);
                            m4.w = warp_max_f32(a[r + 3]);
                            if (lane == 0) *reinterpret_cast<float4*>(mx + qd * R + r) = m4;
                        }
                        if ((tid & (p.page - 1)) == 0) pv[tid >> p.page_shift] = cvs;
                    }
                    if (named_barrier_or(bar, 128, ab)) goto epi_out;
                    // scales of the next leaf's key
                    key_scales(last ? nxt.h : u.h, nid, nks, nvs);
                    if (last && fresh) load_q(nxt, nq + 1);
                    // lane = row: its maximum, and the largest value scale among its visible pages of the leaf
                    {
                        const int row = lane % R, i = diag ? row_i : 127;
                        const float4 v0 = *reinterpret_cast<const float4*>(pv), v1 = *reinterpret_cast<const float4*>(pv + 4);
                        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                        float vm = v[0];
#pragma unroll
                        for (int k = 1; k < 8; ++k)
                            if (k << p.page_shift <= i) vm = fmaxf(vm, v[k]);
                        nm = __fmul_rn(fmaxf(fmax3(mx[row], mx[R + row], mx[2 * R + row]), mx[3 * R + row]), cst[row]);
                        no = __fmul_rn(vm, 0.00390625f);
                        // 256 / vm: scales are powers of two
                        const float iv = __fmul_rn(256.0f, __uint_as_float((254u << 23) - __float_as_uint(vm)));
                        if (lane < R) {
                            rmax[lane] = -nm;
                            rval[lane] = iv;
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 c4 = *reinterpret_cast<const float4*>(cst + r), m4 = *reinterpret_cast<const float4*>(rmax + r);
                        float y[4];
                        upk2(fma2(pk2(a[r], a[r + 1]), pk2(c4.x, c4.y), pk2(m4.x, m4.y)), y[0], y[1]);
                        upk2(fma2(pk2(a[r + 2], a[r + 3]), pk2(c4.z, c4.w), pk2(m4.z, m4.w)), y[2], y[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[r + k] = ex2_hw(y[k]);
                    }
                    float w[R];  // 256 f p
                    if (!diag) {
                        const float f = __fmul_rn(cvs, rval[0]);
                        const f2x f2 = pk2(f, f);
#pragma unroll
                        for (int r = 0; r < R; r += 2) upk2(mul2(pk2(a[r], a[r + 1]), f2), w[r], w[r + 1]);
                    } else {
                        // f <= 1 for a key that the row sees; for others p is 0
#pragma unroll
                        for (int r = 0; r < R; ++r) w[r] = __fmul_rn(a[r], fminf(__fmul_rn(cvs, rval[r]), 256.0f));
                    }
                    // P of the previous leaf is read until its O is there
                    if (l > 0 && !ab) {
                        const uint32_t g1 = g - 1;
                        ab = !catt_wait(&b[4 + g1 % C::OBUF], (g1 / C::OBUF) & 1, abort_flag, lim);
                        ab = __any_sync(0xffffffffu, ab);
                    }
                    if (!ab) {
                        uint32_t hi[R / 4], lo[R / 4];
#pragma unroll
                        for (int r = 0; r < R; r += 4) {
                            const uint32_t h0 = pack_e4m3(w[r], w[r + 1]), h1 = pack_e4m3(w[r + 2], w[r + 3]);
                            const float2 z0 = unpack_e4m3(h0), z1 = unpack_e4m3(h1);
                            hi[r / 4] = h0 | h1 << 16;
                            lo[r / 4] = pack_e4m3(__fsub_rn(w[r], z0.x), __fsub_rn(w[r + 1], z0.y)) |
                                        pack_e4m3(__fsub_rn(w[r + 2], z1.x), __fsub_rn(w[r + 3], z1.y)) << 16;
                        }
                        uint8_t* dst = ps + (tid >> 3) * (8 * C::NC) + (tid & 7) * 16;  // 16 bytes per key and 16 columns
                        if constexpr (R == 8) {
                            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                        } else {
#pragma unroll
                            for (int k = 0; k < R / 16; ++k) {
                                *reinterpret_cast<uint4*>(dst + k * 128) = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                                *reinterpret_cast<uint4*>(dst + (R / 16 + k) * 128) = make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                            }
                        }
                    }
                    if (diag) {
                        // values that no row sees must be finite (0 x NaN): zero behind the tile's last key, and NaN bytes
                        // between its first row's key and that
                        const int st = g % ST;
                        if (!ab) ab = !catt_wait(&vf[st], (g / ST) & 1, abort_flag, lim);
                        ab = __any_sync(0xffffffffu, ab);
                        if (!ab) {
                            if (tid > (u.imin(p) & 127)) {
                                uint8_t* vt = smem + C::OFF_V + st * C::TILE + (tid >> 3) * (D * 8) + (tid & 7) * 16;
                                for (int k = 0; k < D / 16; ++k) {
                                    uint4* at = reinterpret_cast<uint4*>(vt + k * 128);
                                    if (!seen || no_page) {
                                        *at = make_uint4(0, 0, 0, 0);
                                    } else {
                                        const uint4 y = *at;
                                        const uint32_t z[4] = {y.x, y.y, y.z, y.w};
                                        uint32_t o[4];
#pragma unroll
                                        for (int e = 0; e < 4; ++e) o[e] = z[e] & ~__vcmpeq4(z[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                        *at = make_uint4(o[0], o[1], o[2], o[3]);
                                    }
                                }
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && !ab && !(p.debug & TBIK_DEBUG_WITHHOLD_ACC_ARRIVE)) mbar_arrive(&b[8]);
                    // sums over the warp's 32 keys: halves 16, 8, 4, 2, 1 apart; the rows are dealt out on the way
                    {
                        int n = R;
#pragma unroll
                        for (int o = 16; o; o >>= 1) {
                            if (n > 1) {
                                n >>= 1;
#pragma unroll
                                for (int k = 0; k < R / 2; ++k)
                                    if (k < n) {
                                        const float keep = (lane & o) ? a[k + n] : a[k], send = (lane & o) ? a[k] : a[k + n];
                                        a[k] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, o));
                                    }
                            } else {
                                a[0] = __fadd_rn(a[0], __shfl_xor_sync(0xffffffffu, a[0], o));
                            }
                        }
                        if (lane % (32 / R) == 0) x[C::X_SUM + (g & 1) * 4 * R + qd * R + lane / (32 / R)] = a[0];
                    }
                }
                if (l > 0 && !ab) {
                    tc_fence_after();
                    tree_step(g - 1, l - 1);
                }
                if (l == u.size) break;
                ++g;
                prev_m = nm;
                prev_o = no;
                cid = nid;
                cks = nks;
                cvs = nvs;
            }
            u = nxt;
            nq += fresh;
            more = has_next;
            imax = nmax;
            if (more) codes = pop_codes(u.size);
        }
    epi_out:;
    }
    if (marks) catt_mark<D>(p);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

// ------------------------------------------------------------------ the tree above the units
//
// A group of D / 4 threads per row, four dims each.  Trees that are cut a few levels deep are one group's work; for deeper
// ones (few rows over long contexts) the groups of a block take one subtree each.  Several nodes are in flight at a time.
// Empty nodes are passed over.

constexpr int CATT_JOIN_THREADS = 256;

struct CattSum {
    float m, s;
    float4 o;
    bool any;
};
__device__ __forceinline__ CattSum catt_join(const CattSum& a, const CattSum& b) {
    if (!b.any) return a;
    if (!a.any) return b;
    CattSum r;
    float ea, eb;
    catt_factors(a.m, b.m, r.m, ea, eb);
    r.s = __fmaf_rn(b.s, eb, __fmul_rn(a.s, ea));
    r.o.x = __fmaf_rn(b.o.x, eb, __fmul_rn(a.o.x, ea));
    r.o.y = __fmaf_rn(b.o.y, eb, __fmul_rn(a.o.y, ea));
    r.o.z = __fmaf_rn(b.o.z, eb, __fmul_rn(a.o.z, ea));
    r.o.w = __fmaf_rn(b.o.w, eb, __fmul_rn(a.o.w, ea));
    r.any = true;
    return r;
}
__device__ __forceinline__ CattSum catt_node_sum(const CacheAttParams& p, size_t at, int D, int part) {
    CattSum x;
    const float2 ms = p.ms[at];
    x.m = ms.x;
    x.s = ms.y;
    x.o = *reinterpret_cast<const float4*>(p.o + at * D + part * 4);
    x.any = true;
    return x;
}

// The tree over nodes v0 .. v0 + n - 1 of a tile's 2^d, n a power of two, STEP nodes at a time (n a multiple of it);
// PEND: log2(n / STEP) at most.
template <int D, int R, int STEP, int PEND>
__device__ __forceinline__ CattSum catt_join_nodes(const CacheAttParams& p, int slot, int L, int d, int v0, int n, int row, int part) {
    CattSum st[PEND + 1], r;
    r.any = false;
    int depth = 0;
#pragma unroll 1
    for (int v = 0; v < n; v += STEP) {
        CattSum x[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            x[k].any = false;
            if (catt_node_size(L, d, v0 + v + k)) x[k] = catt_node_sum(p, (size_t)(slot + v0 + v + k) * R + row, D, part);
        }
#pragma unroll
        for (int h = 1; h < STEP; h <<= 1)
#pragma unroll
            for (int k = 0; k + h < STEP; k += 2 * h) x[k] = catt_join(x[k], x[k + h]);
        r = x[0];
        for (int c = v / STEP; c & 1; c >>= 1) r = catt_join(st[--depth], r);
        if (v + STEP < n) st[depth++] = r;
    }
    return r;
}

template <int D, int R>
__global__ void __launch_bounds__(CATT_JOIN_THREADS) cache_attention_join_kernel(const __grid_constant__ CacheAttParams p) {
    constexpr int LANES = D / 4, GROUPS = CATT_JOIN_THREADS / LANES;
    static_assert((2 << CATT_JOIN_DEPTH) >= 2 * GROUPS, "deeper trees have two nodes for every group");
    __shared__ CattSum sums[GROUPS][LANES];
    const int part = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = p.count[0], deep = p.count[1];
    // A call that gave up (an expired wait) has left descriptors unwritten: whatever they hold, nothing outside the
    // workspace and the output is touched.
    auto sound = [&](const int4& t0, const int4& t1) {
        return t0.x >= 0 && t0.y > 0 && t0.y < 20 && t0.z > 0 && t0.w > 0 && t0.w <= R && (long long)t0.x + (1 << t0.y) <= p.max_slots &&
               t1.x >= 0 && t1.y >= 0 && t1.y <= CATT_LEAF * p.group - t0.w && t1.z >= 0 && t1.z < p.kv_heads &&
               t1.x <= p.tokens - 1 - catt_div(p, t1.y + t0.w - 1);
    };
    auto put = [&](const int4& t1, int row, const CattSum& x) {
        const int fr = t1.y + row, t = catt_div(p, fr), hd = t1.z * p.group + fr - t * p.group;
        const float is = __frcp_rn(x.s);
        uint2 y;
        y.x = pack_bf2(__fmul_rn(x.o.x, is), __fmul_rn(x.o.y, is));
        y.y = pack_bf2(__fmul_rn(x.o.z, is), __fmul_rn(x.o.w, is));
        *reinterpret_cast<uint2*>(p.out + ((size_t)(t1.x + t) * p.heads + hd) * D + part * 4) = y;
    };
#pragma unroll 1
    for (long long w = (long long)blockIdx.x * GROUPS + grp; w < (long long)count * R; w += (long long)gridDim.x * GROUPS) {
        const int4 t0 = p.tiles[2 * (w / R)], t1 = p.tiles[2 * (w / R) + 1];  // slot, d, L, rows; token, first row, kv head
        const int row = (int)(w % R);
        if (!sound(t0, t1) || row >= t0.w || t0.y > CATT_JOIN_DEPTH) continue;
        if (t0.y == 1)
            put(t1, row, catt_join_nodes<D, R, 2, 0>(p, t0.x, t0.z, 1, 0, 2, row, part));
        else if (t0.y == 2)
            put(t1, row, catt_join_nodes<D, R, 4, 0>(p, t0.x, t0.z, 2, 0, 4, row, part));
        else
            put(t1, row, catt_join_nodes<D, R, 8, CATT_JOIN_DEPTH - 3>(p, t0.x, t0.z, t0.y, 0, 1 << t0.y, row, part));
    }
    if (!deep) return;
#pragma unroll 1
    for (long long w = blockIdx.x; w < (long long)count * R; w += gridDim.x) {
        const int4 t0 = p.tiles[2 * (w / R)], t1 = p.tiles[2 * (w / R) + 1];
        const int row = (int)(w % R);
        if (!sound(t0, t1) || row >= t0.w || t0.y <= CATT_JOIN_DEPTH) continue;  // the same for the whole block
        // as many nodes for each group: 4 (8 groups) or 2 (16 groups) at least
        constexpr int LEAST = (2 << CATT_JOIN_DEPTH) / GROUPS;
        const int per = (1 << t0.y) / GROUPS;
        const CattSum r = catt_join_nodes<D, R, LEAST, 14>(p, t0.x, t0.z, t0.y, grp * per, per, row, part);
        __syncthreads();
        sums[grp][part] = r;
        __syncthreads();
        if (grp == 0) {
            CattSum x[GROUPS];
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) x[k] = sums[k][part];
#pragma unroll
            for (int h = 1; h < GROUPS; h <<= 1)
#pragma unroll
                for (int k = 0; k + h < GROUPS; k += 2 * h) x[k] = catt_join(x[k], x[k + h]);
            put(t1, row, x[0]);
        }
    }
}

}  // namespace tbik

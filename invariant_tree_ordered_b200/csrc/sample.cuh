// Sampling the next token from a row of logits (tbik_sample).
//
//   w_i = exp((z_i - max z) / temperature), held as the integer q_i = rint(2^32 w_i);
//   top-k keeps the k largest logits, then top-p the shortest prefix (by descending logit, lower index first among
//   equal ones) of what is left whose mass reaches p of its mass, then min-p the tokens with w_i >= min_p;
//   the token is the first, by index, at which the running sum of the kept q exceeds floor(u * their total).
//
// Sums of integers do not depend on their order, so a row's token depends on that row alone: not on the batch, not on
// the cluster size, and atomics may be used freely.  A weight below 2^-33 of the largest counts as zero; rounding to
// nearest at 2^-32 moves a border between tokens by about 2^-32 sqrt(V) of the largest weight.
//
// Layout: a cluster of 1..8 blocks holds one row in its shared memory (one read of HBM), every later step runs there.
// What bounds it are the instructions per token, so the common case takes two sweeps over shared memory:
//   1. a histogram of counts over linear bins of (max - z) / temperature, 32 to a unit (one shared atomic per token);
//      with top-k the bin of the k-th token is exact, and the tokens up to it (a few more than k) are sorted in one block,
//      where the rest is decided too;
//   2. with top-p alone, counts times the bins' middle weights estimate the mass up to a bin to a few 0.1 %, which gives
//      a bracket of bins around the limit; the second sweep forms the exact sums: the row's mass, the kept mass above the
//      bracket (per chunk of tokens, for the choice), and a histogram of the tokens inside, whose border bin is sorted.
//      The estimate only chooses the bracket; whether the limit lies inside is checked with the exact sums.
// A row that does not fit (the limit outside the bracket, too many tokens in a list, infinite logits, temperatures near
// 0) takes the general steps: histograms of masses, the border bin split again on the bits of the logits until it
// fits or all its logits are equal.
//
// Measured: 256 rows of 151936 fp32 logits, every row with its own settings, 165 us (an HBM read takes 24 us; two blocks fit
// an SM, and issue slots are 40 % used: of the 17 cycles between a warp's instructions 5 go to block barriers, which wait
// for the cluster's too, 3 to loads and 2 to shared memory); one row 19 to 31 us; 97 rows of 32000 in bf16 29 to 34 us.  A row
// read again from memory by one block for each sweep, without meetings, measured 172 us for the first and is not kept.
// The general steps: top-p 0.95 at temperature 100 takes 97 us for one row of 151936 and 0.95 ms for 256, over equal logits
// 72 us and 0.80 ms, top-k 5000 45 us and 0.50 ms (60 us and 0.64 ms with top-p); 97 rows of 32000 in bf16 47 to 100 us.
// With top-p 0.95 in every row the two sweeps take 28 us for one row and 0.29 ms for 256.
#pragma once

#include "device_common.cuh"

namespace tbik {

constexpr int SMP_THREADS = 512;
constexpr int SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_BINS = 1024;
constexpr int SMP_CAND = 1024;         // tokens that one block sorts
constexpr int SMP_CHUNK_ROUNDS = 8;    // rounds of SMP_THREADS tokens per partial sum
constexpr int SMP_CHUNK = SMP_THREADS * SMP_CHUNK_ROUNDS;
constexpr int SMP_MAX_SEG = 12 * SMP_CHUNK;  // tokens per block
constexpr int SMP_MAX_CLUSTER = 8;
constexpr int SMP_BINS2 = 256;         // of the second histogram
constexpr int SMP_BORDER = 128;        // tokens of its border bin, from each block
constexpr int SMP_LIST = 2048;         // tokens of a top-k set that one block sorts; tokens of a bracket per block
constexpr int SMP_SWEEP = 16;          // tokens per thread and chunk of the second sweep
constexpr int SMP_SWEEP_CHUNKS = (SMP_MAX_SEG + 16) / (SMP_THREADS * SMP_SWEEP) + 1;

struct SampleParams {
    const void* logits;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* out;
    int batch, vocab, seg;  // seg: tokens per block, a multiple of 16
};

struct SampleShared {
    union {
        unsigned long long csum[SMP_MAX_SEG / SMP_CHUNK][SMP_WARPS];  // kept mass of each chunk
        unsigned long long sweep[SMP_SWEEP_CHUNKS][SMP_WARPS];        // and in the two-sweep form
    };
    union {
        unsigned long long wsum[SMP_CHUNK_ROUNDS][SMP_WARPS];  // of the chosen chunk, when the lists are done with
        unsigned long long cand[SMP_LIST];  // key << 32 | ~index: descending order is the order of the tokens
        struct {
            unsigned long long border_list[SMP_MAX_CLUSTER][SMP_BORDER];
            uint32_t loc[SMP_LIST];         // this block's tokens in the bracket
        };
    };
    unsigned long long extra[SMP_SWEEP_CHUNKS];             // and of its tokens in the bracket
    // what each block of the cluster has pushed to this one
    struct {
        unsigned long long total, above, in, kept;
        float max;
        uint32_t nan, first, lists, border;
    } from[SMP_MAX_CLUSTER];
    unsigned long long part[3][SMP_WARPS];
    uint32_t n_loc;
    float wbound;
    unsigned long long scan[SMP_WARPS + 1];
    unsigned long long total;           // this block's kept mass (read by the others)
    unsigned long long mass;            // mass up to and with the last kept token
    unsigned long long base_mass;
    alignas(16) uint32_t cnt[SMP_BINS];
    alignas(16) uint32_t mhi[SMP_BINS];
    uint32_t mlo[SMP_BINS];  // directly behind mhi
    uint32_t wmin[SMP_WARPS], wmax[SMP_WARPS];
    uint32_t kmin, kmax;
    uint32_t n_cand;
    uint32_t lkey, lidx;  // the last kept token
    int border, base_cnt, border_cnt;
    int token;
};

// Order-preserving key of a float (larger float, larger key; -0 below +0 is undone by the + 0.0f of the loads).
__device__ __forceinline__ uint32_t smp_key(float z) {
    const uint32_t b = __float_as_uint(z);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t atom_add_cluster_u32(uint32_t addr, uint32_t x) {
    uint32_t v;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(addr), "r"(x) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(x) : "memory");
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Modulo 2^64, by three reductions of 32-bit integers: 22, 21 and 21 bits, 32 of which stay below 2^32.
__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x3fffffu);
    const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 22) & 0x1fffffu);
    const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 43));
    return a + ((unsigned long long)b << 22) + ((unsigned long long)c << 43);
}

template <typename T>
__device__ __forceinline__ float smp_load(const T* s, int i);
template <>
__device__ __forceinline__ float smp_load<float>(const float* s, int i) { return s[i] + 0.0f; }
template <>
__device__ __forceinline__ float smp_load<uint16_t>(const uint16_t* s, int i) { return bf2f(s[i]) + 0.0f; }

template <typename T>
__device__ __forceinline__ T smp_minus_inf();
template <>
__device__ __forceinline__ float smp_minus_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ uint16_t smp_minus_inf<uint16_t>() { return 0xff80; }

// The values of a 16-byte piece.
template <typename T>
struct SmpPiece;
template <>
struct SmpPiece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& w, float (&z)[4]) {
        z[0] = __uint_as_float(w.x), z[1] = __uint_as_float(w.y), z[2] = __uint_as_float(w.z), z[3] = __uint_as_float(w.w);
    }
};
template <>
struct SmpPiece<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& w, float (&z)[8]) { unpack8(w, z); }
};

// What is kept, and with which weight.
struct SampleFilter {
    float m, min_w;     // row maximum, min_p
    float c, c_lo, low; // log2(e) / temperature in two parts; differences below `low` have weight 0
    bool greedy;        // only tokens at the maximum
    bool ones;          // weights 1 for tokens of key lkey (counting equal ones)
    uint32_t lkey, lidx;

    // 2^(x c) with the product's rounding and c's carried along: an error of c alone would move all of a row's tail
    // against its head by some 10^-6, a few tokens' worth at the top-p border.
    __device__ __forceinline__ float power(float x) const {
        x = fmaxf(x, low);
        const float a = __fmul_rn(x, c), lo = __fmaf_rn(x, -c_lo, __fmaf_rn(x, -c, a)), e = ex2_hw(a);
        return __fmaf_rn(e, __fmul_rn(lo, -0.693147181f), e);
    }
    // The same for two logits.
    __device__ __forceinline__ void power2(float z0, float z1, float& w0, float& w1) const {
        float x0, x1, a0, a1;
        upk2(add2(pk2(z0, z1), pk2(-m, -m)), x0, x1);
        const f2x x = pk2(fmaxf(x0, low), fmaxf(x1, low)), a = mul2(x, pk2(c, c));
        const f2x lo = fma2(x, pk2(-c_lo, -c_lo), fma2(x, pk2(-c, -c), a));
        upk2(a, a0, a1);
        const f2x e = pk2(ex2_hw(a0), ex2_hw(a1));
        upk2(fma2(e, mul2(lo, pk2(-0.693147181f, -0.693147181f)), e), w0, w1);
    }
    __device__ __forceinline__ float weight(float z) const {
        if (z == m) return 1.0f;
        if (z == -INFINITY || m == INFINITY) return 0.0f;
        return power(__fsub_rn(z, m));
    }
    __device__ __forceinline__ unsigned long long units(float z) const { return __float2ull_rn(__fmul_rn(weight(z), 0x1p32f)); }
    __device__ __forceinline__ unsigned long long kept(float z, uint32_t idx) const {
        const uint32_t key = smp_key(z);
        if (ones) return key == lkey;
        if (greedy) return z == m;
        if (key < lkey || (key == lkey && idx > lidx)) return 0;
        const float w = weight(z);
        if (w < min_w && z != m) return 0;
        return __float2ull_rn(__fmul_rn(w, 0x1p32f));
    }
};

// Sum of the kept units of the row; with `find`, the index at which the running sum (by index) first exceeds `target`
// (-1 if none).  Two barriers of the cluster.  Every block of the cluster gets the same result.
template <typename T, typename Pick>
__device__ __forceinline__ unsigned long long sample_select(const T* s, int len, uint32_t base, const SampleFilter& f, SampleShared& sh,
                                                            uint32_t rank, uint32_t cl, Pick target_of, int& token) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = (len + SMP_CHUNK - 1) / SMP_CHUNK;
    unsigned long long mine = 0;
    for (int c = 0; c < chunks; ++c) {
        unsigned long long a = 0;
#pragma unroll
        for (int r = 0; r < SMP_CHUNK_ROUNDS; ++r) {
            const int i = c * SMP_CHUNK + r * SMP_THREADS + tid;
            if (i < len) a += f.kept(smp_load(s, i), base + i);
        }
        a = warp_sum_u64(a);
        if (lane == 0) sh.csum[c][warp] = a;
        mine += a;
    }
    if (lane == 0) sh.scan[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        unsigned long long t = 0;
        for (int w = 0; w < SMP_WARPS; ++w) t += sh.scan[w];
        sh.total = t;
        sh.token = -1;
    }
    cluster_sync();
    unsigned long long before = 0, all = 0, own = 0;
    for (uint32_t r = 0; r < cl; ++r) {
        const unsigned long long t = ld_cluster_u64(mapa_shared(smem_u32(&sh.total), r));
        if (r < rank) before += t;
        if (r == rank) own = t;
        all += t;
    }
    const unsigned long long target = target_of(all);
    if (all > 0 && target >= before && target - before < own) {  // the same for the whole block
        unsigned long long left = target - before;
        int c = 0;
        for (;; ++c) {
            unsigned long long t = 0;
            for (int w = 0; w < SMP_WARPS; ++w) t += sh.csum[c][w];
            if (left < t) break;
            left -= t;
        }
        unsigned long long a[SMP_CHUNK_ROUNDS];
#pragma unroll
        for (int r = 0; r < SMP_CHUNK_ROUNDS; ++r) {
            const int i = c * SMP_CHUNK + r * SMP_THREADS + tid;
            a[r] = i < len ? f.kept(smp_load(s, i), base + i) : 0;
            const unsigned long long t = warp_sum_u64(a[r]);
            if (lane == 0) sh.wsum[r][warp] = t;
        }
        __syncthreads();
        int rr = 0, ww = 0;
        for (;;) {
            const unsigned long long t = sh.wsum[rr][ww];
            if (left < t) break;
            left -= t;
            if (++ww == SMP_WARPS) {
                ww = 0;
                ++rr;
            }
        }
        if (warp == ww) {
            unsigned long long x = 0;
#pragma unroll
            for (int r = 0; r < SMP_CHUNK_ROUNDS; ++r)
                if (r == rr) x = a[r];
            unsigned long long p = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, p, o);
                if (lane >= o) p += y;
            }
            if (p - x <= left && left < p) sh.token = (int)(base + c * SMP_CHUNK + rr * SMP_THREADS + tid);
        }
    }
    cluster_sync();
    token = -1;
    for (uint32_t r = 0; r < cl; ++r) token = max(token, (int)ld_cluster_u32(mapa_shared(smem_u32(&sh.token), r)));
    cluster_sync();  // everybody has read before anything is written again
    return all;
}

// u * total as (floor, whether something is left over), u in [0, 1], total < 2^63.
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long total, bool& rest) {
    const uint32_t bits = __float_as_uint(u);
    const int shift = (int)(bits >> 23) - 127 + 40;  // U = floor(2^63 u)
    const unsigned long long mant = (bits & 0x7fffffu) | 0x800000u;
    const unsigned long long U = shift >= 0 ? mant << shift : shift > -24 ? mant >> -shift : 0ull;
    rest = ((total << 1) * U) != 0;
    return __umul64hi(total << 1, U);
}

// Sum over lower threads, `all` over the block.  Two barriers.
template <typename V>
__device__ __forceinline__ V sample_before(V v, V* buf, V& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = s;
    __syncthreads();
    V b = 0;
    all = 0;
    for (int w = 0; w < SMP_WARPS; ++w) {
        const V t = buf[w];
        if (w < warp) b += t;
        all += t;
    }
    return b + s - v;
}

__device__ __forceinline__ float smp_unkey(uint32_t key) { return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key); }

// The two-sweep form; false (for the whole cluster) if the row does not fit it.  All blocks of the cluster leave together.
template <typename T>
__device__ bool sample_fast(const SampleParams& p, SampleShared& sh, uint8_t* raw, int row, uint32_t rank, uint32_t cl, int len, int mis,
                            int pieces, SampleFilter f, float scale, bool by_k, bool by_p, int k, float tp) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int PER = SmpPiece<T>::N, BPT = 4, ROUNDS = SMP_SWEEP / PER;
    const uint4* img = reinterpret_cast<const uint4*>(raw);
    const uint32_t at = rank * (uint32_t)p.seg;
    const float m = f.m;

    if (f.greedy) {  // the lowest index of the largest logit
        uint32_t best = 0xffffffffu;
        for (int v = tid; v < pieces; v += SMP_THREADS) {
            float z[PER];
            SmpPiece<T>::get(img[v], z);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (z[e] == m) best = min(best, at + (uint32_t)(v * PER + e - mis));
        }
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0) sh.wmin[warp] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < SMP_WARPS; ++w) best = min(best, sh.wmin[w]);
            st_cluster_u32(mapa_shared(smem_u32(&sh.from[rank].first), 0), best);
        }
        cluster_sync();
        if (rank == 0 && tid == 0) {
            for (uint32_t r = 0; r < cl; ++r) best = min(best, sh.from[r].first);
            p.out[row] = (int)best;
        }
        return true;
    }

    float above = INFINITY, inside = INFINITY;  // in bins: kept for certain below `above`, to be decided below `inside`
    const float u = p.u[row];
    if (by_k || by_p) {
        // ---- first sweep: counts
        for (int v = tid; v < pieces; v += SMP_THREADS) {
            float z[PER];
            SmpPiece<T>::get(img[v], z);
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                // floor by an addition that rounds toward zero
                const float y = fminf(__fmul_rn(__fsub_rn(m, z[e]), scale), (float)(SMP_BINS - 1));
                atomicAdd(&sh.cnt[__float_as_uint(__fadd_rz(y, 0x1p23f)) - 0x4b000000u], 1u);
            }
        }
        cluster_sync();
        uint32_t cnt[BPT] = {0, 0, 0, 0};  // threads behind the last bin have none
        if (tid < SMP_BINS / BPT) {
            const uint32_t a = smem_u32(&sh.cnt[tid * BPT]);
            uint4 t[SMP_MAX_CLUSTER];
#pragma unroll
            for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) t[r] = r < cl ? ld_cluster_v4(mapa_shared(a, r)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) cnt[0] += t[r].x, cnt[1] += t[r].y, cnt[2] += t[r].z, cnt[3] += t[r].w;
        }
        if (by_k) {
            uint32_t here = 0, every;
#pragma unroll
            for (int x = 0; x < BPT; ++x) here += cnt[x];
            uint32_t b = sample_before(here, sh.wmin, every);
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                if (b < (uint32_t)k && (uint32_t)k <= b + cnt[x]) {
                    sh.border = tid * BPT + x;
                    sh.border_cnt = (int)(b + cnt[x]);
                }
                if (tid < SMP_BINS / BPT) sh.mhi[tid * BPT + x] = b;  // the bin's first place
                b += cnt[x];
            }
            __syncthreads();
            const int border = sh.border, most = sh.border_cnt;
            // the last bin has no lower end, and holds what lies outside the segments
            if (border == SMP_BINS - 1 || most > SMP_LIST) {
                cluster_sync();  // everybody has read the counts
                for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = 0;
                cluster_sync();
                return false;
            }
            // ---- the tokens up to that bin go to the first block, each bin's to its place
            const float limit = (float)(border + 1);
            const uint32_t list = mapa_shared(smem_u32(sh.cand), 0), num = mapa_shared(smem_u32(sh.mlo), 0);
            auto bin0 = [&](float z) { return (int)__fmul_rn(__fsub_rn(m, z), scale); };
            for (int v = tid; v < pieces; v += SMP_THREADS) {
                float z[PER];
                SmpPiece<T>::get(img[v], z);
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (__fmul_rn(__fsub_rn(m, z[e]), scale) < limit) {
                        const int bin = bin0(z[e]);
                        const uint32_t slot = sh.mhi[bin] + atom_add_cluster_u32(num + 4 * bin, 1u);
                        const uint32_t idx = at + (uint32_t)(v * PER + e - mis);
                        if (slot < SMP_LIST) st_cluster_u64(list + slot * 8, (unsigned long long)smp_key(z[e] + 0.0f) << 32 | (uint32_t)~idx);
                    }
            }
            cluster_sync();
            if (rank != 0) return true;
            // a token's place: its bin's first, and the larger ones in the bin
            constexpr int Q = SMP_LIST / SMP_THREADS;
            unsigned long long c[Q], q[Q];
            int place[Q];
#pragma unroll
            for (int x = 0; x < Q; ++x) {
                const int i = x * SMP_THREADS + tid;
                place[x] = -1;
                if (i < most) {
                    c[x] = sh.cand[i];
                    const int bin = bin0(smp_unkey((uint32_t)(c[x] >> 32)));
                    const int lo = (int)sh.mhi[bin], hi = lo + (int)sh.mlo[bin];
                    place[x] = lo;
                    for (int j = lo; j < hi; ++j) place[x] += sh.cand[j] > c[x];
                }
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < Q; ++x)
                if (place[x] >= 0) sh.cand[place[x]] = c[x];
            for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
            __syncthreads();
            const int n = min(most, k);
            unsigned long long v = 0, all;
#pragma unroll
            for (int x = 0; x < Q; ++x) {
                const int i = tid * Q + x;
                c[x] = q[x] = 0;
                if (i < n) {
                    c[x] = sh.cand[i];
                    q[x] = f.units(smp_unkey((uint32_t)(c[x] >> 32)));
                }
                v += q[x];
            }
            unsigned long long b4 = sample_before(v, sh.scan, all);
            if (by_p) {
                bool rest;
                unsigned long long lim = share_of(tp > 0.0f ? tp : 0.0f, all, rest);
                if (rest) ++lim;
                if (lim < 1) lim = 1;
#pragma unroll
                for (int x = 0; x < Q; ++x) {
                    const unsigned long long e = b4 + q[x];
                    if (b4 >= lim) q[x] = 0;  // mass before it has reached the share
                    b4 = e;
                }
            }
            // what stays, in a histogram of masses over the indices
            int shift = 0;
            while ((p.vocab - 1) >> shift >= SMP_BINS) ++shift;
            v = 0;
#pragma unroll
            for (int x = 0; x < Q; ++x) {
                const float z = smp_unkey((uint32_t)(c[x] >> 32));
                if (q[x] && z != m && f.weight(z) < f.min_w) q[x] = 0;
                if (q[x]) {
                    const int bin = (int)(~(uint32_t)c[x] >> shift);
                    atomicAdd(&sh.mhi[bin], (uint32_t)(q[x] >> 16));
                    atomicAdd(&sh.mlo[bin], (uint32_t)(q[x] & 0xffffu));
                }
            }
            __syncthreads();
            unsigned long long ms[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ms[x] = ((unsigned long long)sh.mhi[tid * 2 + x] << 16) + sh.mlo[tid * 2 + x];
                v += ms[x];
            }
            b4 = sample_before(v, sh.scan, all);
            bool rest;
            unsigned long long target = share_of(u >= 0.0f ? fminf(u, 1.0f) : 0.0f, all, rest);
            if (target >= all) target = all - 1;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (b4 <= target && target < b4 + ms[x]) {
                    sh.border = tid * 2 + x;
                    sh.base_mass = b4;
                }
                b4 += ms[x];
            }
            __syncthreads();
            // its tokens, and the one at which the running sum passes the target
            unsigned long long* units = reinterpret_cast<unsigned long long*>(sh.mhi);  // [SMP_CAND], the bins are read
            unsigned int* fill = &sh.n_loc;
#pragma unroll
            for (int x = 0; x < Q; ++x)
                if (q[x] && (int)(~(uint32_t)c[x] >> shift) == sh.border) {
                    const uint32_t slot = atomicAdd(fill, 1u);  // a bin has at most 2^shift tokens: 512
                    sh.cnt[slot] = ~(uint32_t)c[x];
                    units[slot] = q[x];
                }
            __syncthreads();
            const int few = (int)sh.n_loc;
            for (int i = tid; i < few; i += SMP_THREADS) {
                const uint32_t idx = sh.cnt[i];
                unsigned long long b = sh.base_mass;
                for (int j = 0; j < few; ++j)
                    if (sh.cnt[j] < idx) b += units[j];
                if (b <= target && target < b + units[i]) p.out[row] = (int)idx;
            }
            return true;
        }
        // ---- top-p alone: a bracket of bins around the limit, from counts and the bins' middle weights
        auto mass = [&](int x) { return __fmul_rn((float)cnt[x], ex2_hw(-1.44269504f / 32.0f * ((float)(tid * BPT + x) + 0.5f))); };
        float s1 = 0.0f, s2 = 0.0f, all1, all2;
#pragma unroll
        for (int x = 0; x < BPT; ++x) {
            const float w = mass(x);
            s1 += w;
            if (cnt[x]) s2 += w * w / (float)cnt[x];
        }
        float b = sample_before(s1, reinterpret_cast<float*>(sh.wmin), all1);
        sample_before(s2, reinterpret_cast<float*>(sh.wmax), all2);
        // The limit is where P >= p S.  A token's weight is off by up to 1.6 % of it, evenly spread (0.9 % rms; the margin
        // takes four deviations); above the limit that shifts P and p S together, (1 - p) of it is left, and below it
        // the weights are at most the border's, w: a variance of w times the mass (1 - p) S.  A little more for weights
        // that change across a bin.
        const float share = fminf(fmaxf(tp, 0.0f), 1.0f), want = share * all1;
        if (tid == 0) {
            sh.border = 0;
            sh.border_cnt = SMP_BINS - 1;
            sh.wbound = 1.0f;
        }
        __syncthreads();
        const float b0 = b;
#pragma unroll
        for (int x = 0; x < BPT; ++x) {
            const float e = b + mass(x);
            if (b < want && e >= want) sh.wbound = 1.1f * mass(x) / (float)cnt[x];
            b = e;
        }
        __syncthreads();
        const float w = sh.wbound;
        const float margin = 0.036f * ((1.0f - share) * sqrtf(all2) + share * sqrtf(w * (1.0f - share) * all1)) + 0.0004f * all1;
        b = b0;
#pragma unroll
        for (int x = 0; x < BPT; ++x) {
            const float e = b + mass(x);
            if (b < want - margin && e >= want - margin) sh.border = tid * BPT + x;
            if (b < want + margin && e >= want + margin) sh.border_cnt = tid * BPT + x;
            b = e;
        }
        __syncthreads();
        above = (float)sh.border;
        inside = (float)(sh.border_cnt + 1);
        if (sh.border_cnt >= SMP_BINS - 1) inside = INFINITY;
    }

    // ---- second sweep: the sums
    const float spread = (float)(SMP_BINS2 - 1) / (inside - above);  // bins of the second histogram per bin
    unsigned long long total = 0, sure = 0, in = 0;
    const int chunks = (pieces + SMP_THREADS * ROUNDS - 1) / (SMP_THREADS * ROUNDS);
    const T* simg = reinterpret_cast<const T*>(raw);
    auto bin_of = [&](float z) { return (int)(__fmul_rn(__fsub_rn(__fmul_rn(__fsub_rn(m, z), scale), above), spread)); };
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        // units below 2^23 (weights below about 2^-9): 2^32 w rounds to an integer in the addition of 2^23; 16 of them
        // fit 27 bits, and 32 lanes' 32.  Larger ones (their q is 2^23 or more, if not their units) and those in the
        // bracket (few) are set aside.  The limit is on the rounded units: the largest weight below 2^-9 rounds up to
        // 2^23 of them, and a warp full of it would sum to 2^32.
        uint32_t s_all = 0, s_up = 0, s_kept = 0, large = 0, between = 0;
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int v = (c * ROUNDS + r) * SMP_THREADS + tid;
            if (v < pieces) {
                float z[PER];
                SmpPiece<T>::get(img[v], z);
                float ws[PER];
#pragma unroll
                for (int e = 0; e < PER; e += 2) f.power2(z[e], z[e + 1], ws[e], ws[e + 1]);
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const float w = ws[e], y = __fmul_rn(__fsub_rn(m, z[e]), scale);
                    const uint32_t q = __float_as_uint(__fmaf_rn(w, 0x1p32f, 0x1p23f)) - 0x4b000000u;
                    const bool up = y < above, mid = !up && y < inside && q, big = !mid && q >= 1u << 23;
                    if (mid) between |= 1u << (r * PER + e);
                    if (big) large |= 1u << (r * PER + e);
                    if (!mid && !big) s_all += q;
                    if (up && !big) s_up += q;
                    if (up && !big && w >= f.min_w) s_kept += q;
                }
            }
        }
        auto place = [&](int bit) { return ((c * ROUNDS + bit / PER) * SMP_THREADS + tid) * PER + bit % PER; };
        unsigned long long kept = 0;
        while (large) {
            const int bit = __ffs((int)large) - 1;
            large &= large - 1;
            const float z = smp_load(simg, place(bit)), w = f.weight(z);
            const unsigned long long q = __float2ull_rn(__fmul_rn(w, 0x1p32f));
            total += q;
            if (__fmul_rn(__fsub_rn(m, z), scale) < above) {
                sure += q;
                if (w >= f.min_w || z == m) kept += q;
            }
        }
        if (__any_sync(0xffffffffu, between)) {  // one reservation for the warp
            const uint32_t count = __popc(between);
            uint32_t upto = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            uint32_t first = 0;
            if (lane == 31) first = atomicAdd(&sh.n_loc, upto);
            first = __shfl_sync(0xffffffffu, first, 31) + upto - count;
            while (between) {
                const int bit = __ffs((int)between) - 1;
                between &= between - 1;
                if (first < SMP_LIST) sh.loc[first] = (uint32_t)place(bit);
                ++first;
            }
        }
        // 32 lanes x 16 values of at most 2^23 - 1: below 2^32
        unsigned long long t = __reduce_add_sync(0xffffffffu, s_kept);
        if (__any_sync(0xffffffffu, kept != 0)) t += warp_sum_u64(kept);
        if (lane == 0) sh.sweep[c][warp] = t;
        total += s_all;
        sure += s_up;
    }
    SampleFilter g = f;
    if (by_p) {
        __syncthreads();
        const int mine = min((int)sh.n_loc, SMP_LIST);
        for (int i = tid; i < mine; i += SMP_THREADS) {
            const float z = smp_load(simg, (int)sh.loc[i]);
            const unsigned long long q = f.units(z);
            const int bin = bin_of(z);
            if (q >> 16) atomicAdd(&sh.mhi[bin], (uint32_t)(q >> 16));
            if (q & 0xffffu) atomicAdd(&sh.mlo[bin], (uint32_t)(q & 0xffffu));
            in += q;
        }
        total += in;
        total = warp_sum_u64(total);
        sure = warp_sum_u64(sure);
        in = warp_sum_u64(in);
        if (lane == 0) {
            sh.part[0][warp] = total;
            sh.part[1][warp] = sure;
            sh.part[2][warp] = in;
        }
        __syncthreads();
        if (warp == 0) {
            unsigned long long t[3];
#pragma unroll
            for (int x = 0; x < 3; ++x) t[x] = warp_sum_u64(lane < SMP_WARPS ? sh.part[x][lane] : 0ull);
            if (lane < (int)cl) {
                const uint32_t to = mapa_shared(smem_u32(&sh.from[rank]), lane);
                st_cluster_u64(to, t[0]);
                st_cluster_u64(to + 8, t[1]);
                st_cluster_u64(to + 16, t[2]);
                st_cluster_u32(mapa_shared(smem_u32(&sh.from[rank].lists), lane), sh.n_loc);
            }
        }
        cluster_sync();
        total = sure = in = 0;
        bool fits = true;
#pragma unroll
        for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) {
            const bool there = r < cl;
            total += there ? sh.from[r].total : 0ull;
            sure += there ? sh.from[r].above : 0ull;
            in += there ? sh.from[r].in : 0ull;
            fits &= !there || sh.from[r].lists <= SMP_LIST;
        }
        bool rest;
        unsigned long long limit = share_of(tp > 0.0f ? tp : 0.0f, total, rest);
        if (rest) ++limit;
        if (limit < 1) limit = 1;
        fits &= sure < limit && limit <= sure + in;
        if (fits) {
            unsigned long long ms[BPT] = {0, 0, 0, 0}, all;
            if (tid < SMP_BINS2 / BPT) {
                const uint32_t a1 = smem_u32(&sh.mhi[tid * BPT]), a2 = smem_u32(&sh.mlo[tid * BPT]);
                uint4 t[SMP_MAX_CLUSTER];
                auto pull = [&](uint32_t a) {
#pragma unroll
                    for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) t[r] = r < cl ? ld_cluster_v4(mapa_shared(a, r)) : make_uint4(0, 0, 0, 0);
                };
                pull(a1);
#pragma unroll
                for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) ms[0] += t[r].x, ms[1] += t[r].y, ms[2] += t[r].z, ms[3] += t[r].w;
#pragma unroll
                for (int x = 0; x < BPT; ++x) ms[x] <<= 16;
                pull(a2);
#pragma unroll
                for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) ms[0] += t[r].x, ms[1] += t[r].y, ms[2] += t[r].z, ms[3] += t[r].w;
            }
            unsigned long long b = sure + sample_before(ms[0] + ms[1] + ms[2] + ms[3], sh.scan, all);
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                if (b < limit && limit <= b + ms[x]) {
                    sh.border = tid * BPT + x;
                    sh.base_mass = b;
                }
                b += ms[x];
            }
            __syncthreads();
        }
        if (!fits) {  // the same in every block
            cluster_sync();
            for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
            cluster_sync();
            return false;
        }
        // the border bin's tokens, to every block; each finds the last one that stays
        const int border = sh.border;
        if (tid == 0) sh.n_cand = 0;
        __syncthreads();
        for (int i = tid; i < mine; i += SMP_THREADS) {
            const float z = smp_load(simg, (int)sh.loc[i]);
            if (bin_of(z) == border) {
                const uint32_t idx = at + sh.loc[i] - (uint32_t)mis, slot = atomicAdd(&sh.n_cand, 1u);
                if (slot < SMP_BORDER)
                    for (uint32_t r = 0; r < cl; ++r)
                        st_cluster_u64(mapa_shared(smem_u32(&sh.border_list[rank][slot]), r), (unsigned long long)smp_key(z) << 32 | (uint32_t)~idx);
            }
        }
        __syncthreads();
        if (tid < (int)cl) st_cluster_u32(mapa_shared(smem_u32(&sh.from[rank].border), tid), sh.n_cand);
        cluster_sync();
        // the lists one behind the other; the bins have been read by everybody
        unsigned long long* units = reinterpret_cast<unsigned long long*>(sh.mhi);  // [SMP_CAND]
        static_assert(sizeof(sh.mhi) + sizeof(sh.mlo) >= SMP_MAX_CLUSTER * SMP_BORDER * 8, "units of the border bin");
        for (int i = tid; i < (int)cl * SMP_BORDER; i += SMP_THREADS) {
            const uint32_t r = (uint32_t)i / SMP_BORDER, slot = (uint32_t)i % SMP_BORDER;
            if (slot < sh.from[r].border) units[i] = f.units(smp_unkey((uint32_t)(sh.border_list[r][slot] >> 32)));
            fits &= sh.from[r].border <= SMP_BORDER;
        }
        if (!__syncthreads_and(fits)) {
            cluster_sync();
            if (tid == 0) sh.n_cand = 0;
            for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
            cluster_sync();
            return false;
        }
        for (int i = tid; i < (int)cl * SMP_BORDER; i += SMP_THREADS) {
            const uint32_t r = (uint32_t)i / SMP_BORDER, slot = (uint32_t)i % SMP_BORDER;
            if (slot >= sh.from[r].border) continue;
            const unsigned long long me = sh.border_list[r][slot];
            unsigned long long b = sh.base_mass;
            for (uint32_t t = 0; t < cl; ++t)
                for (uint32_t j = 0; j < sh.from[t].border; ++j)
                    if (sh.border_list[t][j] > me) b += units[t * SMP_BORDER + j];
            if (b < limit && limit <= b + units[i]) {
                sh.lkey = (uint32_t)(me >> 32);
                sh.lidx = ~(uint32_t)me;
            }
        }
        __syncthreads();
        g.lkey = sh.lkey;
        g.lidx = sh.lidx;
        for (int i = tid; i < mine; i += SMP_THREADS) {
            const uint32_t j = sh.loc[i];
            const unsigned long long q = g.kept(smp_load(simg, (int)j), at + j - (uint32_t)mis);
            if (q) atomicAdd(&sh.extra[j / (SMP_THREADS * SMP_SWEEP)], q);
        }
    }

    // ---- the choice: the chunk, the round and warp, the lane, the token
    __syncthreads();
    unsigned long long sum = 0;
    for (int c = warp; c < chunks; c += SMP_WARPS) {
        const unsigned long long t = warp_sum_u64(lane < SMP_WARPS ? sh.sweep[c][lane] : 0ull) + sh.extra[c];
        if (lane == 0) sh.extra[c] = t;
        sum += t;
    }
    if (lane == 0) sh.scan[warp] = sum;
    __syncthreads();
    if (tid < (int)cl) {
        sum = 0;
        for (int w = 0; w < SMP_WARPS; ++w) sum += sh.scan[w];
        st_cluster_u64(mapa_shared(smem_u32(&sh.from[rank].kept), tid), sum);
    }
    cluster_sync();  // the last access to another block's memory lies before this
    unsigned long long before = 0, all = 0, own = 0;
#pragma unroll
    for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r) {
        const unsigned long long t = r < cl ? sh.from[r].kept : 0ull;
        if (r < rank) before += t;
        if (r == rank) own = t;
        all += t;
    }
    bool rest;
    unsigned long long target = share_of(u >= 0.0f ? fminf(u, 1.0f) : 0.0f, all, rest);
    if (target >= all) target = all - 1;
    if (target >= before && target - before < own) {  // the same for the whole block
        unsigned long long left = target - before;
        int c = 0;
        for (; left >= sh.extra[c]; ++c) left -= sh.extra[c];
        unsigned long long mine[ROUNDS];
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int v = (c * ROUNDS + r) * SMP_THREADS + tid;
            mine[r] = 0;
            if (v < pieces) {
                float z[PER];
                SmpPiece<T>::get(img[v], z);
#pragma unroll
                for (int e = 0; e < PER; ++e) mine[r] += g.kept(z[e] + 0.0f, at + (uint32_t)(v * PER + e - mis));
            }
            const unsigned long long t = warp_sum_u64(mine[r]);
            if (lane == 0) sh.wsum[r][warp] = t;
        }
        __syncthreads();
        int rr = 0, ww = 0;
        while (left >= sh.wsum[rr][ww]) {
            left -= sh.wsum[rr][ww];
            if (++ww == SMP_WARPS) {
                ww = 0;
                ++rr;
            }
        }
        if (warp == ww) {
            unsigned long long x = 0;
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r)
                if (r == rr) x = mine[r];
            unsigned long long e = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, e, o);
                if (lane >= o) e += y;
            }
            if (e - x <= left && left < e) {
                left -= e - x;
                const int v = (c * ROUNDS + rr) * SMP_THREADS + tid;
                float z[PER];
                SmpPiece<T>::get(img[v], z);
                int token = -1;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint32_t idx = at + (uint32_t)(v * PER + i - mis);
                    const unsigned long long q = g.kept(z[i] + 0.0f, idx);
                    if (token < 0 && left < q) token = (int)idx;
                    if (token < 0) left -= q;
                }
                p.out[row] = token;
            }
        }
    }
    return true;
}

template <typename T>
__global__ void __launch_bounds__(SMP_THREADS, 2) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank = cluster_rank(), cl;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
    // another block's memory may be written once that block runs: waited for before the first push
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int row = blockIdx.x / cl;
    const long long at = (long long)rank * p.seg;
    const int len = (int)(p.vocab - at < p.seg ? (p.vocab > at ? p.vocab - at : 0) : p.seg);
    const T* g = reinterpret_cast<const T*>(p.logits) + (size_t)row * p.vocab + at;
    // the segment's image in shared memory keeps the address modulo 16, so that whole 16-byte pieces can be copied;
    // the pieces that reach over either end are read element by element
    constexpr int PER = 16 / sizeof(T);
    const int mis = (int)((reinterpret_cast<uintptr_t>(g) & 15) / sizeof(T));
    T* simg = reinterpret_cast<T*>(raw);
    const T* s = simg + mis;
    const int pieces = len > 0 ? (mis + len + PER - 1) / PER : 0;
    float m = -INFINITY;
    bool nan = false;
    if (len > 0) {
        const uint4* ga = reinterpret_cast<const uint4*>(g - mis);
        constexpr int UN = 4;
        for (int base = 0; base < pieces; base += SMP_THREADS * UN) {
            uint4 w[UN];
            bool whole[UN];
#pragma unroll
            for (int x = 0; x < UN; ++x) {
                const int v = base + x * SMP_THREADS + tid;
                whole[x] = v < pieces && v * PER >= mis && (v + 1) * PER <= mis + len;
                if (whole[x]) w[x] = __ldcs(ga + v);
            }
#pragma unroll
            for (int x = 0; x < UN; ++x) {
                const int v = base + x * SMP_THREADS + tid;
                if (whole[x]) {
                    reinterpret_cast<uint4*>(raw)[v] = w[x];
                } else if (v < pieces) {  // what is not of this segment reads as -inf
                    for (int e = 0; e < PER; ++e) {
                        const int i = v * PER + e;
                        if (i >= mis && i < mis + len) simg[i] = g[i - mis];
                        else simg[i] = smp_minus_inf<T>();
                    }
                    w[x] = reinterpret_cast<const uint4*>(raw)[v];
                }
                if (v < pieces) {
                    float z[PER];
                    SmpPiece<T>::get(w[x], z);
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        nan |= z[e] != z[e];
                        m = fmaxf(m, z[e]);
                    }
                }
            }
        }
    }
    {
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) sh.wmax[warp] = __float_as_uint(m);
        nan = __syncthreads_or(nan);
        if (tid == 0) sh.n_cand = sh.n_loc = 0;
        for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
        if (tid < SMP_SWEEP_CHUNKS) sh.extra[tid] = 0;
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (tid < (int)cl) {
            for (int w = 0; w < SMP_WARPS; ++w) m = fmaxf(m, __uint_as_float(sh.wmax[w]));
            st_cluster_u32(mapa_shared(smem_u32(&sh.from[rank].max), tid), __float_as_uint(m));
            st_cluster_u32(mapa_shared(smem_u32(&sh.from[rank].nan), tid), nan);
        }
        cluster_sync();
        m = -INFINITY;
#pragma unroll
        for (uint32_t r = 0; r < SMP_MAX_CLUSTER; ++r)
            if (r < cl) {
                m = fmaxf(m, sh.from[r].max);
                nan |= sh.from[r].nan != 0;
            }
    }
    if (nan || m == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            p.out[row] = -1;
            if (nan) set_error(TBIK_ERR_VALUE);
        }
        return;
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    const int k = p.top_k ? p.top_k[row] : 0;
    const float tp = p.top_p ? p.top_p[row] : 1.0f;
    SampleFilter f;
    f.m = m;
    f.greedy = !(temp > 0.0f) || k == 1;
    f.ones = false;
    {
        const double c = f.greedy ? 1.0 : 1.4426950408889634 / (double)temp;
        f.c = (float)fmin(c, 3e38);
        f.c_lo = c < 1e30 ? (float)(c - (double)f.c) : 0.0f;
        f.low = -__fdiv_rn(200.0f, f.c);
    }
    f.min_w = p.min_p ? fmaxf(p.min_p[row], 0.0f) : 0.0f;  // NaN is off
    f.lkey = 0;
    f.lidx = 0xffffffffu;
    const bool by_k = !f.greedy && k > 0 && k < p.vocab;
    const bool by_p = !f.greedy && tp < 1.0f;
    int token;
    {
        const float scale = f.greedy ? 1.0f : __fdiv_rn(32.0f, temp);
        if (m < INFINITY && scale < 1e30f && scale > 1e-30f &&
            sample_fast<T>(p, sh, raw, row, rank, cl, len, mis, pieces, f, scale, by_k, by_p, k, tp))
            return;
    }
    if (by_k || by_p) {
        // the general steps: histogram over linear bins of (m - z) / temperature, 32 of them to a unit
        const float scale = __fdiv_rn(32.0f, temp);
        auto bin0 = [&](float z) { return min(SMP_BINS - 1, z == m ? 0 : __float2int_rz(__fmul_rn(__fsub_rn(m, z), scale))); };
        auto add = [&](int b, unsigned long long q) {
            atomicAdd(&sh.cnt[b], 1u);
            if (by_p) {
                if (q >> 16) atomicAdd(&sh.mhi[b], (uint32_t)(q >> 16));
                if (q & 0xffffu) atomicAdd(&sh.mlo[b], (uint32_t)(q & 0xffffu));
            }
        };
        for (int i = tid; i < len; i += SMP_THREADS) {
            const float z = smp_load(s, i);
            const unsigned long long q = by_p ? f.units(z) : 1;
            if (by_k || q) add(bin0(z), q);
        }
        constexpr int BPT = SMP_BINS / SMP_THREADS;
        uint32_t cnt[BPT];
        unsigned long long mass[BPT];
        uint32_t cnt0[BPT];
        unsigned long long mass0[BPT], total_mass = 0;
        // totals of every bin over the cluster, then their running sums; `border` is the bin in which the limit falls
        auto gather = [&]() {
            cluster_sync();
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                cnt[x] = 0;
                mass[x] = 0;
                for (uint32_t r = 0; r < cl; ++r) {
                    const int b = tid * BPT + x;
                    cnt[x] += ld_cluster_u32(mapa_shared(smem_u32(&sh.cnt[b]), r));
                    mass[x] += ((unsigned long long)ld_cluster_u32(mapa_shared(smem_u32(&sh.mhi[b]), r)) << 16) +
                               ld_cluster_u32(mapa_shared(smem_u32(&sh.mlo[b]), r));
                }
            }
        };
        auto block_before = [&](unsigned long long v, unsigned long long& all) {  // exclusive prefix over the block
            unsigned long long pfx = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, pfx, o);
                if (lane >= o) pfx += y;
            }
            __syncthreads();
            if (lane == 31) sh.scan[warp] = pfx;
            __syncthreads();
            unsigned long long b = 0;
            all = 0;
            for (int w = 0; w < SMP_WARPS; ++w) {
                if (w < warp) b += sh.scan[w];
                all += sh.scan[w];
            }
            return b + pfx - v;
        };
        auto find_border = [&](bool count, unsigned long long limit, const uint32_t (&cn)[BPT], const unsigned long long (&ms)[BPT],
                               uint32_t base_cnt, unsigned long long base_mass) {
            unsigned long long ca = 0, ma = 0, all;
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                ca += cn[x];
                ma += ms[x];
            }
            unsigned long long cb = base_cnt + block_before(ca, all), mb = base_mass + block_before(ma, all);
#pragma unroll
            for (int x = 0; x < BPT; ++x) {
                const unsigned long long b = count ? cb : mb, e = b + (count ? (unsigned long long)cn[x] : ms[x]);
                if (b < limit && limit <= e) {
                    sh.border = tid * BPT + x;
                    sh.border_cnt = (int)cn[x];
                    sh.base_cnt = (int)cb;
                    sh.base_mass = mb;
                }
                cb += cn[x];
                mb += ms[x];
            }
            __syncthreads();
        };
        // Keeps the tokens whose count (or mass) before them is below the limit: sets f.lkey, f.lidx to the last one
        // and returns the mass up to it.  cn0/ms0: the first histogram's totals.
        auto cut = [&](bool count, unsigned long long limit) {
            find_border(count, limit, cnt0, mass0, 0, 0);
            int border = sh.border, border_cnt = sh.border_cnt;
            unsigned long long bc = (unsigned long long)sh.base_cnt, bm = sh.base_mass;
            bool first = true;           // the border is a bin of the first histogram
            uint32_t klo = 0, khi = 0;   // afterwards: a range of keys
            auto inside = [&](float z, uint32_t idx, unsigned long long q) {
                if (!by_k && !q) return false;
                const uint32_t key = smp_key(z);
                if (key < f.lkey || (key == f.lkey && idx > f.lidx)) return false;  // an earlier cut
                return first ? bin0(z) == border : key >= klo && key <= khi;
            };
            unsigned long long through = 0;
            while (true) {
                if (border_cnt <= SMP_CAND) {
                    // sort the border's tokens in the cluster's first block
                    const uint32_t list = mapa_shared(smem_u32(sh.cand), 0), num = mapa_shared(smem_u32(&sh.n_cand), 0);
                    for (int i = tid; i < len; i += SMP_THREADS) {
                        const float z = smp_load(s, i);
                        const uint32_t idx = (uint32_t)(at + i);
                        if (inside(z, idx, by_k ? 1 : f.units(z))) {
                            const uint32_t slot = atom_add_cluster_u32(num, 1u);
                            if (slot < SMP_CAND) st_cluster_u64(list + slot * 8, (unsigned long long)smp_key(z) << 32 | (uint32_t)~idx);
                        }
                    }
                    cluster_sync();
                    if (rank == 0) {
                        const int n = min((int)sh.n_cand, SMP_CAND);
                        int n2 = 32;
                        while (n2 < n) n2 <<= 1;
                        for (int i = n + tid; i < n2; i += SMP_THREADS) sh.cand[i] = 0;
                        __syncthreads();
                        for (int size = 2; size <= n2; size <<= 1)
                            for (int stride = size >> 1; stride; stride >>= 1) {
                                for (int i = tid; i < n2 / 2; i += SMP_THREADS) {
                                    const int a = 2 * i - (i & (stride - 1)), b = a + stride;
                                    const unsigned long long x = sh.cand[a], y = sh.cand[b];
                                    if ((x < y) == ((a & size) == 0)) {
                                        sh.cand[a] = y;
                                        sh.cand[b] = x;
                                    }
                                }
                                __syncthreads();
                            }
                        // running sums over the sorted list; two tokens per thread
                        unsigned long long q[2], v = 0, all;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int i = tid * 2 + x;
                            q[x] = 0;
                            if (i < n) {
                                const uint32_t key = (uint32_t)(sh.cand[i] >> 32);
                                q[x] = f.units(__uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key));
                            }
                            v += q[x];
                        }
                        unsigned long long mb = bm + block_before(v, all);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int i = tid * 2 + x;
                            const unsigned long long b = count ? bc + i : mb, e = count ? b + 1 : mb + q[x];
                            if (i < n && b < limit && limit <= e) {
                                sh.lkey = (uint32_t)(sh.cand[i] >> 32);
                                sh.lidx = ~(uint32_t)sh.cand[i];
                                sh.mass = mb + q[x];
                            }
                            mb += q[x];
                        }
                    }
                    cluster_sync();
                    f.lkey = ld_cluster_u32(mapa_shared(smem_u32(&sh.lkey), 0));
                    f.lidx = ld_cluster_u32(mapa_shared(smem_u32(&sh.lidx), 0));
                    through = ld_cluster_u64(mapa_shared(smem_u32(&sh.mass), 0));
                    if (tid == 0) sh.n_cand = 0;
                    cluster_sync();
                    return through;
                }
                // too many: the range of their keys, and a histogram over it
                uint32_t lo = 0xffffffffu, hi = 0;
                for (int i = tid; i < len; i += SMP_THREADS) {
                    const float z = smp_load(s, i);
                    if (inside(z, (uint32_t)(at + i), by_k ? 1 : f.units(z))) {
                        lo = min(lo, smp_key(z));
                        hi = max(hi, smp_key(z));
                    }
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                if (lane == 0) {
                    sh.wmin[warp] = lo;
                    sh.wmax[warp] = hi;
                }
                for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
                __syncthreads();
                if (tid == 0) {
                    for (int w = 0; w < SMP_WARPS; ++w) {
                        lo = min(lo, sh.wmin[w]);
                        hi = max(hi, sh.wmax[w]);
                    }
                    sh.kmin = lo;
                    sh.kmax = hi;
                }
                cluster_sync();
                lo = 0xffffffffu;
                hi = 0;
                for (uint32_t r = 0; r < cl; ++r) {
                    lo = min(lo, ld_cluster_u32(mapa_shared(smem_u32(&sh.kmin), r)));
                    hi = max(hi, ld_cluster_u32(mapa_shared(smem_u32(&sh.kmax), r)));
                }
                klo = lo;
                khi = hi;
                first = false;
                if (klo == khi) {
                    // all equal: how many of them stay, and the index of the last of those
                    const unsigned long long q = f.units(__uint_as_float((klo & 0x80000000u) ? (klo & 0x7fffffffu) : ~klo));
                    const unsigned long long stay = count ? limit - bc : (limit - bm + q - 1) / (q ? q : 1);
                    SampleFilter t = f;
                    t.ones = true;
                    t.lkey = klo;
                    cluster_sync();
                    int last;
                    sample_select(s, len, (uint32_t)at, t, sh, rank, cl, [&](unsigned long long) { return stay - 1; }, last);
                    f.lkey = klo;
                    f.lidx = (uint32_t)last;
                    return bm + stay * q;
                }
                int shift = 0;
                while (((khi - klo) >> shift) >= (uint32_t)SMP_BINS) ++shift;
                for (int i = tid; i < len; i += SMP_THREADS) {
                    const float z = smp_load(s, i);
                    const unsigned long long q = by_p ? f.units(z) : 1;
                    if (inside(z, (uint32_t)(at + i), q)) add((int)((khi - smp_key(z)) >> shift), q);
                }
                gather();
                find_border(count, limit, cnt, mass, (uint32_t)bc, bm);
                border = sh.border;
                border_cnt = sh.border_cnt;
                bc = (unsigned long long)sh.base_cnt;
                bm = sh.base_mass;
                khi = khi - ((uint32_t)border << shift);
                const uint32_t width = (1u << shift) - 1u;
                klo = khi - klo > width ? khi - width : klo;
                cluster_sync();  // the bins have been read by everybody
            }
        };
        gather();
#pragma unroll
        for (int x = 0; x < BPT; ++x) {
            cnt0[x] = cnt[x];
            mass0[x] = mass[x];
            total_mass += mass[x];
        }
        unsigned long long all = 0;
        block_before(total_mass, all);
        cluster_sync();
        if (by_k) {
            const unsigned long long t = cut(true, (unsigned long long)k);
            if (by_p) all = t;
        }
        if (by_p) {
            bool rest;
            unsigned long long limit = share_of(tp > 0.0f ? tp : 0.0f, all, rest);
            if (rest) ++limit;         // mass before < share, in integers
            if (limit < 1) limit = 1;  // the first token always stays
            if (limit < all) cut(false, limit);
        }
    }
    const float u = p.u[row];
    sample_select(s, len, (uint32_t)at, f, sh, rank, cl,
                  [&](unsigned long long total) {
                      bool rest;
                      const unsigned long long t = share_of(u >= 0.0f ? fminf(u, 1.0f) : 0.0f, total, rest);
                      return f.greedy ? 0ull : (t < total ? t : total - 1);
                  },
                  token);
    if (rank == 0 && tid == 0) p.out[row] = token;
}

}  // namespace tbik

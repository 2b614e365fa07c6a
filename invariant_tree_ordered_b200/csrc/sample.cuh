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
// The threshold of top-k and top-p is found by a histogram over linear bins of (max - z) / temperature, whose border
// bin (usually some tens of tokens) is sorted in one block; a border bin with more tokens is split again on the bits
// of the logits until it fits or all its logits are equal.
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
    unsigned long long csum[SMP_MAX_SEG / SMP_CHUNK][SMP_WARPS];
    unsigned long long wsum[SMP_CHUNK_ROUNDS][SMP_WARPS];
    unsigned long long cand[SMP_CAND];  // key << 32 | ~index: descending order is the order of the tokens
    unsigned long long scan[SMP_WARPS + 1];
    unsigned long long total;           // this block's kept mass (read by the others)
    unsigned long long mass;            // mass up to and with the last kept token
    unsigned long long base_mass;
    uint32_t cnt[SMP_BINS], mhi[SMP_BINS], mlo[SMP_BINS];
    uint32_t wmin[SMP_WARPS], wmax[SMP_WARPS];
    uint32_t kmin, kmax;
    uint32_t n_cand;
    uint32_t lkey, lidx;  // the last kept token
    float bmax;
    int nan;
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

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__device__ __forceinline__ float smp_load(const T* s, int i);
template <>
__device__ __forceinline__ float smp_load<float>(const float* s, int i) { return s[i] + 0.0f; }
template <>
__device__ __forceinline__ float smp_load<uint16_t>(const uint16_t* s, int i) { return bf2f(s[i]) + 0.0f; }

// What is kept, and with which weight.
struct SampleFilter {
    float m, c, min_w;  // row maximum, log2(e) / temperature, min_p
    bool greedy;        // only tokens at the maximum
    bool ones;          // weights 1 for tokens of key lkey (counting equal ones)
    uint32_t lkey, lidx;

    __device__ __forceinline__ float weight(float z) const {
        if (z == m) return 1.0f;
        if (z == -INFINITY) return 0.0f;
        return ex2_hw(__fmul_rn(__fsub_rn(z, m), c));
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

// u * total as (floor, whether something is left over), u in [0, 1].
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long total, bool& rest) {
    const unsigned long long U = __double2ull_rz((double)u * 9223372036854775808.0);  // exact
    rest = ((total << 1) * U) != 0;
    return __umul64hi(total << 1, U);
}

template <typename T>
__global__ void __launch_bounds__(SMP_THREADS) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank = cluster_rank(), cl;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
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
    float m = -INFINITY;
    bool nan = false;
    if (len > 0) {
        const int pieces = (mis + len + PER - 1) / PER;
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
                } else if (v < pieces) {
                    for (int e = 0; e < PER; ++e) {
                        const int i = v * PER + e;
                        if (i >= mis && i < mis + len) simg[i] = g[i - mis];
                    }
                }
                if (v < pieces)
                    for (int e = 0; e < PER; ++e) {
                        const int i = v * PER + e;
                        if (i >= mis && i < mis + len) {
                            const float z = smp_load(simg, i);
                            nan |= z != z;
                            m = fmaxf(m, z);
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
        if (tid == 0) {
            for (int w = 0; w < SMP_WARPS; ++w) m = fmaxf(m, __uint_as_float(sh.wmax[w]));
            sh.bmax = m;
            sh.nan = nan;
            sh.n_cand = 0;
        }
        for (int i = tid; i < SMP_BINS; i += SMP_THREADS) sh.cnt[i] = sh.mhi[i] = sh.mlo[i] = 0;
        cluster_sync();
        m = -INFINITY;
        for (uint32_t r = 0; r < cl; ++r) {
            m = fmaxf(m, __uint_as_float(ld_cluster_u32(mapa_shared(smem_u32(&sh.bmax), r))));
            nan |= ld_cluster_u32(mapa_shared(smem_u32(&sh.nan), r)) != 0;
        }
    }
    if (nan || m == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) {
            p.out[row] = -1;
            if (nan) set_error(TBIK_ERR_VALUE);
        }
        cluster_sync();
        return;
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    const int k = p.top_k ? p.top_k[row] : 0;
    const float tp = p.top_p ? p.top_p[row] : 1.0f;
    SampleFilter f;
    f.m = m;
    f.greedy = !(temp > 0.0f) || k == 1;
    f.ones = false;
    f.c = f.greedy ? 1.0f : __fdiv_rn(1.44269504088896341f, temp);
    f.min_w = p.min_p ? p.min_p[row] : 0.0f;
    f.lkey = 0;
    f.lidx = 0xffffffffu;
    const bool by_k = !f.greedy && k > 0 && k < p.vocab;
    const bool by_p = !f.greedy && tp < 1.0f;
    int token;
    if (by_k || by_p) {
        // histogram over linear bins of (m - z) / temperature, 32 of them to a unit
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

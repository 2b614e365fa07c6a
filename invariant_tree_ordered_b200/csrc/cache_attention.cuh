// Attention over the paged 8-bit cache (cache.cuh), with the key reduction in tree order.
//
// Query t of sequence b sits at position i = start[b] + t and sees the keys at positions 0..i.  They are reduced like
// in the other attentions of the library: leaves of 128 consecutive positions, each a (max, sum, weighted value sum)
// summary, combined by the halving tree over the ceil((i + 1) / 128) leaves, so a row's bits depend only on its
// query and the cache's contents, never on the batch or on how the work is split.
#pragma once

#include "cache.cuh"

namespace tbik {

constexpr int CATT_LEAF = 128;
constexpr int CATT_MAX_LEVELS = 20;

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
    float scale;  // log2(e) / sqrt(head_dim)
};

__device__ __forceinline__ float e4m3_f32(uint32_t b) {
    const uint32_t m = b & 7u, f = (b >> 3) & 15u;
    float v = f ? __uint_as_float(((f + 120u) << 23) | (m << 20)) : (float)m * 0x1p-9f;
    if ((b & 0x7Fu) == 0x7Fu) v = __uint_as_float(0x7fc00000u);
    return (b & 0x80u) ? -v : v;
}

// One block of 128 threads per (packed token, head): a thread is a key for the scores and a dim for the values.
template <int D>
__global__ void __launch_bounds__(128) cache_attention_simple_kernel(const CacheAttParams p) {
    __shared__ float qs[D], ps[128], red[4], vs[128];
    __shared__ int ids[128];
    const int tid = threadIdx.x, tok = blockIdx.x, head = blockIdx.y, kvh = head / (p.heads / p.kv_heads);
    int b = tok, t = 0;
    if (p.cu) {
        int lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu[mid] <= tok) lo = mid; else hi = mid - 1;
        }
        b = lo;
        t = tok - p.cu[b];
        if (t < 0 || tok >= p.cu[b + 1]) return;  // before the first or behind the last sequence
    }
    uint16_t* out = p.out + ((size_t)tok * p.heads + head) * D;
    const int s = p.start[b], row = p.rows ? p.rows[b] : b;
    const long long n = (long long)s + t + 1;
    bool bad = row < 0 || row >= p.slots || n > p.max_keys || n > (long long)p.max_pages * p.page || t >= p.max_q;
    if (s < 0 || bad) {
        if (tid < D) out[tid] = 0x7fc0;
        if (bad && tid == 0) set_error(TBIK_ERR_PAGE);
        return;
    }
    if (tid < D) qs[tid] = bf2f(p.q[((size_t)tok * p.heads + head) * D + tid]);
    const int L = (int)((n + CATT_LEAF - 1) / CATT_LEAF);
    float sm[CATT_MAX_LEVELS], ss[CATT_MAX_LEVELS], so[CATT_MAX_LEVELS];
    int depth = 0;
    for (int leaf = 0; leaf < L; ++leaf) {
        const int j = leaf * CATT_LEAF + tid;
        __syncthreads();
        float sc = -INFINITY;
        int id = -1;
        if (j < n) {
            id = p.table[(size_t)row * p.max_pages + j / p.page];
            if (id < 0 || id >= p.num_pages) {
                bad = true;
                id = -1;
            }
        }
        if (id >= 0) {
            const size_t ph = (size_t)id * p.kv_heads + kvh;
            const int o = j % p.page;
            const uint8_t* k = p.pages + ph * ((size_t)p.page * D) + (o >> 3) * (D * 8) + (o & 7) * 16;
            float a = 0.0f;
            for (int g = 0; g < D / 16; ++g)
                for (int e = 0; e < 16; ++e) a = __fmaf_rn(e4m3_f32(k[g * 128 + e]), qs[g * 16 + e], a);
            sc = a * p.scales[ph] * p.scale;
            vs[tid] = p.scales[(size_t)p.num_pages * p.kv_heads + ph];
        }
        ids[tid] = id;
        float m = sc;
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        ps[tid] = id >= 0 ? ex2_hw(sc - m) : 0.0f;
        __syncthreads();
        float sum = 0.0f, o = 0.0f;
        const int cnt = n - (long long)leaf * CATT_LEAF < CATT_LEAF ? (int)(n - (long long)leaf * CATT_LEAF) : CATT_LEAF;
        for (int c = 0; c < cnt; ++c) {
            sum += ps[c];
            if (tid < D && ids[c] >= 0) {
                const int pos = (leaf * CATT_LEAF + c) % p.page;
                const uint8_t* v = p.pages + (((size_t)p.num_pages + ids[c]) * p.kv_heads + kvh) * ((size_t)p.page * D);
                o = __fmaf_rn(ps[c] * vs[c], e4m3_f32(v[(pos >> 3) * (D * 8) + (tid >> 4) * 128 + (pos & 7) * 16 + (tid & 15)]), o);
            }
        }
        // close the nodes whose last leaf this is, deepest first
        const LeafOps ops = leaf_ops(L, leaf);
        for (int c = leaf_pops(ops); c > 0; --c) {
            --depth;
            const float M = fmaxf(sm[depth], m);
            const float ea = sm[depth] == M ? 1.0f : ex2_hw(sm[depth] - M), eb = m == M ? 1.0f : ex2_hw(m - M);
            sum = __fmaf_rn(sum, eb, __fmul_rn(ss[depth], ea));
            o = __fmaf_rn(o, eb, __fmul_rn(so[depth], ea));
            m = M;
        }
        sm[depth] = m;
        ss[depth] = sum;
        so[depth] = o;
        ++depth;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) set_error(TBIK_ERR_PAGE);
    if (tid < D) out[tid] = bad ? (uint16_t)0x7fc0 : f2bf(__fmul_rn(so[0], __fdiv_rn(1.0f, ss[0])));
}

}  // namespace tbik

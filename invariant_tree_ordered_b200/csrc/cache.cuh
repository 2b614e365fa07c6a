// The paged 8-bit key/value cache: its layout, the writes into it (tbik_cache_append) and the life of its pages
// (extend, fork, free, compact, copy).  cache_attention.cuh reads it.
//
// A page holds `page` consecutive positions of one sequence for every kv head, keys and values apart; per (page,
// head) the tokens' e4m3 bytes and one fp32 power-of-two scale.  Inside a page, token t's dims 16j..16j+15 are 16
// contiguous bytes at (t / 8) * (D * 8) + j * 128 + (t % 8) * 16: blocks of 8 tokens x 16 dims, 128 bytes each,
// which is the unswizzled operand block of tcgen05.mma for 8-bit types.  The same bytes are K-major for keys (the
// products run over dims) and MN-major for values (they run over tokens), so attention copies a page to shared
// memory in one piece and the tensor cores read it as it lies there, for every page size that is a multiple of 16.
#pragma once

#include "device_common.cuh"

namespace tbik {

constexpr int CACHE_EMIN = -100;         // the smallest scale exponent (a page of zeros has it)
constexpr int CACHE_MAX_BATCH = 8192;    // sequences per call of the page operations (their prefix sums are in shared memory)
constexpr int CACHE_MAX_SLOTS = 65536;   // table rows (one bit each in shared memory)
constexpr int CACHE_MAX_PAGES = 1 << 20; // pages of a pool (one bit each in shared memory)

__device__ __forceinline__ float cache_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int cache_exponent(float s) { return (int)(__float_as_uint(s) >> 23 & 255) - 127; }

// ------------------------------------------------------------------ append
//
// The stored value of x under scale 2^E is cut(r * 2^-E), r = x rounded to 4 significant bits (to nearest, ties to
// even) and cut = truncation to e4m3's grid, which only matters below 2^-6 (spacing 2^-9).  E is the smallest
// exponent with max |r| <= 448 * 2^E over the page's tokens so far, at least CACHE_EMIN.  When a later token raises
// E, the older bytes are cut again on the coarser grid.  Truncations on nested grids compose (cut after cut is the
// coarser cut), and r does not depend on E, so the bytes of a page whose positions are written once and in order are a
// function of its tokens alone and not of how the tokens were split into calls; rounding twice to nearest would not have
// that property.  (A position written again leaves the scale that its first token raised.)  Everything below is integer
// arithmetic on the bit patterns, hence exact.

// bf16 magnitude bits (15) -> magnitude bits rounded to 3 mantissa bits (the low 4 bits are zero afterwards; a carry
// runs into the exponent field, up to 0x7F80 = 2^128 for the largest inputs, which the scale absorbs).
__host__ __device__ __forceinline__ uint32_t cache_round4(uint32_t mag) { return (mag + 7u + ((mag >> 4) & 1u)) & 0x7FF0u; }

// The smallest E with (rounded magnitude) <= 448 * 2^E = 1.75 * 2^(8+E).
__host__ __device__ __forceinline__ int cache_need(uint32_t rmag) {
    const int e = (int)(rmag >> 7) - 127, m = (int)(rmag >> 4) & 7;
    const int E = (m <= 6) ? e - 8 : e - 7;
    return (rmag == 0 || E < CACHE_EMIN) ? CACHE_EMIN : E;
}

// One bf16 pattern -> e4m3 byte under scale 2^E.  Infinities saturate, NaN becomes zero (both are reported).
__host__ __device__ __forceinline__ uint32_t cache_quant(uint32_t h, int E) {
    const uint32_t sign = (h >> 8) & 0x80u, mag = h & 0x7FFFu;
    if (mag >= 0x7F80u) return mag == 0x7F80u ? (sign | 0x7Eu) : 0u;
    const uint32_t r = cache_round4(mag);
    const int f = (int)(r >> 7) - 127 - E + 7;  // e4m3 exponent field of the normal value
    const uint32_t m = (r >> 4) & 7u;
    uint32_t b;
    if (f >= 1)
        b = ((uint32_t)f << 3) | m;
    else {
        const int sh = 1 - f;
        b = (r < 0x80u || sh > 4) ? 0u : (8u + m) >> sh;  // bf16 subnormals are far below the grid
    }
    return sign | b;
}

// The same for the two halves of a word whose magnitudes are finite, as two bytes: round4 on both halves at once (no
// carry leaves a half), cut by an addition of 2^14 that rounds toward zero (fp32's spacing there is e4m3's below 2^-6,
// and finer ones above stay), and a conversion that is then exact.  `down` is 2^-E, E < 120 (there, fp32 holds every
// rounded value).
__device__ __forceinline__ uint32_t cache_quant2(uint32_t w, float down) {
    const uint32_t mag = w & 0x7fff7fffu;
    const uint32_t r = (mag + 0x00070007u + ((mag >> 4) & 0x00010001u)) & 0x7ff07ff0u;
    const float lo = __fsub_rn(__fmaf_rz(__uint_as_float(r << 16), down, 16384.0f), 16384.0f);
    const float hi = __fsub_rn(__fmaf_rz(__uint_as_float(r & 0xffff0000u), down, 16384.0f), 16384.0f);
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi), "f"(lo));
    return (uint32_t)b | (__byte_perm(w, 0, 0x4431) & 0x8080u);  // the signs are in bytes 1 and 3
}

// An e4m3 byte cut to the grid of a scale 2^d times larger.
__host__ __device__ __forceinline__ uint32_t cache_down(uint32_t q, int d) {
    const uint32_t sign = q & 0x80u, b = q & 0x7Fu;
    if (b == 0x7Fu) return q;
    const int f = (int)(b >> 3) - d;
    const uint32_t m = b & 7u;
    uint32_t r;
    if (b < 8u)
        r = d > 3 ? 0u : b >> d;
    else if (f >= 1)
        r = b - ((uint32_t)d << 3);
    else
        r = (1 - f) > 4 ? 0u : (8u + m) >> (1 - f);
    return sign | r;
}

struct CacheAppendParams {
    const uint16_t* k;
    const uint16_t* v;
    uint8_t* pages;   // [2][num_pages][kv_heads][page * D]
    float* scales;    // [2][num_pages][kv_heads]
    const int32_t* table;
    const int32_t* refs;
    const int32_t* start;
    const int32_t* cu;    // null: token b belongs to sequence b
    const int32_t* rows;  // null: sequence b has table row b
    int tokens, batch, slots, max_pages, num_pages, kv_heads, page, page_shift;
};

// One block per (page that a sequence's new tokens touch, kv head, keys or values): the page's new tokens are read
// once into registers (16-byte loads, CH of them in flight per thread), their largest magnitude fixes the scale, and
// the bytes go out 8 at a time (two tokens of a warp fill a 32-byte sector).  The tokens are asked for before the page is
// looked up, so that the chain of loads is sequence, start, tokens.  Bound by integer instructions ahead of HBM: 32 prompts
// of 100 to 4096 tokens, 8 heads of 128 dims, 58 us, 3.9 TB/s; 16 instructions a value (39 M by warps), 9.6 of them on the
// ALU pipe, which is 75 % busy, with issue slots 64 % and DRAM 42 %.  128 threads with eight loads each measured 58 us
// there, 256 with four 65 us.  A decode step (one token each: one warp per token, head and operand, eight to a block) takes
// 2.3 us for 64 sequences and 39 us for 8192 (8 heads of 128; blocks of one warp took 2.5 and 70 us).
//
// Which page a block has: sequence b's pages start at virtual index cu[b] / page + 2 b.  n tokens touch at most
// n / page + 2 pages, so the ranges do not overlap, and the grid is known without reading `start`.  The sequence is
// found in two steps of THREADS looks, whatever the batch (8192 at most; as many steps as it takes to see all of them
// were 1128 us for 8192 sequences of one token, two are 263 us).
//
// With `rows`, a slot that is named twice would be written by two blocks at once.  Up to APPEND_FEW * THREADS sequences a
// block compares its slot with all of the call's.  For more (and for single tokens, GROUPS warps a block) the grid is what
// the device holds; each block marks all slots once, in two maps of a bit per slot, and takes several pages or tokens in
// turn, so that the looks stay in proportion to the call: 8192 single tokens 51 us (356 us with all blocks comparing),
// with `cu` 389 us (1348 us).  Up to 4 looks a thread the comparison is as fast or faster: 512 sequences 22 us either way,
// 64 4.6 us (5.3 us with maps).
constexpr int APPEND_FEW = 4;
template <int THREADS>
__device__ __forceinline__ int append_sequence(const CacheAppendParams& p, int x) {
    static_assert(THREADS * THREADS >= CACHE_MAX_BATCH, "two steps");
    const int tid = threadIdx.x, stride = (p.batch + THREADS - 1) / THREADS;
    auto before = [&](int i) { return i < p.batch && (p.cu[i] >> p.page_shift) + 2 * i <= x; };
    const int b = (__syncthreads_count(before(tid * stride)) - 1) * stride;  // of the looked at, the last that starts at or before x
    if (stride == 1 || b < 0) return b;
    return b + __syncthreads_count(tid + 1 < stride && before(b + tid + 1));
}

// (The ROWS form's bounds on registers keep as many blocks on an SM as the other's: left alone it takes up to 152, and 32
// prompts 76 us in place of 55.)
template <int D, int THREADS, int CH, int GROUPS, bool ROWS>
__global__ void __launch_bounds__(THREADS * GROUPS, ROWS && GROUPS == 1 ? (CH == 8 ? 768 : CH == 4 ? 1024 : 1536) / THREADS : 0)
    cache_append_kernel(const CacheAppendParams p) {
    static_assert(GROUPS == 1 || THREADS == 32, "groups are warps");
    const int tid = threadIdx.x % THREADS;
    const int head = blockIdx.y, kv = blockIdx.z;
    extern __shared__ uint32_t append_maps[];  // slots that the call names, and those it names twice
    uint32_t* twice = append_maps + (p.slots + 31) / 32;
    const bool maps = ROWS && (GROUPS > 1 || p.batch > APPEND_FEW * THREADS);
    if (maps) {
        for (int i = threadIdx.x; i < 2 * ((p.slots + 31) / 32); i += THREADS * GROUPS) append_maps[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.batch; i += THREADS * GROUPS) {
            const int r = p.rows[i];
            if (r >= 0 && r < p.slots) {
                const uint32_t bit = 1u << (r & 31);
                if (atomicOr(&append_maps[r >> 5], bit) & bit) atomicOr(&twice[r >> 5], bit);
            }
        }
        __syncthreads();
    }
    __shared__ uint32_t red[THREADS / 32];
    auto page = [&](int vp) {  // of the touched pages, or (without cu) of the tokens
        int b, t0, n, j;  // sequence, its first token, its tokens, page number among the touched ones
        if constexpr (GROUPS == 1) {
            b = append_sequence<THREADS>(p, vp);
            if (b < 0) return;  // cu[0] > 0 and before the first page
            t0 = p.cu[b];
            n = p.cu[b + 1] - t0;
            j = vp - ((t0 >> p.page_shift) + 2 * b);
            if (t0 < 0 || n < 0 || t0 > p.tokens - n) {
                if (tid == 0) set_error(TBIK_ERR_POSITION);
                return;
            }
        } else {
            b = vp;
            t0 = b;
            n = 1;
            j = 0;
        }
        const int s = p.start[b];
        const int first = s >> p.page_shift;  // the page of the first new token
        if (n <= 0 || j < 0 || s < 0) return;
        const long long end = (long long)s + n;
        const long long pg = (long long)first + j;
        const long long pg0 = pg * p.page;
        if (pg0 >= end) return;  // fewer pages than the bound allows
        const int o0 = pg0 >= s ? 0 : (int)(s - pg0);                          // first new token's place in the page
        const int o1 = (int)(end - pg0 < p.page ? end - pg0 : p.page);         // behind the last
        const int src0 = t0 + (int)(pg0 + o0 - s);                             // its packed token
        const int chunks = (o1 - o0) * (D / 8);
        const uint16_t* x = (kv ? p.v : p.k) + ((size_t)src0 * p.kv_heads + head) * D;
        const size_t tstride = (size_t)p.kv_heads * D;
        uint4 w[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = c * THREADS + tid;
            w[c] = make_uint4(0, 0, 0, 0);
            if (i < chunks) w[c] = __ldg(reinterpret_cast<const uint4*>(x + (size_t)(i / (D / 8)) * tstride) + i % (D / 8));
        }
        // the tokens are on their way while the page is looked up
        const int row = ROWS ? p.rows[b] : b;
        bool bad = row < 0 || row >= p.slots || pg >= p.max_pages;
        if (maps) {
            if (!bad) bad = (twice[row >> 5] >> (row & 31)) & 1u;
        } else if (ROWS && !bad) {
            bool dup = false;
            for (int i = tid; i < p.batch; i += THREADS) dup |= i != b && p.rows[i] == row;
            bad = __syncthreads_or(dup);
        }
        int id = -1;
        if (!bad) {
            id = p.table[(size_t)row * p.max_pages + pg];
            bad = id < 0 || id >= p.num_pages || p.refs[id] != 1;  // a shared page is never written
        }
        if (bad) {
            if (tid == 0) set_error(TBIK_ERR_PAGE);
            return;
        }
        uint32_t top2 = 0;  // largest magnitudes of the even and the odd dims
#pragma unroll
        for (int c = 0; c < CH; ++c)
            top2 = __vmaxu2(__vmaxu2(top2, __vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu)),
                            __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu));
        uint32_t top = max(top2 & 0xffffu, top2 >> 16);
        const bool odd = top >= 0x7F80u;
        if (odd) {  // what is not finite does not count
            top = 0;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint32_t a[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t l = a[q] & 0x7FFFu, h = (a[q] >> 16) & 0x7FFFu;
                    if (l < 0x7F80u) top = max(top, l);
                    if (h < 0x7F80u) top = max(top, h);
                }
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (THREADS > 32) {
            if ((tid & 31) == 0) red[tid >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < THREADS / 32; ++i) top = max(top, red[i]);
        }
        if (odd) set_error(TBIK_ERR_VALUE);
        int E = cache_need(cache_round4(top));  // rounding is monotone: the largest magnitude rounds to the largest
        const size_t ph = ((size_t)kv * p.num_pages + id) * p.kv_heads + head;
        uint8_t* dst = p.pages + ph * ((size_t)p.page * D);
        if (o0 > 0) {
            const int was = cache_exponent(p.scales[ph]);
            if (THREADS > 32)
                __syncthreads();  // every thread has read the old scale before it is replaced
            else
                __syncwarp();
            if (E <= was) {
                E = was;
            } else {  // older tokens follow the larger scale
                const int d = E - was;
                for (int i = tid; i < o0 * (D / 16); i += THREADS) {
                    const int t = i / (D / 16), g = i % (D / 16);
                    uint4* q = reinterpret_cast<uint4*>(dst + (t >> 3) * (D * 8) + g * 128 + (t & 7) * 16);
                    uint4 y = *q;
                    uint32_t* a = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t v = a[k];
                        a[k] = cache_down(v & 255u, d) | cache_down((v >> 8) & 255u, d) << 8 |
                               cache_down((v >> 16) & 255u, d) << 16 | cache_down(v >> 24, d) << 24;
                    }
                    *q = y;
                }
            }
        }
        if (tid == 0) p.scales[ph] = cache_pow2(E);
        const float down = cache_pow2(-E);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = c * THREADS + tid;
            if (i < chunks) {
                const int t = o0 + i / (D / 8), g = i % (D / 8);
                const uint32_t a[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                uint2 y;
                if (!odd && E < 120) {  // at 120 the largest rounded value is 2^128
                    y.x = cache_quant2(a[0], down) | cache_quant2(a[1], down) << 16;
                    y.y = cache_quant2(a[2], down) | cache_quant2(a[3], down) << 16;
                } else {
                    y.x = cache_quant(a[0] & 0xffffu, E) | cache_quant(a[0] >> 16, E) << 8 |
                          cache_quant(a[1] & 0xffffu, E) << 16 | cache_quant(a[1] >> 16, E) << 24;
                    y.y = cache_quant(a[2] & 0xffffu, E) | cache_quant(a[2] >> 16, E) << 8 |
                          cache_quant(a[3] & 0xffffu, E) << 16 | cache_quant(a[3] >> 16, E) << 24;
                }
                *reinterpret_cast<uint2*>(dst + (t >> 3) * (D * 8) + (g >> 1) * 128 + (t & 7) * 16 + (g & 1) * 8) = y;
            }
        }
    };
    if constexpr (GROUPS > 1) {
        for (int x = blockIdx.x * GROUPS + (int)threadIdx.x / THREADS; x < p.batch; x += gridDim.x * GROUPS) page(x);
    } else if constexpr (ROWS) {
        const int pages = p.tokens / p.page + 2 * p.batch;
        for (int x = blockIdx.x; x < pages; x += gridDim.x) {
            page(x);
            __syncthreads();  // `red` and the page's old scale have been read
        }
    } else {
        page(blockIdx.x);
    }
}

// ------------------------------------------------------- page operations
//
// Bookkeeping: table [slots][max_pages] page numbers (-1 behind a sequence's last page), lens [slots] tokens, refs
// [num_pages] table entries that name a page (0: free).  Every call is all or nothing: a kernel of one block looks
// at all of its arguments first and only then changes anything.  New pages are the lowest free ones, handed out in
// the order of the call's sequences, so the outcome does not depend on timing.

constexpr int CACHE_PLAN_THREADS = 1024;

// Exclusive prefix sum over the block; `total` is the block's sum.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return s - v + (warp ? before : 0);
}

// refs of pages 4i..4i+3 (past the pool: `fill`).
__device__ __forceinline__ int4 load_refs4(const int32_t* refs, int i4, int num_pages, int fill) {
    const int p = 4 * i4;
    if (p + 3 < num_pages) return *reinterpret_cast<const int4*>(refs + p);
    int4 r;
    r.x = p < num_pages ? refs[p] : fill;
    r.y = p + 1 < num_pages ? refs[p + 1] : fill;
    r.z = p + 2 < num_pages ? refs[p + 2] : fill;
    r.w = fill;
    return r;
}

// Whether the pool has `want` free pages.  Stops as soon as it has seen that many.
__device__ __forceinline__ bool enough_free(const int32_t* refs, int num_pages, int want, int* warp_sums) {
    int seen = 0;
    for (int base = 0; base * 4 < num_pages && seen < want; base += CACHE_PLAN_THREADS) {
        const int4 r = load_refs4(refs, base + threadIdx.x, num_pages, 1);
        int total;
        block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), warp_sums, total);
        seen += total;
    }
    return seen >= want;
}

// Calls give(rank, page) for the `want` lowest free pages.
template <typename F>
__device__ __forceinline__ void each_free(const int32_t* refs, int num_pages, int want, int* warp_sums, F give) {
    int seen = 0;
    for (int base = 0; base * 4 < num_pages && seen < want; base += CACHE_PLAN_THREADS) {
        const int4 r = load_refs4(refs, base + threadIdx.x, num_pages, 1);
        const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
        int total;
        int rank = seen + block_scan(f[0] + f[1] + f[2] + f[3], warp_sums, total);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (f[q]) {
                if (rank < want) give(rank, 4 * (base + (int)threadIdx.x) + q);
                ++rank;
            }
        seen += total;
    }
}

// In place: need[0..n) -> exclusive prefix sums, need[n] = the sum (saturating far above any pool).
__device__ __forceinline__ int prefix_in_place(int* need, int n, int* warp_sums) {
    int run = 0;
    for (int base = 0; base < n; base += CACHE_PLAN_THREADS) {
        const int i = base + threadIdx.x;
        const int v = i < n ? need[i] : 0;
        int total;
        const int before = block_scan(v, warp_sums, total);
        if (i < n) need[i] = run + before;
        run = (int)min((long long)run + total, 1ll << 30);
    }
    __syncthreads();
    if (threadIdx.x == 0) need[n] = run;
    __syncthreads();
    return run;
}

// The last i of [0, n) with prefix[i] <= rank (skipping the empty ones before it).
__device__ __forceinline__ int owner_of(const int* prefix, int n, int rank) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= rank)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

struct CacheMetaParams {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int slots, max_pages, num_pages, page;
};

// Room for n_new[b] more tokens of each sequence: start[b] = its old length (where they go), or -1 for all when the
// call cannot be granted.
__global__ void __launch_bounds__(CACHE_PLAN_THREADS)
    cache_extend_kernel(const CacheMetaParams m, const int32_t* rows, const int32_t* n_new, int32_t* start, int batch) {
    extern __shared__ int sm[];
    int* need = sm;               // [batch + 1]
    uint32_t* seen = reinterpret_cast<uint32_t*>(sm + batch + 1);  // a bit per slot
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x;
    for (int i = tid; i < (m.slots + 31) / 32; i += CACHE_PLAN_THREADS) seen[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < batch; b += CACHE_PLAN_THREADS) {
        const int r = rows ? rows[b] : b;
        const int n = n_new[b];
        int k = 0;
        if (r < 0 || r >= m.slots || n < 0) {
            bad = true;
        } else {
            const uint32_t bit = 1u << (r & 31);
            if (atomicOr(&seen[r >> 5], bit) & bit) bad = true;
            const int l = m.lens[r];
            const long long last = ((long long)l + n + m.page - 1) / m.page;
            if (l < 0 || last > m.max_pages)
                bad = true;
            else
                k = (int)last - (l + m.page - 1) / m.page;
        }
        need[b] = k;
    }
    bad = __syncthreads_or(bad);
    const int want = prefix_in_place(need, batch, warp_sums);
    if (!bad) bad = !enough_free(m.refs, m.num_pages, want, warp_sums);
    if (bad) {
        if (tid == 0) set_error(TBIK_ERR_PAGE);
        for (int b = tid; b < batch; b += CACHE_PLAN_THREADS) start[b] = -1;
        return;
    }
    // each_free's barriers order its reads of refs before the next chunk only; a page's own thread changes it
    each_free(m.refs, m.num_pages, want, warp_sums, [&](int rank, int id) {
        const int b = owner_of(need, batch, rank);
        const int r = rows ? rows[b] : b;
        const int have = (m.lens[r] + m.page - 1) / m.page;
        m.table[(size_t)r * m.max_pages + have + (rank - need[b])] = id;
        m.refs[id] = 1;
    });
    __syncthreads();  // the lengths above are read before they change
    for (int b = tid; b < batch; b += CACHE_PLAN_THREADS) {
        const int r = rows ? rows[b] : b;
        const int l = m.lens[r];
        start[b] = l;
        m.lens[r] = l + n_new[b];
    }
}

// Page moves that a plan kernel leaves for cache_move_kernel: word 0 is their number, then (from, to) pairs.
__device__ __forceinline__ int2* move_list(int* ws) { return reinterpret_cast<int2*>(ws) + 1; }

// Whether the first n pages of a row are in use, a warp's lanes each for some of them (`lane` of `step`).
__device__ __forceinline__ bool pages_in_use(const CacheMetaParams& m, int row, int n, int lane, int step) {
    bool all = true;
    for (int j = lane; j < n; j += step) {
        const int id = m.table[(size_t)row * m.max_pages + j];
        all &= id >= 0 && id < m.num_pages && m.refs[id] > 0;
    }
    return all;
}

// For the plan kernels that look at many table entries: they run as a cluster whose blocks share the looking, and block 0
// goes on alone with the answer.  True in every thread of block 0 if some thread of the cluster has `bad`; the other
// blocks are done when this returns.
constexpr int CACHE_PLAN_CLUSTER = 8;
__device__ __forceinline__ bool plan_any(bool bad, uint32_t rank, uint32_t cl) {
    __shared__ uint32_t from[CACHE_PLAN_CLUSTER];
    bad = __syncthreads_or(bad);
    cluster_sync();  // block 0 runs: its memory may be written
    if (threadIdx.x == 0) st_cluster_u32(mapa_shared(smem_u32(&from[rank]), 0), bad);
    cluster_sync();
    if (rank == 0)
        for (uint32_t r = 0; r < cl; ++r) bad |= from[r] != 0;
    return bad;
}

// children[i] becomes a copy of parents[i]: full pages are shared, a page that is partly filled gets a copy, since
// both sequences will write into it.  Words 0 and 1 of ws: the number of copies and whether the call is granted.
// A warp per parent looks at its row (in a cluster of up to 8 blocks: 32 parents to a block), so that a row that names no
// page in use is found before anything changes; then one block plans.
__global__ void __launch_bounds__(CACHE_PLAN_THREADS)
    cache_fork_plan_kernel(const CacheMetaParams m, const int32_t* parents, const int32_t* children, int count, int* ws) {
    extern __shared__ int sm[];
    int* need = sm;  // [count + 1]
    uint32_t* child = reinterpret_cast<uint32_t*>(sm + count + 1);
    __shared__ int warp_sums[32];
    const int tid = threadIdx.x;
    uint32_t cl;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
    const uint32_t rank = cluster_rank();
    for (int i = tid; i < (m.slots + 31) / 32; i += CACHE_PLAN_THREADS) child[i] = 0;
    bool bad = false;
    for (int i = (int)rank * 32 + (tid >> 5); i < count; i += (int)cl * 32) {
        const int p = parents[i];
        if (p < 0 || p >= m.slots) continue;  // refused below, and so is a length that cannot be
        const int l = m.lens[p];
        if (l > 0) bad |= !pages_in_use(m, p, min(m.max_pages, (int)(((long long)l + m.page - 1) / m.page)), tid & 31, 32);
    }
    bad = plan_any(bad, rank, cl);
    if (rank != 0) return;
    for (int i = tid; i < count; i += CACHE_PLAN_THREADS) {
        const int p = parents[i], c = children[i];
        int k = 0;
        if (p < 0 || p >= m.slots || c < 0 || c >= m.slots) {
            bad = true;
        } else {
            const uint32_t bit = 1u << (c & 31);
            if (atomicOr(&child[c >> 5], bit) & bit) bad = true;
            const int l = m.lens[p];
            if (m.lens[c] != 0 || l < 0 || (long long)l > (long long)m.max_pages * m.page) bad = true;
            else
                k = l % m.page != 0;
        }
        need[i] = k;
    }
    bad = __syncthreads_or(bad);
    if (!bad)  // a row cannot be parent and child of one call
        for (int i = tid; i < count; i += CACHE_PLAN_THREADS) bad |= (child[parents[i] >> 5] >> (parents[i] & 31)) & 1u;
    bad = __syncthreads_or(bad);
    const int want = prefix_in_place(need, count, warp_sums);
    if (!bad) bad = !enough_free(m.refs, m.num_pages, want, warp_sums);
    if (tid == 0) {
        ws[0] = bad ? 0 : want;
        ws[1] = !bad;
        if (bad) set_error(TBIK_ERR_PAGE);
    }
    if (bad) return;
    int2* moves = move_list(ws);
    each_free(m.refs, m.num_pages, want, warp_sums, [&](int rank, int id) {
        const int i = owner_of(need, count, rank);
        const int p = parents[i], full = m.lens[p] / m.page;
        moves[rank] = make_int2(m.table[(size_t)p * m.max_pages + full], id);
        m.table[(size_t)children[i] * m.max_pages + full] = id;
        m.refs[id] = 1;
    });
}

// Compaction: the k-th live page at or behind index n = (number of live pages) moves to the k-th free index below n.
// Sources and targets are disjoint, so the copies need no order.  ws: count, n (-1 when refused), moves, then the new
// index of each moved page.  A cluster of 8 blocks first looks whether every page of every row is in use: a warp takes
// `per` slots at a time, few when there are few, and at most the 32 lengths that its lanes load at once.
__global__ void __launch_bounds__(CACHE_PLAN_THREADS)
    cache_compact_plan_kernel(const CacheMetaParams m, int32_t* live_out, int* ws) {
    __shared__ int warp_sums[32];
    __shared__ int n_live;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t cl;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
    const uint32_t rank = cluster_rank();
    const int warps = (int)cl * 32, per = min(32, (m.slots + warps - 1) / warps);
    bool bad = false;
    for (int r0 = ((int)rank * 32 + (tid >> 5)) * per; r0 < m.slots; r0 += warps * per) {
        const int l = lane < per && r0 + lane < m.slots ? m.lens[r0 + lane] : 0;
        bad |= l < 0 || (long long)l > (long long)m.max_pages * m.page;
        for (uint32_t some = __ballot_sync(0xffffffffu, l > 0); some; some &= some - 1) {
            const int k = __ffs((int)some) - 1, lk = __shfl_sync(0xffffffffu, l, k);
            bad |= !pages_in_use(m, r0 + k, min(m.max_pages, (int)(((long long)lk + m.page - 1) / m.page)), lane, 32);
        }
    }
    if (tid == 0) n_live = 0;
    bad = plan_any(bad, rank, cl);
    if (rank != 0) return;
    if (bad) {
        if (tid == 0) {
            set_error(TBIK_ERR_PAGE);
            ws[0] = 0;
            ws[1] = -1;
            live_out[0] = -1;
        }
        return;
    }
    int cnt = 0;
    for (int i = tid; 4 * i < m.num_pages; i += CACHE_PLAN_THREADS) {
        const int4 r = load_refs4(m.refs, i, m.num_pages, 0);
        cnt += (r.x != 0) + (r.y != 0) + (r.z != 0) + (r.w != 0);
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) atomicAdd(&n_live, cnt);
    __syncthreads();
    const int n = n_live;
    int2* moves = move_list(ws);
    int* map = ws + 2 + 2 * ((m.num_pages + 1) / 2);
    int holes = 0, highs = 0;
    for (int base = 0; base * 4 < m.num_pages; base += CACHE_PLAN_THREADS) {
        const int4 r = load_refs4(m.refs, base + tid, m.num_pages, 0);
        const int p0 = 4 * (base + tid);
        const int v[4] = {r.x, r.y, r.z, r.w};
        int ho = 0, hi = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            ho += p0 + q < n && v[q] == 0;
            hi += p0 + q >= n && v[q] != 0;
        }
        int th, ti;
        int rh = holes + block_scan(ho, warp_sums, th);
        int ri = highs + block_scan(hi, warp_sums, ti);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (p0 + q < n && v[q] == 0) moves[rh++].y = p0 + q;
            if (p0 + q >= n && v[q] != 0) moves[ri++].x = p0 + q;
        }
        holes += th;
        highs += ti;
    }
    __syncthreads();
    for (int i = tid; i < holes; i += CACHE_PLAN_THREADS) {
        const int2 mv = moves[i];
        map[mv.x] = mv.y;
        m.refs[mv.y] = m.refs[mv.x];
        m.refs[mv.x] = 0;
    }
    if (tid == 0) {
        ws[0] = holes;
        ws[1] = n;
        live_out[0] = n;
    }
}

// tbik_cache_copy: pages must be in range, targets distinct and none of them a source.
__global__ void __launch_bounds__(CACHE_PLAN_THREADS)
    cache_copy_plan_kernel(const int32_t* src, const int32_t* dst, int count, int num_pages, int* ws) {
    extern __shared__ uint32_t target[];
    const int tid = threadIdx.x;
    for (int i = tid; i < (num_pages + 31) / 32; i += CACHE_PLAN_THREADS) target[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < count; i += CACHE_PLAN_THREADS) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
            bad = true;
            continue;
        }
        const uint32_t bit = 1u << (d & 31);
        if (atomicOr(&target[d >> 5], bit) & bit) bad = true;
    }
    bad = __syncthreads_or(bad);
    if (!bad)
        for (int i = tid; i < count; i += CACHE_PLAN_THREADS) bad |= (target[src[i] >> 5] >> (src[i] & 31)) & 1u;
    bad = __syncthreads_or(bad);
    int2* moves = move_list(ws);
    if (!bad)
        for (int i = tid; i < count; i += CACHE_PLAN_THREADS) moves[i] = make_int2(src[i], dst[i]);
    if (tid == 0) {
        ws[0] = bad ? 0 : count;
        if (bad) set_error(TBIK_ERR_PAGE);
    }
}

struct CacheMoveParams {
    uint8_t* pages;
    float* scales;
    int planes;       // layers * 2
    int num_pages, kv_heads;
    int page_bytes;   // kv_heads * page * D
    const int* ws;
};

constexpr int CACHE_MOVE_THREADS = 256;
constexpr int CACHE_MOVE_BYTES = CACHE_MOVE_THREADS * 16 * 4;  // bytes of one step of a block

// The data of the moves in every layer's keys and values: blocks take 16 KB pieces in turn, four 16-byte loads in
// flight per thread.  Bound by HBM: 5.6 TB/s read and written for the moves of a pool of 2048 pages, 60 % live (4 layers,
// 8 heads of 128 dims, pages of 32: 47 us).
__device__ __forceinline__ void move_pages(const CacheMoveParams& p) {
    const int count = p.ws[0];
    const int2* moves = reinterpret_cast<const int2*>(p.ws) + 1;
    const int pieces = (p.page_bytes + CACHE_MOVE_BYTES - 1) / CACHE_MOVE_BYTES;
    const long long units = (long long)count * p.planes * pieces;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int piece = (int)(u % pieces);
        const long long r = u / pieces;
        const int plane = (int)(r % p.planes);
        const int2 mv = moves[r / p.planes];
        const size_t from = ((size_t)plane * p.num_pages + mv.x) * p.page_bytes, to = ((size_t)plane * p.num_pages + mv.y) * p.page_bytes;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int off = piece * CACHE_MOVE_BYTES + (i * CACHE_MOVE_THREADS + threadIdx.x) * 16;
            if (off < p.page_bytes) w[i] = *reinterpret_cast<const uint4*>(p.pages + from + off);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int off = piece * CACHE_MOVE_BYTES + (i * CACHE_MOVE_THREADS + threadIdx.x) * 16;
            if (off < p.page_bytes) *reinterpret_cast<uint4*>(p.pages + to + off) = w[i];
        }
        if (piece == 0)
            for (int h = threadIdx.x; h < p.kv_heads; h += CACHE_MOVE_THREADS)
                p.scales[((size_t)plane * p.num_pages + mv.y) * p.kv_heads + h] =
                    p.scales[((size_t)plane * p.num_pages + mv.x) * p.kv_heads + h];
    }
}

__global__ void __launch_bounds__(CACHE_MOVE_THREADS) cache_move_kernel(const CacheMoveParams p) { move_pages(p); }

// The second kernel of a fork: the children's rows, the shared pages' counts, and the copies.
__global__ void __launch_bounds__(CACHE_MOVE_THREADS)
    cache_fork_kernel(const CacheMoveParams p, const CacheMetaParams m, const int32_t* parents, const int32_t* children,
                      int count) {
    if (!p.ws[1]) return;
    for (int i = blockIdx.x; i < count; i += gridDim.x) {
        const int par = parents[i], c = children[i], l = m.lens[par], full = l / m.page;
        for (int j = threadIdx.x; j < full; j += CACHE_MOVE_THREADS) {
            const int id = m.table[(size_t)par * m.max_pages + j];  // in use: the plan has looked
            m.table[(size_t)c * m.max_pages + j] = id;
            atomicAdd(&m.refs[id], 1);
        }
        if (threadIdx.x == 0) m.lens[c] = l;
    }
    move_pages(p);
}

// The second kernel of a compaction: table entries of moved pages, and the copies.
__global__ void __launch_bounds__(CACHE_MOVE_THREADS) cache_compact_kernel(const CacheMoveParams p, const CacheMetaParams m) {
    const int n = p.ws[1];
    if (n < 0) return;
    const int* map = p.ws + 2 + 2 * ((m.num_pages + 1) / 2);
    const long long entries = (long long)m.slots * m.max_pages;
    for (long long e = (long long)blockIdx.x * CACHE_MOVE_THREADS + threadIdx.x; e < entries; e += (long long)gridDim.x * CACHE_MOVE_THREADS) {
        const int id = m.table[e];
        if (id < n) continue;  // below the front, or none
        const int r = (int)(e / m.max_pages), j = (int)(e % m.max_pages);
        if (j >= (m.lens[r] + m.page - 1) / m.page) continue;
        m.table[e] = map[id];  // in use: the plan has looked
    }
    move_pages(p);
}

// Every block looks at all of the call's slots before it empties any, so that a slot out of range leaves the others
// alone; the grid is bounded, so that the looks stay in proportion to the call (128 threads read 8192 slots in 64 steps).
// Taking the length out by an exchange makes a row that is named twice give up its pages once.
__global__ void __launch_bounds__(128) cache_free_kernel(const CacheMetaParams m, const int32_t* rows, int batch) {
    __shared__ int len;
    bool bad = false;
    if (rows)
        for (int b = threadIdx.x; b < batch; b += 128) bad |= rows[b] < 0 || rows[b] >= m.slots;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_error(TBIK_ERR_PAGE);
        return;
    }
    for (int b = blockIdx.x; b < batch; b += gridDim.x) {
        const int r = rows ? rows[b] : b;
        __syncthreads();  // the length of the sequence before has been read
        if (threadIdx.x == 0) len = atomicExch(&m.lens[r], 0);
        __syncthreads();
        int used = (int)(((long long)max(len, 0) + m.page - 1) / m.page);
        if (used > m.max_pages) used = m.max_pages;
        for (int j = threadIdx.x; j < used; j += 128) {
            int32_t* e = &m.table[(size_t)r * m.max_pages + j];
            const int id = *e;
            *e = -1;
            if (id < 0 || id >= m.num_pages || atomicSub(&m.refs[id], 1) <= 0) {
                if (id >= 0 && id < m.num_pages) atomicAdd(&m.refs[id], 1);
                set_error(TBIK_ERR_PAGE);
            }
        }
    }
}

}  // namespace tbik

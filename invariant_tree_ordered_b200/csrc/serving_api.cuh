// Host side of the cache, its attention and the sampling: argument checks and launches.  Included at the end of
// tbik_api.cu, whose helpers and device error word it shares.
#pragma once

namespace {

struct CacheShape {
    int slots, max_pages, num_pages, kv_heads, head_dim, page;
};

tbik_status check_meta(int batch, int slots, int max_pages, int num_pages, int page) {
    if (batch < 0 || slots <= 0 || max_pages <= 0 || num_pages <= 0) return TBIK_ERR_ARG;
    if (page != 16 && page != 32 && page != 64 && page != 128) return TBIK_ERR_SHAPE;
    if (batch > CACHE_MAX_BATCH || slots > CACHE_MAX_SLOTS || num_pages > CACHE_MAX_PAGES || max_pages > CACHE_MAX_PAGES)
        return TBIK_ERR_SHAPE;
    return TBIK_OK;
}

tbik_status check_data(int layers, int num_pages, int kv_heads, int head_dim, int page) {
    if (layers <= 0 || kv_heads <= 0) return TBIK_ERR_ARG;
    if (head_dim != 64 && head_dim != 128) return TBIK_ERR_SHAPE;
    if (kv_heads > 65535 || (long long)kv_heads * page * head_dim > (1 << 30) || layers > (1 << 20)) return TBIK_ERR_SHAPE;
    return check_meta(0, 1, 1, num_pages, page);
}

CacheMetaParams meta_params(int32_t* table, const int32_t* lens, int32_t* refs, int slots, int max_pages, int num_pages, int page) {
    CacheMetaParams m;
    m.table = table, m.lens = const_cast<int32_t*>(lens), m.refs = refs;
    m.slots = slots, m.max_pages = max_pages, m.num_pages = num_pages, m.page = page;
    return m;
}

CacheMoveParams move_params(uint8_t* pages, float* scales, int layers, int num_pages, int kv_heads, int head_dim, int page, void* ws) {
    CacheMoveParams p;
    p.pages = pages, p.scales = scales, p.planes = 2 * layers, p.num_pages = num_pages, p.kv_heads = kv_heads;
    p.page_bytes = kv_heads * page * head_dim;
    p.ws = reinterpret_cast<const int*>(ws);
    return p;
}

// Scales are read one by one, and one layer of a pool's scales starts at any multiple of 4 bytes.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shared memory of a plan kernel: prefix sums over the call's sequences and a bit per slot.
size_t plan_smem(int count, int slots) { return ((size_t)count + 1) * 4 + ((size_t)slots + 31) / 32 * 4; }

// A plan kernel as one cluster of `blocks` blocks.
template <typename... P, typename... A>
tbik_status launch_plan(void (*kernel)(P...), int blocks, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(CACHE_PLAN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) return TBIK_ERR_CUDA;
    return launch_status();
}

// Blocks of a kernel that walks over page data: eight of 256 threads fill an SM.
int move_grid(const DeviceInfo* info, long long most) {
    const long long full = (long long)info->sms * 8;
    return (int)(most < 1 ? 1 : most < full ? most : full);
}

template <int D, int THREADS, int CH, int GROUPS>
void launch_append(const CacheAppendParams& p, const DeviceInfo* info, cudaStream_t s) {
    long long x = GROUPS > 1 ? (p.batch + GROUPS - 1) / GROUPS : p.tokens / p.page + 2 * p.batch;
    if (!p.rows) {
        cache_append_kernel<D, THREADS, CH, GROUPS, false><<<dim3((unsigned)x, p.kv_heads, 2), THREADS * GROUPS, 0, s>>>(p);
        return;
    }
    const long long most = (2048 / (THREADS * GROUPS) * (long long)info->sms + 2 * p.kv_heads - 1) / (2 * p.kv_heads);
    const bool maps = GROUPS > 1 || p.batch > APPEND_FEW * THREADS;
    if (maps && x > most) x = most;
    cache_append_kernel<D, THREADS, CH, GROUPS, true>
        <<<dim3((unsigned)x, p.kv_heads, 2), THREADS * GROUPS, maps ? ((size_t)p.slots + 31) / 32 * 8 : 0, s>>>(p);
}

template <int D>
void dispatch_append(const CacheAppendParams& p, const DeviceInfo* info, cudaStream_t s) {
    if (!p.cu) return launch_append<D, 32, 1, 8>(p, info, s);
    switch (p.page * D / 8 / 128) {
        case 1: return launch_append<D, 128, 1, 1>(p, info, s);
        case 2: return launch_append<D, 128, 2, 1>(p, info, s);
        case 4: return launch_append<D, 128, 4, 1>(p, info, s);
        case 8: return launch_append<D, 128, 8, 1>(p, info, s);
        default: return launch_append<D, 256, 8, 1>(p, info, s);
    }
}

tbik_status check_attention(int tokens, int batch, int max_q, int max_keys, int heads, int kv_heads, int head_dim, int page) {
    if (tokens < 0 || batch < 0 || max_q <= 0 || max_keys <= 0 || heads <= 0 || kv_heads <= 0) return TBIK_ERR_ARG;
    if (heads % kv_heads || heads / kv_heads > 64 || kv_heads > 65535) return TBIK_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return TBIK_ERR_SHAPE;
    if (batch > CACHE_MAX_BATCH || max_keys > (1 << 26)) return TBIK_ERR_SHAPE;
    return check_meta(batch, 1, 1, 1, page);
}

// Rows of a tile, grid and workspace of an attention call.
struct CattSplit {
    int rows;    // rows per tile: 8, 16 or 32
    int grid, slots;
    size_t off_tiles, off_ms, off_o, bytes;
};

tbik_status plan_cache_attention(int tokens, int batch, int max_q, int max_keys, int heads, int kv_heads, int head_dim,
                                 int sms, CattSplit& c) {
    memset(&c, 0, sizeof(c));
    if (tokens == 0 || batch == 0) return TBIK_OK;
    const int group = heads / kv_heads;
    // Rows of a sequence that share a kv head: at most, or where max_q says nothing (every sequence could have all tokens), on
    // average.  Any tile gives the same bits.  24 sequences of 1 to 5 tokens and 16 heads, max_q left at its default: 43 us
    // in tiles of 8, 82 us in tiles of 32.
    const long long most = (long long)(max_q < tokens ? max_q : (tokens + batch - 1) / batch) * group;
    // The smallest tile that holds them, up to 32.  32 sequences of 8192 keys, 4 kv heads of 128 dims: 8 rows 78 us in
    // tiles of 8 and 88 us in tiles of 16; 16 rows 61 us in tiles of 16, 76 us in tiles of 32 and 74 us in two of 8;
    // 32 rows 125 us, 150 us in two tiles of 16.  (Tiles of 64 rows by eight warps in one block an SM instead of
    // four warps in two were slower: 512 rows 1370 us against 1290 us.)
    c.rows = most <= 8 ? 8 : most <= 16 ? 16 : 32;
    // blocks of 128 positions that hold tokens: a sequence's touch one more than they fill, and each holds one
    const long long items = (long long)batch * (((max_q < tokens ? max_q : tokens) + 126) / 128 + 1);
    const int ctas = c.rows == 8 ? 3 : 2;
    const long long leaves = (max_keys + CATT_LEAF - 1) / CATT_LEAF;
    // tiles: one for each of the blocks where a block's rows fit one, else a full one for every c.rows rows and one more for
    // each block
    const long long held = items < tokens ? items : tokens, rows = (long long)(max_q < 128 ? max_q : 128) * group;
    const long long tiles = kv_heads * (rows <= c.rows ? held : ((long long)tokens * group + held * (c.rows - 1)) / c.rows);
    const long long work = tiles * leaves;
    const long long full = (long long)sms * ctas;
    c.grid = (int)(work < full ? work : full);
    if (leaves > 1) {
        // a cut tile of L leaves has fewer than 2 L / T nodes; T is at least all leaves / (grid * CATT_UNITS), or the
        // kernel's cap (CattCfg::MAX_NODE)
        const long long by_grid = 2ll * c.grid * CATT_UNITS, by_cap = 2 * work / (c.rows == 32 ? CattCfg<128, 32>::MAX_NODE : CattCfg<128, 8>::MAX_NODE);
        static_assert(CattCfg<128, 8>::MAX_NODE == CattCfg<128, 16>::MAX_NODE && CattCfg<64, 32>::MAX_NODE == CattCfg<128, 32>::MAX_NODE, "caps");
        long long slots = by_grid > by_cap ? by_grid : by_cap;
        if (slots > 2 * work) slots = 2 * work;
        slots += 2;
        if (slots * c.rows > (1ll << 30)) return TBIK_ERR_SHAPE;
        c.slots = (int)slots;
        c.off_tiles = 256;
        c.off_ms = c.off_tiles + (size_t)(slots / 2) * 32;
        c.off_o = (c.off_ms + (size_t)slots * c.rows * 8 + 255) / 256 * 256;
        c.bytes = c.off_o + (size_t)slots * c.rows * head_dim * 4;
    }
    return TBIK_OK;
}

template <int D, int R>
tbik_status launch_cache_attention(const CacheAttParams& p, const CattSplit& c, const DeviceInfo* info, int dev, cudaStream_t s) {
    using C = CattCfg<D, R>;
    static bool ready[kMaxDevices];
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!ready[dev]) {
            if (cudaFuncSetAttribute(cache_attention_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
                return TBIK_ERR_CUDA;
            ready[dev] = true;
        }
    }
    cache_attention_kernel<D, R><<<c.grid, C::THREADS, C::SMEM, s>>>(p);
    tbik_status st = launch_status();
    if (st != TBIK_OK || !c.slots) return st;
    // the second kernel's blocks may be set up while the first one ends; they wait for its results themselves
    cudaLaunchConfig_t cfg = {};
    const long long rows = (long long)(c.slots / 2) * c.rows, full = (long long)info->sms * 8;
    cfg.gridDim = dim3((unsigned)(rows < full ? rows : full));
    cfg.blockDim = dim3(CATT_JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<D, R>, p) != cudaSuccess) return TBIK_ERR_CUDA;
    return launch_status();
}

template <int D>
tbik_status dispatch_cache_attention(const CacheAttParams& p, const CattSplit& c, const DeviceInfo* info, int dev, cudaStream_t s) {
    switch (c.rows) {
        case 8: return launch_cache_attention<D, 8>(p, c, info, dev, s);
        case 16: return launch_cache_attention<D, 16>(p, c, info, dev, s);
        default: return launch_cache_attention<D, 32>(p, c, info, dev, s);
    }
}

template <typename T>
tbik_status launch_sample(SampleParams& p, const DeviceInfo* info, int dev, cudaStream_t s) {
    // Blocks per row: as few as hold the row in 80 KB each, more (up to 8) while the device holds all of them at once (two
    // to an SM) and a block has at least 4096 tokens.
    // 97 rows of 32000 in bf16: 37 us with one block each, 33 us with two, 39 us with four; 40 rows of 20000: 31 us with
    // two, 29 us with four, 33 us with eight.
    int cl = 1;
    while (cl < SMP_MAX_CLUSTER && ((long long)p.vocab * (int)sizeof(T) > 80000LL * cl ||
                                    ((long long)p.batch * cl <= info->sms && p.vocab > 4096 * cl)))
        cl *= 2;
    p.seg = ((p.vocab + cl - 1) / cl + 15) / 16 * 16;
    const size_t smem = (size_t)p.seg * sizeof(T) + 32;
    static bool ready[kMaxDevices];
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!ready[dev]) {
            if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     SMP_MAX_SEG * (int)sizeof(T) + 32) != cudaSuccess)
                return TBIK_ERR_CUDA;
            ready[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * cl));
    cfg.blockDim = dim3(SMP_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sample_kernel<T>, (const SampleParams)p) != cudaSuccess) return TBIK_ERR_CUDA;
    return launch_status();
}

}  // namespace

extern "C" {

tbik_status tbik_cache_extend(int32_t* table, int32_t* lens, int32_t* refs, const int32_t* rows, const int32_t* n_new,
                              int32_t* start, int batch, int slots, int max_pages, int num_pages, int page, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_meta(batch, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if (!rows && batch > slots) return TBIK_ERR_SHAPE;
    if (batch == 0) return TBIK_OK;
    if (!table || !lens || !refs || !n_new || !start) return TBIK_ERR_ARG;
    if (!aligned16(refs)) return TBIK_ERR_ALIGN;
    cache_extend_kernel<<<1, CACHE_PLAN_THREADS, plan_smem(batch, slots), reinterpret_cast<cudaStream_t>(stream)>>>(
        meta_params(table, lens, refs, slots, max_pages, num_pages, page), rows, n_new, start, batch);
    return launch_status();
}

size_t tbik_cache_fork_workspace(int count) {
    return count < 0 || count > CACHE_MAX_BATCH ? (size_t)-1 : ((size_t)count + 1) * 8;
}

tbik_status tbik_cache_fork(uint8_t* pages, float* scales, int32_t* table, int32_t* lens, int32_t* refs,
                            const int32_t* parents, const int32_t* children, int count, int layers, int slots,
                            int max_pages, int num_pages, int kv_heads, int head_dim, int page, void* ws,
                            size_t ws_bytes, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_meta(count, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if ((st = check_data(layers, num_pages, kv_heads, head_dim, page)) != TBIK_OK) return st;
    if (count == 0) return TBIK_OK;
    if (!pages || !scales || !table || !lens || !refs || !parents || !children) return TBIK_ERR_ARG;
    if (!aligned16(pages) || !aligned4(scales) || !aligned16(refs) || (ws && !aligned16(ws))) return TBIK_ERR_ALIGN;
    if (!ws || ws_bytes < tbik_cache_fork_workspace(count)) return TBIK_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const CacheMetaParams m = meta_params(table, lens, refs, slots, max_pages, num_pages, page);
    const CacheMoveParams p = move_params(pages, scales, layers, num_pages, kv_heads, head_dim, page, ws);
    int blocks = 1;
    while (blocks < CACHE_PLAN_CLUSTER && 32 * blocks < count) blocks *= 2;
    st = launch_plan(cache_fork_plan_kernel, blocks, plan_smem(count, slots), s, m, parents, children, count, reinterpret_cast<int*>(ws));
    if (st != TBIK_OK) return st;
    const long long most = (long long)count * p.planes * ((p.page_bytes + CACHE_MOVE_BYTES - 1) / CACHE_MOVE_BYTES);
    cache_fork_kernel<<<move_grid(info, most), CACHE_MOVE_THREADS, 0, s>>>(p, m, parents, children, count);
    return launch_status();
}

tbik_status tbik_cache_free(int32_t* table, int32_t* lens, int32_t* refs, const int32_t* rows, int batch, int slots,
                            int max_pages, int num_pages, int page, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_meta(batch, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if (!rows && batch > slots) return TBIK_ERR_SHAPE;
    if (batch == 0) return TBIK_OK;
    if (!table || !lens || !refs) return TBIK_ERR_ARG;
    cache_free_kernel<<<move_grid(info, batch), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        meta_params(table, lens, refs, slots, max_pages, num_pages, page), rows, batch);
    return launch_status();
}

size_t tbik_cache_compact_workspace(int num_pages) {
    if (num_pages <= 0 || num_pages > CACHE_MAX_PAGES) return (size_t)-1;
    return (2 + 2 * (((size_t)num_pages + 1) / 2) + (size_t)num_pages) * 4;
}

tbik_status tbik_cache_compact(uint8_t* pages, float* scales, int32_t* table, const int32_t* lens, int32_t* refs,
                               int32_t* live, int layers, int slots, int max_pages, int num_pages, int kv_heads,
                               int head_dim, int page, void* ws, size_t ws_bytes, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_meta(0, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if ((st = check_data(layers, num_pages, kv_heads, head_dim, page)) != TBIK_OK) return st;
    if (!pages || !scales || !table || !lens || !refs || !live) return TBIK_ERR_ARG;
    if (!aligned16(pages) || !aligned4(scales) || !aligned16(refs) || (ws && !aligned16(ws))) return TBIK_ERR_ALIGN;
    if (!ws || ws_bytes < tbik_cache_compact_workspace(num_pages)) return TBIK_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const CacheMetaParams m = meta_params(table, lens, refs, slots, max_pages, num_pages, page);
    const CacheMoveParams p = move_params(pages, scales, layers, num_pages, kv_heads, head_dim, page, ws);
    st = launch_plan(cache_compact_plan_kernel, slots > 32 ? CACHE_PLAN_CLUSTER : 1, 0, s, m, live, reinterpret_cast<int*>(ws));
    if (st != TBIK_OK) return st;
    const long long most = (long long)(num_pages / 2 + 1) * p.planes * ((p.page_bytes + CACHE_MOVE_BYTES - 1) / CACHE_MOVE_BYTES);
    cache_compact_kernel<<<move_grid(info, most), CACHE_MOVE_THREADS, 0, s>>>(p, m);
    return launch_status();
}

tbik_status tbik_cache_copy(uint8_t* pages, float* scales, const int32_t* src, const int32_t* dst, int count, int layers,
                            int num_pages, int kv_heads, int head_dim, int page, void* ws, size_t ws_bytes, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_meta(count, 1, 1, num_pages, page)) != TBIK_OK) return st;
    if ((st = check_data(layers, num_pages, kv_heads, head_dim, page)) != TBIK_OK) return st;
    if (count == 0) return TBIK_OK;
    if (!pages || !scales || !src || !dst) return TBIK_ERR_ARG;
    if (!aligned16(pages) || !aligned4(scales) || (ws && !aligned16(ws))) return TBIK_ERR_ALIGN;
    if (!ws || ws_bytes < tbik_cache_fork_workspace(count)) return TBIK_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = ((size_t)num_pages + 31) / 32 * 4;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(cache_copy_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CACHE_MAX_PAGES / 8) != cudaSuccess)
        return TBIK_ERR_CUDA;
    const CacheMoveParams p = move_params(pages, scales, layers, num_pages, kv_heads, head_dim, page, ws);
    cache_copy_plan_kernel<<<1, CACHE_PLAN_THREADS, smem, s>>>(src, dst, count, num_pages, reinterpret_cast<int*>(ws));
    if ((st = launch_status()) != TBIK_OK) return st;
    const long long most = (long long)count * p.planes * ((p.page_bytes + CACHE_MOVE_BYTES - 1) / CACHE_MOVE_BYTES);
    cache_move_kernel<<<move_grid(info, most), CACHE_MOVE_THREADS, 0, s>>>(p);
    return launch_status();
}

tbik_status tbik_cache_append(const uint16_t* k, const uint16_t* v, uint8_t* pages, float* scales, const int32_t* table,
                              const int32_t* refs, const int32_t* start, const int32_t* cu, const int32_t* rows,
                              int tokens, int batch, int slots, int max_pages, int num_pages, int kv_heads, int head_dim,
                              int page, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if (tokens < 0) return TBIK_ERR_ARG;
    if ((st = check_meta(batch, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if ((st = check_data(1, num_pages, kv_heads, head_dim, page)) != TBIK_OK) return st;
    if ((!cu && tokens != batch) || (!rows && batch > slots)) return TBIK_ERR_SHAPE;
    if (tokens == 0 || batch == 0) return TBIK_OK;
    if (!k || !v || !pages || !scales || !table || !refs || !start) return TBIK_ERR_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(pages) || !aligned4(scales)) return TBIK_ERR_ALIGN;
    CacheAppendParams p;
    p.k = k, p.v = v, p.pages = pages, p.scales = scales, p.table = table, p.refs = refs, p.start = start;
    p.cu = cu, p.rows = rows, p.tokens = tokens, p.batch = batch, p.slots = slots, p.max_pages = max_pages;
    p.num_pages = num_pages, p.kv_heads = kv_heads, p.page = page;
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    if (head_dim == 128)
        dispatch_append<128>(p, info, reinterpret_cast<cudaStream_t>(stream));
    else
        dispatch_append<64>(p, info, reinterpret_cast<cudaStream_t>(stream));
    return launch_status();
}

size_t tbik_cache_attention_workspace(int tokens, int batch, int max_q, int max_keys, int heads, int kv_heads,
                                      int head_dim, int page) {
    int dev;
    DeviceInfo* info;
    if (device_info(dev, info) != TBIK_OK) return (size_t)-1;
    if (check_attention(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, page) != TBIK_OK) return (size_t)-1;
    CattSplit c;
    if (plan_cache_attention(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, info->sms, c) != TBIK_OK) return (size_t)-1;
    return c.bytes;
}

tbik_status tbik_cache_attention(const uint16_t* q, const uint8_t* pages, const float* scales, const int32_t* table,
                                 const int32_t* start, const int32_t* cu, const int32_t* rows, uint16_t* out, int tokens,
                                 int batch, int slots, int max_pages, int num_pages, int heads, int kv_heads, int head_dim,
                                 int page, int max_q, int max_keys, void* ws, size_t ws_bytes, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if ((st = check_attention(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, page)) != TBIK_OK) return st;
    if ((st = check_meta(batch, slots, max_pages, num_pages, page)) != TBIK_OK) return st;
    if ((!cu && tokens != batch) || (!rows && batch > slots)) return TBIK_ERR_SHAPE;
    CattSplit c;
    if ((st = plan_cache_attention(tokens, batch, max_q, max_keys, heads, kv_heads, head_dim, info->sms, c)) != TBIK_OK) return st;
    if (tokens == 0 || batch == 0) return TBIK_OK;
    if (!q || !pages || !scales || !table || !start || !out) return TBIK_ERR_ARG;
    if (!aligned16(q) || !aligned16(pages) || !aligned4(scales) || !aligned16(out)) return TBIK_ERR_ALIGN;
    if (c.bytes && (!ws || ws_bytes < c.bytes)) return TBIK_ERR_WORKSPACE;
    if (c.bytes && !aligned16(ws)) return TBIK_ERR_ALIGN;
    CacheAttParams p;
    memset(&p, 0, sizeof(p));
    p.q = q, p.pages = pages, p.scales = scales, p.table = table, p.start = start, p.cu = cu, p.rows = rows, p.out = out;
    p.tokens = tokens, p.batch = batch, p.slots = slots, p.max_pages = max_pages, p.num_pages = num_pages;
    p.heads = heads, p.kv_heads = kv_heads, p.page = page, p.max_q = max_q, p.max_keys = max_keys;
    p.group = heads / kv_heads;
    p.group_inv = ((1u << 31) + (unsigned)p.group - 1) / (unsigned)p.group;
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    p.scale = (float)(1.4426950408889634 / std::sqrt((double)head_dim));
    if (c.slots) {
        uint8_t* w = reinterpret_cast<uint8_t*>(ws);
        p.count = reinterpret_cast<int*>(w);
        p.tiles = reinterpret_cast<int4*>(w + c.off_tiles);
        p.ms = reinterpret_cast<float2*>(w + c.off_ms);
        p.o = reinterpret_cast<float*>(w + c.off_o);
        p.max_slots = c.slots;
    }
    p.wait_cycles = wait_cycles(info);
    p.debug = g_debug_flags;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return head_dim == 128 ? dispatch_cache_attention<128>(p, c, info, dev, s) : dispatch_cache_attention<64>(p, c, info, dev, s);
}

tbik_status tbik_sample(const void* logits, const float* u, const float* temperature, const int32_t* top_k,
                        const float* top_p, const float* min_p, int32_t* out, int batch, int vocab, int bf16, void* stream) {
    int dev;
    DeviceInfo* info;
    tbik_status st = device_info(dev, info);
    if (st != TBIK_OK) return st;
    if (batch < 0 || vocab <= 0) return TBIK_ERR_ARG;
    if (vocab > SMP_MAX_SEG * SMP_MAX_CLUSTER || batch > (1 << 24)) return TBIK_ERR_SHAPE;
    if (batch == 0) return TBIK_OK;
    if (!logits || !u || !out) return TBIK_ERR_ARG;
    if (!aligned16(logits)) return TBIK_ERR_ALIGN;
    SampleParams p;
    p.logits = logits, p.u = u, p.temperature = temperature, p.top_k = top_k, p.top_p = top_p, p.min_p = min_p;
    p.out = out, p.batch = batch, p.vocab = vocab;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return bf16 ? launch_sample<uint16_t>(p, info, dev, s) : launch_sample<float>(p, info, dev, s);
}

}  // extern "C"

// paged_api.cuh -- host side of the paged key/value cache: argument checks and
// launches of attn_paged_tables, attn_paged_append and attn_paged_fwd.  Included
// by attn_api.cu, whose helpers it uses.
#pragma once

namespace {

// Bytes from the first to one past the last element of a cache.
size_t cache_extent(int n_pages, int page_size, int Hkv, int D, long long ps, long long ts, long long hs) {
    return ((size_t)(n_pages - 1) * ps + (size_t)(page_size - 1) * ts + (size_t)(Hkv - 1) * hs + D) * 2;
}

// Do the three strides lay the cache's rows (of `row` units, every stride a multiple of
// `step`) out without overlap?  Each axis, from the one with the smallest stride up, has to
// step over all that lies below it.  The stride of an axis of one has no meaning and becomes
// `row`.
bool layout_ok(int n_pages, int page_size, int Hkv, int row, int step, long long& ps, long long& ts, long long& hs) {
    if (n_pages == 1) ps = row;
    if (page_size == 1) ts = row;
    if (Hkv == 1) hs = row;
    if (ps < 1 || ts < 1 || hs < 1 || ps % step != 0 || ts % step != 0 || hs % step != 0) return false;
    struct Axis {
        long long stride;
        int n;
    } a[3] = {{hs, Hkv}, {ts, page_size}, {ps, n_pages}};
    std::sort(a, a + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
    long long below = row;
    for (const Axis& x : a) {
        if (x.n == 1) continue;
        if (x.stride < below) return false;
        if (x.stride > (1ll << 60) / x.n) return false;
        below = x.stride * (x.n - 1) + below;
    }
    return true;
}
bool cache_layout_ok(int n_pages, int page_size, int Hkv, int D, long long& ps, long long& ts, long long& hs) {
    return layout_ok(n_pages, page_size, Hkv, D, 8, ps, ts, hs);
}

// Sizes of a cache and of what it is used with.
attn_status_t check_cache(int n_pages, int page_size, int Hkv, int D, long long& ps, long long& ts, long long& hs) {
    if (n_pages < 1 || page_size < 1 || Hkv < 1 || D < 1) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
    return cache_layout_ok(n_pages, page_size, Hkv, D, ps, ts, hs) ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

bool aligned(const void* ptr, size_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; }

// Shared-memory opt-in of the paged kernels, once per device.
template <bool kF16, int kD, int kNB>
bool opt_in_smem_rows() {
    return cudaFuncSetAttribute(attn::paged::paged_rows_kernel<kF16, kD, kNB>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                attn::paged::RowsGeo<kD, kNB>::kSmemBytes) == cudaSuccess;
}

template <bool kF16, int kD>
bool opt_in_smem_rows_all() {
    if constexpr (kD == 256) return opt_in_smem_rows<kF16, kD, 1>() && opt_in_smem_rows<kF16, kD, 2>();
    else if constexpr (kD == 128)
        return opt_in_smem_rows<kF16, kD, 1>() && opt_in_smem_rows<kF16, kD, 2>() && opt_in_smem_rows<kF16, kD, 3>();
    else return opt_in_smem_rows<kF16, kD, 1>() && opt_in_smem_rows<kF16, kD, 2>() &&
                opt_in_smem_rows<kF16, kD, 3>() && opt_in_smem_rows<kF16, kD, 4>();
}

template <bool kF16, int kD, bool kFold = false>
bool opt_in_smem_tiles() {
    return cudaFuncSetAttribute(attn::paged::paged_tiles_kernel<kF16, kD, kFold>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                attn::paged::TilesGeo<kD>::kSmemBytes) == cudaSuccess;
}

bool paged_device_setup(int dev, int* sm_count) {
    static std::mutex mu;
    static int sms[kMaxDevices] = {};
    if (dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (sms[dev] == 0) {
        int n = 0;
        if (!opt_in_smem_rows_all<false, 64>() || !opt_in_smem_rows_all<true, 64>() ||
            !opt_in_smem_rows_all<false, 128>() || !opt_in_smem_rows_all<true, 128>() ||
            !opt_in_smem_tiles<false, 64>() || !opt_in_smem_tiles<true, 64>() || !opt_in_smem_tiles<false, 128>() ||
            !opt_in_smem_tiles<true, 128>() || !opt_in_smem_tiles<false, 128, true>() ||
            !opt_in_smem_tiles<true, 128, true>() || !opt_in_smem_rows_all<false, 256>() || !opt_in_smem_rows_all<true, 256>() ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            return false;
        sms[dev] = n;
    }
    *sm_count = sms[dev];
    return true;
}

// The workspace's parts, for blocks of `rows` rows.
attn::paged::Workspace split_workspace(void* workspace, int sms, int rows) {
    using namespace attn::paged;
    char* at = static_cast<char*>(workspace);
    Workspace w;
    w.header = reinterpret_cast<PieceHeader*>(at);
    w.ml = reinterpret_cast<float2*>(at + ws_header_bytes(sms));
    w.o = reinterpret_cast<float*>(at + ws_header_bytes(sms) + ws_ml_bytes(sms, rows));
    return w;
}

// The tag of a launch that counts its pieces in a workspace of unknown contents: 48 bits
// of a product, so that they look like nothing a buffer is likely to hold.
unsigned long long next_tag() {
    static std::atomic<unsigned long long> launches{0};
    const unsigned long long tag = (launches.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9E3779B97F4A7C15ull >> 16;
    return tag != 0 ? tag : 1;
}

// Rows that the rows kernel computes together, in blocks of 8: as many as the registers hold
// (at head size 128 a fourth block spills: 32 rows 109 us, 24 rows 62 us, on the same cache).
// At 256 the second block spills too, 158 bytes, and still pays where the cache's bytes bound
// the call: 16 rows on 16 x 2000 to 6000 keys 117 us, as twice 8 rows 137 us, on 2 x 20000 keys
// 89 / 107 us.  Short and computing calls lose: on 1000 keys 23 / 14.5 us, 512 tokens on 8000
// keys 1616 / 1476 us.
int max_row_blocks(int D) { return D == 64 ? 4 : D == 128 ? 3 : 2; }
int row_blocks_for(long long rows, int D) {
    return static_cast<int>(std::min<long long>((rows + 7) / 8, max_row_blocks(D)));
}

// Launched so that its blocks are in place while the kernel before it in the stream still
// runs (if that one allows it); they wait for its end before they read or write anything.
template <class... Params, class... Args>
attn_status_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                            const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return ATTN_OK;
}

template <bool kF16, int kD, int kNB>
attn_status_t launch_rows(const attn::paged::PagedParams& p, void* workspace, int sms, cudaStream_t stream) {
    using namespace attn::paged;
    using G = RowsGeo<kD, kNB>;
    SchedParams sp{};
    sp.map = make_row_map(p.Hkv, p.group, G::kRows, 1);
    sp.ws = split_workspace(workspace, sms, G::kRows);
    sp.tag = next_tag();
    return launch_behind(paged_rows_kernel<kF16, kD, kNB>, dim3(sms), G::kThreads, G::kSmemBytes, stream, p, sp);
}

// Does a call take the tcgen05 kernel?  From more rows a key/value head on than the rows kernel
// computes together (16 sequences of 2000 to 6000 keys, rows / tiles kernel: 24 rows 62 / 63 us
// at head size 128, 32 rows 41 / 49 us at 64; 8 rows 45 / 61 and 29 / 48), where pages can be
// gathered in boxes of 16 rows or more and the head size has a kernel.
bool takes_tiles(long long rows, int D, int page_size) {
    return rows > 8 * max_row_blocks(D) && D <= 128 && page_size % 16 == 0;
}

size_t paged_workspace_bytes(int sms, long long rows, int D, int page_size) {
    return attn::paged::ws_bytes(sms, takes_tiles(rows, D, page_size) ? attn::kTiles * attn::kBM : 8 * row_blocks_for(rows, D), D);
}

// Tensor map of q: boxes of 64 columns x `heads` heads x `tokens` tokens.
bool encode_q_map(EncodeTiledFn fn, CUtensorMap* tm, bool f16, int D, const attn::paged::PagedParams& p, int heads, int tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens}, estr[3] = {1, 1, 1};
    return fn(tm, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF16, int kD>
attn_status_t launch_tiles(const attn::paged::PagedParams& p, long long rows, void* workspace, int sms,
                           cudaStream_t stream) {
    using namespace attn::paged;
    using T = TilesGeo<kD>;
    EncodeTiledFn fn = encoder();
    if (!fn) return ATTN_ERR_CUDA;
    SchedParams sp{};
    sp.map = make_row_map(p.Hkv, p.group, attn::kBM, attn::kTiles);
    sp.ws = split_workspace(workspace, sms, T::kRows);
    TilesParams tp{};
    tp.box_rows = 16;
    while (tp.box_rows < attn::kBN && p.page_size % (2 * tp.box_rows) == 0) tp.box_rows *= 2;
    tp.tile_tokens = sp.map.tokens / attn::kTiles;
    tp.q_rows = sp.map.heads * tp.tile_tokens;
    tp.poll_limit = kDefaultPollLimit;
    const CUtensorMapDataType type = kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapL2promotion promotion =
        kD == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    CUtensorMap tm[3];
    if (!encode_q_map(fn, &tm[0], kF16, kD, p, sp.map.heads, tp.tile_tokens)) return ATTN_ERR_CUDA;
    // K and V: boxes of box_rows rows.  A row of head size 128 is two 128-byte halves of a
    // swizzled tile, which a tensor map of (64 columns, row, head, page) copies apart.  With
    // the axes (64 columns, 8 rows, half, 8-row group, page) one box has both, and a head is
    // a step of the half axis where heads follow one another in a row, or of the group axis
    // where a head's rows of a page do.
    const bool by_half = p.head_stride == kD, by_group = p.head_stride == p.token_stride * p.page_size;
    const bool folded = kD == 128 && (by_half || by_group);
    tp.head_at_half = by_half ? 2 : 0;
    tp.head_at_group = by_half ? 0 : p.page_size / 8;
    const cuuint64_t heads = (cuuint64_t)p.Hkv, groups = (cuuint64_t)p.page_size / 8;
    const cuuint64_t hs = (cuuint64_t)p.head_stride * 2, ts = (cuuint64_t)p.token_stride * 2, ps = (cuuint64_t)p.page_stride * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)kD, heads, (cuuint64_t)p.page_size, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {hs, ts, ps};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)tp.box_rows, 1};
    const cuuint64_t fold_dims[5] = {64, 8, by_half ? 2 * heads : 2, by_half ? groups : groups * heads, (cuuint64_t)p.n_pages};
    const cuuint64_t fold_strides[4] = {ts, 128, 8 * ts, ps};
    const cuuint32_t fold_box[5] = {64, 8, 2, (cuuint32_t)tp.box_rows / 8, 1};
    const cuuint32_t estr5[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (fn(&tm[1 + i], type, folded ? 5 : 4, const_cast<uint16_t*>(i ? p.v : p.k), folded ? fold_dims : dims,
               folded ? fold_strides : strides, folded ? fold_box : box, estr5, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return ATTN_ERR_CUDA;
    auto kernel = paged_tiles_kernel<kF16, kD, false>;
    if constexpr (kD == 128)
        if (folded) kernel = paged_tiles_kernel<kF16, kD, true>;
    const attn_status_t st =
        launch_behind(kernel, dim3(sms), attn::kThreads, T::kSmemBytes, stream, tm[0], tm[1], tm[2], p, sp, tp);
    if (st != ATTN_OK) return st;
    // blocks for the rows that units are likely to have: most find nothing to join
    const int at_once = kCombineThreads / (kD / 4);
    const int parts = static_cast<int>((std::min<long long>(rows, T::kRows) + at_once - 1) / at_once);
    return launch_behind(paged_combine_kernel<kF16, kD, T::kRows, attn::kTiles>, dim3(sms, parts), kCombineThreads, 0,
                         stream, p, sp);
}

// The rows kernel's variant for sequences of at most `rows` rows.
template <bool kF16, int kD>
attn_status_t launch_rows_for(const attn::paged::PagedParams& p, long long rows, void* workspace, int sms,
                              cudaStream_t stream) {
    const int nb = row_blocks_for(rows, kD);
    if (nb == 1) return launch_rows<kF16, kD, 1>(p, workspace, sms, stream);
    if constexpr (kD != 256)
        if (nb == 3) return launch_rows<kF16, kD, 3>(p, workspace, sms, stream);
    if constexpr (kD == 64)
        if (nb == 4) return launch_rows<kF16, kD, 4>(p, workspace, sms, stream);
    return launch_rows<kF16, kD, 2>(p, workspace, sms, stream);
}

// Does a batch with long sequences have so many single tokens that they are worth a kernel of
// their own?  The lengths are on the device; on the host the longest sequence against the
// mean tells.  A row tile with one token in it takes a key tile about as fast as the cache
// can be read, and blocks that read overlap with blocks that compute, so the rows kernel in
// front pays late, and the sooner the longer the contexts.  One chunk of 100 to 700 among 20 to
// 200 tokens, all rows in tiles / shared, longest / mean in brackets: at head size 128, contexts
// of 500 to 3000 keys, 106 / 117 us (52), 149 / 154 (80), 182 / 185 (97), 224 / 216 (116), 285 /
// 269 (156); level at 63 with 2000 to 8000 keys, at 70 with 100 to 1000.  At 64, where a tile's
// step takes as long for half the bytes, 36 / 47 us (17), 60 / 62 (29), 86 / 80 (52), 122 / 101
// (80); with 2000 to 8000 keys 91 / 82 (17), 148 / 117 (29); with 100 to 1000 25 / 29 (17), 62 /
// 66 (63), 73 / 68 (80).
bool is_mixed(const attn::paged::PagedParams& p, int max_q_len, int D) {
    // of a batch padded with empty sequences no more have rows than there are rows beside the longest's
    const long long n = max_q_len < p.total_q ? std::min(p.n_seqs, p.total_q - max_q_len + 1) : p.n_seqs;
    return p.group <= 8 * max_row_blocks(D) && max_q_len * n >= (D == 64 ? 16ll : 96ll) * p.total_q;
}

template <bool kF16, int kD>
attn_status_t launch_paged(const attn::paged::PagedParams& p, int max_q_len, void* workspace, int sms, cudaStream_t stream) {
    const long long rows = (long long)max_q_len * p.group;
    if constexpr (kD != 256) {
        if (takes_tiles(rows, kD, p.page_size)) {
            attn::paged::PagedParams half = p;
            if (is_mixed(p, max_q_len, kD)) {
                half.split_rows = 8 * row_blocks_for(p.group, kD);
                half.take_short = 1;
                const attn_status_t st = launch_rows_for<kF16, kD>(half, p.group, workspace, sms, stream);
                if (st != ATTN_OK) return st;
                half.take_short = 0;
            }
            return launch_tiles<kF16, kD>(half, rows, workspace, sms, stream);
        }
    }
    return launch_rows_for<kF16, kD>(p, rows, workspace, sms, stream);
}

}  // namespace

extern "C" attn_status_t attn_paged_tables(const int* ctx_lens, const int* new_lens, int n_seqs, int page_size,
                                           const int* free_pages, int n_free, const int* free_head, int* block_table,
                                           int max_pages, long long table_stride, int* cu_new, int* kv_lens,
                                           long long* slot_map, int max_tokens, int* counts, cudaStream_t stream) {
    if (!ctx_lens || !new_lens || !block_table || !cu_new || !kv_lens || !slot_map || !counts) return ATTN_ERR_INVALID_ARG;
    if (n_seqs < 1 || page_size < 1 || n_free < 0 || max_pages < 1 || max_tokens < 1) return ATTN_ERR_INVALID_ARG;
    if (n_free > 0 && !free_pages) return ATTN_ERR_INVALID_ARG;
    if (table_stride < max_pages || table_stride > (1ll << 60) / n_seqs) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)ctx_lens, (const void*)new_lens, (const void*)free_pages, (const void*)free_head,
                            (const void*)block_table, (const void*)cu_new, (const void*)kv_lens, (const void*)counts})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(slot_map, 8)) return ATTN_ERR_INVALID_ARG;
    const void* out_p[5] = {block_table, cu_new, kv_lens, slot_map, counts};
    const size_t out_n[5] = {((size_t)(n_seqs - 1) * table_stride + max_pages) * 4, ((size_t)n_seqs + 1) * 4,
                             (size_t)n_seqs * 4, (size_t)max_tokens * 8, 16};
    const void* in_p[4] = {ctx_lens, new_lens, free_pages, free_head};
    const size_t in_n[4] = {(size_t)n_seqs * 4, (size_t)n_seqs * 4, (size_t)n_free * 4, free_head ? 4u : 0u};
    for (int a = 0; a < 5; ++a) {
        for (int c = 0; c < 4; ++c)
            if (in_n[c] > 0 && ranges_overlap(out_p[a], out_n[a], in_p[c], in_n[c])) return ATTN_ERR_INVALID_ARG;
        for (int c = a + 1; c < 5; ++c)
            if (ranges_overlap(out_p[a], out_n[a], out_p[c], out_n[c])) return ATTN_ERR_INVALID_ARG;
    }
    attn::paged::TableParams p{};
    p.ctx_lens = ctx_lens;
    p.new_lens = new_lens;
    p.free_pages = free_pages;
    p.free_head = free_head;
    p.table = block_table;
    p.cu_new = cu_new;
    p.kv_lens = kv_lens;
    p.counts = counts;
    p.slot_map = slot_map;
    p.table_stride = table_stride;
    p.n_seqs = n_seqs;
    p.n_free = n_free;
    p.max_pages = max_pages;
    p.max_tokens = max_tokens;
    p.page_size = page_size;
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    // one block per 1024 tokens, at most 128: each repeats the scan over the sequences
    const int blocks = std::min(128, (max_tokens + attn::paged::kTableThreads - 1) / attn::paged::kTableThreads);
    return launch_behind(attn::paged::paged_tables_kernel, dim3(blocks), attn::paged::kTableThreads, 0, stream, p);
}

extern "C" attn_status_t attn_paged_append(const void* k, const void* v, const long long* slot_map, void* k_cache,
                                           void* v_cache, int n_tokens, int Hkv, int D, int n_pages, int page_size,
                                           long long k_stride, long long v_stride, long long page_stride,
                                           long long token_stride, long long head_stride, cudaStream_t stream) {
    if (!k || !v || !slot_map || !k_cache || !v_cache || n_tokens < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = check_cache(n_pages, page_size, Hkv, D, page_stride, token_stride, head_stride);
    if (st != ATTN_OK) return st;
    const long long row = (long long)Hkv * D;
    for (long long stride : {k_stride, v_stride})
        if (stride % 8 != 0 || stride < row || stride > (1ll << 60) / n_tokens) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {k, v, (const void*)k_cache, (const void*)v_cache})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(slot_map, 8)) return ATTN_ERR_INVALID_ARG;
    // The caches overlap no row and no slot.  K and V of one interleaved tensor share an
    // address range without sharing an element, so the two caches are not compared.
    const size_t cache = cache_extent(n_pages, page_size, Hkv, D, page_stride, token_stride, head_stride);
    const void* in_p[3] = {k, v, slot_map};
    const size_t in_n[3] = {((size_t)(n_tokens - 1) * k_stride + row) * 2, ((size_t)(n_tokens - 1) * v_stride + row) * 2,
                            (size_t)n_tokens * 8};
    for (int c = 0; c < 3; ++c)
        if (ranges_overlap(k_cache, cache, in_p[c], in_n[c]) || ranges_overlap(v_cache, cache, in_p[c], in_n[c]))
            return ATTN_ERR_INVALID_ARG;
    if (k_cache == v_cache) return ATTN_ERR_INVALID_ARG;
    if (row / 8 > (1 << 24)) return ATTN_ERR_UNSUPPORTED;
    attn::paged::AppendParams p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_cache = static_cast<uint16_t*>(k_cache);
    p.v_cache = static_cast<uint16_t*>(v_cache);
    p.slot_map = slot_map;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.page_stride = page_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.n_slots = (long long)n_pages * page_size;
    p.T = n_tokens;
    p.row_chunks = static_cast<int>(row / 8);
    p.head_chunks_log2 = D == 64 ? 3 : D == 128 ? 4 : 5;
    p.per_block = std::max(1, attn::paged::kAppendThreads * 4 / p.row_chunks);
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    p.by_row = attn::paged::make_fastdiv(static_cast<unsigned int>(p.row_chunks));
    const unsigned int blocks = static_cast<unsigned int>(((long long)n_tokens + p.per_block - 1) / p.per_block);
    return launch_behind(attn::paged::paged_append_kernel, dim3(blocks), attn::paged::kAppendThreads, 0, stream, p);
}

extern "C" attn_status_t attn_paged_fwd_workspace_size(int total_q, int max_q_len, int Hq, int Hkv, int D, int page_size,
                                                       size_t* bytes) {
    if (!bytes) return ATTN_ERR_INVALID_ARG;
    *bytes = 0;
    if (total_q < 1 || max_q_len < 1 || page_size < 1 || Hq < 1 || Hkv < 1 || D < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
    if ((long long)total_q * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !paged_device_setup(dev, &sms)) return ATTN_ERR_CUDA;
    *bytes = paged_workspace_bytes(sms, (long long)max_q_len * (Hq / Hkv), D, page_size);
    return ATTN_OK;
}

extern "C" attn_status_t attn_paged_fwd(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                                        const int* block_table, const int* cu_q, const int* kv_lens, int n_seqs,
                                        int total_q, int max_q_len, int Hq, int Hkv, int D, int n_pages, int page_size,
                                        int max_pages, long long q_stride, long long table_stride,
                                        long long page_stride, long long token_stride, long long head_stride,
                                        int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
    // ---- validation: nothing is launched on any error
    if (!q || !k_cache || !v_cache || !o || !block_table || !cu_q || !kv_lens) return ATTN_ERR_INVALID_ARG;
    if (n_seqs < 1 || total_q < 1 || max_q_len < 1 || Hq < 1 || max_pages < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = check_cache(n_pages, page_size, Hkv, D, page_stride, token_stride, head_stride);
    if (st != ATTN_OK) return st;
    if (Hq % Hkv != 0 || (causal != 0 && causal != 1) || !std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_F16) return ATTN_ERR_INVALID_ARG;
    const long long row = (long long)Hq * D;
    if (q_stride % 8 != 0 || q_stride < row || q_stride > (1ll << 60) / total_q) return ATTN_ERR_INVALID_ARG;
    if (table_stride < max_pages || table_stride > (1ll << 60) / n_seqs) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {q, k_cache, v_cache, (const void*)o})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)lse, (const void*)block_table, (const void*)cu_q, (const void*)kv_lens})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, kWorkspaceAlign)) return ATTN_ERR_INVALID_ARG;
    if ((long long)total_q * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    // o, lse and the workspace overlap no input and not each other
    const size_t cache = cache_extent(n_pages, page_size, Hkv, D, page_stride, token_stride, head_stride);
    const void* in_p[8] = {q, k_cache, v_cache, block_table, cu_q, kv_lens, o, lse};
    const size_t o_bytes = (size_t)total_q * row * 2, lse_bytes = lse ? (size_t)total_q * Hq * 4 : 0;
    const size_t in_n[8] = {((size_t)(total_q - 1) * q_stride + row) * 2, cache, cache,
                            ((size_t)(n_seqs - 1) * table_stride + max_pages) * 4, ((size_t)n_seqs + 1) * 4,
                            (size_t)n_seqs * 4, o_bytes, lse_bytes};
    for (int c = 0; c < 6; ++c)
        if (ranges_overlap(o, o_bytes, in_p[c], in_n[c]) || (lse && ranges_overlap(lse, lse_bytes, in_p[c], in_n[c])))
            return ATTN_ERR_INVALID_ARG;
    if (lse && ranges_overlap(lse, lse_bytes, o, o_bytes)) return ATTN_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !paged_device_setup(dev, &sms)) return ATTN_ERR_CUDA;
    const size_t need = paged_workspace_bytes(sms, (long long)max_q_len * (Hq / Hkv), D, page_size);
    if (!workspace || workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    for (int c = 0; c < 8; ++c)
        if (in_n[c] > 0 && ranges_overlap(workspace, need, in_p[c], in_n[c])) return ATTN_ERR_INVALID_ARG;
    attn::paged::PagedParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_cache);
    p.v = static_cast<const uint16_t*>(v_cache);
    p.o = static_cast<uint16_t*>(o);
    p.lse = lse;
    p.table = block_table;
    p.cu_q = cu_q;
    p.kv_lens = kv_lens;
    p.n_seqs = n_seqs;
    p.total_q = total_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.causal = causal;
    // a length is at most what the table's columns name, and leaves room to count tiles past it
    p.max_kv = static_cast<int>(std::min<long long>((long long)max_pages * page_size, 0x7fffffffLL - 4096));
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.page_stride = page_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    const bool f16 = dtype == ATTN_DTYPE_F16;
    if (D == 64) return f16 ? launch_paged<true, 64>(p, max_q_len, workspace, sms, stream) : launch_paged<false, 64>(p, max_q_len, workspace, sms, stream);
    if (D == 128) return f16 ? launch_paged<true, 128>(p, max_q_len, workspace, sms, stream) : launch_paged<false, 128>(p, max_q_len, workspace, sms, stream);
    return f16 ? launch_paged<true, 256>(p, max_q_len, workspace, sms, stream) : launch_paged<false, 256>(p, max_q_len, workspace, sms, stream);
}

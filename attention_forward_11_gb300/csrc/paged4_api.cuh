// paged4_api.cuh -- host side of the paged cache in 4 bits: argument checks and launches of
// attn_paged_coded_append and attn_paged_coded_fwd.  Included by attn_api.cu behind paged_api.cuh and
// paged_pages_api.cuh, whose helpers it uses.
#pragma once

namespace {

// A cache in 4 bits: strides in bytes.
struct Cache4 {
    const void *k_codes, *k_scales, *v_codes, *v_scales;
    int n_pages, page_size, Hkv, D;
    long long code_page, code_token, code_head, scale_page, scale_token, scale_head;
    float k_unit, v_unit;
    size_t code_bytes() const { return extent(code_page, code_token, code_head, D / 2); }
    size_t scale_bytes() const { return extent(scale_page, scale_token, scale_head, D / 16); }
    size_t extent(long long ps, long long ts, long long hs, int row) const {
        return (size_t)(n_pages - 1) * ps + (size_t)(page_size - 1) * ts + (size_t)(Hkv - 1) * hs + row;
    }
};

bool unit_ok(float unit) { return std::isfinite(unit) && unit > 0.f && std::isfinite(1.f / unit); }

// Is the inverse of a unit a power of two, from 2^-101 to 2^99, whose product with any scale's inverse is a normal
// number?
bool short_unit(float inv) {
    int e;  // inv is 2^(e - 1)
    return std::frexp(inv, &e) == 0.5f && e >= -100 && e <= 100;
}

attn_status_t check_cache4(Cache4& c) {
    if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return ATTN_ERR_INVALID_ARG;
    if (c.n_pages < 1 || c.page_size < 1 || c.Hkv < 1 || c.D < 1) return ATTN_ERR_INVALID_ARG;
    if (c.D != 64 && c.D != 128 && c.D != 256) return ATTN_ERR_UNSUPPORTED;
    if (!unit_ok(c.k_unit) || !unit_ok(c.v_unit)) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {c.k_codes, c.v_codes})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {c.k_scales, c.v_scales})
        if (!aligned(ptr, c.D / 16)) return ATTN_ERR_INVALID_ARG;
    return layout_ok(c.n_pages, c.page_size, c.Hkv, c.D / 2, 16, c.code_page, c.code_token, c.code_head) &&
                   layout_ok(c.n_pages, c.page_size, c.Hkv, c.D / 16, c.D / 16, c.scale_page, c.scale_token, c.scale_head)
               ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

template <int kD, int kNB>
bool opt_in_smem_rows4() {
    using namespace attn::paged;
    return cudaFuncSetAttribute(paged4_rows_kernel<kD, kNB, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Rows4Geo<kD, kNB, false>::kSmemBytes) == cudaSuccess &&
           cudaFuncSetAttribute(paged4_rows_kernel<kD, kNB, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Rows4Geo<kD, kNB, true>::kSmemBytes) == cudaSuccess;
}

template <bool kF16, int kD>
bool opt_in_smem_tiles4() {
    return cudaFuncSetAttribute(attn::paged::paged4_tiles_kernel<kF16, kD>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                attn::paged::Tiles4Geo<kD>::kSmemBytes) == cudaSuccess;
}

bool paged4_device_setup(int dev, int* sm_count) {
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    if (!paged_device_setup(dev, sm_count)) return false;  // checks dev
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev])
        done[dev] = opt_in_smem_rows4<64, 1>() && opt_in_smem_rows4<64, 2>() && opt_in_smem_rows4<64, 3>() &&
                    opt_in_smem_rows4<64, 4>() && opt_in_smem_rows4<128, 1>() && opt_in_smem_rows4<128, 2>() &&
                    opt_in_smem_rows4<128, 3>() && opt_in_smem_rows4<256, 1>() && opt_in_smem_rows4<256, 2>() &&
                    opt_in_smem_tiles4<false, 64>() &&
                    opt_in_smem_tiles4<true, 64>() && opt_in_smem_tiles4<false, 128>() && opt_in_smem_tiles4<true, 128>();
    return done[dev];
}

template <int kD, int kNB, bool kMany = false>
attn_status_t launch_rows4(const attn::paged::Paged4Params& p, void* workspace, int sms, cudaStream_t stream) {
    using namespace attn::paged;
    using G = Rows4Geo<kD, kNB, kMany>;
    SchedParams sp{};
    sp.map = make_row_map(p.Hkv, p.group, G::kRows, 1);
    sp.ws = split_workspace(workspace, sms * G::kTeams, G::kRows);
    sp.tag = next_tag();
    sp.o_unit = p.v_unit;
    return launch_behind(paged4_rows_kernel<kD, kNB, kMany>, dim3(sms), G::kThreads, G::kSmemBytes, stream, p, sp);
}

// Teams of four warps (paged4_rows_sm103.cuh) pay where most of them find work of their own, as far
// as the host knows.  300 to 8000 keys, 64/8 heads of 128, sequences x heads with a place / with rows,
// teams / whole blocks: 192 / 64 19.4 / 17.0 us, 320 / 192 33.5 / 38.4, 480 / 352 52.6 / 64.0, 672 /
// 544 78.5 / 98.6, 1280 / 1152 152 / 198; 8 x 1 of 32767 keys 31.6 / 20.0.  More than 8 rows at head
// size 64, 2000 to 6000 keys, 32 units 18.8 / 18.6, 128 38.0 / 39.5, 512 103 / 109; at 128 128 units 57.5 /
// 55.3, 512 144 / 152; at 256 384 units 119 / 135.
bool many_units(const attn::paged::Paged4Params& p, int nb, int D, int sms) {
    const long long units = (long long)std::min(p.total_q, p.n_seqs) * p.Hkv;
    return units >= (D == 64 && nb > 1 ? sms / 2 : 2 * sms);
}

// Does a call take the tcgen05 kernel?  From more rows a key/value head on than the rows kernel
// computes together, on pages of any size (and unless V's unit is tiny: the rows kernel needs less workspace).
// 16 sequences of 2000 to 6000 keys, 8 key heads, rows / tiles kernel: at head size 128 16 rows 41 / 73 us, 24 54 / 71,
// 32 83 / 69, 40 76 / 62, 64 111 / 66; at 64 24 34 / 55, 32 45 / 53, 40 54 / 48, 64 61 / 50.
bool takes_tiles4(long long rows, int D) { return rows > 8 * max_row_blocks(D) && D <= 128; }

size_t paged4_workspace_bytes(int sms, long long rows, int D) {
    if (takes_tiles4(rows, D)) return attn::paged::ws_bytes(sms, attn::kTiles * attn::kBM, D);
    const int nb = row_blocks_for(rows, D);
    return attn::paged::ws_bytes((nb == 1 && D <= 128 ? 4 : 2) * sms, 8 * nb, D);
}

// The rows kernel's variant for sequences of at most `rows` rows.
template <int kD, bool kMany>
attn_status_t launch_rows4_blocks(const attn::paged::Paged4Params& p, int nb, void* workspace, int sms, cudaStream_t stream) {
    if (nb == 1) return launch_rows4<kD, 1, kMany>(p, workspace, sms, stream);
    if constexpr (kD != 256)
        if (nb == 3) return launch_rows4<kD, 3, kMany>(p, workspace, sms, stream);
    if constexpr (kD == 64)
        if (nb == 4) return launch_rows4<kD, 4, kMany>(p, workspace, sms, stream);
    return launch_rows4<kD, 2, kMany>(p, workspace, sms, stream);
}
template <int kD>
attn_status_t launch_rows4_for(const attn::paged::Paged4Params& p, long long rows, void* workspace, int sms, cudaStream_t stream) {
    const int nb = row_blocks_for(rows, kD);
    return many_units(p, nb, kD, sms) ? launch_rows4_blocks<kD, true>(p, nb, workspace, sms, stream)
                                      : launch_rows4_blocks<kD, false>(p, nb, workspace, sms, stream);
}

template <bool kF16, int kD>
attn_status_t launch_tiles4(const attn::paged::Paged4Params& p, long long rows, void* workspace, int sms, cudaStream_t stream) {
    using namespace attn::paged;
    using T = Tiles4Geo<kD>;
    EncodeTiledFn fn = encoder();
    if (!fn) return ATTN_ERR_CUDA;
    SchedParams sp{};
    sp.map = make_row_map(p.Hkv, p.group, attn::kBM, attn::kTiles);
    sp.ws = split_workspace(workspace, sms, T::kRows);
    sp.o_unit = p.v_unit;
    TilesParams tp{};
    tp.tile_tokens = sp.map.tokens / attn::kTiles;
    tp.q_rows = sp.map.heads * tp.tile_tokens;
    tp.poll_limit = kDefaultPollLimit;
    CUtensorMap tm;
    if (!encode_q_map(fn, &tm, kF16, kD, p, sp.map.heads, tp.tile_tokens)) return ATTN_ERR_CUDA;
    const attn_status_t st = launch_behind(paged4_tiles_kernel<kF16, kD>, dim3(sms), attn::kThreads, T::kSmemBytes,
                                           stream, tm, p, sp, tp);
    if (st != ATTN_OK) return st;
    const int at_once = kCombineThreads / (kD / 4);
    const int parts = static_cast<int>((std::min<long long>(rows, T::kRows) + at_once - 1) / at_once);
    return launch_behind(paged_combine_kernel<kF16, kD, T::kRows, attn::kTiles>, dim3(sms, parts), kCombineThreads, 0,
                         stream, static_cast<const PagedParams&>(p), sp);
}

// Batches of long sequences and single tokens are shared by is_mixed, whose thresholds are the 16-bit kernels'.
// Over codes the rows kernel is faster and a tile's step slower, so sharing wins sooner: one chunk among tokens,
// 32/8 heads, longest / mean in brackets, all rows in tiles / shared: at head size 128, contexts of 100 to 1000 keys,
// 34 / 34 us (17), 60 / 53 (36), 80 / 58 (50), 127 / 68 (84), 249 / 107 (156); of 2000 to 8000 119 / 95, 213 / 125,
// 286 / 138, 451 / 195, 857 / 336; at 64 25 / 28, 43 / 41, 56 / 45, 84 / 52, 165 / 74, and 96 / 67, 158 / 96, 213 / 104,
// 334 / 142, 635 / 251.  4 chunks of 100 to 512 among 36 tokens, 500 to 6000 keys, head size 128, 166 / 127 (20).
template <int kD>
attn_status_t launch_paged4(const attn::paged::Paged4Params& p, int max_q_len, void* workspace, int sms, cudaStream_t stream) {
    const long long rows = (long long)max_q_len * p.group;
    if constexpr (kD != 256) {
        if (takes_tiles4(rows, kD) && p.v_unit >= attn::paged::kTiles4LeastUnit) {
            attn::paged::Paged4Params half = p;
            if (is_mixed(p, max_q_len, kD)) {
                half.split_rows = 8 * row_blocks_for(p.group, kD);
                half.take_short = 1;
                const attn_status_t st = launch_rows4_for<kD>(half, p.group, workspace, sms, stream);
                if (st != ATTN_OK) return st;
                half.take_short = 0;
            }
            return p.f16 ? launch_tiles4<true, kD>(half, rows, workspace, sms, stream)
                         : launch_tiles4<false, kD>(half, rows, workspace, sms, stream);
        }
    }
    return launch_rows4_for<kD>(p, rows, workspace, sms, stream);
}

}  // namespace

extern "C" attn_status_t attn_paged_coded_append(const void* k, const void* v, const long long* slot_map, void* k_codes,
                                            void* k_scales, void* v_codes, void* v_scales, int n_tokens, int Hkv, int D,
                                            int n_pages, int page_size, long long k_stride, long long v_stride,
                                            long long code_page_stride, long long code_token_stride,
                                            long long code_head_stride, long long scale_page_stride,
                                            long long scale_token_stride, long long scale_head_stride, float k_unit,
                                            float v_unit, int dtype, cudaStream_t stream) {
    if (!k || !v || !slot_map || n_tokens < 1) return ATTN_ERR_INVALID_ARG;
    Cache4 c{k_codes, k_scales, v_codes, v_scales, n_pages, page_size, Hkv, D, code_page_stride, code_token_stride,
             code_head_stride, scale_page_stride, scale_token_stride, scale_head_stride, k_unit, v_unit};
    const attn_status_t st = check_cache4(c);
    if (st != ATTN_OK) return st;
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_F16) return ATTN_ERR_INVALID_ARG;
    const long long row = (long long)Hkv * D;
    for (long long stride : {k_stride, v_stride})
        if (stride % 8 != 0 || stride < row || stride > (1ll << 60) / n_tokens) return ATTN_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8)) return ATTN_ERR_INVALID_ARG;
    // The caches overlap no row and no slot.  Parts of one interleaved tensor share an address
    // range without sharing a byte, so they are not compared with one another.
    const size_t codes = c.code_bytes(), scales = c.scale_bytes();
    const Range in[3] = {{k, ((size_t)(n_tokens - 1) * k_stride + row) * 2}, {v, ((size_t)(n_tokens - 1) * v_stride + row) * 2},
                         {slot_map, (size_t)n_tokens * 8}};
    for (const Range& out : {Range{k_codes, codes}, Range{v_codes, codes}, Range{k_scales, scales}, Range{v_scales, scales}})
        for (const Range& x : in)
            if (ranges_overlap(out.at, out.n, x.at, x.n)) return ATTN_ERR_INVALID_ARG;
    const void* base[4] = {k_codes, v_codes, k_scales, v_scales};
    for (int a = 0; a < 4; ++a)
        for (int b = a + 1; b < 4; ++b)
            if (base[a] == base[b]) return ATTN_ERR_INVALID_ARG;
    if (row / 16 > (1 << 24)) return ATTN_ERR_UNSUPPORTED;
    attn::paged::Append4Params p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_codes = static_cast<uint8_t*>(k_codes);
    p.k_scales = static_cast<uint8_t*>(k_scales);
    p.v_codes = static_cast<uint8_t*>(v_codes);
    p.v_scales = static_cast<uint8_t*>(v_scales);
    p.slot_map = slot_map;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.code_page = c.code_page;
    p.code_token = c.code_token;
    p.code_head = c.code_head;
    p.scale_page = c.scale_page;
    p.scale_token = c.scale_token;
    p.scale_head = c.scale_head;
    p.n_slots = (long long)n_pages * page_size;
    p.k_inv = static_cast<float>(1.0 / static_cast<double>(k_unit));
    p.v_inv = static_cast<float>(1.0 / static_cast<double>(v_unit));
    p.T = n_tokens;
    p.row_blocks = static_cast<int>(row / 16);
    p.head_blocks_log2 = D == 64 ? 2 : D == 128 ? 3 : 4;
    p.per_block = std::max(1, attn::paged::kAppend4Threads / p.row_blocks);
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    p.by_row = attn::paged::make_fastdiv(static_cast<unsigned int>(p.row_blocks));
    const dim3 blocks(static_cast<unsigned int>(((long long)n_tokens + p.per_block - 1) / p.per_block));
    const bool f16 = dtype == ATTN_DTYPE_F16, brief = short_unit(p.k_inv) && short_unit(p.v_inv);
    auto kernel = f16 ? brief ? attn::paged::paged4_append_kernel<true, true> : attn::paged::paged4_append_kernel<true, false>
                      : brief ? attn::paged::paged4_append_kernel<false, true> : attn::paged::paged4_append_kernel<false, false>;
    return launch_behind(kernel, blocks, attn::paged::kAppend4Threads, 0, stream, p);
}

extern "C" attn_status_t attn_paged_coded_fwd_workspace_size(int total_q, int max_q_len, int Hq, int Hkv, int D, int page_size,
                                                        size_t* bytes) {
    if (!bytes) return ATTN_ERR_INVALID_ARG;
    *bytes = 0;
    if (total_q < 1 || max_q_len < 1 || page_size < 1 || Hq < 1 || Hkv < 1 || D < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
    if ((long long)total_q * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !paged4_device_setup(dev, &sms)) return ATTN_ERR_CUDA;
    *bytes = paged4_workspace_bytes(sms, (long long)max_q_len * (Hq / Hkv), D);
    return ATTN_OK;
}

extern "C" attn_status_t attn_paged_coded_fwd(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                                         const void* v_scales, void* o, float* lse, const int* block_table,
                                         const int* cu_q, const int* kv_lens, int n_seqs, int total_q, int max_q_len,
                                         int Hq, int Hkv, int D, int n_pages, int page_size, int max_pages,
                                         long long q_stride, long long table_stride, long long code_page_stride,
                                         long long code_token_stride, long long code_head_stride,
                                         long long scale_page_stride, long long scale_token_stride,
                                         long long scale_head_stride, int causal, float scale, float k_unit,
                                         float v_unit, int dtype, void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream) {
    // ---- validation: nothing is launched on any error
    if (!q || !o || !block_table || !cu_q || !kv_lens) return ATTN_ERR_INVALID_ARG;
    if (total_q < 1 || max_q_len < 1 || Hq < 1 || !table_ok(n_seqs, max_pages, table_stride)) return ATTN_ERR_INVALID_ARG;
    Cache4 c{k_codes, k_scales, v_codes, v_scales, n_pages, page_size, Hkv, D, code_page_stride, code_token_stride,
             code_head_stride, scale_page_stride, scale_token_stride, scale_head_stride, k_unit, v_unit};
    const attn_status_t st = check_cache4(c);
    if (st != ATTN_OK) return st;
    if (Hq % Hkv != 0 || (causal != 0 && causal != 1) || !std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    const double scale_log2 = static_cast<double>(scale) * k_unit * 1.4426950408889634;
    if (!std::isnormal(static_cast<float>(scale_log2))) return ATTN_ERR_INVALID_ARG;  // fewer bits would move logits
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_F16) return ATTN_ERR_INVALID_ARG;
    const long long row = (long long)Hq * D;
    if (q_stride % 8 != 0 || q_stride < row || q_stride > (1ll << 60) / total_q) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {q, (const void*)o})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)lse, (const void*)block_table, (const void*)cu_q, (const void*)kv_lens})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, kWorkspaceAlign)) return ATTN_ERR_INVALID_ARG;
    if ((long long)total_q * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    // o, lse and the workspace overlap no input and not each other
    int dev = 0, sms = 0;
    const size_t codes = c.code_bytes(), scales = c.scale_bytes();
    const Range in[8] = {{q, ((size_t)(total_q - 1) * q_stride + row) * 2}, {k_codes, codes}, {v_codes, codes},
                         {k_scales, scales}, {v_scales, scales},
                         {block_table, ((size_t)(n_seqs - 1) * table_stride + max_pages) * 4},
                         {cu_q, ((size_t)n_seqs + 1) * 4}, {kv_lens, (size_t)n_seqs * 4}};
    Range out[3] = {{o, (size_t)total_q * row * 2}, {lse, lse ? (size_t)total_q * Hq * 4 : 0}, {workspace, 0}};
    if (outputs_overlap(out, in)) return ATTN_ERR_INVALID_ARG;
    if (cudaGetDevice(&dev) != cudaSuccess || !paged4_device_setup(dev, &sms)) return ATTN_ERR_CUDA;
    const long long rows = (long long)max_q_len * (Hq / Hkv);
    const size_t need = paged4_workspace_bytes(sms, rows, D);
    if (!workspace || workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    out[2].n = need;
    if (outputs_overlap(out, in)) return ATTN_ERR_INVALID_ARG;
    attn::paged::Paged4Params p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k_codes = static_cast<const uint8_t*>(k_codes);
    p.k_scales = static_cast<const uint8_t*>(k_scales);
    p.v_codes = static_cast<const uint8_t*>(v_codes);
    p.v_scales = static_cast<const uint8_t*>(v_scales);
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
    p.max_kv = row_tokens(max_pages, page_size);
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.page_stride = c.code_page;
    p.token_stride = c.code_token;
    p.head_stride = c.code_head;
    p.scale_page = c.scale_page;
    p.scale_token = c.scale_token;
    p.scale_head = c.scale_head;
    p.scale_log2 = static_cast<float>(scale_log2);
    p.v_unit = v_unit;
    p.f16 = dtype == ATTN_DTYPE_F16;
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    if (D == 64) return launch_paged4<64>(p, max_q_len, workspace, sms, stream);
    if (D == 128) return launch_paged4<128>(p, max_q_len, workspace, sms, stream);
    return launch_paged4<256>(p, max_q_len, workspace, sms, stream);
}

// paged_pages_api.cuh -- host side of attn_paged_fork, attn_paged_free and attn_paged_copy:
// argument checks and launches.  Included by attn_api.cu behind paged_api.cuh, whose helpers
// it uses.
#pragma once

namespace {

struct Range {
    const void* at;
    size_t n;
};

// Does an output overlap an input or another output?  (Ranges of no bytes overlap nothing.)
template <int kOut, int kIn>
bool outputs_overlap(const Range (&out)[kOut], const Range (&in)[kIn]) {
    for (int a = 0; a < kOut; ++a) {
        if (out[a].n == 0) continue;
        for (int c = 0; c < kIn; ++c)
            if (in[c].n > 0 && ranges_overlap(out[a].at, out[a].n, in[c].at, in[c].n)) return true;
        for (int c = a + 1; c < kOut; ++c)
            if (out[c].n > 0 && ranges_overlap(out[a].at, out[a].n, out[c].at, out[c].n)) return true;
    }
    return false;
}

bool table_ok(int n_seqs, int max_pages, long long table_stride) {
    return n_seqs >= 1 && max_pages >= 1 && table_stride >= max_pages && table_stride <= (1ll << 60) / n_seqs;
}

// Tokens that a row of the table names, as an int.
int row_tokens(int max_pages, int page_size) {
    return static_cast<int>(std::min<long long>((long long)max_pages * page_size, 0x7fffffffLL - 4096));
}

// Entries of a table from which on its rows are given to the whole GPU (1024 rows of 470 entries, all
// freed, 26 us, in the one cluster 44; 300 rows 16 / 22 us; 128 rows 12.9 / 12.8 us; 256 rows of 256, or of
// 1024, 13.8 / 14.2).  What is given back is on the device, so a wide table takes it for a few pages too: drafts
// of 256 rows 9.2 us, in the one cluster 8.5.
constexpr long long kFreeLarge = 65536;

}  // namespace

extern "C" attn_status_t attn_paged_fork(const int* parents, const int* lens, int* kv_lens, int n_seqs, int page_size,
                                         const int* free_pages, int n_free, const int* free_head, int* block_table,
                                         int max_pages, long long table_stride, int* shares, int n_pages, int* copies,
                                         int* counts, cudaStream_t stream) {
    if (!parents || !kv_lens || !block_table || !shares || !copies || !counts) return ATTN_ERR_INVALID_ARG;
    if (page_size < 1 || n_free < 0 || n_pages < 1 || !table_ok(n_seqs, max_pages, table_stride)) return ATTN_ERR_INVALID_ARG;
    if (n_free > 0 && !free_pages) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)parents, (const void*)lens, (const void*)kv_lens, (const void*)free_pages,
                            (const void*)free_head, (const void*)block_table, (const void*)shares, (const void*)copies,
                            (const void*)counts})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    const size_t n = (size_t)n_seqs * 4;
    const Range out[5] = {{kv_lens, n}, {block_table, ((size_t)(n_seqs - 1) * table_stride + max_pages) * 4},
                          {shares, (size_t)n_pages * 4}, {copies, 3 * n}, {counts, 16}};
    const Range in[4] = {{parents, n}, {lens, lens ? n : 0}, {free_pages, (size_t)n_free * 4}, {free_head, free_head ? 4u : 0u}};
    if (outputs_overlap(out, in)) return ATTN_ERR_INVALID_ARG;
    attn::paged::ForkParams p{};
    p.parents = parents;
    p.lens = lens;
    p.free_pages = free_pages;
    p.free_head = free_head;
    p.kv_lens = kv_lens;
    p.table = block_table;
    p.shares = shares;
    p.copies = copies;
    p.counts = counts;
    p.table_stride = table_stride;
    p.n_seqs = n_seqs;
    p.n_free = n_free;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.max_kv = row_tokens(max_pages, page_size);
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    // four warps for every row, up to 128 blocks: each repeats the scan over the rows
    const int blocks = std::min(128, (n_seqs + attn::paged::kForkRows - 1) / attn::paged::kForkRows);
    return launch_behind(attn::paged::paged_fork_kernel, dim3(blocks), attn::paged::kForkThreads, 0, stream, p);
}

extern "C" attn_status_t attn_paged_free(const int* kv_lens, const int* keep_lens, int n_seqs, int page_size,
                                         const int* block_table, int max_pages, long long table_stride, int* shares,
                                         int n_pages, int* free_pages, int n_free, const int* free_head, int* counts,
                                         cudaStream_t stream) {
    if (!kv_lens || !keep_lens || !block_table || !shares || !free_pages || !free_head || !counts) return ATTN_ERR_INVALID_ARG;
    if (page_size < 1 || n_free < 1 || n_pages < 1 || !table_ok(n_seqs, max_pages, table_stride)) return ATTN_ERR_INVALID_ARG;
    for (const void* ptr : {(const void*)kv_lens, (const void*)keep_lens, (const void*)block_table, (const void*)shares,
                            (const void*)free_pages, (const void*)free_head, (const void*)counts})
        if (!aligned(ptr, 4)) return ATTN_ERR_INVALID_ARG;
    const size_t n = (size_t)n_seqs * 4;
    const Range out[3] = {{shares, (size_t)n_pages * 4}, {free_pages, (size_t)n_free * 4}, {counts, 16}};
    const Range in[4] = {{kv_lens, n}, {keep_lens, n}, {block_table, ((size_t)(n_seqs - 1) * table_stride + max_pages) * 4},
                         {free_head, 4}};
    if (outputs_overlap(out, in)) return ATTN_ERR_INVALID_ARG;
    attn::paged::FreeParams p{};
    p.kv_lens = kv_lens;
    p.keep_lens = keep_lens;
    p.table = block_table;
    p.free_head = free_head;
    p.shares = shares;
    p.free_pages = free_pages;
    p.counts = counts;
    p.table_stride = table_stride;
    p.n_seqs = n_seqs;
    p.n_free = n_free;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.max_kv = row_tokens(max_pages, page_size);
    p.by_page = attn::paged::make_fastdiv(static_cast<unsigned int>(page_size));
    p.phase = (long long)n_seqs * max_pages >= kFreeLarge ? 1 : 0;
    if (p.phase == 1) {
        const attn_status_t st = launch_behind(attn::paged::paged_free_kernel, dim3(18 * attn::paged::kFreeBlocks),
                                               attn::paged::kFreeThreads, 0, stream, p);
        if (st != ATTN_OK) return st;
        p.phase = 2;
    }
    return launch_behind(attn::paged::paged_free_kernel, dim3(attn::paged::kFreeBlocks), attn::paged::kFreeThreads, 0,
                         stream, p);
}

extern "C" attn_status_t attn_paged_copy(const int* copies, int n_copies, void* const* caches, int n_caches, int n_pages,
                                         int page_size, int Hkv, int row_bytes, long long page_stride,
                                         long long token_stride, long long head_stride, cudaStream_t stream) {
    if (!copies || !caches || n_copies < 1 || n_caches < 1 || n_pages < 1 || page_size < 1 || Hkv < 1 || row_bytes < 4)
        return ATTN_ERR_INVALID_ARG;
    if (row_bytes % 4 != 0 || !aligned(copies, 4)) return ATTN_ERR_INVALID_ARG;
    if (!layout_ok(n_pages, page_size, Hkv, row_bytes, 4, page_stride, token_stride, head_stride)) return ATTN_ERR_INVALID_ARG;
    if ((long long)page_size * Hkv > 0x7fffffffLL / row_bytes) return ATTN_ERR_UNSUPPORTED;
    const size_t extent = (size_t)(n_pages - 1) * page_stride + (size_t)(page_size - 1) * token_stride +
                          (size_t)(Hkv - 1) * head_stride + row_bytes;
    uintptr_t bits = 0;
    for (int i = 0; i < n_caches; ++i) {
        if (!caches[i] || !aligned(caches[i], 4)) return ATTN_ERR_INVALID_ARG;
        if (ranges_overlap(caches[i], extent, copies, (size_t)n_copies * 12)) return ATTN_ERR_INVALID_ARG;
        bits |= reinterpret_cast<uintptr_t>(caches[i]);
    }
    // heads that follow one another without a gap are one row
    if (Hkv == 1 || head_stride == row_bytes) {
        row_bytes *= Hkv;
        Hkv = 1;
        head_stride = row_bytes;
    }
    // tokens of a head that follow one another without a gap are one run, in pieces of its own size
    const bool run = page_size > 1 && token_stride == row_bytes;
    bits |= static_cast<uintptr_t>(Hkv == 1 ? 0 : head_stride) | static_cast<uintptr_t>(n_pages == 1 ? 0 : page_stride);
    if (!run) bits |= static_cast<uintptr_t>(row_bytes) | static_cast<uintptr_t>(page_size == 1 ? 0 : token_stride);
    const int piece = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : 4;
    attn::paged::CopyParams p{};
    p.copies = copies;
    p.page_stride = page_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.n_copies = n_copies;
    p.n_pages = n_pages;
    p.page_size = page_size;
    p.heads = Hkv;
    p.run = run ? row_bytes : 0;
    p.pieces = std::max(row_bytes / piece, 1);
    p.head_first = Hkv > 1 && token_stride < head_stride;
    p.by_token = attn::paged::make_fastdiv(static_cast<unsigned int>(Hkv * p.pieces));
    p.by_row = attn::paged::make_fastdiv(static_cast<unsigned int>(p.pieces));
    const long long all = ((long long)page_size * row_bytes + piece - 1) / piece * Hkv;
    constexpr int kAtOnce = 32 * attn::paged::kCopyFly, kMostWarps = 152 * 8 * (attn::paged::kCopyThreads / 32);
    for (int first = 0; first < n_caches; first += attn::paged::kCopyMaxCaches) {
        p.n_caches = std::min(n_caches - first, attn::paged::kCopyMaxCaches);
        p.by_cache = attn::paged::make_fastdiv(static_cast<unsigned int>(p.n_caches));
        // a warp copies a part: up to 8 times what it has in flight, less where that leaves warps idle
        const long long pairs = (long long)n_copies * p.n_caches;
        const long long parts = std::max((all + 8 * kAtOnce - 1) / (8 * kAtOnce), (kMostWarps + pairs - 1) / pairs);
        p.parts = static_cast<int>(std::min(parts, (all + kAtOnce - 1) / kAtOnce));
        p.by_parts = attn::paged::make_fastdiv(static_cast<unsigned int>(p.parts));
        for (int i = 0; i < p.n_caches; ++i) p.caches[i] = static_cast<char*>(caches[first + i]);
        const int warps = attn::paged::kCopyThreads / 32;
        const dim3 grid(static_cast<unsigned int>(std::min((pairs * p.parts + warps - 1) / warps, 152ll * 8)));
        attn_status_t st;
        if (piece == 16) st = launch_behind(attn::paged::paged_copy_kernel<uint4>, grid, attn::paged::kCopyThreads, 0, stream, p);
        else if (piece == 8) st = launch_behind(attn::paged::paged_copy_kernel<uint2>, grid, attn::paged::kCopyThreads, 0, stream, p);
        else st = launch_behind(attn::paged::paged_copy_kernel<uint32_t>, grid, attn::paged::kCopyThreads, 0, stream, p);
        if (st != ATTN_OK) return st;
    }
    return ATTN_OK;
}

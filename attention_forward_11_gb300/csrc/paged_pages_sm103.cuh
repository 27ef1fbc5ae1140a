// paged_pages_sm103.cuh -- pages that several sequences share: forking, freeing, copying.
//
// `shares` counts, for every page, the rows of the block table that name it beyond the
// first, so a page that paged_tables_kernel takes from the free list needs no count, and a
// page goes back to the list once its count would fall below zero.
//
// paged_fork_kernel gives rows the first t tokens of another row: its full pages are named
// twice from then on (shares + 1), a rest of t % P tokens takes a free page, and the copy
// that fills it is listed for paged_copy_kernel.  As in paged_tables_kernel every block
// repeats the scan that hands out the free pages (out of L2) instead of waiting for another
// block, and then writes its own rows.  A row that is rewritten is no source in the same
// call, so nothing that a block reads is written by another.  64 forks of 100 to 8000 tokens on
// pages of 16 take 4.8 us (a warp a row 7.2), three loads one behind another and a launch.
//
// paged_free_kernel takes the pages behind a row's kept tokens from it.  Which of several
// rows gives a shared page its last push depends on timing, so the freed pages are listed by
// number: the counts are lowered first, then every page whose count is below zero is found by
// a scan over all counts.  Both halves are one launch of one cluster of 8 blocks, whose
// hardware barrier stands between them; no workspace.  Where a table is large (kFreeLarge) 8 SMs
// take longer over its rows than a second launch does, and the first half is a launch of its own
// over all of them.
//
// Drafts of 256 rows given back take 8.7 us, 1024 rows of up to 470 pages 26 us.
//
// paged_copy_kernel copies the first tokens of pages to other pages in up to 256 caches (all
// layers' K and V) at once, a warp a part of a page: 64 half-filled pages of 131 KB in 64 caches take
// 90 us, 6.05 TB/s of HBM; of a cache in 4 bits, two layouts and so two launches, 38 us, 4.05 TB/s
// (a block a part: 106 and 44 us).
#pragma once
#include <climits>
#include <cstdint>

#include "paged_common_sm103.cuh"
#include "paged_tables_sm103.cuh"

namespace attn {
namespace paged {

struct ForkParams {
    const int *parents, *lens;  // lens: nullptr takes all of the parent's tokens
    const int *free_pages, *free_head;
    int *kv_lens, *table, *shares, *copies, *counts;
    long long table_stride;
    int n_seqs, n_free, n_pages, max_pages, page_size;
    int max_kv;  // tokens that a row can name
    FastDiv by_page;
};

constexpr int kForkThreads = 1024;  // rows scanned per step
constexpr int kForkRowWarps = 4, kForkRows = kForkThreads / 32 / kForkRowWarps;  // warps of a row, rows written at a time

__global__ void __launch_bounds__(kForkThreads) paged_fork_kernel(const ForkParams p) {
    __shared__ int s_parent[kForkThreads];  // -1: no fork
    __shared__ int s_len[kForkThreads];
    __shared__ int s_last[kForkThreads];    // entry of the column behind the full pages
    __shared__ long long s_part[2][32];
    launch_dependents();
    wait_for_primary();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = gridDim.x, c = blockIdx.x;
    const long long head = p.free_head != nullptr ? max(*p.free_head, 0) : 0;
    auto parent_of = [&](int s) {
        const int x = p.parents[s];
        return x >= 0 && x < p.n_seqs && x != s ? x : -1;
    };
    auto is_page = [&](int x) { return x >= 0 && x < p.n_pages; };
    long long taken = 0, forks = 0, refused = 0;  // of the steps before
    for (int s0 = 0; s0 < p.n_seqs; s0 += kForkThreads) {
        const int s = s0 + tid, n = min(kForkThreads, p.n_seqs - s0);
        int parent = -1, len = 0, rest = 0, src = -1;
        bool refuse = false;
        if (tid < n) parent = parent_of(s);
        if (parent >= 0) {
            refuse = parent_of(parent) >= 0;
            len = min(max(p.kv_lens[parent], 0), p.max_kv);
            if (p.lens != nullptr) len = min(len, max(p.lens[s], 0));
            const int full = static_cast<int>(p.by_page.quot(len));
            rest = len - full * p.page_size;
            if (rest > 0) src = p.table[parent * p.table_stride + full];
            if (refuse) parent = -1;
        }
        const bool needs = parent >= 0 && rest > 0 && is_page(src);
        long long a = needs, b = (parent >= 0 ? 1ll : 0ll) + (refuse ? 1ll << 32 : 0ll);
        block_scan2(a, b, s_part);  // ends with every thread past its last read of the step before
        const long long at = head + taken + a - 1;
        const int dst = needs && at < p.n_free ? p.free_pages[at] : -1;
        s_parent[tid] = parent;
        s_len[tid] = len;
        s_last[tid] = needs ? dst : src;
        if (tid < n && tid % G == c) {  // this block's rows
            int* to = p.copies + 3ll * s;
            const bool copy = needs && at < p.n_free;
            to[0] = copy ? src : -1;
            to[1] = copy ? dst : -1;
            to[2] = copy ? rest : 0;
            if (parent >= 0) p.kv_lens[s] = len;
        }
        taken += s_part[0][31];
        forks += s_part[1][31] & 0xffffffff;
        refused += s_part[1][31] >> 32;
        __syncthreads();
        for (int j = warp / kForkRowWarps * G + c; j < n; j += kForkRows * G) {
            const int from = s_parent[j];
            if (from < 0) continue;
            const int full = static_cast<int>(p.by_page.quot(s_len[j]));
            const int* row = p.table + from * p.table_stride;
            int* to = p.table + (s0 + j) * p.table_stride;
#pragma unroll 4
            for (int col = warp % kForkRowWarps * 32 + lane; col < full; col += 32 * kForkRowWarps) {
                const int x = row[col];
                to[col] = x;
                if (is_page(x)) atomicAdd(p.shares + x, 1);
            }
            if (lane == 0 && warp % kForkRowWarps == 0 && s_len[j] > full * p.page_size) to[full] = s_last[j];
        }
        __syncthreads();
    }
    if (c == 0 && tid == 0) {
        const long long left = max((long long)p.n_free - head, 0ll), got = min(taken, left);
        p.counts[0] = static_cast<int>(forks);
        p.counts[1] = static_cast<int>(min(head + got, (long long)INT_MAX));
        p.counts[2] = static_cast<int>(taken - got);
        p.counts[3] = static_cast<int>(refused);
    }
}

struct FreeParams {
    const int *kv_lens, *keep_lens, *table, *free_head;
    int *shares, *free_pages, *counts;
    long long table_stride;
    int n_seqs, n_free, n_pages, page_size;
    int max_kv;
    int phase;  // 0: all in one cluster; 1: the counts are lowered, by the whole GPU; 2: the rest, behind that
    FastDiv by_page;
};

constexpr int kFreeThreads = 1024, kFreeBlocks = 8;
constexpr int kFreeWarpPages = 256;                                      // pages of a warp in one step
constexpr int kFreeTile = kFreeThreads / 32 * kFreeWarpPages;            // of a block

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_peer_int(const int* mine, int rank) {
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), far;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(far) : "memory");
    return v;
}

__global__ void __cluster_dims__(kFreeBlocks, 1, 1) __launch_bounds__(kFreeThreads) paged_free_kernel(const FreeParams p) {
    constexpr int kWarps = kFreeThreads / 32, kLoads = kFreeWarpPages / 32;
    __shared__ int s_warp[kWarps];
    __shared__ int s_sum[2];  // freed pages and cut rows of this block
    launch_dependents();
    wait_for_primary();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    if (tid < 2) s_sum[tid] = 0;
    auto lens = [&](int s, int& kv, int& keep) {
        kv = min(max(p.kv_lens[s], 0), p.max_kv);
        keep = max(p.keep_lens[s], 0);
    };
    // pages behind the kept tokens: one row less names each
    const int blocks = gridDim.x;
    for (int s = p.phase == 2 ? p.n_seqs : warp * blocks + c; s < p.n_seqs; s += kWarps * blocks) {
        int kv, keep;
        lens(s, kv, keep);
        if (keep >= kv) continue;
        const int col0 = static_cast<int>(p.by_page.quot((long long)keep + p.page_size - 1));
        const int col1 = static_cast<int>(p.by_page.quot((long long)kv + p.page_size - 1));
        const int* row = p.table + s * p.table_stride;
#pragma unroll 4
        for (int col = col0 + lane; col < col1; col += 32) {
            const int x = row[col];
            if (x >= 0 && x < p.n_pages) atomicSub(p.shares + x, 1);
        }
    }
    if (p.phase == 1) return;
    __threadfence();
    cluster_barrier();
    // what is below zero is free; first how many there are in this block's part of the pages
    const int n0 = static_cast<int>((long long)p.n_pages * c / kFreeBlocks);
    const int n1 = static_cast<int>((long long)p.n_pages * (c + 1) / kFreeBlocks);
    auto look = [&](int first, uint32_t (&below)[kLoads]) {  // this warp's pages from `first` on
        int v[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int x = first + 32 * k + lane;
            v[k] = x < n1 ? __ldcg(p.shares + x) : 0;
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) below[k] = __ballot_sync(0xffffffffu, v[k] < 0);
    };
    int found = 0, cut = 0;
    for (int at = n0; at < n1; at += kFreeTile) {
        uint32_t below[kLoads];
        look(at + warp * kFreeWarpPages, below);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) found += __popc(below[k]);
    }
    // rows whose last kept page is partly kept and still shared
    for (int s = tid * kFreeBlocks + c; s < p.n_seqs; s += kFreeThreads * kFreeBlocks) {
        int kv, keep;
        lens(s, kv, keep);
        const int col = static_cast<int>(p.by_page.quot(keep));
        if (keep >= kv || keep == col * p.page_size) continue;
        const int x = p.table[s * p.table_stride + col];
        cut += x >= 0 && x < p.n_pages && __ldcg(p.shares + x) > 0;
    }
    cut = __reduce_add_sync(0xffffffffu, cut);
    if (lane == 0) {
        if (found) atomicAdd(&s_sum[0], found);
        if (cut) atomicAdd(&s_sum[1], cut);
    }
    cluster_barrier();
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kFreeBlocks; ++k) {
        const int x = cluster_peer_int(&s_sum[0], k);
        if (k < c) before += x;
        all += x;
    }
    const int head = min(max(*p.free_head, 0), p.n_free);
    int to = head - all + before;  // of this block's first freed page
    for (int at = n0; at < n1; at += kFreeTile) {
        uint32_t below[kLoads];
        const int first = at + warp * kFreeWarpPages;
        look(first, below);
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) mine += __popc(below[k]);
        __syncthreads();  // the step before has been read
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        int front = 0, step = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int x = s_warp[w];
            if (w < warp) front += x;
            step += x;
        }
        int next = to + front;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int place = next + __popc(below[k] & ((1u << lane) - 1));
            if ((below[k] >> lane) & 1) {
                const int x = first + 32 * k + lane;
                p.shares[x] = 0;
                if (place >= 0) p.free_pages[place] = x;
            }
            next += __popc(below[k]);
        }
        to += step;
    }
    if (c == 0 && tid == 0) {
        int cuts = 0;
#pragma unroll
        for (int k = 0; k < kFreeBlocks; ++k) cuts += cluster_peer_int(&s_sum[1], k);
        const int fit = min(all, head);
        p.counts[0] = fit;
        p.counts[1] = head - fit;
        p.counts[2] = all - fit;
        p.counts[3] = cuts;
    }
    cluster_barrier();  // no block leaves while another reads its sums
}

constexpr int kCopyThreads = 256, kCopyMaxCaches = 256;
constexpr int kCopyChunk = 1024;  // copies looked at together
constexpr int kCopyFly = 4;       // pieces of a thread in flight

struct CopyParams {
    const int* copies;  // [n_copies, 3]: from page, to page, tokens
    long long page_stride, token_stride, head_stride;  // of every cache, in bytes
    int n_copies, n_caches, n_pages, page_size;
    int heads, pieces;  // of a token, of a head's row
    int parts;          // that a page is copied in
    int head_first;     // a head's tokens follow one another more closely than a token's heads
    int run;            // bytes of a token where a head's tokens follow one another without a gap, or 0
    FastDiv by_token, by_row, by_cache, by_parts;  // heads * pieces, pieces, n_caches, parts
    char* caches[kCopyMaxCaches];
};

template <class Piece>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const __grid_constant__ CopyParams p) {
    constexpr int kEach = kCopyChunk / kCopyThreads, kWarps = kCopyThreads / 32;
    __shared__ int s_copy[kCopyChunk][3];
    __shared__ int s_warp[kWarps];
    launch_dependents();
    wait_for_primary();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int first = 0; first < p.n_copies; first += kCopyChunk) {
        // the chunk's copies, in one order for every block
        int src[kEach], dst[kEach], rows[kEach], mine = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = first + threadIdx.x * kEach + j;
            src[j] = dst[j] = rows[j] = 0;
            if (i < min(first + kCopyChunk, p.n_copies)) {
                const int* x = p.copies + 3ll * i;
                src[j] = x[0], dst[j] = x[1], rows[j] = min(x[2], p.page_size);
                if (src[j] < 0 || src[j] >= p.n_pages || dst[j] < 0 || dst[j] >= p.n_pages || src[j] == dst[j]) rows[j] = 0;
            }
            mine += rows[j] > 0;
        }
        int at = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += x;
        }
        __syncthreads();  // the chunk before has been read
        if (lane == 31) s_warp[warp] = at;
        __syncthreads();
        int n = 0;
        at -= mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s_warp[w];
            n += s_warp[w];
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (rows[j] <= 0) continue;
            s_copy[at][0] = src[j];
            s_copy[at][1] = dst[j];
            s_copy[at][2] = rows[j];
            ++at;
        }
        __syncthreads();
        const long long units = (long long)n * p.n_caches * p.parts;
        for (long long u = (long long)blockIdx.x * kWarps + warp; u < units; u += (long long)gridDim.x * kWarps) {  // a warp's
            const long long pair = (long long)p.by_parts.quot(u);
            const int part = static_cast<int>(u - pair * p.parts);
            const int which = static_cast<int>(p.by_cache.quot(pair));
            char* base = p.caches[pair - (long long)which * p.n_caches];
            const char* from = base + s_copy[which][0] * p.page_stride;
            char* to = base + s_copy[which][1] * p.page_stride;
            // pieces of a head; a run's last one may be a part, copied word by word
            const unsigned int rows = s_copy[which][2], run = rows * p.run;
            const unsigned int of_head = p.run != 0 ? (run + sizeof(Piece) - 1) / sizeof(Piece) : rows * p.pieces;
            const unsigned int all = of_head * p.heads;
            const unsigned int end = static_cast<unsigned int>((long long)all * (part + 1) / p.parts);
            for (unsigned int k = static_cast<unsigned int>((long long)all * part / p.parts) + lane; k < end;
                 k += kCopyFly * 32) {
                Piece v[kCopyFly];
                long long at[kCopyFly];
#pragma unroll
                for (int j = 0; j < kCopyFly; ++j) {
                    const unsigned int x = k + j * 32;
                    at[j] = -1;
                    if (x >= end) continue;
                    unsigned int token, head, piece;
                    if (p.run != 0) {
                        head = x / of_head;
                        piece = (x - head * of_head) * sizeof(Piece);
                        const long long off = head * p.head_stride + piece;
                        if (piece + sizeof(Piece) > run) {
                            for (; piece < run; piece += 4)
                                *reinterpret_cast<uint32_t*>(to + head * p.head_stride + piece) =
                                    *reinterpret_cast<const uint32_t*>(from + head * p.head_stride + piece);
                            continue;
                        }
                        at[j] = off;
                        v[j] = *reinterpret_cast<const Piece*>(from + off);
                        continue;
                    }
                    if (p.head_first) {
                        head = x / of_head;
                        piece = x - head * of_head;
                        token = static_cast<unsigned int>(p.by_row.quot(piece));
                        piece -= token * p.pieces;
                    } else {
                        token = static_cast<unsigned int>(p.by_token.quot(x));
                        piece = x - token * p.by_token.d;
                        head = static_cast<unsigned int>(p.by_row.quot(piece));
                        piece -= head * p.pieces;
                    }
                    at[j] = token * p.token_stride + head * p.head_stride + piece * static_cast<long long>(sizeof(Piece));
                    v[j] = *reinterpret_cast<const Piece*>(from + at[j]);
                }
#pragma unroll
                for (int j = 0; j < kCopyFly; ++j)
                    if (at[j] >= 0) *reinterpret_cast<Piece*>(to + at[j]) = v[j];
            }
        }
    }
}

}  // namespace paged
}  // namespace attn

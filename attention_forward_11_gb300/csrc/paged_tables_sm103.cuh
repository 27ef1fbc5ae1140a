// paged_tables_sm103.cuh -- block tables, slot maps and the write into the pages.
//
// paged_tables_kernel extends each sequence's row of the block table by the pages
// its new tokens need, taken in order from the list of free pages, and says in
// which slot (page * page_size + row) every new token goes.  With c_i cached and
// n_i new tokens both are prefix sums over the sequences: of n_i, and of the pages
// ceil((c_i + n_i) / P) - ceil(c_i / P) that start in sequence i.  The call is bound
// by its launch, so one kernel does all of it: every block repeats the scan (8 bytes
// a sequence, out of L2) instead of waiting for another block's, and then writes its
// own share of the table's new entries and of the slots.  A slot whose page is new is
// taken from the free list itself, never from the table entry another block writes.  64
// sequences with a token each take 4.4 us on the device, 1024 with 115000 tokens 5.3 us.
//
// paged_append_kernel copies rows into their slots, 16 bytes a thread and step: a pure
// copy, bound by HBM (twice the rows' bytes): 65000 rows of 16 heads of 64 take 79 us, 6.76
// TB/s.
#pragma once
#include <cstdint>
#include <climits>

#include "paged_common_sm103.cuh"

namespace attn {
namespace paged {

constexpr int kTableThreads = 1024;  // sequences scanned per step

struct TableParams {
    const int *ctx_lens, *new_lens;
    const int *free_pages, *free_head;  // free_head: nullptr starts at the list's front
    int* table;
    int *cu_new, *kv_lens, *counts;
    long long* slot_map;
    long long table_stride;
    int n_seqs, n_free, max_pages, max_tokens, page_size;
    FastDiv by_page;
};

// Inclusive sum over the block of a pair of 64-bit values (every thread calls it).
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long ua = __shfl_up_sync(0xffffffffu, a, d), ub = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) a += ua, b += ub;
    }
    if (lane == 31) part[0][warp] = a, part[1][warp] = b;
    __syncthreads();
    if (warp == 0) {
        long long x = part[0][lane], y = part[1][lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long ux = __shfl_up_sync(0xffffffffu, x, d), uy = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) x += ux, y += uy;
        }
        part[0][lane] = x, part[1][lane] = y;
    }
    __syncthreads();
    if (warp > 0) a += part[0][warp - 1], b += part[1][warp - 1];
}

// Largest i in [0, n) with a[i] <= x, for ascending a with a[0] <= x.
__device__ __forceinline__ int last_at_most(const long long* a, int n, long long x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kTableThreads) paged_tables_kernel(const TableParams p) {
    __shared__ long long s_tok[kTableThreads], s_page[kTableThreads];  // tokens / new pages before the sequence
    __shared__ int s_ctx[kTableThreads], s_have[kTableThreads];
    __shared__ long long s_part[2][32];
    wait_for_primary();
    const int tid = threadIdx.x, G = gridDim.x, c = blockIdx.x;
    const long long head = p.free_head != nullptr ? max(*p.free_head, 0) : 0;
    // this block's share of the slot map
    const int t0 = static_cast<int>((long long)p.max_tokens * c / G);
    const int t1 = static_cast<int>((long long)p.max_tokens * (c + 1) / G);
    long long tok = 0, page = 0;  // of all sequences before the step's
    int too_long = 0;
    for (int s0 = 0; s0 < p.n_seqs; s0 += kTableThreads) {
        const int s = s0 + tid, n = min(kTableThreads, p.n_seqs - s0);
        int ctx = 0, fresh = 0, have = 0, want = 0;
        long long kv = 0;
        if (tid < n) {
            ctx = max(p.ctx_lens[s], 0);
            fresh = max(p.new_lens[s], 0);
            kv = (long long)ctx + fresh;
            const long long last = (long long)p.by_page.quot(kv + p.page_size - 1);
            have = static_cast<int>(min((long long)p.by_page.quot((long long)ctx + p.page_size - 1), (long long)p.max_pages));
            want = static_cast<int>(min(last, (long long)p.max_pages));
            too_long += last > p.max_pages;
        }
        long long a = fresh, b = want - have;
        block_scan2(a, b, s_part);  // ends with every thread past its last read of the step before
        s_tok[tid] = tok + a - fresh;
        s_page[tid] = page + b - (want - have);
        s_ctx[tid] = ctx;
        s_have[tid] = have;
        if (c == 0 && tid < n) {
            p.cu_new[s + 1] = static_cast<int>(min(tok + a, (long long)INT_MAX));
            p.kv_lens[s] = static_cast<int>(min(kv, (long long)INT_MAX));
        }
        const long long tok_end = tok + s_part[0][31], page_end = page + s_part[1][31];
        __syncthreads();
        // this block's share of the step's new table entries
        const long long pages = page_end - page;
        for (long long i = page + pages * c / G + tid; i < page + pages * (c + 1) / G; i += kTableThreads) {
            const int j = last_at_most(s_page, n, i);
            const long long at = head + i;
            p.table[(s0 + j) * p.table_stride + s_have[j] + (i - s_page[j])] = at < p.n_free ? p.free_pages[at] : -1;
        }
        // the slots of this block's tokens that belong to the step's sequences
        for (long long t = max((long long)t0, tok) + tid; t < min((long long)t1, tok_end); t += kTableThreads) {
            const int j = last_at_most(s_tok, n, t);
            const long long pos = s_ctx[j] + (t - s_tok[j]);
            const long long col = (long long)p.by_page.quot(pos);
            int entry = -1;
            if (col < s_have[j]) {
                entry = p.table[(s0 + j) * p.table_stride + col];
            } else if (col < p.max_pages) {
                const long long at = head + s_page[j] + (col - s_have[j]);
                if (at < p.n_free) entry = p.free_pages[at];
            }
            p.slot_map[t] = entry < 0 ? -1ll : (long long)entry * p.page_size + (pos - col * p.page_size);
        }
        tok = tok_end;
        page = page_end;
        __syncthreads();
    }
    launch_dependents();  // late: with it in front the next kernel's blocks cost 1024 sequences 2 us
    for (long long t = max((long long)t0, tok) + tid; t < t1; t += kTableThreads) p.slot_map[t] = -1;
    if (c == 0) {
        long long x = too_long, unused = 0;
        block_scan2(x, unused, s_part);
        if (tid == kTableThreads - 1) {
            const long long left = max((long long)p.n_free - head, 0ll), taken = min(page, left);
            p.cu_new[0] = 0;
            p.counts[0] = static_cast<int>(min(tok, (long long)INT_MAX));
            p.counts[1] = static_cast<int>(min(head + taken, (long long)INT_MAX));
            p.counts[2] = static_cast<int>(min(page - taken, (long long)INT_MAX));
            p.counts[3] = static_cast<int>(x);
        }
    }
}

constexpr int kAppendThreads = 256;

struct AppendParams {
    const uint16_t *k, *v;  // rows [T, Hkv, D], heads contiguous
    uint16_t *k_cache, *v_cache;
    const long long* slot_map;
    long long k_stride, v_stride;                      // elements from row to row
    long long page_stride, token_stride, head_stride;  // of both caches, in elements
    long long n_slots;
    int T, per_block;      // rows, rows of one block
    int row_chunks;        // 16-byte pieces of a row: Hkv * D / 8
    int head_chunks_log2;  // of one head: D / 8
    FastDiv by_page, by_row;
};

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendParams p) {
    launch_dependents();
    wait_for_primary();
    const long long row0 = (long long)blockIdx.x * p.per_block;
    const unsigned int n = static_cast<unsigned int>(min((long long)p.per_block, p.T - row0)) * p.row_chunks;
    for (unsigned int i = threadIdx.x; i < n; i += kAppendThreads) {
        const unsigned int r = static_cast<unsigned int>(p.by_row.quot(i));
        const unsigned int ch = i - r * p.row_chunks;
        const long long slot = p.slot_map[row0 + r];
        if (slot < 0 || slot >= p.n_slots) continue;
        const long long page = (long long)p.by_page.quot(slot);
        const long long to = page * p.page_stride + (slot - page * p.by_page.d) * p.token_stride +
                             (ch >> p.head_chunks_log2) * p.head_stride + ((ch & ((1u << p.head_chunks_log2) - 1)) << 3);
        const uint4 a = *reinterpret_cast<const uint4*>(p.k + (row0 + r) * p.k_stride + ch * 8ll);
        const uint4 b = *reinterpret_cast<const uint4*>(p.v + (row0 + r) * p.v_stride + ch * 8ll);
        *reinterpret_cast<uint4*>(p.k_cache + to) = a;
        *reinterpret_cast<uint4*>(p.v_cache + to) = b;
    }
}

}  // namespace paged
}  // namespace attn

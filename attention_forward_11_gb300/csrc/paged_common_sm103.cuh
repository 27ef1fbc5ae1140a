// paged_common_sm103.cuh -- what the kernels of the paged key/value cache share:
// the division by the page size, the launch parameters, and how a ragged batch's
// lengths are read.
//
// A cache holds pages of `page_size` tokens; token t of sequence s lives at row
// t % page_size of page table[s, t / page_size].  Lengths and tables are device
// data that no host code sees, so every value is clamped where it is read: a
// query range to the rows that exist, a key length to what the table's columns
// can name, and a page that is not in [0, n_pages) holds no keys.
#pragma once
#include <cstdint>

namespace attn {
namespace paged {

// n / d for 0 <= n < 2^64 / d as one high product: with m = floor(2^64 / d) + 1,
// n m / 2^64 exceeds n / d by n (m d - 2^64) / (d 2^64) <= n / 2^64 < 1 / d.
struct FastDiv {
    unsigned long long m = 0;  // 0: the divisor is one
    unsigned int d = 1;
    __device__ __forceinline__ unsigned long long quot(unsigned long long n) const {
        return m == 0 ? n : __umul64hi(n, m);
    }
};
inline FastDiv make_fastdiv(unsigned int d) {
    FastDiv f;
    f.d = d;
    f.m = d == 1 ? 0ull : ~0ull / d + 1;
    return f;
}

struct PagedParams {
    const uint16_t *q, *k, *v;  // queries [total_q, Hq, D] and the two caches
    uint16_t* o;                // [total_q, Hq, D]
    float* lse;                 // [Hq, total_q], or nullptr
    const int *table, *cu_q, *kv_lens;
    int n_seqs, total_q, Hq, Hkv, group, n_pages, page_size, max_pages, causal;
    int max_kv;                                       // keys that a table row can name
    long long q_stride, table_stride;                 // elements from token to token, row to row
    long long page_stride, token_stride, head_stride;  // of both caches, in elements
    float scale_log2;                                 // softmax scale * log2(e)
    FastDiv by_page;
    // A batch shared by two kernels: sequences of at most split_rows (token, head) rows a
    // key/value head are the first one's (take_short), the others the second one's.  0: all.
    int split_rows, take_short;
};

struct Seq {
    int q0, q_len, kv_len;
};

__device__ __forceinline__ Seq seq_of(const PagedParams& p, int s) {
    Seq x;
    x.q0 = min(max(p.cu_q[s], 0), p.total_q);
    x.q_len = max(min(p.cu_q[s + 1], p.total_q) - x.q0, 0);
    x.kv_len = min(max(p.kv_lens[s], 0), p.max_kv);
    if (p.split_rows != 0 && (x.q_len * p.group <= p.split_rows) != (p.take_short != 0)) x.q_len = 0;
    return x;
}

// Keys that token t of a sequence sees: [0, visible).  Causal masks are aligned at
// the end: the last new token sees every key.
__device__ __forceinline__ int visible_keys(const PagedParams& p, const Seq& x, int t) {
    return p.causal ? max(x.kv_len - x.q_len + t + 1, 0) : x.kv_len;
}

// Programmatic launch: a kernel's blocks may be in place before the kernel in front of it
// has ended; every thread waits for that end before it touches memory.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Reads a word of every 64 bytes of a kernel's parameters, whose first reads miss one after
// another otherwise (a block calls it before it waits for the kernel in front).
template <class P>
__device__ __forceinline__ void touch_params(const P& p) {
    const int* w = reinterpret_cast<const int*>(&p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(P) / 4); i += 16) asm volatile("" ::"r"(w[i]));
}

}  // namespace paged
}  // namespace attn

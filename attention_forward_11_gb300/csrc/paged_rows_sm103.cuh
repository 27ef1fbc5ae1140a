// paged_rows_sm103.cuh -- attention of a few query rows over a paged cache (decode,
// drafted tokens, short chunks).
//
// The rows of a unit are the (token, query head) pairs of one sequence that share a
// key/value head, token by token: row r is token r / group, head r % group of the
// group.  Up to 8 kNB rows are computed together, so a cache row is read once for all
// of them.  With so few rows the call is bound by the cache's bytes; the products only
// have to keep up, and the 128 query rows of a tcgen05 tile would be empty.  So keys
// are the long side of the warp-level products m16n8k16, rows the short one:
//   S^T [16 keys x 8 rows]  = K Q^T     A = K from shared memory, B = Q in registers
//   O^T [16 of D x 8 rows] += V^T P^T   A = V from shared memory transposed, B = P^T
// A warp owns a slice of every tile, 16 keys (32 at head size 64), and keeps its own running
// maximum, sum and O^T (online softmax in log2 units, fp32), so warps meet only at the end
// of a unit, where their (m, l, O) are merged in a fixed order.  P is rounded to the
// operands' type for its product, as in the dense forward: the product takes 16-bit operands,
// and a second one for the rest of the rounding would cost as much again.  Against 64 bits O
// is off by 2.1e-3 of its norm in bf16 and 2.7e-4 in fp16; O's own rounding alone is 1.7e-3
// and 2.1e-4.
//
// One block a SM takes an equal share of the batch (paged_sched_sm103.cuh); of the blocks
// that have a piece of one unit, the last to finish joins them.  Each warp
// fills a ring of its own with cp.async, two slices ahead of the one it computes and across
// the ends of units, with no barrier between warps: 16-byte copies follow any page size and
// any strides, and a slice's page numbers are read one slice earlier still.  192 KB of
// slices keep HBM busy: 256 sequences of 100 to 4000 keys take 320 us (6.6 TB/s of cache),
// 48 of 300 to 8000 113 us (6.0 TB/s).  Short calls are a block's start (4 us to the first
// copies) and end (merge and join, 5 us): 8 sequences of 32768 keys 29.1 us (19.8 at HBM's
// rate), one of 1000 keys 9.5 us.
#pragma once
#include <cmath>
#include <cstdint>

#include "paged_common_sm103.cuh"
#include "paged_sched_sm103.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// transpose of an 8x8 matrix of 16-bit values held across the warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// c += a b: a [16 x 16], b [16 x 8], fp32 sums
template <bool kF16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes global -> shared, or 16 zero bytes
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

template <int kD, int kNB>
struct RowsGeo {
    static constexpr int kWarps = kD == 256 ? 4 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * kNB;
    static constexpr int kKS = kD == 64 ? 2 : 1;        // 16-key blocks of a warp's slice
    static constexpr int kSlice = 16 * kKS;             // keys of a slice
    static constexpr int kTileKeys = kSlice * kWarps;   // keys of all warps in one step
    static constexpr int kSliceBytes = kSlice * kD * 2; // K or V rows of a slice
    static constexpr int kChunks = kD / 8;              // 16-byte pieces of a row
    static constexpr int kStages = 3;                   // 192 KB of slices
    static constexpr int kMergeCols = 64;               // columns of O merged at a time
    static constexpr int kMergeStride = kMergeCols + 4; // floats; rows 2 t of a warp fall into different banks
    static constexpr int kRing = kWarps * kStages * 2 * kSliceBytes;
    static constexpr int kMerge = kWarps * 8 * kMergeStride * 4;
    static constexpr int kStats = kWarps * kRows * 8;
    static constexpr int kSmemBytes = kRing + kMerge + kStats;
    static_assert(kSmemBytes <= 231000, "ring, merge buffer and static shared memory exceed 227 KB");
    static_assert(kMerge >= kThreads / (kD / 4) * (kD + 4) * 4, "joined rows do not fit the merge buffer");
    // a piece is worth its merge from two tiles on, and so is a share (one sequence of 1000 or
    // 5000 keys, 8 heads: 9.7 and 10.9 us; shares of at least 4 tiles 11.1 and 11.4, 8 tiles
    // 11.0 and 15.3); units up to 8 tiles longer than a share stay whole
    static constexpr int kMinPiece = 2, kMinShare = 2, kCutTiles = 8;
    using ShareT = Share<kTileKeys, kMinPiece, kMinShare>;
    using CursorT = Cursor<ShareT, kTileKeys>;
};

// Joins the n pieces of a unit that block `first` started: M = max m, L = sum l 2^(m - M),
// O = sum O 2^(m - M) / L.  kD / 4 threads have a row (four columns each), or, when there are
// fewer rows than such groups, a part of a row's pieces; `buf` is shared scratch of a row and
// its sum for every group.  A block does this alone at its end, so what counts is how many
// loads wait on one another: 20 pieces are in flight at once, the first before M is known.
template <bool kF16, int kD, int kRows, int kThreads>
__device__ __forceinline__ void join_pieces(const PagedParams& p, const SchedParams& sp, const Seq& x, int head_unit, int t0,
                                            int first, int n, float* buf) {
    constexpr int kLanes = kD / 4, kGroups = kThreads / kLanes, kFly = 20;
    constexpr int kSpan = kLanes < 32 ? kLanes : 32;  // lanes that share a search for M
    const int group = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 4, lane = threadIdx.x % kSpan;
    const int rows = min(min(sp.map.tokens, x.q_len - t0) * sp.map.heads, kRows);
    int parts = 1;
    while (2 * parts * rows <= kGroups) parts *= 2;
    const int part = group % parts;
    for (int r0 = 0; r0 < rows; r0 += kGroups / parts) {
        const int r = min(r0 + group / parts, kRows - 1);  // rows past the last are computed and not stored
        const Row w = row_of(p, sp.map, x, head_unit, t0, sp.map.tokens, r);
        const bool mine = r0 + group / parts < rows && w.there;
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = part; i0 == part || i0 < n; i0 += kFly * parts) {  // the first step is every thread's
            float2 ml[kFly];
            float4 v[kFly];
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const int i = i0 + j * parts;
                ml[j] = make_float2(-INFINITY, 0.f);
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine && i < n) {
                    const size_t row = (size_t)piece_slot(first, i) * kRows + r;
                    ml[j] = __ldcg(sp.ws.ml + row);
                    v[j] = __ldcg(reinterpret_cast<const float4*>(sp.ws.o + row * kD + col));
                }
            }
            if (i0 == part) {
                for (int i = lane; mine && i < n; i += kSpan)
                    M = fmaxf(M, __ldcg(sp.ws.ml + (size_t)piece_slot(first, i) * kRows + r).x);
#pragma unroll
                for (int d = kSpan / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
            }
            const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const float f = ex2_approx(ml[j].x - use);
                L += ml[j].y * f;
                acc.x += v[j].x * f;
                acc.y += v[j].y * f;
                acc.z += v[j].z * f;
                acc.w += v[j].w * f;
            }
        }
        if (parts > 1) {
            float* to = buf + group * (kD + 4);
            *reinterpret_cast<float4*>(to + col) = acc;
            if (col == 0) to[kD] = L;
            __syncthreads();
            if (part == 0)
                for (int k = 1; k < parts; ++k) {
                    const float* from = buf + (group + k) * (kD + 4);
                    const float4 y = *reinterpret_cast<const float4*>(from + col);
                    acc.x += y.x;
                    acc.y += y.y;
                    acc.z += y.z;
                    acc.w += y.w;
                    L += from[kD];
                }
        }
        if (!mine || part != 0) continue;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const size_t tok = (size_t)x.q0 + w.token;
        *reinterpret_cast<uint2*>(p.o + (tok * p.Hq + w.head) * kD + col) =
            make_uint2(pack_x2<kF16>(acc.x * inv, acc.y * inv), pack_x2<kF16>(acc.z * inv, acc.w * inv));
        if (col == 0 && p.lse != nullptr)
            p.lse[(size_t)w.head * p.total_q + tok] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
}

template <bool kF16, int kD, int kNB>
__global__ void __launch_bounds__(RowsGeo<kD, kNB>::kThreads, 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ SchedParams sp) {
    using G = RowsGeo<kD, kNB>;
    constexpr int kKS = G::kKS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_part[3 * G::kWarps];
    __shared__ StartPos s_start;
    __shared__ uint32_t s_valid[G::kWarps][G::kStages];  // keys of a slice that have a page
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (G::kStages * 2 * G::kSliceBytes);
    float* merge = reinterpret_cast<float*>(smem + G::kRing);
    float2* stats = reinterpret_cast<float2*>(smem + G::kRing + G::kMerge);
    launch_dependents();
    touch_params(p);
    touch_params(sp);
    wait_for_primary();

    typename G::ShareT sh;
    const bool some = find_share<G::kThreads, typename G::ShareT, G::kTileKeys, G::kMinShare, G::kCutTiles, false>(p, sp, s_part, &s_start, sh);
    if (!some) return;
    typename G::CursorT cur;
    cur.first(p, sp, sh, s_start);
    typename G::CursorT ld = cur;  // the copies' position, ahead of the products'
    int ld_tile = ld.tile;
    // the counts of the pieces at this share's ends (ready before any is counted)
    CountWord counts[2];
    if (tid == G::kThreads - 1) {
        counts[0] = look_at_count(sp.ws.count(static_cast<int>(blockIdx.x)));
        counts[1] = look_at_count(sp.ws.count(cur.ok && cur.tile > 0 ? sh.starter(cur.at) : static_cast<int>(blockIdx.x)));
    }

    // The page numbers of the next slices to copy: lane i has that of key i % kSlice.  A slice
    // is looked up when the one before it is copied, the first three together.
    struct Look {
        int page, row;    // page number and row of this lane's key
        int hkv;          // key/value head
        bool some;        // the slice has keys
        bool ok;          // there is such a slice
    };
    auto look_up = [&](Look& k) {
        k.page = -1;
        k.ok = ld.ok;
        if (!ld.ok) return;
        const int key = ld_tile * G::kTileKeys + G::kSlice * warp + (lane & (G::kSlice - 1));
        k.some = ld_tile * G::kTileKeys + G::kSlice * warp < ld.keys;
        k.hkv = sp.map.kv_head(ld.head_unit);
        if (key < ld.keys) {
            const int col = static_cast<int>(p.by_page.quot(key));
            k.page = p.table[ld.s * p.table_stride + col];
            k.row = key - col * p.page_size;
        }
        if (++ld_tile == ld.tile_end) {
            ld.next(p, sp, sh);
            ld_tile = ld.tile;
        }
    };
    // Copies a slice into a stage.  A lane has 16 bytes of every (32 / kChunks)-th row.
    constexpr int kRowsAtOnce = 32 / G::kChunks, kCopies = 16 / kRowsAtOnce;  // of a 16-key block
    const int lane_row = lane / G::kChunks, lane_chunk = lane % G::kChunks;
    const long long lane_at = lane_row * p.token_stride + lane_chunk * 8;
    const bool blocks_in_pages = p.page_size % 16 == 0;
    auto copy = [&](const Look& k, int st) {
        if (k.ok) {
            const bool there = k.page >= 0 && k.page < p.n_pages;
            const long long base = there ? k.page * p.page_stride + k.row * p.token_stride + k.hkv * p.head_stride : 0;
            const uint32_t valid = __ballot_sync(0xffffffffu, there);
            if (lane == 0) s_valid[warp][st] = valid;
            const uint32_t to = ring + st * (2 * G::kSliceBytes);
            auto place = [&](int row) { return to + row * (kD * 2) + ((lane_chunk ^ (row & 7)) << 4); };
            if (blocks_in_pages && valid == 0xffffffffu) {
                // 16 keys of one page each: a third of the instructions of the other way
#pragma unroll
                for (int b = 0; b < kKS; ++b) {
                    const long long at = __shfl_sync(0xffffffffu, base, 16 * b) + lane_at;
                    const uint16_t *pk = p.k + at, *pv = p.v + at;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const uint32_t dst = place(16 * b + lane_row + i * kRowsAtOnce);
                        cp_async16(dst, pk);
                        cp_async16(dst + G::kSliceBytes, pv);
                        pk += kRowsAtOnce * p.token_stride;
                        pv += kRowsAtOnce * p.token_stride;
                    }
                }
            } else if (k.some) {
#pragma unroll
                for (int i = 0; i < kKS * kCopies; ++i) {
                    const int row = lane_row + i * kRowsAtOnce;
                    const long long at = __shfl_sync(0xffffffffu, base, row) + lane_chunk * 8;
                    const bool ok = (valid >> row) & 1;
                    cp_async16(place(row), p.k + at, ok);
                    cp_async16(place(row) + G::kSliceBytes, p.v + at, ok);
                }
            }
        }
        cp_async_commit();
    };
    static_assert(G::kStages == 3, "two slices are copied ahead");
    Look next;
    {
        Look k0, k1;
        look_up(k0);
        look_up(k1);
        look_up(next);
        copy(k0, 0);
        copy(k1, 1);
    }
    if (tid == G::kThreads - 1) {
        begin_count(counts[0], sp.tag);
        if (counts[1].word != counts[0].word) begin_count(counts[1], sp.tag);
    }
    int st = 0;

#pragma unroll 1
    for (; cur.ok; cur.next(p, sp, sh)) {
        const Seq x = cur.x;
        const int t0 = cur.row_unit * sp.map.tokens;
        // Q^T as the products' B operand: row n0 + g, elements 16 ks + 2 t4 (+ 8)
        uint32_t qf[kNB][kD / 16][2];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
            const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + g);
            const uint16_t* src = p.q + (w.there ? (x.q0 + w.token) * p.q_stride + w.head * kD : 0);
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                qf[nb][ks][0] = w.there ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * t4) : 0u;
                qf[nb][ks][1] = w.there ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 + 2 * t4) : 0u;
            }
        }
        // this thread's two rows of every row block: 2 t4 and 2 t4 + 1
        int lim[kNB][2], all_see = 0x7fffffff;  // keys that every row sees
        float m[kNB][2], l[kNB][2], o[kNB][kD / 16][4];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + 2 * t4 + e);
                lim[nb][e] = w.there ? visible_keys(p, x, w.token) : 0x7fffffff;  // a row that is none masks nothing
                all_see = min(all_see, lim[nb][e]);
                m[nb][e] = -INFINITY;
                l[nb][e] = 0.f;
            }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, d));
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][mt][e] = 0.f;

#pragma unroll 1
        for (int tile = cur.tile; tile < cur.tile_end; ++tile) {
            cp_async_wait<G::kStages - 2>();
            __syncwarp();  // the slice is there, and every lane is done with the one before
            copy(next, st == 0 ? G::kStages - 1 : st - 1);
            look_up(next);
            const int k0 = tile * G::kTileKeys + G::kSlice * warp;
            const uint32_t from = ring + st * (2 * G::kSliceBytes);
            const uint32_t valid = s_valid[warp][st];
            if (k0 < cur.keys) {
                // one product after another would wait for the sum: a single chain is cut in two
                constexpr bool kTwoSums = kNB * kKS == 1;
                float sc[kNB][kKS][4], sc2[kNB][kKS][4];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                    for (int b = 0; b < kKS; ++b) {
                        sc[nb][b][0] = sc[nb][b][1] = sc[nb][b][2] = sc[nb][b][3] = 0.f;
                        sc2[nb][b][0] = sc2[nb][b][1] = sc2[nb][b][2] = sc2[nb][b][3] = 0.f;
                    }
                {
                    const int kk = (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t a0 = from + kk * (kD * 2);
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
                        for (int b = 0; b < kKS; ++b) {
                            uint32_t a[4];
                            ldsm_x4(a, a0 + b * (16 * kD * 2) + (((2 * ks + (lane >> 4)) ^ (kk & 7)) << 4));
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb)
                                mma_16816<kF16>(kTwoSums && (ks & 1) ? sc2[nb][b] : sc[nb][b], a, qf[nb][ks][0], qf[nb][ks][1]);
                        }
                    if constexpr (kTwoSums)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[0][0][e] += sc2[0][0][e];
                }
                if (k0 + G::kSlice > all_see || valid != 0xffffffffu) {
#pragma unroll
                    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                        for (int b = 0; b < kKS; ++b)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kk = 16 * b + 8 * (e / 2) + g;
                                if (!((valid >> kk) & 1) || k0 + kk >= lim[nb][e % 2]) sc[nb][b][e] = -INFINITY;
                            }
                }
                uint32_t pf[kNB][kKS][2];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) {
                    // element e of block b: key k0 + 16 b + g + 8 (e / 2), row 2 t4 + e % 2
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int b = 0; b < kKS; ++b)
#pragma unroll
                            for (int u = 0; u < 2; ++u) mx = fmaxf(mx, sc[nb][b][2 * u + e]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        const float mn = fmaxf(m[nb][e], mx * p.scale_log2), use = mn == -INFINITY ? 0.f : mn;
                        al[e] = ex2_approx(m[nb][e] - use);
                        m[nb][e] = mn;
                        float sum = 0.f;
#pragma unroll
                        for (int b = 0; b < kKS; ++b)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float& y = sc[nb][b][2 * u + e];
                                y = ex2_approx(fmaf(y, p.scale_log2, -use));
                                sum += y;
                            }
                        l[nb][e] = l[nb][e] * al[e] + sum;
                    }
                    // the maximum settles after a few slices: most leave O as it is
                    if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
                        for (int mt = 0; mt < kD / 16; ++mt) {
                            o[nb][mt][0] *= al[0];
                            o[nb][mt][1] *= al[1];
                            o[nb][mt][2] *= al[0];
                            o[nb][mt][3] *= al[1];
                        }
                    }
#pragma unroll
                    for (int b = 0; b < kKS; ++b) {
                        pf[nb][b][0] = movmatrix(pack_x2<kF16>(sc[nb][b][0], sc[nb][b][1]));
                        pf[nb][b][1] = movmatrix(pack_x2<kF16>(sc[nb][b][2], sc[nb][b][3]));
                    }
                }
                {
                    const int kk = (lane & 7) + (lane >> 4) * 8;
                    const uint32_t a0 = from + G::kSliceBytes + kk * (kD * 2);
#pragma unroll
                    for (int b = 0; b < kKS; ++b)
#pragma unroll
                        for (int mt = 0; mt < kD / 16; ++mt) {
                            uint32_t a[4];
                            ldsm_x4_trans(a, a0 + b * (16 * kD * 2) + (((2 * mt + ((lane >> 3) & 1)) ^ (kk & 7)) << 4));
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb)
                                mma_16816<kF16>(o[nb][mt], a, pf[nb][b][0], pf[nb][b][1]);
                        }
                }
            }
            st = st + 1 == G::kStages ? 0 : st + 1;
        }

        // merge the warps: M = max m, L = sum l 2^(m - M), O = sum O 2^(m - M) (/ L when the unit is whole)
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
                if (g == 0) stats[warp * G::kRows + 8 * nb + 2 * t4 + e] = make_float2(m[nb][e], l[nb][e]);
            }
        const bool whole = cur.whole();
        const int slot = 2 * static_cast<int>(blockIdx.x) + (cur.tile == 0 ? 1 : 0);
        constexpr int kParts = kD / G::kMergeCols;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                __syncthreads();  // the stats are there; what was merged before has been read
#pragma unroll
                for (int mt = 0; mt < G::kMergeCols / 16; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        merge[(warp * 8 + 2 * t4 + (e & 1)) * G::kMergeStride + 16 * mt + g + 8 * (e >> 1)] =
                            o[nb][part * (G::kMergeCols / 16) + mt][e];
                __syncthreads();
#pragma unroll
                for (int i = tid; i < 8 * (G::kMergeCols / 2); i += G::kThreads) {
                    const int r = i / (G::kMergeCols / 2), dc = (i % (G::kMergeCols / 2)) * 2, d = part * G::kMergeCols + dc;
                    const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + r);
                    if (!w.there) continue;
                    float M = -INFINITY, L = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
                    for (int k = 0; k < G::kWarps; ++k) M = fmaxf(M, stats[k * G::kRows + 8 * nb + r].x);
                    const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int k = 0; k < G::kWarps; ++k) {
                        const float2 ml = stats[k * G::kRows + 8 * nb + r];
                        const float f = ex2_approx(ml.x - use);
                        const float2 v = *reinterpret_cast<const float2*>(merge + (k * 8 + r) * G::kMergeStride + dc);
                        L += ml.y * f;
                        a0 += v.x * f;
                        a1 += v.y * f;
                    }
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        const long long tok = x.q0 + w.token;
                        *reinterpret_cast<uint32_t*>(p.o + (tok * p.Hq + w.head) * kD + d) = pack_x2<kF16>(a0 * inv, a1 * inv);
                        if (d == 0 && p.lse != nullptr)
                            p.lse[(long long)w.head * p.total_q + tok] =
                                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
                    } else {
                        const size_t row = (size_t)slot * G::kRows + 8 * nb + r;
                        *reinterpret_cast<float2*>(sp.ws.o + row * kD + d) = make_float2(a0, a1);
                        if (d == 0) sp.ws.ml[row] = make_float2(M, L);
                    }
                }
            }
        __syncthreads();  // the stats may be overwritten; a piece is written
        if (!whole) {
            const int first = cur.tile == 0 ? static_cast<int>(blockIdx.x) : sh.starter(cur.at);
            const int n = sh.pieces(cur.at, cur.tiles, first);
            if (tid == 0) s_last = count_piece(sp.ws.count(first), n);
            __syncthreads();
            if (s_last) join_pieces<kF16, kD, G::kRows, G::kThreads>(p, sp, x, cur.head_unit, t0, first, n, merge);
            __syncthreads();
        }
    }
    cp_async_wait<0>();
}

}  // namespace paged
}  // namespace attn

// paged4_rows_sm103.cuh -- attention of a few query rows over a paged cache in 4 bits (decode,
// drafted tokens, short chunks).
//
// The kernel is paged_rows_sm103.cuh's: keys are the long side of the products m16n8k16, a warp
// owns a slice of every tile with its own ring of cp.async copies and its own softmax state,
// shares and pieces as in paged_sched_sm103.cuh.  A key has 0.28 of the bytes, so a call is bound
// by its instructions: at HBM's rate a scheduler has 392 cycles for 16 keys of head size 128, and
// the 64 conversions, 64 scalings (two cycles each, on ports that they share) and 16 products
// alone take 256.  What is left is kept small:
//   - No operand is put together from its rows and columns: the products' sums run over any order
//     of their terms, and every lane takes the elements that lie together.
//     S^T = K Q^T: lane (g, t) has the t-th quarter of the rows of keys g and g + 8, elements 4 j to
//     4 j + 3 of it for product j, read as whole words; Q is loaded in the same order.
//     O^T += V^T P^T: lane (g, t) has the g-th eighth of the rows of its four keys, and product j
//     gives elements 2 j and 2 j + 1 of it.  A pair of the operand is one element of two keys, so
//     two keys' nibbles are laid side by side (two instructions for four pairs) before they are
//     converted.  The scales of both are one or two a key and lane.
//   - The maximum that weights are relative to rises only when a logit is past it (kMaxAbove; 164 to
//     154 us for 144 sequences of 300 to 8000 keys, 64/8 heads of 128).
//   - Where there are many units, a block is teams of four warps, each with a share of its own: a
//     unit's start and end are four warps' work, not all of them's.  Up to 8 rows at head sizes 64
//     and 128 there are four teams (198 to 164 us), which leaves 128 registers a thread, so the share
//     and both positions in it live in shared memory; otherwise two (48 sequences at head size 256
//     135 to 119 us, 64 times 5 drafted tokens of 4 heads at 128 152 to 144).
//   - A unit's own cost is reckoned as 512 or 1024 keys (256 in the 16-bit kernel): 223 to 208 us.
// The keys' order within 16 (slot r is key perm(r)) and a swizzle of 16-byte pieces keep all reads
// free of bank conflicts.  L2 is asked for no more than a row of codes, since the next 64 bytes
// belong to another head where pages are stored token by token (280 to 203 us).
//
// 144 sequences as above take 152 us, 4.8 TB/s of cache (48 of them 60, in 16 bits 134); the same heads of 64
// 103 us; 8 of 32768 keys, one key head, 20 us (30 in 16 bits); one of 1000 keys, 8 heads, 11 us (10), a
// block's start and end.  Stored token by token 144 take 204 us (heads of 64 213): a head's 64 or 32 bytes of codes
// and 8 or 4 of scales lie apart from the next token's, and 1.15 GB are read for 0.73.  No unit is full at 152 us:
// 2.6 instructions a cycle of 4, ALU pipe 55 %, DRAM 58 %; what a key costs whatever its head size (look-ups,
// addresses, masks, maximum, exponentials) is a third of the time at 128 and half at 64.  Drafted tokens (16 x 5,
// 4 heads of 64 a key head: 38 us, 6 of bytes) issue 1.1 instructions a cycle: a third of a warp's time waits for
// instructions to be fetched, since three row blocks unrolled are more code than the cache nearest to the
// schedulers holds, and eight warps hide little.  Bulk copies of 1 KB in place of cp.async took 175 us, slices of
// 16 keys 189.
//
// P is rounded to fp16 for its product whatever q's type, which the products' operands are too:
// against 64 bits O is off by 1.7e-3 of its norm in bf16 and 2.5e-4 to 2.9e-4 in fp16, of which O's own rounding is
// 1.65e-3 and 2.1e-4.
#pragma once
#include <cmath>
#include <cstdint>

#include "paged4_common_sm103.cuh"
#include "paged_rows_sm103.cuh"
#include "paged_sched_sm103.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

// 16 bytes global -> shared, or 16 zero bytes, of rows of kRow bytes that may lie apart: L2 is not
// asked for more than a row
template <int kRow>
__device__ __forceinline__ void cp_async_row16(uint32_t dst, const void* src, bool there) {
    if constexpr (kRow >= 128)
        cp_async16(dst, src, there);
    else if constexpr (kRow == 64)
        asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// 4 or 8 bytes global -> shared, or as many zero bytes
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool there) {
    if constexpr (kBytes == 16)
        cp_async16(dst, src, there);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(there ? kBytes : 0)
                     : "memory");
}
template <int kBytes>
__device__ __forceinline__ uint32_t lds_bytes(uint32_t at) {
    uint32_t v;
    if constexpr (kBytes == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    else if constexpr (kBytes == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void lds_x4(uint32_t* r, uint32_t at) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void lds_x2(uint32_t* r, uint32_t at) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
}

template <int kD, int kNB, bool kMany>
struct Rows4Geo {
    // kMany: teams of four warps, as many as the registers allow
    static constexpr int kWarps = kMany && kNB == 1 && kD <= 128 ? 16 : 8;
    static constexpr int kTeams = kMany ? kWarps / 4 : 1;  // of a block, each with a share of its own
    static constexpr int kTeamWarps = kWarps / kTeams;
    static constexpr int kThreads = 32 * kWarps, kTeamThreads = 32 * kTeamWarps;
    static constexpr int kRows = 8 * kNB;
    static constexpr int kKS = kD == 256 ? 1 : 2;       // 16-key blocks of a warp's slice
    static constexpr int kSlice = 16 * kKS;
    static constexpr int kTileKeys = kSlice * kTeamWarps;  // of a team's step
    static constexpr int kCodeRow = kD / 2, kScaleRow = kD / 16;  // bytes of a key
    static constexpr int kCodeBytes = kSlice * kCodeRow, kScaleBytes = kSlice * kScaleRow;
    // a stage: K codes, V codes, K scales, V scales
    static constexpr int kV = kCodeBytes, kScales = 2 * kCodeBytes, kVScales = kScales + kScaleBytes;
    static constexpr int kStageBytes = 2 * (kCodeBytes + kScaleBytes);
    static constexpr int kStages = kWarps == 16 ? (kD == 64 ? 4 : 2) : kD == 64 ? 6 : 4;
    static constexpr int kChunks = kCodeRow / 16;  // 16-byte pieces of a row
    static constexpr int kMergeCols = 64;
    static constexpr int kMergeStride = kMergeCols + 2;  // rows 2 t of a warp, and 2 t + 1, fall into different banks
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kMerge = kWarps * 8 * kMergeStride * 4;
    static constexpr int kStats = kWarps * kRows * 8;
    static constexpr int kSmemBytes = kRing + kMerge + kStats;
    static_assert(kSmemBytes <= 231000, "ring, merge buffer and static shared memory exceed 227 KB");
    static_assert(kMerge / kTeams >= kTeamThreads / (kD / 4) * (kD + 4) * 4, "joined rows do not fit the merge buffer");
    static constexpr int kJoinFly = kWarps == 16 ? 8 : 20;  // pieces in flight, as the registers allow
    static constexpr int kMinPiece = 2, kMinShare = 2, kCutTiles = 8;
    using ShareT = Share<kTileKeys, kMinPiece, kMinShare, kMany ? 512 : 1024>;
    using CursorT = Cursor<ShareT, kTileKeys>;
    // key of slot r of 16, and the 16-byte piece c of row r's place in the row
    __host__ __device__ static constexpr int perm(int r) {
        return kD == 128 ? r ^ ((r >> 1) & 1) : kD == 64 ? r ^ ((r >> 2) & 1) : r;
    }
    __host__ __device__ static constexpr int place(int r, int c) {
        return kD == 128 ? c ^ (((r >> 2) & 1) << 1) : kD == 64 ? c : c ^ (r & 7);
    }
};

// q's type is looked at where a unit begins and ends only, so one kernel takes both.
template <int kD, int kNB, bool kMany>
__global__ void __launch_bounds__(Rows4Geo<kD, kNB, kMany>::kThreads, 1)
    paged4_rows_kernel(const __grid_constant__ Paged4Params p, const __grid_constant__ SchedParams sp) {
    using G = Rows4Geo<kD, kNB, kMany>;
    constexpr int kKS = G::kKS, kStages = G::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_part[3 * G::kWarps];
    __shared__ StartPos s_start[G::kTeams];
    __shared__ uint32_t s_valid[G::kWarps][kStages];  // keys of a slice that have a page
    __shared__ int s_last[G::kTeams];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int team = warp / G::kTeamWarps, mate = warp % G::kTeamWarps;
    const int me = static_cast<int>(blockIdx.x) * G::kTeams + team;  // of all teams
    const int ttid = tid % G::kTeamThreads;
    auto meet = [&]() {  // of the team
        if constexpr (G::kTeams == 1) __syncthreads();
        else named_bar_sync(1 + team, G::kTeamThreads);
    };
    const uint32_t ring = smem_u32(smem) + warp * (kStages * G::kStageBytes);
    float* merge = reinterpret_cast<float*>(smem + G::kRing + team * (G::kMerge / G::kTeams));
    float2* stats = reinterpret_cast<float2*>(smem + G::kRing + G::kMerge + team * (G::kStats / G::kTeams));
    launch_dependents();
    touch_params(p);
    touch_params(sp);
    wait_for_primary();

    // The share and the two positions in it are looked at where a unit begins or ends only; kept in
    // registers they would take a third of a thread's.
    __shared__ typename G::ShareT s_sh[G::kTeams];
    __shared__ typename G::CursorT s_cur[G::kWarps], s_ld[G::kWarps];  // of the products, and of the copies ahead of them
    {
        typename G::ShareT sh;
        const bool some = find_share<G::kThreads, typename G::ShareT, G::kTileKeys, G::kMinShare, G::kCutTiles, false, G::kTeams>(
            p, sp, s_part, s_start, sh, team);
        if (!some || sh.begin == sh.end) return;  // the team's warps: they meet nobody but one another
        typename G::CursorT first;
        first.first(p, sp, sh, s_start[team]);
        if (ttid == 0) s_sh[team] = sh;
        if (lane == 0) s_cur[warp] = s_ld[warp] = first;
        // the counts of the pieces at this share's ends are made ready before any is counted
        if (ttid == G::kTeamThreads - 1) {
            const CountWord a = look_at_count(sp.ws.count(me));
            const CountWord b = look_at_count(sp.ws.count(first.ok && first.tile > 0 ? sh.starter(first.at) : me));
            begin_count(a, sp.tag);
            if (b.word != a.word) begin_count(b, sp.tag);
        }
        meet();
    }
    auto advance = [&](typename G::CursorT* at) {
        typename G::CursorT c = *at;
        c.next(p, sp, s_sh[team]);
        __syncwarp();
        if (lane == 0) *at = c;
        __syncwarp();
    };
    // where the copies are
    struct Ahead {
        const int* row;  // of the table
        int tile, tile_end, keys, hkv;
        bool ok;
    } ld;
    auto take = [&]() {
        const typename G::CursorT& c = s_ld[warp];
        ld.ok = c.ok;
        if (!c.ok) return;
        ld.row = p.table + c.s * p.table_stride;
        ld.tile = c.tile;
        ld.tile_end = c.tile_end;
        ld.keys = c.keys;
        ld.hkv = sp.map.kv_head(c.head_unit);
    };
    take();

    // The page numbers of the next slices to copy: lane i has that of key i % kSlice.  A slice
    // is looked up when the one before it is copied, the first ones together.
    struct Look {
        int page, row;    // page number and row of this lane's key
        int hkv;          // key/value head
        bool some;        // the slice has keys
        bool ok;          // there is such a slice
    };
    auto look_up = [&](Look& k) {
        k.page = -1;
        k.row = 0;
        k.ok = ld.ok;
        if (!ld.ok) return;
        const int first = ld.tile * G::kTileKeys + G::kSlice * mate, key = first + (lane & (G::kSlice - 1));
        k.some = first < ld.keys;
        k.hkv = ld.hkv;
        if (key < ld.keys) {
            const int col = static_cast<int>(p.by_page.quot(key));
            k.page = ld.row[col];
            k.row = key - col * p.page_size;
        }
        if (++ld.tile == ld.tile_end) {
            advance(&s_ld[warp]);
            take();
        }
    };
    // Copies a slice into a stage.  A lane has 16 bytes of every (32 / kChunks)-th row of codes,
    // and the scales of a row.
    constexpr int kRowsAtOnce = 32 / G::kChunks;
    const int lane_row = lane / G::kChunks, lane_chunk = lane % G::kChunks;
    const bool blocks_in_pages = p.page_size % 16 == 0;
    auto copy = [&](const Look& k, int st) {
        if (k.ok) {
            const bool there = k.page >= 0 && k.page < p.n_pages;
            const uint32_t valid = __ballot_sync(0xffffffffu, there);
            const uint32_t to = ring + st * G::kStageBytes;
            if (k.some) {
                if (lane == 0) s_valid[warp][st] = valid;
                const long long page = there ? k.page : 0;
                const long long base = page * p.page_stride + k.row * p.token_stride + k.hkv * p.head_stride;
                const long long scales = page * p.scale_page + k.row * p.scale_token + k.hkv * p.scale_head;
                if constexpr (kKS == 2) {
                    cp_async_small<G::kScaleRow>(to + G::kScales + lane * G::kScaleRow, p.k_scales + scales, there);
                    cp_async_small<G::kScaleRow>(to + G::kVScales + lane * G::kScaleRow, p.v_scales + scales, there);
                } else {
                    cp_async_small<G::kScaleRow>(to + G::kScales + lane * G::kScaleRow,
                                                 (lane < 16 ? p.k_scales : p.v_scales) + scales, there);
                }
                auto place = [&](int row) { return to + row * G::kCodeRow + G::place(row, lane_chunk) * 16; };
                if (blocks_in_pages && valid == 0xffffffffu) {
                    // 16 keys of one page each
                    const long long lane_at = lane_row * p.token_stride + lane_chunk * 16;
#pragma unroll
                    for (int b = 0; b < kKS; ++b) {
                        const long long at = __shfl_sync(0xffffffffu, base, 16 * b) + lane_at;
                        const uint8_t *pk = p.k_codes + at, *pv = p.v_codes + at;
#pragma unroll
                        for (int i = 0; i < 16; i += kRowsAtOnce) {
                            const uint32_t dst = place(16 * b + lane_row + i);
                            cp_async_row16<G::kCodeRow>(dst, pk, true);
                            cp_async_row16<G::kCodeRow>(dst + G::kV, pv, true);
                            pk += kRowsAtOnce * p.token_stride;
                            pv += kRowsAtOnce * p.token_stride;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < G::kSlice; i += kRowsAtOnce) {
                        const int row = lane_row + i;
                        const bool ok = (valid >> row) & 1;
                        const long long from = __shfl_sync(0xffffffffu, base, row);
                        const long long at = ok ? from + lane_chunk * 16 : 0;
                        cp_async_row16<G::kCodeRow>(place(row), p.k_codes + at, ok);
                        cp_async_row16<G::kCodeRow>(place(row) + G::kV, p.v_codes + at, ok);
                    }
                }
            }
        }
        cp_async_commit();
    };
    Look next;
    {
        Look first[kStages - 1];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) look_up(first[i]);
        look_up(next);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy(first[i], i);
    }
    int st = 0;

#pragma unroll 1
    for (; s_cur[warp].ok; advance(&s_cur[warp])) {
        // Q^T as the products' B operand: row n0 + g, elements 4 j to 4 j + 3 of this lane's quarter
        uint32_t qf[kNB][kD / 16][2];
        float back[kNB];  // what undoes the row's factor
        int lim[kNB][2], all_see = 0x7fffffff;  // keys that each of this thread's rows sees, and that every row sees
        float m[kNB][2], l[kNB][2], sl2[kNB][2], o[kNB][kD / 16][4];
        int tile, tile_end, keys;
        {
        const typename G::CursorT& cur = s_cur[warp];
        const Seq x = cur.x;
        const int t0 = cur.row_unit * sp.map.tokens;
        tile = cur.tile, tile_end = cur.tile_end, keys = cur.keys;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
            const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + g);
            const uint16_t* src = p.q + (w.there ? (x.q0 + w.token) * p.q_stride + w.head * kD + t4 * (kD / 4) : 0);
#pragma unroll
            for (int j = 0; j < kD / 16; ++j) {
                const uint2 y = w.there ? *reinterpret_cast<const uint2*>(src + 4 * j) : make_uint2(0u, 0u);
                qf[nb][j][0] = y.x;
                qf[nb][j][1] = y.y;
            }
            back[nb] = 1.f;
            if (!p.f16) {
                uint32_t top2 = 0;
#pragma unroll
                for (int j = 0; j < kD / 16; ++j)
                    top2 = __vmaxu2(top2, __vmaxu2(qf[nb][j][0] & 0x7fff7fffu, qf[nb][j][1] & 0x7fff7fffu));
                uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float factor = row_factor(top, back[nb]);
#pragma unroll
                for (int j = 0; j < kD / 16; ++j) {
                    qf[nb][j][0] = bf16x2_to_f16x2(qf[nb][j][0], factor);
                    qf[nb][j][1] = bf16x2_to_f16x2(qf[nb][j][1], factor);
                }
            }
        }
        // this thread's two rows of every row block: 2 t4 and 2 t4 + 1
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + 2 * t4 + e);
                lim[nb][e] = w.there ? visible_keys(p, x, w.token) : 0x7fffffff;  // a row that is none masks nothing
                all_see = min(all_see, lim[nb][e]);
                m[nb][e] = -INFINITY;
                l[nb][e] = 0.f;
                sl2[nb][e] = row_scale(p.scale_log2, __shfl_sync(0xffffffffu, back[nb], (2 * t4 + e) * 4));
            }
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, d));
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int j = 0; j < kD / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][j][e] = 0.f;

#pragma unroll 1
        for (; tile < tile_end; ++tile) {
            cp_async_wait<kStages - 2>();
            __syncwarp();  // the slice is there, and every lane is done with the one before
            copy(next, st == 0 ? kStages - 1 : st - 1);
            look_up(next);
            const int k0 = tile * G::kTileKeys + G::kSlice * mate;
            const uint32_t from = ring + st * G::kStageBytes;
            const uint32_t valid = s_valid[warp][st];
            if (k0 < keys) {
                float sc[kNB][kKS][4];
#pragma unroll
                for (int b = 0; b < kKS; ++b) {
                    // this lane's quarter of rows perm(g) and perm(g) + 8, and its scales
                    uint32_t kw[2][kD / 32], ks[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int row = 16 * b + 8 * u + G::perm(g);
                        const uint32_t at = from + row * G::kCodeRow;
                        if constexpr (kD == 64) lds_x2(kw[u], at + 8 * t4);
                        else
#pragma unroll
                            for (int c = 0; c < kD / 128; ++c) lds_x4(kw[u] + 4 * c, at + G::place(row, kD / 128 * t4 + c) * 16);
                        ks[u] = lds_bytes<kD / 64>(from + G::kScales + row * G::kScaleRow + kD / 64 * t4);
                    }
#pragma unroll
                    for (int nb = 0; nb < kNB; ++nb) sc[nb][b][0] = sc[nb][b][1] = sc[nb][b][2] = sc[nb][b][3] = 0.f;
                    uint32_t two[2], by[2];
#pragma unroll
                    for (int w = 0; w < kD / 32; ++w) {
                        uint32_t lo[4], hi[4];
                        e2m1_to_f16(lo, kw[0][w]);
                        e2m1_to_f16(hi, kw[1][w]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (w % 4 == 0) two[u] = e4m3_to_f16(ks[u] >> (4 * w));
                            if (w % 2 == 0) by[u] = w % 4 == 0 ? low_twice(two[u]) : high_twice(two[u]);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            lo[c] = hmul2(lo[c], by[0]);
                            hi[c] = hmul2(hi[c], by[1]);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t a[4] = {lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1]};
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb)
                                mma_16816<true>(sc[nb][b], a, qf[nb][2 * w + j][0], qf[nb][2 * w + j][1]);
                        }
                    }
                }
                if (k0 + G::kSlice > all_see || valid != 0xffffffffu) {
#pragma unroll
                    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                        for (int b = 0; b < kKS; ++b)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kk = 16 * b + 8 * (e / 2) + G::perm(g);
                                if (!((valid >> kk) & 1) || k0 + kk >= lim[nb][e % 2]) sc[nb][b][e] = -INFINITY;
                            }
                }
                uint32_t pf[kNB][kKS][2];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) {
                    // element e of block b: slot g + 8 (e / 2), row 2 t4 + e % 2.  Most slices only look
                    // whether the maximum has to rise.
                    float mx[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(sc[nb][0][e], sc[nb][0][2 + e]);
#pragma unroll
                        for (int b = 1; b < kKS; ++b) mx[e] = fmaxf(mx[e], fmaxf(sc[nb][b][e], sc[nb][b][2 + e]));
                        mx[e] *= sl2[nb][e];
                    }
                    if (__any_sync(0xffffffffu, mx[0] > m[nb][0] + kMaxAbove || mx[1] > m[nb][1] + kMaxAbove)) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
                            const float mn = fmaxf(m[nb][e], mx[e] - kMaxBelow);
                            al[e] = ex2_approx(m[nb][e] - (mn == -INFINITY ? 0.f : mn));
                            m[nb][e] = mn;
                            l[nb][e] *= al[e];
                        }
#pragma unroll
                        for (int j = 0; j < kD / 16; ++j) {
                            o[nb][j][0] *= al[0];
                            o[nb][j][1] *= al[1];
                            o[nb][j][2] *= al[0];
                            o[nb][j][3] *= al[1];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float use = m[nb][e] == -INFINITY ? 0.f : m[nb][e];
#pragma unroll
                        for (int b = 0; b < kKS; ++b)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float& y = sc[nb][b][2 * u + e];
                                y = ex2_approx(fmaf(y, sl2[nb][e], -use));
                                l[nb][e] += y;
                            }
                    }
#pragma unroll
                    for (int b = 0; b < kKS; ++b) {
                        pf[nb][b][0] = movmatrix(pack_x2<true>(sc[nb][b][0], sc[nb][b][1]));
                        pf[nb][b][1] = movmatrix(pack_x2<true>(sc[nb][b][2], sc[nb][b][3]));
                    }
                }
#pragma unroll
                for (int b = 0; b < kKS; ++b) {
                    // this lane's eighth of the rows of slots 2 t4 (+ 8) and 2 t4 + 1 (+ 8), and their scales
                    uint32_t vw[4][kD / 64], vs[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int row = 16 * b + 8 * (u / 2) + G::perm(2 * t4 + u % 2);
                        const uint32_t at = from + G::kV + row * G::kCodeRow;
                        if constexpr (kD == 64) vw[u][0] = lds_bytes<4>(at + 4 * g);
                        else if constexpr (kD == 128) lds_x2(vw[u], at + G::place(row, g / 2) * 16 + (g & 1) * 8);
                        else lds_x4(vw[u], at + G::place(row, g) * 16);
                        vs[u] = lds_bytes<kD == 256 ? 2 : 1>(from + G::kVScales + row * G::kScaleRow +
                                                             (kD == 64 ? g / 2 : kD == 128 ? g : 2 * g));
                    }
                    uint32_t by[2];
#pragma unroll
                    for (int w = 0; w < kD / 64; ++w) {
                        uint32_t a[4][4];  // [pair of keys, low and high elements][byte]
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t x0 = vw[2 * u][w], x1 = vw[2 * u + 1][w];
                            e2m1_to_f16(a[2 * u], (x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u));
                            e2m1_to_f16(a[2 * u + 1], ((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u));
                            if (w % 2 == 0) by[u] = e4m3_to_f16(__byte_perm(vs[2 * u], vs[2 * u + 1], w == 0 ? 0x0040 : 0x0051));
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                a[2 * u][c] = hmul2(a[2 * u][c], by[u]);
                                a[2 * u + 1][c] = hmul2(a[2 * u + 1][c], by[u]);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t f[4] = {a[0][c], a[1][c], a[2][c], a[3][c]};
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb) mma_16816<true>(o[nb][4 * w + c], f, pf[nb][b][0], pf[nb][b][1]);
                        }
                    }
                }
            }
            st = st + 1 == kStages ? 0 : st + 1;
        }

        // merge the warps: M = max m, L = sum l 2^(m - M), O = sum O 2^(m - M) (/ L when the unit is whole)
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
                if (g == 0) stats[mate * G::kRows + 8 * nb + 2 * t4 + e] = make_float2(m[nb][e], l[nb][e]);
            }
        const typename G::CursorT& cur = s_cur[warp];
        const Seq x = cur.x;
        const int t0 = cur.row_unit * sp.map.tokens;
        const bool whole = cur.whole();
        const int slot = 2 * me + (cur.tile == 0 ? 1 : 0);
        constexpr int kParts = kD / G::kMergeCols;  // of a row: products 4 part to 4 part + 3 of every lane
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                meet();  // the stats are there; what was merged before has been read
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)  // row 2 t4 + e lies at 4 e + t4
                        *reinterpret_cast<float2*>(merge + (mate * 8 + 4 * e + t4) * G::kMergeStride + 8 * g + 2 * j) =
                            make_float2(o[nb][4 * part + j][e], o[nb][4 * part + j][2 + e]);
                meet();
#pragma unroll
                for (int i = ttid; i < 8 * (G::kMergeCols / 2); i += G::kTeamThreads) {
                    const int at = i / (G::kMergeCols / 2), r = 2 * (at & 3) + (at >> 2);
                    const int dc = (i % (G::kMergeCols / 2)) * 2, d = (kD / 8) * (dc >> 3) + 8 * part + (dc & 7);
                    const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + r);
                    if (!w.there) continue;
                    float M = -INFINITY, L = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
                    for (int k = 0; k < G::kTeamWarps; ++k) M = fmaxf(M, stats[k * G::kRows + 8 * nb + r].x);
                    const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int k = 0; k < G::kTeamWarps; ++k) {
                        const float2 ml = stats[k * G::kRows + 8 * nb + r];
                        const float f = ex2_approx(ml.x - use);
                        const float2 v = *reinterpret_cast<const float2*>(merge + (k * 8 + at) * G::kMergeStride + dc);
                        L += ml.y * f;
                        a0 += v.x * f;
                        a1 += v.y * f;
                    }
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        const long long tok = x.q0 + w.token;
                        a0 *= inv;
                        a1 *= inv;
                        a0 *= p.v_unit;  // last: the sums times the unit may be no numbers of fp32
                        a1 *= p.v_unit;
                        *reinterpret_cast<uint32_t*>(p.o + (tok * p.Hq + w.head) * kD + d) =
                            p.f16 ? pack_x2<true>(a0, a1) : pack_x2<false>(a0, a1);
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
        meet();  // the stats may be overwritten; a piece is written
        if (!whole) {
            const int first = cur.tile == 0 ? me : s_sh[team].starter(cur.at);
            const int n = s_sh[team].pieces(cur.at, cur.tiles, first);
            if (ttid == 0) s_last[team] = count_piece(sp.ws.count(first), n);
            meet();
            if (s_last[team]) {
                if (p.f16) join_pieces<true, kD, G::kRows, G::kTeamThreads, G::kJoinFly>(p, sp, x, cur.head_unit, t0, first, n, merge, G::kTeams == 1 ? 0 : 1 + team);
                else join_pieces<false, kD, G::kRows, G::kTeamThreads, G::kJoinFly>(p, sp, x, cur.head_unit, t0, first, n, merge, G::kTeams == 1 ? 0 : 1 + team);
            }
            meet();
        }
    }
    cp_async_wait<0>();
}

}  // namespace paged
}  // namespace attn

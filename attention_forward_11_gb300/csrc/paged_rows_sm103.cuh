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
// A warp owns 16 keys of every tile and keeps its own running maximum, sum and O^T
// (online softmax in log2 units, fp32), so warps meet only at the end of a unit, where
// their (m, l, O) are merged in a fixed order.  P is rounded to the operands' type for
// its product, as in the dense forward.
//
// One block a SM takes an equal share of the batch (paged_sched_sm103.cuh).  Each warp
// fills a ring of its own with cp.async, kStages - 1 slices ahead of the one it computes
// and across the ends of units, with no barrier between warps: 16-byte copies follow any
// page size and any strides, and a slice's page numbers are read one slice earlier still.
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
    static constexpr int kTileKeys = 16 * kWarps;       // keys of all warps in one step
    static constexpr int kSliceBytes = 16 * kD * 2;     // K or V rows of one warp's step
    static constexpr int kChunks = kD / 8;              // 16-byte pieces of a row
    static constexpr int kStages = kD == 64 ? 6 : 3;    // 192 KB of slices
    static constexpr int kMergeCols = 64;               // columns of O merged at a time
    static constexpr int kMergeStride = kMergeCols + 4; // floats; rows 2 t of a warp fall into different banks
    static constexpr int kRing = kWarps * kStages * 2 * kSliceBytes;
    static constexpr int kMerge = kWarps * 8 * kMergeStride * 4;
    static constexpr int kStats = kWarps * kRows * 8;
    static constexpr int kSmemBytes = kRing + kMerge + kStats;
    static_assert(kSmemBytes <= 231000, "ring, merge buffer and static shared memory exceed 227 KB");
    // a piece is worth its merge from two tiles on, a share from four
    static constexpr int kMinPiece = 2, kMinShare = 4;
    using ShareT = Share<kTileKeys, kMinPiece, kMinShare>;
    using CursorT = Cursor<ShareT, kTileKeys>;
};

template <bool kF16, int kD, int kNB>
__global__ void __launch_bounds__(RowsGeo<kD, kNB>::kThreads, 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ SchedParams sp) {
    using G = RowsGeo<kD, kNB>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_part[G::kWarps];
    __shared__ StartPos s_start;
    __shared__ uint32_t s_valid[G::kWarps][G::kStages];  // keys of a slice that have a page
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (G::kStages * 2 * G::kSliceBytes);
    float* merge = reinterpret_cast<float*>(smem + G::kRing);
    float2* stats = reinterpret_cast<float2*>(smem + G::kRing + G::kMerge);
    launch_dependents();

    typename G::ShareT sh;
    if (tid == 0) sp.ws.header[blockIdx.x].n = 0;
    const bool some = find_share<G::kThreads, typename G::ShareT, G::kTileKeys, G::kMinShare>(p, sp, s_part, &s_start, sh);
    if (!some) return;
    typename G::CursorT cur;
    cur.first(p, sp, sh, s_start);
    typename G::CursorT ld = cur;  // the copies' position, ahead of the products'
    int ld_tile = ld.tile;

    // The page numbers of the next slice to copy: lane i has that of key i % 16.
    int page = -1, page_row = 0;
    auto look_up = [&]() {
        page = -1;
        if (!ld.ok) return;
        const int key = ld_tile * G::kTileKeys + 16 * warp + (lane & 15);
        if (key >= ld.keys) return;
        const int col = static_cast<int>(p.by_page.quot(key));
        page = p.table[ld.s * p.table_stride + col];
        page_row = key - col * p.page_size;
    };
    // Copies that slice into a stage, then moves on.
    auto issue = [&](int st) {
        if (ld.ok) {
            const bool there = page >= 0 && page < p.n_pages;
            const long long base = there ? page * p.page_stride + page_row * p.token_stride +
                                               ld.head_unit / sp.map.splits * p.head_stride
                                         : 0;
            const uint32_t valid = __ballot_sync(0xffffffffu, there) & 0xffffu;
            if (lane == 0) s_valid[warp][st] = valid;
            const uint32_t to = ring + st * (2 * G::kSliceBytes);
            if (ld_tile * G::kTileKeys + 16 * warp < ld.keys) {
#pragma unroll
                for (int i = 0; i < G::kChunks / 2; ++i) {
                    const int idx = lane + 32 * i, kk = idx / G::kChunks, ch = idx % G::kChunks;
                    const long long at = __shfl_sync(0xffffffffu, base, kk) + ch * 8;
                    const bool ok = (valid >> kk) & 1;
                    const uint32_t dst = to + kk * (kD * 2) + ((ch ^ (kk & 7)) << 4);
                    cp_async16(dst, p.k + at, ok);
                    cp_async16(dst + G::kSliceBytes, p.v + at, ok);
                }
            }
            if (++ld_tile == ld.tile_end) {
                ld.next(p, sp, sh);
                ld_tile = ld.tile;
            }
            look_up();
        }
        cp_async_commit();
    };
    look_up();
#pragma unroll 1
    for (int st = 0; st < G::kStages; ++st) issue(st);
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
        int lim[kNB][2];
        float m[kNB][2], l[kNB][2], o[kNB][kD / 16][4];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + 2 * t4 + e);
                lim[nb][e] = w.there ? visible_keys(p, x, w.token) : 0;
                m[nb][e] = -INFINITY;
                l[nb][e] = 0.f;
            }
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][mt][e] = 0.f;

#pragma unroll 1
        for (int tile = cur.tile; tile < cur.tile_end; ++tile) {
            cp_async_wait<G::kStages - 1>();
            __syncwarp();
            const int k0 = tile * G::kTileKeys + 16 * warp;
            const uint32_t from = ring + st * (2 * G::kSliceBytes);
            const uint32_t valid = s_valid[warp][st];
            if (k0 < cur.keys) {
                float sc[kNB][4];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
                {
                    const int kk = (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t a0 = from + kk * (kD * 2);
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks) {
                        uint32_t a[4];
                        ldsm_x4(a, a0 + (((2 * ks + (lane >> 4)) ^ (kk & 7)) << 4));
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) mma_16816<kF16>(sc[nb], a, qf[nb][ks][0], qf[nb][ks][1]);
                    }
                }
                uint32_t pf[kNB][2];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) {
                    // element e of sc: key k0 + g + 8 (e / 2), row 2 t4 + e % 2
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool v0 = ((valid >> g) & 1) && k0 + g < lim[nb][e];
                        const bool v1 = ((valid >> (g + 8)) & 1) && k0 + g + 8 < lim[nb][e];
                        float a = v0 ? sc[nb][e] * p.scale_log2 : -INFINITY;
                        float b = v1 ? sc[nb][e + 2] * p.scale_log2 : -INFINITY;
                        float mx = fmaxf(a, b);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        const float mn = fmaxf(m[nb][e], mx), use = mn == -INFINITY ? 0.f : mn;
                        al[e] = ex2_approx(m[nb][e] - use);
                        m[nb][e] = mn;
                        a = ex2_approx(a - use);
                        b = ex2_approx(b - use);
                        l[nb][e] = l[nb][e] * al[e] + (a + b);
                        sc[nb][e] = a;
                        sc[nb][e + 2] = b;
                    }
#pragma unroll
                    for (int mt = 0; mt < kD / 16; ++mt) {
                        o[nb][mt][0] *= al[0];
                        o[nb][mt][1] *= al[1];
                        o[nb][mt][2] *= al[0];
                        o[nb][mt][3] *= al[1];
                    }
                    pf[nb][0] = movmatrix(pack_x2<kF16>(sc[nb][0], sc[nb][1]));
                    pf[nb][1] = movmatrix(pack_x2<kF16>(sc[nb][2], sc[nb][3]));
                }
                {
                    const int kk = (lane & 7) + (lane >> 4) * 8;
                    const uint32_t a0 = from + G::kSliceBytes + kk * (kD * 2);
#pragma unroll
                    for (int mt = 0; mt < kD / 16; ++mt) {
                        uint32_t a[4];
                        ldsm_x4_trans(a, a0 + (((2 * mt + ((lane >> 3) & 1)) ^ (kk & 7)) << 4));
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) mma_16816<kF16>(o[nb][mt], a, pf[nb][0], pf[nb][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage and its mask
            issue(st);
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
        if (!whole && cur.tile == 0 && tid == 0)
            sp.ws.header[blockIdx.x] = PieceHeader{sh.pieces(cur.at, cur.tiles, static_cast<int>(blockIdx.x)), cur.s,
                                                   cur.head_unit, cur.row_unit};
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
                for (int i = tid; i < 8 * (G::kMergeCols / 4); i += G::kThreads) {
                    const int r = i / (G::kMergeCols / 4), dc = (i % (G::kMergeCols / 4)) * 4, d = part * G::kMergeCols + dc;
                    const Row w = row_of(p, sp.map, x, cur.head_unit, t0, sp.map.tokens, 8 * nb + r);
                    if (!w.there) continue;
                    float M = -INFINITY, L = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
                    for (int k = 0; k < G::kWarps; ++k) M = fmaxf(M, stats[k * G::kRows + 8 * nb + r].x);
                    const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int k = 0; k < G::kWarps; ++k) {
                        const float2 ml = stats[k * G::kRows + 8 * nb + r];
                        const float f = ex2_approx(ml.x - use);
                        const float4 v = *reinterpret_cast<const float4*>(merge + (k * 8 + r) * G::kMergeStride + dc);
                        L += ml.y * f;
                        a0 += v.x * f;
                        a1 += v.y * f;
                        a2 += v.z * f;
                        a3 += v.w * f;
                    }
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        const long long tok = x.q0 + w.token;
                        uint2 out;
                        out.x = pack_x2<kF16>(a0 * inv, a1 * inv);
                        out.y = pack_x2<kF16>(a2 * inv, a3 * inv);
                        *reinterpret_cast<uint2*>(p.o + (tok * p.Hq + w.head) * kD + d) = out;
                        if (d == 0 && p.lse != nullptr)
                            p.lse[(long long)w.head * p.total_q + tok] =
                                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
                    } else {
                        const size_t row = (size_t)slot * G::kRows + 8 * nb + r;
                        *reinterpret_cast<float4*>(sp.ws.o + row * kD + d) = make_float4(a0, a1, a2, a3);
                        if (d == 0) sp.ws.ml[row] = make_float2(M, L);
                    }
                }
            }
        __syncthreads();  // the stats may be overwritten
    }
    cp_async_wait<0>();
}

}  // namespace paged
}  // namespace attn

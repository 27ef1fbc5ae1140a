// paged_sched_sm103.cuh -- how the work of attention over a paged cache is shared out,
// and how the pieces of a shared unit are joined.
//
// A unit is a block of query rows of one sequence that read one key/value head: `tokens`
// consecutive tokens times `heads` query heads of the head's group (a group larger than
// a block is cut into `splits` parts).  Lengths are on the device, so every block works
// out its own share there: units are laid end to end in the order (sequence, head, row
// block), a unit as long as the keys that its last token sees plus kUnitKeys for its
// start and end, and block c of G takes the stretch [c T / G, (c + 1) T / G) of the total
// T.  All shares are equal for any mixture of lengths, which is what a batch of few long
// and many short sequences needs.  A stretch that ends inside a unit leaves a piece: the
// unnormalised sums (m, l, O) of some of its key tiles in fp32, which go to the workspace
// and are joined by paged_combine_kernel.  Cuts that would leave a piece of less than
// kMinPiece key tiles move to the unit's edge, and shares are at least kMinShare tiles.
//
// With d = keys - rows of a sequence, row block i (of t tokens, the last one aside) sees
// max(0, d + (i + 1) t) keys, an arithmetic series: the length of any number of row
// blocks is a closed form and the row block at a position a binary search.
#pragma once
#include <cstdint>

#include "paged_common_sm103.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

constexpr int kUnitKeys = 128;  // a unit's own cost, in keys

struct RowMap {
    int heads;      // query heads of a block
    int splits;     // blocks of heads per key/value head
    int tokens;     // tokens of a unit
    int head_units; // Hkv * splits
};

// How `rows` rows of a block (times `tiles` blocks side by side) cover a group.
inline RowMap make_row_map(int Hkv, int group, int rows, int tiles) {
    RowMap m;
    m.splits = (group + rows - 1) / rows;
    m.heads = (group + m.splits - 1) / m.splits;
    m.tokens = rows / m.heads * tiles;
    m.head_units = Hkv * m.splits;
    return m;
}

// Header of the pieces of one cut unit, written by the block that has its first piece.
struct PieceHeader {
    int n;                   // pieces (0: this block starts no cut unit)
    int seq, head_unit, row_unit;
};

// Workspace: headers [G], (m, l) [2 G][rows], O [2 G][rows][D].  Block c's piece at the
// front of its share (a unit begun by an earlier block) is slot 2 c, the one at its end
// slot 2 c + 1.
struct Workspace {
    PieceHeader* header;
    float2* ml;
    float* o;
};

__host__ __device__ inline size_t ws_header_bytes(int G) { return ((size_t)G * sizeof(PieceHeader) + 255) / 256 * 256; }
__host__ __device__ inline size_t ws_ml_bytes(int G, int rows) { return ((size_t)2 * G * rows * sizeof(float2) + 255) / 256 * 256; }
__host__ __device__ inline size_t ws_bytes(int G, int rows, int D) {
    return ws_header_bytes(G) + ws_ml_bytes(G, rows) + (size_t)2 * G * rows * D * sizeof(float);
}

struct SchedParams {
    RowMap map;
    Workspace ws;
};

__device__ __forceinline__ int row_units(const SchedParams& sp, const Seq& x) {
    return (x.q_len + sp.map.tokens - 1) / sp.map.tokens;
}

// Keys that row unit i sees: those of its last token.
__device__ __forceinline__ int unit_keys(const PagedParams& p, const SchedParams& sp, const Seq& x, int i) {
    return visible_keys(p, x, min((i + 1) * sp.map.tokens, x.q_len) - 1);
}

// Length of the first r row units of a head (r < row_units, or all of them).
__device__ __forceinline__ long long units_length(const PagedParams& p, const SchedParams& sp, const Seq& x, int r) {
    long long keys;
    if (!p.causal) {
        keys = (long long)r * x.kv_len;
    } else {
        const long long t = sp.map.tokens, d = (long long)x.kv_len - x.q_len;
        const bool all = r == row_units(sp, x);
        const long long n = all ? r - 1 : r;                // units of t tokens
        const long long i0 = d >= 0 ? 0 : min(-d / t, n);   // the first that sees a key: d + (i0 + 1) t > 0
        keys = (n - i0) * d + t * ((n * (n + 1) - i0 * (i0 + 1)) / 2) + (all ? x.kv_len : 0);
    }
    return keys + (long long)r * kUnitKeys;
}

__device__ __forceinline__ long long seq_length(const PagedParams& p, const SchedParams& sp, const Seq& x) {
    return x.q_len == 0 ? 0 : sp.map.head_units * units_length(p, sp, x, row_units(sp, x));
}

// A block's share, and a position in it.  kTile: keys of a tile (a power of two).
template <int kTile, int kMinPiece, int kMinShare>
struct Share {
    long long begin, end;  // stretch of this block
    long long total;
    int blocks;            // that have a share

    // Tile at which a cut at length `at` of a unit of `tiles` tiles falls.
    __device__ __forceinline__ static int cut(long long at, int tiles) {
        const long long t = at <= kUnitKeys ? 0 : (at - kUnitKeys) / kTile;
        if (t < kMinPiece) return 0;
        return tiles - t < kMinPiece ? tiles : static_cast<int>(t);
    }
    // Blocks whose cut falls inside a unit that starts at `start`: those before the first
    // whose cut would be at the unit's end.
    __device__ __forceinline__ int pieces(long long start, int tiles, int first) const {
        // cut(x) < tiles  <=>  x < kUnitKeys + kTile * (tiles - kMinPiece + 1)
        const long long y = start + kUnitKeys + (long long)kTile * (tiles - kMinPiece + 1);
        const long long last = (y * blocks + total - 1) / total - 1;  // largest c with floor(c T / G) < y
        return static_cast<int>(min(last, (long long)blocks - 1)) - first + 1;
    }
};

struct StartPos {
    long long total;
    long long seq_at;  // position of the sequence that the share starts in
    int seq;
};

// Sum over the block (every thread calls it; kThreads / 32 <= 32 warps).
template <int kThreads>
__device__ __forceinline__ long long block_sum(long long v, long long* part) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += part[w];
    __syncthreads();
    return v;
}

// The share of block blockIdx.x and the sequence it starts in (block-wide; `part` and
// `found` are shared scratch).  Returns false for a block without work.
template <int kThreads, class ShareT, int kTile, int kMinShare>
__device__ __forceinline__ bool find_share(const PagedParams& p, const SchedParams& sp, long long* part, StartPos* found,
                                           ShareT& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long sum = 0;
    for (int s = tid; s < p.n_seqs; s += kThreads) sum += seq_length(p, sp, seq_of(p, s));
    sh.total = block_sum<kThreads>(sum, part);
    if (sh.total == 0) return false;
    sh.blocks = static_cast<int>(min((long long)gridDim.x, max(sh.total / (kTile * kMinShare), 1ll)));
    const int c = blockIdx.x;
    if (c >= sh.blocks) return false;
    sh.begin = c * sh.total / sh.blocks;
    sh.end = (c + 1) * sh.total / sh.blocks;
    long long at = 0;  // before the step's sequences
    for (int s0 = 0; s0 < p.n_seqs; s0 += kThreads) {
        const int s = s0 + tid;
        const long long len = s < p.n_seqs ? seq_length(p, sp, seq_of(p, s)) : 0;
        long long v = len;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        if (lane == 31) part[warp] = v;
        __syncthreads();
        long long before = at, step = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += part[w];
            step += part[w];
        }
        const long long end = before + v, start = end - len;
        if (sh.begin >= start && sh.begin < end) {
            found->seq = s;
            found->seq_at = start;
        }
        at += step;
        __syncthreads();
        if (at > sh.begin) break;
    }
    return true;
}

// Walks the units of a share.
template <class ShareT, int kTile>
struct Cursor {
    Seq x;
    int s, head_unit, row_unit, n_row_units;
    int keys;         // that the unit sees
    int tiles;        // of the whole unit, at least one
    int tile, tile_end;  // of this block's piece
    long long at, length;  // the unit's position and length
    bool ok;

    __device__ __forceinline__ bool whole() const { return tile == 0 && tile_end == tiles; }

    __device__ __forceinline__ void load_seq(const PagedParams& p, const SchedParams& sp) {
        for (; s < p.n_seqs; ++s) {
            x = seq_of(p, s);
            if (x.q_len > 0) break;
        }
        ok = s < p.n_seqs;
        if (ok) n_row_units = row_units(sp, x);
    }
    __device__ __forceinline__ void measure(const PagedParams& p, const SchedParams& sp) {
        keys = unit_keys(p, sp, x, row_unit);
        tiles = max((keys + kTile - 1) / kTile, 1);
        length = keys + kUnitKeys;
    }
    // This block's piece of the unit; false if it has none.
    __device__ __forceinline__ bool piece(const ShareT& sh) {
        tile = sh.begin > at ? ShareT::cut(sh.begin - at, tiles) : 0;
        tile_end = sh.end >= at + length ? tiles : ShareT::cut(sh.end - at, tiles);
        return tile < tile_end;
    }
    __device__ __forceinline__ void step(const PagedParams& p, const SchedParams& sp) {
        at += length;
        if (++row_unit < n_row_units) return;
        row_unit = 0;
        if (++head_unit < sp.map.head_units) return;
        head_unit = 0;
        ++s;
        load_seq(p, sp);
    }
    // To the next unit of which this block has a piece.
    __device__ __forceinline__ void seek(const PagedParams& p, const SchedParams& sp, const ShareT& sh) {
        while (ok && at < sh.end) {
            measure(p, sp);
            if (piece(sh)) return;
            step(p, sp);
        }
        ok = false;
    }
    __device__ __forceinline__ void next(const PagedParams& p, const SchedParams& sp, const ShareT& sh) {
        step(p, sp);
        seek(p, sp, sh);
    }
    __device__ __forceinline__ void first(const PagedParams& p, const SchedParams& sp, const ShareT& sh, const StartPos& f) {
        s = f.seq;
        x = seq_of(p, s);
        ok = true;
        n_row_units = row_units(sp, x);
        const long long per_head = units_length(p, sp, x, n_row_units);
        head_unit = static_cast<int>((sh.begin - f.seq_at) / per_head);
        const long long head_at = f.seq_at + head_unit * per_head, rest = sh.begin - head_at;
        int lo = 0, hi = n_row_units - 1;  // the last row unit that starts at or before the position
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (units_length(p, sp, x, mid) <= rest) lo = mid;
            else hi = mid - 1;
        }
        row_unit = lo;
        at = head_at + units_length(p, sp, x, lo);
        seek(p, sp, sh);
    }
};

// ---- rows of a unit
// Row r of a block that starts at token t0 of its sequence: token, query head, and
// whether there is such a row.
struct Row {
    int token, head;  // of the sequence, of all query heads
    bool there;
};
__device__ __forceinline__ Row row_of(const PagedParams& p, const RowMap& m, const Seq& x, int head_unit, int t0, int tokens,
                                      int r) {
    Row w;
    const int t = r / m.heads, h = (head_unit % m.splits) * m.heads + r % m.heads;
    w.token = t0 + t;
    w.head = head_unit / m.splits * p.group + h;
    w.there = t < tokens && w.token < x.q_len && h < p.group;
    return w;
}

// ---- programmatic launch: the joining kernel is in place when the last block ends
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the pieces of cut units: M = max m, L = sum l 2^(m - M), O = sum O 2^(m - M) / L.
// Grid (G, row groups): block (c, y) has kRowsPer rows of the unit that block c of the
// first kernel starts; its warps share a row's pieces, in a fixed order, and add up in
// shared memory in the order of the warps.
constexpr int kCombineThreads = 256;

template <bool kF16, int kD, int kRows, int kTokenTiles, int kRowsPer>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedParams p, const SchedParams sp) {
    constexpr int kWarpsPer = kCombineThreads / 32 / kRowsPer;  // warps of a row
    constexpr int kPer = kD / 32;                               // columns of a lane
    __shared__ float s_o[kWarpsPer > 1 ? kCombineThreads / 32 : 1][kD];
    __shared__ float2 s_ml[kCombineThreads / 32];
    wait_for_primary();  // every thread: this kernel's end stands for the first one's too
    const int c = blockIdx.x;
    const PieceHeader h = sp.ws.header[c];
    if (h.n == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rr = warp / kWarpsPer, part = warp % kWarpsPer;
    const int r = blockIdx.y * kRowsPer + rr;  // row of the unit
    const Seq x = seq_of(p, h.seq);
    constexpr int kTileRows = kRows / kTokenTiles;
    const int tile_tokens = sp.map.tokens / kTokenTiles;
    const int tile = r / kTileRows;
    const Row w = row_of(p, sp.map, x, h.head_unit, h.row_unit * sp.map.tokens + tile * tile_tokens, tile_tokens,
                         r % kTileRows);
    float M = -INFINITY, L = 0.f, acc[kPer] = {};
    if (w.there) {
        for (int i = lane; i < h.n; i += 32) {
            const int slot = i == 0 ? 2 * c + 1 : 2 * (c + i);
            M = fmaxf(M, sp.ws.ml[(size_t)slot * kRows + r].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float use = M == -INFINITY ? 0.f : M;
        constexpr int kFly = kD == 256 ? 4 : 8;  // pieces in flight
        for (int i0 = part; i0 < h.n; i0 += kFly * kWarpsPer) {
            float f[kFly], v[kFly][kPer];
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const int i = i0 + j * kWarpsPer;
                const int slot = i == 0 ? 2 * c + 1 : 2 * (c + i);
                f[j] = 0.f;
                if (i < h.n) {
                    const float2 ml = sp.ws.ml[(size_t)slot * kRows + r];
                    f[j] = ex2_approx(ml.x - use);
                    L += ml.y * f[j];
                    const float* src = sp.ws.o + ((size_t)slot * kRows + r) * kD + kPer * lane;
#pragma unroll
                    for (int e = 0; e < kPer; e += 2) {
                        const float2 y = *reinterpret_cast<const float2*>(src + e);
                        v[j][e] = y.x;
                        v[j][e + 1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kPer; ++e) v[j][e] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < kFly; ++j)
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] += v[j][e] * f[j];
        }
    }
    if constexpr (kWarpsPer > 1) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) s_o[warp][kPer * lane + e] = acc[e];
        if (lane == 0) s_ml[warp].y = L;
        __syncthreads();
        if (part != 0) return;
#pragma unroll
        for (int k = 1; k < kWarpsPer; ++k) {
            L += s_ml[warp + k].y;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] += s_o[warp + k][kPer * lane + e];
        }
    }
    if (!w.there) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t tok = (size_t)x.q0 + w.token;
    uint16_t* dst = p.o + (tok * p.Hq + w.head) * kD + kPer * lane;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_x2<kF16>(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[(size_t)w.head * p.total_q + tok] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace paged
}  // namespace attn

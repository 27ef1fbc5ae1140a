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
// and are joined by the last block to finish one (paged_rows_kernel: count_piece below, then
// join_pieces) or by a kernel behind (paged_tiles_kernel: paged_combine_kernel).  Cuts that
// would leave a piece of less than kMinPiece key tiles move to the unit's edge, and no more
// blocks than units take part where their shares would be below kMinShare tiles.
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

constexpr int kUnitKeys = 256;  // a unit's own cost, in keys (about 2 us of 64 KB tiles); kernels
                                // that take a key in less time have a cost of their own (kUnit)

struct RowMap {
    int heads;      // query heads of a block
    int splits;     // blocks of heads per key/value head
    int tokens;     // tokens of a unit
    int head_units; // Hkv * splits
    FastDiv by_heads, by_splits, by_tokens;
    // row of a block -> token; head unit -> key/value head
    __device__ __forceinline__ int token_of(int r) const { return static_cast<int>(by_heads.quot(r)); }
    __device__ __forceinline__ int kv_head(int head_unit) const { return static_cast<int>(by_splits.quot(head_unit)); }
};

// How `rows` rows of a block (times `tiles` blocks side by side) cover a group.
inline RowMap make_row_map(int Hkv, int group, int rows, int tiles) {
    RowMap m;
    m.splits = (group + rows - 1) / rows;
    m.heads = (group + m.splits - 1) / m.splits;
    m.tokens = rows / m.heads * tiles;
    m.head_units = Hkv * m.splits;
    m.by_heads = make_fastdiv(m.heads);
    m.by_splits = make_fastdiv(m.splits);
    m.by_tokens = make_fastdiv(m.tokens);
    return m;
}

// Header of the pieces of one cut unit, written by the block that has its first piece.
struct PieceHeader {
    int n;                   // pieces (0: this block starts no cut unit)
    int seq, head_unit, row_unit;
};

// Workspace: headers [G], (m, l) [2 G][rows], O [2 G][rows][D].  Block c's piece at the
// front of its share (a unit begun by an earlier block) is slot 2 c, the one at its end
// slot 2 c + 1.  Where the last block to finish a unit's pieces joins them, the headers'
// place holds the counts of the pieces that are there (count_piece).
struct Workspace {
    PieceHeader* header;
    __device__ __forceinline__ unsigned long long* count(int c) const {
        return reinterpret_cast<unsigned long long*>(header + c);
    }
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
    unsigned long long tag;  // of this launch, 48 bits, not zero
    float o_unit = 1.f;      // O is what the pieces give times this: last, since their sums times it may be no
                             // numbers of fp32
};

// a / b for a, b >= 0; most fit 32 bits, where a division is several times cheaper
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0)
        return static_cast<long long>(static_cast<unsigned int>(a) / static_cast<unsigned int>(b));
    return a / b;
}

__device__ __forceinline__ int row_units(const SchedParams& sp, const Seq& x) {
    return static_cast<int>(sp.map.by_tokens.quot((long long)x.q_len + sp.map.tokens - 1));
}

// Keys that row unit i sees: those of its last token.
__device__ __forceinline__ int unit_keys(const PagedParams& p, const SchedParams& sp, const Seq& x, int i) {
    return visible_keys(p, x, min((i + 1) * sp.map.tokens, x.q_len) - 1);
}

// Length of the first r row units of a head (r < row_units, or all of them).
template <int kUnit>
__device__ __forceinline__ long long units_length(const PagedParams& p, const SchedParams& sp, const Seq& x, int r) {
    long long keys;
    if (!p.causal) {
        keys = (long long)r * x.kv_len;
    } else {
        const long long t = sp.map.tokens, d = (long long)x.kv_len - x.q_len;
        const bool all = r == row_units(sp, x);
        const long long n = all ? r - 1 : r;                // units of t tokens
        const long long i0 = d >= 0 ? 0 : min((long long)sp.map.by_tokens.quot(-d), n);   // the first that sees a key: d + (i0 + 1) t > 0
        keys = (n - i0) * d + t * ((n * (n + 1) - i0 * (i0 + 1)) / 2) + (all ? x.kv_len : 0);
    }
    return keys + (long long)r * kUnit;
}

template <int kUnit>
__device__ __forceinline__ long long seq_length(const PagedParams& p, const SchedParams& sp, const Seq& x) {
    return x.q_len == 0 ? 0 : sp.map.head_units * units_length<kUnit>(p, sp, x, row_units(sp, x));
}

// A block's share, and a position in it.  kTile: keys of a tile (a power of two).
template <int kTile, int kMinPiece, int kMinShare, int kUnitCost = kUnitKeys>
struct Share {
    static constexpr int kUnit = kUnitCost;
    // two cuts are at least kUnit (as many blocks as units) or kMinShare tiles apart
    static_assert(kTile <= kUnit && kMinShare >= 1, "two cuts never fall on one tile");
    long long begin, end;  // stretch of this block
    long long total;
    int blocks;            // that have a share
    bool whole;            // nothing is cut: a unit counts one, and block c takes unit c

    // Tile at which a cut at length `at` of a unit of `tiles` tiles falls.
    __device__ __forceinline__ static int cut(long long at, int tiles) {
        const long long t = at <= kUnit ? 0 : (at - kUnit) / kTile;
        if (t < kMinPiece) return 0;
        return tiles - t < kMinPiece ? tiles : static_cast<int>(t);
    }
    // Blocks whose cut falls inside a unit that starts at `start`: those before the first
    // whose cut would be at the unit's end.
    __device__ __forceinline__ int pieces(long long start, int tiles, int first) const {
        // cut(x) < tiles  <=>  x < kUnit + kTile * (tiles - kMinPiece + 1)
        const long long y = start + kUnit + (long long)kTile * (tiles - kMinPiece + 1);
        const long long last = quotient(y * blocks + total - 1, total) - 1;  // largest c with floor(c T / G) < y
        return static_cast<int>(min(last, (long long)blocks - 1)) - first + 1;
    }
    // The block that has the first piece of a cut unit: the first whose end is no cut at
    // the unit's start.
    __device__ __forceinline__ int starter(long long start) const {
        const long long y = start + kUnit + (long long)kTile * kMinPiece;
        return static_cast<int>(quotient(y * blocks + total - 1, total)) - 1;  // first c with floor((c + 1) T / G) >= y
    }
};

struct StartPos {
    long long seq_at;  // position of the sequence that the share starts in
    int seq;
    Seq x;
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

// The share of block blockIdx.x and the sequence it starts in (block-wide; `part`, three
// values a warp, and `found` are shared scratch).  Returns false for a block without work.
// With kTeams > 1 a block's threads are that many teams, each with a share, `found` and `sh` of
// its own, as if they were blocks; `team` is the thread's.  A team without work has an empty
// share (begin == end).
template <int kThreads, class ShareT, int kTile, int kMinShare, int kCutTiles, bool kAlign, int kTeams = 1>
__device__ __forceinline__ bool find_share(const PagedParams& p, const SchedParams& sp, long long* part, StartPos* found,
                                           ShareT& sh, int team = 0) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    const bool one_step = p.n_seqs <= kThreads;
    long long total = 0, n_units = 0, longest = 0;
    if (!one_step) {
        for (int s = tid; s < p.n_seqs; s += kThreads) {
            const Seq x = seq_of(p, s);
            total += seq_length<ShareT::kUnit>(p, sp, x);
            n_units += row_units(sp, x);
            if (x.q_len > 0) longest = max(longest, (long long)x.kv_len);
        }
        total = block_sum<kThreads>(total, part);
        n_units = block_sum<kThreads>(n_units, part);
        longest = __reduce_max_sync(0xffffffffu, static_cast<int>(longest));
        if (lane == 0) part[warp] = longest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) longest = max(longest, part[w]);
        __syncthreads();
    }
    long long at = 0, units_at = 0;  // before the step's sequences
    for (int s0 = 0; s0 < p.n_seqs; s0 += kThreads) {
        const int s = s0 + tid;
        Seq x{};
        if (s < p.n_seqs) x = seq_of(p, s);
        const long long len = seq_length<ShareT::kUnit>(p, sp, x);
        const int units = row_units(sp, x);
        long long v = len;
        int u = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long pv = __shfl_up_sync(0xffffffffu, v, d);
            const int pu = __shfl_up_sync(0xffffffffu, u, d);
            if (lane >= d) v += pv, u += pu;
        }
        const int most = __reduce_max_sync(0xffffffffu, x.q_len > 0 ? x.kv_len : 0);
        if (lane == 31) {
            part[warp] = v;
            part[kWarps + warp] = u;
            part[2 * kWarps + warp] = most;
        }
        __syncthreads();
        long long before = at, step = 0, units_before = units_at, units_step = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += part[w], units_before += part[kWarps + w];
            step += part[w];
            units_step += part[kWarps + w];
            if (one_step) longest = max(longest, part[2 * kWarps + w]);
        }
        if (s0 == 0) {
            if (one_step) total = step, n_units = units_step;
            if (total == 0) return false;
            n_units *= sp.map.head_units;
            const long long c0 = (long long)blockIdx.x * kTeams, c = c0 + team, G = (long long)gridDim.x * kTeams;
            // Whole units where the longest is no longer than an equal share and what a cut
            // costs at its end (kCutTiles), or, where units share K/V tiles in L2 and need them
            // as fast as L2 gives them (kAlign; whole units all start at key 0 and keep in step),
            // than 1.35 shares.  576 to 416 tokens, 64/8 heads, on 32000 keys, longest / share 1.06,
            // 1.19, 1.36, 1.46: whole / cut 341 / 435, 345 / 385, 333 / 350, 331 / 317 us at head
            // size 128; on 8000 keys 101 / 110, 101 / 100, 99 / 90.  At 64, where a tile's softmax
            // takes longer than its bytes, 294 / 286, 296 / 256, 296 / 226, 294 / 211: no kAlign.
            const long long share = quotient(total, G);
            longest += ShareT::kUnit;
            sh.whole = n_units <= G && (longest <= share + kCutTiles * kTile || (kAlign && longest * 100 <= share * 135));
            if (sh.whole) {
                sh.total = n_units;
                sh.blocks = static_cast<int>(n_units);
            } else {
                // a block for every unit, and more where that leaves shares of kMinShare tiles
                // (but not for up to half as many more, which cuts units for little: one long sequence
                // among short ones, blocks / units 1.22, 1.41, 1.47: cut / not 9.2 / 9.1, 10.6 / 11.0,
                // 9.7 / 12.0 us, and 20.0 / 19.2 at 1.46 in the tiles kernel; 1.6, 2.5, 3.9: 10.5 / 11.0,
                // 10.4 / 12.6, 10.3 / 15.6)
                sh.total = total;
                const long long most_blocks = quotient(total, kTile * kMinShare);
                sh.blocks = static_cast<int>(min(G, 2 * most_blocks >= 3 * n_units ? most_blocks : n_units));
            }
            if (c0 >= sh.blocks) return false;
            sh.begin = quotient(min(c, (long long)sh.blocks) * sh.total, sh.blocks);
            sh.end = quotient(min(c + 1, (long long)sh.blocks) * sh.total, sh.blocks);
        }
        const long long end = sh.whole ? (units_before + u) * sp.map.head_units : before + v;
        const long long start = end - (sh.whole ? (long long)units * sp.map.head_units : len);
        if constexpr (kTeams == 1) {
            if (sh.begin >= start && sh.begin < end) {
                found->seq = s;
                found->seq_at = start;
                found->x = x;
            }
        } else {
#pragma unroll
            for (int t = 0; t < kTeams; ++t) {
                const long long c = min((long long)blockIdx.x * kTeams + t, (long long)sh.blocks);
                const long long begin = quotient(c * sh.total, sh.blocks);
                if (begin >= start && begin < end) {
                    found[t].seq = s;
                    found[t].seq_at = start;
                    found[t].x = x;
                }
            }
        }
        at += step;
        units_at += units_step;
        __syncthreads();
        const long long last = kTeams == 1 ? sh.begin
                                           : quotient(min((long long)(blockIdx.x + 1) * kTeams, (long long)sh.blocks) * sh.total, sh.blocks) - 1;
        if ((sh.whole ? units_at * sp.map.head_units : at) > last) break;
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
    long long at;     // the unit's position
    bool whole_units;
    bool ok;

    __device__ __forceinline__ int length() const { return whole_units ? 1 : keys + ShareT::kUnit; }
    __device__ __forceinline__ bool whole() const { return tile == 0 && tile_end == tiles; }

    // The next sequence that has rows, from s on (every lane of a warp calls this).  A batch captured
    // for more requests than there are has many without, so 32 are looked at together (12 decoding
    // requests with one head, spread over 1024 places: 23 us, one look after another 33 us, without
    // the other places 20 us).
    __device__ __forceinline__ void load_seq(const PagedParams& p, const SchedParams& sp) {
        for (;; s += 32) {
            ok = s < p.n_seqs;
            if (!ok) return;
            const int mine = s + (threadIdx.x & 31);
            const uint32_t some = __ballot_sync(0xffffffffu, mine < p.n_seqs && seq_of(p, min(mine, p.n_seqs - 1)).q_len > 0);
            if (some == 0) continue;
            s += __ffs(some) - 1;
            break;
        }
        x = seq_of(p, s);
        n_row_units = row_units(sp, x);
    }
    __device__ __forceinline__ void measure(const PagedParams& p, const SchedParams& sp) {
        keys = unit_keys(p, sp, x, row_unit);
        tiles = max((keys + kTile - 1) / kTile, 1);
    }
    // This block's piece of the unit; false if it has none.
    __device__ __forceinline__ bool piece(const ShareT& sh) {
        tile = sh.begin > at ? ShareT::cut(sh.begin - at, tiles) : 0;
        tile_end = sh.end >= at + length() ? tiles : ShareT::cut(sh.end - at, tiles);
        return tile < tile_end;
    }
    __device__ __forceinline__ void step(const PagedParams& p, const SchedParams& sp, const ShareT& sh) {
        at += length();
        if (at >= sh.end) {  // what lies behind the share may be a thousand empty places: no look at them
            ok = false;
            return;
        }
        if (++row_unit < n_row_units) return;
        row_unit = 0;
        if (++head_unit < sp.map.head_units) return;
        head_unit = 0;
        ++s;
        load_seq(p, sp);
    }
    // To the next unit of which this block has a piece.
    __device__ __forceinline__ void seek(const PagedParams& p, const SchedParams& sp, const ShareT& sh) {
        while (ok) {  // at < sh.end
            measure(p, sp);
            if (piece(sh)) return;
            step(p, sp, sh);
        }
    }
    __device__ __forceinline__ void next(const PagedParams& p, const SchedParams& sp, const ShareT& sh) {
        step(p, sp, sh);
        seek(p, sp, sh);
    }
    __device__ __forceinline__ void first(const PagedParams& p, const SchedParams& sp, const ShareT& sh, const StartPos& f) {
        s = f.seq;
        x = f.x;
        ok = true;
        n_row_units = row_units(sp, x);
        whole_units = sh.whole;
        const long long per_head = sh.whole ? n_row_units : units_length<ShareT::kUnit>(p, sp, x, n_row_units);
        head_unit = static_cast<int>(quotient(sh.begin - f.seq_at, per_head));
        const long long head_at = f.seq_at + head_unit * per_head, rest = sh.begin - head_at;
        // the last row unit that starts at or before the position: the warp's lanes try 32 at
        // a time (every lane of a warp calls this)
        const int lane = threadIdx.x & 31;
        int lo = 0, n = n_row_units;  // it is one of [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32, at_lane = lo + lane * step;
            const bool before = lane * step < n && (sh.whole ? at_lane : units_length<ShareT::kUnit>(p, sp, x, at_lane)) <= rest;  // lane 0: true
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, before));
            n = min(step, n - k * step);
            lo += k * step;
        }
        row_unit = lo;
        at = head_at + (sh.whole ? lo : units_length<ShareT::kUnit>(p, sp, x, lo));
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
    const int t = m.token_of(r), g = m.kv_head(head_unit);
    const int h = (head_unit - g * m.splits) * m.heads + r - t * m.heads;
    w.token = t0 + t;
    w.head = g * p.group + h;
    w.there = t < tokens && w.token < x.q_len && h < p.group;
    return w;
}

// ---- the last block to finish a unit's pieces joins them
// Slot of piece i of a unit that block `first` starts.
__device__ __forceinline__ int piece_slot(int first, int i) { return i == 0 ? 2 * first + 1 : 2 * (first + i); }

// The pieces of the unit that block c starts are counted in word c of a workspace of unknown
// contents: the count is a launch's own once the upper 48 bits of the word are the launch's
// tag.  Every block that will count a piece makes sure of that long before (begin_count: a
// word that is not the launch's yet becomes its zero, by whoever comes first), so that the
// counting itself is one atomic addition, however many blocks end together.  The block that
// counts the last piece joins all, and clears the word: a replayed graph's launches share
// their tag.
struct CountWord {
    unsigned long long* word;
    unsigned long long seen;
};
__device__ __forceinline__ CountWord look_at_count(unsigned long long* word) {
    CountWord c{word, 0};
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(c.seen) : "l"(word) : "memory");
    return c;
}
__device__ __forceinline__ void begin_count(const CountWord& c, unsigned long long tag) {
    if ((c.seen >> 16) != tag) atomicCAS(c.word, c.seen, tag << 16);
}
// One thread, behind a barrier that follows the piece's writes; true for the last of n.
__device__ __forceinline__ bool count_piece(unsigned long long* word, int n) {
    unsigned long long old;
    asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
    const bool last = static_cast<int>(old & 0xffff) + 1 == n;
    if (last) *reinterpret_cast<volatile unsigned long long*>(word) = 0ull;
    return last;
}

// Joins the pieces of cut units: M = max m, L = sum l 2^(m - M), O = sum O 2^(m - M) / L (times o_unit), the
// sums in the order of the pieces.  Grid (G, parts of a unit's rows): block (c, y) has a part of the
// rows of the unit that block c of the first kernel starts, kD / 4 threads a row with four
// columns each.  Most units have two or three pieces, so what the kernel costs is its
// instructions a row and how many loads wait on one another: those of the first kFly pieces
// are in flight before M is known, and a thread has one row where units have so many (with
// four rows a thread a chunk of 64 tokens on 16000 took 48 instead of 38 us).  It takes 8 us
// with nothing to join and 15 us for 152 cut units of 256 rows, alone and with cold caches.
constexpr int kCombineThreads = 256;

template <bool kF16, int kD, int kRows, int kTokenTiles>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const __grid_constant__ PagedParams p,
                                                                        const __grid_constant__ SchedParams sp) {
    constexpr int kLanes = kD / 4, kFly = 4;
    constexpr int kTileRows = kRows / kTokenTiles;
    launch_dependents();
    touch_params(sp);
    wait_for_primary();  // every thread: this kernel's end stands for the first one's too
    const int c = blockIdx.x;
    const PieceHeader h = sp.ws.header[c];
    if (h.n == 0) return;
    const int col = threadIdx.x % kLanes * 4;
    const Seq x = seq_of(p, h.seq);
    const int tile_tokens = sp.map.tokens / kTokenTiles;
    constexpr int kAtOnce = kCombineThreads / kLanes;  // rows of a block
    for (int r = blockIdx.y * kAtOnce + threadIdx.x / kLanes; r < kRows; r += gridDim.y * kAtOnce) {  // row of the unit
        const int tile = r / kTileRows;
        const Row w = row_of(p, sp.map, x, h.head_unit, h.row_unit * sp.map.tokens + tile * tile_tokens, tile_tokens,
                             r % kTileRows);
        if (!w.there) continue;
        // row of the workspace that holds piece i
        auto ws_row = [&](int i) { return (size_t)piece_slot(c, i) * kRows + r; };
        float2 ml[kFly];
        float4 v[kFly];
        auto load = [&](int i0) {
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                ml[j] = make_float2(-INFINITY, 0.f);
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + j < h.n) {
                    ml[j] = sp.ws.ml[ws_row(i0 + j)];
                    v[j] = *reinterpret_cast<const float4*>(sp.ws.o + ws_row(i0 + j) * kD + col);
                }
            }
        };
        load(0);
        float M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
        for (int i = kFly; i < h.n; ++i) M = fmaxf(M, sp.ws.ml[ws_row(i)].x);
        const float use = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0;;) {
#pragma unroll
            for (int j = 0; j < kFly; ++j) {
                const float f = ex2_approx(ml[j].x - use);
                L += ml[j].y * f;
                acc.x += v[j].x * f;
                acc.y += v[j].y * f;
                acc.z += v[j].z * f;
                acc.w += v[j].w * f;
            }
            i0 += kFly;
            if (i0 >= h.n) break;
            load(i0);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L, unit = sp.o_unit;
        const size_t tok = (size_t)x.q0 + w.token;
        *reinterpret_cast<uint2*>(p.o + (tok * p.Hq + w.head) * kD + col) =
            make_uint2(pack_x2<kF16>(acc.x * inv * unit, acc.y * inv * unit), pack_x2<kF16>(acc.z * inv * unit, acc.w * inv * unit));
        if (col == 0 && p.lse != nullptr)
            p.lse[(size_t)w.head * p.total_q + tok] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
}

}  // namespace paged
}  // namespace attn

// paged_tiles_sm103.cuh -- attention of many query rows over a paged cache (prompts,
// chunks of prompts, mixed batches) on the tcgen05 tensor cores.
//
// The pipeline is the dense forward's (fmha_fwd_sm103.cuh): two tiles of 128 rows that
// share every K/V tile, S, P and O in tensor memory, a softmax warpgroup per tile, an
// epilogue warpgroup, one MMA warp and one TMA warp.  What the cache changes:
//   - A tile's rows are the (token, query head) pairs of one key/value head, token by
//     token: a TMA box of `heads` heads x 128 / heads tokens of q.  All heads of a group
//     use one K/V tile, and a causal tile spans few tokens, so little of it is masked.
//   - A K/V tile is gathered by TMA boxes of gcd(page_size, 128) rows, issued by the
//     lanes of the TMA warp side by side.  The pages of the next tile are looked up while
//     the warp waits for room.  Boxes behind the last key and boxes without a page read
//     past the last page, which TMA fills with zeros; keys without a page are masked.
//   - Rows of the last page behind the last key hold anything.  Their logits are masked,
//     but 0 x NaN is NaN in P V, so the softmax warps zero those rows of V in shared
//     memory before they hand over the weights of a sequence's last tile.
//   - A warp of its own walks the block's share (paged_sched_sm103.cuh) and posts the
//     pieces in a ring of kItems work items, so that no role waits for a length.
//   - P is rounded to the operands' type for its product, as in the dense forward: the tensor
//     cores take it in 16 bits.  Against 64 bits O is off by 2.1 to 2.4e-3 of its norm in bf16,
//     2.9e-4 in fp16; O's own rounding alone is 1.7e-3 and 2.1e-4.
//   - Rows of a tile that are no rows of the sequence are not stored: O goes through
//     shared memory to rows of 16-byte stores instead of a TMA store.
// Two prompts of 8192 (32/8 heads of 128) take 688 us, 1598 TFLOP/s, and 512 tokens on 32256
// cached ones (64/8 heads) 347 us, 1573 TFLOP/s, where the dense forward of the same shapes
// takes 666 and 343 us: 2640 SM cycles a key tile of two row tiles against 2520, of which
// the products are 2048, at the clock that the power cap leaves (1.65 to 1.8 GHz).
//
// Waits are bounded as in the dense forward: after a timeout all roles leave, copies and
// MMAs in flight are waited for, and tensor memory is freed.
#pragma once
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda.h>

#include "fmha_fwd_sm103.cuh"
#include "paged_common_sm103.cuh"
#include "paged_sched_sm103.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

constexpr int kSchedWarp = kMmaWarp + 3;
constexpr int kItems = 4;       // work items posted ahead
constexpr int kMaskRing = 8;    // page masks of the last K tiles
constexpr int kItemReaders = kSoftmaxWarps + 4 + 2;  // warps that read an item

// Registers a thread, of the launch's 4 x 128: the epilogue's row addresses take more than
// the dense forward's, its softmax can spare them (4 bytes of spills at head size 128, 20 at
// 64; a version without the first and with 12 of the second is as fast).
constexpr int kTilesRegsSoftmax = 168, kTilesRegsEpilogue = 96, kTilesRegsOther = 80;
static_assert(2 * kTilesRegsSoftmax + kTilesRegsEpilogue + kTilesRegsOther <= 4 * (65536 / kThreads),
              "register split exceeds the launch allocation");

struct Item {
    int seq, q0, q_len, kv_len;  // the sequence
    int head_unit, t0;      // head block, first token of tile 0
    int kb;                 // first key tile
    int n0, n1;             // key tiles of the two row tiles, one at least in all; n0 < 0: no more items
    int slot;               // workspace slot of a piece; -1: the unit is whole
    __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
    __device__ __forceinline__ int nmax() const { return n0 > n1 ? n0 : n1; }
};

template <int kD>
struct TilesGeo {
    static_assert(kD == 64 || kD == 128, "head size 64 or 128");
    static constexpr int kTile = kBN;
    static constexpr int kRows = kTiles * kBM;
    // 32 rows on 1000 keys, 8 heads: shares of at least 2 tiles 16.5 us, of 4 19.6 us; 8 sequences
    // of 200 to 600 keys: units up to 8 tiles longer than a share whole 18.1 us, up to 2 21.1 us
    static constexpr int kMinPiece = 2, kMinShare = 2, kCutTiles = 8;
    using ShareT = Share<kTile, kMinPiece, kMinShare>;
    using CursorT = Cursor<ShareT, kTile>;
    // K/V stages in flight, as many as fit beside Q: two of 64 KB at head size 128, four of
    // 32 KB at 64 (where the softmax paces a step and two measured within 1 %).
    static constexpr int kStages = kD == 64 ? 4 : 2;
    static constexpr int kHalves = kD / 64;
    static constexpr int kTileBytes = kBM * kD * 2;  // Q, K or V tile
    // barriers, as in the dense forward, and those of the work items
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQEmpty = kBarQFull + kTiles;
    static constexpr int kBarKvFull = kBarQEmpty + kTiles;     // [stage]: V_{g-1} and K_g landed
    static constexpr int kBarKvEmpty = kBarKvFull + kStages;   // [stage]: both read by their last MMA
    static constexpr int kBarSFull = kBarKvEmpty + kStages;
    static constexpr int kBarODone = kBarSFull + kTiles;
    static constexpr int kBarOFree = kBarODone + kTiles;
    static constexpr int kBarStatsFull = kBarOFree + kTiles;
    static constexpr int kBarStatsFree = kBarStatsFull + kTiles;
    static constexpr int kBarMmaDone = kBarStatsFree + kTiles;
    static constexpr int kBarItemFull = kBarMmaDone + 1;
    static constexpr int kBarItemEmpty = kBarItemFull + kItems;
    static constexpr int kBarCount = kBarItemEmpty + kItems;
    // shared memory, from a 1024-byte aligned base
    static constexpr int kSmemQ = 0;
    static constexpr int kSmemK = kSmemQ + kTiles * kTileBytes;
    static constexpr int kSmemV = kSmemK + kStages * kTileBytes;
    static constexpr int kSmemStage = kSmemV + kStages * kTileBytes;  // O staging: 4 KB a warp
    static constexpr int kSmemStats = kSmemStage + kHalfBytes;        // per tile and row: (m, l)
    static constexpr int kSmemBar = kSmemStats + kTiles * kBM * 8;
    static constexpr int kSmemTmemSlot = kSmemBar + kBarCount * 8;
    static constexpr int kSmemAbort = kSmemTmemSlot + 4;
    static constexpr int kSmemMmaExit = kSmemAbort + 4;
    static constexpr int kSmemMask = kSmemMmaExit + 4;
    static constexpr int kSmemStart = (kSmemMask + kMaskRing * 4 + 7) / 8 * 8;
    static constexpr int kSmemPart = kSmemStart + static_cast<int>(sizeof(StartPos));
    static constexpr int kSmemItems = kSmemPart + 3 * (kThreads / 32) * 8;
    static constexpr int kSmemUsed = kSmemItems + kItems * static_cast<int>(sizeof(Item));
    static constexpr int kSmemBytes = kSmemUsed + 1024;
    static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory limit");
    static_assert(kStages + 2 < kMaskRing, "a K tile's page mask is read before it is replaced");
};

struct TilesParams {
    int box_rows;   // rows of a K/V box: gcd(page_size, 128)
    int head_at_half;    // coordinates of a folded box: third = head * head_at_half,
    int head_at_group;   // fourth = head * head_at_group + row / 8
    int tile_tokens;  // tokens of a row tile
    int q_rows;       // rows that a Q box fills
    unsigned int poll_limit;
};

// 3-d tiled load global -> shared, completion counted on an mbarrier (bytes)
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar), "l"(policy)
        : "memory");
}

// kFold: one box has both 64-column halves of head size 128.  A K/V tile in shared memory
// is 8-row groups of 128-byte rows, kKvGroup bytes apart, the second half's columns kKvHalf
// behind the first's.  Copied half by half the halves are 16 KB blocks; in one box, where the
// cache's strides let a tensor map step over a row's halves inside a group (paged_api.cuh),
// the groups of the halves alternate, and a tile takes half the copies.
template <bool kF16, int kD, bool kFold>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p,
                       const __grid_constant__ SchedParams sp, const __grid_constant__ TilesParams tp) {
    using T = TilesGeo<kD>;
    constexpr int kStages = T::kStages;
    constexpr int kBoxHalves = kFold ? 1 : T::kHalves;  // halves that are copied apart
    constexpr int kKvHalf = kFold ? 1024 : kHalfBytes, kKvGroup = kFold ? 2048 : 1024;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::kSmemAbort);
    volatile int* mma_exit = reinterpret_cast<volatile int*>(smem + T::kSmemMmaExit);
    volatile uint32_t* page_mask = reinterpret_cast<volatile uint32_t*>(smem + T::kSmemMask);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kSmemTmemSlot);
    volatile Item* items = reinterpret_cast<volatile Item*>(smem + T::kSmemItems);
    StartPos* start = reinterpret_cast<StartPos*>(smem + T::kSmemStart);
    auto bar = [&](int i) -> uint32_t { return sbase + T::kSmemBar + 8 * i; };
    launch_dependents();
    touch_params(p);
    touch_params(sp);

    // ---- set-up: barriers, abort flag, tensor memory (the kernel in front may still run)
    if (warp == kLoadWarp && lane == 0) {
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(bar(T::kBarQFull + t), 1);
            mbar_init(bar(T::kBarQEmpty + t), 1);
            mbar_init(bar(T::kBarSFull + t), 1);
            mbar_init(bar(T::kBarODone + t), 1);
            mbar_init(bar(T::kBarOFree + t), 4 * 32);
            mbar_init(bar(T::kBarStatsFull + t), 4 * 32);
            mbar_init(bar(T::kBarStatsFree + t), 4 * 32);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(T::kBarKvFull + s), 1);
            mbar_init(bar(T::kBarKvEmpty + s), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(bar(T::kBarItemFull + i), 1);
            mbar_init(bar(T::kBarItemEmpty + i), kItemReaders);
        }
        mbar_init(bar(T::kBarMmaDone), 1);
        *abort_flag = 0;
        *mma_exit = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const unsigned int limit = tp.poll_limit;
    const int wg = warp / 4;

    // ---- this block's share
    wait_for_primary();
    typename T::ShareT sh;
    if (threadIdx.x == 0) sp.ws.header[blockIdx.x].n = 0;
    if (!find_share<kThreads, typename T::ShareT, T::kTile, T::kMinShare, T::kCutTiles, kD == 128>(
            p, sp, reinterpret_cast<long long*>(smem + T::kSmemPart), start, sh)) {
        if (warp == 0) tmem_dealloc(tmem_base, kTmemCols);
        return;
    }

    // Item j, for every lane of the warp; false: no more items, or the block gives up (*ok).
    auto get_item = [&](int j, Item& w, bool& ok) -> bool {
        const bool got = wait_bounded(bar(T::kBarItemFull + j % kItems), (j / kItems) & 1, abort_flag, limit);
        if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            return false;
        }
        const volatile Item& it = items[j % kItems];
        w.seq = it.seq;
        w.q0 = it.q0;
        w.q_len = it.q_len;
        w.kv_len = it.kv_len;
        w.head_unit = it.head_unit;
        w.t0 = it.t0;
        w.kb = it.kb;
        w.n0 = it.n0;
        w.n1 = it.n1;
        w.slot = it.slot;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T::kBarItemEmpty + j % kItems));
        return w.n0 >= 0;
    };

    if (wg == 3) {
      regs_dec<kTilesRegsOther>();
      if (warp == kSchedWarp) {
        // =========================== work items ============================
        typename T::CursorT cur;
        cur.first(p, sp, sh, *start);
        for (int j = 0;; ++j) {
            // units that see no key are written here: O = 0, LSE = -inf
            while (cur.ok && cur.keys == 0) {
                for (int i = lane; i < T::kRows * (kD / 8); i += 32) {
                    const int r = i / (kD / 8), t = r / kBM;
                    const Row w = row_of(p, sp.map, cur.x, cur.head_unit,
                                         cur.row_unit * sp.map.tokens + t * tp.tile_tokens, tp.tile_tokens, r % kBM);
                    if (!w.there) continue;
                    const size_t tok = static_cast<size_t>(cur.x.q0) + w.token;
                    *reinterpret_cast<uint4*>(p.o + (tok * p.Hq + w.head) * kD + i % (kD / 8) * 8) =
                        make_uint4(0u, 0u, 0u, 0u);
                    if (i % (kD / 8) == 0 && p.lse != nullptr)
                        p.lse[static_cast<size_t>(w.head) * p.total_q + tok] = -INFINITY;
                }
                cur.next(p, sp, sh);
            }
            if (j >= kItems) {
                const bool got = wait_bounded(bar(T::kBarItemEmpty + j % kItems), (j / kItems - 1) & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) break;
            }
            const bool more = cur.ok;
            if (lane == 0) {
                volatile Item& it = items[j % kItems];
                if (more) {
                    const int t0 = cur.row_unit * sp.map.tokens;
                    int n[kTiles];
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        const int a = t0 + t * tp.tile_tokens;
                        const int keys = a < cur.x.q_len
                                             ? visible_keys(p, cur.x, min(a + tp.tile_tokens, cur.x.q_len) - 1) : 0;
                        n[t] = max(min((keys + kBN - 1) / kBN, cur.tile_end) - cur.tile, 0);
                    }
                    it.seq = cur.s;
                    it.q0 = cur.x.q0;
                    it.q_len = cur.x.q_len;
                    it.kv_len = cur.x.kv_len;
                    it.head_unit = cur.head_unit;
                    it.t0 = t0;
                    it.kb = cur.tile;
                    it.n0 = n[0];
                    it.n1 = n[1];
                    it.slot = cur.whole() ? -1 : 2 * static_cast<int>(blockIdx.x) + (cur.tile == 0 ? 1 : 0);
                    if (!cur.whole() && cur.tile == 0)
                        sp.ws.header[blockIdx.x] =
                            PieceHeader{sh.pieces(cur.at, cur.tiles, static_cast<int>(blockIdx.x)), cur.s, cur.head_unit,
                                        cur.row_unit};
                } else {
                    it.n0 = -1;
                }
                mbar_arrive(bar(T::kBarItemFull + j % kItems));
            }
            __syncwarp();
            if (!more) break;
            cur.next(p, sp, sh);
        }
      } else if (warp == kLoadWarp) {
        // =========================== TMA producer ===========================
        // Stages as in the dense forward: stage g holds V of fill g - 1 and K of fill g.
        // Lanes 0-15 copy K boxes, lanes 16-31 V boxes: box (lane % 16) / halves of the
        // tile, half (lane % 16) % halves of its columns.
        const uint64_t pol_q = l2_policy_evict_first();
        const uint64_t pol_kv = l2_policy_evict_last();
        const int box = (lane & 15) / kBoxHalves, half = (lane & 15) % kBoxHalves;
        const int n_boxes = kBM / tp.box_rows;
        const bool copies = box < n_boxes;
        const uint32_t box_at = half * kHalfBytes + box * (tp.box_rows / 8) * kKvGroup;
        int g = 0;                       // stages issued
        int q_issued[kTiles] = {0, 0};   // Q_t fills posted so far
        bool ok = true;
        int jk = 0, ktk = 0;             // items taken; key tile of the last one whose K is next
        Item wk{};
        // page and row of this lane's box of that tile (-1: behind the last key)
        int page = -1, page_row = 0;
        bool in_range = false;
        auto look_up = [&]() {
            const int key = (wk.kb + ktk) * kBN + box * tp.box_rows;
            in_range = copies && key < wk.kv_len;
            page = -1;
            if (in_range) {
                const int col = static_cast<int>(p.by_page.quot(key));
                page = p.table[wk.seq * p.table_stride + col];
                page_row = key - col * p.page_size;
            }
        };
        // Q of a unit; a tile without key tiles needs none
        auto post_q = [&]() -> bool {
            const int h0 = sp.map.kv_head(wk.head_unit) * p.group + wk.head_unit % sp.map.splits * sp.map.heads;
            for (int t = 0; t < kTiles; ++t) {
                const bool got =
                    q_issued[t] == 0 || wait_bounded(bar(T::kBarQEmpty + t), (q_issued[t] - 1) & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) return false;
                if (lane == 0) {
                    if (wk.n(t) > 0) {
                        mbar_arrive_expect_tx(bar(T::kBarQFull + t), T::kHalves * tp.q_rows * 128);
                        for (int h = 0; h < T::kHalves; ++h)
                            tma_load_3d(sbase + T::kSmemQ + t * T::kTileBytes + h * kHalfBytes, &tm_q, h * 64, h0,
                                        wk.q0 + wk.t0 + t * tp.tile_tokens, bar(T::kBarQFull + t), pol_q);
                    } else {
                        mbar_arrive(bar(T::kBarQFull + t));
                    }
                }
                ++q_issued[t];
            }
            return true;
        };
        bool have_k = get_item(jk, wk, ok), have_v = false;
        int v_page = 0, v_row = 0, v_hkv = 0;
        if (have_k) look_up();
        while (ok && (have_k || have_v)) {
            const int st = g % kStages, use = g / kStages;
            const bool got = use == 0 || wait_bounded(bar(T::kBarKvEmpty + st), (use - 1) & 1, abort_flag, limit);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const bool valid = in_range && page >= 0 && page < p.n_pages;
            const int k_page = valid ? page : p.n_pages, k_row = valid ? page_row : 0;  // past the last page: zeros
            const int k_hkv = sp.map.kv_head(wk.head_unit);
            const uint32_t miss = __ballot_sync(0xffffffffu, in_range && !valid);
            if (lane == 0) {
                if (have_k) {
                    uint32_t mask = 0;  // one bit per 16 keys
                    const int per = tp.box_rows / 16;
                    for (int b = 0; miss != 0 && b < n_boxes; ++b)
                        if ((miss >> (b * kBoxHalves)) & 1) mask |= ((1u << per) - 1u) << (b * per);
                    page_mask[g % kMaskRing] = mask;
                }
                mbar_arrive_expect_tx(bar(T::kBarKvFull + st), ((have_k ? 1 : 0) + (have_v ? 1 : 0)) * T::kTileBytes);
            }
            __syncwarp();
            if (copies && (lane < 16 ? have_k : have_v)) {
                const bool is_k = lane < 16;
                const uint32_t to = sbase + box_at + (is_k ? T::kSmemK + st * T::kTileBytes
                                                           : T::kSmemV + ((g - 1) % kStages) * T::kTileBytes);
                const CUtensorMap* map = is_k ? &tm_k : &tm_v;
                const int hkv = is_k ? k_hkv : v_hkv, row = is_k ? k_row : v_row, pg = is_k ? k_page : v_page;
                if constexpr (kFold)
                    tma_load_5d(to, map, 0, 0, hkv * tp.head_at_half, hkv * tp.head_at_group + row / 8, pg,
                                bar(T::kBarKvFull + st), pol_kv);
                else
                    tma_load_4d(to, map, half * 64, hkv, row, pg, bar(T::kBarKvFull + st), pol_kv);
            }
            __syncwarp();
            ++g;  // counted before anything can fail: the drain below waits for these copies
            if (have_k && ktk == 0 && !post_q()) {
                ok = false;
                break;
            }
            have_v = have_k;
            v_page = k_page;
            v_row = k_row;
            v_hkv = k_hkv;
            if (have_k) {
                if (++ktk >= wk.nmax()) {
                    ktk = 0;
                    have_k = get_item(++jk, wk, ok);
                }
                if (have_k) look_up();
            }
        }
        // drain: every copy this warp issued has landed before the block may exit
        if (lane == 0) {
            for (int t = 0; t < kTiles; ++t)
                if (q_issued[t] > 0) drain_bounded(bar(T::kBarQFull + t), (q_issued[t] - 1) & 1, limit);
            for (int st = 0; st < kStages; ++st) {
                const int fills = g > st ? (g - 1 - st) / kStages + 1 : 0;
                if (fills) drain_bounded(bar(T::kBarKvFull + st), (fills - 1) & 1, limit);
            }
        }
        __syncwarp();
      } else if (warp == kMmaWarp) {
        // =========================== MMA issuer =============================
        constexpr uint32_t idesc_qk = idesc_f16kind_f32(kBM, kBN, false, kF16);
        constexpr uint32_t idesc_pv = idesc_f16kind_f32(kBM, kD, true, kF16);
        const uint64_t q_desc0 = sdesc_sw128(sbase + T::kSmemQ, 16, 1024);
        const uint64_t k_desc0 = sdesc_sw128(sbase + T::kSmemK, 16, kKvGroup);
        const uint64_t v_desc0 = sdesc_sw128(sbase + T::kSmemV, kKvHalf, kKvGroup);
        auto issue_qk = [&](int t, int ks) {
            const uint32_t d = tmem_base + kTmemS + 128 * t;
            const uint64_t qd = q_desc0 + static_cast<uint64_t>((t * T::kTileBytes) >> 4);
            const uint64_t kd = k_desc0 + static_cast<uint64_t>((ks * T::kTileBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
                const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
                mma_bf16_ss(d, qd + off, kd + static_cast<uint64_t>(((kk >> 2) * kKvHalf + (kk & 3) * 32) >> 4), idesc_qk,
                            kk > 0 ? 1u : 0u);
            }
        };
        auto issue_pv = [&](int t, int vs, int h, bool accumulate) {
            const uint32_t d = tmem_base + kTmemO + 128 * t;
            const uint32_t pa = tmem_base + kTmemS + 128 * t;
            const uint64_t vd = v_desc0 + static_cast<uint64_t>((vs * T::kTileBytes) >> 4);
#pragma unroll
            for (int q = 0; q < kBN / 32; ++q) {
                const int kk = h * (kBN / 32) + q;
                mma_bf16_ts(d, pa + kk * 8, vd + static_cast<uint64_t>((kk * 2 * kKvGroup) >> 4), idesc_pv,
                            (accumulate || kk > 0) ? 1u : 0u);
            }
        };
        int kv = 0;  // K/V tiles consumed so far (stage kv carries K_kv)
        bool ok = true;
        // S_t(0) of item j from the K of stage `st`, which has landed
        auto first_s = [&](int j, const Item& w, int t, int st) -> bool {
            if (!wait_bounded(bar(T::kBarQFull + t), j & 1, abort_flag, limit)) return false;
            tc_fence_after();
            if (elect_one()) {
                if (w.n(t) > 0) {
                    issue_qk(t, st);
                    mma_commit(bar(T::kBarSFull + t));
                }
                if (w.n(t) <= 1) mma_commit(bar(T::kBarQEmpty + t));  // Q_t no longer read
            }
            __syncwarp();
            return true;
        };
        Item w;
        bool have = get_item(0, w, ok);
        if (have) {
            ok = wait_bounded(bar(T::kBarKvFull), 0, abort_flag, limit) && first_s(0, w, 0, 0) && first_s(0, w, 1, 0);
            if (ok && elect_one()) mma_commit(bar(T::kBarKvEmpty));  // stage 0 holds K_0 alone
            __syncwarp();
        }
        Item wn;
        bool have_n = false;
        // Step kt of item j.  The last step of an item is code of its own and the tiles are
        // unrolled: the loop over the others stays a straight run of MMAs (2900 to 2700
        // cycles a step).
        auto step = [&](auto last_step, int j, int kt) -> bool {
            constexpr bool kLast = decltype(last_step)::value;
            const int vs = kv % kStages;
            const int kn = kv + 1;  // stage kn: V_{kt} and K_{kt+1} (or the next item's K_0)
            if constexpr (kLast) {
                have_n = get_item(j + 1, wn, ok);
                if (!ok) return false;
            }
            if (!wait_bounded(bar(T::kBarKvFull + kn % kStages), (kn / kStages) & 1, abort_flag, limit)) return false;
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const int nt = w.n(t);
                if (kt < nt) {
                    // the first P.V of a unit overwrites O_t: the previous unit's
                    // epilogue must have read it out of tensor memory
                    if (kt == 0 && j > 0 && !wait_bounded(bar(T::kBarOFree + t), (j - 1) & 1, abort_flag, limit))
                        return false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        named_bar_sync(kBarP + 2 * t + h, kBarPThreads);
                        tc_fence_after();
                        if (elect_one()) {
                            issue_pv(t, vs, h, kt > 0);
                            if (h == 1 && kt == nt - 1) mma_commit(bar(T::kBarODone + t));  // O_t final
                        }
                        __syncwarp();
                    }
                } else if (nt == 0 && kt == 0) {
                    // tile without work: its (all-zero) O_t is "final" once the previous
                    // unit's was read, which keeps the barrier in step with the epilogue
                    if (j > 0 && !wait_bounded(bar(T::kBarOFree + t), (j - 1) & 1, abort_flag, limit)) return false;
                    if (elect_one()) mma_commit(bar(T::kBarODone + t));
                    __syncwarp();
                }
                if constexpr (kLast) {
                    // the next item's S_t(0), before the other tile's last P.V: its softmax
                    // starts while this item ends
                    if (have_n && !first_s(j + 1, wn, t, kn % kStages)) return false;
                } else if (kt + 1 < nt) {
                    if (elect_one()) {
                        issue_qk(t, kn % kStages);
                        mma_commit(bar(T::kBarSFull + t));
                        if (kt + 2 == nt) mma_commit(bar(T::kBarQEmpty + t));  // last S_t of the unit
                    }
                    __syncwarp();
                }
            }
            // stage kn is free once its V and its K have been read
            if ((!kLast || have_n) && elect_one()) mma_commit(bar(T::kBarKvEmpty + kn % kStages));
            __syncwarp();
            ++kv;
            return true;
        };
        for (int j = 0; ok && have; ++j) {
            const int nm = w.nmax();
            for (int kt = 0; ok && kt + 1 < nm; ++kt) ok = step(std::false_type{}, j, kt);
            if (ok) ok = step(std::true_type{}, j, nm - 1);
            have = have_n;
            w = wn;
        }
        *mma_exit = 1;  // the release warp may stop
        // every MMA this warp issued has completed before tensor memory is freed
        if (elect_one()) {
            mma_commit(bar(T::kBarMmaDone));
            drain_bounded(bar(T::kBarMmaDone), 0, limit);
        }
        __syncwarp();
      } else {
        // =========================== release warp ===========================
        // As in the dense forward: once the block gives up, completes the P barriers that
        // the MMA warp may be waiting on until that warp has left its loop.
        const unsigned long long cap = 64ull * limit;
        unsigned long long i = 0;
        for (; i < cap && !*mma_exit; ++i) {
            if (*abort_flag) {
                for (int b = 0; b < 2 * kTiles; ++b)
                    for (int k = 0; k < 4; ++k) named_bar_arrive(kBarP + b, kBarPThreads);
            } else {
                nanosleep_ns(1024);
            }
        }
        if (i == cap) atomicOr(&g_attn_status, kStatusTimeout);
      }
    } else if (wg < 2) {
        // =========================== softmax warpgroups =====================
        regs_inc<kTilesRegsSoftmax>();
        const int t = warp / 4;
        const int wq = warp % 4;
        const int r = wq * 32 + lane;  // row within the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem_base + lane_off + kTmemS + 128 * t;
        const uint32_t tO = tmem_base + lane_off + kTmemO + 128 * t;
        const float sl2 = p.scale_log2;
        const int row_token = r / sp.map.heads;  // token of this row within the tile
        int sc = 0;  // S_t products consumed so far
        int kv = 0;  // K/V tiles before this unit
        bool ok = true;

        for (int j = 0; ok; ++j) {
            Item w;
            if (!get_item(j, w, ok)) break;
            const int nt = w.n(t), nm = w.nmax();
            const int token = w.t0 + t * tp.tile_tokens + row_token;
            int nvis = 0;  // visible keys of this row from the item's next key tile on
            if (row_token < tp.tile_tokens && token < w.q_len)
                nvis = (p.causal ? max(w.kv_len - w.q_len + token + 1, 0) : w.kv_len) - w.kb * kBN;
            // keys of the sequence in its last tile, and which of the item's tiles that is
            // (past the last: the item does not reach it, or it is full)
            const int last_kt = w.kv_len % kBN != 0 ? w.kv_len / kBN - w.kb : 0x7fffffff;
            const int last_keys = w.kv_len % kBN;
            float m_run = -INFINITY;  // running max (log2 units of scaled logits) used by the weights
            float l_run = 0.f;        // running sum of weights

            for (int kt = 0; kt < nt; ++kt, ++sc, nvis -= kBN) {
                const bool got = wait_bounded(bar(T::kBarSFull + t), sc & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t missing = page_mask[(kv + kt) % kMaskRing];
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));

                if (nvis < kBN) {
#pragma unroll
                    for (int jj = 0; jj < kBN; ++jj)
                        if (jj >= nvis) s[jj] = __float_as_uint(-INFINITY);
                }
                if (missing != 0) {  // keys without a page
#pragma unroll
                    for (int jj = 0; jj < kBN; ++jj)
                        if ((missing >> (jj / 16)) & 1) s[jj] = __float_as_uint(-INFINITY);
                }
                if (kt == last_kt) {
                    // V's rows behind the last key become zero.  V_kt lands with stage kv + kt + 1,
                    // which is not refilled before this tile's weights have been used.
                    const int sn = kv + kt + 1;
                    const bool landed = wait_bounded(bar(T::kBarKvFull + sn % kStages), (sn / kStages) & 1, abort_flag, limit);
                    if (!__all_sync(0xffffffffu, landed)) {
                        ok = false;
                        break;
                    }
                    uint8_t* v = smem + T::kSmemV + ((kv + kt) % kStages) * T::kTileBytes;
                    const int first = last_keys * 8;  // 16-byte pieces of a half, 64 a group
                    for (int h = 0; h < T::kHalves; ++h)
                        for (int i = first + r; i < kBN * 8; i += 128)
                            *reinterpret_cast<uint4*>(v + h * kKvHalf + (i >> 6) * kKvGroup + (i & 63) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                // tile maximum (three-input max, 8 independent chains)
                float mx[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    mx[q] = fmax3(__uint_as_float(s[q]), __uint_as_float(s[8 + q]), __uint_as_float(s[16 + q]));
#pragma unroll
                for (int base = 24; base + 16 <= kBN; base += 16)
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        mx[q] = fmax3(mx[q], __uint_as_float(s[base + q]), __uint_as_float(s[base + 8 + q]));
                // the last eight logits join the chains' tree
                auto last = [&](int q) { return __uint_as_float(s[kBN - 8 + q]); };
                const float tmax = fmaxf(fmax3(fmax3(mx[0], mx[1], last(0)), fmax3(mx[2], mx[3], last(1)),
                                               fmax3(mx[4], mx[5], last(2))),
                                         fmax3(fmax3(mx[6], mx[7], last(3)), fmax3(last(4), last(5), last(6)), last(7)));
                const float m_tile = tmax * sl2;

                // raise the running max only when the tile max exceeds it by more than 2^15
                float alpha = 1.f;
                if (m_tile - m_run > kRescaleLog2) {
                    alpha = ex2_approx(m_run - m_tile);
                    m_run = m_tile;
                }
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                const bool need = (kt > 0) && (alpha != 1.f);
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int c = 0; c < kD / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(tO + 16 * c, o);
                        tmem_wait_ld_regs16(o);
#pragma unroll
                        for (int q = 0; q < 16; q += 2) {
                            float x0, x1;
                            fmul2_b(x0, x1, __uint_as_float(o[q]), __uint_as_float(o[q + 1]), alpha);
                            o[q] = __float_as_uint(x0);
                            o[q + 1] = __float_as_uint(x1);
                        }
                        tmem_st16(tO + 16 * c, o);
                    }
                }
                // weights 2^(s*scale*log2e - m_use), their row sum, P_t in two halves of 64 keys
                float rs0 = 0.f, rs1 = 0.f, rs2 = 0.f, rs3 = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int c = 2 * h; c < 2 * h + 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int q = 0; q < 16; q += 2) {
                            const int e = 32 * c + 2 * q;
                            float a0, a1, b0, b1;
                            ffma2_bc(a0, a1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), sl2, -m_use);
                            ffma2_bc(b0, b1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]), sl2, -m_use);
                            a0 = ex2_approx(a0);
                            a1 = ex2_approx(a1);
                            b0 = ex2_approx(b0);
                            b1 = ex2_approx(b1);
                            if (q & 2) {
                                fadd2_acc(rs2, rs3, a0, a1);
                                fadd2_acc(rs2, rs3, b0, b1);
                            } else {
                                fadd2_acc(rs0, rs1, a0, a1);
                                fadd2_acc(rs0, rs1, b0, b1);
                            }
                            pk[q] = pack_x2<kF16>(a0, a1);
                            pk[q + 1] = pack_x2<kF16>(b0, b1);
                        }
                        tmem_st16(tS + 16 * c, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    named_bar_arrive(kBarP + 2 * t + h, kBarPThreads);
                }
                l_run = l_run * alpha + ((rs0 + rs1) + (rs2 + rs3));
            }
            if (!ok) break;
            kv += nm;

            // hand (m, l) of every row to the epilogue warpgroup and start the next unit
            const bool got = j == 0 || wait_bounded(bar(T::kBarStatsFree + t), (j - 1) & 1, abort_flag, limit);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            reinterpret_cast<float2*>(smem + T::kSmemStats)[t * kBM + r] = make_float2(m_run, l_run);
            mbar_arrive(bar(T::kBarStatsFull + t));
        }
    } else {
        // =========================== epilogue warpgroup =====================
        regs_dec<kTilesRegsEpilogue>();
        const int wq = warp % 4;
        const int r = wq * 32 + lane;  // row within a tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        uint8_t* stage = smem + T::kSmemStage + wq * 4096;  // this warp's 32 rows of 128 bytes
        const int row_token = r / sp.map.heads, row_head = r % sp.map.heads;
        bool ok = true;
        for (int j = 0; ok; ++j) {
            Item w;
            if (!get_item(j, w, ok)) break;
            const int h_in = w.head_unit % sp.map.splits * sp.map.heads + row_head;  // head within the group
            const int head = w.head_unit / sp.map.splits * p.group + h_in;
            for (int t = 0; t < kTiles; ++t) {
                // O_t final (every P.V of the unit completed) and (m, l) of its rows
                const bool got = wait_bounded(bar(T::kBarODone + t), j & 1, abort_flag, limit) &&
                                 wait_bounded(bar(T::kBarStatsFull + t), j & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 ml = reinterpret_cast<const float2*>(smem + T::kSmemStats)[t * kBM + r];
                mbar_arrive(bar(T::kBarStatsFree + t));
                const int nt = w.n(t);
                const int token = w.t0 + t * tp.tile_tokens + row_token;
                const bool there = row_token < tp.tile_tokens && token < w.q_len && h_in < p.group;
                // row of [total_q, Hq] (at most 2^31 - 1 of them); negative: no such row
                const int out_row = there ? (w.q0 + token) * p.Hq + head : -1;
                const uint32_t tO = tmem_base + lane_off + kTmemO + 128 * t;
                const float inv_l = ml.y == 0.f ? 0.f : 1.f / ml.y;
                const size_t ws_row = static_cast<size_t>(w.slot >= 0 ? w.slot : 0) * T::kRows + t * kBM + r;
#pragma unroll
                for (int h = 0; h < T::kHalves; ++h) {
                    uint32_t o[64];
                    if (nt > 0) {
                        tmem_ld32(tO + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
                        tmem_ld32(tO + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
                        tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[32]>(&o[0]));
                        tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[32]>(&o[32]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 64; ++e) o[e] = 0u;
                    }
                    if (h == T::kHalves - 1) {  // O_t may now be overwritten by the next item's first P.V
                        tc_fence_before();
                        mbar_arrive(bar(T::kBarOFree + t));
                    }
                    if (w.slot >= 0 && !__any_sync(0xffffffffu, there)) continue;
                    if (w.slot >= 0) {  // a piece: raw sums to its workspace slot, 32 columns at a time
                        float* dst = sp.ws.o + (ws_row - lane) * kD + 64 * h;  // of the warp's first row
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                                    make_uint4(o[32 * c + 4 * q], o[32 * c + 4 * q + 1], o[32 * c + 4 * q + 2],
                                               o[32 * c + 4 * q + 3]);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int rr = 4 * i + lane / 8, q = lane % 8;
                                *reinterpret_cast<uint4*>(dst + rr * kD + 32 * c + 4 * q) =
                                    *reinterpret_cast<const uint4*>(stage + rr * 128 + ((q ^ (rr & 7)) * 16));
                            }
                            __syncwarp();
                        }
                        continue;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {  // 16-byte chunk q of this row's half
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            fmul2_b(f[e], f[e + 1], __uint_as_float(o[8 * q + e]), __uint_as_float(o[8 * q + e + 1]),
                                    inv_l);
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                            make_uint4(pack_x2<kF16>(f[0], f[1]), pack_x2<kF16>(f[2], f[3]),
                                       pack_x2<kF16>(f[4], f[5]), pack_x2<kF16>(f[6], f[7]));
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // four rows at a time, eight lanes a row
                        const int rr = 4 * i + lane / 8, q = lane % 8;
                        const int to = __shfl_sync(0xffffffffu, out_row, rr);
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((q ^ (rr & 7)) * 16));
                        if (to >= 0)
                            *reinterpret_cast<uint4*>(p.o + static_cast<size_t>(to) * kD + 64 * h + 8 * q) = x;
                    }
                    __syncwarp();
                }
                if (there) {
                    if (w.slot >= 0)
                        sp.ws.ml[ws_row] = ml;
                    else if (p.lse != nullptr)
                        p.lse[static_cast<size_t>(head) * p.total_q + w.q0 + token] =
                            ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.69314718055994531f;
                }
            }
        }
    }

    // ---- teardown: all tensor-memory traffic is complete; free it
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace paged
}  // namespace attn

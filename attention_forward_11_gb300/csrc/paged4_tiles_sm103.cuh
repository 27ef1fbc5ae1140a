// paged4_tiles_sm103.cuh -- attention of many query rows over a paged cache in 4 bits (prompts,
// chunks of prompts, mixed batches) on the tcgen05 tensor cores.
//
// The pipeline is paged_tiles_sm103.cuh's: two tiles of 128 (token, head) rows that share every
// K/V tile, S, P and O in tensor memory, a softmax warpgroup per tile, work items posted by a
// warp that walks the block's share.  All operands are fp16 (paged4_common_sm103.cuh).  What the
// codes change:
//   - The epilogue's warpgroup fills the stages instead of TMA: a row's codes are copied by D / 32
//     lanes, each for itself and a tile ahead, converted without rounding and stored where TMA
//     would have put them.
//   - Every lane finds the page of a row of its own, so pages of any size are taken; rows without
//     a key become zeros, so V needs no clean-up.
//   - The softmax warps turn bf16 queries into fp16 in shared memory before their first product; a
//     row's power of two goes into its softmax scale.  (Between two fills it cost two prompts of
//     8192, 32/8 heads, 890 instead of 808 us.)
//   - Fills and epilogues are one sequence in a fixed order in which nothing waits for what comes
//     behind it: item j's epilogue runs after the fill of the stage behind the one with its last V.
//     It stores O as it comes out of tensor memory, a row's 64 bytes a thread.
//
// 512 tokens on 32256 cached ones, 64/8 heads of 128, take 418 us, 1300 TFLOP/s (the 16-bit kernel 336);
// at head size 64 287 (254); two prompts of 8192, 32/8 heads, 788 us (629); 4 chunks of 100 to 512 among 36
// tokens 166 us (172).  What bounds it is the fills' warpgroup, 2750 busy cycles a step of two row
// tiles (1150 of conversions and stores, 1175 of page numbers, addresses and copies), and shared memory,
// which the products read at its full rate half of the time.  Measured and not kept: codes by TMA into
// shared staging (614 us); copies or addresses by other warps of the MMA's warpgroup, which slow its
// issue (466 to 564); codes taken into registers before the stage is free (452).
//
// Waits are bounded as in the dense forward: after a timeout all roles leave, copies and
// MMAs in flight are waited for, and tensor memory is freed.
#pragma once
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda.h>

#include "fmha_fwd_sm103.cuh"
#include "paged4_common_sm103.cuh"
#include "paged4_rows_sm103.cuh"
#include "paged_common_sm103.cuh"
#include "paged_sched_sm103.cuh"
#include "paged_tiles_sm103.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace paged {

// Registers a thread, of the launch's 4 x 128: the fills take more than the dense forward's epilogue.
constexpr int kTiles4RegsSoftmax = 168, kTiles4RegsEpilogue = 112, kTiles4RegsOther = 64;
static_assert(2 * kTiles4RegsSoftmax + kTiles4RegsEpilogue + kTiles4RegsOther <= 4 * (65536 / kThreads),
              "register split exceeds the launch allocation");

// The smallest unit of V whose quotient by a row's sum, at most 2^47 (2^31 weights below 2^16), is a normal number:
// the epilogue's one product for both costs two prompts of 8192 786 us, one for each 798.
constexpr float kTiles4LeastUnit = 0x1p-79f;

template <int kD>
struct Tiles4Geo {
    static_assert(kD == 64 || kD == 128, "head size 64 or 128");
    static constexpr int kTile = kBN;
    static constexpr int kRows = kTiles * kBM;
    // 32 rows on 1000 keys, 8 heads: shares of at least 2 tiles 18.4 us, of 4 21.0 us (256 rows 25.1 / 27.6);
    // 8 sequences of 200 to 600 keys: units up to 8 tiles longer than a share whole 18.7 us, up to 2 20.0 us
    // (14.8 / 17.0 at head size 64)
    static constexpr int kMinPiece = 2, kMinShare = 2, kCutTiles = 8;
    using ShareT = Share<kTile, kMinPiece, kMinShare>;
    using CursorT = Cursor<ShareT, kTile>;
    // K/V stages in flight, as many as fit beside Q: two of 64 KB at head size 128, four of
    // 32 KB at 64 (3 or 2 there are as fast: a chunk of 512 on 32256 285 us, two prompts of 8192 600).
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
    static constexpr int kItems = 8;  // posted ahead: the fills are up to four items ahead of the epilogue
    static constexpr int kBarItemFull = kBarMmaDone + 1;
    static constexpr int kBarItemEmpty = kBarItemFull + kItems;
    static constexpr int kBarQReady = kBarItemEmpty + kItems;  // Q_t is fp16
    static constexpr int kBarCount = kBarQReady + kTiles;
    // shared memory, from a 1024-byte aligned base
    static constexpr int kSmemQ = 0;
    static constexpr int kSmemK = kSmemQ + kTiles * kTileBytes;
    static constexpr int kSmemV = kSmemK + kStages * kTileBytes;
    // codes of the next K tile and of the next V tile, 16 bytes a thread and row, and their scales
    static constexpr int kCodeBytes = kBM * kD / 2, kScaleBytes = kBM * (kD / 32) * 4;
    static constexpr int kSmemCodes = kSmemV + kStages * kTileBytes;
    static constexpr int kSmemStats = kSmemCodes + 2 * (kCodeBytes + kScaleBytes);  // per tile and row: (m, l)
    static constexpr int kSmemBar = kSmemStats + kTiles * kBM * 8;
    static constexpr int kSmemTmemSlot = kSmemBar + kBarCount * 8;
    static constexpr int kSmemAbort = kSmemTmemSlot + 4;
    static constexpr int kSmemMmaExit = kSmemAbort + 4;
    static constexpr int kSmemMask = kSmemMmaExit + 4;
    static constexpr int kMaskWords = kBN / 32;  // one bit a key
    static constexpr int kSmemStart = (kSmemMask + kMaskRing * 4 * kMaskWords + 7) / 8 * 8;
    static constexpr int kSmemPart = kSmemStart + static_cast<int>(sizeof(StartPos));
    static constexpr int kSmemItems = kSmemPart + 3 * (kThreads / 32) * 8;
    static constexpr int kSmemUsed = kSmemItems + kItems * static_cast<int>(sizeof(Item));
    static constexpr int kSmemBytes = kSmemUsed + 1024;
    static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-CTA shared memory limit");
    static_assert(kStages + 2 < kMaskRing, "a K tile's page mask is read before it is replaced");
};

// kF16: q's and o's type.
template <bool kF16, int kD>
__global__ void __launch_bounds__(kThreads, 1)
    paged4_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Paged4Params p,
                        const __grid_constant__ SchedParams sp, const __grid_constant__ TilesParams tp) {
    using T = Tiles4Geo<kD>;
    constexpr int kStages = T::kStages;
    constexpr bool kTurnsQ = !kF16;  // Q becomes fp16 in shared memory
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
            mbar_init(bar(T::kBarKvFull + s), 4);
            mbar_init(bar(T::kBarKvEmpty + s), 1);
        }
        for (int i = 0; i < T::kItems; ++i) {
            mbar_init(bar(T::kBarItemFull + i), 1);
            mbar_init(bar(T::kBarItemEmpty + i), kItemReaders);
        }
        for (int t = 0; t < kTiles; ++t) mbar_init(bar(T::kBarQReady + t), 4);
        mbar_init(bar(T::kBarMmaDone), 1);
        *abort_flag = 0;
        *mma_exit = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
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
    // Units up to 1.35 shares whole at head size 128, as in the 16-bit kernel.  Codes need L2 less: 576 to 416
    // tokens on 32000 keys, 64/8 heads, whole / cut 396 / 399, 400 / 379, 398 / 358, 396 / 336, 315 / 315, 295 / 294 us;
    // on 8000 119 / 119, 118 / 124, 117 / 117, 118 / 111, 106 / 106, 99 / 99.
    if (!find_share<kThreads, typename T::ShareT, T::kTile, T::kMinShare, T::kCutTiles, kD == 128>(
            p, sp, reinterpret_cast<long long*>(smem + T::kSmemPart), start, sh)) {
        if (warp == 0) tmem_dealloc(tmem_base, kTmemCols);
        return;
    }

    // Item j, for every lane of the warp; false: no more items, or the block gives up (*ok).
    auto release_item = [&](int j) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T::kBarItemEmpty + j % T::kItems));
    };
    auto look_at_item = [&](int j, Item& w, bool& ok) -> bool {
        const bool got = wait_bounded(bar(T::kBarItemFull + j % T::kItems), (j / T::kItems) & 1, abort_flag, limit);
        if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            return false;
        }
        const volatile Item& it = items[j % T::kItems];
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
        return w.n0 >= 0;
    };
    auto get_item = [&](int j, Item& w, bool& ok) -> bool {
        const bool more = look_at_item(j, w, ok);
        if (ok) release_item(j);
        return more;
    };

    if (wg == 3) {
      regs_dec<kTiles4RegsOther>();
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
            if (j >= T::kItems) {
                const bool got = wait_bounded(bar(T::kBarItemEmpty + j % T::kItems), (j / T::kItems - 1) & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) break;
            }
            const bool more = cur.ok;
            if (lane == 0) {
                volatile Item& it = items[j % T::kItems];
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
                mbar_arrive(bar(T::kBarItemFull + j % T::kItems));
            }
            __syncwarp();
            if (!more) break;
            cur.next(p, sp, sh);
        }
      } else if (warp == kLoadWarp) {
        // =========================== Q ======================================
        const uint64_t pol_q = l2_policy_evict_first();
        int q_issued[kTiles] = {0, 0};   // Q_t fills posted so far
        bool ok = true;
        Item wk{};
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
        for (int j = 0; get_item(j, wk, ok) && (ok = post_q()); ++j) {
        }
        // drain: every copy this warp issued has landed before the block may exit
        if (lane == 0) {
            for (int t = 0; t < kTiles; ++t)
                if (q_issued[t] > 0) drain_bounded(bar(T::kBarQFull + t), (q_issued[t] - 1) & 1, limit);
        }
        __syncwarp();
      } else if (warp == kMmaWarp) {
        // =========================== MMA issuer =============================
        constexpr uint32_t idesc_qk = idesc_f16kind_f32(kBM, kBN, false, true);
        constexpr uint32_t idesc_pv = idesc_f16kind_f32(kBM, kD, true, true);
        const uint64_t q_desc0 = sdesc_sw128(sbase + T::kSmemQ, 16, 1024);
        const uint64_t k_desc0 = sdesc_sw128(sbase + T::kSmemK, 16, 1024);
        const uint64_t v_desc0 = sdesc_sw128(sbase + T::kSmemV, kHalfBytes, 1024);
        auto issue_qk = [&](int t, int ks) {
            const uint32_t d = tmem_base + kTmemS + 128 * t;
            const uint64_t qd = q_desc0 + static_cast<uint64_t>((t * T::kTileBytes) >> 4);
            const uint64_t kd = k_desc0 + static_cast<uint64_t>((ks * T::kTileBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
                const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
                mma_bf16_ss(d, qd + off, kd + static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4), idesc_qk,
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
                mma_bf16_ts(d, pa + kk * 8, vd + static_cast<uint64_t>((kk * 2 * 1024) >> 4), idesc_pv,
                            (accumulate || kk > 0) ? 1u : 0u);
            }
        };
        int kv = 0;  // K/V tiles consumed so far (stage kv carries K_kv)
        bool ok = true;
        // S_t(0) of item j from the K of stage `st`, which has landed
        auto first_s = [&](int j, const Item& w, int t, int st) -> bool {
            if (!wait_bounded(bar((kTurnsQ ? T::kBarQReady : T::kBarQFull) + t), j & 1, abort_flag, limit)) return false;
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
        // unrolled: the loop over the others stays a straight run of MMAs, as in the 16-bit kernel,
        // where that was measured.
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
        regs_inc<kTiles4RegsSoftmax>();
        const int t = warp / 4;
        const int wq = warp % 4;
        const int r = wq * 32 + lane;  // row within the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem_base + lane_off + kTmemS + 128 * t;
        const uint32_t tO = tmem_base + lane_off + kTmemO + 128 * t;
        float sl2 = p.scale_log2;
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
            if constexpr (kTurnsQ) {  // this row of Q_t from bf16 to fp16
                const bool got = wait_bounded(bar(T::kBarQFull + t), j & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                uint8_t* row = smem + T::kSmemQ + t * T::kTileBytes + r * 128;
                auto piece = [&](int q) { return reinterpret_cast<uint4*>(row + q / 8 * kHalfBytes + ((q % 8) ^ (r & 7)) * 16); };
                uint4 x[kD / 8];
                uint32_t top2 = 0;
#pragma unroll
                for (int q = 0; q < kD / 8; ++q) {
                    x[q] = *piece(q);
                    top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(x[q].x & 0x7fff7fffu, x[q].y & 0x7fff7fffu),
                                                   __vmaxu2(x[q].z & 0x7fff7fffu, x[q].w & 0x7fff7fffu)));
                }
                float inverse;
                const float factor = row_factor(max(top2 & 0xffffu, top2 >> 16), inverse);
                sl2 = row_scale(p.scale_log2, inverse);
#pragma unroll
                for (int q = 0; q < kD / 8; ++q)
                    *piece(q) = make_uint4(bf16x2_to_f16x2(x[q].x, factor), bf16x2_to_f16x2(x[q].y, factor),
                                           bf16x2_to_f16x2(x[q].z, factor), bf16x2_to_f16x2(x[q].w, factor));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(T::kBarQReady + t));
            }
            float m_run = -INFINITY;  // what the weights are relative to (log2 units of scaled logits)
            float l_run = 0.f;        // running sum of weights

            for (int kt = 0; kt < nt; ++kt, ++sc, nvis -= kBN) {
                const bool got = wait_bounded(bar(T::kBarSFull + t), sc & 1, abort_flag, limit);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t missing[T::kMaskWords];
#pragma unroll
                for (int c = 0; c < T::kMaskWords; ++c) missing[c] = page_mask[(kv + kt) % kMaskRing * T::kMaskWords + c];
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
                if ((missing[0] | missing[1] | missing[2] | missing[3]) != 0) {  // keys without a page
#pragma unroll
                    for (int jj = 0; jj < kBN; ++jj)
                        if ((missing[jj / 32] >> (jj % 32)) & 1) s[jj] = __float_as_uint(-INFINITY);
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

                // the maximum rises only when the tile's is past it
                float alpha = 1.f;
                if (m_tile - m_run > kMaxAbove) {
                    alpha = ex2_approx(m_run - (m_tile - kMaxBelow));
                    m_run = m_tile - kMaxBelow;
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
                            pk[q] = pack_x2<true>(a0, a1);
                            pk[q + 1] = pack_x2<true>(b0, b1);
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
        regs_dec<kTiles4RegsEpilogue>();
        const int wq = warp % 4;
        const int r = wq * 32 + lane;  // row within a tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const int row_token = r / sp.map.heads, row_head = r % sp.map.heads;
        bool ok = true;
        // stores item j's O and LSE, or its piece
        auto finish = [&](int j, const Item& w) {
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
                const float inv_l = ml.y == 0.f ? 0.f : p.v_unit / ml.y;  // a normal number (kTiles4LeastUnit)
                const size_t ws_row = static_cast<size_t>(w.slot >= 0 ? w.slot : 0) * T::kRows + t * kBM + r;
                // A thread stores its row's 32 columns as they come: whole sectors
#pragma unroll
                for (int h = 0; h < kD / 32; ++h) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tmem_ld32(tO + 32 * h, o);
                        tmem_wait_ld_regs(o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (h == kD / 32 - 1) {  // O_t may now be overwritten by the next item's first P.V
                        tc_fence_before();
                        mbar_arrive(bar(T::kBarOFree + t));
                    }
                    if (!there) continue;
                    if (w.slot >= 0) {  // a piece: sums to its workspace slot
                        float4* dst = reinterpret_cast<float4*>(sp.ws.o + ws_row * kD + 32 * h);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                 __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
                        continue;
                    }
                    uint4* dst = reinterpret_cast<uint4*>(p.o + static_cast<size_t>(out_row) * kD + 32 * h);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            fmul2_b(f[e], f[e + 1], __uint_as_float(o[8 * q + e]), __uint_as_float(o[8 * q + e + 1]),
                                    inv_l);
                        dst[q] = make_uint4(pack_x2<kF16>(f[0], f[1]), pack_x2<kF16>(f[2], f[3]),
                                            pack_x2<kF16>(f[4], f[5]), pack_x2<kF16>(f[6], f[7]));
                    }
                }
                if (there) {
                    if (w.slot >= 0)
                        sp.ws.ml[ws_row] = ml;
                    else if (p.lse != nullptr)
                        p.lse[static_cast<size_t>(head) * p.total_q + w.q0 + token] =
                            ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.69314718055994531f;
                }
            }
        };
        // ======================= K and V from their codes ===================
        constexpr int kLanes = kD / 32;          // of a row, with 32 elements each
        constexpr int kAtOnce = 32 / kLanes;     // rows of a warp in one step; a warp has rows 32 wq to 32 wq + 31
        const int chunk = lane % kLanes, first_row = 32 * wq + lane / kLanes;
        // where the rows of a tile lie: this lane's row 32 wq + lane (page < 0: no such key or no page)
        struct Place {
            int page, row;
            uint32_t there, missing;  // rows of this warp that have a page; keys that have none
        };
        // A thread's codes wait in shared memory: registers that loads were in flight for would be
        // spilled around the epilogue.
        const uint32_t k_codes = sbase + T::kSmemCodes + r * 16, k_scales = sbase + T::kSmemCodes + T::kCodeBytes + r * 4;
        constexpr uint32_t kToV = T::kCodeBytes + T::kScaleBytes;
        auto load = [&](const Place& at, const uint8_t* codes, const uint8_t* scales, int hkv, uint32_t off) {
            const long long page = at.page;
            const long long code = page * p.page_stride + at.row * p.token_stride + hkv * p.head_stride;
            const long long scale = page * p.scale_page + at.row * p.scale_token + hkv * p.scale_head;
            long long c[kLanes], b[kLanes];
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                c[i] = __shfl_sync(0xffffffffu, code, i * kAtOnce + lane / kLanes);
                b[i] = __shfl_sync(0xffffffffu, scale, i * kAtOnce + lane / kLanes);
            }
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const bool there = (at.there >> (i * kAtOnce + lane / kLanes)) & 1;
                cp_async_row16<kD / 2>(k_codes + off + i * (kBM * 16), codes + c[i] + chunk * 16, there);
                cp_async_small<4>(k_scales + off + i * (kBM * 4), scales + b[i] + chunk / 2 * 4, there);
            }
        };
        // As TMA lays out a swizzled tile of 64-column halves.  The halves of a row fall into the same
        // banks, so lanes of the second one store their pieces in another order.
        const uint32_t later = kD == 128 ? chunk / 2 * 2 : 0;  // 0 or 2
        auto store = [&](uint32_t tile, uint32_t off) {
            uint32_t w[kLanes][4], two[kLanes];
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                lds_x2(w[i], k_codes + off + i * (kBM * 16) + later * 4);
                lds_x2(w[i] + 2, k_codes + off + i * (kBM * 16) + (later ^ 2) * 4);
                two[i] = lds_bytes<2>(k_scales + off + i * (kBM * 4) + chunk % 2 * 2);
            }
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const int row = first_row + i * kAtOnce;
                const uint32_t to = tile + chunk / 2 * kHalfBytes + row * 128;
                const uint32_t s2 = e4m3_to_f16(two[i]);
                const uint32_t by[2] = {later ? high_twice(s2) : low_twice(s2), later ? low_twice(s2) : high_twice(s2)};
                uint32_t h[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    e2m1_to_f16(h[q], w[i][q]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[q][e] = hmul2(h[q][e], by[q / 2]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     to + (((chunk % 2 * 4 + (q ^ later)) ^ (row & 7)) << 4)),
                                 "r"(h[q][0]), "r"(h[q][1]), "r"(h[q][2]), "r"(h[q][3])
                                 : "memory");
            }
        };
        // The tile whose K is next: `ahead` is one further, for its page numbers to arrive in time.
        struct Tile {
            int j, kt, n;      // item, key tile of n
            int seq, kb, kv_len, hkv;
            bool ok;
        };
        auto enter = [&](Tile& x, int j) {
            Item w;
            x.ok = look_at_item(j, w, ok);
            x.j = j;
            if (!x.ok) return;
            x.kt = 0;
            x.n = w.nmax();
            x.seq = w.seq;
            x.kb = w.kb;
            x.kv_len = w.kv_len;
            x.hkv = sp.map.kv_head(w.head_unit);
        };
        auto step_on = [&](Tile& x) {
            if (++x.kt == x.n) enter(x, x.j + 1);
        };
        auto look_up = [&](const Tile& x, Place& at) {
            at.page = at.row = 0;
            if (!x.ok) return;
            const int key = (x.kb + x.kt) * kBN + 32 * wq + lane;
            at.page = -1;
            if (key < x.kv_len) {
                const int col = static_cast<int>(p.by_page.quot(key));
                at.page = p.table[x.seq * p.table_stride + col];
                at.row = key - col * p.page_size;
            }
            // judged when the number is there (settle)
        };
        auto settle = [&](const Tile& x, Place& at) {
            const bool in_range = (x.kb + x.kt) * kBN + 32 * wq + lane < x.kv_len;
            const bool there = in_range && at.page >= 0 && at.page < p.n_pages;
            if (!there) at.page = at.row = 0;
            at.there = __ballot_sync(0xffffffffu, there);
            at.missing = __ballot_sync(0xffffffffu, in_range && !there);
        };
        Tile cur, ahead;
        Place here, next;
        enter(cur, 0);
        if (cur.ok) {
            look_up(cur, here);
            ahead = cur;
            step_on(ahead);
            look_up(ahead, next);
            settle(cur, here);
            load(here, p.k_codes, p.k_scales, cur.hkv, 0);
        }
        cp_async_commit();
        bool have_v = false;
        int ends = -1, pending = -1;  // items whose last V is next, or is in the stage before
        for (int g = 0; ok && (cur.ok || have_v); ++g) {
            const int st = g % kStages, use = g / kStages;
            const bool got = use == 0 || wait_bounded(bar(T::kBarKvEmpty + st), (use - 1) & 1, abort_flag, limit);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            cp_async_wait<0>();
            const bool had_v = have_v;
            const int ended = ends;
            if (cur.ok) {
                store(sbase + T::kSmemK + st * T::kTileBytes, 0);
                if (lane == 0) page_mask[g % kMaskRing * T::kMaskWords + wq] = here.missing;
            }
            if (had_v) store(sbase + T::kSmemV + ((g - 1) % kStages) * T::kTileBytes, kToV);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(T::kBarKvFull + st));
            // the codes of this tile's V and of the next one's K, and the page numbers of the one behind
            have_v = cur.ok;
            ends = cur.ok && cur.kt + 1 == cur.n ? cur.j : -1;
            if (cur.ok) {
                load(here, p.v_codes, p.v_scales, cur.hkv, kToV);
                cur = ahead;
                here = next;
                if (cur.ok) {
                    settle(cur, here);
                    load(here, p.k_codes, p.k_scales, cur.hkv, 0);
                    step_on(ahead);
                    look_up(ahead, next);
                }
            }
            cp_async_commit();
            if (pending >= 0) {
                Item w;
                if (!look_at_item(pending, w, ok)) break;
                finish(pending, w);
                if (!ok) break;
                release_item(pending);
            }
            pending = had_v ? ended : -1;
        }
        if (ok && pending >= 0) {
            Item w;
            if (look_at_item(pending, w, ok)) finish(pending, w);
        }
        cp_async_wait<0>();
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

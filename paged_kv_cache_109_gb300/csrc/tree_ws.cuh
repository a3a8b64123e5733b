// tree_ws.cuh -- attention of a tree of drafted tokens over the paged cache on
// the 5th-generation tensor cores (tcgen05, tensor-memory accumulators), bf16.
//
//   out[r] = sum_t softmax_t(scale q_r.k_t) v_t over the cached tokens, the
//   node's ancestors and itself.
//
// What bounds it: K and V are read once per unit and serve all its rows, 6 D
// operations per row and key (P in two parts) against 4 D bytes per key, so with
// one tile in use the cache's bytes decide and with two the products: measured
// on one GB300 (D = 128, 38 sequences x 8 kv heads x 64 key blocks) 203 us = 6270
// GB/s of K and V, 93% of the copy rate, with 64 rows, and 312 us = 4090 GB/s with
// 256 rows, where the GPU then runs into its power limit (1.7 of 2.07 GHz).  P as
// one bf16 part would take 237 us there, at up to 1.4 times the error (against
// 64 bits, normal data, 200 to 16000 keys: 0.0022 to 0.0023 for 0.0017): the second part
// stays, so that a verified row is as near to the decode's as the formula allows.
//
// The kernel is one persistent CTA per SM that keeps a ring of K/V blocks full
// through the whole of its range (tree_sched.cuh), across the ends of units.
//
// A unit has two tiles of 128 rows = (node, query head of the group) pairs,
// head fastest; keys come in blocks of 128.
//   two tiles in use   both take every key block (K and V cross shared memory
//                      once per 256 rows);
//   one tile in use    the two accumulators take the key blocks in turn, block
//                      x goes to accumulator x mod 2, so that one block's
//                      softmax runs beside the other's products; they are
//                      joined by their (m, l) at the end.
//
//   warps 0-3, 4-7  softmax of accumulator 0, 1: thread t owns tensor-memory
//                   lane t (one row); output or workspace cells at the end
//   warps 8, 10     producers of K and of V: block-table lookups, TMA copies.
//                   The K warp walks the range, hands its parts to the other
//                   warps through a short queue and loads Q (TMA), the V warp
//                   the nodes' parents.  The V warp checks the blocks that not
//                   every row may see (tree nodes, rows behind the last key)
//                   before their use: rows behind are cleared, and values that
//                   are not finite are taken out (0 times NaN would reach rows
//                   that do not see the node) and noted; the rows that do see
//                   such a node add its values at the end
//   warp 9          MMA issue: S = Q K^T, O += P V (P from tensor memory as
//                   two bf16 parts, hi + lo: about 16 significant bits of each
//                   weight, as in the prefill kernel)
//
// A copy of K or V covers up to a whole cache block and both 64-column halves:
// the tensor map's dimensions are (64 columns, 8 rows, halves, groups of 8
// rows, block x head), so that shared memory holds [8-row group][half][8 rows].
// (A box per 16 rows and half, twice the instructions at 16-token blocks, took
// one warp 4000 cycles of issue per 128 keys, longer than the 2800 that
// 64 KB take at the copy rate.)
// Head dims between 64 and 128 take a copy per half, [half][8-row group], since
// a row's second half would reach past its end.
//
// Only blocks that reach past the cached tokens are masked.  A row's visible
// keys of such a block are 128 bits: ones up to the cached tokens' end, then
// one bit per ancestor, found by walking up the parents.
//
// Synchronisation is by mbarriers; every wait is bounded, and a timeout raises
// PA_DEVERR_TIMEOUT and ends the role (the others then time out too) without
// leaving copies or MMAs in flight past the CTA's end.
//
// Registers: 168, the most for 352 threads; 8 to 16 bytes a thread spill.
#pragma once

#include <type_traits>

#include "tree_sched.cuh"

namespace pa {

template <int D>
struct TreeWsCfg {
    static constexpr int kThreads = 352;
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kKWarp = 8, kMmaWarp = 9, kVWarp = 10;
    static constexpr int kRows = 128;                     // rows per tile = tensor-memory lanes
    static constexpr int kKeys = 128;
    static constexpr int kHalves = D / 64;                // 64-column (128-byte) slices
    static constexpr int kGroup = kHalves * 1024;         // 8 rows, both halves
    static constexpr int kItem = kKeys / 8 * kGroup;      // K or V of one block
    static constexpr int kQTile = kRows / 8 * kGroup;
    static constexpr int kSlotOff = 2 * kQTile;
    static constexpr int kSmemMax = 232448;               // dynamic shared memory per CTA
    static constexpr int kExtra = 2000;                   // barriers and the small arrays below
    static constexpr int kSlots = (kSmemMax - 1024 - kExtra - kSlotOff) / kItem;
    static constexpr int kBarOff = kSlotOff + kSlots * kItem;
    // K/V full, K/V empty; per accumulator S full, P full, O done; Q full, Q free,
    // O free, (m, l) ready, V to check, V checked, final; queue full, empty
    static constexpr int kQueue = 4;                      // parts announced at once
    static constexpr int kBars = 2 * kSlots + 13 + 2 * kQueue;
    // parents (as parent + 1, a byte each) and flags of V rows with values taken
    // out, of the last four parts (a part's output is read while the part
    // behind it is under way)
    static constexpr int kBufs = 4;
    static constexpr int kParentOff = kBarOff + 8 * kBars;
    static constexpr int kFlagOff = kParentOff + kBufs * PA_MAX_TREE_NODES;
    static constexpr int kQueueOff = kFlagOff + kBufs * (PA_MAX_TREE_NODES / 8);
    static constexpr int kTslotOff = kQueueOff + kQueue * (int)sizeof(TreeSeg);
    static_assert(kTslotOff + 16 - kBarOff <= kExtra, "small arrays");
    static size_t smem_bytes() { return 1024 + kTslotOff + 16; }
    static constexpr uint32_t kTmemCols = 512;            // per accumulator: S (and P) at +0, O at +128
    static constexpr uint32_t kTileCols = 256;
    static constexpr uint32_t kOCol = 128;
    static_assert(D == 64 || D == 128, "tile width");
    // each producer waits for the item a turn before its own, and its previous
    // item is at most four back: so no slot can be a turn further behind
    static_assert(kSlots >= 5, "ring");
    static_assert(sizeof(TreeSeg) % 16 == 0, "queue entries");
};

// 5-D tiled bulk tensor load global -> shared, completion counted on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// A shared-memory matrix descriptor from its low word (start address, LBO) and
// its high word (SBO, version, swizzle).
__device__ __forceinline__ uint64_t umma_desc(uint32_t lo, uint32_t hi) {
    return (uint64_t)hi << 32 | lo;
}

// split_bf16x2 with one packed subtraction.
__device__ __forceinline__ void split_bf16x2_packed(float2 x, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(x.x, x.y);
    const float2 h = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    const float2 d = __ffma2_rn(h, make_float2(-1.f, -1.f), x);
    lo = pack_bf16x2(d.x, d.y);
}

// Any of the two bf16 values not finite (exponent all ones).
__device__ __forceinline__ bool bf16x2_odd(uint32_t x) {
    return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t bf16x2_clean(uint32_t x) {
    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
    return x;
}

// SPLIT: head dims between 64 and 128 (D = 128), copied half by half.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(TreeWsCfg<D>::kThreads, 1)
tree_ws_kernel(const __grid_constant__ CUtensorMap tmap_q,
               const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, const TreeArgs a, const TreeWork w,
               const int32_t box_rows) {
    // box_rows: rows of a copy, a multiple of 8 that divides the block size
    using C = TreeWsCfg<D>;
    extern __shared__ uint8_t sm_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sm_u = smem_u32(sm);
    const uint32_t bar0 = sm_u + C::kBarOff;
    auto kv_full = [&](int32_t s) { return bar0 + 8u * s; };
    auto kv_empty = [&](int32_t s) { return bar0 + 8u * (C::kSlots + s); };
    const uint32_t bar1 = bar0 + 8u * (2 * C::kSlots);
    auto s_full = [&](int32_t t) { return bar1 + 8u * t; };
    auto p_full = [&](int32_t t) { return bar1 + 8u * (2 + t); };
    auto o_done = [&](int32_t t) { return bar1 + 8u * (4 + t); };
    const uint32_t q_full = bar1 + 8u * 6, q_free = bar1 + 8u * 7, o_free = bar1 + 8u * 8;
    const uint32_t ml_ready = bar1 + 8u * 9, v_go = bar1 + 8u * 10, v_ok = bar1 + 8u * 11;
    const uint32_t bar_fin = bar1 + 8u * 12;
    auto seg_full = [&](int32_t s) { return bar1 + 8u * (13 + s); };
    auto seg_empty = [&](int32_t s) { return bar1 + 8u * (13 + C::kQueue + s); };
    uint8_t* parents = sm + C::kParentOff;
    uint32_t* flags = reinterpret_cast<uint32_t*>(sm + C::kFlagOff);
    TreeSeg* queue = reinterpret_cast<TreeSeg*>(sm + C::kQueueOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::kTslotOff);

    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int32_t s = 0; s < C::kSlots; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int32_t t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), 4);                      // one arrival per softmax warp
            mbar_init(o_done(t), 1);
        }
        mbar_init(q_full, 2);                             // the copies', the parents'
        mbar_init(q_free, 1);
        mbar_init(o_free, C::kSoftmaxWarps);
        mbar_init(ml_ready, C::kSoftmaxWarps);
        mbar_init(v_go, 1);
        mbar_init(v_ok, 1);
        mbar_init(bar_fin, 1);
        for (int32_t s = 0; s < C::kQueue; ++s) {
            mbar_init(seg_full(s), 1);
            mbar_init(seg_empty(s), C::kSoftmaxWarps + 2);
        }
        mbar_fence_init();
    }
    if (warp == C::kKWarp && lane == 0) prefetch_tmap(&tmap_k);
    if (warp == C::kVWarp && lane == 0) prefetch_tmap(&tmap_v);
    if (warp == C::kMmaWarp && lane == 0) prefetch_tmap(&tmap_q);
    if (warp == C::kMmaWarp) tmem_alloc(smem_u32(tslot), C::kTmemCols);
    griddep_wait();
    // the range: by the K warp alone where it can (the ring is not in use yet:
    // its start serves the search of larger batches)
    TreeIter it{};
    if (a.num_seqs > kTreeWarpSeqs) {
        it = tree_begin(a, w, reinterpret_cast<int64_t*>(sm + C::kSlotOff));
        fence_proxy_async_smem();
    } else if (warp == C::kKWarp) {
        it = tree_begin_warp(a, w);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    const int32_t G = a.group, BS = a.block_size, hd = a.head_dim;
    const int32_t HT = w.s.heads, tpt = w.s.tokens;
    // bytes from one 8-row group of K or V to the next, and between halves
    constexpr int32_t gs = SPLIT ? 1024 : C::kGroup, ho = SPLIT ? C::kKeys * 128 : 1024;
    // a bounded wait whose outcome is the same in every lane of the warp
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimitCycles)) != 0;
    };
    // Ring items of a part of n blocks in the order they are consumed: step x
    // takes K(x), then V(x - lag); lag is 1 with two tiles in use, 2 with one.
    auto k_item = [](int32_t x, int32_t lag) { return x + max(0, x - lag); };
    auto v_item = [](int32_t y, int32_t lag, int32_t n) { return y + min(y + lag + 1, n); };

    TreeSeg sg;
    bool ok = true;
    int32_t seg = 0;                                      // parts so far
    int32_t item0 = 0;                                    // ring items of earlier parts
    // The next part from the queue (its entry is free again at once: the copy
    // is in registers); false at the end of the range, or with ok false.
    auto next_part = [&]() {
        const int32_t s = seg % C::kQueue;
        ok = warp_wait(seg_full(s), (seg / C::kQueue) & 1);
        if (!ok) return false;
        sg = queue[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(s));
        return sg.n > 0;
    };

    if (warp == C::kKWarp || warp == C::kVWarp) {
        // ---- producers -----------------------------------------------------
        // Lane j copies the j-th box (box_rows keys, all columns) of a block.
        const bool is_v = warp == C::kVWarp;
        const void* map = is_v ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k);
        const int32_t nbox = C::kKeys / box_rows;
        const uint32_t box_step = (uint32_t)(box_rows / 8) * gs;      // in shared memory
        const uint32_t box_bytes = (uint32_t)(box_rows / 8) * C::kGroup;
        const int32_t dcol = C::kKeys / BS, drow = C::kKeys - dcol * BS;
        int32_t mine = -1;                                // lane s: this warp's latest item in slot s
        int32_t checked = 0;                              // V blocks checked so far
        TreeCut cut{};
        bool was_one = false;                             // the part before used one tile
        int32_t q_parts = 0;                              // parts whose Q is asked for
        // K's warp finds the parts and announces them (n = 0: there are no more)
        auto announce = [&]() {
            if (!tree_next(a, w.s, it, sg)) sg.n = 0;
            const int32_t s = seg % C::kQueue;
            if (seg >= C::kQueue) ok = warp_wait(seg_empty(s), ((seg / C::kQueue) - 1) & 1);
            if (!ok) return false;
            if (lane == 0) queue[s] = sg;
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_full(s));
            if (sg.n > 0 && sg.kb0 == 0 && sg.parts > 0)
                cut = TreeCut{sg.q0 + sg.tok0, sg.ntok, sg.g, sg.sg, sg.parts, {0, 0, 0}};
            return sg.n > 0;
        };
        // Q: a copy per tile and half of `tokens` x `heads` rows in place (rows
        // behind the part's last node or head hold whatever comes there: a
        // row's scores reach no other row).
        auto load_q = [&]() {
            const int32_t tiles = sg.ntok > tpt ? 2 : 1;
            if (seg > 0) ok = warp_wait(q_free, (seg - 1) & 1);
            // tile 1's rows hold the (m, l) of a part with one tile until its
            // output has been written
            if (ok && tiles == 2 && was_one) ok = warp_wait(o_free, (seg - 1) & 1);
            if (!ok) return;
            was_one = tiles == 1;
            ++q_parts;
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)(tpt * HT) * 128u * C::kHalves * tiles);
                for (int32_t t = 0; t < tiles; ++t)
                    for (int32_t h = 0; h < C::kHalves; ++h)
                        tma_load_3d(sm_u + t * C::kQTile + h * (C::kRows * 128), &tmap_q, h * 64,
                                    sg.g * G + sg.sg * HT, sg.q0 + sg.tok0 + t * tpt, q_full);
            }
        };
        while (ok && (is_v ? next_part() : announce())) {
            const int32_t n = sg.kb1 - sg.kb0, lag = sg.ntok > tpt ? 1 : 2;
            uint32_t* noted = flags + (seg % C::kBufs) * (PA_MAX_TREE_NODES / 32);
            if (is_v) {
                // the nodes' parents (the K warp is at most one part further, after
                // the output of the part three before this one)
                if (lane < PA_MAX_TREE_NODES / 32) noted[lane] = 0;
                for (int32_t j = lane; j < sg.n; j += 32) {
                    const int32_t p = tree_parent(a.parents[sg.q0 + j], j, true);
                    parents[(seg % C::kBufs) * PA_MAX_TREE_NODES + j] = (uint8_t)(p + 1);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            } else if (seg == 0) {
                load_q();
            }
            // V's block y, if it reaches past the cached tokens: rows of tree
            // nodes, and rows behind the last key up to the end of its 16-key
            // step (the later steps are left out)
            auto check = [&](int32_t y) {
                const int32_t key0 = (sg.kb0 + y) * C::kKeys;
                if (!ok || y < 0 || key0 + C::kKeys <= sg.C) return;
                // (the MMA warp says when the block is there)
                if (!(ok = warp_wait(v_go, checked++ & 1))) return;
                const int32_t vkeys = min(C::kKeys, sg.T - key0);
                const int32_t r0 = max(0, sg.C - key0), r1 = (vkeys + 15) & ~15;
                uint8_t* vt = sm + C::kSlotOff + (item0 + v_item(y, lag, n)) % C::kSlots * C::kItem;
                // 16-byte pieces x of the block's rows in shared memory: row x / 8
                auto piece = [&](int32_t x, int32_t h) {
                    return reinterpret_cast<uint4*>(vt + (x >> 6) * gs + h * ho + (x & 63) * 16);
                };
                for (int32_t x = vkeys * 8 + lane; x < r1 * 8; x += 32)
#pragma unroll
                    for (int32_t h = 0; h < C::kHalves; ++h) *piece(x, h) = make_uint4(0u, 0u, 0u, 0u);
                // 0 x is NaN for a value that is not finite: one product and sum
                // per pair says whether there is any
                __nv_bfloat162 sum = __float2bfloat162_rn(0.f);
#pragma unroll 4
                for (int32_t x = r0 * 8 + lane; x < vkeys * 8; x += 32) {
#pragma unroll
                    for (int32_t h = 0; h < C::kHalves; ++h) {
                        const uint4 v = *piece(x, h);
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int32_t e = 0; e < 4; ++e)
                            sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]),
                                          __float2bfloat162_rn(0.f), sum);
                    }
                }
                const bool odd = __isnan(__low2float(sum)) || __isnan(__high2float(sum));
                if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                    for (int32_t x = r0 * 8 + lane; x < vkeys * 8; x += 32) {
#pragma unroll 1
                        for (int32_t h = 0; h < C::kHalves; ++h) {
                            const uint4 v = *piece(x, h);
                            if (bf16x2_odd(v.x) || bf16x2_odd(v.y) || bf16x2_odd(v.z) || bf16x2_odd(v.w)) {
                                *piece(x, h) = make_uint4(bf16x2_clean(v.x), bf16x2_clean(v.y),
                                                          bf16x2_clean(v.z), bf16x2_clean(v.w));
                                const int32_t node = key0 + (x >> 3) - sg.C;
                                atomicOr(noted + (node >> 5), 1u << (node & 31));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ok);
            };
            const int32_t* table = a.block_tables + (int64_t)sg.i * a.max_blocks;
            // this lane's box of block x: its table entry (read two blocks ahead
            // of use) and its row in the block
            int32_t key = sg.kb0 * C::kKeys + lane * box_rows;   // of the block to look up
            int32_t col = key / BS, row = key - col * BS;        // its table column, first row
            struct Box {
                int32_t id, row;
                bool has;
            };
            auto lookup = [&](int32_t x) {
                Box b{0, row, x < n && lane < nbox && key < sg.T};
                if (b.has) b.id = table[col];
                key += C::kKeys;
                col += dcol;
                row += drow;
                if (row >= BS) {
                    row -= BS;
                    ++col;
                }
                return b;
            };
            Box b0 = lookup(0), b1 = lookup(1);
            for (int32_t x = 0; ok && x < n; ++x) {
                const Box b2 = lookup(x + 2);
                const int32_t item = item0 + (is_v ? v_item(x, lag, n) : k_item(x, lag));
                const int32_t s = item % C::kSlots, turn = item / C::kSlots;
                int32_t z = -1;                            // a bad entry's box reads zeros
                if (b0.has) {
                    if (b0.id < 0 || b0.id >= a.num_blocks)
                        raise_error(PA_DEVERR_TABLE_ENTRY);
                    else
                        z = b0.id * a.num_kv_heads + sg.g;
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, b0.has)) * box_bytes;
                if (turn > 0) ok = warp_wait(kv_empty(s), (turn - 1) & 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(kv_full(s), bytes);
                __syncwarp();
                if (b0.has) {
                    const uint32_t dst = sm_u + C::kSlotOff + s * C::kItem + lane * box_step;
                    tma_load_5d(dst, map, 0, 0, 0, b0.row >> 3, z, kv_full(s));
                    if constexpr (SPLIT)
                        tma_load_5d(dst + ho, map, 64, 0, 0, b0.row >> 3, z, kv_full(s));
                }
                if (lane == s) mine = item;
                b0 = b1;
                b1 = b2;
                // (one block behind the copies: a later copy may wait for a slot
                // that this block's use frees)
                if (is_v)
                    check(x - 1);
                else if (seg > 0 && x == min(n - 1, 1))   // with the part's first keys under way
                    load_q();
            }
            if (is_v) check(n - 1);
            item0 += 2 * n;
            ++seg;
        }
        // every copy has landed before the CTA may end: the MMA warp waits for
        // each, and after a failure this warp does
        if (!is_v && w.cuts != nullptr && lane == 0) w.cuts[blockIdx.x] = cut;
        if (!ok) {
            if (mine >= 0)
                mbar_wait_bounded(kv_full(lane), (mine / C::kSlots) & 1, kWaitLimitCycles);
            if (!is_v && q_parts > 0)
                mbar_wait_bounded(q_full, (q_parts - 1) & 1, kWaitLimitCycles);
            if (lane == 0) raise_error(PA_DEVERR_TIMEOUT);
        }
    } else if (warp == C::kMmaWarp) {
        // ---- MMA issue -----------------------------------------------------
        constexpr uint32_t kIdS = umma_idesc_bf16(128, C::kKeys, 0);
        const uint32_t kIdO = umma_idesc_bf16(128, hd, 1);   // the head dim's columns only
        // Descriptors as two words: a k-step adds its offset / 16 to the low one
        // (addresses stay below 2^18, so the field never carries), the high
        // one is a constant.
        constexpr uint32_t kQHi = (uint32_t)(1024 >> 4) | 1u << 14 | 2u << 29;
        constexpr uint32_t kKvHi = (uint32_t)(gs >> 4) | 1u << 14 | 2u << 29;
        constexpr uint32_t kKLbo = 1u << 16, kVLbo = (uint32_t)(ho >> 4) << 16;   // (K: not used)
        const uint32_t q_lo = sm_u >> 4 | kKLbo;
        const uint32_t slot_lo = (sm_u + C::kSlotOff) >> 4;
        const bool leader = elect_one();
        uint32_t turn[2] = {0, 0};                        // parity of each accumulator's next block
        int32_t checked = 0;                              // V blocks checked so far
        while (ok && next_part()) {
            const int32_t n = sg.kb1 - sg.kb0, lag = sg.ntok > tpt ? 1 : 2;
            ok = warp_wait(q_full, seg & 1);
            for (int32_t x = 0; ok && x < n + lag; ++x) {
                const bool has_k = x < n, has_v = x >= lag;
                const int32_t ki = item0 + k_item(x, lag), vi = item0 + v_item(x - lag, lag, n);
                const int32_t ks = ki % C::kSlots, vs = has_v ? vi % C::kSlots : 0;
                // K: K-major, 128-byte swizzle; V: MN-major, 64-column atoms
                // ho bytes apart (LBO)
                const uint32_t k_lo = (slot_lo + (uint32_t)ks * (C::kItem >> 4)) | kKLbo;
                const uint32_t v_lo = (slot_lo + (uint32_t)vs * (C::kItem >> 4)) | kVLbo;
                int32_t vkeys = C::kKeys;                 // keys of V's block
                if (has_v) {
                    if (!(ok = warp_wait(kv_full(vs), (vi / C::kSlots) & 1))) break;
                    const int32_t key0 = (sg.kb0 + x - lag) * C::kKeys;
                    if (key0 + C::kKeys > sg.C) {
                        vkeys = min(C::kKeys, sg.T - key0);
                        if (lane == 0) mbar_arrive(v_go);
                        if (!(ok = warp_wait(v_ok, checked++ & 1))) break;
                    }
                    // the output of the part before this one has left O
                    if (x == lag && seg > 0 && !(ok = warp_wait(o_free, (seg - 1) & 1))) break;
                }
#pragma unroll
                for (int32_t t = 0; t < 2; ++t) {
                    if (lag == 2 && t != (x & 1)) continue;
                    const uint32_t s_t = tmem + t * C::kTileCols;
                    if (has_v) {
                        const bool fresh = x < (lag == 1 ? 2 : 4);   // O's first block
                        if (!(ok = warp_wait(p_full(t), turn[t]))) break;
                        turn[t] ^= 1u;
                        tc_fence_after();
                        if (leader) {
                            // O += P V: half hf of the keys has hi at columns
                            // 64 hf .. 64 hf + 31 and lo at the next 32, 16 keys =
                            // 8 columns per step (unrolled: descriptors from a
                            // loop's counter took 130 cycles an instruction)
#pragma unroll
                            for (int32_t k = 0; k < 8; ++k)
#pragma unroll
                                for (int32_t lo = 0; lo < 2; ++lo)
                                    if (k * 16 < vkeys)
                                        umma_bf16_ts(s_t + C::kOCol, s_t + (k >> 2) * 64 + lo * 32 + (k & 3) * 8,
                                                     umma_desc(v_lo + k * (gs >> 3), kKvHi), kIdO,
                                                     (!fresh || lo > 0 || k > 0) ? 1u : 0u);
                            umma_commit(o_done(t));
                        }
                        __syncwarp();
                    }
                    if (has_k) {
                        if ((lag == 2 || t == 0) &&
                            !(ok = warp_wait(kv_full(ks), (ki / C::kSlots) & 1)))
                            break;
                        if (leader) {
                            // S(x) = Q K(x)^T over the columns P(x - lag) occupied,
                            // k-steps of the head dim only
                            const uint32_t q_t = q_lo + (lag == 1 ? t * (C::kQTile >> 4) : 0);
#pragma unroll
                            for (int32_t k = 0; k < D / 16; ++k)
                                if (k < hd / 16)
                                    umma_bf16(s_t, umma_desc(q_t + (k >> 2) * (C::kRows * 8) + (k & 3) * 2, kQHi),
                                              umma_desc(k_lo + (k >> 2) * (ho >> 4) + (k & 3) * 2, kKvHi), kIdS,
                                              k > 0 ? 1u : 0u);
                            umma_commit(s_full(t));
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (leader) {
                    if (has_k) umma_commit(kv_empty(ks));
                    if (has_v) umma_commit(kv_empty(vs));
                    // every S of the part is issued, and the output of the part
                    // before it is written (step lag waited for that)
                    if (x == max(n - 1, lag)) umma_commit(q_free);
                }
                __syncwarp();
            }
            item0 += 2 * n;
            ++seg;
        }
        // every MMA issued has finished before tensor memory is released
        if (leader) umma_commit(bar_fin);
        __syncwarp();
        mbar_wait_bounded(bar_fin, 0, kWaitLimitCycles);
        if (!ok && lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    } else {
        // ---- softmax of accumulator wg, lane r -------------------------------
        const int32_t wg = warp >> 2, r = tid & (C::kRows - 1);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + wg * C::kTileCols + lane_base;
        const uint32_t o_tm = s_tm + C::kOCol;
        const float c = a.scale_log2;                     // > 0 on this path
        const int32_t rtok = r / HT, rhead = r - rtok * HT;
        int32_t blocks = 0;                               // blocks of this accumulator so far
        int32_t ones = 0;                                 // parts with one tile so far
        while (ok && next_part()) {
            const int32_t n = sg.kb1 - sg.kb0;
            const bool two = sg.ntok > tpt;
            const int32_t tok = two ? wg * tpt + rtok : rtok;
            const bool row_ok = rtok < tpt && tok < sg.ntok && rhead < min(HT, G - sg.sg * HT);
            const int32_t node = sg.tok0 + tok;
            const uint8_t* up = parents + (seg % C::kBufs) * PA_MAX_TREE_NODES;
            float m_ref = -INFINITY, l = 0.f;
            const int32_t step = two ? 1 : 2;
            const int32_t mine0 = two ? 0 : wg;           // first block of this accumulator
            for (int32_t x = mine0; ok && x < n; x += step) {
                if (!(ok = warp_wait(s_full(wg), blocks & 1))) break;
                tc_fence_after();
                const int32_t key0 = (sg.kb0 + x) * C::kKeys;
                const bool masked = key0 + C::kKeys > sg.C;
                // visible keys of a masked block
                uint64_t vis[2] = {~0ull, ~0ull};
                if (masked) {
                    const int32_t seen = sg.C - key0;      // cached tokens of the block (< 128)
                    vis[0] = seen >= 64 ? ~0ull : seen > 0 ? (1ull << seen) - 1 : 0ull;
                    vis[1] = seen > 64 ? (1ull << (seen - 64)) - 1 : 0ull;
                    if (row_ok) {
                        for (int32_t k = node; k >= 0; k = (int32_t)up[k] - 1) {
                            const int32_t b = seen + k;
                            if (b < 0) break;
                            if (b < 64) vis[0] |= 1ull << b;
                            else if (b < 128) vis[1] |= 1ull << (b - 64);
                        }
                    }
                    __syncwarp();
                }
                const bool first = x == mine0;            // O holds nothing of this part yet
                // 64 keys of S at a time: mask them and take their maximum; move
                // this row's reference m if the block's exceeds it by more than 8
                // (so O is rescaled rarely; p <= 2^8); then again 64 at a time p =
                // 2^(s c - m), as hi + lo over the same columns of S.  (Publishing P
                // by halves, so that its products begin beside the other half's
                // softmax, cost the MMA warp more in waits than it gave: 126 us
                // became 138 on 32 multi-head sequences, and two tiles in use run at
                // the power limit either way.)
                uint32_t sr[2][32];
                float mx = -INFINITY;
                auto load = [&](int32_t hh) {
                    tmem_ld32_async(s_tm + hh * 64, sr[0]);
                    tmem_ld32_async(s_tm + hh * 64 + 32, sr[1]);
                    tmem_wait_ld();
                    tmem_regs_ready(sr[0]);
                    tmem_regs_ready(sr[1]);
                    if (masked) {
                        const uint64_t v = hh ? vis[1] : vis[0];
                        const uint32_t bits[2] = {(uint32_t)v, (uint32_t)(v >> 32)};
#pragma unroll
                        for (int32_t j = 0; j < 64; ++j)
                            if (!(bits[j >> 5] >> (j & 31) & 1u))
                                sr[j >> 5][j & 31] = __float_as_uint(-INFINITY);
                    }
                };
#pragma unroll 1
                for (int32_t hh = 0; hh < 2; ++hh) {
                    load(hh);
                    float mp[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int32_t jj = 0; jj < 32; ++jj)
                        mp[jj & 3] = fmax3(mp[jj & 3], __uint_as_float(sr[(2 * jj) >> 5][(2 * jj) & 31]),
                                           __uint_as_float(sr[(2 * jj + 1) >> 5][(2 * jj + 1) & 31]));
                    mx = fmaxf(fmax3(mp[0], mp[1], mp[2]), mp[3]);
                }
                mx *= c;
                const bool moved = mx > m_ref + 8.f;
                const float al = moved ? ex2_approx(m_ref - mx) : 1.f;   // 0 when m_ref = -inf
                if (moved) m_ref = mx;
                const float ref = m_ref == -INFINITY ? 0.f : m_ref;
                const float2 c2 = make_float2(c, c), nm2 = make_float2(-ref, -ref);
                float2 rs[2] = {make_float2(l * al, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int32_t hh = 1; hh >= 0; --hh) {     // (the second half's are in registers)
                    if (hh == 0) load(0);
                    uint32_t pk[32], plo[32];             // hi and lo parts of P
#pragma unroll
                    for (int32_t jj = 0; jj < 32; ++jj) {
                        const int32_t j = 2 * jj;
                        const float2 xx = __ffma2_rn(make_float2(__uint_as_float(sr[j >> 5][j & 31]),
                                                                 __uint_as_float(sr[(j + 1) >> 5][(j + 1) & 31])),
                                                     c2, nm2);
                        const float2 pp = make_float2(ex2_approx(xx.x), ex2_approx(xx.y));
                        rs[jj & 1] = __fadd2_rn(rs[jj & 1], pp);
                        split_bf16x2_packed(pp, pk[jj], plo[jj]);
                    }
                    tmem_st32_async(s_tm + hh * 64, pk);
                    tmem_st32_async(s_tm + hh * 64 + 32, plo);
                }
                l = (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
                // O holds the P V of the earlier blocks: rescale it once that has
                // finished, before this block is published
                if (!first && __any_sync(0xffffffffu, moved)) {
                    if (!(ok = warp_wait(o_done(wg), (blocks - 1) & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int32_t cc = 0; cc < D / 32; ++cc) {
                        float ov[32];
                        tmem_ld32(o_tm + cc * 32, ov);
#pragma unroll
                        for (int32_t j = 0; j < 32; ++j) ov[j] *= al;
                        tmem_st32(o_tm + cc * 32, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(wg));
                ++blocks;
            }
            if (!ok) break;
            // ---- the part's rows: out, or the workspace cells ----
            const bool any = mine0 < n;                   // this accumulator took a block
            if (any && !(ok = warp_wait(o_done(wg), (blocks - 1) & 1))) break;
            float f[2] = {1.f, 0.f};                      // factors of accumulators 0 and 1
            if (!two) {
                // exchange (m, l); each warpgroup then writes half the columns
                float2* ml = reinterpret_cast<float2*>(sm + C::kQTile) + (ones & 1) * 2 * C::kRows;
                tc_fence_before();
                ml[wg * C::kRows + r] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_ready);
                if (!(ok = warp_wait(ml_ready, ones & 1))) break;
                ++ones;
                tc_fence_after();
                const float2 x0 = ml[r], x1 = ml[C::kRows + r];
                m_ref = fmaxf(x0.x, x1.x);
                const float ref = m_ref == -INFINITY ? 0.f : m_ref;
                f[0] = ex2_approx(x0.x - ref);
                f[1] = ex2_approx(x1.x - ref);
                l = f[0] * x0.y + f[1] * x1.y;
            } else {
                tc_fence_after();
            }
            const bool whole = sg.kb0 == 0 && sg.kb1 == sg.nb;
            if (whole) {
                const float inv = l != 0.f ? 1.f / l : 0.f;   // (NaN: as the formula has it)
                f[0] *= inv;
                f[1] *= inv;
            }
            const uint32_t* noted = flags + (seg % C::kBufs) * (PA_MAX_TREE_NODES / 32);
            uint32_t odd = 0;                             // some V row of the part had values taken out
            if (sg.kb1 * C::kKeys > sg.C) {
#pragma unroll
                for (int32_t x = 0; x < PA_MAX_TREE_NODES / 32; ++x) odd |= noted[x];
            }
            const int32_t urow = two ? wg * C::kRows + r : r;
            float* cell = whole ? nullptr : tree_cell(a, w, sg);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                 ((int64_t)(sg.q0 + node) * a.num_q_heads + (int64_t)sg.g * G +
                                  sg.sg * HT + rhead) * hd;
            // a whole unit's rows are stored 64 bytes at a time by groups of four
            // lanes: after a 4 x 4 transpose lane b of a group has piece b of each
            // of its rows (a row a lane made 32 partial lines a store)
            __nv_bfloat16* dst[4];
#pragma unroll
            for (int32_t k = 0; k < 4; ++k) {
                const int32_t from = (lane & ~3) + k;
                const uint64_t p = reinterpret_cast<uint64_t>(row_ok ? out : nullptr);
                const uint64_t hi = __shfl_sync(0xffffffffu, (uint32_t)(p >> 32), from);
                dst[k] = reinterpret_cast<__nv_bfloat16*>(
                    hi << 32 | __shfl_sync(0xffffffffu, (uint32_t)p, from));
            }
            const int32_t c0 = two ? 0 : wg * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
            const bool both = !two && n > 1;
#pragma unroll 1
            for (int32_t cc = c0; cc < c1; ++cc) {
                __syncwarp();                             // the loads are warp-collective
                float ov[32];
                tmem_ld32((two ? o_tm : tmem + lane_base + C::kOCol) + cc * 32, ov);
#pragma unroll
                for (int32_t j = 0; j < 32; ++j) ov[j] *= f[0];
                if (both) {
                    float o2[32];
                    tmem_ld32(tmem + C::kTileCols + lane_base + C::kOCol + cc * 32, o2);
#pragma unroll
                    for (int32_t j = 0; j < 32; ++j) ov[j] = fmaf(o2[j], f[1], ov[j]);
                }
                if (odd != 0 && row_ok) {
                    for (int32_t k = node; k >= 0; k = (int32_t)up[k] - 1) {
                        if (!(noted[k >> 5] >> (k & 31) & 1u)) continue;
                        const int32_t p = sg.C + k;
                        const int32_t id = a.block_tables[(int64_t)sg.i * a.max_blocks + p / BS];
                        if (id < 0 || id >= a.num_blocks) continue;
                        const __nv_bfloat16* v =
                            static_cast<const __nv_bfloat16*>(a.v_cache) +
                            (((int64_t)id * a.num_kv_heads + sg.g) * BS + p % BS) * hd + cc * 32;
#pragma unroll
                        for (int32_t j = 0; j < 32; ++j) {
                            if (cc * 32 + j < hd) {
                                const float y = __bfloat162float(v[j]);
                                if (!(fabsf(y) <= 3.4028235e38f)) ov[j] += y;
                            }
                        }
                    }
                }
                if (whole) {
                    uint32_t pc[4][4];                    // 16-byte pieces of this lane's row
#pragma unroll
                    for (int32_t q = 0; q < 16; ++q)
                        pc[q >> 2][q & 3] = pack_bf16x2(ov[2 * q], ov[2 * q + 1]);
                    __syncwarp();
#pragma unroll
                    for (int32_t e = 0; e < 4; ++e) {
#pragma unroll
                        for (int32_t s = 1; s < 4; s <<= 1) {
#pragma unroll
                            for (int32_t k = 0; k < 4; ++k) {
                                if (k & s) continue;
                                const bool up1 = lane & s;
                                const uint32_t got = __shfl_xor_sync(
                                    0xffffffffu, up1 ? pc[k][e] : pc[k + s][e], s);
                                if (up1) pc[k][e] = got; else pc[k + s][e] = got;
                            }
                        }
                    }
                    const int32_t col = cc * 32 + (lane & 3) * 8;
#pragma unroll
                    for (int32_t k = 0; k < 4; ++k)
                        if (dst[k] != nullptr && col < hd)
                            *reinterpret_cast<uint4*>(dst[k] + col) =
                                make_uint4(pc[k][0], pc[k][1], pc[k][2], pc[k][3]);
                } else if (row_ok) {
#pragma unroll
                    for (int32_t q4 = 0; q4 < 8; ++q4) {
                        if (cc * 32 + q4 * 4 >= hd) break;   // past the head dim
                        *reinterpret_cast<float4*>(
                            cell + ((size_t)(cc * 8 + q4) * 2 * C::kRows + urow) * 4) =
                            make_float4(ov[q4 * 4], ov[q4 * 4 + 1], ov[q4 * 4 + 2], ov[q4 * 4 + 3]);
                    }
                }
            }
            if (!whole && row_ok && (two || wg == 0))
                *reinterpret_cast<float2*>(cell + (size_t)hd * 2 * C::kRows + 2 * urow) =
                    make_float2(m_ref, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            ++seg;
        }
        if (!ok && lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    }
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace pa

// tree_ws.cuh -- attention of a tree of drafted tokens over the paged cache on
// the 5th-generation tensor cores (tcgen05, tensor-memory accumulators), bf16.
//
//   out[r] = sum_t softmax_t(scale q_r.k_t) v_t over the cached tokens, the
//   node's ancestors and itself.
//
// What bounds it: K and V are read once per unit and serve all its rows, 4 D
// operations per row and key against 4 D bytes per key, so up to about 250
// rows a kv head the cache's bytes decide.  The kernel is therefore one
// persistent CTA per SM that keeps a ring of K/V blocks full through the whole
// of its range (tree_sched.cuh), across the ends of units.
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
//   warp 8          producer: block-table lookups, TMA copies of K and V
//   warp 9          MMA issue: S = Q K^T, O += P V (P from tensor memory as
//                   two bf16 parts, hi + lo: about 16 significant bits of each
//                   weight, as in the prefill kernel)
//   warp 10         Q of the next unit (16-byte cp.async, 128-byte swizzle) and
//                   its nodes' parents
//   warp 11         V rows that not every row may see (tree nodes, rows behind
//                   the last key): rows behind are cleared, and values that
//                   are not finite are taken out (0 times NaN would reach rows
//                   that do not see the node) and noted; the rows that do see
//                   such a node add its values at the end.
//
// Only blocks that reach past the cached tokens are masked.  A row's visible
// keys of such a block are 128 bits: ones up to the cached tokens' end, then
// one bit per ancestor, found by walking up the parents.
//
// Synchronisation is by mbarriers; every wait is bounded, and a timeout raises
// PA_DEVERR_TIMEOUT and ends the role (the others then time out too) without
// leaving copies or MMAs in flight past the CTA's end.
#pragma once

#include <type_traits>

#include "cp_async.cuh"
#include "tree_sched.cuh"

namespace pa {

template <int D>
struct TreeWsCfg {
    static constexpr int kThreads = 384;
    static constexpr int kSoftmaxWarps = 8;
    static constexpr int kProducerWarp = 8, kMmaWarp = 9, kQWarp = 10, kScanWarp = 11;
    static constexpr int kRows = 128;                     // rows per tile = tensor-memory lanes
    static constexpr int kKeys = 128;
    static constexpr int kHalves = D / 64;                // 64-column (128-byte) slices
    static constexpr int kSlice = kKeys * 128;
    static constexpr int kItem = kHalves * kSlice;        // K or V of one block
    static constexpr int kQSlice = kRows * 128;
    static constexpr int kQTile = kHalves * kQSlice;
    static constexpr int kSlotOff = 2 * kQTile;
    static constexpr int kSmemMax = 232448;               // dynamic shared memory per CTA
    static constexpr int kExtra = 2000;                   // barriers and the small arrays below
    static constexpr int kSlots = (kSmemMax - 1024 - kExtra - kSlotOff) / kItem;
    static constexpr int kBarOff = kSlotOff + kSlots * kItem;
    // K/V full, K/V empty; per accumulator S full, P half 0, P full, O half 0,
    // O done; Q full, Q free, O free, (m, l) ready, V to check, V checked, final
    static constexpr int kBars = 2 * kSlots + 17;
    // parents (as parent + 1, a byte each) and flags of V rows with values taken
    // out, of the last four parts (a part's output is read while the part
    // behind it is under way; every part but a CTA's last has blocks to check,
    // so the scan warp is never further ahead)
    static constexpr int kParentBufs = 4, kFlagBufs = 4;
    static constexpr int kParentOff = kBarOff + 8 * kBars;
    static constexpr int kFlagOff = kParentOff + kParentBufs * PA_MAX_TREE_NODES;
    static constexpr int kTslotOff = kFlagOff + kFlagBufs * (PA_MAX_TREE_NODES / 8);
    static_assert(kTslotOff + 16 - kBarOff <= kExtra, "small arrays");
    static size_t smem_bytes() { return 1024 + kTslotOff + 16; }
    static constexpr uint32_t kTmemCols = 512;            // per accumulator: S (and P) at +0, O at +128
    static constexpr uint32_t kTileCols = 256;
    static constexpr uint32_t kOCol = 128;
    static_assert(D == 64 || D == 128, "tile width");
    static_assert(kSlots >= 4, "ring");
};

// Any of the two bf16 values not finite (exponent all ones).
__device__ __forceinline__ bool bf16x2_odd(uint32_t x) {
    return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t bf16x2_clean(uint32_t x) {
    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
    return x;
}

template <int D>
__global__ void __launch_bounds__(TreeWsCfg<D>::kThreads, 1)
tree_ws_kernel(const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, const TreeArgs a, const TreeWork w,
               const int32_t box_rows) {
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
    auto p_half = [&](int32_t t) { return bar1 + 8u * (2 + t); };
    auto p_full = [&](int32_t t) { return bar1 + 8u * (4 + t); };
    auto o_half = [&](int32_t t) { return bar1 + 8u * (6 + t); };
    auto o_done = [&](int32_t t) { return bar1 + 8u * (8 + t); };
    const uint32_t q_full = bar1 + 8u * 10, q_free = bar1 + 8u * 11, o_free = bar1 + 8u * 12;
    const uint32_t ml_ready = bar1 + 8u * 13, v_go = bar1 + 8u * 14, v_ok = bar1 + 8u * 15;
    const uint32_t bar_fin = bar1 + 8u * 16;
    uint8_t* parents = sm + C::kParentOff;
    uint32_t* flags = reinterpret_cast<uint32_t*>(sm + C::kFlagOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::kTslotOff);

    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int32_t s = 0; s < C::kSlots; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int32_t t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_half(t), 4);                      // one arrival per softmax warp
            mbar_init(p_full(t), 4);
            mbar_init(o_half(t), 1);
            mbar_init(o_done(t), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(o_free, C::kSoftmaxWarps);
        mbar_init(ml_ready, C::kSoftmaxWarps);
        mbar_init(v_go, 1);
        mbar_init(v_ok, 1);
        mbar_init(bar_fin, 1);
        mbar_fence_init();
    }
    if (warp == C::kProducerWarp && lane == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    if (warp == C::kMmaWarp) tmem_alloc(smem_u32(tslot), C::kTmemCols);
    griddep_wait();
    // (the ring is not in use yet: its start serves the range's search)
    TreeIter it = tree_begin(a, w, reinterpret_cast<int64_t*>(sm + C::kSlotOff));
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    const int32_t G = a.group, BS = a.block_size, hd = a.head_dim;
    const int32_t HT = w.s.heads, tpt = w.s.tokens;
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
    if (warp == C::kProducerWarp) {
        // ---- producer ------------------------------------------------------
        // Lane j copies the j-th box (box_rows keys) of a block.
        const int32_t nsub = C::kKeys / box_rows;
        const uint32_t box_bytes = (uint32_t)box_rows * 128u;
        int32_t used = 0;
        while (ok && tree_next(a, w.s, it, sg)) {
            const int32_t n = sg.kb1 - sg.kb0, lag = sg.ntok > tpt ? 1 : 2;
            const int32_t* table = a.block_tables + (int64_t)sg.i * a.max_blocks;
            auto lookup = [&](int32_t x) {                 // raw table entry of lane's box
                const int32_t key0 = (sg.kb0 + x) * C::kKeys + lane * box_rows;
                return (x < n && lane < nsub && key0 < sg.T) ? table[key0 / BS] : 0;
            };
            auto issue = [&](int32_t x, int32_t id, bool is_v) {
                const int32_t key0 = (sg.kb0 + x) * C::kKeys + lane * box_rows;
                const bool has = lane < nsub && key0 < sg.T;
                int32_t z = -1;                            // a bad entry's box reads zeros
                if (has) {
                    if (id < 0 || id >= a.num_blocks)
                        raise_error(PA_DEVERR_TABLE_ENTRY);
                    else
                        z = id * a.num_kv_heads + sg.g;
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, has)) * box_bytes * C::kHalves;
                const int32_t s = used % C::kSlots;
                if (used >= C::kSlots && !warp_wait(kv_empty(s), ((used / C::kSlots) - 1) & 1)) {
                    ok = false;
                    return;
                }
                if (lane == 0) mbar_arrive_expect_tx(kv_full(s), bytes);
                __syncwarp();
                if (has) {
                    const uint32_t dst = sm_u + C::kSlotOff + s * C::kItem + lane * box_bytes;
                    const void* map = is_v ? static_cast<const void*>(&tmap_v)
                                           : static_cast<const void*>(&tmap_k);
#pragma unroll
                    for (int32_t h = 0; h < C::kHalves; ++h)
                        tma_load_3d(dst + h * C::kSlice, map, h * 64, key0 % BS, z, kv_full(s));
                }
                ++used;
            };
            // entries of blocks x - 2 .. x + 1: each is read two steps ahead of use
            int32_t e_m2 = 0, e_m1 = 0, e0 = lookup(0), e1 = lookup(1);
            for (int32_t x = 0; ok && x < n + lag; ++x) {
                const int32_t e2 = lookup(x + 2);
                if (x < n) issue(x, e0, false);
                if (ok && x >= lag) issue(x - lag, lag == 1 ? e_m1 : e_m2, true);
                e_m2 = e_m1;
                e_m1 = e0;
                e0 = e1;
                e1 = e2;
            }
        }
        // the last copy into each slot has landed before the CTA may end
        for (int32_t j = max(0, used - C::kSlots); j < used; ++j)
            mbar_wait_bounded(kv_full(j % C::kSlots), (j / C::kSlots) & 1, kWaitLimitCycles);
        if (!ok && lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    } else if (warp == C::kMmaWarp) {
        // ---- MMA issue -----------------------------------------------------
        constexpr uint32_t kIdS = umma_idesc_bf16(128, C::kKeys, 0);
        const uint32_t kIdO = umma_idesc_bf16(128, hd, 1);   // the head dim's columns only
        const uint64_t qdesc0 = umma_sdesc(sm_u, 16, 1024, 2);
        const bool leader = elect_one();
        int32_t done[2] = {0, 0};                         // P V products of earlier blocks
        int32_t checked = 0;                              // masked V blocks so far
        while (ok && tree_next(a, w.s, it, sg)) {
            const int32_t n = sg.kb1 - sg.kb0, lag = sg.ntok > tpt ? 1 : 2;
            ok = warp_wait(q_full, seg & 1);
            for (int32_t x = 0; ok && x < n + lag; ++x) {
                const bool has_k = x < n, has_v = x >= lag;
                const int32_t ki = item0 + k_item(x, lag), vi = item0 + v_item(x - lag, lag, n);
                const int32_t ks = ki % C::kSlots, vs = has_v ? vi % C::kSlots : 0;
                // K: K-major, 128-byte swizzle; V: MN-major, 64-column atoms kSlice
                // bytes apart (LBO)
                const uint64_t kdesc = umma_sdesc(sm_u + C::kSlotOff + ks * C::kItem, 16, 1024, 2);
                const uint64_t vdesc =
                    umma_sdesc(sm_u + C::kSlotOff + vs * C::kItem, C::kSlice, 1024, 2);
                if (has_k) ok = warp_wait(kv_full(ks), (ki / C::kSlots) & 1);
                if (ok && has_v) {
                    ok = warp_wait(kv_full(vs), (vi / C::kSlots) & 1);
                    if (ok && (sg.kb0 + x - lag + 1) * C::kKeys > sg.C) {
                        // (the scan warp does not follow the ring: this warp tells
                        // it that the block is there)
                        if (lane == 0) mbar_arrive(v_go);
                        ok = warp_wait(v_ok, checked++ & 1);
                    }
                    // the output of the part before this one has left O
                    if (ok && x == lag && seg > 0) ok = warp_wait(o_free, (seg - 1) & 1);
                }
                for (int32_t t = lag == 1 ? 0 : x & 1; ok && t < (lag == 1 ? 2 : (x & 1) + 1); ++t) {
                    const uint32_t s_t = tmem + t * C::kTileCols;
                    if (has_v) {
                        const bool fresh = x < (lag == 1 ? 2 : 4);   // O's first block
#pragma unroll
                        for (int32_t hf = 0; hf < 2; ++hf) {
                            if (!warp_wait(hf ? p_full(t) : p_half(t), done[t] & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (leader) {
                                // half hf: hi at columns 64 hf .. 64 hf + 31,
                                // lo at the next 32; 16 keys = 8 columns per step
#pragma unroll
                                for (int32_t k = 0; k < 4; ++k)
                                    umma_bf16_ts(s_t + C::kOCol, s_t + hf * 64 + k * 8,
                                                 vdesc + (uint64_t)((hf * 4 + k) * 128), kIdO,
                                                 (!fresh || hf > 0 || k > 0) ? 1u : 0u);
#pragma unroll
                                for (int32_t k = 0; k < 4; ++k)
                                    umma_bf16_ts(s_t + C::kOCol, s_t + hf * 64 + 32 + k * 8,
                                                 vdesc + (uint64_t)((hf * 4 + k) * 128), kIdO, 1u);
                                umma_commit(hf ? o_done(t) : o_half(t));
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        if (t == 0) ++done[0]; else ++done[1];
                    }
                    if (has_k && leader) {
                        // S(x) = Q K(x)^T over the columns P(x - lag) occupied,
                        // k-steps of the head dim only
                        const uint64_t qdesc = qdesc0 + (uint64_t)(lag == 1 ? t * (C::kQTile >> 4) : 0);
#pragma unroll
                        for (int32_t k = 0; k < D / 16; ++k) {
                            if (k < hd / 16)
                                umma_bf16(s_t,
                                          qdesc + (uint64_t)((k >> 2) * (C::kQSlice >> 4) + (k & 3) * 2),
                                          kdesc + (uint64_t)((k >> 2) * (C::kSlice >> 4) + (k & 3) * 2),
                                          kIdS, k > 0 ? 1u : 0u);
                        }
                        umma_commit(s_full(t));
                    }
                    __syncwarp();
                }
                if (ok && leader) {
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
    } else if (warp == C::kQWarp) {
        // ---- Q and parents -------------------------------------------------
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
        bool was_one = false;                             // the part before used one tile
        while (ok && tree_next(a, w.s, it, sg)) {
            const int32_t tiles = sg.ntok > tpt ? 2 : 1;
            if (seg > 0) ok = warp_wait(q_free, (seg - 1) & 1);
            // tile 1's rows hold the (m, l) of a part with one tile until its
            // output has been written
            if (ok && tiles == 2 && was_one) ok = warp_wait(o_free, (seg - 1) & 1);
            if (!ok) break;
            const int32_t pieces = hd / 8;
            const int32_t heads = min(HT, G - sg.sg * HT);
            // consecutive lanes copy consecutive 16-byte pieces of a row
            constexpr int32_t kPer = D / 8;
            const int32_t c = lane % kPer;
#pragma unroll 4
            for (int32_t r = lane / kPer; r < tiles * C::kRows; r += 32 / kPer) {
                const int32_t t = r >> 7, rr = r & 127;
                const int32_t tk = rr / HT, head = rr - tk * HT, tok = t * tpt + tk;
                // zeros past the head dim and in idle rows
                const bool live = tk < tpt && tok < sg.ntok && head < heads && c < pieces;
                const int64_t row = live ? (int64_t)(sg.q0 + sg.tok0 + tok) * a.num_q_heads +
                                               (int64_t)sg.g * G + sg.sg * HT + head
                                         : 0;
                cp_async16(sm_u + t * C::kQTile + rr * 128 + (c >> 3) * C::kQSlice +
                               (((c & 7) ^ (rr & 7)) << 4),
                           q + row * hd + (live ? c * 8 : 0), live ? 16u : 0u);
            }
            for (int32_t j = lane; j < sg.n; j += 32) {
                const int32_t p = tree_parent(a.parents[sg.q0 + j], j, true);
                parents[(seg % C::kParentBufs) * PA_MAX_TREE_NODES + j] = (uint8_t)(p + 1);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            was_one = tiles == 1;
            ++seg;
        }
        if (!ok && lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    } else if (warp == C::kScanWarp) {
        // ---- V rows that not every row sees ----------------------------------
        int32_t checked = 0;
        while (ok && tree_next(a, w.s, it, sg)) {
            const int32_t n = sg.kb1 - sg.kb0, lag = sg.ntok > tpt ? 1 : 2;
            uint32_t* noted = flags + (seg % C::kFlagBufs) * (PA_MAX_TREE_NODES / 32);
            if (lane < PA_MAX_TREE_NODES / 32) noted[lane] = 0;
            __syncwarp();
            for (int32_t y = max(0, sg.C / C::kKeys - sg.kb0); ok && y < n; ++y) {
                const int32_t vi = item0 + v_item(y, lag, n), vs = vi % C::kSlots;
                ok = warp_wait(v_go, checked++ & 1);
                if (!ok) break;
                uint8_t* vt = sm + C::kSlotOff + vs * C::kItem;
                const int32_t key0 = (sg.kb0 + y) * C::kKeys;
                const int32_t nodes0 = max(0, sg.C - key0);           // first row of a node
                const int32_t valid = min(C::kKeys, sg.T - key0);     // rows of keys
                // a row of a slice is 8 pieces of 16 bytes (any order: swizzled)
                for (int32_t x = nodes0 * 8 + lane; x < C::kKeys * 8; x += 32) {
                    const int32_t row = x >> 3;
#pragma unroll
                    for (int32_t h = 0; h < C::kHalves; ++h) {
                        uint4* p = reinterpret_cast<uint4*>(vt + h * C::kSlice + x * 16);
                        if (row >= valid) {
                            *p = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            uint4 v = *p;
                            if (bf16x2_odd(v.x) || bf16x2_odd(v.y) || bf16x2_odd(v.z) || bf16x2_odd(v.w)) {
                                *p = make_uint4(bf16x2_clean(v.x), bf16x2_clean(v.y),
                                                bf16x2_clean(v.z), bf16x2_clean(v.w));
                                const int32_t node = key0 + row - sg.C;
                                atomicOr(noted + (node >> 5), 1u << (node & 31));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_ok);
            }
            item0 += 2 * n;
            ++seg;
        }
        if (!ok && lane == 0) raise_error(PA_DEVERR_TIMEOUT);
    } else {
        // ---- softmax of accumulator wg, lane r -------------------------------
        const int32_t wg = warp >> 2, r = tid & (C::kRows - 1);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + wg * C::kTileCols + lane_base;
        const uint32_t o_tm = s_tm + C::kOCol;
        const float c = a.scale_log2;                     // >= 0 on this path
        const int32_t rtok = r / HT, rhead = r - rtok * HT;
        int32_t blocks = 0;                               // blocks of this accumulator so far
        int32_t ones = 0;                                 // parts with one tile so far
        while (ok && tree_next(a, w.s, it, sg)) {
            const int32_t n = sg.kb1 - sg.kb0;
            const bool two = sg.ntok > tpt;
            const int32_t tok = two ? wg * tpt + rtok : rtok;
            const bool row_ok = rtok < tpt && tok < sg.ntok && rhead < min(HT, G - sg.sg * HT);
            const int32_t node = sg.tok0 + tok;
            const uint8_t* up = parents + (seg % C::kParentBufs) * PA_MAX_TREE_NODES;
            float m_ref = -INFINITY, l = 0.f;
            const int32_t step = two ? 1 : 2;
            const int32_t mine0 = two ? 0 : wg;           // first block of this accumulator
            for (int32_t x = mine0; x < n; x += step) {
                if (!warp_wait(s_full(wg), blocks & 1)) {
                    ok = false;
                    break;
                }
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
                }
                const float2 c2 = make_float2(c, c);
                const bool first = x == mine0;            // O holds nothing of this part yet
                auto block = [&](auto is_masked) -> bool {
                    constexpr bool kMasked = decltype(is_masked)::value;
                    uint32_t sr[2][32];
                    tmem_ld32_async(s_tm, sr[0]);
                    tmem_ld32_async(s_tm + 32, sr[1]);
                    tmem_wait_ld();
                    tmem_regs_ready(sr[0]);
                    tmem_regs_ready(sr[1]);
#pragma unroll
                    for (int32_t hh = 0; hh < 2; ++hh) {
                        const uint32_t bits[2] = {(uint32_t)vis[hh], (uint32_t)(vis[hh] >> 32)};
                        if constexpr (kMasked) {
#pragma unroll
                            for (int32_t j = 0; j < 64; ++j)
                                if (!(bits[j >> 5] >> (j & 31) & 1u))
                                    sr[j >> 5][j & 31] = __float_as_uint(-INFINITY);
                        }
                        float mp[4];
#pragma unroll
                        for (int32_t u = 0; u < 4; ++u) mp[u] = -INFINITY;
#pragma unroll
                        for (int32_t jj = 0; jj < 32; ++jj)
                            mp[jj & 3] = fmax3(mp[jj & 3], __uint_as_float(sr[(2 * jj) >> 5][(2 * jj) & 31]),
                                               __uint_as_float(sr[(2 * jj + 1) >> 5][(2 * jj + 1) & 31]));
                        const float mraw = fmaxf(fmax3(mp[0], mp[1], mp[2]), mp[3]);
                        const float mx = mraw == -INFINITY ? -INFINITY : mraw * c;
                        // the reference moves only when the maximum exceeds it by
                        // more than 8, so O is rescaled rarely; p <= 2^8
                        const bool moved = mx > m_ref + 8.f;
                        const float al = moved ? ex2_approx(m_ref - mx) : 1.f;   // 0 when m_ref = -inf
                        if (moved) m_ref = mx;
                        l *= al;
                        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
                        const float2 nm2 = make_float2(-ref, -ref);
                        float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        uint32_t pk[32], plo[32];             // hi and lo parts of P
#pragma unroll
                        for (int32_t jj = 0; jj < 32; ++jj) {
                            const int32_t j = 2 * jj;
                            const float2 xx = __ffma2_rn(make_float2(__uint_as_float(sr[j >> 5][j & 31]),
                                                                     __uint_as_float(sr[(j + 1) >> 5][(j + 1) & 31])),
                                                         c2, nm2);
                            float2 pp = make_float2(ex2_approx(xx.x), ex2_approx(xx.y));
                            if constexpr (kMasked) {         // c = 0: -inf * 0 is NaN
                                pp.x = (bits[j >> 5] >> (j & 31) & 1u) ? pp.x : 0.f;
                                pp.y = (bits[j >> 5] >> ((j + 1) & 31) & 1u) ? pp.y : 0.f;
                            }
                            rs[jj & 1] = __fadd2_rn(rs[jj & 1], pp);
                            split_bf16x2(pp.x, pp.y, pk[jj], plo[jj]);
                        }
                        // this half's 64 columns of S are in registers: hi and lo
                        // take them
                        tmem_st32_async(s_tm + hh * 64, pk);
                        tmem_st32_async(s_tm + hh * 64 + 32, plo);
                        l += (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
                        // the second half's scores load while this half is published
                        if (hh == 0) {
                            tmem_ld32_async(s_tm + 64, sr[0]);
                            tmem_ld32_async(s_tm + 96, sr[1]);
                        }
                        // O holds the P V of every earlier half: rescale it once
                        // that has finished, before this half is published
                        if ((!first || hh > 0) && __any_sync(0xffffffffu, moved)) {
                            const bool waited = hh == 0 ? warp_wait(o_done(wg), (blocks - 1) & 1)
                                                        : warp_wait(o_half(wg), blocks & 1);
                            if (!waited) return false;
                            tc_fence_after();
#pragma unroll
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
                        if (lane == 0) mbar_arrive(hh == 0 ? p_half(wg) : p_full(wg));
                        if (hh == 0) {
                            tmem_wait_ld();
                            tmem_regs_ready(sr[0]);
                            tmem_regs_ready(sr[1]);
                        }
                    }
                    return true;
                };
                ok = masked ? block(std::true_type{}) : block(std::false_type{});
                if (!ok) break;
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
            const uint32_t* noted = flags + (seg % C::kFlagBufs) * (PA_MAX_TREE_NODES / 32);
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
            const int32_t c0 = two ? 0 : wg * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
            const bool both = !two && n > 1;
#pragma unroll
            for (int32_t cc = 0; cc < D / 32; ++cc) {
                if (cc < c0 || cc >= c1) continue;
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
                if (!row_ok) continue;
                if (whole) {
#pragma unroll
                    for (int32_t q4 = 0; q4 < 4; ++q4) {
                        if (cc * 32 + q4 * 8 >= hd) break;   // past the head dim
                        uint4 v;
                        v.x = pack_bf16x2(ov[q4 * 8 + 0], ov[q4 * 8 + 1]);
                        v.y = pack_bf16x2(ov[q4 * 8 + 2], ov[q4 * 8 + 3]);
                        v.z = pack_bf16x2(ov[q4 * 8 + 4], ov[q4 * 8 + 5]);
                        v.w = pack_bf16x2(ov[q4 * 8 + 6], ov[q4 * 8 + 7]);
                        *reinterpret_cast<uint4*>(out + cc * 32 + q4 * 8) = v;
                    }
                } else {
#pragma unroll
                    for (int32_t q4 = 0; q4 < 8; ++q4) {
                        if (cc * 32 + q4 * 4 >= hd) break;
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

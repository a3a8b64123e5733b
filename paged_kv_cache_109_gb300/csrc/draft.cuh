// draft.cuh -- host side of the drafted (speculative) step's calls:
// pa_plan_step, pa_decode_tree, pa_accept_tree.  Included by pa.cu, whose
// argument helpers and launch it uses.
#pragma once

#include "accept_tree.cuh"
#include "plan_step.cuh"
#include "tree_args.cuh"
#include "tree_generic.cuh"
#include "tree_mma.cuh"
#include "tree_tf32.cuh"
#include "tree_tiled.cuh"
#include "tree_ws.cuh"

namespace pa {
namespace {

pa_status plan_impl(PlanArgs a, cudaStream_t st) {
    const bool small = a.num_seqs <= kPlanSmallSeqs && a.max_tokens <= kPlanSmallTokens;
    cudaError_t err = launch_pdl(small ? plan_scan_kernel<true> : plan_scan_kernel<false>, dim3(1),
                                 dim3(kPlanScanThreads), 0, st, a);
    if (err != cudaSuccess) return PA_ERR_CUDA;
    if (small) return PA_OK;
    // a thread per four tokens (and at most that many fresh blocks), 8 CTAs a SM
    const int64_t sms = std::max(1, device_sm_count());
    const int64_t want = ((int64_t)a.max_tokens + 4 * kPlanFillThreads - 1) / (4 * kPlanFillThreads);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, sms * 8));
    err = launch_pdl(plan_fill_kernel, dim3(grid), dim3(kPlanFillThreads), 0, st, a);
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int LAYERS>
cudaError_t launch_accept(const AcceptArgs& a, void* const* k, void* const* v, int32_t layers,
                          int32_t num_seqs, int vec, cudaStream_t st) {
    AcceptCaches<LAYERS> c;
    for (int32_t l = 0; l < layers; ++l) {
        c.k[l] = static_cast<uint8_t*>(k[l]);
        c.v[l] = static_cast<uint8_t*>(v[l]);
    }
    const dim3 grid(num_seqs, 2 * layers);
    switch (vec) {
        case 16: return launch_pdl(accept_tree_kernel<16, LAYERS>, grid, dim3(kAcceptThreads), 0, st, a, c);
        case 8: return launch_pdl(accept_tree_kernel<8, LAYERS>, grid, dim3(kAcceptThreads), 0, st, a, c);
        case 4: return launch_pdl(accept_tree_kernel<4, LAYERS>, grid, dim3(kAcceptThreads), 0, st, a, c);
        default: return launch_pdl(accept_tree_kernel<2, LAYERS>, grid, dim3(kAcceptThreads), 0, st, a, c);
    }
}

// ---- tree attention: kernel choice, work division, workspace ---------------------

// Rows of one copy of the tcgen05 tree kernel: it lies inside one block and
// takes whole 8-row groups (a 128-byte swizzle atom); 0: the block size is
// not a multiple of 8.
int32_t tree_box_rows(int32_t block_size) {
    if (block_size % 8 != 0) return 0;
    int32_t rows = 8;
    while (rows < 128 && block_size % (2 * rows) == 0) rows *= 2;
    return rows;
}

// The tcgen05 kernel's shapes: bf16, head dims that are multiples of 16 up to
// 128, block sizes that are multiples of 8.
bool tree_ws_shape(const pa_cache_desc* c) {
    return c->dtype == PA_BF16 && c->head_dim % 16 == 0 && c->head_dim <= 128 &&
           tree_box_rows(c->block_size) > 0;
}

// A tile of `rows` (node, query head) rows, `tiles` of them a unit.
TreeShape tree_shape(int32_t rows, int32_t tiles, int32_t keys, int32_t group) {
    TreeShape s{};
    s.rows = rows;
    s.tiles = tiles;
    s.heads = std::min(group, rows);
    s.tokens = rows / s.heads;
    s.sub_groups = (group + s.heads - 1) / s.heads;
    s.keys = keys;
    s.block_one = s.block_more = 1;
    s.overhead = 1;
    s.min_range = 3;
    return s;
}

// Most that a unit can cost.
int64_t tree_most(const TreeShape& s, int32_t max_q_len, int32_t max_seq_len) {
    return ((int64_t)max_seq_len + s.keys - 1) / s.keys *
               (max_q_len > s.tokens ? s.block_more : s.block_one) +
           s.overhead;
}

// The current device, asked for once a call's sizing.
struct TreeDevice {
    int32_t id, sms;
};
TreeDevice tree_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) dev = -1;
    return {dev, std::max(1, device_sm_count())};
}

// CTAs of a call: `per_sm` a SM, fewer when the host's bounds say that less
// work can be there.
int32_t tree_ctas(const TreeShape& s, int32_t num_seqs, int32_t max_q_len, int32_t max_seq_len,
                  int32_t num_kv_heads, int32_t sms, int32_t per_sm) {
    const int64_t per = (int64_t)s.tokens * s.tiles;
    const int64_t units = (int64_t)num_seqs * num_kv_heads * s.sub_groups * ((max_q_len + per - 1) / per);
    const int64_t cost = tree_most(s, max_q_len, max_seq_len);
    const int64_t ctas = (units * cost + s.min_range - 1) / s.min_range;
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)sms * per_sm));
}

size_t tree_workspace(const TreeShape& s, int32_t ctas, int32_t head_dim) {
    if (s.fixed_cost > 0) return 0;
    return align256((size_t)ctas * sizeof(TreeCut)) +
           align256(2 * (size_t)ctas * tree_cell_floats(s, head_dim) * 4);
}

// Two 128-row tiles, blocks of 128 keys.  Costs in 0.73 us: a block takes 1.45 us
// with one tile in use and 2.25 us with two, a unit about 3 us beside them.
TreeShape tree_ws_tiling(int32_t group) {
    TreeShape s = tree_shape(128, 2, 128, group);
    s.block_one = 2;
    s.block_more = 3;
    s.overhead = 4;
    s.min_range = 8;
    return s;
}

// Warps of a CTA of the mma.sync and tf32 kernels, 16 rows each.  Up to 128
// columns the fewest of one, two and four that cover a sequence's rows, since
// more CTAs then share an SM (16 rows, D = 128, block size 4, 38 sequences x 4000
// tokens: 204 us with one warp, 350 with four of which one works); above, four:
// shared memory leaves room for few CTAs, and the other warps help to copy (D =
// 256: 508 us with four, 725 with one).
int32_t tree_row_warps(int32_t head_dim, int32_t group, int32_t max_q_len) {
    const int64_t rows = head_dim > 128 ? 64 : (int64_t)group * max_q_len;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

// The mma.sync kernel: 64-key chunks up to 128 columns (32-key ones for fewer
// than four warps), 32-key ones up to 256.
bool tree_mma_shape(const pa_cache_desc* c) {
    return c->dtype == PA_BF16 && c->head_dim % 16 == 0 && c->head_dim <= 256;
}
TreeShape tree_mma_tiling(int32_t head_dim, int32_t group, int32_t warps) {
    TreeShape s = tree_shape(16 * warps, 1, head_dim <= 128 && warps == 4 ? 64 : 32, group);
    s.overhead = 2;
    s.min_range = 8;
    return s;
}

// The tf32 kernel of fp32 caches: 32-key chunks for four warps and up to 128
// columns, else 16-key ones.
bool tree_tf_shape(const pa_cache_desc* c) { return c->dtype == PA_F32 && tiled_shape(c); }
TreeShape tree_tf_tiling(int32_t head_dim, int32_t group, int32_t warps) {
    TreeShape s = tree_shape(16 * warps, 1, head_dim <= 128 && warps == 4 ? 32 : 16, group);
    s.overhead = 2;
    s.min_range = 8;
    return s;
}

// The CUDA-core kernel of the other bf16 shapes: 16, 32 or 64 rows by what a
// sequence can have (up to 32 above 128 columns: D = 72, 38 sequences x 16 kv heads
// x 4000 tokens, 16 rows 956 us, 2460 in tiles of 64; 32 rows 1420, 2460); 32-key
// chunks up to 128 columns, 16-key ones up to 256.
int32_t tree_tiled_rpt(int32_t head_dim, int32_t group, int32_t max_q_len) {
    const int64_t rows = (int64_t)group * max_q_len;
    return rows <= 16 ? 1 : rows <= 32 || head_dim > 128 ? 2 : 4;
}
TreeShape tree_tiled_tiling(int32_t head_dim, int32_t group, int32_t max_q_len) {
    TreeShape s = tree_shape(16 * tree_tiled_rpt(head_dim, group, max_q_len), 1,
                             head_dim <= 128 ? 32 : 16, group);
    s.overhead = 2;
    s.min_range = 8;
    return s;
}

// An instance of the mma.sync, the tf32 or the CUDA-core kernel: its number, and its
// shared memory at the call's head dim and at its largest.  An instance's limit is
// set to the largest only, so that host threads with calls of two head dims do not
// set it under one another.
constexpr int kTreeInstances = 15;
struct TreeInstance {
    int number, threads;
    size_t smem, most;
};

template <typename Kern>
bool tree_allow_smem(Kern kern, const TreeInstance& t) {
    static std::atomic<uint64_t> allowed[kTreeInstances];    // (one type for all instances)
    return allow_smem(allowed[t.number], kern, t.most);
}

// CTAs of an instance that one SM of the current device holds, per head dim.
template <typename Kern>
int32_t tree_per_sm(Kern kern, const TreeInstance& t, int32_t device, int32_t head_dim) {
    static std::atomic<uint8_t> table[kMaxDevices][kTreeInstances][257];
    if (device < 0) return 1;
    std::atomic<uint8_t>& cached = table[device][t.number][head_dim];
    int n = cached.load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (tree_allow_smem(kern, t) && cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                    &n, kern, t.threads, t.smem) == cudaSuccess && n > 0) {
        cached.store((uint8_t)n, std::memory_order_relaxed);
        return n;
    }
    cudaGetLastError();
    return 1;
}

// Calls f(kernel, instance) with the instance of a head dim and warps: of the
// mma.sync, the tf32 and the CUDA-core kernel.
template <int DMAX, int KC, int WARPS, typename F>
auto call_tree_mma(int32_t head_dim, F f) {
    using C = TreeMmaCfg<DMAX, KC, WARPS>;
    return f(tree_mma_kernel<DMAX, KC, WARPS>,
             TreeInstance{DMAX > 128 ? 0 : WARPS, C::kThreads, C::smem_bytes(head_dim), C::smem_bytes(DMAX)});
}
template <typename F>
auto with_tree_mma(int32_t head_dim, int32_t warps, F f) {
    if (head_dim > 128) return call_tree_mma<256, 32, 4>(head_dim, f);
    return warps == 1   ? call_tree_mma<128, 32, 1>(head_dim, f)
           : warps == 2 ? call_tree_mma<128, 32, 2>(head_dim, f)
                        : call_tree_mma<128, 64, 4>(head_dim, f);
}
template <int DMAX, int KC, int WARPS, typename F>
auto call_tree_tf(int32_t head_dim, F f) {
    using C = TreeTfCfg<DMAX, KC, WARPS>;
    return f(tree_tf32_kernel<DMAX, KC, WARPS>,
             TreeInstance{5 + (DMAX > 128 ? 0 : WARPS), C::kThreads, C::smem_bytes(head_dim), C::smem_bytes(DMAX)});
}
template <typename F>
auto with_tree_tf(int32_t head_dim, int32_t warps, F f) {
    if (head_dim > 128) return call_tree_tf<256, 16, 4>(head_dim, f);
    return warps == 1   ? call_tree_tf<128, 16, 1>(head_dim, f)
           : warps == 2 ? call_tree_tf<128, 16, 2>(head_dim, f)
                        : call_tree_tf<128, 32, 4>(head_dim, f);
}
template <int RPT, int NF, int KC, typename F>
auto call_tree_tiled(int32_t head_dim, F f) {
    using C = TreeTiledCfg<RPT, NF, KC>;
    return f(tree_tiled_kernel<__nv_bfloat16, RPT, NF, KC>,
             TreeInstance{10 + (NF == 8 ? RPT - 1 : RPT == 4 ? 4 : RPT + 1), kTreeTiledThreads,
                          C::smem_bytes(head_dim, 2), C::smem_bytes(32 * NF, 2)});
}
template <typename F>
auto with_tree_tiled(int32_t head_dim, int32_t rpt, F f) {
    if (head_dim > 128)
        return rpt == 1 ? call_tree_tiled<1, 8, 16>(head_dim, f) : call_tree_tiled<2, 8, 16>(head_dim, f);
    return rpt == 1   ? call_tree_tiled<1, 4, 32>(head_dim, f)
           : rpt == 2 ? call_tree_tiled<2, 4, 32>(head_dim, f)
                      : call_tree_tiled<4, 4, 32>(head_dim, f);
}

// A kernel's tiling and CTAs for a call.
enum TreeKernel { kTreeWs, kTreeMma, kTreeTf, kTreeTiled };
struct TreeLaunch {
    TreeShape s;
    int32_t ctas, warps;
};
TreeLaunch tree_launch(TreeKernel k, const TreeDevice& dev, const pa_cache_desc* c, int32_t group,
                       int32_t num_seqs, int32_t max_q_len, int32_t max_seq_len) {
    TreeLaunch t{};
    t.warps = tree_row_warps(c->head_dim, group, max_q_len);
    int32_t per_sm = 1;
    auto resident = [&](auto kern, const TreeInstance& x) { return tree_per_sm(kern, x, dev.id, c->head_dim); };
    if (k == kTreeWs) {
        t.s = tree_ws_tiling(group);
    } else if (k == kTreeMma) {
        t.s = tree_mma_tiling(c->head_dim, group, t.warps);
        per_sm = with_tree_mma(c->head_dim, t.warps, resident);
    } else if (k == kTreeTf) {
        t.s = tree_tf_tiling(c->head_dim, group, t.warps);
        per_sm = with_tree_tf(c->head_dim, t.warps, resident);
    } else {
        t.s = tree_tiled_tiling(c->head_dim, group, max_q_len);
        const int32_t rpt = tree_tiled_rpt(c->head_dim, group, max_q_len);
        per_sm = with_tree_tiled(c->head_dim, rpt, resident);
    }
    // Short sequences go whole: no range ends inside a unit, so no merge follows.  A
    // unit's parts then cost the same whatever its length.  Whole against cut, 1 and
    // 64 sequences of 8 nodes, 8 kv heads, group 4, D = 128: tcgen05, 500 cached
    // tokens 12.0, 15.1 and 41.3, 53.6 us, 1000 tokens 17.0, 15.7 and 61.8, 69.9 us,
    // 2000 tokens 26.9, 16.2 and 106.5, 103.0 us; mma.sync, 118 tokens 19.2, 33.7 and
    // 24.9, 42.4 us, 500 tokens 48.9, 32.1 and 60.8, 64.5 us; tf32, 118 tokens 35.5,
    // 38.9 and 43.3, 55.0 us, 500 tokens 105, 39.8 and 133, 131 us.
    if (max_seq_len <= (k == kTreeWs ? 512 : 128)) {
        t.s.fixed_cost = (int32_t)tree_most(t.s, max_q_len, max_seq_len);
        t.s.min_range = t.s.fixed_cost;
    }
    t.ctas = tree_ctas(t.s, num_seqs, max_q_len, max_seq_len, c->num_kv_heads, dev.sms, per_sm);
    return t;
}

// Cache viewed as 5-D: (64 columns, 8 rows, 64-column halves, 8-row groups of
// a block, num_blocks * Hkv); one box is `rows` rows of one (block, head) tile,
// swizzled 128 B.  Head dims other than 64 and 128 have all their columns in
// the first dimension and one "half" (a box takes 64 of the columns; those past
// the head dim are filled with zeros).
bool encode_tree_map(CUtensorMap* map, const void* base, const pa_cache_desc* c, int32_t rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t halves = c->head_dim == 128 ? 2 : 1;
    const cuuint64_t row = (cuuint64_t)c->head_dim * 2;
    cuuint64_t dims[5] = {(cuuint64_t)c->head_dim / halves, 8, halves, (cuuint64_t)c->block_size / 8,
                          (cuuint64_t)c->num_blocks * (cuuint64_t)c->num_kv_heads};
    cuuint64_t strides[4] = {row, 128, 8 * row, row * (cuuint64_t)c->block_size};
    if (halves == 1) strides[1] = row;               // one entry: any multiple of 16
    cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, (cuuint32_t)rows / 8, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Queries [total_q][Hq][D] as 3-D; one box is a tile's (token, head) rows, 64
// columns of them.
bool encode_tree_q(CUtensorMap* map, const TreeArgs& a, const TreeShape& s) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row = (cuuint64_t)a.head_dim * 2;
    cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.total_q};
    cuuint64_t strides[2] = {row, row * (cuuint64_t)a.num_q_heads};
    cuuint32_t box[3] = {64, (cuuint32_t)s.heads, (cuuint32_t)s.tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int D, bool SPLIT>
cudaError_t launch_tree_ws(const TreeArgs& a, const TreeWork& w, const pa_cache_desc* c,
                           int32_t ctas, cudaStream_t st) {
    using Cfg = TreeWsCfg<D>;
    const int32_t rows = tree_box_rows(c->block_size);
    CUtensorMap mq, mk, mv;
    if (!encode_tree_q(&mq, a, w.s) || !encode_tree_map(&mk, a.k_cache, c, rows) || !encode_tree_map(&mv, a.v_cache, c, rows))
        return cudaErrorUnknown;
    auto kern = tree_ws_kernel<D, SPLIT>;
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, kern, Cfg::smem_bytes())) return cudaErrorUnknown;
    return launch_pdl(kern, dim3(ctas), dim3(Cfg::kThreads), Cfg::smem_bytes(), st, mq, mk, mv,
                      a, w, rows);
}

template <typename E>
cudaError_t launch_tree_merge(const TreeArgs& a, const TreeWork& w, int32_t ctas, cudaStream_t st) {
    if (w.cuts == nullptr || ctas == 1) return cudaSuccess;
    // (the last CTA's range ends with the work)
    const int32_t rows = std::min(a.max_q_len, w.s.tokens * w.s.tiles) * w.s.heads;
    const int32_t items = std::min(rows, w.s.rows * w.s.tiles) * ((a.head_dim + 7) / 8);
    const int32_t split = std::min(kTreeMergeSplit, (items + kTreeMergeThreads - 1) / kTreeMergeThreads);
    return launch_pdl(tree_merge_kernel<E>, dim3(ctas - 1, split), dim3(kTreeMergeThreads), 0, st, a,
                      w);
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_plan_step(const int32_t* seq_lens, const int32_t* new_tokens,
                       const int32_t* blocks_held, int32_t num_seqs,
                       const int32_t* free_blocks, int32_t num_free, const int32_t* free_head,
                       int32_t* ref_cnt, int32_t num_blocks, int32_t block_size,
                       int32_t* block_tables, int32_t max_blocks_per_seq,
                       int32_t* seq_lens_out, int32_t* blocks_held_out, int32_t* free_head_out,
                       int32_t* query_start_loc, int32_t* block_start, int64_t* slot_mapping,
                       int32_t* positions, int32_t* seq_ids, int32_t max_tokens, void* stream) {
    const CallRange range("pa_plan_step");
    constexpr int32_t kMost = INT32_MAX - (1 << 20);
    if (num_seqs < 0 || num_free < 0 || num_blocks <= 0 || block_size <= 0 ||
        max_blocks_per_seq < 0 || max_tokens < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || max_tokens >= kMost || num_free >= kMost) return PA_ERR_UNSUPPORTED;
    if ((num_seqs > 0 && (!seq_lens || !new_tokens || !blocks_held || !block_tables ||
                          !seq_lens_out || !blocks_held_out)) ||
        !free_head || !free_head_out || !query_start_loc || !block_start ||
        (max_tokens > 0 && !slot_mapping) || (num_free > 0 && !free_blocks))
        return PA_ERR_INVALID_ARG;
    PlanArgs a{seq_lens, new_tokens, blocks_held, free_blocks, free_head, ref_cnt, block_tables,
               seq_lens_out, blocks_held_out, free_head_out, query_start_loc, block_start,
               slot_mapping, positions, seq_ids, num_seqs, num_free, num_blocks, block_size,
               max_blocks_per_seq, max_tokens};
    // every output apart from every other array, but for the three that may be
    // the inputs themselves
    const size_t n = (size_t)num_seqs * 4, tok = (size_t)max_tokens * 4;
    struct Span {
        const void* p;
        size_t bytes, align;
    };
    const Span in[] = {{seq_lens, n, 4}, {new_tokens, n, 4}, {blocks_held, n, 4},
                       {free_blocks, (size_t)num_free * 4, 4}, {free_head, 4, 4}};
    const Span out[] = {{seq_lens_out, n, 4}, {blocks_held_out, n, 4}, {free_head_out, 4, 4},
                        {query_start_loc, n + 4, 4}, {block_start, n + 4, 4},
                        {slot_mapping, 2 * tok, 8}, {positions, tok, 4}, {seq_ids, tok, 4},
                        {block_tables, n * max_blocks_per_seq, 4},
                        {ref_cnt, (size_t)num_blocks * 4, 4}};
    for (const Span& x : in)
        if (!aligned(x.p, x.align)) return PA_ERR_INVALID_ARG;
    for (size_t x = 0; x < sizeof(out) / sizeof(out[0]); ++x) {
        if (!aligned(out[x].p, out[x].align)) return PA_ERR_INVALID_ARG;
        for (size_t y = 0; y < x; ++y)
            if (overlap(out[x].p, out[x].bytes, out[y].p, out[y].bytes)) return PA_ERR_INVALID_ARG;
        for (const Span& y : in) {
            const bool same = out[x].p == y.p && ((out[x].p == seq_lens_out && y.p == seq_lens) ||
                                                  (out[x].p == blocks_held_out && y.p == blocks_held) ||
                                                  (out[x].p == free_head_out && y.p == free_head));
            if (!same && overlap(out[x].p, out[x].bytes, y.p, y.bytes)) return PA_ERR_INVALID_ARG;
        }
    }
    const CallDevice dev;
    if (!dev.map(a.seq_lens) || !dev.map(a.new_tokens) || !dev.map(a.blocks_held) ||
        !dev.map(a.free_blocks) || !dev.map(a.free_head) ||
        !dev.map(a.seq_lens_out) || !dev.map(a.blocks_held_out) ||
        !dev.map(a.free_head_out) || !dev.map(a.query_start) ||
        !dev.map(a.block_start) || !dev.map(a.slot_mapping) ||
        !dev.map(a.positions) || !dev.map(a.seq_ids) ||
        (block_tables && !dev.memory(block_tables)) || (ref_cnt && !dev.memory(ref_cnt)))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass(
            [&] { return debug::check_free(a.free_blocks, num_free, a.free_head, num_blocks, st); });
        if (r != PA_OK) return r;
    }
    return plan_impl(a, st);
}

size_t pa_decode_tree_workspace_bytes(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                      int32_t max_q_len, int32_t max_seq_len,
                                      const pa_cache_desc* cache) {
    if (pa_decode_path(num_q_heads, cache) < 0 || num_seqs <= 0 || total_q <= 0 ||
        max_q_len <= 0 || max_seq_len <= 0)
        return 0;
    // the largest of the kernels that the call's pointers may select, for any number
    // of nodes up to max_q_len: CTAs of fewer row warps are more, so the size does
    // not grow with the nodes by itself
    const int32_t group = num_q_heads / cache->num_kv_heads;
    const TreeDevice dev = tree_device();
    size_t most = 0;
    auto take = [&](TreeKernel k) {
        for (int32_t rows = k == kTreeWs ? 64 : 16; rows <= 64; rows *= 2) {
            // the most nodes that this many rows cover (64 take any number, in turn)
            const int32_t nodes = rows < 64 ? rows / group : max_q_len;
            if (nodes < 1 || nodes > max_q_len) continue;
            const TreeLaunch t = tree_launch(k, dev, cache, group, num_seqs, nodes, max_seq_len);
            most = std::max(most, tree_workspace(t.s, t.ctas, cache->head_dim));
        }
    };
    if (tree_ws_shape(cache)) take(kTreeWs);
    if (tree_mma_shape(cache))
        take(kTreeMma);
    else if (tree_tf_shape(cache))
        take(kTreeTf);
    else if (tiled_shape(cache))
        take(kTreeTiled);
    return most;
}

pa_status pa_decode_tree(const void* q, const int32_t* query_start_loc, const int32_t* parents,
                         int32_t total_q, int32_t max_q_len, const void* k_cache,
                         const void* v_cache, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                         int32_t max_seq_len, int32_t num_q_heads, float scale, void* out,
                         void* workspace, size_t workspace_bytes_given, const pa_cache_desc* cache,
                         void* stream) {
    const CallRange range("pa_decode_tree");
    if (pa_decode_path(num_q_heads, cache) < 0 || num_seqs < 0 || total_q < 0 || max_q_len < 0 ||
        max_seq_len < 0 || max_blocks_per_seq < 0 || max_q_len > max_seq_len)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
    if (!q || !query_start_loc || !parents || !k_cache || !v_cache || !block_tables ||
        !seq_lens || !out)
        return PA_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * cache->block_size < max_seq_len) return PA_ERR_INVALID_ARG;
    // (key positions of a block behind the last stay in 32 bits)
    if (max_q_len > PA_MAX_TREE_NODES || num_seqs > 65535 || cache->num_kv_heads > 65535 ||
        cache->head_dim > 32 * kTreeDimPerLane || max_seq_len > INT32_MAX - 4096)
        return PA_ERR_UNSUPPORTED;
    const int eb = elem_bytes(cache);
    if (!aligned(q, eb) || !aligned(out, eb) || !aligned(k_cache, eb) || !aligned(v_cache, eb) ||
        !aligned(query_start_loc, 4) || !aligned(parents, 4) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4))
        return PA_ERR_INVALID_ARG;
    const CallDevice dev;
    if (!dev.map(q) || !dev.map(query_start_loc) || !dev.map(parents) ||
        !dev.map(block_tables) || !dev.map(seq_lens) || !dev.map(out) ||
        !dev.memory(k_cache) || !dev.memory(v_cache))
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_decode_tree_workspace_bytes(num_seqs, total_q, num_q_heads, max_q_len,
                                                       max_seq_len, cache);
    if (need > 0 && (!workspace || workspace_bytes_given < need || !aligned(workspace, 256) ||
                     !dev.memory(workspace)))
        return PA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass([&] {
            const pa_status x = debug::check_tables(block_tables, max_blocks_per_seq, seq_lens,
                                                    num_seqs, max_seq_len, query_start_loc, total_q,
                                                    cache, st);
            return x != PA_OK ? x
                              : debug::check_tree(query_start_loc, num_seqs, parents, total_q,
                                                  max_q_len, nullptr, st);
        });
        if (r != PA_OK) return r;
    }
    TreeArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.query_start = query_start_loc;
    a.parents = parents;
    a.seq_lens = seq_lens;
    a.block_tables = block_tables;
    a.out = out;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.max_seq_len = max_seq_len;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = cache->num_kv_heads;
    a.group = num_q_heads / cache->num_kv_heads;
    a.head_dim = cache->head_dim;
    a.scale_log2 = scale * kLog2e;
    // the tcgen05 kernel takes a row's maximum before it scales, and masks with
    // -inf: scale > 0; its copies of q are TMA, from device memory
    const bool ws = tree_ws_shape(cache) && aligned(q, 16) && dev.memory(q) &&
                    aligned(out, 16) && aligned(k_cache, 16) && aligned(v_cache, 16) && scale > 0.f;
    const bool caches16 = aligned(k_cache, 16) && aligned(v_cache, 16);
    const bool mma = !ws && tree_mma_shape(cache) && caches16;
    const bool tf = tree_tf_shape(cache) && caches16 && aligned(out, 16);
    const bool tiled = cache->dtype == PA_BF16 && !tree_mma_shape(cache) && tiled_shape(cache) &&
                       caches16 && aligned(out, 16);
    if (ws || mma || tf || tiled) {
        const TreeKernel kernel = ws ? kTreeWs : mma ? kTreeMma : tf ? kTreeTf : kTreeTiled;
        const TreeLaunch t = tree_launch(kernel, tree_device(), cache, a.group, num_seqs, max_q_len, max_seq_len);
        // unit costs are 32-bit in the kernels
        const int64_t per = (int64_t)t.s.tokens * t.s.tiles;
        if ((int64_t)a.num_kv_heads * t.s.sub_groups * ((max_q_len + per - 1) / per) *
                tree_most(t.s, max_q_len, max_seq_len) > INT32_MAX)
            return PA_ERR_UNSUPPORTED;
        TreeWork w{};
        w.s = t.s;
        uint8_t* base = static_cast<uint8_t*>(workspace);
        if (t.s.fixed_cost == 0) {
            w.cuts = reinterpret_cast<TreeCut*>(base);
            w.cells = reinterpret_cast<float*>(base + align256((size_t)t.ctas * sizeof(TreeCut)));
        }
        auto go = [&](auto kern, const TreeInstance& x) {
            if (!tree_allow_smem(kern, x)) return cudaErrorUnknown;
            return launch_pdl(kern, dim3(t.ctas), dim3(x.threads), x.smem, st, a, w);
        };
        cudaError_t err;
        if (mma)
            err = with_tree_mma(a.head_dim, t.warps, go);
        else if (tf)
            err = with_tree_tf(a.head_dim, t.warps, go);
        else if (tiled)
            err = with_tree_tiled(a.head_dim, tree_tiled_rpt(a.head_dim, a.group, max_q_len), go);
        else
            err = cache->head_dim == 128 ? launch_tree_ws<128, false>(a, w, cache, t.ctas, st)
                  : cache->head_dim > 64 ? launch_tree_ws<128, true>(a, w, cache, t.ctas, st)
                                         : launch_tree_ws<64, false>(a, w, cache, t.ctas, st);
        if (err == cudaSuccess)
            err = cache->dtype == PA_F32 ? launch_tree_merge<float>(a, w, t.ctas, st)
                                         : launch_tree_merge<__nv_bfloat16>(a, w, t.ctas, st);
        return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    const dim3 grid(total_q, cache->num_kv_heads);
    const cudaError_t err =
        cache->dtype == PA_F32
            ? launch_pdl(tree_generic_kernel<float>, grid, dim3(128), 0, st, a)
            : launch_pdl(tree_generic_kernel<__nv_bfloat16>, grid, dim3(128), 0, st, a);
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_accept_tree(const int32_t* leaf, const int32_t* parents,
                         const int32_t* query_start_loc, const int32_t* seq_lens,
                         int32_t num_seqs, int32_t total_q, int32_t max_q_len,
                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                         void* const* k_caches, void* const* v_caches, int32_t num_layers,
                         int32_t* new_lens, int32_t* accepted_rows, const pa_cache_desc* cache,
                         void* stream) {
    const CallRange range("pa_accept_tree");
    if (!desc_ok(cache) || num_seqs < 0 || total_q < 0 || max_q_len < 0 || num_layers < 1 ||
        max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (max_q_len > PA_MAX_TREE_NODES || num_layers > kAcceptMaxLayers) return PA_ERR_UNSUPPORTED;
    if (!leaf || (!parents && total_q > 0) || !query_start_loc || !seq_lens || !block_tables ||
        !k_caches || !v_caches || !new_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(leaf, 4) || !aligned(parents, 4) || !aligned(query_start_loc, 4) ||
        !aligned(seq_lens, 4) || !aligned(block_tables, 4) || !aligned(new_lens, 4) ||
        !aligned(accepted_rows, 4))
        return PA_ERR_INVALID_ARG;
    // the outputs apart from the inputs and from one another
    const size_t n = (size_t)num_seqs * 4, rows = (size_t)total_q * 4;
    const size_t tab = n * max_blocks_per_seq;
    if (overlap(new_lens, n, accepted_rows, rows)) return PA_ERR_INVALID_ARG;
    const std::pair<const void*, size_t> in[] = {{leaf, n}, {parents, rows},
                                                 {query_start_loc, n + 4}, {seq_lens, n},
                                                 {block_tables, tab}};
    for (const auto& x : in)
        if (overlap(new_lens, n, x.first, x.second) ||
            overlap(accepted_rows, rows, x.first, x.second))
            return PA_ERR_INVALID_ARG;
    AcceptArgs a{leaf, parents, query_start_loc, seq_lens, block_tables, new_lens, accepted_rows,
                 total_q, max_q_len, max_blocks_per_seq, cache->num_blocks, cache->block_size,
                 cache->num_kv_heads, cache->head_dim * elem_bytes(cache)};
    const CallDevice dev;
    if (!dev.map(a.leaf) || !dev.map(a.parents) || !dev.map(a.query_start) ||
        !dev.map(a.seq_lens) || !dev.map(a.block_tables) ||
        !dev.map(a.new_lens) || !dev.map(a.accepted_rows))
        return PA_ERR_INVALID_ARG;
    int vec = 16;
    while (vec > 2 && a.row_bytes % vec) vec >>= 1;
    // the caches, none of which may share a byte with another (their moves
    // would race)
    uintptr_t bases[2 * kAcceptMaxLayers];
    for (int32_t l = 0; l < num_layers; ++l) {
        for (int which = 0; which < 2; ++which) {
            void* c = which ? v_caches[l] : k_caches[l];
            if (!dev.memory(c) || !aligned(c, elem_bytes(cache)))
                return PA_ERR_INVALID_ARG;
            while (vec > 2 && !aligned(c, vec)) vec >>= 1;
            bases[2 * l + which] = reinterpret_cast<uintptr_t>(c);
        }
    }
    std::sort(bases, bases + 2 * num_layers);
    const size_t cache_bytes = (size_t)cache->num_blocks * cache->num_kv_heads *
                               cache->block_size * (size_t)a.row_bytes;
    for (int32_t x = 1; x < 2 * num_layers; ++x)
        if (bases[x] - bases[x - 1] < cache_bytes) return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass([&] {
            return debug::check_tree(a.query_start, num_seqs, a.parents, total_q, max_q_len, a.leaf, st);
        });
        if (r != PA_OK) return r;
    }
    for (int32_t l0 = 0; l0 < num_layers; l0 += kAcceptLayers) {
        const int32_t nl = std::min(kAcceptLayers, num_layers - l0);
        if (l0 > 0) a.new_lens = nullptr;        // written by the first launch
        const cudaError_t err =
            nl <= kAcceptFew
                ? launch_accept<kAcceptFew>(a, k_caches + l0, v_caches + l0, nl, num_seqs, vec, st)
                : launch_accept<kAcceptLayers>(a, k_caches + l0, v_caches + l0, nl, num_seqs, vec, st);
        if (err != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // extern "C"

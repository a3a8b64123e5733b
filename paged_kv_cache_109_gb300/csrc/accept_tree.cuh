// accept_tree.cuh -- keep the accepted path of each draft tree: the K/V rows of
// its nodes a_0 < a_1 < ... move to the positions right behind the cached
// tokens, cache row C + j <- cache row C + a_j, in every layer.
//
// A path's nodes ascend and a_j >= j, so a row is only ever overwritten after
// the one step that reads it: j ascending, row C + j is a source of no later
// step (a_m > a_j >= j for m > j).  A thread owns the same bytes of every row
// and takes the steps in order, a batch of loads before that batch's stores,
// so no thread depends on another.
//
// Bound: each moved row's bytes, read and written once.  Measured (GPU time): 128
// sequences x 16 layers, 61 MB moved, 9.8 us in back-to-back calls, whose rows stay
// in L2, and 15 us alone with cold caches, where the copy rate allows 9.0; one
// sequence 2.8 us, the launch.
#pragma once

#include "common.cuh"
#include "ptx.cuh"
#include "write_kv.cuh"

namespace pa {

constexpr int kAcceptThreads = 128;
constexpr int kAcceptUnroll = 4;
// Layers of one launch: 16, or 128 (2 KB of pointers, which the host copies for
// every launch).
constexpr int kAcceptFew = 16, kAcceptLayers = 128;
constexpr int kAcceptMaxLayers = 1024;  // layers of one call

template <int LAYERS>
struct AcceptCaches {
    uint8_t* k[LAYERS];
    uint8_t* v[LAYERS];
};

struct AcceptArgs {
    const int32_t* leaf;
    const int32_t* parents;
    const int32_t* query_start;
    const int32_t* seq_lens;
    const int32_t* block_tables;
    int32_t* new_lens;              // nullptr: an earlier launch wrote them
    int32_t* accepted_rows;         // may be nullptr
    int32_t total_q, max_q_len, max_blocks, num_blocks, block_size, num_kv_heads;
    int32_t row_bytes;              // one (token, kv head) row
};

// One CTA per (sequence, layer, K or V).
template <int VEC, int LAYERS>
__global__ void __launch_bounds__(kAcceptThreads)
accept_tree_kernel(const AcceptArgs a, const __grid_constant__ AcceptCaches<LAYERS> caches) {
    using V = typename VecType<VEC>::T;
    __shared__ int32_t s_parent[PA_MAX_TREE_NODES];
    __shared__ int32_t s_path[PA_MAX_TREE_NODES];
    __shared__ int64_t s_src[PA_MAX_TREE_NODES], s_dst[PA_MAX_TREE_NODES];   // row offsets, -1: skip
    __shared__ int32_t s_depth;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x, i = blockIdx.x;
    const bool first = blockIdx.y == 0;
    const int32_t q0 = a.query_start[i], q1 = a.query_start[i + 1];
    const int32_t T = a.seq_lens[i], B = a.block_size;
    if (q1 < q0 || (int64_t)q1 - q0 > min(a.max_q_len, PA_MAX_TREE_NODES) || q0 < 0 ||
        q1 > a.total_q || T < q1 - q0 || T > (int64_t)a.max_blocks * B) {
        if (first && a.new_lens != nullptr) {
            if (tid == 0) {
                raise_error(PA_DEVERR_SEQ_LEN);
                a.new_lens[i] = T;
            }
            // those of its rows that there are, unless starts in no order may have
            // given them to another sequence too
            bool ordered = a.accepted_rows != nullptr;
            for (int32_t j = tid; j < (int32_t)gridDim.x; j += kAcceptThreads)
                ordered = ordered && a.query_start[j] <= a.query_start[j + 1];
            if (__syncthreads_and(ordered))
                for (int64_t r = (int64_t)max(q0, 0) + tid; r < min(q1, a.total_q); r += kAcceptThreads)
                    a.accepted_rows[r] = -1;
        }
        return;
    }
    const int32_t n = q1 - q0;
    const int32_t C = T - n;
    for (int32_t j = tid; j < n; j += kAcceptThreads) s_parent[j] = a.parents[q0 + j];
    __syncthreads();
    if (tid == 0) {
        // depth of the leaf, then its path from the end
        const int32_t leaf = a.leaf[i];
        bool ok = leaf >= -1 && leaf < n;
        int32_t d = 0;
        for (int32_t x = leaf; ok && x >= 0; x = s_parent[x]) {
            ++d;
            ok = s_parent[x] >= -1 && s_parent[x] < x;
        }
        if (!ok) {
            if (first) raise_error(PA_DEVERR_TREE);
            d = 0;
        }
        int32_t x = leaf;
        for (int32_t j = d - 1; j >= 0; --j, x = s_parent[x]) s_path[j] = x;
        s_depth = d;
    }
    __syncthreads();
    const int32_t d = s_depth;
    if (first) {
        if (tid == 0 && a.new_lens != nullptr) a.new_lens[i] = C + d;
        if (a.accepted_rows != nullptr && a.new_lens != nullptr)
            for (int32_t j = tid; j < n; j += kAcceptThreads)
                a.accepted_rows[q0 + j] = j < d ? q0 + s_path[j] : -1;
    }
    const int64_t head_stride = (int64_t)B * a.row_bytes;
    const int32_t* table = a.block_tables + (int64_t)i * a.max_blocks;
    for (int32_t j = tid; j < d; j += kAcceptThreads) {
        const int32_t from = C + s_path[j], to = C + j;
        int64_t src = -1, dst = -1;
        if (from != to) {
            const int32_t sb = table[from / B], db = table[to / B];
            if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                if (first) raise_error(PA_DEVERR_TABLE_ENTRY);
            } else {
                src = sb * (int64_t)a.num_kv_heads * head_stride + (from % B) * (int64_t)a.row_bytes;
                dst = db * (int64_t)a.num_kv_heads * head_stride + (to % B) * (int64_t)a.row_bytes;
            }
        }
        s_src[j] = src;
        s_dst[j] = dst;
    }
    __syncthreads();
    const int32_t layer = blockIdx.y >> 1;
    uint8_t* cache = (blockIdx.y & 1) ? caches.v[layer] : caches.k[layer];
    const int32_t vpr = a.row_bytes / VEC;
    for (int32_t x = tid; x < a.num_kv_heads * vpr; x += kAcceptThreads) {
        const int32_t h = x / vpr, c = x - h * vpr;
        uint8_t* base = cache + h * head_stride + (int64_t)c * VEC;
        for (int32_t j0 = 0; j0 < d; j0 += kAcceptUnroll) {
            V buf[kAcceptUnroll];
#pragma unroll
            for (int u = 0; u < kAcceptUnroll; ++u)
                if (j0 + u < d && s_src[j0 + u] >= 0)
                    buf[u] = *reinterpret_cast<const V*>(base + s_src[j0 + u]);
#pragma unroll
            for (int u = 0; u < kAcceptUnroll; ++u)
                if (j0 + u < d && s_src[j0 + u] >= 0)
                    *reinterpret_cast<V*>(base + s_dst[j0 + u]) = buf[u];
        }
    }
}

}  // namespace pa

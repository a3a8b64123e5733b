// tree_generic.cuh -- attention of a tree of drafted tokens over the paged
// cache, for every shape (head dims up to 256) the other tree kernels do not
// take.
//
// Row r is node j = r - query_start[i] of sequence i; with C = T - n cached
// tokens it sees keys 0 .. C - 1, the keys C + k of its ancestors k, and its
// own key C + j:  out = sum_t softmax_t(scale q.k_t) v_t over those.
//
// One CTA per (row, kv head); warp w takes query heads w, w + 4, ... of the
// group, lanes split the head dimension, keys come one at a time with an
// online softmax.  Keys that the row does not see are not read.  Bound by the
// latency of a key's load and reduction, one after another: 8 sequences x 8 kv
// heads x 2000 tokens, 8 nodes, group 4, D = 42 take 1.48 ms in bf16, 1.67 in fp32.
#pragma once

#include "tree_args.cuh"

namespace pa {

// This CTA's row, which is sequence i's.
template <typename E>
__device__ __forceinline__ void tree_generic_row(const TreeArgs& a, int32_t i, const TreeSeq s) {
    __shared__ uint32_t s_vis[PA_MAX_TREE_NODES / 32];
    const int32_t r = blockIdx.x, g = blockIdx.y;
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t D = a.head_dim, G = a.group, BS = a.block_size;
    const int32_t j = r - s.q0;
    if (threadIdx.x < PA_MAX_TREE_NODES / 32) s_vis[threadIdx.x] = 0;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int32_t x = j; x >= 0;) {
            s_vis[x >> 5] |= 1u << (x & 31);
            x = tree_parent(a.parents[s.q0 + x], x, g == 0);
        }
    }
    __syncthreads();
    const int32_t C = s.T - s.n;
    const int32_t* table = a.block_tables + (int64_t)i * a.max_blocks;
    const E* q = static_cast<const E*>(a.q);
    const E* kc = static_cast<const E*>(a.k_cache);
    const E* vc = static_cast<const E*>(a.v_cache);
    E* out = static_cast<E*>(a.out);
    for (int32_t hh = warp; hh < G; hh += 4) {
        const int64_t row_q = ((int64_t)r * a.num_q_heads + (int64_t)g * G + hh) * D;
        float qv[kTreeDimPerLane], acc[kTreeDimPerLane];
#pragma unroll
        for (int c = 0; c < kTreeDimPerLane; ++c) {
            const int32_t d = lane + 32 * c;
            qv[c] = d < D ? Elem<E>::to_float(q[row_q + d]) : 0.f;
            acc[c] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        for (int32_t t = 0; t <= C + j; ++t) {
            if (t >= C && !(s_vis[(t - C) >> 5] >> ((t - C) & 31) & 1u)) continue;
            const int32_t id = table[t / BS];
            if (id < 0 || id >= a.num_blocks) {
                if (lane == 0) raise_error(PA_DEVERR_TABLE_ENTRY);
                continue;
            }
            const int64_t row = (((int64_t)id * a.num_kv_heads + g) * BS + t % BS) * D;
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < kTreeDimPerLane; ++c) {
                const int32_t d = lane + 32 * c;
                if (d < D) dot = fmaf(qv[c], Elem<E>::to_float(kc[row + d]), dot);
            }
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            const float sc = dot * a.scale_log2;
            const float mn = fmaxf(m, sc);
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float al = exp2f(m - ref), w = exp2f(sc - ref);
            m = mn;
            l = fmaf(l, al, w);
#pragma unroll
            for (int c = 0; c < kTreeDimPerLane; ++c) {
                const int32_t d = lane + 32 * c;
                if (d < D) acc[c] = fmaf(w, Elem<E>::to_float(vc[row + d]), acc[c] * al);
            }
        }
        // (l is NaN where a score is: the row is NaN then, as the formula has it)
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int c = 0; c < kTreeDimPerLane; ++c) {
            const int32_t d = lane + 32 * c;
            if (d < D) out[row_q + d] = Elem<E>::from_float(acc[c] * inv);
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(128) tree_generic_kernel(const TreeArgs a) {
    griddep_wait();
    const int32_t r = blockIdx.x;
    // the first CTA reports the refused sequences (some have no rows)
    if (r == 0 && blockIdx.y == 0)
        for (int32_t x = threadIdx.x; x < a.num_seqs; x += 128) tree_seq(a, x, true);
    // sequence of row r: the last i with query_start[i] <= r
    int32_t lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (a.query_start[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const TreeSeq s = tree_seq(a, lo, false);
    if (r >= s.q0 && r - s.q0 < s.n) {
        tree_generic_row<E>(a, lo, s);
        return;
    }
    // behind the last sequence, refused, or starts that do not ascend (a copy of the
    // row's code: with one for both, fp32 rows took 15% longer)
    __shared__ int32_t s_seq;
    if (threadIdx.x == 0) s_seq = -1;
    __syncthreads();
    for (int32_t x = threadIdx.x; x < a.num_seqs; x += 128) {
        const TreeSeq t = tree_seq(a, x, false);
        if (r >= t.q0 && r - t.q0 < t.n) atomicMax(&s_seq, x);
    }
    __syncthreads();
    const int32_t i = s_seq;
    if (i >= 0) tree_generic_row<E>(a, i, tree_seq(a, i, false));
}

}  // namespace pa

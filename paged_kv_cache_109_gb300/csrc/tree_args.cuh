// tree_args.cuh -- arguments of the draft-tree attention kernels, and what they
// share: a sequence's rows and lengths with their checks, a node's parent.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "ptx.cuh"

namespace pa {

constexpr int kTreeDimPerLane = 8;      // head_dim <= 256

struct TreeArgs {
    const void* q;                  // [total_q][Hq][D]
    const void* k_cache;            // [num_blocks][Hkv][B][D]
    const void* v_cache;
    const int32_t* query_start;     // [N + 1]
    const int32_t* parents;         // [total_q]
    const int32_t* seq_lens;        // [N]
    const int32_t* block_tables;    // [N][max_blocks]
    void* out;                      // [total_q][Hq][D]
    int32_t num_seqs, total_q, max_q_len, max_seq_len;
    int32_t max_blocks, num_blocks, block_size;
    int32_t num_q_heads, num_kv_heads, group, head_dim;
    float scale_log2;               // scale * log2(e)
};

// Rows and length of a sequence; n = 0 where there is nothing to do or the
// sequence is refused (reported once, by the thread that asks with `report`).
struct TreeSeq {
    int32_t q0, n, T;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int32_t i, bool report) {
    TreeSeq s;
    s.q0 = a.query_start[i];
    const int64_t n = (int64_t)a.query_start[i + 1] - s.q0;
    s.T = a.seq_lens[i];
    const int64_t cap = min((int64_t)a.max_seq_len, (int64_t)a.max_blocks * a.block_size);
    const bool ok = n >= 0 && n <= a.max_q_len && s.q0 >= 0 && s.q0 + n <= a.total_q &&
                    s.T >= n && s.T <= cap;
    if (!ok && report) raise_error(PA_DEVERR_SEQ_LEN);
    s.n = ok ? (int32_t)n : 0;
    return s;
}

// Parent of node x: one outside [-1, x) is reported and read as -1 (the walk
// up always ends).
__device__ __forceinline__ int32_t tree_parent(int32_t p, int32_t x, bool report) {
    if (p >= -1 && p < x) return p;
    if (report) raise_error(PA_DEVERR_TREE);
    return -1;
}

}  // namespace pa

// plan_step.cuh -- block tables and slot mapping of a step on the GPU, from the
// requests' lengths: BlockPool.grow of every sequence in order ("vLLM
// PagedAttention: from memory fragmentation to slot mapping" §3-§4, §6).
//
// With C_i cached and n_i new tokens, h_i blocks held and block size B,
//   g_i = max(0, ceil((C_i + n_i) / B) - h_i)
//   Q = exclusive sum of n, S = exclusive sum of g
//   table[i][h_i + k] = free[F + S_i + k],  slot(Q_i + j) through position C_i + j.
// Two launches.  plan_scan_kernel, one CTA: the totals decide whether the step
// fits (all or nothing), then the running sums and the per-sequence outputs
// are written.  plan_fill_kernel, a CTA per tile of tokens and of fresh table
// entries: each finds its sequence by binary search in Q (or S).  A token's
// block is taken from the table below h_i and straight from the queue above
// it, so no thread reads an entry that another one writes.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace pa {

struct PlanArgs {
    const int32_t* seq_lens;
    const int32_t* new_tokens;
    const int32_t* blocks_held;
    const int32_t* free_blocks;
    const int32_t* free_head;
    int32_t* ref_cnt;               // may be nullptr
    int32_t* block_tables;          // [N][max_blocks]
    int32_t* seq_lens_out;          // may be seq_lens
    int32_t* blocks_held_out;       // may be blocks_held
    int32_t* free_head_out;         // may be free_head
    int32_t* query_start;           // [N + 1]
    int32_t* block_start;           // [N + 1]
    int64_t* slot_mapping;          // [max_tokens]
    int32_t* positions;             // may be nullptr
    int32_t* seq_ids;               // may be nullptr
    int32_t num_seqs, num_free, num_blocks, block_size, max_blocks, max_tokens;
};

// One sequence's new tokens and blocks to take; `bad` collects PA_DEVERR_* bits.
struct PlanSeq {
    int32_t len, add, held, grow;
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int32_t i, unsigned int& bad) {
    PlanSeq s{a.seq_lens[i], a.new_tokens[i], a.blocks_held[i], 0};
    const int32_t B = a.block_size;
    const int64_t cap = min((int64_t)a.max_blocks * B, (int64_t)INT32_MAX);
    const int64_t total = (int64_t)s.len + s.add;
    if (s.len < 0 || s.add < 0 || total > cap || s.held < 0 || s.held > a.max_blocks ||
        ((int64_t)s.len + B - 1) / B > s.held) {
        bad |= PA_DEVERR_SEQ_LEN;
        return s;
    }
    s.grow = (int32_t)max((int64_t)0, (total + B - 1) / B - s.held);
    if (a.ref_cnt != nullptr && s.add > 0 && s.len % B != 0) {
        const int32_t id = a.block_tables[(int64_t)i * a.max_blocks + s.len / B];
        if (id >= 0 && id < a.num_blocks && a.ref_cnt[id] > 1) bad |= PA_DEVERR_SHARED;
    }
    return s;
}

constexpr int kPlanScanThreads = 1024;

__global__ void __launch_bounds__(kPlanScanThreads) plan_scan_kernel(const PlanArgs a) {
    __shared__ int64_t s_new[32], s_grow[32];
    __shared__ unsigned int s_bad[32];
    griddep_wait();
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t head = *a.free_head;
    // totals: does the step fit?
    int64_t add = 0, grow = 0;
    unsigned int bad = 0;
    for (int32_t i = tid; i < a.num_seqs; i += kPlanScanThreads) {
        const PlanSeq s = plan_seq(a, i, bad);
        add += s.add;
        grow += s.grow;
    }
    for (int off = 16; off > 0; off >>= 1) {
        add += __shfl_xor_sync(0xffffffffu, add, off);
        grow += __shfl_xor_sync(0xffffffffu, grow, off);
        bad |= __shfl_xor_sync(0xffffffffu, bad, off);
    }
    if (lane == 0) {
        s_new[warp] = add;
        s_grow[warp] = grow;
        s_bad[warp] = bad;
    }
    __syncthreads();
    add = s_new[lane];
    grow = s_grow[lane];
    bad = s_bad[lane];
    for (int off = 16; off > 0; off >>= 1) {
        add += __shfl_xor_sync(0xffffffffu, add, off);
        grow += __shfl_xor_sync(0xffffffffu, grow, off);
        bad |= __shfl_xor_sync(0xffffffffu, bad, off);
    }
    if (bad == 0 && add > a.max_tokens) bad |= PA_DEVERR_SEQ_LEN;
    if (bad == 0 && (head < 0 || head + grow > a.num_free)) bad |= PA_DEVERR_POOL;
    const bool fits = bad == 0;
    if (tid == 0 && !fits) raise_error(bad);
    __syncthreads();
    // running sums over tiles of 1024 sequences (fits: they stay in 32 bits)
    int32_t q0 = 0, b0 = 0;
    for (int32_t i0 = 0; i0 < a.num_seqs; i0 += kPlanScanThreads) {
        const int32_t i = i0 + tid;
        PlanSeq s{0, 0, 0, 0};
        if (i < a.num_seqs) {
            unsigned int ignored = 0;
            s = plan_seq(a, i, ignored);
        }
        if (!fits) s.add = s.grow = 0;
        int32_t qi = s.add, bi = s.grow;
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, qi, off);
            const int32_t y = __shfl_up_sync(0xffffffffu, bi, off);
            if (lane >= off) {
                qi += x;
                bi += y;
            }
        }
        if (lane == 31) {
            s_new[warp] = qi;
            s_grow[warp] = bi;
        }
        __syncthreads();
        int32_t wq = (int32_t)s_new[lane], wb = (int32_t)s_grow[lane];
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, wq, off);
            const int32_t y = __shfl_up_sync(0xffffffffu, wb, off);
            if (lane >= off) {
                wq += x;
                wb += y;
            }
        }
        const int32_t before_q = warp ? __shfl_sync(0xffffffffu, wq, max(warp - 1, 0)) : 0;
        const int32_t before_b = warp ? __shfl_sync(0xffffffffu, wb, max(warp - 1, 0)) : 0;
        if (i < a.num_seqs) {
            a.query_start[i] = q0 + before_q + qi - s.add;
            a.block_start[i] = b0 + before_b + bi - s.grow;
            a.seq_lens_out[i] = s.len + s.add;
            a.blocks_held_out[i] = s.held + s.grow;
        }
        q0 += __shfl_sync(0xffffffffu, wq, 31);
        b0 += __shfl_sync(0xffffffffu, wb, 31);
        __syncthreads();                          // s_new, s_grow free for the next tile
    }
    if (tid == 0) {
        a.query_start[a.num_seqs] = q0;
        a.block_start[a.num_seqs] = b0;
        *a.free_head_out = head + b0;
    }
}

// Last i in [0, n) with start[i] <= x (start[0] <= x).
__device__ __forceinline__ int32_t plan_find(const int32_t* start, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Block of the queue, -1 and a report for an id outside the pool.
__device__ __forceinline__ int32_t plan_free(const PlanArgs& a, int32_t at) {
    const int32_t id = a.free_blocks[at];
    if (id < 0 || id >= a.num_blocks) {
        raise_error(PA_DEVERR_TABLE_ENTRY);
        return -1;
    }
    return id;
}

constexpr int kPlanFillThreads = 256;

__global__ void __launch_bounds__(kPlanFillThreads) plan_fill_kernel(const PlanArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int32_t N = a.num_seqs, B = a.block_size;
    const int32_t tokens = a.query_start[N], blocks = a.block_start[N];
    const int32_t head = *a.free_head_out - blocks;
    const int32_t stride = gridDim.x * kPlanFillThreads;
    const int32_t first = blockIdx.x * kPlanFillThreads + threadIdx.x;
    for (int32_t e = first; e < blocks; e += stride) {
        const int32_t i = plan_find(a.block_start, N, e);
        const int32_t held = a.blocks_held_out[i] - (a.block_start[i + 1] - a.block_start[i]);
        const int32_t id = plan_free(a, head + e);
        a.block_tables[(int64_t)i * a.max_blocks + held + (e - a.block_start[i])] = id;
        if (a.ref_cnt != nullptr && id >= 0) a.ref_cnt[id] = 1;
    }
    for (int32_t t = first; t < a.max_tokens; t += stride) {
        int32_t i = -1, p = -1;
        int64_t slot = -1;
        if (t < tokens) {
            i = plan_find(a.query_start, N, t);
            const int32_t q0 = a.query_start[i], add = a.query_start[i + 1] - q0;
            const int32_t took = a.block_start[i + 1] - a.block_start[i];
            const int32_t held = a.blocks_held_out[i] - took;
            p = a.seq_lens_out[i] - add + (t - q0);
            const int32_t b = p / B;
            int32_t id;
            if (b < held) {
                id = a.block_tables[(int64_t)i * a.max_blocks + b];
                if (id < 0 || id >= a.num_blocks) {
                    raise_error(PA_DEVERR_TABLE_ENTRY);
                    id = -1;
                }
            } else {
                id = plan_free(a, head + a.block_start[i] + (b - held));
            }
            if (id >= 0) slot = (int64_t)id * B + p % B;
        }
        a.slot_mapping[t] = slot;
        if (a.positions != nullptr) a.positions[t] = p;
        if (a.seq_ids != nullptr) a.seq_ids[t] = i;
    }
}

}  // namespace pa

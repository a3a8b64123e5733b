// plan_step.cuh -- block tables and slot mapping of a step on the GPU, from the
// requests' lengths: BlockPool.grow of every sequence in order ("vLLM
// PagedAttention: from memory fragmentation to slot mapping" §3-§4, §6).
//
// With C_i cached and n_i new tokens, h_i blocks held and block size B,
//   g_i = max(0, ceil((C_i + n_i) / B) - h_i)
//   Q = exclusive sum of n, S = exclusive sum of g
//   table[i][h_i + k] = free[F + S_i + k],  slot(Q_i + j) through position C_i + j.
// plan_scan_kernel, one CTA: the totals decide whether the step fits (all or
// nothing), then the running sums and the per-sequence outputs are written.  A
// token's block is taken from the table below h_i and straight from the queue
// above it, so no thread reads an entry that another one writes.  A small step
// (up to kPlanSmallSeqs sequences and kPlanSmallTokens tokens) ends in the same
// CTA: one launch, whose latency is what such a step costs (GPU time, one launch
// against two: 64 sequences with a token each 6.4 us, 10.9; at the limits, 256 x 32
// tokens 9.2, 9.6 and 1024 x 8 10.6, 11.3).  Otherwise plan_fill_kernel writes tokens and fresh
// entries from the whole GPU.  A thread takes four consecutive tokens, with one
// table entry for as long as they share a block and 16-byte stores; in global
// memory a warp searches Q together for its 128 tokens.
//
// Measured (GPU time of the whole call): 2048 sequences with some 2.1 million new
// tokens 19.7 us, where the bytes take 5.0; with a search by each thread 21.0.  It
// is bound by latencies: the one CTA's scan (8 us) and then the fill's dependent
// loads; filling the SMs further (32 registers a thread) changed nothing.  In the
// small form the sums are in shared memory and each thread's own search is the
// faster one: 6.4 us against 6.8 for a decode step, 8.8 against 9.4 for a drafted
// one.
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
    if (a.ref_cnt != nullptr && s.add > 0) {
        // the held blocks that the new tokens go into
        const int32_t end = min(s.held, (int32_t)((total + B - 1) / B));
        for (int32_t b = s.len / B; b < end; ++b) {
            const int32_t id = a.block_tables[(int64_t)i * a.max_blocks + b];
            if (id >= 0 && id < a.num_blocks && a.ref_cnt[id] > 1) bad |= PA_DEVERR_SHARED;
        }
    }
    return s;
}

constexpr int kPlanScanThreads = 1024;
constexpr int kPlanHeld = 4;            // sequences a thread keeps in registers
constexpr int kPlanSmallSeqs = 1024, kPlanSmallTokens = 8192;

// Last i in [0, n) with start[i] <= x (start[0] <= x).
__device__ __forceinline__ int32_t plan_find(const int32_t* start, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The same by a whole warp, all lanes with one x: 32 probes a round.
__device__ __forceinline__ int32_t plan_find_warp(const int32_t* start, int32_t n, int32_t x) {
    const int32_t lane = threadIdx.x & 31;
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t step = (hi - lo + 32) / 32;
        const int32_t at = lo + (lane + 1) * step;
        const uint32_t yes = __ballot_sync(0xffffffffu, at <= hi && start[min(at, hi)] <= x);
        lo += __popc(yes) * step;
        hi = min(hi, lo + step - 1);
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

// What the fill reads: the sums and the per-sequence results, in global memory
// or (small steps) in shared memory.
struct PlanSums {
    const int32_t *query_start, *block_start, *lens, *held;   // [N + 1], [N + 1], [N], [N]
    int32_t tokens, blocks, head;
};

// One sequence of the fill.
struct PlanSpan {
    int32_t i, q0, q1, pos0, held, taken, take0;   // tokens [q0, q1) from position pos0
};
__device__ __forceinline__ PlanSpan plan_span(const PlanSums& s, int32_t i) {
    PlanSpan p;
    p.i = i;
    p.q0 = s.query_start[i];
    p.q1 = s.query_start[i + 1];
    p.take0 = s.block_start[i];
    p.taken = s.block_start[i + 1] - p.take0;
    p.held = s.held[i] - p.taken;
    p.pos0 = s.lens[i] - (p.q1 - p.q0);
    return p;
}

// The sequence of item x of [0, total), all lanes of a warp with consecutive
// groups of PER items from x0 on (x = x0 + PER * lane).  TOGETHER (sums in global
// memory): the warp finds the first and the last one's, and only where they
// differ does each lane search between them.
template <bool TOGETHER, int32_t PER>
__device__ __forceinline__ int32_t plan_seq_of(const int32_t* start, int32_t n, int32_t x0,
                                               int32_t x, int32_t total) {
    if constexpr (!TOGETHER) {
        return x < total ? plan_find(start, n, x) : 0;
    } else {
        if (x0 >= total) return 0;
        const int32_t lo = plan_find_warp(start, n, x0);
        const int32_t end = x0 + min(total - x0, 32 * PER) - 1;
        const int32_t hi = start[lo + 1] > end ? lo : plan_find_warp(start, n, end);
        return lo == hi || x >= total ? lo : lo + plan_find(start + lo, hi - lo + 1, x);
    }
}

// Fresh table entries and tokens: thread `first` of `stride` (whole warps).
template <bool TOGETHER>
__device__ __forceinline__ void plan_fill(const PlanArgs& a, const PlanSums& s, int32_t first,
                                          int32_t stride) {
    const int32_t N = a.num_seqs, B = a.block_size;
    const int32_t lane = threadIdx.x & 31;
    for (int32_t e0 = first - lane; e0 < s.blocks; e0 += stride) {
        const int32_t e = e0 + lane;
        const int32_t i = plan_seq_of<TOGETHER, 1>(s.block_start, N, e0, e, s.blocks);
        if (e >= s.blocks) continue;
        const int32_t b0 = s.block_start[i];
        const int32_t held = s.held[i] - (s.block_start[i + 1] - b0);
        const int32_t id = plan_free(a, s.head + e);
        a.block_tables[(int64_t)i * a.max_blocks + held + (e - b0)] = id;
        if (a.ref_cnt != nullptr && id >= 0) a.ref_cnt[id] = 1;
    }
    const bool wide = ((reinterpret_cast<uintptr_t>(a.slot_mapping) |
                        reinterpret_cast<uintptr_t>(a.positions) |
                        reinterpret_cast<uintptr_t>(a.seq_ids)) & 15) == 0;
    const int32_t groups = a.max_tokens / 4 + (a.max_tokens % 4 != 0);
    for (int32_t g0 = first - lane; g0 < groups; g0 += stride) {
        const int32_t g = g0 + lane;
        const int32_t t0 = g < groups ? 4 * g : s.tokens;
        const int32_t i = plan_seq_of<TOGETHER, 4>(s.query_start, N, 4 * g0, t0, s.tokens);
        if (g >= groups) continue;
        int64_t slot[4];
        int32_t pos[4], seq[4];
        PlanSpan p{-1, 0, 0, 0, 0, 0, 0};
        int32_t block = -1, id = -1;                  // table column of `id`
        if (t0 < s.tokens) p = plan_span(s, i);
#pragma unroll
        for (int32_t u = 0; u < 4; ++u) {
            const int32_t t = t0 + u;
            slot[u] = -1;
            pos[u] = seq[u] = -1;
            if (t >= s.tokens) continue;
            while (t >= p.q1) {                       // (sequences without tokens are passed)
                p = plan_span(s, p.i + 1);
                block = -1;
            }
            pos[u] = p.pos0 + (t - p.q0);
            seq[u] = p.i;
            const int32_t b = pos[u] / B;
            if (b != block) {
                block = b;
                if (b < p.held) {
                    id = a.block_tables[(int64_t)p.i * a.max_blocks + b];
                    if (id < 0 || id >= a.num_blocks) {
                        raise_error(PA_DEVERR_TABLE_ENTRY);
                        id = -1;
                    }
                } else {
                    id = plan_free(a, s.head + p.take0 + (b - p.held));
                }
            }
            if (id >= 0) slot[u] = (int64_t)id * B + (pos[u] - b * B);
        }
        if (wide && t0 + 4 <= a.max_tokens) {
            longlong2* out = reinterpret_cast<longlong2*>(a.slot_mapping + t0);
            out[0] = make_longlong2(slot[0], slot[1]);
            out[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions != nullptr)
                *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            if (a.seq_ids != nullptr)
                *reinterpret_cast<int4*>(a.seq_ids + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        } else {
#pragma unroll
            for (int32_t u = 0; u < 4; ++u) {
                if (t0 + u >= a.max_tokens) continue;
                a.slot_mapping[t0 + u] = slot[u];
                if (a.positions != nullptr) a.positions[t0 + u] = pos[u];
                if (a.seq_ids != nullptr) a.seq_ids[t0 + u] = seq[u];
            }
        }
    }
}

// SMALL: the whole step in this CTA (num_seqs <= kPlanSmallSeqs).
template <bool SMALL>
__global__ void __launch_bounds__(kPlanScanThreads) plan_scan_kernel(const PlanArgs a) {
    __shared__ int64_t s_new[32], s_grow[32];
    __shared__ unsigned int s_bad[32];
    __shared__ int32_t s_sums[SMALL ? 4 * (kPlanSmallSeqs + 1) : 1];
    int32_t* s_query = s_sums;
    int32_t* s_block = s_query + (SMALL ? kPlanSmallSeqs + 1 : 0);
    int32_t* s_lens = s_block + (SMALL ? kPlanSmallSeqs + 1 : 0);
    int32_t* s_held = s_lens + (SMALL ? kPlanSmallSeqs + 1 : 0);
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t head = *a.free_head;
    // A round takes the next 4096 sequences (1024 in a small step), a thread
    // consecutive ones.  The first pass adds them all up: does the step fit?  A
    // batch of one round stays in registers for the second.
    constexpr int32_t kPer = SMALL ? 1 : kPlanHeld;
    const int32_t rounds = (a.num_seqs + kPer * kPlanScanThreads - 1) / (kPer * kPlanScanThreads);
    PlanSeq s[kPer];
    int64_t add = 0, grow = 0;
    unsigned int bad = 0;
    auto read = [&](int32_t round, unsigned int& why) {
#pragma unroll
        for (int32_t u = 0; u < kPer; ++u) {
            const int32_t i = (round * kPlanScanThreads + tid) * kPer + u;
            s[u] = PlanSeq{0, 0, 0, 0};
            if (i < a.num_seqs) s[u] = plan_seq(a, i, why);
        }
    };
    for (int32_t r = 0; r < rounds; ++r) {
        read(r, bad);
#pragma unroll
        for (int32_t u = 0; u < kPer; ++u) {
            add += s[u].add;
            grow += s[u].grow;
        }
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
    // running sums (fits: they stay in 32 bits)
    int32_t q0 = 0, b0 = 0;
    for (int32_t r = 0; r < rounds; ++r) {
        unsigned int ignored = 0;
        if (rounds > 1) read(r, ignored);
        int32_t mq = 0, mb = 0;
#pragma unroll
        for (int32_t u = 0; u < kPer; ++u) {
            if (!fits) s[u].add = s[u].grow = 0;
            mq += s[u].add;
            mb += s[u].grow;
        }
        int32_t qi = mq, bi = mb;
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
        int32_t q = q0 + before_q + qi - mq, b = b0 + before_b + bi - mb;
#pragma unroll
        for (int32_t u = 0; u < kPer; ++u) {
            const int32_t i = (r * kPlanScanThreads + tid) * kPer + u;
            if (i < a.num_seqs) {
                a.query_start[i] = q;
                a.block_start[i] = b;
                a.seq_lens_out[i] = s[u].len + s[u].add;
                a.blocks_held_out[i] = s[u].held + s[u].grow;
                if constexpr (SMALL) {
                    s_query[i] = q;
                    s_block[i] = b;
                    s_lens[i] = s[u].len + s[u].add;
                    s_held[i] = s[u].held + s[u].grow;
                }
                q += s[u].add;
                b += s[u].grow;
            }
        }
        q0 += __shfl_sync(0xffffffffu, wq, 31);
        b0 += __shfl_sync(0xffffffffu, wb, 31);
        __syncthreads();                          // s_new, s_grow free for the next round
    }
    if (tid == 0) {
        a.query_start[a.num_seqs] = q0;
        a.block_start[a.num_seqs] = b0;
        *a.free_head_out = head + b0;
        if constexpr (SMALL) {
            s_query[a.num_seqs] = q0;
            s_block[a.num_seqs] = b0;
        }
    }
    if constexpr (SMALL) {
        __syncthreads();
        plan_fill<false>(a, PlanSums{s_query, s_block, s_lens, s_held, q0, b0, head}, tid,
                         kPlanScanThreads);
    }
}

constexpr int kPlanFillThreads = 256;

__global__ void __launch_bounds__(kPlanFillThreads) plan_fill_kernel(const PlanArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tokens = a.query_start[a.num_seqs], blocks = a.block_start[a.num_seqs];
    plan_fill<true>(a, PlanSums{a.query_start, a.block_start, a.seq_lens_out, a.blocks_held_out,
                                tokens, blocks, *a.free_head_out - blocks},
                    blockIdx.x * kPlanFillThreads + threadIdx.x, gridDim.x * kPlanFillThreads);
}

}  // namespace pa

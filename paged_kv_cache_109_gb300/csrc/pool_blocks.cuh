// pool_blocks.cuh -- the pool's blocks on the GPU beside plan_step: blocks that
// sequences no longer need go back to the free queue (BlockPool.release), forked
// sequences share their source's blocks (BlockPool.fork; the partly filled tail is
// copied at once, as copy_on_write would before the next token).
//
// The free queue is the one plan_step takes from: free_blocks[F ..).  Blocks that come
// back are put right in front of it, first in the order of sequences and tables, so
// the queue needs no other end and what was used last is taken first.
//
// Both number a list of table entries (those dropped, those shared) over all sequences
// and give equal shares of it to the warps of one cluster.  A CTA keeps the running
// sums of a round of sequences in shared memory; a warp finds the sequences of its
// first and last of 256 entries there together, its lanes those in between.
//
// Release with reference counts: every dropped entry takes one off its block's count.
// A block that reaches none is freed once, at its last entry e in the list's order:
// its count then serves to find that entry, as the minimum of -1 - e (no workspace,
// and the order does not depend on which thread came last); the owner sets it to zero.
//
// Bound: latencies.  Measured (GPU time): a release of 1800 entries of 256 sequences 8.2 us
// (a launch, the scan, one exchange between the CTAs); of 220000 entries of 2048 sequences
// 14.8 us, of which the bytes take 0.2.  One prompt forked four times and released with
// counts 20.6 us in three launches; 96 forks of 24 prompts over 16 layers and their release
// 33 us, where the tails' rows take 15 at the copy rate.
#pragma once

#include "cluster.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "write_kv.cuh"

namespace pa {

struct ReleaseArgs {
    const int32_t* seq_lens;        // tokens that stay
    const int32_t* block_tables;
    const int32_t* blocks_held;
    int32_t* free_blocks;
    const int32_t* free_head;
    int32_t* ref_cnt;               // may be nullptr
    int32_t* blocks_held_out;       // may be blocks_held
    int32_t* free_head_out;         // may be free_head
    int32_t num_seqs, num_free, num_blocks, block_size, max_blocks;
    int32_t kept;                   // entries that a CTA has room to keep
};

struct ForkArgs {
    const int32_t* src;             // row that row i starts as a copy of, -1: none
    const int32_t* seq_lens;
    int32_t* block_tables;
    const int32_t* blocks_held;
    int32_t* ref_cnt;
    const int32_t* free_blocks;
    const int32_t* free_head;
    int32_t* seq_lens_out;          // may be seq_lens
    int32_t* blocks_held_out;       // may be blocks_held
    int32_t* free_head_out;         // may be free_head
    int64_t* block_pairs;           // [N][2] blocks to copy, -1: none
    int32_t num_seqs, num_free, num_blocks, block_size, max_blocks;
};

constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPoolPer = 4;                             // sequences a thread scans
constexpr int kPoolRound = kPoolThreads * kPoolPer;     // sequences of a round
constexpr int kPoolMaxCluster = 16;
constexpr int kPoolMaxWarps = kPoolMaxCluster * kPoolWarps;
constexpr int kPoolKept = 40960;                        // entries that a CTA keeps at most (160 KB)
constexpr int kPoolChunk = 8, kForkChunk = 4;           // entries a lane has under way

struct PoolShared {
    int32_t start[kPoolRound + 1];  // running sum of the entries, from the round's first
    int32_t first[kPoolRound];      // release: a sequence's first entry; fork: its source
    int64_t warp_a[kPoolWarps], warp_b[kPoolWarps];
    int32_t count[kPoolMaxWarps];   // freed blocks, by warp of the cluster
    unsigned int bad[kPoolMaxCluster];
    int32_t head;                   // the queue's front, from the first CTA
};

// Exclusive running sums of one or two values over the CTA's threads; the totals too.
template <bool TWO>
__device__ __forceinline__ void pool_scan(PoolShared& s, int64_t& a, int64_t& b, int64_t& sum_a,
                                          int64_t& sum_b) {
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t a0 = a, b0 = b;
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, off);
        const int64_t y = TWO ? __shfl_up_sync(0xffffffffu, b, off) : 0;
        if (lane >= off) {
            a += x;
            b += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.warp_a[warp] = a;
        if (TWO) s.warp_b[warp] = b;
    }
    __syncthreads();
    int64_t wa = s.warp_a[lane], wb = TWO ? s.warp_b[lane] : 0;
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, wa, off);
        const int64_t y = TWO ? __shfl_up_sync(0xffffffffu, wb, off) : 0;
        if (lane >= off) {
            wa += x;
            wb += y;
        }
    }
    sum_a = __shfl_sync(0xffffffffu, wa, 31);
    const int64_t ca = __shfl_sync(0xffffffffu, wa, max(warp - 1, 0));
    a += (warp ? ca : 0) - a0;
    if (TWO) {
        sum_b = __shfl_sync(0xffffffffu, wb, 31);
        const int64_t cb = __shfl_sync(0xffffffffu, wb, max(warp - 1, 0));
        b += (warp ? cb : 0) - b0;
    }
}

// The warp's word (a count, a CTA's bad bits) to every CTA of the cluster.
__device__ __forceinline__ void pool_tell(const void* at, int32_t x) {
    if ((threadIdx.x & 31) < cluster_size()) cluster_store(cluster_map(at, threadIdx.x & 31), x);
}

// Last i in [lo, hi] with start[i] <= e (start[lo] <= e), all lanes of a warp with one e.
__device__ __forceinline__ int32_t pool_find_warp(const int32_t* start, int32_t lo, int32_t hi, int32_t e) {
    while (lo < hi) {
        const int32_t step = (hi - lo + 32) / 32;
        const int32_t at = lo + ((int32_t)(threadIdx.x & 31) + 1) * step;
        const uint32_t yes = __ballot_sync(0xffffffffu, at <= hi && start[min(at, hi)] <= e);
        lo += __popc(yes) * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// The sequences of entries e0 + 32 u + lane of a round, below `end` (-1: none).
template <int CHUNK>
__device__ __forceinline__ void pool_seqs(const PoolShared& s, int32_t e0, int32_t end,
                                          int32_t (&seq)[CHUNK]) {
    const int32_t lane = threadIdx.x & 31;
    const int32_t last = min(end, e0 + 32 * CHUNK) - 1;
    const int32_t lo = pool_find_warp(s.start, 0, kPoolRound - 1, e0);
    const int32_t hi = s.start[lo + 1] > last ? lo : pool_find_warp(s.start, lo, kPoolRound - 1, last);
    int32_t top[CHUNK];
#pragma unroll
    for (int u = 0; u < CHUNK; ++u) {
        seq[u] = lo;
        top[u] = hi;
    }
    // (a lane's searches go on side by side)
    for (int32_t left = hi - lo; left > 0; left >>= 1) {
#pragma unroll
        for (int u = 0; u < CHUNK; ++u) {
            const int32_t mid = (seq[u] + top[u] + 1) / 2;
            if (s.start[mid] <= e0 + 32 * u + lane) seq[u] = mid; else top[u] = mid - 1;
        }
    }
#pragma unroll
    for (int u = 0; u < CHUNK; ++u)
        if (e0 + 32 * u + lane >= end) seq[u] = -1;
}

// ---- release -------------------------------------------------------------------------

struct ReleaseSeq {
    int32_t keep, held;             // entries [keep, held) are dropped
};

__device__ __forceinline__ ReleaseSeq release_seq(const ReleaseArgs& a, int32_t i, unsigned int& bad) {
    const int32_t len = a.seq_lens[i], held = a.blocks_held[i];
    const int64_t keep = ((int64_t)len + a.block_size - 1) / a.block_size;
    if (len < 0 || held < 0 || held > a.max_blocks || keep > held) {
        bad |= PA_DEVERR_SEQ_LEN;
        return {0, 0};
    }
    return {(int32_t)keep, held};
}

// The round's entries into s.start and s.first; how many there are.
__device__ __forceinline__ int64_t release_round(PoolShared& s, const ReleaseArgs& a, int32_t i0,
                                                 unsigned int& bad) {
    ReleaseSeq q[kPoolPer];
    int64_t mine = 0, none = 0, total, ignored;
#pragma unroll
    for (int u = 0; u < kPoolPer; ++u) {
        const int32_t i = i0 + (int32_t)threadIdx.x * kPoolPer + u;
        q[u] = ReleaseSeq{0, 0};
        if (i < a.num_seqs) q[u] = release_seq(a, i, bad);
        mine += q[u].held - q[u].keep;
    }
    pool_scan<false>(s, mine, none, total, ignored);
#pragma unroll
    for (int u = 0; u < kPoolPer; ++u) {
        const int32_t x = (int32_t)threadIdx.x * kPoolPer + u;
        s.start[x] = (int32_t)mine;
        s.first[x] = q[u].keep;
        mine += q[u].held - q[u].keep;
    }
    if (threadIdx.x == 0) s.start[kPoolRound] = (int32_t)total;
    __syncthreads();
    return total;
}

template <bool COUNTED>
__global__ void __launch_bounds__(kPoolThreads) release_blocks_kernel(const ReleaseArgs a) {
    extern __shared__ int32_t s_ids[];  // [a.kept]: the CTA's entries, where they fit
    __shared__ PoolShared s;
    griddep_wait();
    griddep_launch_dependents();
    cluster_arrive();                   // this CTA runs
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const int32_t rank = (int32_t)cluster_rank(), ctas = (int32_t)cluster_size();
    const int32_t warp = rank * kPoolWarps + (tid >> 5), warps = ctas * kPoolWarps;   // of the cluster
    int32_t head = *a.free_head;
    const int32_t rounds = (a.num_seqs + kPoolRound - 1) / kPoolRound;
    unsigned int bad = 0;
    int64_t total = 0;
    for (int32_t r = 0; r < rounds; ++r) total += release_round(s, a, r * kPoolRound, bad);
    bad = __syncthreads_or(bad) ? PA_DEVERR_SEQ_LEN : 0;
    if (head < 0 || head > a.num_free) bad |= PA_DEVERR_POOL;
    if (total > INT32_MAX / 2) bad |= PA_DEVERR_SEQ_LEN;
    const bool off = bad != 0;          // (as this CTA sees it)

    // Entries [e0, e1) of the list are this warp's: f(e, id, in) for 32 at a time, in
    // order, all lanes together (in: the lane has one; id: -1 for none or a bad one).
    const int64_t per = (((total + warps - 1) / warps) + 31) / 32 * 32;
    const int64_t e0 = min(total, warp * per), e1 = off ? e0 : min(total, e0 + per);
    const bool keep = per * kPoolWarps <= a.kept;
    int32_t* const ids = s_ids + (keep ? (tid >> 5) * per : 0);
    bool have = false;
    auto each = [&](auto f) {
        int64_t base = 0;
        for (int32_t r = 0; r < rounds; ++r) {
            unsigned int ignored = 0;
            if (rounds > 1 && !(keep && have)) {
                __syncthreads();
                release_round(s, a, r * kPoolRound, ignored);
            }
            const bool again = keep && have;
            if (again && r > 0) break;  // (all rounds at once)
            const int64_t n = again ? total : s.start[kPoolRound], end = min(base + n, e1);
            for (int64_t t = max(base, e0); t < end; t += 32 * kPoolChunk) {
                int32_t id[kPoolChunk];
                if (again) {
#pragma unroll
                    for (int u = 0; u < kPoolChunk; ++u)
                        id[u] = t + 32 * u + lane < end ? ids[t - e0 + 32 * u + lane] : -1;
                } else {
                    int32_t seq[kPoolChunk];
                    pool_seqs(s, (int32_t)(t - base), (int32_t)(end - base), seq);
#pragma unroll
                    for (int u = 0; u < kPoolChunk; ++u) {
                        const int32_t x = (int32_t)(t - base) + 32 * u + lane;
                        id[u] = -1;
                        if (seq[u] >= 0)
                            id[u] = a.block_tables[(int64_t)(r * kPoolRound + seq[u]) * a.max_blocks +
                                                   s.first[seq[u]] + (x - s.start[seq[u]])];
                    }
#pragma unroll
                    for (int u = 0; u < kPoolChunk; ++u)
                        if (keep && seq[u] >= 0) ids[t - e0 + 32 * u + lane] = id[u];
                }
#pragma unroll
                for (int u = 0; u < kPoolChunk; ++u) {
                    const int64_t e = t + 32 * u + lane;
                    if (t + 32 * u >= end) break;
                    const bool there = e < end && id[u] >= 0 && id[u] < a.num_blocks;
                    f((int32_t)e, there ? id[u] : -1, e < end);
                }
            }
            base += n;
        }
        have = true;
    };
    auto undo = [&]() {
        each([&](int32_t, int32_t id, bool) {
            if (id >= 0) atomicAdd(&a.ref_cnt[id], 1);
        });
    };
    cluster_wait();                     // all CTAs run: their shared memory is there
    if constexpr (COUNTED) {
        unsigned int over = 0;
        each([&](int32_t, int32_t id, bool) {
            if (id >= 0 && atomicSub(&a.ref_cnt[id], 1) <= 0) over = PA_DEVERR_SHARED;
        });
        bad |= __syncthreads_or(over) ? PA_DEVERR_SHARED : 0;
        if (tid < 32) pool_tell(&s.bad[rank], (int32_t)bad);
        if (rank == 0 && tid < 32) pool_tell(&s.head, head);
        cluster_sync();
        for (int32_t c = 0; c < ctas; ++c) bad |= s.bad[c];
        if (bad)
            undo();
        else
            each([&](int32_t e, int32_t id, bool) {
                if (id >= 0 && __ldcg(&a.ref_cnt[id]) <= 0) atomicMin(&a.ref_cnt[id], -1 - e);
            });
        cluster_sync();
    }
    auto owns = [&](int32_t e, int32_t id) {
        return id >= 0 && (!COUNTED || __ldcg(&a.ref_cnt[id]) == -1 - e);
    };
    int32_t mine = 0;
    if (bad == 0)
        each([&](int32_t e, int32_t id, bool in) {
            if (in && id < 0) raise_error(PA_DEVERR_TABLE_ENTRY);
            mine += __popc(__ballot_sync(0xffffffffu, owns(e, id)));
        });
    pool_tell(&s.count[warp], mine);
    if (!COUNTED && tid < 32) pool_tell(&s.bad[rank], (int32_t)bad);
    if (!COUNTED && rank == 0 && tid < 32) pool_tell(&s.head, head);
    cluster_sync();
    head = s.head;                      // (all CTAs decide by the same numbers)
    if (!COUNTED)
        for (int32_t c = 0; c < ctas; ++c) bad |= s.bad[c];
    int32_t freed = 0, before = 0;
    for (int32_t w = lane; w < warps; w += 32) {
        const int32_t n = s.count[w];
        freed += n;
        before += w < warp ? n : 0;
    }
    freed = __reduce_add_sync(0xffffffffu, freed);
    before = __reduce_add_sync(0xffffffffu, before);
    if (bad == 0 && freed > head) {
        bad = PA_DEVERR_POOL;
        if constexpr (COUNTED) {
            each([&](int32_t e, int32_t id, bool) {
                if (owns(e, id)) a.ref_cnt[id] = 0;
            });
            cluster_sync();
            undo();
        }
    } else if (bad == 0) {
        int32_t at = head - freed + before;
        each([&](int32_t e, int32_t id, bool) {
            const bool own = owns(e, id);
            const uint32_t mask = __ballot_sync(0xffffffffu, own);
            const int32_t to = at + __popc(mask & ((1u << lane) - 1));
            if (own) {
                // (behind the front only where somebody writes the inputs meanwhile)
                if (to < head) a.free_blocks[to] = id;
                if (COUNTED) a.ref_cnt[id] = 0;
            }
            at += __popc(mask);
        });
    }
    if (rank == 0 && tid == 0 && bad) raise_error(bad);
    if (rounds > 1) cluster_sync();     // the inputs have been read: they may be the outputs
    for (int32_t i = rank * kPoolThreads + tid; i < a.num_seqs; i += ctas * kPoolThreads) {
        unsigned int ignored = 0;
        const int32_t held = a.blocks_held[i];
        a.blocks_held_out[i] = bad ? held : release_seq(a, i, ignored).keep;
    }
    if (rank == 0 && tid == 0) *a.free_head_out = head - (bad ? 0 : freed);
}

// ---- fork ------------------------------------------------------------------------------

// Row i of a fork: its source's tokens and full blocks.
struct ForkSeq {
    int32_t src, len, full, tail;   // src < 0: not forked; tail: a partly filled block
};

__device__ __forceinline__ ForkSeq fork_seq(const ForkArgs& a, int32_t i, unsigned int& bad) {
    const int32_t p = a.src[i];
    if (p < 0) return {-1, 0, 0, 0};
    if (p >= a.num_seqs || a.blocks_held[i] != 0 || a.src[p] >= 0) {
        bad |= PA_DEVERR_FORK;
        return {-1, 0, 0, 0};
    }
    const int32_t len = a.seq_lens[p], held = a.blocks_held[p];
    if (len < 0 || held < 0 || held > a.max_blocks ||
        ((int64_t)len + a.block_size - 1) / a.block_size > held) {
        bad |= PA_DEVERR_SEQ_LEN;
        return {-1, 0, 0, 0};
    }
    return {p, len, len / a.block_size, len % a.block_size != 0};
}

// The round's shared entries into s; how many there are, and the fresh blocks before
// this thread's first sequence in `take`.
__device__ __forceinline__ int64_t fork_round(PoolShared& s, const ForkArgs& a, int32_t i0,
                                              unsigned int& bad, ForkSeq (&q)[kPoolPer],
                                              int64_t& take, int64_t& fresh) {
    int64_t mine = 0, total;
    take = 0;
#pragma unroll
    for (int u = 0; u < kPoolPer; ++u) {
        const int32_t i = i0 + (int32_t)threadIdx.x * kPoolPer + u;
        q[u] = ForkSeq{-1, 0, 0, 0};
        if (i < a.num_seqs) q[u] = fork_seq(a, i, bad);
        mine += q[u].full;
        take += q[u].tail;
    }
    pool_scan<true>(s, mine, take, total, fresh);
#pragma unroll
    for (int u = 0; u < kPoolPer; ++u) {
        const int32_t x = (int32_t)threadIdx.x * kPoolPer + u;
        s.start[x] = (int32_t)mine;
        s.first[x] = q[u].src;
        mine += q[u].full;
    }
    if (threadIdx.x == 0) s.start[kPoolRound] = (int32_t)total;
    __syncthreads();
    return total;
}

// (Every CTA finds out by itself whether the call can be done, and its one cluster
// barrier is met on every path.)
__global__ void __launch_bounds__(kPoolThreads) fork_blocks_kernel(const ForkArgs a) {
    __shared__ PoolShared s;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const int32_t rank = (int32_t)cluster_rank(), ctas = (int32_t)cluster_size();
    const int32_t warp = rank * kPoolWarps + (tid >> 5), warps = ctas * kPoolWarps;   // of the cluster
    const int32_t head = *a.free_head;
    const int32_t rounds = (a.num_seqs + kPoolRound - 1) / kPoolRound;
    unsigned int bad = 0;
    int64_t total = 0, fresh = 0, take = 0, more = 0;
    ForkSeq q[kPoolPer];
    for (int32_t r = 0; r < rounds; ++r) {
        total += fork_round(s, a, r * kPoolRound, bad, q, take, more);
        fresh += more;
    }
    bad = (__syncthreads_or(bad & PA_DEVERR_FORK) ? PA_DEVERR_FORK : 0) |
          (__syncthreads_or(bad & PA_DEVERR_SEQ_LEN) ? PA_DEVERR_SEQ_LEN : 0);
    if (bad == 0 && (head < 0 || head + fresh > a.num_free)) bad = PA_DEVERR_POOL;
    if (bad == 0 && total > INT32_MAX / 2) bad = PA_DEVERR_SEQ_LEN;
    if (bad && rank == 0 && tid == 0) raise_error(bad);
    // (what a row becomes is read before any output is written: they may be the inputs)
    auto becomes = [&](int32_t i, int32_t& len, int32_t& held) {
        const int32_t p = a.src[i];
        const int32_t from = bad || p < 0 || p >= a.num_seqs ? i : p;
        len = a.seq_lens[from];
        held = from == i ? a.blocks_held[i] : (int32_t)(((int64_t)len + a.block_size - 1) / a.block_size);
    };
    const int32_t own = rank * kPoolThreads + tid;
    int32_t len0 = 0, held0 = 0;
    if (rounds <= 1) {
        if (own < a.num_seqs) becomes(own, len0, held0);
        cluster_arrive();
    }

    const int64_t per = (((total + warps - 1) / warps) + 31) / 32 * 32;
    const int64_t e0 = min(total, warp * per), e1 = min(total, e0 + per);
    int64_t base = 0, taken = 0;
    for (int32_t r = 0; r < rounds; ++r) {
        unsigned int ignored = 0;
        if (rounds > 1) {
            __syncthreads();
            fork_round(s, a, r * kPoolRound, ignored, q, take, more);
        }
        const int64_t n = s.start[kPoolRound], end = bad ? 0 : min(base + n, e1);
        // tails
        if (rank == 0) {
            int64_t at = head + taken + take;
            int32_t old[kPoolPer], id[kPoolPer];
#pragma unroll
            for (int u = 0; u < kPoolPer; ++u) {
                old[u] = id[u] = -1;
                if (!bad && q[u].tail) {
                    old[u] = a.block_tables[(int64_t)q[u].src * a.max_blocks + q[u].full];
                    id[u] = at < a.num_free ? a.free_blocks[at] : -1;
                    ++at;
                }
            }
#pragma unroll
            for (int u = 0; u < kPoolPer; ++u) {
                const int32_t i = r * kPoolRound + tid * kPoolPer + u;
                if (i >= a.num_seqs) continue;
                int64_t from = -1, to = -1;
                if (!bad && q[u].tail) {
                    const bool ok = id[u] >= 0 && id[u] < a.num_blocks;
                    a.block_tables[(int64_t)i * a.max_blocks + q[u].full] = ok ? id[u] : -1;
                    if (ok) a.ref_cnt[id[u]] = 1;
                    if (!ok || old[u] < 0 || old[u] >= a.num_blocks) {
                        raise_error(PA_DEVERR_TABLE_ENTRY);
                    } else {
                        from = old[u];
                        to = id[u];
                    }
                }
                a.block_pairs[2 * (int64_t)i] = from;
                a.block_pairs[2 * (int64_t)i + 1] = to;
            }
        }
        // shared entries
        for (int64_t t = max(base, e0); t < end; t += 32 * kForkChunk) {
            int32_t seq[kForkChunk], id[kForkChunk];
            pool_seqs(s, (int32_t)(t - base), (int32_t)(end - base), seq);
#pragma unroll
            for (int u = 0; u < kForkChunk; ++u) {
                const int32_t x = (int32_t)(t - base) + 32 * u + lane;
                if (seq[u] >= 0)
                    id[u] = a.block_tables[(int64_t)s.first[seq[u]] * a.max_blocks + x - s.start[seq[u]]];
            }
#pragma unroll
            for (int u = 0; u < kForkChunk; ++u) {
                const int32_t x = (int32_t)(t - base) + 32 * u + lane;
                if (seq[u] < 0) continue;
                a.block_tables[(int64_t)(r * kPoolRound + seq[u]) * a.max_blocks + x - s.start[seq[u]]] = id[u];
                if (id[u] >= 0 && id[u] < a.num_blocks)
                    atomicAdd(&a.ref_cnt[id[u]], 1);
                else
                    raise_error(PA_DEVERR_TABLE_ENTRY);
            }
        }
        base += n;
        taken += more;
    }
    if (rounds <= 1)
        cluster_wait();
    else
        cluster_sync();
    // (a source's row is no fork, so its length stays what it is)
    for (int32_t i = own; i < a.num_seqs; i += ctas * kPoolThreads) {
        int32_t len = len0, held = held0;
        if (rounds > 1 || i != own) becomes(i, len, held);
        a.seq_lens_out[i] = len;
        a.blocks_held_out[i] = held;
    }
    if (rank == 0 && tid == 0) *a.free_head_out = head + (bad ? 0 : (int32_t)fresh);
}

// K and V rows of the tails that fork_blocks_kernel paired: of block pair i the first
// seq_lens_out[i] % B rows of every kv head, in one cache.  One CTA per (sequence,
// layer, K or V).
constexpr int kForkThreads = 128;
constexpr int kForkLayers = 128;    // layers of one launch
constexpr int kForkUnroll = 4;

template <int LAYERS>
struct ForkCaches {
    uint8_t* k[LAYERS];
    uint8_t* v[LAYERS];
};

template <int VEC, int LAYERS>
__global__ void __launch_bounds__(kForkThreads)
fork_copy_kernel(const ForkArgs a, int32_t num_kv_heads, int32_t row_bytes,
                 const __grid_constant__ ForkCaches<LAYERS> caches) {
    using V = typename VecType<VEC>::T;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t i = blockIdx.x;
    const int64_t src = a.block_pairs[2 * (int64_t)i], dst = a.block_pairs[2 * (int64_t)i + 1];
    if (src < 0 || dst < 0 || src >= a.num_blocks || dst >= a.num_blocks) return;
    const int32_t rows = max(a.seq_lens_out[i], 0) % a.block_size;
    uint8_t* cache = (blockIdx.y & 1) ? caches.v[blockIdx.y >> 1] : caches.k[blockIdx.y >> 1];
    const int64_t head_bytes = (int64_t)a.block_size * row_bytes;
    const int64_t block_bytes = num_kv_heads * head_bytes;
    const uint8_t* from = cache + src * block_bytes;
    uint8_t* to = cache + dst * block_bytes;
    const int64_t vecs = (int64_t)rows * row_bytes / VEC;        // of one head
    const int64_t total = num_kv_heads * vecs;
    if (total <= INT32_MAX / 2) {
        const uint32_t per = (uint32_t)vecs, all = (uint32_t)total;
        for (uint32_t x0 = threadIdx.x; x0 < all; x0 += kForkUnroll * kForkThreads) {
            V buf[kForkUnroll];
            int64_t off[kForkUnroll];
#pragma unroll
            for (int u = 0; u < kForkUnroll; ++u) {
                const uint32_t x = x0 + u * kForkThreads, h = x / per;
                off[u] = h * head_bytes + (int64_t)(x - h * per) * VEC;
                if (x < all) buf[u] = *reinterpret_cast<const V*>(from + off[u]);
            }
#pragma unroll
            for (int u = 0; u < kForkUnroll; ++u)
                if (x0 + u * kForkThreads < all) *reinterpret_cast<V*>(to + off[u]) = buf[u];
        }
    } else {
        for (int64_t x = threadIdx.x; x < total; x += kForkThreads) {
            const int64_t off = x / vecs * head_bytes + x % vecs * VEC;
            *reinterpret_cast<V*>(to + off) = *reinterpret_cast<const V*>(from + off);
        }
    }
}

}  // namespace pa

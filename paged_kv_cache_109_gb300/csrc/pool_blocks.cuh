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
// and give equal shares of it to the CTAs of one cluster.  A CTA keeps the running
// sums of a round of sequences in shared memory and finds an entry's sequence there.
//
// Release with reference counts: every dropped entry takes one off its block's count.
// A block that reaches none is freed once, at its last entry e in the list's order:
// its count then serves to find that entry, as the minimum of -1 - e (no workspace,
// and the order does not depend on which thread came last); the owner sets it to zero.
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
constexpr int kPoolPer = 4;                             // sequences a thread scans
constexpr int kPoolRound = kPoolThreads * kPoolPer;     // sequences of a round
constexpr int kPoolMaxCluster = 8;

struct PoolShared {
    int32_t start[kPoolRound + 1];  // running sum of the entries, from the round's first
    int32_t first[kPoolRound];      // release: a sequence's first entry; fork: its source
    int64_t warp_a[32], warp_b[32];
    unsigned int bad;
    int64_t from_cta[2][kPoolMaxCluster];
};

// Exclusive running sums of two values over the CTA's threads; the totals too.
__device__ __forceinline__ void pool_scan(PoolShared& s, int64_t& a, int64_t& b, int64_t& sum_a,
                                          int64_t& sum_b) {
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t a0 = a, b0 = b;
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) {
            a += x;
            b += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.warp_a[warp] = a;
        s.warp_b[warp] = b;
    }
    __syncthreads();
    int64_t wa = s.warp_a[lane], wb = s.warp_b[lane];
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, wa, off), y = __shfl_up_sync(0xffffffffu, wb, off);
        if (lane >= off) {
            wa += x;
            wb += y;
        }
    }
    sum_a = __shfl_sync(0xffffffffu, wa, 31);
    sum_b = __shfl_sync(0xffffffffu, wb, 31);
    const int64_t ca = __shfl_sync(0xffffffffu, wa, max(warp - 1, 0));
    const int64_t cb = __shfl_sync(0xffffffffu, wb, max(warp - 1, 0));
    a += (warp ? ca : 0) - a0;
    b += (warp ? cb : 0) - b0;
}

// x of every CTA of the cluster, by rank (turn: 0 and 1 in turn).
__device__ __forceinline__ const int64_t* pool_exchange(PoolShared& s, int32_t turn, int64_t x) {
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    if (threadIdx.x < ctas)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                         cluster_map(&s.from_cta[turn & 1][rank], threadIdx.x)), "l"(x)
                     : "memory");
    cluster_sync();
    return s.from_cta[turn & 1];
}

// Sequence of entry e of the round (s.start[0] <= e < s.start[n]).
__device__ __forceinline__ int32_t pool_find(const PoolShared& s, int32_t n, int32_t e) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (s.start[mid] <= e) lo = mid; else hi = mid - 1;
    }
    return lo;
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

// The round's entries into s.start and s.first; their number and how many there are.
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
    pool_scan(s, mine, none, total, ignored);
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

__global__ void __launch_bounds__(kPoolThreads) release_blocks_kernel(const ReleaseArgs a) {
    __shared__ PoolShared s;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x;
    const int32_t rank = (int32_t)cluster_rank(), ctas = (int32_t)cluster_size();
    const int32_t head = *a.free_head;
    const int32_t rounds = (a.num_seqs + kPoolRound - 1) / kPoolRound;
    unsigned int bad = 0;
    int64_t total = 0;
    if (tid == 0) s.bad = 0;
    for (int32_t r = 0; r < rounds; ++r) total += release_round(s, a, r * kPoolRound, bad);
    __syncthreads();
    if (bad) atomicOr(&s.bad, bad);
    __syncthreads();
    bad = s.bad;
    if (head < 0 || head > a.num_free) bad |= PA_DEVERR_POOL;
    if (total > INT32_MAX / 2) bad |= PA_DEVERR_SEQ_LEN;
    cluster_sync();                     // all CTAs run
    int32_t turn = 0;
    // (the first CTA's word goes, whatever happens to the inputs meanwhile)
    bad = (unsigned int)pool_exchange(s, turn++, bad)[0];

    // Entries [e0, e1) of the list are this CTA's: f(e, id, there) for each, tiles of
    // the CTA in order (there: this thread has one, with a valid id).
    const int64_t per = (total + ctas - 1) / ctas;
    const int64_t e0 = min(total, rank * per), e1 = min(total, e0 + per);
    auto each = [&](auto f) {
        int64_t base = 0;
        for (int32_t r = 0; r < rounds; ++r) {
            unsigned int ignored = 0;
            if (rounds > 1) {
                __syncthreads();
                release_round(s, a, r * kPoolRound, ignored);
            }
            const int64_t n = s.start[kPoolRound];
            const int64_t end = min(base + n, e1);
            for (int64_t t = max(base, e0); t < end; t += kPoolThreads) {
                const int64_t e = t + tid;
                int32_t id = -1;
                if (e < end) {
                    const int32_t x = (int32_t)(e - base), i = pool_find(s, kPoolRound, x);
                    id = a.block_tables[(int64_t)(r * kPoolRound + i) * a.max_blocks + s.first[i] + (x - s.start[i])];
                }
                f((int32_t)e, id, e < end && id >= 0 && id < a.num_blocks, e < end);
            }
            base += n;
        }
    };
    auto undo = [&]() {
        each([&](int32_t, int32_t id, bool there, bool) {
            if (there) atomicAdd(&a.ref_cnt[id], 1);
        });
    };
    int64_t freed = 0;
    if (bad == 0 && a.ref_cnt != nullptr) {
        unsigned int over = 0;
        each([&](int32_t, int32_t id, bool there, bool) {
            if (there && atomicSub(&a.ref_cnt[id], 1) <= 0) over = PA_DEVERR_SHARED;
        });
        over = __syncthreads_or(over) ? PA_DEVERR_SHARED : 0;
        const int64_t* all = pool_exchange(s, turn++, over);
        for (int32_t c = 0; c < ctas; ++c) bad |= (unsigned int)all[c];
        if (bad) {
            undo();
        } else {
            each([&](int32_t e, int32_t id, bool there, bool) {
                if (there && __ldcg(&a.ref_cnt[id]) <= 0) atomicMin(&a.ref_cnt[id], -1 - e);
            });
        }
        cluster_sync();
    }
    auto owns = [&](int32_t e, int32_t id, bool there) {
        return there && (a.ref_cnt == nullptr || __ldcg(&a.ref_cnt[id]) == -1 - e);
    };
    if (bad == 0) {
        int32_t mine = 0;
        each([&](int32_t e, int32_t id, bool there, bool in) {
            if (in && !there) raise_error(PA_DEVERR_TABLE_ENTRY);
            mine += owns(e, id, there);
        });
        int64_t x = mine, none = 0, sum, ignored;
        pool_scan(s, x, none, sum, ignored);
        const int64_t* all = pool_exchange(s, turn++, sum);
        int64_t before = 0;
        for (int32_t c = 0; c < ctas; ++c) {
            if (c < rank) before += all[c];
            freed += all[c];
        }
        if (freed > head) {
            bad = PA_DEVERR_POOL;
            if (a.ref_cnt != nullptr) {
                each([&](int32_t e, int32_t id, bool there, bool) {
                    if (owns(e, id, there)) a.ref_cnt[id] = 0;
                });
                cluster_sync();
                undo();
            }
            freed = 0;
        } else {
            int64_t at = head - freed + before;
            each([&](int32_t e, int32_t id, bool there, bool) {
                const bool own = owns(e, id, there);
                int64_t rank_in = own, zero = 0, got, none2;
                pool_scan(s, rank_in, zero, got, none2);
                if (own) {
                    a.free_blocks[at + rank_in] = id;
                    if (a.ref_cnt != nullptr) a.ref_cnt[id] = 0;
                }
                at += got;
            });
        }
    }
    if (rank == 0 && tid == 0 && bad) raise_error(bad);
    cluster_sync();                     // the inputs have been read: they may be the outputs
    for (int32_t i = rank * kPoolThreads + tid; i < a.num_seqs; i += ctas * kPoolThreads) {
        unsigned int ignored = 0;
        const int32_t held = a.blocks_held[i];
        a.blocks_held_out[i] = bad ? held : release_seq(a, i, ignored).keep;
    }
    if (rank == 0 && tid == 0) *a.free_head_out = head - (int32_t)freed;
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

// The round's shared entries into s; their number, and the fresh blocks before each
// of this thread's sequences in `take`.
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
    pool_scan(s, mine, take, total, fresh);
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

__global__ void __launch_bounds__(kPoolThreads) fork_blocks_kernel(const ForkArgs a) {
    __shared__ PoolShared s;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x;
    const int32_t rank = (int32_t)cluster_rank(), ctas = (int32_t)cluster_size();
    const int32_t head = *a.free_head;
    const int32_t rounds = (a.num_seqs + kPoolRound - 1) / kPoolRound;
    unsigned int bad = 0;
    int64_t total = 0, fresh = 0, take, more;
    ForkSeq q[kPoolPer];
    if (tid == 0) s.bad = 0;
    for (int32_t r = 0; r < rounds; ++r) {
        total += fork_round(s, a, r * kPoolRound, bad, q, take, more);
        fresh += more;
    }
    __syncthreads();
    if (bad) atomicOr(&s.bad, bad);
    __syncthreads();
    bad = s.bad;
    if (bad == 0 && (head < 0 || head + fresh > a.num_free)) bad = PA_DEVERR_POOL;
    if (bad == 0 && total > INT32_MAX / 2) bad = PA_DEVERR_SEQ_LEN;
    cluster_sync();                     // all CTAs run
    bad = (unsigned int)pool_exchange(s, 0, bad)[0];
    if (bad && rank == 0 && tid == 0) raise_error(bad);

    const int64_t per = (total + ctas - 1) / ctas;
    const int64_t e0 = min(total, rank * per), e1 = min(total, e0 + per);
    int64_t base = 0, taken = 0;
    for (int32_t r = 0; r < rounds; ++r) {
        unsigned int ignored = 0;
        if (rounds > 1) {
            __syncthreads();
            fork_round(s, a, r * kPoolRound, ignored, q, take, more);
        }
        const int64_t n = s.start[kPoolRound], end = bad ? 0 : min(base + n, e1);
        // shared entries
        for (int64_t e = max(base, e0) + tid; e < end; e += kPoolThreads) {
            const int32_t x = (int32_t)(e - base), i = pool_find(s, kPoolRound, x);
            const int32_t b = x - s.start[i];
            const int32_t id = a.block_tables[(int64_t)s.first[i] * a.max_blocks + b];
            a.block_tables[(int64_t)(r * kPoolRound + i) * a.max_blocks + b] = id;
            if (id >= 0 && id < a.num_blocks)
                atomicAdd(&a.ref_cnt[id], 1);
            else
                raise_error(PA_DEVERR_TABLE_ENTRY);
        }
        // tails, lengths
        if (rank == 0) {
            int64_t at = head + taken + take;
#pragma unroll
            for (int u = 0; u < kPoolPer; ++u) {
                const int32_t i = r * kPoolRound + tid * kPoolPer + u;
                if (i >= a.num_seqs) continue;
                int64_t from = -1, to = -1;
                if (!bad && q[u].tail) {
                    const int32_t old = a.block_tables[(int64_t)q[u].src * a.max_blocks + q[u].full];
                    int32_t id = a.free_blocks[at++];
                    const bool ok = id >= 0 && id < a.num_blocks;
                    if (!ok) id = -1;
                    a.block_tables[(int64_t)i * a.max_blocks + q[u].full] = id;
                    if (ok) a.ref_cnt[id] = 1;
                    if (!ok || old < 0 || old >= a.num_blocks) {
                        raise_error(PA_DEVERR_TABLE_ENTRY);
                    } else {
                        from = old;
                        to = id;
                    }
                }
                a.block_pairs[2 * (int64_t)i] = from;
                a.block_pairs[2 * (int64_t)i + 1] = to;
            }
        }
        base += n;
        taken += more;
    }
    cluster_sync();                     // the inputs have been read: they may be the outputs
    // (a source's row is no fork, so nobody writes the length read here)
    for (int32_t i = rank * kPoolThreads + tid; i < a.num_seqs; i += ctas * kPoolThreads) {
        const int32_t p = a.src[i];
        const int32_t from = bad || p < 0 ? i : p;
        const int32_t len = a.seq_lens[from];
        const int32_t held = from == i ? a.blocks_held[i]
                                       : (int32_t)(((int64_t)len + a.block_size - 1) / a.block_size);
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
    const int64_t from = a.block_pairs[2 * (int64_t)i], to = a.block_pairs[2 * (int64_t)i + 1];
    if (from < 0 || to < 0) return;
    const int32_t rows = a.seq_lens_out[i] % a.block_size;
    uint8_t* cache = (blockIdx.y & 1) ? caches.v[blockIdx.y >> 1] : caches.k[blockIdx.y >> 1];
    const int64_t head_bytes = (int64_t)a.block_size * row_bytes;
    const int64_t block_bytes = num_kv_heads * head_bytes;
    const int32_t vecs = (int32_t)((int64_t)rows * row_bytes / VEC);      // of one head
    for (int64_t x = threadIdx.x; x < (int64_t)num_kv_heads * vecs; x += kForkThreads) {
        const int64_t h = x / vecs, c = x - h * vecs;
        const int64_t off = h * head_bytes + c * VEC;
        *reinterpret_cast<V*>(cache + to * block_bytes + off) =
            *reinterpret_cast<const V*>(cache + from * block_bytes + off);
    }
}

}  // namespace pa

// verify_tree.cuh -- which drafted tokens hold against the target's probabilities,
// and the token that follows the last of them, from given random numbers.
//
// At a node with target row l and draft row d, temperature T,
//   P = softmax(l / T), q = softmax(d / T),
// its children's tokens t_1, t_2, ... (drawn from q) are tried in order with their
// uniforms u: token t holds iff
//   u q(t) S < max(P(t) - c q(t), 0),          c = 0 and S = 1 for the first,
// and after one that fails c grows by S, S = sum_x max(P(x) - c q(x), 0): what is left
// of P once the earlier tries are taken out (trying again from the rest r = max(P - c q,
// 0) / S subtracts S q from it, so the rests stay of this form).  A child that holds
// is the next node; where none does, the next token is drawn from the rest as
// argmax_x r(x) / e(x) with exponential e.  So the next token and the tokens that
// hold have the target's distribution.  Without draft rows, q is one at the child's
// token: a failed token leaves P.  T <= 0: all of P is on its first largest logit.
//
// Only rows on the path are read, so a walk of a few steps instead of all rows: one
// cluster a sequence, its CTAs with a share of the vocabulary each.  A step reads the
// node's rows once (largest logit, sum of exponentials, by the running maximum), the
// CTAs exchange their parts through shared memory, and each takes the same decision
// from the same numbers.  (What decides is exchanged too, so that the CTAs stay
// together even where somebody writes the inputs meanwhile.)
#pragma once

#include "cluster.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace pa {

struct VerifyArgs {
    const void* logits;             // [total_q][vocab]
    const void* draft;              // the same or nullptr
    int64_t logit_stride, draft_stride, noise_stride;   // elements from row to row
    const int32_t* tokens;          // [total_q]
    const int32_t* parents;         // [total_q]
    const int32_t* query_start;     // [N + 1]
    const float* uniforms;          // [total_q]
    const float* noise;             // [N][vocab]
    const float* temperature;       // [N] or nullptr
    int32_t* leaf;                  // [N]
    int32_t* next;                  // [N]
    int32_t total_q, max_q_len, vocab;
};

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;

// What a CTA tells the others.
struct VerifyPart {
    float top, draft_top;           // largest logit of its share
    double sum, draft_sum;          // sum of exponentials, relative to it
    int32_t index;                  // of `top` (greedy), of the best (next token)
};

struct VerifyShared {
    VerifyPart part[2][kVerifyMaxCluster];
    double chance[PA_MAX_TREE_NODES], draft_chance[PA_MAX_TREE_NODES];   // of a node's token
    float logit[PA_MAX_TREE_NODES], draft_logit[PA_MAX_TREE_NODES];
    float uniform[PA_MAX_TREE_NODES];
    int32_t token[PA_MAX_TREE_NODES], parent[PA_MAX_TREE_NODES];
    uint32_t child[PA_MAX_TREE_NODES / 32];      // children of the current node
    int32_t first, nodes;                        // rows of the sequence (nodes -1: refused)
    float heat;
    double warp_sum[kVerifyWarps];
    float warp_top[kVerifyWarps];
    int32_t warp_index[kVerifyWarps];
    int32_t verdict, tried;                      // of the current node
    float spent;
};

// 8 elements from p on, -inf past `count`.
template <typename E, bool WIDE>
__device__ __forceinline__ void load8(const E* p, int32_t count, float (&x)[8]) {
    if (WIDE && count >= 8) {
        if constexpr (sizeof(E) == 2) {
            const uint4 r = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4 a = reinterpret_cast<const float4*>(p)[0];
            const float4 b = reinterpret_cast<const float4*>(p)[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < count ? Elem<E>::to_float(p[i]) : -INFINITY;
    }
}

// The largest and its sum of exponentials over a share of a row.  A NaN or +inf
// makes the sum NaN.
template <typename E, bool WIDE>
__device__ __forceinline__ void row_sum(const E* row, int32_t lo, int32_t hi, float scale,
                                        float& top, float& sum) {
    top = -INFINITY;
    sum = 0.f;
    for (int32_t o = lo + 8 * (int32_t)threadIdx.x; o < hi; o += 8 * kVerifyThreads) {
        float x[8];
        load8<E, WIDE>(row + o, hi - o, x);
        float m = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = fmaxf(m, x[i]);
        if (m > top) {
            sum *= exp2f((top - m) * scale);
            top = m;
        }
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += exp2f((x[i] - base) * scale);
    }
}

// (value, index): the larger value, the lower index of equal ones.
__device__ __forceinline__ void take_better(float& v, int32_t& i, float w, int32_t j) {
    if (w > v || (w == v && j < i)) {
        v = w;
        i = j;
    }
}

// The CTA's largest and sum, in thread 0.
__device__ __forceinline__ void block_sum(VerifyShared& s, float& top, double& sum, float part,
                                          float scale) {
    float m = top;
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    // (a share without a finite value keeps its zero or NaN)
    sum = top == -INFINITY ? part : part * exp2f((top - m) * scale);
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) {
        s.warp_top[warp] = m;
        s.warp_sum[warp] = sum;
    }
    __syncthreads();
    top = lane < kVerifyWarps ? s.warp_top[lane] : -INFINITY;
    sum = lane < kVerifyWarps ? s.warp_sum[lane] : 0.0;
    m = top;
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (top != -INFINITY) sum *= exp2f((top - m) * scale);
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    top = m;
}

__device__ __forceinline__ void block_best(VerifyShared& s, float& v, int32_t& i) {
    for (int off = 16; off > 0; off >>= 1)
        take_better(v, i, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, i, off));
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) {
        s.warp_top[warp] = v;
        s.warp_index[warp] = i;
    }
    __syncthreads();
    v = lane < kVerifyWarps ? s.warp_top[lane] : -INFINITY;
    i = lane < kVerifyWarps ? s.warp_index[lane] : INT32_MAX;
    for (int off = 16; off > 0; off >>= 1)
        take_better(v, i, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, i, off));
}

// The rows of one node, as weights relative to their sums.
struct VerifyRow {
    float top, inv;                 // largest logit, 1 / sum
};

constexpr int32_t kVerifyNone = -1, kVerifyAgain = -2;   // verdicts beside a node

template <typename E, bool DRAFT, bool WIDE>
__global__ void __launch_bounds__(kVerifyThreads) verify_tree_kernel(const VerifyArgs a) {
    __shared__ VerifyShared s;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int32_t seq = blockIdx.x / ctas;
    const int32_t vocab = a.vocab;
    // this CTA's share of the vocabulary
    const int32_t share = (int32_t)(((int64_t)vocab + 16 * ctas - 1) / (16 * ctas) * 16);
    const int32_t lo = (int32_t)min((int64_t)vocab, (int64_t)share * rank);
    const int32_t hi = (int32_t)min((int64_t)vocab, (int64_t)lo + share);

    // the tree, from the first CTA to all
    if (rank == 0) {
        const int32_t q0 = a.query_start[seq], q1 = a.query_start[seq + 1];
        const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q ||
                         (int64_t)q1 - q0 > min(a.max_q_len, PA_MAX_TREE_NODES);
        const float heat = a.temperature != nullptr ? a.temperature[seq] : 1.f;
        const float scale = kLog2e / heat;
        const bool cold = heat <= 0.f;
        const bool off = !cold && !(scale > 0.f && scale < INFINITY);
        const int32_t nodes = bad || off ? -1 : q1 - q0;
        if (tid == 0 && bad) raise_error(PA_DEVERR_SEQ_LEN);
        if (tid == 0 && !bad && off) raise_error(PA_DEVERR_LOGITS);
        for (int32_t j = tid; j < nodes; j += kVerifyThreads) {
            int32_t up = a.parents[q0 + j];
            if (up < -1 || up >= j) {
                raise_error(PA_DEVERR_TREE);
                up = -1;
            }
            s.parent[j] = up;
            s.token[j] = a.tokens[q0 + j];
            s.uniform[j] = a.uniforms[q0 + j];
        }
        if (tid == 0) {
            s.first = q0;
            s.nodes = nodes;
            s.heat = heat;
        }
        __syncthreads();
    }
    cluster_sync();                     // (also: all CTAs run before any stores to another)
    if (rank == 0 && ctas > 1) {
        for (uint32_t r = 1; r < ctas; ++r) {
            for (int32_t j = tid; j < s.nodes; j += kVerifyThreads) {
                cluster_store(cluster_map(&s.parent[j], r), s.parent[j]);
                cluster_store(cluster_map(&s.token[j], r), s.token[j]);
                cluster_store(cluster_map(&s.uniform[j], r), s.uniform[j]);
            }
            if (tid == 0) {
                cluster_store(cluster_map(&s.first, r), s.first);
                cluster_store(cluster_map(&s.nodes, r), s.nodes);
                cluster_store(cluster_map(&s.heat, r), s.heat);
            }
        }
    }
    if (ctas > 1) cluster_sync();
    const int32_t q0 = s.first, nodes = s.nodes;
    if (nodes <= 0) {
        if (rank == 0 && tid == 0) a.leaf[seq] = a.next[seq] = -1;
        return;
    }
    const bool cold = s.heat <= 0.f;
    const float scale = cold ? 1.f : kLog2e / s.heat;
    const double fine = cold ? 1.0 : 1.4426950408889634 / (double)s.heat;
    const E* target = static_cast<const E*>(a.logits);
    const E* draft = static_cast<const E*>(a.draft);
    uint32_t turn = 0;                  // exchanges so far
    int32_t cur = 0;
    VerifyRow p{}, q{};
    float spent = 0.f;                  // c, once no child holds

    // thread 0's part to every CTA, then all CTAs' parts are in s.part[...]
    auto exchange = [&](const VerifyPart& mine) -> const VerifyPart* {
        const uint32_t at = turn++ & 1;
        if (tid < (int32_t)ctas) {
            VerifyPart* to = &s.part[at][rank];
            cluster_store(cluster_map(&to->top, tid), mine.top);
            cluster_store(cluster_map(&to->draft_top, tid), mine.draft_top);
            cluster_store(cluster_map(&to->sum, tid), mine.sum);
            cluster_store(cluster_map(&to->draft_sum, tid), mine.draft_sum);
            cluster_store(cluster_map(&to->index, tid), mine.index);
        }
        cluster_sync();
        return s.part[at];
    };
    auto give_up = [&](unsigned int why) {
        if (rank == 0 && tid == 0) {
            raise_error(why);
            a.leaf[seq] = a.next[seq] = -1;
        }
    };

    while (true) {
        const E* row = target + (int64_t)(q0 + cur) * a.logit_stride;
        const E* drow = DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr;
        spent = 0.f;
        __syncthreads();
        // the node's children: their logits, from the CTA that has the token
        bool is_child = false;
        if (tid < PA_MAX_TREE_NODES) {
            is_child = tid > cur && tid < nodes && s.parent[tid] == cur;
            const uint32_t mask = __ballot_sync(0xffffffffu, is_child);
            if (lane == 0) s.child[tid >> 5] = mask;
        }
        if (is_child && !cold) {
            const int32_t t = s.token[tid];
            if (t >= lo && t < hi) {
                const float x = Elem<E>::to_float(row[t]);
                const float y = DRAFT ? Elem<E>::to_float(drow[t]) : 0.f;
                for (uint32_t r = 0; r < ctas; ++r) {
                    cluster_store(cluster_map(&s.logit[tid], r), x);
                    if (DRAFT) cluster_store(cluster_map(&s.draft_logit[tid], r), y);
                }
            }
        }
        __syncthreads();
        uint32_t any = 0;
        for (int w = 0; w < PA_MAX_TREE_NODES / 32; ++w) any |= s.child[w];
        if (cold) {
            // the first largest logit
            float v = -INFINITY;
            int32_t best = INT32_MAX;
            bool nan = false;
            for (int32_t o = lo + 8 * tid; o < hi; o += 8 * kVerifyThreads) {
                float x[8];
                load8<E, WIDE>(row + o, hi - o, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    nan |= x[i] != x[i];
                    if (x[i] > v) {
                        v = x[i];
                        best = o + i;
                    }
                }
            }
            if (nan) v = INFINITY;
            block_best(s, v, best);
            const VerifyPart* all = exchange(VerifyPart{v, 0.f, 0.0, 0.0, best});
            v = -INFINITY;
            best = INT32_MAX;
            for (uint32_t r = 0; r < ctas; ++r) take_better(v, best, all[r].top, all[r].index);
            if (!(v > -INFINITY && v < INFINITY)) {
                give_up(PA_DEVERR_LOGITS);
                return;
            }
            int32_t child = -1;
            for (int w = PA_MAX_TREE_NODES / 32 - 1; any != 0 && w >= 0; --w)
                for (uint32_t m = s.child[w]; m != 0; m &= m - 1) {
                    const int32_t j = 32 * w + __ffs(m) - 1;
                    if (s.token[j] == best && (child < 0 || j < child)) child = j;
                }
            if (child < 0) {
                if (rank == 0 && tid == 0) {
                    a.leaf[seq] = cur;
                    a.next[seq] = best;
                }
                return;
            }
            cur = child;
            continue;
        }
        {
            float top, part, dtop = 0.f;
            double sum, dsum = 0.0;
            row_sum<E, WIDE>(row, lo, hi, scale, top, part);
            block_sum(s, top, sum, part, scale);
            if (DRAFT && any) {
                row_sum<E, WIDE>(drow, lo, hi, scale, dtop, part);
                block_sum(s, dtop, dsum, part, scale);
            }
            const VerifyPart* all = exchange(VerifyPart{top, dtop, sum, dsum, 0});
            p.top = q.top = -INFINITY;
            for (uint32_t r = 0; r < ctas; ++r) {
                p.top = fmaxf(p.top, all[r].top);
                q.top = fmaxf(q.top, all[r].draft_top);
            }
            sum = dsum = 0.0;
            for (uint32_t r = 0; r < ctas; ++r) {
                sum += all[r].top == -INFINITY ? all[r].sum : all[r].sum * exp2f((all[r].top - p.top) * scale);
                if (DRAFT && any)
                    dsum += all[r].draft_top == -INFINITY
                                ? all[r].draft_sum
                                : all[r].draft_sum * exp2f((all[r].draft_top - q.top) * scale);
            }
            // (NaN, an infinity, or nothing to choose from)
            if (!(sum >= 0.5) || (DRAFT && any && !(dsum >= 0.5))) {
                give_up(PA_DEVERR_LOGITS);
                return;
            }
            p.inv = (float)(1.0 / sum);
            q.inv = DRAFT && any ? (float)(1.0 / dsum) : 0.f;
            if (is_child) {
                const int32_t t = s.token[tid];
                const bool in = t >= 0 && t < vocab;
                if (!in && rank == 0) raise_error(PA_DEVERR_TREE);
                s.chance[tid] = in ? exp2(((double)s.logit[tid] - p.top) * fine) / sum : 0.0;
                if (DRAFT)
                    s.draft_chance[tid] = in ? exp2(((double)s.draft_logit[tid] - q.top) * fine) / dsum : 0.0;
            }
            __syncthreads();
        }
        // the children in order; thread 0 decides, from numbers that all CTAs have
        int32_t verdict = kVerifyNone;
        if (any) {
            if (tid == 0) s.tried = 0;
            double spent_d = 0.0, rest = 1.0;
            while (true) {
                if (tid == 0) {
                    verdict = kVerifyNone;
                    int32_t j = s.tried;
                    for (; j < nodes; ++j) {
                        if (!(s.child[j >> 5] >> (j & 31) & 1)) continue;
                        if (s.token[j] < 0 || s.token[j] >= vocab) continue;
                        double left = s.chance[j], ask = (double)s.uniform[j] * rest;
                        if (DRAFT) {
                            left = fmax(left - spent_d * s.draft_chance[j], 0.0);
                            ask *= s.draft_chance[j];
                        } else {
                            for (int32_t k = cur + 1; k < j; ++k)     // tried before
                                if ((s.child[k >> 5] >> (k & 31) & 1) && s.token[k] == s.token[j]) left = 0.0;
                        }
                        if (ask < left) {
                            verdict = j;
                            break;
                        }
                        if (DRAFT) {
                            spent_d += rest;
                            bool more = false;
                            for (int32_t k = j + 1; k < nodes; ++k) more |= s.child[k >> 5] >> (k & 31) & 1;
                            if (more) {
                                verdict = kVerifyAgain;
                                ++j;
                                break;
                            }
                        } else {
                            rest = fmax(rest - left, 0.0);
                        }
                    }
                    s.tried = j;
                    s.verdict = verdict;
                    s.spent = (float)spent_d;
                }
                __syncthreads();
                verdict = s.verdict;
                spent = s.spent;
                if (!DRAFT || verdict != kVerifyAgain) break;
                // what is left of P
                float sum = 0.f;
                const float pi = p.inv, qi = spent * q.inv;
                for (int32_t o = lo + 8 * tid; o < hi; o += 8 * kVerifyThreads) {
                    float x[8], y[8];
                    load8<E, WIDE>(row + o, hi - o, x);
                    load8<E, WIDE>(drow + o, hi - o, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum += fmaxf(exp2f((x[i] - p.top) * scale) * pi - exp2f((y[i] - q.top) * scale) * qi, 0.f);
                }
                float top = 0.f;
                double total;
                block_sum(s, top, total, sum, 0.f);
                const VerifyPart* all = exchange(VerifyPart{0.f, 0.f, total, 0.0, 0});
                rest = 0.0;
                for (uint32_t r = 0; r < ctas; ++r) rest += all[r].sum;
            }
        }
        if (verdict >= 0) {
            cur = verdict;
            continue;
        }
        break;
    }

    // the next token: the best of the rest, of P itself where rounding left nothing
    const E* row = target + (int64_t)(q0 + cur) * a.logit_stride;
    const E* drow = DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr;
    const float* noise = a.noise + (int64_t)seq * a.noise_stride;
    for (int round = 0; round < 2; ++round) {
        float v = 0.f;
        int32_t best = INT32_MAX;
        const bool rest = round == 0;
        const float pi = p.inv, qi = rest ? spent * q.inv : 0.f;
        for (int32_t o = lo + 8 * tid; o < hi; o += 8 * kVerifyThreads) {
            float x[8], y[8], e[8];
            load8<E, WIDE>(row + o, hi - o, x);
            load8<float, WIDE>(noise + o, hi - o, e);
            if (DRAFT && qi != 0.f) load8<E, WIDE>(drow + o, hi - o, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float w = exp2f((x[i] - p.top) * scale) * pi;
                if (DRAFT && qi != 0.f) w -= exp2f((y[i] - q.top) * scale) * qi;
                w = w / e[i];
                if (o + i < hi && w > v) {
                    bool out = false;
                    if (!DRAFT && rest)
                        for (int32_t j = cur + 1; j < nodes; ++j)
                            out |= s.parent[j] == cur && s.token[j] == o + i;
                    if (!out) {
                        v = w;
                        best = o + i;
                    }
                }
            }
        }
        block_best(s, v, best);
        const VerifyPart* all = exchange(VerifyPart{v, 0.f, 0.0, 0.0, best});
        v = 0.f;
        best = INT32_MAX;
        for (uint32_t r = 0; r < ctas; ++r) take_better(v, best, all[r].top, all[r].index);
        if (best != INT32_MAX || round == 1) {
            if (rank == 0 && tid == 0) {
                const bool none = best == INT32_MAX;
                if (none) raise_error(PA_DEVERR_LOGITS);
                a.leaf[seq] = none ? -1 : cur;
                a.next[seq] = none ? -1 : best;
            }
            return;
        }
    }
}

}  // namespace pa

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
// node's rows once (largest logit, sum of exponentials, by the running maximum), every
// warp tells every CTA its part through shared memory, and behind one cluster barrier
// all warps take the same decision from the same numbers.  (What decides is told by
// the first CTA, the tree with the first step, so that the CTAs stay together even
// where somebody writes the inputs meanwhile.)
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

constexpr int kVerifyThreads = 256;                 // one a node
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;
static_assert(kVerifyThreads >= PA_MAX_TREE_NODES, "a thread per node");

// What a warp tells the CTAs: the largest logit of its share and the sum of
// exponentials relative to it, of the target's and the draft's row.
struct VerifyPart {
    float top, sum, draft_top, draft_sum;
};

struct VerifyShared {
    VerifyPart part[2][kVerifyMaxCluster * kVerifyWarps];
    // the tree, from the first CTA
    float logit[PA_MAX_TREE_NODES], draft_logit[PA_MAX_TREE_NODES];   // of a node's token
    float uniform[PA_MAX_TREE_NODES];
    int32_t token[PA_MAX_TREE_NODES];
    int32_t child[PA_MAX_TREE_NODES], sibling[PA_MAX_TREE_NODES];     // first, next; -1: none
    int32_t parent[PA_MAX_TREE_NODES];
    int32_t first, nodes;                            // rows of the sequence (nodes -1: refused)
    float heat;
};

// ---- packed pairs of floats ------------------------------------------------------------

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---- rows --------------------------------------------------------------------------------

// 16 bytes of a row: 8 bf16 or 4 fp32.
template <typename E>
struct RowVec {
    static constexpr int kCount = 16 / (int)sizeof(E);
    uint4 r;
    __device__ __forceinline__ void load(const E* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() {        // -inf
        const uint32_t x = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;
        r = make_uint4(x, x, x, x);
    }
    // largest, NaN left out
    __device__ __forceinline__ float top() const {
        if constexpr (sizeof(E) == 2) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            const float* f = reinterpret_cast<const float*>(&r);
            return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
        }
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ uint64_t pair(int i) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
        if constexpr (sizeof(E) == 2)
            return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else
            return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

// The running maximum of a share and its sum of exponentials.  A NaN or +inf makes
// the sum NaN; -inf counts as nothing.
struct RowSum {
    float top, scale;
    uint64_t sum;                   // two parts
    __device__ __forceinline__ void start(float s) {
        top = -INFINITY;
        scale = s;
        sum = 0;
    }
    __device__ __forceinline__ void raise(float m) {
        if (m > top) {
            const float f = ex2_approx((top - m) * scale);
            sum = mul2(sum, pack2(f, f));
            top = m;
        }
    }
    template <typename E, int U>
    __device__ __forceinline__ void take(const RowVec<E> (&v)[U]) {
        float m = v[0].top();
#pragma unroll
        for (int u = 1; u < U; ++u) m = fmaxf(m, v[u].top());
        raise(m);
        const float base = top == -INFINITY ? 0.f : -top;
        const uint64_t off = pack2(base, base), by = pack2(scale, scale);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < RowVec<E>::kCount / 2; ++i) {
                float a, b;
                unpack2(mul2(add2(v[u].pair(i), off), by), a, b);
                sum = add2(sum, pack2(ex2_approx(a), ex2_approx(b)));
            }
    }
    __device__ __forceinline__ void take(float x) {
        raise(x);
        const float w = ex2_approx((x - (top == -INFINITY ? 0.f : top)) * scale);
        sum = add2(sum, pack2(w, 0.f));
    }
    // of the warp: top and sum in all lanes
    __device__ __forceinline__ void reduce(float& all_top, float& all_sum) const {
        float a, b, m = top;
        unpack2(sum, a, b);
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        // (a share without a finite value keeps its zero or NaN)
        float s = a + b;
        if (top != -INFINITY) s *= ex2_approx((top - m) * scale);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        all_top = m;
        all_sum = s;
    }
};

// A share [lo, hi) of a row: the 16-byte pieces inside it, and the elements before and
// behind them.
template <typename E>
struct RowShare {
    const E* body;
    int32_t pieces, front, back;    // front elements before body, back elements behind
    __device__ __forceinline__ RowShare(const E* row, int32_t lo, int32_t hi) {
        const int32_t off = (int32_t)((reinterpret_cast<uintptr_t>(row + lo) & 15) / sizeof(E));
        front = min(hi - lo, (RowVec<E>::kCount - off) % RowVec<E>::kCount);
        body = row + lo + front;
        pieces = (hi - lo - front) / RowVec<E>::kCount;
        back = hi - lo - front - pieces * RowVec<E>::kCount;
    }
    // fetch the pieces into L2
    __device__ __forceinline__ void prefetch() const {
        if (pieces > 0)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(body), "r"(pieces * 16)
                         : "memory");
    }
    __device__ __forceinline__ void ends(RowSum& s) const {
        const int32_t tid = threadIdx.x;
        if (tid < front) s.take(Elem<E>::to_float(body[tid - front]));
        if (tid >= 32 && tid - 32 < back)
            s.take(Elem<E>::to_float(body[pieces * RowVec<E>::kCount + tid - 32]));
    }
};

// One row, or two at once (their shares may be cut differently).
constexpr int kRowUnroll = 4;
template <typename E, bool TWO>
__device__ __forceinline__ void row_sums(const RowShare<E>& x, const RowShare<E>& y, RowSum& sx,
                                         RowSum& sy) {
    constexpr int U = kRowUnroll;
    const int32_t n = TWO ? max(x.pieces, y.pieces) : x.pieces;
    for (int32_t v = threadIdx.x; v < n; v += U * kVerifyThreads) {
        RowVec<E> a[U], b[TWO ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t at = v + u * kVerifyThreads;
            if (at < x.pieces) a[u].load(x.body + (int64_t)at * RowVec<E>::kCount);
            else a[u].clear();
        }
        if constexpr (TWO) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t at = v + u * kVerifyThreads;
                if (at < y.pieces) b[u].load(y.body + (int64_t)at * RowVec<E>::kCount);
                else b[u].clear();
            }
        }
        sx.take(a);
        if constexpr (TWO) sy.take(b);
    }
    x.ends(sx);
    if constexpr (TWO) y.ends(sy);
}

// 8 elements from p on, -inf past `count`.
template <typename E, bool WIDE>
__device__ __forceinline__ void load8(const E* p, int32_t count, float (&x)[8]) {
    if (WIDE && count >= 8) {
        constexpr int N = RowVec<E>::kCount;
#pragma unroll
        for (int u = 0; u < 8 / N; ++u) {
            RowVec<E> v;
            v.load(p + u * N);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) unpack2(v.pair(i), x[u * N + 2 * i], x[u * N + 2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < count ? Elem<E>::to_float(p[i]) : -INFINITY;
    }
}

// (value, index): the larger value, the lower index of equal ones.
__device__ __forceinline__ void take_better(float& v, int32_t& i, float w, int32_t j) {
    if (w > v || (w == v && j < i)) {
        v = w;
        i = j;
    }
}
__device__ __forceinline__ void warp_best(float& v, int32_t& i) {
    for (int off = 16; off > 0; off >>= 1)
        take_better(v, i, __shfl_xor_sync(0xffffffffu, v, off), __shfl_xor_sync(0xffffffffu, i, off));
}

// Scale of the exponents, log2(e) / T, as two floats, and 2^((x - top) scale) with
// it: the product's rounding is taken into the result.
struct FineScale {
    float hi, lo;
    __device__ __forceinline__ explicit FineScale(float heat) {
        constexpr float kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);
        hi = kLog2e / heat;
        lo = (fmaf(-hi, heat, kLog2e) + kLog2eRest) / heat;
    }
    __device__ __forceinline__ float power(float x, float top) const {
        const float d = x - top, y = d * hi;
        const float rest = fmaf(d, lo, fmaf(d, hi, -y));
        return y < -200.f ? 0.f : exp2f(y) * fmaf(rest, 0.6931472f, 1.f);
    }
};

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A node's row: largest logit, 1 / sum.
struct VerifyRow {
    float top, inv;
};

template <typename E, bool DRAFT, bool WIDE>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_tree_kernel(const VerifyArgs a) {
    __shared__ VerifyShared s;
    griddep_wait();
    griddep_launch_dependents();
    cluster_arrive();                   // this CTA runs
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int32_t seq = blockIdx.x / ctas;
    const int32_t vocab = a.vocab;
    // this CTA's share of the vocabulary
    const int32_t share = (int32_t)(((int64_t)vocab + 16 * ctas - 1) / (16 * ctas) * 16);
    const int32_t lo = (int32_t)min((int64_t)vocab, (int64_t)share * rank);
    const int32_t hi = (int32_t)min((int64_t)vocab, (int64_t)lo + share);
    const E* target = static_cast<const E*>(a.logits);
    const E* draft = static_cast<const E*>(a.draft);
    const float* noise = a.noise + (int64_t)seq * a.noise_stride;

    // The sequence as this CTA sees it; from the first exchange on, as the first CTA
    // does.
    int32_t q0 = a.query_start[seq];
    float heat = a.temperature != nullptr ? a.temperature[seq] : 1.f;
    unsigned int bad = 0;
    int32_t nodes;
    {
        const int32_t q1 = a.query_start[seq + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.total_q ||
            (int64_t)q1 - q0 > min(a.max_q_len, PA_MAX_TREE_NODES))
            bad = PA_DEVERR_SEQ_LEN;
        const float x = kLog2e / heat;
        if (!bad && !(heat <= 0.f) && !(x > 0.f && x < INFINITY)) bad = PA_DEVERR_LOGITS;
        nodes = bad ? -1 : q1 - q0;
    }
    if (tid == 0 && nodes > 0) {
        RowShare<E>(target + (int64_t)q0 * a.logit_stride, lo, hi).prefetch();
        if (!(heat <= 0.f)) RowShare<float>(noise, lo, hi).prefetch();
    }
    int32_t parent = -1, token = -1;    // of node tid
    float uniform = 0.f;
    if (tid < nodes) {
        parent = a.parents[q0 + tid];
        if (rank == 0) {
            token = a.tokens[q0 + tid];
            uniform = a.uniforms[q0 + tid];
        }
        if (parent < -1 || parent >= tid) {
            if (rank == 0) raise_error(PA_DEVERR_TREE);
            parent = -1;
        }
    }
    const bool inner = __syncthreads_or(parent == 0);        // node 0 has children
    if (tid == 0 && nodes > 0 && DRAFT && inner && !(heat <= 0.f))
        RowShare<E>(draft + (int64_t)q0 * a.draft_stride, lo, hi).prefetch();
    int32_t child = -1, sibling = -1;
    if (rank == 0) {
        s.parent[tid] = parent;
        __syncthreads();
        for (int32_t j = nodes - 1; j > tid; --j) {
            const int32_t p = s.parent[j];
            if (p == tid) child = j;
            if (p == parent) sibling = j;
        }
    }

    uint32_t turn = 0;                  // exchanges so far
    // the warp's part to every CTA; all warps' parts
    auto exchange = [&](const VerifyPart& mine) -> const VerifyPart* {
        const uint32_t at = turn++ & 1;
        if (lane < (int32_t)ctas) {
            const uint32_t to = cluster_map(&s.part[at][rank * kVerifyWarps + warp], lane);
            cluster_store(to, mine.top);
            cluster_store(to + 4, mine.sum);
            cluster_store(to + 8, mine.draft_top);
            cluster_store(to + 12, mine.draft_sum);
        }
        cluster_sync();
        return s.part[at];
    };
    const int32_t parts = (int32_t)ctas * kVerifyWarps;
    auto best_of = [&](const VerifyPart* all, float floor, int32_t& index) {
        float v = floor;
        index = INT32_MAX;
        for (int32_t e = lane; e < parts; e += 32) take_better(v, index, all[e].top, __float_as_int(all[e].sum));
        warp_best(v, index);
        return v;
    };
    auto give_up = [&](unsigned int why) {
        if (rank == 0 && tid == 0) {
            if (why) raise_error(why);
            a.leaf[seq] = a.next[seq] = -1;
        }
    };

    int32_t cur = 0;
    bool any = inner;
    VerifyRow p{}, q{};
    float spent = 0.f;                  // c, once no child holds
    for (bool begin = true;; begin = false) {
        const bool cold = heat <= 0.f;
        const E* row = target + (int64_t)(q0 + cur) * a.logit_stride;
        const E* drow = DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr;
        // the children's logits
        const bool told = rank == 0 && !cold && parent == cur && token >= 0 && token < vocab;
        float tl = 0.f, dl = 0.f;
        if (told) {
            tl = Elem<E>::to_float(row[token]);
            if (DRAFT) dl = Elem<E>::to_float(drow[token]);
        }
        VerifyPart mine{-INFINITY, 0.f, -INFINITY, 0.f};
        const float scale = cold ? 1.f : kLog2e / heat;
        if (nodes > 0 && cold) {
            // the first largest logit; a NaN counts as an infinity
            int32_t best = INT32_MAX;
            float v = -INFINITY;
            const RowShare<E> x(row, lo, hi);
            auto one = [&](int32_t at) {
                const float y = Elem<E>::to_float(row[at]);
                take_better(v, best, y != y ? INFINITY : y, at);
            };
            if (tid < x.front) one(lo + tid);
            for (int32_t u = tid; u < x.pieces; u += kVerifyThreads) {
                RowVec<E> w;
                w.load(x.body + (int64_t)u * RowVec<E>::kCount);
                float m = 0.f;          // (a NaN leaves one in the sum)
                float y[RowVec<E>::kCount];
#pragma unroll
                for (int i = 0; i < RowVec<E>::kCount / 2; ++i) unpack2(w.pair(i), y[2 * i], y[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < RowVec<E>::kCount; ++i) m += y[i] * 0.f;
                if (w.top() > v || m != m) {
                    const int32_t at = lo + x.front + u * RowVec<E>::kCount;
                    for (int i = 0; i < RowVec<E>::kCount; ++i) one(at + i);
                }
            }
            if (tid >= 32 && tid - 32 < x.back) one(hi - x.back + tid - 32);
            warp_best(v, best);
            mine.top = v;
            mine.sum = __int_as_float(best);
        } else if (nodes > 0) {
            RowSum sx, sy;
            sx.start(scale);
            sy.start(scale);
            const RowShare<E> x(row, lo, hi);
            if (DRAFT && any) {
                row_sums<E, true>(x, RowShare<E>(drow, lo, hi), sx, sy);
                sy.reduce(mine.draft_top, mine.draft_sum);
            } else {
                row_sums<E, false>(x, x, sx, sx);
            }
            sx.reduce(mine.top, mine.sum);
        }
        if (begin) cluster_wait();      // all CTAs run: their shared memory is there
        if (begin && rank == 0) {
            for (uint32_t r = 0; r < ctas; ++r) {
                if (tid < nodes) {
                    cluster_store(cluster_map(&s.token[tid], r), token);
                    cluster_store(cluster_map(&s.uniform[tid], r), uniform);
                    cluster_store(cluster_map(&s.child[tid], r), child);
                    cluster_store(cluster_map(&s.sibling[tid], r), sibling);
                }
                if (tid == 0) {
                    cluster_store(cluster_map(&s.first, r), q0);
                    cluster_store(cluster_map(&s.nodes, r), nodes);
                    cluster_store(cluster_map(&s.heat, r), heat);
                }
            }
        }
        if (told)
            for (uint32_t r = 0; r < ctas; ++r) {
                cluster_store(cluster_map(&s.logit[tid], r), tl);
                if (DRAFT) cluster_store(cluster_map(&s.draft_logit[tid], r), dl);
            }
        const VerifyPart* all = exchange(mine);
        if (begin) {
            q0 = s.first;
            nodes = s.nodes;
            heat = s.heat;
            if (nodes <= 0) {
                give_up(bad);
                return;
            }
            any = s.child[0] >= 0;
        }
        if (heat <= 0.f) {
            int32_t best;
            const float v = best_of(all, -INFINITY, best);
            if (!(v > -INFINITY && v < INFINITY)) {
                give_up(PA_DEVERR_LOGITS);
                return;
            }
            int32_t j = s.child[cur];
            while (j >= 0 && s.token[j] != best) j = s.sibling[j];
            if (j < 0) {
                if (rank == 0 && tid == 0) {
                    a.leaf[seq] = cur;
                    a.next[seq] = best;
                }
                return;
            }
            cur = j;
            continue;
        }
        const FineScale fine(heat);
        {
            float top = -INFINITY, dtop = -INFINITY, sum = 0.f, dsum = 0.f;
            for (int32_t e = lane; e < parts; e += 32) {
                top = fmaxf(top, all[e].top);
                dtop = fmaxf(dtop, all[e].draft_top);
            }
            for (int off = 16; off > 0; off >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                dtop = fmaxf(dtop, __shfl_xor_sync(0xffffffffu, dtop, off));
            }
            for (int32_t e = lane; e < parts; e += 32) {
                const VerifyPart x = all[e];
                sum += x.top == -INFINITY ? x.sum : x.sum * ex2_approx((x.top - top) * scale);
                dsum += x.draft_top == -INFINITY ? x.draft_sum
                                                 : x.draft_sum * ex2_approx((x.draft_top - dtop) * scale);
            }
            for (int off = 16; off > 0; off >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, off);
                dsum += __shfl_xor_sync(0xffffffffu, dsum, off);
            }
            // (NaN, an infinity, or nothing to choose from)
            if (!(sum >= 0.5f) || (DRAFT && any && !(dsum >= 0.5f))) {
                give_up(PA_DEVERR_LOGITS);
                return;
            }
            p = VerifyRow{top, 1.f / sum};
            q = VerifyRow{dtop, DRAFT && any ? 1.f / dsum : 0.f};
        }
        // the children in order
        int32_t held = -1;
        float rest = 1.f;
        spent = 0.f;
        for (int32_t j = s.child[cur]; j >= 0; j = s.sibling[j]) {
            const int32_t t = s.token[j];
            if (t < 0 || t >= vocab) {
                if (rank == 0 && tid == 0) raise_error(PA_DEVERR_TREE);
                continue;
            }
            float left = fine.power(s.logit[j], p.top) * p.inv, ask = s.uniform[j] * rest;
            if (DRAFT) {
                const float qt = fine.power(s.draft_logit[j], q.top) * q.inv;
                left = fmaxf(fmaf(-spent, qt, left), 0.f);
                ask *= qt;
            } else {
                for (int32_t k = s.child[cur]; k != j; k = s.sibling[k])      // tried before
                    if (s.token[k] == t) left = 0.f;
            }
            if (ask < left) {
                held = j;
                break;
            }
            if (!DRAFT) {
                rest = fmaxf(rest - left, 0.f);
                continue;
            }
            spent += rest;
            if (s.sibling[j] < 0) break;
            // what is left of P
            float sum = 0.f;
            const float pi = p.inv, qi = spent * q.inv;
            for (int32_t o = lo + 8 * tid; o < hi; o += 8 * kVerifyThreads) {
                float x[8], y[8];
                load8<E, WIDE>(row + o, hi - o, x);
                load8<E, WIDE>(drow + o, hi - o, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum += fmaxf(ex2_approx((x[i] - p.top) * scale) * pi - ex2_approx((y[i] - q.top) * scale) * qi, 0.f);
            }
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const VerifyPart* sums = exchange(VerifyPart{0.f, sum, 0.f, 0.f});
            rest = 0.f;
            for (int32_t e = lane; e < parts; e += 32) rest += sums[e].sum;
            for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
        }
        if (held < 0) break;
        cur = held;
        any = s.child[cur] >= 0;
    }

    // the next token: the best of the rest, of P itself where rounding left nothing
    const E* row = target + (int64_t)(q0 + cur) * a.logit_stride;
    const E* drow = DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr;
    const FineScale fine(heat);
    for (int round = 0; round < 2; ++round) {
        float v = 0.f;
        int32_t best = INT32_MAX;
        const bool rest = round == 0;
        const float scale = fine.hi, pi = p.inv, qi = rest ? spent * q.inv : 0.f;
        for (int32_t o = lo + 8 * tid; o < hi; o += 8 * kVerifyThreads) {
            float x[8], y[8], e[8];
            load8<E, WIDE>(row + o, hi - o, x);
            load8<float, WIDE>(noise + o, hi - o, e);
            if (DRAFT && qi != 0.f) load8<E, WIDE>(drow + o, hi - o, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // (first about, without the exponent's second part)
                const float up = ex2_approx((x[i] - p.top) * scale) * pi;
                float w = up;
                float room = up;
                if (DRAFT && qi != 0.f) {
                    const float down = ex2_approx((y[i] - q.top) * scale) * qi;
                    w = up - down;
                    room = up + down;
                }
                if (o + i >= hi || !(fmaf(room, 0x1p-14f, w) * rcp_approx(e[i]) > v)) continue;
                w = fine.power(x[i], p.top) * pi;
                if (DRAFT && qi != 0.f) w -= fine.power(y[i], q.top) * qi;
                w = w / e[i];
                if (w > v) {
                    bool out = false;
                    if (!DRAFT && rest)
                        for (int32_t j = s.child[cur]; j >= 0; j = s.sibling[j]) out |= s.token[j] == o + i;
                    if (!out) {
                        v = w;
                        best = o + i;
                    }
                }
            }
        }
        warp_best(v, best);
        const VerifyPart* all = exchange(VerifyPart{v, __int_as_float(best), 0.f, 0.f});
        best_of(all, 0.f, best);
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

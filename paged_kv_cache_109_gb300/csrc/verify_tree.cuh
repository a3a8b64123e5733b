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
// each CTA's first warp takes the same decision from the same numbers.  (What decides is
// told by the first CTA, the tree with the first step, so that the CTAs meet at the same
// barriers even where somebody writes the inputs meanwhile.)
//
// Bound: the bytes of the rows on the walks and of one row of noise a sequence; in
// practice the walk, whose steps wait for one another.  A step of 131072 tokens on bf16 in
// 8 CTAs takes some 7500 clocks alone: 4300 for the two rows, 1050 for the barrier, 1200
// for the decision, the rest for the warps' sums; three times as many CTAs on an SM make
// it 11000.  Measured (GPU time): 64 chains of 5 nodes, 115 MB, 45 us (the copy rate:
// 17); 128 trees of up to 40, 243 MB, 79 us (36); 48 trees on fp32 with 100003 tokens and
// no draft rows, 63 MB, 34 us from memory (9.3); one chain of 6 at 32000 tokens 18 us, a
// launch and 6 steps; sampling alone (one node) 64 rows of 131072, 50 MB, 18 us from memory
// (7.4).  Half of the issue slots are in use then; deeper copies, a fetch of
// the likely next rows ahead, 16 CTAs a sequence or 512 threads a CTA did not help.  64
// registers, for 4 CTAs an SM; five of the eight instances spill 20 to 92 bytes.
#pragma once

#include "cluster.cuh"
#include "common.cuh"
#include "cp_async.cuh"
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
constexpr int kVerifyMaxCluster = 8;
static_assert(kVerifyThreads >= PA_MAX_TREE_NODES, "a thread per node");

// What a warp tells the CTAs: the largest logit of its share and the sum of
// exponentials relative to it, of the target's and the draft's row.
struct __align__(16) VerifyPart {
    float top, sum, draft_top, draft_sum;
};

// A node as the first CTA tells it: first child and next sibling, -1 where there is
// none.
struct __align__(16) VerifyNode {
    int32_t token, child, sibling;
    float uniform;
};

// What a CTA's first warp decides for its other warps.
enum VerifyVerdict : int32_t { kVerifyHolds, kVerifyRest, kVerifyNext, kVerifyFinely, kVerifyDone };
struct VerifyStep {
    int32_t verdict, node;                           // node: that holds, to try next; token
    float top, draft_top, inv, draft_inv;            // the node's rows
    float spent, rest;                               // c, S
    float floor;
};

struct VerifyShared {
    VerifyPart part[2][kVerifyMaxCluster * kVerifyWarps];
    VerifyNode node[PA_MAX_TREE_NODES];
    float2 logit[PA_MAX_TREE_NODES];                 // of a node's token: target, draft
    int32_t parent[PA_MAX_TREE_NODES];
    VerifyStep step;
    int4 tree;                                       // first row, nodes (-1: refused), temperature, scale
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

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
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
    // the same, NaN where one is
    __device__ __forceinline__ float top_or_nan() const {
        if constexpr (sizeof(E) == 2) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
            const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
            const float x = __low2float(m), y = __high2float(m);
            return x != x ? x : y != y ? y : fmaxf(x, y);
        } else {
            const float* f = reinterpret_cast<const float*>(&r);
            float m = f[0];
#pragma unroll
            for (int i = 1; i < 4; ++i) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(f[i]));
            return m;
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

// The running maximum of a share and its sum of exponentials, in 32 bits: all terms are
// positive and at most V / 8192 + 30 additions follow one another, each off by 2^-24 of
// itself, so 131072 tokens' sum is off by 2^-18 with the exponentials' own 2^-20 to 2^-22
// (sums in 64 bits and exp2f made 64 chains 272 us).  A NaN or +inf makes
// the sum NaN; -inf counts as nothing.  The maximum starts at the lowest finite value:
// a row of nothing but that has weights of one, and no -inf is subtracted from another.
constexpr float kLowest = -3.402823466e38f;
struct RowSum {
    float top, scale;
    uint64_t sum;                   // two parts
    __device__ __forceinline__ void start(float s) {
        top = kLowest;
        scale = s;
        sum = 0;
    }
    __device__ __forceinline__ void raise(float m) {
        m = fmaxf(m, top);
        const float f = ex2_approx((top - m) * scale);
        sum = mul2(sum, pack2(f, f));
        top = m;
    }
    template <typename E, int U>
    __device__ __forceinline__ void take(const RowVec<E> (&v)[U]) {
        float m = v[0].top();
#pragma unroll
        for (int u = 1; u < U; ++u) m = fmaxf(m, v[u].top());
        raise(m);
        const uint64_t off = pack2(-top, -top), by = pack2(scale, scale);
        uint64_t part[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            part[u] = 0;
#pragma unroll
            for (int i = 0; i < RowVec<E>::kCount / 2; ++i) {
                float a, b;
                unpack2(mul2(add2(v[u].pair(i), off), by), a, b);
                const uint64_t w = pack2(ex2_approx(a), ex2_approx(b));
                part[u] = i == 0 ? w : add2(part[u], w);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) sum = add2(sum, part[u]);
    }
    __device__ __forceinline__ void take(float x) {
        raise(x);
        sum = add2(sum, pack2(ex2_approx((x - top) * scale), 0.f));
    }
    __device__ __forceinline__ float total() const {
        float a, b;
        unpack2(sum, a, b);
        return a + b;
    }
};

// Two sums of the warp (their tops and totals in all lanes).
__device__ __forceinline__ void reduce_sums(const RowSum& x, const RowSum& y, float& top_x, float& sum_x,
                                            float& top_y, float& sum_y) {
    top_x = warp_max(x.top);
    top_y = warp_max(y.top);
    sum_x = x.total() * ex2_approx((x.top - top_x) * x.scale);
    sum_y = y.total() * ex2_approx((y.top - top_y) * y.scale);
    for (int off = 16; off > 0; off >>= 1) {
        sum_x += __shfl_xor_sync(0xffffffffu, sum_x, off);
        sum_y += __shfl_xor_sync(0xffffffffu, sum_y, off);
    }
}

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

// The rows' sums of a step: one row, or two at once (their shares may be cut
// differently).  Pieces come by asynchronous copies into shared memory, each thread's
// own ones, so that none waits for another; kVerifyDepth steps of four pieces are under
// way at a time, which registers would not hold.
constexpr int kVerifyDepth = 2;
constexpr size_t kVerifyRing = (size_t)kVerifyDepth * 4 * kVerifyThreads * 16;

template <typename E, bool TWO>
__device__ __forceinline__ void row_sums(uint4* ring, const RowShare<E>& x, const RowShare<E>& y,
                                         RowSum& sx, RowSum& sy) {
    constexpr int N = RowVec<E>::kCount, T = kVerifyThreads;
    constexpr int X = TWO ? 2 : 4;      // x's pieces of a step
    const int32_t tid = threadIdx.x;
    const int32_t most = TWO ? max(x.pieces, y.pieces) : x.pieces;
    uint4* mine = ring + tid;
    // step k has x's pieces k X T + u T + tid; where all threads have all of theirs
    // (`whole` steps), nothing is asked
    const int32_t whole = (TWO ? min(x.pieces, y.pieces) : x.pieces) / (X * T);
    const int32_t steps = (most + X * T - 1) / (X * T);
    const E* px = x.body + (int64_t)tid * N;
    const E* py = TWO ? y.body + (int64_t)tid * N : nullptr;
    auto issue = [&](int32_t k, int32_t d) {
        const uint32_t slot = smem_u32(mine) + d * (4 * T * 16);
        if (k < whole) {
#pragma unroll
            for (int u = 0; u < 4; ++u) cp_async16(slot + u * T * 16, u < X ? px + u * T * N : py + (u - X) * T * N, 16);
        } else {
            const int32_t at = k * X * T + tid;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t p = at + (u < X ? u : u - X) * T;
                if (p < (u < X ? x.pieces : y.pieces))
                    cp_async16(slot + u * T * 16, u < X ? px + u * T * N : py + (u - X) * T * N, 16);
            }
        }
        px += X * T * N;
        if (TWO) py += X * T * N;
        cp_async_commit();
    };
#pragma unroll
    for (int d = 0; d < kVerifyDepth; ++d) issue(d, d);
    int d = 0;
    for (int32_t k = 0; k < steps; ++k) {
        cp_async_wait<kVerifyDepth - 1>();
        const uint4* slot = mine + d * 4 * T;
        RowVec<E> a[X], b[TWO ? 2 : 1];
#pragma unroll
        for (int u = 0; u < X; ++u) a[u].r = slot[u * T];
        if constexpr (TWO) {
#pragma unroll
            for (int u = 0; u < 2; ++u) b[u].r = slot[(X + u) * T];
        }
        if (k >= whole) {               // (what is behind the rows is whatever was there)
            const int32_t at = k * X * T + tid;
#pragma unroll
            for (int u = 0; u < X; ++u)
                if (at + u * T >= x.pieces) a[u].clear();
            if constexpr (TWO) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (at + u * T >= y.pieces) b[u].clear();
            }
        }
        sx.take(a);
        if constexpr (TWO) sy.take(b);
        issue(k + kVerifyDepth, d);     // (the slots have been read: their values are used)
        d = d + 1 == kVerifyDepth ? 0 : d + 1;
    }
    cp_async_wait<0>();
    x.ends(sx);
    if constexpr (TWO) y.ends(sy);
}

// 8 elements of a share: neighbours where rows are aligned to 16 bytes (WIDE), else
// kVerifyThreads apart, so that a warp's loads are neighbours.
template <bool WIDE>
struct Eight {
    static constexpr int32_t kApart = WIDE ? 1 : kVerifyThreads, kNext = 8 * kVerifyThreads;
    static __device__ __forceinline__ int32_t first(int32_t lo) {
        return lo + (int32_t)threadIdx.x * (WIDE ? 8 : 1);
    }
};

// Them as they are stored.
template <typename E, bool WIDE>
struct Octet {
    static constexpr int N = RowVec<E>::kCount;
    RowVec<E> v[8 / N];
    // of a row, from element o on; -inf from `hi` on
    __device__ __forceinline__ void load(const E* row, int32_t o, int32_t hi) {
        if (WIDE && hi - o >= 8) {
#pragma unroll
            for (int u = 0; u < 8 / N; ++u) v[u].load(row + o + u * N);
        } else {
#pragma unroll
            for (int u = 0; u < 8 / N; ++u) v[u].clear();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (o + i * Eight<WIDE>::kApart < hi)
                    reinterpret_cast<E*>(&v[i / N])[i % N] = row[o + i * Eight<WIDE>::kApart];
        }
    }
    __device__ __forceinline__ void load_all(const E* p) {
#pragma unroll
        for (int u = 0; u < 8 / N; ++u) v[u].load(p + u * N);
    }
    __device__ __forceinline__ uint64_t pair(int i) const { return v[2 * i / N].pair(i % (N / 2)); }
    // exponentials relative to the largest
    __device__ __forceinline__ void powers(float top, float scale, float (&w)[8]) const {
        const uint64_t off = pack2(-top, -top), by = pack2(scale, scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(mul2(add2(pair(i), off), by), a, b);
            w[2 * i] = ex2_approx(a);
            w[2 * i + 1] = ex2_approx(b);
        }
    }
};

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
    __device__ __forceinline__ FineScale() {}
    __device__ __forceinline__ explicit FineScale(float heat) {
        constexpr float kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e);
        hi = kLog2e / heat;
        lo = (fmaf(-hi, heat, kLog2e) + kLog2eRest) / heat;
    }
    __device__ __forceinline__ float power(float x, float top) const {
        const float d = x - top, y = d * hi;
        const float rest = fmaf(d, lo, fmaf(d, hi, -y));
        return y < -126.f ? 0.f : ex2_approx(y) * fmaf(rest, 0.6931472f, 1.f);
    }
};

// 1 / x, off by a unit in the last place at most (the instruction's documented bound;
// subnormal numbers are zero).
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The race for the next token: the largest key, its place and least value, and the
// next largest key (all >= 0).
struct Race {
    float first, least, second;
    int32_t index;
    __device__ __forceinline__ void start() {
        first = least = second = 0.f;
        index = INT32_MAX;
    }
    __device__ __forceinline__ void take(float key, float low, int32_t at) {
        second = fmaxf(second, fminf(first, key));
        if (key > first) {
            index = at;
            least = low;
        }
        first = fmaxf(first, key);
    }
    __device__ __forceinline__ void join(const Race& o) {
        second = fmaxf(fmaxf(second, o.second), fminf(first, o.first));
        if (o.first > first || (o.first == first && o.index < index)) {
            first = o.first;
            least = o.least;
            index = o.index;
        }
    }
    // of the warp, in all lanes
    __device__ __forceinline__ void reduce() {
        const float m = warp_max(first);
        const int32_t at = __reduce_min_sync(0xffffffffu, first == m ? index : INT32_MAX);
        const bool mine = first == m && index == at;
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        second = warp_max((threadIdx.x & 31) == __ffs(who) - 1 ? second : fmaxf(first, second));
        least = __shfl_sync(0xffffffffu, least, __ffs(who) - 1);
        first = m;
        index = at;
    }
};

// What a race runs over: a share of the node's rows and of the noise.  The weights are
// those of P, or (with a share) of max(P - c q, 0), relative to P's largest.
//
// Keys are first taken with short exponentials and reciprocals.  A weight's exponent y
// is off by 2^-23 |y|, its exponential, the reciprocal and the products by less: kOpen
// = 2^-16 of each term covers them for weights down to 2^-64.  A key is the most that
// this leaves open, divided by 1 + kOpen; only where another key reaches the least
// value of the best one are those that can still win computed finely.  (Noise below
// 2^-126 counts as zero.)
constexpr float kOpen = 0x1p-16f;

template <typename E, bool DRAFT, bool WIDE>
struct RaceField {
    const E* row;
    const E* drow;
    const float* noise;
    const VerifyNode* node;         // the tree
    FineScale fine;
    float top, draft_top, share;    // share: c sum(P) / sum(q)
    int32_t lo, hi, child;          // child: first of the tokens that are out (DRAFT: none)

    struct Tokens {                 // 8 of them
        Octet<E, WIDE> x, y;
        Octet<float, WIDE> e;
    };
    __device__ __forceinline__ void load(Tokens& t, int32_t o) const {
        t.x.load(row, o, hi);
        t.e.load(noise, o, hi);
        if (DRAFT && share != 0.f) t.y.load(drow, o, hi);
    }
    __device__ __forceinline__ void load_all(Tokens& t, int32_t o) const {
        t.x.load_all(row + o);
        t.e.load_all(noise + o);
        if (DRAFT && share != 0.f) t.y.load_all(drow + o);
    }
    // Their keys, with `share` times `bound`.
    __device__ __forceinline__ void keys(const Tokens& t, int32_t o, float bound, float (&key)[8]) const {
        float up[8];
        t.x.powers(top, fine.hi, up);
        if (DRAFT && share != 0.f) {
            float down[8];
            t.y.powers(draft_top, fine.hi, down);
#pragma unroll
            for (int i = 0; i < 8; ++i) up[i] = fmaf(down[i], -share * bound, up[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(t.e.pair(i), a, b);
            key[2 * i] = up[2 * i] * rcp_approx(a);
            key[2 * i + 1] = up[2 * i + 1] * rcp_approx(b);
        }
        if (!DRAFT)
            for (int32_t j = child; j >= 0; j = node[j].sibling) {
                const int32_t at = node[j].token - o;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (at == i * Eight<WIDE>::kApart) key[i] = 0.f;
            }
    }
    __device__ __forceinline__ Race run() const {
        constexpr float kMost = (1.f - kOpen) / (1.f + kOpen), kLeast = (1.f + kOpen) / (1.f - kOpen);
        constexpr int32_t kStep = Eight<WIDE>::kNext;
        float first = 0.f, second = 0.f;
        int32_t at = -1;                // group of the largest
        auto take = [&](const Tokens& t, int32_t o) {
            float key[8];
            keys(t, o, kMost, key);
            // (a NaN, as of no weight and no noise, is left out)
            const float m = fmaxf(fmaxf(fmaxf(key[0], key[1]), fmaxf(key[2], key[3])),
                                  fmaxf(fmaxf(key[4], key[5]), fmaxf(key[6], key[7])));
            second = fmaxf(second, fminf(first, m));
            if (m > first) at = o;
            first = fmaxf(first, m);
        };
        int32_t o = Eight<WIDE>::first(lo);
        if constexpr (WIDE && sizeof(E) == 2) {
            // all threads have all of their 8: the next ones are on their way meanwhile
            // (fp32 rows have no registers for that)
            const int32_t whole = (hi - lo) / kStep;
            Tokens a, b;
            if (whole > 0) load_all(a, o);
            int32_t k = 0;
            for (; k + 2 <= whole; k += 2, o += 2 * kStep) {
                load_all(b, o + kStep);
                take(a, o);
                if (k + 2 < whole) load_all(a, o + 2 * kStep);
                take(b, o + kStep);
            }
            if (k < whole) {
                take(a, o);
                o += kStep;
            }
        }
        for (; o < hi; o += kStep) {
            Tokens t;
            load(t, o);
            take(t, o);
        }
        Tokens t;
        Race r;
        r.start();
        if (at >= 0) {
            float key[8], low[8];
            load(t, at);
            keys(t, at, kMost, key);
            keys(t, at, kLeast, low);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r.take(fmaxf(key[i], 0.f), low[i] * (1.f - 2.f * kOpen), at + i * Eight<WIDE>::kApart);
        }
        r.second = fmaxf(r.second, second);
        return r;
    }
    // Finely, those whose key is `floor` or more.
    __device__ __forceinline__ Race run_finely(float floor) const {
        constexpr float kMost = (1.f - kOpen) / (1.f + kOpen);
        Race r;
        r.start();
#pragma unroll 1
        for (int32_t o = lo + (int32_t)threadIdx.x; o < hi; o += kVerifyThreads) {
            const float x = Elem<E>::to_float(row[o]), e = noise[o];
            const float y = DRAFT && share != 0.f ? Elem<E>::to_float(drow[o]) : -INFINITY;
            float key = ex2_approx((x - top) * fine.hi);
            if (DRAFT && share != 0.f) key = fmaf(ex2_approx((y - draft_top) * fine.hi), -share * kMost, key);
            if (!(key * rcp_approx(e) >= floor)) continue;
            bool out = false;
            if (!DRAFT)
                for (int32_t j = child; j >= 0; j = node[j].sibling) out |= node[j].token == o;
            if (out) continue;
            float w = fine.power(x, top);
            if (DRAFT && share != 0.f) w -= fine.power(y, draft_top) * share;
            r.take(fmaxf(w / (e < 0x1p-126f ? 0.f : e), 0.f), 0.f, o);
        }
        return r;
    }
};

template <typename E, bool DRAFT, bool WIDE>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_tree_kernel(const VerifyArgs a) {
    extern __shared__ uint4 ring[];     // kVerifyRing
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
    if (rank == 0) {
        if (tid < PA_MAX_TREE_NODES) s.parent[tid] = parent;
        __syncthreads();
        VerifyNode n{token, -1, -1, uniform};
        for (int32_t j = nodes - 1; j > tid; --j) {
            const int32_t p = s.parent[j];
            if (p == tid) n.child = j;
            if (p == parent) n.sibling = j;
        }
        if (tid < PA_MAX_TREE_NODES) s.node[tid] = n;
    }

    uint32_t turn = 0;                  // exchanges so far
    // the warp's part to every CTA; all warps' parts
    auto exchange = [&](const VerifyPart& mine) -> const VerifyPart* {
        const uint32_t at = turn++ & 1;
        if (lane < (int32_t)ctas)
            cluster_store(cluster_map(&s.part[at][rank * kVerifyWarps + warp], lane),
                          make_float4(mine.top, mine.sum, mine.draft_top, mine.draft_sum));
        cluster_sync();
        return s.part[at];
    };
    const int32_t parts = (int32_t)ctas * kVerifyWarps;
    // the first CTA gives the sequence's results
    auto finish = [&](unsigned int why, int32_t leaf, int32_t next) {
        if (rank == 0 && tid == 0) {
            if (why) raise_error(why);
            a.leaf[seq] = leaf;
            a.next[seq] = next;
        }
    };

    int32_t cur = 0;
    bool any = inner;
    FineScale fine(heat <= 0.f ? 1.f : heat);
    for (bool begin = true;; begin = false) {
        const bool cold = heat <= 0.f;
        const E* row = target + (int64_t)(q0 + cur) * a.logit_stride;
        const E* drow = DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr;
        // the children's logits
        const bool told = rank == 0 && !cold && parent == cur && token >= 0 && token < vocab;
        float2 logit = make_float2(0.f, 0.f);
        if (told) {
            logit.x = Elem<E>::to_float(row[token]);
            if (DRAFT) logit.y = Elem<E>::to_float(drow[token]);
        }
        // (the sum of a CTA that sees no sequence: where the first one sees one, somebody
        // writes the inputs, and all refuse it)
        VerifyPart mine{kLowest, NAN, kLowest, 0.f};
        const float scale = fine.hi;
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
            constexpr int U = 8;        // pieces under way
            for (int32_t u0 = tid; u0 < x.pieces; u0 += U * kVerifyThreads) {
                RowVec<E> w[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    w[u].clear();
                    if (u0 + u * kVerifyThreads < x.pieces)
                        w[u].load(x.body + (int64_t)(u0 + u * kVerifyThreads) * RowVec<E>::kCount);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (w[u].top_or_nan() <= v) continue;
                    const int32_t at = lo + x.front + (u0 + u * kVerifyThreads) * RowVec<E>::kCount;
#pragma unroll 1
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
                row_sums<E, true>(ring, x, RowShare<E>(drow, lo, hi), sx, sy);
            } else {
                row_sums<E, false>(ring, x, x, sx, sx);
            }
            reduce_sums(sx, sy, mine.top, mine.sum, mine.draft_top, mine.draft_sum);
        }
        if (begin) cluster_wait();      // all CTAs run: their shared memory is there
        if (begin && rank == 0) {
            __syncthreads();
            for (int32_t x = tid; x < nodes * (int32_t)ctas; x += kVerifyThreads) {
                const int32_t r = x / nodes, j = x - r * nodes;
                cluster_store(cluster_map(&s.node[j], r), *reinterpret_cast<const int4*>(&s.node[j]));
            }
            if (tid < (int32_t)ctas)
                cluster_store(cluster_map(&s.tree, tid), make_int4(q0, nodes, __float_as_int(heat), __float_as_int(fine.hi)));
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, told); m != 0; m &= m - 1) {
            const int32_t l = __ffs(m) - 1;
            const float2 x = make_float2(__shfl_sync(0xffffffffu, logit.x, l), __shfl_sync(0xffffffffu, logit.y, l));
            if (lane < (int32_t)ctas) cluster_store(cluster_map(&s.logit[warp * 32 + l], lane), x);
        }
        const VerifyPart* all = exchange(mine);
        if (begin) {
            q0 = s.tree.x;
            nodes = s.tree.y;
            heat = __int_as_float(s.tree.z);
            fine = FineScale(heat <= 0.f ? 1.f : heat);
            if (nodes <= 0) {
                finish(bad, -1, -1);
                return;
            }
            any = s.node[0].child >= 0;
        }
        if (heat <= 0.f) {
            int32_t best = INT32_MAX;
            float v = -INFINITY;
            for (int32_t e = lane; e < parts; e += 32) take_better(v, best, all[e].top, __float_as_int(all[e].sum));
            warp_best(v, best);
            if (!(v > -INFINITY && v < INFINITY)) {
                finish(PA_DEVERR_LOGITS, -1, -1);
                return;
            }
            int32_t j = s.node[cur].child;
            while (j >= 0 && s.node[j].token != best) {
                const uint32_t t = s.node[j].token;     // (outside the vocabulary: met here)
                if (t >= (uint32_t)vocab && rank == 0 && tid == 0) raise_error(PA_DEVERR_TREE);
                j = s.node[j].sibling;
            }
            if (j < 0) {
                finish(0, cur, best);
                return;
            }
            cur = j;
            any = s.node[cur].child >= 0;
            continue;
        }
        // the children in order: the first warp decides, for all with its numbers
        int32_t verdict = kVerifyNext;
        while (true) {
            if (warp == 0) {
                VerifyStep step;
                if (verdict != kVerifyRest) {
                    // (up to four parts a lane)
                    VerifyPart x[kVerifyMaxCluster * kVerifyWarps / 32];
                    RowSum sx, sy;
                    const float scale = __int_as_float(s.tree.w);   // (as told: all decide by the same)
                    sx.start(scale);
                    sy.start(scale);
#pragma unroll
                    for (int u = 0; u < kVerifyMaxCluster * kVerifyWarps / 32; ++u) {
                        x[u] = VerifyPart{kLowest, 0.f, kLowest, 0.f};
                        if (lane + 32 * u < parts) x[u] = all[lane + 32 * u];
                        sx.top = fmaxf(sx.top, x[u].top);
                        sy.top = fmaxf(sy.top, x[u].draft_top);
                    }
                    float sum = 0.f, dsum = 0.f;
#pragma unroll
                    for (int u = 0; u < kVerifyMaxCluster * kVerifyWarps / 32; ++u) {
                        sum += x[u].sum * ex2_approx((x[u].top - sx.top) * scale);
                        dsum += x[u].draft_sum * ex2_approx((x[u].draft_top - sy.top) * scale);
                    }
                    sx.sum = pack2(sum, 0.f);
                    sy.sum = pack2(dsum, 0.f);
                    step = VerifyStep{kVerifyNext, any ? s.node[cur].child : -1, 0.f, 0.f, 0.f, 0.f, 0.f, 1.f, 0.f};
                    reduce_sums(sx, sy, step.top, sum, step.draft_top, dsum);
                    step.inv = rcp_approx(sum);
                    step.draft_inv = DRAFT && any ? rcp_approx(dsum) : 0.f;
                    // (NaN, an infinity, or nothing to choose from)
                    if (!(sum >= 0.5f) || (DRAFT && any && !(dsum >= 0.5f))) step.verdict = kVerifyDone;
                } else {
                    step = s.step;
                    step.rest = 0.f;
                    for (int32_t e = lane; e < parts; e += 32) step.rest += all[e].sum;
                    for (int off = 16; off > 0; off >>= 1) step.rest += __shfl_xor_sync(0xffffffffu, step.rest, off);
                    step.verdict = kVerifyNext;
                }
                while (step.verdict == kVerifyNext && step.node >= 0) {
                    const int32_t j = step.node;
                    const VerifyNode n = s.node[j];
                    step.node = n.sibling;
                    if (n.token < 0 || n.token >= vocab) {
                        if (rank == 0 && lane == 0) raise_error(PA_DEVERR_TREE);
                        continue;
                    }
                    const float2 l = s.logit[j];
                    float left = fine.power(l.x, step.top) * step.inv, ask = n.uniform * step.rest;
                    if (DRAFT) {
                        const float qt = fine.power(l.y, step.draft_top) * step.draft_inv;
                        left = fmaxf(fmaf(-step.spent, qt, left), 0.f);
                        ask *= qt;
                    } else {
                        for (int32_t k = s.node[cur].child; k != j; k = s.node[k].sibling)   // tried before
                            if (s.node[k].token == n.token) left = 0.f;
                    }
                    if (ask < left) {
                        step.verdict = kVerifyHolds;
                        step.node = j;
                    } else if (DRAFT) {
                        step.spent += step.rest;
                        if (step.node >= 0) step.verdict = kVerifyRest;
                    } else {
                        step.rest = fmaxf(step.rest - left, 0.f);
                    }
                }
                __syncwarp();
                if (lane == 0) s.step = step;
            }
            __syncthreads();
            verdict = s.step.verdict;
            if (!DRAFT || verdict != kVerifyRest) break;
            // what is left of P
            float sum = 0.f;
            const float top = s.step.top, draft_top = s.step.draft_top, inv = s.step.inv;
            const float share = s.step.spent * s.step.draft_inv;
            for (int32_t o = Eight<WIDE>::first(lo); o < hi; o += Eight<WIDE>::kNext) {
                Octet<E, WIDE> x, y;
                float up[8], down[8];
                x.load(row, o, hi);
                y.load(drow, o, hi);
                x.powers(top, scale, up);
                y.powers(draft_top, scale, down);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += fmaxf(fmaf(down[i], -share, up[i] * inv), 0.f);
            }
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            all = exchange(VerifyPart{0.f, sum, 0.f, 0.f});
        }
        if (verdict == kVerifyDone) {
            finish(PA_DEVERR_LOGITS, -1, -1);
            return;
        }
        if (verdict != kVerifyHolds) break;
        cur = s.step.node;
        any = s.node[cur].child >= 0;
    }

    // the next token: of the rest, or of P itself where rounding left none
    RaceField<E, DRAFT, WIDE> field{target + (int64_t)(q0 + cur) * a.logit_stride,
                                    DRAFT ? draft + (int64_t)(q0 + cur) * a.draft_stride : nullptr,
                                    noise, s.node, fine, s.step.top, s.step.draft_top,
                                    s.step.spent * s.step.draft_inv / s.step.inv, lo, hi,
                                    any ? s.node[cur].child : -1};
    bool finely = false;
    while (true) {
        Race best = finely ? field.run_finely(s.step.floor) : field.run();
        best.reduce();
        // the warps' best
        const VerifyPart* all = exchange(VerifyPart{best.first, __int_as_float(best.index), best.second, best.least});
        if (warp == 0) {
            best.start();
            for (int32_t e = lane; e < parts; e += 32) {
                const VerifyPart x = all[e];
                best.join(Race{x.top, x.draft_sum, x.draft_top, __float_as_int(x.sum)});
            }
            best.reduce();
            // all have it
            if (lane == 0) {
                s.step.node = best.index;
                s.step.floor = fmaxf(best.least, 0x1p-149f);
                s.step.verdict = best.index == INT32_MAX ? kVerifyRest
                                 : !finely && best.second >= best.least ? kVerifyFinely
                                                                        : kVerifyDone;
            }
        }
        __syncthreads();
        const int32_t verdict = s.step.verdict;
        if (verdict == kVerifyDone) {
            finish(0, cur, s.step.node);
            return;
        }
        finely = verdict == kVerifyFinely;
        if (!finely) {
            if (field.share == 0.f && field.child < 0) {
                finish(PA_DEVERR_LOGITS, -1, -1);
                return;
            }
            field.share = 0.f;
            field.child = -1;
        }
    }
}

}  // namespace pa

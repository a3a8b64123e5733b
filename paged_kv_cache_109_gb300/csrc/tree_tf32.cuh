// tree_tf32.cuh -- attention of a tree of drafted tokens over fp32 paged caches
// on the warp-level tensor cores, at fp32's accuracy: each operand goes in as
// two tf32 parts, x = hi + lo (hi: x rounded to 11 bits, lo = x - hi, of which
// the unit takes 11 more), and a product as hi hi + hi lo + lo hi.  What is
// dropped (lo lo, and lo's last bits) is under 2^-20 of the product, below what
// a 32-bit sum over a head dim of terms loses.  Head dims up to 256 whose rows
// are whole 16-byte pieces.
//
// A unit is one tile of 16 rows a warp ((node, query head) pairs, head fastest);
// a persistent CTA of one, two or four warps, the fewest that cover a sequence's
// rows, takes the parts of its range (tree_sched.cuh) one after another.  Keys
// come in chunks of KC through a double buffer of 16-byte cp.async copies:
//   S = Q K^T, online softmax in base 2 (S times scale log2 e), O += P V.
// A contraction's index may be taken in any order that both operands share, so
// the fragments are read 16 bytes at a time:
//   S: lane (g, t) holds columns 4 t .. 4 t + 3 of each 16 of Q's row g and K's
//      row g, two k-steps' worth;
//   O: step k takes keys 2 t (k = t) and 2 t + 1 (k = t + 4), which is where the
//      scores' accumulator has them, and column n of tile j is 4 n + j of each
//      32: lane (g, t) reads V[key][4 g .. 4 g + 3] for four tiles.
// Row strides put the 16-byte reads of eight lanes in different banks: Q and K
// 64 bytes off a multiple of 128, V 16 bytes off a multiple of 64.
//
// Bound: the products, 12 D operations per row and key (three for one) at the
// mma.sync tf32 rate (measured 300 TFLOP/s, so 100 of the operator's, against 73
// for FMAs); with one warp's rows in use, the copies.  Measured (D = 128, 38
// sequences x 8 kv heads x 4000 tokens): 64 rows 776 us = 51 TFLOP/s, 16 rows 438 us
// = 2840 GB/s; 16-key chunks with three CTAs an SM reached 47 TFLOP/s.
//
// In chunks that reach past the cached tokens, values of V that are not finite
// are taken out before the product, and added for the rows that see them.
//
// Two parts cannot hold an infinity, nor a value that 11 bits round up to 2^128
// (|x| >= 0x7f7ff000 as bits): hi - lo is then inf - inf, and what they meet, even
// with weight 0, becomes NaN.  No later step takes a NaN out of l or O (a NaN score
// is in l), so rows that end finite are right as they are; a CTA with one that does
// not goes through its range again and does such rows by FMAs (tree_plain_part),
// where a hidden key is not read and a visible infinity gives what the formula
// gives.  Without that look at the rows and with it, which finds nothing: 16 sequences
// of up to 24 nodes 140.6, 142.2 us; D = 256, 64 rows, 38 sequences x 2000 tokens 1060,
// 1078.  (Clamping each hi part instead took 152 and 1157, and would leave infinite
// operands to be told apart.)
#pragma once

#include "cp_async.cuh"
#include "tree_sched.cuh"
#include "tree_tiled.cuh"

namespace pa {

template <int DMAX, int KC, int WARPS>
struct TreeTfCfg {
    static_assert(DMAX % 32 == 0 && KC % 8 == 0, "tile shape");
    static constexpr int kThreads = 32 * WARPS;
    static constexpr int kRows = 16 * WARPS;
    // CTAs an SM holds at DMAX columns (the registers' limit for the compiler)
    static constexpr int kPerSm = DMAX > 128 ? (WARPS == 1 ? 2 : 1) : WARPS == 4 ? 2 : 4;
    // row strides in floats
    static __host__ __device__ int32_t k_stride(int32_t D) {
        const int32_t p = (D + 15) / 16 * 16;
        return p % 32 == 16 ? p : p + 16;
    }
    static __host__ __device__ int32_t v_stride(int32_t D) { return (D + 15) / 16 * 16 + 4; }
    // dynamic shared bytes: q [rows], K [2][KC], V [2][KC] rows | visible nodes
    // [rows][8] words | parents | odd keys of the chunk | a row to do again
    static size_t smem_bytes(int32_t D) {
        return 4 * ((size_t)(kRows + 2 * KC) * k_stride(D) + 2 * (size_t)KC * v_stride(D) +
                    kRows * (PA_MAX_TREE_NODES / 32) + PA_MAX_TREE_NODES + KC + 1);
    }
};

__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// hi: x rounded to tf32's 11 bits (half away from zero), lo: what is left.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ bool f32_odd(float x) { return !(fabsf(x) <= 3.4028235e38f); }

// Those rows of a part that did not end finite again, in 32-bit FMAs: a warp takes
// a row and 32 keys at a time, a lane a key's score and then every 32nd column of O.
// Keys that the row does not see are not read.  An infinite value or sum stays one
// under weights that underflow.
template <int DMAX, int WARPS>
__device__ __forceinline__ void tree_plain_part(const TreeArgs& a, const TreeWork& w, const TreeSeg& sg,
                                                int32_t keys, const uint32_t* bits) {
    constexpr int32_t kWords = PA_MAX_TREE_NODES / 32;
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t D = a.head_dim, HT = w.s.heads, hs = min(HT, a.group - sg.sg * HT);
    const int32_t* table = a.block_tables + (int64_t)sg.i * a.max_blocks;
    const float* kc = static_cast<const float*>(a.k_cache);
    const float* vc = static_cast<const float*>(a.v_cache);
    const int32_t key0 = sg.kb0 * keys, key1 = min((int64_t)sg.kb1 * keys, (int64_t)sg.T);
    const bool whole = sg.kb0 == 0 && sg.kb1 == sg.nb;
    float* cell = whole ? nullptr : tree_cell(a, w, sg);
#pragma unroll 1
    for (int32_t rho = warp; rho < sg.ntok * HT; rho += WARPS) {
        const int32_t tk = rho / HT, hh = rho - tk * HT;
        if (hh >= hs) continue;
        const int64_t row = ((int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + (int64_t)sg.g * a.group +
                             sg.sg * HT + hh) * D;
        const float* q = static_cast<const float*>(a.q) + row;
        float* out = static_cast<float*>(a.out) + row;
        float* ml = whole ? nullptr : cell + (size_t)D * 16 * WARPS + 2 * rho;
        auto sum_at = [&](int32_t d) { return cell + ((size_t)(d >> 2) * 16 * WARPS + rho) * 4 + (d & 3); };
        bool odd = !whole && f32_odd(ml[1]);
        for (int32_t d = lane; d < D; d += 32) odd |= f32_odd(whole ? out[d] : *sum_at(d));
        if (!__any_sync(0xffffffffu, odd)) continue;
        float m = -INFINITY, l = 0.f, acc[DMAX / 32];
#pragma unroll
        for (int32_t c = 0; c < DMAX / 32; ++c) acc[c] = 0.f;
#pragma unroll 1
        for (int32_t t0 = key0; t0 < key1; t0 += 32) {
            const int32_t t = t0 + lane, node = t - sg.C;
            bool sees = t < key1 && (node < 0 || (bits[tk * kWords + (node >> 5)] >> (node & 31) & 1u));
            int64_t at = 0;
            if (sees) {
                const int32_t id = table[t / a.block_size];
                sees = id >= 0 && id < a.num_blocks;
                at = (((int64_t)id * a.num_kv_heads + sg.g) * a.block_size + t % a.block_size) * D;
            }
            float s = sees ? 0.f : -INFINITY;
            for (int32_t d = 0; sees && d < D; d += 4) {
                const float4 y = *reinterpret_cast<const float4*>(kc + at + d);
                s = fmaf(q[d] * a.scale_log2, y.x, s);
                s = fmaf(q[d + 1] * a.scale_log2, y.y, s);
                s = fmaf(q[d + 2] * a.scale_log2, y.z, s);
                s = fmaf(q[d + 3] * a.scale_log2, y.w, s);
            }
            float mx = s;
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
            const float al = exp2f(m - ref), p = exp2f(s - ref);
            float sum = p;
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l = fmaf(l, al, sum);
            m = mn;
#pragma unroll
            for (int32_t c = 0; c < DMAX / 32; ++c)
                if (!f32_odd(acc[c])) acc[c] *= al;
            for (uint32_t left = __ballot_sync(0xffffffffu, sees); left != 0; left &= left - 1) {
                const int32_t k = __ffs(left) - 1;
                const float pk = __shfl_sync(0xffffffffu, p, k);
                const float* v = vc + __shfl_sync(0xffffffffu, at, k);
#pragma unroll
                for (int32_t c = 0; c < DMAX / 32; ++c) {
                    const int32_t d = lane + 32 * c;
                    if (d >= D) continue;
                    const float y = v[d];
                    acc[c] = f32_odd(y) ? acc[c] + y : fmaf(pk, y, acc[c]);
                }
            }
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int32_t c = 0; c < DMAX / 32; ++c) {
            const int32_t d = lane + 32 * c;
            if (d < D) *(whole ? out + d : sum_at(d)) = whole ? acc[c] * inv : acc[c];
        }
        if (!whole && lane == 0) *reinterpret_cast<float2*>(ml) = make_float2(m, l);
    }
}

// This CTA's range by tree_plain_part.
template <int DMAX, int WARPS>
__device__ __forceinline__ void tree_plain_range(const TreeArgs& a, const TreeWork& w, int32_t keys,
                                                 uint32_t* bits, int32_t* up) {
    TreeIter it = tree_begin(a, w, reinterpret_cast<int64_t*>(bits));
    TreeSeg sg;
    __syncthreads();                     // the search's scratch is free
    while (tree_next(a, w.s, it, sg)) {
        tree_visible(a, sg, up, bits);
        tree_plain_part<DMAX, WARPS>(a, w, sg, keys, bits);
        __syncthreads();                 // the node masks are free
    }
}

template <int DMAX, int KC, int WARPS>
__global__ void __launch_bounds__(TreeTfCfg<DMAX, KC, WARPS>::kThreads, TreeTfCfg<DMAX, KC, WARPS>::kPerSm)
tree_tf32_kernel(const TreeArgs a, const TreeWork w) {
    using C = TreeTfCfg<DMAX, KC, WARPS>;
    constexpr int NT = KC / 8;           // key tiles
    constexpr int CG = DMAX / 32;        // 32-column groups of O
    constexpr int kWords = PA_MAX_TREE_NODES / 32;
    extern __shared__ __align__(16) float sm_tf[];
    griddep_wait();                      // inputs may come from the previous kernel
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t grp = lane >> 2, tig = lane & 3;
    const int32_t D = a.head_dim, G = a.group, BS = a.block_size;
    const int32_t HT = w.s.heads;
    const int32_t kst = C::k_stride(D), vst = C::v_stride(D), ppr = D / 4;
    float* qs = sm_tf;                                          // [rows][kst]
    float* ks = qs + C::kRows * kst;                         // [2][KC][kst]
    float* vs = ks + 2 * KC * kst;                              // [2][KC][vst]
    uint32_t* bits = reinterpret_cast<uint32_t*>(vs + 2 * KC * vst);   // [tokens][8]
    int32_t* up = reinterpret_cast<int32_t*>(bits + C::kRows * kWords);
    int32_t* odd = up + PA_MAX_TREE_NODES;                      // [KC] key's V had values taken out
    int32_t* redo = odd + KC;                                   // a row did not end finite
    const float* q = static_cast<const float*>(a.q);
    const float* vc = static_cast<const float*>(a.v_cache);

    // columns of Q and K past the head dim stay zero
    for (int32_t x = tid; x < (C::kRows + 2 * KC) * kst; x += C::kThreads) qs[x] = 0.f;
    TreeIter it = tree_begin(a, w, reinterpret_cast<int64_t*>(bits));
    TreeSeg sg;
    TreeCut cut{};
    if (tid == 0) *redo = 0;
    __syncthreads();                     // the search's scratch is free
    while (tree_next(a, w.s, it, sg)) {
        if (sg.kb0 == 0 && sg.parts > 0)
            cut = TreeCut{sg.q0 + sg.tok0, sg.ntok, sg.g, sg.sg, sg.parts, {0, 0, 0}};
        const int32_t hs = min(HT, G - sg.sg * HT);
        const int64_t head_base = (int64_t)sg.g * G + sg.sg * HT;
        const int32_t* table = a.block_tables + (int64_t)sg.i * a.max_blocks;
        // Copies of chunk c (keys c KC ..) into buffer c & 1; keys past the last
        // and keys behind a bad table entry are filled with zeros.
        auto find = [&](int32_t c) {
            return tree_entry(a, sg, lane < KC && c < sg.kb1 ? c * KC + lane : sg.T);
        };
        auto issue = [&](int32_t c, TreeEntry e) {
            tree_copy<KC, WARPS>(a, tree_row(a, sg, e, warp == 0), ppr, smem_u32(ks + (c & 1) * KC * kst), kst * 4,
                          smem_u32(vs + (c & 1) * KC * vst), vst * 4);
            cp_async_commit();
        };
        // rows in use of Q (idle rows' scores reach no other row), a warp a row at a
        // time; plain loads where q is not 16-byte aligned
        const bool q16 = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0;
        for (int32_t rho = warp; rho < sg.ntok * HT; rho += WARPS) {
            const int32_t tk = rho / HT, hh = rho - tk * HT;
            if (hh >= hs) continue;
            const float* src = q + ((int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh) * D;
            for (int32_t d = 4 * lane; d < D; d += 128) {
                float* dst = qs + rho * kst + d;
                if (q16)
                    cp_async16(smem_u32(dst), src + d, 16u);
                else
                    *reinterpret_cast<float4*>(dst) =
                        make_float4(src[d], src[d + 1], src[d + 2], src[d + 3]);
            }
        }
        issue(sg.kb0, find(sg.kb0));       // q and the first chunk
        TreeEntry next = find(sg.kb0 + 1);
        tree_visible(a, sg, up, bits);

        // this lane's two rows: warp * 16 + grp (half 0) and + 8 (half 1)
        bool rvalid[2];
        int32_t rtok[2];
#pragma unroll
        for (int32_t h = 0; h < 2; ++h) {
            const int32_t rho = warp * 16 + grp + 8 * h, tk = rho / HT, hh = rho - tk * HT;
            rvalid[h] = tk < sg.ntok && hh < hs;
            rtok[h] = min(tk, sg.ntok - 1);
        }
        const bool busy = warp * 16 / HT < sg.ntok;      // the warp has rows in use
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float acc[CG][4][4];
#pragma unroll
        for (int32_t cg = 0; cg < CG; ++cg)
#pragma unroll
            for (int32_t j = 0; j < 4; ++j) acc[cg][j][0] = acc[cg][j][1] = acc[cg][j][2] = acc[cg][j][3] = 0.f;

        for (int32_t c = sg.kb0; c < sg.kb1; ++c) {
            if (c + 1 < sg.kb1) {          // next chunk in flight while this one is used
                issue(c + 1, next);
                next = find(c + 2);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            const int32_t t0 = c * KC;
            const bool masked = t0 + KC > sg.C;
            for (int32_t k = tid; masked && k < KC; k += C::kThreads) odd[k] = 0;
            __syncthreads();               // chunk c (and q) visible to every warp
            const float* kb = ks + (c & 1) * KC * kst;
            float* vb = vs + (c & 1) * KC * vst;
            if (masked) {
                for (int32_t x = tid; x < KC * D; x += C::kThreads) {
                    const int32_t k = x / D;
                    float* p = vb + k * vst + (x - k * D);
                    if (f32_odd(*p)) {
                        *p = 0.f;
                        odd[k] = 1;
                    }
                }
                __syncthreads();
            }
            if (busy) {
                // (the corrections are summed apart: a tensor-core sum cuts off
                // what it cannot hold, so long chains drift)
                float s[NT][4], sc[NT][4], sd[NT][4];
#pragma unroll
                for (int32_t n = 0; n < NT; ++n)
#pragma unroll
                    for (int32_t e = 0; e < 4; ++e) s[n][e] = sc[n][e] = sd[n][e] = 0.f;
                const float* qa = qs + (warp * 16 + grp) * kst + 4 * tig;
                const float* ka = kb + grp * kst + 4 * tig;
#pragma unroll 2
                for (int32_t d0 = 0; d0 < D; d0 += 16) {
                    const float4 x0 = *reinterpret_cast<const float4*>(qa + d0);
                    const float4 x1 = *reinterpret_cast<const float4*>(qa + 8 * kst + d0);
                    uint32_t ah[2][4], al[2][4];
                    split_tf32(x0.x, ah[0][0], al[0][0]);
                    split_tf32(x1.x, ah[0][1], al[0][1]);
                    split_tf32(x0.y, ah[0][2], al[0][2]);
                    split_tf32(x1.y, ah[0][3], al[0][3]);
                    split_tf32(x0.z, ah[1][0], al[1][0]);
                    split_tf32(x1.z, ah[1][1], al[1][1]);
                    split_tf32(x0.w, ah[1][2], al[1][2]);
                    split_tf32(x1.w, ah[1][3], al[1][3]);
#pragma unroll
                    for (int32_t n = 0; n < NT; ++n) {
                        const float4 y = *reinterpret_cast<const float4*>(ka + n * 8 * kst + d0);
                        uint32_t bh[4], bl[4];
                        split_tf32(y.x, bh[0], bl[0]);
                        split_tf32(y.y, bh[1], bl[1]);
                        split_tf32(y.z, bh[2], bl[2]);
                        split_tf32(y.w, bh[3], bl[3]);
#pragma unroll
                        for (int32_t e = 0; e < 2; ++e) {
                            mma_tf32_1688(s[n], ah[e], bh[2 * e], bh[2 * e + 1]);
                            mma_tf32_1688(sc[n], al[e], bh[2 * e], bh[2 * e + 1]);
                            mma_tf32_1688(sd[n], ah[e], bl[2 * e], bl[2 * e + 1]);
                        }
                    }
                }
#pragma unroll
                for (int32_t n = 0; n < NT; ++n)
#pragma unroll
                    for (int32_t e = 0; e < 4; ++e)
                        s[n][e] = (s[n][e] + (sc[n][e] + sd[n][e])) * a.scale_log2;

                // mask, online softmax of rows grp (h = 0) and grp + 8 (h = 1);
                // a row's columns are spread over its 4 lanes
                float al[2];
#pragma unroll
                for (int32_t h = 0; h < 2; ++h) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int32_t n = 0; n < NT; ++n)
#pragma unroll
                        for (int32_t e = 0; e < 2; ++e) {
                            float& x = s[n][2 * h + e];
                            bool sees = rvalid[h];
                            if (masked && sees) {
                                const int32_t k = t0 + n * 8 + 2 * tig + e - sg.C;
                                sees = k < 0 || (k < sg.n && (bits[rtok[h] * kWords + (k >> 5)] >> (k & 31) & 1u));
                            }
                            x = sees ? x : -INFINITY;
                            mx = fmaxf(mx, x);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m[h], mx);
                    const float mref = mn == -INFINITY ? 0.f : mn;   // no visible key yet
                    al[h] = exp2f(m[h] - mref);                       // 0 while m = -inf
                    float sum = 0.f;
#pragma unroll
                    for (int32_t n = 0; n < NT; ++n)
#pragma unroll
                        for (int32_t e = 0; e < 2; ++e) {
                            float& x = s[n][2 * h + e];
                            x = exp2f(x - mref);                      // 0 for masked keys
                            sum += x;
                        }
                    l[h] = l[h] * al[h] + sum;                        // this lane's columns only
                    m[h] = mn;
                }

                // O = a O + P V: a chunk's products from zero, then one rounded sum
                uint32_t ph[NT][4], pl[NT][4];
#pragma unroll
                for (int32_t n = 0; n < NT; ++n) {
                    split_tf32(s[n][0], ph[n][0], pl[n][0]);
                    split_tf32(s[n][2], ph[n][1], pl[n][1]);
                    split_tf32(s[n][1], ph[n][2], pl[n][2]);
                    split_tf32(s[n][3], ph[n][3], pl[n][3]);
                }
                const float* va = vb + 2 * tig * vst + 4 * grp;
#pragma unroll
                for (int32_t cg = 0; cg < CG; ++cg) {
                    if (cg * 32 < D) {
                        float o[4][4], oc[4][4];
#pragma unroll
                        for (int32_t j = 0; j < 4; ++j)
#pragma unroll
                            for (int32_t e = 0; e < 4; ++e) o[j][e] = oc[j][e] = 0.f;
#pragma unroll
                        for (int32_t n = 0; n < NT; ++n) {
                            // (columns past the head dim hold anything: they are
                            // never stored)
                            const float4 y0 = *reinterpret_cast<const float4*>(va + n * 8 * vst + cg * 32);
                            const float4 y1 = *reinterpret_cast<const float4*>(va + (n * 8 + 1) * vst + cg * 32);
                            const float e0[4] = {y0.x, y0.y, y0.z, y0.w}, e1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                            for (int32_t j = 0; j < 4; ++j) {
                                uint32_t h0, l0, h1, l1;
                                split_tf32(e0[j], h0, l0);
                                split_tf32(e1[j], h1, l1);
                                mma_tf32_1688(o[j], ph[n], h0, h1);
                                mma_tf32_1688(oc[j], pl[n], h0, h1);
                                mma_tf32_1688(oc[j], ph[n], l0, l1);
                            }
                        }
#pragma unroll
                        for (int32_t j = 0; j < 4; ++j)
#pragma unroll
                            for (int32_t e = 0; e < 4; ++e)
                                acc[cg][j][e] = fmaf(acc[cg][j][e], al[e >> 1], o[j][e] + oc[j][e]);
                    }
                }
                // values of V that were taken out, for the rows that see them
                // (infinite or NaN: any positive weight gives the same)
                for (int32_t k = 0; masked && k < KC && t0 + k < sg.T; ++k) {
                    if (!odd[k]) continue;
                    const int32_t node = t0 + k - sg.C, id = table[(t0 + k) / BS];
                    if (id < 0 || id >= a.num_blocks) continue;
                    const float* v = vc + (((int64_t)id * a.num_kv_heads + sg.g) * BS + (t0 + k) % BS) * D;
#pragma unroll
                    for (int32_t h = 0; h < 2; ++h) {
                        if (!rvalid[h] ||
                            !(node < 0 || (bits[rtok[h] * kWords + (node >> 5)] >> (node & 31) & 1u)))
                            continue;
#pragma unroll
                        for (int32_t cg = 0; cg < CG; ++cg)
#pragma unroll
                            for (int32_t j = 0; j < 4; ++j)
#pragma unroll
                                for (int32_t e = 0; e < 2; ++e) {
                                    const int32_t col = cg * 32 + 8 * tig + 4 * e + j;
                                    if (col < D && f32_odd(v[col])) acc[cg][j][2 * h + e] += v[col];
                                }
                    }
                }
            }
            __syncthreads();               // buffer c & 1 is free
        }

        // row sums over the row's 4 lanes, then out = O / l, or the cells
#pragma unroll
        for (int32_t h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        const bool whole = sg.kb0 == 0 && sg.kb1 == sg.nb;
        float* cell = whole ? nullptr : tree_cell(a, w, sg);
#pragma unroll
        for (int32_t h = 0; h < 2; ++h) {
            if (!rvalid[h]) continue;
            const int32_t rho = warp * 16 + grp + 8 * h, tk = rho / HT, hh = rho - tk * HT;
            const int64_t row = (int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh;
            const float inv = whole ? (l[h] != 0.f ? 1.f / l[h] : 0.f) : 1.f;
            float* dst = whole ? static_cast<float*>(a.out) + row * D : cell + (size_t)rho * 4;
#pragma unroll
            for (int32_t cg = 0; cg < CG; ++cg)
#pragma unroll
                for (int32_t e = 0; e < 2; ++e) {
                    const int32_t col = cg * 32 + 8 * tig + 4 * e;
                    if (col < D) {
                        const float4 o = make_float4(acc[cg][0][2 * h + e] * inv, acc[cg][1][2 * h + e] * inv,
                                                     acc[cg][2][2 * h + e] * inv, acc[cg][3][2 * h + e] * inv);
                        *reinterpret_cast<float4*>(dst + (whole ? col : (size_t)col * C::kRows)) = o;
                        if (f32_odd(o.x) || f32_odd(o.y) || f32_odd(o.z) || f32_odd(o.w)) *redo = 1;
                    }
                }
            if (f32_odd(l[h])) *redo = 1;
            if (!whole && tig == 0)
                *reinterpret_cast<float2*>(cell + (size_t)D * C::kRows + 2 * rho) =
                    make_float2(m[h], l[h]);
        }
        __syncthreads();                   // q and the node masks are free
    }
    if (w.cuts != nullptr && tid == 0) w.cuts[blockIdx.x] = cut;
    __syncthreads();
    if (*redo) tree_plain_range<DMAX, WARPS>(a, w, KC, bits, up);
    griddep_launch_dependents();
}

}  // namespace pa

// tree_mma.cuh -- attention of a tree of drafted tokens over the paged cache on
// the warp-level tensor-core path (mma.sync m16n8k16), bf16: head dims that are
// multiples of 16 up to 256 which the tcgen05 kernel does not take (above 128,
// block sizes that are not multiples of 8, queries in host memory, unaligned
// outputs, scale <= 0).
//
// A unit is one tile of 16 rows a warp ((node, query head) pairs, head fastest);
// a persistent CTA of one, two or four warps, the fewest that cover a sequence's
// rows, takes the parts of its range (tree_sched.cuh) one after another.  Keys
// come in chunks of KC through a double buffer of 16-byte cp.async copies, rows
// padded by 16 bytes so that an ldmatrix reads eight bank groups:
//   S = Q K^T, online softmax in base 2, O += P V with P as bf16 hi + lo (about
//   16 significant bits, as in the other tensor-core kernels).
// Bound: the products of mma.sync, 6 D operations per row and key with both
// parts of P; a chunk's copies run beside the chunk before.  Measured (38 sequences
// x 8 kv heads x 4000 tokens, 64 rows): D = 256 567 us = 141 TFLOP/s of the
// operator's 4 D, D = 128 with 4-token blocks 345 us = 115 TFLOP/s, where mma.sync
// reaches 603 (402 of the operator's); 16 rows, D = 128: 204 us = 3060 GB/s.
//
// In chunks that reach past the cached tokens, values of V that are not finite
// are taken out of shared memory before the product (0 times NaN would reach
// rows that do not see the node); the rows that see such a node add them at
// the end of the chunk.
#pragma once

#include "cp_async.cuh"
#include "tree_sched.cuh"
#include "tree_tiled.cuh"
#include "tree_ws.cuh"

namespace pa {

template <int DMAX, int KC, int WARPS>
struct TreeMmaCfg {
    static_assert(DMAX % 16 == 0 && KC % 32 == 0, "tile shape");
    static constexpr int kThreads = 32 * WARPS;
    static constexpr int kRows = 16 * WARPS;
    // CTAs an SM holds at DMAX columns (the registers' limit for the compiler)
    static constexpr int kPerSm = WARPS == 4 ? 2 : 4;

    // dynamic shared bytes: q [rows][row + 16] | K, V double buffer [KC][row + 16]
    // | visible nodes [rows][8] words | parents | odd rows of the chunk
    static size_t smem_bytes(int32_t head_dim) {
        const size_t stride = (size_t)head_dim * 2 + 16;
        return kRows * stride + 4 * (size_t)KC * stride +
               kRows * (PA_MAX_TREE_NODES / 8) + PA_MAX_TREE_NODES * 4 + KC * 4;
    }
};

template <int DMAX, int KC, int WARPS>
__global__ void __launch_bounds__(TreeMmaCfg<DMAX, KC, WARPS>::kThreads, TreeMmaCfg<DMAX, KC, WARPS>::kPerSm)
tree_mma_kernel(const TreeArgs a, const TreeWork w) {
    using C = TreeMmaCfg<DMAX, KC, WARPS>;
    constexpr int NT = KC / 8;           // key n-tiles of S
    constexpr int DT = DMAX / 8;         // column n-tiles of O
    constexpr int kWords = PA_MAX_TREE_NODES / 32;
    extern __shared__ __align__(16) uint8_t sm_tm[];
    griddep_wait();                      // inputs may come from the previous kernel
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t grp = lane >> 2, tig = lane & 3;
    const int32_t lm = lane >> 3, lr = lane & 7;      // ldmatrix: matrix, row in matrix
    const int32_t D = a.head_dim, G = a.group, BS = a.block_size;
    const int32_t HT = w.s.heads;
    const int32_t rowb = D * 2, stride = rowb + 16, ppr = rowb / 16;
    uint8_t* qsm = sm_tm;                                       // [rows][stride]
    uint8_t* kvs = sm_tm + C::kRows * stride;               // [2][K, V][KC][stride]
    uint32_t* bits = reinterpret_cast<uint32_t*>(kvs + 4 * KC * stride);   // [tokens][8]
    int32_t* up = reinterpret_cast<int32_t*>(bits + C::kRows * kWords);
    int32_t* odd = up + PA_MAX_TREE_NODES;                      // [KC] key's V had values taken out
    const uint32_t q_u = smem_u32(qsm), kv_u = smem_u32(kvs);
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.v_cache);

    TreeIter it = tree_begin(a, w, reinterpret_cast<int64_t*>(sm_tm));
    TreeSeg sg;
    TreeCut cut{};
    __syncthreads();                     // the search's scratch is the queries' place
    while (tree_next(a, w.s, it, sg)) {
        if (sg.kb0 == 0 && sg.parts > 0)
            cut = TreeCut{sg.q0 + sg.tok0, sg.ntok, sg.g, sg.sg, sg.parts, {0, 0, 0}};
        const int32_t hs = min(HT, G - sg.sg * HT);
        const int64_t head_base = (int64_t)sg.g * G + sg.sg * HT;
        const int32_t* table = a.block_tables + (int64_t)sg.i * a.max_blocks;
        // Q rows of the tile (zeros for idle rows; plain loads where q is not
        // 16-byte aligned)
        const bool q16 = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0;
        for (int32_t x = tid; x < C::kRows * ppr; x += C::kThreads) {
            const int32_t rho = x / ppr, piece = x - rho * ppr;
            const int32_t tk = rho / HT, hh = rho - tk * HT;
            const bool ok = tk < sg.ntok && hh < hs;
            const int64_t row = ok ? (int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh : 0;
            const __nv_bfloat16* src = q + row * D + piece * 8;
            if (q16) {
                cp_async16(q_u + rho * stride + piece * 16, src, ok ? 16u : 0u);
            } else {
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(qsm + rho * stride + piece * 16);
#pragma unroll
                for (int32_t e = 0; e < 8; ++e) dst[e] = ok ? src[e] : __float2bfloat16(0.f);
            }
        }
        // Copies of chunk c (keys c KC ..) into buffer c & 1, 32 keys at a time;
        // keys past the last and keys behind a bad table entry are filled with
        // zeros.
        constexpr int32_t kSub = KC / 32;
        auto find = [&](int32_t c, TreeEntry (&e)[kSub]) {
#pragma unroll
            for (int32_t u = 0; u < kSub; ++u)
                e[u] = tree_entry(a, sg, c < sg.kb1 ? c * KC + u * 32 + lane : sg.T);
        };
        auto issue = [&](int32_t c, const TreeEntry (&e)[kSub]) {
            const uint32_t kb = kv_u + (c & 1) * 2 * KC * stride;
#pragma unroll
            for (int32_t u = 0; u < kSub; ++u)
                tree_copy<32, WARPS>(a, tree_row(a, sg, e[u], warp == 0), ppr, kb + u * 32 * stride, stride,
                              kb + (KC + u * 32) * stride, stride);
            cp_async_commit();
        };
        TreeEntry next[kSub];
        find(sg.kb0, next);
        issue(sg.kb0, next);             // q and the first chunk
        find(sg.kb0 + 1, next);
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
        float acc[DT][4];
#pragma unroll
        for (int32_t nd = 0; nd < DT; ++nd) acc[nd][0] = acc[nd][1] = acc[nd][2] = acc[nd][3] = 0.f;

        for (int32_t c = sg.kb0; c < sg.kb1; ++c) {
            if (c + 1 < sg.kb1) {          // next chunk in flight while this one is used
                issue(c + 1, next);
                find(c + 2, next);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            const int32_t t0 = c * KC;
            const bool masked = t0 + KC > sg.C;
            for (int32_t k = tid; masked && k < KC; k += C::kThreads) odd[k] = 0;
            __syncthreads();               // chunk c (and q) visible to every warp
            uint8_t* vsm = kvs + ((c & 1) * 2 + 1) * KC * stride;
            if (masked) {
                for (int32_t x = tid; x < KC * ppr; x += C::kThreads) {
                    const int32_t k = x / ppr, piece = x - k * ppr;
                    uint4* p = reinterpret_cast<uint4*>(vsm + k * stride + piece * 16);
                    const uint4 v = *p;
                    if (bf16x2_odd(v.x) || bf16x2_odd(v.y) || bf16x2_odd(v.z) || bf16x2_odd(v.w)) {
                        *p = make_uint4(bf16x2_clean(v.x), bf16x2_clean(v.y), bf16x2_clean(v.z),
                                        bf16x2_clean(v.w));
                        odd[k] = 1;
                    }
                }
                __syncthreads();
            }
            if (busy) {
                const uint32_t kb = kv_u + (c & 1) * 2 * KC * stride;
                const uint32_t vb = kb + KC * stride;

                // S = Q K^T: per 16 columns of D, one Q fragment against every
                // 16-key pair of n-tiles
                float s[NT][4];
#pragma unroll
                for (int32_t n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                for (int32_t ks = 0; ks < DMAX / 16; ++ks) {
                    if (ks < D / 16) {
                        uint32_t qa[4];
                        ldsm_x4(q_u + (warp * 16 + (lm & 1) * 8 + lr) * stride + (ks * 16 + (lm >> 1) * 8) * 2,
                                qa[0], qa[1], qa[2], qa[3]);
#pragma unroll
                        for (int32_t kp = 0; kp < KC / 16; ++kp) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(kb + (kp * 16 + (lm >> 1) * 8 + lr) * stride +
                                        (ks * 16 + (lm & 1) * 8) * 2,
                                    b0, b1, b2, b3);
                            mma_bf16_16816(s[2 * kp], qa, b0, b1);
                            mma_bf16_16816(s[2 * kp + 1], qa, b2, b3);
                        }
                    }
                }

                // scale, mask, online softmax of rows grp (h = 0) and grp + 8
                // (h = 1); a row's columns are spread over its 4 lanes
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
                            x = sees ? x * a.scale_log2 : -INFINITY;
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
#pragma unroll
                for (int32_t nd = 0; nd < DT; ++nd) {
                    acc[nd][0] *= al[0];
                    acc[nd][1] *= al[0];
                    acc[nd][2] *= al[1];
                    acc[nd][3] *= al[1];
                }

                // O += P V, P from the S registers (two key n-tiles = one k
                // step), hi and lo against the same V fragments
#pragma unroll
                for (int32_t kp = 0; kp < KC / 16; ++kp) {
                    uint32_t pf[4], pl[4];
                    split_bf16x2(s[2 * kp][0], s[2 * kp][1], pf[0], pl[0]);
                    split_bf16x2(s[2 * kp][2], s[2 * kp][3], pf[1], pl[1]);
                    split_bf16x2(s[2 * kp + 1][0], s[2 * kp + 1][1], pf[2], pl[2]);
                    split_bf16x2(s[2 * kp + 1][2], s[2 * kp + 1][3], pf[3], pl[3]);
#pragma unroll
                    for (int32_t dp = 0; dp < DMAX / 16; ++dp) {
                        if (dp < D / 16) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4_trans(vb + (kp * 16 + (lm & 1) * 8 + lr) * stride +
                                              (dp * 16 + (lm >> 1) * 8) * 2,
                                          b0, b1, b2, b3);
                            mma_bf16_16816(acc[2 * dp], pf, b0, b1);
                            mma_bf16_16816(acc[2 * dp + 1], pf, b2, b3);
                            mma_bf16_16816(acc[2 * dp], pl, b0, b1);
                            mma_bf16_16816(acc[2 * dp + 1], pl, b2, b3);
                        }
                    }
                }
                // values of V that were taken out, for the rows that see them
                // (infinite or NaN: any positive weight gives the same)
                for (int32_t k = 0; masked && k < KC && t0 + k < sg.T; ++k) {
                    if (!odd[k]) continue;
                    const int32_t node = t0 + k - sg.C, id = table[(t0 + k) / BS];
                    if (id < 0 || id >= a.num_blocks) continue;
                    const __nv_bfloat16* v =
                        vc + (((int64_t)id * a.num_kv_heads + sg.g) * BS + (t0 + k) % BS) * D;
#pragma unroll
                    for (int32_t h = 0; h < 2; ++h) {
                        if (!rvalid[h] ||
                            !(node < 0 || (bits[rtok[h] * kWords + (node >> 5)] >> (node & 31) & 1u)))
                            continue;
#pragma unroll
                        for (int32_t nd = 0; nd < DT; ++nd)
#pragma unroll
                            for (int32_t e = 0; e < 2; ++e)
                                if (nd < D / 8) {
                                    const float y = __bfloat162float(v[nd * 8 + 2 * tig + e]);
                                    if (!(fabsf(y) <= 3.4028235e38f)) acc[nd][2 * h + e] += y;
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
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
#pragma unroll
        for (int32_t h = 0; h < 2; ++h) {
            if (!rvalid[h]) continue;
            const int32_t rho = warp * 16 + grp + 8 * h, tk = rho / HT, hh = rho - tk * HT;
            const int64_t row = (int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh;
            const float inv = l[h] != 0.f ? 1.f / l[h] : 0.f;
#pragma unroll
            for (int32_t nd = 0; nd < DT; ++nd) {
                if (nd >= D / 8) continue;
                const int32_t col = nd * 8 + 2 * tig;
                const float x = acc[nd][2 * h], y = acc[nd][2 * h + 1];
                if (whole) {
                    out[row * D + col] = __float2bfloat16_rn(x * inv);
                    out[row * D + col + 1] = __float2bfloat16_rn(y * inv);
                } else {
                    *reinterpret_cast<float2*>(cell + ((size_t)(col >> 2) * C::kRows + rho) * 4 +
                                               (col & 3)) = make_float2(x, y);
                }
            }
            if (!whole && tig == 0)
                *reinterpret_cast<float2*>(cell + (size_t)D * C::kRows + 2 * rho) =
                    make_float2(m[h], l[h]);
        }
        __syncthreads();                   // q and the node masks are free
    }
    if (w.cuts != nullptr && tid == 0) w.cuts[blockIdx.x] = cut;
    griddep_launch_dependents();
}

}  // namespace pa

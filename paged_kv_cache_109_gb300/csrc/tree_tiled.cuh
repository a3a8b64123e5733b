// tree_tiled.cuh -- attention of a tree of drafted tokens over the paged cache on
// CUDA cores, in 32-bit arithmetic, for the bf16 shapes that no tensor-core
// kernel takes: head dims up to 256 that are multiples of 8 but not of 16.
//
// A unit is one tile of R = 16 RPT rows ((node, query head) pairs, head
// fastest); a persistent CTA of 128 threads takes the parts of its range
// (tree_sched.cuh) one after another.  Keys come in chunks of KC through a
// double buffer of 16-byte cp.async copies; thread (rg, kg), rg = tid / 8 and
// kg = tid % 8, owns rows rg RPT .. rg RPT + RPT - 1, the scores of keys kg,
// kg + 8, ... and float4 column groups kg, kg + 8, ... of the accumulator:
//   S = Q K^T (q scaled by scale log2 e), online softmax in base 2, O += P V.
// Rows in shared memory are padded by 16 bytes: the four row groups of a warp
// then read Q and P from different banks.
//
// Bound: the FMAs, 4 D per row and key; K and V are read once per R rows.
// Measured: D = 72, 38 sequences x 16 kv heads x 4000 tokens, 64 rows 2.46 ms (18
// TFLOP/s of the 73 that FMAs reach), 16 rows 0.96 ms.  Two rows a thread above 128
// columns spill (144 bytes stored a thread).
// RPT is the smallest of 1, 2, 4 (up to 128 columns) that covers a sequence's
// rows, so a small tree does not pay for idle rows.
//
// In chunks that reach past the cached tokens a key that a row does not see
// has weight -1, which the product skips: its V (NaN, say) leaves no trace.
#pragma once

#include "cp_async.cuh"
#include "prefill_tiled.cuh"
#include "tree_sched.cuh"

namespace pa {

constexpr int kTreeTiledThreads = 128;

template <int RPT, int NF, int KC>
struct TreeTiledCfg {
    static constexpr int kRows = 16 * RPT;
    static constexpr int kKeysPerThread = KC / 8;
    static_assert(KC % 8 == 0 && NF >= 1 && RPT >= 1, "tile shape");
    // dynamic shared bytes: q [rows][D + 4] fp32 | K, V double buffer
    // [KC][row + 16] | P [rows][KC + 4] | visible nodes [rows][8] | parents
    static size_t smem_bytes(int32_t head_dim, int32_t elem) {
        const size_t stride = (size_t)head_dim * elem + 16;
        return (size_t)kRows * (head_dim + 4) * 4 + 4 * (size_t)KC * stride +
               (size_t)kRows * (KC + 4) * 4 + (size_t)kRows * (PA_MAX_TREE_NODES / 8) +
               PA_MAX_TREE_NODES * 4;
    }
};

// Nodes each of the part's tokens sees: word x of token t in bits[t * 8 + x].
// All threads of the block; parents' staging in `up`.
__device__ __forceinline__ void tree_visible(const TreeArgs& a, const TreeSeg& sg, int32_t* up,
                                             uint32_t* bits) {
    constexpr int32_t kWords = PA_MAX_TREE_NODES / 32;
    for (int32_t j = threadIdx.x; j < sg.n; j += blockDim.x)
        up[j] = tree_parent(a.parents[sg.q0 + j], j, sg.g == 0 && sg.sg == 0 && sg.tok0 == 0);
    for (int32_t x = threadIdx.x; x < sg.ntok * kWords; x += blockDim.x) bits[x] = 0;
    __syncthreads();
    for (int32_t t = threadIdx.x; t < sg.ntok; t += blockDim.x)
        for (int32_t k = sg.tok0 + t; k >= 0; k = up[k]) bits[t * kWords + (k >> 5)] |= 1u << (k & 31);
    __syncthreads();
}

template <typename E, int RPT, int NF, int KC>
__global__ void __launch_bounds__(kTreeTiledThreads)
tree_tiled_kernel(const TreeArgs a, const TreeWork w) {
    using C = TreeTiledCfg<RPT, NF, KC>;
    constexpr int R = C::kRows, KPT = C::kKeysPerThread;
    constexpr int kE = (int)sizeof(E);
    constexpr int kWords = PA_MAX_TREE_NODES / 32;
    extern __shared__ __align__(16) uint8_t sm_tt[];
    griddep_wait();                 // inputs may come from the previous kernel
    const int32_t tid = threadIdx.x, rg = tid >> 3, kg = tid & 7;
    const int32_t D = a.head_dim, G = a.group;
    const int32_t HT = w.s.heads;
    const int32_t rowb = D * kE, stride = rowb + 16, ppr = rowb / 16;
    const int32_t qst = D + 4, pst = KC + 4;
    float* qs = reinterpret_cast<float*>(sm_tt);                          // [R][D + 4]
    uint8_t* kvs = sm_tt + (size_t)R * qst * 4;                           // [2][K, V][KC][stride]
    float* ps = reinterpret_cast<float*>(kvs + 2 * 2 * KC * stride);      // [R][KC + 4]
    uint32_t* bits = reinterpret_cast<uint32_t*>(ps + R * pst);           // [tokens][8]
    int32_t* up = reinterpret_cast<int32_t*>(bits + R * kWords);
    const E* q = static_cast<const E*>(a.q);

    TreeIter it = tree_begin(a, w, reinterpret_cast<int64_t*>(sm_tt));
    TreeSeg sg;
    TreeCut cut{};
    __syncthreads();                // the search's scratch is the queries' place
    while (tree_next(a, w.s, it, sg)) {
        if (sg.kb0 == 0 && sg.parts > 0)
            cut = TreeCut{sg.q0 + sg.tok0, sg.ntok, sg.g, sg.sg, sg.parts, {0, 0, 0}};
        const int32_t hs = min(HT, G - sg.sg * HT);
        const int64_t head_base = (int64_t)sg.g * G + sg.sg * HT;
        // Copies of chunk c (keys c KC ..) into buffer c & 1; keys past the last
        // and keys behind a bad table entry are filled with zeros.
        auto find = [&](int32_t c) {
            return tree_entry(a, sg, (tid & 31) < KC && c < sg.kb1 ? c * KC + (tid & 31) : sg.T);
        };
        auto issue = [&](int32_t c, TreeEntry e) {
            const uint32_t kb = smem_u32(kvs + (c & 1) * 2 * KC * stride);
            tree_copy<KC, kTreeTiledThreads / 32>(a, tree_row(a, sg, e, tid < 32), ppr, kb, stride, kb + KC * stride, stride);
            cp_async_commit();
        };
        issue(sg.kb0, find(sg.kb0));
        TreeEntry next = find(sg.kb0 + 1);
        // Q rows, eight rows' loads of a warp at a time (zeros in idle rows)
        for (int32_t r0 = tid >> 5; r0 < R; r0 += 8 * (kTreeTiledThreads / 32)) {
            for (int32_t d = tid & 31; d < D; d += 32) {
                float v[8];
#pragma unroll
                for (int32_t u = 0; u < 8; ++u) {
                    const int32_t rho = r0 + u * (kTreeTiledThreads / 32), tk = rho / HT, hh = rho - tk * HT;
                    v[u] = 0.f;
                    if (tk < sg.ntok && hh < hs)
                        v[u] = Elem<E>::to_float(
                            q[((int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh) * D + d]);
                }
#pragma unroll
                for (int32_t u = 0; u < 8; ++u) {
                    const int32_t rho = r0 + u * (kTreeTiledThreads / 32);
                    if (rho < R) qs[rho * qst + d] = v[u] * a.scale_log2;
                }
            }
        }
        tree_visible(a, sg, up, bits);

        // this thread's rows: validity and token
        bool rvalid[RPT];
        int32_t rtok[RPT];
        float m[RPT], l[RPT];
        float4 acc[RPT][NF];
#pragma unroll
        for (int32_t r = 0; r < RPT; ++r) {
            const int32_t rho = rg * RPT + r, tk = rho / HT, hh = rho - tk * HT;
            rvalid[r] = tk < sg.ntok && hh < hs;
            rtok[r] = min(tk, sg.ntok - 1);
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int32_t f = 0; f < NF; ++f) acc[r][f] = make_float4(0.f, 0.f, 0.f, 0.f);
        }

        for (int32_t c = sg.kb0; c < sg.kb1; ++c) {
            if (c + 1 < sg.kb1) {      // next chunk in flight while this one is used
                issue(c + 1, next);
                next = find(c + 2);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncthreads();           // chunk c (and q) visible to every thread
            const uint8_t* kb = kvs + (c & 1) * 2 * KC * stride;
            const uint8_t* vb = kb + KC * stride;
            const int32_t t0 = c * KC;
            const bool masked = t0 + KC > sg.C;

            // scores of rows rg RPT + r and keys kg + 8 j
            float s[RPT][KPT];
#pragma unroll
            for (int32_t r = 0; r < RPT; ++r)
#pragma unroll
                for (int32_t j = 0; j < KPT; ++j) s[r][j] = 0.f;
#pragma unroll 4
            for (int32_t d4 = 0; d4 < D / 4; ++d4) {
                float4 qv[RPT], kv4[KPT];
#pragma unroll
                for (int32_t r = 0; r < RPT; ++r)
                    qv[r] = *reinterpret_cast<const float4*>(qs + (rg * RPT + r) * qst + 4 * d4);
#pragma unroll
                for (int32_t j = 0; j < KPT; ++j)
                    kv4[j] = smem_load4<E>(kb + (kg + 8 * j) * stride + d4 * 4 * kE);
#pragma unroll
                for (int32_t r = 0; r < RPT; ++r)
#pragma unroll
                    for (int32_t j = 0; j < KPT; ++j) {
                        float x = s[r][j];
                        x = fmaf(qv[r].x, kv4[j].x, x);
                        x = fmaf(qv[r].y, kv4[j].y, x);
                        x = fmaf(qv[r].z, kv4[j].z, x);
                        x = fmaf(qv[r].w, kv4[j].w, x);
                        s[r][j] = x;
                    }
            }

            // mask, online softmax per row (its eight threads), p to shared
            // memory for the eight threads' P V
            float al[RPT];
#pragma unroll
            for (int32_t r = 0; r < RPT; ++r) {
                uint32_t hidden = rvalid[r] ? 0u : ~0u;          // bit j: key kg + 8 j
                if (masked && rvalid[r]) {
#pragma unroll
                    for (int32_t j = 0; j < KPT; ++j) {
                        const int32_t k = t0 + kg + 8 * j - sg.C;    // node, < 0: a cached token
                        const bool sees = k < 0 || (k < sg.n && (bits[rtok[r] * kWords + (k >> 5)] >> (k & 31) & 1u));
                        hidden |= (sees ? 0u : 1u) << j;
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int32_t j = 0; j < KPT; ++j) {
                    s[r][j] = hidden >> j & 1u ? -INFINITY : s[r][j];
                    mx = fmaxf(mx, s[r][j]);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                const float mn = fmaxf(m[r], mx);
                const float mref = mn == -INFINITY ? 0.f : mn;    // no visible key yet
                al[r] = exp2f(m[r] - mref);                        // 0 while m = -inf
                float sum = 0.f;
#pragma unroll
                for (int32_t j = 0; j < KPT; ++j) {
                    const float p = exp2f(s[r][j] - mref);         // 0 for masked keys
                    sum += p;
                    ps[(rg * RPT + r) * pst + kg + 8 * j] = hidden >> j & 1u ? -1.f : p;
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                l[r] = l[r] * al[r] + sum;
                m[r] = mn;
#pragma unroll
                for (int32_t f = 0; f < NF; ++f) {
                    acc[r][f].x *= al[r];
                    acc[r][f].y *= al[r];
                    acc[r][f].z *= al[r];
                    acc[r][f].w *= al[r];
                }
            }
            __syncwarp();              // a row group's p, written by its own warp

            auto product = [&](auto skip) {
#pragma unroll 2
                for (int32_t k4 = 0; k4 < KC; k4 += 4) {
                    float4 pv[RPT];
#pragma unroll
                    for (int32_t r = 0; r < RPT; ++r)
                        pv[r] = *reinterpret_cast<const float4*>(ps + (rg * RPT + r) * pst + k4);
#pragma unroll
                    for (int32_t kk = 0; kk < 4; ++kk) {
                        const uint8_t* vrow = vb + (k4 + kk) * stride;
#pragma unroll
                        for (int32_t f = 0; f < NF; ++f) {
                            const int32_t col = 4 * (kg + 8 * f);
                            if (col < D) {
                                const float4 v = smem_load4<E>(vrow + col * kE);
#pragma unroll
                                for (int32_t r = 0; r < RPT; ++r) {
                                    const float p = kk == 0 ? pv[r].x : kk == 1 ? pv[r].y
                                                  : kk == 2 ? pv[r].z : pv[r].w;
                                    if (decltype(skip)::value && p < 0.f) continue;
                                    acc[r][f].x = fmaf(p, v.x, acc[r][f].x);
                                    acc[r][f].y = fmaf(p, v.y, acc[r][f].y);
                                    acc[r][f].z = fmaf(p, v.z, acc[r][f].z);
                                    acc[r][f].w = fmaf(p, v.w, acc[r][f].w);
                                }
                            }
                        }
                    }
                }
            };
            if (masked)
                product(std::true_type{});
            else
                product(std::false_type{});   // (idle rows' -1 weights are never stored)
            __syncthreads();           // buffer c & 1 and p are free
        }

        const bool whole = sg.kb0 == 0 && sg.kb1 == sg.nb;
        float* cell = whole ? nullptr : tree_cell(a, w, sg);
        E* out = static_cast<E*>(a.out);
#pragma unroll
        for (int32_t r = 0; r < RPT; ++r) {
            if (!rvalid[r]) continue;
            const int32_t rho = rg * RPT + r, tk = rho / HT, hh = rho - tk * HT;
            const int64_t row = (int64_t)(sg.q0 + sg.tok0 + tk) * a.num_q_heads + head_base + hh;
            const float inv = whole ? (l[r] != 0.f ? 1.f / l[r] : 0.f) : 1.f;
#pragma unroll
            for (int32_t f = 0; f < NF; ++f) {
                const int32_t col = 4 * (kg + 8 * f);
                if (col >= D) continue;
                const float4 o = make_float4(acc[r][f].x * inv, acc[r][f].y * inv,
                                             acc[r][f].z * inv, acc[r][f].w * inv);
                if (!whole) {
                    *reinterpret_cast<float4*>(cell + ((size_t)(kg + 8 * f) * R + rho) * 4) = o;
                } else if constexpr (kE == 2) {
                    *reinterpret_cast<uint2*>(out + row * D + col) =
                        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                } else {
                    *reinterpret_cast<float4*>(out + row * D + col) = o;
                }
            }
            if (!whole && kg == 0)
                *reinterpret_cast<float2*>(cell + (size_t)D * R + 2 * rho) = make_float2(m[r], l[r]);
        }
        __syncthreads();               // q, p and the node masks are free
    }
    if (w.cuts != nullptr && tid == 0) w.cuts[blockIdx.x] = cut;
    griddep_launch_dependents();
}

}  // namespace pa

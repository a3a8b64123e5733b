// tree_sched.cuh -- how the draft-tree attention kernels divide their work, and
// the merge of the parts.
//
// A unit is one (sequence, kv head, sub-group of query heads, tile of tree
// tokens) with all its keys; its cost is `overhead` for its prologue and
// epilogue, and for each key block one weight or the other by whether its
// sequence's units have one tile of rows or more.  A block belongs to the range
// that its cost begins in.  The units' costs laid end to end are cut into
// equal ranges, one per CTA of a grid that fills the GPU once, so the load is
// even whatever the lengths are: a CTA takes the tail of one unit, some whole
// units and the head of another.  A unit inside one range is written to the
// output at once.  Of a unit cut by a range's end every part leaves (acc, m,
// l) in its CTA's workspace cells -- at most two a CTA: cell 0 the part that
// continues an earlier CTA's, cell 1 the one that starts here -- and
// tree_merge_kernel joins them by log-sum-exp:
//   M = max_p m_p,  w_p = 2^(m_p - M),  out = sum w_p acc_p / sum w_p l_p.
// The cells' number depends on the grid alone, not on the batch.
#pragma once

#include "cp_async.cuh"
#include "tree_args.cuh"

namespace pa {

// Tiling of a kernel (host constants of a launch).
struct TreeShape {
    int32_t rows;           // rows of a tile: (token, query head) pairs, head fastest
    int32_t tiles;          // tiles of a unit
    int32_t heads;          // query heads of a tile: min(group, rows)
    int32_t tokens;         // tokens of a tile: rows / heads
    int32_t sub_groups;     // ceil(group / heads)
    int32_t keys;           // keys of a block
    int32_t block_one, block_more;   // cost of a key block, with one tile in use or more
    int32_t overhead;       // cost of a unit beside its key blocks
    int32_t min_range;      // least cost of a CTA's range
    int32_t fixed_cost;     // > 0: every unit counts as this much, and no range ends inside one
};

// A unit cut by the end of a CTA's range, for the merge: written by the CTA
// that starts it.  parts: the CTAs behind that hold the rest (0: none).
struct TreeCut {
    int32_t row0, ntok, g, sg;      // packed row of its first token, tokens, heads
    int32_t parts, pad[3];
};

struct TreeWork {
    TreeShape s;
    TreeCut* cuts;          // [CTAs] (nullptr: no unit can be cut, no merge follows)
    float* cells;           // [2 * CTAs]: acc [D / 4][rows * tiles][4], then (m, l) [rows * tiles][2]
};

__host__ __device__ inline size_t tree_cell_floats(const TreeShape& s, int32_t head_dim) {
    return (size_t)s.rows * s.tiles * (head_dim + 2);
}

__device__ __forceinline__ int32_t tree_units(const TreeArgs& a, const TreeShape& s, int32_t n) {
    const int32_t per = s.tokens * s.tiles;
    return n > 0 ? a.num_kv_heads * s.sub_groups * ((n + per - 1) / per) : 0;
}

__device__ __forceinline__ int32_t tree_weight(const TreeShape& s, int32_t n) {
    return n > s.tokens ? s.block_more : s.block_one;
}

__device__ __forceinline__ int32_t tree_cost(const TreeShape& s, int32_t n, int32_t T) {
    return s.fixed_cost > 0 ? s.fixed_cost
                            : (T + s.keys - 1) / s.keys * tree_weight(s, n) + s.overhead;
}

// One unit's part within a CTA's range.
struct TreeSeg {
    int32_t i, q0, n, T, C;         // sequence, its rows, lengths (C: cached tokens)
    int32_t g, sg;                  // kv head, sub-group
    int32_t tok0, ntok;             // tokens (nodes) tok0 .. tok0 + ntok - 1
    int32_t kb0, kb1, nb;           // key blocks of this part, of the unit
    int32_t parts;                  // of a unit that starts here: the CTAs behind with the rest
    int32_t pad[3];
};

// Position in the cost line.
struct TreeIter {
    int64_t pos, end, seq0;         // next cost, range end, cost before sequence i
    int64_t range;                  // cost of a CTA's range
    int32_t i;
};

// The next part of the range; false at its end.  Uniform over the threads
// that call it with equal state.
__device__ __forceinline__ bool tree_next(const TreeArgs& a, const TreeShape& sh, TreeIter& it,
                                          TreeSeg& o) {
    while (it.pos < it.end) {
        const TreeSeq s = tree_seq(a, it.i, false);
        // (a sequence's cost stays in 32 bits: the launch refuses others)
        const int32_t units = tree_units(a, sh, s.n);
        const int32_t cost = tree_cost(sh, s.n, s.T);
        const int64_t seq1 = it.seq0 + (int64_t)units * cost;
        if (it.pos >= seq1) {
            it.seq0 = seq1;
            if (++it.i >= a.num_seqs) return false;
            continue;
        }
        const int32_t at = (int32_t)(it.pos - it.seq0);
        const int32_t u = at / cost, from = at - u * cost;
        const int32_t to = (int32_t)min((int64_t)cost, from + (it.end - it.pos));
        it.pos += to - from;
        o.nb = (s.T + sh.keys - 1) / sh.keys;
        const int32_t wt = tree_weight(sh, s.n);
        // blocks whose cost begins in [from, to)
        o.kb0 = max(0, from - sh.overhead + wt - 1) / wt;
        o.kb1 = to == cost ? o.nb : min(o.nb, max(0, to - sh.overhead + wt - 1) / wt);
        if (o.kb0 >= o.kb1) continue;
        // the ranges behind that hold the unit's other blocks
        const int32_t left = sh.overhead + (o.nb - 1) * wt - to;
        o.parts = o.kb1 < o.nb ? (int32_t)(left / it.range) + 1 : 0;
        const int32_t per = sh.tokens * sh.tiles, tiles = (s.n + per - 1) / per;
        const int32_t hs = tiles == 1 ? u : u / tiles, tile = u - hs * tiles;
        o.i = it.i;
        o.q0 = s.q0;
        o.n = s.n;
        o.T = s.T;
        o.C = s.T - s.n;
        o.g = sh.sub_groups == 1 ? hs : hs / sh.sub_groups;
        o.sg = hs - o.g * sh.sub_groups;
        o.tok0 = tile * per;
        o.ntok = min(per, s.n - o.tok0);
        return true;
    }
    return false;
}

// This CTA's range of a line of `total` cost.
__device__ __forceinline__ void tree_range(const TreeShape& s, int64_t total, TreeIter& it) {
    const uint32_t ctas = gridDim.x;
    it.range = total <= 0x7fffffff ? (int64_t)(((uint32_t)total + ctas - 1) / ctas)
                                   : (total + ctas - 1) / ctas;
    it.range = s.fixed_cost > 0 ? (it.range + s.fixed_cost - 1) / s.fixed_cost * s.fixed_cost
                                : max(it.range, (int64_t)s.min_range);
    it.pos = min(total, it.range * blockIdx.x);
    it.end = min(total, it.pos + it.range);
}

// This CTA's range: all threads of the block, `scratch` holding 2 + threads /
// 32 values.  Every CTA sums the batch's costs; CTA 0 reports refused
// sequences.
__device__ __forceinline__ TreeIter tree_begin(const TreeArgs& a, const TreeWork& w,
                                               int64_t* scratch) {
    const int32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t threads = blockDim.x, warps = threads / 32;
    const int32_t chunk = (a.num_seqs + threads - 1) / threads;
    const int32_t i0 = min(a.num_seqs, tid * chunk), i1 = min(a.num_seqs, i0 + chunk);
    int64_t sum = 0;
    for (int32_t i = i0; i < i1; ++i) {
        const TreeSeq s = tree_seq(a, i, blockIdx.x == 0);
        sum += (int64_t)tree_units(a, w.s, s.n) * tree_cost(w.s, s.n, s.T);
    }
    int64_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    if (lane == 31) scratch[2 + warp] = incl;
    if (tid == 0) {
        scratch[0] = 0;                         // read for an empty range only
        scratch[1] = 0;
    }
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int32_t x = 0; x < warps; ++x) {
        const int64_t v = scratch[2 + x];
        if (x < warp) before += v;
        total += v;
    }
    int64_t at = before + incl - sum;           // cost before sequence i0
    TreeIter it;
    tree_range(w.s, total, it);
    // the thread whose sequences hold the range's start names the sequence
    if (at <= it.pos && it.pos < at + sum) {
        int32_t i = i0;
        if (chunk > 1) {
            for (;; ++i) {
                const TreeSeq s = tree_seq(a, i, false);
                const int64_t c = (int64_t)tree_units(a, w.s, s.n) * tree_cost(w.s, s.n, s.T);
                if (it.pos < at + c) break;
                at += c;
            }
        }
        scratch[0] = i;
        scratch[1] = at;
    }
    __syncthreads();
    it.i = (int32_t)scratch[0];
    it.seq0 = scratch[1];
    return it;
}

// The same by one warp, for up to 128 sequences (four a lane): no barrier, so
// the block's other warps set up meanwhile.
constexpr int32_t kTreeWarpSeqs = 128;
__device__ __forceinline__ TreeIter tree_begin_warp(const TreeArgs& a, const TreeWork& w) {
    const int32_t lane = threadIdx.x & 31;
    int64_t c[4];
#pragma unroll
    for (int32_t u = 0; u < 4; ++u) {
        const int32_t i = 4 * lane + u;
        c[u] = 0;
        if (i < a.num_seqs) {
            const TreeSeq s = tree_seq(a, i, blockIdx.x == 0);
            c[u] = (int64_t)tree_units(a, w.s, s.n) * tree_cost(w.s, s.n, s.T);
        }
    }
    int64_t incl = c[0] + c[1] + c[2] + c[3];
    const int64_t sum = incl;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    TreeIter it;
    tree_range(w.s, __shfl_sync(0xffffffffu, incl, 31), it);
    int64_t at = incl - sum;
    int32_t i = 4 * lane;
    const bool mine = at <= it.pos && it.pos < incl;
#pragma unroll
    for (int32_t u = 0; u < 3; ++u) {
        if (it.pos >= at + c[u] && i == 4 * lane + u) {
            at += c[u];
            ++i;
        }
    }
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    const int32_t src = who ? __ffs(who) - 1 : 0;         // (none: an empty range)
    it.i = who ? __shfl_sync(0xffffffffu, i, src) : 0;
    it.seq0 = who ? __shfl_sync(0xffffffffu, at, src) : 0;
    return it;
}

// Copies of a chunk of keys by the WARPS warps of a block.  A lane finds the
// cache row of one key: one table entry and one division a lane, not one a
// piece.  The entry is read a chunk ahead of use (tree_entry) and looked at when
// the copies are issued (tree_row), so its latency passes beside the chunk's
// work.  The warps then take the rows in turn, 16 bytes a lane.
struct TreeEntry {
    int32_t id, off;        // table entry; the key's place in its block, < 0: no key
};
__device__ __forceinline__ TreeEntry tree_entry(const TreeArgs& a, const TreeSeg& s, int32_t key) {
    TreeEntry e{0, -1};
    if (key < s.T) {
        const int32_t b = key / a.block_size;
        e.id = a.block_tables[(int64_t)s.i * a.max_blocks + b];
        e.off = key - b * a.block_size;
    }
    return e;
}
__device__ __forceinline__ int64_t tree_row(const TreeArgs& a, const TreeSeg& s, TreeEntry e,
                                            bool report) {
    if (e.off < 0) return -1;
    if (e.id < 0 || e.id >= a.num_blocks) {
        if (report) raise_error(PA_DEVERR_TABLE_ENTRY);
        return -1;
    }
    return ((int64_t)e.id * a.num_kv_heads + s.g) * a.block_size + e.off;
}

// row: this lane's (lane < KC) cache row of its key, -1: zeros.  pieces: 16-byte
// pieces of a row; kst, vst: row strides in shared memory, bytes.
template <int KC, int WARPS>
__device__ __forceinline__ void tree_copy(const TreeArgs& a, int64_t row, int32_t pieces, uint32_t kb,
                                          int32_t kst, uint32_t vb, int32_t vst) {
    static_assert(KC <= 32 && KC % WARPS == 0, "a key a lane");
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
    const uint8_t* vc = static_cast<const uint8_t*>(a.v_cache);
    const int64_t off = row < 0 ? -1 : row * pieces * 16;
    if (pieces > 16) {
        // a row a warp at a time
#pragma unroll
        for (int32_t u = 0; u < KC / WARPS; ++u) {
            const int32_t k = warp + u * WARPS;
            const int64_t r = __shfl_sync(0xffffffffu, off, k);
            const uint32_t bytes = r < 0 ? 0u : 16u;
            const int64_t src = r < 0 ? 0 : r + lane * 16;
            if (lane < pieces) {
                cp_async16(kb + k * kst + lane * 16, kc + src, bytes);
                cp_async16(vb + k * vst + lane * 16, vc + src, bytes);
            }
            for (int32_t p = lane + 32; p < pieces; p += 32) {
                const int64_t more = r < 0 ? 0 : r + p * 16;
                cp_async16(kb + k * kst + p * 16, kc + more, bytes);
                cp_async16(vb + k * vst + p * 16, vc + more, bytes);
            }
        }
        return;
    }
    // short rows: several at a time, lanes per row a power of two
    int32_t shift = 4;
    while (shift > 0 && (1 << (shift - 1)) >= pieces) --shift;
    const int32_t p = lane & ((1 << shift) - 1), sub = lane >> shift, rows = 32 >> shift;
#pragma unroll 4
    for (int32_t k0 = warp * rows; k0 < KC; k0 += WARPS * rows) {
        const int32_t k = k0 + sub;
        const int64_t r = __shfl_sync(0xffffffffu, off, k & 31);
        if (k >= KC || p >= pieces) continue;
        const int64_t src = r < 0 ? 0 : r + p * 16;
        const uint32_t bytes = r < 0 ? 0u : 16u;
        cp_async16(kb + k * kst + p * 16, kc + src, bytes);
        cp_async16(vb + k * vst + p * 16, vc + src, bytes);
    }
}

// The cell of this CTA's part.
__device__ __forceinline__ float* tree_cell(const TreeArgs& a, const TreeWork& w, const TreeSeg& s) {
    return w.cells + (2 * (size_t)blockIdx.x + (s.kb0 == 0 ? 1 : 0)) * tree_cell_floats(w.s, a.head_dim);
}

// Joins the parts of the unit that CTA blockIdx.x of the attention kernel
// starts and does not end.  A thread takes one row and eight columns at a
// time, lanes along the rows.  Measured alone with cold caches: 13.5 us for the 19 MB
// of parts that 128 sequences of up to 64 nodes leave (1.4 TB/s, 42% of the warps
// active, so neither bytes nor instructions bound it), 7.4 us for 1.8 MB, with up to
// 8 CTAs a cut.  16 give a thread one item of the largest tile: a whole call on 24
// sequences of up to 48 nodes, group 5, D = 96 took 53.5 us with 8, 52.8 with 16,
// larger batches the same either way.
constexpr int kTreeMergeThreads = 256;
constexpr int kTreeMergeSplit = 16;     // CTAs per cut

template <typename E>
__global__ void __launch_bounds__(kTreeMergeThreads)
tree_merge_kernel(const TreeArgs a, const TreeWork w) {
    griddep_wait();
    griddep_launch_dependents();
    const TreeShape& sh = w.s;
    const TreeCut cut = w.cuts[blockIdx.x];
    if (cut.parts == 0) return;
    const int32_t heads = min(sh.heads, a.group - cut.sg * sh.heads);
    const int32_t D = a.head_dim, urows = sh.rows * sh.tiles;
    const int32_t live = cut.ntok <= sh.tokens ? cut.ntok * sh.heads : urows;
    const int32_t groups = (D + 7) / 8;
    const size_t cell = tree_cell_floats(sh, D);
    const float* first = w.cells + (2 * (size_t)blockIdx.x + 1) * cell;
    const float* next = w.cells + 2 * ((size_t)blockIdx.x + 1) * cell;  // cell 0 of the CTAs behind
    E* out = static_cast<E*>(a.out);
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & (4 * sizeof(E) - 1)) == 0;
    for (int32_t at = blockIdx.y * kTreeMergeThreads + threadIdx.x; at < live * groups;
         at += gridDim.y * kTreeMergeThreads) {
        const int32_t row = at % live, col = (at / live) * 8;
        const int32_t t = row / sh.rows, r = row - t * sh.rows;
        const int32_t tk = r / sh.heads, h = r - tk * sh.heads, tok = t * sh.tokens + tk;
        if (tk >= sh.tokens || tok >= cut.ntok || h >= heads) continue;
        const size_t ml = (size_t)D * urows + 2 * (size_t)row;
        float M = first[ml];
#pragma unroll 4
        for (int32_t p = 0; p < cut.parts; ++p) M = fmaxf(M, next[p * 2 * cell + ml]);
        const float ref = M == -INFINITY ? 0.f : M;
        float l = 0.f, o[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = 0.f;
        const bool wide = col + 4 < D;
#pragma unroll 4
        for (int32_t p = -1; p < cut.parts; ++p) {
            const float* c = p < 0 ? first : next + p * 2 * cell;
            const float2 v = *reinterpret_cast<const float2*>(c + ml);
            const float4 x0 = *reinterpret_cast<const float4*>(c + ((size_t)(col / 4) * urows + row) * 4);
            float4 x1 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (wide) x1 = *reinterpret_cast<const float4*>(c + ((size_t)(col / 4 + 1) * urows + row) * 4);
            const float wp = exp2f(v.x - ref);                 // 0 for a part without visible keys
            l += wp * v.y;
            const float xs[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            // (an infinite sum stays one under a weight that underflows)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += fabsf(xs[e]) <= 3.4028235e38f ? wp * xs[e] : xs[e];
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        E* dst = out + ((int64_t)(cut.row0 + tok) * a.num_q_heads + (int64_t)cut.g * a.group +
                        cut.sg * sh.heads + h) * D + col;
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] *= inv;
        // (head dims with parts are multiples of 4; an output may be aligned to
        // its elements only)
        if (!vec) {
            for (int c = 0; c < 8 && col + c < D; ++c) dst[c] = Elem<E>::from_float(o[c]);
        } else if constexpr (sizeof(E) == 2) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            if (wide)
                *reinterpret_cast<uint2*>(dst + 4) =
                    make_uint2(pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
        } else {
            *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
            if (wide) *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace pa

// rope_write.cuh -- a layer's projected rows on their way to its attention: the
// queries and keys of each head are normed and rotated by their positions, the
// queries go to their own array, the keys and values to their cache slots.
//
// With a head's row x of D values, weight w and position axes p_0 .. p_{A-1}:
//   y = x / sqrt(mean(x^2) + eps) * w                 (without w: y = x)
//   angle_j = p_{a(j)} * inv_freq[j]                  for pair j of rot_dim / 2
//   (y1, y2) -> scale * (y1 cos - y2 sin, y1 sin + y2 cos)
// Pair j is (j, j + rot_dim / 2) or the neighbours (2 j, 2 j + 1); dimensions from
// rot_dim on keep y.  All in 32 bits, rounded once.
//
// Angles: a position of up to 2^31 times a frequency has more whole turns than 32
// bits can hold beside the fraction that matters.  A frequency is therefore taken
// as a 64-bit fraction of a turn, F = inv_freq / 2 pi * 2^64 (whole numbers only:
// the 24 bits of inv_freq times 1 / 2 pi to 96 bits), and p * F modulo 2^64 drops the
// whole turns without a rounding; what is left is off by p * 2^-64 turns.
//
// Bound: each row read and written once.  Measured (GPU time): 16384 tokens of 64 + 8
// heads of 128 on bf16, 671 MB, 101 us (98% of the copy rate); 2303 tokens of 32 + 8 with
// norms, 57 MB, 13.2 us from L2, 16.8 from memory (the rate allows 8.3, and a launch takes
// 2.5): few warps a SM then, and a row after the other in each; more rows under way
// changed nothing.  5001 tokens of 15 + 5 heads of 80 on fp32 with norms, 80 MB, 15.4 us
// (11.8), where instructions bound it; one token 3.6 us.
#pragma once

#include "common.cuh"
#include "cp_async.cuh"
#include "ptx.cuh"
#include "write_kv.cuh"

namespace pa {

struct RopeArgs {
    const uint8_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* q_weight;        // may be nullptr
    const uint8_t* k_weight;        // may be nullptr
    const int32_t* positions;       // [axes][num_tokens]
    const float* inv_freq;          // [rot_dim / 2]
    const int64_t* slot_mapping;    // [num_tokens]
    uint8_t* out;                   // [num_tokens][Hq][D]
    uint8_t* k_cache;
    uint8_t* v_cache;
    int64_t q_stride, k_stride, v_stride;   // elements from token to token
    int64_t num_slots;
    int32_t num_tokens, num_q_heads, num_kv_heads, head_dim, block_size;
    int32_t rot_dim, axes, cyclic, neighbours;
    int32_t section[3];
    float eps, scale;
};

// Axis of pair j.
__device__ __forceinline__ int32_t rope_axis(const RopeArgs& a, int32_t j) {
    if (a.axes == 1) return 0;
    if (a.cyclic) {
        const int32_t x = j % a.axes;
        const int32_t pairs = x == 0 ? a.section[0] : x == 1 ? a.section[1] : a.section[2];
        return j / a.axes < pairs ? x : 0;
    }
    return j < a.section[0] ? 0 : j < a.section[0] + a.section[1] ? 1 : 2;
}

// A frequency in radians as a 64-bit fraction of a turn, whole turns dropped.
// |f| below 2^32 (ok is false for others).
__device__ __forceinline__ uint64_t turn_fraction(float f, bool& ok) {
    // floor(2^96 / (2 pi))
    constexpr unsigned __int128 kInvTurn =
        ((unsigned __int128)0x28be60db9391054aull << 32) | 0x7f09d5f4u;
    const uint32_t bits = __float_as_uint(f);
    const int32_t e = (int32_t)((bits >> 23) & 255);
    const uint32_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);   // |f| = m 2^(max(e, 1) - 150)
    ok = e < 127 + 32;
    const int32_t shift = 32 + 150 - max(e, 1);                     // >= 24 where ok
    if (!ok || shift >= 128) return 0;
    const uint64_t x = (uint64_t)((m * kInvTurn) >> shift);
    return (bits >> 31) ? 0 - x : x;
}

// cos and sin of a 64-bit fraction of a turn: the nearest quarter turn taken off,
// the rest (at most an eighth, 32 bits) in radians of pi.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t t) {
    const uint64_t near = t + (1ull << 61);
    const uint32_t quarter = (uint32_t)(near >> 62);
    const int64_t rest = (int64_t)((near & ((1ull << 62) - 1))) - (1ll << 61);
    float s, c;
    sincospif((float)(int32_t)(rest >> 30) * (1.0f / 8589934592.0f), &s, &c);   // * 2^-33
    const float x = (quarter & 1) ? s : c, y = (quarter & 1) ? c : s;
    return make_float2((quarter == 1 || quarter == 2) ? -x : x, (quarter & 2) ? -y : y);
}

template <typename E, int VEC>
struct RopeVec {
    static constexpr int kBytes = VEC * (int)sizeof(E);
    using Raw = typename VecType<kBytes>::T;
    Raw raw;
    __device__ __forceinline__ void clear() { raw = Raw{}; }
    // Unpacked again from here on: keeping what was unpacked would cost more registers
    // than it saves time.
    __device__ __forceinline__ void repack() {
        if constexpr (kBytes == 16)
            asm volatile("" : "+r"(raw.x), "+r"(raw.y), "+r"(raw.z), "+r"(raw.w));
    }
    __device__ __forceinline__ void load(const E* p) { raw = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    __device__ __forceinline__ float get(int i) const {
        return Elem<E>::to_float(reinterpret_cast<const E*>(&raw)[i]);
    }
    __device__ __forceinline__ void set(int i, float x) {
        reinterpret_cast<E*>(&raw)[i] = Elem<E>::from_float(x);
    }
};

// A warp works on one token (`splits` warps share one where there are few), so that
// each lane computes and keeps the cos and sin of its own pairs for all heads.  A row
// is D / (2 VEC) pairs of VEC-element pieces, whose rotated pairs lie inside a piece
// (neighbours) or between its two pieces (halves); `lanes` lanes share a row (as many as
// it has piece pairs, so that other dims than powers of two leave few lanes idle: 5001 tokens of
// 15 + 5 heads of 80 on fp32 take 15.4 us in 10 lanes a row, 20.3 in 16) and a lane has up to C of its piece pairs.
constexpr int kRopeWarps = 4;
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeMaxDim = 256;

template <typename E, int VEC, int C, bool NEIGHBOURS>
struct RopeRows {
    using Vec = RopeVec<E, VEC>;
    int32_t dim, lanes, lane, pieces, across;   // `lanes` lanes share a row, this one is `lane`
    int32_t at0[C], at1[C];         // a piece pair's two places (dim: none)
    float cs[C][VEC], sn[C][VEC];   // of its pairs
    uint32_t turned;                // bit c * VEC + i: that pair is rotated

    __device__ __forceinline__ int32_t piece(int c) const {
        return lane + c * lanes;
    }
    __device__ __forceinline__ void place(const RopeArgs& a, int32_t of, int32_t mine) {
        dim = a.head_dim;
        lanes = of;
        lane = mine;
        pieces = VEC == 1 ? (dim + 1) / 2 : dim / (2 * VEC);
        across = a.rot_dim / (2 * VEC);              // rotated piece pairs, halves
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t p = piece(c);
            if (NEIGHBOURS) {
                at0[c] = VEC == 1 ? 2 * p : p * VEC;
                at1[c] = VEC == 1 ? 2 * p + 1 : (p + pieces) * VEC;
            } else {
                at0[c] = (p < across ? p : across + p) * VEC;
                at1[c] = (p < across ? p + across : pieces + p) * VEC;
            }
            if (p >= pieces) at0[c] = at1[c] = dim;
            if (at1[c] >= dim) at1[c] = dim;
        }
    }
    // The pairs' cos and sin.
    __device__ __forceinline__ void turn(int32_t half, const float2* of) {
        turned = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                // pair i of the pieces (halves), of one piece, then the other (neighbours)
                const int32_t p = piece(c);
                int32_t j;
                if (VEC > 1 && NEIGHBOURS)
                    j = (i < VEC / 2 ? at0[c] : at1[c]) / 2 + i % (VEC > 1 ? VEC / 2 : 1);
                else
                    j = NEIGHBOURS ? p : p < across ? p * VEC + i : half;
                const bool in = p < pieces && j < half;
                const float2 x = in ? of[j] : make_float2(1.f, 0.f);
                cs[c][i] = x.x;
                sn[c][i] = x.y;
                turned |= in ? 1u << (c * VEC + i) : 0u;
            }
    }
    __device__ __forceinline__ void turn_piece(int c, float (&y0)[VEC], float (&y1)[VEC]) const {
        constexpr uint32_t kAll = (1u << VEC) - 1;
        const uint32_t bits = turned >> (c * VEC) & kAll;
        if (bits == 0) return;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const bool one = VEC > 1 && NEIGHBOURS;
            float& a = !one ? y0[i] : i < VEC / 2 ? y0[2 * i % VEC] : y1[2 * i % VEC];
            float& b = !one ? y1[i] : i < VEC / 2 ? y0[(2 * i + 1) % VEC] : y1[(2 * i + 1) % VEC];
            const float x = a, y = b;
            const float u = x * cs[c][i] - y * sn[c][i], w = x * sn[c][i] + y * cs[c][i];
            const bool in = bits == kAll || (bits >> i & 1);
            a = in ? u : x;
            b = in ? w : y;
        }
    }
    struct Weights {
        Vec lo[C], hi[C];
    };
    __device__ __forceinline__ void load(Weights& w, const E* weight) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            w.lo[c].clear();
            w.hi[c].clear();
            if (weight != nullptr && at0[c] < dim) w.lo[c].load(weight + at0[c]);
            if (weight != nullptr && at1[c] < dim) w.hi[c].load(weight + at1[c]);
        }
    }
    // One row of each group of lanes, normed (NORM) and rotated.
    template <bool NORM>
    __device__ __forceinline__ void row(Vec (&lo)[C], Vec (&hi)[C], const Weights& w, float inv_dim,
                                        float eps) const {
        float norm = 1.f;
        if constexpr (NORM) {
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    sum = fmaf(lo[c].get(i), lo[c].get(i), sum);
                    sum = fmaf(hi[c].get(i), hi[c].get(i), sum);
                }
            if ((lanes & (lanes - 1)) == 0) {
                for (int32_t off = lanes >> 1; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            } else {
                for (int32_t off = 16; off > 0; off >>= 1) {
                    if (off >= lanes) continue;
                    const float x = __shfl_down_sync(0xffffffffu, sum, off);
                    if (lane < off && lane + off < lanes) sum += x;
                }
                sum = __shfl_sync(0xffffffffu, sum, (threadIdx.x & 31) - lane);
            }
            norm = rsqrtf(fmaf(sum, inv_dim, eps));
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (NORM && sizeof(E) == 2) {
                lo[c].repack();
                hi[c].repack();
            }
            float y0[VEC], y1[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                y0[i] = lo[c].get(i);
                y1[i] = hi[c].get(i);
                if constexpr (NORM) {
                    y0[i] = y0[i] * norm * w.lo[c].get(i);
                    y1[i] = y1[i] * norm * w.hi[c].get(i);
                }
            }
            turn_piece(c, y0, y1);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                lo[c].set(i, y0[i]);
                hi[c].set(i, y1[i]);
            }
        }
    }
    __device__ __forceinline__ void store(const Vec (&lo)[C], const Vec (&hi)[C], E* dst) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (at0[c] < dim) lo[c].store(dst + at0[c]);
            if (at1[c] < dim) hi[c].store(dst + at1[c]);
        }
    }
};

// Rows come by asynchronous copies into shared memory, each lane's own pieces, so that
// kRopeDepth rows a lane are under way without registers to hold them (16-byte
// pieces; smaller ones are loaded as they are needed).
constexpr int kRopeDepth = 3;

template <typename E, int VEC, int C, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads, (sizeof(E) == 2 && VEC == 8 ? 24 : 32) / kRopeWarps) rope_write_kernel(const RopeArgs a, int32_t splits,
                                                                    int32_t lanes) {
    constexpr bool kRing = VEC * sizeof(E) == 16;
    using Rows = RopeRows<E, VEC, C, NEIGHBOURS>;
    extern __shared__ uint4 s_ring[];               // [kRopeDepth][2][kRopeThreads], then cos, sin
    float2* s_turn = reinterpret_cast<float2*>(s_ring + (kRing ? kRopeDepth * 2 * kRopeThreads : 0));
    griddep_wait();
    griddep_launch_dependents();
    const int32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t D = a.head_dim, half = a.rot_dim / 2, B = a.block_size;
    const int64_t id = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = id / splits;
    const int32_t part = (int32_t)(id - tok * splits);
    if (tok >= a.num_tokens) return;
    Rows rows;
    // This warp's groups of lanes take heads base + group, then those a step further,
    // ...: of the queries, the keys, the values.  (Lanes left over are of no group.)
    const int32_t groups = 32 / lanes, base = part * groups, step = splits * groups;
    const int32_t group = lane / lanes < groups ? lane / lanes : INT32_MAX / 2;
    rows.place(a, lanes, lane % lanes);
    const E* const q = reinterpret_cast<const E*>(a.q) + tok * a.q_stride;
    const E* const k = reinterpret_cast<const E*>(a.k) + tok * a.k_stride;
    const E* const v = reinterpret_cast<const E*>(a.v) + tok * a.v_stride;
    // the next row to fetch: its kind (3: none left), first head of the warp, slots
    int32_t kind = base < a.num_q_heads ? 0 : base < a.num_kv_heads ? 1 : 3, head = base, fetched = 0;
    uint4* const mine = s_ring + threadIdx.x;
    auto fetch = [&]() {
        if constexpr (kRing) {
            if (kind < 3) {
                const int32_t h = head + group, heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
                const E* src = (kind == 0 ? q : kind == 1 ? k : v) + (int64_t)h * D;
                uint4* slots = mine + fetched * 2 * kRopeThreads;
                if (h < heads && rows.at0[0] < D) cp_async16(smem_u32(slots), src + rows.at0[0], 16);
                if (h < heads && rows.at1[0] < D) cp_async16(smem_u32(slots + kRopeThreads), src + rows.at1[0], 16);
                head += step;
                if (head >= heads) {
                    head = base;
                    kind = base < a.num_kv_heads ? kind + 1 : 3;
                }
            }
            fetched = fetched + 1 == kRopeDepth ? 0 : fetched + 1;
            cp_async_commit();
        }
    };
#pragma unroll
    for (int x = 0; x < kRopeDepth; ++x) fetch();
    // (the rows are on their way before anything is known of the token: nothing below
    // waits for more than one load)
    int64_t slot = a.slot_mapping[tok];
    const int32_t pos = a.positions[tok];
    float2* turn = s_turn + warp * half;
    for (int32_t j = lane; j < half; j += 32) {
        const int32_t axis = rope_axis(a, j);
        const int32_t p = axis == 0 ? pos : a.positions[(int64_t)axis * a.num_tokens + tok];
        bool ok;
        const uint64_t f = turn_fraction(a.inv_freq[j], ok);
        float2 cs = turn_cos_sin((uint64_t)((int64_t)p) * f);
        if (!ok) cs = make_float2(NAN, NAN);
        turn[j] = make_float2(a.scale * cs.x, a.scale * cs.y);
    }
    __syncwarp();
    rows.turn(half, turn);
    if (slot >= a.num_slots) {
        if (pos >= 0 && lane == 0 && part == 0) raise_error(PA_DEVERR_SLOT);
        slot = -1;
    }
    const int64_t block = slot / B;
    const int64_t at = (block * a.num_kv_heads * B + (slot - block * B)) * (int64_t)D;
    const float inv_dim = 1.f / (float)D;
    typename Rows::Weights w;
    int32_t taken = 0;
    // the rows of one kind, f(lo, hi) between the fetch and the store
    auto each = [&](const E* src, E* dst, int64_t apart, int32_t heads, auto f) {
        for (int32_t h0 = base; h0 < heads; h0 += step) {
            const int32_t h = h0 + group;
            RopeVec<E, VEC> lo[C], hi[C];
            if constexpr (kRing) cp_async_wait<kRopeDepth - 1>();
#pragma unroll
            for (int c = 0; c < C; ++c) {
                lo[c].clear();
                hi[c].clear();
                if constexpr (kRing) {
                    const uint4* slots = mine + taken * 2 * kRopeThreads;
                    if (h < heads && rows.at0[c] < D) lo[c].raw = slots[0];
                    if (h < heads && rows.at1[c] < D) hi[c].raw = slots[kRopeThreads];
                } else {
                    if (h < heads && rows.at0[c] < D) lo[c].load(src + (int64_t)h * D + rows.at0[c]);
                    if (h < heads && rows.at1[c] < D) hi[c].load(src + (int64_t)h * D + rows.at1[c]);
                }
            }
            taken = taken + 1 == kRopeDepth ? 0 : taken + 1;
            f(lo, hi);
            if (h < heads) rows.store(lo, hi, dst + h * apart);
            fetch();                    // (the slots have been read: their values are used)
        }
    };
    auto turned = [&](const E* src, E* dst, int64_t apart, int32_t heads, const E* weight) {
        // (fp32 rows leave registers for the weights; else they come from L1 each time)
        constexpr bool kKeep = sizeof(E) == 4;
        if (kKeep) rows.load(w, weight);
        if (weight != nullptr)
            each(src, dst, apart, heads, [&](auto& lo, auto& hi) {
                if (!kKeep) rows.load(w, weight);
                rows.template row<true>(lo, hi, w, inv_dim, a.eps);
            });
        else
            each(src, dst, apart, heads, [&](auto& lo, auto& hi) { rows.template row<false>(lo, hi, w, inv_dim, a.eps); });
    };
    if (pos >= 0) {
        turned(q, reinterpret_cast<E*>(a.out) + tok * a.num_q_heads * D, D, a.num_q_heads,
               reinterpret_cast<const E*>(a.q_weight));
        if (slot >= 0) {
            turned(k, reinterpret_cast<E*>(a.k_cache) + at, (int64_t)B * D, a.num_kv_heads,
                   reinterpret_cast<const E*>(a.k_weight));
            each(v, reinterpret_cast<E*>(a.v_cache) + at, (int64_t)B * D, a.num_kv_heads, [](auto&, auto&) {});
        }
    }
    if constexpr (kRing) cp_async_wait<0>();
}

}  // namespace pa

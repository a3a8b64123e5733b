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
#pragma once

#include "common.cuh"
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

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;

template <typename E, int VEC>
struct RopeVec {
    static constexpr int kBytes = VEC * (int)sizeof(E);
    using Raw = typename VecType<kBytes>::T;
    Raw raw;
    __device__ __forceinline__ void load(const E* p) { raw = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    __device__ __forceinline__ float get(int i) const {
        return Elem<E>::to_float(reinterpret_cast<const E*>(&raw)[i]);
    }
    __device__ __forceinline__ void set(int i, float x) {
        reinterpret_cast<E*>(&raw)[i] = Elem<E>::from_float(x);
    }
};

// A row is D / (2 VEC) pairs of VEC-element pieces, whose rotated pairs lie inside it
// (neighbours) or between its two pieces (halves).  2^LOG lanes share a row, a lane
// has up to C of its piece pairs.  One CTA: `tile` tokens.
template <typename E, int VEC, int C>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs a, int32_t tile,
                                                                  int32_t log_lanes) {
    extern __shared__ float2 s_turn[];              // [tile][rot_dim / 2] cos, sin
    using Vec = RopeVec<E, VEC>;
    griddep_wait();
    griddep_launch_dependents();
    const int32_t D = a.head_dim, half = a.rot_dim / 2, B = a.block_size;
    const int32_t t0 = blockIdx.x * tile;
    const int32_t tokens = min(tile, a.num_tokens - t0);
    for (int32_t x = threadIdx.x; x < half * tokens; x += kRopeThreads) {
        const int32_t t = x / half, j = x - t * half;
        const int32_t p = a.positions[(int64_t)rope_axis(a, j) * a.num_tokens + t0 + t];
        bool ok;
        const uint64_t f = turn_fraction(a.inv_freq[j], ok);
        float2 cs = turn_cos_sin((uint64_t)((int64_t)p) * f);
        if (!ok) cs = make_float2(NAN, NAN);
        s_turn[x] = make_float2(a.scale * cs.x, a.scale * cs.y);
    }
    __syncthreads();
    const int32_t lanes = 1 << log_lanes;
    const int32_t lane = threadIdx.x & (lanes - 1);
    const int32_t pieces = VEC == 1 ? (D + 1) / 2 : D / (2 * VEC);
    const int32_t turned = a.neighbours ? 0 : a.rot_dim / (2 * VEC);   // piece pairs, halves
    const int32_t rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int32_t groups = kRopeThreads >> log_lanes;
    const float inv_dim = 1.0f / (float)D;
    // (whole warps go round together: the sums are taken by shuffles)
    for (int32_t x0 = 0; x0 < tokens * rows; x0 += groups) {
        const int32_t x = x0 + (threadIdx.x >> log_lanes);
        const int32_t t = min(x / rows, tokens - 1), r = x - t * rows;
        const int64_t tok = t0 + t;
        bool live = x < tokens * rows && a.positions[tok] >= 0;
        const int32_t kind = r < a.num_q_heads ? 0 : r < a.num_q_heads + a.num_kv_heads ? 1 : 2;
        const int32_t h = kind == 0 ? r : r - a.num_q_heads - (kind - 1) * a.num_kv_heads;
        const E* src;
        E* dst;
        if (kind == 0) {
            src = reinterpret_cast<const E*>(a.q) + tok * a.q_stride + (int64_t)h * D;
            dst = reinterpret_cast<E*>(a.out) + (tok * a.num_q_heads + h) * D;
        } else {
            src = reinterpret_cast<const E*>(kind == 1 ? a.k : a.v) +
                  tok * (kind == 1 ? a.k_stride : a.v_stride) + (int64_t)h * D;
            const int64_t slot = a.slot_mapping[tok];
            if (live && slot >= a.num_slots && lane == 0) raise_error(PA_DEVERR_SLOT);
            live = live && slot >= 0 && slot < a.num_slots;
            const int64_t block = slot / B;
            dst = reinterpret_cast<E*>(kind == 1 ? a.k_cache : a.v_cache) +
                  ((block * a.num_kv_heads + h) * B + (slot - block * B)) * (int64_t)D;
        }
        Vec lo[C], hi[C];
        int32_t at0[C], at1[C];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t p = lane + (c << log_lanes);
            // the piece pair's two places
            if (a.neighbours) {
                at0[c] = VEC == 1 ? 2 * p : p * VEC;
                at1[c] = VEC == 1 ? 2 * p + 1 : (p + pieces) * VEC;
            } else {
                at0[c] = (p < turned ? p : turned + p) * VEC;
                at1[c] = (p < turned ? p + turned : pieces + p) * VEC;
            }
            if (p >= pieces) at0[c] = at1[c] = D;
            if (live && at0[c] < D) lo[c].load(src + at0[c]);
            if (live && at1[c] < D) hi[c].load(src + at1[c]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (at0[c] < D) sum += lo[c].get(i) * lo[c].get(i);
                if (at1[c] < D) sum += hi[c].get(i) * hi[c].get(i);
            }
        }
        for (int32_t off = lanes >> 1; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (!live) continue;
        const E* weight = reinterpret_cast<const E*>(kind == 0 ? a.q_weight : a.k_weight);
        const float norm = rsqrtf(sum * inv_dim + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (at0[c] >= D) continue;
            const int32_t p = lane + (c << log_lanes);
            const bool two = at1[c] < D;
            if (kind < 2) {
                float y0[VEC], y1[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    y0[i] = lo[c].get(i);
                    y1[i] = two ? hi[c].get(i) : 0.f;
                }
                if (weight != nullptr) {
                    Vec w0, w1;
                    w0.load(weight + at0[c]);
                    if (two) w1.load(weight + at1[c]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        y0[i] = y0[i] * norm * w0.get(i);
                        if (two) y1[i] = y1[i] * norm * w1.get(i);
                    }
                }
                const float2* turn = s_turn + t * half;
                if (a.neighbours && VEC > 1) {
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) {
                        const int32_t j0 = (at0[c] + i) / 2, j1 = (at1[c] + i) / 2;
                        if (j0 < half) {
                            const float2 cs = turn[j0];
                            const float u = y0[i], w = y0[i + 1];
                            y0[i] = u * cs.x - w * cs.y;
                            y0[i + 1] = u * cs.y + w * cs.x;
                        }
                        if (j1 < half) {
                            const float2 cs = turn[j1];
                            const float u = y1[i], w = y1[i + 1];
                            y1[i] = u * cs.x - w * cs.y;
                            y1[i + 1] = u * cs.y + w * cs.x;
                        }
                    }
                } else if (a.neighbours ? p < half : p < turned) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float2 cs = turn[p * VEC + i];
                        const float u = y0[i], w = y1[i];
                        y0[i] = u * cs.x - w * cs.y;
                        y1[i] = u * cs.y + w * cs.x;
                    }
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    lo[c].set(i, y0[i]);
                    if (two) hi[c].set(i, y1[i]);
                }
            }
            lo[c].store(dst + at0[c]);
            if (two) hi[c].store(dst + at1[c]);
        }
    }
}

}  // namespace pa

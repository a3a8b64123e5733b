// serving.cu -- C-ABI entry points of the steps around paged attention: pa_rope_write,
// pa_verify_tree, pa_release_blocks, pa_fork_blocks.  Host side only, as pa.cu; a
// source file of its own so that both compile at the same time.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <iterator>

#include "common.cuh"
#include "debug_checks.h"
#include "host_util.cuh"
#include "pool_blocks.cuh"
#include "rope_write.cuh"
#include "verify_tree.cuh"

namespace pa {

bool take_serving_error(unsigned int* bits) {
    const unsigned int zero = 0;
    return cudaMemcpyFromSymbol(bits, g_device_error, sizeof(*bits)) == cudaSuccess &&
           (*bits == 0 || cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) == cudaSuccess);
}

namespace {

// launch_pdl of a grid whose CTAs form clusters of `ctas` along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, unsigned ctas, size_t smem,
                           cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PA_USE_PDL ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// An array of a call: its span in bytes, and what it may be the same array as.
struct Span {
    const void* p;
    size_t bytes, align;
    const void* may_be;             // an output may be this input itself
};

// Alignment of all, and every output apart from the other arrays.
template <size_t I, size_t O>
bool spans_ok(const Span (&in)[I], const Span (&out)[O]) {
    for (const Span& x : in)
        if (!aligned(x.p, x.align)) return false;
    for (size_t x = 0; x < O; ++x) {
        if (!aligned(out[x].p, out[x].align)) return false;
        for (size_t y = 0; y < x; ++y)
            if (overlap(out[x].p, out[x].bytes, out[y].p, out[y].bytes)) return false;
        for (const Span& y : in)
            if (!(out[x].p == y.p && y.p == out[x].may_be) &&
                overlap(out[x].p, out[x].bytes, y.p, y.bytes))
                return false;
    }
    return true;
}

// Bytes from the first to the last element of `rows` rows of `width` elements, `stride`
// apart.
size_t strided_bytes(int64_t rows, int64_t stride, int64_t width, int elem) {
    return rows == 0 ? 0 : (size_t)((rows - 1) * stride + width) * elem;
}

// ---- rope_write ------------------------------------------------------------------------

template <typename E, int VEC>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    constexpr int C = std::max(1, 4 / VEC);
    const int32_t pieces = VEC == 1 ? (a.head_dim + 1) / 2 : a.head_dim / (2 * VEC);
    const int32_t per = (pieces + 31) / 32, lanes = (pieces + per - 1) / per;
    // warps of a token: more while 8 a SM hold them and they find a row each (32 + 8 heads
    // of 128 on bf16, 1, 2, 4 and 8 warps a token, rows from memory: 150 tokens 9.3, 6.4, 5.4,
    // 5.0 us, 600 tokens 9.7, 7.4, 7.9, 9.3, 1200 tokens 11.2, 11.2, 12.7, 14.2)
    const int32_t rows = std::max(a.num_q_heads, a.num_kv_heads), groups = 32 / lanes;
    const int64_t room = (int64_t)std::max(1, device_sm_count()) * 8;
    int32_t splits = 1;
    while (splits < 16 && 2 * splits * (int64_t)a.num_tokens <= room && splits * groups < rows) splits *= 2;
    // two also where one would leave a third of the 24 a SM that 16-byte pieces of bf16 have,
    // and has 8 turns of query rows or more.  One and two warps, rows from memory, with norms:
    // 2303 tokens of 64 + 8 heads of 128 27.0, 22.8 us, of 32 + 8 17.7, 16.5, 1300 of them 11.6,
    // 11.4; but 1000 10.6, 11.1 and 3000 18.4, 18.7, and with 4 turns, 2303 of 16 + 4 heads of
    // 128 11.2, 12.7, of 32 + 8 heads of 64 10.5, 11.5.  (fp32, of 32 a SM: 2303 tokens of 15 + 5
    // heads of 80 9.9, 10.0.)
    if (sizeof(E) == 2 && VEC == 8 && a.num_tokens > room && a.num_tokens <= 2 * room && rows >= 8 * groups)
        splits = 2;
    const size_t ring = VEC * sizeof(E) == 16 ? (size_t)kRopeDepth * 2 * kRopeThreads * 16 : 0;
    const size_t smem = ring + (size_t)kRopeWarps * (a.rot_dim / 2) * sizeof(float2);
    const int64_t ctas = ((int64_t)a.num_tokens * splits + kRopeWarps - 1) / kRopeWarps;
    const dim3 grid((unsigned)ctas), block(kRopeThreads);
    return a.neighbours
               ? launch_pdl(rope_write_kernel<E, VEC, C, true>, grid, block, smem, st, a, splits, lanes)
               : launch_pdl(rope_write_kernel<E, VEC, C, false>, grid, block, smem, st, a, splits, lanes);
}

// Widest pieces that the head dim and the rotated part hold whole, and the pointers
// and strides are aligned to.
int rope_vec(const RopeArgs& a, int elem) {
    for (int vec = 16 / elem; vec > 1; vec /= 2) {
        const size_t bytes = (size_t)vec * elem;
        const bool fits = a.head_dim % (2 * vec) == 0 &&
                          (a.neighbours || a.rot_dim % (2 * vec) == 0) &&
                          (a.q_stride * elem) % bytes == 0 && (a.k_stride * elem) % bytes == 0 &&
                          (a.v_stride * elem) % bytes == 0;
        if (fits && aligned(a.q, bytes) && aligned(a.k, bytes) && aligned(a.v, bytes) &&
            aligned(a.q_weight, bytes) && aligned(a.k_weight, bytes) && aligned(a.out, bytes) &&
            aligned(a.k_cache, bytes) && aligned(a.v_cache, bytes))
            return vec;
    }
    return 1;
}

// ---- verify_tree -----------------------------------------------------------------------

template <typename E, bool DRAFT, bool WIDE>
cudaError_t launch_verify(const VerifyArgs& a, int32_t num_seqs, cudaStream_t st) {
    // CTAs of a sequence: up to 8, each with 2048 tokens of the vocabulary or more while
    // all CTAs find room at once (4 a SM), else with 8192 or more, where a step's fixed
    // costs count once a CTA.  1, 2, 4 and 8 CTAs, chains of 5 nodes on bf16: one of 16000
    // tokens 18.2, 13.8, 11.8, 11.4 us, one of 131072 84, 47, 29, 19; 128 of 8000 18.3,
    // 17.7, 22.1, 34.5, of 32000 35, 30, 30, 40; 400 of 32000 83, 69, 76, 109, of 131072
    // 295, 241, 217, 211.  Sequences of one node, from memory: 64 of 131072 32.6, 22.7, 18.7, 18.2,
    // 256 of 128256 57, 62, 56, 58 (greedy 47, 42, 45, 51), 400 of 32000 25, 28, 33, 53: more CTAs
    // than these need, as chains of 5 want them.
    const int64_t room = (int64_t)std::max(1, device_sm_count()) * 4;
    unsigned ctas = 1;
    while (ctas < 8 && a.vocab / (2 * (int32_t)ctas) >= ((int64_t)num_seqs * 2 * ctas <= room ? 2048 : 8192)) ctas *= 2;
    auto kern = verify_tree_kernel<E, DRAFT, WIDE>;
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, kern, kVerifyRing)) return cudaErrorUnknown;
    return launch_cluster(kern, dim3(num_seqs * ctas), dim3(kVerifyThreads), ctas, kVerifyRing, st, a);
}

template <typename E>
cudaError_t dispatch_verify(const VerifyArgs& a, int32_t num_seqs, bool wide, cudaStream_t st) {
    if (a.draft != nullptr)
        return wide ? launch_verify<E, true, true>(a, num_seqs, st) : launch_verify<E, true, false>(a, num_seqs, st);
    return wide ? launch_verify<E, false, true>(a, num_seqs, st) : launch_verify<E, false, false>(a, num_seqs, st);
}

// ---- release, fork -----------------------------------------------------------------------

// Whether the current device runs clusters of 16 of the release kernel (8 is what every
// device does), asked for once.
bool pool_sixteen() {
    static std::atomic<uint8_t> known[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    uint8_t x = known[dev].load(std::memory_order_acquire);
    if (x == 0) {
        auto can = [](auto kern) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kPoolMaxCluster);
            cfg.blockDim = dim3(kPoolThreads);
            cfg.dynamicSmemBytes = kPoolKept * 4;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = kPoolMaxCluster;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPoolKept * 4) == cudaSuccess &&
                   cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                   cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
        };
        x = can(release_blocks_kernel<false>) && can(release_blocks_kernel<true>) ? 2 : 1;
        cudaGetLastError();
        known[dev].store(x, std::memory_order_release);
    }
    return x == 2;
}

// CTAs of the cluster, by the entries that there can be: a CTA for every 2048 of them up
// to 8, then 16 where each has 16384 or more.  (256 rows of 258, of which 1800 entries
// come back: 8.1 us with 2 CTAs, 8.3 with 8, 8.5 with 16.  96 forks in 128 rows of 130 and
// their release with counts: 40 us with 2, 34 with 8.  2048 rows of 377, 220000 entries
// back: 91 us with 2, 20.8 with 8, 14.8 with 16.)
unsigned pool_ctas(int32_t num_seqs, int32_t max_blocks, unsigned most) {
    const int64_t entries = (int64_t)num_seqs * max_blocks;
    unsigned ctas = 1;
    while (ctas < most && entries > (int64_t)ctas * (ctas < 8 ? 2048 : 16384)) ctas *= 2;
    return ctas;
}

// The entries of a CTA stay in shared memory between the kernel's passes, up to 160 KB.
template <bool COUNTED>
cudaError_t launch_release(ReleaseArgs a, cudaStream_t st) {
    auto kern = release_blocks_kernel<COUNTED>;
    const unsigned ctas = pool_ctas(a.num_seqs, a.max_blocks, pool_sixteen() ? 16 : 8);
    // (a warp's share is rounded up to 32)
    const int64_t share = ((int64_t)a.num_seqs * a.max_blocks + ctas - 1) / ctas + 33 * kPoolWarps;
    a.kept = (int32_t)std::min<int64_t>(share, kPoolKept);
    static std::atomic<uint64_t> allowed;
    if (!allow_smem(allowed, kern, kPoolKept * 4)) return cudaErrorUnknown;
    return launch_cluster(kern, dim3(ctas), dim3(kPoolThreads), ctas, (size_t)a.kept * 4, st, a);
}

template <int LAYERS>
cudaError_t launch_fork_copy(const ForkArgs& a, const pa_cache_desc* cache, void* const* k,
                             void* const* v, int32_t layers, int vec, cudaStream_t st) {
    ForkCaches<LAYERS> c;
    for (int32_t l = 0; l < layers; ++l) {
        c.k[l] = static_cast<uint8_t*>(k[l]);
        c.v[l] = static_cast<uint8_t*>(v[l]);
    }
    const dim3 grid(a.num_seqs, 2 * layers), block(kForkThreads);
    const int32_t row = cache->head_dim * elem_bytes(cache), heads = cache->num_kv_heads;
    switch (vec) {
        case 16: return launch_pdl(fork_copy_kernel<16, LAYERS>, grid, block, 0, st, a, heads, row, c);
        case 8: return launch_pdl(fork_copy_kernel<8, LAYERS>, grid, block, 0, st, a, heads, row, c);
        case 4: return launch_pdl(fork_copy_kernel<4, LAYERS>, grid, block, 0, st, a, heads, row, c);
        default: return launch_pdl(fork_copy_kernel<2, LAYERS>, grid, block, 0, st, a, heads, row, c);
    }
}

constexpr int32_t kMostBlocks = INT32_MAX - (1 << 20);
constexpr int32_t kForkMaxLayers = 1024;        // layers of one call

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_rope_write(const void* q, const void* k, const void* v, int64_t q_stride,
                        int64_t k_stride, int64_t v_stride, int32_t num_tokens,
                        int32_t num_q_heads, const int32_t* positions, const float* inv_freq,
                        const void* q_weight, const void* k_weight, const pa_rope_desc* rope,
                        const int64_t* slot_mapping, void* out, void* k_cache, void* v_cache,
                        const pa_cache_desc* cache, void* stream) {
    const CallRange range("pa_rope_write");
    if (!desc_ok(cache) || !rope || num_tokens < 0 || num_q_heads <= 0 ||
        num_q_heads % cache->num_kv_heads || rope->rot_dim < 0 || rope->rot_dim % 2 ||
        rope->rot_dim > cache->head_dim || rope->num_axes < 1 || rope->num_axes > 3 ||
        !(rope->eps >= 0.f) || !std::isfinite(rope->eps) || !std::isfinite(rope->scale))
        return PA_ERR_INVALID_ARG;
    const int32_t D = cache->head_dim, half = rope->rot_dim / 2;
    int64_t pairs = 0;
    for (int x = 0; x < rope->num_axes; ++x) {
        if (rope->num_axes > 1 && rope->sections[x] < 0) return PA_ERR_INVALID_ARG;
        pairs += rope->sections[x];
    }
    if (rope->num_axes > 1 && pairs != half) return PA_ERR_INVALID_ARG;
    if (rope->num_axes > 1 && rope->cyclic) {
        // every pair of the later axes inside the head's rotated part
        for (int x = 1; x < rope->num_axes; ++x)
            if (rope->sections[x] > 0 &&
                (int64_t)(rope->sections[x] - 1) * rope->num_axes + x >= half)
                return PA_ERR_INVALID_ARG;
    }
    if (num_tokens == 0) return PA_OK;
    if (D > kRopeMaxDim) return PA_ERR_UNSUPPORTED;
    const int64_t q_row = (int64_t)num_q_heads * D, kv_row = (int64_t)cache->num_kv_heads * D;
    if (!q || !k || !v || !positions || (half > 0 && !inv_freq) || !slot_mapping || !out ||
        !k_cache || !v_cache || q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 1) {              // (no other token is anywhere)
        q_stride = q_row;
        k_stride = v_stride = kv_row;
    }
    const int eb = elem_bytes(cache);
    const int64_t most = INT64_MAX / 16 / num_tokens;
    if (q_stride > most || k_stride > most || v_stride > most) return PA_ERR_INVALID_ARG;
    const size_t cache_bytes = (size_t)cache->num_blocks * cache->block_size * kv_row * eb;
    const size_t n = (size_t)num_tokens;
    const Span in[] = {{q, strided_bytes(num_tokens, q_stride, q_row, eb), (size_t)eb, nullptr},
                       {k, strided_bytes(num_tokens, k_stride, kv_row, eb), (size_t)eb, nullptr},
                       {v, strided_bytes(num_tokens, v_stride, kv_row, eb), (size_t)eb, nullptr},
                       {positions, n * 4 * rope->num_axes, 4, nullptr},
                       {inv_freq, (size_t)half * 4, 4, nullptr},
                       {q_weight, (size_t)D * eb, (size_t)eb, nullptr},
                       {k_weight, (size_t)D * eb, (size_t)eb, nullptr},
                       {slot_mapping, n * 8, 8, nullptr}};
    // (in place: rows of q that follow one another)
    const Span outs[] = {{out, n * q_row * eb, (size_t)eb, q_stride == q_row ? q : nullptr},
                         {k_cache, cache_bytes, (size_t)eb, nullptr},
                         {v_cache, cache_bytes, (size_t)eb, nullptr}};
    if (!spans_ok(in, outs)) return PA_ERR_INVALID_ARG;
    RopeArgs a{};
    a.q = static_cast<const uint8_t*>(q);
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.q_weight = static_cast<const uint8_t*>(q_weight);
    a.k_weight = static_cast<const uint8_t*>(k_weight);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.slot_mapping = slot_mapping;
    a.out = static_cast<uint8_t*>(out);
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.num_slots = (int64_t)cache->num_blocks * cache->block_size;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = cache->num_kv_heads;
    a.head_dim = D;
    a.block_size = cache->block_size;
    a.rot_dim = rope->rot_dim;
    a.axes = rope->num_axes;
    a.cyclic = rope->cyclic != 0;
    a.neighbours = rope->neighbours != 0;
    for (int x = 0; x < 3; ++x) a.section[x] = x < rope->num_axes ? rope->sections[x] : 0;
    a.eps = rope->eps;
    a.scale = rope->scale;
    const CallDevice dev;
    if (!dev.map(a.q) || !dev.map(a.k) || !dev.map(a.v) ||
        !dev.map(a.q_weight) || !dev.map(a.k_weight) ||
        !dev.map(a.positions) || !dev.map(a.inv_freq) ||
        !dev.map(a.slot_mapping) || !dev.map(a.out) ||
        !dev.memory(k_cache) || !dev.memory(v_cache))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass(
            [&] { return debug::check_live_slots(a.slot_mapping, a.positions, num_tokens, a.num_slots, st); });
        if (r != PA_OK) return r;
    }
    const int vec = rope_vec(a, eb);
    cudaError_t err;
    if (cache->dtype == PA_F32)
        err = vec == 4   ? launch_rope<float, 4>(a, st)
              : vec == 2 ? launch_rope<float, 2>(a, st)
                         : launch_rope<float, 1>(a, st);
    else
        err = vec == 8   ? launch_rope<__nv_bfloat16, 8>(a, st)
              : vec == 4 ? launch_rope<__nv_bfloat16, 4>(a, st)
              : vec == 2 ? launch_rope<__nv_bfloat16, 2>(a, st)
                         : launch_rope<__nv_bfloat16, 1>(a, st);
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_verify_tree(const void* logits, const void* draft_logits, int64_t logit_stride,
                         int64_t draft_stride, int32_t vocab_size, int32_t dtype,
                         const int32_t* tokens, const int32_t* parents,
                         const int32_t* query_start_loc, int32_t num_seqs, int32_t total_q,
                         int32_t max_q_len, const float* uniforms, const float* noise,
                         int64_t noise_stride, const float* temperature, int32_t* leaf,
                         int32_t* next_tokens, void* stream) {
    const CallRange range("pa_verify_tree");
    if (num_seqs < 0 || total_q < 0 || max_q_len < 0 || vocab_size <= 0 ||
        (dtype != PA_F32 && dtype != PA_BF16))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (max_q_len > PA_MAX_TREE_NODES || num_seqs > 65535 || vocab_size > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (!query_start_loc || !noise || !leaf || !next_tokens || logit_stride < vocab_size ||
        noise_stride < vocab_size || (draft_logits && draft_stride < vocab_size) ||
        (total_q > 0 && (!logits || !tokens || !parents || !uniforms)))
        return PA_ERR_INVALID_ARG;
    const int eb = dtype == PA_F32 ? 4 : 2;
    const int64_t most = INT64_MAX / 16 / std::max(std::max(total_q, num_seqs), 1);
    if (logit_stride > most || noise_stride > most || (draft_logits && draft_stride > most))
        return PA_ERR_INVALID_ARG;
    const size_t n = (size_t)num_seqs * 4, rows = (size_t)total_q * 4;
    const Span in[] = {{logits, strided_bytes(total_q, logit_stride, vocab_size, eb), (size_t)eb, nullptr},
                       {draft_logits, strided_bytes(total_q, draft_stride, vocab_size, eb), (size_t)eb, nullptr},
                       {tokens, rows, 4, nullptr}, {parents, rows, 4, nullptr},
                       {query_start_loc, n + 4, 4, nullptr}, {uniforms, rows, 4, nullptr},
                       {noise, strided_bytes(num_seqs, noise_stride, vocab_size, 4), 4, nullptr},
                       {temperature, n, 4, nullptr}};
    const Span outs[] = {{leaf, n, 4, nullptr}, {next_tokens, n, 4, nullptr}};
    if (!spans_ok(in, outs)) return PA_ERR_INVALID_ARG;
    VerifyArgs a{logits, draft_logits, logit_stride, draft_stride, noise_stride, tokens, parents,
                 query_start_loc, uniforms, noise, temperature, leaf, next_tokens, total_q,
                 max_q_len, vocab_size};
    const CallDevice dev;
    if (!dev.map(a.logits) || !dev.map(a.draft) || !dev.map(a.tokens) ||
        !dev.map(a.parents) || !dev.map(a.query_start) ||
        !dev.map(a.uniforms) || !dev.map(a.noise) ||
        !dev.map(a.temperature) || !dev.map(a.leaf) || !dev.map(a.next))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass([&] {
            return debug::check_tree(a.query_start, num_seqs, a.parents, total_q, max_q_len, nullptr, st);
        });
        if (r != PA_OK) return r;
    }
    const bool wide = aligned(a.logits, 16) && aligned(a.draft, 16) && aligned(a.noise, 16) &&
                      logit_stride * eb % 16 == 0 && noise_stride * 4 % 16 == 0 &&
                      (!a.draft || draft_stride * eb % 16 == 0);
    const cudaError_t err = dtype == PA_F32 ? dispatch_verify<float>(a, num_seqs, wide, st)
                                            : dispatch_verify<__nv_bfloat16>(a, num_seqs, wide, st);
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_release_blocks(const int32_t* seq_lens, const int32_t* block_tables,
                            int32_t max_blocks_per_seq, const int32_t* blocks_held,
                            int32_t num_seqs, int32_t* free_blocks, int32_t num_free,
                            const int32_t* free_head, int32_t* ref_cnt, int32_t num_blocks,
                            int32_t block_size, int32_t* blocks_held_out, int32_t* free_head_out,
                            void* stream) {
    const CallRange range("pa_release_blocks");
    if (num_seqs < 0 || num_free < 0 || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_free >= kMostBlocks) return PA_ERR_UNSUPPORTED;
    if ((num_seqs > 0 && (!seq_lens || !blocks_held || !blocks_held_out ||
                          (max_blocks_per_seq > 0 && !block_tables))) ||
        !free_head || !free_head_out || (num_free > 0 && !free_blocks))
        return PA_ERR_INVALID_ARG;
    const size_t n = (size_t)num_seqs * 4;
    const Span in[] = {{seq_lens, n, 4, nullptr}, {blocks_held, n, 4, nullptr},
                       {block_tables, n * max_blocks_per_seq, 4, nullptr}, {free_head, 4, 4, nullptr}};
    const Span outs[] = {{blocks_held_out, n, 4, blocks_held}, {free_head_out, 4, 4, free_head},
                         {free_blocks, (size_t)num_free * 4, 4, nullptr},
                         {ref_cnt, (size_t)num_blocks * 4, 4, nullptr}};
    if (!spans_ok(in, outs)) return PA_ERR_INVALID_ARG;
    ReleaseArgs a{seq_lens, block_tables, blocks_held, free_blocks, free_head, ref_cnt,
                  blocks_held_out, free_head_out, num_seqs, num_free, num_blocks, block_size,
                  max_blocks_per_seq, 0};
    const CallDevice dev;
    if (!dev.map(a.seq_lens) || !dev.map(a.blocks_held) || !dev.map(a.free_head) ||
        !dev.map(a.blocks_held_out) || !dev.map(a.free_head_out) ||
        !dev.map(a.free_blocks) || (block_tables && !dev.memory(block_tables)) ||
        (ref_cnt && !dev.memory(ref_cnt)))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass([&] {
            return debug::check_release(a.seq_lens, a.blocks_held, num_seqs, block_tables, max_blocks_per_seq,
                                        a.free_blocks, num_free, a.free_head, ref_cnt, num_blocks, block_size, st);
        });
        if (r != PA_OK) return r;
    }
    const cudaError_t err = ref_cnt ? launch_release<true>(a, st) : launch_release<false>(a, st);
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_fork_blocks(const int32_t* src, const int32_t* seq_lens, int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* blocks_held, int32_t num_seqs,
                         int32_t* ref_cnt, const int32_t* free_blocks, int32_t num_free,
                         const int32_t* free_head, void* const* k_caches, void* const* v_caches,
                         int32_t num_layers, int32_t* seq_lens_out, int32_t* blocks_held_out,
                         int32_t* free_head_out, int64_t* block_pairs, const pa_cache_desc* cache,
                         void* stream) {
    const CallRange range("pa_fork_blocks");
    if (!desc_ok(cache) || num_seqs < 0 || num_free < 0 || max_blocks_per_seq < 0 || num_layers < 1)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_free >= kMostBlocks || num_layers > kForkMaxLayers)
        return PA_ERR_UNSUPPORTED;
    if ((num_seqs > 0 && (!src || !seq_lens || !blocks_held || !seq_lens_out || !blocks_held_out ||
                          !block_pairs || (max_blocks_per_seq > 0 && !block_tables))) ||
        !ref_cnt || !free_head || !free_head_out || (num_free > 0 && !free_blocks) || !k_caches || !v_caches)
        return PA_ERR_INVALID_ARG;
    const size_t n = (size_t)num_seqs * 4;
    const Span in[] = {{src, n, 4, nullptr}, {seq_lens, n, 4, nullptr}, {blocks_held, n, 4, nullptr},
                       {free_blocks, (size_t)num_free * 4, 4, nullptr}, {free_head, 4, 4, nullptr}};
    const Span outs[] = {{seq_lens_out, n, 4, seq_lens}, {blocks_held_out, n, 4, blocks_held},
                         {free_head_out, 4, 4, free_head}, {block_pairs, 4 * n, 8, nullptr},
                         {block_tables, n * max_blocks_per_seq, 4, nullptr},
                         {ref_cnt, (size_t)cache->num_blocks * 4, 4, nullptr}};
    if (!spans_ok(in, outs)) return PA_ERR_INVALID_ARG;
    ForkArgs a{src, seq_lens, block_tables, blocks_held, ref_cnt, free_blocks, free_head,
               seq_lens_out, blocks_held_out, free_head_out, block_pairs, num_seqs, num_free,
               cache->num_blocks, cache->block_size, max_blocks_per_seq};
    const CallDevice dev;
    if (!dev.map(a.src) || !dev.map(a.seq_lens) || !dev.map(a.blocks_held) ||
        !dev.map(a.free_blocks) || !dev.map(a.free_head) ||
        !dev.map(a.seq_lens_out) || !dev.map(a.blocks_held_out) ||
        !dev.map(a.free_head_out) || !dev.map(a.block_pairs) ||
        (block_tables && !dev.memory(block_tables)) || !dev.memory(ref_cnt))
        return PA_ERR_INVALID_ARG;
    // the caches, none of which may share a byte with another
    const int32_t row = cache->head_dim * elem_bytes(cache);
    int vec = 16;
    while (vec > 2 && row % vec) vec >>= 1;
    uintptr_t bases[2 * kForkMaxLayers];
    CallMemory known[2] = {CallMemory(dev), CallMemory(dev)};
    for (int32_t l = 0; l < num_layers; ++l) {
        for (int which = 0; which < 2; ++which) {
            void* c = which ? v_caches[l] : k_caches[l];
            if (!known[which].memory(c) || !aligned(c, elem_bytes(cache))) return PA_ERR_INVALID_ARG;
            while (vec > 2 && !aligned(c, vec)) vec >>= 1;
            bases[2 * l + which] = reinterpret_cast<uintptr_t>(c);
        }
    }
    std::sort(bases, bases + 2 * num_layers);
    const size_t cache_bytes = (size_t)cache->num_blocks * cache->num_kv_heads * cache->block_size * (size_t)row;
    for (int32_t x = 1; x < 2 * num_layers; ++x)
        if (bases[x] - bases[x - 1] < cache_bytes) return PA_ERR_INVALID_ARG;
    // ... nor with the other arrays: the last cache that starts before an array's end
    auto inside = [&](const Span& x) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(x.p);
        const uintptr_t* last = std::lower_bound(bases, bases + 2 * num_layers, p + x.bytes);
        return last != bases && overlap(x.p, x.bytes, reinterpret_cast<const void*>(last[-1]), cache_bytes);
    };
    if (std::any_of(std::begin(in), std::end(in), inside) || std::any_of(std::begin(outs), std::end(outs), inside))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug::enabled()) {
        const pa_status r = debug_pass([&] {
            const pa_status x = debug::check_fork(a.src, a.seq_lens, a.blocks_held, num_seqs, block_tables,
                                                  max_blocks_per_seq, ref_cnt, cache, st);
            return x != PA_OK ? x
                              : debug::check_free(a.free_blocks, num_free, a.free_head, cache->num_blocks, st);
        });
        if (r != PA_OK) return r;
    }
    const unsigned ctas = pool_ctas(num_seqs, max_blocks_per_seq, 8);
    cudaError_t err = launch_cluster(fork_blocks_kernel, dim3(ctas), dim3(kPoolThreads), ctas, 0, st, a);
    for (int32_t l0 = 0; err == cudaSuccess && num_seqs > 0 && l0 < num_layers; l0 += kForkLayers) {
        const int32_t nl = std::min(kForkLayers, num_layers - l0);
        err = nl <= 16 ? launch_fork_copy<16>(a, cache, k_caches + l0, v_caches + l0, nl, vec, st)
                       : launch_fork_copy<kForkLayers>(a, cache, k_caches + l0, v_caches + l0, nl, vec, st);
    }
    return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"

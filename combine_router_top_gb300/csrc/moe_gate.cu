// moe_gate.cu -- the gated route (softmax or sigmoid scores, a balance bias,
// groups, top-k, renormalised weights) and its gradient.
//
// The choice goes by key_e = s_e + bias_e, or by the logit itself where there is
// no bias: logits order as their scores do, with no rounding in between. Every
// key is one 32-bit word that orders as the float does, so that a round of the
// warp's arg-max is one redux.sync. The words 1 and 0 lie below every number's:
//   1  masked, or of a group that was not chosen: taken only when nothing else
//      is left, and then no pair;
//   0  already taken, or past the last expert.
//
// One warp per token. Lane l holds consecutive experts of one group: L = 32 / G
// lanes to a group, v = ceil((E/G) / L) experts to a lane, so that lanes ascend
// with the experts and the lowest tied lane holds the lowest tied index.
// The route's counting is that of moe_route.cu: tiles of 8 or 32 tokens, a mask
// word per expert whose bits are the tile's tokens, and the slot kernels there.
// Up to 32 tokens one block does the whole route in one launch. Small batches are
// bound by latency (1 token x 256 experts 6.2 us a call, 1024 tokens 9.9), large ones
// by the choice's instructions (16384 tokens, bf16: 36.7 us, 1127 of a warp a token).
#include <math.h>

#include <algorithm>

#include "moe_gate.cuh"

namespace moe {
namespace {

enum GateTile { kOneTile, kTiles8, kTiles32 };

// One block per tile of tokens, the warps taking its tokens in turn. kOneTile:
// the batch is one tile, and the block ends the route by itself. kTiles8 and
// kTiles32: each pair's rank within its tile goes to slot, the tile's count per
// expert to the workspace, and the slot kernels of moe_route.cu follow. A choice
// that is no pair gets a rank past every capacity, so that its slot becomes -1.
// Lanes of up to 16 experts leave room for 32 warps to a block; wider ones keep
// their keys in registers with 8.
template <typename T, int V>
__global__ void __launch_bounds__(V <= 16 ? 1024 : 256)
gate_kernel(const T *__restrict__ logits, const float *__restrict__ bias, GateArgs a, GateTile mode,
            int32_t *__restrict__ topk_idx, float *__restrict__ topk_w, int32_t *__restrict__ slot,
            void *__restrict__ tile_counts, int stride, int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
            int32_t *__restrict__ rank_counts, int32_t *__restrict__ dropped) {
    __shared__ uint32_t mask[kMaxExperts];
    __shared__ int32_t chosen[kTileTokens * kMaxTopK];                 // expert of each pair, -1: no pair
    __shared__ int wsum[32];
    constexpr int32_t kNoPair = 1 << 30;                               // + any count stays below 2^31
    const int lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) mask[e] = 0u;
    __syncthreads();
    pdl_enter();
    const int tile_tokens = mode == kTiles8 ? kSmallTileTokens : kTileTokens;
    const int t0 = blockIdx.x * tile_tokens;
    const int tokens = min(a.T - t0, tile_tokens);
    for (int i = threadIdx.x >> 5; i < tokens; i += blockDim.x >> 5) {
        int e;
        float w;
        bool ok;
        warp_gate<T, V>(logits + (size_t)(t0 + i) * a.E, bias, a, lane, e, w, ok);
        if (lane < a.k) {
            topk_idx[(size_t)(t0 + i) * a.k + lane] = e;
            topk_w[(size_t)(t0 + i) * a.k + lane] = w;
            chosen[i * a.k + lane] = ok ? e : -1;
            if (ok) atomicOr(&mask[e], 1u << i);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * a.k; i += blockDim.x) {
        const int e = chosen[i];
        const int rank = e >= 0 ? __popc(mask[e] & ((1u << (i / a.k)) - 1u)) : kNoPair;
        slot[(size_t)t0 * a.k + i] = mode == kOneTile ? (rank < a.C ? rank : -1) : rank;
    }
    if (mode == kTiles8) {
        uint8_t *c8 = static_cast<uint8_t *>(tile_counts);
        for (int e = threadIdx.x; e < a.E; e += blockDim.x)
            c8[(size_t)e * stride + blockIdx.x] = (uint8_t)__popc(mask[e]);
    } else if (mode == kTiles32) {
        int32_t *c = static_cast<int32_t *>(tile_counts);
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) c[(size_t)blockIdx.x * a.E + e] = __popc(mask[e]);
    } else {
        __syncthreads();                                               // every rank above is formed
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) mask[e] = __popc(mask[e]);
        __syncthreads();
        route_totals(reinterpret_cast<const int *>(mask), a.E, a.R, a.C, counts, offsets, rank_counts, dropped, wsum);
    }
}

// ---- gradient -----------------------------------------------------------------

// The factor on the weights, and its reciprocal in two steps that stay in range for every finite scale: w / scale =
// w up inv with up a power of two (so that w up is exact) and |scale| up within [1, 4), or 2^-23 and more for subnormal
// scales, whose own reciprocal overflows.
struct GateScale {
    float scale, up, inv;
};

// LP lanes to a token, NV 16-byte words of its row to a lane. The lanes form the
// chosen experts' gradients between them, then write the row whole (zeros, or
// -a s_e dot for a softmax over all experts) and the chosen places after it, within
// the same warp. Bound by the T*E elements written (and, for a softmax over all
// experts, read, which stay in registers from the sum to the product).
template <typename T, bool DENSE, int LP, int NV>
__global__ void __launch_bounds__(256)
gate_backward_kernel(const T *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                     const float *__restrict__ topk_w, const float *__restrict__ d_topk_w, T *__restrict__ d_logits,
                     int T_, int E, int k, int sigm, int renorm, GateScale by) {
    constexpr int kVec = 16 / (int)sizeof(T), kTokens = 256 / LP, kPer = LP < kMaxTopK ? kMaxTopK / LP : 1;
    pdl_enter();
    const int sub = threadIdx.x % LP;
    const int words = E / kVec;
    for (int t0 = blockIdx.x * kTokens; t0 < T_; t0 += gridDim.x * kTokens) {
        const int t = t0 + threadIdx.x / LP;
        const bool live = t < T_;                                      // lanes past the end go through the motions
        const T *row = logits + (size_t)t * E;
        T *out = d_logits + (size_t)t * E;
        uint4 word[NV];
        if constexpr (DENSE) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (live && v * LP + sub < words) word[v] = ld_stream_v4(reinterpret_cast<const uint4 *>(row) + v * LP + sub);
        }
        int e[kPer];
        float w[kPer], gw[kPer], f[kPer], part = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = i * LP + sub;
            e[i] = -1;
            w[i] = gw[i] = f[i] = 0.0f;
            if (live && j < k) {
                e[i] = __ldg(topk_idx + (size_t)t * k + j);
                w[i] = __ldg(topk_w + (size_t)t * k + j);
                gw[i] = __ldg(d_topk_w + (size_t)t * k + j);
                if ((unsigned)e[i] >= (unsigned)E) e[i] = -1;
                if (e[i] >= 0 && sigm) f[i] = to_f32(row[e[i]]);
                if (e[i] < 0 || w[i] == 0.0f) w[i] = gw[i] = 0.0f;     // no pair: whatever d_topk_w holds
            }
            part = __fmaf_rn(__fmul_rn(w[i], by.up), gw[i], part);
        }
        const float dot = (DENSE || renorm) ? __fmul_rn(lanes_sum<LP>(part), by.inv) : 0.0f;
        if constexpr (DENSE) {
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (live && v * LP + sub < words) {
                    float x[kVec];
                    unpack16(word[v], x);
#pragma unroll
                    for (int q = 0; q < kVec; ++q) top = fmaxf(top, x[q]);         // NaN stays out
                }
            }
            top = lanes_max<LP>(top);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (live && v * LP + sub < words) {
                    float x[kVec];
                    unpack16(word[v], x);
#pragma unroll
                    for (int q = 0; q < kVec; ++q)
                        if (open_logit(x[q])) total = __fadd_rn(total, exp_below(x[q], top));
                }
            }
            total = lanes_sum<LP>(total);
            const float c = total > 0.0f ? __fdiv_rn(-__fmul_rn(by.scale, dot), total) : 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (live && v * LP + sub < words) {
                    float x[kVec];
                    unpack16(word[v], x);
#pragma unroll
                    for (int q = 0; q < kVec; ++q) x[q] = open_logit(x[q]) ? __fmul_rn(exp_below(x[q], top), c) : 0.0f;
                    st_v4(reinterpret_cast<uint4 *>(out) + v * LP + sub, pack16(x));
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (live && v * LP + sub < words)
                    st_v4(reinterpret_cast<uint4 *>(out) + v * LP + sub, make_uint4(0u, 0u, 0u, 0u));
        }
        __syncwarp();                                                  // the row before the chosen places
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float d = __fmul_rn(w[i], __fsub_rn(gw[i], dot));
            // 1 - sigmoid(f) = 1 / (1 + exp(f)); exp(f) = inf gives 0
            if (sigm) d = __fdiv_rn(d, __fadd_rn(1.0f, expf(f[i])));
            if (w[i] != 0.0f) from_f32(out + e[i], d);
        }
    }
}

// The same for rows that are no multiple of 16 bytes: a warp to a token, an element
// at a time.
template <typename T, bool DENSE>
__global__ void __launch_bounds__(256)
gate_backward_odd_kernel(const T *__restrict__ logits, const int32_t *__restrict__ topk_idx,
                         const float *__restrict__ topk_w, const float *__restrict__ d_topk_w,
                         T *__restrict__ d_logits, int T_, int E, int k, int sigm, int renorm, GateScale by) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    for (int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < T_; t += gridDim.x * (blockDim.x >> 5)) {
        const T *row = logits + (size_t)t * E;
        T *out = d_logits + (size_t)t * E;
        int e = -1;
        float w = 0.0f, gw = 0.0f, f = 0.0f;
        if (lane < k) {
            e = __ldg(topk_idx + (size_t)t * k + lane);
            w = __ldg(topk_w + (size_t)t * k + lane);
            gw = __ldg(d_topk_w + (size_t)t * k + lane);
            if ((unsigned)e >= (unsigned)E) e = -1;
            if (e >= 0 && sigm) f = to_f32(row[e]);
            if (e < 0 || w == 0.0f) w = gw = 0.0f;
        }
        const float dot = (DENSE || renorm) ? __fmul_rn(lanes_sum<32>(__fmul_rn(__fmul_rn(w, by.up), gw)), by.inv) : 0.0f;
        if constexpr (DENSE) {
            float top = -INFINITY, total = 0.0f;
            for (int i = lane; i < E; i += 32) top = fmaxf(top, to_f32(row[i]));
            top = lanes_max<32>(top);
            for (int i = lane; i < E; i += 32) {
                const float x = to_f32(row[i]);
                if (open_logit(x)) total = __fadd_rn(total, exp_below(x, top));
            }
            total = lanes_sum<32>(total);
            const float c = total > 0.0f ? __fdiv_rn(-__fmul_rn(by.scale, dot), total) : 0.0f;
            for (int i = lane; i < E; i += 32) {
                const float x = to_f32(row[i]);
                from_f32(out + i, open_logit(x) ? __fmul_rn(exp_below(x, top), c) : 0.0f);
            }
        } else {
            for (int i = lane; i < E; i += 32) from_f32(out + i, 0.0f);
        }
        __syncwarp();
        float d = __fmul_rn(w, __fsub_rn(gw, dot));
        if (sigm) d = __fdiv_rn(d, __fadd_rn(1.0f, expf(f)));
        if (w != 0.0f) from_f32(out + e, d);
    }
}

template <typename T, int V>
int launch_gate(const Dims &d, const GateArgs &a, cudaStream_t st, const void *logits, const float *bias,
                int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *slot,
                int32_t *rank_counts, int32_t *dropped, void *workspace) {
    const GateTile mode = d.T <= kTileTokens ? kOneTile : route_small(d.T, d.E) ? kTiles8 : kTiles32;
    const int tile = mode == kTiles8 ? kSmallTileTokens : kTileTokens;
    const int blocks = (d.T + tile - 1) / tile;
    const int most = V <= 16 ? 32 : 8;                                 // warps to a block
    // one tile: a warp per token, and at least 8 for the totals
    int warps = mode == kOneTile ? (d.T > 8 ? d.T : 8) : tile;
    if (warps > most) warps = most;
    if (launch_pdl(gate_kernel<T, V>, blocks, warps * 32, st, static_cast<const T *>(logits), bias, a, mode, topk_idx,
                   topk_w, slot, workspace, (int)route_small_stride(d.T), counts, offsets, rank_counts, dropped) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    if (mode == kOneTile) return MOE_OK;
    if (mode == kTiles8)
        return launch_route_slots_small(d, st, static_cast<const uint8_t *>(workspace), topk_idx, slot, counts,
                                        offsets, rank_counts, dropped);
    return launch_route_slots_large(d, st, static_cast<int32_t *>(workspace), topk_idx, slot, counts, offsets,
                                    rank_counts, dropped);
}

template <typename T, typename... A>
int launch_gate_v(const Dims &d, const GateArgs &a, A... args) {
    if (a.v <= 2) return launch_gate<T, 2>(d, a, args...);
    if (a.v <= 4) return launch_gate<T, 4>(d, a, args...);
    if (a.v <= 8) return launch_gate<T, 8>(d, a, args...);
    if (a.v <= 16) return launch_gate<T, 16>(d, a, args...);
    if (a.v <= 32) return launch_gate<T, 32>(d, a, args...);
    return launch_gate<T, 64>(d, a, args...);                          // v <= 61: E <= 1024, G <= 32
}

template <typename T, bool DENSE, int LP, int NV, typename... A>
int launch_backward_one(const Dims &d, cudaStream_t st, A... args) {
    static PerContext<int> resident_cache;
    const int resident = resident_blocks_cached(resident_cache, gate_backward_kernel<T, DENSE, LP, NV>, 256);
    const int grid = persistent_grid(((long long)d.T + 256 / LP - 1) / (256 / LP), resident, d.max_blocks);
    return launch_pdl(gate_backward_kernel<T, DENSE, LP, NV>, grid, 256, st, args...) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T, bool DENSE, typename... A>
int launch_backward_rows(const Dims &d, cudaStream_t st, A... args) {
    constexpr int kVec = 16 / (int)sizeof(T);
    const int words = d.E / kVec;
    if (d.E % kVec != 0) {
        static PerContext<int> resident_cache;
        const int resident = resident_blocks_cached(resident_cache, gate_backward_odd_kernel<T, DENSE>, 256);
        const int grid = persistent_grid(((long long)d.T + 7) / 8, resident, d.max_blocks);
        return launch_pdl(gate_backward_odd_kernel<T, DENSE>, grid, 256, st, args...) == cudaSuccess ? MOE_OK
                                                                                                     : MOE_ERR_CUDA;
    }
    if (words <= 8) return launch_backward_one<T, DENSE, 8, 1>(d, st, args...);
    if (words <= 16) return launch_backward_one<T, DENSE, 16, 1>(d, st, args...);
    if (words <= 32) return launch_backward_one<T, DENSE, 16, 2>(d, st, args...);
    if (words <= 64) return launch_backward_one<T, DENSE, 16, 4>(d, st, args...);
    if (words <= 128) return launch_backward_one<T, DENSE, 32, 4>(d, st, args...);
    return launch_backward_one<T, DENSE, 32, 8>(d, st, args...);        // 1024 fp32 logits are 256 words
}

template <typename T>
int launch_backward(const Dims &d, const GateArgs &a, cudaStream_t st, const void *logits, const int32_t *idx,
                    const float *w, const float *dw, void *out) {
    const T *l = static_cast<const T *>(logits);
    T *o = static_cast<T *>(out);
    const float up = ldexpf(1.0f, -std::max(-126, std::min(126, ilogbf(a.scale))));
    const GateScale by = {a.scale, up, 1.0f / (a.scale * up)};
    if (!a.sigmoid && !a.renorm)
        return launch_backward_rows<T, true>(d, st, l, idx, w, dw, o, d.T, d.E, d.k, a.sigmoid, a.renorm, by);
    return launch_backward_rows<T, false>(d, st, l, idx, w, dw, o, d.T, d.E, d.k, a.sigmoid, a.renorm, by);
}

}  // namespace
}  // namespace moe

extern "C" int moe_route_gated(const moe_problem *p, const moe_gate *gate, const void *logits, const float *bias,
                               int32_t *topk_idx, float *topk_w, int32_t *counts, int32_t *offsets, int32_t *slot,
                               int32_t *rank_counts, int32_t *dropped, void *workspace, size_t workspace_bytes,
                               void *stream) {
    using namespace moe;
    Dims d;
    int rc = check_problem(p, &d);
    if (rc != MOE_OK) return rc;
    GateArgs a;
    rc = check_gate(d, gate, &a);
    if (rc != MOE_OK) return rc;
    if (!counts || !offsets || !rank_counts || !dropped || !workspace) return MOE_ERR_INVALID_ARG;
    if (d.T > 0 && (!logits || !topk_idx || !topk_w || !slot)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_route_workspace_bytes(p)) return MOE_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(rank_counts, 4) ||
        !aligned(dropped, 4) || !aligned(bias, 4))
        return MOE_ERR_INVALID_ARG;
    if (d.T > 0 && (!aligned(logits, logits_align(gate, d.E)) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
                    !aligned(slot, 4)))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (d.T == 0)                                                      // the zero counts of an empty batch
        return launch_route_slots_small(d, st, static_cast<const uint8_t *>(workspace), topk_idx, slot, counts,
                                        offsets, rank_counts, dropped);
    if (gate->logits_type == MOE_LOGITS_BF16)
        return launch_gate_v<__nv_bfloat16>(d, a, st, logits, bias, topk_idx, topk_w, counts, offsets, slot,
                                            rank_counts, dropped, workspace);
    return launch_gate_v<float>(d, a, st, logits, bias, topk_idx, topk_w, counts, offsets, slot, rank_counts, dropped,
                                workspace);
}

extern "C" int moe_route_gated_backward(const moe_problem *p, const moe_gate *gate, const void *logits,
                                        const int32_t *topk_idx, const float *topk_w, const float *d_topk_w,
                                        void *d_logits, void *stream) {
    using namespace moe;
    Dims d;
    int rc = check_problem(p, &d);
    if (rc != MOE_OK) return rc;
    GateArgs a;
    rc = check_gate(d, gate, &a);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    if (!topk_idx || !topk_w || !d_topk_w || !d_logits) return MOE_ERR_INVALID_ARG;
    if (!logits && (a.sigmoid || !a.renorm)) return MOE_ERR_INVALID_ARG;
    const size_t al = logits_align(gate, d.E);
    if (!aligned(logits, al) || !aligned(d_logits, al) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        !aligned(d_topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (gate->logits_type == MOE_LOGITS_BF16)
        return launch_backward<__nv_bfloat16>(d, a, st, logits, topk_idx, topk_w, d_topk_w, d_logits);
    return launch_backward<float>(d, a, st, logits, topk_idx, topk_w, d_topk_w, d_logits);
}

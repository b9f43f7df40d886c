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

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr uint32_t kTaken = 0u, kMasked = 1u;
constexpr uint32_t kFirstNumber = 0x007FFFFFu;          // key of -inf, the lowest of all numbers
constexpr float kMaskLogit = -3.38953138925153547590470800371487866880e38f;   // the lowest finite bf16

struct GateArgs {
    int T, E, k, R, C;
    int G, top_g, per, L, v;                            // per = E / G; L lanes of v experts to a group
    int sigmoid, top2, renorm;
    float scale;
};

enum GateTile { kOneTile, kTiles8, kTiles32 };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Four fp32 or eight bf16 logits of one 16-byte word.
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[4]) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack16(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Not masked: above the mask value and not NaN.
__device__ __forceinline__ bool open_logit(float l) { return l > kMaskLogit; }

// 1 / (1 + exp(-l)): expf and the correctly rounded reciprocal, 1 at +inf, 0 once exp(-l) overflows.
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }
// sigmoid(l) exp(-top) for a whole number top <= 0 with l <= top, or l positive and top 0, as exp(l - top) / (1 + exp(l))
// where l is not positive: the factor leaves quotients of a row's sigmoids as they are and keeps them from underflowing
// with their row. l - top is exact wherever its exp is not 0: both are multiples of l's last place, or near each other.
__device__ __forceinline__ float sigmoid_above(float l, float top) {
    return l > 0.0f ? sigmoid(l) : __fdiv_rn(expf(__fsub_rn(l, top)), __fadd_rn(1.0f, expf(l)));
}
// logit_key of a number (no NaN) in three instructions: -0 becomes +0 by adding 0.
__device__ __forceinline__ uint32_t number_key(float f) {
    const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
    return u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
// exp(l - top), 1 where l is the top (also where both are +inf).
__device__ __forceinline__ float exp_below(float l, float top) { return l == top ? 1.0f : expf(__fsub_rn(l, top)); }

// Sum and maximum over LP neighbouring lanes, every lane the same value.
template <int LP>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
    return x;
}
template <int LP>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

// hi + lo += x without loss (Knuth's two-sum): the softmax's denominator comes
// out as the rounded exact sum whatever the order, so that a choice by biased
// softmax scores does not hang on how experts are laid over lanes.
__device__ __forceinline__ void two_sum(float &hi, float &lo, float x) {
    const float s = __fadd_rn(hi, x);
    const float b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
}

// The choice of one token by its warp: lane j < k returns choice j's expert and
// weight, ok = false where it is no pair.
template <typename T, int V>
__device__ __forceinline__ void warp_gate(const T *__restrict__ row, const float *__restrict__ bias, const GateArgs &a,
                                          int lane, int &my_e, float &my_w, bool &ok) {
    const int g = lane / a.L, r = lane - g * a.L;
    const int e0 = g * a.per + r * a.v;                                // first expert of this lane
    int n = g < a.G ? min(a.v, a.per - r * a.v) : 0;                   // and how many it holds
    n = max(n, 0);
    float l[V];
    constexpr int kVec = 16 / (int)sizeof(T);
    if (V % kVec == 0 && n == V && e0 % kVec == 0 && a.E % kVec == 0) {
#pragma unroll
        for (int i = 0; i < V / kVec; ++i) {
            float f[kVec];
            unpack16(__ldg(reinterpret_cast<const uint4 *>(row + e0) + i), f);
#pragma unroll
            for (int q = 0; q < kVec; ++q)
                if (i * kVec + q < V) l[i * kVec + q] = f[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = i < n ? to_f32(row[e0 + i]) : -INFINITY;
    }

    // softmax: the row's largest logit and the sum of exp below it
    float top = 0.0f, sum = 1.0f;
    const bool by_score = bias != nullptr || (a.top2 && a.G > 1);      // scores enter the choice
    if (!a.sigmoid && (by_score || !a.renorm)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (open_logit(l[i])) m = max(m, number_key(l[i]));
        m = __reduce_max_sync(kFull, m);
        top = m == 0 ? 0.0f : key_logit(m);
        float hi = 0.0f, lo = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (open_logit(l[i])) two_sum(hi, lo, exp_below(l[i], top));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h2 = __shfl_xor_sync(kFull, hi, o), l2 = __shfl_xor_sync(kFull, lo, o);
            // the larger first: both lanes of a pair then form the same sum
            const float big = fmaxf(hi, h2), small = fminf(hi, h2);
            float h = big, e = __fadd_rn(lo, l2);
            two_sum(h, e, small);
            hi = h;
            lo = e;
        }
        sum = __fadd_rn(hi, lo);
    }

    uint32_t key[V];
    if (bias != nullptr) {
        float b[V];
        if (V % 4 == 0 && n == V && e0 % 4 == 0 && (reinterpret_cast<uintptr_t>(bias) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(bias + e0) + i);
                b[4 * i] = f.x;
                b[4 * i + 1] = f.y;
                b[4 * i + 2] = f.z;
                b[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) b[i] = i < n ? __ldg(bias + e0 + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = a.sigmoid ? sigmoid(l[i]) : __fdiv_rn(exp_below(l[i], top), sum);
            const bool open = open_logit(l[i]) && b[i] > -INFINITY;
            key[i] = i >= n ? kTaken : open ? number_key(__fadd_rn(s, b[i])) : kMasked;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            key[i] = i >= n ? kTaken : open_logit(l[i]) ? number_key(l[i]) : kMasked;
    }

    // Lanes of up to 8 experts sort theirs once, largest first, ties by index: a round of the choice then looks at
    // the first key alone. `order` holds the sorted experts' places within the lane, 4 bits each.
    uint32_t order = 0;
    if constexpr (V <= 8) {
        uint32_t id[V];
#pragma unroll
        for (int i = 0; i < V; ++i) id[i] = i;
        const auto swap = [&](int x, int y) {                          // x < y: the larger to x
            const bool s = key[y] > key[x] || (key[y] == key[x] && id[y] < id[x]);
            const uint32_t kx = key[x], ix = id[x];
            key[x] = s ? key[y] : kx;
            key[y] = s ? kx : key[y];
            id[x] = s ? id[y] : ix;
            id[y] = s ? ix : id[y];
        };
        if constexpr (V == 2) swap(0, 1);
        if constexpr (V >= 4) {                                        // Batcher's odd-even merge
#pragma unroll
            for (int h = 0; h < V; h += 4) {
                swap(h, h + 1);
                swap(h + 2, h + 3);
                swap(h, h + 2);
                swap(h + 1, h + 3);
                swap(h + 1, h + 2);
            }
        }
        if constexpr (V == 8) {
            swap(0, 4);
            swap(1, 5);
            swap(2, 6);
            swap(3, 7);
            swap(2, 4);
            swap(3, 5);
            swap(1, 2);
            swap(3, 4);
            swap(5, 6);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) order |= id[i] << (4 * i);
    }

    if (a.G > 1) {
        // this lane's two best keys, then its group's by a turn around the group's lanes
        uint32_t k1 = 0, k2 = 0;
        if constexpr (V <= 8) {
            k1 = key[0];
            k2 = key[1];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
        }
        const uint32_t own1 = k1, own2 = k2;
        const int base = lane - r;
        for (int o = 1; o < a.L; ++o) {
            int src = r + o;
            src = base + (src >= a.L ? src - a.L : src);
            const uint32_t o1 = __shfl_sync(kFull, own1, src & 31), o2 = __shfl_sync(kFull, own2, src & 31);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        }
        uint32_t gk = k1;
        if (a.top2) {
            float s1 = key_logit(k1), s2 = key_logit(k2);
            if (bias == nullptr) {
                s1 = a.sigmoid ? sigmoid(s1) : exp_below(s1, top);
                s2 = a.sigmoid ? sigmoid(s2) : exp_below(s2, top);
            }
            gk = k2 >= kFirstNumber ? logit_key(__fadd_rn(s1, s2)) : kFirstNumber;
        }
        int better = 0;
#pragma unroll 4
        for (int o = 0; o < a.G; ++o) {
            const uint32_t ok_ = __shfl_sync(kFull, gk, o * a.L);
            better += ok_ > gk || (ok_ == gk && o < g);
        }
        if (better >= a.top_g) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = min(key[i], kMasked);
        }
    }

    uint32_t my_key = 0;
    my_e = 0;
    if constexpr (V <= 8) {
        for (int j = 0; j < a.k; ++j) {
            const uint32_t m = __reduce_max_sync(kFull, key[0]);       // >= kMasked: k <= E
            const int wl = __ffs(__ballot_sync(kFull, key[0] == m)) - 1;
            const int e = __shfl_sync(kFull, e0 + (int)(order & 15u), wl);
            if (lane == wl) {
#pragma unroll
                for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
                key[V - 1] = kTaken;
                order >>= 4;
            }
            if (lane == j) {
                my_key = m;
                my_e = e;
            }
        }
    } else {
        // A lane's best remaining key changes only when the lane wins, and which of its experts has it is looked
        // for by the winner alone: the lowest of its tied ones, in the lowest tied lane.
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i]);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t m = __reduce_max_sync(kFull, best);
            const int wl = __ffs(__ballot_sync(kFull, best == m)) - 1;
            int bi = 0;
            if (lane == wl) {
                best = 0;
                bool found = false;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool hit = !found && key[i] == m;
                    if (hit) {
                        bi = i;
                        key[i] = kTaken;
                    }
                    found |= hit;
                    best = max(best, key[i]);
                }
            }
            const int e = __shfl_sync(kFull, e0 + bi, wl);
            if (lane == j) {
                my_key = m;
                my_e = e;
            }
        }
    }

    ok = lane < a.k && my_key > kMasked;
    const float f = ok ? to_f32(row[my_e]) : 0.0f;
    float s = 0.0f;
    if (a.renorm) {
        const uint32_t m = __reduce_max_sync(kFull, ok ? logit_key(f) : 0u);
        const float most = key_logit(m);                               // the largest chosen logit
        if (ok) s = a.sigmoid ? sigmoid_above(f, ceilf(fminf(most, 0.0f))) : exp_below(f, most);
        const float total = lanes_sum<32>(s);                             // 0 only where nothing was chosen
        s = ok ? __fdiv_rn(s, total) : 0.0f;
    } else if (ok) {
        s = a.sigmoid ? sigmoid(f) : __fdiv_rn(exp_below(f, top), sum);
    }
    my_w = __fmul_rn(s, a.scale);
}

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

int check_gate(const Dims &d, const moe_gate *g, GateArgs *a) {
    if (g == nullptr) return MOE_ERR_INVALID_ARG;
    if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (g->group_rule != MOE_GROUP_MAX && g->group_rule != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
    if (g->logits_type != MOE_LOGITS_F32 && g->logits_type != MOE_LOGITS_BF16) return MOE_ERR_INVALID_ARG;
    if (g->num_groups < 1 || d.E % g->num_groups != 0) return MOE_ERR_INVALID_ARG;
    if (g->top_groups < 1 || g->top_groups > g->num_groups) return MOE_ERR_INVALID_ARG;
    const int per = d.E / g->num_groups;
    if ((long long)g->top_groups * per < d.k) return MOE_ERR_INVALID_ARG;
    if (g->group_rule == MOE_GROUP_TOP2 && g->num_groups > 1 && per < 2) return MOE_ERR_INVALID_ARG;
    if (!(fabsf(g->scale) <= 3.4028234e38f) || g->scale == 0.0f) return MOE_ERR_INVALID_ARG;
    if (g->num_groups > 32) return MOE_ERR_UNSUPPORTED;
    a->T = d.T;
    a->E = d.E;
    a->k = d.k;
    a->R = d.R;
    a->C = d.C;
    a->G = g->num_groups;
    a->top_g = g->top_groups;
    a->per = per;
    a->L = 32 / a->G;
    a->v = (per + a->L - 1) / a->L;
    a->sigmoid = g->score == MOE_SCORE_SIGMOID;
    a->top2 = g->group_rule == MOE_GROUP_TOP2;
    a->renorm = g->renormalise != 0;
    a->scale = g->scale;
    return MOE_OK;
}

size_t logits_align(const moe_gate *g, int E) {
    const size_t size = g->logits_type == MOE_LOGITS_BF16 ? 2 : 4;
    return (size_t)E * size % 16 == 0 ? 16 : size;
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

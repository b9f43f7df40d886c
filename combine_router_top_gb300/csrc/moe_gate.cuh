// moe_gate.cuh -- one token's choice by a warp, and the gate's checks: what the gated
// route (moe_gate.cu) and the layer for a few tokens (moe_few.cu) share.
#pragma once

#include <math.h>

#include "moe_internal.cuh"

namespace moe {

constexpr uint32_t kTaken = 0u, kMasked = 1u;
constexpr uint32_t kFirstNumber = 0x007FFFFFu;          // key of -inf, the lowest of all numbers
constexpr float kMaskLogit = -3.38953138925153547590470800371487866880e38f;   // the lowest finite bf16

struct GateArgs {
    int T, E, k, R, C;
    int G, top_g, per, L, v;                            // per = E / G; L lanes of v experts to a group
    int sigmoid, top2, renorm;
    float scale;
};

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

// ---- host checks --------------------------------------------------------------

inline int check_gate(const Dims &d, const moe_gate *g, GateArgs *a) {
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

inline size_t logits_align(const moe_gate *g, int E) {
    const size_t size = g->logits_type == MOE_LOGITS_BF16 ? 2 : 4;
    return (size_t)E * size % 16 == 0 ? 16 : size;
}

}  // namespace moe

// moe_few.cu -- a whole mixture-of-experts layer for up to 32 tokens: the choice by one block,
// and two kernels for the products; with 8- and 4-bit weights blocks that make the tokens' x fp16
// beside the choice, and a kernel that does so with h between the products.
//
//   up:    h[t][j] = round(silu(x Wg_e^T) (x Wu_e^T)) of every pair (t, j), e its expert
//   down:  out[t] = bf16(sum_j w_j h[t][j] Wd_e^T)
//
// With few tokens every chosen expert's weights are read once for a handful of rows: the
// layer is bound by HBM, then by what it costs to make operands of 8- and 4-bit weights. So
//   - the weights are the 16-row operand of mma.m16n8k16 and up to 8 of an expert's tokens its 8
//     columns (a tcgen05 tile of 128 rows would leave most SMs without work, and its tensor
//     rate is not what is short). In the up kernel 8 of the rows are the gate's and 8 the up's,
//     so that a lane holds both factors of its h;
//   - every warp fetches its own weights, a 5-d TMA box of 16 rows x 256 bytes at a time, laid out
//     so that a fragment's 64 bytes of each row are contiguous, into a ring of its own: no barrier
//     between warps but where several share a tile of rows;
//   - the down kernel's blocks start as the up kernel's end and fill their rings before h is there;
//   - weights of 8 and 4 bits are made fp16 operands, which costs least: an e4m3 pair one conversion (a bf16
//     pair takes five instructions), a 4-bit pair one logic operation, which leaves 1024 + q, or 1024 + 16 q where
//     the code stands 4 bits higher. The inputs of such weights are fp16 too, each row behind a power of two that
//     brings its largest value to 2^14 .. 2^15 and is 2^112 at most: half of fp16's lowest step, 2^-25, is then 2^-39 of the
//     largest value, or 2^-137 where that is below 2^-98. h, kept in fp32 meanwhile, is rounded to fp16's 11 bits.
//     With bf16 weights h is rounded to bf16, since a product's operands are of one type: the output is then 0.0023 of its
//     norm off the value in 64 bits, of which its own rounding makes 0.0017. h in two bf16 parts would mend that for a second
//     product of each; the layer is defined with the one.
//     4-bit weights: inputs whose code stands higher are divided by 16 (their error is 2^-35 of the largest, or 2^-133), and
//     what 1024 (or 64) and the codes' middle, 8, add to a group's sum is taken off it in fp32: sum x (1024 + q) - 1032 sum x.
//
// us on GB300, with the floor of the chosen experts' bytes at the measured copy rate:
//   1 token, 2 of 8 experts of 14336 x 4096, bf16             112    (floor 105)
//   1 token, 8 of 256 of 2048 x 7168 and a shared one, 4-bit   61    (30.5)
//   13 tokens, top-6 of 64 of 1408 x 2048 and shared, e4m3     97    (62.9; 48 experts live and the shared one)
//   32 tokens, top-8 of 256 of 2048 x 7168, e4m3              804    (664; 101 live)
// A call of next to no work (256 experts of 128 x 128) takes 12.5 us with one token, four launches one behind the other;
// 18.6 with 8 tokens and 25.3 with 32. Each by itself, with 1, 8 and 32: the choice 6.5, 6.6 and 10.9, up 5.5, 5.6 and 6.4,
// h's fp16 3.4, down 6.2, 12.6 and 14.1, where eight units each go through all lists. What the slower ones
// spend: 4-bit weights are bound by the instructions that make operands and scale their sums; lists of more than 8 rows by
// those that load the inputs of each 16 of them; the down kernel of 8- and 4-bit weights by a list's sums at nearly every
// piece, and by spills (128 registers; in the up kernel of e4m3 weights, for up to 32 tokens, too).
#include <algorithm>
#include <type_traits>

#include "moe_gate.cuh"
#include "moe_tc.cuh"
#include "moe_w4.cuh"

namespace moe {
namespace {

constexpr int kFewTokens = 32;
constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 16;                       // matrix rows of a unit
constexpr int kFewBlocks = 4;                      // blocks (64 bytes of each row) in a slot of a warp's ring
constexpr int kFewSlot = kFewBlocks * kFewRows * 64;
// For each warp. What the ring leaves of an SM's memory is L1 for the inputs and the scales: 32 tokens, top-6 of 64 experts
// of 1408 x 2048, e4m3, take 116 us with two slots, 146 with three; one token 20.8 and 21.4.
constexpr int kFewSlots = 2;
constexpr int kFewRing = kFewWarps * kFewSlots * kFewSlot;
constexpr int kFewMaxPairs = kFewTokens * kMaxTopK + kFewTokens;       // with the shared expert's
constexpr int kFewMaxLists = kFewTokens * kMaxTopK + 1;                // experts with rows

struct FewArgs {
    GateArgs gate;
    int H, I, E, T, k, shared;
};

// The kernels' kind of weights: moe_weights, the 4-bit ones by their group.
enum FewKind { kBf16, kFp8, kW4G32, kW4G64, kW4G128 };
template <int WT>
constexpr bool kIsW4 = WT >= kW4G32;
template <int WT>
constexpr int kFewGroup = WT == kW4G32 ? 32 : WT == kW4G64 ? 64 : 128;
template <int WT>
constexpr bool kFewHalf = WT != kBf16;             // inputs as fp16

// A block of a row: the 64 bytes that the four lanes of a fragment's row read at once.
template <int WT>
constexpr int kFewBlockInputs = WT == kBf16 ? 32 : WT == kFp8 ? 64 : 128;
// Blocks whose inputs a lane loads together, one such step ahead of the products.
template <int WT>
constexpr int kFewStepBlocks = WT == kBf16 ? 4 : WT == kFp8 ? 2 : 1;

// The experts that have rows, in the order of their first pair, the shared one last; list d holds rows off[d] .. off[d + 1] - 1.
struct alignas(16) FewLists {
    uint16_t expert[kFewMaxLists + 1];
    uint16_t off[kFewMaxLists + 2];
    uint16_t pair[kFewMaxPairs];                   // t (k + shared) + j of a row
    uint8_t token[kFewMaxPairs];
    float weight[kFewMaxPairs];
    int n;
};

// Loads whose addresses are only good where the program order comes to them: volatile, so that none is made earlier.
// OFF: bytes on from the address, within the instruction.
template <int OFF>
__device__ __forceinline__ uint32_t ld_u16(const void *p) {
    uint16_t r;
    asm volatile("ld.global.nc.u16 %0, [%1+%2];" : "=h"(r) : "l"(p), "n"(OFF));
    return r;
}
template <int OFF>
__device__ __forceinline__ uint32_t ld_u32(const void *p) {
    uint32_t r;
    asm volatile("ld.global.nc.u32 %0, [%1+%2];" : "=r"(r) : "l"(p), "n"(OFF));
    return r;
}
template <int OFF>
__device__ __forceinline__ uint2 ld_v2(const void *p) {
    uint2 r;
    asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2+%3];" : "=r"(r.x), "=r"(r.y) : "l"(p), "n"(OFF));
    return r;
}
template <int OFF>
__device__ __forceinline__ float ld_f32(const void *p) {
    float r;
    asm volatile("ld.global.f32 %0, [%1+%2];" : "=f"(r) : "l"(p), "n"(OFF));
    return r;
}
template <int OFF = 0>
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4+%5];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "n"(OFF));
    return r;
}
// f of the numbers 0 .. N - 1 as types.
template <int I, int N, typename F>
__device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<I + 1, N>(f);
    }
}
__device__ __forceinline__ uint4 ld_l2_v4(const void *p) {
    uint4 r;
    asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// Inputs as fp16: the rows, their scales, and with 4-bit weights what each group's sum starts from.
struct FewInputs {
    uint16_t *x;
    float *scale, *less;
};

// Eight values of a row.
__device__ __forceinline__ void load8(const uint16_t *p, float (&f)[8]) {
    const uint4 v = ld_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const uint4 u = ld_v4(p), v = ld_v4(p + 4);
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
// A row of n (a multiple of 128) values as fp16 behind a power of two that brings its largest to 2^14 .. 2^15, and that
// power's inverse; group 32, 64 or 128: as the inputs of 4-bit weights. By a block, all of whose threads come here; rows of up
// to eight values a thread are read once.
template <typename T>
__device__ __forceinline__ void row_to_half(const T *row, int n, int group, const FewInputs &to, size_t at) {
    __shared__ float most[32];
    const int nt = 8 * blockDim.x, first = 8 * threadIdx.x;
    float f[8], m = 0.0f;
    for (int i = first; i < n; i += nt) {
        load8(row + i, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(f[q]));         // NaN stays out
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < (int)blockDim.x >> 5; ++i) m = fmaxf(m, most[i]);
    // the power of two from the exponent's bits; a row with infinities stays as it is. 2^112 at most: a tiny row's sums with large
    // weights stay within fp32, and its scale times a routing weight down to 2^-14 within fp32's normal numbers
    const int e = (int)(__float_as_uint(m) >> 23) - 127;
    const int s = m == 0.0f || e == 128 ? 0 : max(e - 14, -112);
    const float by = __uint_as_float((uint32_t)(127 - s) << 23);
    for (int i0 = 0; i0 < n; i0 += nt) {
        const int i = i0 + first;
        float less = 0.0f;
        if (i < n) {
            if (n > nt) load8(row + i, f);
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float b = group != 0 && (q & 1) ? by * 0.0625f : by;
                const __half2 v = __floats2half2_rn(__fmul_rn(f[2 * q], b), __fmul_rn(f[2 * q + 1], b));
                w[q] = *reinterpret_cast<const uint32_t *>(&v);
                // codes behind 1024 + q (1032 at the middle), or 1024 + 16 q (1152)
                const float2 r = __half22float2(v);
                less -= (q & 1 ? 1152.0f : 1032.0f) * (r.x + r.y);
            }
            st_v4(to.x + at * n + i, make_uint4(w[0], w[1], w[2], w[3]));
        }
        if (group != 0) {                          // 4, 8 or 16 lanes to a group, all of them on the same side of n
            for (int o = 1; o < group / 8; o <<= 1) less += __shfl_xor_sync(kFull, less, o);
            if (i < n && i % group == 0) to.less[at * (n / group) + i / group] = less;
        }
    }
    if (threadIdx.x == 0) to.scale[at] = __uint_as_float((uint32_t)(127 + s) << 23);
}

// h as fp16, a block to a pair. Lets the down kernel start at once. A choice that is no pair has a row too, whatever the
// workspace held, which nothing reads: so this kernel needs no list, and reads nothing before its wait.
__global__ void __launch_bounds__(256)
few_half_kernel(const float *h, int I, int group, FewInputs to) {
    pdl_launch_dependents();
    pdl_wait();
    row_to_half(h + (size_t)blockIdx.x * I, I, group, to, blockIdx.x);
}

// The choice of all tokens, a warp to a token, and the lists: block 0. With weights of 8 or 4 bits the other blocks, one
// to a token, make its x fp16. The up and down kernels' blocks read the lists; the
// down kernel's may do so before the up kernel has ended, which lets others start only once this one has.
template <typename T, int V>
__global__ void __launch_bounds__(V <= 16 ? 1024 : 256)
few_choice_kernel(const __grid_constant__ FewArgs a, const T *__restrict__ logits, const float *__restrict__ bias,
                  int32_t *__restrict__ topk_idx, float *__restrict__ topk_w, FewLists *__restrict__ l,
                  unsigned *__restrict__ there, const uint16_t *x, int group, FewInputs half) {
    __shared__ uint32_t mask[kMaxExperts];         // an expert's tokens
    __shared__ uint16_t off_of[kMaxExperts];       // its first row
    __shared__ int16_t chosen[kFewTokens * kMaxTopK];                  // expert of a pair, -1: no pair
    __shared__ float weight[kFewTokens * kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += blockDim.x) mask[e] = 0u;
    __syncthreads();
    pdl_enter();
    if (blockIdx.x > 0) {
        const int t = blockIdx.x - 1;
        row_to_half(x + (size_t)t * a.H, a.H, group, half, t);
        return;
    }
    for (int i = tid; i < a.H / 16; i += blockDim.x) there[i] = 0u;
    for (int t = warp; t < a.T; t += blockDim.x >> 5) {
        int e;
        float w;
        bool ok;
        warp_gate<T, V>(logits + (size_t)t * a.E, bias, a.gate, lane, e, w, ok);
        if (lane < a.k) {
            chosen[t * a.k + lane] = (int16_t)(ok ? e : -1);
            weight[t * a.k + lane] = w;
            if (ok) atomicOr(&mask[e], 1u << t);
            if (topk_idx) topk_idx[t * a.k + lane] = e;
            if (topk_w) topk_w[t * a.k + lane] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {                               // a list for the pair of each expert's first token
        int n = 0, rows = 0;
        for (int i0 = 0; i0 < a.T * a.k; i0 += 32) {
            const int i = i0 + lane;
            const int e = i < a.T * a.k ? chosen[i] : -1;
            const uint32_t m = e >= 0 ? mask[e] : 0u;
            const bool first = e >= 0 && (m & ((1u << (i / a.k)) - 1u)) == 0u;
            const unsigned all = __ballot_sync(kFull, first);
            int incl = first ? __popc(m) : 0;
            const int own = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            if (first) {
                const int d = n + __popc(all & ((1u << lane) - 1u));
                l->expert[d] = (uint16_t)e;
                l->off[d] = (uint16_t)(rows + incl - own);
                off_of[e] = (uint16_t)(rows + incl - own);
            }
            n += __popc(all);
            rows += __shfl_sync(kFull, incl, 31);
        }
        if (a.shared) {
            if (lane < a.T) {
                l->pair[rows + lane] = (uint16_t)(lane * (a.k + 1) + a.k);
                l->token[rows + lane] = (uint8_t)lane;
                l->weight[rows + lane] = 1.0f;
            }
            if (lane == 0) {
                l->expert[n] = (uint16_t)a.E;
                l->off[n] = (uint16_t)rows;
            }
            ++n;
            rows += a.T;
        }
        if (lane == 0) {
            l->off[n] = (uint16_t)rows;
            l->n = n;
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * a.k; i += blockDim.x) {
        const int e = chosen[i];
        if (e < 0) continue;
        const int t = i / a.k;
        const int r = off_of[e] + __popc(mask[e] & ((1u << t) - 1u));
        l->pair[r] = (uint16_t)(t * (a.k + a.shared) + (i - t * a.k));
        l->token[r] = (uint8_t)t;
        l->weight[r] = weight[i];
    }
}

// The pieces of one warp's work, in order. A unit is 16 matrix rows: up, 8 of the gate's and 8 of the up's of a list's
// expert; down, 16 of each list's expert in turn. A unit belongs to a team of `team` warps, which take its pieces in
// turn; down, where the units are few, to 2^split teams of different blocks, and counts as so many units.
struct FewPlan {
    int units, lists, pieces, per, all, first, team, step, split, stride;
};
template <bool DOWN>
struct FewWalk {
    int unit, q, d, c;                             // q: piece of the unit; d: its list, c: its place in the rows
    __device__ __forceinline__ void start(const FewPlan &p) {
        q = c = p.first + (DOWN ? p.team * (unit & ((1 << p.split) - 1)) : 0);
        d = DOWN ? 0 : unit / p.per;
        if (DOWN) wrap(p);
    }
    __device__ __forceinline__ bool wrap(const FewPlan &p) {
        if (c < p.pieces) return false;
        do {
            c -= p.pieces;
            ++d;
        } while (c >= p.pieces);
        return true;
    }
    __device__ __forceinline__ int row(const FewPlan &p) const { return DOWN ? unit >> p.split : unit - d * p.per; }
};

// What a step needs from global memory besides the weights: 8 columns' inputs, the scales of the fragment's rows g
// and g + 8, and with 4-bit weights what each group's sum starts from in the lane's columns 2 t and 2 t + 1.
template <int WT>
struct FewOperand {
    uint4 x[4];
    uint2 sa, sb;
    float less[kIsW4<WT> ? 128 / kFewGroup<WT> : 1][2];
};

// A box of the weights: x within a block of 64 bytes (0), row, gate or up, block, expert.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int row, int block, int expert) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(block), "r"(expert)
        : "memory");
}

// A packed word's 8 codes as four pairs of fp16, pair (2i, 2i + 1) to r[i]: 1024 + q, and for odd i 1024 + 16 q.
__device__ __forceinline__ void w4_raw_pairs(uint32_t word, uint32_t (&r)[4]) {
    const uint32_t up = word >> 8;
    r[0] = (word & 0x000F000Fu) | 0x64006400u;
    r[1] = (word & 0x00F000F0u) | 0x64006400u;
    r[2] = (up & 0x000F000Fu) | 0x64006400u;
    r[3] = (up & 0x00F000F0u) | 0x64006400u;
}
__device__ __forceinline__ void add_scaled(float (&c)[4], const float (&part)[4], float sa, float sb) {
    c[0] = fmaf(part[0], sa, c[0]);
    c[1] = fmaf(part[1], sa, c[1]);
    c[2] = fmaf(part[2], sb, c[2]);
    c[3] = fmaf(part[3], sb, c[3]);
}

// A step's products: the blocks at pa (rows g; rows g + 8 are 512 bytes on) with the inputs of NT times 8 columns, the
// weights made operands once for all.
template <int WT, int NT>
__device__ __forceinline__ void few_step(float (*c)[4], const FewOperand<WT> (&o)[NT], const uint8_t *pa, int blocks) {
    if constexpr (WT == kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= blocks) break;
            const uint4 va = *reinterpret_cast<const uint4 *>(pa + 1024 * i), vb = *reinterpret_cast<const uint4 *>(pa + 1024 * i + 512);
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                mma16816<false>(c[m], va.x, vb.x, va.y, vb.y, o[m].x[i].x, o[m].x[i].y);
                mma16816<false>(c[m], va.z, vb.z, va.w, vb.w, o[m].x[i].z, o[m].x[i].w);
            }
        }
    } else if constexpr (WT == kFp8) {
        float part[NT][4];
#pragma unroll
        for (int m = 0; m < NT; ++m) part[m][0] = part[m][1] = part[m][2] = part[m][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 va = *reinterpret_cast<const uint4 *>(pa + 1024 * i), vb = *reinterpret_cast<const uint4 *>(pa + 1024 * i + 512);
            const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t a0 = e4m3x2_to_f16x2(wa[q]), a1 = e4m3x2_to_f16x2(wb[q]);
                const uint32_t a2 = e4m3x2_to_f16x2(wa[q] >> 16), a3 = e4m3x2_to_f16x2(wb[q] >> 16);
#pragma unroll
                for (int m = 0; m < NT; ++m) {
                    const uint4 b = o[m].x[2 * i + q / 2];
                    mma16816<true>(part[m], a0, a1, a2, a3, q % 2 ? b.z : b.x, q % 2 ? b.w : b.y);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) add_scaled(c[m], part[m], __uint_as_float(o[0].sa.x), __uint_as_float(o[0].sb.x));
    } else {
        const uint4 va = *reinterpret_cast<const uint4 *>(pa), vb = *reinterpret_cast<const uint4 *>(pa + 512);
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        constexpr int kPer = kFewGroup<WT> / 32;                       // blocks of 32 inputs to a group
        float part[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t ra[4], rb[4];
            w4_raw_pairs(wa[j], ra);
            w4_raw_pairs(wb[j], rb);
            const uint32_t sa = j / kPer < 2 ? o[0].sa.x : o[0].sa.y, sb = j / kPer < 2 ? o[0].sb.x : o[0].sb.y;
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                if (j % kPer == 0) {               // from what the group's sum is too large by
                    part[m][0] = part[m][2] = o[m].less[j / kPer][0];
                    part[m][1] = part[m][3] = o[m].less[j / kPer][1];
                }
                mma16816<true>(part[m], ra[0], rb[0], ra[1], rb[1], o[m].x[j].x, o[m].x[j].y);
                mma16816<true>(part[m], ra[2], rb[2], ra[3], rb[3], o[m].x[j].z, o[m].x[j].w);
                if (j % kPer == kPer - 1) {
                    if (j / kPer % 2 == 0) add_scaled(c[m], part[m], bf16_lo(sa), bf16_lo(sb));
                    else add_scaled(c[m], part[m], bf16_hi(sa), bf16_hi(sb));
                }
            }
        }
    }
}

// down, a unit split between several blocks: their sums [unit][2^split][T][16], and how many of them are there.
struct FewParts {
    float *sums;
    unsigned *there;
};

// x: up, the tokens' inputs; down, the pairs' h; where they are fp16 with their rows' scales. h: what the up kernel writes,
// fp32 where it is made fp16 after, else bf16.
// NTM times 8 columns at most: one for up to 8 tokens, whose registers are few and whose code has no loop over columns. 8 tokens,
// top-6 of 64 experts of 1408 x 2048, e4m3: 64.8 us, with four 67.8; 4-bit, 53.4 and 55.8.
template <int WT, bool DOWN, int NTM>
__global__ void __launch_bounds__(kFewThreads, 2)
few_kernel(const __grid_constant__ CUtensorMap map, FewArgs a, int team, int split, const FewLists *made, FewInputs in,
           const void *__restrict__ w_scale, void *h, uint16_t *__restrict__ out, FewParts parts, unsigned *status) {
    extern __shared__ __align__(128) uint8_t few_smem[];
    __shared__ __align__(8) uint64_t full[kFewWarps][kFewSlots];
    __shared__ FewLists lists;
    __shared__ float4 red[DOWN ? 1 : kFewWarps][32];
    __shared__ float token_scale[kFewTokens];
    __shared__ bool last_here;
    // down: each warp's share of its unit's outputs, [warp][token][16]
    float *acc_out = reinterpret_cast<float *>(few_smem + kFewRing);
    constexpr int kBlockIn = kFewBlockInputs<WT>, kPieceIn = kBlockIn * kFewBlocks;
    constexpr int kGroup = kFewGroup<WT>, kStep = kFewStepBlocks<WT>, kSteps = kFewBlocks / kStep;
    // bytes of a row's scales in a piece
    constexpr int kScaleBytes = WT == kFp8 ? kPieceIn / 128 * 4 : kPieceIn / kGroup * 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int K = DOWN ? a.I : a.H, M = DOWN ? a.H : 2 * a.I;
    if (lane < kFewSlots) {
        mbar_init(&full[warp][lane], 1u);
        fence_mbar_init();
    }
    if constexpr (!DOWN) {
        pdl_wait();
        pdl_launch_dependents();
        if (kFewHalf<WT> && tid < a.T) token_scale[tid] = in.scale[tid];
    }
    // down: before its wait. The choice's kernel has ended and flushed them by then: the up kernel lets the next one start only
    // behind its own wait for that, and all loads of them are from L2, so that no earlier call's are found in an L1.
    for (int i = tid; i < (int)(sizeof(FewLists) / 16); i += kFewThreads)
        reinterpret_cast<uint4 *>(&lists)[i] = ld_l2_v4(reinterpret_cast<const uint4 *>(made) + i);
    __syncthreads();

    FewPlan plan;
    plan.lists = lists.n;
    plan.pieces = (K + kPieceIn - 1) / kPieceIn;
    plan.per = DOWN ? a.H / 16 : a.I / 8;
    plan.units = DOWN ? (plan.lists > 0 ? plan.per << split : 0) : plan.per * plan.lists;
    plan.all = DOWN ? plan.lists * plan.pieces : plan.pieces;
    plan.team = team;
    plan.first = warp & (team - 1);
    plan.split = split;
    plan.step = team << split;
    plan.stride = gridDim.x * (kFewWarps / team);
    const int tail = (K - (plan.pieces - 1) * kPieceIn) / kBlockIn;    // blocks of a row's last piece
    const unsigned scale_row = (unsigned)(K / kGroup) * 2u;
    // from the unit's row 0 to its row 8
    const unsigned row8 = DOWN ? 8u : (unsigned)a.I;

    // Fetching: lane 0 asks for the box; with 4-bit weights lane r < 16 for row r's scales, as far as L2.
    FewWalk<DOWN> fw;
    fw.unit = blockIdx.x + gridDim.x * (warp / team);
    int expert = 0, row0 = 0;
    const uint8_t *from = static_cast<const uint8_t *>(w_scale);
    const auto aim = [&]() {                       // for the walk's list and place, or the next unit's that has one for us
        while (fw.q >= plan.all && fw.unit < plan.units) {
            fw.unit += plan.stride;
            fw.start(plan);
        }
        if (fw.unit >= plan.units) return;
        expert = lists.expert[fw.d];
        row0 = fw.row(plan) * (DOWN ? 16 : 8);
        if (kIsW4<WT>)
            from = static_cast<const uint8_t *>(w_scale) +
                   ((size_t)expert * M + row0 + (lane & 7) + (lane & 8 ? row8 : 0u)) * scale_row + (size_t)fw.c * kScaleBytes;
    };
    fw.start(plan);
    aim();
    unsigned fetched = 0;
    const auto fetch = [&](unsigned s) {
        if (fw.unit >= plan.units) return;
        if (lane == 0) {
            mbar_expect_tx(&full[warp][s], kFewSlot);              // blocks past the row's end count, as zeros
            tma_load_5d(few_smem + (warp * kFewSlots + s) * kFewSlot, &map, &full[warp][s], row0, fw.c * kFewBlocks, expert);
        }
        if (kIsW4<WT> && lane < 16) asm volatile("prefetch.global.L2 [%0];" ::"l"(from));
        ++fetched;
        fw.q += plan.step;
        fw.c += plan.step;
        if (fw.q >= plan.all || (DOWN && fw.wrap(plan))) {
            aim();
        } else if (kIsW4<WT>) {
            from += plan.step * kScaleBytes;
        }
    };
#pragma unroll
    for (int i = 0; i < kFewSlots; ++i) fetch(i);

    if constexpr (DOWN) {
        for (int i = lane; i < a.T * 16; i += 32) acc_out[warp * a.T * 16 + i] = 0.0f;
        pdl_wait();                                // h is there
        pdl_launch_dependents();
        if (kFewHalf<WT>) {
            for (int i = tid; i < lists.off[lists.n]; i += kFewThreads) lists.weight[i] *= in.scale[lists.pair[i]];
            __syncthreads();
        }
        __syncwarp();
    }
    const int first_warp = warp & ~(team - 1);
    const auto team_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + first_warp), "r"(team * 32) : "memory"); };
    float acc[NTM][4];
#pragma unroll
    for (int i = 0; i < NTM; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    unsigned n = 0, lost = 0, slot = 0, parity = 0;
    bool alive = true;
    int first = 0, rows = 0;
    // down: the list's rows into this warp's sums of their tokens
    const auto fold = [&]() {
        float *mine = acc_out + warp * a.T * 16;
#pragma unroll
        for (int nt = 0; nt < NTM; ++nt) {
            if (8 * nt >= rows) break;
            const int r = 8 * nt + 2 * t;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (r + q < rows) {
                    const float by = lists.weight[first + r + q];
                    float *to = mine + lists.token[first + r + q] * 16 + g;
                    to[0] = fmaf(acc[nt][q], by, to[0]);
                    to[8] = fmaf(acc[nt][2 + q], by, to[8]);
                }
            }
            acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        }
    };
    // A row of the inputs, that of row r of the list; rows past the list's last are the last one again: their columns are
    // not stored.
    const auto input_row = [&](int r) {
        r = first + min(r, rows - 1);
        return DOWN ? (int)lists.pair[r] : (int)lists.token[r];
    };

    // Where a lane reads at a piece: its inputs of its column of the list's first eight, the starts of its two columns' sums,
    // its rows' scales.
    struct Place {
        const uint16_t *x;
        const float *l0, *l1;
        const uint8_t *sa, *sb;
    };
    FewWalk<DOWN> walk;
    for (walk.unit = blockIdx.x + gridDim.x * (warp / team); walk.unit < plan.units; walk.unit += plan.stride) {
        walk.start(plan);
        const auto place = [&](Place &p) {         // for the walk's list and piece
            first = lists.off[walk.d];
            rows = lists.off[walk.d + 1] - first;
            const size_t e = lists.expert[walk.d];
            if constexpr (WT == kFp8) {
                const int ma = walk.row(plan) * (DOWN ? 16 : 8), mb = DOWN ? ma : a.I + ma;
                const uint8_t *sc = static_cast<const uint8_t *>(w_scale) + 4 * (e * (M / 128) * (K / 128)) + walk.c * kScaleBytes;
                p.sa = sc + 4 * (size_t)((ma / 128) * (K / 128));
                p.sb = sc + 4 * (size_t)((mb / 128) * (K / 128));
            }
            if constexpr (kIsW4<WT>) {
                p.sa = static_cast<const uint8_t *>(w_scale) + (e * M + walk.row(plan) * (DOWN ? 16 : 8) + g) * scale_row +
                       walk.c * kScaleBytes;
                p.sb = p.sa + (size_t)row8 * scale_row;
            }
        };
        const auto columns = [&](Place &p, int nt) {                   // and for the list's rows 8 nt and on
            p.x = in.x + (size_t)input_row(8 * nt + g) * K + walk.c * kPieceIn + (WT == kFp8 ? 16 : 8) * t;
            if constexpr (kIsW4<WT>) {
                p.l0 = in.less + (size_t)input_row(8 * nt + 2 * t) * (K / kGroup) + walk.c * (kPieceIn / kGroup);
                p.l1 = in.less + (size_t)input_row(8 * nt + 2 * t + 1) * (K / kGroup) + walk.c * (kPieceIn / kGroup);
            }
        };
        // step `number` of a piece that has `blocks` blocks
        const auto load = [&](FewOperand<WT> &to, const Place &p, auto number, int blocks, bool scales) {
            constexpr int step = decltype(number)::value, at = step * kStep * kBlockIn * 2;
            if constexpr (WT == kBf16) {
                to.x[0] = ld_v4<at>(p.x);          // a row's length is a multiple of two blocks
                to.x[1] = ld_v4<at + 64>(p.x);
                if (blocks > 2) {
                    to.x[2] = ld_v4<at + 128>(p.x);
                    to.x[3] = ld_v4<at + 192>(p.x);
                }
            } else if constexpr (WT == kFp8) {
                to.x[0] = ld_v4<at>(p.x);
                to.x[1] = ld_v4<at + 16>(p.x);
                to.x[2] = ld_v4<at + 128>(p.x);
                to.x[3] = ld_v4<at + 144>(p.x);
            } else {
                to.x[0] = ld_v4<at>(p.x);
                to.x[1] = ld_v4<at + 64>(p.x);
                to.x[2] = ld_v4<at + 128>(p.x);
                to.x[3] = ld_v4<at + 192>(p.x);
                each<0, 128 / kGroup>([&](auto i) {
                    constexpr int off = 4 * (step * (128 / kGroup) + decltype(i)::value);
                    to.less[decltype(i)::value][0] = ld_f32<off>(p.l0);
                    to.less[decltype(i)::value][1] = ld_f32<off>(p.l1);
                });
            }
            if (!scales) return;
            if constexpr (WT == kFp8 || WT == kW4G64) {
                to.sa.x = ld_u32<4 * step>(p.sa);
                to.sb.x = ld_u32<4 * step>(p.sb);
            } else if constexpr (WT == kW4G128) {
                to.sa.x = ld_u16<2 * step>(p.sa);
                to.sb.x = ld_u16<2 * step>(p.sb);
            } else if constexpr (WT == kW4G32) {
                to.sa = ld_v2<8 * step>(p.sa);
                to.sb = ld_v2<8 * step>(p.sb);
            }
        };
        constexpr std::integral_constant<int, 0> kFirst{};
        Place at;
        FewOperand<WT> o[1];
        const auto blocks_of = [&](int c) { return c == plan.pieces - 1 ? tail : kFewBlocks; };
        if (walk.q < plan.all) {
            place(at);
            columns(at, 0);
            load(o[0], at, kFirst, blocks_of(walk.c), true);
        }
        while (walk.q < plan.all) {
            const int blocks = blocks_of(walk.c);
            if (alive && !__all_sync(kFull, mbar_try_wait(smem_u32(&full[warp][slot]), parity)) &&
                !__all_sync(kFull, mbar_wait_bounded(&full[warp][slot], parity))) {
                alive = false;                     // outputs stay wrong; the barriers below still meet
                lost = n;
                if (lane == 0) atomicOr(status, kStatusWaitGaveUp);
            }
            const uint8_t *pa = few_smem + (warp * kFewSlots + slot) * kFewSlot + 16 * lane;       // row g, 16 t bytes in
            if ((NTM == 1 || rows <= 8) && blocks == kFewBlocks) {                   // most pieces: steps and offsets known
                each<0, kSteps>([&](auto number) {
                    constexpr int step = decltype(number)::value;
                    FewOperand<WT> next;
                    if constexpr (step + 1 < kSteps) load(next, at, std::integral_constant<int, step + 1>{}, kFewBlocks, true);
                    few_step<WT, 1>(acc, o, pa + 1024 * kStep * step, kStep);
                    if constexpr (step + 1 < kSteps) o[0] = next;
                });
            } else {
                // 16 rows of the list at a time, for which the weights are made operands once; the tails of few rows
#pragma unroll
                for (int nt = 0; nt < NTM; nt += 2) {
                    if (8 * nt >= rows) break;     // warp-uniform
                    const bool pair = NTM > 1 && rows > 8 * (nt + 1);
                    Place p0 = at, p1 = at;
                    columns(p0, nt);
                    if (pair) columns(p1, nt + 1);
#pragma unroll 1
                    for (int b = 0; b < blocks; b += kStep) {
                        load(o[0], p0, kFirst, blocks - b, true);
                        if (NTM > 1 && pair) {
                            FewOperand<WT> two[2];
                            two[0] = o[0];
                            load(two[1], p1, kFirst, blocks - b, false);
                            few_step<WT, 2>(acc + nt, two, pa + 1024 * b, blocks - b);
                        } else {
                            few_step<WT, 1>(acc + nt, o, pa + 1024 * b, blocks - b);
                        }
                        p0.x += kStep * kBlockIn;
                        p1.x += kStep * kBlockIn;
                        p0.sa += kScaleBytes / kSteps;
                        p0.sb += kScaleBytes / kSteps;
                        if (kIsW4<WT>) {
                            p0.l0 += 128 / kGroup;
                            p0.l1 += 128 / kGroup;
                            p1.l0 += 128 / kGroup;
                            p1.l1 += 128 / kGroup;
                        }
                    }
                }
            }
            // on to the next piece, whose first step's operands come while this warp frees the slot and waits
            walk.q += plan.step;
            walk.c += plan.step;
            const bool other = DOWN && walk.wrap(plan);
            if (DOWN && (other || walk.q >= plan.all)) fold();
            if (walk.q < plan.all) {
                if (other) {
                    place(at);
                    columns(at, 0);
                } else {
                    at.x += plan.step * kPieceIn;
                    at.sa += plan.step * kScaleBytes;
                    at.sb += plan.step * kScaleBytes;
                    if (kIsW4<WT>) {
                        at.l0 += plan.step * (kPieceIn / kGroup);
                        at.l1 += plan.step * (kPieceIn / kGroup);
                    }
                }
                load(o[0], at, kFirst, blocks_of(walk.c), true);
            }
            ++n;
            __syncwarp();                          // every lane has read the slot
            if (alive) fetch(slot);
            if (++slot == kFewSlots) {
                slot = 0;
                parity ^= 1u;
            }
        }

        if constexpr (!DOWN) {
            // h from the sums of the unit's list, joined over the team's warps
            walk.start(plan);
            first = lists.off[walk.d];
            rows = lists.off[walk.d + 1] - first;
#pragma unroll
            for (int nt = 0; nt < NTM; ++nt) {
                if (8 * nt >= rows) break;
                float4 v = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
                acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
                if (team > 1) {
                    red[warp][lane] = v;
                    team_sync();
                    if (warp == first_warp) {
                        for (int i = 1; i < team; ++i) {
                            const float4 u = red[warp + i][lane];
                            v.x += u.x;
                            v.y += u.y;
                            v.z += u.z;
                            v.w += u.w;
                        }
                    }
                    team_sync();
                    if (warp != first_warp) continue;
                }
                const int r = first + 8 * nt + 2 * t, o = walk.row(plan) * 8 + g;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (r + q >= first + rows) break;
                    const float by = kFewHalf<WT> ? token_scale[lists.token[r + q]] : 1.0f;
                    const float u = silu((q ? v.y : v.x) * by) * ((q ? v.w : v.z) * by);
                    const size_t to = (size_t)lists.pair[r + q] * a.I + o;
                    if (kFewHalf<WT>) static_cast<float *>(h)[to] = u;
                    else put_bf16(static_cast<uint16_t *>(h) + to, u);
                }
            }
        } else {
            team_sync();
            const float *sums = acc_out + first_warp * a.T * 16;
            const int in_team = (warp - first_warp) * 32 + lane;
            const auto put = [&](int i, float v) { put_bf16(out + (size_t)(i >> 4) * a.H + walk.row(plan) * 16 + (i & 15), v); };
            float *part = parts.sums + (size_t)walk.unit * a.T * 16;
            for (int i = in_team; i < a.T * 16; i += team * 32) {
                float v = 0.0f;
                for (int j = 0; j < team; ++j) v += sums[j * a.T * 16 + i];
                if (split == 0) put(i, v);
                else part[i] = v;
            }
            if (split > 0) {                       // the team is the block; the last one of the unit joins the sums, in order
                __threadfence();
                team_sync();
                const int unit = walk.unit >> split;
                if (tid == 0) last_here = atomicAdd(parts.there + unit, 1u) == (1u << split) - 1u;
                team_sync();
                if (last_here) {
                    __threadfence();
                    part = parts.sums + ((size_t)unit << split) * a.T * 16;
                    for (int i = in_team; i < a.T * 16; i += team * 32) {
                        float v = 0.0f;
                        for (int j = 0; j < 1 << split; ++j) v += __ldcg(part + j * a.T * 16 + i);
                        put(i, v);
                    }
                }
            }
            team_sync();
            for (int i = lane; i < a.T * 16; i += 32) acc_out[warp * a.T * 16 + i] = 0.0f;
            __syncwarp();
        }
    }
    if constexpr (DOWN) {
        if (lists.n == 0)                          // not one pair in the whole batch
            for (int i = blockIdx.x * kFewThreads + tid; i < a.T * a.H; i += gridDim.x * kFewThreads) out[i] = 0;
    }
    // after a wait that gave up: no copy outlives the block
    if (!alive)
        for (; lost < fetched; ++lost) mbar_wait_bounded(&full[warp][lost % kFewSlots], (lost / kFewSlots) & 1u);
}

int check_mlp(const moe_mlp *m) {
    if (m == nullptr) return MOE_ERR_INVALID_ARG;
    if (m->weights < MOE_WEIGHTS_BF16 || m->weights > MOE_WEIGHTS_W4) return MOE_ERR_INVALID_ARG;
    if (m->inner < 1 || m->inner > kMaxHidden) return MOE_ERR_INVALID_ARG;
    if (m->shared != 0 && m->shared != 1) return MOE_ERR_INVALID_ARG;
    if (m->weights == MOE_WEIGHTS_W4 && m->group != 32 && m->group != 64 && m->group != 128) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}
int check_few(const Dims &d, const moe_mlp *m) {
    const int step = m->weights == MOE_WEIGHTS_BF16 ? 64 : 128;
    if (d.T > kFewTokens || d.H % step != 0 || m->inner % step != 0 || d.dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Blocks, and warps to a unit: as many as all units at work at once leave it of the warps of GB300's 152 SMs, two blocks on
// each. By the sizes alone: the grid does not change a sum's order.
int few_team(long long units) {
    int team = 1;
    while (team < kFewWarps && units * team * 2 <= 2LL * 152 * kFewWarps) team *= 2;
    return team;
}
int few_grid(long long units, int max_blocks) { return persistent_grid(units, 2 * sm_count(), max_blocks); }

// Matrices [S][parts][rows][row_bytes] in boxes of `box_rows` rows of each part x kFewBlocks blocks of 64 bytes.
bool encode_few(CUtensorMap *map, const void *base, uint64_t rows, uint64_t parts, uint64_t row_bytes, uint64_t S,
                uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[5] = {64, rows, parts, row_bytes / 64, S};
    const cuuint64_t strides[4] = {row_bytes, rows * row_bytes, 64, parts * rows * row_bytes};
    const cuuint32_t box[5] = {64, box_rows, (cuuint32_t)parts, kFewBlocks, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the workspace holds.
struct FewSpace {
    FewLists *lists;
    FewParts parts;
    void *h;                                       // [T (k + shared)][I]: bf16, or fp32 where h_half follows
    FewInputs x_half, h_half;
    int split;
    size_t bytes;
};
// The binary logarithm of how many blocks share a down unit: where the units are too few for the SMs' warps (2048 outputs
// are 128 units) and leave each of those warps at least four pieces. us with one block to a unit and with two, 2048 outputs
// of 1408 inputs, top-6 of 64 experts: 32 tokens, bf16, 212 and 182; e4m3, 152 and 116; one token, bf16 (8 pieces a warp with
// one), 20.4 and 19.9; e4m3 (5), 20.5 and 20.8; 4-bit (2), 18.8 and 20.3.
int few_split(const Dims &d, const moe_mlp *m) {
    const int piece = kFewBlocks * (m->weights == MOE_WEIGHTS_BF16 ? kFewBlockInputs<kBf16>
                                    : m->weights == MOE_WEIGHTS_W4 ? kFewBlockInputs<kW4G32>
                                                                   : kFewBlockInputs<kFp8>);
    const long long pieces = (std::min<long long>((long long)d.T * d.k, d.E) + m->shared) * ((m->inner + piece - 1) / piece);
    int split = 0;
    while (split < 3 && ((long long)(d.H / 16) * kFewWarps << (split + 1)) <= 2LL * 152 * kFewWarps &&
           pieces >= 4LL * kFewWarps << (split + 1))
        ++split;
    return split;
}
FewSpace few_space(void *base, const Dims &d, const moe_mlp *m) {
    FewSpace s = {};
    uint8_t *at = static_cast<uint8_t *>(base);
    const auto take = [&](size_t bytes) {
        void *p = at + s.bytes;
        s.bytes += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t T = d.T, pairs = T * (d.k + m->shared), I = m->inner;
    const int split = few_split(d, m);
    const bool half = m->weights != MOE_WEIGHTS_BF16, w4 = m->weights == MOE_WEIGHTS_W4;
    const auto inputs = [&](size_t rows, size_t n) {
        FewInputs f;
        f.x = static_cast<uint16_t *>(take(rows * n * 2));
        f.scale = static_cast<float *>(take(rows * 4));
        f.less = static_cast<float *>(take(w4 ? rows * (n / m->group) * 4 : 0));
        return f;
    };
    s.split = split;
    s.lists = static_cast<FewLists *>(take(sizeof(FewLists)));
    s.parts.there = static_cast<unsigned *>(take((size_t)d.H / 16 * sizeof(unsigned)));
    s.parts.sums = static_cast<float *>(take(split > 0 ? ((size_t)d.H << split) * T * sizeof(float) : 0));
    s.h = take(pairs * I * (half ? 4 : 2));
    if (half) {
        s.x_half = inputs(T, d.H);
        s.h_half = inputs(pairs, I);
    }
    return s;
}

template <typename T, int V>
int launch_choice(const FewArgs &a, cudaStream_t st, const void *logits, const float *bias, int32_t *idx, float *w,
                  const void *x, int group, const FewSpace &s) {
    const bool half = s.x_half.x != nullptr;
    const int most = V <= 16 ? 32 : 8;             // warps; at least 8 for the clearing, and 8 values of x to a thread
    const int warps = std::min(most, std::max(std::max(a.T, 8), half ? a.H / 256 : 0));
    return launch_pdl(few_choice_kernel<T, V>, half ? 1 + a.T : 1, warps * 32, st, a, static_cast<const T *>(logits), bias, idx,
                      w, s.lists, s.parts.there, static_cast<const uint16_t *>(x), group, s.x_half) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
template <typename T, typename... A>
int launch_choice_v(const FewArgs &a, A... args) {
    if (a.gate.v <= 2) return launch_choice<T, 2>(a, args...);
    if (a.gate.v <= 4) return launch_choice<T, 4>(a, args...);
    if (a.gate.v <= 8) return launch_choice<T, 8>(a, args...);
    if (a.gate.v <= 16) return launch_choice<T, 16>(a, args...);
    if (a.gate.v <= 32) return launch_choice<T, 32>(a, args...);
    return launch_choice<T, 64>(a, args...);
}

template <int WT, int NTM>
int launch_few(const Dims &d, const FewArgs &a, cudaStream_t st, const void *x, const void *w_up, const void *up_scale,
               const void *w_down, const void *down_scale, void *out, const FewSpace &s, unsigned *status) {
    static PerContext<int> up_done, down_done;
    const size_t most = kFewRing + kFewWarps * kFewTokens * 16 * sizeof(float);
    if (!set_smem_once(up_done, few_kernel<WT, false, NTM>, kFewRing) || !set_smem_once(down_done, few_kernel<WT, true, NTM>, (int)most))
        return MOE_ERR_CUDA;
    CUtensorMap up, down;
    const uint64_t S = a.E + a.shared, block = kFewBlockInputs<WT>;
    if (!encode_few(&up, w_up, a.I, 2, a.H / block * 64, S, 8) || !encode_few(&down, w_down, a.H, 1, a.I / block * 64, S, 16))
        return MOE_ERR_CUDA;
    uint16_t *o = static_cast<uint16_t *>(out);
    constexpr bool half = kFewHalf<WT>;
    constexpr int group = kIsW4<WT> ? kFewGroup<WT> : 0;
    FewInputs up_x = s.x_half, down_x = s.h_half;
    if (!half) {
        up_x.x = static_cast<uint16_t *>(const_cast<void *>(x));
        down_x.x = static_cast<uint16_t *>(s.h);
    }
    long long units = (std::min<long long>((long long)d.T * d.k, d.E) + a.shared) * (a.I / 8);
    if (launch_pdl_smem(few_kernel<WT, false, NTM>, few_grid(units, d.max_blocks), kFewThreads, kFewRing, st, up, a, few_team(units), 0,
                        s.lists, up_x, up_scale, s.h, o, s.parts, status) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (half && launch_pdl(few_half_kernel, d.T * (d.k + a.shared), 256, st, static_cast<const float *>(s.h), a.I, group, s.h_half) !=
                    cudaSuccess)
        return MOE_ERR_CUDA;
    const int split = s.split;
    units = (long long)(d.H / 16) << split;
    if (launch_pdl_smem(few_kernel<WT, true, NTM>, few_grid(units, d.max_blocks), kFewThreads,
                        kFewRing + (size_t)kFewWarps * d.T * 16 * sizeof(float), st, down, a, few_team(units), split, s.lists,
                        down_x, down_scale, s.h, o, s.parts, status) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_layer_few_workspace_bytes(const moe_problem *p, const moe_mlp *mlp) {
    using namespace moe;
    Dims d;
    if (check_problem(p, &d) != MOE_OK || check_mlp(mlp) != MOE_OK || check_few(d, mlp) != MOE_OK) return 0;
    return few_space(nullptr, d, mlp).bytes;
}

extern "C" int moe_layer_few(const moe_problem *p, const moe_gate *gate, const moe_mlp *mlp, const void *x,
                             const void *logits, const float *bias, const void *w_up, const void *up_scale,
                             const void *w_down, const void *down_scale, int32_t *topk_idx, float *topk_w, void *out,
                             void *workspace, size_t workspace_bytes, void *stream) {
    using namespace moe;
    Dims d;
    FewArgs a;
    int rc = check_problem(p, &d);
    if (rc == MOE_OK) rc = check_gate(d, gate, &a.gate);
    if (rc == MOE_OK) rc = check_mlp(mlp);
    if (rc == MOE_OK) rc = check_few(d, mlp);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    const bool scaled = mlp->weights != MOE_WEIGHTS_BF16;
    if (!x || !logits || !w_up || !w_down || !out || !workspace) return MOE_ERR_INVALID_ARG;
    if (scaled != (up_scale != nullptr) || scaled != (down_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_layer_few_workspace_bytes(p, mlp)) return MOE_ERR_INVALID_ARG;
    const size_t scale_align = mlp->weights == MOE_WEIGHTS_W4 ? 16 : 4;
    if (!aligned(x, 16) || !aligned(logits, logits_align(gate, d.E)) || !aligned(bias, 4) || !aligned(w_up, 16) ||
        !aligned(w_down, 16) || !aligned(up_scale, scale_align) || !aligned(down_scale, scale_align) ||
        !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(out, 16) || !aligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    a.H = d.H;
    a.I = mlp->inner;
    a.E = d.E;
    a.T = d.T;
    a.k = d.k;
    a.shared = mlp->shared;
    unsigned *status = device_status_word();
    if (status == nullptr) return MOE_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    const FewSpace s = few_space(workspace, d, mlp);
    const int group = mlp->weights == MOE_WEIGHTS_W4 ? mlp->group : 0;
    rc = gate->logits_type == MOE_LOGITS_BF16 ? launch_choice_v<__nv_bfloat16>(a, st, logits, bias, topk_idx, topk_w, x, group, s)
                                              : launch_choice_v<float>(a, st, logits, bias, topk_idx, topk_w, x, group, s);
    if (rc != MOE_OK) return rc;
    const auto go = [&](auto kind) {
        if (d.T <= 8) return launch_few<decltype(kind)::value, 1>(d, a, st, x, w_up, up_scale, w_down, down_scale, out, s, status);
        return launch_few<decltype(kind)::value, 4>(d, a, st, x, w_up, up_scale, w_down, down_scale, out, s, status);
    };
    if (mlp->weights == MOE_WEIGHTS_BF16) return go(std::integral_constant<int, kBf16>{});
    if (mlp->weights == MOE_WEIGHTS_FP8_B128) return go(std::integral_constant<int, kFp8>{});
    if (mlp->group == 32) return go(std::integral_constant<int, kW4G32>{});
    if (mlp->group == 64) return go(std::integral_constant<int, kW4G64>{});
    return go(std::integral_constant<int, kW4G128>{});
}

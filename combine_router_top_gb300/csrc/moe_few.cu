// moe_few.cu -- a whole mixture-of-experts layer for up to 32 tokens, in two kernels.
//
//   up:    choice; h[t][j] = bf16(silu(x Wg_e^T) (x Wu_e^T)) of every pair (t, j), e its expert
//   down:  choice; out[t] = bf16(sum_j w_j h[t][j] Wd_e^T)
//
// With few tokens every chosen expert's weights are read once for a handful of rows: the
// layer is bound by HBM, then by latency. So
//   - the weights are the 16-row operand of mma.m16n8k16 and up to 8 of an expert's tokens its 8
//     columns (a tcgen05 tile of 128 rows would leave most SMs without work, and its tensor
//     rate is not what is short). In the up kernel 8 of the rows are the gate's and 8 the up's,
//     so that a lane holds both factors of its h;
//   - they come by bulk copies into a ring in shared memory that one warp keeps full, over the
//     end of one tile of rows into the next, and that leaves room for a second block on the SM:
//     the down kernel's blocks start while the up kernel's are at work, choose for themselves
//     (the choice costs a warp about a microsecond a token) and fill their rings before h is there;
//   - every block forms the choice itself, from the logits: no launch and no wait between
//     the router and the products.
#include <algorithm>

#include "moe_gate.cuh"
#include "moe_w4.cuh"

namespace moe {
namespace {

constexpr int kFewTokens = 32;
constexpr int kFewWarps = 8;                       // that multiply; one more fetches
constexpr int kFewThreads = (kFewWarps + 1) * 32;
constexpr int kFewRows = 16;                       // matrix rows of a tile
constexpr int kFewPiece = 1024;                    // bytes of a row in a stage of the ring: 128 for each warp
constexpr int kFewPitch = kFewPiece + 64;          // rows 64 bytes apart in the banks: two rows' 64 bytes meet no twice
constexpr int kFewStage = kFewRows * kFewPitch;
constexpr int kFewStages = 5;
constexpr int kFewMaxPairs = kFewTokens * kMaxTopK + kFewTokens;       // with the shared expert's
constexpr int kFewMaxLists = kFewTokens * kMaxTopK + 1;                // experts with rows

struct FewArgs {
    GateArgs gate;
    int H, I, E, T, k, shared, group, logits_bf16;
};

// Inputs of a row in a warp's 128 bytes, and in one step of its loop.
template <int WT>
constexpr int kFewWarpInputs = WT == MOE_WEIGHTS_BF16 ? 64 : WT == MOE_WEIGHTS_FP8_B128 ? 128 : 256;
template <int WT>
constexpr int kFewStepInputs = WT == MOE_WEIGHTS_BF16 ? 64 : 128;

// The choice by whatever lane width the experts need. Not inlined: one copy of each serves every kernel here.
template <typename T, int V>
__device__ __noinline__ void few_gate_v(const void *logits, const float *bias, const GateArgs *a, int token, int lane,
                                        int *e, float *w, bool *ok) {
    int my_e;
    float my_w;
    bool my_ok;
    warp_gate<T, V>(static_cast<const T *>(logits) + (size_t)token * a->E, bias, *a, lane, my_e, my_w, my_ok);
    *e = my_e;
    *w = my_w;
    *ok = my_ok;
}
template <typename T>
__device__ __forceinline__ void few_gate(const void *logits, const float *bias, const GateArgs *a, int token, int lane,
                                         int *e, float *w, bool *ok) {
    if (a->v <= 2) few_gate_v<T, 2>(logits, bias, a, token, lane, e, w, ok);
    else if (a->v <= 4) few_gate_v<T, 4>(logits, bias, a, token, lane, e, w, ok);
    else if (a->v <= 8) few_gate_v<T, 8>(logits, bias, a, token, lane, e, w, ok);
    else if (a->v <= 16) few_gate_v<T, 16>(logits, bias, a, token, lane, e, w, ok);
    else if (a->v <= 32) few_gate_v<T, 32>(logits, bias, a, token, lane, e, w, ok);
    else few_gate_v<T, 64>(logits, bias, a, token, lane, e, w, ok);
}

// The experts that have rows, in the order of their first pair, the shared one last; list d holds rows off[d] .. off[d + 1] - 1.
struct FewLists {
    uint16_t expert[kFewMaxLists + 1];
    uint16_t off[kFewMaxLists + 2];
    uint16_t pair[kFewMaxPairs];                   // t (k + shared) + j of a row
    uint8_t token[kFewMaxPairs];
    float weight[kFewMaxPairs];
    int n;
    int dead;                                      // a wait gave up
};
// Needed only while the lists are made; lies where the ring is later.
struct FewScratch {
    uint32_t mask[kMaxExperts];                    // the expert's tokens
    uint16_t list_of[kMaxExperts];
    int16_t chosen[kFewTokens * kMaxTopK];         // expert of a pair, -1: no pair
    float w[kFewTokens * kMaxTopK];
};
static_assert(sizeof(FewScratch) <= kFewStages * kFewStage, "the scratch lies within the ring");

__device__ __forceinline__ void few_lists(const FewArgs &a, const void *logits, const float *bias, FewLists &l,
                                          FewScratch &s, int32_t *topk_idx, float *topk_w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += kFewThreads) s.mask[e] = 0u;
    if (tid == 0) l.dead = 0;
    __syncthreads();
    for (int t = warp; t < a.T; t += kFewWarps + 1) {
        int e;
        float w;
        bool ok;
        if (a.logits_bf16) few_gate<__nv_bfloat16>(logits, bias, &a.gate, t, lane, &e, &w, &ok);
        else few_gate<float>(logits, bias, &a.gate, t, lane, &e, &w, &ok);
        if (lane < a.k) {
            s.chosen[t * a.k + lane] = (int16_t)(ok ? e : -1);
            s.w[t * a.k + lane] = w;
            if (ok) atomicOr(&s.mask[e], 1u << t);
            if (topk_idx) topk_idx[t * a.k + lane] = e;
            if (topk_w) topk_w[t * a.k + lane] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {                               // a list for the pair of each expert's first token
        int n = 0, rows = 0;
        for (int i0 = 0; i0 < a.T * a.k; i0 += 32) {
            const int i = i0 + lane;
            const int e = i < a.T * a.k ? s.chosen[i] : -1;
            const uint32_t m = e >= 0 ? s.mask[e] : 0u;
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
                l.expert[d] = (uint16_t)e;
                l.off[d] = (uint16_t)(rows + incl - own);
                s.list_of[e] = (uint16_t)d;
            }
            n += __popc(all);
            rows += __shfl_sync(kFull, incl, 31);
        }
        if (a.shared) {
            if (lane < a.T) {
                l.pair[rows + lane] = (uint16_t)(lane * (a.k + 1) + a.k);
                l.token[rows + lane] = (uint8_t)lane;
                l.weight[rows + lane] = 1.0f;
            }
            if (lane == 0) {
                l.expert[n] = (uint16_t)a.E;
                l.off[n] = (uint16_t)rows;
            }
            ++n;
            rows += a.T;
        }
        if (lane == 0) {
            l.off[n] = (uint16_t)rows;
            l.n = n;
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * a.k; i += kFewThreads) {
        const int e = s.chosen[i];
        if (e < 0) continue;
        const int t = i / a.k;
        const int r = l.off[s.list_of[e]] + __popc(s.mask[e] & ((1u << t) - 1u));
        l.pair[r] = (uint16_t)(t * (a.k + a.shared) + (i - t * a.k));
        l.token[r] = (uint8_t)t;
        l.weight[r] = s.w[i];
    }
    fence_proxy_async_smem();                      // the ring's copies come over the scratch
    __syncthreads();
}

// The stages of a block's work, in order: for its tiles of 16 matrix rows (up: of one list's expert; down: of each list's
// expert in turn), the rows' inputs in pieces.
template <bool DOWN>
struct FewWalk {
    int tile, d, c;                                // up: tile runs over (list, tile of the list's expert)
    int tiles, lists, pieces, per, stride;
    __device__ __forceinline__ FewWalk(int lists_, int per_, int pieces_)
        : d(0), c(0), lists(lists_), pieces(pieces_), per(per_), stride(gridDim.x) {
        tile = blockIdx.x;
        tiles = DOWN ? per : per * lists;
        if (!DOWN) d = tile / per;
    }
    __device__ __forceinline__ bool more() const { return tile < tiles && lists > 0; }
    __device__ __forceinline__ int row() const { return DOWN ? tile : tile - d * per; }      // tile within the matrix
    __device__ __forceinline__ void next() {
        if (++c < pieces) return;
        c = 0;
        if (DOWN) {
            if (++d < lists) return;
            d = 0;
            tile += stride;
        } else {
            tile += stride;
            d = tile / per;
        }
    }
};

// Two bytes of e4m3 at a time -> two bf16: a code's exponent and mantissa bits under a bf16's are its value times
// 2^-120, exactly, subnormals among them.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w, uint32_t pick) {
    const uint32_t b = __byte_perm(w, 0u, pick);   // each code in the upper byte of its half
    const uint32_t v = (b & 0x80008000u) | (b >> 4 & 0x07F007F0u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7B807B80u));
    return r;
}

// What a step needs from global memory besides the weights: 8 columns' inputs and the scales.
template <int WT>
struct FewOperand {
    uint4 x[WT == MOE_WEIGHTS_BF16 ? 2 : 4];
    uint2 sa, sb;                                  // scales of the fragment's rows g and g + 8
};

__device__ __forceinline__ uint4 ld_l2_v4(const void *p) { return __ldcg(static_cast<const uint4 *>(p)); }

template <int WT, bool DOWN>
__global__ void __launch_bounds__(kFewThreads, 2)
few_kernel(const __grid_constant__ FewArgs a, const uint16_t *__restrict__ x, const void *__restrict__ logits, const float *__restrict__ bias,
           const uint8_t *__restrict__ w, const void *__restrict__ w_scale, uint16_t *h, int32_t *__restrict__ topk_idx,
           float *__restrict__ topk_w, uint16_t *__restrict__ out, unsigned *status) {
    extern __shared__ __align__(128) uint8_t few_smem[];
    __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages];
    __shared__ FewLists lists;
    __shared__ float4 red[DOWN ? 1 : 2][DOWN ? 1 : kFewWarps][32];
    uint8_t *ring = few_smem;
    // down: each warp's share of out's tile, [warp][token][16]
    float *acc_out = reinterpret_cast<float *>(few_smem + kFewStages * kFewStage);
    constexpr int kWarpIn = kFewWarpInputs<WT>, kStep = kFewStepInputs<WT>, kPieceIn = kWarpIn * kFewWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    constexpr int kAhead = WT == MOE_WEIGHTS_W4 ? 1 : 2;
    const int K = DOWN ? a.I : a.H, M = DOWN ? a.H : 2 * a.I;
    if (tid < kFewStages) {
        mbar_init(&full[tid], 1u);
        mbar_init(&empty[tid], kFewWarps);
        fence_mbar_init();
    }
    if constexpr (!DOWN) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // The up kernel lets this one start once it has itself waited for all before it: the inputs of the call are there.
    few_lists(a, logits, bias, lists, *reinterpret_cast<FewScratch *>(ring), DOWN || blockIdx.x != 0 ? nullptr : topk_idx,
              DOWN || blockIdx.x != 0 ? nullptr : topk_w);
    const int pieces = (K + kPieceIn - 1) / kPieceIn;
    const size_t row_bytes = WT == MOE_WEIGHTS_BF16 ? 2 * (size_t)K : WT == MOE_WEIGHTS_FP8_B128 ? (size_t)K : (size_t)K / 2;
    FewWalk<DOWN> walk(lists.n, DOWN ? a.H / 16 : a.I / 8, pieces);

    if (warp == kFewWarps) {
        // lane r fetches row r of the tile
        unsigned n = 0;
        bool alive = true;
        for (; walk.more() && alive; walk.next(), ++n) {
            const unsigned s = n % kFewStages;
            if (n >= kFewStages && !mbar_wait_bounded(&empty[s], (n / kFewStages - 1u) & 1u)) {
                alive = false;
                if (lane == 0) atomicOr(status, kStatusWaitGaveUp);
                break;
            }
            const unsigned bytes = (unsigned)min((size_t)kFewPiece, row_bytes - (size_t)walk.c * kFewPiece);
            if (lane == 0) mbar_expect_tx(&full[s], kFewRows * bytes);
            __syncwarp();
            const int r = lane & 15;
            const int m = DOWN ? walk.row() * 16 + r : (r < 8 ? 0 : a.I) + walk.row() * 8 + (r & 7);
            const size_t row = (size_t)lists.expert[walk.d] * M + m;
            if (lane < 16)
                bulk_g2s(ring + s * kFewStage + r * kFewPitch, w + row * row_bytes + (size_t)walk.c * kFewPiece, bytes, &full[s]);
            if (WT == MOE_WEIGHTS_W4 && lane >= 16) {
                const char *p = static_cast<const char *>(w_scale) + 2 * (row * (size_t)(K / a.group) + (size_t)walk.c * (kPieceIn / a.group));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
            }
        }
        // no copy outlives the block
        for (unsigned i = n > kFewStages ? n - kFewStages : 0u; i < n; ++i)
            mbar_wait_bounded(&full[i % kFewStages], (i / kFewStages) & 1u);
        return;
    }

    if constexpr (DOWN) {
        for (int i = tid; i < kFewWarps * a.T * 16; i += kFewWarps * 32) acc_out[i] = 0.0f;
        pdl_wait();                                // h is there
        pdl_launch_dependents();
        asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
    }
    // The steps of the loop, two ahead of the products: a stage's inputs of this warp, for each 8 rows of the list.
    FewWalk<DOWN> at = walk;
    int at_nt = 0, at_h = 0;
    const auto load = [&](FewOperand<WT> &o) {
        // to the next step that has inputs
        int k0 = 0;
        for (; at.more(); at.next()) {
            k0 = at.c * kPieceIn + warp * kWarpIn + at_h * kStep;
            if (k0 < K) break;
        }
        if (!at.more()) return;
        const int first = lists.off[at.d], rows = lists.off[at.d + 1] - first;
        const int r = at_nt * 8 + g;
        constexpr int kVec = WT == MOE_WEIGHTS_BF16 ? 2 : 4;
#pragma unroll
        for (int i = 0; i < kVec; ++i) o.x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
            const uint16_t *p = (DOWN ? h + (size_t)lists.pair[first + r] * K : x + (size_t)lists.token[first + r] * K) + k0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint16_t *q = p + (WT == MOE_WEIGHTS_FP8_B128 ? 64 * (i / 2) + 16 * t + 8 * (i % 2) : 32 * i + 8 * t);
                o.x[i] = DOWN ? ld_l2_v4(q) : __ldg(reinterpret_cast<const uint4 *>(q));
            }
        }
        const size_t e = lists.expert[at.d];
        if constexpr (WT == MOE_WEIGHTS_FP8_B128) {
            const float *sc = static_cast<const float *>(w_scale) + e * (size_t)(M / 128) * (K / 128) + k0 / 128;
            const int ma = DOWN ? at.row() * 16 : at.row() * 8, mb = DOWN ? ma : a.I + ma;
            o.sa.x = __float_as_uint(__ldg(sc + (size_t)(ma / 128) * (K / 128)));
            o.sb.x = __float_as_uint(__ldg(sc + (size_t)(mb / 128) * (K / 128)));
        }
        if constexpr (WT == MOE_WEIGHTS_W4) {
            const int ma = DOWN ? at.row() * 16 + g : at.row() * 8 + g, mb = DOWN ? ma + 8 : a.I + ma;
            const uint16_t *sc = static_cast<const uint16_t *>(w_scale) + k0 / a.group;
            const uint16_t *pa = sc + (e * M + ma) * (size_t)(K / a.group), *pb = sc + (e * M + mb) * (size_t)(K / a.group);
            if (a.group == 128) {
                o.sa.x = __ldg(pa);
                o.sb.x = __ldg(pb);
            } else if (a.group == 64) {
                o.sa.x = __ldg(reinterpret_cast<const uint32_t *>(pa));
                o.sb.x = __ldg(reinterpret_cast<const uint32_t *>(pb));
            } else {
                o.sa = __ldg(reinterpret_cast<const uint2 *>(pa));
                o.sb = __ldg(reinterpret_cast<const uint2 *>(pb));
            }
        }
        // the step after it: the warp's second block of 128, the next 8 rows, the next stage
        if (WT == MOE_WEIGHTS_W4 && at_h == 0 && k0 + kStep < K) {
            at_h = 1;
            return;
        }
        at_h = 0;
        if (8 * ++at_nt < rows) return;
        at_nt = 0;
        at.next();
    };
    FewOperand<WT> o0, o1, o2;
    load(o0);
    if (kAhead == 2) load(o1);

    unsigned n = 0, turn = 0;
    bool alive = true;
    float acc[kFewTokens / 8][4];
#pragma unroll
    for (int i = 0; i < kFewTokens / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    for (; walk.more(); ++n) {
        const unsigned s = n % kFewStages;
        if (alive && !mbar_wait_bounded(&full[s], (n / kFewStages) & 1u)) {
            alive = false;                         // outputs stay wrong; the barriers below still meet
            if (lane == 0) atomicOr(status, kStatusWaitGaveUp);
        }
        const int first = lists.off[walk.d], rows = lists.off[walk.d + 1] - first;
        const uint8_t *base = ring + s * kFewStage + 128 * warp + 16 * t;
        const int kw = walk.c * kPieceIn + warp * kWarpIn;
#pragma unroll
        for (int nt = 0; nt < kFewTokens / 8; ++nt) {
            if (8 * nt >= rows || kw >= K) continue;                   // warp-uniform
            float(&c)[4] = acc[nt];
#pragma unroll
            for (int hh = 0; hh < kWarpIn / kStep; ++hh) {
                if (kw + hh * kStep >= K) continue;
                load(kAhead == 2 ? o2 : o1);
                const uint8_t *pa = base + g * kFewPitch + 64 * hh, *pb = pa + 8 * kFewPitch;
                if constexpr (WT == MOE_WEIGHTS_BF16) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 va = *reinterpret_cast<const uint4 *>(pa + 64 * i);
                        const uint4 vb = *reinterpret_cast<const uint4 *>(pb + 64 * i);
                        mma16816<false>(c, va.x, vb.x, va.y, vb.y, o0.x[i].x, o0.x[i].y);
                        mma16816<false>(c, va.z, vb.z, va.w, vb.w, o0.x[i].z, o0.x[i].w);
                    }
                } else if constexpr (WT == MOE_WEIGHTS_FP8_B128) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 va = *reinterpret_cast<const uint4 *>(pa + 64 * i);
                        const uint4 vb = *reinterpret_cast<const uint4 *>(pb + 64 * i);
                        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint4 b = o0.x[2 * i + q / 2];
                            mma16816<false>(part, e4m3x2_to_bf16x2(wa[q], 0x1404), e4m3x2_to_bf16x2(wb[q], 0x1404),
                                            e4m3x2_to_bf16x2(wa[q], 0x3424), e4m3x2_to_bf16x2(wb[q], 0x3424),
                                            q % 2 ? b.z : b.x, q % 2 ? b.w : b.y);
                        }
                    }
                    const float sa = __uint_as_float(o0.sa.x), sb = __uint_as_float(o0.sb.x);
                    c[0] = fmaf(part[0], sa, c[0]);
                    c[1] = fmaf(part[1], sa, c[1]);
                    c[2] = fmaf(part[2], sb, c[2]);
                    c[3] = fmaf(part[3], sb, c[3]);
                } else {
                    const uint4 va = *reinterpret_cast<const uint4 *>(pa), vb = *reinterpret_cast<const uint4 *>(pb);
                    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
                    // the scale of each 32 inputs
                    float sa[4], sb[4];
                    if (a.group == 32) {
                        sa[0] = bf16_lo(o0.sa.x), sa[1] = bf16_hi(o0.sa.x), sa[2] = bf16_lo(o0.sa.y), sa[3] = bf16_hi(o0.sa.y);
                        sb[0] = bf16_lo(o0.sb.x), sb[1] = bf16_hi(o0.sb.x), sb[2] = bf16_lo(o0.sb.y), sb[3] = bf16_hi(o0.sb.y);
                    } else {
                        sa[0] = sa[1] = bf16_lo(o0.sa.x);
                        sb[0] = sb[1] = bf16_lo(o0.sb.x);
                        sa[2] = sa[3] = a.group == 64 ? bf16_hi(o0.sa.x) : sa[0];
                        sb[2] = sb[3] = a.group == 64 ? bf16_hi(o0.sb.x) : sb[0];
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t ra[4], rb[4];
                        w4_pairs<false>(wa[j], ra);
                        w4_pairs<false>(wb[j], rb);
                        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816<false>(part, ra[0], rb[0], ra[1], rb[1], o0.x[j].x, o0.x[j].y);
                        mma16816<false>(part, ra[2], rb[2], ra[3], rb[3], o0.x[j].z, o0.x[j].w);
                        c[0] = fmaf(part[0], sa[j], c[0]);
                        c[1] = fmaf(part[1], sa[j], c[1]);
                        c[2] = fmaf(part[2], sb[j], c[2]);
                        c[3] = fmaf(part[3], sb[j], c[3]);
                    }
                }
                o0 = o1;
                if (kAhead == 2) o1 = o2;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);

        const FewWalk<DOWN> was = walk;
        walk.next();
        if (was.c + 1 < was.pieces) continue;      // the rows go on
        constexpr float kUnit = WT == MOE_WEIGHTS_W4 ? kW4Unit<false> : 1.0f;
        if constexpr (!DOWN) {
            // the warps' sums joined by one of them in turn, which makes h of them. Two buffers: who writes one again
            // has passed the barrier of the other, which its readers pass after reading
#pragma unroll
            for (int nt = 0; nt < kFewTokens / 8; ++nt) {
                if (8 * nt >= rows) continue;
                red[turn & 1u][warp][lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
                acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
                asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
                if ((unsigned)warp == turn % kFewWarps) {
                    float4 v = red[turn & 1u][0][lane];
#pragma unroll
                    for (int i = 1; i < kFewWarps; ++i) {
                        const float4 u = red[turn & 1u][i][lane];
                        v.x += u.x;
                        v.y += u.y;
                        v.z += u.z;
                        v.w += u.w;
                    }
                    const int r = 8 * nt + 2 * t, o = was.row() * 8 + g;
                    if (r < rows) put_bf16(h + (size_t)lists.pair[first + r] * a.I + o, silu(v.x * kUnit) * (v.z * kUnit));
                    if (r + 1 < rows)
                        put_bf16(h + (size_t)lists.pair[first + r + 1] * a.I + o, silu(v.y * kUnit) * (v.w * kUnit));
                }
                ++turn;
            }
        } else {
            // this list's rows into the warp's sums of their tokens
            float *mine = acc_out + warp * a.T * 16;
#pragma unroll
            for (int nt = 0; nt < kFewTokens / 8; ++nt) {
                if (8 * nt >= rows) continue;
                const int r = 8 * nt + 2 * t;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (r + q < rows) {
                        const float by = lists.weight[first + r + q] * kUnit;
                        float *to = mine + lists.token[first + r + q] * 16 + g;
                        to[0] = fmaf(acc[nt][q], by, to[0]);
                        to[8] = fmaf(acc[nt][2 + q], by, to[8]);
                    }
                }
                acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
            }
            __syncwarp();
            if (was.d + 1 < was.lists) continue;
            asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
            for (int i = tid; i < a.T * 16; i += kFewWarps * 32) {
                float v = 0.0f;
#pragma unroll
                for (int j = 0; j < kFewWarps; ++j) {
                    v += acc_out[j * a.T * 16 + i];
                    acc_out[j * a.T * 16 + i] = 0.0f;
                }
                put_bf16(out + (size_t)(i >> 4) * a.H + was.row() * 16 + (i & 15), v);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
        }
    }
    if constexpr (DOWN) {
        if (lists.n == 0)                          // not one pair in the whole batch
            for (int i = blockIdx.x * kFewWarps * 32 + tid; i < a.T * a.H; i += gridDim.x * kFewWarps * 32) out[i] = 0;
    }
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

template <int WT>
int launch_few(const Dims &d, const FewArgs &a, cudaStream_t st, const void *x, const void *logits, const float *bias,
               const void *w_up, const void *up_scale, const void *w_down, const void *down_scale, int32_t *idx, float *w,
               void *out, void *h, unsigned *status) {
    static PerContext<int> up_done, down_done;
    const size_t ring = (size_t)kFewStages * kFewStage, most = ring + kFewWarps * kFewTokens * 16 * sizeof(float);
    if (!set_smem_once(up_done, few_kernel<WT, false>, (int)ring) || !set_smem_once(down_done, few_kernel<WT, true>, (int)most))
        return MOE_ERR_CUDA;
    const long long lists = std::min<long long>((long long)d.T * d.k, d.E) + a.shared;
    int grid = persistent_grid(lists * (a.I / 8), sm_count(), d.max_blocks);
    if (launch_pdl_smem(few_kernel<WT, false>, grid, kFewThreads, ring, st, a, static_cast<const uint16_t *>(x), logits, bias,
                        static_cast<const uint8_t *>(w_up), up_scale, static_cast<uint16_t *>(h), idx, w,
                        static_cast<uint16_t *>(out), status) != cudaSuccess)
        return MOE_ERR_CUDA;
    grid = persistent_grid(d.H / 16, sm_count(), d.max_blocks);
    if (launch_pdl_smem(few_kernel<WT, true>, grid, kFewThreads, ring + (size_t)kFewWarps * d.T * 16 * sizeof(float), st, a,
                        static_cast<const uint16_t *>(x), logits, bias, static_cast<const uint8_t *>(w_down), down_scale,
                        static_cast<uint16_t *>(h), idx, w, static_cast<uint16_t *>(out), status) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_layer_few_workspace_bytes(const moe_problem *p, const moe_mlp *mlp) {
    using namespace moe;
    Dims d;
    if (check_problem(p, &d) != MOE_OK || check_mlp(mlp) != MOE_OK || check_few(d, mlp) != MOE_OK) return 0;
    const size_t n = (size_t)d.T * (d.k + mlp->shared) * mlp->inner * 2;
    return n < 256 ? 256 : (n + 255) & ~(size_t)255;
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
    a.group = mlp->group;
    a.logits_bf16 = gate->logits_type == MOE_LOGITS_BF16;
    unsigned *status = device_status_word();
    if (status == nullptr) return MOE_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    if (mlp->weights == MOE_WEIGHTS_BF16)
        return launch_few<MOE_WEIGHTS_BF16>(d, a, st, x, logits, bias, w_up, up_scale, w_down, down_scale, topk_idx, topk_w,
                                            out, workspace, status);
    if (mlp->weights == MOE_WEIGHTS_FP8_B128)
        return launch_few<MOE_WEIGHTS_FP8_B128>(d, a, st, x, logits, bias, w_up, up_scale, w_down, down_scale, topk_idx,
                                                topk_w, out, workspace, status);
    return launch_few<MOE_WEIGHTS_W4>(d, a, st, x, logits, bias, w_up, up_scale, w_down, down_scale, topk_idx, topk_w, out,
                                      workspace, status);
}

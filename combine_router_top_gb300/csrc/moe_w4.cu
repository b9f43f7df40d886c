// moe_w4.cu -- the experts' products with 4-bit weights and group scales.
//
//   r[m] = sum_g scale[m][g] * sum_{i in g} x[i] (q[m][i] - 8)
//   y[n] = bf16(r[n])  or  bf16(silu(r[n]) r[N + n])
//
// q - 8 is an integer of -8..7, exact in bf16 and in fp16, and so is its product
// with a bf16 (or e4m3) x in fp32: each group's sum runs on the tensor cores as
// it is, the scale multiplies the sum in fp32, and the only rounding to 16 bits
// is the output's.
//
// Few rows per expert (this file's first kernel): every weight is read once for
// few products, so the call is bound by HBM. The weights are the 16-row operand
// of mma.m16n8k16 and 8 rows of x its 8 columns. A block takes 16 rows of one
// expert's matrix; its warps split the inputs in blocks of 128 and join their
// sums through shared memory in the warps' order. Within 128 inputs lane
// (g, t) of the fragment holds bytes 16 t .. 16 t + 15 of row g, one 16-byte
// load: the packing puts there 8 inputs of each 32, which are the lane's
// share of two MMA steps, so that every step stays within one group of 32.
#include "moe_w4.cuh"

namespace moe {
namespace {

constexpr int kW4Warps = 8;

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight inputs of one row as four 16-bit pairs.
template <bool F8>
__device__ __forceinline__ void load_x8(const uint8_t *p, uint32_t (&b)[4]) {
    if constexpr (F8) {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p));
        b[0] = e4m3x2_to_f16x2(q.x);
        b[1] = e4m3x2_to_f16x2(q.x >> 16);
        b[2] = e4m3x2_to_f16x2(q.y);
        b[3] = e4m3x2_to_f16x2(q.y >> 16);
    } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
        b[0] = q.x;
        b[1] = q.y;
        b[2] = q.z;
        b[3] = q.w;
    }
}

// The scales of one row's 128 inputs: group 128: one bf16; 64: two; 32: four.
template <int GS>
__device__ __forceinline__ void load_scales(const uint16_t *p, float (&s)[128 / GS]) {
    if constexpr (GS == 128) {
        s[0] = __uint_as_float((uint32_t)__ldg(p) << 16);
    } else if constexpr (GS == 64) {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(p));
        s[0] = bf16_lo(v);
        s[1] = bf16_hi(v);
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        s[0] = bf16_lo(v.x);
        s[1] = bf16_hi(v.x);
        s[2] = bf16_lo(v.y);
        s[3] = bf16_hi(v.y);
    }
}

// Exclusive scan over e of the token tiles (of `tile` rows) of min(counts[e], C)
// rows into off[0..E]; one block of kW4Warps * 32 threads.
__device__ __forceinline__ void token_tile_offsets(const int32_t *__restrict__ counts, int E, int C, int tile, int *off,
                                                   int *warp_tot) {
    const int nt = kW4Warps * 32, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + nt - 1) / nt;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) local += (min(__ldg(counts + e), C) + tile - 1) / tile;
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int run = incl - local;
    for (int i = 0; i < warp; ++i) run += warp_tot[i];
    for (int e = e0; e < e1; ++e) {
        off[e] = run;
        run += (min(__ldg(counts + e), C) + tile - 1) / tile;
    }
    if (tid == nt - 1) off[E] = run;
    __syncthreads();
}

template <bool F8, int GS, bool GATE, int NT>
__global__ void __launch_bounds__(kW4Warps * 32)
expert_w4_rows_kernel(W4Args a, const uint8_t *__restrict__ x, const float *__restrict__ x_scale,
                      const int32_t *__restrict__ counts, const uint8_t *__restrict__ w_q,
                      const uint16_t *__restrict__ w_scale, uint16_t *__restrict__ y) {
    constexpr int kTokens = 8 * NT, kOut = GATE ? 8 : 16, kGroups = 128 / GS;
    __shared__ int off[kMaxExperts + 1];
    __shared__ int warp_tot[kW4Warps];
    __shared__ float4 red[kW4Warps][NT][32];
    pdl_enter();
    token_tile_offsets(counts, a.E, a.C, kTokens, off, warp_tot);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const unsigned tiles = off[a.E], row_tiles = (a.N + kOut - 1) / kOut;
    const size_t w_row = (size_t)a.K / 2, s_row = (size_t)a.K / GS, x_row = F8 ? (size_t)a.K : 2 * (size_t)a.K;

    for (UnitWalk wk(blockIdx.x, gridDim.x, row_tiles); wk.row < tiles; wk.next()) {
        const int e = expert_of_row(off, a.E, (int)wk.row);
        const int kept = min(__ldg(counts + e), a.C);
        const int tok0 = (int)(wk.row - off[e]) * kTokens;
        const int n0 = (int)wk.seg * kOut;
        // rows past the matrix read its last row, and their sums are not stored
        const int ra = min(n0 + g, a.N - 1);
        const int rb = GATE ? a.N + ra : min(n0 + 8 + g, a.N - 1);
        const uint8_t *qa = w_q + ((size_t)e * a.M + ra) * w_row + 16 * t;
        const uint8_t *qb = w_q + ((size_t)e * a.M + rb) * w_row + 16 * t;
        const uint16_t *sa = w_scale + ((size_t)e * a.M + ra) * s_row;
        const uint16_t *sb = w_scale + ((size_t)e * a.M + rb) * s_row;
        const uint8_t *px[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)           // columns past the rows read the last row, not stored either
            px[n] = x + ((size_t)e * a.C + min(tok0 + 8 * n + g, kept - 1)) * x_row + (F8 ? 8 : 16) * t;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;

        for (int kb = warp; kb < a.nkb; kb += kW4Warps) {
            const uint4 va = ld_stream_v4(qa + (size_t)kb * 64), vb = ld_stream_v4(qb + (size_t)kb * 64);
            float fa[kGroups], fb[kGroups];
            load_scales<GS>(sa + kb * kGroups, fa);
            load_scales<GS>(sb + kb * kGroups, fb);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                fa[q] *= kW4Unit<F8>;
                fb[q] *= kW4Unit<F8>;
            }
            const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float blk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                float part[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j % (GS / 32) == 0) part[0] = part[1] = part[2] = part[3] = 0.0f;
                    uint32_t b[4], pa[4], pb[4];
                    load_x8<F8>(px[n] + (size_t)kb * (F8 ? 128 : 256) + j * (F8 ? 32 : 64), b);
                    w4_pairs<F8>(wa[j], pa);
                    w4_pairs<F8>(wb[j], pb);
                    mma16816<F8>(part, pa[0], pb[0], pa[1], pb[1], b[0], b[1]);
                    mma16816<F8>(part, pa[2], pb[2], pa[3], pb[3], b[2], b[3]);
                    if (j % (GS / 32) == GS / 32 - 1) {
                        const int q = j / (GS / 32);
                        float(&to)[4] = F8 ? blk : acc[n];
                        to[0] = fmaf(part[0], fa[q], to[0]);
                        to[1] = fmaf(part[1], fa[q], to[1]);
                        to[2] = fmaf(part[2], fb[q], to[2]);
                        to[3] = fmaf(part[3], fb[q], to[3]);
                    }
                }
                if constexpr (F8) {
                    const int c0 = min(tok0 + 8 * n + 2 * t, kept - 1), c1 = min(tok0 + 8 * n + 2 * t + 1, kept - 1);
                    const float s0 = __ldg(x_scale + ((size_t)e * a.C + c0) * a.nkb + kb);
                    const float s1 = __ldg(x_scale + ((size_t)e * a.C + c1) * a.nkb + kb);
                    acc[n][0] = fmaf(blk[0], s0, acc[n][0]);
                    acc[n][1] = fmaf(blk[1], s1, acc[n][1]);
                    acc[n][2] = fmaf(blk[2], s0, acc[n][2]);
                    acc[n][3] = fmaf(blk[3], s1, acc[n][3]);
                }
            }
        }
        __syncthreads();                       // the previous unit's sums have been read
#pragma unroll
        for (int n = 0; n < NT; ++n) red[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (warp < NT) {                       // warp n joins the sums of columns 8n .. 8n+7
            float4 r = red[0][warp][lane];
#pragma unroll
            for (int i = 1; i < kW4Warps; ++i) {
                const float4 v = red[i][warp][lane];
                r.x += v.x;
                r.y += v.y;
                r.z += v.z;
                r.w += v.w;
            }
            const int c = tok0 + 8 * warp + 2 * t;
            uint16_t *o = y + ((size_t)e * a.C + c) * a.N + n0 + g;
            if constexpr (GATE) {
                if (n0 + g < a.N) {
                    if (c < kept) put_bf16(o, silu(r.x) * r.z);
                    if (c + 1 < kept) put_bf16(o + a.N, silu(r.y) * r.w);
                }
            } else {
                if (n0 + g < a.N) {
                    if (c < kept) put_bf16(o, r.x);
                    if (c + 1 < kept) put_bf16(o + a.N, r.y);
                }
                if (n0 + 8 + g < a.N) {
                    if (c < kept) put_bf16(o + 8, r.z);
                    if (c + 1 < kept) put_bf16(o + 8 + a.N, r.w);
                }
            }
        }
    }
}

template <bool F8, int GS, bool GATE, int NT>
int launch_rows(const Dims &d, const W4Args &a, cudaStream_t st, const void *x, const float *x_scale,
                const int32_t *counts, const void *w_q, const void *w_scale, void *y) {
    static PerContext<int> resident_cache;
    const int resident = resident_blocks_cached(resident_cache, expert_w4_rows_kernel<F8, GS, GATE, NT>, kW4Warps * 32);
    const long long tiles = (long long)(d.T * (long long)d.k < (long long)d.E * d.C ? d.T * (long long)d.k : (long long)d.E * d.C);
    const int grid = persistent_grid(tiles * ((a.N + (GATE ? 8 : 16) - 1) / (GATE ? 8 : 16)), resident, d.max_blocks);
    if (launch_pdl(expert_w4_rows_kernel<F8, GS, GATE, NT>, grid, kW4Warps * 32, st, a, static_cast<const uint8_t *>(x),
                   x_scale, counts, static_cast<const uint8_t *>(w_q), static_cast<const uint16_t *>(w_scale),
                   static_cast<uint16_t *>(y)) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <bool F8, int GS, bool GATE, typename... A>
int launch_nt(const Dims &d, A... args) {
    if ((d.T < d.C ? d.T : d.C) <= 8) return launch_rows<F8, GS, GATE, 1>(d, args...);
    return launch_rows<F8, GS, GATE, 2>(d, args...);
}
template <bool F8, int GS, typename... A>
int launch_gate_act(const Dims &d, const W4Args &a, A... args) {
    return a.M == 2 * a.N ? launch_nt<F8, GS, true>(d, a, args...) : launch_nt<F8, GS, false>(d, a, args...);
}
template <bool F8, typename... A>
int launch_group(const Dims &d, const W4Args &a, A... args) {
    if (a.group == 32) return launch_gate_act<F8, 32>(d, a, args...);
    if (a.group == 64) return launch_gate_act<F8, 64>(d, a, args...);
    return launch_gate_act<F8, 128>(d, a, args...);
}

int check_w4(const moe_w4 *w) {
    if (w == nullptr) return MOE_ERR_INVALID_ARG;
    if (w->n_in < 128 || w->n_in > kMaxHidden || w->n_in % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (w->n_out < 8 || w->n_out > kMaxHidden || w->n_out % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_ERR_INVALID_ARG;
    if (w->act != MOE_ACT_NONE && w->act != MOE_ACT_SILU_GATE) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

W4Args w4_args(const Dims &d, const moe_w4 *w) {
    W4Args a;
    a.E = d.E;
    a.C = d.C;
    a.K = w->n_in;
    a.N = w->n_out;
    a.M = w->act == MOE_ACT_SILU_GATE ? 2 * w->n_out : w->n_out;
    a.group = w->group;
    a.nkb = a.K / 128;
    return a;
}

// Many rows per expert take the tiles.
bool w4_many_rows(const Dims &d) {
    return (d.T < d.C ? d.T : d.C) > 8 && (long long)d.T * d.k >= 4LL * d.E;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_expert_w4_workspace_bytes(const moe_problem *p, const moe_w4 *w) {
    using namespace moe;
    Dims d;
    if (check_problem(p, &d) != MOE_OK || check_w4(w) != MOE_OK) return 0;
    const size_t n = w4_many_rows(d) ? w4_tiles_workspace_bytes(d, w4_args(d, w)) : 0;
    return n < 256 ? 256 : n;
}

extern "C" int moe_expert_w4(const moe_problem *p, const moe_w4 *w, const void *x, const float *x_scale,
                             const int32_t *counts, const void *w_q, const void *w_scale, void *y, void *workspace,
                             size_t workspace_bytes, void *stream) {
    using namespace moe;
    Dims d;
    int rc = check_problem(p, &d);
    if (rc != MOE_OK) return rc;
    rc = check_w4(w);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    const bool f8 = d.dtype == MOE_DTYPE_FP8_E4M3_B128;
    if (f8 != (x_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!x || !counts || !w_q || !w_scale || !y || !workspace) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_expert_w4_workspace_bytes(p, w)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w_q, 16) || !aligned(y, 16) || !aligned(workspace, 16) || !aligned(w_scale, 16) ||
        !aligned(counts, 4) || !aligned(x_scale, 4))
        return MOE_ERR_INVALID_ARG;
    const W4Args a = w4_args(d, w);
    cudaStream_t st = as_stream(stream);
    if (w4_many_rows(d)) return launch_w4_tiles(d, a, st, x, x_scale, counts, w_q, w_scale, y, workspace);
    if (f8) return launch_group<true>(d, a, st, x, x_scale, counts, w_q, w_scale, y);
    return launch_group<false>(d, a, st, x, x_scale, counts, w_q, w_scale, y);
}

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
// Few rows per expert (this file; moe_w4_tiles.cu has the kernel for many): every
// weight is read once for few products, so the call is bound by HBM. The weights are
// the 16-row operand of mma.m16n8k16 and up to 8 rows of x its 8 columns: a tcgen05
// tile of 128 rows would leave most SMs without work for one token's few experts.
// Within 128 inputs lane (g, t) of the fragment holds bytes 16 t .. 16 t + 15 of row
// g, one 16-byte copy: the packing puts there 8 inputs of each 32, which are the
// lane's share of two MMA steps, so that every step stays within one group of 32.
// One token, 8 experts of 2 x 2048 x 7168 (121 MB): 29 us, 0.61 of the copy
// bandwidth; of it about 7 us are the launch, the wait for the counts and the
// unequal last round of units. 64 such experts: 0.76.
#include "moe_w4.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Depth = 4;            // blocks of codes that a warp has in flight or at hand
constexpr int kW4Stage = 1024 + 128;   // a block of 16 rows: 64 bytes of codes and up to 8 of scales each
constexpr int kW4TileMap = 1024;       // token tiles whose expert is looked up instead of searched

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

// The scales of one row's 128 inputs from shared memory: group 128: one bf16, the
// upper one of its word if odd; 64: two; 32: four.
template <int GS>
__device__ __forceinline__ void read_scales(const uint8_t *p, unsigned odd, float (&s)[128 / GS]) {
    if constexpr (GS == 128) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
        s[0] = odd ? bf16_hi(v) : bf16_lo(v);
    } else if constexpr (GS == 64) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
        s[0] = bf16_lo(v);
        s[1] = bf16_hi(v);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        s[0] = bf16_lo(v.x);
        s[1] = bf16_hi(v.x);
        s[2] = bf16_lo(v.y);
        s[3] = bf16_hi(v.y);
    }
}

// kept[e] = min(counts[e], C); the exclusive scan over e of their token tiles (of
// `tile` rows) into off[0..E]; and the expert of each of the first kW4TileMap tiles
// into tile_e. One block of kW4Warps * 32 threads.
__device__ __forceinline__ void token_tile_offsets(const int32_t *__restrict__ counts, int E, int C, int tile, int *kept,
                                                   int *off, uint16_t *tile_e, int *warp_tot) {
    const int nt = kW4Warps * 32, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + nt - 1) / nt;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int local = 0;
    for (int e = e0; e < e1; ++e) {
        kept[e] = min(__ldg(counts + e), C);
        local += (kept[e] + tile - 1) / tile;
    }
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
        const int n = (kept[e] + tile - 1) / tile;
        for (int i = run; i < min(run + n, kW4TileMap); ++i) tile_e[i] = (uint16_t)e;
        run += n;
    }
    if (tid == nt - 1) off[E] = run;
    __syncthreads();
}

// BYTES (4, 8 or 16) of global memory to shared memory, tracked by this thread's groups.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// What a block needs to know of a unit of its work.
struct W4Unit {
    int e, n0, tok0, kept;             // expert, first output, first row of x, rows of the expert
};

// A block takes 16 MT rows of one expert's matrix (with the gate 8 MT outputs) and
// up to 8 of the expert's rows of x; its 8 warps split the inputs in blocks of
// 128, warp w the blocks w, w + 8, ... Each warp keeps kW4Depth blocks of codes and
// scales coming to a ring of its own by asynchronous copies, over the end of one
// unit of work into the next, so that the joining of the sums at the unit's end does
// not empty it. A lane reads the codes that it copied itself.
template <bool F8, int GS, bool GATE, int MT>
__global__ void __launch_bounds__(kW4Warps * 32, MT == 1 ? 3 : 2)
expert_w4_rows_kernel(W4Args a, const uint8_t *__restrict__ x, const float *__restrict__ x_scale,
                      const int32_t *__restrict__ counts, const uint8_t *__restrict__ w_q,
                      const uint16_t *__restrict__ w_scale, uint16_t *__restrict__ y) {
    constexpr int kTokens = 8, kOut = (GATE ? 8 : 16) * MT, kGroups = 128 / GS;
    constexpr int kScaleBytes = GS == 32 ? 8 : 4;    // copied for a row's block: its scales, or the word they are in
    constexpr int kStage = MT * kW4Stage;
    __shared__ __align__(16) uint8_t ring[kW4Warps][kW4Depth][kStage];
    __shared__ int rows_of[kMaxExperts], off[kMaxExperts + 1];
    __shared__ uint16_t tile_e[kW4TileMap];
    __shared__ int warp_tot[kW4Warps];
    __shared__ float4 red[2][kW4Warps][MT][32];
    pdl_enter();
    token_tile_offsets(counts, a.E, a.C, kTokens, rows_of, off, tile_e, warp_tot);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const unsigned tiles = off[a.E], row_tiles = (a.N + kOut - 1) / kOut;
    const size_t w_row = (size_t)a.K / 2, s_row = (size_t)a.K / GS, x_row = F8 ? (size_t)a.K : 2 * (size_t)a.K;
    const auto expert_of = [&](unsigned p) { return p < kW4TileMap ? (int)tile_e[p] : expert_of_row(off, a.E, (int)p); };

    // matrix rows g and g + 8 of a fragment; rows past the matrix read its last, and their sums are not stored
    const auto row_a = [&](int n0, int m) { return min(n0 + (GATE ? 8 : 16) * m + g, a.N - 1); };
    const auto row_b = [&](int n0, int m) { return GATE ? a.N + row_a(n0, m) : min(n0 + 16 * m + 8 + g, a.N - 1); };
    // the blocks to fetch, in the order that they are used
    UnitWalk fw(blockIdx.x, gridDim.x, row_tiles);
    int fkb = a.nkb;                                 // past the end: unit fw is the next
    const uint8_t *fa[MT], *fb[MT], *fs[MT];
    const uint32_t dst = smem_u32(&ring[warp][0][0]) + 16 * lane;
    const uint32_t sdst = smem_u32(&ring[warp][0][1024 * MT]) + 64 * t + 8 * g;  // lanes t = 0, 1: rows g and g + 8
    const auto fetch = [&](unsigned slot) {
        if (fkb >= a.nkb && warp < a.nkb) {
            if (fw.row < tiles) {
                const size_t m0 = (size_t)expert_of(fw.row) * a.M;
                const int n0 = (int)fw.seg * kOut;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int ra = row_a(n0, m), rb = row_b(n0, m);
                    fa[m] = w_q + (m0 + ra) * w_row + 64 * warp + 16 * t;
                    fb[m] = w_q + (m0 + rb) * w_row + 64 * warp + 16 * t;
                    fs[m] = reinterpret_cast<const uint8_t *>(w_scale + (m0 + (t == 0 ? ra : rb)) * s_row + warp * kGroups);
                    fs[m] -= reinterpret_cast<uintptr_t>(fs[m]) & (kScaleBytes - 1);
                }
                fkb = warp;
                fw.next();
            }
        }
        if (fkb < a.nkb) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                cp_async<16>(dst + slot * kStage + 1024 * m, fa[m]);
                cp_async<16>(dst + slot * kStage + 1024 * m + 512, fb[m]);
                if (t < 2) cp_async<kScaleBytes>(sdst + slot * kStage + 128 * m, fs[m]);
                fa[m] += 64 * kW4Warps;
                fb[m] += 64 * kW4Warps;
                fs[m] += 2 * kGroups * kW4Warps;
            }
            fkb += kW4Warps;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (unsigned i = 0; i < kW4Depth - 1; ++i) fetch(i);

    unsigned step = 0;
    unsigned n_unit = 0;
    for (UnitWalk wk(blockIdx.x, gridDim.x, row_tiles); wk.row < tiles; wk.next(), ++n_unit) {
        W4Unit u;
        u.e = expert_of(wk.row);
        u.n0 = (int)wk.seg * kOut;
        u.tok0 = (int)(wk.row - off[u.e]) * kTokens;
        u.kept = rows_of[u.e];
        // columns past the rows read the last row, and are not stored
        const uint8_t *px = x + ((size_t)u.e * a.C + min(u.tok0 + g, u.kept - 1)) * x_row + (F8 ? 8 : 16) * t +
                            (size_t)warp * (F8 ? 128 : 256);
        // which half of its word holds the scale of a group of 128: the same for all of a warp's blocks of a row
        unsigned odd = 0;
        if constexpr (GS == 128) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                odd |= (((unsigned)row_a(u.n0, m) * a.nkb + warp) & 1u) << (2 * m) |
                       (((unsigned)row_b(u.n0, m) * a.nkb + warp) & 1u) << (2 * m + 1);
        }
        float acc[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;

        for (int kb = warp; kb < a.nkb; kb += kW4Warps, ++step) {
            uint32_t b[4][4];                        // the block's x, before the wait for its codes
#pragma unroll
            for (int j = 0; j < 4; ++j) load_x8<F8>(px + j * (F8 ? 32 : 64), b[j]);
            px += kW4Warps * (F8 ? 128 : 256);
            asm volatile("cp.async.wait_group %0;" ::"n"(kW4Depth - 2) : "memory");
            __syncwarp();                            // this block is there, and the last one's slot has been read
            fetch((step + kW4Depth - 1) % kW4Depth);
            const uint8_t *at = &ring[warp][step % kW4Depth][0];
            uint4 va[MT], vb[MT];
            float sa[MT][kGroups], sb[MT][kGroups];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                va[m] = *reinterpret_cast<const uint4 *>(at + 1024 * m + 16 * lane);
                vb[m] = *reinterpret_cast<const uint4 *>(at + 1024 * m + 512 + 16 * lane);
                read_scales<GS>(at + 1024 * MT + 128 * m + 8 * g, odd >> (2 * m) & 1u, sa[m]);
                read_scales<GS>(at + 1024 * MT + 128 * m + 64 + 8 * g, odd >> (2 * m + 1) & 1u, sb[m]);
            }
            float part[MT][4], blk[F8 ? MT : 1][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t pa[4], pb[4];
                    w4_pairs<F8>(j == 0 ? va[m].x : j == 1 ? va[m].y : j == 2 ? va[m].z : va[m].w, pa);
                    w4_pairs<F8>(j == 0 ? vb[m].x : j == 1 ? vb[m].y : j == 2 ? vb[m].z : vb[m].w, pb);
                    float(&p)[4] = part[m];
                    if (j % (GS / 32) == 0) p[0] = p[1] = p[2] = p[3] = 0.0f;
                    mma16816<F8>(p, pa[0], pb[0], pa[1], pb[1], b[j][0], b[j][1]);
                    mma16816<F8>(p, pa[2], pb[2], pa[3], pb[3], b[j][2], b[j][3]);
                    if (j % (GS / 32) == GS / 32 - 1) {
                        const int q = j / (GS / 32);
                        float(&to)[4] = F8 ? blk[m] : acc[m];
                        if (F8 && q == 0) to[0] = to[1] = to[2] = to[3] = 0.0f;
                        to[0] = fmaf(p[0], sa[m][q], to[0]);
                        to[1] = fmaf(p[1], sa[m][q], to[1]);
                        to[2] = fmaf(p[2], sb[m][q], to[2]);
                        to[3] = fmaf(p[3], sb[m][q], to[3]);
                    }
                }
            }
            if constexpr (F8) {
                const int c0 = min(u.tok0 + 2 * t, u.kept - 1), c1 = min(u.tok0 + 2 * t + 1, u.kept - 1);
                const float s0 = __ldg(x_scale + ((size_t)u.e * a.C + c0) * a.nkb + kb);
                const float s1 = __ldg(x_scale + ((size_t)u.e * a.C + c1) * a.nkb + kb);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    acc[m][0] = fmaf(blk[m][0], s0, acc[m][0]);
                    acc[m][1] = fmaf(blk[m][1], s1, acc[m][1]);
                    acc[m][2] = fmaf(blk[m][2], s0, acc[m][2]);
                    acc[m][3] = fmaf(blk[m][3], s1, acc[m][3]);
                }
            }
        }
        // two buffers of sums: a warp that writes unit u + 2's has passed the barrier of unit u + 1, which the
        // readers of unit u's pass after reading
        float4(&sums)[kW4Warps][MT][32] = red[n_unit & 1];
#pragma unroll
        for (int m = 0; m < MT; ++m) sums[warp][m][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        __syncthreads();
        if (warp < MT) {                       // one warp for each fragment of 16 matrix rows
            float4 r = sums[0][warp][lane];
#pragma unroll
            for (int i = 1; i < kW4Warps; ++i) {
                const float4 v = sums[i][warp][lane];
                r.x += v.x;
                r.y += v.y;
                r.z += v.z;
                r.w += v.w;
            }
            r.x *= kW4Unit<F8>;
            r.y *= kW4Unit<F8>;
            r.z *= kW4Unit<F8>;
            r.w *= kW4Unit<F8>;
            const int c = u.tok0 + 2 * t, out = u.n0 + (GATE ? 8 : 16) * warp + g;
            uint16_t *o = y + ((size_t)u.e * a.C + c) * a.N + out;
            if constexpr (GATE) {
                if (out < a.N) {
                    if (c < u.kept) put_bf16(o, silu(r.x) * r.z);
                    if (c + 1 < u.kept) put_bf16(o + a.N, silu(r.y) * r.w);
                }
            } else {
                if (out < a.N) {
                    if (c < u.kept) put_bf16(o, r.x);
                    if (c + 1 < u.kept) put_bf16(o + a.N, r.y);
                }
                if (out + 8 < a.N) {
                    if (c < u.kept) put_bf16(o + 8, r.z);
                    if (c + 1 < u.kept) put_bf16(o + 8 + a.N, r.w);
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool F8, int GS, bool GATE, int MT>
int launch_rows(const Dims &d, const W4Args &a, cudaStream_t st, const void *x, const float *x_scale,
                const int32_t *counts, const void *w_q, const void *w_scale, void *y) {
    static PerContext<int> resident_cache;
    const auto kernel = expert_w4_rows_kernel<F8, GS, GATE, MT>;
    const int resident = resident_blocks_cached(resident_cache, kernel, kW4Warps * 32);
    constexpr int kOut = (GATE ? 8 : 16) * MT;
    const long long tiles = std::min<long long>((long long)d.T * d.k, (long long)d.E * d.C);
    const int grid = persistent_grid(tiles * ((a.N + kOut - 1) / kOut), resident, d.max_blocks);
    if (launch_pdl(kernel, grid, kW4Warps * 32, st, a, static_cast<const uint8_t *>(x), x_scale, counts,
                   static_cast<const uint8_t *>(w_q), static_cast<const uint16_t *>(w_scale),
                   static_cast<uint16_t *>(y)) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <bool F8, int GS, bool GATE, typename... A>
int launch_mt(const Dims &d, const W4Args &a, A... args) {
    // Two fragments of matrix rows to a warp halve what it spends beside the products (8 tokens of 64 live experts
    // of 2 x 2048 x 7168: 189 us, with one 209), where the experts that can have rows still give every resident
    // block a few units.
    const long long live = std::min<long long>((long long)d.T * d.k, d.E);
    if (live * a.N / (GATE ? 16 : 32) >= 3LL * sm_count()) return launch_rows<F8, GS, GATE, 2>(d, a, args...);
    return launch_rows<F8, GS, GATE, 1>(d, a, args...);
}
template <bool F8, int GS, typename... A>
int launch_gate_act(const Dims &d, const W4Args &a, A... args) {
    return a.M == 2 * a.N ? launch_mt<F8, GS, true>(d, a, args...) : launch_mt<F8, GS, false>(d, a, args...);
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

// Many rows per expert take the tiles: from 4 rows on the mean, where some expert can have over 8. 64 experts of
// 2 x 2048 x 7168, groups of 128, us: 1 row 187 here, 199 with the tiles; 4 rows 195 and 199; 8 rows 214 and 199, and
// past 8 rows this file's kernel reads the weights again for every 8. The figures are for even loads: the mean is all that
// is known on the host, and an expert far above it pays that way here.
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

// moe_combine_bwd.cu -- the gradient of the top-k weighted combine.
//
// out[t] = sum_j w_j y[e_j][slot_j] gives, for every kept pair,
//   d_y[e_j][slot_j] = bf16(w_j d_out[t])        d_w[t][j] = <d_out[t], y[e_j][slot_j]>.
// One pass: a row of d_out is read once into registers, each of the token's k
// rows of y meets it there, and the scaled copy leaves for d_y. Bound by HBM:
// two bytes read and two written per kept element, two read per token element.
// The dot products are summed in fp32, per lane over its chunks in order, then
// over the warp by a butterfly, then over the token's warps in order: the order
// depends on the sizes alone.
#include "moe_internal.cuh"

namespace moe {
namespace {

// A block of WPT warps takes a token at a time and walks its row in segments of
// WPT*32 chunks of 16 bytes (8 elements), one chunk to a lane. Many small blocks
// with one load in flight a lane keep HBM busier than few with several: 4096 x 7168
// top-8, 4 warps with 7 chunks a lane 189 us, 7 warps with 4, 2 and 1 174, 164 and
// 161 (0.92 of the copy bandwidth), 14 and 28 warps with 1 163 and 233.
template <int WPT, int KMAX>
__global__ void __launch_bounds__(WPT * 32)
combine_backward_kernel(const uint4 *__restrict__ y, const uint4 *__restrict__ d_out,
                        const int32_t *__restrict__ topk_idx, const float *__restrict__ topk_w,
                        const int32_t *__restrict__ slot, uint4 *__restrict__ d_y, float *__restrict__ d_w, int T,
                        int H8, int k, int C) {
    __shared__ float part[2][WPT][KMAX];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int buf = 0;
    for (int t = blockIdx.x; t < T; t += gridDim.x, buf ^= 1) {
        int row = -1;
        float w = 0.0f;
        if (lane < k) {
            const int s = __ldg(slot + (size_t)t * k + lane);
            const int e = __ldg(topk_idx + (size_t)t * k + lane);
            w = __ldg(topk_w + (size_t)t * k + lane);
            if (s >= 0) row = e * C + s;
        }
        const unsigned kept = __ballot_sync(kFull, row >= 0);
        const int n_kept = __popc(kept);
        float dot[KMAX];
#pragma unroll
        for (int j = 0; j < KMAX; ++j) dot[j] = 0.0f;
        for (int c = threadIdx.x; c - (int)threadIdx.x < H8; c += WPT * 32) {
            uint4 g = make_uint4(0u, 0u, 0u, 0u);
            if (c < H8) g = ld_stream_v4(d_out + (size_t)t * H8 + c);
            const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
            unsigned rem = kept;
#pragma unroll
            for (int j = 0; j < KMAX; ++j) {
                if (j < n_kept) {                                      // warp-uniform
                    const int src = __ffs(rem) - 1;
                    rem &= rem - 1;
                    const size_t at = (size_t)__shfl_sync(kFull, row, src) * H8;
                    const float wj = __shfl_sync(kFull, w, src);
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (c < H8) v = ld_stream_v4(y + at + c);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        dot[j] = __fmaf_rn(bf16_lo(gw[q]), bf16_lo(vw[q]), dot[j]);
                        dot[j] = __fmaf_rn(bf16_hi(gw[q]), bf16_hi(vw[q]), dot[j]);
                        o[q] = pack_bf16x2(__fmul_rn(wj, bf16_lo(gw[q])), __fmul_rn(wj, bf16_hi(gw[q])));
                    }
                    if (c < H8) st_v4(d_y + at + c, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            if (j < n_kept) {
                float s = dot[j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                if (lane == 0) part[buf][warp][j] = s;
            }
        }
        // two buffers: the next token's parts do not touch these, and the one
        // after it comes behind the next token's barrier
        __syncthreads();
        if (warp == 0 && lane < k) {
            float s = 0.0f;
            if (row >= 0) {
                const int j = __popc(kept & ((1u << lane) - 1u));
#pragma unroll
                for (int i = 0; i < WPT; ++i) s += part[buf][i][j];
            }
            d_w[(size_t)t * k + lane] = s;
        }
    }
}

template <int WPT, int KMAX>
int launch_one(const Dims &d, cudaStream_t st, const void *y, const void *d_out, const int32_t *idx, const float *w,
               const int32_t *slot, void *d_y, float *d_w) {
    static PerContext<int> resident_cache;
    const int resident = resident_blocks_cached(resident_cache, combine_backward_kernel<WPT, KMAX>, WPT * 32);
    const int grid = persistent_grid(d.T, resident, d.max_blocks);
    if (launch_pdl(combine_backward_kernel<WPT, KMAX>, grid, WPT * 32, st, static_cast<const uint4 *>(y),
                   static_cast<const uint4 *>(d_out), idx, w, slot, static_cast<uint4 *>(d_y), d_w, d.T, d.H / 8, d.k,
                   d.C) != cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <int KMAX, typename... A>
int launch_k(const Dims &d, A... args) {
    const int H8 = d.H / 8;
    if (H8 <= 32) return launch_one<1, KMAX>(d, args...);
    if (H8 <= 64) return launch_one<2, KMAX>(d, args...);
    if (H8 <= 128) return launch_one<4, KMAX>(d, args...);
    // few tokens: the time is a block's own, which more warps to a row shorten (237 x 2056 top-6: 5.3 us with 16
    // warps, 6.9 with 7); many: the width that wastes fewer lanes at the row's end
    if (d.T <= 2 * sm_count()) return launch_one<16, KMAX>(d, args...);
    if ((H8 + 223) / 224 * 224 < (H8 + 255) / 256 * 256) return launch_one<7, KMAX>(d, args...);
    return launch_one<8, KMAX>(d, args...);
}

}  // namespace
}  // namespace moe

extern "C" int moe_combine_backward(const moe_problem *p, const void *y, const void *d_out, const int32_t *topk_idx,
                                    const float *topk_w, const int32_t *slot, void *d_y, float *d_topk_w,
                                    void *stream) {
    using namespace moe;
    Dims d;
    int rc = check_problem(p, &d);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    if (!y || !d_out || !topk_idx || !topk_w || !slot || !d_y || !d_topk_w) return MOE_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(d_out, 16) || !aligned(d_y, 16) || !aligned(topk_idx, 4) ||
        !aligned(topk_w, 4) || !aligned(slot, 4) || !aligned(d_topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    if (d.k <= 2) return launch_k<2>(d, st, y, d_out, topk_idx, topk_w, slot, d_y, d_topk_w);
    if (d.k <= 8) return launch_k<8>(d, st, y, d_out, topk_idx, topk_w, slot, d_y, d_topk_w);
    return launch_k<16>(d, st, y, d_out, topk_idx, topk_w, slot, d_y, d_topk_w);
}

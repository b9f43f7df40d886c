// moe_norm.cu -- the norms around a block of the residual stream, fused with the
// block's gate and residual scale, alone or behind the combine; and their gradient.
//
//   b = y  or  N(y; w_post)          N(v; w) = v (mean(v^2) + eps)^(-1/2) w
//   r = residual + a g b             g: 1, a factor for each channel or for each token
//   n = N(r; w_pre)
//
// y is read (moe_block_norm) or formed as the combine forms it (moe_combine_norm). Everything
// between the loads and the stores is fp32: n comes from the r before it is rounded.
//
// Gradient, with ^ for a row divided by its root mean square and 1/s for that root's inverse:
//   D   = d_r + (w_pre d_n - r^ mean(r^ w_pre d_n)) / s_r                 = d_residual
//   d_y = (w_post c - y^ mean(y^ w_post c)) / s_y,  c = a g D
//   d_w_pre = sum_t d_n r^    d_w_post = sum_t c y^    d_gate = a sum D b  (over t, or over h)
// Both norms' statistics come from the row itself again, which is in shared memory: the forward
// pass keeps nothing but y and r. The second mean, over D, is taken from sums of its parts,
//   sum y w_post g D = sum y w_post g d_r + 1/s_r (sum y w_post g w_pre d_n - 1/s_r mean sum y w_post g r),
// so that one sum over the block makes all of a row's means.
//
// All of it is bound by HBM where there are many rows, and by a launch and two sums over a block
// where there are few. us on GB300, call behind call on inputs in turn (floor: bytes at the measured copy rate):
//   norm, 1 x 7168                           5.2  (2.9 in a graph; launch, load, two sums, store)
//   norm, 16384 x 7168, bf16               156    (floor 140; a copy and two sums a row)
//   combine and norm, 1024 x 7168, top-8    34.8  (floor 24)
//   gradient, 4096 x 7168, channel gate     74    (floor 53)
//   gradient, 16381 x 4096, no norm after  129    (floor 120)
// The norm of the stream alone (no y) takes a row straight into registers whatever the number of rows: 16384 x 7168 in 170,
// with a floor of 70.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kNormMaxHidden = 16384;
constexpr int kNormMaxDepth = 4;                   // rows on their way or at hand in a ring
// Threads of the ring kernel on an SM: so many warps that one row's sums leave others to run.
constexpr int kNormThreadsPerSM = 1024;
constexpr int kCombineSlots = 16, kCombineSmem = 160 * 1024;       // experts' rows in a ring

struct NormArgs {
    int T, H8, k, C;                   // H8 chunks of 8 elements to a row
    float eps, scale, inv_h;
    int channel, token;                // the gate's kind
};

// Eight elements of a row as they are stored, and as fp32.
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    uint4 a;
};
template <>
struct Raw8<true> {
    uint4 a, b;
};
// fp32 in pairs: a product or a sum of two is one instruction.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ void to_floats(const Raw8<false> &v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}
__device__ __forceinline__ void to_floats(const Raw8<true> &v, float2 (&f)[4]) {
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
// Chunk c of a row that is read once. Not volatile as ld_stream_v4 is, whose loads of a token's rows would not all be under
// way at once (combine and norm, 237 x 2056, top-6: 6.6 us instead of 4.6): the row's pointer has to come from
// pdl_enter_before().
__device__ __forceinline__ void load_row8(const void *row, int c, Raw8<false> &v) {
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w)
        : "l"(static_cast<const uint4 *>(row) + c));
}
// The residual's: the same memory may be written as r, by the thread that read it.
__device__ __forceinline__ uint4 ld_once_v4(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void load_residual8(const void *row, int c, Raw8<false> &v) {
    v.a = ld_once_v4(static_cast<const uint4 *>(row) + c);
}
__device__ __forceinline__ void load_residual8(const void *row, int c, Raw8<true> &v) {
    v.a = ld_once_v4(static_cast<const uint4 *>(row) + 2 * c);
    v.b = ld_once_v4(static_cast<const uint4 *>(row) + 2 * c + 1);
}
// Chunk c of a vector that every row uses.
__device__ __forceinline__ void load_param8(const void *p, int c, Raw8<false> &v) {
    v.a = __ldg(static_cast<const uint4 *>(p) + c);
}
__device__ __forceinline__ void load_param8(const void *p, int c, Raw8<true> &v) {
    v.a = __ldg(static_cast<const uint4 *>(p) + 2 * c);
    v.b = __ldg(static_cast<const uint4 *>(p) + 2 * c + 1);
}
// The same where it is not to stay in registers from row to row: volatile.
__device__ __forceinline__ uint4 ld_again_v4(const uint4 *p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ void load_param8_again(const void *p, int c, Raw8<false> &v) {
    v.a = ld_again_v4(static_cast<const uint4 *>(p) + c);
}
__device__ __forceinline__ void load_param8_again(const void *p, int c, Raw8<true> &v) {
    v.a = ld_again_v4(static_cast<const uint4 *>(p) + 2 * c);
    v.b = ld_again_v4(static_cast<const uint4 *>(p) + 2 * c + 1);
}
template <bool F32>
__device__ __forceinline__ void store8(void *row, int c, const float2 (&f)[4]) {
    if constexpr (F32) {
        uint4 *o = static_cast<uint4 *>(row) + 2 * c;
        st_v4(o, make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y)));
        st_v4(o + 1, make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y)));
    } else {
        st_v4(static_cast<uint4 *>(row) + c, make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                                        pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y)));
    }
}

// Sums of N values over the block, every thread the same result: by a butterfly over the warp,
// then by one over the warps' sums. `turn` alternates between two buffers: a thread writes to one
// again only behind the next sum's barrier, which all reach after reading it.
template <int N>
struct BlockSum {
    float part[2][N][32];
};
// `threads`: the block's first ones, whole warps, which alone come here.
template <int N>
__device__ __forceinline__ void block_sum(BlockSum<N> &s, float (&v)[N], unsigned &turn, int threads) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = threads >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
    if (warps == 1) return;
    const unsigned b = turn & 1u;
    ++turn;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s.part[b][i][warp] = v[i];
    }
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < warps ? s.part[b][i][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
    }
}

// The sum over the block where a thread holds two chunks of a row, `threads` apart (a: from the first, b: from the second),
// in the order that block_sum has with one chunk to a thread: 32 neighbouring chunks by a butterfly, a half of the lanes for
// each of a warp's two, then those sums. A row's sum is then the same in the kernel that has one chunk to a thread, so that
// the number of rows, by which the kernel is chosen, leaves a row's results as they are. 2 to 16 warps.
__device__ __forceinline__ float block_sum_pairs(BlockSum<1> &s, float a, float b, unsigned &turn, int threads) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = threads >> 5;
    float x = lane & 16 ? b : a;
    x += __shfl_xor_sync(kFull, lane & 16 ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    const unsigned at = turn & 1u;
    ++turn;
    if ((lane & 15) == 0) s.part[at][0][(lane >> 4) * warps + warp] = x;
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
    x = lane < 2 * warps ? s.part[at][0][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}
// A row's sum of squares from a thread's: PAIRS, of each of its two chunks.
template <bool PAIRS>
__device__ __forceinline__ float row_sum(BlockSum<1> &s, const float2 (&sq)[PAIRS ? 2 : 1], unsigned &turn, int threads) {
    if constexpr (PAIRS) {
        return block_sum_pairs(s, __fadd_rn(sq[0].x, sq[0].y), __fadd_rn(sq[1].x, sq[1].y), turn, threads);
    } else {
        float f[1] = {__fadd_rn(sq[0].x, sq[0].y)};
        block_sum(s, f, turn, threads);
        return f[0];
    }
}

// Sums of eight values over the block: over the warp by halves, four values to a lane after one exchange, two after the
// next, one after three, which takes 9 shuffles instead of 40; then over the warps, a lane to a value of a warp.
struct BlockSum8 {
    float part[2][32][8];
};
__device__ __forceinline__ void block_sum8(BlockSum8 &s, float (&v)[8], unsigned &turn) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float a[4], b[2], x;
    // lanes with bit 2 go on with values 4 to 7, the others with 0 to 3; then bits 1 and 0 choose among those
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = lane & 4 ? v[4 + i] : v[i];
        a[i] += __shfl_xor_sync(kFull, lane & 4 ? v[i] : v[4 + i], 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        b[i] = lane & 2 ? a[2 + i] : a[i];
        b[i] += __shfl_xor_sync(kFull, lane & 2 ? a[i] : a[2 + i], 2);
    }
    x = lane & 1 ? b[1] : b[0];
    x += __shfl_xor_sync(kFull, lane & 1 ? b[0] : b[1], 1);
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
    if (warps > 1) {
        const unsigned at = turn & 1u;
        ++turn;
        if (lane < 8) s.part[at][warp][lane] = x;
        __syncthreads();
        x = 0.0f;
        for (int i = lane >> 3; i < warps; i += 4) x += s.part[at][i][lane & 7];
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(kFull, x, i);
}

__device__ __forceinline__ float inv_rms(float sum_sq, const NormArgs &a) {
    return __frsqrt_rn(__fmaf_rn(sum_sq, a.inv_h, a.eps));
}

// From the block's output v, of which a thread has NC chunks of 8 elements in registers, and the residual to r and n. g: the
// scale and a token's gate. param(k, c): chunk c of w_post (k = 0), of the gate for each channel (1) or of w_pre (2). PAIRS:
// the sums in the order of one chunk to a thread.
template <bool HAS_Y, bool RES32, int NC, bool PAIRS, typename Param>
__device__ __forceinline__ void finish_row(const NormArgs &a, int t, float g, float2 (&v)[NC][4], const Raw8<RES32> (&res)[NC],
                                           bool w_post, bool w_pre, Param param, void *r_out, void *n_out, BlockSum<1> &sums,
                                           unsigned &turn, int threads) {
    const size_t res_row = (size_t)a.H8 * (RES32 ? 32 : 16), bf_row = (size_t)a.H8 * 16;
    const auto times = [&](int k, int c, float2 (&f)[4]) {
        float2 p[4];
        to_floats(param(k, c), p);
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = mul2(f[q], p[q]);
    };
    constexpr int kSums = PAIRS ? 2 : 1;
    float2 sq[kSums];
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < kSums; ++i) sq[i] = both(0.0f);
    };
    clear();
    if (HAS_Y && w_post) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (i * threads + (int)threadIdx.x < a.H8)
#pragma unroll
                for (int q = 0; q < 4; ++q) sq[i % kSums] = fma2(v[i][q], v[i][q], sq[i % kSums]);
        g = __fmul_rn(g, inv_rms(row_sum<PAIRS>(sums, sq, turn, threads), a));
    }
    clear();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = i * threads + (int)threadIdx.x;
        if (c < a.H8) {
            float2 x[4];
            to_floats(res[i], x);
            if constexpr (HAS_Y) {
                if (w_post) times(0, c, v[i]);
                if (a.channel) times(1, c, v[i]);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = fma2(v[i][q], both(g), x[q]);
            }
            if (r_out) store8<RES32>(static_cast<char *>(r_out) + t * res_row, c, x);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                sq[i % kSums] = fma2(x[q], x[q], sq[i % kSums]);
                v[i][q] = x[q];
            }
        }
    }
    if (!w_pre) return;
    const float s = inv_rms(row_sum<PAIRS>(sums, sq, turn, threads), a);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = i * threads + (int)threadIdx.x;
        if (c < a.H8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], both(s));
            times(2, c, v[i]);
            store8<false>(static_cast<char *>(n_out) + t * bf_row, c, v[i]);
        }
    }
}

// moe_block_norm for few rows, or very long ones: a block takes a row at a time, NC chunks of 8 elements to a thread,
// straight into registers, which has the shortest chain: no ring to set up, the vectors' loads beside the row's.
// HAS_Y: there is a block before the norm.
template <bool HAS_Y, bool RES32, bool PAR32, int NC>
__global__ void __launch_bounds__(1024)
norm_kernel(NormArgs a, const void *__restrict__ y, const void *residual, const void *__restrict__ w_post,
            const void *__restrict__ w_pre, const void *__restrict__ gate, void *r_out, void *n_out) {
    // one chunk to a thread: the vectors come along with the first row, and stay
    constexpr bool kHold = NC == 1;
    __shared__ BlockSum<1> sums;
    pdl_enter_before(y);
    unsigned turn = 0;
    const size_t res_row = (size_t)a.H8 * (RES32 ? 32 : 16), bf_row = (size_t)a.H8 * 16;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        int c[NC];
        Raw8<RES32> res[NC];
        Raw8<false> yy[NC];
        Raw8<PAR32> p_post, p_pre, p_gate;
        float2 v[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            c[i] = i * (int)blockDim.x + (int)threadIdx.x;
            if (c[i] < a.H8) {
                load_residual8(static_cast<const char *>(residual) + t * res_row, c[i], res[i]);
                if (HAS_Y) load_row8(static_cast<const char *>(y) + t * bf_row, c[i], yy[i]);
            }
        }
        if constexpr (kHold) {
            if (c[0] < a.H8) {
                if (HAS_Y && w_post) load_param8(w_post, c[0], p_post);
                if (HAS_Y && a.channel) load_param8(gate, c[0], p_gate);
                if (w_pre) load_param8(w_pre, c[0], p_pre);
            }
        }
        float g = a.scale;
        if (HAS_Y && a.token) g = __fmul_rn(g, __ldg(static_cast<const float *>(gate) + t));
        if constexpr (HAS_Y) {
#pragma unroll
            for (int i = 0; i < NC; ++i) to_floats(yy[i], v[i]);
        }
        const auto param = [&](int k, int ch) {
            if constexpr (kHold) {
                return k == 0 ? p_post : k == 1 ? p_gate : p_pre;
            } else {
                Raw8<PAR32> raw;
                load_param8_again(k == 0 ? w_post : k == 1 ? gate : w_pre, ch, raw);
                return raw;
            }
        };
        finish_row<HAS_Y, RES32, NC, false>(a, t, g, v, res, w_post != nullptr, w_pre != nullptr, param, r_out, n_out, sums, turn, (int)blockDim.x);
    }
}

// The kept choices of a token, in order.
struct Choices {
    int n;
    float w[kMaxTopK];
    size_t at[kMaxTopK];                             // bytes from y to the row
};
// Lane j < k of one warp: choice j of a token; none past the last token.
struct Choice {
    int s, e;
    float w;
};
__device__ __forceinline__ Choice load_choice(const NormArgs &a, const int32_t *topk_idx, const float *topk_w, const int32_t *slot,
                                              long long t) {
    const int lane = threadIdx.x & 31;
    Choice c = {-1, 0, 0.0f};
    if (lane < a.k && t < a.T) {
        c.s = __ldg(slot + t * a.k + lane);
        c.e = __ldg(topk_idx + t * a.k + lane);
        c.w = __ldg(topk_w + t * a.k + lane);
    }
    return c;
}
__device__ __forceinline__ void put_choices(const NormArgs &a, const Choice &c, Choices &to) {
    const int lane = threadIdx.x & 31;
    const unsigned kept = __ballot_sync(kFull, c.s >= 0);
    if (c.s >= 0) {
        const int j = __popc(kept & ((1u << lane) - 1u));
        to.w[j] = c.w;
        to.at[j] = (size_t)(c.e * a.C + c.s) * ((size_t)a.H8 * 16);
    }
    if (lane == 0) to.n = __popc(kept);
}

// moe_combine_norm: the same behind the weighted sum of SRC experts' rows at a time, a token after the other, whose
// choices are loaded a token ahead. Few tokens or short rows: all of a token's rows are asked for at once. 237 x 2056,
// top-6: 7.2 us, 4.6 in a graph.
template <int SRC, bool RES32, bool PAR32, int NC, int MAXT>
__global__ void __launch_bounds__(MAXT)
combine_norm_kernel(NormArgs a, const void *__restrict__ y, const int32_t *__restrict__ topk_idx,
                    const float *__restrict__ topk_w, const int32_t *__restrict__ slot, const void *residual,
                    const void *__restrict__ w_post, const void *__restrict__ w_pre, const void *__restrict__ gate, void *out,
                    void *r_out, void *n_out) {
    __shared__ Choices choices[2];
    __shared__ BlockSum<1> sums;
    const size_t res_row = (size_t)a.H8 * (RES32 ? 32 : 16), bf_row = (size_t)a.H8 * 16;
    pdl_enter_before(y, topk_idx, topk_w, slot);
    if (threadIdx.x < 32) put_choices(a, load_choice(a, topk_idx, topk_w, slot, blockIdx.x), choices[0]);
    __syncthreads();
    unsigned turn = 0, at = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, at ^= 1u) {
        const Choices &now = choices[at];
        Raw8<RES32> res[NC];
        float2 v[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i * (int)blockDim.x + (int)threadIdx.x;
            if (c < a.H8) load_residual8(static_cast<const char *>(residual) + t * res_row, c, res[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = both(0.0f);
        }
        for (int j0 = 0; j0 < now.n; j0 += SRC) {                      // once, or more past SRC choices
            Raw8<false> in[SRC][NC];
#pragma unroll
            for (int j = 0; j < SRC; ++j)
                if (j0 + j < now.n)
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int c = i * (int)blockDim.x + (int)threadIdx.x;
                        if (c < a.H8) load_row8(static_cast<const char *>(y) + now.at[j0 + j], c, in[j][i]);
                    }
#pragma unroll
            for (int j = 0; j < SRC; ++j) {
                if (j0 + j < now.n) {
                    const float w = now.w[j0 + j];
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        float2 f[4];
                        to_floats(in[j][i], f);
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[i][q] = fma2(both(w), f[q], v[i][q]);
                    }
                }
            }
        }
        // the other buffer was last read before the barriers of the token before
        if (threadIdx.x < 32) put_choices(a, load_choice(a, topk_idx, topk_w, slot, (long long)t + gridDim.x), choices[at ^ 1u]);
        float g = a.scale;
        if (a.token) g = __fmul_rn(g, __ldg(static_cast<const float *>(gate) + t));
        if (out != nullptr) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * (int)blockDim.x + (int)threadIdx.x;
                if (c < a.H8) store8<false>(static_cast<char *>(out) + t * bf_row, c, v[i]);
            }
        }
        const auto param = [&](int k, int ch) {
            Raw8<PAR32> raw;
            load_param8_again(k == 0 ? w_post : k == 1 ? gate : w_pre, ch, raw);
            return raw;
        };
        finish_row<true, RES32, NC, false>(a, t, g, v, res, w_post != nullptr, w_pre != nullptr, param, r_out, n_out, sums, turn, (int)blockDim.x);
        if ((!w_post && !w_pre) || blockDim.x == 32) __syncthreads();  // the choices' buffers turn behind a barrier
    }
}

// The same for many tokens. The block's last warp sees to the tokens' choices and to the experts' rows, which come by bulk
// copies into a ring of `slots` rows, tokens ahead; the others add each row as it arrives. (Loads to registers a token ahead
// would fill the SM's load queue, behind which the sums' shared memory accesses then wait: 48 us for 1024 x 7168, top-8,
// where this takes 35 and the kernel above 45.)
template <bool RES32, bool PAR32, int NC>
__global__ void __launch_bounds__(544, NC == 4 ? 1 : 2)
combine_norm_rows_kernel(NormArgs a, const void *__restrict__ y, const int32_t *__restrict__ topk_idx,
                         const float *__restrict__ topk_w, const int32_t *__restrict__ slot, const void *residual,
                         const void *__restrict__ w_post, const void *__restrict__ w_pre, const void *__restrict__ gate,
                         void *out, void *r_out, void *n_out, int slots, unsigned *status) {
    constexpr int kAhead = 4;                                          // tokens whose choices are at hand
    extern __shared__ __align__(128) char norm_ring[];
    __shared__ __align__(8) uint64_t full[kCombineSlots], empty[kCombineSlots], known[kAhead], done[kAhead];
    __shared__ Choices choices[kAhead];
    __shared__ BlockSum<1> sums;
    const int tid = threadIdx.x, threads = (int)blockDim.x - 32, lane = tid & 31;
    const unsigned bf_row = (unsigned)a.H8 * 16u;
    const size_t res_row = (size_t)a.H8 * (RES32 ? 32 : 16);
    if (tid < slots) {
        mbar_init(&full[tid], 1u);
        mbar_init(&empty[tid], threads >> 5);
        fence_mbar_init();
    }
    if (tid < kAhead) {
        mbar_init(&known[tid], 1u);
        mbar_init(&done[tid], threads >> 5);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter_before(topk_idx, topk_w, slot);
    bool alive = true;
    const auto wait = [&](uint64_t *bar, unsigned use) {               // one warp, all lanes
        if (alive && !__all_sync(kFull, mbar_wait_bounded(bar, use & 1u))) {
            alive = false;                           // outputs stay wrong; the barriers below still meet
            if (lane == 0) atomicOr(status, kStatusWaitGaveUp);
        }
    };
    if (tid >= threads) {
        unsigned n_token = 0, n_row = 0, s = 0, use = 0;
        Choice next = load_choice(a, topk_idx, topk_w, slot, blockIdx.x);
        for (long long t = blockIdx.x; t < a.T; t += gridDim.x, ++n_token) {
            const unsigned at = n_token % kAhead;
            if (n_token >= kAhead) wait(&done[at], n_token / kAhead - 1u);
            const Choice now = next;
            next = load_choice(a, topk_idx, topk_w, slot, t + gridDim.x);
            put_choices(a, now, choices[at]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&known[at]);
            const int n = choices[at].n;
            for (int j = 0; j < n && alive; ++j, ++n_row) {
                if (n_row >= (unsigned)slots) wait(&empty[s], use - 1u);
                if (alive && lane == 0) {
                    mbar_expect_tx(&full[s], bf_row);
                    bulk_g2s(norm_ring + (size_t)s * bf_row, static_cast<const char *>(y) + choices[at].at[j], bf_row, &full[s]);
                }
                if (++s == (unsigned)slots) {
                    s = 0;
                    ++use;
                }
            }
        }
        // no copy outlives the block
        for (unsigned i = n_row > (unsigned)slots ? n_row - slots : 0u; i < n_row; ++i)
            mbar_wait_bounded(&full[i % (unsigned)slots], (i / (unsigned)slots) & 1u);
        return;
    }
    unsigned turn = 0, s = 0, use = 0, n_token = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, ++n_token) {
        const unsigned at = n_token % kAhead;
        Raw8<RES32> res[NC];
        float2 v[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i * threads + tid;
            if (c < a.H8) load_residual8(static_cast<const char *>(residual) + t * res_row, c, res[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = both(0.0f);
        }
        wait(&known[at], n_token / kAhead);
        const int n = alive ? choices[at].n : 0;
        for (int j = 0; j < n; ++j) {
            const float w = choices[at].w[j];
            wait(&full[s], use);
            const char *in = norm_ring + (size_t)s * bf_row;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * threads + tid;
                if (c < a.H8) {
                    float2 f[4];
                    to_floats(*reinterpret_cast<const Raw8<false> *>(in + (size_t)c * 16), f);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = fma2(both(w), f[q], v[i][q]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == (unsigned)slots) {
                s = 0;
                ++use;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&done[at]);
        float g = a.scale;
        if (a.token) g = __fmul_rn(g, __ldg(static_cast<const float *>(gate) + t));
        if (out != nullptr) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * threads + tid;
                if (c < a.H8) store8<false>(static_cast<char *>(out) + (size_t)t * bf_row, c, v[i]);
            }
        }
        const auto param = [&](int k, int ch) {
            Raw8<PAR32> raw;
            load_param8_again(k == 0 ? w_post : k == 1 ? gate : w_pre, ch, raw);
            return raw;
        };
        finish_row<true, RES32, NC, NC == 2>(a, t, g, v, res, w_post != nullptr, w_pre != nullptr, param, r_out, n_out, sums, turn, threads);
    }
}

// moe_block_norm for many rows. A block of threads takes a row at a time, NC chunks of 8 elements to a thread; the rows of
// y and of the residual come by bulk copies into a ring, `depth` rows deep, so that loads run on while a row's sums meet:
// 4864 x 7168 in 52 us, straight into registers 87.
template <bool RES32, bool PAR32, int NC>
__global__ void __launch_bounds__(512, 2)
norm_rows_kernel(NormArgs a, const void *y, const void *residual, const void *__restrict__ w_post,
                 const void *__restrict__ w_pre, const void *__restrict__ gate, void *r_out, void *n_out, int depth,
                 unsigned *status) {
    extern __shared__ __align__(128) char norm_ring[];
    __shared__ __align__(8) uint64_t full[kNormMaxDepth];
    __shared__ BlockSum<1> sums;
    constexpr int kSums = NC == 2 ? 2 : 1;
    const int tid = threadIdx.x;
    const unsigned bf_row = (unsigned)a.H8 * 16u, res_row = RES32 ? 2u * bf_row : bf_row, stage = bf_row + res_row;
    if (tid < depth) {
        mbar_init(&full[tid], 1u);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();
    bool alive = true;
    unsigned fetched = 0;
    const auto fetch = [&](unsigned s) {             // thread 0
        const long long row = blockIdx.x + (long long)fetched * gridDim.x;
        if (row >= a.T || !alive) return;
        char *to = norm_ring + (size_t)s * stage;
        mbar_expect_tx(&full[s], stage);
        bulk_g2s(to, static_cast<const char *>(y) + (size_t)row * bf_row, bf_row, &full[s]);
        bulk_g2s(to + bf_row, static_cast<const char *>(residual) + (size_t)row * res_row, res_row, &full[s]);
        ++fetched;
    };
    if (tid == 0)
        for (int i = 0; i < depth; ++i) fetch(i);
    unsigned turn = 0, n_row = 0, lost = 0, s = 0, parity = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, ++n_row) {
        if (alive && !mbar_wait_bounded(&full[s], parity)) {
            alive = false;                           // outputs stay wrong; the barriers below still meet
            lost = n_row;
            atomicOr(status, kStatusWaitGaveUp);
        }
        const char *in = norm_ring + (size_t)s * stage;
        Raw8<false> yy[NC];
        Raw8<RES32> res[NC];
        float2 sq[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) sq[i] = both(0.0f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i * (int)blockDim.x + tid;
            if (c < a.H8) {
                yy[i] = *reinterpret_cast<const Raw8<false> *>(in + (size_t)c * 16);
                res[i] = *reinterpret_cast<const Raw8<RES32> *>(in + bf_row + (size_t)c * sizeof(Raw8<RES32>));
                float2 v[4];
                to_floats(yy[i], v);
#pragma unroll
                for (int q = 0; q < 4; ++q) sq[i % kSums] = fma2(v[q], v[q], sq[i % kSums]);
            }
        }
        float g = a.scale;
        if (a.token) g = __fmul_rn(g, __ldg(static_cast<const float *>(gate) + t));
        if (w_post) {
            g = __fmul_rn(g, inv_rms(row_sum<NC == 2>(sums, sq, turn, (int)blockDim.x), a));
        } else {
            __syncthreads();
        }
        if (blockDim.x == 32) __syncwarp();
        if (tid == 0) fetch(s);                      // all have read the row's place in the ring
        if (++s == (unsigned)depth) {
            s = 0;
            parity ^= 1u;
        }
        float2 v[NC][4];
#pragma unroll
        for (int i = 0; i < kSums; ++i) sq[i] = both(0.0f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i * (int)blockDim.x + tid;
            if (c < a.H8) {
                float2 x[4];
                to_floats(yy[i], v[i]);
                to_floats(res[i], x);
                if (w_post) {
                    Raw8<PAR32> w;
                    float2 p[4];
                    load_param8(w_post, c, w);
                    to_floats(w, p);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], p[q]);
                }
                if (a.channel) {
                    Raw8<PAR32> w;
                    float2 p[4];
                    load_param8(gate, c, w);
                    to_floats(w, p);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], p[q]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[i][q] = fma2(v[i][q], both(g), x[q]);
                    sq[i % kSums] = fma2(v[i][q], v[i][q], sq[i % kSums]);
                }
                if (r_out) store8<RES32>(static_cast<char *>(r_out) + (size_t)t * res_row, c, v[i]);
            }
        }
        if (w_pre) {
            const float by = inv_rms(row_sum<NC == 2>(sums, sq, turn, (int)blockDim.x), a);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * (int)blockDim.x + tid;
                if (c < a.H8) {
                    Raw8<PAR32> w;
                    float2 p[4];
                    load_param8(w_pre, c, w);
                    to_floats(w, p);
#pragma unroll
                    for (int q = 0; q < 4; ++q) p[q] = mul2(mul2(v[i][q], both(by)), p[q]);
                    store8<false>(static_cast<char *>(n_out) + (size_t)t * bf_row, c, p);
                }
            }
        }
    }
    if (tid == 0 && !alive)                          // no copy outlives the block
        for (; lost < fetched; ++lost) mbar_wait_bounded(&full[lost % (unsigned)depth], (lost / (unsigned)depth) & 1u);
}

struct NormPtrs {
    const void *y;
    const int32_t *idx;
    const float *w;
    const int32_t *slot;
    const void *residual, *w_post, *w_pre, *gate;
    void *out, *r, *n;
};

template <bool HAS_Y, bool RES32, bool PAR32, int NC>
int launch_norm(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    const int threads = ((a.H8 + NC - 1) / NC + 31) / 32 * 32;
    // blocks do not wait on one another: a few more than an SM holds even out its end
    const int grid = persistent_grid(d.T, sm_count() * std::min(32, 2048 / threads), d.max_blocks);
    return launch_pdl(norm_kernel<HAS_Y, RES32, PAR32, NC>, grid, threads, st, a, p.y, p.residual, p.w_post, p.w_pre, p.gate,
                      p.r, p.n) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
template <bool HAS_Y, bool RES32, bool PAR32>
int launch_norm_nc(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    if (a.H8 <= 1024) return launch_norm<HAS_Y, RES32, PAR32, 1>(d, a, st, p);
    return launch_norm<HAS_Y, RES32, PAR32, 2>(d, a, st, p);
}
template <int SRC, bool RES32, bool PAR32, int NC, int MAXT>
int launch_combine_norm(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    const int threads = ((a.H8 + NC - 1) / NC + 31) / 32 * 32;
    const int grid = persistent_grid(d.T, sm_count() * std::min(32, 2048 / threads), d.max_blocks);
    return launch_pdl(combine_norm_kernel<SRC, RES32, PAR32, NC, MAXT>, grid, threads, st, a, p.y, p.idx, p.w, p.slot, p.residual,
                      p.w_post, p.w_pre, p.gate, p.out, p.r, p.n) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
template <int SRC, bool RES32, bool PAR32>
int launch_combine_norm_nc(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    if (a.H8 <= 512) return launch_combine_norm<SRC, RES32, PAR32, 1, 512>(d, a, st, p);
    if (a.H8 <= 1024) return launch_combine_norm<SRC, RES32, PAR32, 1, 1024>(d, a, st, p);
    return launch_combine_norm<(SRC < 4 ? SRC : 4), RES32, PAR32, 4, 512>(d, a, st, p);
}
template <bool RES32, bool PAR32, int NC>
int launch_combine_norm_rows(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    const auto kernel = combine_norm_rows_kernel<RES32, PAR32, NC>;
    const int threads = ((a.H8 + NC - 1) / NC + 31) / 32 * 32 + 32, row = d.H * 2;
    int per_sm = std::max(1, std::min(16, 1088 / threads));
    while (per_sm > 1 && kCombineSmem / per_sm / row < 4) --per_sm;
    const int slots = std::min(kCombineSlots, kCombineSmem / per_sm / row);
    static PerContext<int> smem_done;
    if (!set_smem_once(smem_done, kernel, kCombineSmem)) return MOE_ERR_CUDA;
    unsigned *status = device_status_word();
    if (status == nullptr) return MOE_ERR_CUDA;
    const int grid = persistent_grid(d.T, sm_count() * per_sm, d.max_blocks);
    return launch_pdl_smem(kernel, grid, threads, (size_t)slots * row, st, a, p.y, p.idx, p.w, p.slot, p.residual, p.w_post,
                           p.w_pre, p.gate, p.out, p.r, p.n, slots, status) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
template <bool RES32, bool PAR32>
int launch_combine_norm_k(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    // the ring, where a block has several tokens and a row is long. us, direct and ring, with 2 choices a token: 304 tokens of
    // 2048 channels, 3.7 and 3.9; 4096 of 2048, 21 and 28; 304 of 4096, 4.4 and 4.9; 4096 of 4096, 48 and 40; with 8: 4096 of
    // 2048, 49 and 51; 304 of 4096, 8.0 and 6.8; 304 of 7168, 11.4 and 8.5; 4096 of 7168, 146 and 104; of 16384, 273 and 254.
    if (d.T >= 2 * 152 && a.H8 > 256) {
        if (a.H8 <= 1024) return launch_combine_norm_rows<RES32, PAR32, 2>(d, a, st, p);
        return launch_combine_norm_rows<RES32, PAR32, 4>(d, a, st, p);
    }
    if (d.k <= 2) return launch_combine_norm_nc<2, RES32, PAR32>(d, a, st, p);
    if (d.k <= 4) return launch_combine_norm_nc<4, RES32, PAR32>(d, a, st, p);
    return launch_combine_norm_nc<8, RES32, PAR32>(d, a, st, p);
}

// Where the ring pays, with a block's output of its own: from about four rows to an SM on, up to 8192 channels. us, direct
// and ring: 304 rows of 2048, 2.9 and 3.2; 608, 3.4 and 3.5; 4864, 17.2 and 16.5; 608 of 7168, 9.7 and 7.7; 2432, 44 and 30;
// 608 of 16384 (a ring of two rows at most), 14.7 and 16.7; 4864, 130 and 138.
bool norm_many_rows(const Dims &d) { return d.T >= 4 * 152 && d.H <= 8192; }

template <bool RES32, bool PAR32, int NC>
int launch_norm_rows(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    const auto kernel = norm_rows_kernel<RES32, PAR32, NC>;
    constexpr int kMaxSmem = 200 * 1024;
    const int threads = ((a.H8 + NC - 1) / NC + 31) / 32 * 32, row = d.H * (RES32 ? 6 : 4);
    int per_sm = std::max(1, std::min(16, kNormThreadsPerSM / threads));
    while (per_sm > 1 && kMaxSmem / per_sm / row < 2) --per_sm;
    const int depth = std::max(1, std::min(kNormMaxDepth, kMaxSmem / per_sm / row));
    static PerContext<int> smem_done;
    if (!set_smem_once(smem_done, kernel, kMaxSmem)) return MOE_ERR_CUDA;
    unsigned *status = device_status_word();
    if (status == nullptr) return MOE_ERR_CUDA;
    const int grid = persistent_grid(d.T, sm_count() * per_sm, d.max_blocks);
    return launch_pdl_smem(kernel, grid, threads, (size_t)depth * row, st, a, p.y, p.residual, p.w_post, p.w_pre, p.gate, p.r,
                           p.n, depth, status) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}
template <bool RES32, bool PAR32>
int launch_norm_rows_nc(const Dims &d, const NormArgs &a, cudaStream_t st, const NormPtrs &p) {
    if (a.H8 <= 256) return launch_norm_rows<RES32, PAR32, 1>(d, a, st, p);
    return launch_norm_rows<RES32, PAR32, 2>(d, a, st, p);
}
// By the types that the call names: f(residual fp32, parameters fp32).
template <typename F>
int by_types(const moe_norm *n, F f) {
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    const bool res = n->residual_type == MOE_VALUE_F32, par = n->param_type == MOE_VALUE_F32;
    if (res) return par ? f(yes, yes) : f(yes, no);
    return par ? f(no, yes) : f(no, no);
}

int check_norm(const Dims &d, const moe_norm *n, NormArgs *a) {
    if (n == nullptr) return MOE_ERR_INVALID_ARG;
    if (n->branch_gate < MOE_BRANCH_PLAIN || n->branch_gate > MOE_BRANCH_TOKEN) return MOE_ERR_INVALID_ARG;
    if (n->residual_type != MOE_VALUE_BF16 && n->residual_type != MOE_VALUE_F32) return MOE_ERR_INVALID_ARG;
    if (n->param_type != MOE_VALUE_BF16 && n->param_type != MOE_VALUE_F32) return MOE_ERR_INVALID_ARG;
    if (!(n->eps > 0.0f && n->eps <= 3.4028234e38f) || !(fabsf(n->scale) <= 3.4028234e38f)) return MOE_ERR_INVALID_ARG;
    if (d.H > kNormMaxHidden) return MOE_ERR_UNSUPPORTED;
    a->T = d.T;
    a->H8 = d.H / 8;
    a->k = d.k;
    a->C = d.C;
    a->eps = n->eps;
    a->scale = n->scale;
    a->inv_h = 1.0f / (float)d.H;
    a->channel = n->branch_gate == MOE_BRANCH_CHANNEL;
    a->token = n->branch_gate == MOE_BRANCH_TOKEN;
    return MOE_OK;
}

// What the two forward calls have in common; has_y: there is a block's output.
int check_forward(const moe_norm *n, bool has_y, const NormPtrs &p) {
    if (!p.residual || (!p.r && !p.n)) return MOE_ERR_INVALID_ARG;
    if ((p.w_pre != nullptr) != (p.n != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!has_y && (p.w_post || n->branch_gate != MOE_BRANCH_PLAIN || p.r)) return MOE_ERR_INVALID_ARG;
    if ((p.gate != nullptr) != (n->branch_gate != MOE_BRANCH_PLAIN)) return MOE_ERR_INVALID_ARG;
    if (!aligned(p.y, 16) || !aligned(p.residual, 16) || !aligned(p.w_post, 16) || !aligned(p.w_pre, 16) ||
        !aligned(p.gate, n->branch_gate == MOE_BRANCH_TOKEN ? 4 : 16) || !aligned(p.out, 16) || !aligned(p.r, 16) ||
        !aligned(p.n, 16))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// ---- gradient -----------------------------------------------------------------

struct NormBwdPtrs {
    const void *y, *r, *d_r, *d_n, *w_post, *w_pre, *gate;
    void *d_y, *d_residual;
    float *d_gate_token, *part;
    unsigned *status;
};

// A block takes the rows of one part (rows p, p + parts, ...) at a time and keeps that part's column
// sums in registers: NC chunks of 8 columns to a thread. The rows of y, r, d_r and d_n come by
// bulk copies into a ring, `depth` rows deep, so that loads run on while a row's sums meet; they are
// read there again for the second of the two passes over a row, which leaves registers for the column sums. One sum over the
// block a row, of six values: with a second one for the mean over D, and a third pass behind it, 4096 x 7168 takes 85 us, so 74.
// DOTS: that mean, or a token's gate's gradient, is wanted. (Known when compiled: its six sums would cost the other kernel
// spills, 16381 x 4096 without a norm after the block in 160 us instead of 129.) Bound by the chain of a row's passes, one row of 7168 to an SM at a time:
// 2.7 us a row, of which its bytes need 1.9.
template <bool RES32, bool PAR32, int NC, int MAXT, bool DOTS>
__global__ void __launch_bounds__(MAXT)
norm_backward_kernel(NormArgs a, NormBwdPtrs p, int parts, int depth) {
    extern __shared__ __align__(128) char bwd_ring[];
    __shared__ __align__(8) uint64_t full[kNormMaxDepth];
    __shared__ BlockSum8 sums8;
    __shared__ BlockSum<2> sums2;
    const int tid = threadIdx.x;
    const unsigned bf_row = (unsigned)a.H8 * 16u, res_row = RES32 ? 2u * bf_row : bf_row;
    const unsigned y_bytes = p.y ? bf_row : 0u, r_bytes = p.w_pre ? res_row : 0u;
    const unsigned dr_bytes = p.d_r ? res_row : 0u, dn_bytes = p.w_pre ? bf_row : 0u;
    const unsigned at_r = y_bytes, at_dr = at_r + r_bytes, at_dn = at_dr + dr_bytes, stage = at_dn + dn_bytes;
    if (tid < depth) {
        mbar_init(&full[tid], 1u);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();

    // the rows that this block reads, in order
    int f_part = blockIdx.x, f_row = blockIdx.x;
    unsigned fetched = 0;
    bool alive = true;
    const auto fetch = [&](unsigned s) {             // thread 0
        if (f_part >= parts || !alive) return;
        char *to = bwd_ring + (size_t)s * stage;
        mbar_expect_tx(&full[s], stage);
        if (y_bytes) bulk_g2s(to, static_cast<const char *>(p.y) + (size_t)f_row * bf_row, y_bytes, &full[s]);
        if (r_bytes) bulk_g2s(to + at_r, static_cast<const char *>(p.r) + (size_t)f_row * res_row, r_bytes, &full[s]);
        if (dr_bytes) bulk_g2s(to + at_dr, static_cast<const char *>(p.d_r) + (size_t)f_row * res_row, dr_bytes, &full[s]);
        if (dn_bytes) bulk_g2s(to + at_dn, static_cast<const char *>(p.d_n) + (size_t)f_row * bf_row, dn_bytes, &full[s]);
        ++fetched;
        f_row += parts;
        if (f_row >= a.T) {
            f_part += gridDim.x;
            f_row = f_part;
        }
    };
    if (tid == 0)
        for (int i = 0; i < depth; ++i) fetch(i);

    // w_post and a channel's gate in one: where a thread has one chunk, once for all rows
    constexpr bool kHold = NC == 1 && MAXT <= 896;
    const auto post_of = [&](int c, float2 (&f)[4]) {
        Raw8<PAR32> raw;
        float2 g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = both(1.0f);
        if (p.w_post) {
            load_param8_again(p.w_post, c, raw);
            to_floats(raw, f);
        }
        if (a.channel) {
            load_param8_again(p.gate, c, raw);
            to_floats(raw, g);
#pragma unroll
            for (int q = 0; q < 4; ++q) f[q] = mul2(f[q], g[q]);
        }
    };
    float2 held[4];
    if (kHold && tid < a.H8) post_of(tid, held);
    unsigned turn = 0, n_row = 0, lost = 0, s = 0, parity = 0;
    for (int part = blockIdx.x; part < parts; part += gridDim.x) {
        float2 sum_pre[NC][4], sum_post[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) sum_pre[i][q] = sum_post[i][q] = both(0.0f);
        for (int t = part; t < a.T; t += parts, ++n_row) {
            if (alive && !mbar_wait_bounded(&full[s], parity)) {
                alive = false;                       // outputs stay wrong; the barriers below still meet
                lost = n_row;
                atomicOr(p.status, kStatusWaitGaveUp);
            }
            const char *in = bwd_ring + (size_t)s * stage;
            const auto y_of = [&](int c, float2 (&f)[4]) {
                to_floats(*reinterpret_cast<const Raw8<false> *>(in + (size_t)c * 16), f);
            };
            const auto r_of = [&](int c, float2 (&f)[4]) {
                to_floats(*reinterpret_cast<const Raw8<RES32> *>(in + at_r + (size_t)c * sizeof(Raw8<RES32>)), f);
            };
            const auto dr_of = [&](int c, float2 (&f)[4]) {
                to_floats(*reinterpret_cast<const Raw8<RES32> *>(in + at_dr + (size_t)c * sizeof(Raw8<RES32>)), f);
            };
            const auto dn_of = [&](int c, float2 (&f)[4]) {
                to_floats(*reinterpret_cast<const Raw8<false> *>(in + at_dn + (size_t)c * 16), f);
            };
            float2 v[NC][4];                         // w_pre d_n
            float2 rr = both(0.0f), rn = both(0.0f), yy = both(0.0f), yd = both(0.0f), yn = both(0.0f), yr = both(0.0f);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * (int)blockDim.x + tid;
                if (c < a.H8) {
                    float2 x[4], y[4], w[4];
                    if constexpr (DOTS) {
                        y_of(c, y);
#pragma unroll
                        for (int q = 0; q < 4; ++q) yy = fma2(y[q], y[q], yy);
                        if constexpr (!kHold) post_of(c, w);
#pragma unroll
                        for (int q = 0; q < 4; ++q) y[q] = mul2(y[q], kHold ? held[q] : w[q]);
                        if (dr_bytes) {
                            dr_of(c, x);
#pragma unroll
                            for (int q = 0; q < 4; ++q) yd = fma2(y[q], x[q], yd);
                        }
                    }
                    if (r_bytes) {
                        Raw8<PAR32> raw;
                        load_param8_again(p.w_pre, c, raw);
                        to_floats(raw, w);
                        dn_of(c, v[i]);
                        r_of(c, x);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            v[i][q] = mul2(v[i][q], w[q]);
                            rr = fma2(x[q], x[q], rr);
                            rn = fma2(x[q], v[i][q], rn);
                        }
                        if constexpr (DOTS) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                yn = fma2(y[q], v[i][q], yn);
                                yr = fma2(y[q], x[q], yr);
                            }
                        }
                    }
                }
            }
            float f[DOTS ? 8 : 2];
            f[0] = __fadd_rn(rr.x, rr.y);
            f[1] = __fadd_rn(rn.x, rn.y);
            if constexpr (DOTS) {
                f[2] = __fadd_rn(yy.x, yy.y);
                f[3] = __fadd_rn(yd.x, yd.y);
                f[4] = __fadd_rn(yn.x, yn.y);
                f[5] = __fadd_rn(yr.x, yr.y);
                f[6] = f[7] = 0.0f;
                block_sum8(sums8, f, turn);
            } else {
                block_sum(sums2, f, turn, (int)blockDim.x);
            }
            if (blockDim.x == 32) __syncwarp();
            // all are done with the row before this one
            if (tid == 0 && n_row > 0 && depth > 1) fetch(s == 0 ? depth - 1 : s - 1);

            const float rs = inv_rms(f[0], a), ys = DOTS && p.w_post ? inv_rms(f[DOTS ? 2 : 0], a) : 1.0f;
            const float mean = __fmul_rn(__fmul_rn(f[1], rs), a.inv_h);         // of r^ w_pre d_n
            const float g = a.token ? __ldg(static_cast<const float *>(p.gate) + t) : 1.0f, gy = __fmul_rn(g, ys);
            // the sum of y w_post D from its parts' sums: D = d_r + rs (w_pre d_n - r rs mean)
            float e = 0.0f;
            if constexpr (DOTS) e = __fmaf_rn(rs, __fmaf_rn(-__fmul_rn(rs, mean), f[5], f[4]), f[3]);
            if (DOTS && p.d_gate_token && tid == 0) p.d_gate_token[t] = __fmul_rn(__fmul_rn(a.scale, ys), e);
            const float m = __fmul_rn(__fmul_rn(e, ys), a.inv_h);               // of y^ w_post D
            const float by_y = __fmul_rn(__fmul_rn(a.scale, g), ys), less = DOTS && p.w_post ? __fmul_rn(ys, m) : 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = i * (int)blockDim.x + tid;
                if (c < a.H8) {
                    float2 D[4], x[4], w[4];
                    if (dr_bytes)
                        dr_of(c, D);
                    else
#pragma unroll
                        for (int q = 0; q < 4; ++q) D[q] = both(0.0f);
                    if (r_bytes) {
                        float2 n[4];
                        r_of(c, x);
                        dn_of(c, n);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 rh = mul2(x[q], both(rs));
                            sum_pre[i][q] = fma2(n[q], rh, sum_pre[i][q]);
                            D[q] = fma2(both(rs), fma2(rh, both(-mean), v[i][q]), D[q]);
                        }
                    }
                    store8<RES32>(static_cast<char *>(p.d_residual) + (size_t)t * res_row, c, D);
                    if (y_bytes) {
                        y_of(c, x);
                        if constexpr (!kHold) post_of(c, w);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            sum_post[i][q] = fma2(D[q], mul2(x[q], both(gy)), sum_post[i][q]);
                            D[q] = mul2(D[q], kHold ? held[q] : w[q]);
                            x[q] = mul2(DOTS ? fma2(x[q], both(-less), D[q]) : D[q], both(by_y));
                        }
                        store8<false>(static_cast<char *>(p.d_y) + (size_t)t * bf_row, c, x);
                    }
                }
            }
            if (depth == 1) {                        // a row of its own at a time
                __syncthreads();
                if (tid == 0) fetch(0);
            }
            if (++s == (unsigned)depth) {
                s = 0;
                parity ^= 1u;
            }
        }
        float *to = p.part + (size_t)part * 16 * a.H8;                          // [part][pre, post][H]
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i * (int)blockDim.x + tid;
            if (c < a.H8) {
                store8<true>(to, c, sum_pre[i]);
                store8<true>(to + 8 * a.H8, c, sum_post[i]);
            }
        }
    }
    if (tid == 0 && !alive)                          // no copy outlives the block
        for (; lost < fetched; ++lost) mbar_wait_bounded(&full[lost % (unsigned)depth], (lost / (unsigned)depth) & 1u);
}

// The parts' column sums into the gradients of the norms' weights and of a gate for each channel. A block
// takes 128 columns of one of the two sums, four to a lane, 32 warps the parts in turn, joined in order.
template <bool PAR32>
__global__ void __launch_bounds__(1024)
norm_columns_kernel(NormArgs a, const float *part, int parts, const void *__restrict__ w_post,
                    const void *__restrict__ gate, float *__restrict__ d_w_post, float *__restrict__ d_w_pre,
                    float *__restrict__ d_gate) {
    __shared__ float4 sums[32][32];
    pdl_enter_before(part);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.H8 * 8;
    const bool post = blockIdx.y != 0;
    if (post ? !d_w_post && !d_gate : !d_w_pre) return;
    const int h4 = blockIdx.x * 128 + 4 * lane;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h4 < H) {
        const float *from = part + (post ? H : 0) + h4;
#pragma unroll 8
        for (int i = warp; i < parts; i += 32) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(from + (size_t)i * 2 * H));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    sums[warp][lane] = s;
    __syncthreads();
    const int h = blockIdx.x * 128 + (int)threadIdx.x;
    if (threadIdx.x < 128 && h < H) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += reinterpret_cast<const float *>(&sums[i][0])[threadIdx.x];
        if (!post) {
            d_w_pre[h] = v;
        } else {
            const auto at = [&](const void *p) {
                return PAR32 ? static_cast<const float *>(p)[h] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[h]);
            };
            v = __fmul_rn(v, a.scale);
            if (d_w_post) d_w_post[h] = a.channel ? __fmul_rn(v, at(gate)) : v;
            if (d_gate) d_gate[h] = w_post ? __fmul_rn(v, at(w_post)) : v;
        }
    }
}

// Parts of the column sums: by the sizes alone, so that neither the grid nor the device changes a
// sum's order. About as many as blocks that GB300's 152 SMs hold at once; each part costs two rows of fp32 to
// write and to read again.
int norm_parts(long long T, int H) {
    const long long most = 152LL * std::max(1, std::min(8, 8192 / H));
    return (int)std::max(1LL, std::min(most, (T + 1) / 2));
}

template <bool PAR32>
int launch_columns(const Dims &d, const NormArgs &a, cudaStream_t st, const float *part, int parts, const void *w_post,
                   const void *gate, float *d_w_post, float *d_w_pre, float *d_gate) {
    if (!d_w_post && !d_w_pre && !d_gate) return MOE_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((d.H + 127) / 128), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_columns_kernel<PAR32>, a, part, parts, w_post, gate, d_w_post, d_w_pre, d_gate) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

template <bool RES32, bool PAR32, int NC, int MAXT, bool DOTS>
int launch_backward_nc(const Dims &d, const NormArgs &a, cudaStream_t st, const NormBwdPtrs &p, float *d_w_post,
                       float *d_w_pre, float *d_gate) {
    const auto kernel = norm_backward_kernel<RES32, PAR32, NC, MAXT, DOTS>;
    const int threads = ((a.H8 + NC - 1) / NC + 31) / 32 * 32;
    const int row = d.H * ((p.y ? 2 : 0) + (p.w_pre ? (RES32 ? 6 : 4) : 0) + (p.d_r ? (RES32 ? 4 : 2) : 0));
    const int parts = norm_parts(d.T, d.H);
    constexpr int kMaxSmem = 200 * 1024;
    const int blocks_per_sm = std::max(1, std::min(8, 8192 / d.H));
    const int depth = std::max(1, std::min(kNormMaxDepth, kMaxSmem / blocks_per_sm / row));
    static PerContext<int> smem_done;
    if (!set_smem_once(smem_done, kernel, kMaxSmem)) return MOE_ERR_CUDA;
    const size_t smem = (size_t)depth * row;
    const int grid = persistent_grid(parts, sm_count() * blocks_per_sm, d.max_blocks);
    if (launch_pdl_smem(kernel, grid, threads, smem, st, a, p, parts, depth) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_columns<PAR32>(d, a, st, p.part, parts, p.w_post, p.gate, d_w_post, d_w_pre, d_gate);
}
template <bool RES32, bool PAR32, bool DOTS, typename... A>
int launch_norm_backward(const Dims &d, const NormArgs &a, A... args) {
    if (a.H8 <= 256) return launch_backward_nc<RES32, PAR32, 1, 256, DOTS>(d, a, args...);
    // A chunk to a thread, as many warps as there can be, though that leaves no registers for the vectors: they are read again
    // for each row. us with one chunk a thread and with two and the vectors held, both with two sums a row: 4096 x 7168, 85 and
    // 95; 16381 x 4096, 149 and 152; 237 x 2056, 15.0 and 17.1. Up to 896 threads there are more registers for each: 4096 x 7168
    // within 64 took 89.
    if (a.H8 > 512 && a.H8 <= 896) return launch_backward_nc<RES32, PAR32, 1, 896, DOTS>(d, a, args...);
    if (a.H8 <= 1024) return launch_backward_nc<RES32, PAR32, 1, 1024, DOTS>(d, a, args...);
    return launch_backward_nc<RES32, PAR32, 4, 512, DOTS>(d, a, args...);
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm(const moe_problem *p, const moe_norm *norm, const void *y, const void *residual,
                              const void *w_post, const void *w_pre, const void *gate, void *r, void *n,
                              void *stream) {
    using namespace moe;
    Dims d;
    NormArgs a;
    int rc = check_problem(p, &d);
    if (rc == MOE_OK) rc = check_norm(d, norm, &a);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    const NormPtrs ptrs = {y, nullptr, nullptr, nullptr, residual, w_post, w_pre, gate, nullptr, r, n};
    rc = check_forward(norm, y != nullptr, ptrs);
    if (rc != MOE_OK) return rc;
    cudaStream_t st = as_stream(stream);
    return by_types(norm, [&](auto res, auto par) {
        constexpr bool kRes = decltype(res)::value, kPar = decltype(par)::value;
        if (y == nullptr) return launch_norm_nc<false, kRes, kPar>(d, a, st, ptrs);
        if (norm_many_rows(d)) return launch_norm_rows_nc<kRes, kPar>(d, a, st, ptrs);
        return launch_norm_nc<true, kRes, kPar>(d, a, st, ptrs);
    });
}

extern "C" int moe_combine_norm(const moe_problem *p, const moe_norm *norm, const void *y, const int32_t *topk_idx,
                                const float *topk_w, const int32_t *slot, const void *residual, const void *w_post,
                                const void *w_pre, const void *gate, void *out, void *r, void *n, void *stream) {
    using namespace moe;
    Dims d;
    NormArgs a;
    int rc = check_problem(p, &d);
    if (rc == MOE_OK) rc = check_norm(d, norm, &a);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) return MOE_OK;
    if (!y || !topk_idx || !topk_w || !slot) return MOE_ERR_INVALID_ARG;
    if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(slot, 4)) return MOE_ERR_INVALID_ARG;
    const NormPtrs ptrs = {y, topk_idx, topk_w, slot, residual, w_post, w_pre, gate, out, r, n};
    rc = check_forward(norm, true, ptrs);
    if (rc != MOE_OK) return rc;
    cudaStream_t st = as_stream(stream);
    return by_types(norm, [&](auto res, auto par) {
        return launch_combine_norm_k<decltype(res)::value, decltype(par)::value>(d, a, st, ptrs);
    });
}

extern "C" size_t moe_block_norm_backward_workspace_bytes(const moe_problem *p, const moe_norm *norm) {
    using namespace moe;
    Dims d;
    NormArgs a;
    if (check_problem(p, &d) != MOE_OK || check_norm(d, norm, &a) != MOE_OK) return 0;
    return ((size_t)norm_parts(d.T, d.H) * 2 * d.H * sizeof(float) + 255) & ~(size_t)255;
}

extern "C" int moe_block_norm_backward(const moe_problem *p, const moe_norm *norm, const void *y, const void *r,
                                       const void *d_r, const void *d_n, const void *w_post, const void *w_pre,
                                       const void *gate, void *d_y, void *d_residual, float *d_w_post, float *d_w_pre,
                                       float *d_gate, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace moe;
    Dims d;
    NormArgs a;
    int rc = check_problem(p, &d);
    if (rc == MOE_OK) rc = check_norm(d, norm, &a);
    if (rc != MOE_OK) return rc;
    if (d.T == 0) {                                                    // the sums of no rows
        if (!aligned(d_w_post, 4) || !aligned(d_w_pre, 4) || !aligned(d_gate, 4)) return MOE_ERR_INVALID_ARG;
        NormArgs none = a;
        none.channel = 0;
        return launch_columns<true>(d, none, as_stream(stream), nullptr, 0, nullptr, nullptr, d_w_post, d_w_pre,
                                    a.channel ? d_gate : nullptr);
    }
    const bool gated = norm->branch_gate != MOE_BRANCH_PLAIN;
    if ((!y && (w_post || gated)) || (y != nullptr) != (d_y != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!d_residual || (!w_pre && !d_r) || (w_pre != nullptr) != (d_n != nullptr) || (w_pre && !r)) return MOE_ERR_INVALID_ARG;
    if ((gate != nullptr) != gated || (d_w_post && !w_post) || (d_w_pre && !w_pre) || (d_gate && !gate)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_block_norm_backward_workspace_bytes(p, norm)) return MOE_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(r, 16) || !aligned(d_r, 16) || !aligned(d_n, 16) || !aligned(w_post, 16) ||
        !aligned(w_pre, 16) || !aligned(gate, a.token ? 4 : 16) || !aligned(d_y, 16) || !aligned(d_residual, 16) ||
        !aligned(d_w_post, 4) || !aligned(d_w_pre, 4) || !aligned(d_gate, 4) || !aligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    NormBwdPtrs b = {y, r, d_r, d_n, w_post, w_pre, gate, d_y, d_residual, a.token ? d_gate : nullptr,
                     static_cast<float *>(workspace), device_status_word()};
    if (b.status == nullptr) return MOE_ERR_CUDA;
    cudaStream_t st = as_stream(stream);
    if (a.token) d_gate = nullptr;                                     // a token's comes from its row
    return by_types(norm, [&](auto res, auto par) {
        constexpr bool kRes = decltype(res)::value, kPar = decltype(par)::value;
        if (y && (w_post || b.d_gate_token)) return launch_norm_backward<kRes, kPar, true>(d, a, st, b, d_w_post, d_w_pre, d_gate);
        return launch_norm_backward<kRes, kPar, false>(d, a, st, b, d_w_post, d_w_pre, d_gate);
    });
}

// moe_w4_tiles.cu -- the experts' products with 4-bit weights for many rows per
// expert, on the tcgen05 tensor cores.
//
//   r[m] = sum_g scale[m][g] * sum_{i in g} x[i] (q[m][i] - 8)
//
// The weights are the 128-row operand and the expert's rows of x the columns
// (16 to 64 of them), so that a TMEM lane is a row of the matrix: the thread that
// reads a lane's sums has one scale to multiply them by, and the one that writes
// the lane's weights has one row of codes to turn into bf16. The codes go from
// shared memory through registers into TMEM, from where tcgen05.mma takes its
// first operand; the 16-bit weights exist nowhere else. Each group's sum is exact
// products added in fp32 into a fresh accumulator, then scaled in fp32.
//
// A persistent grid, one CTA per SM, walks tiles of (expert, 2 x 128 matrix rows,
// up to 64 rows of x): rows n .. n+127 of the gate and of the up matrix, or 256
// rows of a matrix without the gate. In each CTA:
//   warp 0      one lane issues the TMA loads of x, 128 inputs of the tile's rows in
//               two boxes, into a ring of 4;
//   warps 1, 3  the MMAs of a tile's even and odd blocks, one elected lane each: per
//               group, the steps of both halves into fresh accumulators. All 512 TMEM
//               columns are held: for each half and parity 64 columns of accumulators
//               (one group of up to 64 rows of x, two of 32 or four of 16) and 64 of
//               operand (128 inputs);
//   warp 2      brings the group scales (and fp8 rows' block scales), 8 groups at a
//               time, from HBM to a ring in shared memory;
//   warps 4-19  four TMEM quadrants x two halves x even and odd blocks: copy the codes
//               of their 32 rows to rings of their own and turn them into operands;
//   warps 20-27 four quadrants x two halves: add up the groups' sums, and write y.
// Bound by the conversion of codes (144 instructions of a warp for 32 rows x 128
// inputs, half of them on the half-rate ALU pipe) and by the chain operand -> MMA ->
// sums -> accumulator; the split into these roles is what overlaps the links. 256
// experts of 2 x 2048 x 7168 with 32 rows each, groups of 128: 964 us, 0.61 of the
// copy bandwidth; 32 such experts 136 us with 32 rows, 122 with 16, 185 with 64;
// groups of 32 and 16 rows 140 us.
// Every mbarrier wait is bounded; one that gives up raises the status word and an
// abort flag, the CTA drains what it has in flight, frees its TMEM and returns.
#include "moe_tc.cuh"
#include "moe_w4.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kTRows = 128;                          // matrix rows of one half (TMEM lanes)
constexpr int kTTok = 64;                            // rows of x to a tile, at most
constexpr int kTXStages = 4;                         // rings of x blocks: two of even and two of odd blocks
constexpr int kTThreads = 896;                       // 28 warps of 72 registers
constexpr int kTWDepth = 4;                          // blocks of codes that a warp has in flight or at hand
constexpr uint32_t kTWBytes = 32 * 64;               // codes of a warp's 32 rows of a block
constexpr uint32_t kTXBytes = kTTok * 128;           // x of 64 inputs
constexpr int kTChunks = 3, kTChunk = 8;             // scale ring: 3 chunks of 8 groups
constexpr size_t kTExBytes = (size_t)16 * kTRows * 4;
constexpr size_t kTScaleBytes = (size_t)kTChunks * 2 * kTRows * kTChunk * 2;
constexpr size_t kTXsBytes = (size_t)kTChunks * kTChunk * kTTok * 4;
constexpr size_t kTSmemBytes = 1024 + kTXStages * 2 * (size_t)kTXBytes + 16 * kTWDepth * (size_t)kTWBytes + kTExBytes +
                               kTScaleBytes + kTXsBytes;

// How a tile of up to CAP rows of x uses a parity's 64 columns of accumulators: the
// sums of kBatch groups of CAP columns go to one slot and are waited for together,
// kSlots slots.
template <int GPB, int CAP>
struct W4Acc {
    static constexpr int kRoom = kTTok / CAP;                          // 4, 2, 1
    static constexpr int kBatch = GPB < kRoom ? GPB : kRoom;
    static constexpr int kSlots = kRoom / kBatch;
};

// 16 bytes of global memory to shared memory, asynchronously.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The same for BYTES (4, 8 or 16), or as many zeros where there is nothing to copy.
template <int BYTES>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool some) {
    const int n = some ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
// Arrives on the mbarrier once all of this thread's copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D[128 x N] (+)= A (TMEM) B: one step of 16 inputs.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The tiles holding kept rows, in the order (expert, matrix rows, rows of x), so
// that the tiles that share weights run at about the same time.
struct W4Tiles {
    const int *first;                                // first tile of expert e; first[E] = their number
    int E, n_tiles;
    __device__ __forceinline__ void decode(int t, int &e, int &nt, int &tt) const {
        e = expert_of_row(first, E, t);
        const int per = (first[e + 1] - first[e]) / n_tiles;
        const int local = t - first[e];
        nt = local / per;
        tt = local - nt * per;
    }
};

// x of [E][C][K] in boxes of 16, 32, 48 and 64 rows x 64 inputs.
struct W4Maps {
    CUtensorMap x[4];
};

template <int N>
struct Int {
    static constexpr int value = N;
};

// acc[i] += v[i] * scale (times the fp8 row's own scale), 16 columns.
template <bool F8>
__device__ __forceinline__ void add16(float *acc, const uint32_t *v, float ws, const float *xs) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float4 f = make_float4(ws, ws, ws, ws);
        if constexpr (F8) {
            f = *reinterpret_cast<const float4 *>(xs + i);
            f = make_float4(f.x * ws, f.y * ws, f.z * ws, f.w * ws);
        }
        acc[i] = fmaf(__uint_as_float(v[i]), f.x, acc[i]);
        acc[i + 1] = fmaf(__uint_as_float(v[i + 1]), f.y, acc[i + 1]);
        acc[i + 2] = fmaf(__uint_as_float(v[i + 2]), f.z, acc[i + 2]);
        acc[i + 3] = fmaf(__uint_as_float(v[i + 3]), f.w, acc[i + 3]);
    }
}

// One warp brings the scales of groups c .. c+7 of 128 matrix rows, `valid` of them
// in the matrix, to `to` (16 bytes a row), W bytes of a row to a copy; zeros for rows
// and groups past the end. Rows of an odd number of scales, which 4-byte copies
// cannot reach, go through registers.
template <int W>
__device__ __forceinline__ void scale_chunk(const uint16_t *__restrict__ src, int groups, int c, int valid,
                                            uint16_t *to, int lane) {
#pragma unroll
    for (int i = 0; i < kTRows / 32; ++i) {
        const int r = 32 * i + lane;
        const uint16_t *from = src + (size_t)min(r, max(valid - 1, 0)) * groups + c;
#pragma unroll
        for (int q = 0; q < kTChunk; q += W / 2) {
            const bool some = r < valid && c + q < groups;
            if constexpr (W >= 4)
                cp_async_or_zero<W>(smem_u32(to + r * kTChunk + q), some ? from + q : src, some);
            else
                to[r * kTChunk + q] = some ? __ldg(from + q) : (uint16_t)0;
        }
    }
}

template <bool F8, int GS, bool GATE>
__global__ void __launch_bounds__(kTThreads, 1)
expert_w4_tiles_kernel(const __grid_constant__ W4Maps maps, W4Args a, const uint8_t *__restrict__ w_q,
                       const int32_t *__restrict__ counts, const uint16_t *__restrict__ w_scale,
                       const float *__restrict__ x_scale, uint16_t *__restrict__ y, unsigned *status) {
    constexpr int GPB = 128 / GS;                    // groups to a block of 128 inputs
    constexpr int kOut = GATE ? kTRows : 2 * kTRows; // outputs of a tile
    extern __shared__ uint8_t w4_smem_raw[];
    constexpr int SX = kTXStages;
    __shared__ __align__(8) uint64_t x_full[SX];
    __shared__ __align__(8) uint64_t a_full[2], a_free[4];                // operands of even and odd blocks; [2 (odd block) + odd use]
    __shared__ __align__(8) uint64_t d_full[8], d_free[8];                // accumulators: [4 (odd block) + slot]
    __shared__ __align__(8) uint64_t sc_full[kTChunks], sc_empty[kTChunks];
    __shared__ __align__(8) uint64_t ex_full[4], ex_free[4];           // sums traded between the halves
    __shared__ __align__(8) uint64_t s_drain[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ int s_first[kMaxExperts + 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t smem0 = (smem_u32(w4_smem_raw) + 1023u) & ~1023u;
    uint8_t *const base = w4_smem_raw + (smem0 - smem_u32(w4_smem_raw));
    uint8_t *const codes = base + SX * 2 * kTXBytes;
    float *const ex = reinterpret_cast<float *>(codes + 16 * kTWDepth * kTWBytes);
    uint16_t *const sc = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(ex) + kTExBytes);
    float *const xs = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(sc) + kTScaleBytes);   // fp8 rows only
    const int nkb = a.nkb, groups = nkb * GPB;
    const int n_tiles = (a.N + kOut - 1) / kOut;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SX; ++i) {
            mbar_init(&x_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&a_full[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&a_free[i], 1);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_free[i], 8);
        }
        for (int i = 0; i < kTChunks; ++i) {
            mbar_init(&sc_full[i], 32);
            mbar_init(&sc_empty[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&ex_full[i], 2);
            mbar_init(&ex_free[i], 2);
        }
        mbar_init(&s_drain[0], 1);
        mbar_init(&s_drain[1], 1);
        s_abort = 0;
        fence_mbar_init();
    }
    pdl_wait();                                      // counts and x are final from here on
    if (warp == 0) {
        const int per = (a.E + 31) / 32;
        int sum = 0;
        for (int e = lane * per; e < min(a.E, lane * per + per); ++e)
            sum += (min(__ldg(counts + e), a.C) + kTTok - 1) / kTTok * n_tiles;
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - sum;
        for (int e = lane * per; e < min(a.E, lane * per + per); ++e) {
            s_first[e] = run;
            run += (min(__ldg(counts + e), a.C) + kTTok - 1) / kTTok * n_tiles;
        }
        if (lane == 31) s_first[a.E] = incl;
    }
    __syncthreads();
    const int total = s_first[a.E];
    if ((int)blockIdx.x >= total) {
        pdl_launch_dependents();
        return;
    }
    const W4Tiles tiles{s_first, a.E, n_tiles};
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;                    // half h, odd block or even p: accumulators at 128 h + 64 p, operand 256 on

    uint32_t x_even = 0, x_odd = 0;                  // blocks of x loaded, also for the drain
    // setmaxnreg is one instruction of a whole warpgroup (warps 0-3, 4-7, ...). 896 threads of 72 registers are
    // 64512; 20 warps give up 16 of theirs for the 8 that hold 64 sums: 20 x 32 x 56 + 8 x 32 x 112 = 64512
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            const bool elected = elect_one();
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                int e, nt, tt;
                tiles.decode(t, e, nt, tt);
                const int rows = min(min(__ldg(counts + e), a.C) - tt * kTTok, kTTok);
                const int n16 = __shfl_sync(kFull, (rows + 15) / 16, 0);
                const int ez = __shfl_sync(kFull, e, 0), row_x = __shfl_sync(kFull, tt * kTTok, 0);
                const CUtensorMap *map = &maps.x[n16 - 1];
                for (int kb = 0; kb < nkb; ++kb) {
                    uint32_t &use = kb & 1 ? x_odd : x_even;
                    const uint32_t s = 2 * (kb & 1) + (use & 1);
                    // the block two uses ago has been multiplied: its x stage is its operand use's
                    if (use >= 2 && !(ok = warp_wait(smem_u32(&a_free[0]) + 8 * s, ((use >> 1) + 1) & 1, &s_abort))) break;
                    if (elected) {
                        const uint32_t at = smem0 + s * 2 * kTXBytes, bar = smem_u32(&x_full[0]) + 8 * s;
                        mbar_expect_tx(&x_full[s], n16 * 4096);
                        tma_load_3d(at, map, bar, kb * 128, row_x, ez);
                        tma_load_3d(at + kTXBytes, map, bar, kb * 128 + 64, row_x, ez);
                    }
                    __syncwarp();
                    ++use;
                }
            }
        } else if (warp == 1 || warp == 3) {
            // The whole warp runs the loop and one elected lane issues: the operands of
            // tcgen05.mma are then warp-uniform values, and a step of 128 x 32 x 16 takes
            // 17 cycles to issue where a loop of one lane by itself takes 45 (measured).
            // One warp for the even blocks of a tile and one for the odd ones: between
            // two blocks a warp spends as long in its waits as in its MMAs.
            const uint32_t par = __shfl_sync(kFull, (uint32_t)warp >> 1, 0);
            const uint32_t op = __shfl_sync(kFull, tmem, 0) + 256 + 64 * par;       // + 128 per half
            const uint32_t d0 = __shfl_sync(kFull, tmem, 0) + 64 * par;             // + 128 per half, 32 per slot
            const bool elected = elect_one();
            const uint32_t b_afull = smem_u32(&a_full[par]), b_afree = smem_u32(&a_free[2 * par]);
            const uint32_t b_dfull = smem_u32(&d_full[4 * par]), b_dfree = smem_u32(&d_free[4 * par]);
            uint32_t use = 0;                        // blocks so far: of the operand, and of the parity's two x stages
            uint32_t d_phase = 0;                    // odd or even use of the slots (bits)
            int last_cap = 0;
            bool ok = true;
            const auto tile = [&](auto cap_, uint32_t n16) {
                constexpr int CAP = decltype(cap_)::value;
                using Acc = W4Acc<GPB, CAP>;
                // fp32 sums; both operands fp16 (0) or bf16 (1); 128 x n16
                const uint32_t idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) | ((n16 >> 3) << 17) |
                                       ((uint32_t)(kTRows >> 4) << 24);
                if (last_cap != CAP) {               // slots of other widths: every one of the last tile's has been read
                    for (int i = 0; i < 4; ++i)
                        if (!warp_wait(b_dfree + 8 * i, (d_phase >> i & 1u) ^ 1u, &s_abort)) return false;
                    last_cap = CAP;
                }
                uint32_t slot = 0;
                for (int kb = (int)par; kb < nkb; kb += 2, ++use) {
                    const uint32_t s = 2 * par + (use & 1);
                    const uint64_t bx = umma_desc_sw128(smem0 + s * 2 * kTXBytes);
                    if (!warp_wait(smem_u32(&x_full[0]) + 8 * s, use >> 1 & 1u, &s_abort)) return false;
                    if (!warp_wait(b_afull, use & 1u, &s_abort)) return false;
#pragma unroll
                    for (int q = 0; q < GPB; q += Acc::kBatch) {
                        if (!warp_wait(b_dfree + 8 * slot, (d_phase >> slot & 1u) ^ 1u, &s_abort)) return false;
                        d_phase ^= 1u << slot;
                        tc_fence_after();
                        const uint32_t d = d0 + slot * (Acc::kBatch * CAP);
                        if (elected) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int k = 0; k < Acc::kBatch * GS / 16; ++k) {
                                    const int k16 = q * (GS / 16) + k;
                                    mma_ts(d + 128 * h + k / (GS / 16) * CAP, op + 128 * h + 8 * k16,
                                           bx + ((k16 >> 2) * kTXBytes + 32 * (k16 & 3)) / 16, idesc,
                                           k % (GS / 16) > 0 ? 1u : 0u);
                                }
                            }
                            mma_commit(b_dfull + 8 * slot);
                            if (q + Acc::kBatch == GPB) mma_commit(b_afree + 8 * (use & 1));   // operand and x are read
                        }
                        __syncwarp();
                        if (++slot == Acc::kSlots) slot = 0;
                    }
                }
                return true;
            };
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                int e, nt, tt;
                tiles.decode(t, e, nt, tt);
                const int rows = __shfl_sync(kFull, min(min(__ldg(counts + e), a.C) - tt * kTTok, kTTok), 0);
                const uint32_t n16 = (uint32_t)(rows + 15) / 16 * 16;
                ok = rows <= 16 ? tile(Int<16>(), n16) : rows <= 32 ? tile(Int<32>(), n16) : tile(Int<64>(), n16);
            }
        } else {
            constexpr int KPC = kTChunk / GPB;       // blocks of 128 inputs to a chunk
            const int chunks = (groups + kTChunk - 1) / kTChunk;
            uint32_t cg = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total && !s_abort; t += gridDim.x) {
                int e, nt, tt;
                tiles.decode(t, e, nt, tt);
                // first outputs and matrix rows of the two halves, and how many of their 128 rows there are
                const int n0 = nt * kOut, n1 = GATE ? n0 : n0 + kTRows;
                const int valid0 = min(a.N - n0, kTRows), valid1 = min(a.N - n1, kTRows);
                const uint16_t *src0 = w_scale + ((size_t)e * a.M + n0) * groups;
                const uint16_t *src1 = w_scale + ((size_t)e * a.M + (GATE ? a.N + n0 : n1)) * groups;
                const int kept = min(__ldg(counts + e), a.C) - tt * kTTok;
                const float *xsrc = F8 ? x_scale + ((size_t)e * a.C + tt * kTTok) * nkb : nullptr;
                for (int c = 0; c < chunks; ++c, ++cg) {
                    const int buf = cg % kTChunks;
                    if (cg >= kTChunks &&              // the ring's slot has been read
                        !(ok = warp_wait(smem_u32(&sc_empty[buf]), ((cg / kTChunks) + 1) & 1, &s_abort)))
                        break;
                    uint16_t *to = sc + (size_t)buf * 2 * kTRows * kTChunk;
                    const auto both = [&](auto w) {
                        constexpr int W = decltype(w)::value;
                        scale_chunk<W>(src0, groups, c * kTChunk, valid0, to, lane);
                        scale_chunk<W>(src1, groups, c * kTChunk, valid1, to + kTRows * kTChunk, lane);
                    };
                    // rows of a multiple of 8 scales are copied 16 bytes at a time, others as their alignment lets
                    const bool odd_rows = GPB == 1 && groups % 2 != 0;
                    if (groups % 8 == 0) both(Int<16>());
                    else if (GPB == 4 || groups % 4 == 0) both(Int<8>());
                    else if (!odd_rows) both(Int<4>());
                    else both(Int<2>());
                    if constexpr (F8) {
#pragma unroll
                        for (int r = lane; r < kTTok; r += 32) {
#pragma unroll
                            for (int i = 0; i < KPC; ++i) {
                                const bool some = r < kept && c * KPC + i < nkb;
                                cp_async_or_zero<4>(smem_u32(xs + ((size_t)buf * kTChunk + i) * kTTok + r),
                                                    some ? xsrc + (size_t)r * nkb + c * KPC + i : x_scale, some);
                            }
                        }
                    }
                    if (odd_rows) {
                        // scales stored by this thread itself: only an ordinary arrive releases those to the readers,
                        // after the row scales' copies
                        cp_async_wait_all();
                        mbar_arrive(&sc_full[buf]);
                    } else {
                        cp_async_arrive(&sc_full[buf]);
                    }
                }
            }
            cp_async_wait_all();
        }
    } else if (warp < 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int quad = warp & 3, h = ((warp - 4) >> 2) & 1, par = (warp - 4) >> 3;
        const uint32_t op0 = tmem + ((uint32_t)(quad * 32) << 16) + 256 + 128 * h + 64 * par;
        const uint32_t b_afull = smem_u32(&a_full[par]), b_afree = smem_u32(&a_free[2 * par]);
        // The codes of this warp's 32 rows come to a ring of the warp's own, by its own asynchronous copies: no other
        // warp waits for them. Lane l copies chunk l % 4 (16 bytes) of rows l / 4 + 8 i; chunk t of row r stands at
        // t ^ (r / 2 % 4), so that neither the copies nor the reads of a row a lane meet in a bank.
        uint8_t *const ring = codes + (warp - 4) * kTWDepth * kTWBytes;
        const uint32_t dst = smem_u32(ring) + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
        const uint8_t *const src = ring + lane * 64;
        const int swz = ((lane >> 1) & 3) << 4;
        const int mine = (total - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;       // tiles of this CTA
        const uint32_t blocks = (uint32_t)mine * (uint32_t)((nkb - par + 1) / 2);  // every other block of each
        const uint8_t *from = nullptr;               // the tile's rows, at this lane's first chunk of the next block
        uint32_t off[4] = {};                        // and the offsets of its four rows
        int it = (int)blockIdx.x - (int)gridDim.x, ikb = nkb;
        const auto fetch = [&](uint32_t n) {         // block n of this warp's, in turn
            if (n < blocks) {
                if (ikb >= nkb) {
                    int e, nt, tt;
                    tiles.decode(it += gridDim.x, e, nt, tt);
                    const int n0 = GATE ? nt * kOut : nt * kOut + h * kTRows;
                    from = w_q + ((size_t)e * a.M + (GATE ? h * a.N : 0)) * (a.K / 2) + 16 * (lane & 3) + 64 * par;
                    const int last = a.N - 1;        // rows past the matrix are read as its last: their scales are 0
#pragma unroll
                    for (int i = 0; i < 4; ++i) off[i] = (uint32_t)min(n0 + quad * 32 + (lane >> 2) + 8 * i, last) * (a.K / 2);
                    ikb = par;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) cp_async16(dst + (n % kTWDepth) * kTWBytes + i * 512, from + off[i]);
                from += 128;
                ikb += 2;
            }
            cp_async_commit();
        };
#pragma unroll
        for (int n = 0; n < kTWDepth - 1; ++n) fetch(n);
        for (uint32_t n = 0; n < blocks; ++n) {
            cp_async_wait<kTWDepth - 2>();
            __syncwarp();                            // every lane's copies of block n are there, and block n - 1 is read
            fetch(n + kTWDepth - 1);
            uint4 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = *reinterpret_cast<const uint4 *>(src + (n % kTWDepth) * kTWBytes + ((i << 4) ^ swz));
            if (n > 0 && !warp_wait(b_afree + 8 * ((n - 1) & 1), (n - 1) >> 1 & 1u, &s_abort)) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t r[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w4_pairs<F8>(j == 0 ? q[i].x : j == 1 ? q[i].y : j == 2 ? q[i].z : q[i].w, r[i]);
                tmem_st16(op0 + 16 * j, reinterpret_cast<const uint32_t(&)[16]>(r));
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(b_afull);
        }
        cp_async_wait<0>();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        const int quad = warp & 3, h = (warp - 20) >> 2;
        const int row = quad * 32 + lane;            // TMEM lane: row of this half
        const uint32_t d0 = tmem + ((uint32_t)(quad * 32) << 16) + 128 * h;
        const uint32_t b_dfull = smem_u32(&d_full[0]), b_dfree = smem_u32(&d_free[0]);
        uint32_t cg = 0, n_ex = 0;                   // chunks and trades so far
        uint32_t d_phase = 0;                        // odd or even use of the accumulators (bits)
        bool ok = true;
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
            int e, nt, tt;
            tiles.decode(t, e, nt, tt);
            const int rows = min(min(__ldg(counts + e), a.C) - tt * kTTok, kTTok);
            const auto tile = [&](auto cap_) {       // with sums for CAP columns only: registers
                constexpr int CAP = decltype(cap_)::value;
                using Acc = W4Acc<GPB, CAP>;
                float acc[CAP];
#pragma unroll
                for (int i = 0; i < CAP; ++i) acc[i] = 0.0f;
                for (int c = 0; c < groups; c += kTChunk, ++cg) {
                    const uint32_t buf = cg % kTChunks;
                    if (!warp_wait(smem_u32(&sc_full[buf]), (cg / kTChunks) & 1, &s_abort)) return false;
                    const uint4 s8 = *reinterpret_cast<const uint4 *>(sc + ((buf * 2 + h) * kTRows + row) * kTChunk);
                    const uint16_t *s1 = sc + ((buf * 2 + h) * kTRows + row) * kTChunk;
                    const uint32_t s2[4] = {s8.x, s8.y, s8.z, s8.w};   // this row's 8 scales
                    const float *xr = xs + buf * kTChunk * kTTok;
                    const int n = min(kTChunk, groups - c);
                    // a chunk's batches: of an even and an odd block in turn, as their MMAs run side by side. A parity's
                    // batches in a chunk are a multiple of its slots, so that each chunk begins with slot 0.
                    constexpr int kSteps = kTChunk / 2 / Acc::kBatch, kPerBlock = GPB / Acc::kBatch;
                    static_assert(kSteps % Acc::kSlots == 0, "slots");
#pragma unroll(CAP == 64 ? 2 : 8)
                    for (int i = 0; i < 2 * kSteps; ++i) {
                        const int p = i & 1, step = i >> 1;
                        // the batch's first group: block 2 (step / kPerBlock) + p of the chunk
                        const int group = (2 * (step / kPerBlock) + p) * GPB + step % kPerBlock * Acc::kBatch;
                        if (group < n) {
                            const int which = 4 * p + step % Acc::kSlots;
                            if (!warp_wait(b_dfull + 8 * which, d_phase >> which & 1u, &s_abort)) return false;
                            d_phase ^= 1u << which;
                            tc_fence_after();
                            const uint32_t d = d0 + 64 * p + step % Acc::kSlots * (Acc::kBatch * CAP);
                            const float *xg = xr + group / GPB * kTTok;
                            constexpr int kCols = Acc::kBatch * CAP, kNow = kCols < 32 ? 16 : 32;
#pragma unroll
                            for (int b = 0; b < kCols; b += kNow) {    // some columns at a time: registers
                                uint32_t v[kNow];
                                tmem_ld16(d + b, v);
                                if constexpr (kNow > 16) tmem_ld16(d + b + 16, v + 16);
                                tmem_ld_wait();
                                if (b + kNow >= kCols) {               // the last of them is read
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive_at(b_dfree + 8 * which);
                                }
#pragma unroll
                                for (int u = 0; u < kNow; u += 16) {
                                    const int gi = group + (b + u) / CAP;
                                    const float ws = CAP == 64 ? bf16_lo((uint32_t)s1[gi]) : gi & 1 ? bf16_hi(s2[gi >> 1]) : bf16_lo(s2[gi >> 1]);
                                    add16<F8>(acc + (b + u) % CAP, v + u, ws, xg + (b + u) % CAP);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_empty[buf]);
                }
#pragma unroll
                for (int i = 0; i < CAP; ++i) acc[i] *= kW4Unit<F8>;
                uint16_t *const out = y + ((size_t)e * a.C + tt * kTTok) * a.N;
                if constexpr (GATE) {
                    // the halves' warps of the same rows trade, 16 columns at a time: each gets the other's sums of 8
                    // of them, and finishes those
                    const int n = nt * kOut + row;
#pragma unroll
                    for (int b = 0; b < CAP; b += 16) {
                        if (b >= rows) break;
                        if (!warp_wait(smem_u32(&ex_free[quad]), (n_ex & 1u) ^ 1u, &s_abort)) return false;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            ex[(8 * (1 - h) + i) * kTRows + row] = h == 0 ? acc[b + 8 + i] : acc[b + i];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ex_full[quad]);
                        if (!warp_wait(smem_u32(&ex_full[quad]), n_ex & 1u, &s_abort)) return false;
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float other = ex[(8 * h + i) * kTRows + row];
                            o[i] = h == 0 ? silu(acc[b + i]) * other : silu(other) * acc[b + 8 + i];
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ex_free[quad]);
                        ++n_ex;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (b + 8 * h + i < rows && n < a.N)
                                put_bf16(out + (size_t)(b + 8 * h + i) * a.N + n, o[i]);
                    }
                } else {
                    const int n = nt * kOut + h * kTRows + row;
#pragma unroll
                    for (int i = 0; i < CAP; ++i)
                        if (i < rows && n < a.N) put_bf16(out + (size_t)i * a.N + n, acc[i]);
                }
                return true;
            };
            ok = rows <= 16 ? tile(Int<16>()) : rows <= 32 ? tile(Int<32>()) : tile(Int<64>());
        }
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (s_abort) {
        // drain: the loads and MMAs this CTA started must land before its
        // shared memory and TMEM are released
        volatile int no_abort = 0;
        if (warp == 0 && lane == 0) {
            atomicOr(status, kStatusWaitGaveUp);
            for (uint32_t p = 0; p < 2; ++p) {
                const uint32_t n = p ? x_odd : x_even;
                for (uint32_t u = n > 2 ? n - 2 : 0; u < n; ++u)
                    gemm_wait(smem_u32(&x_full[2 * p + (u & 1)]), u >> 1 & 1, &no_abort);
            }
        }
        if ((warp == 1 || warp == 3) && elect_one()) {   // the lanes that issued the MMAs
            mma_commit(smem_u32(&s_drain[warp >> 1]));
            gemm_wait(smem_u32(&s_drain[warp >> 1]), 0, &no_abort);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// fp8 rows as fp16 (exact): the operand of the tiles' MMAs. Kept rows only.
__global__ void __launch_bounds__(256)
w4_rows_to_f16_kernel(const uint4 *__restrict__ x, const int32_t *__restrict__ counts, uint4 *__restrict__ out, int E,
                      int C, int K) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ int32_t warp_tot[32];
    pdl_enter();
    kept_row_offsets(counts, E, C, off, warp_tot);
    const unsigned rows = off[E], tasks = K / 16;    // a task is 16 codes
    for (UnitWalk wk(blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8, (tasks + 31) / 32); wk.row < rows; wk.next()) {
        const int e = expert_of_row(off, E, (int)wk.row);
        const size_t row = (size_t)e * C + (wk.row - off[e]);
        const unsigned c = wk.seg * 32 + (threadIdx.x & 31);
        if (c >= tasks) continue;
        const uint4 q = ld_stream_v4(x + row * tasks + c);
        uint4 *o = out + (row * tasks + c) * 2;
        o[0] = make_uint4(e4m3x2_to_f16x2(q.x), e4m3x2_to_f16x2(q.x >> 16), e4m3x2_to_f16x2(q.y),
                          e4m3x2_to_f16x2(q.y >> 16));
        o[1] = make_uint4(e4m3x2_to_f16x2(q.z), e4m3x2_to_f16x2(q.z >> 16), e4m3x2_to_f16x2(q.w),
                          e4m3x2_to_f16x2(q.w >> 16));
    }
}

// x [E][rows][K] of 16-bit numbers in boxes of box_rows x 64, 128-byte swizzled; rows past the end read as zero.
bool encode_3d(CUtensorMap *map, const void *base, uint64_t K, uint64_t rows, uint64_t E, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {K, rows, E};
    const cuuint64_t strides[2] = {K * 2, K * rows * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long kept_at_most(const Dims &d) {
    return std::min<long long>((long long)d.T * d.k, (long long)d.E * d.C);
}

template <bool F8, int GS, bool GATE>
int launch_one(const Dims &d, const W4Args &a, cudaStream_t st, const void *x, const float *x_scale,
               const int32_t *counts, const void *w_q, const void *w_scale, void *y, void *workspace) {
    const int n_tiles = (a.N + (GATE ? kTRows : 2 * kTRows) - 1) / (GATE ? kTRows : 2 * kTRows);
    const long long tiles = (kept_at_most(d) / kTTok + d.E) * n_tiles;
    if (tiles * a.nkb >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;    // blocks are counted in 32 bits
    W4Maps maps;
    for (int i = 0; i < 4; ++i)
        if (!encode_3d(&maps.x[i], F8 ? workspace : x, a.K, a.C, a.E, 16 * (i + 1))) return MOE_ERR_CUDA;
    unsigned *status = device_status_word();
    if (status == nullptr) return MOE_ERR_CUDA;
    static PerContext<int> smem_done;
    if (!set_smem_once(smem_done, expert_w4_tiles_kernel<F8, GS, GATE>, (int)kTSmemBytes)) return MOE_ERR_CUDA;
    if constexpr (F8) {
        static PerContext<int> resident_cache;
        const int resident = resident_blocks_cached(resident_cache, w4_rows_to_f16_kernel, 256);
        const int grid = persistent_grid((kept_at_most(d) * ((a.K / 16 + 31) / 32) + 7) / 8, resident, d.max_blocks);
        if (launch_pdl(w4_rows_to_f16_kernel, grid, 256, st, static_cast<const uint4 *>(x), counts,
                       static_cast<uint4 *>(workspace), a.E, a.C, a.K) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    const int grid = persistent_grid(tiles, sm_count(), d.max_blocks);
    if (launch_pdl_smem(expert_w4_tiles_kernel<F8, GS, GATE>, grid, kTThreads, kTSmemBytes, st, maps, a,
                        static_cast<const uint8_t *>(w_q), counts,
                        static_cast<const uint16_t *>(w_scale), x_scale, static_cast<uint16_t *>(y), status) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    return MOE_OK;
}

template <bool F8, int GS, typename... A>
int launch_act(const Dims &d, const W4Args &a, A... args) {
    return a.M == 2 * a.N ? launch_one<F8, GS, true>(d, a, args...) : launch_one<F8, GS, false>(d, a, args...);
}
template <bool F8, typename... A>
int launch_group(const Dims &d, const W4Args &a, A... args) {
    if (a.group == 32) return launch_act<F8, 32>(d, a, args...);
    if (a.group == 64) return launch_act<F8, 64>(d, a, args...);
    return launch_act<F8, 128>(d, a, args...);
}

}  // namespace

size_t w4_tiles_workspace_bytes(const Dims &d, const W4Args &a) {
    return d.dtype == MOE_DTYPE_FP8_E4M3_B128 ? (size_t)a.E * a.C * a.K * 2 : 0;
}

int launch_w4_tiles(const Dims &d, const W4Args &a, cudaStream_t st, const void *x, const float *x_scale,
                    const int32_t *counts, const void *w_q, const void *w_scale, void *y, void *workspace) {
    if (d.dtype == MOE_DTYPE_FP8_E4M3_B128)
        return launch_group<true>(d, a, st, x, x_scale, counts, w_q, w_scale, y, workspace);
    return launch_group<false>(d, a, st, x, x_scale, counts, w_q, w_scale, y, workspace);
}

}  // namespace moe

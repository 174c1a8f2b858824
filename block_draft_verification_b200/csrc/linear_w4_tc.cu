// linear_w4_tc.cu -- the products of linear_w4.cu for more tokens than a few, on
// the tensor cores (tcgen05): bf16 activations, any output type.
//
// A tile is 128 weight rows (four units) by up to 128 tokens.  Its K loop:
//   warp 0       one bulk copy per packed step (64 or 128 k) of the tile into the W
//                ring
//   warp 2       TMA of the tokens' x (64 k boxes, 128-byte swizzle) into the chunk's
//                stage
//   warps 4-19   codes to exact bf16 integers q - zero, stored as the K-major,
//                128-byte swizzled A tile of a 64 k chunk; a warp takes a unit, and
//                each four warps every fourth chunk
//   warp 1       tcgen05.mma (M = 128, N = tokens, K = 16) of a group's k into one
//                of four TMEM accumulators
//   warps 20-27  tcgen05.ld of the group's sums, times the row's scale, added to
//                fp32 sums in registers while the next group's MMAs run
// so the weights are never rounded: a group's integer-weighted sums come out of
// the tensor core and the scale multiplies them in fp32.  The scaling costs 128 x
// N fused multiply-adds a group beside 128 x N x group on the tensor core.
//
// Measured: 20,480 x 5,120 with 64 tokens (groups of 64) in 50 us, 5,120 x 20,480 with
// 256 in 84 us (640 TFLOP/s), the conv of 32 x 8 tokens at H = 5,120 in 50 us.  With
// codes, sums and tile ends left out the pipeline alone takes 30, 61 and 29 us: about
// 480 cycles a chunk, the way from a free stage over the copy of x (about 1,100
// cycles) to its MMAs in a ring of four; a tile's end costs 9 to 16 us of the rest.
//
// Tiles are taken by clusters of S CTAs that split K; the sums meet in
// distributed shared memory in rank order: no workspace, no atomics.  S is the
// one that leaves the SMs least idle.  Every wait is bounded (tw_wait); after one
// that ran out the roles pass through their loops without waiting, a flag is set,
// copies and MMAs in flight are waited for (bounded) and TMEM is released.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "linear_w4.cuh"
#include "stream.cuh"
#include "tc.cuh"
#include "w4.cuh"

namespace dfl {

namespace cg = cooperative_groups;

constexpr int TW_ROWS = 128;            // weight rows per tile: four units
constexpr int TW_DEQ = 16, TW_SUM = 8;  // warps
constexpr int TW_THREADS = 32 * (4 + TW_DEQ + TW_SUM);
constexpr int TW_SUB = TW_ROWS * 128;   // bytes of 64 k of A
constexpr int TW_NA = 4;                // chunks in the operand rings (A and x)
// Registers: 896 threads are launched with 72 each, 64,512; 128 x 40 + 512 x 48 +
// 256 x 136 use all of them after the split.

struct W4TcArgs {
    const uint8_t* packed;
    int64_t tokens, n_rows;         // n_rows: rows of W
    int64_t ld;                     // linear: N; conv: H
    int steps, S, C, tt;            // K steps, cluster size, clusters, token tiles
    int64_t tiles;
    void* y;
    int y_bf16, y_vec;              // y_vec: four rows of a token may be stored at once
    const __nv_bfloat16* x;         // conv
    const __nv_bfloat16* x_prev;    // conv; NULL: linear
    int T;
};

__host__ __device__ constexpr int tw_w_stage(int kb, int sg, int fmt) {
    return 4 * (kb * W4_CHUNK_BYTES + sg * w4_scale_bytes(fmt));
}
// Tokens whose sums are joined at a time at a tile's end: all of them, where shared
// memory holds them beside a W ring long enough (not 128 with float scales or steps
// of one chunk).
__host__ __device__ constexpr int tw_round(int n, int kb, int fmt) {
    return n == 128 && (kb == 1 || (fmt & DFLASH2_W4_SCALE_F32)) ? 64 : n;
}
// Shared memory but for the W ring: the operand rings, a round's sums, the barriers.
__host__ __device__ constexpr int tw_fixed(int n, int kb, int fmt) {
    return TW_NA * (TW_SUB + n * 128) + tw_round(n, kb, fmt) * TW_ROWS * 4 + 384;
}
// Steps in the W ring: what is left, and no more than 12.
__host__ __device__ constexpr int tw_w_stages(int n, int kb, int sg, int fmt) {
    const int w = (227 * 1024 - tw_fixed(n, kb, fmt)) / tw_w_stage(kb, sg, fmt);
    return w < 12 ? w : 12;
}
__host__ __device__ constexpr int tw_smem(int n, int kb, int sg, int fmt) {
    return tw_fixed(n, kb, fmt) + tw_w_stages(n, kb, sg, fmt) * tw_w_stage(kb, sg, fmt);
}
constexpr int TW_AHEAD = 3;      // pairs of groups by which the scales are read before their sums
constexpr int TW_PREFETCH = 12;  // steps between the request to L2 and the copy

__device__ __forceinline__ void tw_load_x(uint32_t dst, const CUtensorMap* map, int k, int tok,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(k), "r"(tok), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar, int rank) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(bar),
        "r"(rank)
        : "memory");
}
// Waits, bounded: `tries` tries of up to a microsecond each; a wait that runs out
// leaves `tries` at 1, so that everything after it passes at once and the role runs
// to its end (with results that do not count: tw_report sets the error flag).
// The loop is one piece of assembly without a result to branch on: the code around
// it stays on the warp's common path, where the MMA warp's operands are uniform.
// tried: the barrier was tested before and found done.
constexpr uint32_t TW_TRIES = 1000000u;
__device__ __forceinline__ void tw_wait(uint32_t bar, uint32_t parity, uint32_t& tries, bool tried = false) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "setp.ne.u32 q, %4, 0;\n\t@q bra DONE;\n\t"
        "mov.u32 n, %0;\n"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 n, n, -1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra TRY;\n\t"
        "mov.u32 %0, 1;\n"
        "DONE:\n\t}"
        : "+r"(tries)
        : "r"(bar), "r"(parity), "r"(1000u), "r"((uint32_t)tried)
        : "memory");
}
__device__ __forceinline__ void tw_wait_cluster(uint32_t bar, uint32_t parity, uint32_t& tries) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %0;\n"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 n, n, -1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra TRY;\n\t"
        "mov.u32 %0, 1;\n"
        "DONE:\n\t}"
        : "+r"(tries)
        : "r"(bar), "r"(parity), "r"(1000u)
        : "memory");
}
__device__ __forceinline__ void tw_report(uint32_t tries, unsigned flag) {
    if (tries == 1u) atomicOr(&g_dev_err, flag);
}
__device__ __forceinline__ void unpack4(uint2 q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xFFFF0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// The MMA warp's instructions, issued by its one elected lane without leaving the
// warp's common path: operands then stay in the warp's uniform registers (a
// product takes 15 cycles to issue; about 85 from a branch that one lane takes).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_bf16_elect(uint32_t elected, uint32_t tmem_d, uint64_t a, uint64_t b,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected));
}
__device__ __forceinline__ void mma_commit_elect(uint32_t elected, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(elected)
        : "memory");
}
// 32 lanes x 16 consecutive fp32 columns, no wait.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// What a summing thread needs at a tile's end.
struct TwEnd {
    const W4TcArgs* a;
    float* sp;            // [rank of origin][token of the share][row]
    uint32_t tries;
    int rank, rt, tok0, ntok, e, half, q;
    uint32_t pready, pfree;
    int round;            // rounds before this tile's
};

// The sums of this CTA's K go to the CTAs of the cluster that write them, NR
// tokens at a time (half of them of either half of the columns), each CTA a share of
// them; then they are added in rank order and written.
template <int NTOK, int NR, int S>
__device__ __forceinline__ uint32_t tw_tile_end(const TwEnd& f, const uint64_t (&acc)[NTOK / 4]) {
    constexpr int NC = NTOK / 2, CPR = NR / 2, SHARE = NR / S;
    const W4TcArgs& a = *f.a;
    uint32_t tries = f.tries;
    const int e = f.e, lane = e & 31;
    const uint32_t spu = smem_u32(f.sp);
    auto token_of = [](int t, int rd) { return (t / CPR) * NC + rd * CPR + t % CPR; };
#pragma unroll
    for (int rd = 0; rd < NC / CPR; ++rd) {
        const int round = f.round + rd;
        if (rd * CPR >= f.ntok) break;  // the same in every CTA of the cluster
        if (S > 1 && round > 0) tw_wait_cluster(f.pfree, (round - 1) & 1, tries);
        const uint32_t own = spu + 4 * (f.rank * SHARE * TW_ROWS + 32 * f.q + lane);
        if constexpr (S == 1) {
            const uint32_t o = own + 4 * f.half * CPR * TW_ROWS;
#pragma unroll
            for (int n = 0; n < CPR; ++n) {
                const uint64_t pr = acc[(rd * CPR + n) / 2];
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(o + 4 * n * TW_ROWS),
                             "f"((n & 1) ? f2_hi(pr) : f2_lo(pr))
                             : "memory");
            }
        } else {
            // this half's CPR tokens are CPR / SHARE whole shares (S = 2: one)
            static_assert(CPR % SHARE == 0, "a half of a round is whole shares");
#pragma unroll
            for (int b = 0; b < CPR / SHARE; ++b) {
                uint32_t o;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(o)
                             : "r"(own), "r"(f.half * (CPR / SHARE) + b));
#pragma unroll
                for (int n = 0; n < SHARE; ++n) {
                    const int i = rd * CPR + b * SHARE + n;
                    const uint64_t pr = acc[i / 2];
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(o + 4 * n * TW_ROWS),
                                 "f"((i & 1) ? f2_hi(pr) : f2_lo(pr))
                                 : "memory");
                }
            }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (S > 1 && e < S) cluster_arrive(f.pready, e);
        auto sum4 = [&](int row, int tl) {  // four rows of a token, over the cluster
            const uint32_t p = spu + 4 * (tl * TW_ROWS + row);
            float4 v[S];
#pragma unroll
            for (int k = 0; k < S; ++k) {
                const uint4 u = lds128(p + 4 * k * SHARE * TW_ROWS);
                v[k] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                   __uint_as_float(u.w));
            }
#pragma unroll
            for (int k = 1; k < S; ++k)
                v[0].x += v[k].x, v[0].y += v[k].y, v[0].z += v[k].z, v[0].w += v[k].w;
            return v[0];
        };
        if (!a.x_prev) {
            const int row = (e & 31) * 4;
            const int64_t n = (int64_t)f.rt * TW_ROWS + row;
            const bool vec = a.y_vec && n + 4 <= a.n_rows;
            if (S > 1) tw_wait_cluster(f.pready, round & 1, tries);
#pragma unroll
            for (int i = 0; i < (SHARE + 7) / 8; ++i) {
                const int tl = (e >> 5) + 8 * i, t = token_of(f.rank * SHARE + tl, rd);
                if ((SHARE % 8 != 0 && tl >= SHARE) || t >= f.ntok) continue;
                const float4 v = sum4(row, tl);
                const int64_t o = (f.tok0 + t) * a.ld + n;
                const float w4[4] = {v.x, v.y, v.z, v.w};
                if (vec) {
                    if (a.y_bf16)
                        *(uint2*)((__nv_bfloat16*)a.y + o) = pack4(w4);
                    else
                        *(float4*)((float*)a.y + o) = v;
                } else {
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (n + p < a.n_rows) {
                            if (a.y_bf16)
                                ((__nv_bfloat16*)a.y)[o + p] = __float2bfloat16_rn(w4[p]);
                            else
                                ((float*)a.y)[o + p] = w4[p];
                        }
                }
            }
        } else {
            // a and b of a channel: rows 8 apart (w4_pack, taps); H is a multiple of 64,
            // so a tile's 64 channels are all there.  x is on its way while the
            // cluster's sums come in.
            const int c4 = (e & 15) * 4, ch = f.rt * 64 + c4, row = (c4 >> 3) * 16 + (c4 & 7);
            constexpr int M = (SHARE + 15) / 16;  // items of a thread
            uint2 xc[M], xp[M];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const int t = token_of(f.rank * SHARE + (e >> 4) + 16 * i, rd);
                const int tok = f.tok0 + min(t, f.ntok - 1), sq = tok / a.T;
                const __nv_bfloat16* x = a.x + tok * a.ld + ch;
                xc[i] = __ldg((const uint2*)x);
                xp[i] = __ldg((const uint2*)(tok == sq * a.T ? a.x_prev + sq * a.ld + ch : x - a.ld));
            }
            if (S > 1) tw_wait_cluster(f.pready, round & 1, tries);
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const int tl = (e >> 4) + 16 * i, t = token_of(f.rank * SHARE + tl, rd);
                if ((SHARE % 16 != 0 && tl >= SHARE) || t >= f.ntok) continue;
                const float4 av = sum4(row, tl), bv = sum4(row + 8, tl);
                const float a4[4] = {av.x, av.y, av.z, av.w}, b4[4] = {bv.x, bv.y, bv.z, bv.w};
                float c[4], p[4];
                unpack4(xc[i], c);
                unpack4(xp[i], p);
#pragma unroll
                for (int z = 0; z < 4; ++z) c[z] = fmaf(b4[z], p[z], fmaf(a4[z], c[z], c[z]));
                *(uint2*)((__nv_bfloat16*)a.y + (int64_t)(f.tok0 + t) * a.ld + ch) = pack4(c);
            }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (S > 1 && e < S) cluster_arrive(f.pfree, e);
    }
    return tries;
}

// NTOK: tokens per tile (32, 64, 128); FMT: scale format; G32: groups of 32, two
// per step; KB: chunks per step.
template <int NTOK, int FMT, bool G32, int KB>
__global__ void __launch_bounds__(TW_THREADS, 1)
    linear_w4_tc_kernel(const __grid_constant__ CUtensorMap map_x, const W4TcArgs a) {
    constexpr int SG = G32 ? 2 : 1;
    constexpr int SB = w4_scale_bytes(FMT), LB = SB / 8;
    constexpr int STEP = KB * W4_CHUNK_BYTES + SG * SB;
    constexpr int NA = TW_NA, NW = tw_w_stages(NTOK, KB, SG, FMT);
    constexpr int WST = tw_w_stage(KB, SG, FMT);
    constexpr int XSUB = NTOK * 128;       // bytes of 64 k of x
    constexpr int NC = NTOK / 2;           // columns per summing warp
    constexpr int NR = tw_round(NTOK, KB, FMT);  // tokens per round of a tile's end
    // TMEM holds two pairs of groups' accumulators; a pair is waited for, read and
    // given back at once (a wait that finds its barrier done still takes about 107
    // cycles, a good part of a group's products)
    constexpr int NB = 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sa = smem_raw;
    if ((smem_u32(sa) & 1023u) != 0) {  // the swizzle's alignment, as declared
        if (threadIdx.x == 0) atomicOr(&g_dev_err, (unsigned)ERR_PRODUCER);
        return;
    }
    uint8_t* sx = sa + NA * TW_SUB;
    float* sp = (float*)(sx + NA * XSUB);  // [token][row] sums of a round
    uint8_t* sw = (uint8_t*)sp + NR * TW_ROWS * 4;
    uint64_t* bars = (uint64_t*)(sw + NW * WST);
    uint32_t* s_tmem = (uint32_t*)(bars + 44);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.S, cl = blockIdx.x / a.S;
    const int k0 = (int)((int64_t)a.steps * rank / a.S);
    const int nst = (int)((int64_t)a.steps * (rank + 1) / a.S) - k0;

    const uint32_t wfull = smem_u32(bars), wempty = wfull + 8 * NW, full = wempty + 8 * NW,
                   empty = full + 8 * NA, tfull = empty + 8 * NA, tempty = tfull + 8 * NB,
                   mdone = tempty + 8 * NB, pready = mdone + 8, pfree = pready + 8;
    // full: a chunk's A tile (an arrival per code warp) and its x (one, and the bytes)
    static_assert(2 * NW + 2 * NA + 2 * NB + 3 <= 44, "barriers");

    if (threadIdx.x == 0) {
        for (int i = 0; i < NW; ++i) {
            mbar_init(wfull + 8 * i, 1);
            mbar_init(wempty + 8 * i, 4 * KB);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(full + 8 * i, 4 + 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, TW_SUM);
        }
        mbar_init(mdone, 1);
        mbar_init(pready, (uint32_t)a.S);
        mbar_init(pfree, (uint32_t)a.S);
        mbar_fence_init();
    }
    constexpr uint32_t NCOLS = NB * 2 * NTOK;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(s_tmem)),
                     "r"(NCOLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    // the barriers of every CTA are set up: waited for before the first use of
    // another CTA's
    if (a.S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    uint32_t tries = TW_TRIES;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            // ---------------- packed weights; L2 is asked for them TW_PREFETCH steps
            // before their copy, four at a time, so that the ring need only cover its
            // latency, not DRAM's
            int i = 0;
            for (int64_t tile = cl; tile < a.tiles; tile += a.C) {
                const uint8_t* src = a.packed + w4_block(tile / a.tt * 4, a.steps, k0, STEP);
                const int64_t next = tile + a.C;
                const uint8_t* src1 =
                    a.packed + w4_block((next < a.tiles ? next : tile) / a.tt * 4, a.steps, k0, STEP);
                for (int s = 0; s < nst; ++s, ++i) {
                    const int w = i % NW;
                    if (i >= NW) tw_wait(wempty + 8 * w, (i / NW - 1) & 1, tries);
                    bulk_g2s(smem_u32(sw + w * WST), src + (int64_t)s * WST, WST, wfull + 8 * w);
                    if (s % 4 == 3 && i >= NW - 1) {
                        // steps s + TW_PREFETCH .. of this tile or, past its end, of the next
                        const int p = s + TW_PREFETCH, over = p - nst;
                        if (over < 0)
                            prefetch_l2(src + (int64_t)p * WST, min(4, -over) * WST);
                        else if (next < a.tiles && over < nst)
                            prefetch_l2(src1 + (int64_t)over * WST, min(4, nst - over) * WST);
                    }
                }
            }
            // the last copies have landed before the CTA may leave
            for (int q = i > NW ? i - NW : 0; q < i; ++q) tw_wait(wfull + 8 * (q % NW), (q / NW) & 1, tries);
            tw_report(tries, ERR_PRODUCER);
        } else if (warp == 2 && lane == 0) {
            // ---------------- x
            int ci = 0;
            for (int64_t tile = cl; tile < a.tiles; tile += a.C) {
                const int tok0 = (int)(tile % a.tt) * NTOK;
                for (int s = 0; s < nst * KB; ++s, ++ci) {
                    const int x = ci % NA;
                    if (ci >= NA) tw_wait(empty + 8 * x, (ci / NA - 1) & 1, tries);
                    mbar_expect_tx(full + 8 * x, (uint32_t)XSUB);
                    tw_load_x(smem_u32(sx + x * XSUB), &map_x, (k0 * KB + s) * W4_CHUNK, tok0,
                              full + 8 * x);
                }
            }
            for (int q = ci > NA ? ci - NA : 0; q < ci; ++q) tw_wait(full + 8 * (q % NA), (q / NA) & 1, tries);
            tw_report(tries, ERR_PRODUCER);
        } else if (warp == 1) {
            // ---------------- MMA issuer: the whole warp waits, one lane issues
            const uint32_t elected = elect_lane();
            int st = 0, pb = 0;
            uint32_t par = 0, tpar = 1;  // phases of the ring and (waited for) of TMEM
            bool tried = false;
            for (int64_t tile = cl; tile < a.tiles; tile += a.C) {
                const int64_t left = a.tokens - (tile % a.tt) * NTOK;
                const uint32_t idesc =
                    instr_desc(TW_ROWS, (int)min((int64_t)NTOK, (left + 15) / 16 * 16));
                for (int s = 0; s < nst; ++s) {
                    // a pair of groups: two steps, or a step of two groups; its
                    // accumulators have been read (their first use: the phase before
                    // the first counts as done)
                    const bool opens = SG == 2 || s % 2 == 0, closes = SG == 2 || s % 2 == 1 || s + 1 == nst;
                    if (opens) tw_wait(tempty + 8 * pb, tpar, tries);
                    const uint32_t d0 = tmem + (uint32_t)((2 * pb + (opens ? 0 : 1)) * NTOK);
#pragma unroll
                    for (int c = 0; c < KB; ++c) {
                        tw_wait(full + 8 * st, par, tries, tried);
                        tc_fence_after();
                        const uint64_t ao = smem_desc(smem_u32(sa + st * TW_SUB));
                        const uint64_t xo = smem_desc(smem_u32(sx + st * XSUB));
                        const uint32_t done = empty + 8 * st;
                        if (++st == NA) {
                            st = 0;
                            par ^= 1u;
                        }
                        tried = mbar_test(full + 8 * st, par);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const bool first = SG == 2 ? kk % 2 == 0 : kk == 0 && c == 0;
                            mma_bf16_elect(elected, d0 + (SG == 2 ? kk / 2 * NTOK : 0), ao + 2 * kk, xo + 2 * kk,
                                           idesc, first ? 0u : 1u);
                        }
                        mma_commit_elect(elected, done);
                    }
                    if (closes) {
                        mma_commit_elect(elected, tfull + 8 * pb);
                        pb ^= 1;
                        if (pb == 0) tpar ^= 1u;
                    }
                }
            }
            if (lane == 0) tw_report(tries, ERR_MMA);
            mma_commit_elect(elected, mdone);  // fires when every MMA issued has completed
        }
    } else if (warp < 4 + TW_DEQ) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // ---------------- codes to operands: a warp takes a unit's 32 rows of every
        // fourth chunk, always into the same stage of A
        static_assert(NA == 4 && TW_DEQ == 16, "a stage for each four warps");
        const int u = warp & 3, grp = (warp - 4) >> 2;
        const int r = lane >> 2, c = lane & 3;
        const bool odd = (r & 1) != 0;  // odd rows store their second half first: the
                                        // eight lanes of a store then hit all banks
        const uint32_t src = smem_u32(sw) + u * STEP + lane * 16 + (KB == 2 ? (grp & 1) * W4_CHUNK_BYTES : 0);
        // the zero points of the lane's rows r, r + 8, r + 16, r + 24
        const uint32_t zsrc = smem_u32(sw) + u * STEP + KB * W4_CHUNK_BYTES + r * LB +
                              ((FMT & DFLASH2_W4_SCALE_F32) ? 16 : 8);
        const uint32_t dst = smem_u32(sa) + grp * TW_SUB + (u * 32 + r) * 128;
        const uint32_t d0 = dst + ((4 * (odd ? 1 : 0) + c) ^ r) * 16, d1 = dst + ((4 * (odd ? 0 : 1) + c) ^ r) * 16;
        int left = 0;  // chunks of this CTA's tiles that these four warps take
        for (int64_t tile = cl; tile < a.tiles; tile += a.C) left += nst * KB;
        left = (left - grp + 3) / 4;
        int w = (KB == 2 ? grp >> 1 : grp) % NW;
        uint32_t wpar = 0, apar = 1;  // A's stage: the phase before the first counts as done
        // W is tested while the chunk before is worked on.  A test by parity must not
        // come two phases early: chunk i - 4, waited for here, had its W, and a stage's
        // use before is no later than that one's
        static_assert(KB == 2 ? NW >= 4 : NW >= 8, "the phase before is complete");
        bool ready = false;
        for (int k = 0; k < left; ++k) {
            tw_wait(wfull + 8 * w, wpar, tries, ready);
            tw_wait(empty + 8 * grp, apar, tries);
            apar ^= 1u;
            const uint32_t wo = (uint32_t)(w * WST), wdone = wempty + 8 * w;
            const uint4 v[2] = {lds128(src + wo), lds128(src + wo + 512)};
            uint2 zq[SG];
            if constexpr (FMT != 0)
#pragma unroll
                for (int h = 0; h < SG; ++h) zq[h] = lds64(zsrc + wo + h * SB);
            w += KB == 2 ? 2 : 4;
            if (w >= NW) {
                w -= NW;
                wpar ^= 1u;
            }
            ready = mbar_test(wfull + 8 * w, wpar);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // rows r + 16 b + 8 q
                    uint32_t z0 = 0x41C041C0u, z1 = 0x41C041C0u;  // 16 + 8; of either half
                    if constexpr (FMT != 0) {
                        z0 = z1 = __byte_perm(b ? zq[0].y : zq[0].x, 0, q ? 0x3232 : 0x1010);
                        if constexpr (G32) z1 = __byte_perm(b ? zq[SG - 1].y : zq[SG - 1].x, 0, q ? 0x3232 : 0x1010);
                    }
                    const uint32_t h0 = q ? v[b].z : v[b].x, h1 = q ? v[b].w : v[b].y;
                    const uint32_t wa = odd ? h1 : h0, wb = odd ? h0 : h1;
                    const uint32_t za = G32 && odd ? z1 : z0, zb = G32 && odd ? z0 : z1;
                    sts128(d0 + b * 2048 + q * 1024, w4_pair_exact(wa, 0, za), w4_pair_exact(wa, 1, za),
                           w4_pair_exact(wa, 2, za), w4_pair_exact(wa, 3, za));
                    sts128(d1 + b * 2048 + q * 1024, w4_pair_exact(wb, 0, zb), w4_pair_exact(wb, 1, zb),
                           w4_pair_exact(wb, 2, zb), w4_pair_exact(wb, 3, zb));
                }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full + 8 * grp);
                mbar_arrive(wdone);
            }
        }
        if (lane == 0) tw_report(tries, ERR_EPILOGUE);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        // ---------------- scaling and sums
        const int q = warp & 3;                     // TMEM lanes 32 q .. 32 q + 31 = unit q
        const int half = (warp - 4 - TW_DEQ) >> 2;  // columns half * NC ..
        const int e = threadIdx.x - 32 * (4 + TW_DEQ);
        const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * NC);
        if (a.S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        int round = 0, pb = 0;
        uint32_t tpar = 0;
        bool tried = false;
        for (int64_t tile = cl; tile < a.tiles; tile += a.C) {
            const int rt = (int)(tile / a.tt);
            const int tok0 = (int)(tile - (int64_t)rt * a.tt) * NTOK;
            const int ntok = (int)min((int64_t)NTOK, a.tokens - tok0);
            // this row's scales, TW_AHEAD pairs ahead of their use, straight from the
            // packed steps (in L2 by then)
            const uint8_t* sp0 = a.packed + w4_block((int64_t)rt * 4 + q, a.steps, k0, STEP) + KB * W4_CHUNK_BYTES +
                                 (lane & 7) * LB + (lane >> 3) * ((FMT & DFLASH2_W4_SCALE_F32) ? 4 : 2);
            auto read_scales = [&](int s, float (&f)[SG]) {
                const uint8_t* p = sp0 + (int64_t)min(s, nst - 1) * WST;
#pragma unroll
                for (int h = 0; h < SG; ++h) {
                    if constexpr ((FMT & DFLASH2_W4_SCALE_F32) != 0)
                        f[h] = __ldg((const float*)(p + h * SB));
                    else
                        f[h] = __uint_as_float((uint32_t)__ldg((const unsigned short*)(p + h * SB)) << 16);
                }
            };
            constexpr int PS = SG == 1 ? 2 : 1;  // steps of a pair of groups
            float sc[TW_AHEAD][PS][SG];          // of the pair at hand and the next ones, in turn
#pragma unroll
            for (int z = 0; z < TW_AHEAD; ++z)
#pragma unroll
                for (int y = 0; y < PS; ++y) read_scales(z * PS + y, sc[z][y]);
            uint64_t acc[NC / 2];  // pairs of tokens
#pragma unroll
            for (int n = 0; n < NC / 2; ++n) acc[n] = 0;
            // (a register that a load is still to fill is not moved: the pairs take the
            // scale registers in turn)
            for (int s0 = 0; s0 < nst; s0 += TW_AHEAD * PS) {
#pragma unroll
                for (int z0 = 0; z0 < TW_AHEAD; ++z0) {
                    const int s = s0 + z0 * PS;
                    if (s >= nst) break;
                    tw_wait(tfull + 8 * pb, tpar, tries, tried);
                    tc_fence_after();
                    const int done = pb;
                    pb ^= 1;
                    if (pb == 0) tpar ^= 1u;
                    tried = mbar_test(tfull + 8 * pb, tpar);
                    const uint32_t ta = tb + (uint32_t)(done * 2 * NTOK);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float f = SG == 2 ? sc[z0][0][g % SG] : sc[z0][g % PS][0];
                        constexpr int G = NC >= 32 ? 2 : 1;  // 16-column loads in flight
                        if (SG == 2 || g == 0 || s + 1 < nst)  // an odd last step goes alone
#pragma unroll
                            for (int n = 0; n < NC; n += 16 * G) {
                                if (half * NC + n < ntok) {  // the same for the whole warp
                                    uint32_t v[G][16];
#pragma unroll
                                    for (int z = 0; z < G; ++z) tmem_ld(ta + g * NTOK + n + 16 * z, v[z]);
                                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                                    for (int z = 0; z < G; ++z)
#pragma unroll
                                        for (int x = 0; x < 16; x += 2) {
                                            uint64_t& p = acc[(n + 16 * z + x) / 2];
                                            p = f2_fma(f2_pack(f, f),
                                                       f2_pack(__uint_as_float(v[z][x]),
                                                               __uint_as_float(v[z][x + 1])),
                                                       p);
                                        }
                                }
                            }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty + 8 * done);
#pragma unroll
                    for (int y = 0; y < PS; ++y) read_scales(s + TW_AHEAD * PS + y, sc[z0][y]);
                }
            }
            // The tile's end, written out for each cluster size: its loops are short and
            // unrolled, their addresses constants.
            const TwEnd t{&a, sp, tries, rank, rt, tok0, ntok, e, half, q, pready, pfree, round};
            if (a.S == 1)
                tries = tw_tile_end<NTOK, NR, 1>(t, acc);
            else if (a.S == 2)
                tries = tw_tile_end<NTOK, NR, 2>(t, acc);
            else if (a.S == 4)
                tries = tw_tile_end<NTOK, NR, 4>(t, acc);
            else
                tries = tw_tile_end<NTOK, NR, 8>(t, acc);
            round += min(NTOK / NR, (ntok + NR / 2 - 1) / (NR / 2));
        }
        if (lane == 0) tw_report(tries, ERR_EPILOGUE);
    }
    if (a.S > 1 && warp < 4 + TW_DEQ) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __syncthreads();
    if (warp == 1) {
        tw_wait(mdone, 0, tries);
        if (lane == 0) tw_report(tries, ERR_DRAIN);
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(NCOLS));
    }
    if (a.S > 1) cg::this_cluster().sync();  // the others may still read this CTA's sums
}

}  // namespace dfl

using namespace dfl;

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                           cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? (EncodeTiledFn)p
                   : (EncodeTiledFn) nullptr;
    }();
    return fn;
}

template <int NTOK, int FMT, bool G32, int KB>
int launch(const CUtensorMap& map, const W4TcArgs& a, int dev, cudaStream_t s) {
    constexpr int smem = tw_smem(NTOK, KB, G32 ? 2 : 1, FMT);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto* k = linear_w4_tc_kernel<NTOK, FMT, G32, KB>;
    {
        static std::mutex mu;
        static bool attr_set[64] = {};
        std::lock_guard<std::mutex> g(mu);
        if (dev >= 64 || !attr_set[dev]) {
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return DFLASH2_ECUDA;
            if (dev < 64) attr_set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.S * a.C));
    cfg.blockDim = dim3(TW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.S;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, map, a) == cudaSuccess ? DFLASH2_OK
                                                              : (cudaGetLastError(), DFLASH2_ECUDA);
}
template <int NTOK, int FMT>
int launch_group(const CUtensorMap& map, const W4TcArgs& a, const W4Layout& L, int dev, cudaStream_t s) {
    if (L.kb == 2) return launch<NTOK, FMT, false, 2>(map, a, dev, s);
    return L.sg == 2 ? launch<NTOK, FMT, true, 1>(map, a, dev, s)
                     : launch<NTOK, FMT, false, 1>(map, a, dev, s);
}
template <int NTOK>
int launch_fmt(const CUtensorMap& map, const W4TcArgs& a, const W4Layout& L, int format, int dev,
               cudaStream_t s) {
    if (format & DFLASH2_W4_SCALE_F32) return launch_group<NTOK, 2>(map, a, L, dev, s);
    if (format & DFLASH2_W4_ZERO) return launch_group<NTOK, 1>(map, a, L, dev, s);
    return launch_group<NTOK, 0>(map, a, L, dev, s);
}

}  // namespace

bool dfl_linear_w4_tc_ok(const W4Call& c) {
    return c.x_vec && !c.x_f32 && encode_fn() != nullptr;
}

// Tokens per tile and cluster size: rounds of tiles times the length of one, in
// cycles.  A chunk takes about 300 for its barriers and codes and, per group, 250,
// 370 or 690 for the sums of 32, 64 or 128 tokens (its MMAs and its weights'
// share of memory bandwidth are below that); each round of a tile's end about 1,500,
// 6,500 where sums cross CTAs.  (10,240 x 5,120: 23.9, 24.9 and 32.8 us at
// 32, 64 and 128 tokens in groups of 128; 20,480 x 5,120 in groups of 64: 46, 50
// and 95 us.)
W4TcPlan dfl_linear_w4_tc_plan(const W4Call& c, const W4Dev& d) {
    const W4Layout& L = c.L;
    W4TcPlan P{};
    int64_t best = -1;
    for (int n : {32, 64, 128}) {
        const int tt = (int)((c.tokens + n - 1) / n);
        const int64_t tiles = (L.units + 3) / 4 * tt;
        const int ends = n / tw_round(n, L.kb, c.format);
        const int64_t step = L.kb * 300 + L.sg * (n == 32 ? 250 : n == 64 ? 370 : 690);
        for (int S = 1; S <= 8 && S <= L.steps; S *= 2) {
            const int64_t C = std::min<int64_t>(tiles, d.clusters[S]);
            const int64_t cost = ((tiles + C - 1) / C) * ((L.steps + S - 1) / S * step +
                                                          ends * (S > 1 ? 6500 : 1500));
            if (best < 0 || cost < best) {
                best = cost;
                P = {n, tt, S, (int)C, tiles};
            }
        }
    }
    return P;
}

int dfl_linear_w4_tc(const W4Call& c, const W4Dev& d, cudaStream_t s) {
    const W4Layout& L = c.L;
    const W4TcPlan P = dfl_linear_w4_tc_plan(c, d);
    W4TcArgs a{};
    a.packed = (const uint8_t*)c.packed;
    a.tokens = c.tokens;
    a.n_rows = L.N;
    a.ld = c.x_prev ? L.K : L.N;
    a.steps = L.steps;
    a.y = c.y;
    a.y_bf16 = c.y_bf16;
    a.y_vec = L.N % 4 == 0 && (uintptr_t)c.y % 16 == 0;
    a.x = (const __nv_bfloat16*)c.x;
    a.x_prev = (const __nv_bfloat16*)c.x_prev;
    a.T = c.T;
    a.S = P.S;
    a.C = P.C;
    a.tt = P.tt;
    a.tiles = P.tiles;
    CUtensorMap map;
    cuuint64_t dims[2] = {(cuuint64_t)L.K, (cuuint64_t)c.tokens};
    cuuint64_t strides[1] = {(cuuint64_t)(c.tokens > 1 ? c.x_stride : L.K) * 2};
    cuuint32_t box[2] = {W4_CHUNK, (cuuint32_t)P.ntok};
    cuuint32_t estr[2] = {1, 1};
    if (encode_fn()(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(c.x), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return DFLASH2_ECUDA;
    if (P.ntok == 32) return launch_fmt<32>(map, a, L, c.format, d.id, s);
    if (P.ntok == 64) return launch_fmt<64>(map, a, L, c.format, d.id, s);
    return launch_fmt<128>(map, a, L, c.format, d.id, s);
}

unsigned dfl_errors_w4_tc(int clear) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_dev_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    if (clear && v) {
        unsigned z = 0;
        cudaMemcpyToSymbol(g_dev_err, &z, sizeof z);
    }
    return v;
}

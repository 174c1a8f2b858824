// linear_w4.cu -- products with 4-bit weights: y = x W^T for the few tokens of
// a decode step, and the two-tap dynamic conv (dynconv2.cu) whose tap
// projection is held the same way.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) * x[t, k]
//
// The inner sums run on the warp matrix instruction (m16n8k16, bf16 operands,
// fp32 sums) with 16 weight rows as the M side and 8 tokens as the N side: a
// block of 8 fills it.  The codes become exact bf16 integers (w4.cuh), so
// nothing is rounded before the fp32 sum; a chunk's sum is scaled and added to
// the row's in fp32.  fp32 activations are split into three bf16 planes whose
// sum is the value exactly (8 + 8 + 8 bits, each plane cut off, not rounded),
// three products into the same fp32 sum.
//
// Work: a cluster of S CTAs takes a range of 32-row units, each CTA one S-th of
// K, so its share of x stays in shared memory for all of them; the (unit,
// step) items of a CTA are cut into one contiguous run per warp, the sums of
// a unit's runs meet in shared memory (in K order, within the CTA and then over
// the cluster): no workspace, no atomics, one order of summation for a given
// shape and device.  Every warp streams its own run through a ring of
// asynchronous copies; a lane copies and reads its own pieces only, so the
// stream needs no barrier.
//
// Measured (8 tokens, groups of 128, bf16): 151,936 x 5,120 in 92 us, 4.4 TB/s of
// packed weights; the codes bound it before memory does: eight of them take three turns,
// four masks and four subtractions, 2.4 of 4 issue slots a cycle are taken and the logic
// pipe is 56 % busy.  5,120 x 5,120 with one token: 8.7 to 9.0 us, of which the stream is
// a third: x is laid out first and the cluster's sums joined last.
// More tokens than 16 go to linear_w4_tc.cu (bf16 activations).
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "linear_w4.cuh"
#include "stream.cuh"
#include "w4.cuh"

namespace dfl {

namespace cg = cooperative_groups;

constexpr int W4_WARPS = 16;
constexpr int W4_THREADS = 32 * W4_WARPS;
constexpr int W4_SMEM = 224 * 1024;  // dynamic shared memory a CTA may take

struct W4Args {
    const uint8_t* packed;
    int64_t N, K, units, tokens;
    const void* x;
    int64_t x_stride;
    int x_vec;           // rows of x start on 16 bytes
    void* y;             // linear: [tokens, N] in y_bf16's type; conv: [tokens, H] in x's
    int y_bf16;
    const void* x_prev;  // conv; NULL: linear
    int T;               // conv: tokens per sequence
    // plan
    int S, C;            // cluster size, clusters
    int steps;           // of K, one or two chunks each
    int tile;            // tokens per tile (8 NT at most)
    int phase, phases;   // steps of x in shared memory at a time, and how often
    int batch;           // units whose sums are in shared memory at a time
    int slots;           // partial sums per unit
    int x_off, part_off, counts_off;  // byte offsets in shared memory
};

// Shared memory of a step in a warp's ring: the lanes' 16-byte pieces of its
// chunks, then every lane's scales.  Lanes copy (and read) their own pieces
// only, so a warp's ring needs no barrier.
__host__ __device__ constexpr int w4_stage_bytes(int kb, int sg, int fmt) {
    return kb * W4_CHUNK_BYTES + sg * 32 * (w4_scale_bytes(fmt) / 8);
}
// Steps in the ring: what fits 7.5 KB a warp, two at least.
__host__ __device__ constexpr int w4_stages(int kb, int sg, int fmt) {
    const int n = 7680 / w4_stage_bytes(kb, sg, fmt);
    return n < 2 ? 2 : n;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void store_out(void* y, int64_t i, float v, bool bf16) {
    if (bf16)
        ((__nv_bfloat16*)y)[i] = __float2bfloat16_rn(v);  // the one rounding of a bf16 output
    else
        ((float*)y)[i] = v;
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight consecutive k of one token as bf16 words: NP planes of 4 words.
template <typename XT, int NP>
__device__ __forceinline__ void load_x8(const XT* row, int64_t k, int64_t K, bool vec,
                                        uint4 (&out)[NP]) {
    if constexpr (NP == 1) {
        if (vec && k + 8 <= K) {
            out[0] = __ldg((const uint4*)(row + k));
            return;
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t a = k + 2 * i;
            const uint32_t lo = a < K ? __ldg((const unsigned short*)row + a) : 0u;
            const uint32_t hi = a + 1 < K ? __ldg((const unsigned short*)row + a + 1) : 0u;
            w[i] = lo | (hi << 16);
        }
        out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float v[8];
        if (vec && k + 8 <= K) {
            const float4 a = __ldg((const float4*)(row + k)), b = __ldg((const float4*)(row + k + 4));
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + i < K ? __ldg((const float*)row + k + i) : 0.0f;
        }
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                // the upper 16 bits of an fp32 are its bf16 cut toward zero; the
                // rest is exact, and after two cuts it has 8 bits
                const uint32_t ua = __float_as_uint(a) & 0xFFFF0000u;
                const uint32_t ub = __float_as_uint(b) & 0xFFFF0000u;
                w[p][i] = (ua >> 16) | ub;
                a -= __uint_as_float(ua);
                b -= __uint_as_float(ub);
            }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
}

// XT: activation type; NT: 8-token tiles; FMT: scale format; G32: groups of
// 32 (two per chunk); KB: chunks per step (2 where the group is a multiple of
// 128: one scaling, one set of loads and one turn of the loop for 128 k).
template <typename XT, int NT, int FMT, bool G32, int KB>
__global__ void __launch_bounds__(W4_THREADS, 1) linear_w4_kernel(const W4Args a) {
    static_assert(!(G32 && KB > 1), "groups of 32 end inside a chunk");
    constexpr int NP = sizeof(XT) == 4 ? 3 : 1;
    constexpr int SG = G32 ? 2 : 1;  // scale groups per step
    constexpr int LB = W4Scale<FMT>::BYTES;
    constexpr int STAGE = w4_stage_bytes(KB, SG, FMT), D = w4_stages(KB, SG, FMT);
    constexpr int STEP = KB * W4_CHUNK_BYTES + SG * w4_scale_bytes(FMT);  // packed bytes
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.S, cl = blockIdx.x / a.S;
    const int64_t tok0 = (int64_t)blockIdx.y * a.tile;
    const int nt = (int)min((int64_t)a.tile, a.tokens - tok0);

    // this CTA's steps of K and units
    const int k0 = a.steps * rank / a.S, k1 = a.steps * (rank + 1) / a.S;
    const int64_t u0 = a.units * cl / a.C, u1 = a.units * (cl + 1) / a.C;

    // shared memory: the warps' rings, x [chunk][half][plane][8 NT tokens][32 k]
    // bf16 (64-byte rows), then the partial sums [unit of the batch][slot][NT * 8]
    // [32 lanes] fp32 and the units' slot counts
    constexpr int XROW = NT * 8 * 64, XSTEP = KB * 2 * NP * XROW;
    const uint32_t ring = smem_u32(smem + warp * (D * STAGE));
    const uint32_t ring_u = ring + lane * 16, ring_s = ring + KB * W4_CHUNK_BYTES + lane * LB;
    uint8_t* xs = smem + a.x_off;
    float* part = (float*)(smem + a.part_off);
    constexpr int PU = NT * 8 * 32;  // floats of one slot

    const int phases = a.phases;

    // n items are cut into min(warps, n) runs, none empty: run w is items
    // n w / R .. n (w + 1) / R - 1, so a unit's items lie in adjacent runs and
    // run w fills slot w - (the run of the unit's first item).
    // (n is at most 2^24, batch x steps of a phase)
    auto runs_of = [](int n) { return min(W4_WARPS, n); };
    auto run_of = [&](int i, int n) { return (int)((unsigned)((i + 1) * runs_of(n) - 1) / (unsigned)n); };

    // The run at hand, of batch ub and phase ph: its items are cu, cc (unit and
    // step) onward; `left` of them are not yet requested.
    int c0 = 0, nc = 0, n = 0, cu = 0, cc = 0, len = 0, left = 0, lc = 0;
    int64_t lu = 0;  // unit and step (of the run's part of K) of the next request
    const uint8_t* lw = nullptr;
    // the next step into a stage of the ring (an empty group at the run's end)
    auto request = [&](int stage) {
        if (left > 0) {
            --left;
            const uint32_t dst = ring_u + stage * STAGE;
            const uint8_t* src = lw + lane * 16;
#pragma unroll
            for (int q = 0; q < 2 * KB; ++q) cp_async16(dst + q * 512, src + q * 512);
            const uint32_t dsc = ring_s + stage * STAGE;
            const uint8_t* ssc = lw + KB * W4_CHUNK_BYTES + (lane >> 2) * LB;
#pragma unroll
            for (int h = 0; h < SG; ++h) {
                if constexpr (LB == 8) {
                    cp_async8(dsc + h * 32 * LB, ssc + h * 8 * LB);
                } else {
#pragma unroll
                    for (int q = 0; q < LB / 16; ++q)
                        cp_async16(dsc + h * 32 * LB + 16 * q, ssc + h * 8 * LB + 16 * q);
                }
            }
            lw += 4 * STEP;
            if (++lc == nc) {
                lc = 0;
                lw = a.packed + w4_block(++lu, a.steps, c0, STEP);
            }
        }
        cp_async_commit();
    };
    auto start = [&](int64_t ub, int ph) {
        const int nu = (int)min((int64_t)a.batch, u1 - ub);
        c0 = k0 + ph * a.phase;
        nc = max(0, min(a.phase, k1 - c0));
        n = nu * nc;
        const int runs = runs_of(n);
        const int i0 = warp < runs ? (int)((unsigned)(n * warp) / (unsigned)runs) : 0;
        const int i1 = warp < runs ? (int)((unsigned)(n * (warp + 1)) / (unsigned)runs) : 0;
        left = len = i1 - i0;
        cu = nc > 0 ? i0 / nc : 0;
        lc = cc = i0 - cu * nc;
        lu = ub + cu;
        lw = a.packed + w4_block(lu, a.steps, c0 + cc, STEP);
#pragma unroll
        for (int d = 0; d < D - 1; ++d) request(d);
    };

    start(u0, 0);
    for (int64_t ub = u0; ub < u1; ub += a.batch) {
        const int nu = (int)min((int64_t)a.batch, u1 - ub);
        for (int ph = 0; ph < phases; ++ph) {
            // x of this phase (kept over the batches when there is one phase)
            const bool new_x = phases > 1 || ub == u0;
            if (new_x) {
                const int items = nc * KB * 8 * nt;  // (chunk, half, 8 k) per token
                for (int i = threadIdx.x; i < items; i += W4_THREADS) {
                    const int c8 = i & 3, r = i >> 2;
                    const int ch = r / nt, t = r - ch * nt;  // ch = 2 * chunk + half
                    const XT* row = (const XT*)a.x + (tok0 + t) * a.x_stride;
                    uint4 v[NP];
                    load_x8<XT, NP>(row, (int64_t)(2 * KB * c0 + ch) * 32 + 8 * c8, a.K, a.x_vec != 0, v);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        *(uint4*)(xs + (size_t)(ch * NP + p) * XROW + t * 64 + c8 * 16) = v[p];
                }
                if (phases > 1 && ph == 0)
                    for (int i = threadIdx.x; i < nu * a.slots * PU; i += W4_THREADS) part[i] = 0.0f;
                __syncthreads();
            }
            // a lane's rows of x: tokens past the tile's last read that one's, and
            // their columns of the products are never looked at
            uint32_t xoff[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) xoff[t] = min(8 * t + (lane >> 2), nt - 1) * 64 + (lane & 3) * 16;
            float acc[2][NT][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[b][t][j] = 0.0f;
            const uint32_t xs_u = smem_u32(xs);
            uint32_t xc = xs_u + cc * XSTEP;
            for (int i0 = 0; i0 < len; i0 += D) {
#pragma unroll
              for (int d = 0; d < D; ++d) {  // the ring's stages in turn
                const int i = i0 + d;
                if (i >= len) break;
                cp_async_wait<D - 2>();
                request((d + D - 1) % D);  // the stage that the step before this one has left
                W4Scale<FMT> w4s[SG];
#pragma unroll
                for (int h = 0; h < SG; ++h) w4s[h].load_shared(ring_s + d * STAGE + h * 32 * LB);
                uint4 wv[KB][2];
#pragma unroll
                for (int c = 0; c < KB; ++c)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        wv[c][b] = lds128(ring_u + d * STAGE + c * W4_CHUNK_BYTES + b * 512);
                float s[2][NT][4];
#pragma unroll
                for (int h = 0; h < 2 * KB; ++h) {  // 32 k each: two matrix steps
                    const W4Scale<FMT>& ws = w4s[G32 ? h : 0];
                    if (h == 0 || G32) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int j = 0; j < 4; ++j) s[b][t][j] = 0.0f;
                    }
                    uint32_t A[2][2][4];  // [16-row half][matrix step]
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint4& w = wv[h >> 1][b];
                        const uint32_t wl = (h & 1) ? w.y : w.x, wh = (h & 1) ? w.w : w.z;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                A[b][q][2 * e] = w4_pair_exact(wl, 2 * q + e, ws.zero2(2 * b));
                                A[b][q][2 * e + 1] = w4_pair_exact(wh, 2 * q + e, ws.zero2(2 * b + 1));
                            }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            const uint4 xv = lds128(xc + xoff[t] + (h * NP + p) * XROW);
#pragma unroll
                            for (int b = 0; b < 2; ++b) mma_16816(s[b][t], A[b][0], xv.x, xv.y);
#pragma unroll
                            for (int b = 0; b < 2; ++b) mma_16816(s[b][t], A[b][1], xv.z, xv.w);
                        }
                        if (h == 2 * KB - 1 || G32)
#pragma unroll
                            for (int b = 0; b < 2; ++b)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    acc[b][t][j] = fmaf(ws.scale(2 * b + (j >> 1)), s[b][t][j], acc[b][t][j]);
                    }
                }
                xc += XSTEP;
                if (++cc == nc || i + 1 == len) {
                    // the run leaves the unit: its sum into the run's slot
                    const int first = run_of(cu * nc, n);
                    float* p = part + ((size_t)cu * a.slots + (warp - first)) * PU + lane;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float* q = p + ((b * NT + t) * 4 + j) * 32;
                                *q = phases > 1 ? *q + acc[b][t][j] : acc[b][t][j];
                                acc[b][t][j] = 0.0f;
                            }
                    cc = 0;
                    ++cu;
                    xc = xs_u;
                }
              }
            }
            // the next run's first steps are on their way while this one is wound up
            if (ph + 1 < phases) {
                start(ub, ph + 1);
                __syncthreads();  // x is replaced
            } else if (ub + a.batch < u1) {
                start(ub + a.batch, 0);
            }
        }

        // Sums of the batch: over the slots and then the cluster, in K order;
        // this CTA takes every S-th unit.  How many slots a unit has in CTA r
        // is worked out once per unit.
        uint8_t* counts = smem + a.counts_off;  // [S][batch]
        for (int i = threadIdx.x; i < a.S * nu; i += W4_THREADS) {
            const int r = i / nu, j = i - r * nu;
            int m = a.slots;
            if (phases == 1) {
                const int nc = a.steps * (r + 1) / a.S - a.steps * r / a.S;
                m = run_of(j * nc + nc - 1, nu * nc) - run_of(j * nc, nu * nc) + 1;
            }
            counts[r * a.batch + j] = (uint8_t)m;
        }
        if (a.S > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        auto unit_sum = [&](int j, int off) {  // off: position within the slot
            float v = 0.0f;
            const float* own = part + (size_t)j * a.slots * PU + off;
            for (int r = 0; r < a.S; ++r) {
                const float* base = a.S > 1 ? cg::this_cluster().map_shared_rank(own, r) : own;
                const int m = counts[r * a.batch + j];
                for (int q = 0; q < m; ++q) v += base[(size_t)q * PU];
            }
            return v;
        };
        // position of (row of the unit, token of the tile) in a slot
        auto slot_pos = [&](int row, int t) {
            const int b = row >> 4, rr = row & 15;
            return ((b * NT + (t >> 3)) * 4 + 2 * (rr >> 3) + (t & 1)) * 32 + (rr & 7) * 4 +
                   ((t & 7) >> 1);
        };
        const int mine = (nu - rank + a.S - 1) / a.S;
        if (!a.x_prev) {
            for (int i = threadIdx.x; i < mine * nt * W4_UNIT; i += W4_THREADS) {
                const int row = i & 31, r = i >> 5, t = r % nt, j = (r / nt) * a.S + rank;
                const int64_t nn = (ub + j) * W4_UNIT + row;
                const float v = unit_sum(j, slot_pos(row, t));
                if (nn < a.N) store_out(a.y, (tok0 + t) * a.N + nn, v, a.y_bf16 != 0);
            }
        } else {
            // rows 0..7 of a unit's halves are a, rows 8..15 b of the same 8 channels
            const XT* x = (const XT*)a.x;
            for (int i = threadIdx.x; i < mine * nt * 16; i += W4_THREADS) {
                const int c = i & 15, r = i >> 4, t = r % nt, j = (r / nt) * a.S + rank;
                const int64_t ch = (ub + j) * 16 + c, tok = tok0 + t;
                const int ra = (c & 8) * 2 + (c & 7);
                const float av = unit_sum(j, slot_pos(ra, t));
                const float bv = unit_sum(j, slot_pos(ra + 8, t));
                const float xc = to_f32(x[tok * a.K + ch]);
                const float xp = to_f32(tok % a.T == 0 ? ((const XT*)a.x_prev)[tok / a.T * a.K + ch]
                                                       : x[(tok - 1) * a.K + ch]);
                store_out(a.y, tok * a.K + ch, fmaf(bv, xp, fmaf(av, xc, xc)), a.y_bf16 != 0);
            }
        }
        // the sums are read (by the whole cluster) before they are replaced,
        // and before a CTA whose memory is still read may leave
        if (a.S > 1)
            cg::this_cluster().sync();
        else if (ub + a.batch < u1)
            __syncthreads();
    }
}

// Codes [N, K / 2] (the even k in the low half of a byte), scales and zero
// points [N, K / group] into the packed layout.  One thread per 16 bytes of
// weights, then one per scale entry.
__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* __restrict__ q,
                                                      const void* __restrict__ scale,
                                                      const uint8_t* __restrict__ zero,
                                                      W4Layout L, int format,
                                                      uint8_t* __restrict__ packed) {
    const bool taps = (format & DFLASH2_W4_TAPS) != 0;
    const bool f32s = (format & DFLASH2_W4_SCALE_F32) != 0;
    const int sbytes = w4_scale_bytes(format);
    const int64_t kg = L.K / L.group;  // groups per row as given
    // packed row -> row as given (taps: 8 rows of a, the same 8 of b)
    auto source = [&](int64_t r) {
        return taps ? (r / 16) * 8 + (r & 7) + ((r & 8) ? L.N / 2 : 0) : r;
    };
    auto zero_at = [&](int64_t row, int64_t g) -> uint32_t {
        if (!zero) return 8u;
        const uint32_t z = zero[row * kg + g];
        if (z > 15u) atomicOr(&g_dev_err, (unsigned)ERR_INPUT);
        return min(z, 15u);
    };
    const int64_t blocks = (L.units + 3) / 4 * 4 * L.steps;
    const int vecs = L.kb * (W4_CHUNK_BYTES / 16);  // per block
    const int64_t nv = blocks * vecs, ns = blocks * L.sg * W4_UNIT;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < nv + ns;
         i += (int64_t)gridDim.x * blockDim.x) {
        if (i < nv) {
            const int64_t blk = i / vecs, u = (blk >> 2) / L.steps * 4 + (blk & 3);
            const int v = (int)(i - blk * vecs), b = (v >> 5) & 1, lane = v & 31;
            const int64_t c = (blk >> 2) % L.steps * L.kb + (v >> 6);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // row r or r + 8, half h
                const int64_t row = u * W4_UNIT + 16 * b + (lane >> 2) + 8 * (j >> 1);
                const int64_t k = c * W4_CHUNK + 32 * (j & 1) + 8 * (lane & 3);
                if (row < L.N && k < L.K) {
                    const uint32_t in = *(const uint32_t*)(q + (source(row) * L.K + k) / 2);
                    uint32_t o = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o |= ((in >> (4 * e)) & 15u) << (4 * ((e >> 1) + 4 * (e & 1)));
                    w[j] = (o << 3) | (o >> 29);
                } else {
                    w[j] = 0x44444444u;  // eight codes of 8, turned by three bits
                }
            }
            *(uint4*)(packed + blk * L.step_bytes + v * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            const int64_t e = i - nv;
            const int j = (int)(e & 3), g8 = (int)((e >> 2) & 7);  // row = 8 j + g8
            const int64_t bg = e >> 5, blk = bg / L.sg, u = (blk >> 2) / L.steps * 4 + (blk & 3);
            const int h = (int)(bg - blk * L.sg);
            const int64_t row = u * W4_UNIT + 8 * j + g8;
            const int64_t g = ((blk >> 2) % L.steps * L.kb * W4_CHUNK + 32 * h) / L.group;
            const bool in = row < L.N && g < kg;
            const int64_t src = in ? source(row) * kg + g : 0;
            uint8_t* dst = packed + blk * L.step_bytes + L.kb * W4_CHUNK_BYTES + h * sbytes +
                           (size_t)g8 * (sbytes / 8);
            const unsigned short z16 =
                (unsigned short)(0x4180u + ((in ? zero_at(source(row), g) : 8u) << 3));
            if (f32s) {
                ((float*)dst)[j] = in ? ((const float*)scale)[src] : 0.0f;
                ((unsigned short*)(dst + 16))[j] = z16;
                ((unsigned short*)(dst + 24))[j] = 0;
            } else {
                ((unsigned short*)dst)[j] = in ? ((const unsigned short*)scale)[src] : 0;
                if (format & DFLASH2_W4_ZERO) ((unsigned short*)(dst + 8))[j] = z16;
            }
        }
    }
}

}  // namespace dfl

using namespace dfl;
using namespace dfl_host;

namespace {

bool device_info(W4Dev& d) {
    static std::mutex mu;
    static W4Dev known[64] = {};
    if (cudaGetDevice(&d.id) != cudaSuccess) return false;
    std::lock_guard<std::mutex> g(mu);
    if (d.id < 64 && known[d.id].clusters[1] > 0) {
        d = known[d.id];
        return true;
    }
    auto* k = linear_w4_kernel<__nv_bfloat16, 1, 0, false, 1>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM) != cudaSuccess)
        return false;
    for (int S = 1; S <= 8; S *= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)S * 128);
        cfg.blockDim = dim3(W4_THREADS);
        cfg.dynamicSmemBytes = W4_SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)S;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) return false;
        d.clusters[S] = std::max(1, n);
    }
    if (d.id < 64) known[d.id] = d;
    return true;
}

// Cluster size, clusters, and the shared-memory split of one call.
struct W4Plan {
    int S, C, tile, NT, KB, SG, steps, phase, phases, batch, slots, x_off, part_off, counts_off;
    size_t smem;
};
W4Plan w4_plan(const W4Layout& L, int format, int64_t tokens, bool x_f32, const W4Dev& d) {
    W4Plan best{};
    int64_t best_cost = -1;
    const int planes = x_f32 ? 3 : 1;
    const int NT = tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4;
    const int tile = (int)std::min<int64_t>(tokens, 8 * NT);
    const int KB = L.kb, SG = L.sg, fmt = format & (DFLASH2_W4_SCALE_F32 | DFLASH2_W4_ZERO);
    const int x_off = W4_WARPS * w4_stages(KB, SG, fmt & 2 ? 2 : fmt) * w4_stage_bytes(KB, SG, fmt & 2 ? 2 : fmt);
    const size_t slot = (size_t)NT * 8 * 32 * sizeof(float);
    const int steps = L.steps;
    for (int S = 1; S <= 8 && S <= steps; S *= 2) {
        W4Plan P{};
        P.S = S;
        P.NT = NT;
        P.tile = tile;
        P.KB = KB;
        P.SG = SG;
        P.steps = steps;
        P.C = (int)std::min<int64_t>(L.units, d.clusters[S]);
        const int kc = (steps + S - 1) / S;  // a CTA's share of K
        const int64_t cu = (L.units + P.C - 1) / P.C;
        const size_t xb = (size_t)KB * 2 * planes * 8 * NT * 64;  // bytes of a step's x
        // at most this much for x, the rest for the sums; phases of one length
        const int most_x = std::max(1, (int)((W4_SMEM - x_off - W4_WARPS * (slot + 8)) / xb));
        P.phases = (kc + most_x - 1) / most_x;
        P.phase = (kc + P.phases - 1) / P.phases;
        P.x_off = x_off;
        P.part_off = x_off + (int)(P.phase * xb);
        const size_t left = W4_SMEM - P.part_off;
        // a unit's items are in ceil((nc - 1) / shortest run) + 1 runs at most
        for (P.batch = (int)std::min<int64_t>(cu, left / slot); P.batch >= 1; --P.batch) {
            int most = 1;
            // the batches of the range: full ones and the last one; the phases
            // of a longer and of a shorter share of K
            for (int64_t nu : {(int64_t)P.batch, cu % P.batch, (cu - 1) % P.batch}) {
                if (nu <= 0) continue;
                for (int nc : {P.phase, kc - (P.phases - 1) * P.phase,
                               steps / S - (P.phases - 1) * P.phase, steps / S}) {
                    nc = std::min(nc, P.phase);
                    if (nc <= 0) continue;
                    const int64_t run = nu * nc / W4_WARPS;
                    const int64_t m = run == 0 ? nc : (nc - 1 + run - 1) / run + 1;
                    most = (int)std::max<int64_t>(most, std::min<int64_t>(m, W4_WARPS));
                }
            }
            P.slots = most;
            if (P.batch * (P.slots * slot + S) <= left) break;
        }
        P.counts_off = P.part_off + (int)(P.batch * P.slots * slot);
        P.smem = P.counts_off + (size_t)P.batch * S;
        // chunks a CTA streams, and some for the joining of each batch's sums and
        // for each filling of x (a chunk of a unit takes an SM about 25 ns)
        const int64_t batches = (cu + P.batch - 1) / P.batch;
        const int64_t fills = P.phases > 1 ? P.phases * batches : 1;
        const int64_t cost = cu * kc * KB + batches * (S > 1 ? 30 + 10 * S : 20) +
                             fills * (20 + (int64_t)P.phase * (int64_t)xb / 8192);
        if (best_cost < 0 || cost < best_cost) {
            best = P;
            best_cost = cost;
        }
    }
    return best;
}

template <typename XT, int NT, int FMT, bool G32, int KB>
int launch(const W4Args& a, const W4Plan& P, int dev, cudaStream_t s) {
    auto* k = linear_w4_kernel<XT, NT, FMT, G32, KB>;
    {
        static std::mutex mu;
        static bool attr_set[64] = {};
        std::lock_guard<std::mutex> g(mu);
        if (dev >= 64 || !attr_set[dev]) {
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W4_SMEM) !=
                cudaSuccess)
                return DFLASH2_ECUDA;
            if (dev < 64) attr_set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.S * P.C), (unsigned)((a.tokens + P.tile - 1) / P.tile));
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = P.smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)P.S;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a) == cudaSuccess ? DFLASH2_OK
                                                         : (cudaGetLastError(), DFLASH2_ECUDA);
}
template <typename XT, int FMT, bool G32, int KB>
int launch_nt(const W4Args& a, const W4Plan& P, int dev, cudaStream_t s) {
    switch (P.NT) {
        case 1: return launch<XT, 1, FMT, G32, KB>(a, P, dev, s);
        case 2: return launch<XT, 2, FMT, G32, KB>(a, P, dev, s);
        default: return launch<XT, 4, FMT, G32, KB>(a, P, dev, s);
    }
}
template <typename XT, int FMT>
int launch_group(const W4Args& a, const W4Plan& P, int dev, cudaStream_t s) {
    if (P.KB == 2) return launch_nt<XT, FMT, false, 2>(a, P, dev, s);
    return P.SG == 2 ? launch_nt<XT, FMT, true, 1>(a, P, dev, s)
                         : launch_nt<XT, FMT, false, 1>(a, P, dev, s);
}
template <typename XT>
int launch_fmt(const W4Args& a, const W4Plan& P, int format, int dev, cudaStream_t s) {
    if (format & DFLASH2_W4_SCALE_F32) return launch_group<XT, 2>(a, P, dev, s);
    if (format & DFLASH2_W4_ZERO) return launch_group<XT, 1>(a, P, dev, s);
    return launch_group<XT, 0>(a, P, dev, s);
}
int launch_any(const W4Args& a, const W4Plan& P, int format, bool x_f32, int dev, cudaStream_t s) {
    return x_f32 ? launch_fmt<float>(a, P, format, dev, s) : launch_fmt<__nv_bfloat16>(a, P, format, dev, s);
}

constexpr int W4_FORMATS = DFLASH2_W4_ZERO | DFLASH2_W4_SCALE_F32 | DFLASH2_W4_TAPS;
constexpr int64_t W4_MAX_TOKENS = 1 << 18;

// The plan of the few-token kernel, or NULL where the call goes to the tensor cores.
const W4Plan* few_plan(const W4Call& c, const W4Dev& d) {
    const bool tc = dfl_linear_w4_tc_ok(c);
    if (tc && c.tokens > W4_FEW_TOKENS) return nullptr;
    // the plan of the thread's last shape is kept: a decode calls the same ones over
    struct Last {
        int64_t N, K, tokens;
        int group, format, x_f32, dev;
        W4Plan P;
    };
    static thread_local Last last = {};
    if (last.N != c.L.N || last.K != c.L.K || last.tokens != c.tokens || last.group != c.L.group ||
        last.format != c.format || last.x_f32 != c.x_f32 || last.dev != d.id)
        last = {c.L.N, c.L.K, c.tokens, c.L.group, c.format, c.x_f32, d.id,
                w4_plan(c.L, c.format, c.tokens, c.x_f32, d)};
    return tc && c.tokens > 8 && last.P.phases > 2 ? nullptr : &last.P;
}

// A checked call: by token count and type to one of the two kernels.
int run(const W4Call& c, cudaStream_t s) {
    W4Dev d;
    if (!device_info(d)) return DFLASH2_ECUDA;
    const W4Plan* few = few_plan(c, d);
    if (!few) return dfl_linear_w4_tc(c, d, s);
    const W4Plan& P = *few;
    W4Args a{};
    a.packed = (const uint8_t*)c.packed;
    a.N = c.L.N;
    a.K = c.L.K;
    a.units = c.L.units;
    a.tokens = c.tokens;
    a.x = c.x;
    a.x_stride = c.x_stride;
    a.x_vec = c.x_vec;
    a.y = c.y;
    a.y_bf16 = c.y_bf16;
    a.x_prev = c.x_prev;
    a.T = c.T;
    a.S = P.S;
    a.C = P.C;
    a.steps = P.steps;
    a.tile = P.tile;
    a.phase = P.phase;
    a.phases = P.phases;
    a.batch = P.batch;
    a.slots = P.slots;
    a.x_off = P.x_off;
    a.part_off = P.part_off;
    a.counts_off = P.counts_off;
    return launch_any(a, P, c.format, c.x_f32, d.id, s);
}

}  // namespace

extern "C" size_t dflash2_w4_packed_bytes(int64_t N, int64_t K, int group, int format) {
    if (format < 0 || (format & ~W4_FORMATS) || !w4_shape_ok(N, K, group)) return 0;
    return w4_layout(N, K, group, format).total;
}

extern "C" int dflash2_w4_pack(const uint8_t* q, const void* scale, const uint8_t* zero, int64_t N,
                               int64_t K, int group, int format, void* packed,
                               dflash2_stream_t stream) {
    if (format < 0 || (format & ~W4_FORMATS)) return DFLASH2_EINVAL;
    if (!w4_shape_ok(N, K, group)) return DFLASH2_ESHAPE;
    if ((format & DFLASH2_W4_TAPS) && (N != 2 * K || K % 64 != 0)) return DFLASH2_ESHAPE;
    if (!q || !scale || !packed || ((format & DFLASH2_W4_ZERO) && !zero)) return DFLASH2_EINVAL;
    if (zero && !(format & DFLASH2_W4_ZERO)) return DFLASH2_EINVAL;
    if (!aligned(q, 16) || !aligned(scale, (format & DFLASH2_W4_SCALE_F32) ? 4 : 2) ||
        !aligned(packed, 256))
        return DFLASH2_EALIGN;
    const W4Layout L = w4_layout(N, K, group, format);
    const int64_t n = (int64_t)(L.total / L.step_bytes) * (L.kb * (W4_CHUNK_BYTES / 16) + L.sg * W4_UNIT);
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 148 * 32);
    w4_pack_kernel<<<blocks, 256, 0, (cudaStream_t)stream>>>(q, scale, zero, L, format,
                                                             (uint8_t*)packed);
    return launch_status();
}

extern "C" int dflash2_linear_w4(const void* x, int dtype, int64_t x_stride, int64_t tokens,
                                 const void* packed, int64_t N, int64_t K, int group, int format,
                                 void* y, int out_dtype, dflash2_stream_t stream) {
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return DFLASH2_EDTYPE;
    if (format < 0 || (format & ~(DFLASH2_W4_ZERO | DFLASH2_W4_SCALE_F32))) return DFLASH2_EINVAL;
    if (!w4_shape_ok(N, K, group) || tokens < 0 || tokens > W4_MAX_TOKENS || x_stride < K)
        return DFLASH2_ESHAPE;
    if (tokens == 0) return DFLASH2_OK;
    if (!x || !packed || !y) return DFLASH2_EINVAL;
    const int es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(packed, 256) || !aligned(y, elem_size(out_dtype)))
        return DFLASH2_EALIGN;
    W4Call c{};
    c.L = w4_layout(N, K, group, format);
    c.format = format;
    c.packed = packed;
    c.x = x;
    c.x_stride = x_stride;
    c.tokens = tokens;
    c.x_f32 = dtype == DFLASH2_F32;
    c.x_vec = aligned(x, 16) && (tokens == 1 || x_stride * es % 16 == 0);
    c.y = y;
    c.y_bf16 = out_dtype == DFLASH2_BF16;
    return run(c, (cudaStream_t)stream);
}

extern "C" int dflash2_linear_w4_plan(int64_t tokens, int64_t N, int64_t K, int group, int format,
                                      int dtype, int* tile, int* cluster) {
    if (!dtype_ok(dtype)) return DFLASH2_EDTYPE;
    if (format < 0 || (format & ~W4_FORMATS) || !tile || !cluster) return DFLASH2_EINVAL;
    if (!w4_shape_ok(N, K, group) || tokens < 1 || tokens > W4_MAX_TOKENS) return DFLASH2_ESHAPE;
    W4Dev d;
    if (!device_info(d)) return DFLASH2_ECUDA;
    W4Call c{};
    c.L = w4_layout(N, K, group, format);
    c.format = format & ~DFLASH2_W4_TAPS;
    c.tokens = tokens;
    c.x_f32 = dtype == DFLASH2_F32;
    c.x_vec = true;
    if (const W4Plan* few = few_plan(c, d)) {
        *tile = 0;
        *cluster = few->S;
    } else {
        const W4TcPlan P = dfl_linear_w4_tc_plan(c, d);
        *tile = P.ntok;
        *cluster = P.S;
    }
    return DFLASH2_OK;
}

extern "C" int dflash2_dynconv2_w4(const void* x, const void* x_prev, const void* packed, int group,
                                   int format, int dtype, int B, int T, int H, void* out,
                                   dflash2_stream_t stream) {
    if (!dtype_ok(dtype)) return DFLASH2_EDTYPE;
    if (format < 0 || (format & ~W4_FORMATS) || !(format & DFLASH2_W4_TAPS)) return DFLASH2_EINVAL;
    if (B < 0 || T < 0 || H < 64 || H % 64 != 0 || !w4_shape_ok(2 * (int64_t)H, H, group) ||
        (int64_t)B * T > W4_MAX_TOKENS)
        return DFLASH2_ESHAPE;
    if ((int64_t)B * T == 0) return DFLASH2_OK;
    if (!x || !x_prev || !packed || !out) return DFLASH2_EINVAL;
    if (!aligned(x, 16) || !aligned(x_prev, 16) || !aligned(packed, 256) || !aligned(out, 16))
        return DFLASH2_EALIGN;
    W4Call c{};
    c.L = w4_layout(2 * (int64_t)H, H, group, format);
    c.format = format & ~DFLASH2_W4_TAPS;
    c.packed = packed;
    c.x = x;
    c.x_stride = H;
    c.tokens = (int64_t)B * T;
    c.x_f32 = dtype == DFLASH2_F32;
    c.x_vec = true;
    c.y = out;
    c.y_bf16 = dtype == DFLASH2_BF16;
    c.x_prev = x_prev;
    c.T = T;
    return run(c, (cudaStream_t)stream);
}

unsigned dfl_errors_w4(int clear) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_dev_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    if (clear && v) {
        unsigned z = 0;
        cudaMemcpyToSymbol(g_dev_err, &z, sizeof z);
    }
    return v;
}

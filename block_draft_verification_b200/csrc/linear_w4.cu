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
// chunk) items of a CTA are cut into one contiguous run per warp, the sums of
// a unit's runs meet in shared memory (in K order, within the CTA and then over
// the cluster): no workspace, no atomics, one order of summation for a given
// shape and device.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "stream.cuh"
#include "w4.cuh"

namespace dfl {

namespace cg = cooperative_groups;

constexpr int W4_WARPS = 16;
constexpr int W4_THREADS = 32 * W4_WARPS;
constexpr int W4_SMEM = 224 * 1024;  // dynamic shared memory a CTA may take

struct W4Args {
    const uint8_t* weights;
    const uint8_t* scales;
    int64_t N, K, units, tokens;
    int chunks, groups, group;
    const void* x;
    int64_t x_stride;
    int x_vec;           // rows of x start on 16 bytes
    int gdiv;            // chunks per group, and the reciprocal that divides by it
    uint32_t gmagic;
    void* y;             // linear: [tokens, N] in y_bf16's type; conv: [tokens, H] in x's
    int y_bf16;
    const void* x_prev;  // conv; NULL: linear
    int T;               // conv: tokens per sequence
    // plan
    int S, C;            // cluster size, clusters
    int tile;            // tokens per tile (8 NT at most)
    int phase, phases;   // chunks of x in shared memory at a time, and how often
    int batch;           // units whose sums are in shared memory at a time
    int slots;           // partial sums per unit
};

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
// 32 (two per chunk).
template <typename XT, int NT, int FMT, bool G32>
__global__ void __launch_bounds__(W4_THREADS, 1) linear_w4_kernel(const W4Args a) {
    constexpr int NP = sizeof(XT) == 4 ? 3 : 1;
    constexpr int D = NT <= 2 ? 4 : 2;  // items in flight per warp
    constexpr int SG = G32 ? 2 : 1;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.S, cl = blockIdx.x / a.S;
    const int64_t tok0 = (int64_t)blockIdx.y * a.tile;
    const int nt = (int)min((int64_t)a.tile, a.tokens - tok0);

    const int ck0 = (int)((int64_t)a.chunks * rank / a.S);
    const int ck1 = (int)((int64_t)a.chunks * (rank + 1) / a.S);
    const int64_t u0 = a.units * cl / a.C, u1 = a.units * (cl + 1) / a.C;

    // shared memory: x [chunk][half][plane][token][32 k] bf16 (64-byte rows),
    // then the partial sums [unit of the batch][slot][NT * 8][32 lanes] fp32
    const int xrow = nt * 64, xchunk = 2 * NP * xrow;
    uint8_t* xs = smem;
    float* part = (float*)(smem + (size_t)a.phase * 2 * NP * a.tile * 64);
    constexpr int PU = NT * 8 * 32;  // floats of one slot

    const int phases = a.phases;

    // n items are cut into min(warps, n) runs, none empty: run w is items
    // n w / R .. n (w + 1) / R - 1, so a unit's items lie in adjacent runs and
    // run w fills slot w - (the run of the unit's first item).
    auto runs_of = [](int64_t n) { return (int)min((int64_t)W4_WARPS, n); };
    auto run_of = [&](int64_t i, int64_t n) { return (int)(((i + 1) * runs_of(n) - 1) / n); };

    for (int64_t ub = u0; ub < u1; ub += a.batch) {
        const int nu = (int)min((int64_t)a.batch, u1 - ub);
        for (int ph = 0; ph < phases; ++ph) {
            const int c0 = ck0 + ph * a.phase, nc = max(0, min(a.phase, ck1 - c0));
            const int64_t n = (int64_t)nu * nc;
            const int runs = runs_of(n);
            const int i0 = warp < runs ? (int)(n * warp / runs) : 0;
            const int i1 = warp < runs ? (int)(n * (warp + 1) / runs) : 0;

            // the run's first items are on their way while x is laid out
            uint4 wb[D][2];
            W4Scale<FMT> sb[D][SG];
            int lu = 0, lc = 0;  // unit and chunk of the next item to load
            if (nc > 0) {
                lu = i0 / nc;
                lc = i0 - lu * nc;
            }
            auto load = [&](int d) {
                const int64_t u = ub + lu;
                const int c = c0 + lc;
                const uint4* p = (const uint4*)(a.weights + (u * a.chunks + c) * W4_BLOCK) + lane;
                wb[d][0] = __ldcs(p);
                wb[d][1] = __ldcs(p + 32);
                const int g = G32 ? 2 * c : a.gdiv == 1 ? c : (int)__umulhi((unsigned)c, a.gmagic);
                const uint8_t* s = a.scales + (u * a.groups + g) * w4_scale_bytes(FMT);
#pragma unroll
                for (int h = 0; h < SG; ++h) sb[d][h].load(s + h * w4_scale_bytes(FMT), lane >> 2);
                if (++lc == nc) {
                    lc = 0;
                    ++lu;
                }
            };
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (i0 + d < i1) load(d);

            // x of this phase (kept over the batches when there is one phase)
            if (phases > 1 || ub == u0) {
                const int items = nc * 8 * nt;  // (chunk, half, 8 k) per token
                for (int i = threadIdx.x; i < items; i += W4_THREADS) {
                    const int c8 = i & 3, r = i >> 2;
                    const int t = r % nt, ch = r / nt;  // ch = 2 * chunk + half
                    const XT* row = (const XT*)a.x + (tok0 + t) * a.x_stride;
                    uint4 v[NP];
                    load_x8<XT, NP>(row, (int64_t)(2 * c0 + ch) * 32 + 8 * c8, a.K, a.x_vec != 0, v);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        *(uint4*)(xs + (size_t)(ch * NP + p) * xrow + t * 64 + c8 * 16) = v[p];
                }
            }
            if (phases > 1 && ph == 0)
                for (int i = threadIdx.x; i < nu * a.slots * PU; i += W4_THREADS) part[i] = 0.0f;
            __syncthreads();

            float acc[2][NT][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[b][t][j] = 0.0f;
            int cu = 0, cc = 0;  // unit and chunk of the item at hand
            if (nc > 0) {
                cu = i0 / nc;
                cc = i0 - cu * nc;
            }
            for (int i = i0; i < i1; i += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (i + d < i1) {
                        // operands of the 16-row halves: [half b][k step][4]
                        uint32_t A[2][4][4];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t w[4] = {wb[d][b].x, wb[d][b].y, wb[d][b].z, wb[d][b].w};
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const W4Scale<FMT>& s = sb[d][G32 ? h : 0];
                                const uint32_t zl = s.zero2(2 * b), zh = s.zero2(2 * b + 1);
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    A[b][2 * h + q][0] = w4_pair(w[h], 2 * q, zl);
                                    A[b][2 * h + q][1] = w4_pair(w[2 + h], 2 * q, zh);
                                    A[b][2 * h + q][2] = w4_pair(w[h], 2 * q + 1, zl);
                                    A[b][2 * h + q][3] = w4_pair(w[2 + h], 2 * q + 1, zh);
                                }
                            }
                        }
                        float sc[SG][4];
#pragma unroll
                        for (int h = 0; h < SG; ++h)
#pragma unroll
                            for (int j = 0; j < 4; ++j) sc[h][j] = sb[d][h].scale(j);
                        if (i + d + D < i1) load(d);
                        const uint8_t* xc = xs + (size_t)cc * xchunk + lane * 16;
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const bool live = 8 * t + (lane >> 2) < nt;
                            float s[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h == 0 || G32)
#pragma unroll
                                    for (int b = 0; b < 2; ++b)
#pragma unroll
                                        for (int j = 0; j < 4; ++j) s[b][j] = 0.0f;
#pragma unroll
                                for (int p = 0; p < NP; ++p) {
                                    uint4 xv = make_uint4(0, 0, 0, 0);
                                    if (live)
                                        xv = *(const uint4*)(xc + (h * NP + p) * xrow + t * 512);
#pragma unroll
                                    for (int b = 0; b < 2; ++b) {
                                        mma_16816(s[b], A[b][2 * h], xv.x, xv.y);
                                        mma_16816(s[b], A[b][2 * h + 1], xv.z, xv.w);
                                    }
                                }
                                if (h == 1 || G32)
#pragma unroll
                                    for (int b = 0; b < 2; ++b)
#pragma unroll
                                        for (int j = 0; j < 4; ++j)
                                            acc[b][t][j] = fmaf(sc[G32 ? h : 0][2 * b + (j >> 1)],
                                                                s[b][j], acc[b][t][j]);
                            }
                        }
                        if (++cc == nc || i + d + 1 == i1) {
                            // the run leaves the unit: its sum into the run's slot
                            const int first = run_of((int64_t)cu * nc, n);
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
                        }
                    }
                }
            }
            if (ph + 1 < phases) __syncthreads();  // x is replaced
        }

        // Sums of the batch: over the slots and then the cluster, in K order;
        // this CTA takes every S-th unit.
        if (a.S > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        auto unit_sum = [&](int j, int off) {  // off: position within the slot
            float v = 0.0f;
            for (int r = 0; r < a.S; ++r) {
                const float* base = a.S > 1 ? cg::this_cluster().map_shared_rank(part, r) : part;
                int m = a.slots;
                const int nc = (int)((int64_t)a.chunks * (r + 1) / a.S) -
                               (int)((int64_t)a.chunks * r / a.S);
                if (phases == 1) {
                    const int64_t n = (int64_t)nu * nc;
                    m = nc > 0 ? run_of((int64_t)j * nc + nc - 1, n) - run_of((int64_t)j * nc, n) + 1
                               : 0;
                }
                base += (size_t)j * a.slots * PU + off;
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
            // rows 0..15 of a unit are a, rows 16..31 b of the same 16 channels
            const XT* x = (const XT*)a.x;
            for (int i = threadIdx.x; i < mine * nt * 16; i += W4_THREADS) {
                const int c = i & 15, r = i >> 4, t = r % nt, j = (r / nt) * a.S + rank;
                const int64_t ch = (ub + j) * 16 + c, tok = tok0 + t;
                const float av = unit_sum(j, slot_pos(c, t));
                const float bv = unit_sum(j, slot_pos(16 + c, t));
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
    const int64_t kg = L.K / L.group;  // groups per row as given
    // packed row -> row as given (taps: 16 rows of a, the same 16 of b)
    auto source = [&](int64_t r) {
        return taps ? (r / 32) * 16 + (r & 15) + ((r & 16) ? L.N / 2 : 0) : r;
    };
    auto zero_at = [&](int64_t row, int64_t g) -> uint32_t {
        if (!zero) return 8u;
        const uint32_t z = zero[row * kg + g];
        if (z > 15u) atomicOr(&g_dev_err, (unsigned)ERR_INPUT);
        return min(z, 15u);
    };
    const int64_t nv = L.units * L.chunks * (W4_BLOCK / 16);
    const int64_t ns = L.units * L.groups * W4_UNIT;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < nv + ns;
         i += (int64_t)gridDim.x * blockDim.x) {
        if (i < nv) {
            const int64_t blk = i >> 6;
            const int v = (int)(i & 63), b = v >> 5, lane = v & 31;
            const int64_t u = blk / L.chunks;
            const int c = (int)(blk - u * L.chunks);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // row r or r + 8, half h
                const int64_t row = u * W4_UNIT + 16 * b + (lane >> 2) + 8 * (j >> 1);
                const int64_t k = (int64_t)c * W4_CHUNK + 32 * (j & 1) + 8 * (lane & 3);
                if (row < L.N && k < L.K) {
                    const int64_t src = source(row);
                    const uint32_t in = *(const uint32_t*)(q + (src * L.K + k) / 2);
                    uint32_t o = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o |= ((in >> (4 * e)) & 15u) << (4 * ((e >> 1) + 4 * (e & 1)));
                    w[j] = o;
                } else {
                    // K tail: codes equal to the zero point of the group that the
                    // chunk's first half is scaled with (groups of 32 have scale 0 there)
                    w[j] = 0x88888888u;
                }
            }
            *(uint4*)(packed + blk * W4_BLOCK + v * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            const int64_t e = i - nv;
            const int j = (int)(e & 3), g8 = (int)((e >> 2) & 7);  // row = 8 j + g8
            const int64_t ug = e >> 5, u = ug / L.groups, g = ug - u * L.groups;
            const int64_t row = u * W4_UNIT + 8 * j + g8;
            const bool in = row < L.N && g < kg;
            const int64_t src = in ? source(row) * kg + g : 0;
            uint8_t* dst = packed + L.scale_off + ug * L.sbytes + (size_t)g8 * (L.sbytes / 8);
            const unsigned short z16 =
                (unsigned short)(0x4300u + (in ? zero_at(source(row), g) : 8u));
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

struct Dev {
    int id, sms;
};
bool device_info(Dev& d) {
    return cudaGetDevice(&d.id) == cudaSuccess &&
           cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.id) == cudaSuccess;
}

// Cluster size, clusters, and the shared-memory split of one call.
struct W4Plan {
    int S, C, tile, NT, phase, batch, slots;
    size_t smem;
};
W4Plan w4_plan(const W4Layout& L, int64_t tokens, int planes, int sms) {
    W4Plan best{};
    int64_t best_cost = -1;
    const int NT = tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4;
    const int tile = (int)std::min<int64_t>(tokens, 8 * NT);
    const size_t slot = (size_t)NT * 8 * 32 * sizeof(float);
    for (int S = 1; S <= 8 && S <= L.chunks; S *= 2) {
        W4Plan P{};
        P.S = S;
        P.NT = NT;
        P.tile = tile;
        P.C = (int)std::min<int64_t>(L.units, std::max(1, sms / S));
        const int kc = (L.chunks + S - 1) / S;  // a CTA's share of K
        const int64_t cu = (L.units + P.C - 1) / P.C;
        const size_t xc = (size_t)2 * planes * tile * 64;  // bytes of x per chunk
        // at most this much for x, the rest for the sums
        P.phase = (int)std::min<int64_t>(kc, (int64_t)(160 * 1024 / xc));
        const size_t left = W4_SMEM - P.phase * xc;
        // a unit's items are in ceil((nc - 1) / shortest run) + 1 runs at most
        for (P.batch = (int)std::min<int64_t>(cu, 1024); P.batch >= 1; --P.batch) {
            int most = 1;
            // the batches of the range: full ones and the last one
            for (int64_t nu : {(int64_t)P.batch, cu % P.batch, (cu - 1) % P.batch}) {
                if (nu <= 0) continue;
                for (int nc : {P.phase, kc % P.phase, (L.chunks / S) % P.phase, L.chunks / S}) {
                    nc = std::min(nc, P.phase);
                    if (nc <= 0) continue;
                    const int64_t run = nu * nc / W4_WARPS;
                    const int64_t m = run == 0 ? nc : (nc - 1 + run - 1) / run + 1;
                    most = (int)std::max<int64_t>(most, std::min<int64_t>(m, W4_WARPS));
                }
            }
            P.slots = most;
            if ((size_t)P.batch * P.slots * slot <= left) break;
        }
        P.smem = P.phase * xc + (size_t)P.batch * P.slots * slot;
        // items a CTA streams, and about a microsecond's worth for the cluster's barriers
        const int64_t cost = cu * kc + (S > 1 ? 40 : 0);
        if (best_cost < 0 || cost < best_cost) {
            best = P;
            best_cost = cost;
        }
    }
    return best;
}

template <typename XT, int NT, int FMT, bool G32>
int launch(const W4Args& a, const W4Plan& P, int dev, cudaStream_t s) {
    auto* k = linear_w4_kernel<XT, NT, FMT, G32>;
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
template <typename XT, int FMT, bool G32>
int launch_nt(const W4Args& a, const W4Plan& P, int dev, cudaStream_t s) {
    switch (P.NT) {
        case 1: return launch<XT, 1, FMT, G32>(a, P, dev, s);
        case 2: return launch<XT, 2, FMT, G32>(a, P, dev, s);
        default: return launch<XT, 4, FMT, G32>(a, P, dev, s);
    }
}
template <typename XT>
int launch_fmt(const W4Args& a, const W4Plan& P, int format, int dev, cudaStream_t s) {
    const bool g32 = a.group == 32;
    if (format & DFLASH2_W4_SCALE_F32)
        return g32 ? launch_nt<XT, 2, true>(a, P, dev, s)
                   : launch_nt<XT, 2, false>(a, P, dev, s);
    if (format & DFLASH2_W4_ZERO)
        return g32 ? launch_nt<XT, 1, true>(a, P, dev, s)
                   : launch_nt<XT, 1, false>(a, P, dev, s);
    return g32 ? launch_nt<XT, 0, true>(a, P, dev, s)
               : launch_nt<XT, 0, false>(a, P, dev, s);
}

constexpr int W4_FORMATS = DFLASH2_W4_ZERO | DFLASH2_W4_SCALE_F32 | DFLASH2_W4_TAPS;
constexpr int64_t W4_MAX_TOKENS = 1 << 18;

W4Args w4_args(const W4Layout& L, const W4Plan& P, const void* packed) {
    W4Args a{};
    a.weights = (const uint8_t*)packed;
    a.scales = (const uint8_t*)packed + L.scale_off;
    a.N = L.N;
    a.K = L.K;
    a.units = L.units;
    a.chunks = L.chunks;
    a.groups = L.groups;
    a.group = L.group;
    a.S = P.S;
    a.C = P.C;
    a.tile = P.tile;
    a.phase = P.phase;
    a.phases = ((L.chunks + P.S - 1) / P.S + P.phase - 1) / P.phase;
    a.gdiv = std::max(1, L.group / W4_CHUNK);
    // ceil(2^32 / gdiv): exact for chunk * gdiv < 2^32, and both are at most 2^14
    a.gmagic = (uint32_t)(((1ull << 32) + a.gdiv - 1) / a.gdiv);
    a.batch = P.batch;
    a.slots = P.slots;
    return a;
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
    const int64_t n = L.units * L.chunks * (W4_BLOCK / 16) + L.units * L.groups * W4_UNIT;
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
    Dev d;
    if (!device_info(d)) return DFLASH2_ECUDA;
    const W4Layout L = w4_layout(N, K, group, format);
    const W4Plan P = w4_plan(L, tokens, dtype == DFLASH2_F32 ? 3 : 1, d.sms);
    W4Args a = w4_args(L, P, packed);
    a.x = x;
    a.x_stride = x_stride;
    a.x_vec = aligned(x, 16) && (tokens == 1 || x_stride * es % 16 == 0);
    a.tokens = tokens;
    a.y = y;
    a.y_bf16 = out_dtype == DFLASH2_BF16;
    cudaStream_t s = (cudaStream_t)stream;
    return dtype == DFLASH2_BF16 ? launch_fmt<__nv_bfloat16>(a, P, format, d.id, s)
                                 : launch_fmt<float>(a, P, format, d.id, s);
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
    Dev d;
    if (!device_info(d)) return DFLASH2_ECUDA;
    const int64_t tokens = (int64_t)B * T;
    const W4Layout L = w4_layout(2 * (int64_t)H, H, group, format);
    const W4Plan P = w4_plan(L, tokens, dtype == DFLASH2_F32 ? 3 : 1, d.sms);
    W4Args a = w4_args(L, P, packed);
    a.x = x;
    a.x_stride = H;
    a.x_vec = 1;
    a.x_prev = x_prev;
    a.T = T;
    a.tokens = tokens;
    a.y = out;
    a.y_bf16 = dtype == DFLASH2_BF16;
    cudaStream_t s = (cudaStream_t)stream;
    const int fmt = format & ~DFLASH2_W4_TAPS;
    return dtype == DFLASH2_BF16 ? launch_fmt<__nv_bfloat16>(a, P, fmt, d.id, s)
                                 : launch_fmt<float>(a, P, fmt, d.id, s);
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

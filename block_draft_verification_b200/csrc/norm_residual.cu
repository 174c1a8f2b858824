// norm_residual.cu -- the norms around a block, fused with the block's gate and
// residual scale:
//
//   r' = r + alpha * act(g) * rms(y; w_post),   h = rms(r'; w_pre),
//   rms(v; w)_i = v_i / sqrt(mean_j v_j^2 + eps) * (w_i + w_offset)
//
// One pass over memory: a row's y and r are read once, kept in registers while
// the sum of squares of y, then of r', is formed in fp32, and r' and h are
// written once.  h is taken from r' before its rounding.  A row is worked on
// by one CTA sized to it; rows too long for its registers are read again from
// cache (three passes).
//
// Sums of squares that leave fp32's range are formed again from the row scaled by a
// power of two, so finite rows of any size are right; no other row pays more than a test.
//
// Measured: 4,096 rows of 5,120 with an fp32 residual and a gate per token in 50 us,
// 5.9 TB/s (91 % of the copy rate; two vectors a thread, 320 threads); 256 rows in 4.8 us and 8 rows in
// 3.9 us, which is the two barriers and a launch; 1,001 rows of 6,001, by element in three
// passes, in 40 us, 1.5 TB/s.
#include <cfloat>

#include "common.cuh"

namespace dfl {

struct NormArgs {
    const void* res;
    const void* y;
    const void* gate;    // NULL: none
    const void* w_post;  // NULL: y is taken as it is
    const void* w_pre;   // NULL: no second norm, h is not written
    void* res_out;
    void* h;
    int64_t rows, H, res_stride, y_stride, gate_stride, gate_rep;
    float alpha, eps, w_offset;
    int sigmoid;
};

// W consecutive elements as they are stored (W = 8: 16-byte loads, W = 1: one
// element), widened to fp32 when used.
template <typename T, int W>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *(const uint4*)p; }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? q.x : i < 4 ? q.y : i < 6 ? q.z : q.w;
        return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
};
template <>
struct Pack<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *(const float4*)p;
        b = *(const float4*)(p + 4);
    }
    __device__ __forceinline__ float get(int i) const {
        const float4& v = i < 4 ? a : b;
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *p; }
    __device__ __forceinline__ float get(int) const { return __bfloat162float(q); }
};
template <>
struct Pack<float, 1> {
    float q;
    __device__ __forceinline__ void load(const float* p) { q = *p; }
    __device__ __forceinline__ float get(int) const { return q; }
};
__device__ __forceinline__ void store_pack(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_pack(float* p, const float (&v)[8]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_pack(__nv_bfloat16* p, const float (&v)[1]) {
    *p = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void store_pack(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ float ld_1(const float* p) { return *p; }
__device__ __forceinline__ float ld_1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float act(float g, int sigmoid) {
    if (!sigmoid) return g;
    float r;  // within one unit in the last place, for a division's worth of instructions less
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-g)));
    return r;
}

// Sum over the block, the same value in every thread (`buf`: 32 floats, to be used
// again one barrier later).
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) v += __shfl_xor_sync(FULL, v, j);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < nw ? buf[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) v += __shfl_xor_sync(FULL, v, j);
    return v;
}

// Whether fp32 holds a mean square (with eps) in full: not where values lie beyond about
// 1e19 / sqrt(H), nor where all lie below 1e-18 with no eps to cover them.
__device__ __forceinline__ bool in_range(float m) { return m >= 0x1p-120f && m <= FLT_MAX; }

// 1 / sqrt(sum / H + eps), `sum` a row's sum of squares.  Out of range, the row is summed
// once more, `again(c)` the thread's sum of (c v)^2 with c a power of two that brings it
// back; the whole block takes the same branch.
template <typename Again>
__device__ __forceinline__ float inv_rms(float sum, float H, float eps, float* buf, const Again& again) {
    float m = sum / H + eps;
    if (in_range(m)) return rsqrtf(m);
    const float c = m > 1.0f ? 0x1p-80f : 0x1p100f;
    __syncthreads();  // `buf` is read
    m = block_sum(again(c), buf) / H + eps * c * c;
    return c * rsqrtf(m);
}

// XT: y, gate, weights and h; RT: the residual; a thread holds V packs of W
// elements of the row (blockDim V W >= H; W = 8 wants H a multiple of 8 and
// 16-byte rows, W = 1 takes any).  A row's y, residual and gate are requested before
// its first sum; the weights ahead of the sum before their use where they are at most 32
// bytes a thread (requested behind it, 256 rows of 5,120 take 5.2 us instead of 4.8; with
// more bytes ahead, 1,024 fp32 rows of 16,384 take 87 instead of 79).  A CTA takes one
// row: in a loop over rows the two packs of 5,120 bf16 columns take 94 registers a thread
// and two rows fit an SM, without it about 60 and three (63.6 and 52.9 us at 4,096 rows).
template <typename XT, typename RT, int W, int V>
__global__ void __launch_bounds__(512) norm_residual_kernel(const NormArgs a) {
    __shared__ float buf[2][32];
    const int np = (int)(a.H / W);
    const int64_t row = blockIdx.x;
    const XT* y = (const XT*)a.y + row * a.y_stride;
    const RT* r = (const RT*)a.res + row * a.res_stride;
    const XT* g = a.gate ? (const XT*)a.gate + row / a.gate_rep * a.gate_stride : nullptr;
    Pack<XT, W> py[V], pg[V];
    Pack<RT, W> pr[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int q = threadIdx.x + i * blockDim.x;
        if (q < np) {
            py[i].load(y + W * q);
            pr[i].load(r + W * q);
            if (g) pg[i].load(g + W * q);
        }
    }
    float inv = a.alpha;
    Pack<XT, W> pw[V];  // of w_post, then of w_pre
    constexpr bool EARLY = V * W * sizeof(XT) <= 32;
    auto load_w = [&](const void* w, int i) {
        const int q = threadIdx.x + i * blockDim.x;
        if (q < np) pw[i].load((const XT*)w + W * q);
    };
    if (a.w_post) {
        if (EARLY)
#pragma unroll
            for (int i = 0; i < V; ++i) load_w(a.w_post, i);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (threadIdx.x + i * blockDim.x < np)
#pragma unroll
                for (int e = 0; e < W; ++e) ss = fmaf(py[i].get(e), py[i].get(e), ss);
        inv *= inv_rms(block_sum(ss, buf[0]), (float)a.H, a.eps, buf[0], [&](float c) {
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (threadIdx.x + i * blockDim.x < np)
#pragma unroll
                    for (int e = 0; e < W; ++e) t = fmaf(c * py[i].get(e), c * py[i].get(e), t);
            return t;
        });
    }
    float vr[V][W];
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int q = threadIdx.x + i * blockDim.x;
        if (q < np) {
            if (!EARLY && a.w_post) load_w(a.w_post, i);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float f = inv;
                if (a.w_post) f *= pw[i].get(e) + a.w_offset;
                if (g) f *= act(pg[i].get(e), a.sigmoid);
                vr[i][e] = fmaf(f, py[i].get(e), pr[i].get(e));
                s2 = fmaf(vr[i][e], vr[i][e], s2);
            }
            store_pack((RT*)a.res_out + row * a.H + W * q, vr[i]);
        }
    }
    if (a.w_pre) {
        if (EARLY)
#pragma unroll
            for (int i = 0; i < V; ++i) load_w(a.w_pre, i);
        const float inv2 = inv_rms(block_sum(s2, buf[1]), (float)a.H, a.eps, buf[1], [&](float c) {
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (threadIdx.x + i * blockDim.x < np)
#pragma unroll
                    for (int e = 0; e < W; ++e) t = fmaf(c * vr[i][e], c * vr[i][e], t);
            return t;
        });
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int q = threadIdx.x + i * blockDim.x;
            if (q < np) {
                if (!EARLY) load_w(a.w_pre, i);
                float o[W];
#pragma unroll
                for (int e = 0; e < W; ++e) o[e] = vr[i][e] * inv2 * (pw[i].get(e) + a.w_offset);
                store_pack((XT*)a.h + row * a.H + W * q, o);
            }
        }
    }
}

// A row of any width, stride and alignment: element by element, y and r read again from
// cache after each sum.  r' is recomputed in the last pass, not read back, so that h comes
// from the unrounded value; where the output is written over the residual, r' is written
// only after its last read.  A row with a sum out of range returns false, with nothing
// written, unless SCALED, which takes such a sum once more of c v.
template <typename XT, typename RT, bool SCALED>
__device__ __forceinline__ bool row_by_element(const NormArgs& a, int64_t row, float* buf) {
    constexpr int U = SCALED ? 1 : 4;  // loads in flight
    const XT* y = (const XT*)a.y + row * a.y_stride;
    const RT* r = (const RT*)a.res + row * a.res_stride;
    const XT* g = a.gate ? (const XT*)a.gate + row / a.gate_rep * a.gate_stride : nullptr;
    const XT* wpost = (const XT*)a.w_post;
    const XT* wpre = (const XT*)a.w_pre;
    // 1 / sqrt(mean square + eps) of value(0) .. value(H - 1), or 0 for out of range
    auto inv_rms = [&](float* buf, auto&& value) {
        float c = 1.0f;
        for (;;) {
            float t = 0.0f;
#pragma unroll U
            for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
                const float v = SCALED ? c * value(i) : value(i);
                t = fmaf(v, v, t);
            }
            if (SCALED) __syncthreads();  // `buf` is read
            const float m = block_sum(t, buf) / (float)a.H + (SCALED ? a.eps * c * c : a.eps);
            if (!SCALED) return in_range(m) ? rsqrtf(m) : 0.0f;
            if (in_range(m) || c != 1.0f) return c * rsqrtf(m);
            c = m > 1.0f ? 0x1p-80f : 0x1p100f;
        }
    };
    float inv = a.alpha;
    if (wpost) {
        const float f = inv_rms(buf, [&](int64_t i) { return ld_1(y + i); });
        if (!SCALED && f == 0.0f) return false;
        inv *= f;
    }
    auto sum_at = [&](int64_t i) {
        float f = inv;
        if (wpost) f *= ld_1(wpost + i) + a.w_offset;
        if (g) f *= act(ld_1(g + i), a.sigmoid);
        return fmaf(f, ld_1(y + i), ld_1(r + i));
    };
    float inv2 = 0.0f;
    if (wpre) {
        inv2 = inv_rms(buf + 32, sum_at);
        if (!SCALED && inv2 == 0.0f) return false;
    }
#pragma unroll U
    for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float v = sum_at(i);
        st_1((RT*)a.res_out + row * a.H + i, v);
        if (wpre) st_1((XT*)a.h + row * a.H + i, v * inv2 * (ld_1(wpre + i) + a.w_offset));
    }
    return true;
}
template <typename XT, typename RT>
__global__ void __launch_bounds__(512) norm_residual_any_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float buf[64];
    if (!row_by_element<XT, RT, false>(a, blockIdx.x, buf)) row_by_element<XT, RT, true>(a, blockIdx.x, buf);
}

}  // namespace dfl

using namespace dfl;
using namespace dfl_host;

namespace {

template <typename XT, typename RT>
int launch(const NormArgs& a, bool vec, cudaStream_t s) {
    const unsigned grid = (unsigned)a.rows;  // at most 2^30
    // packs of a row; up to 512 threads take V of them each, all but evenly
    const int64_t np = vec ? a.H / 8 : a.H;
    auto threads = [&](int v) { return (int)(((np + v - 1) / v + 31) / 32 * 32); };
    if (vec && np <= 4 * 512) {
        if (np <= 512)
            norm_residual_kernel<XT, RT, 8, 1><<<grid, threads(1), 0, s>>>(a);
        else if (np <= 2 * 512)
            norm_residual_kernel<XT, RT, 8, 2><<<grid, threads(2), 0, s>>>(a);
        else
            norm_residual_kernel<XT, RT, 8, 4><<<grid, threads(4), 0, s>>>(a);
    } else if (!vec && np <= 8 * 512) {
        if (np <= 2 * 512)
            norm_residual_kernel<XT, RT, 1, 4><<<grid, threads(4), 0, s>>>(a);
        else
            norm_residual_kernel<XT, RT, 1, 8><<<grid, threads(8), 0, s>>>(a);
    } else {
        norm_residual_any_kernel<XT, RT><<<grid, 512, 0, s>>>(a);
    }
    return launch_status();
}

}  // namespace

extern "C" int dflash2_norm_residual(const void* res, int res_dtype, int64_t res_stride,
                                     const void* y, int dtype, int64_t y_stride, const void* gate,
                                     int64_t gate_stride, int64_t gate_rep, int gate_act,
                                     const void* w_post, const void* w_pre, float w_offset,
                                     float alpha, float eps, int64_t rows, int64_t H,
                                     void* res_out, void* h, dflash2_stream_t stream) {
    if (!dtype_ok(dtype) || !dtype_ok(res_dtype)) return DFLASH2_EDTYPE;
    if (dtype == DFLASH2_F32 && res_dtype == DFLASH2_BF16) return DFLASH2_EDTYPE;
    if (rows < 0 || rows > (1 << 30) || H < 1 || H > (1 << 24) || res_stride < H || y_stride < H)
        return DFLASH2_ESHAPE;
    if (gate && (gate_rep < 1 || (gate_stride < H && gate_rep < rows))) return DFLASH2_ESHAPE;
    if (!isfinite(alpha) || !isfinite(w_offset) || !isfinite(eps) || eps < 0.0f) return DFLASH2_EINVAL;
    if (gate_act != DFLASH2_GATE_LINEAR && gate_act != DFLASH2_GATE_SIGMOID) return DFLASH2_EINVAL;
    if (rows == 0) return DFLASH2_OK;
    if (!res || !y || !res_out || (w_pre != nullptr) != (h != nullptr)) return DFLASH2_EINVAL;
    const size_t es = (size_t)elem_size(dtype), rs = (size_t)elem_size(res_dtype);
    if (!aligned(res, rs) || !aligned(y, es) || !aligned(gate, es) || !aligned(w_post, es) ||
        !aligned(w_pre, es) || !aligned(res_out, rs) || !aligned(h, es))
        return DFLASH2_EALIGN;
    if (res_out == res && res_stride != H && rows > 1) return DFLASH2_EINVAL;  // rows would overlap
    // 16-byte loads where every row of every operand starts on 16 bytes
    const bool vec = H % 8 == 0 && aligned(res, 16) && aligned(y, 16) && aligned(gate, 16) &&
                     aligned(w_post, 16) && aligned(w_pre, 16) && aligned(res_out, 16) &&
                     aligned(h, 16) &&
                     (rows == 1 || (res_stride * rs % 16 == 0 && y_stride * es % 16 == 0)) &&
                     (!gate || gate_rep >= rows || gate_stride * es % 16 == 0);
    NormArgs a{res, y, gate, w_post, w_pre, res_out, h, rows, H, res_stride, y_stride, gate_stride,
               gate ? gate_rep : 1, alpha, eps, w_offset, gate_act == DFLASH2_GATE_SIGMOID};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == DFLASH2_F32) return launch<float, float>(a, vec, s);
    return res_dtype == DFLASH2_F32 ? launch<__nv_bfloat16, float>(a, vec, s)
                                    : launch<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}

// w4.cuh -- 4-bit weights with group scales: the packed layout every kernel
// that reads them shares, and the step from codes to matrix operands.
//
//   W[n, k] = scale[n, k / group] * (q[n, k] - zero[n, k / group])
//
// Rows are taken in units of 32, K in chunks of 64, and chunks in steps of two
// where the group is a multiple of 128 (else one).  The packed buffer is one
// block per unit and step: the step's chunks, 1 KB each, then its scales.  The
// blocks of four units follow one another (128 rows of a step are one piece of
// memory: a bulk copy costs about 60 cycles whatever its size, and 4 KB pieces
// reach the full rate where 1 KB ones stay below a third), then comes the next
// step; N is padded to 128 rows.
//
// A chunk holds two 16-row halves of 512 bytes, each the operand of four
// m16n8k16 products: the 16 bytes of lane l are rows r = l / 4 and r + 8, and of
// each row the 8 codes at k = 64 c + 32 h + 8 (l mod 4) for h = 0, 1 (words:
// r h0, r h1, r+8 h0, r+8 h1).  So one 16-byte load per lane, contiguous over the
// warp, feeds four products, and 8 consecutive k of a row are one word, one
// 16-byte piece of a
// K-major bf16 tile.  A word is eight nibbles turned left by three bits; code
// e is nibble e / 2 (e even) or 4 + e / 2 (e odd), so turning the word right by
// 4 j leaves the pair (2 j, 2 j + 1) in bits 3..6 of its two halves, the top of
// a bf16 mantissa (j = 0 needs no turn).
//
// Scales: per group of the step (two where the group is 32), the 32 rows'
// entries in the order (r mod 8, r / 8), so the four rows a lane works on are
// adjacent:
//   format 0 (bf16 scales, zero = 8): 4 bf16 per lane-row, 64 bytes a group
//   DFLASH2_W4_ZERO:                  4 bf16 + 4 bf16 of (16 + zero), 128 bytes
//   DFLASH2_W4_SCALE_F32:             4 float + 4 bf16 of (16 + zero) + 8 pad, 256 bytes
// Rows past N have scale 0; the K tail of a last half chunk has codes equal
// to its zero point and, where it is a group of its own, scale 0.
//
// Codes to operands: 0x4180 | q << 3 is the bf16 value 16 + q; subtracting
// (16 + zero) leaves q - zero, an integer below 16 in magnitude, exactly.  The
// products with x then accumulate in fp32 with no rounding of the weights, and the
// group's scale multiplies the fp32 sum.  (Leaving 16 + zero in and starting the sum
// at -(16 + zero) times the sum of x saves the subtraction, but the sum then passes
// through 16 to 31 times |x| of every channel, and a channel far above the rest
// takes the others' last bits even where its own code is the zero point: not done.)
#pragma once

#include "common.cuh"

namespace dfl {

constexpr int W4_UNIT = 32;         // rows per unit
constexpr int W4_CHUNK = 64;        // K per chunk
constexpr int W4_CHUNK_BYTES = 1024;  // of one unit

// Bytes of one unit's scales for one group of K, by format.
__host__ __device__ constexpr int w4_scale_bytes(int format) {
    return (format & DFLASH2_W4_SCALE_F32) ? 256 : (format & DFLASH2_W4_ZERO) ? 128 : 64;
}

struct W4Layout {
    int64_t N, K;
    int64_t units;    // of 32 rows
    int chunks;       // of 64 k, the last one possibly half
    int kb, sg;       // chunks and groups (1, or 2 of 32) of a step
    int steps;        // chunks / kb
    int group;
    int step_bytes;
    size_t total;
};

__host__ __device__ inline bool w4_shape_ok(int64_t N, int64_t K, int group) {
    if (N < 1 || K < 32 || N > INT32_MAX || K > (1 << 20)) return false;
    if (group != 32 && (group < 64 || group % 64 != 0)) return false;
    return K % group == 0;
}

__host__ __device__ inline W4Layout w4_layout(int64_t N, int64_t K, int group, int format) {
    W4Layout L;
    L.N = N;
    L.K = K;
    L.units = (N + W4_UNIT - 1) / W4_UNIT;
    L.chunks = (int)((K + W4_CHUNK - 1) / W4_CHUNK);
    L.kb = group % 128 == 0 ? 2 : 1;
    L.sg = group == 32 ? 2 : 1;
    L.steps = L.chunks / L.kb;
    L.group = group;
    L.step_bytes = L.kb * W4_CHUNK_BYTES + L.sg * w4_scale_bytes(format);
    L.total = (size_t)((L.units + 3) / 4) * L.steps * 4 * L.step_bytes;
    return L;
}
// Byte offset of a unit's block of a step.
__host__ __device__ inline int64_t w4_block(int64_t unit, int steps, int step, int step_bytes) {
    return (((unit >> 2) * steps + step) * 4 + (unit & 3)) * step_bytes;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t w4_turn(uint32_t w, int bits) {
    return bits == 0 ? w : __funnelshift_r(w, w, bits);
}
// (w & mask) | magic in one three-input operation
__device__ __forceinline__ uint32_t w4_and_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t t;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t) : "r"(w), "r"(mask), "r"(magic));
    return t;
}
// The pair (2 j, 2 j + 1) of a word as bf16x2, minus the zero points; zz = bf16x2
// of (16 + zero) twice.
__device__ __forceinline__ uint32_t w4_pair_exact(uint32_t w, int j, uint32_t zz) {
    const uint32_t t = w4_and_or(w4_turn(w, 4 * j), 0x00780078u, 0x41804180u);
    __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                               *reinterpret_cast<const __nv_bfloat162*>(&zz));
    return *reinterpret_cast<uint32_t*>(&d);
}

// The scales (and zero points) of the four rows r, r + 8, r + 16, r + 24 of a
// unit for one group.
template <int FMT>
struct W4Scale {
    uint32_t raw[(FMT & DFLASH2_W4_SCALE_F32) ? 6 : (FMT & DFLASH2_W4_ZERO) ? 4 : 2];
    static constexpr int BYTES = w4_scale_bytes(FMT) / 8;
    // a: shared address of the entries of this lane's four rows
    __device__ __forceinline__ void load_shared(uint32_t a) {
        if constexpr ((FMT & DFLASH2_W4_SCALE_F32) != 0) {
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[0]), "=r"(raw[1]), "=r"(raw[2]), "=r"(raw[3])
                         : "r"(a));
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(raw[4]), "=r"(raw[5]) : "r"(a + 16));
        } else if constexpr ((FMT & DFLASH2_W4_ZERO) != 0) {
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[0]), "=r"(raw[1]), "=r"(raw[2]), "=r"(raw[3])
                         : "r"(a));
        } else {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(raw[0]), "=r"(raw[1]) : "r"(a));
        }
    }
    // i: 0 .. 3 for rows r, r + 8, r + 16, r + 24
    __device__ __forceinline__ float scale(int i) const {
        if constexpr ((FMT & DFLASH2_W4_SCALE_F32) != 0) return __uint_as_float(raw[i]);
        return __uint_as_float((i & 1) ? (raw[i >> 1] & 0xFFFF0000u) : (raw[i >> 1] << 16));
    }
    __device__ __forceinline__ uint32_t zero2(int i) const {
        if constexpr (FMT == 0) return 0x41C041C0u;  // 16 + 8
        const uint32_t w = raw[((FMT & DFLASH2_W4_SCALE_F32) ? 4 : 2) + (i >> 1)];
        return (i & 1) ? __byte_perm(w, 0, 0x3232) : __byte_perm(w, 0, 0x1010);
    }
};

}  // namespace dfl

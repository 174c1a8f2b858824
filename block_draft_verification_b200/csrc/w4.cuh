// w4.cuh -- 4-bit weights with group scales: the packed layout every kernel
// that reads them shares, and the step from codes to matrix operands.
//
//   W[n, k] = scale[n, k / group] * (q[n, k] - zero[n, k / group])
//
// The packed buffer is [weights][scales].
//
// Weights: rows in units of 32, K in chunks of 64; unit u, chunk c is the
// 1 KB block at (u * KC + c) * 1024 (KC chunks per row).  A block holds two
// 16-row halves of 512 bytes, each the operand of four m16n8k16 products: the
// 16 bytes of lane l are rows r = l / 4 and r + 8, and of each row the 8 codes
// at k = 64 c + 32 h + 8 (l mod 4) for h = 0, 1 (words: r h0, r h1, r+8 h0,
// r+8 h1).  So one 16-byte load per lane, contiguous over the warp, feeds four
// products, and 8 consecutive k of a row are one word, one 16-byte piece of a
// K-major bf16 tile.  Within a word, code e sits at nibble e / 2 (e even) or
// 4 + e / 2 (e odd): (word >> 4 j) & 0x000F000F is the pair (2 j, 2 j + 1).
//
// Scales: per unit and group of K, the 32 rows' entries in the order
// (r mod 8, r / 8), so the four rows a lane works on are adjacent:
//   format 0 (bf16 scales, zero = 8): 4 bf16 per lane-row, 64 bytes a group
//   DFLASH2_W4_ZERO:                  4 bf16 + 4 bf16 of (128 + zero), 128 bytes
//   DFLASH2_W4_SCALE_F32:             4 float + 4 bf16 of (128 + zero) + 8 pad, 256 bytes
// Rows past N have scale 0; the K tail of a last half chunk has codes equal
// to its zero point and, where it is a group of its own, scale 0.
//
// Codes to operands: 0x4300 | q is the bf16 value 128 + q; subtracting
// (128 + zero) leaves q - zero, an integer of at most 8 bits, exactly.  The
// products with x then accumulate in fp32 with no rounding of the weights, and
// the group's scale multiplies the fp32 sum.
#pragma once

#include "common.cuh"

namespace dfl {

constexpr int W4_UNIT = 32;         // rows per unit
constexpr int W4_CHUNK = 64;        // K per chunk
constexpr int W4_BLOCK = 1024;      // bytes per unit and chunk

// Bytes of one unit's scales for one group of K, by format.
__host__ __device__ constexpr int w4_scale_bytes(int format) {
    return (format & DFLASH2_W4_SCALE_F32) ? 256 : (format & DFLASH2_W4_ZERO) ? 128 : 64;
}

struct W4Layout {
    int64_t N, K;
    int64_t units;    // of 32 rows
    int chunks;       // of 64 k, the last one possibly half
    int groups;       // per row as packed: K / group, or 2 per chunk for group 32
    int group;
    int sbytes;       // scale bytes per unit and group
    size_t scale_off; // bytes
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
    L.group = group;
    L.groups = group == 32 ? 2 * L.chunks : (int)(K / group);
    L.sbytes = w4_scale_bytes(format);
    L.scale_off = (size_t)L.units * L.chunks * W4_BLOCK;
    L.total = L.scale_off + (size_t)L.units * L.groups * L.sbytes;
    return L;
}

// The pair (2 j, 2 j + 1) of a word, minus the zero points, as bf16x2.
// zz = bf16x2 of (128 + zero) twice.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int j, uint32_t zz) {
    uint32_t t;
    // (w >> 4 j & 0x000F000F) | 0x43004300 in one three-input operation
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(t)
        : "r"(w >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
    __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&t),
                               *reinterpret_cast<const __nv_bfloat162*>(&zz));
    return *reinterpret_cast<uint32_t*>(&d);
}

// The scales (and zero points) of the four rows r, r + 8, r + 16, r + 24 of a
// unit for one group.
template <int FMT>
struct W4Scale {
    uint32_t raw[(FMT & DFLASH2_W4_SCALE_F32) ? 6 : (FMT & DFLASH2_W4_ZERO) ? 4 : 2];
    // p: the group's entries of this unit; g = r mod 8
    __device__ __forceinline__ void load(const uint8_t* p, int g) {
        if constexpr ((FMT & DFLASH2_W4_SCALE_F32) != 0) {
            const uint4 a = __ldg((const uint4*)(p + 32 * g));
            const uint2 b = __ldg((const uint2*)(p + 32 * g + 16));
            raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w, raw[4] = b.x, raw[5] = b.y;
        } else if constexpr ((FMT & DFLASH2_W4_ZERO) != 0) {
            const uint4 a = __ldg((const uint4*)(p + 16 * g));
            raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w;
        } else {
            const uint2 a = __ldg((const uint2*)(p + 8 * g));
            raw[0] = a.x, raw[1] = a.y;
        }
    }
    // i: 0 .. 3 for rows r, r + 8, r + 16, r + 24
    __device__ __forceinline__ float scale(int i) const {
        if constexpr ((FMT & DFLASH2_W4_SCALE_F32) != 0) return __uint_as_float(raw[i]);
        return __uint_as_float((i & 1) ? (raw[i >> 1] & 0xFFFF0000u) : (raw[i >> 1] << 16));
    }
    __device__ __forceinline__ uint32_t zero2(int i) const {
        if constexpr (FMT == 0) return 0x43084308u;  // 128 + 8
        const uint32_t w = raw[((FMT & DFLASH2_W4_SCALE_F32) ? 4 : 2) + (i >> 1)];
        return (i & 1) ? __byte_perm(w, 0, 0x3232) : __byte_perm(w, 0, 0x1010);
    }
};

}  // namespace dfl

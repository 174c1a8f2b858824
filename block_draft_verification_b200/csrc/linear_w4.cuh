// linear_w4.cuh -- what the two kernels for products with 4-bit weights share on
// the host: one call's arguments, checked, and the device they run on.
#pragma once

#include "w4.cuh"

struct W4Call {
    dfl::W4Layout L;
    int format;           // without DFLASH2_W4_TAPS
    const void* packed;
    const void* x;
    int64_t x_stride, tokens;
    bool x_f32, x_vec;    // x_vec: rows of x start on 16 bytes
    void* y;
    bool y_bf16;
    const void* x_prev;   // conv; NULL: linear
    int T;                // conv: tokens per sequence
};

// The device at hand and how many clusters of each size it holds at once, one
// CTA per SM (of 148 SMs: 148, 74, 33 and 15 of size 1, 2, 4 and 8; larger
// clusters fit a GPU's processing clusters less well).
struct W4Dev {
    int id;
    int clusters[9];
};

// The tensor-core kernel takes more than this many tokens, and fewer (above 8) where
// the other kernel would have to fill its shared memory with x more than twice over.
// Other kernel and this one: 10,240 x 5,120, 14.0 and 21.4 us at 8 tokens, 21.7 and
// 21.6 at 16, 47.8 and 22.0 at 17; 20,480 x 5,120 (x in two parts), 34.4 and 37.5 at
// 9, 39.7 and 37.8 at 16; 5,120 x 20,480 (x in four parts), 26.1 and 36.1 at 8, 84.0
// and 36.2 at 9.  (At 16 tokens this one is also ahead at 5,120 x 5,120, 14.7 against
// 16.9, and at 151,936 x 5,120, 161 against 202.)
constexpr int64_t W4_FEW_TOKENS = 16;

// Tiles of the tensor-core kernel: tokens per tile and tiles of tokens, cluster size,
// clusters, tiles.
struct W4TcPlan {
    int ntok, tt, S, C;
    int64_t tiles;
};

bool dfl_linear_w4_tc_ok(const W4Call& c);
W4TcPlan dfl_linear_w4_tc_plan(const W4Call& c, const W4Dev& d);
int dfl_linear_w4_tc(const W4Call& c, const W4Dev& d, cudaStream_t s);

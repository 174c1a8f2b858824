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
// Other kernel and this one: 10,240 x 5,120, 13.6 and 23.2 us at 8 tokens, 20.9 and
// 23.4 at 16, 51.5 and 23.7 at 17; 20,480 x 5,120 (x in two parts), 27.7 and 43.4 at
// 9; 5,120 x 20,480 (x in four parts), 22.6 and 37.0 at 8, 83.5 and 37.1 at 9.
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

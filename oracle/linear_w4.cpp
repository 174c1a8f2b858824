/*
 * linear_w4.cpp -- the product with 4-bit weights and group scales, in fp64.
 * TEST INFRASTRUCTURE ONLY (see oracle.h).
 *
 *   W[n, k] = scale[n, k / group] * (q[n, k] - zero[n, k / group])
 *   y[t, n] = sum_k W[n, k] x[t, k],   abs[t, n] = sum_k |W[n, k] x[t, k]|
 * q [N, K/2] bytes, the even k in the low half; zero NULL stands for 8; abs
 * (optional) is the magnitude that a bound on the summation's error refers to.
 */
#include <math.h>

#include "oracle_util.h"

extern "C" int orc_linear_w4(const void* x, int dtype, int64_t tokens, const uint8_t* q,
                             const void* scale, int scale_dtype, const uint8_t* zero, int64_t N,
                             int64_t K, int64_t group, double* y, double* abs_sum) {
    if (!x || !q || !scale || !y || !orc_dtype_ok(dtype) || !orc_dtype_ok(scale_dtype) ||
        tokens < 0 || N < 1 || K < 2 || K % 2 || group < 1 || K % group)
        return -1;
    for (int64_t n = 0; n < N; ++n) {
        for (int64_t t = 0; t < tokens; ++t) {
            double sum = 0.0, mag = 0.0;
            for (int64_t k = 0; k < K; ++k) {
                const int64_t g = n * (K / group) + k / group;
                const uint8_t byte = q[(n * K + k) / 2];
                const int code = (k & 1) ? byte >> 4 : byte & 15;
                const double w = orc_load(scale, scale_dtype, g) * (code - (zero ? zero[g] : 8));
                const double p = w * orc_load(x, dtype, t * K + k);
                sum += p;
                mag += fabs(p);
            }
            y[t * N + n] = sum;
            if (abs_sum) abs_sum[t * N + n] = mag;
        }
    }
    return 0;
}

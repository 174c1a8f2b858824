/*
 * norm_residual.cpp -- the norms around a block with its gate and residual
 * scale, in fp64.
 * TEST INFRASTRUCTURE ONLY (see oracle.h).
 *
 *   r'_i = r_i + alpha * act(g_i) * rms(y; w_post)_i,   h = rms(r'; w_pre),
 *   rms(v; w)_i = v_i / sqrt(mean_j v_j^2 + eps) * (w_i + w_offset)
 * gate row of row r: r / gate_rep; NULL gate, w_post, w_pre (with h) as in the
 * formula without them.
 */
#include <math.h>

#include <vector>

#include "oracle_util.h"

static double inv_rms(const std::vector<double>& v, double eps) {
    double s = 0.0;
    for (double x : v) s += x * x;
    return 1.0 / sqrt(s / (double)v.size() + eps);
}

extern "C" int orc_norm_residual(const void* res, int res_dtype, const void* y, int dtype,
                                 const void* gate, int64_t gate_rep, int sigmoid, const void* w_post,
                                 const void* w_pre, double w_offset, double alpha, double eps,
                                 int64_t rows, int64_t H, double* res_out, double* h) {
    if (!res || !y || !res_out || !orc_dtype_ok(dtype) || !orc_dtype_ok(res_dtype) || rows < 0 ||
        H < 1 || gate_rep < 1)
        return -1;
    std::vector<double> v(H);
    for (int64_t r = 0; r < rows; ++r) {
        for (int64_t i = 0; i < H; ++i) v[i] = orc_load(y, dtype, r * H + i);
        const double s = w_post ? inv_rms(v, eps) : 1.0;
        for (int64_t i = 0; i < H; ++i) {
            if (w_post) v[i] *= s * (orc_load(w_post, dtype, i) + w_offset);
            if (gate) {
                const double g = orc_load(gate, dtype, r / gate_rep * H + i);
                v[i] *= sigmoid ? 1.0 / (1.0 + exp(-g)) : g;
            }
            v[i] = orc_load(res, res_dtype, r * H + i) + alpha * v[i];
            res_out[r * H + i] = v[i];
        }
        if (w_pre) {
            const double s2 = inv_rms(v, eps);
            for (int64_t i = 0; i < H; ++i)
                h[r * H + i] = v[i] * s2 * (orc_load(w_pre, dtype, i) + w_offset);
        }
    }
    return 0;
}

// la_gated_common.cuh — what the gated linear-attention kernels share.
//
// Per key/value head, with a_t = exp(log_gate_t) and G_t = sum_{s<=t} log a_s:
//
//     S_t = a_t S_{t-1} + k_t v_t^T,        o_t = scale * S_t^T q_t
//
// cut into chunks.  With S the state entering a chunk (G counted from there),
//
//     o_i = scale ( sum_{j<=i} e^{G_i-G_j} (q_i.k_j) v_j + e^{G_i} S^T q_i )
//     S'  = e^{G_C} S + sum_j e^{G_C-G_j} k_j v_j^T
//
// and backwards, with R the gradient of the state leaving the chunk,
//
//     dq_i = scale ( sum_{j<=i} e^{G_i-G_j} (dO_i.v_j) k_j + e^{G_i} S dO_i )
//     dk_j = scale sum_{i>=j} e^{G_i-G_j} (dO_i.v_j) q_i  + e^{G_C-G_j} R v_j
//     dv_j = scale sum_{i>=j} e^{G_i-G_j} (q_i.k_j) dO_i  + e^{G_C-G_j} R^T k_j
//     R'   = e^{G_C} R + scale sum_i e^{G_i} q_i dO_i^T
//
// so o, dq, dk and dv are one product, "rows against columns weighted by the
// gates between them, times values, plus rows through a state", with the
// three operands permuted (and time reversed for dk and dv).
//
// The gate at t scales everything that passes from the tokens j < t to the
// tokens i >= t, so its gradient is a sum over such pairs,
//
//     dlog_t = sum_{i>=t} sum_{j<t} M_ij + sum_{i>=t} q_i.dq^S_i
//              + sum_{j<t} k_j.dk^R_j + e^{G_C} <S, R>
//
// (M_ij = scale e^{G_i-G_j} (q_i.k_j)(dO_i.v_j) inside the chunk; dq^S, dk^R
// the parts of dq and dk that come through S and R).  The shorter form
// sum_{i>=t} (q_i.dq_i - k_i.dk_i) over the whole sequence cancels: its
// rounding errors grow with the tokens behind t while the value does not.
#pragma once

#include "la_common.cuh"

namespace la {

// log2 of a gate in 64 bits (sums of them keep the differences that the
// weights are made of).  A gate of zero (log -inf) is taken as 2^-160: its
// weight is zero in float32, and sums with it stay finite, so the weights on
// either side of it are unaffected.  NaN stays NaN.
__device__ __forceinline__ double gate_log2(float lg) {
    const double x = double(lg) * 1.4426950408889634;
    return x < -160.0 ? -160.0 : x;
}

// A gate below 2^-126, the least that float32 holds in full (NaN is not): its
// gradient is written as 0.  What the sums over pairs and states would leave
// there is their float32 rounding.
__device__ __forceinline__ bool gate_is_zero(double log2_gate) { return log2_gate < -126.0; }

__device__ __forceinline__ double warp_scan_sum(double x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

}  // namespace la

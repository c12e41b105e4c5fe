// la_gated_decode.cuh — one step of gated linear attention, in place, for
// every key/value head and its G query heads:
//
//     S = e^{log_gate} S + k v^T,      o_g = scale * S^T q_g
//
// One streaming pass over the float32 state (8 bytes an element, HBM bound).
// The value columns of S are independent of each other (column e of S meets
// only v_e and gives only o_e), so a block takes DC of a head's columns.  Thread
// (rg, cg) holds one float4 of columns of the rows rg, rg + RG, ...: all of its
// loads are issued before any arithmetic, and the updated state answers the
// group's queries, QB at a time, from registers.
//
// Measured (B200, bf16): B256 H32 D128, 1.08 GB, 161 us (6.7 TB/s, what a copy
// reaches); B1 H16 Hkv4 D64, 9 us, of which most is the launch.
#pragma once

#include "la_gated_common.cuh"

namespace la {

// Columns a block takes: all at D <= 64, 32 of 128.  Whole and cut in four, us:
// D = 128 with 32 heads 8.7, 8.2; 1000: 27.1, 25.3; 2000: 45.8, 44.6; 8192: 162.5,
// 160.9.  D = 64: 7.7, 7.5; 10.9, 12.7; 16.7, 18.8; 45.8, 53.9 (16 columns leave a
// thread two rows, so the block's fixed work is most of it).
template <int D>
constexpr int gated_step_columns = D == 128 ? 32 : D;

template <typename T, int D, int DC>
__global__ void __launch_bounds__(2 * D)
gated_step_kernel(float* __restrict__ S, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, const T* __restrict__ lg, T* __restrict__ o, int G,
                  float scale) {
    constexpr int NT = 2 * D;
    constexpr int CG = DC / 4;      // float4 column groups of the block
    constexpr int RG = NT / CG;     // row groups
    constexpr int RPT = D / RG;     // rows a thread
    constexpr int QB = 4;
    static_assert(RPT >= 1 && RPT * RG == D, "thread layout");
    __shared__ float k_s[D], q_s[QB][D];
    __shared__ float4 part[QB][RG][CG];
    constexpr int NB = D / DC;
    const size_t hk = blockIdx.x / NB;
    const int e0 = int(blockIdx.x % NB) * DC;  // first column of the block
    const int tid = threadIdx.x;
    const int cg = tid % CG, rg = tid / CG;
    float4* Sh = reinterpret_cast<float4*>(S + hk * D * D + e0);
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r] = __ldcs(Sh + (rg + RG * r) * (D / 4) + cg);
    const float a = exp2f(float(gate_log2(to_f32(lg[hk]))));
    if (tid < D) k_s[tid] = to_f32(k[hk * D + tid]);
    float4 vv;
    {
        const T* vp = v + hk * D + e0 + 4 * cg;
        vv = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    }
    // QB queries, loaded one batch ahead: thread t holds element t % D of the
    // queries t / D, t / D + 2, ...
    float xq[QB / 2];
    auto load_q = [&](int g0) {
#pragma unroll
        for (int i = 0; i < QB / 2; ++i) {
            const int g = g0 + tid / D + 2 * i;
            xq[i] = g < G ? to_f32(q[(hk * G + g) * D + tid % D]) : 0.f;
        }
    };
    load_q(0);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int f = rg + RG * r;
        const float kf = k_s[f];
        float4 x = s[r];
        x.x = fmaf(kf, vv.x, a * x.x);
        x.y = fmaf(kf, vv.y, a * x.y);
        x.z = fmaf(kf, vv.z, a * x.z);
        x.w = fmaf(kf, vv.w, a * x.w);
        __stcs(Sh + f * (D / 4) + cg, x);
        s[r] = x;
    }
    for (int g0 = 0; g0 < G; g0 += QB) {
        const int nq = min(QB, G - g0);
        if (g0) __syncthreads();  // q_s and part of the batch before are consumed
#pragma unroll
        for (int i = 0; i < QB / 2; ++i) q_s[tid / D + 2 * i][tid % D] = xq[i];
        if (g0 + QB < G) load_q(g0 + QB);
        __syncthreads();
        for (int i = 0; i < nq; ++i) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float qf = q_s[i][rg + RG * r];
                acc.x = fmaf(qf, s[r].x, acc.x);
                acc.y = fmaf(qf, s[r].y, acc.y);
                acc.z = fmaf(qf, s[r].z, acc.z);
                acc.w = fmaf(qf, s[r].w, acc.w);
            }
            // rows of one warp that share a column group, summed in registers
#pragma unroll
            for (int off = CG; off < 32; off <<= 1) {
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
                acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
                acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
            }
            constexpr int RW = CG < 32 ? 32 / CG : 1;  // row groups of one warp
            if (rg % RW == 0) part[i][rg / RW][cg] = acc;
        }
        __syncthreads();
        constexpr int RP = CG < 32 ? RG * CG / 32 : RG;  // partial sums a column
        for (int t = tid; t < nq * DC; t += NT) {
            const int i = t / DC, e = t % DC;
            const float* pf = reinterpret_cast<const float*>(&part[i][0][0]);
            float x = 0.f;
#pragma unroll
            for (int u = 0; u < RP; ++u) x += pf[u * DC + e];
            o[(hk * G + g0 + i) * D + e0 + e] = from_f32<T>(scale * x);
        }
    }
}

}  // namespace la

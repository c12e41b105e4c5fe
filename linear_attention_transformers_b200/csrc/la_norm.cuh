// la_norm.cuh — group norm of an attention output's head rows with the gate's
// activation, from the library's layout [B, H, N, D] to channels last
// [B, N, H*D], and its gradients.  With c = h*D + d, x_hat the row x[b,h,n,:]
// less its mean over sqrt(variance + eps), and m = w_c x_hat + bias_c:
//
//     y[b,n,c] = m act(gate[b,n,c])        (act(m) without a gate)
//
// The norm is what an unnormalised recurrence has in place of the
// denominator.  Everything is one pass: a row is D elements, held by
// D * sizeof(T) / 16 neighbouring lanes (16 bytes each), its statistics are
// shuffles in float32, and the transposition to channels last costs nothing
// because rows stay whole.  HBM bound: 6 bytes an element forward (bf16: x,
// gate, y), 10 backward (x, gate, dy, dx, dgate).
//
// A thread keeps its channels for all of its tokens, so the weights are read
// once and the backward's channel sums stay in registers; each block writes
// one row of partial sums, added in order by norm_sum_kernel (no atomics, so
// runs are bitwise repeatable).
//
// Measured (B200, bf16, gate, silu): forward B4 H16 N4096 D128, 201 MB, 38 us
// (5.3 TB/s); backward B8 H16 N8192 D64, 671 MB, 112 us (6.0 TB/s).  Loads held
// in registers instead of the ring took 46 and 145 us: the rows' reductions and
// the activation leave too few registers to keep enough bytes in flight.
#pragma once

#include "la_async_copy.cuh"
#include "la_common.cuh"

namespace la {

enum : int { ACT_IDENTITY = 0, ACT_SILU = 1 };

struct NormParams {
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float* part;       // [2][blocks][C]: sums for weight and bias
    int64_t tokens;    // B * N
    int64_t N;
    int H;
    int groups;        // 16-byte groups of a token, H * D * sizeof(T) / 16
    int span;          // groups a block covers (groups if they fit, else 256)
    int slots;         // tokens a block takes at once
    float eps;
};

// bf16 tensors take the hardware's base-2 exponential and reciprocal: with the
// rounding of the exponent 2^-19 of the value for |x| up to 16, far below the half
// step of the bf16 outputs (2^-8).  The float32 sums for weight and bias take it
// too: over many tokens its errors add up as the terms do.
// An exponential that overflows gives 1 / inf = 0.
template <bool EXACT>
__device__ __forceinline__ float norm_sigmoid(float x) {
    if (EXACT) return 1.f / (1.f + expf(-x));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

template <typename T> struct NormVec {
    static constexpr int V = 16 / sizeof(T);
    float f[V];
    __device__ __forceinline__ void set(const uint4& u) {
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = to_f32(e[j]);
    }
    __device__ __forceinline__ uint4 get() const {
        uint4 u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = from_f32<T>(f[j]);
        return u;
    }
};

// sum over the LPR lanes that hold a row
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A token's place in x: offsets (in 16-byte groups) of one head's row, advanced
// by a fixed number of tokens at a time without a division.
struct NormPlace {
    int64_t off, nn, N, step_n, step_off, wrap;
    __device__ __forceinline__ NormPlace(int64_t tok, int64_t step, const NormParams& p, int h,
                                         int lpr, int lane_in_row)
        : N(p.N) {
        const int64_t bb = tok / N;
        nn = tok % N;
        off = ((bb * p.H + h) * N + nn) * lpr + lane_in_row;
        const int64_t step_b = step / N;
        step_n = step % N;
        step_off = (step_b * p.H * N + step_n) * lpr;
        wrap = (int64_t(p.H) * N - N) * lpr;  // nn - N in the next sequence
    }
    __device__ __forceinline__ void next() {
        off += step_off;
        nn += step_n;
        if (nn >= N) {
            nn -= N;
            off += wrap;
        }
    }
};

// One kernel for both directions (BWD).  Thread t of a block: slot t / span,
// group g = span * blockIdx.y + t % span; it takes the tokens blockIdx.x *
// slots + slot, then every gridDim.x * slots on.  Its 16 bytes of x, gate and
// dy travel through a ring of kNormStages in shared memory that only it reads
// (so no barrier), which keeps the loads of the next tokens in flight without
// registers to hold them.
constexpr int kNormStages = 4;

// Blocks an SM holds.  Fewer leave too little in flight, more too few
// registers: at B8 H16 N8192 D64 bf16 the backward takes 116 us with 2 and 142
// with 3 (spills), at B2 H12 N4096 D64 float32 29.8 and 25.6; the forward at B4
// H16 N4096 D128 bf16 takes 42 us with 4, 44 with 5 and 49 with 6.
template <typename T, bool BWD>
constexpr int kNormBlocks = BWD ? (sizeof(T) == 4 ? 3 : 2) : 4;

template <typename T, int D, bool BWD, bool GATE, int ACT>
__global__ void __launch_bounds__(256, (kNormBlocks<T, BWD>))
group_norm_kernel(const NormParams p) {
    constexpr int V = NormVec<T>::V, LPR = D / V;
    constexpr bool kExact = sizeof(T) == sizeof(float);
    constexpr int kArrays = 1 + (GATE ? 1 : 0) + (BWD ? 1 : 0);
    extern __shared__ uint4 ring[];  // [kNormStages][kArrays][blockDim.x]
    const int slot = threadIdx.x / p.span, t = threadIdx.x % p.span;
    const int g = p.span * int(blockIdx.y) + t;
    const bool live = slot < p.slots && g < p.groups;
    const int h = live ? g / LPR : 0, d0 = (g % LPR) * V;
    const int C = p.H * D, c0 = h * D + d0;
    float w[V], b[V], dw[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        w[j] = live ? p.weight[c0 + j] : 0.f;
        b[j] = live && p.bias ? p.bias[c0 + j] : 0.f;
        dw[j] = db[j] = 0.f;
    }
    const uint4* x4 = reinterpret_cast<const uint4*>(p.x);
    const uint4* g4 = reinterpret_cast<const uint4*>(p.gate);
    const uint4* dy4 = reinterpret_cast<const uint4*>(p.dy);
    const int64_t step = int64_t(gridDim.x) * p.slots;
    const int64_t start = int64_t(blockIdx.x) * p.slots;
    NormPlace ahead(start + slot, step, p, h, LPR, g % LPR);
    NormPlace here = ahead;
    int64_t atok = start + slot;  // the token fetched next
    auto fetch = [&](int stage) {
        const bool ok = live && atok < p.tokens;
        uint4* dst = ring + stage * kArrays * blockDim.x + threadIdx.x;
        const int64_t yo = ok ? atok * p.groups + g : 0;
        copy16_async(dst, x4 + (ok ? ahead.off : 0), ok);
        if (GATE) copy16_async(dst + blockDim.x, g4 + yo, ok);
        if (BWD) copy16_async(dst + (kArrays - 1) * blockDim.x, dy4 + yo, ok);
        ahead.next();
        atok += step;
    };
#pragma unroll
    for (int i = 0; i < kNormStages - 1; ++i) {
        fetch(i);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    int64_t tok = start + slot;
    // every thread of the block takes the same number of rounds (the shuffles
    // below need whole warps)
    for (int64_t n0 = start; n0 < p.tokens; n0 += step, tok += step) {
        fetch(stage == 0 ? kNormStages - 1 : stage - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kNormStages - 1) : "memory");
        const uint4* src = ring + stage * kArrays * blockDim.x + threadIdx.x;
        stage = stage == kNormStages - 1 ? 0 : stage + 1;
        const bool ok = live && tok < p.tokens;
        const int64_t xo = here.off, yo = tok * p.groups + g;
        if (BWD) here.next();
        {
            NormVec<T> x, ga, dy;
            x.set(src[0]);
            if (GATE) ga.set(src[blockDim.x]);
            if (BWD) dy.set(src[(kArrays - 1) * blockDim.x]);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) s += x.f[j];
            const float mean = row_sum<LPR>(s) * (1.f / D);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x.f[j] -= mean;
                ss = fmaf(x.f[j], x.f[j], ss);
            }
            const float rstd = rsqrtf(fmaf(row_sum<LPR>(ss), 1.f / D, p.eps));
            if (!BWD) {
                NormVec<T> y;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float m = fmaf(x.f[j] * rstd, w[j], b[j]);
                    const float at = GATE ? ga.f[j] : m;
                    const float act = ACT == ACT_SILU ? at * norm_sigmoid<kExact>(at) : at;
                    y.f[j] = GATE ? m * act : act;
                }
                if (ok) __stcs(reinterpret_cast<uint4*>(p.y) + yo, y.get());
            } else {
                NormVec<T> dx, dg;
                float s1 = 0.f, s2 = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = x.f[j] * rstd;
                    x.f[j] = xh;
                    const float m = fmaf(xh, w[j], b[j]);
                    const float at = GATE ? ga.f[j] : m;
                    float act = at, dact = 1.f;
                    if (ACT == ACT_SILU) {
                        const float e = norm_sigmoid<kExact>(at);
                        act = at * e;
                        dact = fmaf(act, 1.f - e, e);
                    }
                    float dm;
                    if (GATE) {
                        dg.f[j] = dy.f[j] * m * dact;
                        dm = dy.f[j] * act;
                    } else {
                        dm = dy.f[j] * dact;
                    }
                    dw[j] = fmaf(dm, xh, dw[j]);
                    db[j] += dm;
                    dm *= w[j];
                    dx.f[j] = dm;
                    s1 += dm;
                    s2 = fmaf(dm, xh, s2);
                }
                s1 = row_sum<LPR>(s1) * (1.f / D);
                s2 = row_sum<LPR>(s2) * (1.f / D);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    dx.f[j] = rstd * (dx.f[j] - s1 - x.f[j] * s2);
                if (ok) {
                    __stcs(reinterpret_cast<uint4*>(p.dx) + xo, dx.get());
                    if (GATE) __stcs(reinterpret_cast<uint4*>(p.dgate) + yo, dg.get());
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (BWD) {
        // the block's slots, added in order through shared memory
        __shared__ float red[256 * V];
        const int64_t row = blockIdx.x;
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j)
                red[int(threadIdx.x) * V + j] = k ? db[j] : dw[j];
            __syncthreads();
            if (slot == 0 && live) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float a = 0.f;
                    for (int i = 0; i < p.slots; ++i) a += red[(i * p.span + t) * V + j];
                    p.part[(int64_t(k) * gridDim.x + row) * C + c0 + j] = a;
                }
            }
        }
    }
}

// out[c] = sum over rows of part[rows][C], in a fixed order: 32 channels a
// block, 16 threads a channel, then the 16 sums.  blockIdx.y picks weight (0)
// or bias (1); a null output is skipped.
__global__ void __launch_bounds__(512)
norm_sum_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                float* __restrict__ dbias, int rows, int C) {
    float* out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    part += int64_t(blockIdx.y) * rows * C;
    __shared__ float red[16][33];
    const int c = int(blockIdx.x) * 32 + int(threadIdx.x % 32), i0 = threadIdx.x / 32;
    float a = 0.f;
    if (c < C)
        for (int i = i0; i < rows; i += 16) a += part[int64_t(i) * C + c];
    red[i0][threadIdx.x % 32] = a;
    __syncthreads();
    if (i0 == 0 && c < C) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += red[i][threadIdx.x];
        out[c] = a;
    }
}

}  // namespace la

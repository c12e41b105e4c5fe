// la_gated_generic.cuh — gated linear attention on the plain cores, for every
// type and head size (float32, bf16 with D = 16 or 32, and calls of a few tokens
// take it; see la_gated_common.cuh for the formulas).  Chunks of 64 tokens, every chunk of
// every head a block of its own; the states at the chunks' borders are float32
// records in the workspace:
//
//   gated_part_kernel   the chunks' own parts of the state, both directions
//   gated_carry_kernel  the records' recurrence over the chunks, in place
//   gated_o_kernel      o of one chunk
//   gated_grad_kernel   dlog_gate, dk, dv and dq: each of a chunk a block's work
//
// What does not depend on each other shares a launch (the backward's four
// gradients, the two directions of the states), since the sizes that come here
// leave most SMs idle: B2 H6 Hkv2 N333 D64 float32, backward, took 132 us in
// eight launches and takes 66 in three.  B3 H6 N1000 D32 float32, forward: 26 us.
//
// All products are register-tiled float32 (4 rows x D/16 columns a thread)
// from float32 tiles in shared memory, so nothing is rounded below float32;
// the kernels are bound by the cores' multiply-adds.
#pragma once

#include "la_gated_common.cuh"

namespace la {

constexpr int kGatedC = 64;          // tokens a chunk
constexpr int kGatedThreads = 256;   // 16 x 16

struct GatedTile {
    static constexpr int C = kGatedC;
    // padded row lengths, in floats, that keep float4 accesses aligned
    static constexpr int ld(int cols) { return cols + 4; }
};

// rows [n0, n0 + 64) of x [N][D] to float32; zeros from row N on
template <typename T, int D>
__device__ __forceinline__ void gated_load_tile(float* dst, const T* __restrict__ x, int64_t n0,
                                                int64_t N) {
    constexpr int V = 16 / sizeof(T), G = D / V, LD = GatedTile::ld(D);
    for (int i = threadIdx.x; i < kGatedC * G; i += kGatedThreads) {
        const int r = i / G, g = i % G;
        float f[V];
        if (n0 + r < N) {
            uint4 raw = *reinterpret_cast<const uint4*>(x + (n0 + r) * D + g * V);
            const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = to_f32(e[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4*>(dst + r * LD + g * V + j) =
                make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    }
}

// Tokens of the chunk from n0 on, up to a multiple of 4 (a thread's rows): what
// the products go over.  A call of a few tokens takes a fraction of a chunk's time.
__device__ __forceinline__ int gated_rows(int64_t n0, int64_t N) {
    return N - n0 >= kGatedC ? kGatedC : (int(N - n0) + 3) & ~3;
}

// Inclusive sums of log2 gates of one chunk (0 past N); every thread may read
// G[0..63] after the next __syncthreads.
template <typename T>
__device__ __forceinline__ void gated_load_gates(double* G, const T* __restrict__ lg, int64_t n0,
                                                 int64_t N) {
    if (threadIdx.x < 32) {
        const int l = threadIdx.x;
        const double a = n0 + 2 * l < N ? gate_log2(to_f32(lg[n0 + 2 * l])) : 0.0;
        const double b = n0 + 2 * l + 1 < N ? gate_log2(to_f32(lg[n0 + 2 * l + 1])) : 0.0;
        const double s = warp_scan_sum(a + b, l);
        G[2 * l] = s - b;
        G[2 * l + 1] = s;
    }
}

// acc[r][c] += sum_k X[row r][k] Y[col c][k]: rows 4*ty.., columns tx + 16 c
template <int K, int NC>
__device__ __forceinline__ void gated_mm_nt(float (&acc)[4][NC], const float* X, int ldx,
                                            const float* Y, int ldy, int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float4 x[4], y[NC];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = *reinterpret_cast<const float4*>(X + (4 * ty + r) * ldx + k);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            y[c] = *reinterpret_cast<const float4*>(Y + (tx + 16 * c) * ldy + k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                acc[r][c] = fmaf(x[r].x, y[c].x, acc[r][c]);
                acc[r][c] = fmaf(x[r].y, y[c].y, acc[r][c]);
                acc[r][c] = fmaf(x[r].z, y[c].z, acc[r][c]);
                acc[r][c] = fmaf(x[r].w, y[c].w, acc[r][c]);
            }
    }
}

// acc[r][c] += sum_{k<K} X[row r][k] Y[k][col c]: columns tx + 16 c
template <int NC>
__device__ __forceinline__ void gated_mm_nn(float (&acc)[4][NC], const float* X, int ldx,
                                            const float* Y, int ldy, int K, int ty, int tx) {
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = *reinterpret_cast<const float4*>(X + (4 * ty + r) * ldx + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float y[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) y[c] = Y[(k + kk) * ldy + tx + 16 * c];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float xv = kk == 0 ? x[r].x : kk == 1 ? x[r].y : kk == 2 ? x[r].z : x[r].w;
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[r][c] = fmaf(xv, y[c], acc[r][c]);
            }
        }
    }
}

// ------------------------------------------------------------ a chunk's part
// rec[head][chunk] = sum over the chunk (and the G query heads of a group for
// REV) of w_t A_t B_t^T: forward w_t = e^{G_C - G_t}, REV w_t = mul e^{G_t}.
// gtot[head][chunk] = e^{G_C}.
struct GatedPartJob {
    const void *A, *B;
    float *rec, *gtot;
    int64_t blocks;             // heads * run; 0: nothing to do
    int run, chunk0, group;     // chunks that are run, from chunk0 on
    float mul;
};

template <typename T, int D, bool REV>
__device__ __forceinline__ void gated_part_block(const GatedPartJob& job, const T* __restrict__ lg,
                                                 int64_t N, int nchunk, int64_t block) {
    constexpr int LD = GatedTile::ld(D);
    extern __shared__ __align__(16) float sm[];
    float* ta = sm;
    float* tb = sm + kGatedC * LD;
    __shared__ double G[kGatedC];
    const T* A = static_cast<const T*>(job.A);
    const T* B = static_cast<const T*>(job.B);
    const int group = job.group;
    const float mul = job.mul;
    const int64_t head = block / job.run;
    const int chunk = job.chunk0 + int(block % job.run);
    const int64_t n0 = int64_t(chunk) * kGatedC;
    gated_load_gates(G, lg + head * N, n0, N);
    __syncthreads();
    if (threadIdx.x == 0) job.gtot[head * nchunk + chunk] = exp2f(float(G[kGatedC - 1]));
    // rows of the record: RD = max(1, D/16) a thread, columns tx + 16 c
    constexpr int NC = D / 16, NR = D / 16;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[NR][NC] = {};
    const int ng = REV ? group : 1;
    for (int g = 0; g < ng; ++g) {
        if (g) __syncthreads();
        const int64_t src = (REV ? head * group + g : head) * N * D;
        gated_load_tile<T, D>(ta, A + src, n0, N);
        gated_load_tile<T, D>(tb, B + src, n0, N);
        __syncthreads();
        for (int i = threadIdx.x; i < kGatedC * D; i += kGatedThreads) {
            const int r = i / D, c = i % D;
            const float w = REV ? mul * exp2f(float(G[r])) : exp2f(float(G[kGatedC - 1] - G[r]));
            ta[r * LD + c] *= w;
        }
        __syncthreads();
        for (int t = 0; t < kGatedC; ++t) {
            float x[NR], y[NC];
#pragma unroll
            for (int r = 0; r < NR; ++r) x[r] = ta[t * LD + ty + 16 * r];
#pragma unroll
            for (int c = 0; c < NC; ++c) y[c] = tb[t * LD + tx + 16 * c];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[r][c] = fmaf(x[r], y[c], acc[r][c]);
        }
    }
    float* out = job.rec + (head * nchunk + chunk) * int64_t(D) * D;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c) out[(ty + 16 * r) * D + tx + 16 * c] = acc[r][c];
}

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads)
gated_part_kernel(const GatedPartJob fwd, const GatedPartJob rev, const T* __restrict__ lg,
                  int64_t N, int nchunk) {
    const int64_t b = blockIdx.x;
    if (b < rev.blocks)  // the longer ones (group heads each) first
        gated_part_block<T, D, true>(rev, lg, N, nchunk, b);
    else
        gated_part_block<T, D, false>(fwd, lg, N, nchunk, b - rev.blocks);
}

// ------------------------------------------------------- the chunks' recurrence
// In place over a head's records: what enters chunk c replaces its part, from
// `first` (null: zero) on; the state after the last chunk goes to `last` (may
// be null; then the part of the chunk walked last is neither computed nor
// read).  One float4 of the state a thread; the next records are loaded while
// the recurrence runs.
struct GatedCarryJob {
    float4* rec;
    const float* gtot;
    const float4* first;
    float4* last;
};

template <bool REV>
__device__ __forceinline__ void gated_carry(const GatedCarryJob& job, int64_t i, int per_head,
                                            int nchunk) {
    float4* __restrict__ rec = job.rec;
    const float* __restrict__ gtot = job.gtot;
    const float4* __restrict__ first = job.first;
    float4* __restrict__ last = job.last;
    const int64_t head = i / per_head, e = i % per_head;
    float4* r = rec + head * nchunk * per_head + e;
    const float* gt = gtot + head * nchunk;
    float4 run = first ? first[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    const int steps = last ? nchunk : nchunk - 1;  // chunks whose part is added
    for (int c0 = 0; c0 < steps; c0 += U) {
        float4 p[U];
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = REV ? nchunk - 1 - (c0 + u) : c0 + u;
            if (c0 + u < steps) {
                p[u] = r[int64_t(c) * per_head];
                a[u] = gt[c];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + u >= steps) break;
            const int c = REV ? nchunk - 1 - (c0 + u) : c0 + u;
            r[int64_t(c) * per_head] = run;
            run.x = fmaf(a[u], run.x, p[u].x);
            run.y = fmaf(a[u], run.y, p[u].y);
            run.z = fmaf(a[u], run.z, p[u].z);
            run.w = fmaf(a[u], run.w, p[u].w);
        }
    }
    if (last)
        last[i] = run;
    else
        r[int64_t(REV ? 0 : nchunk - 1) * per_head] = run;
}

// blockIdx.y: 0 the first job, forwards; 1 the second, backwards; a job without
// records is skipped
__global__ void __launch_bounds__(128)
gated_carry_kernel(const GatedCarryJob fwd, const GatedCarryJob rev, int64_t total, int per_head,
                   int nchunk) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    if (blockIdx.y == 0) {
        if (fwd.rec) gated_carry<false>(fwd, i, per_head, nchunk);
    } else {
        if (rev.rec) gated_carry<true>(rev, i, per_head, nchunk);
    }
}

// acc[r][c] += sum_e X[row r][e] Y[e][col c] with Y the record S (TRANS false,
// Y[e][c] = S[e][c]) or its transpose (Y[e][c] = S[c][e]), 64 rows of Y at a
// time through the shared tile `buf` ([64][D + 4] floats); rows from `rows` on
// are left out.
template <int D, bool TRANS>
__device__ __forceinline__ void gated_mm_state(float (&acc)[4][D / 16], const float* X,
                                               const float* __restrict__ S, float* buf, int rows,
                                               int ty, int tx) {
    constexpr int LD = GatedTile::ld(D);
    constexpr int KB = D < kGatedC ? D : kGatedC;
    for (int k0 = 0; k0 < D; k0 += KB) {
        __syncthreads();
        for (int i = threadIdx.x; i < KB * D; i += kGatedThreads) {
            // global reads run along the record's rows
            const int a = TRANS ? i / KB : i / D, b = TRANS ? i % KB : i % D;
            if (TRANS)
                buf[b * LD + a] = S[a * D + k0 + b];
            else
                buf[a * LD + b] = S[(k0 + a) * D + b];
        }
        __syncthreads();
        if (4 * ty < rows) gated_mm_nn<D / 16>(acc, X + k0, LD, buf, LD, KB, ty, tx);
    }
}

// ------------------------------------------------------------- o, dq, dk, dv
// One chunk of one row head:
//   out_i = in_mul sum_j w_ij (R_i . K_j) V_j + st_mul r_i (R_i through S)
// forward (REV false): j <= i, w = e^{G_i-G_j}, r = e^{G_i}; row heads are
// query heads, columns come from key/value head / group.  REV: j >= i, w =
// e^{G_j-G_i}, r = e^{G_C-G_i}; row heads are key/value heads and the columns
// run over the group's query heads.  TRANS: rows meet S^T (dq, dk).
template <typename T, int D, bool REV, bool TRANS>
__device__ __forceinline__ void gated_rows_block(
    const T* __restrict__ R, const T* __restrict__ K, const T* __restrict__ V,
    const T* __restrict__ lg, const float* __restrict__ rec, T* __restrict__ out, int64_t N,
    int nchunk, int group, float in_mul, float st_mul, int64_t block) {
    constexpr int LD = GatedTile::ld(D), LP = GatedTile::ld(kGatedC), NC = D / 16;
    extern __shared__ __align__(16) float sm[];
    float* tr = sm;
    float* tk = tr + kGatedC * LD;
    float* tv = tk + kGatedC * LD;
    float* tp = tv + kGatedC * LD;
    __shared__ double G[kGatedC];
    const int64_t head = block / nchunk;
    const int chunk = int(block % nchunk);
    const int64_t kvh = REV ? head : head / group;
    const int64_t n0 = int64_t(chunk) * kGatedC;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int rows = gated_rows(n0, N);
    const bool live = 4 * ty < rows;
    gated_load_gates(G, lg + kvh * N, n0, N);
    gated_load_tile<T, D>(tr, R + head * N * D, n0, N);
    float acc[4][NC] = {};
    const int ng = REV ? group : 1;
    for (int g = 0; g < ng; ++g) {
        const int64_t src = (REV ? head * group + g : kvh) * N * D;
        gated_load_tile<T, D>(tk, K + src, n0, N);
        gated_load_tile<T, D>(tv, V + src, n0, N);
        __syncthreads();
        float p[4][4] = {};
        if (live) gated_mm_nt<D, 4>(p, tr, LD, tk, LD, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = 4 * ty + r, j = tx + 16 * c;
                const bool in = REV ? j >= i : j <= i;
                const float w = in ? exp2f(float(REV ? G[j] - G[i] : G[i] - G[j])) : 0.f;
                tp[i * LP + j] = in ? in_mul * w * p[r][c] : 0.f;
            }
        __syncthreads();
        if (live) gated_mm_nn<NC>(acc, tp, LP, tv, LD, rows, ty, tx);
        __syncthreads();
    }
    if (rec) {
        float s[4][NC] = {};
        gated_mm_state<D, TRANS>(s, tr, rec + (kvh * nchunk + chunk) * int64_t(D) * D, tk, rows,
                                 ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * ty + r;
            const float w = st_mul * exp2f(float(REV ? G[kGatedC - 1] - G[i] : G[i]));
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[r][c] = fmaf(w, s[r][c], acc[r][c]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t n = n0 + 4 * ty + r;
        if (n < N)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                out[(head * N + n) * D + tx + 16 * c] = from_f32<T>(acc[r][c]);
    }
}

// ------------------------------------------------------------------ dlog_gate
template <typename T, int D>
__device__ __forceinline__ void gated_dgate_block(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const T* __restrict__ dO, const T* __restrict__ lg, const float* __restrict__ recS,
    const float* __restrict__ recR, T* __restrict__ dlg, int64_t N, int nchunk, int group,
    float scale, int64_t block) {
    constexpr int LD = GatedTile::ld(D), NC = D / 16;
    extern __shared__ __align__(16) float sm[];
    float* ta = sm;                     // q, then k
    float* tb = ta + kGatedC * LD;      // dO, then v
    float* tk = tb + kGatedC * LD;
    float* tv = tk + kGatedC * LD;
    __shared__ double G[kGatedC];
    __shared__ float rows[kGatedC];           // sum_j M_ij (j < i) and q_i.dq^S_i, by i
    __shared__ float cols[16][kGatedC];       // sum_i M_ij (i > j), by j, one row a ty
    __shared__ float through[kGatedC];        // k_j.dk^R_j
    __shared__ float wsum[kGatedThreads / 32];
    const int64_t head = block / nchunk;
    const int chunk = int(block % nchunk);
    const int64_t n0 = int64_t(chunk) * kGatedC;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const float* S = recS ? recS + (head * nchunk + chunk) * int64_t(D) * D : nullptr;
    const float* R = recR ? recR + (head * nchunk + chunk) * int64_t(D) * D : nullptr;
    const int n_rows = gated_rows(n0, N);
    const bool live = 4 * ty < n_rows;
    gated_load_gates(G, lg + head * N, n0, N);
    gated_load_tile<T, D>(tk, k + head * N * D, n0, N);
    gated_load_tile<T, D>(tv, v + head * N * D, n0, N);
    float rs[4] = {}, cs[4] = {};
    for (int g = 0; g < group; ++g) {
        const int64_t src = (head * group + g) * N * D;
        __syncthreads();
        gated_load_tile<T, D>(ta, q + src, n0, N);
        gated_load_tile<T, D>(tb, dO + src, n0, N);
        __syncthreads();
        float p[4][4] = {}, w[4][4] = {};
        if (live) {
            gated_mm_nt<D, 4>(p, ta, LD, tk, LD, ty, tx);
            gated_mm_nt<D, 4>(w, tb, LD, tv, LD, ty, tx);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = 4 * ty + r, j = tx + 16 * c;
                if (j < i) {
                    const float m = scale * exp2f(float(G[i] - G[j])) * p[r][c] * w[r][c];
                    rs[r] += m;
                    cs[c] += m;
                }
            }
        if (S) {  // scale e^{G_i} q_i^T S dO_i
            float s[4][NC] = {};
            // the state passes through no tile that is still read: k and v are
            // reloaded below
            gated_mm_state<D, false>(s, ta, S, tk, n_rows, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                float d = 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c) d = fmaf(s[r][c], tb[i * LD + tx + 16 * c], d);
                rs[r] = fmaf(scale * exp2f(float(G[i])), d, rs[r]);
            }
            __syncthreads();
            gated_load_tile<T, D>(tk, k + head * N * D, n0, N);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float x = rs[r];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (tx == 0) rows[4 * ty + r] = x;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) cols[ty][tx + 16 * c] = cs[c];
    __syncthreads();
    if (R) {  // e^{G_C-G_j} k_j^T R v_j
        float s[4][NC] = {};
        gated_mm_state<D, false>(s, tk, R, ta, n_rows, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 4 * ty + r;
            float d = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) d = fmaf(s[r][c], tv[j * LD + tx + 16 * c], d);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            if (tx == 0) through[j] = d * exp2f(float(G[kGatedC - 1] - G[j]));
        }
    } else if (tid < kGatedC) {
        through[tid] = 0.f;
    }
    float x = 0.f;  // <S, R>
    if (S && R)
        for (int i = tid; i < D * D; i += kGatedThreads) x = fmaf(S[i], R[i], x);
    x = warp_sum(x);
    if ((tid & 31) == 0) wsum[tid >> 5] = x;
    __syncthreads();
    if (tid < 32) {
        // tokens 2 l and 2 l + 1 of lane l: sums from the end of rows less
        // columns, from the start of what passes through R
        float all = 0.f;
#pragma unroll
        for (int u = 0; u < kGatedThreads / 32; ++u) all += wsum[u];
        all *= exp2f(float(G[kGatedC - 1]));
        float d0 = rows[2 * tid], d1 = rows[2 * tid + 1];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            d0 -= cols[u][2 * tid];
            d1 -= cols[u][2 * tid + 1];
        }
        const float t0 = through[2 * tid], t1 = through[2 * tid + 1];
        float s = d0 + d1, t = t0 + t1;  // inclusive suffix / prefix sums over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, s, o);
            const float b = __shfl_up_sync(0xffffffffu, t, o);
            if (tid + o < 32) s += a;
            if (tid >= o) t += b;
        }
        // shifted, not subtracted: a token's own term may be larger than the rest
        // by more than float32 holds
        float before = __shfl_up_sync(0xffffffffu, t, 1);
        float behind = __shfl_down_sync(0xffffffffu, s, 1);
        if (tid == 0) before = 0.f;
        if (tid == 31) behind = 0.f;
        const int64_t n = n0 + 2 * tid;
        auto put = [&](int64_t at, float x) {
            if (at >= N) return;
            const double gate = gate_log2(to_f32(lg[head * N + at]));
            dlg[head * N + at] = from_f32<T>(gate_is_zero(gate) ? 0.f : x);
        };
        put(n, s + before + all);
        put(n + 1, d1 + behind + (before + t0) + all);
    }
}

// -------------------------------------------------------------------- launches
template <typename T>
struct GatedTensors {
    const T *q, *k, *v, *lg, *dO;
    T *o, *dq, *dk, *dv, *dlg;
    const float *S, *R;         // records, or null
    int64_t N, qheads, kvh;
    int nchunk, group;
    float scale;
};

template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads) gated_o_kernel(const GatedTensors<T> p) {
    gated_rows_block<T, D, false, false>(p.q, p.k, p.v, p.lg, p.S, p.o, p.N, p.nchunk, p.group,
                                         p.scale, p.scale, blockIdx.x);
}

// A block a chunk and gradient; the longest work first.
template <typename T, int D>
__global__ void __launch_bounds__(kGatedThreads) gated_grad_kernel(const GatedTensors<T> p) {
    const int64_t kvb = p.kvh * p.nchunk;
    int64_t b = blockIdx.x;
    if (b < kvb) {
        gated_dgate_block<T, D>(p.q, p.k, p.v, p.dO, p.lg, p.S, p.R, p.dlg, p.N, p.nchunk, p.group,
                                p.scale, b);
    } else if ((b -= kvb) < kvb) {
        gated_rows_block<T, D, true, true>(p.v, p.dO, p.q, p.lg, p.R, p.dk, p.N, p.nchunk, p.group,
                                           p.scale, 1.f, b);
    } else if ((b -= kvb) < kvb) {
        gated_rows_block<T, D, true, false>(p.k, p.q, p.dO, p.lg, p.R, p.dv, p.N, p.nchunk, p.group,
                                            p.scale, 1.f, b);
    } else {
        gated_rows_block<T, D, false, true>(p.dO, p.v, p.k, p.lg, p.S, p.dq, p.N, p.nchunk, p.group,
                                            p.scale, p.scale, b - kvb);
    }
}

}  // namespace la

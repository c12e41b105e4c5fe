// la_gated_tc.cuh — gated linear attention on the tensor cores (bf16, D = 64
// or 128; formulas in la_gated_common.cuh).
//
// The sequence is cut into blocks of C = 128 tokens and spans of L = 128 nb
// tokens; states exist at the spans' borders only, and inside a span every
// block meets the span's blocks before it (forward) or behind it (REV)
// directly.  No block waits for another: all of the sequence is in flight at
// once, whatever the number of heads, and the only serial step is the states'
// recurrence over the spans (gated_border_kernel), which is elementwise.
//
//   gated_span_kernel    a span's own part of the state, sum_t w_t A_t B_t^T
//   gated_border_kernel  the recurrence; bf16 states entering every span
//   gated_block_kernel   o, dq, dk or dv of a 128-token block
//   gated_dgate_sum_kernel  dlog_gate from the pieces the blocks leave
//
// Bytes a token and head (D = 128, nb = 2): k and v once for the parts (4 D),
// the records written, read and written again in bf16, and read (4 + 4 + 2 + 2
// bytes of D^2 / 256 each: 6 D), q, k, v and o once (8 D).
//
// Weights.  Between tokens j <= i the weight is e^{G_i - G_j}.  Sums of log2
// gates are formed in 64 bits per span; a 32-token sub-block J then splits the
// exponent at its border, e^{G_i - G_j} = e^{G_i - G_end(J)} e^{G_end(J) - G_j},
// two factors that are at most 1 for gates of at most 1 and of which the first
// is one exponential per row and sub-block and the second one per token; only
// the 32 x 32 sub-blocks on the diagonal take an exponential per element.
//
// Rounding.  q, k, v, dO are read exactly.  The weighted C x C product and the
// border states are rounded to bf16 once, as tensor-core operands; the scaled
// operand of the parts is held as two bf16 values (hi + lo, 2^-17), so that
// the float32 states returned to the caller keep float32 accuracy; the row
// factors of what comes through a state are applied to the float32 result.
#pragma once

#include "la_chunk_fwd.cuh"
#include "la_gated_common.cuh"

namespace la {

constexpr int kGtC = 128;     // tokens a block
constexpr int kGtMaxNb = 4;   // blocks a span, at most

struct alignas(16) GateTab {
    float loc[kGtMaxNb * kGtC];   // sums of log2 gates from the sub-block's start, inclusive
    float fac[kGtMaxNb * kGtC];   // forward: 2^(to the sub-block's end); REV: 2^loc
    double start[4 * kGtMaxNb + 2];  // sums before each 32-token sub-block; [nsub] = all
};

// MMAs issued by one lane of a warp that runs the issue loop together: the
// descriptors stay warp-uniform values and only the instruction is predicated.
// Inside `if (lane == 0)` the issuing thread needs more instructions an MMA
// (131072 tokens, D = 128, forward blocks: 1554 us, 1368 this way on the same
// GPU), and in gated_bwd64_kernel, with its many tiles, 180 cycles an MMA
// against 45 to 60.
__device__ __forceinline__ void umma_one(uint32_t one, uint32_t d_tmem, uint64_t adesc,
                                         uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void umma_ts_one(uint32_t one, uint32_t d_tmem, uint32_t a_tmem,
                                            uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::
            "r"(sm100::smem_u32(bar)),
        "r"(one)
        : "memory");
}
// One lane of the (converged) warp, the same one every time.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(one));
    return one;
}
// All lanes wait; false for all when one of the waits gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort));
}

__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sums of the span's log2 gates by one warp: lane l takes the tokens l*nsub ..
// l*nsub + nsub - 1 (nsub = 4 nb = 4, 8 or 16), so a sub-block of 32 tokens is
// 32 / nsub neighbouring lanes.  Tokens from N on count as gates of 1.
// use(t, sum, before, start, end, all): token t of the span, the sums up to
// and with it, before its sub-block, to its sub-block's end, and of the span.
template <typename F>
__device__ __forceinline__ void gate_sums(const __nv_bfloat16* lg, int64_t n0, int64_t N,
                                          int nsub, int lane, double* start, F use) {
    const int64_t first = n0 + lane * nsub;
    double s = 0.0;
    for (int u = 0; u < nsub; ++u)
        if (first + u < N) s += gate_log2(__bfloat162float(lg[first + u]));
    const double incl = warp_scan_sum(s, lane);
    const int per = 32 / nsub;  // lanes a sub-block
    const int lo = lane & ~(per - 1);
    const double before = __shfl_sync(0xffffffffu, incl - s, lo);
    const double end = __shfl_sync(0xffffffffu, incl, lo + per - 1);
    const double all = __shfl_sync(0xffffffffu, incl, 31);
    if (start) {
        if (lane == lo) start[lane / per] = before;
        if (lane == 31) start[nsub] = all;
    }
    double run = incl - s;
    for (int u = 0; u < nsub; ++u) {
        if (first + u < N) run += gate_log2(__bfloat162float(lg[first + u]));
        use(lane * nsub + u, run, before, end, all);
    }
}

// ------------------------------------------------------------ a span's part
struct GatedSpanParams {
    CUtensorMap tm_a, tm_b;   // the scaled operand (k; REV: q) and the other (v; dO)
    const __nv_bfloat16* lg;
    float* rec;               // [kvh][nspan][D][D]
    float* tot;               // [kvh][nspan]: product of the span's gates
    int64_t N;
    int64_t items;            // kvh * spans_run
    int nspan, spans_run, span0;
    int nb, nblk, group;
    float mul;
};

template <int D>
struct GatedSpanCfg {
    static constexpr int TILE = kGtC * D * 2;
    static constexpr int NS = 4;                      // ring slots: A, B, A, B
    static constexpr int OFF_SC = NS * TILE;          // the scaled operand: hi tile, lo tile
    static constexpr int OFF_W = OFF_SC + 2 * TILE;   // weights [2][512]
    static constexpr int OFF_BAR = OFF_W + 2 * kGtMaxNb * kGtC * 4;
    static constexpr int NBAR = 2 * NS + 11;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int ACC = 2 * D;                 // columns: hi part, lo part
    static constexpr int T_COLS = 2 * ACC;
    static constexpr int CTAS = D == 64 ? 2 : 1;
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
    static_assert(CTAS * T_COLS <= 512, "TMEM budget");
};

// Warps: 0 TMA, 1 MMA, 2 gate sums, 3 idle, 4-11 scale, 12-15 write the record.
constexpr int kGatedSpanThreads = 512;

// The accumulator is transposed, acc[e][d] = sum_t B_t[e] (w_t A_t)[d], with
// the scaled operand's two parts side by side in columns: one MMA of N = 2 D
// per 16 tokens, and a thread adds the two parts of its row.
template <int D, bool REV>
__global__ void __launch_bounds__(kGatedSpanThreads, GatedSpanCfg<D>::CTAS)
gated_span_kernel(const __grid_constant__ GatedSpanParams prm) {
    using namespace sm100;
    using Cfg = GatedSpanCfg<D>;
    constexpr int C = kGtC, NS = Cfg::NS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [NS] TMA
    uint64_t* empty = full + NS;       // [NS] A: scaled (256); B: MMA done (commit)
    uint64_t* sc_full = empty + NS;    // scaled operand written          (256)
    uint64_t* sc_free = sc_full + 1;   // MMAs have read it               (commit)
    uint64_t* acc_full = sc_full + 2;  // [2] record complete             (commit)
    uint64_t* acc_free = sc_full + 4;  // [2] record read                 (128)
    uint64_t* w_full = sc_full + 6;    // [2] weights written             (32)
    uint64_t* w_free = sc_full + 8;    // [2] weights read                (256)
    uint64_t* drain = sc_full + 10;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    float* wtab = reinterpret_cast<float*>(smem + Cfg::OFF_W);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], (s & 1) ? 1 : 256);
        }
        mbar_init(sc_full, 256);
        mbar_init(sc_free, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 128);
            mbar_init(&w_full[b], 32);
            mbar_init(&w_free[b], 256);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int64_t items = prm.items;
    // item -> key/value head, span, blocks of the span (times the group's heads)
    auto head_of = [&](int64_t it) { return it / prm.spans_run; };
    auto span_of = [&](int64_t it) { return prm.span0 + int(it % prm.spans_run); };
    auto blocks_of = [&](int span) { return min(prm.nb, prm.nblk - span * prm.nb); };
    const int ng = REV ? prm.group : 1;

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&prm.tm_a);
            tma_prefetch_desc(&prm.tm_b);
            uint32_t n = 0;  // tiles issued
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x) {
                const int64_t head = head_of(it);
                const int span = span_of(it), nbv = blocks_of(span);
                for (int b = 0; ok && b < ng * nbv; ++b) {
                    const int src = int(REV ? head * prm.group + b / nbv : head);
                    const int row = (span * prm.nb + b % nbv) * C;
                    for (int t = 0; t < 2; ++t, ++n) {
                        const int s = n % NS;
                        if (n >= NS &&
                            !(ok = mbar_wait(&empty[s], ((n / NS) - 1) & 1, abort_flag)))
                            break;
                        mbar_arrive_expect_tx(&full[s], Cfg::TILE);
                        for (int a = 0; a < D / 64; ++a)
                            tma_load_3d(smem + s * Cfg::TILE + a * C * 128,
                                        t ? &prm.tm_b : &prm.tm_a, &full[s], 64 * a, row, src);
                    }
                }
            }
            for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i)
                mbar_wait_drain(&full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1) {
        {
            const uint32_t one = elect_lane();
            constexpr uint32_t id = idesc_bf16(D, 2 * D, 1, 1);
            const uint64_t dsc = desc_mn_base(sbase + Cfg::OFF_SC, C);
            uint32_t n = 0, blk = 0, m = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x, ++m) {
                const int cnt = ng * blocks_of(span_of(it));
                const uint32_t acc = tmem + (m & 1) * Cfg::ACC;
                if (m >= 2 && !(ok = warp_wait(&acc_free[m & 1], ((m >> 1) - 1) & 1, abort_flag)))
                    break;
                for (int b = 0; b < cnt; ++b, ++blk, n += 2) {
                    const int s = (n + 1) % NS;
                    if (!(ok = warp_wait(&full[s], ((n + 1) / NS) & 1, abort_flag))) break;
                    if (!(ok = warp_wait(sc_full, blk & 1, abort_flag))) break;
                    tc_fence_after();
                    const uint64_t db = desc_mn_base(sbase + s * Cfg::TILE, C);
#pragma unroll
                    for (int k = 0; k < C; k += 16)
                        umma_one(one, acc, db + kstep_mn(k), dsc + kstep_mn(k), id, b > 0 || k > 0);
                    commit_one(one, &empty[s]);
                    commit_one(one, sc_free);
                }
                if (ok) commit_one(one, &acc_full[m & 1]);
            }
            commit_one(one, drain);
            if (lane == 0) mbar_wait_drain(drain, 0);
        }
    } else if (warp == 2) {
        uint32_t m = 0;
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x, ++m) {
            const int buf = m & 1;
            if (!__all_sync(0xffffffffu, m < 2 || mbar_wait(&w_free[buf], ((m >> 1) - 1) & 1,
                                                            abort_flag)))
                break;
            const int64_t head = head_of(it);
            const int span = span_of(it);
            float* w = wtab + buf * kGtMaxNb * C;
            double total = 0.0;
            gate_sums(prm.lg + head * prm.N, int64_t(span) * prm.nb * C, prm.N, 4 * prm.nb, lane,
                      nullptr, [&](int t, double run, double, double, double all) {
                          w[t] = REV ? prm.mul * exp2f(float(run)) : exp2f(float(all - run));
                          total = all;
                      });
            if (lane == 0) prm.tot[head * prm.nspan + span] = exp2f(float(total));
            mbar_arrive(&w_full[buf]);
        }
    } else if (warp >= 4 && warp < 12) {
        // scale A's rows: thread u takes half a row (D / 2 elements)
        const int u = tid - 128;
        const int row = u >> 1, q0 = (u & 1) * (D / 16);
        uint8_t* sc = smem + Cfg::OFF_SC;
        uint32_t n = 0, blk = 0, m = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x, ++m) {
            const int nbv = blocks_of(span_of(it));
            const float* w = wtab + (m & 1) * kGtMaxNb * C;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&w_full[m & 1], (m >> 1) & 1,
                                                         abort_flag))))
                break;
            for (int b = 0; b < ng * nbv; ++b, ++blk, n += 2) {
                const int s = n % NS;
                if (!(ok = __all_sync(0xffffffffu,
                                      mbar_wait(&full[s], (n / NS) & 1, abort_flag))))
                    break;
                const uint8_t* src = smem + s * Cfg::TILE;
                uint4 x[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    x[i] = *reinterpret_cast<const uint4*>(src + tile_chunk_off(C, row, q0 + i));
                mbar_arrive(&empty[s]);
                if (!(ok = __all_sync(0xffffffffu, blk == 0 || mbar_wait(sc_free, (blk - 1) & 1,
                                                                         abort_flag))))
                    break;
                const float wr = w[(b % nbv) * C + row];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t h[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, l[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 f = unpack_bf16(h[j]);
                        f.x *= wr;
                        f.y *= wr;
                        h[j] = pack_bf16(f.x, f.y);
                        const float2 r = unpack_bf16(h[j]);
                        l[j] = pack_bf16(f.x - r.x, f.y - r.y);
                    }
                    const uint32_t off = tile_chunk_off(C, row, q0 + i);
                    *reinterpret_cast<uint4*>(sc + off) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(sc + Cfg::TILE + off) =
                        make_uint4(l[0], l[1], l[2], l[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(sc_full);
            }
            if (ok) mbar_arrive(&w_free[m & 1]);
        }
    } else if (warp >= 12) {
        const int sp = warp & 3;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int e = acc_row<D>(sp, lane);  // row of the accumulator: column of the state
        uint32_t m = 0;
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x, ++m) {
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[m & 1], (m >> 1) & 1, abort_flag)))
                break;
            tc_fence_after();
            const uint32_t acc = tmem + lane_base + (m & 1) * Cfg::ACC;
            float* out = prm.rec + (head_of(it) * prm.nspan + span_of(it)) * int64_t(D) * D;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 16) {
                float hi[16], lo[16];
                tmem_ld16(acc + d0, hi);
                tmem_load<16>(acc + D + d0, lo);
                if (e >= 0) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[(d0 + j) * D + e] = hi[j] + lo[j];
                }
            }
            tc_fence_before();
            mbar_arrive(&acc_free[m & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::T_COLS);
}

// --------------------------------------------------------- the spans' recurrence
// The state entering every span in bf16 (operands of the blocks), from the
// spans' float32 parts; run itself stays float32.  One float4 a thread.
// `last` may be null; then the part of the span walked last is not read.
template <bool REV>
__global__ void __launch_bounds__(128)
gated_border_kernel(const float4* __restrict__ rec, const float* __restrict__ tot,
                    const float4* __restrict__ first, float4* __restrict__ last,
                    uint2* __restrict__ enter, int64_t total, int per_head, int nspan) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int64_t head = i / per_head, e = i % per_head;
    const float4* r = rec + head * nspan * per_head + e;
    uint2* out = enter + head * nspan * per_head + e;
    const float* gt = tot + head * nspan;
    float4 run = first ? first[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    const int steps = last ? nspan : nspan - 1;
    auto put = [&](int c) {
        out[int64_t(c) * per_head] =
            make_uint2(sm100::pack_bf16(run.x, run.y), sm100::pack_bf16(run.z, run.w));
    };
    for (int c0 = 0; c0 < steps; c0 += U) {
        float4 p[U];
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = REV ? nspan - 1 - (c0 + u) : c0 + u;
            if (c0 + u < steps) {
                p[u] = __ldcs(r + int64_t(c) * per_head);
                a[u] = gt[c];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + u >= steps) break;
            put(REV ? nspan - 1 - (c0 + u) : c0 + u);
            run.x = fmaf(a[u], run.x, p[u].x);
            run.y = fmaf(a[u], run.y, p[u].y);
            run.z = fmaf(a[u], run.z, p[u].z);
            run.w = fmaf(a[u], run.w, p[u].w);
        }
    }
    if (last)
        last[i] = run;
    else
        put(REV ? 0 : nspan - 1);
}

// ------------------------------------------------------------- o, dq, dk, dv
// out_i = in_mul sum_j w_ij (R_i . K_j) V_j + st_mul r_i (R_i through the state)
// (see gated_rows_kernel).  XTRA = 0: no more.  XTRA = 1: also the dot of a
// second row tile with what came through the state, rowv_i = R2_i . st_mul r_i
// (R_i S).  XTRA = 2: besides, M_ij = in_mul w_ij (R_i . K_j)(R2_i . V_j), its
// sums over j < i added to rowv_i and its sums over the 32 rows of each
// sub-block to colv.
struct GatedBlockParams {
    CUtensorMap tm_row, tm_col, tm_val, tm_st, tm_out, tm_row2;
    const __nv_bfloat16* lg;
    float* rowv;      // [2][row heads][N]
    float* colv;      // [row heads][4 nb][N]
    int64_t N, items, heads;
    int nblk, nb, nspan, group, has_state;
    float in_mul, st_mul;
};

template <int D, int XTRA>
struct GatedBlockCfg {
    static constexpr int TILE = kGtC * D * 2;
    static constexpr int CTAS = D == 64 && XTRA < 2 ? 2 : 1;
    // an item's row tiles stay for all of its column blocks, so they have
    // buffers of their own (NR each) beside the ring of the others (NS)
    static constexpr int NS = D == 64 && XTRA == 2 ? 8 : 4;
    static constexpr int NR = XTRA == 0 || (D == 64 && XTRA == 2) ? 2 : 1;
    static constexpr int ROWT = XTRA ? 2 : 1;                // row tiles of an item
    static constexpr int NP = D == 128 && XTRA < 2 ? 2 : 1;  // P buffers
    static constexpr int OFF_ROW = NS * TILE;
    static constexpr int OFF_TAB = OFF_ROW + NR * ROWT * TILE;
    static constexpr int OFF_BAR = OFF_TAB + 2 * int(sizeof(GateTab));
    static constexpr int NBAR = 2 * NS + 21;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int T_P = 0;
    static constexpr int T_P2 = kGtC;                        // XTRA = 2
    static constexpr int T_ST = kGtC * (XTRA == 2 ? 2 : NP); // through the state
    static constexpr int T_IN = T_ST + D;                    // inside the span
    static constexpr int T_USED = T_IN + D;
    static constexpr int T_COLS = T_USED <= 256 ? 256 : 512;
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
    static_assert(CTAS * T_COLS <= 512, "TMEM budget");
};

// Warps: 0 TMA loads of the ring, 1 MMA, 2 gate tables and TMA loads of the
// rows, 3 TMA stores, 4-11 compute: two groups of four warps, group h for the column half h of every C x C product
// and of the output.
constexpr int kGatedBlockThreads = 384;

template <int D, bool REV, bool TRANS, int XTRA>
__global__ void __launch_bounds__(kGatedBlockThreads, GatedBlockCfg<D, XTRA>::CTAS)
gated_block_kernel(const __grid_constant__ GatedBlockParams prm) {
    using namespace sm100;
    using Cfg = GatedBlockCfg<D, XTRA>;
    constexpr int C = kGtC, NS = Cfg::NS, NP = Cfg::NP;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [NS] TMA
    uint64_t* empty = full + NS;        // [NS] released (commit, or the store warp)
    uint64_t* p_full = empty + NS;      // [2] P complete                (commit)
    uint64_t* pt_full = p_full + 2;     // [2] weighted P packed         (256)
    uint64_t* p_free = p_full + 4;      // [2] ... consumed              (commit)
    uint64_t* o_full = p_full + 6;      // output accumulators complete  (commit)
    uint64_t* o_free = p_full + 7;      // ... read                      (256)
    uint64_t* out_full = p_full + 8;    // [2] output staged             (256)
    uint64_t* out_free = p_full + 10;   // [2] ... stored                (1)
    uint64_t* tab_full = p_full + 12;   // [2] gate tables written       (32)
    uint64_t* tab_free = p_full + 14;   // [2] ... read                  (256)
    uint64_t* row_full = p_full + 16;   // [2] row tiles landed           (1 + tx)
    uint64_t* row_free = p_full + 18;   // [2] ... read (commit; XTRA: and the epilogue)
    uint64_t* drain = p_full + 20;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    GateTab* tabs = reinterpret_cast<GateTab*>(smem + Cfg::OFF_TAB);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&p_full[b], 1);
            mbar_init(&pt_full[b], 256);
            mbar_init(&p_free[b], 1);
            mbar_init(&out_full[b], 256);
            mbar_init(&out_free[b], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, 256);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tab_full[b], 32);
            mbar_init(&tab_free[b], 256);
            mbar_init(&row_full[b], 1);
            mbar_init(&row_free[b], XTRA ? 2 : 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // One item: 128 rows.  Its other tiles arrive in the ring in the order
    // col 0, [state], val 0, col 1, val 1, ...
    struct Item {
        int64_t head, kvh;  // row head, key/value head
        int span, rb;       // span of the head, block of the span
        int nbv;            // blocks of this span
        int per;            // column blocks a head
        int ncb;            // column blocks (times the group's heads, REV)
        int loads;          // tiles through the ring
    };
    auto item_of = [&](int64_t it) {
        Item x;
        x.head = int(unsigned(it) / unsigned(prm.nblk));
        const int blk = int(unsigned(it) % unsigned(prm.nblk));
        x.kvh = REV ? x.head : int(unsigned(x.head) / unsigned(prm.group));
        x.span = blk / prm.nb;
        x.nbv = min(prm.nb, prm.nblk - x.span * prm.nb);
        // the blocks of a span differ in cost by their place in it: turn the
        // order from span to span, so that a stride over the items (the grid)
        // meets every place
        const unsigned s = unsigned(x.head * prm.nspan + x.span);
        x.rb = int((unsigned(blk % prm.nb) + s + (s >> 1)) % unsigned(x.nbv));
        x.per = REV ? x.nbv - x.rb : x.rb + 1;
        x.ncb = REV ? x.per * prm.group : x.per;
        x.loads = (prm.has_state ? 1 : 0) + 2 * x.ncb;
        return x;
    };
    // block of the span that column block b stands for
    auto col_of = [&](const Item& x, int b) { return REV ? x.rb + b % x.per : b; };

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&prm.tm_col);
            tma_prefetch_desc(&prm.tm_val);
            uint32_t n = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap* map, int rows, int row, int64_t head) {
                const int s = n % NS;
                if (n >= NS && !mbar_wait(&empty[s], ((n / NS) - 1) & 1, abort_flag)) return false;
                mbar_arrive_expect_tx(&full[s], uint32_t(rows) * D * 2);
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(smem + s * Cfg::TILE + a * rows * 128, map, &full[s], 64 * a, row,
                                int(head));
                ++n;
                return true;
            };
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x) {
                const Item x = item_of(it);
                const int base = x.span * prm.nb;
                for (int b = 0; ok && b < x.ncb; ++b) {
                    const int64_t src = REV ? x.head * prm.group + b / x.per : x.kvh;
                    const int row = (base + col_of(x, b)) * C;
                    ok = load(&prm.tm_col, C, row, src);
                    if (ok && b == 0 && prm.has_state)
                        ok = load(&prm.tm_st, D, 0, x.kvh * prm.nspan + x.span);
                    if (ok) ok = load(&prm.tm_val, C, row, src);
                }
            }
            for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i)
                mbar_wait_drain(&full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1) {
        {
            const uint32_t one = elect_lane();
            constexpr uint32_t idP = idesc_bf16(C, C, 0, 0);             // rows x columns
            constexpr uint32_t idS = idesc_bf16(C, D, 0, TRANS ? 0 : 1); // rows through S or S^T
            constexpr uint32_t idV = idesc_bf16(C, D, 0, 1);             // weighted P, values
            uint32_t n = 0, pc = 0, m = 0;
            bool ok = true;
            auto tile = [&](uint32_t i) { return sbase + (i % NS) * Cfg::TILE; };
            auto landed = [&](uint32_t i) {
                return warp_wait(&full[i % NS], (i / NS) & 1, abort_flag);
            };
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
                const Item x = item_of(it);
                const uint32_t st = n + 1, hs = prm.has_state ? 1 : 0;
                auto col_at = [&](int b) { return b == 0 ? n : n + hs + 2 * b; };
                auto val_at = [&](int b) { return n + hs + 1 + 2 * b; };
                const uint32_t rbuf = m % Cfg::NR;
                const uint32_t row = sbase + Cfg::OFF_ROW + rbuf * Cfg::ROWT * Cfg::TILE;
                const uint64_t drow = desc_k_base(row);
                // P of column block b, into the buffer that block b - NP is done with
                auto p_part = [&](int b) {
                    const uint32_t i = pc + b, buf = i % NP;
                    if (i >= NP && !warp_wait(&p_free[buf], (i / NP - 1) & 1, abort_flag))
                        return false;
                    if (b == 0 && !warp_wait(&row_full[rbuf], (m / Cfg::NR) & 1, abort_flag))
                        return false;
                    if (!landed(col_at(b))) return false;
                    if (XTRA == 2 && !landed(val_at(b))) return false;
                    tc_fence_after();
                    const uint64_t dcol = desc_k_base(tile(col_at(b)));
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma_one(one, tmem + Cfg::T_P + buf * C, drow + kstep_k(C, k),
                                  dcol + kstep_k(C, k), idP, k > 0);
                    if constexpr (XTRA == 2) {
                        const uint64_t dr2 = desc_k_base(row + Cfg::TILE),
                                       dv = desc_k_base(tile(val_at(b)));
#pragma unroll
                        for (int k = 0; k < D; k += 16)
                            umma_one(one, tmem + Cfg::T_P2, dr2 + kstep_k(C, k), dv + kstep_k(C, k),
                                      idP, k > 0);
                    }
                    commit_one(one, &p_full[buf]);
                    commit_one(one, &empty[col_at(b) % NS]);
                    return true;
                };
                if (!(ok = p_part(0))) break;
                if (m > 0 && !(ok = warp_wait(o_free, (m - 1) & 1, abort_flag))) break;
                if (hs) {
                    if (!(ok = landed(st))) break;
                    tc_fence_after();
                    const uint64_t ds = TRANS ? desc_k_base(tile(st)) : desc_mn_base(tile(st), D);
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma_one(one, tmem + Cfg::T_ST, drow + kstep_k(C, k),
                                  ds + (TRANS ? kstep_k(D, k) : kstep_mn(k)), idS, k > 0);
                    commit_one(one, &empty[st % NS]);
                }
                if (x.ncb == 1) commit_one(one, &row_free[rbuf]);
                for (int b = 0; b < x.ncb; ++b) {
                    if (NP == 2 && b + 1 < x.ncb) {
                        if (!(ok = p_part(b + 1))) break;
                        if (b + 2 == x.ncb) commit_one(one, &row_free[rbuf]);
                    }
                    const uint32_t i = pc + b;
                    if (!(ok = warp_wait(&pt_full[i % NP], (i / NP) & 1, abort_flag))) break;
                    if (!(ok = landed(val_at(b)))) break;
                    tc_fence_after();
                    const uint32_t tp = tmem + Cfg::T_P + (i % NP) * C;
                    const uint64_t dv = desc_mn_base(tile(val_at(b)), C);
                    // packed halves: columns 0.. and 64.. of the buffer
#pragma unroll
                    for (int k = 0; k < C; k += 16)
                        umma_ts_one(one, tmem + Cfg::T_IN, tp + (k < 64 ? k / 2 : 32 + k / 2),
                                     dv + kstep_mn(k), idV, b > 0 || k > 0);
                    commit_one(one, &p_free[i % NP]);
                    if (b + 1 < x.ncb)
                        commit_one(one, &empty[val_at(b) % NS]);  // the last one: the store warp
                    else
                        commit_one(one, o_full);
                    if (NP == 1 && b + 1 < x.ncb) {
                        if (!(ok = p_part(b + 1))) break;
                        if (b + 2 == x.ncb) commit_one(one, &row_free[rbuf]);
                    }
                }
                pc += x.ncb;
                n += x.loads;
            }
            commit_one(one, drain);
            if (lane == 0) mbar_wait_drain(drain, 0);
        }
    } else if (warp == 2) {
        uint32_t m = 0, issued = 0;
        auto load_rows = [&](const Item& x) {  // of item `issued`
            const uint32_t r = issued % Cfg::NR;
            if (lane == 0) {
                uint8_t* dst = smem + Cfg::OFF_ROW + r * Cfg::ROWT * Cfg::TILE;
                mbar_arrive_expect_tx(&row_full[r], Cfg::ROWT * Cfg::TILE);
                const int row = (x.span * prm.nb + x.rb) * C;
                for (int a = 0; a < D / 64; ++a) {
                    tma_load_3d(dst + a * C * 128, &prm.tm_row, &row_full[r], 64 * a, row,
                                int(x.head));
                    if (XTRA)
                        tma_load_3d(dst + Cfg::TILE + a * C * 128, &prm.tm_row2, &row_full[r],
                                    64 * a, row, int(x.head));
                }
            }
            ++issued;
        };
        for (int64_t it = blockIdx.x; it < prm.items; it += gridDim.x, ++m) {
            const int buf = m & 1;
            const Item x = item_of(it);
            if (m < Cfg::NR) load_rows(x);
            if (!__all_sync(0xffffffffu, m < 2 || mbar_wait(&tab_free[buf], ((m >> 1) - 1) & 1,
                                                            abort_flag)))
                break;
            GateTab& tab = tabs[buf];
            gate_sums(prm.lg + x.kvh * prm.N, int64_t(x.span) * prm.nb * C, prm.N, 4 * prm.nb,
                      lane, tab.start, [&](int t, double run, double before, double end, double) {
                          tab.loc[t] = float(run - before);
                          tab.fac[t] = ex2_fast(float(REV ? run - before : end - run));
                      });
            mbar_arrive(&tab_full[buf]);
            if (m >= Cfg::NR) {
                if (!__all_sync(0xffffffffu, mbar_wait(&row_free[m % Cfg::NR],
                                                       (m / Cfg::NR - 1) & 1, abort_flag)))
                    break;
                load_rows(x);
            }
        }
        if (lane == 0)
            for (uint32_t i = issued > Cfg::NR ? issued - Cfg::NR : 0; i < issued; ++i)
                mbar_wait_drain(&row_full[i % Cfg::NR], (i / Cfg::NR) & 1);
    } else if (warp == 3) {
        if (lane == 0) {
            uint32_t n = 0, m = 0;
            for (int64_t it = blockIdx.x; it < prm.items; it += gridDim.x, ++m) {
                const Item x = item_of(it);
                if (!mbar_wait(&out_full[m & 1], (m >> 1) & 1, abort_flag)) break;
                const uint32_t last = n + x.loads - 1;
                const uint8_t* src = smem + (last % NS) * Cfg::TILE;
                for (int a = 0; a < D / 64; ++a)
                    tma_store_3d(&prm.tm_out, src + a * C * 128, 64 * a,
                                 (x.span * prm.nb + x.rb) * C, int(x.head));
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(&empty[last % NS]);
                if (XTRA) mbar_arrive(&row_free[m % Cfg::NR]);  // the compute warps are done with it
                mbar_arrive(&out_free[m & 1]);
                n += x.loads;
            }
            bulk_wait0();
        }
    } else {
        const int sp = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int irow = 32 * sp + lane;
        uint32_t n = 0, pc = 0, m = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const Item x = item_of(it);
            const GateTab& tab = tabs[m & 1];
            if (!(ok = __all_sync(0xffffffffu,
                                  mbar_wait(&tab_full[m & 1], (m >> 1) & 1, abort_flag))))
                break;
            const int I = 4 * x.rb + sp;  // the warp's sub-block of rows
            const float gi = tab.loc[32 * I + lane];
            const double gI = tab.start[I];
            const int64_t tok0 = int64_t(x.span * prm.nb + x.rb) * C;
            float rsum = 0.f;
            for (int b = 0; b < x.ncb; ++b, ++pc) {
                const int buf = pc % NP;
                if (!(ok = __all_sync(0xffffffffu,
                                      mbar_wait(&p_full[buf], (pc / NP) & 1, abort_flag))))
                    break;
                tc_fence_after();
                const uint32_t reg = tmem + lane_base + Cfg::T_P + buf * C + 64 * half;
                const int cb = col_of(x, b);
#pragma unroll 1
                for (int s = 0; s < 2; ++s) {
                    const int J = 4 * cb + 2 * half + s;  // sub-block of columns
                    float pv[32];
                    const bool in = REV ? J >= I : J <= I;
                    if (in) {
                        tmem_load<32>(reg + 32 * s, pv);
                        if (J == I) {
#pragma unroll
                            for (int t = 0; t < 32; t += 4) {
                                const float4 g = *reinterpret_cast<const float4*>(&tab.loc[32 * J + t]);
                                const float gj[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                                for (int w = 0; w < 4; ++w) {
                                    const bool on = REV ? t + w >= lane : t + w <= lane;
                                    pv[t + w] = on ? pv[t + w] * ex2_fast(REV ? gj[w] - gi : gi - gj[w])
                                                   : 0.f;
                                }
                            }
                        } else {
                            const float r = ex2_fast(REV ? float(tab.start[J] - gI) - gi
                                                         : gi + float(gI - tab.start[J + 1]));
#pragma unroll
                            for (int t = 0; t < 32; t += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(&tab.fac[32 * J + t]);
                                pv[t] *= r * f.x;
                                pv[t + 1] *= r * f.y;
                                pv[t + 2] *= r * f.z;
                                pv[t + 3] *= r * f.w;
                            }
                        }
                        if constexpr (XTRA == 2) {
                            float p2[32];
                            tmem_load<32>(tmem + lane_base + Cfg::T_P2 + 64 * half + 32 * s, p2);
#pragma unroll
                            for (int t = 0; t < 32; ++t) {
                                // the diagonal itself passes no gate
                                p2[t] *= J == I && t == lane ? 0.f : pv[t] * prm.in_mul;
                                rsum += p2[t];
                            }
                            // column sums over the warp's rows: lane l ends with column l
#pragma unroll
                            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                                for (int t = 0; t < off; ++t) {
                                    const bool up = (lane & off) != 0;
                                    const float give = up ? p2[t] : p2[t + off];
                                    const float keep = up ? p2[t + off] : p2[t];
                                    p2[t] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                                }
                            const int64_t tok = int64_t(x.span) * prm.nb * C + 32 * J + lane;
                            if (tok < prm.N)
                                prm.colv[(x.head * (4 * prm.nb) + I) * prm.N + tok] = p2[0];
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 32; ++t) pv[t] = 0.f;
                    }
                    float pk[16];
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        pk[t] = __uint_as_float(pack_bf16(pv[2 * t], pv[2 * t + 1]));
                    tmem_st16(reg + 16 * s, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&pt_full[buf]);
            }
            if (!ok) break;
            if (!(ok = __all_sync(0xffffffffu,
                                  mbar_wait(o_full, m & 1, abort_flag) &&
                                      (m < 2 || mbar_wait(&out_free[m & 1], ((m >> 1) - 1) & 1,
                                                          abort_flag)))))
                break;
            tc_fence_after();
            if (XTRA > 0 &&
                !(ok = __all_sync(0xffffffffu, mbar_wait(&row_full[m % Cfg::NR],
                                                         (m / Cfg::NR) & 1, abort_flag))))
                break;
            const float rr = prm.st_mul *
                             ex2_fast(REV ? float(tab.start[4 * prm.nb] - gI) - gi : gi + float(gI));
            uint8_t* ost = smem + ((n + x.loads - 1) % NS) * Cfg::TILE;
            const uint8_t* row2 =
                smem + Cfg::OFF_ROW + ((m % Cfg::NR) * Cfg::ROWT + Cfg::ROWT - 1) * Cfg::TILE;
#pragma unroll 1
            for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                float ov[32];
                tmem_load<32>(tmem + lane_base + Cfg::T_IN + c0, ov);
#pragma unroll
                for (int t = 0; t < 32; ++t) ov[t] *= prm.in_mul;
                if (prm.has_state) {
                    float sv[32];
                    tmem_load<32>(tmem + lane_base + Cfg::T_ST + c0, sv);
#pragma unroll
                    for (int t = 0; t < 32; ++t) {
                        sv[t] *= rr;
                        ov[t] += sv[t];
                    }
                    if constexpr (XTRA > 0) {
#pragma unroll
                        for (int t = 0; t < 32; t += 8) {
                            const uint4 u = *reinterpret_cast<const uint4*>(
                                row2 + tile_chunk_off(C, irow, (c0 + t) / 8));
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = unpack_bf16(w[j]);
                                rsum = fmaf(f.x, sv[t + 2 * j], rsum);
                                rsum = fmaf(f.y, sv[t + 2 * j + 1], rsum);
                            }
                        }
                    }
                }
                store_row_bf16<32>(ost, C, irow, c0, ov);
            }
            if (XTRA > 0 && tok0 + irow < prm.N)
                prm.rowv[(half * prm.heads + x.head) * prm.N + tok0 + irow] = rsum;
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(o_free);
            mbar_arrive(&out_full[m & 1]);
            mbar_arrive(&tab_free[m & 1]);
            n += x.loads;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::T_COLS);
}

// ------------------------------------------------------------------ dlog_gate
// One block a span and key/value head: sums over the group's heads of the row
// values (rows' M sums and what came through S) less the column sums, from the
// span's end on; of what passes through R, from its start on; and the product
// of the two border states with all of the span's gates.
struct GatedDgateParams {
    const float* qrow;   // [2][B H][N]
    const float* colv;   // [B H][4 nb][N]
    const float* krow;   // [2][B Hkv][N], or null
    const __nv_bfloat16* S;  // [kvh][nspan][D][D] or null
    const __nv_bfloat16* R;
    const __nv_bfloat16* lg;
    __nv_bfloat16* dlg;
    int64_t N, qheads, kvh;
    int nspan, nb, nblk, group;
};

template <int D>
__global__ void __launch_bounds__(256)
gated_dgate_sum_kernel(const GatedDgateParams p) {
    __shared__ float wsum[8];
    __shared__ double gsum[8];
    __shared__ float head_s[16], head_t[16];
    const int64_t head = blockIdx.x / p.nspan;
    const int span = int(blockIdx.x % p.nspan);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n0 = int64_t(span) * p.nb * kGtC;
    const int nsub = 4 * min(p.nb, p.nblk - span * p.nb);
    float x = 0.f;
    if (p.S && p.R) {
        const uint4* s4 = reinterpret_cast<const uint4*>(p.S + (head * p.nspan + span) * D * D);
        const uint4* r4 = reinterpret_cast<const uint4*>(p.R + (head * p.nspan + span) * D * D);
        for (int i = tid; i < D * D / 8; i += 256) {
            const uint4 a = s4[i], b = r4[i];
            const uint32_t u[4] = {a.x, a.y, a.z, a.w}, w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = sm100::unpack_bf16(u[j]), g = sm100::unpack_bf16(w[j]);
                x = fmaf(f.x, g.x, x);
                x = fmaf(f.y, g.y, x);
            }
        }
    }
    x = warp_sum(x);
    if (lane == 0) wsum[warp] = x;
    double lsum = 0.0;  // the span's gates
    for (int64_t n = n0 + tid; n < min(p.N, n0 + 32 * nsub); n += 256)
        lsum += gate_log2(__bfloat162float(p.lg[head * p.N + n]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
    if (lane == 0) gsum[warp] = lsum;
    // sub-block J of warp J mod 8: d = rows less columns, t = through R, by lane
    float d[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int J = warp + 8 * u;
        const int64_t n = n0 + 32 * J + lane;
        if (J < nsub && n < p.N) {
            for (int g = 0; g < p.group; ++g) {
                const int64_t h = head * p.group + g;
                d[u] += p.qrow[h * p.N + n] + p.qrow[(p.qheads + h) * p.N + n];
                for (int I = J; I < nsub; ++I)
                    d[u] -= p.colv[(h * (4 * p.nb) + I) * p.N + n];
            }
            if (p.krow) t[u] = p.krow[head * p.N + n] + p.krow[(p.kvh + head) * p.N + n];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float a = warp_sum(d[u]), b = warp_sum(t[u]);
        if (lane == 0) {
            head_s[warp + 8 * u] = a;
            head_t[warp + 8 * u] = b;
        }
    }
    __syncthreads();
    float all = 0.f;
    double gall = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        all += wsum[w];
        gall += gsum[w];
    }
    all *= exp2f(float(gall));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int J = warp + 8 * u;
        if (J >= nsub) continue;
        float s = d[u], q = t[u];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float a = __shfl_down_sync(0xffffffffu, s, o);
            const float b = __shfl_up_sync(0xffffffffu, q, o);
            if (lane + o < 32) s += a;
            if (lane >= o) q += b;
        }
        // before the token: shifted, not subtracted, since a token's own term may
        // be larger than all before it by more than float32 holds
        q = __shfl_up_sync(0xffffffffu, q, 1);
        if (lane == 0) q = 0.f;
        for (int w = J + 1; w < nsub; ++w) s += head_s[w];
        for (int w = 0; w < J; ++w) q += head_t[w];
        const int64_t n = n0 + 32 * J + lane;
        if (n < p.N) p.dlg[head * p.N + n] = __float2bfloat16_rn(s + q + all);
    }
}

}  // namespace la

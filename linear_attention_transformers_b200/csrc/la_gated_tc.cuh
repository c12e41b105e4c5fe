// la_gated_tc.cuh — gated linear attention on the tensor cores (bf16, D = 64
// or 128; formulas in la_gated_common.cuh).
//
// The sequence is cut into blocks of C = 128 tokens and spans of L = 128 nb
// tokens; states exist at the spans' borders only, and inside a span every
// block meets the span's blocks before it directly (the backward takes spans of
// one block).  No block waits for another: all of the sequence is in flight at
// once, whatever the number of heads, and the only serial step is the states'
// recurrence over the spans, which is elementwise.
//
//   gated_span_kernel    a span's own part of the state, sum_t w_t A_t B_t^T
//   gated_border_kernel  the recurrence; bf16 states entering every span
//   gated_chain_kernel   both, walking the sequence (la_gated_chain.cuh)
//   gated_block_kernel   o of a 128-token block
//   gated_bwd_kernel     dq, dk, dv and dlog_gate of one (la_gated_bwd.cuh)
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
// the 32 x 32 sub-blocks on the diagonal take an exponential per element, of the
// difference of two sums that are float32 from the sub-block's start: each is off
// by at most 2^-24 of itself, and since a gate of 0 counts as 2^-160 that is
// 2^-12 where nearly every token of the 32 has one (a weight is then off by
// 2^-11.5, a tenth of a bf16 half step).
//
// Rounding.  q, k, v, dO are read exactly.  The weighted C x C products (P~; W~)
// and the border states are rounded to bf16 once, as tensor-core operands, S as
// well in <S, R>; the scaled operand of the parts is held as two bf16 values, or
// three where a state goes to the caller in float32; the row factors of what comes
// through a state are applied to the float32 result.  All sums, and the terms of
// dlog_gate, are float32.  So an output has an error of about 0.0024 of its 2-norm
// where its own rounding to bf16 alone gives 0.0017.
#pragma once

#include "la_chunk_fwd.cuh"
#include "la_gated_common.cuh"

namespace la {

constexpr int kGtC = 128;     // tokens a block
constexpr int kGtMaxNb = 4;   // blocks a span, at most

struct alignas(16) GateTab {
    float loc[kGtMaxNb * kGtC];   // sums of log2 gates from the sub-block's start, inclusive
    float fac[kGtMaxNb * kGtC];   // 2^(sum from behind the token to the sub-block's end)
    double start[4 * kGtMaxNb + 2];  // sums before each 32-token sub-block; [nsub] = all
};

// MMAs issued by one lane of a warp that runs the issue loop together: the
// descriptors stay warp-uniform values and only the instruction is predicated.
// Inside `if (lane == 0)` the issuing thread needs more instructions an MMA: the
// forward's blocks take 1029 us that way and 940 this way at 131072 tokens, 32
// heads, D = 128, and 127 and 114 at B8 H16 N8192 D64; in gated_bwd_kernel, with
// its many tiles, an MMA took 180 cycles to issue against 45 to 60.
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
// One arrival for a warp, after what each of its lanes did before (as fast as an
// arrival by every thread, with 32 times fewer operations on shared memory).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(bar);
}
// All lanes wait; false for all when one of the waits gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort));
}

// A box of a tensor map to L2 only.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(c0),
                 "r"(c1), "r"(c2)
                 : "memory");
}
// Two float32 operations an instruction (each rounded as the single one is).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 y, {%4, %5};\n\t"
        "mov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
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

template <int D, int SPLIT>
struct GatedSpanCfg {
    static constexpr int TILE = kGtC * D * 2;
    static constexpr int NS = 4;                      // ring slots: A, B, A, B
    static constexpr int OFF_LO = NS * TILE;          // the scaled operand's later parts
    static constexpr int OFF_W = OFF_LO + (SPLIT - 1) * TILE;  // weights [2][512]
    static constexpr int OFF_BAR = OFF_W + 2 * kGtMaxNb * kGtC * 4;
    static constexpr int NBAR = 2 * NS + 11;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int T_COLS = 2 * D;              // two records
    static constexpr int CTAS = D == 64 ? 2 : 1;
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
    static_assert(CTAS * T_COLS <= 512, "TMEM budget");
};

// Warps: 0 TMA, 1 MMA, 2 gate sums, 3 idle, 4-11 scale, 12-15 write the record.
constexpr int kGatedSpanThreads = 512;

// The accumulator is transposed, acc[e][d] = sum_t B_t[e] (w_t A_t)[d]: a thread
// of the epilogue has one e, so a warp writes rows of the record.  The scaled
// operand is SPLIT bf16 parts, the first over A in its ring slot, the others
// behind the ring, with a product each into the same accumulator: two (2^-17 of
// the value) where the states only enter the blocks, as bf16, three (2^-24) where
// the caller is given the last in float32.
template <int D, bool REV, int SPLIT>
__global__ void __launch_bounds__(kGatedSpanThreads, (GatedSpanCfg<D, SPLIT>::CTAS))
gated_span_kernel(const __grid_constant__ GatedSpanParams prm) {
    using namespace sm100;
    using Cfg = GatedSpanCfg<D, SPLIT>;
    constexpr int C = kGtC, NS = Cfg::NS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [NS] TMA
    uint64_t* empty = full + NS;       // [NS] MMAs done                  (commit)
    uint64_t* sc_full = empty + NS;    // scaled operand written          (8 warps)
    uint64_t* sc_free = sc_full + 1;   // MMAs have read it               (commit)
    uint64_t* acc_full = sc_full + 2;  // [2] record complete             (commit)
    uint64_t* acc_free = sc_full + 4;  // [2] record read                 (4 warps)
    uint64_t* w_full = sc_full + 6;    // [2] weights written             (1)
    uint64_t* w_free = sc_full + 8;    // [2] weights read                (8 warps)
    uint64_t* drain = sc_full + 10;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    float* wtab = reinterpret_cast<float*>(smem + Cfg::OFF_W);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(sc_full, 8);
        mbar_init(sc_free, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 4);
            mbar_init(&w_full[b], 1);
            mbar_init(&w_free[b], 8);
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
            constexpr uint32_t id = idesc_bf16(D, D, 1, 1);
            uint32_t n = 0, blk = 0, m = 0;
            bool ok = true;
            for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x, ++m) {
                const int cnt = ng * blocks_of(span_of(it));
                const uint32_t acc = tmem + (m & 1) * D;
                if (m >= 2 && !(ok = warp_wait(&acc_free[m & 1], ((m >> 1) - 1) & 1, abort_flag)))
                    break;
                for (int b = 0; b < cnt; ++b, ++blk, n += 2) {
                    const int s = (n + 1) % NS;
                    if (!(ok = warp_wait(&full[s], ((n + 1) / NS) & 1, abort_flag))) break;
                    if (!(ok = warp_wait(sc_full, blk & 1, abort_flag))) break;
                    tc_fence_after();
                    const uint64_t db = desc_mn_base(sbase + s * Cfg::TILE, C);
#pragma unroll
                    for (int i = 0; i < SPLIT; ++i) {
                        const uint64_t da = desc_mn_base(
                            sbase + (i == 0 ? (n % NS) * Cfg::TILE : Cfg::OFF_LO + (i - 1) * Cfg::TILE),
                            C);
#pragma unroll
                        for (int k = 0; k < C; k += 16)
                            umma_one(one, acc, db + kstep_mn(k), da + kstep_mn(k), id,
                                     b > 0 || i > 0 || k > 0);
                    }
                    commit_one(one, &empty[n % NS]);
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
            warp_arrive(&w_full[buf]);
        }
    } else if (warp >= 4 && warp < 12) {
        // scale A's rows: thread u takes half a row (D / 2 elements)
        const int u = tid - 128;
        const int row = u >> 1, q0 = (u & 1) * (D / 16);
        uint8_t* lo = smem + Cfg::OFF_LO;
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
                uint8_t* src = smem + s * Cfg::TILE;
                uint4 x[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    x[i] = *reinterpret_cast<const uint4*>(src + tile_chunk_off(C, row, q0 + i));
                const float wr = w[(b % nbv) * C + row];
                // the first part in place; the others wait for the products that
                // still read the block before's
                uint4 later[SPLIT - 1][D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t raw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t part[SPLIT][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 f = mul2(unpack_bf16(raw[j]), make_float2(wr, wr));
#pragma unroll
                        for (int c = 0; c < SPLIT; ++c) {
                            part[c][j] = pack_bf16(f.x, f.y);
                            if (c + 1 < SPLIT)
                                f = fma2(unpack_bf16(part[c][j]), make_float2(-1.f, -1.f), f);
                        }
                    }
                    *reinterpret_cast<uint4*>(src + tile_chunk_off(C, row, q0 + i)) =
                        make_uint4(part[0][0], part[0][1], part[0][2], part[0][3]);
#pragma unroll
                    for (int c = 1; c < SPLIT; ++c)
                        later[c - 1][i] =
                            make_uint4(part[c][0], part[c][1], part[c][2], part[c][3]);
                }
                if (!(ok = blk == 0 || warp_wait(sc_free, (blk - 1) & 1, abort_flag))) break;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int c = 0; c + 1 < SPLIT; ++c)
                        *reinterpret_cast<uint4*>(lo + c * Cfg::TILE +
                                                  tile_chunk_off(C, row, q0 + i)) = later[c][i];
                fence_proxy_async_smem();
                warp_arrive(sc_full);
            }
            if (ok) warp_arrive(&w_free[m & 1]);
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
            const uint32_t acc = tmem + lane_base + (m & 1) * D;
            float* out = prm.rec + (head_of(it) * prm.nspan + span_of(it)) * int64_t(D) * D;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += 16) {
                float x[16];
                tmem_load<16>(acc + d0, x);
                if (e >= 0) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[(d0 + j) * D + e] = x[j];
                }
            }
            tc_fence_before();
            warp_arrive(&acc_free[m & 1]);
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
// `last` may be null; then the part of the span walked last is not read.  Whole
// warps: per_head is a multiple of 128.
template <bool REV>
__global__ void __launch_bounds__(128)
gated_border_kernel(const float4* __restrict__ rec, const float* __restrict__ tot,
                    const float4* __restrict__ first, float4* __restrict__ last,
                    uint2* __restrict__ enter, const uint2* __restrict__ S,
                    float* __restrict__ dots, int64_t total, int per_head, int nspan) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int64_t head = i / per_head, e = i % per_head;
    const float4* r = rec + head * nspan * per_head + e;
    uint2* out = enter + head * nspan * per_head + e;
    const float* gt = tot + head * nspan;
    float4 run = first ? first[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;
    const int steps = last ? nspan : nspan - 1;
    // REV with S: a warp's share of <S, R> at the span (per_head / 32 of them), from
    // R in float32 (see gated_chain_kernel); a warp is always within one head
    auto put = [&](int c) {
        if (REV && S) {
            const uint2 u = S[(head * nspan + c) * per_head + e];
            const float2 f = sm100::unpack_bf16(u.x), h = sm100::unpack_bf16(u.y);
            const float dot =
                warp_sum(fmaf(f.x, run.x, fmaf(f.y, run.y, fmaf(h.x, run.z, h.y * run.w))));
            if ((threadIdx.x & 31) == 0)
                dots[(head * nspan + c) * (per_head / 32) + e / 32] = dot;
        }
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

// -------------------------------------------------------------------------- o
// o_i = scale sum_j e^{G_i-G_j} (q_i . k_j) v_j + scale e^{G_i} (q_i through S)
struct GatedBlockParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_st, tm_o;
    const __nv_bfloat16* lg;
    int64_t N, items;
    int nblk, nb, nspan, group, has_state;
    float scale;
};

template <int D>
struct GatedBlockCfg {
    static constexpr int TILE = kGtC * D * 2;
    static constexpr int CTAS = D == 64 ? 2 : 1;
    static constexpr int NS = 4;                     // ring of the k, v and state tiles
    static constexpr int NR = 2;                     // q stays for all of its column blocks
    static constexpr int NP = D == 128 ? 2 : 1;      // P buffers
    static constexpr int NG = D == 128 ? 4 : 2;      // groups of four compute warps
    static constexpr int THREADS = 128 + 128 * NG;
    static constexpr int OFF_ROW = NS * TILE;
    static constexpr int OFF_TAB = OFF_ROW + NR * TILE;
    static constexpr int OFF_BAR = OFF_TAB + 2 * int(sizeof(GateTab));
    static constexpr int NBAR = 2 * NS + 21;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int T_P = 0;
    static constexpr int T_ST = kGtC * NP;           // through the state
    static constexpr int T_IN = T_ST + D;            // inside the span
    static constexpr int T_COLS = T_IN + D <= 256 ? 256 : 512;
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
    static_assert(CTAS * T_COLS <= 512, "TMEM budget");
};

// Measured: B8 H16 N8192 D64 112 us (604 MB of tiles, states and output: 5.4 TB/s,
// 0.83 of a copy's bandwidth; single blocks), 32 heads of 131072 tokens, D = 128,
// 950 us in a short run (4.83 GB: 5.1 TB/s, 0.78; spans of two blocks), 1043 to 1094
// in one of a hundred milliseconds and more.  Cores issue in half of
// the cycles at most and the tensor pipe is busy in a quarter: what is left of the
// bandwidth is the latency from P to its weights to the product that reads them.
//
// Warps: 0 TMA loads of the ring, 1 MMA, 2 gate tables and TMA loads of q, 3
// TMA stores, from 4 on compute: NG groups of four warps, group h for 128 / NG
// columns of every C x C product and D / NG of the output.
template <int D>
__global__ void __launch_bounds__(GatedBlockCfg<D>::THREADS, GatedBlockCfg<D>::CTAS)
gated_block_kernel(const __grid_constant__ GatedBlockParams prm) {
    using namespace sm100;
    using Cfg = GatedBlockCfg<D>;
    constexpr int C = kGtC, NS = Cfg::NS, NP = Cfg::NP, NG = Cfg::NG;
    constexpr int PW = C / NG;  // columns of P a group packs
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [NS] TMA
    uint64_t* empty = full + NS;        // [NS] released (commit, or the store warp)
    uint64_t* p_full = empty + NS;      // [2] P complete                (commit)
    uint64_t* pt_full = p_full + 2;     // [2] weighted P packed         (compute warps)
    uint64_t* p_free = p_full + 4;      // [2] ... consumed              (commit)
    uint64_t* o_full = p_full + 6;      // output accumulators complete  (commit)
    uint64_t* o_free = p_full + 7;      // ... read                      (compute warps)
    uint64_t* out_full = p_full + 8;    // [2] output staged             (compute warps)
    uint64_t* out_free = p_full + 10;   // [2] ... stored                (1)
    uint64_t* tab_full = p_full + 12;   // [2] gate tables written       (1)
    uint64_t* tab_free = p_full + 14;   // [2] ... read                  (compute warps)
    uint64_t* row_full = p_full + 16;   // [2] q landed                  (1 + tx)
    uint64_t* row_free = p_full + 18;   // [2] ... read                  (commit)
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
            mbar_init(&pt_full[b], 4 * NG);
            mbar_init(&p_free[b], 1);
            mbar_init(&out_full[b], 4 * NG);
            mbar_init(&out_free[b], 1);
            mbar_init(&tab_full[b], 1);
            mbar_init(&tab_free[b], 4 * NG);
            mbar_init(&row_full[b], 1);
            mbar_init(&row_free[b], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, 4 * NG);
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

    // One item: 128 rows of a query head.  Its other tiles arrive in the ring in
    // the order k 0, [state], v 0, k 1, v 1, ...
    struct Item {
        int head, kvh;  // query head, key/value head
        int span, rb;   // span of the head, block of the span
        int ncb;        // column blocks: rb + 1
        int loads;      // tiles through the ring
    };
    auto item_of = [&](int64_t it) {
        Item x;
        x.head = int(unsigned(it) / unsigned(prm.nblk));
        const int blk = int(unsigned(it) % unsigned(prm.nblk));
        x.kvh = int(unsigned(x.head) / unsigned(prm.group));
        x.span = blk / prm.nb;
        const int nbv = min(prm.nb, prm.nblk - x.span * prm.nb);
        // the blocks of a span differ in cost by their place in it: turn the
        // order from span to span, so that a stride over the items (the grid)
        // meets every place
        const unsigned s = unsigned(x.head) * unsigned(prm.nspan) + unsigned(x.span);
        x.rb = int((unsigned(blk % prm.nb) + s + (s >> 1)) % unsigned(nbv));
        x.ncb = x.rb + 1;
        x.loads = (prm.has_state ? 1 : 0) + 2 * x.ncb;
        return x;
    };

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&prm.tm_k);
            tma_prefetch_desc(&prm.tm_v);
            uint32_t n = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap* map, int rows, int row, int head) {
                const int s = n % NS;
                if (n >= NS && !mbar_wait(&empty[s], ((n / NS) - 1) & 1, abort_flag)) return false;
                mbar_arrive_expect_tx(&full[s], uint32_t(rows) * D * 2);
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(smem + s * Cfg::TILE + a * rows * 128, map, &full[s], 64 * a, row,
                                head);
                ++n;
                return true;
            };
            for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x) {
                const Item x = item_of(it);
                for (int b = 0; ok && b < x.ncb; ++b) {
                    const int row = (x.span * prm.nb + b) * C;
                    ok = load(&prm.tm_k, C, row, x.kvh);
                    if (ok && b == 0 && prm.has_state)
                        ok = load(&prm.tm_st, D, 0, x.kvh * prm.nspan + x.span);
                    if (ok) ok = load(&prm.tm_v, C, row, x.kvh);
                }
            }
            for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i)
                mbar_wait_drain(&full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1) {
        const uint32_t one = elect_lane();
        constexpr uint32_t idP = idesc_bf16(C, C, 0, 0);  // rows x columns
        constexpr uint32_t idV = idesc_bf16(C, D, 0, 1);  // rows through S; weighted P, values
        uint32_t n = 0, pc = 0, m = 0;
        bool ok = true;
        auto tile = [&](uint32_t i) { return sbase + (i % NS) * Cfg::TILE; };
        auto landed = [&](uint32_t i) {
            return warp_wait(&full[i % NS], (i / NS) & 1, abort_flag);
        };
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const Item x = item_of(it);
            const uint32_t st = n + 1, hs = prm.has_state ? 1 : 0;
            auto k_at = [&](int b) { return b == 0 ? n : n + hs + 2 * b; };
            auto v_at = [&](int b) { return n + hs + 1 + 2 * b; };
            const uint32_t rbuf = m % Cfg::NR;
            const uint64_t dq = desc_k_base(sbase + Cfg::OFF_ROW + rbuf * Cfg::TILE);
            // P of column block b, into the buffer that block b - NP is done with
            auto p_part = [&](int b) {
                const uint32_t i = pc + b, buf = i % NP;
                if (i >= NP && !warp_wait(&p_free[buf], (i / NP - 1) & 1, abort_flag)) return false;
                if (b == 0 && !warp_wait(&row_full[rbuf], (m / Cfg::NR) & 1, abort_flag))
                    return false;
                if (!landed(k_at(b))) return false;
                tc_fence_after();
                const uint64_t dk = desc_k_base(tile(k_at(b)));
#pragma unroll
                for (int k = 0; k < D; k += 16)
                    umma_one(one, tmem + Cfg::T_P + buf * C, dq + kstep_k(C, k),
                             dk + kstep_k(C, k), idP, k > 0);
                commit_one(one, &p_full[buf]);
                commit_one(one, &empty[k_at(b) % NS]);
                return true;
            };
            if (!(ok = p_part(0))) break;
            if (m > 0 && !(ok = warp_wait(o_free, (m - 1) & 1, abort_flag))) break;
            if (hs) {
                if (!(ok = landed(st))) break;
                tc_fence_after();
                const uint64_t ds = desc_mn_base(tile(st), D);
#pragma unroll
                for (int k = 0; k < D; k += 16)
                    umma_one(one, tmem + Cfg::T_ST, dq + kstep_k(C, k), ds + kstep_mn(k), idV, k > 0);
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
                if (!(ok = landed(v_at(b)))) break;
                tc_fence_after();
                const uint32_t tp = tmem + Cfg::T_P + (i % NP) * C;
                const uint64_t dv = desc_mn_base(tile(v_at(b)), C);
                // a group packs its PW columns into the first half of them
#pragma unroll
                for (int k = 0; k < C; k += 16)
                    umma_ts_one(one, tmem + Cfg::T_IN, tp + (k / PW) * PW + (k % PW) / 2,
                                dv + kstep_mn(k), idV, b > 0 || k > 0);
                commit_one(one, &p_free[i % NP]);
                if (b + 1 < x.ncb)
                    commit_one(one, &empty[v_at(b) % NS]);  // the last one: the store warp
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
    } else if (warp == 2) {
        uint32_t m = 0, issued = 0;
        auto load_rows = [&](const Item& x) {  // of item `issued`
            const uint32_t r = issued % Cfg::NR;
            if (lane == 0) {
                uint8_t* dst = smem + Cfg::OFF_ROW + r * Cfg::TILE;
                mbar_arrive_expect_tx(&row_full[r], Cfg::TILE);
                for (int a = 0; a < D / 64; ++a)
                    tma_load_3d(dst + a * C * 128, &prm.tm_q, &row_full[r], 64 * a,
                                (x.span * prm.nb + x.rb) * C, x.head);
            }
            ++issued;
        };
        for (int64_t it = blockIdx.x; it < prm.items; it += gridDim.x, ++m) {
            const int buf = m & 1;
            const Item x = item_of(it);
            if (m < Cfg::NR) load_rows(x);
            if (m >= 2 && !warp_wait(&tab_free[buf], ((m >> 1) - 1) & 1, abort_flag)) break;
            GateTab& tab = tabs[buf];
            gate_sums(prm.lg + int64_t(x.kvh) * prm.N, int64_t(x.span) * prm.nb * C, prm.N,
                      4 * prm.nb, lane, tab.start,
                      [&](int t, double run, double before, double end, double) {
                          tab.loc[t] = float(run - before);
                          tab.fac[t] = ex2_fast(float(end - run));
                      });
            warp_arrive(&tab_full[buf]);
            if (m >= Cfg::NR) {
                if (!warp_wait(&row_free[m % Cfg::NR], (m / Cfg::NR - 1) & 1, abort_flag)) break;
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
                    tma_store_3d(&prm.tm_o, src + a * C * 128, 64 * a,
                                 (x.span * prm.nb + x.rb) * C, x.head);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(&empty[last % NS]);
                mbar_arrive(&out_free[m & 1]);
                n += x.loads;
            }
            bulk_wait0();
        }
    } else {
        const int sp = warp & 3, grp = (warp - 4) >> 2;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int irow = 32 * sp + lane;
        uint32_t n = 0, pc = 0, m = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < prm.items; it += gridDim.x, ++m) {
            const Item x = item_of(it);
            const GateTab& tab = tabs[m & 1];
            if (!(ok = warp_wait(&tab_full[m & 1], (m >> 1) & 1, abort_flag))) break;
            const int I = 4 * x.rb + sp;  // the warp's sub-block of rows
            const float gi = tab.loc[32 * I + lane];
            const double gI = tab.start[I];
            for (int b = 0; b < x.ncb; ++b, ++pc) {
                const int buf = pc % NP;
                if (!(ok = warp_wait(&p_full[buf], (pc / NP) & 1, abort_flag))) break;
                tc_fence_after();
                const uint32_t reg = tmem + lane_base + Cfg::T_P + buf * C + PW * grp;
#pragma unroll 1
                for (int s = 0; s < PW / 32; ++s) {
                    const int J = 4 * b + (PW / 32) * grp + s;  // sub-block of columns
                    float pv[32];
                    if (J <= I) {
                        tmem_load<32>(reg + 32 * s, pv);
                        if (J == I) {
#pragma unroll
                            for (int t = 0; t < 32; t += 4) {
                                const float4 g = *reinterpret_cast<const float4*>(&tab.loc[32 * J + t]);
                                const float gj[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                                for (int w = 0; w < 4; ++w)
                                    pv[t + w] = t + w <= lane ? pv[t + w] * ex2_fast(gi - gj[w]) : 0.f;
                            }
                        } else {
                            const float r = ex2_fast(gi + float(gI - tab.start[J + 1]));
#pragma unroll
                            for (int t = 0; t < 32; t += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(&tab.fac[32 * J + t]);
                                pv[t] *= r * f.x;
                                pv[t + 1] *= r * f.y;
                                pv[t + 2] *= r * f.z;
                                pv[t + 3] *= r * f.w;
                            }
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
                warp_arrive(&pt_full[buf]);
            }
            if (!ok) break;
            if (!(ok = warp_wait(o_full, m & 1, abort_flag) &&
                       (m < 2 || warp_wait(&out_free[m & 1], ((m >> 1) - 1) & 1, abort_flag))))
                break;
            tc_fence_after();
            const float rr = prm.scale * ex2_fast(gi + float(gI));
            uint8_t* ost = smem + ((n + x.loads - 1) % NS) * Cfg::TILE;
#pragma unroll 1
            for (int c0 = grp * (D / NG); c0 < (grp + 1) * (D / NG); c0 += 32) {
                float ov[32];
                tmem_load<32>(tmem + lane_base + Cfg::T_IN + c0, ov);
#pragma unroll
                for (int t = 0; t < 32; ++t) ov[t] *= prm.scale;
                if (prm.has_state) {
                    float sv[32];
                    tmem_load<32>(tmem + lane_base + Cfg::T_ST + c0, sv);
#pragma unroll
                    for (int t = 0; t < 32; ++t) ov[t] = fmaf(rr, sv[t], ov[t]);
                }
                store_row_bf16<32>(ost, C, irow, c0, ov);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(o_free);
            warp_arrive(&out_full[m & 1]);
            warp_arrive(&tab_free[m & 1]);
            n += x.loads;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::T_COLS);
}

}  // namespace la

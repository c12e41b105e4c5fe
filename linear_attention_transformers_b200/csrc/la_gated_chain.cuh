// la_gated_chain.cuh — border states of gated linear attention by walking the
// sequence (bf16, D = 64 or 128): in place of gated_span_kernel and
// gated_border_kernel where there are heads enough, or blocks few enough.
//
// One CTA takes EC of the D value columns of one key/value head through all of
// its 128-token blocks.  The recurrence is elementwise in the state, so columns
// are independent of each other and the state never leaves the registers of the
// threads that update it; what enters each span goes out in bf16, and the
// float32 records of the other way (4 D^2 bytes written and read a span) do not
// exist.  Per block
//
//     S <- e^{G_C} S + A^T (w B),     w_t = e^{G_C - G_t}  (REV: mul e^{G_t})
//
// with A the block's keys (REV: queries), read through a TMA ring, and B the
// values (dO), read by the threads that scale them and write them as bf16 parts
// side by side: one MMA of M = D, N = SPLIT EC per 16 tokens.  Two parts (2^-17
// of the value) where the state only enters the blocks, as bf16; three (2^-24)
// where the caller is given it in float32.
//
// REV with S (the states entering the blocks, formed before): also the sums
// <S, R> that dlog_gate needs, from R in float32, since R in bf16 as well would
// put two roundings into a sum that dlog_gate often mostly is.
//
// The steps of a block (scale, products, update) belong to different warps and
// overlap across blocks; a block takes as long as the longest of them, the scale
// (1.5 us with EC = 64, 0.9 with 32; sixteen scaling warps in place of eight
// spill and are slower).  Measured: B8 H16 N8192 D64, S 94 us, R with <S, R> 131;
// B4 H16 N4096 D128, 62 and 82.  One CTA an SM and a serial walk: the time is the
// blocks' number times that latency, at about half of a copy's bandwidth.
#pragma once

#include "la_async_copy.cuh"
#include "la_gated_tc.cuh"

namespace la {

struct GatedChainParams {
    CUtensorMap tm_a;
    const __nv_bfloat16 *b, *lg;
    const float* first;        // [kvh][D][D] or null
    float* last;               // [kvh][D][D] or null
    __nv_bfloat16* enter;      // [kvh][nspan][D][D]
    const __nv_bfloat16* S;    // REV: the forward's `enter`, or null
    float* dots;               // REV: [kvh][nspan][D / EC * 8] parts of <S, R>
    int64_t N;
    int nblk, nb, nspan, group, blocks;  // blocks: walked (the last span may be left out)
    float mul;
};

template <int D, int EC, int SPLIT>
struct GatedChainCfg {
    static constexpr int TILE = kGtC * D * 2;          // A
    // ring of A, tiles of B on their way: what fits beside the scaled parts
    static constexpr int NS = (D == 128 && EC == 64 ? 3 : 4) -
                              (SPLIT == 3 && (D == 128 || EC == 64) ? 1 : 0);
    static constexpr int SC = kGtC * 128 * ((SPLIT * EC + 63) / 64);  // scaled B, 64-column atoms
    static constexpr int NB = NS;
    static constexpr int OFF_SC = NS * TILE;           // [2]
    static constexpr int OFF_B = OFF_SC + 2 * SC;      // [NB][EC / 16][256 threads] 16 bytes
    static constexpr int OFF_W = OFF_B + NB * kGtC * EC * 2;  // [4][128] weights
    static constexpr int OFF_TOT = OFF_W + 4 * kGtC * 4;  // [4] the block's gates' product
    static constexpr int OFF_BAR = OFF_TOT + 16;
    static constexpr int NBAR = 2 * NS + 17;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int ACC = SPLIT * EC;
    static constexpr int T_COLS = 2 * ACC <= 128 ? 128 : 2 * ACC <= 256 ? 256 : 512;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// Warps: 0 TMA, 1 MMA, 2 gates, 3 idle, 4-11 scale, 12-19 update.
constexpr int kGatedChainThreads = 640;

template <int D, int EC, bool REV, int SPLIT>
__global__ void __launch_bounds__(kGatedChainThreads, 1)
gated_chain_kernel(const __grid_constant__ GatedChainParams prm) {
    using namespace sm100;
    using Cfg = GatedChainCfg<D, EC, SPLIT>;
    constexpr int C = kGtC, NS = Cfg::NS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // [NS] TMA
    uint64_t* empty = full + NS;        // [NS] products done             (commit)
    uint64_t* sc_full = empty + NS;     // [2] scaled                     (8 warps)
    uint64_t* sc_free = sc_full + 2;    // [2] products done              (commit)
    uint64_t* acc_full = sc_full + 4;   // [2] a block's sum complete     (commit)
    uint64_t* acc_free = sc_full + 6;   // [2] ... read                   (update warps)
    uint64_t* w_full = sc_full + 8;     // [4] weights written            (1)
    uint64_t* w_free = sc_full + 12;    // [4] ... read (scale and update warps)
    uint64_t* drain = sc_full + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    float* wtab = reinterpret_cast<float*>(smem + Cfg::OFF_W);
    float* tots = reinterpret_cast<float*>(smem + Cfg::OFF_TOT);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int NPART = D / EC;
    const int head = int(blockIdx.x) / NPART;          // key/value head
    const int e0 = (int(blockIdx.x) % NPART) * EC;     // first value column
    const int ng = REV ? prm.group : 1;
    const int steps = prm.blocks;
    // block walked at step i
    auto blk_of = [&](int i) { return REV ? prm.nblk - 1 - i : i; };
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sc_full[b], 8);
            mbar_init(&sc_free[b], 1);
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 8);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&w_full[b], 1);
            mbar_init(&w_free[b], 16);
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

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&prm.tm_a);
            uint32_t n = 0;
            bool ok = true;
            for (int i = 0; ok && i < steps; ++i)
                for (int g = 0; g < ng; ++g, ++n) {
                    const int s = n % NS;
                    if (n >= NS && !(ok = mbar_wait(&empty[s], ((n / NS) - 1) & 1, abort_flag)))
                        break;
                    mbar_arrive_expect_tx(&full[s], Cfg::TILE);
                    for (int a = 0; a < D / 64; ++a)
                        tma_load_3d(smem + s * Cfg::TILE + a * C * 128, &prm.tm_a, &full[s],
                                    64 * a, blk_of(i) * C, head * ng + g);
                }
            for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i)
                mbar_wait_drain(&full[i % NS], (i / NS) & 1);
        }
    } else if (warp == 1) {
        const uint32_t one = elect_lane();
        constexpr uint32_t id = idesc_bf16(D, SPLIT * EC, 1, 1);
        uint32_t n = 0;
        bool ok = true;
        for (int i = 0; ok && i < steps; ++i) {
            const uint32_t acc = tmem + (i & 1) * Cfg::ACC;
            if (i >= 2 && !(ok = warp_wait(&acc_free[i & 1], ((i >> 1) - 1) & 1, abort_flag))) break;
            for (int g = 0; g < ng; ++g, ++n) {
                const int s = n % NS, b = n & 1;
                if (!(ok = warp_wait(&full[s], (n / NS) & 1, abort_flag) &&
                           warp_wait(&sc_full[b], (n >> 1) & 1, abort_flag)))
                    break;
                tc_fence_after();
                const uint64_t da = desc_mn_base(sbase + s * Cfg::TILE, C);
                const uint64_t db = desc_mn_base(sbase + Cfg::OFF_SC + b * Cfg::SC, C);
#pragma unroll
                for (int k = 0; k < C; k += 16)
                    umma_one(one, acc, da + kstep_mn(k), db + kstep_mn(k), id, g > 0 || k > 0);
                commit_one(one, &empty[s]);
                commit_one(one, &sc_free[b]);
            }
            if (ok) commit_one(one, &acc_full[i & 1]);
        }
        commit_one(one, drain);
        if (lane == 0) mbar_wait_drain(drain, 0);
    } else if (warp == 2) {
        // Lane l holds tokens 4 l .. 4 l + 3, loaded kAhead blocks ahead (a load may
        // take longer than a block).  Weights need only the sums to the block's end
        // (REV: from its start), formed from that end: an exponent is then off by
        // float32's share of itself, not of the sums over the whole block.
        constexpr int kAhead = 4;
        const __nv_bfloat16* lg = prm.lg + int64_t(head) * prm.N;
        __nv_bfloat16 nx[kAhead][4];
        auto fetch = [&](int i, __nv_bfloat16 (&to)[4]) {
            const int64_t n0 = int64_t(blk_of(i)) * C + 4 * lane;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[j] = i < steps && n0 + j < prm.N ? lg[n0 + j] : __nv_bfloat16(0.f);
        };
#pragma unroll
        for (int r = 0; r < kAhead; ++r) fetch(r, nx[r]);
        bool ok = true;
        for (int i0 = 0; ok && i0 < steps; i0 += kAhead) {
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = i0 + r;
                if (i >= steps) break;
                float x[4], s = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // as gate_log2, in float32: the weights are sums of these alone
                    const float y = __bfloat162float(nx[r][j]) * 1.4426950408889634f;
                    x[j] = y < -160.f ? -160.f : y;
                    s += x[j];
                }
                fetch(i + kAhead, nx[r]);
                float sc = s;  // inclusive, from the lane's end of the block
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = REV ? __shfl_up_sync(0xffffffffu, sc, o)
                                        : __shfl_down_sync(0xffffffffu, sc, o);
                    if (REV ? lane >= o : lane + o < 32) sc += y;
                }
                float run =
                    REV ? __shfl_up_sync(0xffffffffu, sc, 1) : __shfl_down_sync(0xffffffffu, sc, 1);
                if (REV ? lane == 0 : lane == 31) run = 0.f;
                if (!(ok = i < 4 || warp_wait(&w_free[i & 3], ((i >> 2) - 1) & 1, abort_flag)))
                    break;
                float4 w;
                float* wv = reinterpret_cast<float*>(&w);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const int j = REV ? jj : 3 - jj;
                    if (REV) run += x[j];  // the token's own gate is passed backwards
                    wv[j] = REV ? prm.mul * exp2f(run) : exp2f(run);
                    if (!REV) run += x[j];
                }
                *reinterpret_cast<float4*>(wtab + (i & 3) * C + 4 * lane) = w;
                if (lane == (REV ? 31 : 0)) tots[i & 3] = exp2f(sc);
                warp_arrive(&w_full[i & 3]);
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // thread u: half of the columns of row u / 2
        const int u = tid - 128, row = u >> 1, h = u & 1;
        constexpr int NV = EC / 16;  // 16-byte pieces
        // its pieces of B arrive by cp.async in a ring that only it reads
        uint4* ring = reinterpret_cast<uint4*>(smem + Cfg::OFF_B) + u;
        // where the next piece is: its token, and steps to the next head and block
        int fi = 0, fg = 0, fs = 0;
        int64_t ft = int64_t(blk_of(0)) * C + row;
        const int64_t head_step = prm.N * D;
        const __nv_bfloat16* base = prm.b + int64_t(head) * ng * head_step + e0 + h * (EC / 2);
        const __nv_bfloat16* fp = base + ft * D;
        auto fetch = [&]() {
            if (fi < steps) {
                const bool in = ft < prm.N;
                const uint4* src = reinterpret_cast<const uint4*>(in ? fp : base);
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    copy16_async(ring + (fs * NV + j) * 256, src + j, in);
                fs = fs == Cfg::NB - 1 ? 0 : fs + 1;
                if (++fg < ng) {
                    fp += head_step;
                } else {
                    fg = 0;
                    ++fi;
                    ft += REV ? -C : C;
                    fp += (REV ? -C : C) * D - (ng - 1) * head_step;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int rs = 0;  // slot read next
        uint32_t n = 0;
        bool ok = true;
        for (int j = 0; j < Cfg::NB - 1; ++j) fetch();
        for (int i = 0; ok && i < steps; ++i) {
            if (!(ok = warp_wait(&w_full[i & 3], (i >> 2) & 1, abort_flag))) break;
            const float w = wtab[(i & 3) * C + row];
            for (int g = 0; g < ng; ++g, ++n) {
                fetch();
                asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::NB - 1) : "memory");
                uint4 x[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j) x[j] = ring[(rs * NV + j) * 256];
                rs = rs == Cfg::NB - 1 ? 0 : rs + 1;
                if (!(ok = n < 2 || warp_wait(&sc_free[n & 1], ((n >> 1) - 1) & 1, abort_flag)))
                    break;
                uint8_t* sc = smem + Cfg::OFF_SC + (n & 1) * Cfg::SC;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    uint32_t part[SPLIT][4];
                    const uint32_t raw[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float2 f = mul2(unpack_bf16(raw[c]), make_float2(w, w));
#pragma unroll
                        for (int i2 = 0; i2 < SPLIT; ++i2) {
                            part[i2][c] = pack_bf16(f.x, f.y);
                            if (i2 + 1 < SPLIT)
                                f = fma2(unpack_bf16(part[i2][c]), make_float2(-1.f, -1.f), f);
                        }
                    }
#pragma unroll
                    for (int i2 = 0; i2 < SPLIT; ++i2)
                        *reinterpret_cast<uint4*>(
                            sc + tile_chunk_off(C, row, h * NV + j + i2 * (EC / 8))) =
                            make_uint4(part[i2][0], part[i2][1], part[i2][2], part[i2][3]);
                }
                fence_proxy_async_smem();
                warp_arrive(&sc_full[n & 1]);
            }
            if (ok) warp_arrive(&w_free[i & 3]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 12) {
        const int sp = warp & 3, h = (warp - 12) >> 2;
        const uint32_t lane_base = uint32_t(32 * sp) << 16;
        const int d = acc_row<D>(sp, lane);  // row of the state, -1: none
        constexpr int W = EC / 2;
        float run[W];
        const int64_t at = int64_t(d < 0 ? 0 : d) * D + e0 + h * W;
        const float* first = prm.first ? prm.first + int64_t(head) * D * D + at : nullptr;
#pragma unroll
        for (int j = 0; j < W; j += 4) {
            const float4 x = first && d >= 0 ? *reinterpret_cast<const float4*>(first + j)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
            run[j] = x.x, run[j + 1] = x.y, run[j + 2] = x.z, run[j + 3] = x.w;
        }
        // S of the span that is written next, loaded one ahead
        uint4 sx[REV ? W / 8 : 1];
        auto fetch_s = [&](int span) {
            if (!REV || !prm.S || d < 0 || span < 0) return;
            const uint4* s4 = reinterpret_cast<const uint4*>(
                prm.S + (int64_t(head) * prm.nspan + span) * D * D + at);
#pragma unroll
            for (int j = 0; j < W / 8; ++j) sx[j] = __ldcs(s4 + j);
        };
        fetch_s(prm.nspan - 1);
        auto put = [&](int span) {
            if (REV && prm.S) {  // this thread's share of <S, R>, a value a warp
                float2 d2 = make_float2(0.f, 0.f);
                if (d >= 0) {
#pragma unroll
                    for (int j = 0; j < W / 8; ++j) {
                        const uint4 x = sx[j];
                        const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            d2 = fma2(unpack_bf16(p[c]),
                                      make_float2(run[8 * j + 2 * c], run[8 * j + 2 * c + 1]), d2);
                    }
                }
                fetch_s(span - 1);
                const float dot = warp_sum(d2.x + d2.y);
                if (lane == 0)
                    prm.dots[((int64_t(head) * prm.nspan + span) * NPART + int(blockIdx.x) % NPART) * 8 +
                             warp - 12] = dot;
            }
            if (d < 0) return;
            __nv_bfloat16* out = prm.enter + (int64_t(head) * prm.nspan + span) * D * D + at;
#pragma unroll
            for (int j = 0; j < W; j += 8)
                *reinterpret_cast<uint4*>(out + j) =
                    make_uint4(pack_bf16(run[j], run[j + 1]), pack_bf16(run[j + 2], run[j + 3]),
                               pack_bf16(run[j + 4], run[j + 5]), pack_bf16(run[j + 6], run[j + 7]));
        };
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int blk = blk_of(i);
            if (REV ? (blk % prm.nb == prm.nb - 1 || i == 0) : blk % prm.nb == 0) put(blk / prm.nb);
            if (!(ok = warp_wait(&w_full[i & 3], (i >> 2) & 1, abort_flag) &&
                       warp_wait(&acc_full[i & 1], (i >> 1) & 1, abort_flag)))
                break;
            tc_fence_after();
            const float a = tots[i & 3];
            const uint32_t acc = tmem + lane_base + (i & 1) * Cfg::ACC + h * W;
#pragma unroll
            for (int j = 0; j < W; j += 16) {
                float hi[16], lo[16];
                tmem_ld16(acc + j, hi);
                tmem_load<16>(acc + EC + j, lo);
                if (SPLIT == 3) {
                    float l2[16];
                    tmem_load<16>(acc + 2 * EC + j, l2);
#pragma unroll
                    for (int c = 0; c < 16; ++c) lo[c] += l2[c];
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) run[j + c] = fmaf(a, run[j + c], hi[c] + lo[c]);
            }
            tc_fence_before();
            warp_arrive(&acc_free[i & 1]);
            warp_arrive(&w_free[i & 3]);
        }
        if (ok) {
            if (prm.last) {
                if (d >= 0) {
                    float* out = prm.last + int64_t(head) * D * D + at;
#pragma unroll
                    for (int j = 0; j < W; j += 4)
                        *reinterpret_cast<float4*>(out + j) =
                            make_float4(run[j], run[j + 1], run[j + 2], run[j + 3]);
                }
            } else {
                put(REV ? 0 : prm.nspan - 1);  // the span whose own part was left out
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::T_COLS);
}

}  // namespace la
